// The bf16 tile product of the gradient GEMMs: acc += A B over K with fp32
// accumulation, for either memory order of each operand, on four waves.
//
// K is walked in 64-deep stages through two LDS slots filled by
// direct-to-LDS loads; while a 32-deep sub-step's MFMAs issue, the fragment
// reads of the next one and the loads of the stage after next go between
// them.  The MFMAs are volatile asm, so that order is the issue order and
// the accumulators stay where their constraint puts them.  The slots are
// two arrays named statically (two stages per loop trip), so the compiler
// sees that the loads into one and the reads of the other do not alias.
//
// Orders.  K_LAST: element (r, k) at r * ld + k (k contiguous): a slot holds
// rows of 64 k, 16-byte chunks XOR-swizzled by the row, read 16 bytes per
// lane.  K_FIRST: element (r, k) at k * ld + r (r contiguous), as both
// operands of a weight gradient and the weights of a row gradient lie: a
// slot holds 64 rows of k, and ds_read_b64_tr_b16 transposes on the way to
// the registers: of 16 lanes, lane i names 4 r of row k0 + i / 4 and
// receives the 4 k of r0 + i % 16.  Its 32-byte pieces of 8 k rows would
// fall on the same banks, so they are XOR-swizzled by k.
#pragma once

#include "common.h"

namespace mt {

constexpr int SK = 64;                   // stage depth

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ void dma16(const char *src, u32x4 *lds) {
    __builtin_amdgcn_global_load_lds(
        (const void *)src, (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}

// s_waitcnt vmcnt(n) only.
template <int N> __device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

__device__ __forceinline__ void mfma(floatx4 &acc, const bf16x8 &a, const bf16x8 &b) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}

// A zeroed line that lanes past the end of a K_FIRST operand read from.
static __device__ __align__(1024) const char zero_line[1024] = {};

// One operand of a tile.  base: element (0, 0) of the tile (uniform); ld:
// bytes.  K_LAST: rows >= valid re-read row 0.  K_FIRST: columns >= valid
// (a multiple of 8) re-read column 0, and rows of k >= kvalid are zero.
// base2: second panel (K_LAST B of a gated product).
struct Operand {
    const char *base, *base2;
    size_t ld;
    int valid, kvalid;
};

// W rows (columns) of one operand in a slot, PANELS of them: the addresses
// of its loads and of a wave's NQ fragments (of one panel).  ZK: K is ragged
// (kvalid holds).
template <bool KF, int W, int PANELS, int NQ, bool ZK>
struct Side {
    static constexpr int UNITS = W * 8 * PANELS;     // 16-byte units a stage
    static constexpr int LOADS = UNITS / 256;        // per wave and stage
    static constexpr int PER = W / 32;               // loads of one panel
    static constexpr int READS = KF ? 2 : 1;         // per fragment
    static constexpr int CPK = W / 8;                // K_FIRST: chunks per k
    static constexpr int KSTEP = 256 / CPK;          // K_FIRST: k per load
    static_assert(!KF || ((W == 64 || W == 128 || W == 256) && PANELS == 1), "");
    static_assert(W % 32 == 0, "whole loads");

    const char *base, *base2;
    size_t ld;
    uint32_t off[KF ? 2 : PER];
    int kl, kvalid;

    // the swizzle of k row k, in 32-byte pieces
    static __device__ __forceinline__ int swz(int k) {
        return W == 64 ? ((k >> 1) & 1) | ((k >> 2) & 2) : (k & 3) | ((k >> 1) & 4);
    }

    __device__ __forceinline__ void init(const Operand &o, int wave, int lane) {
        base = o.base;
        base2 = PANELS > 1 ? o.base2 : o.base;
        ld = o.ld;
        kvalid = ZK ? o.kvalid : 0;
        if (KF) {
            kl = (wave * 64 + lane) / CPK;           // + KSTEP q
            const int cs = lane % CPK;
#pragma unroll
            for (int v = 0; v < 2; ++v) {            // even and odd loads
                const int f = swz(kl + v * KSTEP);
                int c = ((cs >> 1) ^ f) * 2 + (cs & 1);
                if (c * 8 >= o.valid) c = 0;
                off[v] = (uint32_t)(kl * (uint32_t)ld + c * 16);
            }
        } else {
            kl = 0;
            const int lr = lane >> 3;
            const int ch = (lane & 7) ^ ((4 * wave + (lr >> 1)) & 7);
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                int rr = (wave + 4 * q) * 8 + lr;
                if (rr >= o.valid) rr = 0;
                off[KF ? 0 : q] = (uint32_t)(rr * (uint32_t)ld + ch * 16);
            }
        }
    }

    // load q of stage s into the slot's part of this operand (at unit u0)
    __device__ __forceinline__ void load(int s, int q, u32x4 *st, int u0, int wave) const {
        if (KF) {
            const int k0 = s * SK + q * KSTEP;
            const char *p = base + (size_t)k0 * ld + off[q & 1];
            if (ZK && k0 + kl >= kvalid) p = zero_line + (threadIdx.x & 63) * 16;
            dma16(p, st + (u0 + (q * 4 + wave) * 64));
        } else {
            const char *b = PANELS > 1 && q >= PER ? base2 : base;
            dma16(b + (size_t)s * (SK * 2) + off[KF ? 0 : q % PER],
                  st + (u0 + (wave + 4 * q) * 64));
        }
    }

    // Slot index of this lane's part of fragment q (16 rows from row
    // r0 + 16 q) at sub-step 0, in reads (8 bytes for K_FIRST, else 16),
    // K_LAST: for both sub-steps.  Opaque, so that a read is one index off
    // the slot: through longer address arithmetic the compiler loses track
    // of which slot is read, and waits for every load in flight.
    int rd[KF ? NQ : 2];
    __device__ __forceinline__ void init_reads(int u0, int r0, int lane) {
        const int l16 = lane & 15, b = lane >> 4;
#pragma unroll
        for (int q = 0; q < (KF ? NQ : 2); ++q) {
            if (KF) {
                const int k = 8 * b + (l16 >> 2);
                rd[q] = u0 * 2 + k * (W / 4) + ((((r0 >> 4) + q) ^ swz(k)) * 4) + (l16 & 3);
            } else {
                rd[q] = u0 + (r0 + l16) * 8 + ((q * 4 + b) ^ ((l16 >> 1) & 7));
            }
            asm("" : "+v"(rd[q]));
        }
    }
    // part h of fragment q, sub-step kk; row0: rows from r0 on (K_LAST)
    __device__ __forceinline__ void read(bf16x8 &f, const u32x4 *st, int kk, int q,
                                         int row0, int h) const {
        if (KF) {
            const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4 *)st +
                (rd[KF ? q : 0] + (kk * 32 + 4 * h) * (W / 4)));
            s16x8 w = __builtin_bit_cast(s16x8, f);
            const s16x8 x = __builtin_shufflevector(v, v, 0, 1, 2, 3, 0, 1, 2, 3);
            w = h == 0 ? __builtin_shufflevector(x, w, 0, 1, 2, 3, 12, 13, 14, 15)
                       : __builtin_shufflevector(w, x, 0, 1, 2, 3, 12, 13, 14, 15);
            f = __builtin_bit_cast(bf16x8, w);
        } else {
            f = as_bf16x8(st[rd[kk] + row0 * 8]);
        }
    }
};

// A tile of WM x WN waves of RB x TN 16 x 16 blocks (times B's PANELS).
template <int RB, int TN, int WM, int WN, int PANELS, bool AF, bool BF, bool ZK,
          bool ODD>
struct Product {
    static_assert(WM * WN == 4, "four waves");
    static constexpr int BM = RB * 16 * WM, BN = TN * 16 * WN;
    typedef Side<AF, BM, 1, RB, ZK> SA;
    typedef Side<BF, BN, PANELS, TN, ZK> SB;
    static constexpr int STAGE = SA::UNITS + SB::UNITS;
    static constexpr int NC = TN * PANELS;           // column blocks a wave
    static constexpr int NM = RB * NC;               // MFMAs per sub-step
    static constexpr int NA = RB * SA::READS, NR = NA + NC * SB::READS;
    static constexpr int NL = SA::LOADS + SB::LOADS;
    // reads go between the first three quarters of the MFMAs, loads between
    // all of them
    // (item z of n in `span` slots goes to slot z * span / n; first(q) is
    // the first item at or after slot q)
    static constexpr int RSPAN = NM * 3 / 4;
    static constexpr int first(int q, int n, int span) {
        const int z = (q * n + span - 1) / span;
        return z < n ? z : n;
    }
    static constexpr int MAXR = (NR + RSPAN - 1) / RSPAN;
    static constexpr int MAXL = (NL + NM - 1) / NM;

    // acc += A B over KT stages.  Leaves loads in flight and both slots in
    // use: wait and barrier before using the slots for anything else.
    static __device__ __forceinline__ void run(floatx4 (&acc)[RB][NC], const Operand &oa,
                                               const Operand &ob, u32x4 *slot0,
                                               u32x4 *slot1, int KT, int wave,
                                               int lane) {
        if (KT <= 0) return;
        const int wm = wave / WN, wn = wave % WN;
        SA a;
        SB b;
        a.init(oa, wave, lane);
        b.init(ob, wave, lane);
        a.init_reads(0, wm * RB * 16, lane);
        b.init_reads(SA::UNITS, wn * TN * 16, lane);
        auto load = [&](int s, u32x4 *st, int q) __attribute__((always_inline)) {
            if (q < SA::LOADS) a.load(s, q, st, 0, wave);
            else b.load(s, q - SA::LOADS, st, SA::UNITS, wave);
        };
        auto read = [&](bf16x8 (&fa)[RB], bf16x8 (&fb)[NC], const u32x4 *st, int kk,
                        int r) __attribute__((always_inline)) {
            if (r < NA) {
                const int q = r / SA::READS;
                a.read(fa[q], st, kk, q, q * 16, r % SA::READS);
            } else {
                const int q = (r - NA) / SB::READS;
                b.read(fb[q], st, kk, q % TN, (q / TN) * BN + (q % TN) * 16,
                       (r - NA) % SB::READS);
            }
        };
        bf16x8 fa0[RB], fb0[NC], fa1[RB], fb1[NC];
        __builtin_amdgcn_s_waitcnt(0);
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int q = 0; q < NL; ++q) load(0, slot0, q);
#pragma unroll
        for (int q = 0; q < NL; ++q) load(min(1, KT - 1), slot1, q);
        wait_vmcnt<NL>();
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int r = 0; r < NR; ++r) read(fa0, fb0, slot0, 0, r);

        auto stage = [&](int s, u32x4 *cur, u32x4 *nxt) __attribute__((always_inline)) {
            __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));   // lgkmcnt(0)
#pragma unroll
            for (int q = 0; q < NM; ++q) {
                mfma(acc[q / NC][q % NC], fb0[q % NC], fa0[q / NC]);
#pragma unroll
                for (int u = 0; u < MAXR; ++u)
                    if (first(q, NR, RSPAN) + u < first(q + 1, NR, RSPAN))
                        read(fa1, fb1, cur, 1, first(q, NR, RSPAN) + u);
            }
            // own reads done, stage s + 1 landed, then every wave's part
            __builtin_amdgcn_s_waitcnt(0x0 | (0x7 << 4));
            __builtin_amdgcn_s_barrier();
            const int nx = min(s + 2, KT - 1);
#pragma unroll
            for (int q = 0; q < NM; ++q) {
                mfma(acc[q / NC][q % NC], fb1[q % NC], fa1[q / NC]);
#pragma unroll
                for (int u = 0; u < MAXR; ++u)
                    if (first(q, NR, RSPAN) + u < first(q + 1, NR, RSPAN))
                        read(fa0, fb0, nxt, 0, first(q, NR, RSPAN) + u);
#pragma unroll
                for (int u = 0; u < MAXL; ++u)
                    if (first(q, NL, NM) + u < first(q + 1, NL, NM))
                        load(nx, cur, first(q, NL, NM) + u);
            }
        };
        // wait states that the compiler does not know the asm needs: before
        // the first MFMA (a VALU write of its accumulator) and after the
        // last (a read of its result)
        // ODD: KT may be odd.  (A way round the loop that skips a stage
        // leaves loads into slot0 to be waited for at its head.)
        for (int s = 0; s < KT; s += 2) {
            asm volatile("s_nop 4");
            stage(s, slot0, slot1);
            if (!ODD || s + 1 < KT) stage(s + 1, slot1, slot0);
            asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7");
        }
    }
};

template <int RB, int NC>
__device__ __forceinline__ void clear(floatx4 (&acc)[RB][NC]) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < NC; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
}

}  // namespace mt
