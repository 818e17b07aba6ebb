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

#include <type_traits>

#include "common.h"

namespace mt {

constexpr int SK = 64;                   // stage depth

// A tile's number of stages.
enum Stages { EVEN, ODD, NONE };

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// 64 lanes' 16 bytes at base (uniform) + off (the lane's) to LDS.
__device__ __forceinline__ void dma16(uint64_t base, uint32_t off, u32x4 *lds) {
    typedef const __attribute__((address_space(1))) char *gptr;
    __builtin_amdgcn_global_load_lds(
        (const __attribute__((address_space(1))) void *)((gptr)base + off),
        (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}

// The same from any address of the lane's.
__device__ __forceinline__ void dma16_lanes(const char *src, u32x4 *lds) {
    __builtin_amdgcn_global_load_lds(
        (const void *)src, (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}

// Waits until at most N memory operations (63: the counter's range) of the
// wave are outstanding; they end in order.
template <int N> __device__ __forceinline__ void wait_loads() {
    constexpr int n = N < 63 ? N : 63;
    __builtin_amdgcn_s_waitcnt((n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// HAND: as volatile asm.  The compiler then keeps the issue order as written
// and 256 accumulators in AGPRs (the builtin splits them between AGPRs and
// VGPRs and copies them back and forth every step), but knows nothing of the
// wait states around an MFMA: only for straight loops over a register file
// full of accumulators, where it has no room and no reason to copy one.
// Tiles of fewer accumulators use the builtin.
template <bool HAND>
__device__ __forceinline__ void mfma(floatx4 &acc, const bf16x8 &a, const bf16x8 &b) {
    if (HAND)
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    else
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}

// W rows (columns) of one operand in a slot from unit U0 on, PANELS of them:
// a wave's loads of a stage.  A load's address is a uniform base, one per
// operand and stage, and a 32-bit lane offset that stays in a register for
// the whole kernel: with one wave per SIMD an MFMA leaves issue slots for
// about three other instructions, and address arithmetic would take them.
template <bool KF, int W, int PANELS, int U0>
struct Loader {
    static constexpr int UNITS = W * 8 * PANELS;     // 16-byte units a stage
    static constexpr int LOADS = UNITS / 256;        // per wave and stage
    static constexpr int PER = W / 32;               // loads of one panel
    static constexpr int CPK = W / 8;                // K_FIRST: chunks per k
    static constexpr int KSTEP = 256 / CPK;          // K_FIRST: k per load
    static_assert(!KF || ((W == 64 || W == 128 || W == 256) && PANELS == 1), "");
    static_assert(W % 32 == 0, "whole loads");

    // K_FIRST: the swizzle, and with it the lane's offset, repeats every 16
    // rows of k: loads OFFS apart differ by a uniform hop only.
    static constexpr int OFFS = !KF ? PER : W == 256 ? 2 : 1;
    static constexpr int HOP = KSTEP * OFFS;

    uint32_t off[OFFS];
    uint32_t hop;                                    // K_FIRST: HOP rows of k

    // the swizzle of k row k, in 32-byte pieces
    static __device__ __forceinline__ int swz(int k) {
        return W == 64 ? ((k >> 1) & 1) | ((k >> 2) & 2) : (k & 3) | ((k >> 1) & 4);
    }

    // ld: bytes between rows (of k: K_FIRST); valid < W: rows (K_FIRST:
    // columns, a multiple of 8) from valid on re-read the first
    __device__ __forceinline__ void init(uint32_t ld, int valid, int wave, int lane) {
        hop = KF ? HOP * ld : 0;
#pragma unroll
        for (int q = 0; q < OFFS; ++q) {
            if (KF) {
                const int k = (wave * 64 + lane) / CPK + KSTEP * q;
                const int cs = lane % CPK;
                int c = ((cs >> 1) ^ swz(k)) * 2 + (cs & 1);
                if (c * 8 >= valid) c = 0;
                off[q] = (uint32_t)k * ld + (uint32_t)(c * 16);
            } else {
                const int lr = lane >> 3;
                const int ch = (lane & 7) ^ ((4 * wave + (lr >> 1)) & 7);
                int rr = (wave + 4 * q) * 8 + lr;
                if (rr >= valid) rr = 0;
                off[q] = (uint32_t)rr * ld + (uint32_t)(ch * 16);
            }
        }
    }
    // bytes from a stage to the next
    static __device__ __forceinline__ uint32_t step(uint32_t ld) {
        return KF ? SK * ld : SK * 2;
    }
    // the lane's offset in load q
    __device__ __forceinline__ uint32_t at(int q) const {
        return off[q % OFFS] + (KF ? hop * (uint32_t)(q / OFFS) : 0u);
    }
    // load q of the stage at base (and base2, the second panel's)
    __device__ __forceinline__ void load(uint64_t base, uint64_t base2, int q, u32x4 *st,
                                         int wave) const {
        uint32_t o = off[q % OFFS];
        // opaque: else the offsets, widened to 64 bits, are kept as well
        asm("" : "+v"(o));
        dma16((PANELS > 1 && q >= PER ? base2 : base) +
                  (KF ? hop * (uint32_t)(q / OFFS) : 0u), o,
              st + (U0 + (KF ? q * 4 + wave : wave + 4 * q) * 64));
    }
};

// A wave's NQ fragments (16 rows each from row r0 on) of one operand (of
// one panel).
template <bool KF, int W, int U0, int NQ>
struct Reader {
    static constexpr int READS = KF ? 2 : 1;         // per fragment
    // Slot index of this lane's part of fragment q at sub-step 0, in reads
    // (8 bytes for K_FIRST, else 16); K_LAST: of fragment 0, both sub-steps.
    // Opaque, so that a read is one index off the slot: through longer
    // address arithmetic the compiler loses track of which slot is read, and
    // waits for every load in flight.
    int rd[KF ? NQ : 2];
    __device__ __forceinline__ void init(int r0, int lane) {
        const int l16 = lane & 15, b = lane >> 4;
#pragma unroll
        for (int q = 0; q < (KF ? NQ : 2); ++q) {
            if (KF) {
                const int k = 8 * b + (l16 >> 2);
                rd[q] = U0 * 2 + k * (W / 4) +
                        ((((r0 >> 4) + q) ^ (Loader<KF, W, 1, U0>::swz(k))) * 4) + (l16 & 3);
            } else {
                rd[q] = U0 + (r0 + l16) * 8 + ((q * 4 + b) ^ ((l16 >> 1) & 7));
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

// Tiles of up to BM x BN (times B's PANELS), WM x WN waves.  SPLIT: the sum
// of two products one after the other.
template <int BM, int BN, int WM, int WN, int PANELS, bool AF, bool BF, bool SPLIT = false>
struct Tiles {
    static_assert(WM * WN == 4, "four waves");
    static constexpr int TN = BN / 16 / WN, NC = TN * PANELS;   // column blocks a wave
    typedef Loader<AF, BM, 1, 0> LA;
    typedef Loader<BF, BN, PANELS, LA::UNITS> LB;
    static constexpr int STAGE = LA::UNITS + LB::UNITS;

    // 256 x 256 tiles fill the AGPRs.
    static constexpr bool HAND = BM * BN * PANELS == 256 * 256;

    // The operands of one tile: element (0, 0) of each (uniform).  SPLIT:
    // a2, b2 of the second product; PANELS 2: b2 of the second panel.  kt:
    // stages (maybe 0; a stage's worth of either operand can be read all the
    // same).
    // s0: the first stage (of a range of K).
    struct Source {
        uint64_t a, b, a2, b2;
        int kt, s0;
    };
    // What the loads of every tile share.
    struct Lanes {
        LA a;
        LB b;
        uint32_t step_a, step_b;
        int split;                      // stages of the first product
        __device__ __forceinline__ void init(uint32_t lda, int valid_a, uint32_t ldb,
                                             int valid_b, int wave, int lane) {
            a.init(lda, valid_a, wave, lane);
            b.init(ldb, valid_b, wave, lane);
            step_a = LA::step(lda);
            step_b = LB::step(ldb);
        }
    };
    // A stage to load: the bases of its loads.  (Past the last stage, the
    // last again.)
    struct Stage {
        uint64_t a, b, b2;
        __device__ __forceinline__ void set(const Source &src, const Lanes &ln, int s) {
            s = max(min(s, src.kt - 1), 0) + src.s0;
            const bool second = SPLIT && s >= ln.split;
            const int n = second ? s - ln.split : s;
            a = (second ? src.a2 : src.a) + (uint64_t)n * ln.step_a;
            b = (second ? src.b2 : src.b) + (uint64_t)n * ln.step_b;
            b2 = PANELS > 1 ? src.b2 + (uint64_t)n * ln.step_b : b;
            // opaque: else the compiler adds lane offset and first base ahead
            // of the loop, and the rest by 64-bit vector additions in it
            asm("" : "+s"(a), "+s"(b));
            if (PANELS > 1) asm("" : "+s"(b2));
        }
    };
    // load l of a stage of RBA 32-row parts of A (of BM / 32) and all of B
    template <int RBA>
    static __device__ __forceinline__ void load(const Stage &g, const Lanes &ln, int l,
                                                u32x4 *st, int wave) {
        if (l < RBA) ln.a.load(g.a, g.a, l, st, wave);
        else ln.b.load(g.b, g.b2, l - RBA, st, wave);
    }
    // Asks for stage s at once.
    static __device__ __forceinline__ void load_stage(const Source &src, const Lanes &ln,
                                                      int s, u32x4 *st, int wave) {
        Stage g;
        g.set(src, ln, s);
        load_all(g, ln, st, wave);
    }

    // item z of n in `span` slots goes to slot z * span / n; first(q) is the
    // first item at or after slot q
    static constexpr int first(int q, int n, int span) {
        const int z = (q * n + span - 1) / span;
        return z < n ? z : n;
    }

    // A wave's work on a stage of a tile of RB 16-row blocks per wave.
    template <int RB> struct Worker {
        typedef Reader<AF, BM, 0, RB> RA;
        typedef Reader<BF, BN, LA::UNITS, TN> RBd;
        static constexpr int NM = RB * NC;               // MFMAs per sub-step
        static constexpr int NA = RB * RA::READS, NR = NA + NC * RBd::READS;
        // reads go between the first three quarters of the MFMAs, loads
        // between all of them
        static constexpr int RSPAN = NM * 3 / 4, MAXR = (NR + RSPAN - 1) / RSPAN;
        RA a;
        RBd b;
        bf16x8 fa0[RB], fb0[NC], fa1[RB], fb1[NC];

        __device__ __forceinline__ void read(bf16x8 (&fa)[RB], bf16x8 (&fb)[NC],
                                             const u32x4 *st, int kk, int r) {
            if (r < NA) {
                const int q = r / RA::READS;
                a.read(fa[q], st, kk, q, q * 16, r % RA::READS);
            } else {
                const int q = (r - NA) / RBd::READS;
                b.read(fb[q], st, kk, q % TN, (q / TN) * BN + (q % TN) * 16,
                       (r - NA) % RBd::READS);
            }
        }
        // Reads the first fragments, of a stage that has landed in every wave.
        __device__ __forceinline__ void begin(const u32x4 *slot0, int wave, int lane) {
            // opaque: else the indexes of several kinds of tile are worked
            // out, and kept, ahead of the branch between them
            asm volatile("" : "+v"(lane));
            a.init((wave / WN) * RB * 16, lane);
            b.init((wave % WN) * TN * 16, lane);
            __builtin_amdgcn_s_barrier();
#pragma unroll
            for (int r = 0; r < NR; ++r) read(fa0, fb0, slot0, 0, r);
        }
        // Stage in cur: its sub-step 0 on fa0 while the other half is read
        // into fa1, then sub-step 1 while nxt's first half is read into fa0
        // (unless LAST) and stage g (PARTS 32-row parts of A) is loaded into
        // cur.  AHEAD: loads that may still be in flight when the stage after
        // this one has landed.
        template <bool LAST, int PARTS, int AHEAD>
        __device__ __forceinline__ void stage(floatx4 (&acc)[RB][NC], const Stage &g,
                                              const Lanes &gl, u32x4 *cur, u32x4 *nxt,
                                              int wave) {
            constexpr int NL = PARTS + LB::LOADS;
            constexpr int MAXL = (NL + NM - 1) / NM;
            static_assert(AHEAD < 64, "vmcnt range");
            __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));   // lgkmcnt(0)
#pragma unroll
            for (int q = 0; q < NM; ++q) {
                mfma<HAND>(acc[q / NC][q % NC], fb0[q % NC], fa0[q / NC]);
#pragma unroll
                for (int u = 0; u < MAXR; ++u)
                    if (first(q, NR, RSPAN) + u < first(q + 1, NR, RSPAN))
                        read(fa1, fb1, cur, 1, first(q, NR, RSPAN) + u);
            }
            // own reads done, the next stage landed, then every wave's part
            __builtin_amdgcn_s_waitcnt((AHEAD & 0xF) | ((AHEAD >> 4) << 14) | (0x7 << 4));
            __builtin_amdgcn_s_barrier();
#pragma unroll
            for (int q = 0; q < NM; ++q) {
                mfma<HAND>(acc[q / NC][q % NC], fb1[q % NC], fa1[q / NC]);
                if (!LAST) {
#pragma unroll
                    for (int u = 0; u < MAXR; ++u)
                        if (first(q, NR, RSPAN) + u < first(q + 1, NR, RSPAN))
                            read(fa0, fb0, nxt, 0, first(q, NR, RSPAN) + u);
                }
#pragma unroll
                for (int u = 0; u < MAXL; ++u)
                    if (first(q, NL, NM) + u < first(q + 1, NL, NM))
                        load<PARTS>(g, gl, first(q, NL, NM) + u, cur, wave);
            }
        }
    };
    // Wait states that the compiler does not know the asm MFMAs need: before
    // the first (a VALU write of its accumulator) and after the last (a read
    // of its result).
    static __device__ __forceinline__ void before() {
        if (HAND) asm volatile("s_nop 4");
    }
    static __device__ __forceinline__ void after() {
        if (HAND) asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7");
    }
    // Puts every write of the accumulators above this point and every later
    // read below it (volatile asm keeps its order): above before(), or a
    // constant may be written right ahead of its MFMA, below after().  At the
    // head of each of two ways that read them: below the branch.
    template <int RB>
    static __device__ __forceinline__ void pin(floatx4 (&acc)[RB][NC]) {
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < NC; ++j)
                if (HAND) asm volatile("" : "+a"(acc[i][j]));
    }
    // All loads of stage g.
    static __device__ __forceinline__ void load_all(const Stage &g, const Lanes &ln,
                                                    u32x4 *st, int wave) {
#pragma unroll
        for (int l = 0; l < LA::LOADS + LB::LOADS; ++l) load<LA::LOADS>(g, ln, l, st, wave);
    }

    // acc += A B of a tile of RB 16-row blocks per wave over its src.kt
    // stages, the first two of which have landed in slot0 and slot1 as far as
    // this wave's part goes (asked for by load_stage(), or by this function
    // for the tile before; the caller waits, so that it need not wait for its
    // own stores): while the last two are worked on, the first two of `next`
    // are loaded.
    // RBA: 32-row parts of A that the tile's rows need.  KIND: of src.kt.
    template <int RB, int RBA, Stages KIND>
    static __device__ __forceinline__ void run(floatx4 (&acc)[RB][NC], const Source &src,
                                               const Lanes &ln, const Source &next,
                                               const Lanes &lnext, u32x4 *slot0,
                                               u32x4 *slot1, int wave, int lane) {
        Stage g, h;
        if constexpr (KIND == NONE) {
            __builtin_amdgcn_s_barrier();
            g.set(next, lnext, 0);
            h.set(next, lnext, 1);
            load_all(g, lnext, slot0, wave);
            if (next.kt > 1) load_all(h, lnext, slot1, wave);
            pin(acc);
            return;
        }
        Worker<RB> w;
        pin(acc);
        w.begin(slot0, wave, lane);
        const int kt = src.kt;
        for (int s = 0; s + 2 < kt; s += 2) {
            g.set(src, ln, s + 2);
            h.set(src, ln, s + 3);
            before();
            w.template stage<false, RBA, 0>(acc, g, ln, slot0, slot1, wave);
            w.template stage<false, RBA, 0>(acc, h, ln, slot1, slot0, wave);
            after();
        }
        g.set(next, lnext, 0);
        h.set(next, lnext, 1);
        before();
        w.template stage<KIND == ODD, LA::LOADS, 0>(acc, g, lnext, slot0, slot1, wave);
        after();
        if (KIND == EVEN) {
            before();
            w.template stage<true, LA::LOADS, 0>(acc, h, lnext, slot1, slot0, wave);
            after();
        } else if (HAND || next.kt > 1) {    // (no branch between the large tiles' AGPRs)
            load_all(h, lnext, slot1, wave);
        }
        pin(acc);
        __builtin_amdgcn_sched_barrier(0);
    }

    // f(integral_constant<Stages, KIND>) for a tile of kt stages.
    template <typename F> static __device__ __forceinline__ void by_stages(int kt, F f) {
        if (kt == 0) f(std::integral_constant<Stages, NONE>{});
        else if (!(kt & 1)) f(std::integral_constant<Stages, EVEN>{});
        else f(std::integral_constant<Stages, ODD>{});
    }

    // The same through NS slots, NS - 1 stages ahead (kt >= 1): for products
    // that stream weights through small tiles, whose stages are worked on in
    // far less time than a load takes.
    template <int RB, int NS>
    static __device__ __forceinline__ void run_ring(floatx4 (&acc)[RB][NC],
                                                    const Source &src, const Lanes &ln,
                                                    const Source &next, const Lanes &lnext,
                                                    u32x4 *const (&slot)[NS], int wave,
                                                    int lane) {
        constexpr int NL = LA::LOADS + LB::LOADS, AHEAD = (NS - 2) * NL;
        Worker<RB> w;
        pin(acc);
        w.begin(slot[0], wave, lane);
        Stage g;
        int left = src.kt;
        for (int s = NS; left > NS; s += NS, left -= NS) {
            before();
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                g.set(src, ln, s + i);
                w.template stage<false, LA::LOADS, AHEAD>(acc, g, ln, slot[i],
                                                          slot[(i + 1) % NS], wave);
            }
            after();
        }
        // the last LEFT stages, and the first NS of the next tile (one way
        // for each LEFT: joining on the way would make the compiler wait for
        // every load)
        auto finish = [&](auto count) __attribute__((always_inline)) {
            constexpr int LEFT = decltype(count)::value;
            before();
            auto one = [&](auto at) __attribute__((always_inline)) {
                constexpr int i = decltype(at)::value;
                g.set(next, lnext, i);
                if constexpr (i < LEFT)
                    w.template stage<i + 1 == LEFT, LA::LOADS, AHEAD>(
                        acc, g, lnext, slot[i], slot[(i + 1) % NS], wave);
                else
                    load_all(g, lnext, slot[i], wave);
            };
            one(std::integral_constant<int, 0>{});
            one(std::integral_constant<int, 1>{});
            one(std::integral_constant<int, 2>{});
            after();
        };
        static_assert(NS == 3, "the ways below");
        if (left == 3) finish(std::integral_constant<int, 3>{});
        else if (left == 2) finish(std::integral_constant<int, 2>{});
        else finish(std::integral_constant<int, 1>{});
        pin(acc);
        __builtin_amdgcn_sched_barrier(0);
    }
};

// Stores 16 rows of a wave's TN column blocks as bf16, whole rows of 32 TN
// bytes at a time, TN / 2 stores: the MFMA layout (lane: row l % 16, 4
// columns from 4 (l / 16)) goes through the wave's own 32 TN 16-byte units of
// LDS, from unit u0.  turn() writes and reads them, store() stores what was
// read: a wave's LDS operations run in order, so the next turn() may come
// first and hide the reads.  (Opaque indexes as in Reader: the next tile's
// loads are in flight.  Straight from the registers, in pieces of 64 bytes a
// row, the fine-grained weight gradient took 0.78 ms instead of 0.74.)
template <int TN> struct RowStore {
    static constexpr int CPR = TN * 2;           // 16-byte chunks per row
    u32x4 q[CPR / 4];
    __device__ __forceinline__ void turn(u32x4 *scr, int u0, const float (&v)[TN][4], int lane) {
        const int l16 = lane & 15, hq = lane >> 4;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            u32x2 o;
            o.x = pack_bf16x2(v[j][0], v[j][1]);
            o.y = pack_bf16x2(v[j][2], v[j][3]);
            int at = (u0 + l16 * CPR + ((j * 2 + (hq >> 1)) ^ (l16 & (CPR - 1)))) * 2 + (hq & 1);
            asm("" : "+v"(at));
            ((u32x2 *)scr)[at] = o;
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < CPR / 4; ++i) {
            const int r = i * (64 / CPR) + lane / CPR, c = lane % CPR;
            int at = u0 + r * CPR + (c ^ (r & (CPR - 1)));
            asm("" : "+v"(at));
            q[i] = scr[at];
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
    }
    __device__ __forceinline__ void store(uint16_t *out, size_t ld, int lane) const {
#pragma unroll
        for (int i = 0; i < CPR / 4; ++i)
            *(u32x4 *)(out + (size_t)(i * (64 / CPR) + lane / CPR) * ld + lane % CPR * 8) = q[i];
    }
};

// The tile of round r: persistent blocks, each XCD (block index mod 8)
// taking consecutive tiles.
__device__ __forceinline__ int tile_of(int r) {
    const int nb = gridDim.x, per = nb >> 3;
    return r * nb + (blockIdx.x & 7) * per + (blockIdx.x >> 3);
}

// The lane index, counted anew (opaque), so that neither it nor per-lane
// addresses are kept in registers across tiles.
__device__ __forceinline__ int tile_lane() {
    uint32_t ones = ~0u;
    asm volatile("" : "+s"(ones));
    return __builtin_amdgcn_mbcnt_hi(ones, __builtin_amdgcn_mbcnt_lo(ones, 0));
}

// First column of a tile: the last of an axis of n >= size ends with it, so
// that no operand is read past its end.  (What it shares with the tile before
// it is computed again, to the same bits; axes shorter than a tile have the
// small tiles, which store only their own columns.)
__device__ __forceinline__ int tile_start(int i, int size, int n) {
    return n >= size ? min(i * size, n - size) : 0;
}

inline int cus() {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        n < 8)
        return 256;
    return n / 8 * 8;
}

// Blocks of a persistent grid.
inline int grid_for(long long tiles, int per_cu) {
    const int n = cus() * per_cu;
    const long long g = (tiles + 7) / 8 * 8;
    return (int)(g < n ? (g < 8 ? 8 : g) : n);
}

template <int RB, int NC>
__device__ __forceinline__ void clear(floatx4 (&acc)[RB][NC]) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < NC; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
}

}  // namespace mt
