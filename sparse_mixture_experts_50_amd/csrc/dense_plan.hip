// How the dense layer's products are cut into tiles and ranges of K: host
// code, functions of the sizes alone (for 256 CUs), as workspaces depend on
// them.
#include "dense.h"

namespace {

constexpr int CUS = 256;

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Time estimates in us, fitted to kernel times: stage[o - 1] is one 64-deep
// stage of a tile while o tiles share a CU, tile a tile's start and epilogue.
struct Cost {
    int occupancy;
    double stage[4], tile;
};
// Tiles in rounds of all CUs' places; the last one's share what they find.
double product_us(const Cost &c, long long units, int per) {
    const long long places = (long long)CUS * c.occupancy, rounds = units / places;
    const int rest = ceil_div(units - rounds * places, CUS);
    return 2.5 + rounds * (c.stage[c.occupancy - 1] * per + c.tile) +
           (rest ? c.stage[rest - 1] * per + c.tile : 0.0);
}
// The same for one place a CU, where the last nt2 columns of tiles are lower:
// us1 a tile of mt * nt1, then us2 of mt2 * nt2, first by those with one less.
double two_heights_us(double us1, long long tiles1, double us2, long long tiles2) {
    const long long r1 = tiles1 / CUS, rest1 = tiles1 % CUS;
    const long long r2 = tiles2 / CUS, rest2 = tiles2 % CUS;
    double most = 0;
    for (int o = 0; o < CUS; ++o) {
        const long long place = (o - rest1 + CUS) % CUS, n2 = r2 + (place < rest2);
        const double us = (r1 + (o < rest1)) * us1 + n2 * us2 + (n2 && r1 + rest1 ? 2.0 : 0.0);
        most = us > most ? us : most;
    }
    return 2.5 + most;
}
// Planes of fp32 sums, written and read, and the launch that joins them.
double plane_us(double elements, int splits) {
    return splits > 1 ? 6.0 + elements * splits * 8.0 / 7e6 : 0.0;
}

// The best number of ranges of `stages`, at least two stages each; even: of
// an even number of stages.
template <typename F>
int best_splits(int stages, int most, bool even, double &us, int &per, F cost) {
    int best = 0;
    for (int s = 1; s <= most; ++s) {
        int len = ceil_div(stages, s);
        if (s > 1 && even) len = (len + 1) & ~1;
        if (s > 1 && (len < 2 || (even && (stages & 1)) || (s - 1) * (long long)len >= stages))
            continue;
        const double t = cost(s, len);
        if (best == 0 || t < us) {
            us = t;
            best = s;
            per = len;
        }
    }
    return best;
}

// Row blocks per wave of tiles of one height that M rows need: an even split
// into ceil(M / 256) tiles, rounded up to 4, 6, 7 or 8.
int split_blocks(int M) {
    const int m = ceil_div(M, 256);
    const int rb = (ceil_div(M, m) + 31) >> 5;
    return rb <= 4 ? 4 : rb <= 6 ? 6 : rb;
}

// The best tiles, and their time.
DensePlan tiles_plan(int dtype, int M, int N, int K, int panels, bool two, double &us) {
    DensePlan p = {};
    p.rb = 2;
    p.splits = 1;
    const int stages = K / 64;
    const double elements = (double)M * N * panels;
    if (dtype != 1) {
        p.small = true;
        p.mt = ceil_div(M, 64);
        p.nt = ceil_div(N, 64 / panels);
        // (4096 x 4096 x 4096: 4096 tiles 962 us; 2048 x 2048 x 2048: 1024
        // 127; 1021 x 1984 x 1024: 496 37; 512 x 1024 x 2048: 128 51, in four
        // ranges 25)
        const int n = two ? 2 : 1;
        const Cost c = {4, {1.5 * n, 2.05 * n, 3.2 * n, 3.85 * n}, 2.0};
        double big = 0;
        p.splits = best_splits(stages, 16, false, us, p.per, [&](int s, int len) {
            return product_us(c, (long long)p.mt * p.nt * s, len) + plane_us(elements, s);
        });
        if (N < 128 / panels) return p;
        // (of those: 944 us, 127, 64, 122 and 40)
        const Cost l = {2, {3.7 * n, 7.25 * n}, 3.0};
        DensePlan b = p;
        b.small = false;
        b.mt = ceil_div(M, 128);
        b.nt = ceil_div(N, 128 / panels);
        b.splits = best_splits(stages, 16, false, big, b.per, [&](int s, int len) {
            return product_us(l, (long long)b.mt * b.nt * s, len) + plane_us(elements, s);
        });
        // (as good: the small ones share launches)
        if (big < 0.98 * us) {
            us = big;
            return b;
        }
        return p;
    }
    const int all = two ? 2 * stages : stages;
    // small tiles
    DensePlan a = p;
    a.small = true;
    a.mt = ceil_div(M, 64);
    a.nt = ceil_div(N, 128 / panels);
    {
        // (512 x 4096 x 4096: 256 tiles 25 us; 1024 x 4096 x 4096: 512 41;
        // 2048 x 8192 x 1024: 2048 45)
        const Cost c = {2, {0.3, 0.57}, 2.0};
        const long long tiles = (long long)a.mt * a.nt;
        a.splits = best_splits(all, 16, false, us, a.per, [&](int s, int len) {
            return product_us(c, tiles * s, len) + plane_us(elements, s);
        });
    }
    if (M <= 64 || N < 256 / panels) return a;
    DensePlan b = p;
    b.rb = split_blocks(M);
    b.mt = ceil_div(M, 256);
    b.nt = ceil_div(N, 256 / panels);
    double big = 0;
    {
        // (8192 x 7168 x 2048: 896 tiles 185 us; 2048 x 8192 x 1024: 256 31;
        // with half of the CUs at work the clock is higher: 2048 x 4096 x
        // 4096: 128 tiles 73.  With the small tiles 275, 45 and 75.)
        const long long tiles = (long long)b.mt * b.nt;
        b.splits = best_splits(all, 16, true, big, b.per, [&](int s, int len) {
            const double rate = tiles * s <= CUS / 2 ? 1.08 : 1.4;
            const Cost c = {1, {rate * (0.3 + 0.7 * b.rb / 8)}, 6.0};
            return product_us(c, tiles * s, len) + plane_us(elements, s);
        });
    }
    if (big > us) return a;
    if (b.splits == 1 && b.rb == 8) {
        // lower tiles in the last columns, where they leave less of the last
        // round empty (8192 x 7168 x 2048 with a residual, 896 tiles: 227 us,
        // the last 128 as 256 of half the height 218; 5100 x 4480 x 1024: 60
        // and 54)
        auto tile_us = [&](int rb) { return 1.4 * (0.3 + 0.7 * rb / 8) * all + 6.0; };
        const DensePlan whole = b;
        for (int n = 1; n <= whole.nt && n <= 32; ++n) {
            const int rb2 = 4, mt2 = ceil_div(M, 32 * rb2);
            const double t = two_heights_us(tile_us(whole.rb), (long long)whole.mt * (whole.nt - n),
                                            tile_us(rb2), (long long)mt2 * n);
            if (t < big * 0.97) {
                big = t;
                b.rb2 = rb2;
                b.mt2 = mt2;
                b.nt2 = n;
            }
        }
    }
    us = big;
    return b;
}

// The kernel for few rows: a block's runs of 16 columns, its rows of x and of
// the weights at 90 GB/s and its MFMAs, or all weights at the memory's rate.
double stream_us(int dtype, int M, int N, int K, int panels) {
    const int units = N / 16, per = ceil_div(units, 512), rows = ceil_div(M, 16);
    const double es = dtype == 1 ? 2 : 4, products = (double)rows * panels * K;
    const double block = per * ((rows + panels) * 16 * K * es / 90e3 +
                                products * (dtype == 1 ? 1 / 128.0 * 16 : 1 / 16.0 * 32) / 2400);
    const double all = N * es * panels * K / 5.2e6;
    return 3.0 + (block > all ? block : all);
}

}  // namespace

DensePlan dense_rows_plan(int dtype, int M, int N, int K, int panels, bool bk, bool two) {
    double us = 0;
    const DensePlan p = tiles_plan(dtype, M, N, K, panels, two, us);
    if (bk || M > 64) return p;
    // few columns leave most CUs without a block, where tiles have ranges of K
    // (45 x 128 x 8000, bf16: 17 us, in ranges 10; 64 x 4096 x 14336 37 and 31;
    // 64 x 1024 x 8192, fp32: 60 and 20)
    const double stream = stream_us(dtype, M, N, K, panels);
    const double all = 3.0 + (double)N * panels * K * (dtype == 1 ? 2 : 4) / 4.5e6;
    if ((us > all ? us : all) < stream) return p;
    DensePlan s = {};
    s.stream = true;
    s.rb = 2;
    s.splits = 1;
    return s;
}

size_t dense_weights_plan(DenseWeights &p, int dtype) {
    const int stages = ceil_div(p.M, 64);
    double elements = 0;
    bool big = dtype == 1;
    for (int k = 0; k < p.count; ++k) {
        elements += (double)p.m[k].R * p.m[k].C;
        big = big && p.m[k].R >= 256 && p.m[k].C >= 256;
    }
    auto cut = [&](int tile, Cost c, double &us, int &per) {
        long long tiles = 0;
        for (int k = 0; k < p.count; ++k)
            tiles += (long long)ceil_div(p.m[k].R, tile) * ceil_div(p.m[k].C, tile);
        return best_splits(stages, 16, false, us, per, [&](int s, int len) {
            if (tile == 256) c.stage[0] = tiles * s <= CUS / 2 ? 1.08 : 1.45;
            return product_us(c, tiles * s, len) + plane_us(elements, s);
        });
    };
    double us = 0, us_big = 0;
    int per = 0, per_big = 0;
    if (dtype != 1) {
        p.small = true;
        // (4096 rows, 4096 x 4096: 1047 us, the large tiles 975; 6836, three of
        // 960 x 2240: 1575 tiles 790, in four ranges 727, the large tiles 742)
        p.splits = cut(64, Cost{4, {1.6, 2.2, 3.4, 4.05}, 2.0}, us, p.per);
        const int s = cut(128, Cost{2, {3.9, 7.55}, 3.0}, us_big, per_big);
        if (us_big < 0.98 * us) {
            p.small = false;
            p.splits = s;
            p.per = per_big;
        }
    } else {
        p.small = true;
        // (4096 rows, 1024 x 1024: 64 tiles 43 us, in four ranges 23; 2048 x
        // 2048: 256 tiles 52; 4096 x 4096: 1024 137 us, the large tiles 98)
        p.splits = cut(128, Cost{2, {0.7, 1.05}, 2.5}, us, per);
        p.per = per;
        if (big) {
            const int s = cut(256, Cost{1, {1.45}, 6.0}, us_big, per_big);
            if (us_big <= us) {
                p.small = false;
                p.splits = s;
                p.per = per_big;
            }
        }
    }
    size_t total = 0;
    for (int k = 0; k < p.count; ++k) {
        p.offset[k] = total;
        if (p.splits > 1) total += (size_t)p.splits * p.m[k].R * p.m[k].C;
    }
    return total;
}
