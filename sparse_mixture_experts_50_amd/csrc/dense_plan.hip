// How the dense layer's products are cut into tiles and ranges of K: host
// code, functions of the sizes alone (for 256 CUs), as workspaces depend on
// them.
#include "dense.h"

namespace {

constexpr int CUS = 256;

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Time estimates in us.  Each tile of a round runs beside the others.
struct Cost {
    double stage;             // one 64-deep stage of a tile
    double tile;              // start and epilogue
    int places;               // tiles at a time
};

double product_us(const Cost &c, long long units, int per) {
    return ceil_div(units, c.places) * (c.tile + per * c.stage);
}
// Planes of fp32 sums, written and read, and the launch that joins them.
double plane_us(double elements, int splits) {
    return splits > 1 ? 4.0 + elements * splits * 8.0 / 4e6 : 0.0;
}

// The best number of ranges of `stages`, at least four stages each; even: of
// an even number of stages.
template <typename F>
int best_splits(int stages, int most, bool even, double &us, int &per, F cost) {
    int best = 0;
    for (int s = 1; s <= most; ++s) {
        int len = ceil_div(stages, s);
        if (s > 1 && even) len = (len + 1) & ~1;
        if (s > 1 && (len < 4 || (even && (stages & 1)) || (s - 1) * (long long)len >= stages))
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

}  // namespace

DensePlan dense_rows_plan(int dtype, int M, int N, int K, int panels, bool bk, bool two) {
    DensePlan p = {};
    p.rb = 2;
    p.splits = 1;
    if (M <= 64 && !bk) {
        p.stream = true;
        return p;
    }
    const int stages = K / 64;
    if (dtype != 1) {
        p.small = true;
        p.mt = ceil_div(M, 64);
        p.nt = N / 64;
        const long long tiles = (long long)p.mt * p.nt;
        const Cost c = {3.0 * panels * (two ? 2 : 1), 4.0, 4 * CUS};
        double us = 0;
        p.splits = best_splits(stages, 16, false, us, p.per, [&](int s, int len) {
            return product_us(c, tiles * s, len) + plane_us((double)M * N * panels, s);
        });
        return p;
    }
    const int all = two ? 2 * stages : stages;
    // small tiles
    DensePlan a = p;
    a.small = true;
    a.mt = ceil_div(M, 64);
    a.nt = ceil_div(N, 128 / panels);
    double us = 0;
    const double elements = (double)M * N * panels;
    {
        const Cost c = {0.9, 3.0, 2 * CUS};
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
        const Cost c = {0.6 + 1.4 * b.rb / 8, 6.0, CUS};
        const long long tiles = (long long)b.mt * b.nt;
        b.splits = best_splits(all, 16, true, big, b.per, [&](int s, int len) {
            return product_us(c, tiles * s, len) + plane_us(elements, s);
        });
    }
    return big <= us ? b : a;
}

size_t dense_weights_plan(DenseWeights &p, int dtype) {
    const int stages = ceil_div(p.M, 64);
    double elements = 0;
    bool big = dtype == 1;
    for (int k = 0; k < p.count; ++k) {
        elements += (double)p.m[k].R * p.m[k].C;
        big = big && p.m[k].R >= 256 && p.m[k].C >= 256;
    }
    auto cut = [&](int tile, const Cost &c, double &us, int &per) {
        long long tiles = 0;
        for (int k = 0; k < p.count; ++k)
            tiles += (long long)ceil_div(p.m[k].R, tile) * ceil_div(p.m[k].C, tile);
        return best_splits(stages, 16, false, us, per, [&](int s, int len) {
            return product_us(c, tiles * s, len) + plane_us(elements, s);
        });
    };
    double us = 0, us_big = 0;
    int per = 0, per_big = 0;
    if (dtype != 1) {
        p.small = true;
        p.splits = cut(64, Cost{3.0, 4.0, 4 * CUS}, us, p.per);
    } else {
        p.small = true;
        p.splits = cut(128, Cost{1.5, 4.0, 2 * CUS}, us, per);
        p.per = per;
        if (big) {
            const int s = cut(256, Cost{2.0, 8.0, CUS}, us_big, per_big);
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
