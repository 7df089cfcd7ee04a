// What ds_gemm_fp8's two kernels share: gemm_fp8.cu (few rows of X) and
// gemm_fp8_wide.cu (many).
#pragma once

#include "internal.h"

namespace ds {

constexpr int kF8WideRows = 256, kF8WideFeatures = 256;  // a pair's tile

struct F8Args {
    CUtensorMap tw, tx;  // bytes, boxes {128, a tile's features} and {128, bn} (wide: {128, 128} both), 128-byte swizzle
    const float *ws, *xs;
    int rows, n, kb;
    int bn;              // columns of an MMA: rows of X, or features (wide)
    int m_tiles, n_tiles;
    int rounds, split;   // whole tiles a CTA (a pair) takes; tiles behind them that are cut
    unsigned runs;       // into so many runs
    void *y;
    int y_dtype;
    long long ldy;
    float *partials;
    int *counters;       // a split tile's arrivals, zero between launches
    int *err;
};

// The split tiles' steps are cut into runs, one a CTA (a pair): as many a tile as
// cost least, counted in steps.  A tile in one run costs its steps; cut, the
// partial sums' way out, their counting and their joining take as long as some
// twelve steps (with the pairs' second launch 18, and a sixth for each run), and
// more for every few that are joined: 64 rows by 4,096 x 4,096 take 15.6 us with
// one run a tile, 12.0 with three, 15.2 with seven.  Runs of equal length without
// regard to the tiles leave most CTAs the parts of two, with an end and a partial
// sum each: 64 rows by 28,672 x 4,096 take 29.9 us like that, with 112 CTAs of 152
// and a tile each 22.5; 28,672 x 1,024 15.7 and 8.1.  They pay where whole tiles
// would leave many SMs idle for long.  (Measured on three matrices in turn, which
// fit L2 together but for those of 28,672 x 4,096: of the smaller ones' steps from
// HBM a join may cost fewer.)  Steps times runs stay below 2^32: fewer split tiles
// than CTAs, 2^17 steps a tile.
inline unsigned f8_runs(int split, int kb, int ctas, int bn) {
    if (split == 0) return 1;
    const auto join = [&](int m) {  // of m partial sums a tile
        return bn == kF8WideFeatures ? 18 + split * m / 6 + 9 * ((m - 1) / 6) : bn >= 64 ? 12 + 7 * ((m - 1) / 3) : 12 + 3 * ((m - 1) / 4);
    };
    unsigned best = (unsigned)split;
    int least = kb;
    for (int m = 2; m <= kb && m * split <= ctas; ++m) {
        const int cost = (kb + m - 1) / m + join(m);
        if (cost < least) least = cost, best = (unsigned)(m * split);
    }
    const long long steps = (long long)split * kb;
    if (steps >= ctas && steps / ctas + 24 + join(ctas / split + 1) < least) best = (unsigned)ctas;
    return best;
}
// Whether there are partial sums.
inline bool f8_cut(int split, unsigned runs) { return split > 0 && runs != (unsigned)split; }
// The first and last run that hold steps of a split tile.
__device__ __forceinline__ void f8_contributors(const F8Args &p, int split, int &first, int &last) {
    const unsigned w = (unsigned)p.split * p.kb, t = (unsigned)split * p.kb;
    first = (int)(((t + 1) * p.runs - 1) / w);
    last = (int)(((t + p.kb) * p.runs - 1) / w);
}

// A run's segments: whole tiles in rounds, then its steps of the split tiles.
struct F8Seg {
    int tile, k0, k1;
    int split;  // number of the split tile, or -1 (a whole tile)
};
struct F8Walk {
    int id, grid, round = 0;
    unsigned u, u1;
    __device__ F8Walk(const F8Args &p, int id_, int grid_) : id(id_), grid(grid_) {
        const unsigned w = (unsigned)p.split * p.kb;
        u = w * min((unsigned)id, p.runs) / p.runs;
        u1 = w * min((unsigned)id + 1, p.runs) / p.runs;
    }
    __device__ bool next(const F8Args &p, F8Seg &s) {
        if (round < p.rounds) {
            s.tile = id + grid * round++;
            s.k0 = 0;
            s.k1 = p.kb;
            s.split = -1;
            return true;
        }
        if (u >= u1) return false;
        s.split = (int)(u / (unsigned)p.kb);
        s.tile = p.rounds * grid + s.split;
        s.k0 = (int)(u - (unsigned)s.split * p.kb);
        s.k1 = min(p.kb, s.k0 + (int)(u1 - u));
        u += s.k1 - s.k0;
        if (s.k0 == 0 && s.k1 == p.kb) s.split = -1;
        return true;
    }
};

// Adds `parts` partial sums of C columns, COLS floats apart, in order; several
// partials' loads under way at a time.
template <int C, int COLS>
__device__ __forceinline__ void f8_join(const float *from, size_t part, int parts, float (&acc)[C]) {
    constexpr int AT = C >= 32 ? 3 : C >= 16 ? 4 : 6;
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] = 0.0f;
    for (int c = 0; c < parts; c += AT) {
        float v[AT][C];
#pragma unroll
        for (int a = 0; a < AT; ++a)
#pragma unroll
            for (int i = 0; i < C; ++i) v[a][i] = __ldcg(from + (size_t)min(c + a, parts - 1) * part + i * COLS);
#pragma unroll
        for (int a = 0; a < AT; ++a)
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] += c + a < parts ? v[a][i] : 0.0f;
    }
}

// Pairs of SMs take more than 128 rows of X, and more than 64 unless the features
// are more tiles than pairs (the other kernel's tiles have as many features and
// twice as many CTAs): 128 rows by 4,096 x 4,096 take 15.9 us against 19.8, 65 by
// 14,336 x 4,096 17.4 against 22.3, 128 by 28,672 x 4,096 33.7 against 27.0.
constexpr int kF8Narrow = 64, kF8NarrowMost = 128;
size_t f8_wide_partial_floats(int split, unsigned runs);
int f8_wide_pairs();
cudaError_t f8_wide_launch(const F8Args &a, int pairs, cudaStream_t stream);

}  // namespace ds
