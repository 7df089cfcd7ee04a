// What ds_gemm_fp8's two kernels share: gemm_fp8.cu (up to 128 rows of X) and
// gemm_fp8_wide.cu (more).
#pragma once

#include "internal.h"

namespace ds {

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

// The split tiles' steps are cut into runs, one a CTA (a pair), of four steps at
// least, or a tile's if it has fewer: joining what shorter ones leave takes
// longer than they do (333 rows by 1,000 x 1,416 in runs of one or two: 21 us,
// of four 11).  `most`: runs that meet in a tile at most, where one CTA adds them
// up.  Steps times runs stay below 2^32: fewer split tiles than CTAs, 2^17 steps
// a tile.
__host__ __device__ inline unsigned f8_runs(int split, int kb, int grid, int most) {
    const long long w = (long long)split * kb;
    long long r = w / 4 < split ? split : w / 4;
    if (r > grid) r = grid;
    if (most && r > (long long)split * (most - 1)) r = (long long)split * (most - 1);
    return r < 1 ? 1u : (unsigned)r;
}
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

constexpr int kF8WideRows = 256, kF8WideFeatures = 256;  // a pair's tile
// More rows of X than this run on pairs of SMs.
constexpr int kF8Narrow = 128;
size_t f8_wide_partial_floats(int split);
int f8_wide_pairs();
cudaError_t f8_wide_launch(F8Args &a, cudaStream_t stream);

}  // namespace ds
