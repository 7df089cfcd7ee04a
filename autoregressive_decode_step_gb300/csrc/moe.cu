// A mixture-of-experts layer for few tokens in one launch (ds_moe_layer):
//   logits = x R^T;  the k largest of a token (lower index first among equals);
//   y = (residual +) sum_i w_i D[e_i] (silu(G[e_i] x) * (U[e_i] x))
// with w the softmax of the logits at the chosen experts, divided by their sum
// or not.
//
// What bounds it is the chosen experts' weight bytes, each of which is wanted
// by few tokens.  So the weights go through shared memory once, as 128 rows by
// 128 bytes of the sum a stage (64 gate and 64 up rows, or 128 down rows), and
// a stage belongs to one warp, which multiplies it with up to 32 tokens by
// mma.sync: eight warps have eight stages in hand, none waits for another
// until a tile of outputs is complete.  (tcgen05 would want 8-bit weights and
// activations in one format; here fp32 activations meet e4m3 or bf16 weights.)
// All tiles of a phase, expert after expert, are one line of stages cut into
// equal runs, one a CTA; a tile that is cut is added up by the CTA that is last.
//
// Four phases with a barrier of the whole grid between them (a cooperative
// launch; waits are bounded): logits; gate and up; down; the weighted sum.
// Every CTA draws up the tokens' choices for itself.  The copying warp goes on
// to the next phase's weights while the others wait.
//
// Digits: fp32 activations meet bf16 weights as three bf16 pieces (24 bits,
// exact), e4m3 weights as two f16 pieces behind a power of two per token and
// 128 values that brings the largest below 2^15 (22 bits, and no value loses
// more than 2^-40 of its block's largest; e4m3 is exact in f16).  Where
// outputs are bf16 the intermediate has 16 bits or more.  Sums are fp32.  The
// logits are sums of exact products with their rounding errors carried along
// (two floats, added up in 64 bits): the choice of experts is that of 64 bits.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "tc.h"

#include <cuda_fp16.h>

namespace ds {

constexpr int kMoeMaxTokens = 256, kMoeMaxExperts = 512, kMoeMaxK = 16;
constexpr int kMoeMaxPairs = kMoeMaxTokens * kMoeMaxK;
constexpr int kMoeGroup = 32;  // tokens a stage is multiplied with
constexpr int kMoeMaxJobs = kMoeMaxExperts + kMoeMaxPairs / kMoeGroup;
constexpr int kMoeWarps = 8;
constexpr int kMoeThreads = 384;  // two warpgroups that multiply, one whose first warp copies
// Registers a thread: 168 at launch (384 x 168), moved to the warps that hold
// a tile's sums: 2 x 216 + 72 = 3 x 168.
constexpr int kMoeRegsMain = 216, kMoeRegsOther = 72;
constexpr int kMoeStages = 10, kMoeStageBytes = 128 * 128;
constexpr int kMoeSums = kMoeGroup * 128;  // floats of a tile

struct MoeArgs {
    CUtensorMap tgu, td;  // {d, ff, 2 experts} boxes {128 B, 64, 1}; {ff, d, experts} boxes {128 B, 128, 1}; swizzled
    const void *x, *router, *residual;
    const float *gu_scales, *d_scales;
    void *y;
    int *ids;
    float *weights;
    int x_dtype, r_dtype;
    int n, d, ff, experts, k, renormalize;
    // workspace
    int *err, *bars, *counters;  // counters [2][grid]: arrivals at the tile that a CTA's run ends in
    double *logits;              // [n][experts]
    float *wts;                  // [n k]
    float *h;                    // [n k][ff]
    float *parts;                // [grid][2][32 x 128]
    float *out;                  // [n k][d]
};

struct MoeShared {
    uint64_t full[kMoeStages], empty[kMoeStages];
    int dead, last;
    int offset[kMoeMaxExperts + 1], jobs[kMoeMaxExperts + 1];
    unsigned short job_expert[kMoeMaxJobs];
    unsigned short list[kMoeMaxPairs];  // pairs (token * k + slot) by expert
    union {
        unsigned short chosen[kMoeMaxPairs];
        float sums[kMoeWarps][128 * 8];
    };
};
constexpr size_t kMoeSmem = 1024 + (size_t)kMoeStages * kMoeStageBytes + sizeof(MoeShared);
static_assert(kMoeSmem <= 227 * 1024, "shared memory");

// ------------------------------------------------------------------ waits
__device__ __forceinline__ bool moe_wait(uint64_t *bar, uint32_t parity, volatile int *dead, int *err) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*dead) return false;
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                flag_error(err, DS_ERR_WAIT_TIMEOUT);
                *dead = 1;
                return false;
            }
        }
    }
}
// One thread of every CTA: all of them have arrived, and what they wrote is seen.
__device__ __forceinline__ void moe_meet(int *bar, volatile int *dead, int *err) {
    __threadfence();
    atomicAdd(bar, 1);
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        int v;
        asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(bar) : "memory");
        if (v >= (int)gridDim.x || *dead) break;
        if ((it & 63u) == 0 && global_timer_ns() - t0 > kWaitLimitNs) {
            flag_error(err, DS_ERR_WAIT_TIMEOUT);
            *dead = 1;
            break;
        }
    }
    __threadfence();
}

// ------------------------------------------------------------------ router
__device__ __forceinline__ void moe_load8(const void *base, long long i, int dtype, float (&v)[8]) {
    if (dtype == DS_BF16) {
        widen16(__ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + i)), v);
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + i);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}
// s + c += a b, c holding what the roundings of the product and of s lost.
__device__ __forceinline__ void moe_dot2(float a, float b, float &s, float &c) {
    const float p = __fmul_rn(a, b), e = __fmaf_rn(a, b, -p);
    const float t = __fadd_rn(s, p), z = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(p, z))));
    s = t;
}
// One expert's logits of T tokens by a warp.
template <int T>
__device__ __forceinline__ void moe_logits(const MoeArgs &p, int e, int t0) {
    const int lane = threadIdx.x & 31;
    float s[T], c[T];
#pragma unroll
    for (int i = 0; i < T; ++i) s[i] = c[i] = 0.0f;
    for (int j = lane * 8; j < p.d; j += 256) {
        float r[8], x[T][8];
        moe_load8(p.router, (long long)e * p.d + j, p.r_dtype, r);
#pragma unroll
        for (int i = 0; i < T; ++i) moe_load8(p.x, (long long)min(t0 + i, p.n - 1) * p.d + j, p.x_dtype, x[i]);
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
            for (int q = 0; q < 8; ++q) moe_dot2(x[i][q], r[q], s[i], c[i]);
    }
#pragma unroll
    for (int i = 0; i < T; ++i) {
        // an infinite sum's lost part is NaN: the sum says it all
        double v = fabsf(s[i]) < INFINITY ? (double)s[i] + (double)c[i] : (double)s[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0 && t0 + i < p.n) p.logits[(long long)(t0 + i) * p.experts + e] = v;
    }
}

// Numbers in their order as unsigned ones: NaN above infinity, 0 below all.
__device__ __forceinline__ unsigned long long moe_key(double v) {
    if (v != v) return ~0ull;
    if (v == 0.0) v = 0.0;  // -0 is 0
    const unsigned long long b = (unsigned long long)__double_as_longlong(v);
    return b >> 63 ? ~b : b | 1ull << 63;
}
// A token's k experts by a warp; PER: experts a lane holds.
template <int PER>
__device__ __forceinline__ void moe_choose(const MoeArgs &p, int t, unsigned short *chosen, bool tell) {
    const int lane = threadIdx.x & 31;
    unsigned long long key[PER];
    double v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        v[i] = e < p.experts ? __ldcg(p.logits + (long long)t * p.experts + e) : 0.0;
        key[i] = e < p.experts ? moe_key(v[i]) : 0ull;
    }
    double top = 0.0;
    float mine = 0.0f;  // lane i: the i-th choice's exponential
    int mine_e = 0;
    for (int c = 0; c < p.k; ++c) {
        unsigned long long best = 0ull;
        int at = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) best = key[i], at = i;
        const unsigned hi = __reduce_max_sync(0xffffffffu, (unsigned)(best >> 32));
        const unsigned lo = __reduce_max_sync(0xffffffffu, (unsigned)(best >> 32) == hi ? (unsigned)best : 0u);
        const bool is = (unsigned)(best >> 32) == hi && (unsigned)best == lo;
        const int e = (int)__reduce_min_sync(0xffffffffu, is ? (unsigned)(lane + 32 * at) : 0xffffffffu);
        double val = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 32 * i == e) {
                key[i] = 0ull;
                val = v[i];
            }
        val = __shfl_sync(0xffffffffu, val, e & 31);
        if (c == 0) top = val;
        if (lane == c) {
            mine = expf((float)(val - top));
            mine_e = e;
        }
    }
    if (lane < p.k) chosen[t * p.k + lane] = (unsigned short)mine_e;
    if (!tell) return;
    float sum = 0.0f;
    if (p.renormalize) {
        for (int c = 0; c < p.k; ++c) sum += __shfl_sync(0xffffffffu, mine, c);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 32 * i < p.experts) sum += expf((float)(v[i] - top));
        sum = warp_sum(sum);
    }
    if (lane < p.k) {
        const int at = t * p.k + lane;
        const float w = mine / sum;
        p.wts[at] = w;
        if (p.weights) p.weights[at] = w;
        if (p.ids) p.ids[at] = mine_e;
    }
}

// Every token's choices, and from them each expert's pairs in order and the
// jobs (an expert with up to 32 of its pairs).  All threads.
__device__ __forceinline__ void moe_route(const MoeArgs &p, MoeShared &sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pairs = p.n * p.k;
    for (int t = warp; t < p.n; t += kMoeThreads / 32) {
        const bool tell = t % gridDim.x == blockIdx.x;
        if (p.experts <= 64) moe_choose<2>(p, t, sh.chosen, tell);
        else if (p.experts <= 128) moe_choose<4>(p, t, sh.chosen, tell);
        else moe_choose<16>(p, t, sh.chosen, tell);
    }
    for (int e = threadIdx.x; e <= p.experts; e += kMoeThreads) sh.offset[e] = 0;
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kMoeThreads) {
        int c = 0;
        for (int i = 0; i < pairs; ++i) c += sh.chosen[i] == e;
        sh.offset[e + 1] = c;
    }
    __syncthreads();
    if (warp == 0) {  // running sums of the pairs and of the jobs
        int o = 0, j = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane, c = e < p.experts ? sh.offset[e + 1] : 0, g = (c + kMoeGroup - 1) / kMoeGroup;
            int so = c, sj = g;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int a = __shfl_up_sync(0xffffffffu, so, d), b = __shfl_up_sync(0xffffffffu, sj, d);
                if (lane >= d) so += a, sj += b;
            }
            if (e < p.experts) {
                sh.offset[e + 1] = o + so;
                sh.jobs[e + 1] = j + sj;
                for (int i = 0; i < g; ++i) sh.job_expert[j + sj - g + i] = (unsigned short)e;
            }
            o += __shfl_sync(0xffffffffu, so, 31);
            j += __shfl_sync(0xffffffffu, sj, 31);
        }
        if (lane == 0) sh.jobs[0] = 0;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kMoeThreads) {
        int at = sh.offset[e];
        if (at == sh.offset[e + 1]) continue;
        for (int i = 0; i < pairs; ++i)
            if (sh.chosen[i] == e) sh.list[at++] = (unsigned short)i;
    }
    __syncthreads();
}

// ------------------------------------------------------------------ stages
// A phase's line of stages: jobs x tiles x steps of the sum, an expert's jobs
// side by side for each tile (its weights are then still in L2).
struct MoeLine {
    int tiles, steps, runs;   // runs: CTAs that have one, at least a stage each
    long long total, s0, s1;  // this CTA's run
    __device__ MoeLine(int jobs, int tiles_, int steps_) : tiles(tiles_), steps(steps_) {
        total = (long long)jobs * tiles * steps;
        runs = (int)min((long long)gridDim.x, total);
        s0 = total * min((int)blockIdx.x, runs) / runs;
        s1 = total * min((int)blockIdx.x + 1, runs) / runs;
    }
    __device__ int holder(long long s) const { return (int)(((s + 1) * runs - 1) / total); }
};
struct MoeTile {
    int expert, tile, start, count;  // its pairs: list[start ...]
};
__device__ __forceinline__ MoeTile moe_tile(const MoeShared &sh, const MoeLine &l, int unit) {
    MoeTile t;
    t.expert = sh.job_expert[unit / l.tiles];
    const int j0 = sh.jobs[t.expert], g = sh.jobs[t.expert + 1] - j0, in = unit - j0 * l.tiles;
    t.tile = in / g;
    t.start = sh.offset[t.expert] + in % g * kMoeGroup;
    t.count = min(kMoeGroup, sh.offset[t.expert + 1] - t.start);
    return t;
}

__device__ __forceinline__ void moe_box(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, "
        "%4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// The copying thread's share of a phase; returns false once a wait gave up.
__device__ __forceinline__ bool moe_fetch(const MoeArgs &p, MoeShared &sh, uint32_t ring, const MoeLine &l, bool down, int step,
                                          long long &fill, uint64_t policy) {
    int unit = (int)(l.s0 / l.steps), k = (int)(l.s0 - (long long)unit * l.steps);
    MoeTile t;
    if (l.s0 < l.s1) t = moe_tile(sh, l, unit);
    for (long long s = l.s0; s < l.s1; ++s) {
        const int slot = (int)(fill % kMoeStages);
        if (!moe_wait(&sh.empty[slot], (uint32_t)(fill / kMoeStages + 1) & 1, &sh.dead, p.err)) return false;
        mbar_arrive_expect_tx(&sh.full[slot], kMoeStageBytes);
        const uint32_t dst = ring + slot * kMoeStageBytes;
        if (down) {
            moe_box(dst, &p.td, k * step, t.tile * 128, t.expert, &sh.full[slot], policy);
        } else {
            moe_box(dst, &p.tgu, k * step, t.tile * 64, 2 * t.expert, &sh.full[slot], policy);
            moe_box(dst + kMoeStageBytes / 2, &p.tgu, k * step, t.tile * 64, 2 * t.expert + 1, &sh.full[slot], policy);
        }
        ++fill;
        if (++k == l.steps) {
            k = 0;
            ++unit;
            if (s + 1 < l.s1) t = moe_tile(sh, l, unit);
        }
    }
    return true;
}

__device__ __forceinline__ uint4 moe_lds(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void moe_mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void moe_mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four e4m3 values as two f16 pairs.
__device__ __forceinline__ void moe_widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t moe_top2(float a, float b) {  // leading 8 bits, cut off, a in the low half
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float moe_rest(float a) { return a - __uint_as_float(__float_as_uint(a) & 0xffff0000u); }
__device__ __forceinline__ uint32_t moe_bf16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t moe_f16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// A lane's values of one token for a stage: runs t and t + 4 of eight (bf16
// weights) or sixteen (e4m3); zeros behind the sum's end and for no token.
template <typename SRC, int RUN>
__device__ __forceinline__ void moe_values(const SRC *row, int k0, int len, float (&v)[2 * RUN]) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int k = k0 + (t + 4 * h) * RUN;
        const bool in = row != nullptr && k < len;
#pragma unroll
        for (int i = 0; i < RUN; i += 8) {
            float w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (in) {
                if (sizeof(SRC) == 2) {
                    widen16(__ldcg(reinterpret_cast<const uint4 *>(row + k + i)), w);
                } else {
                    const float4 a = __ldcg(reinterpret_cast<const float4 *>(row + k + i));
                    const float4 b = __ldcg(reinterpret_cast<const float4 *>(row + k + i) + 1);
                    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
                }
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) v[h * RUN + i + q] = w[q];
        }
    }
}

// The MMA's row g is row (g >> 1 | (g & 1) << 2) of eight, so that the eight
// lanes of a shared-memory access meet all banks of the swizzled stage.
__device__ __forceinline__ int moe_row(int g) { return g >> 1 | (g & 1) << 2; }

// acc += (128 rows of the stage) x (8 tokens), bf16 weights: P pieces of the tokens' values.
template <int P>
__device__ __forceinline__ void moe_stage_bf16(float (&acc)[8][4], uint32_t stage, const float (&v)[16]) {
    uint32_t b[P][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float x = v[2 * i], y = v[2 * i + 1];
        b[0][i] = moe_top2(x, y);
        if (P > 1) {
            x = moe_rest(x), y = moe_rest(y);
            b[P > 1 ? 1 : 0][i] = P == 2 ? moe_bf16x2(x, y) : moe_top2(x, y);
        }
        if (P > 2) b[P - 1][i] = moe_bf16x2(moe_rest(x), moe_rest(y));
    }
    const int lane = threadIdx.x & 31, t = lane & 3, r = moe_row(lane >> 2);
    // The tensor core cuts its sums off rather than rounding them, so a stage's
    // are kept short, small pieces first, and added outside.
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        uint4 lo[2], hi[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = stage + (m * 16 + r) * 128 + (((t + 4 * h) ^ r) << 4);
            lo[h] = moe_lds(at), hi[h] = moe_lds(at + 8 * 128);
        }
        float d[4] = {0, 0, 0, 0};
#pragma unroll
        for (int q = P - 1; q >= 0; --q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                moe_mma_bf16(d, lo[h].x, hi[h].x, lo[h].y, hi[h].y, b[q][4 * h], b[q][4 * h + 1]);
                moe_mma_bf16(d, lo[h].z, hi[h].z, lo[h].w, hi[h].w, b[q][4 * h + 2], b[q][4 * h + 3]);
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] += d[i];
    }
}

// The same with e4m3 weights; s0, s1: scales of rows 0 to 63 and 64 to 127.
template <int P>
__device__ __forceinline__ void moe_stage_e4m3(float (&acc)[8][4], uint32_t stage, const float (&v)[32], float s0, float s1) {
    const int lane = threadIdx.x & 31, t = lane & 3, r = moe_row(lane >> 2);
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the largest to [2^14, 2^15), but by no more than 2^114; what is not finite stays so
    const int e = top >= 0x7f800000u ? 14 : max((int)(top >> 23) - 127, -100);
    const float up = __uint_as_float((unsigned)(127 + 14 - e) << 23), back = __uint_as_float((unsigned)(127 - 14 + e) << 23);
    uint32_t b[P][16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float x = v[2 * i] * up, y = v[2 * i + 1] * up;
        b[0][i] = moe_f16x2(x, y);
        if (P > 1) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&b[0][i]));
            b[P - 1][i] = moe_f16x2(x - f.x, y - f.y);
        }
    }
    const float b0 = __shfl_sync(0xffffffffu, back, t * 8), b1 = __shfl_sync(0xffffffffu, back, t * 8 + 4);
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        float d[4] = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = stage + (m * 16 + r) * 128 + (((t + 4 * h) ^ r) << 4);
            const uint4 lo = moe_lds(at), hi = moe_lds(at + 8 * 128);
            const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a0, a1, a2, a3;
                moe_widen(wl[i], a0, a2);
                moe_widen(wh[i], a1, a3);
#pragma unroll
                for (int q = P - 1; q >= 0; --q) moe_mma_f16(d, a0, a1, a2, a3, b[q][8 * h + 2 * i], b[q][8 * h + 2 * i + 1]);
            }
        }
        const float s = m < 4 ? s0 : s1;
        acc[m][0] += d[0] * (s * b0);
        acc[m][1] += d[1] * (s * b1);
        acc[m][2] += d[2] * (s * b0);
        acc[m][3] += d[3] * (s * b1);
    }
}

// ------------------------------------------------------------------ phases
// Two sums (rows f and f + 64) of two tokens of a tile, finished: the
// intermediate's value, or two of the down product.
template <bool DOWN>
__device__ __forceinline__ void moe_finish(const MoeArgs &p, const MoeShared &sh, const MoeTile &t, int token, int f, float2 a, float2 b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (token + i >= t.count) return;
        const long long pair = sh.list[t.start + token + i];
        const float x = i ? a.y : a.x, z = i ? b.y : b.x;
        if (DOWN) {
            const int r = t.tile * 128 + f;
            if (r < p.d) __stcg(p.out + pair * p.d + r, x);
            if (r + 64 < p.d) __stcg(p.out + pair * p.d + r + 64, z);
        } else {
            const int r = t.tile * 64 + f;
            if (r < p.ff) __stcg(p.h + pair * p.ff + r, x / (1.0f + expf(-x)) * z);
        }
    }
}

// The eight warps' share of a phase.
template <bool W8, bool DOWN, typename SRC, int P>
__device__ __forceinline__ void moe_phase(const MoeArgs &p, MoeShared &sh, uint32_t ring, const MoeLine &l, long long &fill) {
    constexpr int RUN = W8 ? 16 : 8, STEP = 8 * RUN;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int len = DOWN ? p.ff : p.d, db = (p.d + 127) / 128, fb = (p.ff + 127) / 128;
    const SRC *src = DOWN ? reinterpret_cast<const SRC *>(p.h) : static_cast<const SRC *>(p.x);
    for (long long s = l.s0; s < l.s1;) {
        const int unit = (int)(s / l.steps), k0 = (int)(s - (long long)unit * l.steps);
        const int k1 = (int)min((long long)l.steps, k0 + l.s1 - s);
        const MoeTile tile = moe_tile(sh, l, unit);
        const int groups = (tile.count + 7) / 8;
        const SRC *row[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int i = n * 8 + g;
            row[n] = nullptr;
            if (i < tile.count) {
                const int pair = sh.list[tile.start + i];
                row[n] = src + (DOWN ? (long long)pair * p.ff : (long long)(pair / p.k) * p.d);
            }
        }
        const float *scale = nullptr, *scale1 = nullptr;
        if (W8) {
            if (DOWN) {
                scale = scale1 = p.d_scales + ((long long)tile.expert * db + tile.tile) * fb;
            } else {
                scale = p.gu_scales + ((long long)tile.expert * 2 * fb + tile.tile / 2) * db;
                scale1 = scale + (long long)fb * db;
            }
        }
        float acc[4][8][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][m][i] = 0.0f;
        // this warp's stages: every eighth
        for (int k = k0 + (int)((warp - fill) & (kMoeWarps - 1)); k < k1; k += kMoeWarps) {
            const long long f = fill + (k - k0);
            const int slot = (int)(f % kMoeStages);
            const uint32_t stage = ring + slot * kMoeStageBytes;
            float s0 = 1.0f, s1 = 1.0f;
            if (W8) s0 = __ldg(scale + k), s1 = __ldg(scale1 + k);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (n < groups) {
                    float v[2 * RUN];
                    moe_values<SRC, RUN>(row[n], k * STEP, len, v);
                    if (n == 0) moe_wait(&sh.full[slot], (uint32_t)(f / kMoeStages) & 1, &sh.dead, p.err);
                    if constexpr (W8) moe_stage_e4m3<P>(acc[n], stage, v, s0, s1);
                    else moe_stage_bf16<P>(acc[n], stage, v);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[slot]);
        }
        fill += k1 - k0;
        // the eight warps' sums, eight tokens at a time, added in order
        const bool whole = k0 == 0 && k1 == l.steps;
        const int f = threadIdx.x >> 2;
        float *mine = p.parts + ((long long)blockIdx.x * 2 + (k0 == 0)) * kMoeSums;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (n >= groups) break;
            float *to = sh.sums[warp];
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                const int r = m * 16 + moe_row(g);
                *reinterpret_cast<float2 *>(to + r * 8 + 2 * t) = make_float2(acc[n][m][0], acc[n][m][1]);
                *reinterpret_cast<float2 *>(to + (r + 8) * 8 + 2 * t) = make_float2(acc[n][m][2], acc[n][m][3]);
            }
            named_sync(1, kMoeWarps * 32);
            float2 a = make_float2(0, 0), b = make_float2(0, 0);
#pragma unroll
            for (int w = 0; w < kMoeWarps; ++w) {
                const float2 x = *reinterpret_cast<const float2 *>(sh.sums[w] + f * 8 + 2 * t);
                const float2 z = *reinterpret_cast<const float2 *>(sh.sums[w] + (f + 64) * 8 + 2 * t);
                a.x += x.x, a.y += x.y, b.x += z.x, b.y += z.y;
            }
            if (whole) {
                moe_finish<DOWN>(p, sh, tile, n * 8 + 2 * t, f, a, b);
            } else {
                __stcg(reinterpret_cast<float2 *>(mine + n * 1024 + f * 8 + 2 * t), a);
                __stcg(reinterpret_cast<float2 *>(mine + n * 1024 + (f + 64) * 8 + 2 * t), b);
            }
            named_sync(1, kMoeWarps * 32);
        }
        if (!whole) {
            const long long u0 = (long long)unit * l.steps;
            const int first = l.holder(u0), last = l.holder(u0 + l.steps - 1);
            int *counter = p.counters + (DOWN ? gridDim.x : 0) + first;
            __threadfence();
            named_sync(1, kMoeWarps * 32);
            if (threadIdx.x == 0) sh.last = atomicAdd(counter, 1) == last - first;
            named_sync(1, kMoeWarps * 32);
            if (sh.last) {
                __threadfence();
                for (int n = 0; n < groups; ++n) {
                    float2 a = make_float2(0, 0), b = make_float2(0, 0);
                    for (int c = first; c <= last; ++c) {
                        const float *from = p.parts + ((long long)c * 2 + (c == first)) * kMoeSums + n * 1024;
                        const float2 x = __ldcg(reinterpret_cast<const float2 *>(from + f * 8 + 2 * t));
                        const float2 z = __ldcg(reinterpret_cast<const float2 *>(from + (f + 64) * 8 + 2 * t));
                        a.x += x.x, a.y += x.y, b.x += z.x, b.y += z.y;
                    }
                    moe_finish<DOWN>(p, sh, tile, n * 8 + 2 * t, f, a, b);
                }
                if (threadIdx.x == 0) *counter = 0;
            }
            named_sync(1, kMoeWarps * 32);
        }
        s += k1 - k0;
    }
}

template <bool W8, typename X>
__global__ __launch_bounds__(kMoeThreads, 1) void moe_kernel(const __grid_constant__ MoeArgs p) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    MoeShared &sh = *reinterpret_cast<MoeShared *>(smem_raw + (ring - smem_u32(smem_raw)) + kMoeStages * kMoeStageBytes);
    const int warp = threadIdx.x >> 5;
    constexpr bool XB = sizeof(X) == 2;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMoeStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        sh.dead = 0;
        fence_mbarrier_init();
    }
    // logits: a warp takes an expert with one token, or with four where that still gives every warp some
    const int gw = blockIdx.x * (kMoeThreads / 32) + warp, gn = gridDim.x * (kMoeThreads / 32);
    if ((long long)p.n * p.experts <= 2 * gn) {
        for (int i = gw; i < p.n * p.experts; i += gn) moe_logits<1>(p, i % p.experts, i / p.experts);
    } else {
        for (int i = gw; i < (p.n + 3) / 4 * p.experts; i += gn) moe_logits<4>(p, i % p.experts, i / p.experts * 4);
    }
    __syncthreads();
    if (threadIdx.x == 0) moe_meet(p.bars, &sh.dead, p.err);
    __syncthreads();
    if (!sh.dead) {  // (the same for all: read between two barriers of the block)
        moe_route(p, sh);
        constexpr int step = W8 ? 128 : 64;
        const int jobs = sh.jobs[p.experts];
        const MoeLine gu(jobs, (p.ff + 63) / 64, (p.d + step - 1) / step), dn(jobs, (p.d + 127) / 128, (p.ff + step - 1) / step);
        long long fill = 0;
        if (warp >= kMoeWarps) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMoeRegsOther));
            if (threadIdx.x == kMoeWarps * 32) {
                const uint64_t policy = policy_evict_first();
                if (moe_fetch(p, sh, ring, gu, false, step, fill, policy)) moe_fetch(p, sh, ring, dn, true, step, fill, policy);
                // the copies still under way land before the CTA ends
                for (long long i = max(0ll, fill - kMoeStages); i < fill; ++i)
                    mbar_wait(&sh.full[i % kMoeStages], (uint32_t)(i / kMoeStages) & 1, p.err);
            }
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMoeRegsMain));
            moe_phase<W8, false, X, W8 ? (XB ? 1 : 2) : (XB ? 1 : 3)>(p, sh, ring, gu, fill);
            named_sync(1, kMoeWarps * 32);
            if (threadIdx.x == 0) moe_meet(p.bars + 1, &sh.dead, p.err);
            named_sync(1, kMoeWarps * 32);
            moe_phase<W8, true, float, W8 ? 2 : (XB ? 2 : 3)>(p, sh, ring, dn, fill);
            named_sync(1, kMoeWarps * 32);
            if (threadIdx.x == 0) moe_meet(p.bars + 2, &sh.dead, p.err);
            named_sync(1, kMoeWarps * 32);
            // the weighted sum, four values a thread
            const int quads = p.d / 4;
            for (long long i = (long long)blockIdx.x * kMoeWarps * 32 + threadIdx.x; i < (long long)p.n * quads; i += (long long)gridDim.x * kMoeWarps * 32) {
                const int tok = (int)(i / quads), j = (int)(i - (long long)tok * quads) * 4;
                const long long at = (long long)tok * p.d + j;
                float4 v = make_float4(0, 0, 0, 0);
                for (int c = 0; c < p.k; ++c) {
                    const long long pair = (long long)tok * p.k + c;
                    const float w = __ldcg(p.wts + pair);
                    const float4 o = __ldcg(reinterpret_cast<const float4 *>(p.out + pair * p.d + j));
                    v.x += w * o.x, v.y += w * o.y, v.z += w * o.z, v.w += w * o.w;
                }
                X *y = static_cast<X *>(p.y) + at;
                const float o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float r = p.residual ? load_as(p.residual, at + q, p.x_dtype) : 0.0f;
                    store_as(y, q, p.x_dtype, r + o[q]);
                }
            }
        }
    }
    __syncthreads();
    // the last CTA leaves the meeting counts as they were found
    if (threadIdx.x == 0) {
        if (atomicAdd(p.bars + 3, 1) == (int)gridDim.x - 1) {
            p.bars[0] = p.bars[1] = p.bars[2] = p.bars[3] = 0;
            __threadfence();
        }
    }
}

// ---------------------------------------------------------------- host
struct MoeSpace {
    size_t bars, counters, logits, wts, h, parts, out, total;
};
static MoeSpace moe_space(int64_t n, int64_t d, int64_t ff, int64_t experts, int64_t k) {
    MoeSpace s;
    const size_t g = (size_t)sm_count(), pairs = (size_t)(n * k);
    size_t at = kWsHeader;
    s.bars = at, at += 256;
    s.counters = at, at += align_up(2 * g * 4, 256);
    s.parts = at, at += g * 2 * kMoeSums * 4;
    s.logits = at, at += align_up((size_t)(n * experts) * 8, 256);
    s.wts = at, at += align_up(pairs * 4, 256);
    s.h = at, at += align_up(pairs * ff * 4, 256);
    s.out = at, at += align_up(pairs * d * 4, 256);
    s.total = at;
    return s;
}

template <bool W8, typename X>
static cudaError_t moe_launch(const MoeArgs &a, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};  // devices whose limit is raised, a bit each
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(moe_kernel<W8, X>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMoeSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sm_count());
    cfg.blockDim = dim3(kMoeThreads);
    cfg.dynamicSmemBytes = kMoeSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_kernel<W8, X>, a);
}

}  // namespace ds

using namespace ds;

static int moe_sizes(int64_t n, int64_t d, int64_t ff, int n_experts, int top_k) {
    if (n < 1 || d < 1 || ff < 1 || n_experts < 1 || top_k < 1) return DS_EMPTY_DIMENSION;
    if (n > kMoeMaxTokens || n_experts > kMoeMaxExperts || top_k > kMoeMaxK || d > DS_MAX_DIM || ff > DS_MAX_DIM) return DS_DIMENSION_TOO_LARGE;
    if (d * ff * 2 * n_experts > (int64_t)1 << 42) return DS_DIMENSION_TOO_LARGE;
    return DS_OK;
}

extern "C" DS_API size_t ds_moe_layer_workspace_bytes(int64_t n, int64_t d, int64_t ff, int n_experts, int top_k) {
    if (moe_sizes(n, d, ff, n_experts, top_k) != DS_OK) return 0;
    return moe_space(n, d, ff, n_experts, top_k).total;
}

extern "C" DS_API int ds_moe_layer(const void *x, int64_t x_len, int x_dtype, int64_t n, int64_t d, const void *w_router,
                                   int64_t router_len, int router_dtype, int n_experts, int top_k, int renormalize,
                                   const void *w_gate_up, int64_t gate_up_len, const float *gate_up_scales,
                                   int64_t gate_up_scales_len, const void *w_down, int64_t down_len, const float *down_scales,
                                   int64_t down_scales_len, int w_dtype, int64_t ff, const void *residual, void *y,
                                   int64_t y_len, int32_t *expert_ids, float *expert_weights, void *workspace,
                                   size_t workspace_bytes, ds_stream_t stream) {
    const int st = moe_sizes(n, d, ff, n_experts, top_k);
    if (st != DS_OK) return st;
    if ((x_dtype != DS_F32 && x_dtype != DS_BF16) || (router_dtype != DS_F32 && router_dtype != DS_BF16) ||
        (w_dtype != DS_BF16 && w_dtype != DS_E4M3))
        return DS_BAD_DTYPE;
    const bool w8 = w_dtype == DS_E4M3;
    const int64_t db = (d + 127) / 128, fb = (ff + 127) / 128, unit = w8 ? 16 : 8;
    if (x_len != n * d) return DS_GEMV_X_LENGTH_MISMATCH;
    if (router_len != n_experts * d || gate_up_len != n_experts * 2 * ff * d || down_len != n_experts * d * ff) return DS_GEMV_A_LENGTH_MISMATCH;
    if (w8 && (gate_up_scales_len != n_experts * 2 * fb * db || down_scales_len != n_experts * db * fb)) return DS_GEMV_A_LENGTH_MISMATCH;
    if (y_len != n * d) return DS_A_LENGTH_MISMATCH;
    if (top_k > n_experts || d % unit || ff % unit) return DS_BAD_ARGUMENT;
    if (!x || !w_router || !w_gate_up || !w_down || !y || (w8 && (!gate_up_scales || !down_scales))) return DS_BAD_ARGUMENT;
    if (((uintptr_t)x | (uintptr_t)w_router | (uintptr_t)w_gate_up | (uintptr_t)w_down) & 15) return DS_BAD_ARGUMENT;
    const int es = x_dtype == DS_BF16 ? 2 : 4;
    if (((uintptr_t)y | (uintptr_t)residual) % es || ((uintptr_t)expert_ids | (uintptr_t)expert_weights) & 3) return DS_BAD_ARGUMENT;
    if (w8 && (((uintptr_t)gate_up_scales | (uintptr_t)down_scales) & 3)) return DS_BAD_ARGUMENT;
    const MoeSpace sp = moe_space(n, d, ff, n_experts, top_k);
    if (!workspace || workspace_bytes < sp.total) return DS_WORKSPACE_TOO_SMALL;
    if ((uintptr_t)workspace & 255) return DS_BAD_ARGUMENT;
    // y may be x or the residual itself (each value is read before it is written); nothing else is shared
    const int64_t ws = w8 ? 1 : 2, rs = router_dtype == DS_BF16 ? 2 : 4, yb = n * d * es;
    const struct {
        const void *p;
        int64_t n;
    } span[] = {{y, yb}, {expert_ids, n * top_k * 4}, {expert_weights, n * top_k * 4}, {x, yb}, {residual, yb},
                {w_router, router_len * rs}, {w_gate_up, gate_up_len * ws}, {w_down, down_len * ws},
                {w8 ? gate_up_scales : nullptr, gate_up_scales_len * 4}, {w8 ? down_scales : nullptr, down_scales_len * 4}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 10; ++j) {
            if (!span[i].p || !span[j].p || (i == 0 && (j == 3 || j == 4) && span[j].p == y)) continue;
            if ((uintptr_t)span[i].p < (uintptr_t)span[j].p + span[j].n && (uintptr_t)span[j].p < (uintptr_t)span[i].p + span[i].n) return DS_BAD_ARGUMENT;
        }
    MoeArgs a = {};
    a.x = x;
    a.router = w_router;
    a.residual = residual;
    a.gu_scales = gate_up_scales;
    a.d_scales = down_scales;
    a.y = y;
    a.ids = expert_ids;
    a.weights = expert_weights;
    a.x_dtype = x_dtype;
    a.r_dtype = router_dtype;
    a.n = (int)n;
    a.d = (int)d;
    a.ff = (int)ff;
    a.experts = n_experts;
    a.k = top_k;
    a.renormalize = renormalize != 0;
    char *w = static_cast<char *>(workspace);
    a.err = reinterpret_cast<int *>(w);
    a.bars = reinterpret_cast<int *>(w + sp.bars);
    a.counters = reinterpret_cast<int *>(w + sp.counters);
    a.logits = reinterpret_cast<double *>(w + sp.logits);
    a.wts = reinterpret_cast<float *>(w + sp.wts);
    a.h = reinterpret_cast<float *>(w + sp.h);
    a.parts = reinterpret_cast<float *>(w + sp.parts);
    a.out = reinterpret_cast<float *>(w + sp.out);
    const int box = w8 ? 128 : 64;
    const long long gdims[3] = {d, ff, 2LL * n_experts}, gst[2] = {d * ws, ff * d * ws};
    const long long ddims[3] = {ff, d, n_experts}, dst[2] = {ff * ws, ff * d * ws};
    const int gbox[3] = {box, 64, 1}, dbox[3] = {box, 128, 1};
    if (!encode_tiled_3d(&a.tgu, w_gate_up, w_dtype, gdims, gst, gbox, true) ||
        !encode_tiled_3d(&a.td, w_down, w_dtype, ddims, dst, dbox, true))
        return DS_CUDA_ERROR;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool xb = x_dtype == DS_BF16;
    const cudaError_t e = w8 ? (xb ? moe_launch<true, __nv_bfloat16>(a, s) : moe_launch<true, float>(a, s))
                             : (xb ? moe_launch<false, __nv_bfloat16>(a, s) : moe_launch<false, float>(a, s));
    return e == cudaSuccess ? DS_OK : DS_CUDA_ERROR;
}
