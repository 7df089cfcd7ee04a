// A mixture-of-experts layer for few tokens in one launch (ds_moe_layer):
//   logits = x R^T;  the k largest of a token (lower index first among equals);
//   y = (residual +) sum_i w_i D[e_i] (silu(G[e_i] x) * (U[e_i] x))
// with w the softmax of the logits at the chosen experts, divided by their sum
// or not.
//
// What bounds it is the chosen experts' weight bytes, each of which is wanted
// by few tokens.  A step takes 256 rows by 128 bytes of the sum (an expert's 128
// gate and 128 up rows, or 256 down rows) through shared memory into two
// tcgen05.mma whose N are the tokens; all tiles of a phase, expert after expert,
// are one line of steps cut into equal runs, one a CTA, so that every SM streams
// the same bytes.  A tile that is cut is added up by the CTA that is last.
//
// Phases with a meeting of the whole grid between them (a cooperative launch;
// every wait is bounded): logits; for more than eight tokens the choices, a
// token a CTA, and the tokens' rows in the order of the experts; gate and up;
// down; the weighted sum.  Up to eight tokens every CTA chooses for itself, and
// every expert's columns are all the tokens.  The copying warp has the next
// phase's weights under way while the others meet.
//
// Digits: an activation goes to the tensor core in pieces of the weights' own
// type, side by side as further columns, that add up to it: one bf16 piece for
// bf16 activations, three (24 bits, exact) for fp32; e4m3 pieces of four bits
// each, a sixteenth apart, behind a power of two per token and 128 values that
// brings the largest to [2^7, 2^8): six for fp32 (24 bits, to 2^-37 of the largest:
// the last piece is off by half of e4m3's least step, 2^-10, and counts 2^-20), three
// for bf16 (two hold its 8 bits; the third those of values below 2^-14 of the
// largest, to 2^-25 of it).  The intermediate is fp32 and goes in three bf16
// pieces (24 bits) or six e4m3 ones, before bf16 outputs in four of e4m3 (16 bits
// and more: see MoeCfg).  Sums leave the tensor core every 128 products (e4m3: a
// block, for its scale; bf16: see kMoeBatch) and are fp32.  The logits are sums of
// products with the rounding errors of both carried along (two floats, some 45 bits
// of the products' magnitudes, fewer of products below 2^-102, whose errors leave
// fp32's range; compared in 64 bits): the choice of experts is that of 64 bits
// unless two are as close as that.
//
// Measured in a graph: 64 tokens through 2 of 8 experts of 4,096 x 14,336 (fp32,
// bf16 weights) 476 us, 5.9 TB/s of 6.8; 64 through 8 of 128 of 2,048 x 768 (bf16,
// e4m3) 138 us, 4.3 TB/s; one token through those in bf16 37 us, 2.1 TB/s: some 20
// us are the phases' latencies (a layer of no size takes 21), 6 of them the ends of
// the two products (partial sums out, counted, read, and code that runs once: some
// 25 cycles an instruction until it is fetched).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "mma_stream.cuh"
#include "tc.h"

namespace ds {

constexpr int kMoeMaxTokens = 256, kMoeMaxExperts = 512, kMoeMaxK = 16;
constexpr int kMoeMaxPairs = kMoeMaxTokens * kMoeMaxK;
constexpr int kMoeGroup = 32;  // tokens a step is multiplied with at most
constexpr int kMoeByToken = 8; // up to so many tokens every expert's columns are all the tokens
constexpr int kMoeMaxJobs = kMoeMaxExperts + kMoeMaxPairs / 16;
constexpr int kMoeThreads = 384;  // two warpgroups that add up; copies, products, scales, one idle
// Registers a thread: 168 at launch (384 x 168), moved to the warps that add
// up: 2 x 216 + 72 = 3 x 168.
constexpr int kMoeRegsSum = 216, kMoeRegsOther = 72;
constexpr int kMoeMaxStages = 5;
constexpr int kMoeWeightBytes = 2 * 128 * 128;  // of a step
constexpr int kMoeRing = 200 * 1024;  // four stages with 128 columns, five with 64 or 32
constexpr int kMoeSlots = 8;  // steps' scales ahead
// Steps between two sums of bf16 products in registers.  The tensor cores cut an
// fp32 sum's low bits off at every addition, always towards zero, so a long run of
// them drifts: 64 fp32 tokens, 8 experts of 14336, are 3.2e-6 off the exact result
// with 16 steps, 8e-7 with 4 and 5e-7 with 2, at 475, 477 and 477 us.
constexpr int kMoeBatch = 2;
constexpr int kMoeAtOnce = 2; // partial sums of a cut tile under way at a time
constexpr int kMoeSums = 2 * kMoeGroup * 128;  // floats of a tile

// How many pieces an activation and the intermediate are cut into, and how many
// tokens fit beside one another in 128 columns.  e4m3 before bf16 outputs: four
// pieces, so that 32 tokens fit.  Six, and 16 tokens, read an expert's weights twice
// as often: 64 tokens through 2 of 8 experts of 4,096 x 14,336 337 us against 260,
// 256 of them 1,080 against 642; of 131,072 outputs 31 against 50 were not the exact
// result rounded (plain fp32: 184).  (Of bf16 two in the place of three gained
// nothing: 463 us against 462, one token 35.1 against 34.5.)
template <bool W8, bool XB>
struct MoeCfg {
    static constexpr int kX = W8 ? (XB ? 3 : 6) : (XB ? 1 : 3);
    static constexpr int kH = W8 ? (XB ? 4 : 6) : 3;
    static constexpr int kGroup = W8 && !XB ? 16 : 32;
    static constexpr int kElem = W8 ? 1 : 2, kStep = 128 / kElem;  // values of a step
    // Both phases share the ring and TMEM: columns of a half of the sums, buffers
    // of two halves, stages.
    static constexpr int kCols = kH * kGroup <= 32 ? 32 : kH * kGroup <= 64 ? 64 : 128;
    static constexpr int kBufs = 256 / kCols < 4 ? 256 / kCols : 4;
    static constexpr int kStageBytes = kMoeWeightBytes + kCols * 128;
    static constexpr int kStages = kMoeRing / kStageBytes < kMoeMaxStages ? kMoeRing / kStageBytes : kMoeMaxStages;
    static_assert(kX <= kH && kH * kGroup <= 128, "columns");
};

struct MoeArgs {
    CUtensorMap tgu, td;  // {d, ff, 2 experts}, {ff, d, experts}: boxes of 128 B x 128 rows; swizzled
    CUtensorMap tx, th;   // the pieces: {d, rows, pieces}, {ff, pairs, pieces}: boxes of 128 B x 8 rows x all pieces
    const void *x, *router, *residual;
    const float *gu_scales, *d_scales;
    void *y;
    int *ids;
    float *weights;
    int x_dtype, r_dtype;
    int n, d, ff, experts, k, renormalize, splits;
    // workspace
    int *err, *bars, *counters;  // counters [2][grid]: arrivals at the tile that a CTA's run ends in
    float2 *logits;              // [splits][n][experts]: a sum and what its roundings lost
    unsigned short *choices;     // [n k]
    float *wts;                  // [n k]
    float *parts;                // [grid][4][2 x 32 x 128]: a run's first and last tile, whole tiles of either warpgroup
    float *out;                  // [n k][d]
    unsigned char *xp, *hp;      // pieces of x (by token, or by pair in the experts' order) and of the intermediate
    float *xs, *hs;              // e4m3: a scale for each 128 of their rows
};

struct MoeShared {
    uint64_t full[kMoeMaxStages], empty[kMoeMaxStages];
    uint64_t s_full[kMoeSlots], s_empty[kMoeSlots];
    uint64_t t_full[2][4], t_empty[4];  // (a warpgroup sees every phase of its own t_full, and no other)
    uint64_t go, done;
    uint32_t tmem;
    int dead, last[2];
    alignas(16) float scale[kMoeSlots][2][kMoeGroup];
    unsigned top[2][4][8];
    int offset[kMoeMaxExperts + 1], jobs[kMoeMaxExperts + 1];
    unsigned short job_expert[kMoeMaxJobs];
    unsigned short list[kMoeMaxPairs];  // pairs (token * k + slot) by expert
};
constexpr size_t kMoeSmem = 1024 + (size_t)kMoeRing + sizeof(MoeShared);
static_assert(kMoeSmem <= 227 * 1024, "shared memory");

// ------------------------------------------------------------------ waits
// One thread of every CTA: all of them have arrived, and what they wrote is seen.
__device__ __forceinline__ void moe_meet(int *bar, volatile int *dead, int *err) {
    asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(bar) : "memory");
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        int v;
        asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(bar) : "memory");
        if (v >= (int)gridDim.x || *dead) break;
        if ((it & 63u) == 0 && clock64() - t0 > kStreamWaitCycles) {
            flag_error(err, DS_ERR_WAIT_TIMEOUT);
            *dead = 1;
            break;
        }
    }
}

// The same for all threads of the CTA; whether a wait gave up.
__device__ __forceinline__ bool moe_meet_all(const MoeArgs &p, MoeShared &sh, int bar) {
    if (threadIdx.x == 0) moe_meet(p.bars + bar, &sh.dead, p.err);
    __syncthreads();
    const bool dead = sh.dead;
    __syncthreads();
    return dead;
}

// ------------------------------------------------------------------ router
// (Plain loads: x may be y, which the kernel writes in the end.)
__device__ __forceinline__ void moe_load8(const void *base, long long i, int dtype, float (&v)[8]) {
    if (dtype == DS_BF16) {
        widen16(*reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + i), v);
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + i);
        const float4 a = p[0], b = p[1];
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
// (s, c) += (s2, c2).  The same whichever is added to which: a two-sum's results
// do not depend on its operands' order.
__device__ __forceinline__ void moe_add2(float &s, float &c, float s2, float c2) {
    const float t = __fadd_rn(s, s2), z = __fsub_rn(t, s);
    c = __fadd_rn(__fadd_rn(c, c2), __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(s2, z)));
    s = t;
}
// How many parts the logits' sums are cut into (each a whole number of 256
// values): a part with an expert and four tokens is a warp's work, and several
// of them a warp even out.  Few tokens: one part, a CTA's work.
__host__ __device__ inline int moe_splits(long long n, long long d, long long experts, int warps) {
    if (n <= kMoeByToken) return 1;
    const long long items = (n + 3) / 4 * experts, whole = (d + 255) / 256;
    long long s = 8LL * warps / items;
    s = s < 1 ? 1 : s > whole ? whole : s > 16 ? 16 : s;
    const long long per = (whole + s - 1) / s;
    return (int)((whole + per - 1) / per);
}
// Part `split` of the sum of one expert's logits of tokens t0 ... t0 + T - 1, by a
// warp, a token's `stride` behind the one before's.
template <int T>
__device__ __forceinline__ void moe_logits(const MoeArgs &p, int e, int t0, int split, int splits, float2 *to, int stride) {
    const int lane = threadIdx.x & 31, per = ((p.d + 255) / 256 + splits - 1) / splits * 256;
    const int end = min(p.d, (split + 1) * per);
    float s[T], c[T];
#pragma unroll
    for (int i = 0; i < T; ++i) s[i] = c[i] = 0.0f;
    for (int j = split * per + lane * 8; j < end; j += 256) {
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
    for (int o = 16; o > 0; o >>= 1)  // (in two floats: doubles add at a sixty-fourth of the rate)
#pragma unroll
        for (int i = 0; i < T; ++i)
            moe_add2(s[i], c[i], __shfl_xor_sync(0xffffffffu, s[i], o), __shfl_xor_sync(0xffffffffu, c[i], o));
    if (lane < T && t0 + lane < p.n) {
        float sum = s[0], lost = c[0];
#pragma unroll
        for (int i = 1; i < T; ++i)
            if (lane == i) sum = s[i], lost = c[i];
        to[(long long)lane * stride] = make_float2(sum, lost);
    }
}

// Numbers in their order as unsigned ones: NaN above infinity, 0 below all.
__device__ __forceinline__ unsigned long long moe_key(double v) {
    if (v != v) return ~0ull;
    if (v == 0.0) v = 0.0;  // -0 is 0
    const unsigned long long b = (unsigned long long)__double_as_longlong(v);
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double moe_value(unsigned long long key) {
    return __longlong_as_double((long long)(key >> 63 ? key & ~(1ull << 63) : ~key));
}
// The logits of tokens t0 ... t0 + n - 1, the parts of their sums added, as keys;
// `id` of `step` threads.
__device__ __forceinline__ void moe_keys(const MoeArgs &p, int t0, int n, unsigned long long *key, int id, int step) {
    for (int i = id; i < n * p.experts; i += step) {
        const float2 *from = p.logits + (long long)t0 * p.experts + i;
        float sum = 0.0f, lost = 0.0f;
#pragma unroll 8
        for (int s = 0; s < p.splits; ++s) {
            const float2 v = __ldcg(from + (long long)s * p.n * p.experts);
            moe_add2(sum, lost, v.x, v.y);
        }
        // an infinite sum's lost part is NaN: the sum says it all
        key[i] = moe_key(fabsf(sum) < INFINITY ? (double)sum + (double)lost : (double)sum);
    }
}
// n tokens' choices: an expert's place is the number of experts ahead of it, so
// all are found at once.  All threads, several an expert where there are few.
__device__ __forceinline__ void moe_choose(const MoeArgs &p, int n, const unsigned long long *key, int *ahead, unsigned short *chosen) {
    const int m = n * p.experts, parts = max(1, min(4, kMoeThreads / m)), per = (p.experts + parts - 1) / parts;
    for (int i = threadIdx.x; i < m; i += kMoeThreads) ahead[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < m * parts; i += kMoeThreads) {
        const int part = i / m, at = i - part * m, t = at / p.experts, e = at - t * p.experts;
        const unsigned long long *of = key + t * p.experts, mine = of[e];
        int count = 0;
#pragma unroll 4
        for (int j = part * per; j < min(p.experts, (part + 1) * per); ++j) count += of[j] > mine || (of[j] == mine && j < e);
        atomicAdd(ahead + at, count);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < m; i += kMoeThreads)
        if (ahead[i] < p.k) chosen[i / p.experts * p.k + ahead[i]] = (unsigned short)(i % p.experts);
    __syncthreads();
}
// A token's weights, and what is told of its choices, by a warp.
__device__ __forceinline__ void moe_weights(const MoeArgs &p, int t, const unsigned long long *key, const unsigned short *chosen) {
    const int lane = threadIdx.x & 31, e = lane < p.k ? chosen[lane] : 0;
    const double top = moe_value(key[chosen[0]]);
    const float mine = lane < p.k ? expf((float)(moe_value(key[e]) - top)) : 0.0f;
    float sum = 0.0f;
    if (p.renormalize) {
        for (int c = 0; c < p.k; ++c) sum += __shfl_sync(0xffffffffu, mine, c);
    } else {
        for (int i = lane; i < p.experts; i += 32) sum += expf((float)(moe_value(key[i]) - top));
        sum = warp_sum(sum);
    }
    if (lane < p.k) {
        const int at = t * p.k + lane;
        const float w = mine / sum;
        p.wts[at] = w;
        if (p.weights) p.weights[at] = w;
        if (p.ids) p.ids[at] = e;
    }
}

// From every token's choices each expert's pairs in order and the jobs (an
// expert with up to G of its pairs).  A warp counts a stretch of the pairs;
// lanes with the same expert find one another.  All threads.
struct MoeRoute {
    unsigned short chosen[kMoeMaxPairs], place[kMoeMaxPairs], count[kMoeThreads / 32][kMoeMaxExperts];
    unsigned long long key[kMoeByToken][kMoeMaxExperts];  // logits
    int ahead[kMoeByToken * kMoeMaxExperts];
};
static_assert(sizeof(MoeRoute) <= kMoeRing, "the choices lie in the ring until it is used");
template <int G>
__device__ __forceinline__ void moe_route(const MoeArgs &p, MoeShared &sh, MoeRoute &r) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pairs = p.n * p.k;
    if (pairs <= 32) {  // a lane a pair; only the entries of chosen experts are written, and read
        if (warp == 0) {
            const int e = lane < pairs ? r.chosen[lane] : 0x7fffffff;
            int at = 0, behind = 0;
            bool head = true;
            for (int j = 0; j < pairs; ++j) {
                const int o = __shfl_sync(0xffffffffu, e, j);
                at += o < e || (o == e && j < lane);
                behind += o == e;
                head &= o != e || j >= lane;
            }
            // heads in the order of their places: jobs (a pair's expert has one: at most 32 tokens, G at a time)
            int job = 0;
            for (int j = 0; j < pairs; ++j) {
                const int o = __shfl_sync(0xffffffffu, e, j), n = __shfl_sync(0xffffffffu, behind, j);
                const bool h = __shfl_sync(0xffffffffu, (int)head, j);
                if (h && o < e) job += (n + G - 1) / G;
            }
            if (lane < pairs) sh.list[at] = (unsigned short)lane;
            const int jobs = (behind + G - 1) / G;
            __syncwarp();
            if (lane < pairs && head) {
                sh.offset[e] = at;
                sh.offset[e + 1] = at + behind;
                sh.jobs[e] = job;
                sh.jobs[e + 1] = job + jobs;
                for (int i = 0; i < jobs; ++i) sh.job_expert[job + i] = (unsigned short)e;
            }
            const int total = __reduce_max_sync(0xffffffffu, lane < pairs ? job + jobs : 0);
            if (lane == 0) sh.jobs[p.experts] = total;
        }
        __syncthreads();
        return;
    }
    const int per = (pairs + kMoeThreads - 1) / kMoeThreads * 32;  // pairs of a warp
    for (int e = lane; e < p.experts; e += 32) r.count[warp][e] = 0;
    __syncwarp();
    for (int i = warp * per + lane; i - lane < min(pairs, (warp + 1) * per); i += 32) {
        const unsigned e = i < pairs ? r.chosen[i] : 0xffffu;
        const unsigned same = __match_any_sync(0xffffffffu, e), before = __popc(same & ((1u << lane) - 1));
        const int base = i < pairs ? r.count[warp][e] : 0;
        __syncwarp();
        if (i < pairs) {
            r.place[i] = (unsigned short)(base + before);
            if (before == 0) r.count[warp][e] = (unsigned short)(base + __popc(same));
        }
        __syncwarp();
    }
    if (threadIdx.x == 0) sh.offset[0] = sh.jobs[0] = 0;
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kMoeThreads) {
        int sum = 0;
        for (int w = 0; w < kMoeThreads / 32; ++w) {
            const int c = r.count[w][e];
            r.count[w][e] = (unsigned short)sum;
            sum += c;
        }
        sh.offset[e + 1] = sum;
    }
    __syncthreads();
    if (warp == 0) {  // running sums of the pairs and of the jobs
        int o = 0, j = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane, c = e < p.experts ? sh.offset[e + 1] : 0, g = (c + G - 1) / G;
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
    }
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += kMoeThreads) {
        const int e = r.chosen[i];
        sh.list[sh.offset[e] + r.count[i / per][e] + r.place[i]] = (unsigned short)i;
    }
    __syncthreads();
}

// ------------------------------------------------------------------ pieces
__device__ __forceinline__ uint32_t moe_e4m3x2(float a, float b) {  // a in the low byte
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ float2 moe_from_e4m3x2(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)v));
    float2 f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}
// The power of two that brings a block's largest (its bits) to [2^7, 2^8), by no
// more than 2^107, and its inverse; NaN for a block that is not finite.
__device__ __forceinline__ void moe_scale(unsigned top, float &up, float &back) {
    if (top >= 0x7f800000u) {
        up = back = __int_as_float(0x7fffffff);
        return;
    }
    const int e = max((int)(top >> 23) - 127, -100);
    up = __uint_as_float((unsigned)(127 + 7 - e) << 23);
    back = __uint_as_float((unsigned)(127 - 7 + e) << 23);
}
// Two neighbouring values' pieces, `step` bytes from piece to piece.
template <bool W8, int P>
__device__ __forceinline__ void moe_put2(unsigned char *to, size_t step, float a, float b, float up) {
    if (W8) {
        a *= up, b *= up;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const uint32_t v = moe_e4m3x2(a, b);
            *reinterpret_cast<unsigned short *>(to + q * step) = (unsigned short)v;
            const float2 f = moe_from_e4m3x2(v);
            a = (a - f.x) * 16.0f, b = (b - f.y) * 16.0f;
        }
    } else {
#pragma unroll
        for (int q = 0; q < P; ++q) {
            // cut off but for the last, which is rounded
            const float x = __uint_as_float(__float_as_uint(a) & 0xffff0000u), z = __uint_as_float(__float_as_uint(b) & 0xffff0000u);
            *reinterpret_cast<uint32_t *>(to + q * step) = q < P - 1 ? __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632) : stream_bf16x2(a, b);
            a -= x, b -= z;
        }
    }
}
// The same for one value.
template <bool W8, int P>
__device__ __forceinline__ void moe_put(unsigned char *to, size_t step, float a, float up) {
    if (W8) {
        a *= up;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const uint32_t v = moe_e4m3x2(a, 0.0f);
            to[q * step] = (unsigned char)v;
            a = (a - moe_from_e4m3x2(v).x) * 16.0f;
        }
    } else {
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const float x = __uint_as_float(__float_as_uint(a) & 0xffff0000u);
            *reinterpret_cast<unsigned short *>(to + q * step) =
                q < P - 1 ? (unsigned short)(__float_as_uint(a) >> 16) : __bfloat16_as_ushort(__float2bfloat16_rn(a));
            a -= x;
        }
    }
}
// Rows of x in pieces, a warp for each 128 values: row r is token r, or that of
// the pair at place r of the experts' order.
template <bool W8, int P>
__device__ __forceinline__ void moe_split_x(const MoeArgs &p, const unsigned short *list, int rows) {
    const int lane = threadIdx.x & 31, blocks = (p.d + 127) / 128, warps = kMoeThreads / 32;
    constexpr int E = W8 ? 1 : 2;
    for (int i = blockIdx.x * warps + (threadIdx.x >> 5); i < rows * blocks; i += gridDim.x * warps) {
        const int r = i / blocks, j = (i - r * blocks) * 128 + lane * 4, tok = list ? list[r] / p.k : r;
        float v[4] = {0, 0, 0, 0};
        if (j < p.d) {  // (d is a multiple of 8)
            if (p.x_dtype == DS_BF16) {
                const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.x) + (size_t)tok * p.d + j);
                v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
                v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
            } else {
                const float4 w = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + (size_t)tok * p.d + j);
                v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
            }
        }
        float up = 1.0f, back;
        if (W8) {
            unsigned top = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) top = max(top, __float_as_uint(v[q]) & 0x7fffffffu);
            moe_scale(__reduce_max_sync(0xffffffffu, top), up, back);
            if (lane == 0) p.xs[(size_t)r * blocks + (j >> 7)] = back;
        }
        if (j < p.d) {
            unsigned char *to = p.xp + ((size_t)r * p.d + j) * E;
            const size_t step = (size_t)rows * p.d * E;
            moe_put2<W8, P>(to, step, v[0], v[1], up);
            moe_put2<W8, P>(to + 2 * E, step, v[2], v[3], up);
        }
    }
}
// What this thread wrote is seen by copies of whoever it meets next.
__device__ __forceinline__ void moe_fence_copies() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// ------------------------------------------------------------------ steps
// A phase's line of steps: jobs x tiles x steps of the sum, an expert's jobs
// side by side for each tile (its weights are then still in L2).
struct MoeLine {
    int tiles, steps, runs;   // runs: CTAs that have one, at least a step each
    long long total, s0, s1;  // this CTA's run
    __device__ MoeLine(int jobs, int tiles_, int steps_) : tiles(tiles_), steps(steps_) {
        total = (long long)jobs * tiles * steps;
        runs = (int)min((long long)gridDim.x, total);
        s0 = quotient(total * min((int)blockIdx.x, runs), runs);
        s1 = quotient(total * min((int)blockIdx.x + 1, runs), runs);
    }
    __device__ int holder(long long s) const { return (int)quotient((s + 1) * runs - 1, total); }
    // (64-bit divisions take some 500 cycles each)
    __device__ static long long quotient(long long a, long long b) { return a >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b); }
};
struct MoeTile {
    int expert, tile, start, count;  // its pairs: list[start ...]
};
template <int G>
__device__ __forceinline__ MoeTile moe_tile(const MoeShared &sh, const MoeLine &l, int unit) {
    MoeTile t;
    t.expert = sh.job_expert[unit / l.tiles];
    const int j0 = sh.jobs[t.expert], g = sh.jobs[t.expert + 1] - j0, in = unit - j0 * l.tiles;
    t.tile = in / g;
    t.start = sh.offset[t.expert] + in % g * G;
    t.count = min(G, sh.offset[t.expert + 1] - t.start);
    return t;
}
// A run's segments: the part of a tile's steps that lies in it.
struct MoeSeg {
    int unit, k0, k1;
};
__device__ __forceinline__ bool moe_next(const MoeLine &l, long long &s, MoeSeg &g) {
    if (s >= l.s1) return false;
    g.unit = (int)(s / l.steps);
    g.k0 = (int)(s - (long long)g.unit * l.steps);
    g.k1 = (int)min((long long)l.steps, g.k0 + l.s1 - s);
    s += g.k1 - g.k0;
    return true;
}
// Eight-token groups of a tile and the MMA's columns (a multiple of 16): a
// group's pieces one after the other, eight tokens each.
template <int P>
struct MoeCols {
    int groups, n;
    __device__ explicit MoeCols(int count) : groups((count + 7) / 8), n((8 * P * groups + 15) & ~15) {}
};
__device__ __forceinline__ void moe_box(uint32_t one, uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(one)
        : "memory");
}
__device__ __forceinline__ void moe_box_once(uint32_t one, uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], "
        "%7;\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(one), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void moe_expect(uint32_t one, uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes), "r"(one)
        : "memory");
}
__device__ __forceinline__ void moe_mma_bf16(uint32_t one, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "setp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}

// State of the ring and of the buffers that goes on from phase to phase.
struct MoeRing {
    int s = 0, b = 0, slot = 0;
    uint32_t ph = 0, bph = 0, sph = 0;
    __device__ void stage(int stages) {
        if (++s == stages) s = 0, ph ^= 1;
    }
    __device__ void buffer(int bufs) {
        if (++b == bufs) b = 0, bph ^= 1;
    }
    __device__ void scales() {
        if (++slot == kMoeSlots) slot = 0, sph ^= 1;
    }
};
__device__ __forceinline__ uint64_t moe_policy_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
// Copies of a step's weights, and of its tokens' pieces: two arrivals a stage.
template <int STAGE, bool DOWN>
__device__ __forceinline__ void moe_copy_weights(const MoeArgs &p, MoeShared &sh, uint32_t one, uint32_t ring, int s, const MoeTile &t, int x, uint64_t policy) {
    const uint32_t dst = ring + s * STAGE, bar = smem_u32(&sh.full[s]);
    moe_expect(one, bar, kMoeWeightBytes);
    if (DOWN) {
        moe_box_once(one, dst, &p.td, x, t.tile * 256, t.expert, bar, policy);
        moe_box_once(one, dst + kMoeWeightBytes / 2, &p.td, x, t.tile * 256 + 128, t.expert, bar, policy);
    } else {
        moe_box_once(one, dst, &p.tgu, x, t.tile * 128, 2 * t.expert, bar, policy);
        moe_box_once(one, dst + kMoeWeightBytes / 2, &p.tgu, x, t.tile * 128, 2 * t.expert + 1, bar, policy);
    }
}
template <int STAGE, int P>
__device__ __forceinline__ void moe_copy_tokens(const MoeArgs &p, MoeShared &sh, uint32_t one, uint32_t ring, int s, const CUtensorMap *map, int row, int count, int x) {
    const uint32_t dst = ring + s * STAGE + kMoeWeightBytes, bar = smem_u32(&sh.full[s]);
    const int groups = (count + 7) / 8;
    moe_expect(one, bar, groups * P * 1024);
    for (int j = 0; j < groups; ++j) moe_box(one, dst + j * P * 1024, map, x, row + 8 * j, 0, bar);
}

// The copying warp's share of a phase.  The tokens of the down products are there
// when the CTAs have met (`go`); until then the ring fills with weights.
template <typename C, bool DOWN, int P>
__device__ __forceinline__ void moe_copies(const MoeArgs &p, MoeShared &sh, uint32_t ring, const MoeLine &l, MoeRing &r) {
    constexpr int G = C::kGroup, step = C::kStep;
    const uint32_t one = stream_elect();
    const uint64_t once = policy_evict_first(), again = moe_policy_normal();  // an expert's weights are read for each of its jobs
    const bool by_token = !DOWN && p.n <= kMoeByToken;
    MoeSeg g;
    long long at = l.s0;
    int ahead = 0;
    if (DOWN) {
        MoeRing w = r;
        while (ahead < C::kStages && moe_next(l, at, g)) {
            const MoeTile t = moe_tile<G>(sh, l, g.unit);
            for (int k = g.k0; k < g.k1 && ahead < C::kStages; ++k, ++ahead) {
                stream_wait(&sh.empty[w.s], w.ph ^ 1, &sh.dead, p.err);
                if (*(volatile int *)&sh.dead) return;
                moe_copy_weights<C::kStageBytes, DOWN>(p, sh, one, ring, w.s, t, k * step, sh.jobs[t.expert + 1] - sh.jobs[t.expert] > 1 ? again : once);
                w.stage(C::kStages);
            }
        }
        stream_wait(&sh.go, 0, &sh.dead, p.err);
        moe_fence_copies();
        at = l.s0;
    }
    while (moe_next(l, at, g)) {
        const MoeTile t = moe_tile<G>(sh, l, g.unit);
        for (int k = g.k0; k < g.k1; ++k) {
            if (ahead > 0) {
                --ahead;
            } else {
                stream_wait(&sh.empty[r.s], r.ph ^ 1, &sh.dead, p.err);
                if (*(volatile int *)&sh.dead) return;
                moe_copy_weights<C::kStageBytes, DOWN>(p, sh, one, ring, r.s, t, k * step, sh.jobs[t.expert + 1] - sh.jobs[t.expert] > 1 ? again : once);
            }
            moe_copy_tokens<C::kStageBytes, P>(p, sh, one, ring, r.s, DOWN ? &p.th : &p.tx, by_token ? 0 : t.start, by_token ? p.n : t.count, k * step);
            r.stage(C::kStages);
        }
    }
}

// The products.
template <typename C, bool DOWN, int P>
__device__ __forceinline__ void moe_products(const MoeArgs &p, MoeShared &sh, uint32_t ring, const MoeLine &l, MoeRing &r, uint32_t tmem, int &turn) {
    constexpr int G = C::kGroup;
    constexpr bool W8 = C::kElem == 1;
    const uint32_t one = stream_elect();
    const bool by_token = !DOWN && p.n <= kMoeByToken;
    MoeSeg g;
    long long at = l.s0;
    for (; moe_next(l, at, g); turn ^= 1) {
        const MoeTile t = moe_tile<G>(sh, l, g.unit);
        const MoeCols<P> c(by_token ? p.n : t.count);
        const uint32_t idesc = (1u << 4) | (W8 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)(c.n >> 3) << 17) | (8u << 24);
        for (int k = g.k0; k < g.k1;) {
            stream_wait(&sh.t_empty[r.b], r.bph ^ 1, &sh.dead, p.err);
            tc_fence_after();
            const uint32_t d = tmem + r.b * 2 * C::kCols;
            const int end = W8 ? k + 1 : min(g.k1, k + kMoeBatch);
            for (uint32_t more = 0; k < end; ++k, more = 1) {
                if (W8) {  // a step's scales are there before its products start
                    stream_wait(&sh.s_full[r.slot], r.sph, &sh.dead, p.err);
                    r.scales();
                }
                stream_wait(&sh.full[r.s], r.ph, &sh.dead, p.err);
                tc_fence_after();
                const uint32_t a = ring + r.s * C::kStageBytes;
                const uint64_t a0 = smem_desc(a, 16, 1024), a1 = smem_desc(a + kMoeWeightBytes / 2, 16, 1024), bd = smem_desc(a + kMoeWeightBytes, 16, 1024);
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // 32 bytes of every row a product
                    if (W8) {
                        stream_mma_f8(one, d, a0 + 2 * i, bd + 2 * i, idesc, i > 0 || more);
                        stream_mma_f8(one, d + C::kCols, a1 + 2 * i, bd + 2 * i, idesc, i > 0 || more);
                    } else {
                        moe_mma_bf16(one, d, a0 + 2 * i, bd + 2 * i, idesc, i > 0 || more);
                        moe_mma_bf16(one, d + C::kCols, a1 + 2 * i, bd + 2 * i, idesc, i > 0 || more);
                    }
                }
                stream_commit(one, &sh.empty[r.s]);
                r.stage(C::kStages);
            }
            stream_commit(one, &sh.t_full[turn][r.b]);
            r.buffer(C::kBufs);
        }
    }
}

// e4m3: a step's scales, of each token's block times those of the weights' two blocks.
template <int G, bool DOWN>
__device__ __forceinline__ void moe_scales(const MoeArgs &p, MoeShared &sh, const MoeLine &l, MoeRing &r) {
    const int lane = threadIdx.x & 31, db = (p.d + 127) / 128, fb = (p.ff + 127) / 128;
    const bool by_token = !DOWN && p.n <= kMoeByToken;
    if (DOWN) stream_wait(&sh.go, 0, &sh.dead, p.err);
    MoeSeg g;
    long long at = l.s0;
    while (moe_next(l, at, g)) {
        const MoeTile t = moe_tile<G>(sh, l, g.unit);
        const int cols = by_token ? p.n : t.count, blocks = DOWN ? fb : db;
        const float *xs = (DOWN ? p.hs : p.xs) + (size_t)(by_token ? 0 : t.start) * blocks;
        const float *w0, *w1;
        if (DOWN) {
            w0 = p.d_scales + ((size_t)t.expert * db + 2 * t.tile) * fb;
            w1 = 2 * t.tile + 1 < db ? w0 + fb : w0;
        } else {
            w0 = p.gu_scales + ((size_t)t.expert * 2 * fb + t.tile) * db;
            w1 = w0 + (size_t)fb * db;
        }
        for (int k = g.k0; k < g.k1; k += 4) {
            float x[4], a[4], b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = k + j < g.k1;
                x[j] = in && lane < cols ? __ldcg(xs + (size_t)lane * blocks + k + j) : 0.0f;
                a[j] = in ? __ldg(w0 + k + j) : 0.0f;
                b[j] = in ? __ldg(w1 + k + j) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (k + j >= g.k1) break;
                stream_wait(&sh.s_empty[r.slot], r.sph ^ 1, &sh.dead, p.err);
                sh.scale[r.slot][0][lane] = x[j] * a[j];
                sh.scale[r.slot][1][lane] = x[j] * b[j];
                __syncwarp();
                stream_arrive(lane == 0, smem_u32(&sh.s_full[r.slot]));
                r.scales();
            }
        }
    }
}

// silu(gate) * up; a function of its own, so that its code is fetched once.
__device__ __noinline__ float moe_act(float gate, float up) { return gate / (1.0f + expf(-gate)) * up; }

template <int N>
__device__ __forceinline__ void moe_ld(uint32_t t, float *v) {
    if constexpr (N == 24) {
        stream_ld<16>(t, v);
        stream_ld<8>(t + 16, v + 16);
    } else if constexpr (N == 48) {
        stream_ld<32>(t, v);
        stream_ld<16>(t + 32, v + 32);
    } else {
        stream_ld<N>(t, v);
    }
}

// Two warpgroups add up, a segment each in turn: thread r is row r of either half.
template <typename C, bool DOWN, int P>
__device__ __forceinline__ void moe_sums(const MoeArgs &p, MoeShared &sh, const MoeLine &l, MoeRing &r, uint32_t tmem, int &turn, uint32_t &seen) {
    constexpr int G = C::kGroup, NG = G / 8, PH = C::kH;
    constexpr bool W8 = C::kElem == 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2, f = threadIdx.x & 127;
    const uint32_t from = tmem + ((uint32_t)(warp & 3) << 21), one = lane == 0;
    const bool by_token = !DOWN && p.n <= kMoeByToken;
    MoeSeg g;
    long long at = l.s0;
    for (; moe_next(l, at, g); turn ^= 1) {
        if (turn != wg) {  // the other's: its buffers and slots pass by
            const int batches = W8 ? g.k1 - g.k0 : (g.k1 - g.k0 + kMoeBatch - 1) / kMoeBatch;
            for (int i = 0; i < batches; ++i) {
                r.buffer(C::kBufs);
                if (W8) r.scales();
            }
            continue;
        }
        const MoeTile t = moe_tile<G>(sh, l, g.unit);
        const MoeCols<P> cols(by_token ? p.n : t.count);
        float acc[2][G];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < G; ++i) acc[h][i] = 0.0f;
        for (int k = g.k0; k < g.k1; k += W8 ? 1 : kMoeBatch) {
            stream_wait(&sh.t_full[wg][r.b], seen >> r.b & 1, &sh.dead, p.err);
            seen ^= 1u << r.b;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                if (j < cols.groups) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v[8 * P];
                        moe_ld<8 * P>(from + r.b * 2 * C::kCols + h * C::kCols + j * 8 * P, v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float x = v[8 * (P - 1) + i];
#pragma unroll
                            for (int q = P - 2; q >= 0; --q) x = W8 ? __fmaf_rn(x, 0.0625f, v[8 * q + i]) : x + v[8 * q + i];
                            acc[h][8 * j + i] = W8 ? __fmaf_rn(x, sh.scale[r.slot][h][8 * j + i], acc[h][8 * j + i]) : acc[h][8 * j + i] + x;
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            stream_arrive(one, smem_u32(&sh.t_empty[r.b]));
            if (W8) {
                stream_arrive(one, smem_u32(&sh.s_empty[r.slot]));
                r.scales();
            }
            r.buffer(C::kBufs);
        }
        // Sums go through memory, cut tile or not, so that what follows is one
        // short loop over groups of eight tokens: a tile ends once or twice a
        // phase and CTA, and code that runs once is paid for in fetches of it.
        const bool whole = g.k0 == 0 && g.k1 == l.steps;
        float *mine = p.parts + ((size_t)blockIdx.x * 4 + (whole ? 2 + wg : g.k0 == 0)) * kMoeSums + f;
#pragma unroll
        for (int j = 0; j < NG; ++j)
            if (j < cols.groups) {
#pragma unroll
                for (int i = 8 * j; i < 8 * j + 8; ++i) {
                    __stcg(mine + i * 128, acc[0][i]);
                    __stcg(mine + (kMoeGroup + i) * 128, acc[1][i]);
                }
            }
        int first = blockIdx.x, last = blockIdx.x;
        if (!whole) {  // a cut tile: whoever is last goes on
            const long long u0 = (long long)g.unit * l.steps;
            first = l.holder(u0);
            last = l.holder(u0 + l.steps - 1);
            int *counter = p.counters + (DOWN ? gridDim.x : 0) + first;
            named_sync(1 + wg, 128);
            if (f == 0) {
                const bool is = stream_count(counter) == last - first;
                if (is) *counter = 0;
                sh.last[wg] = is;
            }
            named_sync(1 + wg, 128);
            if (!sh.last[wg]) continue;
        }
        for (int j = 0; j < cols.groups; ++j) {
            float a[8], b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = b[i] = 0.0f;
            const float *parts = p.parts + (size_t)first * 4 * kMoeSums + j * 1024 + f;
            for (int c = 0; c <= last - first; c += kMoeAtOnce) {  // in CTA order, several requested together
                float v[kMoeAtOnce][16];
#pragma unroll
                for (int q = 0; q < kMoeAtOnce; ++q) {
                    const int k = min(c + q, last - first);
                    const float *part = parts + (size_t)(4 * k + (whole ? 2 + wg : k == 0)) * kMoeSums;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[q][i] = __ldcg(part + i * 128), v[q][8 + i] = __ldcg(part + (kMoeGroup + i) * 128);
                }
#pragma unroll
                for (int q = 0; q < kMoeAtOnce; ++q)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (c + q <= last - first) a[i] += v[q][i], b[i] += v[q][8 + i];
            }
            if (DOWN) {
                const int row = t.tile * 256 + f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (8 * j + i < t.count) {
                        float *to = p.out + (size_t)sh.list[t.start + 8 * j + i] * p.d + row;
                        if (row < p.d) __stcg(to, a[i]);
                        if (row + 128 < p.d) __stcg(to + 128, b[i]);
                    }
                continue;
            }
            // the intermediate, in pieces at the pair's place in the experts' order
            constexpr int E = W8 ? 1 : 2;
            const int feature = t.tile * 128 + f;
            const size_t step = (size_t)p.n * p.k * p.ff * E;
            for (int i = 0; i < 8; ++i) a[i] = moe_act(a[i], b[i]);
            if (W8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(a[i]) & 0x7fffffffu);
                    if (lane == 0) sh.top[wg][warp & 3][i] = top;
                }
                named_sync(1 + wg, 128);
            }
            // by token: column c is token c's, and its place is looked for
            for (int q = 0; q < (by_token ? t.count : min(8, t.count - 8 * j)); ++q) {
                const int at = t.start + 8 * j + q, col = by_token ? sh.list[at] / p.k : q;
                float h = a[0], up = 1.0f, back;
#pragma unroll
                for (int i = 1; i < 8; ++i)
                    if (i == col) h = a[i];
                if (W8) {
                    moe_scale(max(max(sh.top[wg][0][col], sh.top[wg][1][col]), max(sh.top[wg][2][col], sh.top[wg][3][col])), up, back);
                    if (f == 0) p.hs[(size_t)at * ((p.ff + 127) / 128) + t.tile] = back;
                }
                if (feature < p.ff) moe_put<W8, PH>(p.hp + ((size_t)at * p.ff + feature) * E, step, h, up);
            }
            if (W8) named_sync(1 + wg, 128);  // before sh.top is written again
        }
    }
}

template <bool W8, typename X>
__global__ __launch_bounds__(kMoeThreads, 1) void moe_kernel(const __grid_constant__ MoeArgs p) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *ring_p = smem_raw + (ring - smem_u32(smem_raw));
    MoeShared &sh = *reinterpret_cast<MoeShared *>(ring_p + kMoeRing);
    const int warp = threadIdx.x >> 5;
    constexpr bool XB = sizeof(X) == 2;
    using C = MoeCfg<W8, XB>;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMoeMaxStages; ++i) {
            mbar_init(&sh.full[i], 2);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kMoeSlots; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_empty[i], 4);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sh.t_full[0][i], 1);
            mbar_init(&sh.t_full[1][i], 1);
            mbar_init(&sh.t_empty[i], 4);
        }
        mbar_init(&sh.go, 1);
        mbar_init(&sh.done, 1);
        sh.dead = 0;
        fence_mbarrier_init();
    }
    if (warp == 9) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    const bool by_token = p.n <= kMoeByToken;
    const int gw = blockIdx.x * (kMoeThreads / 32) + warp, gn = gridDim.x * (kMoeThreads / 32);
    if (by_token) {  // a CTA an expert and up to four tokens, its warps' parts added here
        const int parts = kMoeThreads / 32;
        float2(&part)[2][kMoeThreads / 32][4] = *reinterpret_cast<float2(*)[2][kMoeThreads / 32][4]>(ring_p);
        for (int i = blockIdx.x, odd = 0; i < (p.n + 3) / 4 * p.experts; i += gridDim.x, odd ^= 1) {
            const int e = i % p.experts, t0 = i / p.experts * 4;
            if (p.n == 1) moe_logits<1>(p, e, t0, warp, parts, part[odd][warp], 1);
            else moe_logits<4>(p, e, t0, warp, parts, part[odd][warp], 1);
            __syncthreads();
            if (threadIdx.x < min(4, p.n - t0)) {
                float2 v = part[odd][0][threadIdx.x];
                for (int w = 1; w < parts; ++w) moe_add2(v.x, v.y, part[odd][w][threadIdx.x].x, part[odd][w][threadIdx.x].y);
                p.logits[(long long)(t0 + threadIdx.x) * p.experts + e] = v;
            }
        }
    } else {
        const int each = p.experts * p.splits;
        for (int i = gw; i < (p.n + 3) / 4 * each; i += gn) {
            const int e = i % each / p.splits, t0 = i / each * 4, split = i % p.splits;
            moe_logits<4>(p, e, t0, split, p.splits, p.logits + ((long long)split * p.n + t0) * p.experts + e, p.experts);
        }
    }
    if (by_token) {
        moe_split_x<W8, C::kX>(p, nullptr, p.n);
        moe_fence_copies();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    MoeRoute &route = *reinterpret_cast<MoeRoute *>(ring_p);
    bool dead = moe_meet_all(p, sh, 0);
    if (!dead) {
        if (by_token) {
            moe_keys(p, 0, p.n, route.key[0], threadIdx.x, kMoeThreads);
            __syncthreads();
            moe_choose(p, p.n, route.key[0], route.ahead, route.chosen);
            if (blockIdx.x == 0 && warp < p.n) moe_weights(p, warp, route.key[0] + warp * p.experts, route.chosen + warp * p.k);
        } else {  // a token's by one CTA, for all
            for (int t = blockIdx.x; t < p.n; t += gridDim.x) {
                moe_keys(p, t, 1, route.key[0], threadIdx.x, kMoeThreads);
                __syncthreads();
                moe_choose(p, 1, route.key[0], route.ahead, route.chosen);
                if (warp == 0) moe_weights(p, t, route.key[0], route.chosen);
                if (threadIdx.x < p.k) p.choices[t * p.k + threadIdx.x] = route.chosen[threadIdx.x];
                __syncthreads();
            }
            dead = moe_meet_all(p, sh, 1);
            for (int i = threadIdx.x; i < p.n * p.k; i += kMoeThreads) route.chosen[i] = __ldcg(p.choices + i);
        }
        __syncthreads();
    }
    if (!dead) {
        moe_route<C::kGroup>(p, sh, route);
        if (!by_token) {
            moe_split_x<W8, C::kX>(p, sh.list, p.n * p.k);
            moe_fence_copies();
            __syncthreads();
            dead = moe_meet_all(p, sh, 2);
        }
        // the choices lay in the ring: copies may overwrite them now
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        moe_fence_copies();
        __syncthreads();
    }
    if (!dead) {
        const int jobs = sh.jobs[p.experts];
        const MoeLine gu(jobs, (p.ff + 127) / 128, (p.d + C::kStep - 1) / C::kStep), dn(jobs, (p.d + 255) / 256, (p.ff + C::kStep - 1) / C::kStep);
        if (warp >= 8) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMoeRegsOther));
            MoeRing r;
            if (warp == 8) {
                moe_copies<C, false, C::kX>(p, sh, ring, gu, r);
                moe_copies<C, true, C::kH>(p, sh, ring, dn, r);
                // After a wait that gave up, copies may be under way that nobody waits for: they land within microseconds.
                if (*(volatile int *)&sh.dead)
                    for (const long long t0 = clock64(); clock64() - t0 < 20000000ll;) {}
            } else if (warp == 9) {
                int turn = 0;
                moe_products<C, false, C::kX>(p, sh, ring, gu, r, tmem, turn);
                moe_products<C, true, C::kH>(p, sh, ring, dn, r, tmem, turn);
                const uint32_t one = stream_elect();
                stream_commit(one, &sh.done);
                mbar_wait(&sh.done, 0, p.err);
            } else if (W8 && warp == 10) {
                moe_scales<C::kGroup, false>(p, sh, gu, r);
                moe_scales<C::kGroup, true>(p, sh, dn, r);
            }
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMoeRegsSum));
            MoeRing r;
            int turn = 0;
            uint32_t seen = 0;  // phases of its buffers, a bit each
            moe_sums<C, false, C::kX>(p, sh, gu, r, tmem, turn, seen);
            moe_fence_copies();
            named_sync(3, 256);
            if (threadIdx.x == 0) {
                moe_meet(p.bars + 3, &sh.dead, p.err);
                moe_fence_copies();
                mbar_arrive(&sh.go);
            }
            moe_sums<C, true, C::kH>(p, sh, dn, r, tmem, turn, seen);
            named_sync(3, 256);
            if (threadIdx.x == 0) moe_meet(p.bars + 4, &sh.dead, p.err);
            named_sync(3, 256);
            // the weighted sum, four values a thread
            const int quads = p.d / 4;
            for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < (long long)p.n * quads; i += (long long)gridDim.x * 256) {
                const int tok = (int)(i / quads), j = (int)(i - (long long)tok * quads) * 4;
                const long long at = (long long)tok * p.d + j;
                float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 2
                for (int c = 0; c < p.k; ++c) {
                    const long long pair = (long long)tok * p.k + c;
                    const float w = __ldcg(p.wts + pair);
                    const float4 o = __ldcg(reinterpret_cast<const float4 *>(p.out + pair * p.d + j));
                    v.x += w * o.x, v.y += w * o.y, v.z += w * o.z, v.w += w * o.w;
                }
                const float o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float res = p.residual ? load_as(p.residual, at + q, p.x_dtype) : 0.0f;
                    store_as(p.y, at + q, p.x_dtype, res + o[q]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, 512);
    // the last CTA leaves the meeting counts as they were found
    if (threadIdx.x == 0) {
        if (atomicAdd(p.bars + 5, 1) == (int)gridDim.x - 1) {
            for (int i = 0; i < 6; ++i) p.bars[i] = 0;
            __threadfence();
        }
    }
}

// ---------------------------------------------------------------- host
struct MoeSpace {
    size_t parts, logits, choices, wts, out, xp, xs, hp, hs, total;
    int splits;
};
static MoeSpace moe_space(int64_t n, int64_t d, int64_t ff, int64_t experts, int64_t k) {
    MoeSpace s;
    const size_t g = (size_t)sm_count(), pairs = (size_t)(n * k), rows = n <= kMoeByToken ? (size_t)n : pairs;
    size_t at = stream_ws_data();
    const auto take = [&](size_t bytes) {
        const size_t was = at;
        at += align_up(bytes, 256);
        return was;
    };
    s.parts = take(g * 4 * kMoeSums * 4);
    s.splits = moe_splits(n, d, experts, sm_count() * (kMoeThreads / 32));
    s.logits = take((size_t)(n * experts) * s.splits * 8);
    s.choices = take(pairs * 2);
    s.wts = take(pairs * 4);
    s.out = take(pairs * d * 4);
    s.xp = take(rows * d * 6);  // three pieces of two bytes or six of one
    s.xs = take(rows * ((d + 127) / 128) * 4);
    s.hp = take(pairs * ff * 6);
    s.hs = take(pairs * ((ff + 127) / 128) * 4);
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
    if (d * ff > ((int64_t)1 << 38) / n_experts) return DS_DIMENSION_TOO_LARGE;  // past any memory, and a copy's strides
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
    if (gate_up_scales_len != (w8 ? n_experts * 2 * fb * db : 0) || down_scales_len != (w8 ? n_experts * db * fb : 0)) return DS_GEMV_A_LENGTH_MISMATCH;
    if (y_len != n * d) return DS_A_LENGTH_MISMATCH;
    if (top_k > n_experts || d % unit || ff % unit) return DS_BAD_ARGUMENT;
    if (!x || !w_router || !w_gate_up || !w_down || !y || w8 != (gate_up_scales != nullptr) || w8 != (down_scales != nullptr)) return DS_BAD_ARGUMENT;
    if (((uintptr_t)x | (uintptr_t)w_router | (uintptr_t)w_gate_up | (uintptr_t)w_down) & 15) return DS_BAD_ARGUMENT;
    const int es = x_dtype == DS_BF16 ? 2 : 4;
    if (((uintptr_t)y | (uintptr_t)residual) % es || ((uintptr_t)expert_ids | (uintptr_t)expert_weights) & 3) return DS_BAD_ARGUMENT;
    if (((uintptr_t)gate_up_scales | (uintptr_t)down_scales) & 3) return DS_BAD_ARGUMENT;
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
                {gate_up_scales, gate_up_scales_len * 4}, {down_scales, down_scales_len * 4}};
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
    a.bars = reinterpret_cast<int *>(w + kWsHeader);
    a.counters = reinterpret_cast<int *>(w + stream_ws_counters());
    a.logits = reinterpret_cast<float2 *>(w + sp.logits);
    a.choices = reinterpret_cast<unsigned short *>(w + sp.choices);
    a.splits = sp.splits;
    a.wts = reinterpret_cast<float *>(w + sp.wts);
    a.xp = reinterpret_cast<unsigned char *>(w + sp.xp);
    a.hp = reinterpret_cast<unsigned char *>(w + sp.hp);
    a.xs = reinterpret_cast<float *>(w + sp.xs);
    a.hs = reinterpret_cast<float *>(w + sp.hs);
    a.parts = reinterpret_cast<float *>(w + sp.parts);
    a.out = reinterpret_cast<float *>(w + sp.out);
    const bool xb = x_dtype == DS_BF16;
    const int box = w8 ? 128 : 64, px = w8 ? (xb ? MoeCfg<true, true>::kX : MoeCfg<true, false>::kX) : (xb ? MoeCfg<false, true>::kX : MoeCfg<false, false>::kX);
    const int ph = w8 ? (xb ? MoeCfg<true, true>::kH : MoeCfg<true, false>::kH) : (xb ? MoeCfg<false, true>::kH : MoeCfg<false, false>::kH);
    const long long pairs = n * top_k, xrows = n <= kMoeByToken ? n : pairs;
    const long long gdims[3] = {d, ff, 2LL * n_experts}, gst[2] = {d * ws, ff * d * ws};
    const long long ddims[3] = {ff, d, n_experts}, dst[2] = {ff * ws, ff * d * ws};
    const long long xdims[3] = {d, xrows, px}, xst[2] = {d * ws, xrows * d * ws};
    const long long hdims[3] = {ff, pairs, ph}, hst[2] = {ff * ws, pairs * ff * ws};
    const int wbox[3] = {box, 128, 1}, xbox[3] = {box, 8, px}, hbox[3] = {box, 8, ph};
    if (!encode_tiled_3d(&a.tgu, w_gate_up, w_dtype, gdims, gst, wbox, true) ||
        !encode_tiled_3d(&a.td, w_down, w_dtype, ddims, dst, wbox, true) ||
        !encode_tiled_3d(&a.tx, a.xp, w_dtype, xdims, xst, xbox, true) ||
        !encode_tiled_3d(&a.th, a.hp, w_dtype, hdims, hst, hbox, true))
        return DS_CUDA_ERROR;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = w8 ? (xb ? moe_launch<true, __nv_bfloat16>(a, s) : moe_launch<true, float>(a, s))
                             : (xb ? moe_launch<false, __nv_bfloat16>(a, s) : moe_launch<false, float>(a, s));
    return e == cudaSuccess ? DS_OK : DS_CUDA_ERROR;
}
