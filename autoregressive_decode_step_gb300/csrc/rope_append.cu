// Rotary positions of one or several axes for the rows of a fused q|k|v
// projection, the rotated k and the v written to their cache slots ("Inside
// the engine", section 1: qkPrep, RoPE and the K/V write in one pass;
// "decode-ops", "API - Method": rope).
//
// Pair p of a head turns by pos[axis(p)] * f_p, f_p = base^(-2p / rot_dim).
// Only the fraction of a full turn matters, so f_p / (2 pi) is held as a
// 64-bit fixed-point fraction F_p of a turn, right to a unit (ra_turns), and
// the product pos * F_p modulo 2^64 is the angle, reduced exactly by integer
// overflow: a position of 2^31 - 1 leaves an error under 2^-33 of a turn (for
// bases from 1e-8 up), where an fp32 angle of a far position has lost whole
// digits.  The quadrant comes off the top two bits before the rest is rounded
// to fp32, so sine and cosine are those of an argument within an eighth of a
// turn.
//
// Bound by bytes (each element read once and written once).  Two kernels:
//  - few rows: a thread keeps the same place of a row for all the rows of its
//    block, so what it does there is worked out once, and the next row's
//    element, slot and position are requested before this row's are used;
//  - from kRaBulkRows on: whole rows come through a shared-memory ring by bulk
//    copies, so the bytes in flight do not hang on the threads that wait for
//    them.
// A row's angles are formed once, in shared memory, for all its heads.
// Measured in a graph, us, heads of 128; up to 2,048 rows stay in L2:
//   rows                            512   1,001  1,500  2,048  4,096  8,192
//   32 + 8 + 8 bf16          first  4.3    6.4    8.1   10.3   20.5   44.4
//                            second 4.6    6.5    8.1    9.7   15.9   35.1  (5.7 TB/s)
//   32 + 8 + 8 fp32 to bf16  first  4.9    7.3    9.2   11.9   25.0   53.7
//                            second 5.6    8.2   10.1   12.9   23.7   48.9
//   32 + 8 + 8 fp32 to fp32  first  6.2    9.7   12.9   16.8   35.9   67.6
//                            second 6.7    9.7   12.4   15.6   35.6   69.3
//   4 + 2 + 2 bf16           first  3.2    4.0    4.5    5.4    8.0   13.3
//                            second 3.3    4.2    5.1    6.0    8.8   15.0
// So kRaBulkRows suits wide bf16 rows; wide fp32 rows lose up to 8 % or win 9 %
// by it and narrow rows lose 10 %.  Rows of single elements (see the entry
// point) always take the first kernel: 1,001 rows of 14 + 2 + 2 fp32 heads of
// 80, 40 dims of them rotated, 8.8 us, 8,192 rows 65.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "tc.h"

namespace ds {

constexpr int kRaThreads = 256;
constexpr int kRaBlocksPerSm = 4;
constexpr int kRaBulkRows = 2048;
constexpr int kRaMaxHd = 256;
constexpr int kRaMaxAxes = 8;

template <int P>
struct RopeTurns {
    unsigned long long turn[P];  // f_p / (2 pi) as a fraction of a turn, in units of 2^-64
    unsigned char axis[P];
};

struct RopeAppendArgs {
    const void *x;         // [n_rows][row_stride]: q heads, then k, then v
    long long row_stride;
    int n_rows;
    const int *positions;  // [n_axes][n_rows]
    int n_qh, n_kvh, hd, rot, layout;
    void *q;               // [n_rows][n_qh * hd]
    void *k_cache, *v_cache;
    long long cache_rows;
    const int *slots;      // [n_rows]
    int *err;
};

__device__ __forceinline__ float2 ra_cos_sin(unsigned long long turn) {
    const unsigned quad = (unsigned)((turn + (1ull << 61)) >> 62);  // nearest quarter turn
    const long long rest = (long long)(turn - ((unsigned long long)quad << 62));
    float s, c;
    sincospif((float)rest * 0x1p-63f, &s, &c);  // an eighth of a turn at most
    switch (quad & 3u) {
        case 0: return make_float2(c, s);
        case 1: return make_float2(-s, c);
        case 2: return make_float2(-c, -s);
        default: return make_float2(s, -c);
    }
}

// W consecutive elements as they are loaded (W 8: 16-byte accesses), as fp32,
// and back.
template <typename T, int W>
struct RaChunk;
template <>
struct RaChunk<float, 8> {
    float4 a, b;
    __device__ void load(const float *p) {
        a = __ldcs(reinterpret_cast<const float4 *>(p));
        b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};
template <>
struct RaChunk<__nv_bfloat16, 8> {
    uint4 a;
    __device__ void load(const __nv_bfloat16 *p) { a = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ void get(float (&v)[8]) const { widen16(a, v); }
};
template <typename T>
struct RaChunk<T, 1> {
    T a;
    __device__ void load(const T *p) { a = *p; }
    __device__ void get(float (&v)[1]) const { v[0] = to_f32(a); }
};
__device__ __forceinline__ void ra_store(float *p, const float (&v)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void ra_store(__nv_bfloat16 *p, const float (&v)[8]) {
    __nv_bfloat16 b[8];  // the one rounding of a rotated value
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float2bfloat16_rn(v[i]);
    *reinterpret_cast<uint4 *>(p) = pack8_bf16(b);
}
__device__ __forceinline__ void ra_store(float *p, const float (&v)[1]) { *p = v[0]; }
__device__ __forceinline__ void ra_store(__nv_bfloat16 *p, const float (&v)[1]) { *p = __float2bfloat16_rn(v[0]); }

__device__ __forceinline__ void ra_get8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void ra_get8(const __nv_bfloat16 *p, float (&v)[8]) {
    widen16(*reinterpret_cast<const uint4 *>(p), v);
}

// Rotate W pairs.  Half-split: pair e is (u[e], w[e]).  Interleaved: u holds
// pairs 0 .. W/2 - 1, w the others (W 1: the pair's two elements).
template <int W>
__device__ __forceinline__ void ra_rotate(const float (&u)[W], const float (&w)[W], const float (&c)[W],
                                          const float (&s)[W], bool split, float (&y0)[W], float (&y1)[W]) {
    if (split || W == 1) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            y0[e] = u[e] * c[e] - w[e] * s[e];
            y1[e] = w[e] * c[e] + u[e] * s[e];
        }
    } else {
        constexpr int h = W / 2;
#pragma unroll
        for (int e = 0; e < h; ++e) {
            y0[2 * e] = u[2 * e] * c[e] - u[2 * e + 1] * s[e];
            y0[2 * e + 1] = u[2 * e + 1] * c[e] + u[2 * e] * s[e];
            y1[2 * e] = w[2 * e] * c[h + e] - w[2 * e + 1] * s[h + e];
            y1[2 * e + 1] = w[2 * e + 1] * c[h + e] + w[2 * e] * s[h + e];
        }
    }
}

// A thread has one item of a row: W pairs of a q or k head (two chunks of W
// elements), or W elements as they are (the tail of a q or k head, or v).
// (Two a thread: half the blocks stay resident, 47 us against 44 at 8,192.)
template <typename XT, typename QT, typename KT, int W, int P>
__global__ void __launch_bounds__(kRaThreads)
    rope_append_kernel(const __grid_constant__ RopeAppendArgs a, const __grid_constant__ RopeTurns<P> turns) {
    __shared__ __align__(16) float cosine[2][P], sine[2][P];
    const int half = a.rot >> 1, hd = a.hd, n_rot = a.n_qh + a.n_kvh;
    const bool split = a.layout == DS_ROPE_HALF_SPLIT;
    const int tid = threadIdx.x;

    // what this thread's item is
    int src = 0, apart = 0, pair = 0, dst = 0, to = -1;  // to: 0 q, 1 k, 2 v, -1 none
    {
        const int per_rot = half / W, per_cp = (hd - a.rot) / W, per_v = hd / W;
        const int n1 = n_rot * per_rot, n2 = n1 + n_rot * per_cp, n3 = n2 + a.n_kvh * per_v;
        const int i = blockIdx.y * kRaThreads + tid;
        int head = 0, d = 0;
        if (i < n1) {
            head = i / per_rot;
            pair = (i % per_rot) * W;
            d = split ? pair : 2 * pair;
            apart = split ? half : W;  // the second chunk is so far behind the first; 0: none
        } else if (i < n2) {
            head = (i - n1) / per_cp;
            d = a.rot + ((i - n1) % per_cp) * W;
        } else if (i < n3) {
            head = n_rot + (i - n2) / per_v;
            d = ((i - n2) % per_v) * W;
        }
        to = i >= n3 ? -1 : head < a.n_qh ? 0 : head < n_rot ? 1 : 2;
        src = head * hd + d;
        dst = (to <= 0 ? head : to == 1 ? head - a.n_qh : head - n_rot) * hd + d;
    }

    RaChunk<XT, W> x0, x1;
    const int step = gridDim.x;
    int r = blockIdx.x;
    const int axis_row = tid < half ? turns.axis[tid] : 0;
    const unsigned long long turn = tid < half ? turns.turn[tid] : 0;
    auto pos_of = [&](int row) { return tid < half ? __ldg(a.positions + (long long)axis_row * a.n_rows + row) : 0; };
    auto fetch = [&](int row) {
        const XT *x = static_cast<const XT *>(a.x) + (long long)row * a.row_stride;
        if (to >= 0) x0.load(x + src);
        if (apart) x1.load(x + src + apart);
    };
    int slot = __ldg(a.slots + r), pos = pos_of(r);
    if (slot >= 0) fetch(r);  // a negative slot: a row of padding
    for (int turn_no = 0; r < a.n_rows; r += step, ++turn_no) {
        const int buf = turn_no & 1, next = r + step;
        int slot_n = -1, pos_n = 0;
        if (next < a.n_rows) {
            slot_n = __ldg(a.slots + next);
            pos_n = pos_of(next);
        }
        if (slot >= 0 && tid < half) {
            const float2 t = ra_cos_sin((unsigned long long)(unsigned)pos * turn);
            cosine[buf][tid] = t.x;
            sine[buf][tid] = t.y;
        }
        // (two sets of angles: a thread may be a row ahead, not two)
        const int bad = __syncthreads_or(slot >= 0 && (pos < 0 || slot >= a.cache_rows));
        if (bad && tid == 0) flag_error(a.err, DS_ERR_POSITION);
        const bool ok = slot >= 0 && !bad && to >= 0;
        float y0[W], y1[W];
        if (ok) x0.get(y0);
        if (ok && apart) {
            float u[W], w[W], c[W], s[W];
            x0.get(u);
            x1.get(w);
            if constexpr (W == 8) {
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float4 c4 = *reinterpret_cast<const float4 *>(&cosine[buf][pair + e]);
                    const float4 s4 = *reinterpret_cast<const float4 *>(&sine[buf][pair + e]);
                    c[e] = c4.x; c[e + 1] = c4.y; c[e + 2] = c4.z; c[e + 3] = c4.w;
                    s[e] = s4.x; s[e + 1] = s4.y; s[e + 2] = s4.z; s[e + 3] = s4.w;
                }
            } else {
                c[0] = cosine[buf][pair];
                s[0] = sine[buf][pair];
            }
            ra_rotate(u, w, c, s, split, y0, y1);
        }
        if (slot_n >= 0) fetch(next);
        if (ok && to == 0) {
            QT *q = static_cast<QT *>(a.q) + (long long)r * a.n_qh * hd + dst;
            ra_store(q, y0);
            if (apart) ra_store(q + apart, y1);
        } else if (ok) {
            KT *p = static_cast<KT *>(to == 1 ? a.k_cache : a.v_cache) + (long long)slot * a.n_kvh * hd + dst;
            ra_store(p, y0);
            if (apart) ra_store(p + apart, y1);
        }
        slot = slot_n;
        pos = pos_n;
    }
}

// Many rows: rows of x through a ring of bulk copies; what an item is stands in
// a table in shared memory.  A row of padding is fetched and not looked at.
struct RaItem {
    int src, apart, pair, dst;  // dst: offset within its buffer's row, x 4, + 0 q, 1 k, 2 v
};
constexpr int kRaStages = 3;
constexpr int kRaBulkBlocks = 4;         // blocks an SM, registers and shared memory permitting
constexpr int kRaBulkSmem = 100 * 1024;  // most shared memory a block takes

template <typename XT, typename QT, typename KT, int P>
__global__ void __launch_bounds__(kRaThreads, 4)
    rope_append_bulk_kernel(const __grid_constant__ RopeAppendArgs a, const __grid_constant__ RopeTurns<P> turns,
                            int n_items, int row_bytes) {
    extern __shared__ __align__(128) unsigned char ra_smem[];
    __shared__ __align__(16) float cosine[2][P], sine[2][P];
    __shared__ uint64_t full[kRaStages];
    RaItem *items = reinterpret_cast<RaItem *>(ra_smem + (size_t)kRaStages * row_bytes);
    const int half = a.rot >> 1, hd = a.hd, n_rot = a.n_qh + a.n_kvh, tid = threadIdx.x;
    const bool split = a.layout == DS_ROPE_HALF_SPLIT;
    const int step = gridDim.x, first = blockIdx.x;
    const uint64_t policy = policy_evict_first();
    auto fetch = [&](int n) {  // the block's n-th row, by one thread
        const long long row = first + (long long)n * step;
        if (row >= a.n_rows) return;
        mbar_arrive_expect_tx(&full[n % kRaStages], (uint32_t)row_bytes);
        bulk_g2s(ra_smem + (size_t)(n % kRaStages) * row_bytes, static_cast<const XT *>(a.x) + row * a.row_stride,
                 (uint32_t)row_bytes, &full[n % kRaStages], policy);
    };
    if (tid == 0) {
        for (int i = 0; i < kRaStages; ++i) mbar_init(&full[i], 1);
        fence_mbarrier_init();
        for (int i = 0; i < kRaStages - 1; ++i) fetch(i);
    }
    const int per_rot = half / 8, per_cp = (hd - a.rot) / 8, per_v = hd / 8;
    const int n1 = n_rot * per_rot, n2 = n1 + n_rot * per_cp;
    for (int i = tid; i < n_items; i += kRaThreads) {
        RaItem it = {0, 0, 0, 0};
        int head, d;
        if (i < n1) {
            head = i / per_rot;
            it.pair = (i % per_rot) * 8;
            d = split ? it.pair : 2 * it.pair;
            it.apart = split ? half : 8;
        } else if (i < n2) {
            head = (i - n1) / per_cp;
            d = a.rot + ((i - n1) % per_cp) * 8;
        } else {
            head = n_rot + (i - n2) / per_v;
            d = ((i - n2) % per_v) * 8;
        }
        it.src = head * hd + d;
        const int to = head < a.n_qh ? 0 : head < n_rot ? 1 : 2;
        it.dst = ((head - (to == 0 ? 0 : to == 1 ? a.n_qh : n_rot)) * hd + d) * 4 + to;
        items[i] = it;
    }
    const int axis_row = tid < half ? turns.axis[tid] : 0;
    const unsigned long long turn = tid < half ? turns.turn[tid] : 0;
    auto pos_of = [&](int row) { return tid < half ? __ldg(a.positions + (long long)axis_row * a.n_rows + row) : 0; };
    int slot = __ldg(a.slots + first), pos = pos_of(first);
    for (int n = 0, r = first; r < a.n_rows; r += step, ++n) {
        const int buf = n & 1, next = r + step;
        int slot_n = -1, pos_n = 0;
        if (next < a.n_rows) {
            slot_n = __ldg(a.slots + next);
            pos_n = pos_of(next);
        }
        if (slot >= 0 && tid < half) {
            const float2 t = ra_cos_sin((unsigned long long)(unsigned)pos * turn);
            cosine[buf][tid] = t.x;
            sine[buf][tid] = t.y;
        }
        // (also: every thread is done with the row before, whose stage is free)
        const int bad = __syncthreads_or(slot >= 0 && (pos < 0 || slot >= a.cache_rows));
        if (tid == 0) {
            if (bad) flag_error(a.err, DS_ERR_POSITION);
            fetch(n + kRaStages - 1);
        }
        const bool there = mbar_wait(&full[n % kRaStages], (n / kRaStages) & 1, a.err);
        if (there && slot >= 0 && !bad) {
            const XT *x = reinterpret_cast<const XT *>(ra_smem + (size_t)(n % kRaStages) * row_bytes);
            for (int i = tid; i < n_items; i += kRaThreads) {
                const int4 e4 = *reinterpret_cast<const int4 *>(items + i);
                const RaItem it = {e4.x, e4.y, e4.z, e4.w};
                float u[8], w[8];
                ra_get8(x + it.src, u);
                const int to = it.dst & 3, at = it.dst >> 2;
                QT *q = static_cast<QT *>(a.q) + (long long)r * a.n_qh * hd + at;
                KT *k = static_cast<KT *>(to == 1 ? a.k_cache : a.v_cache) + (long long)slot * a.n_kvh * hd + at;
                if (it.apart) {
                    ra_get8(x + it.src + it.apart, w);
                    float c[8], s[8], y0[8], y1[8];
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 c4 = *reinterpret_cast<const float4 *>(&cosine[buf][it.pair + e]);
                        const float4 s4 = *reinterpret_cast<const float4 *>(&sine[buf][it.pair + e]);
                        c[e] = c4.x; c[e + 1] = c4.y; c[e + 2] = c4.z; c[e + 3] = c4.w;
                        s[e] = s4.x; s[e + 1] = s4.y; s[e + 2] = s4.z; s[e + 3] = s4.w;
                    }
                    ra_rotate(u, w, c, s, split, y0, y1);
                    if (to == 0) {
                        ra_store(q, y0);
                        ra_store(q + it.apart, y1);
                    } else {
                        ra_store(k, y0);
                        ra_store(k + it.apart, y1);
                    }
                } else if (to == 0) {
                    ra_store(q, u);
                } else {
                    ra_store(k, u);
                }
            }
        }
        slot = slot_n;
        pos = pos_n;
    }
}

template <typename XT, typename QT, typename KT, int P>
static cudaError_t launch_ra_bulk(const RopeAppendArgs &a, const RopeTurns<P> &t, int items, int row_bytes, int smem,
                                  cudaStream_t s) {
    // (the most any call takes: the limit is the kernel's, and another thread's
    // call may set it between this one's two lines)
    const cudaError_t e = cudaFuncSetAttribute((const void *)rope_append_bulk_kernel<XT, QT, KT, P>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kRaBulkSmem);
    if (e != cudaSuccess) return e;
    const int per_sm = std::min(kRaBulkBlocks, 220 * 1024 / (smem + 2 * 1024));
    return launch_ex(rope_append_bulk_kernel<XT, QT, KT, P>, dim3(std::min(a.n_rows, per_sm * sm_count())),
                     dim3(kRaThreads), smem, s, false, a, t, items, row_bytes);
}

template <typename XT, typename QT, typename KT, int P>
static cudaError_t launch_ra(const RopeAppendArgs &a, const RopeTurns<P> &t, bool vec, cudaStream_t s) {
    const int w = vec ? 8 : 1;
    const int items = (a.n_qh + a.n_kvh) * (a.rot / 2 / w + (a.hd - a.rot) / w) + a.n_kvh * (a.hd / w);
    const int ny = (items + kRaThreads - 1) / kRaThreads;
    const int row_bytes = (a.n_qh + 2 * a.n_kvh) * a.hd * (int)sizeof(XT);
    const long long smem = (long long)kRaStages * row_bytes + (long long)items * sizeof(RaItem);
    if (vec && a.n_rows >= kRaBulkRows && smem <= kRaBulkSmem)
        return launch_ra_bulk<XT, QT, KT, P>(a, t, items, row_bytes, (int)smem, s);
    // as many blocks as stay resident; a block with several rows keeps loads in flight
    const int nx = std::min(a.n_rows, std::max(1, kRaBlocksPerSm * sm_count() / ny));
    return vec ? launch_ex(rope_append_kernel<XT, QT, KT, 8, P>, dim3(nx, ny), dim3(kRaThreads), 0, s, false, a, t)
               : launch_ex(rope_append_kernel<XT, QT, KT, 1, P>, dim3(nx, ny), dim3(kRaThreads), 0, s, false, a, t);
}

// A number as the sum of two doubles, about 104 bits.
struct Dd {
    double hi, lo;
};
static Dd dd_mul(Dd a, Dd b) {
    // (a fused multiply-add with zero: a plain product might be fused into the sum below)
    const double p = std::fma(a.hi, b.hi, 0.0);
    const double e = std::fma(a.hi, b.lo, std::fma(a.lo, b.hi, std::fma(a.hi, b.hi, -p)));
    const double s = p + e;
    return {s, e - (s - p)};
}

// x modulo 1 in units of 2^-64, to the nearest.
static unsigned long long ra_fraction(Dd x) {
    if (!std::isfinite(x.hi) || !std::isfinite(x.lo)) return 0;
    unsigned long long sum = 0;
    double rest = 0.0;
    for (const double part : {x.hi, x.lo}) {
        const double a = std::fabs(part), units = std::ldexp(a - std::floor(a), 64), whole = std::floor(units);
        const unsigned long long u = (unsigned long long)whole;
        sum += part < 0.0 ? 0ull - u : u;
        rest += part < 0.0 ? whole - units : units - whole;
    }
    return sum + (unsigned long long)std::llrint(rest);
}

// F_p = base^(-2p / rot) / (2 pi) modulo 1 in units of 2^-64.  A double holds
// 53 bits of it, which a far position would multiply into the angle (2^-25 of
// a turn at 2^31), so: the root r = base^(-2 / rot) by one step of Newton's
// method from the double's, r^(rot / 2) base = 1, and its powers by repeated
// products.  An error of 2^-95 of the frequency remains, a unit of F_p while
// that is below 2^30 turns a position (bases from 1e-8 up).
static void ra_turns(unsigned long long *turn, int n, double base) {
    const double r0 = std::pow(base, -1.0 / n);
    Dd one = {base, 0.0};
    for (int i = 0; i < n; ++i) one = dd_mul(one, {r0, 0.0});  // from base down to 1
    const Dd r = {r0, -r0 * (((one.hi - 1.0) + one.lo) / n)};
    Dd f = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / (2 pi)
    for (int p = 0; p < n; ++p) {
        turn[p] = ra_fraction(f);
        f = dd_mul(f, r);
    }
}

template <int P>
static cudaError_t launch_ra_types(const RopeAppendArgs &a, const unsigned char *axes, double base, int xd, int qd,
                                   int kd, bool vec, cudaStream_t s) {
    RopeTurns<P> t = {};
    ra_turns(t.turn, a.rot / 2, base);
    for (int p = 0; p < a.rot / 2; ++p) t.axis[p] = axes ? axes[p] : 0;
    using B = __nv_bfloat16;
    switch ((xd == DS_BF16) * 4 + (qd == DS_BF16) * 2 + (kd == DS_BF16)) {
        case 0: return launch_ra<float, float, float>(a, t, vec, s);
        case 1: return launch_ra<float, float, B>(a, t, vec, s);
        case 2: return launch_ra<float, B, float>(a, t, vec, s);
        case 3: return launch_ra<float, B, B>(a, t, vec, s);
        case 4: return launch_ra<B, float, float>(a, t, vec, s);
        case 5: return launch_ra<B, float, B>(a, t, vec, s);
        case 6: return launch_ra<B, B, float>(a, t, vec, s);
        default: return launch_ra<B, B, B>(a, t, vec, s);
    }
}

}  // namespace ds

using namespace ds;

extern "C" DS_API size_t ds_rope_append_workspace_bytes(void) { return kWsHeader; }

extern "C" DS_API int ds_rope_append(const void *qkv, int64_t qkv_len, int qkv_dtype, int64_t row_stride,
                                     int64_t n_rows, const int32_t *positions, int n_axes, const uint8_t *pair_axis,
                                     int n_qh, int n_kvh, int head_dim, int rot_dim, double base, int layout,
                                     void *q_out, int64_t q_len, int q_dtype, void *k_cache, void *v_cache,
                                     int kv_dtype, int64_t cache_rows, const int32_t *slots, void *workspace,
                                     size_t workspace_bytes, ds_stream_t stream) {
    if (n_rows < 1 || n_axes < 1 || n_qh < 1 || n_kvh < 1 || head_dim < 1 || rot_dim < 1 || cache_rows < 1)
        return DS_EMPTY_DIMENSION;
    const int64_t cols = ((int64_t)n_qh + 2 * (int64_t)n_kvh) * head_dim;
    if (n_rows > DS_MAX_DIM || cache_rows > DS_MAX_DIM || cols > DS_MAX_DIM || row_stride > DS_MAX_DIM)
        return DS_DIMENSION_TOO_LARGE;
    if (row_stride < cols || qkv_len < (n_rows - 1) * row_stride + cols) return DS_A_LENGTH_MISMATCH;
    if (q_len != n_rows * n_qh * head_dim) return DS_B_LENGTH_MISMATCH;
    if ((qkv_dtype != DS_F32 && qkv_dtype != DS_BF16) || (q_dtype != DS_F32 && q_dtype != DS_BF16) ||
        (kv_dtype != DS_F32 && kv_dtype != DS_BF16) ||
        (layout != DS_ROPE_HALF_SPLIT && layout != DS_ROPE_INTERLEAVED))
        return DS_BAD_DTYPE;
    if (head_dim > kRaMaxHd || rot_dim > head_dim || rot_dim % 2 || n_axes > kRaMaxAxes || !(base > 0.0) ||
        !std::isfinite(base))
        return DS_BAD_ARGUMENT;
    if (!qkv || !positions || !q_out || !k_cache || !v_cache || !slots || (n_axes > 1 && !pair_axis))
        return DS_BAD_ARGUMENT;
    for (int p = 0; pair_axis && p < rot_dim / 2; ++p)
        if (pair_axis[p] >= n_axes) return DS_BAD_ARGUMENT;
    const int xe = qkv_dtype == DS_BF16 ? 2 : 4, qe = q_dtype == DS_BF16 ? 2 : 4;
    // Blocks read a row while others write theirs.  (To the last row's end:
    // qkv_len may reach on, into a buffer that holds the outputs too.)
    const uintptr_t x0 = (uintptr_t)qkv, x1 = x0 + (size_t)((n_rows - 1) * row_stride + cols) * xe;
    const uintptr_t q0 = (uintptr_t)q_out, q1 = q0 + (size_t)q_len * qe;
    if (q0 < x1 && x0 < q1) return DS_BAD_ARGUMENT;
    if (!workspace || workspace_bytes < kWsHeader) return DS_WORKSPACE_TOO_SMALL;
    if ((uintptr_t)workspace & 255) return DS_BAD_ARGUMENT;
    const uintptr_t k0 = (uintptr_t)k_cache, v0 = (uintptr_t)v_cache;
    const size_t cb = (size_t)cache_rows * n_kvh * head_dim * (kv_dtype == DS_BF16 ? 2 : 4);
    if ((k0 < v0 + cb && v0 < k0 + cb) || (k0 < x1 && x0 < k0 + cb) || (v0 < x1 && x0 < v0 + cb) ||
        (k0 < q1 && q0 < k0 + cb) || (v0 < q1 && q0 < v0 + cb))
        return DS_BAD_ARGUMENT;
    RopeAppendArgs a = {};
    a.x = qkv;
    a.row_stride = row_stride;
    a.n_rows = (int)n_rows;
    a.positions = positions;
    a.n_qh = n_qh;
    a.n_kvh = n_kvh;
    a.hd = head_dim;
    a.rot = rot_dim;
    a.layout = layout;
    a.q = q_out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.cache_rows = cache_rows;
    a.slots = slots;
    a.err = static_cast<int *>(workspace);
    // 16-byte accesses need every head, half and row to start on 16 bytes
    const bool vec = (((uintptr_t)qkv | (uintptr_t)q_out | (uintptr_t)k_cache | (uintptr_t)v_cache) & 15) == 0 &&
                     row_stride % 8 == 0 && head_dim % 8 == 0 && rot_dim % 16 == 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = head_dim <= 128
                              ? launch_ra_types<64>(a, pair_axis, base, qkv_dtype, q_dtype, kv_dtype, vec, s)
                              : launch_ra_types<128>(a, pair_axis, base, qkv_dtype, q_dtype, kv_dtype, vec, s);
    return e == cudaSuccess ? DS_OK : DS_CUDA_ERROR;
}
