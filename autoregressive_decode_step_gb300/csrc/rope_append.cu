// Rotary positions of one or several axes for the rows of a fused q|k|v
// projection, the rotated k and the v written to their cache slots ("Inside
// the engine", section 1: qkPrep, RoPE and the K/V write in one pass;
// "decode-ops", "API - Method": rope).
//
// Pair p of a head turns by pos[axis(p)] * f_p, f_p = base^(-2p / rot_dim).
// Only the fraction of a full turn matters, so f_p / (2 pi) is held as a
// 64-bit fixed-point fraction F_p of a turn and the product pos * F_p modulo
// 2^64 is the angle, reduced exactly by integer overflow: a position of
// 2^31 - 1 leaves an error under 2^-33 of a turn, where an fp32 angle of a far
// position has lost whole digits.  The quadrant comes off the top two bits
// before the rest is rounded to fp32, so sine and cosine are those of an
// argument within an eighth of a turn.
//
// Bound by bytes (each element read once and written once); a row's angles
// are formed once, in shared memory, for all its heads.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "tc.h"

namespace ds {

constexpr int kRaThreads = 256;
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

// Eight consecutive elements as fp32, and back (16-byte aligned addresses).
__device__ __forceinline__ void ra_load8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void ra_load8(const __nv_bfloat16 *p, float (&v)[8]) {
    widen16(*reinterpret_cast<const uint4 *>(p), v);
}
__device__ __forceinline__ void ra_store8(float *p, const float (&v)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void ra_store8(__nv_bfloat16 *p, const float (&v)[8]) {
    __nv_bfloat16 b[8];  // the one rounding of a rotated value
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float2bfloat16_rn(v[i]);
    *reinterpret_cast<uint4 *>(p) = pack8_bf16(b);
}
__device__ __forceinline__ void ra_store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void ra_store1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// One block per row.  VEC: eight pairs (or sixteen untouched elements' half)
// per item with 16-byte accesses; else one pair or element per item.
template <typename XT, typename QT, typename KT, bool VEC, int P>
__global__ void __launch_bounds__(kRaThreads)
    rope_append_kernel(const RopeAppendArgs a, const __grid_constant__ RopeTurns<P> turns) {
    __shared__ float2 cs[P];
    const int half = a.rot >> 1, hd = a.hd, n_rot = a.n_qh + a.n_kvh;
    for (int r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
        const int slot = a.slots[r];
        bool ok = slot >= 0;  // a negative slot: a row of padding
        if (ok && slot >= a.cache_rows) {
            ok = false;
            if (threadIdx.x == 0) flag_error(a.err, DS_ERR_POSITION);
        }
        int bad = 0;
        if (ok && threadIdx.x < half) {
            const int pr = threadIdx.x;
            const int pos = a.positions[(long long)turns.axis[pr] * a.n_rows + r];
            bad = pos < 0;
            cs[pr] = ra_cos_sin((unsigned long long)(unsigned)pos * turns.turn[pr]);
        }
        if (__syncthreads_or(bad)) {
            if (threadIdx.x == 0) flag_error(a.err, DS_ERR_POSITION);
            ok = false;
        }
        if (ok) {
            const XT *x = static_cast<const XT *>(a.x) + (long long)r * a.row_stride;
            QT *q = static_cast<QT *>(a.q) + (long long)r * a.n_qh * hd;
            KT *k = static_cast<KT *>(a.k_cache) + (long long)slot * a.n_kvh * hd;
            KT *v = static_cast<KT *>(a.v_cache) + (long long)slot * a.n_kvh * hd;
            constexpr int W = VEC ? 8 : 1;
            const bool split = a.layout == DS_ROPE_HALF_SPLIT;
            const int per_rot = half / W, per_cp = (hd - a.rot) / W, per_v = hd / W;
            const int n1 = n_rot * per_rot, n2 = n1 + n_rot * per_cp, n3 = n2 + a.n_kvh * per_v;
            for (int i = threadIdx.x; i < n3; i += kRaThreads) {
                if (i < n1) {  // W pairs of a q or k head
                    const int head = i / per_rot, pr = (i % per_rot) * W;
                    const int ia = split ? pr : 2 * pr, ib = split ? pr + half : 2 * pr + W;
                    const XT *src = x + head * hd;
                    if constexpr (VEC) {
                        float u[8], w[8], yu[8], yw[8];
                        ra_load8(src + ia, u);
                        ra_load8(src + ib, w);
                        if (split) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 t = cs[pr + e];
                                yu[e] = u[e] * t.x - w[e] * t.y;
                                yw[e] = w[e] * t.x + u[e] * t.y;
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; e += 2) {
                                const float2 t = cs[pr + (e >> 1)], t2 = cs[pr + 4 + (e >> 1)];
                                yu[e] = u[e] * t.x - u[e + 1] * t.y;
                                yu[e + 1] = u[e + 1] * t.x + u[e] * t.y;
                                yw[e] = w[e] * t2.x - w[e + 1] * t2.y;
                                yw[e + 1] = w[e + 1] * t2.x + w[e] * t2.y;
                            }
                        }
                        if (head < a.n_qh) {
                            ra_store8(q + head * hd + ia, yu);
                            ra_store8(q + head * hd + ib, yw);
                        } else {
                            ra_store8(k + (head - a.n_qh) * hd + ia, yu);
                            ra_store8(k + (head - a.n_qh) * hd + ib, yw);
                        }
                    } else {
                        const float2 t = cs[pr];
                        const float u = to_f32(src[ia]), w = to_f32(src[ib]);
                        const float yu = u * t.x - w * t.y, yw = w * t.x + u * t.y;
                        if (head < a.n_qh) {
                            ra_store1(q + head * hd + ia, yu);
                            ra_store1(q + head * hd + ib, yw);
                        } else {
                            ra_store1(k + (head - a.n_qh) * hd + ia, yu);
                            ra_store1(k + (head - a.n_qh) * hd + ib, yw);
                        }
                    }
                } else {  // W elements as they are: the tail of a q or k head, or v
                    int head, d;
                    if (i < n2) {
                        head = (i - n1) / per_cp;
                        d = a.rot + ((i - n1) % per_cp) * W;
                    } else {
                        head = n_rot + (i - n2) / per_v;
                        d = ((i - n2) % per_v) * W;
                    }
                    const XT *src = x + head * hd + d;
                    if constexpr (VEC) {
                        float u[8];
                        ra_load8(src, u);
                        if (head < a.n_qh)
                            ra_store8(q + head * hd + d, u);
                        else if (head < n_rot)
                            ra_store8(k + (head - a.n_qh) * hd + d, u);
                        else
                            ra_store8(v + (head - n_rot) * hd + d, u);
                    } else {
                        const float u = to_f32(*src);
                        if (head < a.n_qh)
                            ra_store1(q + head * hd + d, u);
                        else if (head < n_rot)
                            ra_store1(k + (head - a.n_qh) * hd + d, u);
                        else
                            ra_store1(v + (head - n_rot) * hd + d, u);
                    }
                }
            }
        }
        __syncthreads();  // the row's angles are read before the next row's are written
    }
}

template <typename XT, typename QT, typename KT, int P>
static cudaError_t launch_ra(const RopeAppendArgs &a, const RopeTurns<P> &t, bool vec, cudaStream_t s) {
    const int grid = (int)std::min<long long>(a.n_rows, 1LL << 20);
    return vec ? launch_ex(rope_append_kernel<XT, QT, KT, true, P>, dim3(grid), dim3(kRaThreads), 0, s, false, a, t)
               : launch_ex(rope_append_kernel<XT, QT, KT, false, P>, dim3(grid), dim3(kRaThreads), 0, s, false, a, t);
}

template <int P>
static cudaError_t launch_ra_types(const RopeAppendArgs &a, const unsigned char *axes, double base, int xd, int qd,
                                   int kd, bool vec, cudaStream_t s) {
    RopeTurns<P> t = {};
    for (int p = 0; p < a.rot / 2; ++p) {
        const double turns = std::pow(base, -2.0 * p / a.rot) / 6.283185307179586476925286766559;
        const double frac = turns - std::floor(turns);
        t.turn[p] = frac < 1.0 ? (unsigned long long)std::ldexp(frac, 64) : 0ull;
        t.axis[p] = axes ? axes[p] : 0;
    }
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
    const uintptr_t x0 = (uintptr_t)qkv, x1 = x0 + (size_t)qkv_len * xe, q0 = (uintptr_t)q_out, q1 = q0 + (size_t)q_len * qe;
    if (q0 < x1 && x0 < q1) return DS_BAD_ARGUMENT;  // blocks read a row while others write theirs
    if (!workspace || workspace_bytes < kWsHeader) return DS_WORKSPACE_TOO_SMALL;
    if ((uintptr_t)workspace & 255) return DS_BAD_ARGUMENT;
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
