// Rows or weights in e4m3 with a scale for each block (ds_fp8_quantize).
//
// Per block of 1 x 128 or 128 x 128 values: top = max |x| (at least 2^-96),
// scale = top / 448, q = e4m3(x (448 / top)), rounded to nearest, ties to
// even.  The quotient is formed once a block; its rounding (2^-24) and the
// product's move a value by 2^-23 at most, beside the 2^-4 of e4m3 itself, and
// the largest product, 448 (1 + 2^-23), still rounds to 448.
//
// Sixteen threads hold a block's row, eight values each: one 16-byte load of
// bf16 (two of fp32), a maximum over four shuffles, one 8-byte store.  The
// values stay in registers between the maximum and the rounding, so each is
// read once.  A 128 x 128 block is one CTA of sixteen such groups, eight rows
// each.
#include "common.cuh"
#include "internal.h"

#include <algorithm>

namespace ds {

constexpr int kFqThreads = 256;
constexpr int kFqGroups = kFqThreads / 16;  // rows of a block worked on at a time
constexpr float kFqTiny = 0x1p-96f;         // least maximum: 448 / top and the scale stay normal numbers

struct FqArgs {
    const void *x;
    long long ldx, ldq;
    int rows, cols, kb;
    unsigned char *q;
    float *scales;
};

// Eight values from column c on, zeros behind the row's end; VEC: 16-byte loads.
template <typename T, bool VEC>
__device__ __forceinline__ void fq_load(const T *row, int c, int cols, float (&v)[8]) {
    if (VEC && c + 8 <= cols) {
        if (sizeof(T) == 2) {
            widen16(__ldg(reinterpret_cast<const uint4 *>(row + c)), v);
        } else {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(row + c));
            const float4 b = __ldg(reinterpret_cast<const float4 *>(row + c) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_f32(row[c + i]) : 0.0f;
}

// The largest magnitude as the bits of a float: NaN above infinity above numbers.
__device__ __forceinline__ unsigned fq_top(const float (&v)[8], unsigned top) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    return top;
}

// Scale and factor of a block; NaN for one that holds a NaN or an infinity.
__device__ __forceinline__ void fq_scale(unsigned top, float &scale, float &factor) {
    const float t = top < 0x7f800000u ? fmaxf(__uint_as_float(top), kFqTiny) : __int_as_float(0x7fffffff);
    scale = __fdiv_rn(t, 448.0f);
    factor = __fdiv_rn(448.0f, t);
}

__device__ __forceinline__ unsigned fq_pair(float a, float b) {  // a in the low byte
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

template <bool VEC>
__device__ __forceinline__ void fq_store(unsigned char *row, int c, int cols, const float (&v)[8], float factor) {
    const unsigned lo = fq_pair(v[0] * factor, v[1] * factor) | fq_pair(v[2] * factor, v[3] * factor) << 16;
    const unsigned hi = fq_pair(v[4] * factor, v[5] * factor) | fq_pair(v[6] * factor, v[7] * factor) << 16;
    if (VEC && c + 8 <= cols) {
        *reinterpret_cast<uint2 *>(row + c) = make_uint2(lo, hi);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols) row[c + i] = (unsigned char)((i < 4 ? lo : hi) >> (8 * (i & 3)));
}

// Blocks of 1 x 128: a group of sixteen threads takes block after block, the
// next UNROLL of them requested together.
template <typename T, bool VEC, int UNROLL>
__global__ __launch_bounds__(kFqThreads) void fp8_rows_kernel(const FqArgs p) {
    const int lane = threadIdx.x & 15;
    const long long n = (long long)p.rows * p.kb, step = (long long)gridDim.x * kFqGroups;
    for (long long b0 = (long long)blockIdx.x * kFqGroups + (threadIdx.x >> 4); b0 - (threadIdx.x >> 4) < n; b0 += step * UNROLL) {
        float v[UNROLL][8];
        long long row[UNROLL];
        int j[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const long long b = min(b0 + u * step, n - 1);
            row[u] = n <= 0x7fffffffll ? (long long)((unsigned)b / (unsigned)p.kb) : b / p.kb;
            j[u] = (int)(b - row[u] * p.kb);
            fq_load<T, VEC>(static_cast<const T *>(p.x) + row[u] * p.ldx, j[u] * 128 + lane * 8, p.cols, v[u]);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            unsigned top = fq_top(v[u], 0);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            float scale, factor;
            fq_scale(top, scale, factor);
            if (b0 + u * step < n) {
                fq_store<VEC>(p.q + row[u] * p.ldq, j[u] * 128 + lane * 8, p.cols, v[u], factor);
                if (lane == 0) p.scales[row[u] * p.kb + j[u]] = scale;
            }
        }
    }
}

// Blocks of 128 x 128, a CTA each.
template <typename T, bool VEC>
__global__ __launch_bounds__(kFqThreads) void fp8_blocks_kernel(const FqArgs p) {
    constexpr int kRows = 128 / kFqGroups;
    __shared__ unsigned tops[kFqThreads / 32];
    const int lane = threadIdx.x & 15, r0 = (int)(blockIdx.x / p.kb) * 128 + (threadIdx.x >> 4), c = (int)(blockIdx.x % p.kb) * 128 + lane * 8;
    float v[kRows][8];
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = r0 + i * kFqGroups;
        fq_load<T, VEC>(static_cast<const T *>(p.x) + (long long)min(r, p.rows - 1) * p.ldx, c, r < p.rows ? p.cols : 0, v[i]);
        top = fq_top(v[i], top);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFqThreads / 32; ++i) top = max(top, tops[i]);
    float scale, factor;
    fq_scale(top, scale, factor);
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        if (r0 + i * kFqGroups < p.rows) fq_store<VEC>(p.q + (long long)(r0 + i * kFqGroups) * p.ldq, c, p.cols, v[i], factor);
    if (threadIdx.x == 0) p.scales[blockIdx.x] = scale;
}

template <typename T, bool VEC>
static cudaError_t fq_launch(const FqArgs &a, int block_rows, cudaStream_t s) {
    if (block_rows == 128) {
        const long long grid = (long long)((a.rows + 127) / 128) * a.kb;
        return launch_ex(fp8_blocks_kernel<T, VEC>, dim3((unsigned)grid), dim3(kFqThreads), 0, s, false, a);
    }
    const long long groups = ((long long)a.rows * a.kb + kFqGroups - 1) / kFqGroups;
    constexpr int kUnroll = sizeof(T) == 2 ? 4 : 2;
    const long long most = 8LL * sm_count();
    if (groups <= most) return launch_ex(fp8_rows_kernel<T, VEC, 1>, dim3((unsigned)groups), dim3(kFqThreads), 0, s, false, a);
    return launch_ex(fp8_rows_kernel<T, VEC, kUnroll>, dim3((unsigned)std::min(most, (groups + kUnroll - 1) / kUnroll)),
                     dim3(kFqThreads), 0, s, false, a);
}

}  // namespace ds

using namespace ds;

extern "C" DS_API int ds_fp8_quantize(const void *x, int64_t x_len, int x_dtype, int64_t x_stride, int64_t rows,
                                      int64_t cols, int block_rows, void *q, int64_t q_len, int64_t q_stride,
                                      float *scales, int64_t scales_len, ds_stream_t stream) {
    if (rows < 1 || cols < 1) return DS_EMPTY_DIMENSION;
    if (rows > DS_MAX_DIM || cols > DS_MAX_DIM || x_stride > DS_MAX_DIM || q_stride > DS_MAX_DIM) return DS_DIMENSION_TOO_LARGE;
    if (x_dtype != DS_F32 && x_dtype != DS_BF16) return DS_BAD_DTYPE;
    if (block_rows != 1 && block_rows != 128) return DS_BAD_ARGUMENT;
    if (x_stride < cols || x_len < (rows - 1) * x_stride + cols) return DS_A_LENGTH_MISMATCH;
    const int64_t kb = (cols + 127) / 128, rb = (rows + block_rows - 1) / block_rows;
    if (q_stride < cols || q_len < (rows - 1) * q_stride + cols || scales_len != rb * kb) return DS_B_LENGTH_MISMATCH;
    if (rb * kb > 0x7fffffffLL && block_rows == 128) return DS_DIMENSION_TOO_LARGE;
    const int es = x_dtype == DS_BF16 ? 2 : 4;
    if (!x || !q || !scales || (uintptr_t)x % es || (uintptr_t)scales % 4) return DS_BAD_ARGUMENT;
    // a block's values are read before its codes are written, but not another block's
    const struct {
        uintptr_t at;
        int64_t n;
    } span[] = {{(uintptr_t)x, ((rows - 1) * x_stride + cols) * es}, {(uintptr_t)q, (rows - 1) * q_stride + cols},
                {(uintptr_t)scales, rb * kb * 4}};
    for (int i = 1; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (span[i].at < span[j].at + span[j].n && span[j].at < span[i].at + span[i].n) return DS_BAD_ARGUMENT;
    FqArgs a = {};
    a.x = x;
    a.ldx = x_stride;
    a.ldq = q_stride;
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.kb = (int)kb;
    a.q = static_cast<unsigned char *>(q);
    a.scales = scales;
    const bool vec = (uintptr_t)x % 16 == 0 && (rows == 1 || x_stride * es % 16 == 0) && (uintptr_t)q % 8 == 0 && (rows == 1 || q_stride % 8 == 0);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = x_dtype == DS_BF16 ? (vec ? fq_launch<__nv_bfloat16, true>(a, block_rows, s) : fq_launch<__nv_bfloat16, false>(a, block_rows, s))
                                             : (vec ? fq_launch<float, true>(a, block_rows, s) : fq_launch<float, false>(a, block_rows, s));
    return e == cudaSuccess ? DS_OK : DS_CUDA_ERROR;
}
