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
// read once.
//
// Measured in a graph: 8,192 x 14,336 bf16 in rows 55.6 us (6.4 TB/s, 94 % of the
// copy rate), a row of 4,096 fp32 1.4 us, weights of 4,099 x 1,001 bf16 with codes
// in odd rows 6.2 us (3.3 us in aligned ones).
#include "common.cuh"
#include "internal.h"

#include <algorithm>

namespace ds {

constexpr int kFqThreads = 256;
constexpr int kFqGroups = kFqThreads / 16;  // rows of a block worked on at a time
constexpr int kFqBlockThreads = 1024;       // of a 128 x 128 block
constexpr int kFqCtas = 4;                  // at a time on an SM
constexpr float kFqTiny = 0x1p-96f;         // least maximum: 448 / top and the scale stay normal numbers

struct FqArgs {
    const void *x;
    long long ldx, ldq;
    int rows, cols, kb, q8;  // q8: rows of q start on 8 bytes
    unsigned char *q;
    float *scales;
};

// Eight values as they are stored: 16 bytes of bf16, 32 of fp32.  (Plain loads: the
// launch in front may have written them.)
template <typename T>
struct FqRaw;
template <>
struct FqRaw<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void set(int i, __nv_bfloat16 v) { reinterpret_cast<__nv_bfloat16 *>(&w)[i] = v; }
    // the largest magnitude's bits: NaN above infinity above numbers
    __device__ __forceinline__ unsigned top() const {
        const unsigned m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
        return max(m << 16, m & 0xffff0000u);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const { widen16(w, v); }
};
template <>
struct FqRaw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
    __device__ __forceinline__ void set(int i, float v) { (i < 4 ? &a.x : &b.x)[i & 3] = v; }
    __device__ __forceinline__ unsigned top() const {
        float v[8];
        get(v);
        unsigned t = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(v[i]) & 0x7fffffffu);
        return t;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};
// From column c of a row on, zeros behind its end, value by value.  (Functions of
// their own where a path is rare or long: its code is then fetched once, and a
// small call's time is fetching code.)
template <typename T>
__device__ __noinline__ FqRaw<T> fq_load_slow(const T *row, int c, int cols) {
    FqRaw<T> r;
    r.zero();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols) r.set(i, row[c + i]);
    return r;
}
template <typename T, bool VEC>
__device__ __forceinline__ void fq_load(FqRaw<T> &r, const T *row, int c, int cols) {
    if (VEC && c + 8 <= cols) r.load(row + c);
    else r = fq_load_slow<T>(row, c, cols);
}

// A block's maximum from its bits; NaN for one that holds a NaN or an infinity.
__device__ __forceinline__ float fq_top(unsigned top) {
    return top < 0x7f800000u ? fmaxf(__uint_as_float(top), kFqTiny) : __int_as_float(0x7fffffff);
}

__device__ __forceinline__ unsigned fq_pair(float a, float b) {  // a in the low byte
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Eight codes from column c of a row on that are not eight bytes at once: a row's
// end, or (q8 false) rows that do not start on 8 bytes, where the sixteen threads
// store sixteen neighbouring bytes at a time.
__device__ __noinline__ void fq_store_slow(unsigned char *row, int c, int cols, unsigned lo, unsigned hi, bool q8) {
    if (q8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) row[c + i] = (unsigned char)((i < 4 ? lo : hi) >> (8 * (i & 3)));
        return;
    }
    const int lane = threadIdx.x & 15, half = threadIdx.x & 16, c0 = c - lane * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int from = half + (lane >> 3) + 2 * i;
        const unsigned a = __shfl_sync(0xffffu << half, lo, from), b = __shfl_sync(0xffffu << half, hi, from);
        if (c0 + 16 * i + lane < cols) row[c0 + 16 * i + lane] = (unsigned char)((lane & 4 ? b : a) >> (8 * (lane & 3)));
    }
}
template <typename T>
__device__ __forceinline__ void fq_store(unsigned char *row, int c, int cols, const FqRaw<T> &r, float factor, bool q8) {
    float v[8];
    r.get(v);
    const unsigned lo = fq_pair(v[0] * factor, v[1] * factor) | fq_pair(v[2] * factor, v[3] * factor) << 16;
    const unsigned hi = fq_pair(v[4] * factor, v[5] * factor) | fq_pair(v[6] * factor, v[7] * factor) << 16;
    if (q8 && c + 8 <= cols) *reinterpret_cast<uint2 *>(row + c) = make_uint2(lo, hi);
    else fq_store_slow(row, c, cols, lo, hi, q8);
}

// Blocks of 1 x 128: a group of sixteen threads takes block after block, U of
// them requested together.  Their 2 U quotients are formed side by side, one a
// thread: an IEEE division costs as much as the rest of a block's eight values
// (with one in every thread, and fewer CTAs at a time than the grid was made
// for, 8,192 x 14,336 bf16 took 141 us).  DENSE: whole blocks, no gaps between
// rows, so a block's place follows from its number.
template <typename T, bool VEC, bool DENSE, int U>
__global__ __launch_bounds__(kFqThreads, kFqCtas) void fp8_rows_kernel(const FqArgs p) {
    allow_dependent_launch();
    grid_dependency_wait();
    const int lane = threadIdx.x & 15, half = threadIdx.x & 16;
    const long long n = (long long)p.rows * p.kb, step = (long long)gridDim.x * kFqGroups;
    for (long long b0 = (long long)blockIdx.x * kFqGroups + (threadIdx.x >> 4); b0 - (threadIdx.x >> 4) < n; b0 += step * U) {
        FqRaw<T> v[U];
        long long row[U];
        int c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long b = min(b0 + u * step, n - 1);
            if (DENSE) {
                v[u].load(static_cast<const T *>(p.x) + b * 128 + lane * 8);
            } else {
                row[u] = n <= 0x7fffffffll ? (long long)((unsigned)b / (unsigned)p.kb) : b / p.kb;
                c[u] = (int)(b - row[u] * p.kb) * 128 + lane * 8;
                fq_load<T, VEC>(v[u], static_cast<const T *>(p.x) + row[u] * p.ldx, c[u], p.cols);
            }
        }
        float mine = 0.0f;  // lane: the maximum of block lane % U
#pragma unroll
        for (int u = 0; u < U; ++u) {
            unsigned top = v[u].top();
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (lane % U == u) mine = fq_top(top);
        }
        // lanes below U: 448 / top; the next U: top / 448
        const bool is_scale = lane >= U;
        const float quotient = __fdiv_rn(is_scale ? mine : 448.0f, is_scale ? 448.0f : mine);
        if (is_scale && lane < 2 * U && b0 + (lane - U) * step < n) p.scales[b0 + (lane - U) * step] = quotient;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float factor = __shfl_sync(0xffffffffu, quotient, half + u);
            if (b0 + u * step >= n) continue;
            if (DENSE) fq_store<T>(p.q + (b0 + u * step) * 128, lane * 8, 128, v[u], factor, true);
            else fq_store<T>(p.q + row[u] * p.ldq, c[u], p.cols, v[u], factor, p.q8);
        }
    }
}

// Blocks of 128 x 128, a CTA of 64 groups each, two rows a group (of sixteen
// groups, eight rows each: 4,099 x 1,001 bf16 8.4 us, the loads' latency one row
// after another).
template <typename T, bool VEC>
__global__ __launch_bounds__(kFqBlockThreads) void fp8_blocks_kernel(const FqArgs p) {
    constexpr int kGroups = kFqBlockThreads / 16, kRows = 128 / kGroups;
    __shared__ unsigned tops[kFqBlockThreads / 32];
    allow_dependent_launch();
    grid_dependency_wait();
    const int lane = threadIdx.x & 15, r0 = (int)(blockIdx.x / p.kb) * 128 + (threadIdx.x >> 4), c = (int)(blockIdx.x % p.kb) * 128 + lane * 8;
    FqRaw<T> v[kRows];
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = r0 + i * kGroups;
        fq_load<T, VEC>(v[i], static_cast<const T *>(p.x) + (long long)min(r, p.rows - 1) * p.ldx, c, r < p.rows ? p.cols : 0);
        top = max(top, v[i].top());
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, tops[threadIdx.x & 31]);
    const float t = fq_top(top), factor = __fdiv_rn(448.0f, t);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = r0 + i * kGroups;
        if (r < p.rows) fq_store<T>(p.q + (long long)r * p.ldq, c, p.cols, v[i], factor, p.q8);
    }
    if (threadIdx.x == 0) p.scales[blockIdx.x] = __fdiv_rn(t, 448.0f);
}

template <typename T, bool VEC>
static cudaError_t fq_launch(const FqArgs &a, int block_rows, cudaStream_t s) {
    if (block_rows == 128) {
        const long long grid = (long long)((a.rows + 127) / 128) * a.kb;
        return launch_ex(fp8_blocks_kernel<T, VEC>, dim3((unsigned)grid), dim3(kFqBlockThreads), 0, s, true, a);
    }
    const long long groups = ((long long)a.rows * a.kb + kFqGroups - 1) / kFqGroups, most = (long long)kFqCtas * sm_count();
    const bool dense = VEC && a.q8 && a.cols % 128 == 0 && a.ldx == a.cols && a.ldq == a.cols;
    constexpr int U = sizeof(T) == 2 ? 4 : 2;
    const unsigned grid = (unsigned)std::min(most, groups <= most ? groups : (groups + U - 1) / U);
    const dim3 g(grid), b(kFqThreads);
    // few blocks: one a group; many: U, on a full card
    if (groups <= most)
        return dense ? launch_ex(fp8_rows_kernel<T, VEC, VEC, 1>, g, b, 0, s, true, a) : launch_ex(fp8_rows_kernel<T, VEC, false, 1>, g, b, 0, s, true, a);
    return dense ? launch_ex(fp8_rows_kernel<T, VEC, VEC, U>, g, b, 0, s, true, a) : launch_ex(fp8_rows_kernel<T, VEC, false, U>, g, b, 0, s, true, a);
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
    const bool vec = (uintptr_t)x % 16 == 0 && (rows == 1 || x_stride * es % 16 == 0);
    a.q8 = (uintptr_t)q % 8 == 0 && (rows == 1 || q_stride % 8 == 0);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = x_dtype == DS_BF16 ? (vec ? fq_launch<__nv_bfloat16, true>(a, block_rows, s) : fq_launch<__nv_bfloat16, false>(a, block_rows, s))
                                             : (vec ? fq_launch<float, true>(a, block_rows, s) : fq_launch<float, false>(a, block_rows, s));
    return e == cudaSuccess ? DS_OK : DS_CUDA_ERROR;
}
