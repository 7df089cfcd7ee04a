// Y = X W^T of e4m3 operands with a scale for each 128 of the sum
// (ds_gemm_fp8), on the fifth-generation tensor cores:
//   Y[s][r] = sum_b xs[s][b] ws[r / 128][b] sum_{c in block b} X[s][c] W[r][c]
// A step is one block of 128 of the sum: its products go to TMEM and from there,
// times the block's scale, to fp32 registers.  No scale enters the tensor core,
// so scales need not be powers of two, and every sum in it is short.
//
// This file: up to 64 rows of X, and up to 128 by very many features, where the
// weights' bytes are the bound (gemm_fp8_wide.cu: the others).  A tile is 128
// features (an MMA's M: lane r of TMEM is feature r), for more than 32 rows 256 in
// two halves, by all the rows of X, rounded up to 16, 32, 64 or 128 (the MMA's N):
// one token costs 16 columns.  Tiles, or equal runs of their steps (f8_runs), go
// one to a CTA; a cut tile's partial sums meet in the workspace and are added in
// CTA order by whichever CTA arrives last (a second launch for the wider ones took
// 12 us of 35 with 64 rows by 28,672 x 4,096).  No CTA waits for another.  A launch
// may begin while the one in front ends.
//
// A step brings its weights in one copy (16 KB for few rows, where the runs are
// short and even ones count: one token 9.9 us against 11.2; else 32 KB: 64 rows by
// 28,672 x 4,096 29 us against 33; both in equal runs), and up to four steps'
// columns are a batch: barriers and the latency of TMEM are paid once a batch.  A
// warpgroup for each half of the features adds it up.
//
// Measured in a graph: one token through 6,144 x 4,096 7.7 us (3.3 TB/s: eleven
// steps, the rest start and end), 64 through 28,672 x 4,096 22.6 us (5.4 TB/s), 128
// 27 us.
#include <algorithm>
#include <atomic>

#include "gemm_fp8.h"
#include "mma_stream.cuh"
#include "tc.h"

namespace ds {

constexpr int kF8K = 128;
constexpr int kF8Threads = 384;  // two warpgroups that add up; copies, products, scales, one idle
// Registers a thread: 168 at launch (384 x 168), moved to the warps that add
// up: 2 x 216 + 72 = 3 x 168.
constexpr int kF8RegsSum = 216, kF8RegsOther = 72;
constexpr int kF8MaxStages = 10;
constexpr int kF8Slots = 8;   // batches' scales ahead
constexpr int kF8MaxBufs = 4; // batches in TMEM
constexpr size_t kF8SmemLimit = 227 * 1024;

struct F8Shared {
    uint64_t full[kF8MaxStages], empty[kF8MaxStages];
    uint64_t s_full[kF8Slots], s_empty[kF8Slots];
    uint64_t t_full[kF8MaxBufs], t_empty[kF8MaxBufs];
    uint64_t done;
    uint32_t tmem;
    int dead, last;
    alignas(16) float scale[kF8Slots][2][128];
};

template <int NB>
struct F8Cfg {
    static constexpr int kHalves = NB <= 32 ? 1 : 2, kM = 128 * kHalves;
    static constexpr int kBatch = NB >= 64 ? 1 : NB >= 32 ? 2 : 4;  // steps of a batch
    static constexpr int kCols = kBatch * NB;                       // TMEM columns of a batch and half
    static constexpr int kBufs = NB >= 128 ? 2 : 4, kTmem = kBufs * kHalves * kCols;
    static constexpr int kStageBytes = (kM + NB) * kF8K;
    static constexpr int kFit = (int)((kF8SmemLimit - 1024 - sizeof(F8Shared)) / kStageBytes);
    static constexpr int kStages = kFit < kF8MaxStages ? kFit : kF8MaxStages;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + sizeof(F8Shared);
};

// A feature's outputs of rows row0 ... row0 + N - 1.
template <int N>
__device__ __forceinline__ void f8_store(const F8Args &p, int row0, int feature, const float (&v)[N]) {
    if (feature >= p.rows) return;
    const int n = p.n - row0;
    const long long at = row0 * p.ldy + feature;
    if (p.y_dtype == DS_BF16) {
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.y) + at;
#pragma unroll
        for (int i = 0; i < N; ++i, y += p.ldy)
            if (i < n) *y = __float2bfloat16_rn(v[i]);
    } else {
        float *y = static_cast<float *>(p.y) + at;
#pragma unroll
        for (int i = 0; i < N; ++i, y += p.ldy)
            if (i < n) *y = v[i];
    }
}

// NB: columns of an MMA, rows of X rounded up.
template <int NB>
__global__ __launch_bounds__(kF8Threads, 1) void fp8_gemm_kernel(const __grid_constant__ F8Args p) {
    using C = F8Cfg<NB>;
    constexpr int BS = C::kBatch, CH = NB < 32 ? NB : 32, kBufs = C::kBufs, HV = C::kHalves, kM = C::kM;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    F8Shared &sh = *reinterpret_cast<F8Shared *>(smem_raw + (base - smem_u32(smem_raw)) + C::kStages * C::kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *dead = &sh.dead;

    if (threadIdx.x == 0) {
        stream_prefetch_map(&p.tw);
        stream_prefetch_map(&p.tx);
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kF8Slots; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_empty[i], 4 * HV);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&sh.t_full[i], 1);
            mbar_init(&sh.t_empty[i], 4 * HV);
        }
        mbar_init(&sh.done, 1);
        sh.dead = 0;
        fence_mbarrier_init();
    }
    if (warp == 9) {
        tmem_alloc(&sh.tmem, C::kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    allow_dependent_launch();
    grid_dependency_wait();

    F8Walk walk(p, blockIdx.x, gridDim.x);
    F8Seg sg;
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kF8RegsOther));
        if (warp == 8) {
            // copies
            const uint32_t one = stream_elect();
            const uint64_t policy = policy_evict_first();  // weights are read once
            int s = 0;
            uint32_t ph = 1;
            long long issued = 0;
            while (walk.next(p, sg)) {
                for (int k = sg.k0; k < sg.k1; ++k) {
                    if (issued >= C::kStages) stream_wait(&sh.empty[s], ph, dead, p.err);
                    if (*dead) break;
                    if (one) mbar_arrive_expect_tx(&sh.full[s], C::kStageBytes);
                    const uint32_t dst = base + s * C::kStageBytes, bar = smem_u32(&sh.full[s]);
                    stream_box2(one, dst, &p.tw, k * kF8K, sg.tile * kM, bar, policy);
                    stream_box2(one, dst + kM * kF8K, &p.tx, k * kF8K, 0, bar);
                    ++issued;
                    if (++s == C::kStages) s = 0, ph ^= 1;
                }
                if (*dead) break;
            }
            // the copies still under way land before the CTA ends
            for (long long i = max(0ll, issued - C::kStages); i < issued; ++i)
                mbar_wait(&sh.full[i % C::kStages], (uint32_t)(i / C::kStages) & 1, p.err);
        } else if (warp == 9) {
            // products
            const uint32_t one = stream_elect();
            constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(NB >> 3) << 17) | (8u << 24);
            int s = 0, b = 0;
            uint32_t ph = 0, bph = 1;
            while (walk.next(p, sg)) {
                for (int k = sg.k0; k < sg.k1; k += BS) {
                    stream_wait(&sh.t_empty[b], bph, dead, p.err);
                    tc_fence_after();
                    for (int j = 0; j < BS && k + j < sg.k1; ++j) {
                        stream_wait(&sh.full[s], ph, dead, p.err);
                        tc_fence_after();
                        const uint64_t ad = smem_desc(base + s * C::kStageBytes, 16, 1024);
                        const uint64_t bd = smem_desc(base + s * C::kStageBytes + kM * kF8K, 16, 1024);
#pragma unroll
                        for (int h = 0; h < HV; ++h)
#pragma unroll
                            for (int i = 0; i < 4; ++i)  // 32 bytes of every row a product
                                stream_mma_f8(one, tmem + (HV * b + h) * C::kCols + j * NB, ad + h * (128 * 128 / 16) + 2 * i, bd + 2 * i, idesc, i > 0);
                        stream_commit(one, &sh.empty[s]);
                        if (++s == C::kStages) s = 0, ph ^= 1;
                    }
                    stream_commit(one, &sh.t_full[b]);
                    if (++b == kBufs) b = 0, bph ^= 1;
                }
            }
            stream_commit(one, &sh.done);
            mbar_wait(&sh.done, 0, p.err);
        } else if (warp == 10) {
            // scales: four steps' requested together, so that a batch's come before its products are done
            // (plain loads: the launch in front may have written them, weights' as well)
            constexpr int kVals = 4 * NB / 32, kPer = BS * NB / 32;  // values a lane holds, and of a batch
            int slot = 0;
            uint32_t ph = 1;
            while (walk.next(p, sg)) {
                const float *w0 = p.ws + (long long)(HV * sg.tile) * p.kb, *w1 = HV > 1 && 2 * sg.tile + 1 < (p.rows + 127) / 128 ? w0 + p.kb : w0;
                for (int k = sg.k0; k < sg.k1; k += 4) {
                    float v[kVals], a[kVals], b[kVals];
#pragma unroll
                    for (int i = 0; i < kVals; ++i) {
                        const int at = i * 32 + lane, j = k + at / NB, c = at % NB;
                        v[i] = j < sg.k1 && c < p.n ? p.xs[(long long)c * p.kb + j] : 0.0f;
                        a[i] = j < sg.k1 ? w0[j] : 0.0f;
                        b[i] = HV > 1 && j < sg.k1 ? w1[j] : 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 4; j += BS) {
                        if (k + j >= sg.k1) break;
                        stream_wait(&sh.s_empty[slot], ph, dead, p.err);
#pragma unroll
                        for (int i = 0; i < kPer; ++i) {
                            const int q = j / BS * kPer + i;
                            sh.scale[slot][0][i * 32 + lane] = v[q] * a[q];
                            if (HV > 1) sh.scale[slot][1][i * 32 + lane] = v[q] * b[q];
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.s_full[slot]);
                        if (++slot == kF8Slots) slot = 0, ph ^= 1;
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kF8RegsSum));
        // sums: thread r of warpgroup h is feature r of half h
        const int half = warp >> 2, r = threadIdx.x & 127;
        const uint32_t from = tmem + ((uint32_t)(warp & 3) << 21) + half * C::kCols, one = lane == 0;
        const uint32_t s_full0 = smem_u32(&sh.s_full[0]), s_empty0 = smem_u32(&sh.s_empty[0]), t_full0 = smem_u32(&sh.t_full[0]), t_empty0 = smem_u32(&sh.t_empty[0]);
        unsigned batch = 0;
        while (half < HV && walk.next(p, sg)) {
            float acc[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) acc[i] = 0.0f;
            for (int k = sg.k0; k < sg.k1; k += BS, ++batch) {
                const unsigned b = batch % kBufs, slot = batch % kF8Slots;
                stream_wait(s_full0 + slot * 8, (batch / kF8Slots) & 1, dead, p.err);
                stream_wait(t_full0 + b * 8, (batch / kBufs) & 1, dead, p.err);
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < BS; ++j) {
                    if (k + j < sg.k1) {
                        const float *scale = sh.scale[slot][half] + j * NB;
#pragma unroll
                        for (int c = 0; c < NB; c += CH) {
                            float v[CH];
                            stream_ld<CH>(from + b * HV * C::kCols + j * NB + c, v);
#pragma unroll
                            for (int i = 0; i < CH; i += 4) {
                                const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(scale + c + i);
                                stream_fma2(acc[c + i], acc[c + i + 1], v[i], v[i + 1], f.x);
                                stream_fma2(acc[c + i + 2], acc[c + i + 3], v[i + 2], v[i + 3], f.y);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                stream_arrive(one, t_empty0 + b * 8);
                stream_arrive(one, s_empty0 + slot * 8);
            }
            const int feature = sg.tile * kM + half * 128 + r;
            if (sg.split < 0) {
                f8_store<NB>(p, 0, feature, acc);
                continue;
            }
            constexpr size_t part = HV * NB * 128;  // floats of a partial sum, a half after the other
            float *mine = p.partials + ((size_t)blockIdx.x + sg.split) * part + half * NB * 128 + r;
#pragma unroll
            for (int i = 0; i < NB; ++i) __stcg(mine + i * 128, acc[i]);
            int first, last;
            f8_contributors(p, sg.split, first, last);
            named_sync(1, 128 * HV);
            if (threadIdx.x == 0) {
                const bool is = stream_count(p.counters + sg.split) == last - first;
                if (is) p.counters[sg.split] = 0;
                sh.last = is;
            }
            named_sync(1, 128 * HV);
            if (sh.last) {
                constexpr int AT = NB < 32 ? NB : 32;  // columns at a time
#pragma unroll 1
                for (int c = 0; c < min(NB, p.n); c += AT) {
                    float sum[AT];
                    f8_join<AT, 128>(p.partials + ((size_t)first + sg.split) * part + (half * NB + c) * 128 + r, part, last - first + 1, sum);
                    f8_store<AT>(p, c, feature, sum);
                }
            }
            named_sync(1, 128 * HV);  // before sh.last is written again
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, C::kTmem);
}

// ---------------------------------------------------------------- host
struct F8Plan {
    bool wide;
    int bn, m_tiles, n_tiles, grid, rounds, split;
    unsigned runs;
};

static F8Plan f8_plan(int64_t n, int64_t rows, int64_t cols) {
    F8Plan t;
    const int64_t kb = (cols + kF8K - 1) / kF8K;
    t.wide = n > kF8NarrowMost || (n > kF8Narrow && (rows + kF8WideFeatures - 1) / kF8WideFeatures <= f8_wide_pairs());
    int64_t tiles;
    if (t.wide) {  // m_tiles: features, n_tiles: rows of X
        t.bn = kF8WideFeatures;
        t.m_tiles = (int)((rows + kF8WideFeatures - 1) / kF8WideFeatures);
        t.n_tiles = (int)((n + kF8WideRows - 1) / kF8WideRows);
        tiles = (int64_t)t.m_tiles * t.n_tiles;
        t.grid = f8_wide_pairs();
    } else {
        t.bn = 16;
        while (t.bn < n) t.bn *= 2;
        const int m = t.bn <= 32 ? F8Cfg<32>::kM : F8Cfg<64>::kM;
        tiles = t.m_tiles = (int)((rows + m - 1) / m);
        t.n_tiles = 1;
        t.grid = sm_count();
    }
    t.rounds = (int)(tiles / t.grid);
    t.split = (int)(tiles - (int64_t)t.rounds * t.grid);
    t.runs = f8_runs(t.split, (int)kb, t.grid, t.bn);
    if (t.rounds == 0) t.grid = (int)t.runs;
    return t;
}
static size_t f8_ws_bytes(const F8Plan &t) {
    const size_t floats = t.wide ? f8_wide_partial_floats(t.split, t.runs) : f8_cut(t.split, t.runs) ? ((size_t)t.runs + t.split) * t.bn * F8Cfg<64>::kM : 0;
    return stream_ws_data() + floats * 4;
}

template <int NB>
static cudaError_t f8_launch(const F8Args &a, const F8Plan &t, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};  // devices whose limit is raised, a bit each
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(fp8_gemm_kernel<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kF8SmemLimit);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    return launch_ex(fp8_gemm_kernel<NB>, dim3(t.grid), dim3(kF8Threads), F8Cfg<NB>::kSmem, s, true, a);
}

}  // namespace ds

using namespace ds;

extern "C" DS_API size_t ds_gemm_fp8_workspace_bytes(int64_t n, int64_t rows, int64_t cols) {
    if (n < 1 || rows < 1 || cols < 1 || n > DS_MAX_DIM || rows > DS_MAX_DIM || cols > DS_MAX_DIM) return 0;
    return f8_ws_bytes(f8_plan(n, rows, cols));
}

extern "C" DS_API int ds_gemm_fp8(const void *W, int64_t w_len, int64_t w_stride, const float *w_scales,
                                  int64_t w_scales_len, const void *X, int64_t x_len, int64_t x_stride,
                                  const float *x_scales, int64_t x_scales_len, int64_t n, int64_t rows, int64_t cols,
                                  void *Y, int64_t y_len, int y_dtype, int64_t y_stride, void *workspace,
                                  size_t workspace_bytes, ds_stream_t stream) {
    if (n < 1 || rows < 1 || cols < 1) return DS_EMPTY_DIMENSION;
    if (n > DS_MAX_DIM || rows > DS_MAX_DIM || cols > DS_MAX_DIM || w_stride > DS_MAX_DIM || x_stride > DS_MAX_DIM ||
        y_stride > DS_MAX_DIM)
        return DS_DIMENSION_TOO_LARGE;
    const int64_t kb = (cols + kF8K - 1) / kF8K, blocks = (rows + 127) / 128;
    if (blocks * ((n + 255) / 256) > 0x3fffffffLL) return DS_DIMENSION_TOO_LARGE;
    if (y_dtype != DS_F32 && y_dtype != DS_BF16) return DS_BAD_DTYPE;
    if (w_stride < cols || w_len < (rows - 1) * w_stride + cols || w_scales_len != blocks * kb) return DS_GEMV_A_LENGTH_MISMATCH;
    if (x_stride < cols || x_len < (n - 1) * x_stride + cols || x_scales_len != n * kb) return DS_GEMV_X_LENGTH_MISMATCH;
    if (y_stride < rows || y_len < (n - 1) * y_stride + rows) return DS_A_LENGTH_MISMATCH;
    const int es = y_dtype == DS_BF16 ? 2 : 4;
    if (!W || !X || !Y || !w_scales || !x_scales) return DS_BAD_ARGUMENT;
    if ((((uintptr_t)W | (uintptr_t)X) & 15) || w_stride % 16 || x_stride % 16) return DS_BAD_ARGUMENT;
    if ((uintptr_t)Y % es || (uintptr_t)w_scales % 4 || (uintptr_t)x_scales % 4) return DS_BAD_ARGUMENT;
    const F8Plan t = f8_plan(n, rows, cols);
    if (!workspace || workspace_bytes < f8_ws_bytes(t)) return DS_WORKSPACE_TOO_SMALL;
    if ((uintptr_t)workspace & 255) return DS_BAD_ARGUMENT;
    const uintptr_t y0 = (uintptr_t)Y, y1 = y0 + ((n - 1) * y_stride + rows) * es;
    const struct {
        uintptr_t at;
        int64_t n;
    } in[] = {{(uintptr_t)W, (rows - 1) * w_stride + cols}, {(uintptr_t)X, (n - 1) * x_stride + cols},
              {(uintptr_t)w_scales, blocks * kb * 4}, {(uintptr_t)x_scales, n * kb * 4}};
    for (const auto &i : in)
        if (y0 < i.at + i.n && i.at < y1) return DS_BAD_ARGUMENT;
    F8Args a = {};
    a.ws = w_scales;
    a.xs = x_scales;
    a.rows = (int)rows;
    a.n = (int)n;
    a.kb = (int)kb;
    a.bn = t.bn;
    a.m_tiles = t.m_tiles;
    a.n_tiles = t.n_tiles;
    a.rounds = t.rounds;
    a.split = t.split;
    a.runs = t.runs;
    a.y = Y;
    a.y_dtype = y_dtype;
    a.ldy = y_stride;
    char *w = static_cast<char *>(workspace);
    a.err = reinterpret_cast<int *>(w);
    a.counters = reinterpret_cast<int *>(w + stream_ws_counters());
    a.partials = reinterpret_cast<float *>(w + stream_ws_data());
    if (!encode_tiled_2d(&a.tw, W, DS_E4M3, cols, rows, w_stride, kF8K, t.wide || t.bn <= 32 ? 128 : 256, true) ||
        !encode_tiled_2d(&a.tx, X, DS_E4M3, cols, n, x_stride, kF8K, t.wide ? 128 : t.bn, true))
        return DS_CUDA_ERROR;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = t.wide ? f8_wide_launch(a, t.grid, s) : t.bn == 16 ? f8_launch<16>(a, t, s) : t.bn == 32 ? f8_launch<32>(a, t, s)
                        : t.bn == 64 ? f8_launch<64>(a, t, s) : f8_launch<128>(a, t, s);
    return e == cudaSuccess ? DS_OK : DS_CUDA_ERROR;
}
