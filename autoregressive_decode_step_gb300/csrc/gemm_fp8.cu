// Y = X W^T of e4m3 operands with a scale for each 128 of the sum
// (ds_gemm_fp8), on the fifth-generation tensor cores:
//   Y[s][r] = sum_b xs[s][b] ws[r / 128][b] sum_{c in block b} X[s][c] W[r][c]
//
// A tile is 128 features (the MMA's M: lane r of TMEM is feature r) by up to
// 256 rows of X (its N), a step of the ring one block of 128 of the sum: four
// tcgen05.mma of kind::f8f6f4 into one TMEM buffer, which two warpgroups take
// out, half of the columns each, and add to fp32 registers times the block's
// scale.  So no scale ever enters the tensor core, and scales need not be
// powers of two.  Features are M whatever n is: a single token costs an MMA of
// 16 columns, and the weights' bytes bound it.
//
// Tiles are dealt out whole, one a CTA and round, as long as a round fills the
// card; what is left is cut into equal runs of steps, one a CTA, whose partial
// sums meet in the workspace and are added in CTA order: by whichever CTA
// arrives last for tiles of up to 32 rows (16 KB a partial), by a second launch
// for wider ones.  No CTA waits for another.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "tc.h"
#include "tcgen05.cuh"

namespace ds {

constexpr int kF8M = 128, kF8K = 128;
constexpr int kF8Threads = 352;  // two warpgroups that add up, the copying, the MMA and the scales' warp
constexpr int kF8MaxStages = 12;
constexpr int kF8Slots = 8;      // blocks' scales ahead
constexpr int kF8MaxBufs = 4;
constexpr int kF8Inline = 32;    // widest tile whose partials the last CTA adds
constexpr int kF8Group = 8;      // column tiles that follow one another before the next row of tiles
constexpr size_t kF8SmemLimit = 227 * 1024;

struct F8Args {
    CUtensorMap tw, tx;  // bytes, boxes {128, 128} and {128, bn}, 128-byte swizzle
    const float *ws, *xs;
    int rows, n, kb;
    int bn, m_tiles, n_tiles;
    int rounds, split;   // whole tiles a CTA takes; tiles behind them that are cut
    int stages;
    void *y;
    int y_dtype;
    long long ldy;
    float *partials;     // [CTA + split tile][bn][128]
    int *counters;       // a split tile's arrivals, zero between launches
    int *err;
};

struct F8Shared {
    uint64_t full[kF8MaxStages], empty[kF8MaxStages];
    uint64_t s_full[kF8Slots], s_empty[kF8Slots];
    uint64_t t_full[kF8MaxBufs], t_empty[kF8MaxBufs];
    uint64_t done;
    uint32_t tmem;
    int dead, last;
    alignas(16) float scale[kF8Slots][256];
};

constexpr size_t f8_smem(int bn, int stages) { return 1024 + (size_t)stages * (kF8M + bn) * kF8K + sizeof(F8Shared); }

// Wait for a phase; once any wait of the block has given up, at once.
__device__ __forceinline__ void f8_wait(uint64_t *bar, uint32_t parity, volatile int *dead, int *err) {
    if (mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return;
        if ((it & 63u) == 0) {
            if (*dead) return;
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                flag_error(err, DS_ERR_WAIT_TIMEOUT);
                *dead = 1;
                return;
            }
        }
    }
}

__device__ __forceinline__ uint32_t f8_elect() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one;
}
__device__ __forceinline__ void f8_box(uint32_t one, uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(one)
        : "memory");
}
__device__ __forceinline__ void f8_mma(uint32_t one, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "setp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
__device__ __forceinline__ void f8_commit(uint32_t one, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(one)
        : "memory");
}
// CH columns of this thread's lane, complete on return.
template <int CH>
__device__ __forceinline__ void f8_ld(uint32_t t, float *v);
template <>
__device__ __forceinline__ void f8_ld<8>(uint32_t t, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
        : "r"(t)
        : "memory");
}
template <>
__device__ __forceinline__ void f8_ld<16>(uint32_t t, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(t)
        : "memory");
}
template <>
__device__ __forceinline__ void f8_ld<32>(uint32_t t, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(t)
        : "memory");
}
// (a0, a1) += (x0, x1) (s0, s1)
__device__ __forceinline__ void f8_fma2(float &a0, float &a1, float x0, float x1, float s0, float s1) {
    asm("{\n\t.reg .b64 a, x, s;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 s, {%4, %5};\n\t"
        "fma.rn.f32x2 a, x, s, a;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(x0), "f"(x1), "f"(s0), "f"(s1));
}

// A CTA's segments: whole tiles in rounds, then its run of the split tiles' steps.
struct F8Seg {
    int mt, nt, k0, k1;
    int split;  // number of the split tile, or -1 (a whole tile)
};
// CTAs that have a run of the split tiles' w steps, at least a step each.
__device__ __forceinline__ int f8_runs(long long w, int grid) { return (int)max(1ll, min((long long)grid, w)); }
struct F8Walk {
    int round = 0;
    long long u, u1;
    __device__ explicit F8Walk(const F8Args &p) {
        const long long w = (long long)p.split * p.kb;
        const int runs = f8_runs(w, gridDim.x);
        u = w * min((int)blockIdx.x, runs) / runs;
        u1 = w * min((int)blockIdx.x + 1, runs) / runs;
    }
    __device__ bool next(const F8Args &p, F8Seg &s) {
        int tile;
        if (round < p.rounds) {
            tile = blockIdx.x + gridDim.x * round++;
            s.k0 = 0;
            s.k1 = p.kb;
            s.split = -1;
        } else if (u < u1) {
            s.split = (int)(u / p.kb);
            tile = p.rounds * gridDim.x + s.split;
            s.k0 = (int)(u - (long long)s.split * p.kb);
            s.k1 = (int)min((long long)p.kb, s.k0 + u1 - u);
            u += s.k1 - s.k0;
            if (s.k0 == 0 && s.k1 == p.kb) s.split = -1;
        } else {
            return false;
        }
        // kF8Group column tiles for each row of tiles: what runs at one time shares weights and rows in L2
        const int per = kF8Group * p.m_tiles, g = tile / per, nn = min(kF8Group, p.n_tiles - g * kF8Group);
        s.mt = (tile - g * per) / nn;
        s.nt = g * kF8Group + (tile - g * per) % nn;
        return true;
    }
};
// The CTAs that hold a split tile's first and last step.
__device__ __forceinline__ void f8_contributors(const F8Args &p, int grid, int split, int &first, int &last) {
    const long long w = (long long)p.split * p.kb, t = (long long)split * p.kb;
    const int runs = f8_runs(w, grid);
    first = (int)(((t + 1) * runs - 1) / w);
    last = (int)(((t + p.kb) * runs - 1) / w);
}

__device__ __forceinline__ void f8_store(const F8Args &p, int row, int feature, float v) {
    if (row < p.n && feature < p.rows) store_as(p.y, row * p.ldy + feature, p.y_dtype, v);
}

// NC: columns that a warpgroup adds up (half of the widest tile).
template <int NC>
__global__ __launch_bounds__(kF8Threads, 1) void fp8_gemm_kernel(const __grid_constant__ F8Args p) {
    constexpr int kBufs = 256 / NC < kF8MaxBufs ? 256 / NC : kF8MaxBufs;
    constexpr int kTmemCols = kBufs * 2 * NC < 32 ? 32 : kBufs * 2 * NC;
    constexpr int CH = NC < 32 ? NC : 32;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t stage_bytes = (uint32_t)(kF8M + p.bn) * kF8K;
    F8Shared &sh = *reinterpret_cast<F8Shared *>(smem_raw + (base - smem_u32(smem_raw)) + (size_t)p.stages * stage_bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *dead = &sh.dead;

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kF8Slots; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_empty[i], 8);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&sh.t_full[i], 1);
            mbar_init(&sh.t_empty[i], 8);
        }
        mbar_init(&sh.done, 1);
        sh.dead = 0;
        fence_mbarrier_init();
    }
    if (warp == 9) {
        tmem_alloc(&sh.tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    allow_dependent_launch();

    F8Walk walk(p);
    F8Seg sg;
    if (warp == 8) {
        // copies
        const uint32_t one = f8_elect();
        int s = 0;
        uint32_t ph = 1;
        long long issued = 0;
        while (walk.next(p, sg)) {
            for (int k = sg.k0; k < sg.k1; ++k) {
                f8_wait(&sh.empty[s], ph, dead, p.err);
                if (*dead) break;
                if (one) mbar_arrive_expect_tx(&sh.full[s], stage_bytes);
                const uint32_t dst = base + s * stage_bytes, bar = smem_u32(&sh.full[s]);
                f8_box(one, dst, &p.tw, k * kF8K, sg.mt * kF8M, bar);
                f8_box(one, dst + kF8M * kF8K, &p.tx, k * kF8K, sg.nt * p.bn, bar);
                ++issued;
                if (++s == p.stages) s = 0, ph ^= 1;
            }
            if (*dead) break;
        }
        // the copies still under way land before the CTA ends
        const int open = (int)min(issued, (long long)p.stages);
        for (long long i = issued - open; i < issued; ++i) mbar_wait(&sh.full[i % p.stages], (uint32_t)(i / p.stages) & 1, p.err);
    } else if (warp == 9) {
        // products
        const uint32_t one = f8_elect();
        const uint32_t idesc = (1u << 4) | ((uint32_t)(p.bn >> 3) << 17) | ((uint32_t)(kF8M >> 4) << 24);
        int s = 0, b = 0;
        uint32_t ph = 0, bph = 1;
        while (walk.next(p, sg)) {
            for (int k = sg.k0; k < sg.k1; ++k) {
                f8_wait(&sh.t_empty[b], bph, dead, p.err);
                f8_wait(&sh.full[s], ph, dead, p.err);
                tc_fence_after();
                const uint64_t ad = smem_desc(base + s * stage_bytes, 16, 1024);
                const uint64_t bd = smem_desc(base + s * stage_bytes + kF8M * kF8K, 16, 1024);
#pragma unroll
                for (int i = 0; i < 4; ++i)  // 32 bytes of every row a product
                    f8_mma(one, tmem + b * 2 * NC, ad + 2 * i, bd + 2 * i, idesc, i > 0);
                f8_commit(one, &sh.empty[s]);
                f8_commit(one, &sh.t_full[b]);
                if (++s == p.stages) s = 0, ph ^= 1;
                if (++b == kBufs) b = 0, bph ^= 1;
            }
        }
        f8_commit(one, &sh.done);
        mbar_wait(&sh.done, 0, p.err);
    } else if (warp == 10) {
        // scales: four blocks' requested together, so that a block's come before its product is done
        int slot = 0;
        uint32_t ph = 1;
        constexpr int kCols = (2 * NC + 31) / 32;
        while (walk.next(p, sg)) {
            const float *xs = p.xs + (long long)sg.nt * p.bn * p.kb, *ws = p.ws + (long long)sg.mt * p.kb;
            const int left = min(p.bn, p.n - sg.nt * p.bn);
            for (int k = sg.k0; k < sg.k1; k += 4) {
                float v[4][kCols];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float w = k + j < sg.k1 ? __ldg(ws + k + j) : 0.0f;
#pragma unroll
                    for (int i = 0; i < kCols; ++i) {
                        const int c = i * 32 + lane;
                        v[j][i] = k + j < sg.k1 && c < left ? __ldg(xs + (long long)c * p.kb + k + j) * w : 0.0f;
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (k + j >= sg.k1) break;
                    f8_wait(&sh.s_empty[slot], ph, dead, p.err);
#pragma unroll
                    for (int i = 0; i < kCols; ++i) sh.scale[slot][i * 32 + lane] = v[j][i];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.s_full[slot]);
                    if (++slot == kF8Slots) slot = 0, ph ^= 1;
                }
            }
        }
    } else {
        // sums: thread r of a warpgroup is feature r, its columns [col0, col0 + cw)
        const int cw = p.bn / 2, col0 = (warp >> 2) * cw, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        int b = 0, slot = 0;
        uint32_t bph = 0, ph = 0;
        while (walk.next(p, sg)) {
            float acc[NC];
#pragma unroll
            for (int i = 0; i < NC; ++i) acc[i] = 0.0f;
            for (int k = sg.k0; k < sg.k1; ++k) {
                f8_wait(&sh.s_full[slot], ph, dead, p.err);
                f8_wait(&sh.t_full[b], bph, dead, p.err);
                tc_fence_after();
                const float *scale = sh.scale[slot] + col0;
#pragma unroll
                for (int c = 0; c < NC; c += CH) {
                    if (c < cw) {
                        float v[CH];
                        f8_ld<CH>(tmem + lanes + b * 2 * NC + col0 + c, v);
                        if (c + CH >= cw) {  // the buffer is read out
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sh.t_empty[b]);
                        }
#pragma unroll
                        for (int i = 0; i < CH; i += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(scale + c + i);
                            f8_fma2(acc[c + i], acc[c + i + 1], v[i], v[i + 1], f.x, f.y);
                            f8_fma2(acc[c + i + 2], acc[c + i + 3], v[i + 2], v[i + 3], f.z, f.w);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.s_empty[slot]);
                if (++b == kBufs) b = 0, bph ^= 1;
                if (++slot == kF8Slots) slot = 0, ph ^= 1;
            }
            const int feature = sg.mt * kF8M + r, row0 = sg.nt * p.bn + col0;
            if (sg.split < 0) {
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (i < cw) f8_store(p, row0 + i, feature, acc[i]);
                continue;
            }
            const size_t part = (size_t)p.bn * kF8M;
            float *mine = p.partials + ((size_t)blockIdx.x + sg.split) * part + (size_t)col0 * kF8M + r;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (i < cw) __stcg(mine + i * kF8M, acc[i]);
            if (2 * NC > kF8Inline) continue;
            int first, last;
            f8_contributors(p, gridDim.x, sg.split, first, last);
            __threadfence();
            named_sync(1, 256);
            if (threadIdx.x == 0) sh.last = atomicAdd(p.counters + sg.split, 1) == last - first;
            named_sync(1, 256);
            if (sh.last) {
                __threadfence();
#pragma unroll
                for (int i = 0; i < NC; ++i) acc[i] = 0.0f;
                for (int c = first; c <= last; ++c) {
                    const float *from = p.partials + ((size_t)c + sg.split) * part + (size_t)col0 * kF8M + r;
#pragma unroll
                    for (int i = 0; i < NC; ++i)
                        if (i < cw) acc[i] += __ldcg(from + i * kF8M);
                }
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (i < cw) f8_store(p, row0 + i, feature, acc[i]);
                if (threadIdx.x == 0) p.counters[sg.split] = 0;
            }
            named_sync(1, 256);  // before sh.last is written again
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, kTmemCols);
}

// Adds a split tile's partials, 32 of its rows a block; thread r is feature r.
__global__ __launch_bounds__(kF8M) void fp8_join_kernel(const __grid_constant__ F8Args p, int grid) {
    grid_dependency_wait();
    const int chunks = (p.bn + 31) / 32, split = blockIdx.x / chunks, c0 = (int)(blockIdx.x % chunks) * 32;
    int first, last;
    f8_contributors(p, grid, split, first, last);
    if (first == last) return;  // one CTA had all of it
    const size_t part = (size_t)p.bn * kF8M;
    float acc[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i] = 0.0f;
    for (int c = first; c <= last; ++c) {
        const float *from = p.partials + ((size_t)c + split) * part + (size_t)c0 * kF8M + threadIdx.x;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (c0 + i < p.bn) acc[i] += __ldcg(from + i * kF8M);
    }
    const int tile = p.rounds * grid + split, per = kF8Group * p.m_tiles, g = tile / per;
    const int nn = min(kF8Group, p.n_tiles - g * kF8Group);
    const int mt = (tile - g * per) / nn, nt = g * kF8Group + (tile - g * per) % nn;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (c0 + i < p.bn) f8_store(p, nt * p.bn + c0 + i, mt * kF8M + threadIdx.x, acc[i]);
}

// ---------------------------------------------------------------- host
struct F8Plan {
    int bn, nc, m_tiles, n_tiles, grid, rounds, split, stages;
};

// Rows of X in equal tiles of at most 256, rounded up to the MMA's 16.
static F8Plan f8_plan(int64_t n, int64_t rows, int64_t cols) {
    F8Plan t;
    t.n_tiles = (int)((n + 255) / 256);
    t.bn = (int)(((n + t.n_tiles - 1) / t.n_tiles + 15) / 16 * 16);
    t.n_tiles = (int)((n + t.bn - 1) / t.bn);
    t.nc = 8;
    while (2 * t.nc < t.bn) t.nc *= 2;
    t.m_tiles = (int)((rows + kF8M - 1) / kF8M);
    const int64_t tiles = (int64_t)t.m_tiles * t.n_tiles, kb = (cols + kF8K - 1) / kF8K;
    t.grid = (int)std::min<int64_t>(sm_count(), tiles * kb);
    t.rounds = (int)(tiles / t.grid);
    t.split = (int)(tiles - (int64_t)t.rounds * t.grid);
    t.stages = (int)std::min<size_t>(kF8MaxStages, (kF8SmemLimit - f8_smem(t.bn, 0)) / ((kF8M + t.bn) * kF8K));
    return t;
}
static size_t f8_ws_bytes(const F8Plan &t) {
    return kWsHeader + align_up((size_t)sm_count() * 4, 256) + ((size_t)t.grid + t.split) * t.bn * kF8M * 4;
}

template <int NC>
static cudaError_t f8_launch(const F8Args &a, const F8Plan &t, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};  // devices whose limit is raised, a bit each
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(fp8_gemm_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kF8SmemLimit);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    e = launch_ex(fp8_gemm_kernel<NC>, dim3(t.grid), dim3(kF8Threads), f8_smem(t.bn, t.stages), s, false, a);
    if (e != cudaSuccess || 2 * NC <= kF8Inline || t.split == 0) return e;
    return launch_ex(fp8_join_kernel, dim3(t.split * ((t.bn + 31) / 32)), dim3(kF8M), 0, s, true, a, t.grid);
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
    const int64_t kb = (cols + kF8K - 1) / kF8K, m_tiles = (rows + kF8M - 1) / kF8M;
    if (m_tiles * ((n + 255) / 256) > 0x3fffffffLL) return DS_DIMENSION_TOO_LARGE;
    if (y_dtype != DS_F32 && y_dtype != DS_BF16) return DS_BAD_DTYPE;
    if (w_stride < cols || w_len < (rows - 1) * w_stride + cols || w_scales_len != m_tiles * kb) return DS_GEMV_A_LENGTH_MISMATCH;
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
              {(uintptr_t)w_scales, m_tiles * kb * 4}, {(uintptr_t)x_scales, n * kb * 4}};
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
    a.stages = t.stages;
    a.y = Y;
    a.y_dtype = y_dtype;
    a.ldy = y_stride;
    char *w = static_cast<char *>(workspace);
    a.err = reinterpret_cast<int *>(w);
    a.counters = reinterpret_cast<int *>(w + kWsHeader);
    a.partials = reinterpret_cast<float *>(w + kWsHeader + align_up((size_t)sm_count() * 4, 256));
    if (!encode_tiled_2d(&a.tw, W, DS_E4M3, cols, rows, w_stride, kF8K, kF8M, true) ||
        !encode_tiled_2d(&a.tx, X, DS_E4M3, cols, n, x_stride, kF8K, t.bn, true))
        return DS_CUDA_ERROR;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = t.nc == 8 ? f8_launch<8>(a, t, s) : t.nc == 16 ? f8_launch<16>(a, t, s)
                        : t.nc == 32 ? f8_launch<32>(a, t, s) : t.nc == 64 ? f8_launch<64>(a, t, s) : f8_launch<128>(a, t, s);
    return e == cudaSuccess ? DS_OK : DS_CUDA_ERROR;
}
