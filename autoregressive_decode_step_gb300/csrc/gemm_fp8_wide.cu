// ds_gemm_fp8 for many rows of X (kF8Narrow): pairs of SMs on tiles of 256 rows by
// 256 features.
//
// One tcgen05.mma of cta_group::2 spans both SMs of a pair: each holds 128 rows
// of X and half of the tile's weights in shared memory and gets its own 128
// rows of the product, lane r of its TMEM row r.  So an SM fetches 32 KB a step
// (a block of 128 of the sum) for 128 x 256 x 128 products: 512 tensor cycles
// against 64 bytes a cycle from L2; alone it would fetch 48 KB.
//
// A row's scale and its block of 128 features' make one factor a thread and
// step, so the sums cost one packed multiply-add per two columns.  Two warps issue
// the products of half a step each (64 of either SM's features: 128 columns of
// TMEM, four buffers); four warpgroups take 64 columns each out of TMEM, add
// them to registers and free the buffer before they do.
//
// Tiles are dealt out whole, one a pair and round; what is left over goes
// one to a pair or is cut into runs of steps (f8_runs) whose partial sums a second
// launch adds in order.
//
// Measured in a graph: 8,192 rows by 28,672 x 4,096 661 us (2.91 PFLOP/s, 1.52 of
// the measured bf16 rate) until the card is at its power limit, where an SM runs at
// 1.58 GHz, 750 us then; the tensor pipe active 63 % of the cycles (the issue slots
// 54 %: half of it the sums); 256 by 4,096 x 14,336 25 us, some 8 of them joining
// four partial sums a tile.
#include <algorithm>
#include <atomic>

#include "gemm_fp8.h"
#include "mma_stream.cuh"

namespace ds {

constexpr int kFwThreads = 640;  // sixteen warps that add up; copies, products of one half, scales, products of the other
// Registers a thread: 96 at launch (640 x 96), moved to the warps that add up:
// 4 x 104 + 64 = 5 x 96.
constexpr int kFwRegsSum = 104, kFwRegsOther = 64;
constexpr int kFwStages = 5, kFwHalf = 128 * 128, kFwStageBytes = 2 * kFwHalf;
constexpr int kFwFactors = 4;  // slots of factors, four steps each
constexpr int kFwBufs = 4;    // TMEM buffers of 128 columns, two a step
constexpr int kFwGroup = 8;   // row tiles that follow one another before the next features
constexpr int kFwOutRow = 80;  // 64 bytes of a row and 16 that keep rows apart on the banks
constexpr int kFwPart = 128 * kF8WideFeatures;  // floats of one SM's share of a tile

struct FwShared {
    uint64_t full[kFwStages], empty[kFwStages];
    uint64_t t_full[kFwBufs], t_empty[kFwBufs];
    uint64_t f_full[kFwFactors], f_empty[kFwFactors];
    uint64_t done;
    uint32_t tmem;
    int dead;
    alignas(16) float factor[kFwFactors][4][2][128];
    alignas(16) unsigned char out[16][32 * kFwOutRow];  // a warp's outputs on their way
};
constexpr size_t kFwSmem = 1024 + (size_t)kFwStages * kFwStageBytes + sizeof(FwShared);
static_assert(kFwSmem <= 227 * 1024, "shared memory");

__device__ __forceinline__ uint32_t fw_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The address of the first CTA's copy of a shared variable.
__device__ __forceinline__ uint32_t fw_lead(const void *p) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}
__device__ __forceinline__ void fw_pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Both CTAs' copies count on the first one's barrier.
__device__ __forceinline__ void fw_box(uint32_t one, uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(one)
        : "memory");
}
__device__ __forceinline__ void fw_mma(uint32_t one, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "setp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
// Arrive on both CTAs' barriers when the products issued so far are done.
__device__ __forceinline__ void fw_commit(uint32_t one, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            smem_u32(bar)),
        "h"((unsigned short)3), "r"(one)
        : "memory");
}
// Arrive on a barrier of either CTA: a TMEM buffer is read out.  (Release at CTA
// scope: what it orders are TMEM loads alone, complete and fenced by tcgen05.fence.
// At cluster scope each arrival cost a memory barrier: 1.62 ms for 8,192 rows by
// 28,672 x 4,096.)
__device__ __forceinline__ void fw_arrive(uint32_t one, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "@q mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(one)
        : "memory");
}

// Row and feature tile: kFwGroup row tiles for each feature tile, so that what
// runs at one time shares both operands in L2.
__device__ __forceinline__ void fw_tile(const F8Args &p, int tile, int &rt, int &ft) {
    const int per = kFwGroup * p.m_tiles, g = tile / per, nn = min(kFwGroup, p.n_tiles - g * kFwGroup);
    ft = (tile - g * per) / nn;
    rt = g * kFwGroup + (tile - g * per) % nn;
}

// A warp's 32 rows (lane r row row0 + r) by 64 outputs, through shared memory.
// Rows that start on 16 bytes (Dense): four lanes store 64 neighbouring bytes of a
// row, where a thread's own row at a time took a quarter of the kernel (a line a
// lane).  Others: a value a lane, side by side (128 rows by 300 x 128: 8 us, where 16
// bytes of a row a lane took 19).  Kernels of their own: one with both had registers
// spilled, and 8,192 rows by 28,672 x 4,096 took 686 us against 677.
template <bool Dense>
__device__ __forceinline__ void fw_store_tile(const F8Args &p, unsigned char *out, int row0, int f0, const float (&acc)[64]) {
    const int lane = threadIdx.x & 31, es = p.y_dtype == DS_BF16 ? 2 : 4, per = 64 / es;
    char *y = static_cast<char *>(p.y);
#pragma unroll
    for (int i = 0; i < 64; i += 16) {  // 16 values: 64 bytes of fp32, half of that of bf16
        uint4 *to = reinterpret_cast<uint4 *>(out + lane * kFwOutRow);
        if (es == 2) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float *v = acc + i + 8 * j;
                to[(i >> 3 & 2) + j] = make_uint4(stream_bf16x2(v[0], v[1]), stream_bf16x2(v[2], v[3]), stream_bf16x2(v[4], v[5]), stream_bf16x2(v[6], v[7]));
            }
            if ((i & 16) == 0) continue;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float *v = acc + i + 4 * j;
                to[j] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            }
        }
        __syncwarp();
        const int c0 = f0 + i / per * per;  // first column of these 64 bytes
        if (Dense) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = j * 32 + lane, row = row0 + (at >> 2), col = c0 + (at & 3) * (16 / es);
                if (row >= p.n || col >= p.rows) continue;
                const unsigned char *v = out + (at >> 2) * kFwOutRow + (at & 3) * 16;
                char *q = y + (row * p.ldy + col) * es;
                if (col + 16 / es <= p.rows) {
                    *reinterpret_cast<uint4 *>(q) = *reinterpret_cast<const uint4 *>(v);
                } else {
#pragma unroll 1
                    for (int k = 0; k < (p.rows - col) * es; k += 2) *reinterpret_cast<unsigned short *>(q + k) = *reinterpret_cast<const unsigned short *>(v + k);
                }
            }
        } else {
            const int col = lane & (per - 1);
#pragma unroll 4
            for (int r = lane / per; r < 32; r += 32 / per) {
                if (row0 + r >= p.n || c0 + col >= p.rows) continue;
                const unsigned char *v = out + r * kFwOutRow + col * es;
                char *q = y + ((row0 + r) * p.ldy + c0 + col) * es;
                if (es == 4) *reinterpret_cast<uint32_t *>(q) = *reinterpret_cast<const uint32_t *>(v);
                else *reinterpret_cast<unsigned short *>(q) = *reinterpret_cast<const unsigned short *>(v);
            }
        }
        __syncwarp();
    }
}

template <bool Dense>
__global__ __cluster_dims__(2, 1, 1) __launch_bounds__(kFwThreads, 1) void fp8_gemm_wide_kernel(const __grid_constant__ F8Args p) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    FwShared &sh = *reinterpret_cast<FwShared *>(smem_raw + (base - smem_u32(smem_raw)) + kFwStages * kFwStageBytes);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (uniform, so that addresses of barriers are)
    const int rank = (int)fw_rank();
    volatile int *dead = &sh.dead;

    if (threadIdx.x == 0) {
        stream_prefetch_map(&p.tw);
        stream_prefetch_map(&p.tx);
        for (int i = 0; i < kFwStages; ++i) {
            mbar_init(&sh.full[i], 1);  // the first one's: the copies of both CTAs
            mbar_init(&sh.empty[i], 2);  // a commit of either half's products
        }
        for (int i = 0; i < kFwBufs; ++i) {
            mbar_init(&sh.t_full[i], 1);
            mbar_init(&sh.t_empty[i], 16);
        }
        for (int i = 0; i < kFwFactors; ++i) {
            mbar_init(&sh.f_full[i], 1);
            mbar_init(&sh.f_empty[i], 16);
        }
        mbar_init(&sh.done, 2);
        sh.dead = 0;
        fence_mbarrier_init();
    }
    if (warp == 19) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    fw_pair_sync();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    allow_dependent_launch();
    grid_dependency_wait();

    F8Walk walk(p, blockIdx.x >> 1, gridDim.x >> 1);
    F8Seg sg;
    int rt, ft;
    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFwRegsOther));
        if (warp == 16) {
            // copies: this CTA's rows of X and its half of the weights
            const uint32_t one = stream_elect();
            int s = 0;
            uint32_t ph = 1;
            long long issued = 0;
            while (walk.next(p, sg)) {
                fw_tile(p, sg.tile, rt, ft);
                for (int k = sg.k0; k < sg.k1; ++k) {
                    if (issued >= kFwStages) stream_wait(&sh.empty[s], ph, dead, p.err);
                    if (*dead) break;
                    if (one && rank == 0) mbar_arrive_expect_tx(&sh.full[s], 2 * kFwStageBytes);
                    const uint32_t dst = base + s * kFwStageBytes, bar = fw_lead(&sh.full[s]);
                    fw_box(one, dst, &p.tx, k * 128, rt * kF8WideRows + rank * 128, bar);
                    fw_box(one, dst + kFwHalf, &p.tw, k * 128, ft * kF8WideFeatures + rank * 128, bar);
                    ++issued;
                    if (++s == kFwStages) s = 0, ph ^= 1;
                }
                if (*dead) break;
            }
            // the copies still under way land before either CTA ends
            if (rank == 0)
                for (long long i = max(0ll, issued - kFwStages); i < issued; ++i)
                    mbar_wait(&sh.full[i % kFwStages], (uint32_t)(i / kFwStages) & 1, p.err);
        } else if (warp != 18) {
            // Products, from the first CTA: a warp for each half, 64 of either
            // CTA's 128 features.  (From one warp its four waits a step, some 100
            // cycles each however long done, took longer than the products.)
            const uint32_t one = stream_elect();
            const int h = warp == 17 ? 0 : 1;
            if (rank == 0) {
                constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(kF8WideRows >> 4) << 24);
                int s = 0;
                uint32_t ph = 0, n = 0;  // n: steps so far
                while (walk.next(p, sg)) {
                    for (int k = sg.k1 - sg.k0; k > 0; --k, ++n) {
                        const uint32_t b = n & 1;
                        stream_wait(&sh.t_empty[2 * b + h], (n >> 1 & 1) ^ 1, dead, p.err);
                        stream_wait(&sh.full[s], ph, dead, p.err);
                        tc_fence_after();
                        const uint64_t ad = smem_desc(base + s * kFwStageBytes, 16, 1024);
                        const uint64_t bd = smem_desc(base + s * kFwStageBytes + kFwHalf + h * 64 * 128, 16, 1024);
#pragma unroll
                        for (int i = 0; i < 4; ++i)  // 32 bytes of every row a product
                            fw_mma(one, tmem + b * 256 + h * 128, ad + 2 * i, bd + 2 * i, idesc, i > 0);
                        fw_commit(one, &sh.t_full[2 * b + h]);
                        fw_commit(one, &sh.empty[s]);
                        if (++s == kFwStages) s = 0, ph ^= 1;
                    }
                }
                fw_commit(one, &sh.done);
            }
            mbar_wait(&sh.done, 0, p.err);
        } else {
            // Factors: four steps' scales requested together, and four steps' factors
            // handed over together (a segment's last with the next one's first), by
            // barriers of this CTA alone: memory that one CTA writes and reads is
            // ordered within it.  (Plain loads: the launch in front may have written
            // any of the scales.)
            uint32_t n = 0;  // steps so far
            while (walk.next(p, sg)) {
                fw_tile(p, sg.tile, rt, ft);
                const int row = rt * kF8WideRows + rank * 128 + lane, blocks = (p.rows + 127) / 128;
                const float *xs = p.xs + (long long)row * p.kb;
                const float *w0 = p.ws + (long long)(2 * ft) * p.kb, *w1 = p.ws + (long long)min(2 * ft + 1, blocks - 1) * p.kb;
                for (int k = sg.k0; k < sg.k1; k += 4) {
                    float v[4][4], a[4], b[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool in = k + j < sg.k1;
                        a[j] = in ? w0[k + j] : 0.0f;
                        b[j] = in ? w1[k + j] : 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[j][i] = in && row + 32 * i < p.n ? xs[(long long)(32 * i) * p.kb + k + j] : 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (k + j >= sg.k1) break;
                        const uint32_t at = (n >> 2) % kFwFactors;
                        if ((n & 3) == 0) stream_wait(&sh.f_empty[at], (n / (4 * kFwFactors) & 1) ^ 1, dead, p.err);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            sh.factor[at][n & 3][0][32 * i + lane] = v[j][i] * a[j];
                            sh.factor[at][n & 3][1][32 * i + lane] = v[j][i] * b[j];
                        }
                        __syncwarp();
                        stream_arrive(lane == 0 && (n & 3) == 3, smem_u32(&sh.f_full[at]));
                        ++n;
                    }
                }
            }
            stream_arrive(lane == 0 && (n & 3) != 0, smem_u32(&sh.f_full[(n >> 2) % kFwFactors]));
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFwRegsSum));
        // sums: thread r of a warpgroup is row r; the warpgroup's 64 columns are
        // features f0 on, half `half` of CTA `sub`'s
        const int wg = warp >> 2, half = wg >> 1, sub = wg & 1, r = threadIdx.x & 127, f0 = sub * 128 + half * 64;
        const uint32_t from = tmem + ((uint32_t)(warp & 3) << 21) + half * 128 + sub * 64;
        const uint32_t full0 = smem_u32(&sh.t_full[half]), freed0 = fw_lead(&sh.t_empty[half]);
        const uint32_t factor0 = smem_u32(&sh.factor[0][0][sub][r]), f_full0 = smem_u32(&sh.f_full[0]), one = stream_elect();
        uint32_t n = 0;  // steps so far
        while (walk.next(p, sg)) {
            float acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
            for (int k = sg.k1 - sg.k0; k > 0; --k, ++n) {
                const uint32_t b = n & 1;
                if ((n & 3) == 0) stream_wait(f_full0 + (n >> 2) % kFwFactors * 8, n / (4 * kFwFactors) & 1, dead, p.err);
                float factor;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(factor) : "r"(factor0 + n % (4 * kFwFactors) * 1024));
                stream_wait(full0 + b * 16, n >> 1 & 1, dead, p.err);
                tc_fence_after();
                const uint64_t f = stream_pair(factor, factor);
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    float v[32];
                    stream_ld<32>(from + b * 256 + c, v);
                    if (c == 32) {  // the buffer is read out
                        tc_fence_before();
                        __syncwarp();
                        fw_arrive(one, freed0 + b * 16);
                        stream_arrive(one && (n & 3) == 3, f_full0 + ((n >> 2) % kFwFactors + kFwFactors) * 8);  // f_empty
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 2) stream_fma2(acc[c + i], acc[c + i + 1], v[i], v[i + 1], f);
                }
            }
            fw_tile(p, sg.tile, rt, ft);
            if (sg.split < 0) {
                fw_store_tile<Dense>(p, sh.out[warp], rt * kF8WideRows + rank * 128 + (warp & 3) * 32, ft * kF8WideFeatures + f0, acc);
            } else {
                float *mine = p.partials + (((size_t)walk.id + sg.split) * 2 + rank) * kFwPart + (size_t)f0 * 128 + r;
#pragma unroll
                for (int i = 0; i < 64; ++i) __stcg(mine + i * 128, acc[i]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    fw_pair_sync();  // neither CTA ends while the other's products or arrivals may reach it
    tc_fence_after();
    if (warp == 19) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// Adds a split tile's partials, 8 columns of one SM's rows a block; thread r is row r.
constexpr int kFwJoinCols = 8;
__global__ __launch_bounds__(128) void fp8_join_wide_kernel(const __grid_constant__ F8Args p, int pairs) {
    constexpr int C = kFwJoinCols, kChunks = kF8WideFeatures / C;
    allow_dependent_launch();
    grid_dependency_wait();
    const int chunk = blockIdx.x % kChunks, rank = blockIdx.x / kChunks % 2, split = blockIdx.x / (2 * kChunks);
    int first, last, rt, ft;
    f8_contributors(p, split, first, last);
    if (first == last) return;  // one pair had all of it
    fw_tile(p, p.rounds * pairs + split, rt, ft);
    const int row = rt * kF8WideRows + rank * 128 + threadIdx.x, f0 = ft * kF8WideFeatures + chunk * C;
    if (row - (int)threadIdx.x >= p.n || f0 >= p.rows) return;
    float acc[C];
    f8_join<C, 128>(p.partials + (((size_t)first + split) * 2 + rank) * kFwPart + (size_t)chunk * C * 128 + threadIdx.x, 2 * (size_t)kFwPart,
                    last - first + 1, acc);
    if (row >= p.n) return;
    char *to = static_cast<char *>(p.y) + (row * p.ldy + f0) * (p.y_dtype == DS_BF16 ? 2 : 4);
    if (f0 + C <= p.rows && ((uintptr_t)to & 31) == 0 && p.y_dtype == DS_F32) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < C; ++i) w[i] = __float_as_uint(acc[i]);
        stream_store32(to, w);
    } else if (f0 + C <= p.rows && ((uintptr_t)to & 15) == 0 && p.y_dtype == DS_BF16) {
        *reinterpret_cast<uint4 *>(to) = make_uint4(stream_bf16x2(acc[0], acc[1]), stream_bf16x2(acc[2], acc[3]), stream_bf16x2(acc[4], acc[5]), stream_bf16x2(acc[6], acc[7]));
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (f0 + i < p.rows) store_as(p.y, row * p.ldy + f0 + i, p.y_dtype, acc[i]);
    }
}

// ---------------------------------------------------------------- host
int f8_wide_pairs() { return std::max(1, sm_count() / 2); }
size_t f8_wide_partial_floats(int split, unsigned runs) { return f8_cut(split, runs) ? ((size_t)runs + split) * 2 * kFwPart : 0; }

template <bool Dense>
static cudaError_t f8_wide_kernel(const F8Args &a, int pairs, cudaStream_t stream) {
    static std::atomic<unsigned long long> ready{0};  // devices whose limit is raised, a bit each
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(fp8_gemm_wide_kernel<Dense>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFwSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    return launch_ex(fp8_gemm_wide_kernel<Dense>, dim3(2 * pairs), dim3(kFwThreads), kFwSmem, stream, true, a);
}
cudaError_t f8_wide_launch(const F8Args &a, int pairs, cudaStream_t stream) {
    const bool dense = (((uintptr_t)a.y | (uintptr_t)(a.ldy * (a.y_dtype == DS_BF16 ? 2 : 4))) & 15) == 0;
    const cudaError_t e = dense ? f8_wide_kernel<true>(a, pairs, stream) : f8_wide_kernel<false>(a, pairs, stream);
    if (e != cudaSuccess || !f8_cut(a.split, a.runs)) return e;
    return launch_ex(fp8_join_wide_kernel, dim3(a.split * 2 * (kF8WideFeatures / kFwJoinCols)), dim3(128), 0, stream, true, a, pairs);
}

}  // namespace ds
