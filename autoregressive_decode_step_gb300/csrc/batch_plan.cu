// Block tables, row starts, positions and cache slots of a ragged step, built
// on the GPU from the requests' lengths ("Inside the engine", section 2: a
// step runs prompt chunks and decode rows side by side; section 3: the K/V
// pool's blocks and a request's block table).
//
// With c_s cached and n_s new positions of sequence s and blocks of bt
// positions:
//   need_s = ceil((c_s + n_s) / bt) - ceil(c_s / bt)
//   row_starts[s] = sum of n_i over i < s;   taken_s = sum of need_i over i < s
//   block ceil(c_s / bt) + i of s is free_blocks[taken_s + i], i < need_s
//   row r of s: pos = c_s + r - row_starts[s], slot = block * bt + pos % bt
// Two prefix sums over the sequences, then one independent lookup per row.
//
// The work is a few kilobytes, so the launch and two dependent trips to
// memory bound it, not bytes.  Every block therefore scans all the lengths
// itself (8 bytes a sequence, from L2 after the first block) instead of a
// first launch scanning once for a second to read: one launch in place of
// two.  Both prefix sums stay in shared memory and a row finds its sequence
// there by bisection.  Measured: 3.5 us for 64 sequences of one row, 3.9 us for
// 250 sequences and 16,384 rows.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace ds {

constexpr int kPlThreads = 256;
constexpr int kPlMaxSeqs = 4096;     // both prefix sums in shared memory: 32 KB
constexpr int kPlRowsPerBlock = 256;  // rows a block maps

struct PlanArgs {
    const int *cached, *fresh;  // lengths before the step, new positions
    int n_seqs;
    const int *free_blocks;
    int n_free, bt;
    long long pool_blocks;  // whole blocks of the cache
    int *block_table;
    int max_blocks;
    int *row_starts, *seq_lens, *row_seq, *positions, *slots;
    int max_rows;
    int *n_taken;
    int *err;
};

__device__ __forceinline__ int pl_blocks(long long len, int bt) { return (int)((len + bt - 1) / bt); }

// Last index i in [0, n) with a[i] <= v (a[0] = 0 <= v, a nondecreasing); the
// run of equal entries ends in the sequence that holds v.
__device__ __forceinline__ int pl_find(const int *a, int n, int v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlThreads) paged_plan_kernel(const PlanArgs p) {
    extern __shared__ int sm[];
    int *rows = sm;                     // [n_seqs + 1] exclusive sums of the new rows
    int *taken = sm + p.n_seqs + 1;     // [n_seqs + 1] exclusive sums of the new blocks
    __shared__ long long w_rows[kPlThreads / 32], w_taken[kPlThreads / 32];
    __shared__ int s_cut;               // sequences served
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long cap = (long long)p.max_blocks * p.bt;
    int flags = 0;
    if (tid == 0) s_cut = p.n_seqs;
    __syncthreads();

    long long base_r = 0, base_t = 0;
    for (int s0 = 0; s0 < p.n_seqs; s0 += kPlThreads) {
        const int s = s0 + tid;
        long long nr = 0, nt = 0;
        bool bad = false;
        if (s < p.n_seqs) {
            const long long c = p.cached[s], n = p.fresh[s];
            bad = c < 0 || n < 0 || c + n > cap;
            if (!bad) {
                nr = n;
                nt = pl_blocks(c + n, p.bt) - pl_blocks(c, p.bt);
            } else {
                flags |= DS_ERR_POSITION;
            }
        }
        long long ir = nr, it = nt;  // inclusive sums over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long a = __shfl_up_sync(0xffffffffu, ir, o), b = __shfl_up_sync(0xffffffffu, it, o);
            if (lane >= o) {
                ir += a;
                it += b;
            }
        }
        if (lane == 31) {
            w_rows[warp] = ir;
            w_taken[warp] = it;
        }
        __syncthreads();
        long long br = base_r, bt_ = base_t;
#pragma unroll
        for (int w = 0; w < kPlThreads / 32; ++w) {
            if (w < warp) {
                br += w_rows[w];
                bt_ += w_taken[w];
            }
            base_r += w_rows[w];
            base_t += w_taken[w];
        }
        ir += br;
        it += bt_;
        if (s < p.n_seqs) {
            // the first sequence whose rows or blocks do not fit ends the step
            if (ir > p.max_rows || it > p.n_free) atomicMin(&s_cut, s);
            rows[s + 1] = (int)min(ir, (long long)p.max_rows);
            taken[s + 1] = (int)min(it, (long long)p.n_free);
        }
        __syncthreads();
    }
    if (tid == 0) rows[0] = taken[0] = 0;
    const int cut = s_cut;
    __syncthreads();
    if (cut < p.n_seqs) {
        flags |= DS_ERR_NO_BLOCKS;
        const int r = rows[cut], t = taken[cut];
        __syncthreads();
        for (int s = cut + tid; s < p.n_seqs; s += kPlThreads) {
            rows[s + 1] = r;
            taken[s + 1] = t;
        }
        __syncthreads();
    }
    const int total = rows[p.n_seqs], n_taken = taken[p.n_seqs];
    const int gtid = blockIdx.x * kPlThreads + tid, gn = gridDim.x * kPlThreads;

    // per sequence
    for (int s = gtid; s <= p.n_seqs; s += gn) {
        p.row_starts[s] = rows[s];
        if (s < p.n_seqs) {
            const long long c = p.cached[s];
            p.seq_lens[s] = (int)min(max(c, 0ll), cap) + rows[s + 1] - rows[s];
        } else {
            *p.n_taken = n_taken;
        }
    }
    // per new block: the table entry
    for (int i = gtid; i < n_taken; i += gn) {
        const int s = pl_find(taken, p.n_seqs, i);
        int id = p.free_blocks[i];
        if (id < 0 || id >= p.pool_blocks) {
            flags |= DS_ERR_POSITION;
            id = -1;
        }
        p.block_table[(long long)s * p.max_blocks + pl_blocks(p.cached[s], p.bt) + i - taken[s]] = id;
    }
    // per row; a new block's number comes from the free list, so no row reads
    // a table entry that this launch writes
    for (int r = gtid; r < p.max_rows; r += gn) {
        int s = -1, pos = -1, slot = -1;
        if (r < total) {
            s = pl_find(rows, p.n_seqs, r);
            const int c = p.cached[s];
            pos = c + r - rows[s];
            const int b = pos / p.bt, had = pl_blocks(c, p.bt);
            const int id = b >= had ? p.free_blocks[taken[s] + b - had] : p.block_table[(long long)s * p.max_blocks + b];
            if (id < 0 || id >= p.pool_blocks)
                flags |= DS_ERR_POSITION;
            else
                slot = id * p.bt + pos % p.bt;
        }
        p.row_seq[r] = s;
        p.positions[r] = pos;
        p.slots[r] = slot;
    }
    if (flags) flag_error(p.err, flags);
}

}  // namespace ds

using namespace ds;

extern "C" DS_API size_t ds_paged_plan_workspace_bytes(void) { return kWsHeader; }

extern "C" DS_API int ds_paged_plan(const int32_t *cached_lens, const int32_t *new_lens, int n_seqs,
                                    const int32_t *free_blocks, int64_t n_free, int block_tokens, int64_t cache_rows,
                                    int32_t *block_table, int max_blocks_per_seq, int32_t *row_starts,
                                    int32_t *seq_lens, int32_t *row_seq, int32_t *positions, int32_t *slots,
                                    int64_t max_rows, int32_t *n_taken, void *workspace, size_t workspace_bytes,
                                    ds_stream_t stream) {
    if (n_seqs < 1 || n_free < 0 || block_tokens < 1 || cache_rows < 1 || max_blocks_per_seq < 1 || max_rows < 1)
        return DS_EMPTY_DIMENSION;
    if (n_seqs > kPlMaxSeqs || n_free > DS_MAX_DIM || cache_rows > DS_MAX_DIM || max_rows > DS_MAX_DIM ||
        (int64_t)max_blocks_per_seq * block_tokens > DS_MAX_DIM)
        return DS_DIMENSION_TOO_LARGE;
    if (!cached_lens || !new_lens || (n_free > 0 && !free_blocks) || !block_table || !row_starts || !seq_lens ||
        !row_seq || !positions || !slots || !n_taken)
        return DS_BAD_ARGUMENT;
    if (!workspace || workspace_bytes < kWsHeader) return DS_WORKSPACE_TOO_SMALL;
    if ((uintptr_t)workspace & 255) return DS_BAD_ARGUMENT;
    // Blocks read all the lengths while others write theirs: every output
    // (the last seven) stands apart from the inputs and the other outputs.
    const struct {
        const int32_t *p;
        int64_t n;
    } span[] = {{cached_lens, n_seqs}, {new_lens, n_seqs}, {free_blocks, n_free},
                {block_table, (int64_t)n_seqs * max_blocks_per_seq}, {row_starts, n_seqs + 1}, {seq_lens, n_seqs},
                {row_seq, max_rows}, {positions, max_rows}, {slots, max_rows}, {n_taken, 1}};
    for (int i = 3; i < 10; ++i)
        for (int j = 0; j < i; ++j)
            if ((uintptr_t)span[i].p < (uintptr_t)(span[j].p + span[j].n) &&
                (uintptr_t)span[j].p < (uintptr_t)(span[i].p + span[i].n))
                return DS_BAD_ARGUMENT;
    PlanArgs a = {};
    a.cached = cached_lens;
    a.fresh = new_lens;
    a.n_seqs = n_seqs;
    a.free_blocks = free_blocks;
    a.n_free = (int)n_free;
    a.bt = block_tokens;
    a.pool_blocks = cache_rows / block_tokens;
    a.block_table = block_table;
    a.max_blocks = max_blocks_per_seq;
    a.row_starts = row_starts;
    a.seq_lens = seq_lens;
    a.row_seq = row_seq;
    a.positions = positions;
    a.slots = slots;
    a.max_rows = (int)max_rows;
    a.n_taken = n_taken;
    a.err = static_cast<int *>(workspace);
    const int grid = (int)std::min<int64_t>((max_rows + kPlRowsPerBlock - 1) / kPlRowsPerBlock, 2LL * sm_count());
    const size_t smem = 2 * (size_t)(n_seqs + 1) * sizeof(int);
    const cudaError_t e = launch_ex(paged_plan_kernel, dim3(grid), dim3(kPlThreads), smem,
                                    reinterpret_cast<cudaStream_t>(stream), false, a);
    return e == cudaSuccess ? DS_OK : DS_CUDA_ERROR;
}
