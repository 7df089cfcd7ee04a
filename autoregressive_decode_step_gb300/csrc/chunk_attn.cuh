// Work split of the chunk attention (attention of every request's new rows
// over its blocks of the paged K/V pool), shared by its two kernels.
//
// A tile is up to `tile_tokens` consecutive new rows of one sequence times the
// query heads that share one KV head (a group of more than `sub_heads` heads
// is cut into equal parts, each with tiles of its own).  Its cost is the
// number of positions its last row attends, times a weight, and a constant
// for its beginning and end.  The costs of all tiles, ordered by sequence,
// head and row, form one line that is cut into equal ranges, one per CTA, so
// the load is even whatever the mix of chunks and single tokens.  A cut inside
// a tile is rounded down to a whole K/V step of `step` positions, or to the
// tile's beginning or end where it would leave a piece of fewer than `piece`
// positions (an eighth of a CTA's range, within bounds): a record is not worth
// that.  Each contributor leaves its (max, sum, accumulator) record in the
// workspace and a second launch joins them in CTA order, so results do not
// depend on timing.  (The last contributor to arrive joining them inside the
// first launch was measured and dropped: one CTA reading up to 128 pairs'
// records took 15 to 28 us at the end of the launch when the others had left;
// in the second every SM reads a few.)
//
// Costs have a closed form (a sum over a sequence's tiles is a quadratic in
// their number), so no plan is kept in memory: a CTA finds its range by one
// scan over the sequences' lengths and walks on from there.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace ds {

constexpr int kChunkMaxTileRows = 256;  // (row, head) pairs of the largest tile

struct ChunkArgs {
    const void *q;          // [n_rows][n_qh * hd]
    void *out;              // same
    const void *k_cache, *v_cache;  // [cache_rows][n_kvh * hd]
    int q_dtype, kv_dtype;
    int n_rows;
    const int *row_starts;  // [n_seqs + 1]
    const int *seq_lens;    // [n_seqs]
    int n_seqs;
    long long cache_rows;
    const int *block_table;  // [n_seqs][max_blocks] or nullptr (contiguous slots)
    int max_blocks, bt;
    long long pool_blocks;   // whole blocks of the cache
    int n_qh, n_kvh, hd, gq;
    float scale;
    int head_parts;   // tiles' heads: each KV head's gq query heads in so many parts
    int part_heads;   // query heads of a part (the last may have fewer)
    int tile_tokens;  // rows of a sequence per tile
    int step;         // positions of one K/V step
    int half_tokens;  // tiles of at most so many rows weigh w_half a position, others w_full
    int w_half, w_full;
    int tile_cost;    // what beginning and ending a tile costs
    int piece;        // most positions a piece may need to be worth a record, at least one step
    int rec_rows;     // rows of a partial record
    struct ChunkJoin *joins;  // [grid]: the split tile whose first contributor the CTA is
    float *partials;  // [grid][2] records of rec_rows * (hd + 2) floats (max, sum, then the accumulators)
    int *err;
};

// A split tile, for the joining launch.  pairs 0: the CTA has none.
struct ChunkJoin {
    int pairs;       // rows x part_heads
    int r0, part;    // first row; head part
    int first, last; // contributing CTAs
    int first_slot;  // record of the first of them (the others': 0)
};

int chunk_simt_grid();  // the largest grid of any of the kernels
// The first launch; *grid gets its CTA count and `a` the tile shape that the
// joining launch needs too.
cudaError_t launch_chunk_simt(ChunkArgs &a, int *grid, cudaStream_t stream);
bool chunk_tc_supported(const ChunkArgs &a);
cudaError_t launch_chunk_tc(ChunkArgs &a, int *grid, cudaStream_t stream);
// Set head_parts, part_heads and tile_tokens for tiles of `subs` parts of
// sub_rows (row, head) pairs, each part holding whole rows.
void chunk_tile_shape(ChunkArgs &a, int sub_rows, int subs);

// One sequence of the batch as the walk sees it: its rows that attend
// something, n of them from row r0 on, behind ctx earlier positions.
struct ChunkSeq {
    int s, r0, n, ctx;
    int tiles;
    int w_last;      // weight of the last tile's positions (the others': w_full)
    long long cost;  // of one head part
};

// flags: DS_ERR_POSITION for lengths outside the buffers (clamped).
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkArgs &a, int s, int &flags) {
    const int b = __ldg(a.row_starts + s), e = __ldg(a.row_starts + s + 1);
    const int len = __ldg(a.seq_lens + s);
    const int cap = a.max_blocks * a.bt;
    ChunkSeq q;
    q.s = s;
    q.r0 = min(max(b, 0), a.n_rows);
    const int r1 = min(max(e, q.r0), a.n_rows);
    const int L = min(max(len, 0), cap);
    if (q.r0 != b || r1 != e || L != len) flags |= DS_ERR_POSITION;
    // rows before the first position attend nothing: they are no part of a tile
    const int empty = max(0, r1 - q.r0 - L);
    q.r0 += empty;
    q.n = r1 - q.r0;
    q.ctx = L - q.n;
    q.tiles = (q.n + a.tile_tokens - 1) / a.tile_tokens;
    const long long T = q.tiles;
    q.w_last = q.n - (q.tiles - 1) * a.tile_tokens <= a.half_tokens ? a.w_half : a.w_full;
    q.cost = T ? a.w_full * ((T - 1) * q.ctx + (long long)a.tile_tokens * (T * (T - 1) / 2)) +
                     (long long)q.w_last * (q.ctx + q.n) + T * a.tile_cost
               : 0;
    return q;
}

// Cost of a sequence's tiles before tile t < tiles.
__device__ __forceinline__ long long chunk_cost_before(const ChunkArgs &a, const ChunkSeq &q, long long t) {
    return a.w_full * (t * q.ctx + (long long)a.tile_tokens * (t * (t + 1) / 2)) + t * a.tile_cost;
}

// One piece of work: a tile's K/V steps [b0, b1).
struct ChunkSeg {
    int r0;          // first row of the tile in the batch
    int tokens;      // rows
    int pos0;        // position of the first row: row j attends positions 0 .. pos0 + j
    int len;         // positions the tile attends
    int seq, part;   // sequence; head part (kv head * head_parts + part)
    int b0, b1;      // K/V steps of this CTA
    int slot;        // partial record of this CTA (0 / 1) if others contribute
    int split;       // they do
    int weight;      // of its positions
    long long start, cost;  // place of the tile on the line of costs
};

// The K/V step that a cut at x behind the tile's start falls to.  (The
// constant comes first: a cut inside it is one at position 0.)
__device__ __forceinline__ int chunk_cut(const ChunkArgs &a, const ChunkSeg &g, int piece, long long x) {
    const int pos = (int)max(0ll, x - a.tile_cost) / g.weight;
    if (pos < piece) return 0;
    if (g.len - pos < piece) return (g.len + a.step - 1) / a.step;
    return pos / a.step;
}

// The walk of one CTA over its range.  init() is called by every thread of
// the block (it synchronises the block); then each role walks its own copy.
struct ChunkWalk {
    long long u, u1, unit;  // place, end of the range, range of one CTA
    long long seq_start;    // of the current sequence
    ChunkSeq q;
    int part, tile;
    int piece;
    int flags;

    // s_red: 34 long longs of shared memory.  WHOLE: short ranges are whole
    // steps (for weights of 1 and no tile_cost).
    template <bool WHOLE>
    __device__ void init(const ChunkArgs &a, long long *s_red) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
        const int parts = a.n_kvh * a.head_parts;
        flags = 0;
        long long mine = 0;
        for (int s = tid; s < a.n_seqs; s += blockDim.x) mine += chunk_seq(a, s, flags).cost;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        if (lane == 0) s_red[warp] = mine;
        __syncthreads();
        long long total = 0;
        for (int w = 0; w < nw; ++w) total += s_red[w];
        total *= parts;
        unit = (total + gridDim.x - 1) / gridDim.x;
        piece = (int)min((long long)a.piece, max((long long)a.step, unit / (8 * a.w_full)));
        unit = max(unit, (long long)a.step * a.w_full);  // no two cuts inside one step
        // A range of a few steps is a whole number of them: otherwise the
        // rounding of the cuts gives some CTAs a step more than others (plain
        // cores, 512 fp32 rows of 16 heads: 67 -> 63 us; longer ranges the same).
        if (WHOLE && unit < 4 * a.step) unit = (unit + a.step - 1) / a.step * a.step;
        u = min((long long)blockIdx.x * unit, total);
        u1 = min(u + unit, total);
        // the sequence that holds u
        if (tid == 0) s_red[32] = -1;
        long long base = 0;
        for (int s0 = 0; s0 < a.n_seqs && u < u1; s0 += blockDim.x) {
            const int s = s0 + tid;
            int dummy = 0;
            const long long c = s < a.n_seqs ? chunk_seq(a, s, dummy).cost * parts : 0;
            long long inc = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            __syncthreads();
            if (lane == 31) s_red[warp] = inc;
            __syncthreads();
            long long before = base;
            for (int w = 0; w < nw; ++w) {
                if (w < warp) before += s_red[w];
                base += s_red[w];
            }
            inc += before;
            if (u < inc && u >= inc - c) {
                s_red[32] = s;
                s_red[33] = inc - c;
            }
            if (base > u) break;  // the same for all threads
        }
        __syncthreads();
        part = tile = 0;
        q.s = -1;
        q.tiles = 0;
        if (u < u1) {
            int dummy = 0;
            q = chunk_seq(a, (int)s_red[32], dummy);
            seq_start = s_red[33];
            long long rem = u - seq_start;
            part = (int)(rem / q.cost);
            rem -= (long long)part * q.cost;
            int lo = 0, hi = q.tiles;  // last tile with cost before it <= rem
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (chunk_cost_before(a, q, mid) <= rem)
                    lo = mid;
                else
                    hi = mid;
            }
            tile = lo;
        }
        __syncthreads();
    }

    // The next piece of work, or false at the range's end.
    __device__ bool next(const ChunkArgs &a, ChunkSeg &g) {
        const int parts = a.n_kvh * a.head_parts;
        while (u < u1) {
            if (tile == q.tiles) {
                tile = 0;
                if (++part == parts) {
                    part = 0;
                    seq_start += q.cost * parts;
                    int dummy = 0;
                    do {
                        q = chunk_seq(a, q.s + 1, dummy);
                    } while (q.tiles == 0);
                }
            }
            const int j0 = tile * a.tile_tokens;
            g.tokens = min(a.tile_tokens, q.n - j0);
            g.r0 = q.r0 + j0;
            g.pos0 = q.ctx + j0;
            g.len = q.ctx + j0 + g.tokens;
            g.seq = q.s;
            g.part = part;
            g.weight = tile == q.tiles - 1 ? q.w_last : a.w_full;
            g.cost = (long long)g.weight * g.len + a.tile_cost;
            g.start = seq_start + (long long)part * q.cost + chunk_cost_before(a, q, tile);
            const long long end = min(u1, g.start + g.cost);
            g.b0 = u == g.start ? 0 : chunk_cut(a, g, piece, u - g.start);
            g.b1 = end == g.start + g.cost ? (g.len + a.step - 1) / a.step : chunk_cut(a, g, piece, end - g.start);
            const long long u0 = (long long)blockIdx.x * unit;
            g.slot = g.start < u0 ? 0 : 1;
            ++tile;
            u = end;
            if (g.b0 >= g.b1) continue;
            g.split = g.b0 > 0 || g.b1 < (g.len + a.step - 1) / a.step;
            return true;
        }
        return false;
    }

    // The joining launch's word of a split tile whose first contributor this
    // CTA is.  CTAs that the rounding of the cuts left nothing of it do not
    // count; those in between have a step at least.
    __device__ ChunkJoin join(const ChunkArgs &a, const ChunkSeg &g) const {
        ChunkJoin j;
        j.pairs = g.tokens * a.part_heads;
        j.r0 = g.r0;
        j.part = g.part;
        j.first = blockIdx.x;
        j.first_slot = g.slot;
        j.last = (int)((g.start + g.cost - 1) / unit);
        while (chunk_cut(a, g, piece, j.last * unit - g.start) == (g.len + a.step - 1) / a.step) --j.last;
        return j;
    }
};

// A sequence's block number as the table has it, and the block's first cache
// row; a number outside the pool reads block 0 and flags.  (Two calls, so that
// a caller can fetch ahead.)
__device__ __forceinline__ int chunk_block_id(const ChunkArgs &a, int seq, int blk) {
    return a.block_table ? __ldg(a.block_table + (long long)seq * a.max_blocks + blk) : seq * a.max_blocks + blk;
}
__device__ __forceinline__ long long chunk_id_row(const ChunkArgs &a, int id, int &flags) {
    if (id < 0 || id >= a.pool_blocks) {
        flags |= DS_ERR_POSITION;
        id = 0;
    }
    return (long long)id * a.bt;
}
__device__ __forceinline__ long long chunk_block_row(const ChunkArgs &a, int seq, int blk, int &flags) {
    return chunk_id_row(a, chunk_block_id(a, seq, blk), flags);
}

// Query heads of a head part: count heads from `first` on, of KV head kv.
struct ChunkHeads {
    int kv, first, count;
};
__device__ __forceinline__ ChunkHeads chunk_heads(const ChunkArgs &a, int part) {
    ChunkHeads h;
    h.kv = part / a.head_parts;
    const int skip = (part % a.head_parts) * a.part_heads;
    h.first = h.kv * a.gq + skip;
    h.count = min(a.part_heads, a.gq - skip);
    return h;
}

// Partial record of CTA c: (max in units of log2, sum) per (row, head) pair,
// then rec_rows x hd accumulators.
__device__ __forceinline__ float *chunk_record(const ChunkArgs &a, int c, int slot) {
    return a.partials + ((size_t)c * 2 + slot) * a.rec_rows * (a.hd + 2);
}

// Rows in front of a sequence's first position (a length below the number of
// new rows) attend nothing: their output is zero.
__device__ inline void chunk_zero_empty_rows(const ChunkArgs &a) {
    for (int s = blockIdx.x; s < a.n_seqs; s += gridDim.x) {
        const int r0 = min(max(__ldg(a.row_starts + s), 0), a.n_rows);
        const int r1 = min(max(__ldg(a.row_starts + s + 1), r0), a.n_rows);
        const int L = min(max(__ldg(a.seq_lens + s), 0), a.max_blocks * a.bt);
        if (r1 - r0 <= L) continue;
        const long long w = (long long)a.n_qh * a.hd;
        for (long long i = r0 * w + threadIdx.x; i < (r1 - L) * w; i += blockDim.x) store_as(a.out, i, a.q_dtype, 0.0f);
    }
}

// a * b + c and a + b, two numbers at a time.
__device__ __forceinline__ float2 chunk_fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 chunk_add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

}  // namespace ds
