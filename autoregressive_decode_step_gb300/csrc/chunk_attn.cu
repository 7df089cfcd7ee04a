// Attention of every request's new rows over its blocks of the paged K/V pool
// ("Inside the engine", section 1: prefill runs a chunk of prompt tokens as a
// batch of rows, causal flash attention over the chunk; section 2: chunks and
// decode rows side by side in one step): the entry point, and the plain-core
// kernel for the shapes and types that the tensor-core kernel does not take.
//
// Row j of a sequence's n new rows, L positions long with them, attends
// positions t <= L - n + j:
//   s_t = scale * q . k_t,  m = max s_t,  out = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m)
// in one pass over the positions with a running maximum and sum.
//
// chunk_simt_kernel keeps everything in fp32 (an fp32 cache has more digits
// than a bf16 product keeps): 16 RT (row, head) pairs by 64 positions a step,
// 256 threads of RT x 4 scores and RT x hd/16 outputs in registers, Q, K and V
// in shared memory; work split as in chunk_attn.cuh.  Two sizes of tile:
//  - RT 4, 64 pairs.  Bound by the fp32 FMA and the reads of shared memory:
//    2,048 fp32 rows of 32 heads of 128 take 1,022 us, 34 TFLOP/s.  (Eight
//    rows a thread, half the warps with fewer reads each: 1,190 against 1,074
//    us then.)
//  - RT 1, 16 pairs, for batches with 16 pairs a sequence or fewer on average
//    (single tokens): 64 fp32 tokens over 1,024 to 4,096 positions 370 us
//    against 640 with RT 4, one over 1,024 16.0 against 21.5, three rows each
//    630 against 739.  A step's fetch and work in turns bound it: 3.6 TB/s.
// Warps whose pairs are all behind the tile's last skip a step's work (without
// that and with loads waited for one by one the 64 tokens took 1,210 us).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "chunk_attn.cuh"

namespace ds {

constexpr int kCsThreads = 256;
constexpr int kCsStep = 64;
constexpr int kCsPiece = 128;
constexpr float kLog2e = 1.4426950408889634f;

// Four consecutive elements (the row starts on 4 elements) as fp32.
__device__ __forceinline__ float4 cs_load4(const float *base, long long i) {
    return __ldg(reinterpret_cast<const float4 *>(base + i));
}
__device__ __forceinline__ float4 cs_load4(const __nv_bfloat16 *base, long long i) {
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(base + i));
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float4 cs_load4(const void *base, long long i, int dtype) {
    return dtype == DS_F32 ? cs_load4(static_cast<const float *>(base), i)
                           : cs_load4(static_cast<const __nv_bfloat16 *>(base), i);
}

template <int HD, int RT>
__global__ void __launch_bounds__(kCsThreads, HD <= 128 ? 2 : 1) chunk_simt_kernel(const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int rows = 16 * RT;  // (row, head) pairs of a tile
    constexpr int kFetch = RT == 1 && HD >= 128 ? 8 : 4;
    static_assert(kCsStep * (HD / 4) % (kFetch * kCsThreads) == 0, "");
    constexpr int KS = HD + 4;  // K rows padded: sixteen rows read at once fall into different banks
    constexpr int PS = kCsStep + 4;
    static_assert(PS <= KS || HD < 64, "");
    float *sQ = sm, *sK = sQ + rows * HD, *sV = sK + kCsStep * KS;
    float *sP = sK;  // the weights take K's place once the scores are formed
    __shared__ long long s_red[34];
    __shared__ int s_row[2][kCsStep];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    int flags = 0;

    chunk_zero_empty_rows(a);
    ChunkWalk walk;
    walk.init<true>(a, s_red);
    allow_dependent_launch();
    flags |= walk.flags;
    if (tid == 0) a.joins[blockIdx.x].pairs = 0;
    ChunkSeg g;
    while (walk.next(a, g)) {
        const ChunkHeads hh = chunk_heads(a, g.part);
        for (int i = tid; i < rows * (HD / 4); i += kCsThreads) {
            const int m = i / (HD / 4), d = (i % (HD / 4)) * 4;
            const int tok = m / a.part_heads, h = m % a.part_heads;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (tok < g.tokens && h < hh.count && d < a.hd)
                v = cs_load4(a.q, ((long long)(g.r0 + tok) * a.n_qh + hh.first + h) * a.hd + d, a.q_dtype);
            *reinterpret_cast<float4 *>(sQ + m * HD + d) = v;
        }
        float2 acc[RT][HD / 32];
        float mx[RT], sum[RT];
        int lim[RT];  // last position of each row
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            mx[i] = -INFINITY;
            sum[i] = 0.0f;
            lim[i] = g.pos0 + (ty * RT + i) / a.part_heads;
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) acc[i][c] = make_float2(0.0f, 0.0f);
        }
        // a step's cache rows, worked out by 64 threads while the step before runs
        auto find_rows = [&](int b) {
            const int pos = b * kCsStep + tid;
            if (tid < kCsStep && pos < g.len)
                s_row[b & 1][tid] = (int)(chunk_block_row(a, g.seq, pos / a.bt, flags) + pos % a.bt);
        };
        // a step's K and V, several rows' loads on their way at a time
        auto fetch = [&](const auto *k_cache, const auto *v_cache, int b, int nt) {
            for (int i0 = tid; i0 < kCsStep * (HD / 4); i0 += kFetch * kCsThreads) {
                float4 k[kFetch], v[kFetch];
#pragma unroll
                for (int u = 0; u < kFetch; ++u) {
                    const int i = i0 + u * kCsThreads, t = i / (HD / 4), d = (i % (HD / 4)) * 4;
                    k[u] = v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (t < nt && d < a.hd) {
                        const long long e = ((long long)s_row[b & 1][t] * a.n_kvh + hh.kv) * a.hd + d;
                        k[u] = cs_load4(k_cache, e);
                        v[u] = cs_load4(v_cache, e);
                    }
                }
#pragma unroll
                for (int u = 0; u < kFetch; ++u) {
                    const int i = i0 + u * kCsThreads, t = i / (HD / 4), d = (i % (HD / 4)) * 4;
                    *reinterpret_cast<float4 *>(sK + t * KS + d) = k[u];
                    *reinterpret_cast<float4 *>(sV + t * HD + d) = v[u];
                }
            }
        };
        // a warp whose rows are all behind the tile's last has nothing to work out
        const bool busy = (ty & ~1) * RT < g.tokens * a.part_heads;
        find_rows(g.b0);
        for (int b = g.b0; b < g.b1; ++b) {
            const int t0 = b * kCsStep, nt = min(kCsStep, g.len - t0);
            __syncthreads();  // the last step's weights and values are read, this one's rows found
            if (b + 1 < g.b1) find_rows(b + 1);
            if (a.kv_dtype == DS_F32)
                fetch(static_cast<const float *>(a.k_cache), static_cast<const float *>(a.v_cache), b, nt);
            else
                fetch(static_cast<const __nv_bfloat16 *>(a.k_cache), static_cast<const __nv_bfloat16 *>(a.v_cache), b, nt);
            __syncthreads();
            float2 s2[RT][4] = {};  // sums over even and odd dims
#pragma unroll 4
            for (int d = 0; d < (busy ? HD : 0); d += 4) {
                float4 qv[RT], kv[4];
#pragma unroll
                for (int i = 0; i < RT; ++i) qv[i] = *reinterpret_cast<const float4 *>(sQ + (ty * RT + i) * HD + d);
#pragma unroll
                for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4 *>(sK + (tx + 16 * j) * KS + d);
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s2[i][j] = chunk_fma2(make_float2(qv[i].x, qv[i].y), make_float2(kv[j].x, kv[j].y), s2[i][j]);
                        s2[i][j] = chunk_fma2(make_float2(qv[i].z, qv[i].w), make_float2(kv[j].z, kv[j].w), s2[i][j]);
                    }
            }
            float s[RT][4];
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j].x + s2[i][j].y;
            __syncthreads();  // K is read
            if (!busy) continue;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // a masked score is replaced, not added to: K may hold anything there
                    s[i][j] = t0 + tx + 16 * j <= lim[i] ? s[i][j] * (a.scale * kLog2e) : -INFINITY;
                    top = fmaxf(top, s[i][j]);
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float m_new = fmaxf(mx[i], top);
                const float m_use = m_new == -INFINITY ? 0.0f : m_new;
                const float keep = exp2f(mx[i] - m_use);
                float add = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = exp2f(s[i][j] - m_use);
                    sP[(ty * RT + i) * PS + tx + 16 * j] = p;
                    add += p;
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
                sum[i] = sum[i] * keep + add;
                mx[i] = m_new;
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    acc[i][c].x *= keep;
                    acc[i][c].y *= keep;
                }
            }
            __syncwarp();  // a warp reads the weights of its own rows only
            auto add_values = [&](auto masked) {
                for (int t = 0; t < nt; t += 4) {
                    float4 p4[RT];
#pragma unroll
                    for (int i = 0; i < RT; ++i) p4[i] = *reinterpret_cast<const float4 *>(sP + (ty * RT + i) * PS + t);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
#pragma unroll
                        for (int c = 0; c < HD / 64; ++c) {
                            const float4 v = *reinterpret_cast<const float4 *>(sV + (t + k) * HD + 64 * c + tx * 4);
#pragma unroll
                            for (int i = 0; i < RT; ++i) {
                                // a row skips what it does not attend: 0 x an infinity there would be NaN
                                if (masked.value && t0 + t + k > lim[i]) continue;
                                const float p = k == 0 ? p4[i].x : k == 1 ? p4[i].y : k == 2 ? p4[i].z : p4[i].w;
                                const float2 p2 = make_float2(p, p);
                                acc[i][2 * c] = chunk_fma2(p2, make_float2(v.x, v.y), acc[i][2 * c]);
                                acc[i][2 * c + 1] = chunk_fma2(p2, make_float2(v.z, v.w), acc[i][2 * c + 1]);
                            }
                        }
                    }
                }
            };
            if (t0 + kCsStep - 1 > g.pos0)
                add_values(std::true_type{});
            else
                add_values(std::false_type{});
        }
        const bool split = g.split;
        if (split && g.b0 == 0 && tid == 0) a.joins[blockIdx.x] = walk.join(a, g);
        float *rec = split ? chunk_record(a, blockIdx.x, g.slot) : nullptr;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int m = ty * RT + i, tok = m / a.part_heads, h = m % a.part_heads;
            if (tok >= g.tokens || h >= hh.count) continue;
            if (split) {
                if (tx == 0) {
                    rec[2 * m] = mx[i];
                    rec[2 * m + 1] = sum[i];
                }
#pragma unroll
                for (int c = 0; c < HD / 64; ++c) {
                    const int d = 64 * c + tx * 4;
                    if (d < a.hd)
#pragma unroll
                        for (int e = 0; e < 4; ++e) rec[2 * a.rec_rows + m * a.hd + d + e] = (e & 1) ? acc[i][2 * c + e / 2].y : acc[i][2 * c + e / 2].x;
                }
            } else {
                const long long o = ((long long)(g.r0 + tok) * a.n_qh + hh.first + h) * a.hd;
#pragma unroll
                for (int c = 0; c < HD / 64; ++c) {
                    const int d = 64 * c + tx * 4;
                    if (d < a.hd)
#pragma unroll
                        for (int e = 0; e < 4; ++e) store_as(a.out, o + d + e, a.q_dtype, ((e & 1) ? acc[i][2 * c + e / 2].y : acc[i][2 * c + e / 2].x) / sum[i]);
                }
            }
        }
    }
    if (flags) flag_error(a.err, flags);
}

// Join the records of the split tiles: block (c, y) takes its share of the
// pairs of the tile whose first contributor CTA c was.
//   M = max_c m_c,  out = sum_c 2^(m_c - M) acc_c / sum_c 2^(m_c - M) l_c
// A thread takes four dims of a pair, four records' loads in flight; the
// latency of L2 bounds it, so the items are spread over the grid.  (A warp per
// pair, four pairs one after the other: 12 us behind the ragged chunks' first
// launch, more than half of what that takes.)
constexpr int kCjThreads = 256;
constexpr int kCjShares = 16;
__global__ void __launch_bounds__(kCjThreads) chunk_join_kernel(const __grid_constant__ ChunkArgs a) {
    grid_dependency_wait();
    const ChunkJoin t = a.joins[blockIdx.x];
    const ChunkHeads hh = chunk_heads(a, t.part);
    const size_t rec_floats = (size_t)a.rec_rows * (a.hd + 2);
    const float *rec0 = a.partials + ((size_t)t.first * 2 + t.first_slot) * rec_floats;
    const int per = a.hd / 4;
    for (int i = blockIdx.y * kCjThreads + threadIdx.x; i < t.pairs * per; i += gridDim.y * kCjThreads) {
        const int m = i / per, d = (i % per) * 4;
        const int tok = m / a.part_heads, head = m % a.part_heads;
        if (head >= hh.count) continue;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float M = -INFINITY, L = 0.0f;
        for (int c0 = t.first; c0 <= t.last; c0 += 4) {
            float2 ml[4];
            float4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = min(c0 + k, t.last);
                const float *rec = c == t.first ? rec0 : a.partials + (size_t)c * 2 * rec_floats;
                ml[k] = __ldcg(reinterpret_cast<const float2 *>(rec + 2 * m));
                v[k] = __ldcg(reinterpret_cast<const float4 *>(rec + 2 * a.rec_rows + (size_t)m * a.hd + d));
            }
            float top = M;
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, ml[k].x);
            const float keep = M == top ? 1.0f : exp2f(M - top);  // (equal: both may be -inf)
            M = top;
            L *= keep;
            acc.x *= keep;
            acc.y *= keep;
            acc.z *= keep;
            acc.w *= keep;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (c0 + k > t.last) break;
                const float e = ml[k].x == top ? 1.0f : exp2f(ml[k].x - top);
                L = fmaf(ml[k].y, e, L);
                acc.x = fmaf(v[k].x, e, acc.x);
                acc.y = fmaf(v[k].y, e, acc.y);
                acc.z = fmaf(v[k].z, e, acc.z);
                acc.w = fmaf(v[k].w, e, acc.w);
            }
        }
        const long long o = ((long long)(t.r0 + tok) * a.n_qh + hh.first + head) * a.hd + d;
        store_as(a.out, o, a.q_dtype, acc.x / L);
        store_as(a.out, o + 1, a.q_dtype, acc.y / L);
        store_as(a.out, o + 2, a.q_dtype, acc.z / L);
        store_as(a.out, o + 3, a.q_dtype, acc.w / L);
    }
}

static size_t cs_smem(int HD, int rows) {
    return (size_t)(rows * HD + kCsStep * (HD + 4) + kCsStep * HD) * sizeof(float);
}
static int cs_hd(int hd) { return hd <= 64 ? 64 : hd <= 128 ? 128 : 256; }

int chunk_simt_grid() { return 2 * sm_count(); }

template <int RT>
static cudaError_t launch_cs(ChunkArgs &a, int *grid, cudaStream_t stream) {
    chunk_tile_shape(a, 16 * RT, 1);
    a.step = kCsStep;
    a.half_tokens = 0;
    a.w_half = a.w_full = 1;
    a.tile_cost = 0;
    a.piece = kCsPiece;
    const int HD = cs_hd(a.hd);
    const size_t smem = cs_smem(HD, 16 * RT);
    *grid = HD == 256 ? sm_count() : chunk_simt_grid();
    void (*fn)(ChunkArgs) = HD == 64    ? chunk_simt_kernel<64, RT>
                            : HD == 128 ? chunk_simt_kernel<128, RT>
                                        : chunk_simt_kernel<256, RT>;
    const cudaError_t e = cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_ex(fn, dim3(*grid), dim3(kCsThreads), smem, stream, false, a);
}

cudaError_t launch_chunk_simt(ChunkArgs &a, int *grid, cudaStream_t stream) {
    // (the lengths are on the device: the average decides, every tile size is right for every batch)
    return (long long)a.n_rows * a.gq <= 16ll * a.n_seqs ? launch_cs<1>(a, grid, stream) : launch_cs<4>(a, grid, stream);
}

void chunk_tile_shape(ChunkArgs &a, int sub_rows, int subs) {
    a.head_parts = (a.gq + sub_rows - 1) / sub_rows;
    a.part_heads = (a.gq + a.head_parts - 1) / a.head_parts;
    a.tile_tokens = subs * (sub_rows / a.part_heads);
}

}  // namespace ds

using namespace ds;

// (row, head) pairs of the largest tile any kernel uses, and so of a record
// (a multiple of four: records and their accumulators start on 16 bytes).
static int chunk_rec_rows(int64_t n_rows, int gq) {
    return (int)std::min<int64_t>(kChunkMaxTileRows, (n_rows * gq + 3) / 4 * 4);
}

extern "C" DS_API size_t ds_chunk_attention_workspace_bytes(int n_seqs, int64_t n_rows, int n_qh, int n_kvh,
                                                            int head_dim) {
    if (n_seqs < 1 || n_rows < 1 || n_kvh < 1 || n_qh < n_kvh || n_qh % n_kvh || head_dim < 1 || head_dim > 256 ||
        n_rows > DS_MAX_DIM || n_qh > DS_MAX_DIM)
        return 0;
    const size_t grid = chunk_simt_grid();
    return kWsHeader + align_up(grid * sizeof(ChunkJoin), 256) +
           grid * 2 * (size_t)chunk_rec_rows(n_rows, n_qh / n_kvh) * (head_dim + 2) * sizeof(float);
}

extern "C" DS_API int ds_gqa_chunk_attn(const void *q, int64_t q_len, int q_dtype, int64_t n_rows,
                                        const int32_t *row_starts, const int32_t *seq_lens, int n_seqs,
                                        const void *k_cache, const void *v_cache, int kv_dtype, int64_t cache_rows,
                                        const int32_t *block_table, int max_blocks_per_seq, int block_tokens,
                                        int n_qh, int n_kvh, int head_dim, float scale, void *out, int64_t out_len,
                                        void *workspace, size_t workspace_bytes, ds_stream_t stream) {
    if (n_rows < 1 || n_seqs < 1 || n_qh < 1 || n_kvh < 1 || head_dim < 1 || block_tokens < 1 ||
        max_blocks_per_seq < 1 || cache_rows < 1)
        return DS_EMPTY_DIMENSION;
    if (n_rows > DS_MAX_DIM || n_seqs > DS_MAX_DIM || n_qh > DS_MAX_DIM || cache_rows > DS_MAX_DIM ||
        (int64_t)max_blocks_per_seq * block_tokens > DS_MAX_DIM)
        return DS_DIMENSION_TOO_LARGE;
    if ((q_dtype != DS_F32 && q_dtype != DS_BF16) || (kv_dtype != DS_F32 && kv_dtype != DS_BF16)) return DS_BAD_DTYPE;
    if (n_qh % n_kvh || head_dim % 4 || head_dim > 256 || !(scale > 0.0f) || !std::isfinite(scale)) return DS_BAD_ARGUMENT;
    if (q_len != n_rows * n_qh * head_dim) return DS_A_LENGTH_MISMATCH;
    if (out_len != q_len) return DS_B_LENGTH_MISMATCH;
    if (!q || !row_starts || !seq_lens || !k_cache || !v_cache || !out) return DS_BAD_ARGUMENT;
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)k_cache | (uintptr_t)v_cache) & 15) return DS_BAD_ARGUMENT;
    // a split tile's rows may be written while another block still reads their q
    const size_t qb = (size_t)q_len * (q_dtype == DS_BF16 ? 2 : 4);
    if ((uintptr_t)q < (uintptr_t)out + qb && (uintptr_t)out < (uintptr_t)q + qb) return DS_BAD_ARGUMENT;
    if (!block_table && (int64_t)n_seqs * max_blocks_per_seq * block_tokens > cache_rows)
        return DS_CACHE_CAPACITY_EXCEEDED;
    if (cache_rows < block_tokens) return DS_CACHE_CAPACITY_EXCEEDED;
    if (!workspace || workspace_bytes < ds_chunk_attention_workspace_bytes(n_seqs, n_rows, n_qh, n_kvh, head_dim))
        return DS_WORKSPACE_TOO_SMALL;
    if ((uintptr_t)workspace & 255) return DS_BAD_ARGUMENT;
    ChunkArgs a = {};
    a.q = q;
    a.out = out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.q_dtype = q_dtype;
    a.kv_dtype = kv_dtype;
    a.n_rows = (int)n_rows;
    a.row_starts = row_starts;
    a.seq_lens = seq_lens;
    a.n_seqs = n_seqs;
    a.cache_rows = cache_rows;
    a.block_table = block_table;
    a.max_blocks = max_blocks_per_seq;
    a.bt = block_tokens;
    a.pool_blocks = cache_rows / block_tokens;
    a.n_qh = n_qh;
    a.n_kvh = n_kvh;
    a.hd = head_dim;
    a.gq = n_qh / n_kvh;
    a.scale = scale;
    a.rec_rows = chunk_rec_rows(n_rows, a.gq);
    char *ws = static_cast<char *>(workspace);
    a.err = reinterpret_cast<int *>(ws);
    a.joins = reinterpret_cast<ChunkJoin *>(ws + kWsHeader);
    a.partials = reinterpret_cast<float *>(ws + kWsHeader + align_up((size_t)chunk_simt_grid() * sizeof(ChunkJoin), 256));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int grid = 0;
    cudaError_t e = chunk_tc_supported(a) ? launch_chunk_tc(a, &grid, s) : launch_chunk_simt(a, &grid, s);
    if (e == cudaSuccess)
        e = launch_ex(chunk_join_kernel,
                      dim3(grid, std::min(kCjShares, (a.rec_rows * (a.hd / 4) + kCjThreads - 1) / kCjThreads)),
                      dim3(kCjThreads), 0, s, true, a);
    return e == cudaSuccess ? DS_OK : DS_CUDA_ERROR;
}
