// The chunk attention on the fifth-generation tensor cores (tcgen05), for a
// bf16 cache of whole pages and heads of 64 or 128; the mathematics, the work
// split and the joining of split tiles are those of chunk_attn.cuh.
//
// A tile's (row, head) pairs fill up to two parts of 128 MMA rows, a K/V step
// is 128 positions.  Per part and step:
//   S = Q K^T   (M 128, N 128, K hd): Q and K from shared memory, S in TMEM
//   P = 2^(c S - c m)   by the part's warpgroup, thread r owning row r; P
//       goes back to TMEM as bf16 over the columns S was in
//   O += P V    (M 128, N hd, K 128): P from TMEM, V from shared memory
// While one warpgroup turns its S into P the tensor core works for the other.
// Each part has a warp that issues its MMAs, a PV and the next QK at a time:
// tcgen05.mma of one thread complete in issue order, so S may overwrite the P
// it follows, and the two warps fill each other's waits (from one warp the
// tensor core ran dry for some 900 of 4,400 cycles a step).
//
// Two parts share one stream of K and V (one fetch serves 256 MMA rows; at
// 128 rows a step takes as long to fetch from L2 as to multiply).  A tile that
// fits one part (a single token's group of heads, or the end of a chunk) is
// put in both parts instead, which then take turns at the K/V steps with a
// running maximum and sum each, joined at the end: the same overlap.
//
// fp32 q (PARTS 3): q and P each go to the tensor core as three bf16 numbers
// that add up to them (24 bits cut in three; where q has fewer bits its empty
// pieces are 2^-30 and 2^-60 of it, see load_q).  The pieces of q are three MMAs
// into one S.  The pieces of P are rows of one MMA: a part has 40 pairs, each
// in three rows of a warp with the same S (10 pairs a warp), and row by row
// the warp writes the high, the middle and the low piece; O is the sum of the
// three rows.  (q in rows too costs half the MMAs, but S then is a sum over
// lanes: 384 shuffles a step, which took longer than everything else.)  Both
// parts work on the one tile, in turns.
//
// The running maximum that P is taken relative to is moved (and O rescaled)
// only when a row's maximum has grown by more than 2^8: P then stays below
// 2^8, which costs bf16 and fp32 no digits, and O is rescaled a few times in
// a tile instead of every step.  P is rounded to bf16 (PARTS 1), because a
// second piece of it would double the second product: 2^-8 of a weight at most,
// in the mean 1.3e-3 of the output beside the 1.6e-3 of its own rounding.  The
// sum adds the fp32 weights.
//
// A step that reaches past the first row's position is masked per row.  V
// there may hold anything (another row's NaN, the stale rest of a page), and
// 0 x NaN is NaN, so the warpgroups check the step's V in shared memory:
// positions past the end are zeroed, and a non-finite value at a position
// that only some of the rows attend is zeroed and noted, to be added to the
// rows that do attend it at the end.
//
// Measured in a graph, heads of 128, 32 on 8, pages of 16: a bf16 prompt of
// 8,192 in 456 us (1,206 TFLOP/s; the tensor pipe is active 55 % of the cycles,
// the softmax between a step's two products and the tiles' ends bound it); 64
// single tokens over up to 4,096 positions with bf16 q in 110 us (4.7 TB/s),
// with fp32 q in 137 (3.8 TB/s; idle from a tile's last step to the next one's
// first, 8,000 to 10,000 cycles); one bf16 token over 1,024 in 13.9 us with the
// joining launch (latency); 256 fp32 rows behind 768 positions in 51 us, 2,048
// from position 0 in 306 (40 pairs a tile).
// Registers: 168 a thread in every variant; spilled: none with bf16 q, 20 bytes
// <64, 3>, 116 bytes <128, 3>.
//
// Every wait is bounded; after one gives up all others return at once and the
// kernel runs to its end without them (its barriers still pair up), flagged.
#include <algorithm>
#include <atomic>

#include "chunk_attn.cuh"
#include "tc.h"
#include "tcgen05.cuh"

namespace ds {

constexpr int kCtStep = 128;
constexpr int kCtThreads = 384;  // two softmax warpgroups; one with two MMA, the K/V and the walking warp
// Registers a thread: 168 at launch (384 x 168), moved to the softmax
// warpgroups, whose thread holds a row's 128 scores: 2 x 216 + 72 = 3 x 168.
constexpr int kCtRegsSoftmax = 216, kCtRegsOther = 72;
constexpr int kCtAhead = 8;      // steps one part may be ahead of the other, and more: half the ring's tiles
constexpr int kCtSegs = 4;       // segments handed out and not yet done with
// Weights of the work split (chunk_attn.cuh): a K/V step of both parts takes
// about 1.5 times as long as one of a tile that takes turns; beginning and
// ending a tile takes about as long as two steps, with fp32 q as four (swept
// from 256 to 2048: 64 single fp32 tokens 158 us at 256, 148 at 512, 138 at
// 1024, 146 at 2048; a bf16 prompt of 8192 464, 446, 452, 470).  With fp32 q
// every tile takes turns, so the weights rate its whole tiles above the last
// one of a sequence without cause; equal ones have not been measured.
constexpr int kCtWeightTurns = 2, kCtWeightShared = 3, kCtTileCost = 2 * 256, kCtTileCostF32 = 2 * 512;
constexpr int kCtPiece = 256;
constexpr int kCtHalf = 128 * 128;  // bytes of 128 rows of one 64-element (128-byte) half
constexpr int kCtMaxStages = 10;
constexpr int kCtSmall = 3 * 1024;     // barriers, segments, notes
constexpr size_t kCtSmemLimit = 227 * 1024;
constexpr float kCtLog2e = 1.4426950408889634f;
constexpr float kCtLag = 8.0f;      // log2 of the growth that moves the reference maximum

template <int HD, int PARTS>
struct CtCfg {
    static constexpr int kHalves = HD / 64;
    static constexpr int kTileBytes = kHalves * kCtHalf;  // 128 rows of one head
    static constexpr int kQTiles = PARTS == 1 ? 2 : 3;    // both parts' q, or the three pieces of one
    static constexpr int kFixed = kCtSmall + kQTiles * kTileBytes;
    static constexpr int kFit = (int)((kCtSmemLimit - kFixed) / kTileBytes);
    static constexpr int kStages = kFit < kCtMaxStages ? kFit : kCtMaxStages;
    static constexpr size_t kSmem = kFixed + (size_t)kStages * kTileBytes;
};

struct CtMaps {
    CUtensorMap k, v;  // {64, cache_rows, n_kvh * hd / 64}, boxes {64, box_rows, 1}, 128-byte swizzle
    CUtensorMap q;     // bf16 q: {hd, n_qh, n_rows}, boxes {64, heads of a part, rows of a part}, the same swizzle
    int box_rows;
};

// An MMA warp runs its loop with all its lanes and one of them issues, by a
// predicate: addresses and descriptors then stay in uniform registers, where
// the instruction wants them.  (From a branch of one lane each of them has to
// be moved there first: about 100 cycles an MMA against the 64 it runs.)
__device__ __forceinline__ uint32_t ct_elect() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one;
}
// D[tmem] (+)= A[smem] x B[smem], and A[tmem] x B[smem].
__device__ __forceinline__ void ct_mma_ss(uint32_t one, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "setp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
__device__ __forceinline__ void ct_mma_ts(uint32_t one, uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "setp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
__device__ __forceinline__ void ct_commit(uint32_t one, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(one)
        : "memory");
}
// 32 columns of this thread's lane; complete only after ct_wait_ld().
__device__ __forceinline__ void ct_ld32(uint32_t taddr, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void ct_ld16(uint32_t taddr, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void ct_st16(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// The loads of this warp are complete, v's 32 among them (named, so that no
// use of them is moved in front of the wait).
__device__ __forceinline__ void ct_wait_ld32(float *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                   "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                   "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void ct_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void ct_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void ct_fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float ct_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// bf16 pair, a in the low half.
__device__ __forceinline__ uint32_t ct_pack(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// The leading 8 bits of two numbers (cut off, not rounded) as a bf16 pair.
__device__ __forceinline__ uint32_t ct_top2(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float ct_top(float a, uint32_t mask) { return __uint_as_float(__float_as_uint(a) & mask); }

__device__ __forceinline__ void ct_box(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// The same from the one lane of the warp that `one` marks.
__device__ __forceinline__ void ct_box_one(uint32_t one, uint32_t dst, const CUtensorMap *map, int y, int z, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(bar), "r"(one)
        : "memory");
}

// Wait for a phase; once any wait of the block has given up, at once.
__device__ __forceinline__ void ct_wait(uint64_t *bar, uint32_t parity, volatile int *dead, int *err) {
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

// The same for a counter in shared memory that reaches n.
__device__ __forceinline__ void ct_wait_count(const int *count, int n, volatile int *dead, int *err) {
    const uint64_t t0 = global_timer_ns();
    while (*reinterpret_cast<const volatile int *>(count) < n && !*dead)
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            flag_error(err, DS_ERR_WAIT_TIMEOUT);
            *dead = 1;
        }
}

// Order of the 2 nb tiles of a segment in the ring, the order they are first
// needed in.  Shared steps: K0 V0 K1 V1 ...  Steps taken in turns:
// K0 K1 V0 K2 V1 K3 ... V(nb-2) V(nb-1).
__device__ __forceinline__ int ct_v_place(bool turns, int j, int nb) {
    return !turns ? 2 * j + 1 : j == nb - 1 ? 2 * nb - 1 : 2 * j + 2;
}

// A segment as the walking warp hands it to the other roles.
struct CtSeg {
    ChunkSeg g;
    ChunkHeads heads;
    int nb;     // K/V steps; 0: the walk is over
    int turns;  // the parts take turns at the steps
};

struct CtShared {
    CtSeg seg[kCtSegs];
    uint64_t seg_full[kCtSegs], seg_empty[kCtSegs];
    uint64_t full[kCtMaxStages], empty[kCtMaxStages];
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], v_clean[kCtAhead], done[2];
    uint32_t tmem;
    int dead;
    union {
        long long red[34];  // ChunkWalk::init
        float2 ml[128];     // turns: a row's (max, sum) of part 1, for part 0
    };
    // non-finite V per dim, by the segment's parity: 10-bit first positions of
    // NaN, +inf, -inf behind the tile's pos0; noted: there are some
    int noted[2];
    int readers[2];  // warps that have read this segment's notes
    int left[2];  // segments a part's warps are done with, four counts each
    unsigned note[2][128];
};
static_assert(sizeof(CtShared) <= kCtSmall, "shared words");

constexpr unsigned kCtNoNote = 0x3fffffffu;

// Note a non-finite value of dim d at position rel behind the first row's.
__device__ inline void ct_note(unsigned *w, int rel, float v) {
    const int sh = v != v ? 0 : v > 0.0f ? 10 : 20;
    unsigned old = *reinterpret_cast<volatile unsigned *>(w);
    while (((old >> sh) & 1023u) > (unsigned)rel) {
        const unsigned want = (old & ~(1023u << sh)) | ((unsigned)rel << sh);
        const unsigned was = atomicCAS(w, old, want);
        if (was == old) break;
        old = was;
    }
}
// What the noted values add to a row that attends positions up to rel.
__device__ __forceinline__ float ct_noted(unsigned w, int rel) {
    const bool nan = (int)(w & 1023u) <= rel, pinf = (int)((w >> 10) & 1023u) <= rel, ninf = (int)(w >> 20) <= rel;
    if (nan || (pinf && ninf)) return __int_as_float(0x7fffffff);
    return pinf ? INFINITY : ninf ? -INFINITY : 0.0f;
}

// The sum of a row's weights times column d of V over positions [t0, t1), of
// which the tensor core made NaN although the weights are finite: a weight (or
// a part of it) that is zero or negative met an infinity.  Weights are taken as
// positive, so the infinities decide (also behind a key that is infinite).
__device__ __noinline__ float ct_infinite(const ChunkArgs &a, int seq, int kv, int d, int t0, int t1) {
    float sum = 0.0f;
    int flags = 0;
    for (int t = t0; t < t1 && sum == sum; ++t) {
        const long long row = chunk_block_row(a, seq, t / a.bt, flags) + t % a.bt;
        const float v = load_as(a.v_cache, (row * a.n_kvh + kv) * a.hd + d, DS_BF16);
        if (!(fabsf(v) < INFINITY)) sum += v;
    }
    return sum == 0.0f ? __int_as_float(0x7fffffff) : sum;
}

// Hand-over of segments: these waits are not cut short when another wait has
// given up (the roles must go on agreeing on the segments, their barriers pair
// up by them) and outlast it by far: every role then runs through.
__device__ __forceinline__ void ct_wait_seg(uint64_t *bar, uint32_t parity, int *err) {
    for (int k = 0; k < 8; ++k) {
        if (mbar_wait(bar, parity, k == 7 ? err : nullptr)) return;
    }
}

template <int HD, int PARTS>
__global__ void __launch_bounds__(kCtThreads, 1)
    chunk_tc_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ CtMaps maps) {
    using Cfg = CtCfg<HD, PARTS>;
    constexpr int ST = Cfg::kStages;
    constexpr int RPW = PARTS == 1 ? 32 : 10;  // rows a warp
    constexpr int SUB = 4 * RPW;               // rows of a part
    extern __shared__ __align__(1024) unsigned char ct_smem[];
    CtShared &sh = *reinterpret_cast<CtShared *>(ct_smem);
    unsigned char *s_q = ct_smem + kCtSmall, *s_ring = s_q + Cfg::kQTiles * Cfg::kTileBytes;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *dead = &sh.dead;
    if (smem_u32(ct_smem) & 1023u) {  // swizzled tiles start on 1 KB; the same answer in every thread
        if (tid == 0) flag_error(a.err, DS_ERR_WAIT_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 2);  // both parts
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&sh.q_full[w], PARTS == 1 ? 1 : 8);
            mbar_init(&sh.q_empty[w], 1);
            mbar_init(&sh.s_full[w], 1);
            mbar_init(&sh.p_full[w], 4);
            mbar_init(&sh.o_full[w], 1);
            mbar_init(&sh.done[w], 1);
            sh.noted[w] = sh.readers[w] = sh.left[w] = 0;
        }
        for (int i = 0; i < kCtSegs; ++i) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.seg_empty[i], 11);  // K/V producer, two MMA warps, eight softmax warps
        }
        for (int i = 0; i < kCtAhead; ++i) mbar_init(&sh.v_clean[i], 4);
        sh.dead = 0;
        fence_mbarrier_init();
    }
    for (int i = tid; i < 256; i += kCtThreads) sh.note[i >> 7][i & 127] = kCtNoNote;
    if (warp == 8) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    grid_dependency_wait();  // everything up to here may run before the launch in front is through
    chunk_zero_empty_rows(a);
    ChunkWalk walk;
    walk.init<false>(a, sh.red);  // synchronises the block
    // The joining launch may take its place as blocks of this one end; it
    // waits for the end of all before it reads.
    allow_dependent_launch();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const int half_tokens = a.half_tokens;  // rows of the sequence in one part
    int flags = walk.flags;
    auto seg_get = [&](uint32_t k) -> const CtSeg & {
        ct_wait_seg(&sh.seg_full[k % kCtSegs], (k / kCtSegs) & 1, a.err);
        return sh.seg[k % kCtSegs];
    };
    auto seg_done = [&](uint32_t k) { mbar_arrive(&sh.seg_empty[k % kCtSegs]); };  // one thread of the warp

    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtRegsOther));
    if (warp == 10) {
        // ------------------------------------------------ the walk over this CTA's range, and bf16 q
        // A segment is handed out before the q of the one before it is waited
        // for.  A part's q is free once the tensor core is through with its
        // last QK; MMA rows without a (row, head) pair hold anything: no row
        // reaches another.
        if (lane == 0) {
            a.joins[blockIdx.x].pairs = 0;
            uint32_t issued = 0;
            int q_first = 0, q_row[2] = {0, 0};
            for (uint32_t k = 0;; ++k) {
                CtSeg c;
                c.nb = 0;
                if (walk.next(a, c.g)) {
                    c.nb = c.g.b1 - c.g.b0;
                    c.turns = c.g.tokens <= half_tokens;
                    c.heads = chunk_heads(a, c.g.part);
                    if (c.g.split && c.g.b0 == 0) a.joins[blockIdx.x] = walk.join(a, c.g);
                }
                if (k >= kCtSegs) ct_wait_seg(&sh.seg_empty[k % kCtSegs], ((k / kCtSegs) - 1) & 1, a.err);
                sh.seg[k % kCtSegs] = c;
                mbar_arrive(&sh.seg_full[k % kCtSegs]);
                if (PARTS == 1 && k > 0) {
                    for (int w = 0; w < 2; ++w)
                        if (k > 1) ct_wait(&sh.q_empty[w], k & 1, dead, a.err);  // the segment's before: k - 2
                    if (!*dead) {
                        ++issued;
                        for (int w = 0; w < 2; ++w) {
                            mbar_arrive_expect_tx(&sh.q_full[w],
                                                  (uint32_t)(Cfg::kHalves * 128 * a.part_heads * half_tokens));
                            for (int h = 0; h < Cfg::kHalves; ++h)
                                ct_box(smem_u32(s_q) + w * Cfg::kTileBytes + h * kCtHalf, &maps.q, h * 64, q_first,
                                       q_row[w], &sh.q_full[w]);
                        }
                    }
                }
                if (c.nb == 0) break;
                q_first = c.heads.first;
                q_row[0] = c.g.r0;
                q_row[1] = c.turns ? c.g.r0 : c.g.r0 + half_tokens;
            }
            // every copy issued has landed before the block may end
            for (int w = 0; w < 2; ++w)
                if (issued) mbar_wait(&sh.q_full[w], (issued - 1) & 1, *dead ? nullptr : a.err);
        }
        __syncwarp();
    } else if (warp == 9) {
        // ------------------------------------------------ K/V producer
        uint32_t n = 0;
        const int R = maps.box_rows;
        const uint32_t one = ct_elect(), ring = smem_u32(s_ring);
        for (uint32_t seg = 0;; ++seg) {
            const CtSeg &c = seg_get(seg);
            const int nb = __shfl_sync(0xffffffffu, c.nb, 0);
            if (nb == 0) break;
            const bool turns = __shfl_sync(0xffffffffu, c.turns, 0);
            const int kv = __shfl_sync(0xffffffffu, c.heads.kv, 0), b0 = __shfl_sync(0xffffffffu, c.g.b0, 0);
            const int len = __shfl_sync(0xffffffffu, c.g.len, 0), seq = c.g.seq;
            __syncwarp();
            if (one) seg_done(seg);
            // Lane l holds box l's block number (16 boxes at most); the next
            // tile's is fetched before the stage of this one is awaited: the
            // table is a trip to L2 away.
            auto tile_of = [&](int i, int &j, bool &is_v) {
                if (!turns) {
                    is_v = i & 1;
                    j = i >> 1;
                } else if (i < 2) {
                    is_v = i == nb;  // one step: K0 V0
                    j = is_v ? 0 : i;
                } else {
                    const int m = i - 2;
                    is_v = !(m & 1) || m / 2 + 2 >= nb;
                    j = !is_v ? m / 2 + 2 : (m + 1) / 2;
                }
            };
            auto id_of = [&](int i) {
                int j;
                bool is_v;
                tile_of(i, j, is_v);
                const int pos = (b0 + j) * kCtStep + lane * R;
                return pos < len && lane * R < kCtStep ? chunk_block_id(a, seq, pos / a.bt) : 0;
            };
            int id = id_of(0);
            for (int i = 0; i < 2 * nb; ++i, ++n) {
                int j;
                bool is_v;
                tile_of(i, j, is_v);
                const int boxes = (min(kCtStep, len - (b0 + j) * kCtStep) + R - 1) / R;
                const int id_next = i + 1 < 2 * nb ? id_of(i + 1) : 0;
                const int row = (int)chunk_id_row(a, id, flags) + ((b0 + j) * kCtStep + lane * R) % a.bt;
                id = id_next;
                const int s = n % ST;
                if (n >= ST) ct_wait(&sh.empty[s], ((n / ST) - 1) & 1, dead, a.err);
                // one decision for the warp; a block that has given up fetches no more
                if (__any_sync(0xffffffffu, *dead)) continue;
                if (one) mbar_arrive_expect_tx(&sh.full[s], (uint32_t)(boxes * R * 128 * Cfg::kHalves));
                __syncwarp();
                const uint32_t dst = ring + (uint32_t)s * Cfg::kTileBytes, bar = smem_u32(&sh.full[s]);
                const CUtensorMap *map = is_v ? &maps.v : &maps.k;
                for (int b = 0; b < boxes; ++b) {
                    const int y = __shfl_sync(0xffffffffu, row, b);
#pragma unroll
                    for (int h = 0; h < Cfg::kHalves; ++h)
                        ct_box_one(one, dst + h * kCtHalf + b * R * 128, map, y, kv * Cfg::kHalves + h, bar);
                }
            }
        }
        // every copy issued has landed before the block may end
        if (lane == 0) {
            for (uint32_t f = n > ST ? n - ST : 0; f < n; ++f)
                if (!mbar_wait(&sh.full[f % ST], (f / ST) & 1, *dead ? nullptr : a.err)) break;
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ MMA issue, a warp for each part
        {
            const uint32_t w = warp == 8 ? 0 : 1;
            constexpr uint32_t kIdQk = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
            constexpr uint32_t kIdPv =
                (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) | ((128u >> 4) << 24);
            const uint32_t one = ct_elect();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);  // the same in all lanes, for the compiler too
            // Everything the next MMA needs is at hand before its wait is over:
            // this warp's own instructions are on the critical path.
            const uint64_t q0 = smem_desc(smem_u32(s_q), 16, 1024);
            const uint64_t k0 = smem_desc(smem_u32(s_ring), 16, 1024), v0 = smem_desc(smem_u32(s_ring), kCtHalf, 1024);
            uint32_t at = 0, at_par = 0, p_par = 0;
            auto take = [&]() {  // the next tile of the ring is there
                ct_wait(&sh.full[at], at_par, dead, a.err);
                const uint32_t s = at;
                if (++at == ST) {
                    at = 0;
                    at_par ^= 1;
                }
                return s;
            };
            auto pass = [&]() {  // the next tile is the other part's alone
                const uint32_t s = take();
                if (one) mbar_arrive(&sh.empty[s]);
            };
            auto wait_p = [&]() {
                ct_wait(&sh.p_full[w], p_par, dead, a.err);
                p_par ^= 1;
                tc_fence_after();
            };
            auto qk = [&](uint32_t s) {
                const uint64_t ad = q0 + (uint64_t)(PARTS == 1 ? w * (Cfg::kTileBytes >> 4) : 0);
                const uint64_t bd = k0 + (uint64_t)(s * (Cfg::kTileBytes >> 4));
                const uint32_t d = tm + w * 128;
#pragma unroll
                for (int z = PARTS - 1; z >= 0; --z)  // the smallest piece first
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k) {
                        const uint64_t o = (uint64_t)((k / 4) * (kCtHalf >> 4) + (k % 4) * 2);
                        ct_mma_ss(one, d, ad + (uint64_t)(z * (Cfg::kTileBytes >> 4)) + o, bd + o, kIdQk,
                                  k || z < PARTS - 1 ? 1u : 0u);
                    }
            };
            auto pv = [&](uint32_t s, bool first) {
                const uint64_t bd = v0 + (uint64_t)(s * (Cfg::kTileBytes >> 4));
                const uint32_t d = tm + 256 + w * HD, p = tm + w * 128;
#pragma unroll
                for (int k = 0; k < kCtStep / 16; ++k)
                    ct_mma_ts(one, d, p + k * 8, bd + (uint64_t)(k * 128), kIdPv, (k || !first) ? 1u : 0u);
            };
            for (uint32_t seg = 0;; ++seg) {
                const CtSeg &c = seg_get(seg);
                const int nb = __shfl_sync(0xffffffffu, c.nb, 0);
                if (nb == 0) break;
                const int turns = __shfl_sync(0xffffffffu, c.turns, 0);
                if (one) seg_done(seg);
                uint32_t ks, vs;
                const int stride = turns ? 2 : 1, mine = turns ? (int)w : 0;  // steps mine, mine + stride, ...
                // (also where this part has no step: a barrier tells two phases
                // apart, so each is awaited, and q_empty below lets the next come)
                ct_wait(&sh.q_full[PARTS == 1 ? w : 0], seg & 1, dead, a.err);
                for (int j = 0; j < min(stride, nb); ++j) {
                    if (j != mine) {
                        pass();
                        continue;
                    }
                    ks = take();
                    tc_fence_after();
                    qk(ks);
                    ct_commit(one, &sh.s_full[w]);
                    ct_commit(one, &sh.empty[ks]);
                }
                if (mine + stride >= nb) ct_commit(one, &sh.q_empty[w]);  // no further use of this tile's q
                for (int j = 0; j < nb; ++j) {
                    const bool more = j + stride < nb;
                    if (turns && (j & 1) != mine) {
                        pass();
                        if (more) pass();
                        continue;
                    }
                    vs = take();
                    if (more) ks = take();
                    wait_p();
                    pv(vs, j < stride);
                    if (more) {
                        qk(ks);
                        ct_commit(one, &sh.s_full[w]);
                        if (j + 2 * stride >= nb) ct_commit(one, &sh.q_empty[w]);
                    } else {
                        ct_commit(one, &sh.o_full[w]);
                    }
                    ct_commit(one, &sh.empty[vs]);
                    if (more) ct_commit(one, &sh.empty[ks]);
                }
            }
            // nothing of ours runs on the tensor cores when the block ends
            ct_commit(one, &sh.done[w]);
            mbar_wait(&sh.done[w], 0, *dead ? nullptr : a.err);
        }
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kCtRegsSoftmax));
        // ------------------------------------------------ softmax, part w
        const int w = warp >> 2, q4 = warp & 3, t = tid & 127;
        const int r = PARTS == 1 ? t : q4 * RPW + lane % RPW;  // row of the part
        const int piece = PARTS == 1 ? 0 : lane / RPW;         // hi, mid, lo (3: an unused lane)
        const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
        const uint32_t ts = tmem + lane_base + w * 128, to = tmem + lane_base + 256 + w * HD;
        const float c = a.scale * kCtLog2e;
        const int tok_r = r / a.part_heads, head_r = r % a.part_heads;
        uint32_t n0 = 0, sc = 0, oc0 = 0, oc1 = 0, vc = 0;
        // fp32 q: eight values of a pair an item, as three bf16 numbers each
        // (cut, not rounded: 8 bits of the 24 a piece), one MMA operand per
        // piece; pair p is rows 32 (p / 10) + p % 10 and 10 and 20 further of
        // each.  Both warpgroups load.  A piece with nothing left in it is
        // 2^-30 of the one before, below fp32's digits: zero times an infinite
        // key would be NaN where q times it is an infinity.
        auto load_q = [&](const CtSeg &c) {
            const int n_items = c.g.tokens * a.part_heads * (HD / 8);
            constexpr int kItems = (SUB * (HD / 8) + 255) / 256;
            float4 x[kItems][2];
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int it = tid + 256 * i, p = it / (HD / 8), ch = it % (HD / 8);
                const int tk = p / a.part_heads, h = p - tk * a.part_heads;
                x[i][0] = x[i][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (it < n_items && h < c.heads.count) {
                    const float4 *src = reinterpret_cast<const float4 *>(
                        static_cast<const float *>(a.q) +
                        ((long long)(c.g.r0 + tk) * a.n_qh + c.heads.first + h) * HD + ch * 8);
                    x[i][0] = __ldg(src);
                    x[i][1] = __ldg(src + 1);
                }
            }
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int it = tid + 256 * i, p = it / (HD / 8), ch = it % (HD / 8);
                if (it >= n_items) break;
                float y[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
                const int m0 = (p / RPW) * 32 + p % RPW;
                unsigned char *dst = s_q + (ch >> 3) * kCtHalf;
#pragma unroll
                for (int z = 0; z < 3; ++z) {
                    const uint4 v = make_uint4(ct_top2(y[0], y[1]), ct_top2(y[2], y[3]), ct_top2(y[4], y[5]),
                                               ct_top2(y[6], y[7]));
#pragma unroll
                    for (int m = m0; m < m0 + 3 * RPW; m += RPW)
                        *reinterpret_cast<uint4 *>(dst + z * Cfg::kTileBytes + m * 128 + (((ch & 7) ^ (m & 7)) << 4)) = v;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float t = ct_top(y[k], 0xffff0000u), rest = y[k] - t;
                        y[k] = rest == 0.0f ? t * 0x1p-30f : rest;
                    }
                }
            }
            ct_fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full[0]);
        };
        if (PARTS == 3) {
            const CtSeg &c = seg_get(0);
            if (c.nb) load_q(c);
        }
        for (uint32_t seg = 0;; ++seg) {
            const CtSeg *cur = &seg_get(seg);
            if (cur->nb == 0) break;
            const ChunkSeg &g = cur->g;
            const bool turns = cur->turns;
            const int nb = cur->nb;
            const int steps = turns ? (nb + 1 - w) >> 1 : nb;
            const int rel = (turns ? 0 : w * half_tokens) + tok_r;  // this row attends positions up to pos0 + rel
            const bool valid = tok_r < half_tokens && rel < g.tokens && head_r < cur->heads.count &&
                               (PARTS == 1 || piece < PARTS);
            const bool busy = __any_sync(0xffffffffu, valid);
            const int par = seg & 1;
            float m_ref = -INFINITY, sum = 0.0f;
            for (int i = 0; i < steps; ++i, ++sc) {
                const int j = turns ? 2 * i + w : i;
                const int t0 = (g.b0 + j) * kCtStep;
                const bool masked = t0 + kCtStep - 1 > g.pos0;
                ct_wait(&sh.s_full[w], sc & 1, dead, a.err);
                __syncwarp();  // tensor memory is read by whole warps
                tc_fence_after();
                if (masked && (turns || w == 0)) {
                    // Check the step's V: this thread position t0 + t.  Part 0
                    // does it for both where they share the step.
                    const uint32_t place = n0 + (uint32_t)ct_v_place(turns, j, nb);
                    ct_wait(&sh.full[place % ST], (place / ST) & 1, dead, a.err);
                    unsigned char *row = s_ring + (size_t)(place % ST) * Cfg::kTileBytes + t * 128;
                    const int behind = t0 + t - g.pos0;
                    if (t0 + t >= g.len) {
#pragma unroll
                        for (int ch = 0; ch < HD / 8; ++ch)
                            *reinterpret_cast<uint4 *>(row + (ch >> 3) * kCtHalf + (((ch & 7) ^ (t & 7)) << 4)) =
                                make_uint4(0, 0, 0, 0);
                    } else if (behind > 0) {
                        // an exponent of all ones carries into the sign's place
                        uint32_t bad = 0;
#pragma unroll
                        for (int ch = 0; ch < HD / 8; ++ch) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(row + (ch >> 3) * kCtHalf +
                                                                             (((ch & 7) ^ (t & 7)) << 4));
                            bad |= ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                                   ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
                        }
                        if (bad & 0x80008000u) {
                            // the notes were those of the segment before the last:
                            // the other part is done with it before they change
                            ct_wait_count(&sh.left[1 - w], 4 * ((int)seg - 1), dead, a.err);
                            for (int d = 0; d < HD; ++d) {
                                __nv_bfloat16 *p = reinterpret_cast<__nv_bfloat16 *>(
                                    row + (d >> 6) * kCtHalf + ((((d >> 3) & 7) ^ (t & 7)) << 4) + (d & 7) * 2);
                                const float x = __bfloat162float(*p);
                                if (fabsf(x) < INFINITY) continue;
                                ct_note(&sh.note[par][d], behind, x);
                                *p = __float2bfloat16_rn(0.0f);
                            }
                            sh.noted[par] = 1;
                        }
                    }
                    ct_fence_async();
                    __syncwarp();
                    if (turns)
                        named_sync(2 + w, 128);
                    else if (lane == 0)
                        mbar_arrive(&sh.v_clean[vc % kCtAhead]);
                }
                if (busy) {
                    // bf16: the row's 128 scores stay in registers between their
                    // maximum and their weights.  fp32: short loops that read S
                    // twice, because a whole row's code, three pieces a weight,
                    // is fetched more slowly than it runs (64 single tokens:
                    // 165 -> 142 us; for bf16 the same costs 448 -> 485 us on a
                    // prompt of 8192, where the tensor core waits for P).
                    constexpr int kHeld = PARTS == 1 ? kCtStep : 64;
                    const int lim = masked ? g.pos0 + rel - t0 : kCtStep;  // the row's last column
                    float s[kHeld], top;
                    auto hide = [&](float *v, int k0, int n) {
#pragma unroll
                        for (int k = 0; k < n; ++k) v[k] = k0 + k <= lim ? v[k] : -INFINITY;
                    };
                    auto highest = [&](const float *v, int n) {  // chains of three-input maxima
                        float t4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                        for (int k = 4; k + 1 < n; k += 2)
                            t4[(k >> 1) & 3] = fmaxf(fmaxf(t4[(k >> 1) & 3], v[k]), v[k + 1]);
                        return fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                    };
                    if constexpr (PARTS == 1) {
#pragma unroll
                        for (int k = 0; k < kHeld; k += 32) ct_ld32(ts + k, s + k);
                        ct_wait_ld();
                        if (masked) hide(s, 0, kHeld);
                        top = highest(s, kHeld);
                    } else {
                        top = -INFINITY;
#pragma unroll 1
                        for (int k0 = 0; k0 < kCtStep; k0 += 64) {
                            ct_ld32(ts + k0, s);
                            ct_ld32(ts + k0 + 32, s + 32);
                            ct_wait_ld32(s);
                            ct_wait_ld32(s + 32);
                            if (masked) hide(s, k0, 64);
                            top = fmaxf(top, highest(s, 64));
                        }
                    }
                    const float m_new = fmaxf(m_ref, top);
                    if (i == 0) {
                        m_ref = m_new;
                    } else if (__any_sync(0xffffffffu, valid && (m_new - m_ref) * c > kCtLag)) {
                        const float f = m_new == -INFINITY ? 1.0f : ct_exp2((m_ref - m_new) * c);
                        m_ref = m_new;
                        sum *= f;
#pragma unroll 1
                        for (int k = 0; k < HD; k += 16) {
                            float o[16];
                            uint32_t u[16];
                            ct_ld16(to + k, o);
                            ct_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * f);
                            ct_st16(to + k, u);
                        }
                    }
                    const float mc = m_ref == -INFINITY ? 0.0f : m_ref * c;
                    // two scores an instruction where the machine has the pair form
                    const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
                    // this lane's piece: what the pieces before it hold is taken off
                    const uint32_t cut1 = piece > 0 ? 0xffff0000u : 0u, cut2 = piece > 1 ? 0xffff0000u : 0u;
                    float2 add[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    auto weigh = [&](float *v, int k0) {  // 32 scores to weights, back to where S was
                        if (PARTS == 3 && masked) hide(v, k0, 32);
                        uint32_t p[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float2 x = chunk_fma2(make_float2(v[2 * k], v[2 * k + 1]), c2, mc2);
                            x.x = ct_exp2(x.x);
                            x.y = ct_exp2(x.y);
                            add[k & 1] = chunk_add2(add[k & 1], x);
                            if (PARTS == 1) {
                                p[k] = ct_pack(x.x, x.y);
                            } else {
                                x = chunk_add2(x, make_float2(-ct_top(x.x, cut1), -ct_top(x.y, cut1)));
                                x = chunk_add2(x, make_float2(-ct_top(x.x, cut2), -ct_top(x.y, cut2)));
                                p[k] = ct_top2(x.x, x.y);
                            }
                        }
                        ct_st16(ts + k0 / 2, p);  // (columns whose S has been read)
                    };
                    if constexpr (PARTS == 1) {
#pragma unroll
                        for (int k0 = 0; k0 < kHeld; k0 += 32) weigh(s + k0, k0);
                    } else {
                        float *s_a = s, *s_b = s + 32;  // the next 32 on their way while these are worked on
                        ct_ld32(ts, s_a);
#pragma unroll 1
                        for (int k0 = 0; k0 < kCtStep; k0 += 64) {
                            ct_wait_ld32(s_a);
                            ct_ld32(ts + k0 + 32, s_b);
                            weigh(s_a, k0);
                            ct_wait_ld32(s_b);
                            if (k0 + 64 < kCtStep) ct_ld32(ts + k0 + 64, s_a);
                            weigh(s_b, k0 + 32);
                        }
                    }
                    sum += (add[0].x + add[0].y) + (add[1].x + add[1].y);
                    ct_wait_st();
                    tc_fence_before();
                }
                if (masked && !turns) {
                    // part 0 has checked this V; it may be as far ahead as the
                    // ring reaches, so the checked steps go round several barriers
                    if (w == 1) ct_wait(&sh.v_clean[vc % kCtAhead], (vc / kCtAhead) & 1, dead, a.err);
                    ++vc;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[w]);
            }
            n0 += 2 * nb;

            if (turns) {
                if (w == 1) sh.ml[t] = make_float2(m_ref, sum);
                named_sync(1, 256);  // part 1's maxima and notes are written
            }
            if (PARTS == 3) {  // this tile's S are all there: its q is free
                const CtSeg &next = seg_get(seg + 1);
                for (int u = 0; u < 2; ++u) ct_wait(&sh.q_empty[u], seg & 1, dead, a.err);
                if (next.nb) load_q(next);
            }

            const int steps0 = turns ? (nb + 1) >> 1 : nb, steps1 = turns ? nb >> 1 : nb;
            if (w == 0 || !turns) {
                ct_wait(&sh.o_full[w], (w ? oc1 : oc0) & 1, dead, a.err);
                if (turns && steps1) ct_wait(&sh.o_full[1], oc1 & 1, dead, a.err);
                __syncwarp();
                tc_fence_after();
                // (only a masked step notes, and only after one are they here to be read)
                const bool notes = g.b1 * kCtStep - 1 > g.pos0 && sh.noted[par];
                const bool split = g.split;
                float f0 = 1.0f, f1 = 0.0f;
                if (turns && steps1) {  // join the two parts' turns
                    const float2 o = sh.ml[t];
                    const float top = fmaxf(m_ref, o.x);
                    f0 = m_ref == top ? 1.0f : ct_exp2((m_ref - top) * c);
                    f1 = o.x == top ? 1.0f : ct_exp2((o.x - top) * c);
                    m_ref = top;
                    sum = sum * f0 + o.y * f1;
                }
                if (busy) {
                    const int m = (turns ? 0 : w * half_tokens * a.part_heads) + r;  // pair in the tile's record
                    float *rec = split ? chunk_record(a, blockIdx.x, g.slot) : nullptr;
                    // where the row goes, in elements; -1: nowhere
                    const long long row_at =
                        !valid || piece != 0 ? -1
                        : split ? 2 * a.rec_rows + (long long)m * HD
                                : ((long long)(g.r0 + rel) * a.n_qh + cur->heads.first + head_r) * HD;
                    const float inv = split ? 1.0f : 1.0f / sum;
                    if (split && row_at >= 0) {
                        rec[2 * m] = m_ref * c;
                        rec[2 * m + 1] = sum;
                    }
                    float any = 0.0f;  // NaN once a value is NaN or infinite
#pragma unroll 1
                    for (int k = 0; k < HD; k += 32) {
                        float v[32];
                        ct_ld32(to + k, v);
                        ct_wait_ld();
                        if (turns && steps1) {
                            float v1[32];
                            ct_ld32(to + HD + k, v1);
                            ct_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = v[e] * f0 + v1[e] * f1;
                        }
                        if (PARTS == 3) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float mid = __shfl_down_sync(0xffffffffu, v[e], RPW);
                                const float lo = __shfl_down_sync(0xffffffffu, v[e], 2 * RPW);
                                v[e] = (lo + mid) + v[e];
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e) any = fmaf(v[e], 0.0f, any);
                        if (row_at >= 0) {
                            if (PARTS == 3 || split) {
                                float4 *d = reinterpret_cast<float4 *>((split ? rec : static_cast<float *>(a.out)) + row_at + k);
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    d[e] = make_float4(v[4 * e] * inv, v[4 * e + 1] * inv, v[4 * e + 2] * inv,
                                                       v[4 * e + 3] * inv);
                            } else {
                                uint4 *d = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + row_at + k);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    d[e] = make_uint4(ct_pack(v[8 * e] * inv, v[8 * e + 1] * inv),
                                                      ct_pack(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                                                      ct_pack(v[8 * e + 4] * inv, v[8 * e + 5] * inv),
                                                      ct_pack(v[8 * e + 6] * inv, v[8 * e + 7] * inv));
                            }
                        }
                        __syncwarp();
                    }
                    if (row_at >= 0 && ((any != any && sum > 0.0f) || notes)) {
                        // rare: columns with infinities or NaN, put right where they went
                        void *to_mem = split ? static_cast<void *>(rec) : a.out;
                        const int dt = split ? DS_F32 : a.q_dtype;
                        for (int d = 0; d < HD; ++d) {
                            float x = load_as(to_mem, row_at + d, dt);
                            if (x != x && sum > 0.0f)  // (0: every score is -inf, the row is NaN)
                                x = ct_infinite(a, g.seq, cur->heads.kv, d, g.b0 * kCtStep,
                                                min(g.b1 * kCtStep, g.pos0 + rel + 1));
                            if (notes) x += ct_noted(sh.note[par][d], rel);
                            store_as(to_mem, row_at + d, dt, x);
                        }
                    }
                    __syncwarp();
                }
                if (notes) {
                    // Read: one warp clears them for the segment after the next
                    // when all readers are through.  (Counted and with a limit,
                    // not at a hardware barrier: after a wait has given up, the
                    // warps may have read different answers.)
                    __threadfence_block();
                    __syncwarp();
                    if (lane == 0) atomicAdd(&sh.readers[par], 1);
                    if (warp == 0) {
                        ct_wait_count(&sh.readers[par], turns ? 4 : 8, dead, a.err);
                        __syncwarp();
                        for (int d = lane; d < HD; d += 32) sh.note[par][d] = kCtNoNote;
                        if (lane == 0) sh.noted[par] = sh.readers[par] = 0;
                        __threadfence_block();
                        __syncwarp();
                    }
                }
            }
            if (turns) named_sync(1, 256);  // part 0 has read part 1's accumulator, maxima and notes
            if (steps0) ++oc0;
            if (steps1) ++oc1;
            __syncwarp();
            if (lane == 0) {
                seg_done(seg);
                atomicAdd(&sh.left[w], 1);
            }
        }
    }
    if (flags) flag_error(a.err, flags);
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

bool chunk_tc_supported(const ChunkArgs &a) {
    return a.kv_dtype == DS_BF16 && (a.hd == 64 || a.hd == 128) && a.bt % 8 == 0;
}

template <int HD, int PARTS>
static cudaError_t launch_ct(const ChunkArgs &a, const CtMaps &maps, int grid, cudaStream_t stream) {
    static std::atomic<unsigned long long> ready{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load() & bit)) {
        e = cudaFuncSetAttribute((const void *)chunk_tc_kernel<HD, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)CtCfg<HD, PARTS>::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(bit);
    }
    return launch_ex(chunk_tc_kernel<HD, PARTS>, dim3(grid), dim3(kCtThreads), CtCfg<HD, PARTS>::kSmem, stream, true,
                     a, maps);
}

cudaError_t launch_chunk_tc(ChunkArgs &a, int *grid, cudaStream_t stream) {
    static_assert(CtCfg<128, 1>::kSmem <= kCtSmemLimit && CtCfg<128, 3>::kSmem <= kCtSmemLimit, "shared memory");
    a.q_dtype == DS_BF16 ? chunk_tile_shape(a, 128, 2) : chunk_tile_shape(a, 40, 1);
    a.step = kCtStep;
    a.half_tokens = a.q_dtype == DS_BF16 ? a.tile_tokens / 2 : a.tile_tokens;
    a.w_half = kCtWeightTurns;
    a.w_full = kCtWeightShared;
    a.tile_cost = a.q_dtype == DS_BF16 ? kCtTileCost : kCtTileCostF32;
    a.piece = kCtPiece;
    *grid = sm_count();
    CtMaps maps = {};
    maps.box_rows = 8;
    while (maps.box_rows < 128 && a.bt % (2 * maps.box_rows) == 0) maps.box_rows *= 2;
    const long long dims[3] = {64, a.cache_rows, (long long)a.n_kvh * a.hd / 64};
    const long long strides[2] = {(long long)a.n_kvh * a.hd * 2, 128};
    const int box[3] = {64, maps.box_rows, 1};
    if (!encode_tiled_3d(&maps.k, a.k_cache, DS_BF16, dims, strides, box, true) ||
        !encode_tiled_3d(&maps.v, a.v_cache, DS_BF16, dims, strides, box, true))
        return cudaErrorInvalidValue;
    if (a.q_dtype == DS_BF16) {
        const long long qdims[3] = {a.hd, a.n_qh, a.n_rows};
        const long long qstrides[2] = {(long long)a.hd * 2, (long long)a.n_qh * a.hd * 2};
        const int qbox[3] = {64, a.part_heads, a.tile_tokens / 2};
        if (!encode_tiled_3d(&maps.q, a.q, DS_BF16, qdims, qstrides, qbox, true)) return cudaErrorInvalidValue;
    }
    if (a.hd == 128)
        return a.q_dtype == DS_BF16 ? launch_ct<128, 1>(a, maps, *grid, stream) : launch_ct<128, 3>(a, maps, *grid, stream);
    return a.q_dtype == DS_BF16 ? launch_ct<64, 1>(a, maps, *grid, stream) : launch_ct<64, 3>(a, maps, *grid, stream);
}

}  // namespace ds
