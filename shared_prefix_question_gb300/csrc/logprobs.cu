// logprobs.cu -- log probabilities of given tokens, entropy and top alternatives over the whole
// vocabulary (blink_token_logprobs), without writing the logits.
//
// Mathematics.  With c = log2(e) / T and the raw product z = h . w, a part of the vocabulary is
// summarised by m = max z, s = sum 2^x and u = sum 2^x x, x = c (z - m); two parts merge by
// rescaling to the larger m:  s = a s1 + b s2,  u = a (u1 + s1 d1) + b (u2 + s2 d2) with
// d1 = c (m1 - m), a = 2^d1 and so on.  Then lse = ln2 (c m + log2 s), entropy = ln2 (log2 s - u / s),
// whose two terms are both small when the distribution is peaked, and a log probability is
// ln2 (c (z - m) - log2 s).  The difference is taken before the scaling: c z itself may have lost its
// digits (at T = 10^-6 its last place is a whole unit), and a fused c z - c m leaves what the rounding of c m
// did, 2^80 at T = 10^-30.  It is one instruction more for two logits.  Alternatives and the target
// keep the raw z, which the temperature does not reorder.
//
// Work.  Hidden rows are the M rows of the product (a tensor-memory lane, so a thread, holds one row
// and folds the logits into its state without any exchange), vocabulary rows the N columns, 256 per
// tile.  Up to 128 rows one block works alone (M = 128: the call is bound by reading the unembedding
// once, and the tensor time of 128 rows stays below that); above, a pair of blocks works on 256
// rows (cta_group::2, M = 256, N = 256: each block loads half of the vocabulary tile, so a byte
// staged in shared memory feeds twice the products).
// Rows beyond one tile run in passes of up to a few row tiles; within a pass every row tile is cut
// into the same vocabulary chunks, and the workers on one chunk run side by side so that the
// unembedding comes from HBM once per pass.  A worker carries its rows' state in registers through its
// chunk and writes it once; the merge launch joins the chunks of a row.
//
// Precision.  The tensor core's fp32 accumulator truncates: over a sum of H / 16 steps the loss grows
// with H (measured against 64 bits, logits of 12: 2.7e-6 of the logit at H = 2560, 5.4e-6 at 5120, and
// four times that where all products have one sign).  So a product runs over at most 512 of H only (256 for few rows),
// and the row's thread adds the parts in registers, rounded to nearest: the loss stays that of one part
// whatever H is.
//
// Roles (384 threads a block): warps 0-7 the states (threads t and t + 128 share row t, 128 of a tile's
// columns each, held in registers: 232 a thread, 40 for the other warps), warp 8 TMA producer, warp 9
// MMA issuer (of the even block).
// Tensor memory: two accumulators of 256 columns, so one part is read out and folded while the next is
// multiplied.  Warps 10 and 11 keep the rows' bounds (below) up to date in shared memory.
//
// What bounds it.  Up to 128 rows the unembedding is read once: 151936 x 2560 takes 122 us for one row or 64
// (6.4 TB/s), 127 with the merge.  Above, the tensor core: 512 rows of 5120 take 490 us alone (82 % busy), 4096 rows
// of 2560 1.75 ms (88 %); in a row, where the power limit lowers the clock, 570 us and 2.05 ms.
//
// Lists.  A thread's alternatives are in registers, sorted.  While the tensor core reads its operands
// from shared memory, a dependent shared-memory access of another warp takes hundreds of cycles:
// lists there cost 1,500 cycles per product inserted, whichever way they were worked on.
#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace blink {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxTop = BLINK_MAX_TOP_TOKENS;
constexpr int kVocabTile = 256;
constexpr int kBlockRows = 128;
constexpr int kThreadsLP = 384;
constexpr int kRegsNeeded = 256 * 232 + 128 * 40;
constexpr int kStateWarps = 8;
constexpr int kProducerLP = 8, kIssuerLP = 9;
constexpr int kHalves = 2;      // threads that share a row
constexpr int kHalfCols = kVocabTile / kHalves;
// At most this many 64-wide blocks of H per product.  Measured at H = 2560, entropy against 64 bits: 1.5e-6
// off with 10 blocks, 0.95e-6 with 8, 0.7e-6 with 6, 0.4e-6 with 4; pairs take 4 % longer with 6 than with 8,
// and 1 % less with 10; one block with 64 rows takes 3 % longer with 4.  Up to 32 rows only a quarter of the
// threads have a row and the shorter parts cost 0.5 %.
constexpr int kPartBlocks = 8, kPartBlocksFew = 4;
constexpr int kFewRows = 32;
// 64-wide blocks of H per stage of the ring.  A pair's issuer loses some 120 cycles of the tensor core at every
// barrier it waits for: with two blocks a stage 4096 tokens take 1.73 ms instead of 1.82.  One block alone
// waits for memory, and more, smaller stages suit it.
constexpr int kStageBlocksOne = 1, kStageBlocksPair = 2;  // 64-wide blocks of H per stage of the ring
constexpr int kNoToken = 0x7FFFFFFF;
constexpr int kMaxWorkers = 160;
constexpr int kLaunchRows = 8192;  // rows of one launch: bounds the workspace (86 MB with 32 alternatives, and 16 KB x H of rows)
constexpr int kMaxStages = 8;
constexpr int kSmemMax = 227 * 1024;
constexpr int kBatchCols = 8;  // columns searched for alternatives at a time

// How the rows and the vocabulary are shared out (computed on the host, walked by every role).
struct LogprobPlan {
    int blocks_per_worker;  // 1, or 2 (a pair)
    int workers;
    int row_tiles, tile_rows;  // rows per tile: 128 per block
    int vocab_tiles;
    int group;                // row tiles of a full pass
    int full_passes, chunks;  // vocabulary chunks of a full pass
    int rest, rest_chunks;    // row tiles and chunks of the last, smaller pass (rest = 0: none)
    __host__ __device__ int passes() const { return full_passes + (rest > 0 ? 1 : 0); }
    __host__ __device__ int tiles_of(int pass) const { return pass < full_passes ? group : rest; }
    __host__ __device__ int chunks_of(int pass) const { return pass < full_passes ? chunks : rest_chunks; }
    __host__ __device__ int64_t first_cell(int pass) const
    {
        return static_cast<int64_t>(pass) * group * chunks * kHalves * tile_rows;
    }
    __host__ __device__ int64_t cells() const
    {
        return first_cell(full_passes) + static_cast<int64_t>(rest) * rest_chunks * kHalves * tile_rows;
    }
};

// A worker's part of one pass: vocabulary tiles [v0, v1) of one row tile, and the cell its states go to.
struct Share {
    int row_tile, chunk, v0, v1;
    int64_t cell, half_step;  // of the first half's states; from there to the second half's
    bool any;
};

__host__ __device__ inline Share share_of(const LogprobPlan &p, int pass, int worker)
{
    Share s;
    const int g = p.tiles_of(pass), nc = p.chunks_of(pass);
    s.any = worker < g * nc;
    const int t = worker % g;
    // chunks differ by one tile; each pass deals them to the workers from another place
    const int chunk = (worker / g + pass * 7) % nc;
    s.row_tile = pass * p.group + t;
    s.chunk = chunk;
    s.v0 = static_cast<int>(static_cast<int64_t>(p.vocab_tiles) * chunk / nc);
    s.v1 = static_cast<int>(static_cast<int64_t>(p.vocab_tiles) * (chunk + 1) / nc);
    s.cell = p.first_cell(pass) + (static_cast<int64_t>(chunk) * kHalves * g + t) * p.tile_rows;
    s.half_step = static_cast<int64_t>(g) * p.tile_rows;
    return s;
}

// Row tiles per full pass: the count of 2..6 that leaves the fewest workers idle, the larger of
// equals (fewer passes over the unembedding); all of them when there are no more than that.
int full_group(int workers)
{
    int best = 1, best_used = 0;
    for (int g = 2; g <= 6 && g <= workers; ++g) {
        const int used = workers / g * g;
        if (used >= best_used) best = g, best_used = used;
    }
    return best;
}

LogprobPlan make_plan(int n, int V, int sms)
{
    LogprobPlan p{};
    p.blocks_per_worker = n > kBlockRows ? 2 : 1;
    p.tile_rows = kBlockRows * p.blocks_per_worker;
    p.workers = sms / p.blocks_per_worker;
    if (p.workers < 1) p.workers = 1;
    if (p.workers > kMaxWorkers) p.workers = kMaxWorkers;
    p.row_tiles = (n + p.tile_rows - 1) / p.tile_rows;
    p.vocab_tiles = (V + kVocabTile - 1) / kVocabTile;
    auto chunks_for = [&](int tiles) {
        const int c = p.workers / tiles;
        return c < p.vocab_tiles ? c : p.vocab_tiles;
    };
    const int best = full_group(p.workers);
    p.group = best < p.row_tiles ? best : p.row_tiles;
    p.full_passes = p.row_tiles / p.group;
    p.chunks = chunks_for(p.group);
    p.rest = p.row_tiles - p.full_passes * p.group;
    p.rest_chunks = p.rest > 0 ? chunks_for(p.rest) : 0;
    return p;
}

struct LogprobArgs {
    LogprobPlan plan;
    int V, H, n, top;
    int a_rows;  // rows of one copy of hidden states (a multiple of 8, at most 128)
    const int32_t *row_idx;
    int hidden_rows;
    const int32_t *targets;
    float c;       // log2(e) / T
    float4 *stat;  // [cells]: m (a raw product), s, u, target's raw product (NaN: not in this part)
    int2 *best;    // [cells][top]: raw product (as bits) and token, descending
    float *logprob, *entropy, *lse, *top_lp;
    int32_t *top_ids;
    int *err;
    uint32_t *bounds;  // [n][kMaxTop]: see RowBound
    int prepared;      // a launch before gathered the hidden rows and cleared the bounds
    // shared memory: the stages, with alternatives the rows' bounds, then the barriers
    int stages, block_bytes, a_bytes, bound_off, bar_off, smem_bytes;
};

// Divides the shared memory of a block: as many stages as fit.
void lay_out(LogprobArgs &a)
{
    const bool one = a.plan.blocks_per_worker == 1;
    a.a_rows = a.n < kBlockRows ? (a.n + 7) / 8 * 8 : kBlockRows;
    a.a_bytes = a.a_rows * 128;
    a.block_bytes = a.a_bytes + kVocabTile / (one ? 1 : 2) * 128;
    const int stage_bytes = a.block_bytes * (one ? kStageBlocksOne : kStageBlocksPair);
    const int bounds = a.top > 0 ? kBlockRows * static_cast<int>(sizeof(uint64_t)) : 0;
    a.stages = (kSmemMax - bounds - 256) / stage_bytes;
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    a.bound_off = a.stages * stage_bytes;
    a.bar_off = a.bound_off + bounds;
    a.smem_bytes = a.bar_off + 256;
}

// State of one row: running (m, s, u), the target's product, the row's bound as last read (+inf where
// the thread has no row) and the best products so far.  The list holds `top` entries in its last
// places; the places before them are +inf and never move.
template <int kTop>
struct RowState {
    float m, s, u, tz, bound;
    float v[kTop > 0 ? kTop : 1];
    int32_t id[kTop > 0 ? kTop : 1];
    __device__ __forceinline__ void clear(int top, bool has_row)
    {
        m = -INFINITY;
        s = u = 0.f;
        tz = __int_as_float(0x7FC00000);
        bound = has_row ? -INFINITY : INFINITY;
#pragma unroll
        for (int j = 0; j < kTop; ++j) {
            v[j] = j < kTop - top ? INFINITY : -INFINITY;
            id[j] = kNoToken;
        }
    }
    __device__ __forceinline__ float last() const { return v[kTop > 0 ? kTop - 1 : 0]; }
    // Tokens come in ascending id, so an equal product goes behind those already listed.  No entry
    // waits for another: the list is descending, so entry j moves one place down exactly when the one
    // before it is below z.  No change for a z that is not above the last.
    __device__ __forceinline__ void insert(float z, int32_t i)
    {
#pragma unroll
        for (int j = kTop - 1; j > 0; --j) {
            const bool here = z > v[j], shift = z > v[j - 1];
            v[j] = shift ? v[j - 1] : here ? z : v[j];
            id[j] = shift ? id[j - 1] : here ? i : id[j];
        }
        if (z > v[0]) v[0] = z, id[0] = i;
    }
};

__device__ __forceinline__ uint32_t order_of(float z)  // larger unsigned = larger z; 0 below every number
{
    const uint32_t b = __float_as_uint(z + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t o) { return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o); }

// A row's bound.  Each of kMaxTop words per row holds the largest product seen so far in its own share
// of the vocabulary (a thread's groups of 32 columns are dealt to the words), kept by every worker with
// atomic maxima.  So at least `top` products are no smaller than the top-th largest word, and a
// product below that is no alternative of the row and need not enter a list.  With 20 of 32 words
// about 31 products of the whole row are at or above it, where a thread's own list alone would let in
// its first 20, about half of the next 20 and so on.  How far the others have come varies from run to
// run, and with it what the lists hold, but not the best `top` of them: the result does not vary.

// The k-th largest (k = 1..32) of one word per lane.
__device__ __forceinline__ uint32_t kth_largest(uint32_t v, int k)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
        for (int o = size / 2; o > 0; o /= 2) {
            const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, v, o);
            const bool first = (lane & o) == 0, down = (lane & size) == 0;  // descending runs
            v = first == down ? max(v, other) : min(v, other);
        }
    }
    return __shfl_sync(0xFFFFFFFFu, v, k - 1);
}

// A looser bound that one thread reads by itself: the smallest of the first `top` words.
__device__ __forceinline__ float row_bound(const uint32_t *words, int top)
{
    uint32_t lo = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < kMaxTop; j += 4) {
        if (j < top) {
            const uint4 w = __ldcg(reinterpret_cast<const uint4 *>(words + j));
            lo = min(lo, w.x);
            if (j + 1 < top) lo = min(lo, w.y);
            if (j + 2 < top) lo = min(lo, w.z);
            if (j + 3 < top) lo = min(lo, w.w);
        }
    }
    return lo == 0u ? -INFINITY : of_order(lo);
}

// Where a row's bound is kept.
struct BoundPlace {
    uint32_t *words;  // of this thread's row
    uint32_t kept;    // as warps 10 and 11 last saw it: tag << 32 | order (shared address)
    int top, slot0, tag;
};

// The tag (pass + 1) and the order of a bound are one scalar of 8 bytes, which a reader sees whole: a bound never
// comes with the tag of another pass, whose row is another.  (Of a vector access each element is one by itself.)
__device__ __forceinline__ void publish_bound(uint32_t place, int tag, uint32_t order)
{
    const uint64_t word = static_cast<uint64_t>(static_cast<uint32_t>(tag)) << 32 | order;
    asm volatile("st.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(place), "l"(word) : "memory");
}

// 0: none yet in this pass.
__device__ __forceinline__ uint32_t published_bound(uint32_t place, int tag)
{
    uint64_t word;
    asm volatile("ld.relaxed.cta.shared::cta.b64 %0, [%1];" : "=l"(word) : "r"(place) : "memory");
    return static_cast<int>(word >> 32) == tag ? static_cast<uint32_t>(word) : 0u;
}

// The first of columns 8 b .. 8 b + 7 that is at least `least` and not in `done` (b the same in the warp).
__device__ __forceinline__ void next_candidate(const float (&z)[kHalfCols], int b, float least, uint32_t done, float &zc,
                                               int &jc)
{
    static_assert(kBatchCols == 8 && kHalfCols == 128, "sixteen batches of eight columns");
    zc = -INFINITY;
    jc = -1;
#define BLINK_SEARCH(B)                                                                     \
    case B:                                                                                 \
        _Pragma("unroll") for (int j = 7; j >= 0; --j) if (z[8 * B + j] >= least && !(done >> j & 1u)) \
            zc = z[8 * B + j], jc = j;                                                      \
        break;
    switch (b) {
        BLINK_SEARCH(0) BLINK_SEARCH(1) BLINK_SEARCH(2) BLINK_SEARCH(3) BLINK_SEARCH(4) BLINK_SEARCH(5)
        BLINK_SEARCH(6) BLINK_SEARCH(7) BLINK_SEARCH(8) BLINK_SEARCH(9) BLINK_SEARCH(10) BLINK_SEARCH(11)
        BLINK_SEARCH(12) BLINK_SEARCH(13) BLINK_SEARCH(14) BLINK_SEARCH(15)
    }
#undef BLINK_SEARCH
}

// Folds a row's logits of a tile, tokens id0 .. id0 + kHalfCols - 1, into its state.
template <int kTop>
__device__ __forceinline__ void fold_tile(RowState<kTop> &r, float (&z)[kHalfCols], int id0, int V, float c, int target,
                                          const BoundPlace &bp)
{
    constexpr int kBatches = kHalfCols / kBatchCols;
    const bool whole = id0 + kHalfCols <= V;
    if (!whole) {
#pragma unroll
        for (int j = 0; j < kHalfCols; ++j)
            if (id0 + j >= V) z[j] = -INFINITY;
    }
    float bmax[kBatches];  // of eight columns
#pragma unroll
    for (int b = 0; b < kBatches; ++b) {
        const float *y = z + 8 * b;
        bmax[b] = ptx::max3(ptx::max3(y[0], y[1], y[2]), ptx::max3(y[3], y[4], y[5]), fmaxf(y[6], y[7]));
    }
    float zmax = -INFINITY;
#pragma unroll
    for (int q = 0; q < kHalfCols / 32; ++q) {
        const float gmax = ptx::max3(bmax[4 * q], bmax[4 * q + 1], fmaxf(bmax[4 * q + 2], bmax[4 * q + 3]));
        zmax = fmaxf(zmax, gmax);
        if constexpr (kTop > 0) {
            if (gmax > r.bound) atomicMax(bp.words + bp.slot0 + q, order_of(gmax));
        }
    }
    if (zmax > r.m) {
        const float d = r.m == -INFINITY ? 0.f : (r.m - zmax) * c, f = ptx::ex2(d);
        r.u = f == 0.f ? 0.f : f * fmaf(r.s, d, r.u);  // s d may overflow
        r.s *= f;
        r.m = zmax;
    }
    const float nm = r.m == -INFINITY ? 0.f : -r.m;  // all NaN so far
    if (whole) {
        // two columns an instruction for all but the exp2
        const uint64_t cc = ptx::f32x2(c, c), mm = ptx::f32x2(nm, nm);
        uint64_t s0 = 0ull, s1 = 0ull, u0 = 0ull, u1 = 0ull;
#pragma unroll
        for (int j = 0; j < kHalfCols; j += 4) {
            const uint64_t x0 = ptx::mul_f32x2(ptx::add_f32x2(ptx::f32x2(z[j], z[j + 1]), mm), cc);
            const uint64_t x1 = ptx::mul_f32x2(ptx::add_f32x2(ptx::f32x2(z[j + 2], z[j + 3]), mm), cc);
            float a0, a1, a2, a3;
            ptx::f32x2_split(x0, a0, a1);
            ptx::f32x2_split(x1, a2, a3);
            const uint64_t e0 = ptx::f32x2(ptx::ex2(a0), ptx::ex2(a1)), e1 = ptx::f32x2(ptx::ex2(a2), ptx::ex2(a3));
            s0 = ptx::add_f32x2(s0, e0);
            s1 = ptx::add_f32x2(s1, e1);
            u0 = ptx::fma_f32x2(e0, x0, u0);
            u1 = ptx::fma_f32x2(e1, x1, u1);
        }
        float lo, hi;
        ptx::f32x2_split(ptx::add_f32x2(s0, s1), lo, hi);
        r.s += lo + hi;
        ptx::f32x2_split(ptx::add_f32x2(u0, u1), lo, hi);
        r.u += lo + hi;
    } else {
        float s0 = 0.f, u0 = 0.f;
#pragma unroll
        for (int j = 0; j < kHalfCols; ++j) {
            if (id0 + j < V) {
                const float x0 = (z[j] + nm) * c, e0 = ptx::ex2(x0);
                s0 += e0;
                u0 = fmaf(e0, x0, u0);
            }
        }
        r.s += s0;
        r.u += u0;
    }
    if (__any_sync(0xFFFFFFFFu, static_cast<uint32_t>(target - id0) < static_cast<uint32_t>(kHalfCols))) {
#pragma unroll
        for (int j = 0; j < kHalfCols; ++j)
            if (target == id0 + j) r.tz = z[j];
    }
    if constexpr (kTop > 0) {
        const uint32_t kept = published_bound(bp.kept, bp.tag);
        if (kept != 0u) r.bound = fmaxf(r.bound, of_order(kept));
        if (__any_sync(0xFFFFFFFFu, zmax > r.last() && zmax >= r.bound)) {
            if (r.bound == -INFINITY) r.bound = row_bound(bp.words, bp.top);  // the first tile
            uint32_t mine = 0u;  // this row's batches with a candidate
#pragma unroll
            for (int b = 0; b < kBatches; ++b)
                if (bmax[b] > r.last() && bmax[b] >= r.bound) mine |= 1u << b;
            // Batch by batch, every row takes its next candidate in each round.  One copy of the insertion: it
            // runs seldom (measured: for 1 to 2 batches of a warp's 16 in a tile, once the first tiles are
            // done), and a copy for every column would miss the instruction cache every time.
            uint32_t todo = __reduce_or_sync(0xFFFFFFFFu, mine);
            while (todo != 0u) {
                const int b = __ffs(todo) - 1;
                todo &= todo - 1;
                uint32_t done = 0u;
                while (true) {
                    float zc;
                    int jc;
                    next_candidate(z, b, fmaxf(r.bound, r.last()), done, zc, jc);  // one equal to the last changes nothing
                    if (!__any_sync(0xFFFFFFFFu, jc >= 0)) break;
                    if (jc >= 0) done |= 1u << jc;
                    r.insert(zc, id0 + 8 * b + jc);
                }
            }
        }
    }
}

template <int kCtas, int kTop>
__global__ void __launch_bounds__(kThreadsLP, 1)
    logprob_kernel(const __grid_constant__ CUtensorMap tm_h, const __grid_constant__ CUtensorMap tm_w, const LogprobArgs a)
{
    constexpr bool kList = kTop > 0;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + a.bar_off);
    uint64_t *full = bars, *empty = bars + kMaxStages;
    uint64_t *acc_full = bars + 2 * kMaxStages, *acc_empty = acc_full + 2;
    uint64_t *mma_done = acc_empty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + 1);
    int *abort_word = reinterpret_cast<int *>(tmem_holder + 1);
    volatile int *abort_flag = abort_word;
    volatile int *turn = abort_word + 1;  // pass + 1 the states are at; 0 before, -1 after
    const uint32_t kept_bounds = ptx::smem_u32(smem + a.bound_off);  // [128]: see publish_bound
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kCtas == 2 ? ptx::cluster_rank() : 0u;
    const int worker = blockIdx.x / kCtas;
    const int passes = a.plan.passes();
    const int k_blocks = (a.H + 63) / 64;
    constexpr int kStageBlocks = kCtas == 1 ? kStageBlocksOne : kStageBlocksPair;
    const int most = kCtas == 1 && a.n <= kFewRows ? kPartBlocksFew : kPartBlocks;
    const int n_parts = (k_blocks + most - 1) / most;
    const int part_blocks = ((k_blocks + n_parts - 1) / n_parts + kStageBlocks - 1) / kStageBlocks * kStageBlocks;
    const bool aligned = (ptx::smem_u32(smem) & 1023u) == 0;  // the swizzled tiles need it
    if (!aligned && threadIdx.x == 0) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);

    if (warp == kProducerLP && lane == 0) {
        for (int i = 0; i < a.stages; ++i) {
            ptx::mbar_init(full + i, 1);
            ptx::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(acc_full + i, 1);
            ptx::mbar_init(acc_empty + i, kStateWarps * kCtas);
        }
        ptx::mbar_init(mma_done, 1);
        ptx::fence_mbar_init();
        *abort_word = aligned ? 0 : 1;
        *turn = 0;
        ptx::tma_prefetch_desc(&tm_h);
        ptx::tma_prefetch_desc(&tm_w);
    }
    if (kList && threadIdx.x < kBlockRows)
        reinterpret_cast<uint64_t *>(smem + a.bound_off)[threadIdx.x] = 0ull;
    if (warp == 0) {
        if constexpr (kCtas == 2) {
            ptx::tmem_alloc_pair(tmem_holder, 512);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(tmem_holder, 512);
            ptx::tmem_relinquish();
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    if constexpr (kCtas == 2)
        ptx::cluster_sync();
    else
        __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    // Registers by role: 128 threads at 40 and 256 at 232 are the 384 at 168 of the launch.
    if (warp >= kStateWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (!aligned) {
        // nothing was started: straight to the end
    } else if (warp == kProducerLP) {
        if (lane == 0) {
            const uint32_t bytes = static_cast<uint32_t>(a.block_bytes) * kCtas;  // of both blocks, counted on the even one
            int it = 0, st = 0;
            uint32_t ph = 1u;
            bool ok = true, waited = a.prepared == 0;
            for (int ps = 0; ok && ps < passes; ++ps) {
                const Share sh = share_of(a.plan, ps, worker);
                if (!sh.any) continue;
                const int row0 = sh.row_tile * a.plan.tile_rows + static_cast<int>(rank) * kBlockRows;
                for (int vt = sh.v0; ok && vt < sh.v1; ++vt) {
                    const int col0 = vt * kVocabTile + static_cast<int>(rank) * (kVocabTile / kCtas);
                    for (int k0 = 0; k0 < k_blocks; k0 += kStageBlocks, ++it) {
                        if (!(ok = ptx::mbar_wait(empty + st, ph, abort_flag, a.err, BLINK_DEVICE_TIMEOUT))) break;
                        const int kn = min(kStageBlocks, k_blocks - k0);
                        const uint32_t bar = kCtas == 2 ? ptx::map_to_rank(ptx::smem_u32(full + st), 0) : 0u;
                        if (rank == 0) ptx::mbar_arrive_expect_tx(full + st, bytes * kn);
#pragma unroll
                        for (int kb = 0; kb < kStageBlocks; ++kb) {
                            if (kb >= kn) break;
                            uint8_t *dst = smem + (st * kStageBlocks + kb) * a.block_bytes;
                            if constexpr (kCtas == 2) {
                                ptx::tma_load_3d_pair(dst + a.a_bytes, &tm_w, (k0 + kb) * 64, col0, 0, bar);
                                if (!waited) ptx::grid_dep_wait(), waited = true;
                                ptx::tma_load_3d_pair(dst, &tm_h, (k0 + kb) * 64, row0, 0, bar);
                            } else {
                                ptx::tma_load_3d(dst + a.a_bytes, &tm_w, (k0 + kb) * 64, col0, 0, full + st);
                                if (!waited) ptx::grid_dep_wait(), waited = true;
                                ptx::tma_load_3d(dst, &tm_h, (k0 + kb) * 64, row0, 0, full + st);
                            }
                        }
                        if (++st == a.stages) st = 0, ph ^= 1u;
                    }
                }
            }
            ptx::grid_launch_dependents();
            // Every copy issued must have landed before a block of the pair may exit; they are counted
            // on the even block, which the other waits for at the cluster barrier below.
            if (rank == 0) {
                volatile int no_abort = 0;
                for (int n = it > a.stages ? it - a.stages : 0; n < it; ++n, no_abort = 0)
                    ptx::mbar_wait(full + n % a.stages, (n / a.stages) & 1, &no_abort, a.err, BLINK_DEVICE_TIMEOUT);
            }
        }
    } else if (warp == kIssuerLP) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = ptx::idesc_bf16_f32(kBlockRows * kCtas, kVocabTile, false);
            const uint64_t desc0 = ptx::smem_desc_sw128(ptx::smem_u32(smem), 16, 1024);  // in units of 16 bytes
            const uint32_t block16 = static_cast<uint32_t>(a.block_bytes) >> 4, a16 = static_cast<uint32_t>(a.a_bytes) >> 4;
            int st = 0, part = 0;
            uint32_t ph = 0u;
            bool ok = true;
            for (int ps = 0; ok && ps < passes; ++ps) {
                const Share sh = share_of(a.plan, ps, worker);
                if (!sh.any) continue;
                for (int vt = sh.v0; ok && vt < sh.v1; ++vt) {
                    for (int k0 = 0; ok && k0 < k_blocks; k0 += part_blocks, ++part) {
                        const int buf = part & 1;
                        if (!(ok = ptx::mbar_wait(acc_empty + buf, ((part >> 1) & 1) ^ 1, abort_flag, a.err,
                                                  BLINK_DEVICE_TIMEOUT)))
                            break;
                        ptx::tc_fence_after();
                        const uint32_t d = tmem + buf * kVocabTile;
                        const int kn = min(part_blocks, k_blocks - k0);
                        for (int kb = 0; kb < kn; kb += kStageBlocks) {
                            if (!(ok = ptx::mbar_wait(full + st, ph, abort_flag, a.err, BLINK_DEVICE_TIMEOUT))) break;
                            ptx::tc_fence_after();
                            const uint64_t ad = desc0 + st * kStageBlocks * block16, bd = ad + a16;
                            if constexpr (kCtas == 2) {
                                ptx::mma_ss_pair_x4(d, ad, bd, idesc, kb > 0);
                                if (kb + 1 < kn) ptx::mma_ss_pair_x4(d, ad + block16, bd + block16, idesc, 1u);
                                ptx::mma_commit_pair(empty + st);
                            } else {
                                ptx::mma_ss_x4(d, ad, bd, idesc, kb > 0);
                                ptx::mma_commit(empty + st);
                            }
                            if (++st == a.stages) st = 0, ph ^= 1u;
                        }
                        if (!ok) break;
                        if constexpr (kCtas == 2)
                            ptx::mma_commit_pair(acc_full + buf);
                        else
                            ptx::mma_commit(acc_full + buf);
                    }
                }
            }
            // every product issued must be complete before tensor memory is released
            if constexpr (kCtas == 2)
                ptx::mma_commit_pair(mma_done);
            else
                ptx::mma_commit(mma_done);
            volatile int no_abort = 0;
            ptx::mbar_wait(mma_done, 0, &no_abort, a.err, BLINK_DEVICE_TIMEOUT);
        }
    } else if (warp < kStateWarps) {
        // ------------------------------------------------------------ states: a row per two threads
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int half = warp >> 2, lane_row = (warp & 3) * 32 + lane;
        const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * kHalfCols;
        const float c = a.c;
        BoundPlace bp;
        bp.top = a.top;
        bp.kept = kept_bounds + lane_row * 8;
        if (kList) ptx::grid_dep_wait();  // the bounds have been cleared
        int part = 0;
        bool ok = true;
        for (int ps = 0; ok && ps < passes; ++ps) {
            const Share sh = share_of(a.plan, ps, worker);
            if (!sh.any) continue;
            const int row_w = sh.row_tile * a.plan.tile_rows + static_cast<int>(rank) * kBlockRows + (warp & 3) * 32;
            const int row = row_w + lane;
            const bool live = row_w < a.n;  // of the warp: it has rows at all
            const int target = a.targets && row < a.n ? __ldg(a.targets + row) : -1;
            RowState<kTop> r;
            r.clear(a.top, row < a.n);
            if (kList) {
                bp.words = a.bounds + static_cast<int64_t>(min(row, a.n - 1)) * kMaxTop;
                bp.slot0 = ((sh.chunk * kHalves + half) * (kHalfCols / 32)) % kMaxTop;
                bp.tag = ps + 1;
                if (threadIdx.x == 0) *turn = ps + 1;
            }
            for (int vt = sh.v0; vt < sh.v1; ++vt) {
                float z[kHalfCols];
                for (int k0 = 0; k0 < k_blocks; k0 += part_blocks, ++part) {
                    const int buf = part & 1;
                    if (!(ok = ptx::mbar_wait_warp(acc_full + buf, (part >> 1) & 1, abort_flag, a.err,
                                                   BLINK_DEVICE_TIMEOUT)))
                        break;
                    ptx::tc_fence_after();
                    if (live) {
                        const bool add = k0 > 0;
#pragma unroll
                        for (int q = 0; q < kHalfCols / 32; ++q) {
                            uint32_t raw[32];
                            ptx::tmem_ld32(trow + buf * kVocabTile + q * 32, raw);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const float x = __uint_as_float(raw[j]);
                                z[q * 32 + j] = add ? z[q * 32 + j] + x : x;
                            }
                        }
                    }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (kCtas == 2)
                            ptx::mbar_arrive_cluster(ptx::map_to_rank(ptx::smem_u32(acc_empty + buf), 0));
                        else
                            ptx::mbar_arrive(acc_empty + buf);
                    }
                }
                if (!ok) break;
                const int first_id = vt * kVocabTile + half * kHalfCols;
                if (live && first_id < a.V)
                    fold_tile<kTop>(r, z, first_id, a.V, c, target, bp);
            }
            if (!ok) break;
            if (row < a.n) {
                const int64_t cell = sh.cell + half * sh.half_step + static_cast<int>(rank) * kBlockRows + lane_row;
                a.stat[cell] = make_float4(r.m, r.s, r.u, r.tz);
#pragma unroll
                for (int j = 0; j < kTop; ++j) {
                    const int o = j - (kTop - a.top);
                    if (o >= 0) a.best[cell * a.top + o] = make_int2(__float_as_int(r.v[j]), r.id[j]);
                }
            }
        }
        if (threadIdx.x == 0) *turn = -1;
    } else if (kList) {
        // ------------------------------------------------------------ bounds: warps 10 and 11, 64 rows each
        // Reads the words of the rows that the states are at, again and again, until they are done.  A value
        // that comes late is only looser.  The states change *turn at any time, so lane 0 reads it for the
        // whole warp: kth_largest needs all lanes, at the same rows.
        ptx::grid_dep_wait();
        constexpr unsigned kAll = 0xFFFFFFFFu;
        const auto still_at = [&](int now) { return __shfl_sync(kAll, lane == 0 ? *turn : 0, 0) == now; };
        int seen = 0;
        uint64_t since = ptx::globaltimer_ns();
        while (true) {
            int now = 0;
            if (lane == 0) {
                now = *turn;
                if (now != seen) {
                    seen = now;
                    since = ptx::globaltimer_ns();
                } else if (ptx::globaltimer_ns() - since > 10000000000ull) {
                    now = -1;  // the states' own waits end long before
                }
                if (*abort_flag) now = -1;
            }
            now = __shfl_sync(kAll, now, 0);
            if (now < 0) break;
            if (now > 0) {
                const Share sh = share_of(a.plan, now - 1, worker);
                const int first = (warp - 10) * 64;
                const int row0 = sh.row_tile * a.plan.tile_rows + static_cast<int>(rank) * kBlockRows + first;
                for (int i = 0; i < 64 && row0 + i < a.n && still_at(now); i += 4) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = row0 + i + j < a.n ? __ldcg(a.bounds + static_cast<int64_t>(row0 + i + j) * kMaxTop + lane) : 0u;
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = kth_largest(w[j], a.top);
                    if (lane < 4) {
                        const uint32_t b = lane == 0 ? w[0] : lane == 1 ? w[1] : lane == 2 ? w[2] : w[3];
                        publish_bound(kept_bounds + (first + i + lane) * 8, now, b);
                    }
                    __syncwarp();
                }
            }
            if (still_at(now)) __nanosleep(500);
            __syncwarp();
        }
        __syncwarp();
    }
    __syncwarp();
    if (aligned && rank == 1 && warp == 0 && lane == 0) {
        // the last commit arrives on this block's barrier too: not to leave before it has
        volatile int no_abort = 0;
        ptx::mbar_wait(mma_done, 0, &no_abort, a.err, BLINK_DEVICE_TIMEOUT);
    }
    __syncwarp();
    ptx::tc_fence_before();
    if constexpr (kCtas == 2)
        ptx::cluster_sync();
    else
        __syncthreads();
    ptx::tc_fence_after();
    if (warp == 0) {
        if constexpr (kCtas == 2)
            ptx::tmem_dealloc_pair(tmem, 512);
        else
            ptx::tmem_dealloc(tmem, 512);
    }
}

// What the products need first: hidden rows of an index list gathered into consecutive rows (a row
// outside the tensor: zeros), and the rows' bounds cleared.
__global__ void __launch_bounds__(256) logprob_prepare_kernel(const uint4 *__restrict__ hidden, int64_t stride, int hidden_rows,
                                                              const int32_t *__restrict__ idx, int64_t pieces,
                                                              int row_pieces, uint4 *__restrict__ dst,
                                                              uint4 *__restrict__ bounds, int64_t bound_pieces)
{
    ptx::grid_launch_dependents();
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256, t0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    for (int64_t t = t0; t < bound_pieces; t += step) bounds[t] = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t t = t0; t < pieces; t += step) {
        const int r = static_cast<int>(t / row_pieces), p = static_cast<int>(t - static_cast<int64_t>(r) * row_pieces);
        const int hr = __ldg(idx + r);
        dst[t] = hr >= 0 && hr < hidden_rows ? __ldg(hidden + hr * stride + p) : make_uint4(0u, 0u, 0u, 0u);
    }
}

constexpr int kMaxLists = kMaxWorkers * kHalves;
constexpr int kWideRow = kMaxLists;  // threads of a row with many parts: one per part
constexpr int kMaxCand = 256;

// A listed product as one number: larger is better (larger product, then lower token); 0: none.
__device__ __forceinline__ unsigned long long rank_key(int2 e)
{
    if (e.y == kNoToken) return 0ull;
    return static_cast<unsigned long long>(order_of(__int_as_float(e.x))) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(e.y));
}

template <int kRowThreads>
__device__ __forceinline__ void row_sync()
{
    if constexpr (kRowThreads == 32)
        __syncwarp();
    else
        __syncthreads();
}

// Joins the parts of a row: kRowThreads threads a row, a warp where there are at most 64 parts, else
// one thread per part.  Only listed products at or above the row's bound can be among the best
// `top`: a few dozen, which are collected and ranked by counting.
template <int kRowThreads>
__global__ void __launch_bounds__(kRowThreads == 32 ? 128 : kRowThreads) logprob_merge_kernel(const LogprobArgs a)
{
    constexpr int kRows = kRowThreads == 32 ? 4 : 1, kWarps = kRowThreads / 32;
    constexpr int kMine = kRowThreads == 32 ? 2 : 1;
    __shared__ unsigned long long cand_all[kRows][kMaxCand];
    __shared__ unsigned long long best_all[kWarps];
    __shared__ int count_all[kRows];
    __shared__ float4 red[kWarps];
    const int sub = threadIdx.x / kRowThreads, t = threadIdx.x % kRowThreads;
    const int warp = t >> 5, lane = t & 31;
    const int r = blockIdx.x * kRows + sub;
    ptx::grid_dep_wait();
    if (r >= a.n) return;  // a whole warp, or the whole block
    unsigned long long *cand = cand_all[sub];
    const int rt = r / a.plan.tile_rows;
    const int pass = min(rt / a.plan.group, a.plan.passes() - 1);
    const int g = a.plan.tiles_of(pass), lists = a.plan.chunks_of(pass) * kHalves;
    const int64_t cell0 = a.plan.first_cell(pass) + static_cast<int64_t>(rt - pass * a.plan.group) * a.plan.tile_rows +
                          r % a.plan.tile_rows;
    const int64_t step = static_cast<int64_t>(g) * a.plan.tile_rows;
    const int top = a.top;
    const float nan = __int_as_float(0x7FC00000);
    const int target = a.targets ? __ldg(a.targets + r) : -1;
    const int hr = a.row_idx ? __ldg(a.row_idx + r) : r;
    float4 st[kMine];
    int2 head[kMine];
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
        const int l = t + q * kRowThreads;
        st[q] = l < lists ? __ldcg(a.stat + cell0 + l * step) : make_float4(-INFINITY, 0.f, 0.f, nan);
        head[q] = l < lists && top > 0 ? __ldcg(a.best + (cell0 + l * step) * top) : make_int2(0, kNoToken);
    }
    uint32_t word = top > 0 ? __ldcg(a.bounds + static_cast<int64_t>(r) * kMaxTop + lane) : 0u;
    if (t == 0) count_all[sub] = 0;

    float m = -INFINITY, tz = -INFINITY;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
        m = fmaxf(m, st[q].x);
        tz = fmaxf(tz, st[q].w);  // NaN in every part but the target's
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        tz = fmaxf(tz, __shfl_xor_sync(0xFFFFFFFFu, tz, o));
    }
    float s = 0.f, u = 0.f;
    auto join = [&](float pm, float ps, float pu) {
        const float d = pm == -INFINITY ? 0.f : (pm - m) * a.c, f = exp2f(d);  // an empty part, or one of NaN alone
        s = fmaf(f, ps, s);
        if (f != 0.f) u = fmaf(f, fmaf(ps, d, pu), u);  // s d may overflow
    };
#pragma unroll
    for (int q = 0; q < kMine; ++q) join(st[q].x, st[q].y, st[q].z);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
    }
    if constexpr (kRowThreads > 32) {  // the warps' parts, joined by every thread in the same order
        if (lane == 0) red[warp] = make_float4(m, s, u, tz);
        __syncthreads();
        m = -INFINITY;
        for (int w = 0; w < kWarps; ++w) {
            m = fmaxf(m, red[w].x);
            tz = fmaxf(tz, red[w].w);
        }
        s = u = 0.f;
        for (int w = 0; w < kWarps; ++w) join(red[w].x, red[w].y, red[w].z);
    }
    const bool bad = hr < 0 || hr >= a.hidden_rows;
    const float l2s = log2f(s);
    if (t == 0) {
        if (bad || target < -1 || target >= a.V) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
        if (a.lse) a.lse[r] = bad ? nan : fmaf(m, a.c, l2s) * kLn2;
        if (a.entropy) a.entropy[r] = bad ? nan : (l2s - u / s) * kLn2;
        if (a.logprob) a.logprob[r] = !bad && target >= 0 && target < a.V ? fmaf(tz - m, a.c, -l2s) * kLn2 : nan;
    }
    if (top == 0) return;

    auto put = [&](int place, unsigned long long key) {
        const bool no = bad || key == 0ull;
        a.top_ids[static_cast<int64_t>(r) * top + place] = no ? -1 : static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
        a.top_lp[static_cast<int64_t>(r) * top + place] =
            no ? nan : fmaf(of_order(static_cast<uint32_t>(key >> 32)) - m, a.c, -l2s) * kLn2;
    };
    const unsigned long long bound = static_cast<unsigned long long>(kth_largest(word, top)) << 32;
    row_sync<kRowThreads>();  // the count starts at zero
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
        const int l = t + q * kRowThreads;
        unsigned long long key = rank_key(head[q]);
        for (int j = 0; key != 0ull && key >= bound;) {
            const int at = atomicAdd(&count_all[sub], 1);
            if (at < kMaxCand) cand[at] = key;
            if (++j == top) break;
            key = rank_key(__ldcg(a.best + (cell0 + l * step) * top + j));
        }
    }
    row_sync<kRowThreads>();
    const int count = count_all[sub];
    if (count <= kMaxCand) {
        for (int e = t; e < count; e += kRowThreads) {
            const unsigned long long key = cand[e];
            int place = 0;
            for (int o = 0; o < count; ++o) place += cand[o] > key;  // tokens differ, so keys do
            if (place < top) put(place, key);
        }
        for (int k = count + t; k < top; k += kRowThreads) put(k, 0ull);  // NaN logits left fewer than `top`
        return;
    }
    // More products at or above the bound than the room (many equal ones): the best first entry,
    // `top` times.
    int next[kMine];
#pragma unroll
    for (int q = 0; q < kMine; ++q) next[q] = 0;
    for (int k = 0; k < top; ++k) {
        unsigned long long mine = 0ull;
#pragma unroll
        for (int q = 0; q < kMine; ++q) mine = max(mine, rank_key(head[q]));
        unsigned long long best = mine;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
        if constexpr (kRowThreads > 32) {
            if (lane == 0) best_all[warp] = best;
            __syncthreads();
            for (int w = 0; w < kWarps; ++w) best = max(best, best_all[w]);
            __syncthreads();
        }
        if (t == 0) put(k, best);
        if (mine == best && best != 0ull) {
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                if (rank_key(head[q]) == best) {
                    const int l = t + q * kRowThreads;
                    head[q] = ++next[q] < top ? __ldcg(a.best + (cell0 + l * step) * top + next[q]) : make_int2(0, kNoToken);
                }
            }
        }
    }
}

struct WsLayout {
    size_t stat, best, bounds, rows, total;
};

WsLayout ws_layout(int64_t n_cells, int n, int H, int top)
{
    WsLayout l{};
    const size_t cells = static_cast<size_t>(n_cells);
    l.stat = kHeaderBytes;
    l.best = l.stat + align_up(cells * sizeof(float4), 256);
    l.bounds = l.best + align_up(cells * top * sizeof(int2), 256);
    l.rows = l.bounds + (top > 0 ? static_cast<size_t>(n) * kMaxTop * sizeof(uint32_t) : 0);
    l.total = l.rows + align_up(static_cast<size_t>(n) * H * sizeof(uint16_t), 256);
    return l;
}

// No fewer cells than the plan of any launch of up to n rows has, and never fewer for more rows: a pass has at
// most a cell per worker and tile row (256 rows for each of two workers where pairs work), and no more
// than the row tiles and the vocabulary tiles make.  The plans' own counts go up and down with n, as
// the workers that a pass leaves idle do.
int64_t most_cells(int n, int V, int sms)
{
    const int blocks = sms < 2 * kMaxWorkers ? sms : 2 * kMaxWorkers;
    const int64_t row_tiles = (n + 2 * kBlockRows - 1) / (2 * kBlockRows), vocab_tiles = (V + kVocabTile - 1) / kVocabTile;
    const int workers = blocks / 2 < 1 ? 1 : blocks / 2 < kMaxWorkers ? blocks / 2 : kMaxWorkers;
    const int group = full_group(workers);
    const int64_t by_workers = (row_tiles + group - 1) / group * (blocks < 2 ? 2 : blocks), by_tiles = 2 * row_tiles * vocab_tiles;
    return (by_workers < by_tiles ? by_workers : by_tiles) * kHalves * kBlockRows;
}

// Bytes that serve every launch of a call of n rows, and those of a call of fewer.
size_t ws_bytes_needed(int n, int H, int V, int top, int sms)
{
    const int rows = n < kLaunchRows ? n : kLaunchRows;
    return ws_layout(most_cells(rows, V, sms > 0 ? sms : 1), rows, H, top).total;
}

// The sizes that workspaces are given out for.
bool ws_sizes_ok(int n, int H, int V, int top)
{
    return n >= 1 && n <= BLINK_MAX_INPUT_TOKENS && H >= 1 && H <= 32768 && V >= 1 && V <= (1 << 24) && top >= 0 && top <= kMaxTop;
}

int sm_count()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
}

template <int kCtas, int kTop>
cudaError_t launch_logprob(const CUtensorMap &tm_h, const CUtensorMap &tm_w, const LogprobArgs &a, cudaStream_t stream)
{
    auto kern = logprob_kernel<kCtas, kTop>;
    // The split of registers by role has to fit the registers of the launch: checked once.
    static const bool fits = [kern] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, kern) == cudaSuccess && fa.numRegs * kThreadsLP >= kRegsNeeded;
    }();
    if (!fits) return cudaErrorLaunchOutOfResources;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (kCtas > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = kCtas;
        attr[na].val.clusterDim.y = 1;
        attr[na++].val.clusterDim.z = 1;
    }
    if (a.prepared) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(a.plan.workers * kCtas));
    cfg.blockDim = dim3(kThreadsLP);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.smem_bytes);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(na);
    return cudaLaunchKernelEx(&cfg, kern, tm_h, tm_w, a);
}

// One launch sequence over at most kLaunchRows rows; the workspace serves one after the other.
blink_status run_logprobs(const blink_bf16 *hidden, int64_t hidden_row_stride, int32_t hidden_rows, const int32_t *d_row_idx,
                          const blink_bf16 *unembed, int32_t V, int32_t H, const int32_t *d_targets, int32_t n,
                          float temperature, int32_t top, float *d_logprob, float *d_entropy, float *d_lse,
                          int32_t *d_top_ids, float *d_top_logprobs, void *d_ws, cudaStream_t stream)
{
    const int sms = sm_count();
    if (sms < 2) return BLINK_CUDA_ERROR;
    LogprobArgs a{};
    a.plan = make_plan(n, V, sms);
    const WsLayout l = ws_layout(a.plan.cells(), n, H, top);
    auto *wsb = static_cast<uint8_t *>(d_ws);
    a.V = V;
    a.H = H;
    a.n = n;
    a.top = top;
    lay_out(a);
    a.row_idx = d_row_idx;
    a.hidden_rows = hidden_rows;
    a.targets = d_targets;
    a.c = kLog2e / temperature;
    a.stat = reinterpret_cast<float4 *>(wsb + l.stat);
    a.best = reinterpret_cast<int2 *>(wsb + l.best);
    a.logprob = d_logprob;
    a.entropy = d_entropy;
    a.lse = d_lse;
    a.top_lp = d_top_logprobs;
    a.top_ids = d_top_ids;
    a.err = &static_cast<WorkspaceHeader *>(d_ws)->error;
    a.prepared = d_row_idx != nullptr || top > 0;
    a.bounds = reinterpret_cast<uint32_t *>(wsb + l.bounds);

    const blink_bf16 *rows = hidden;
    int64_t row_stride = hidden_row_stride;
    if (a.prepared) {
        auto *dst = reinterpret_cast<blink_bf16 *>(wsb + l.rows);
        const int64_t pieces = d_row_idx ? static_cast<int64_t>(n) * (H / 8) : 0;
        const int64_t bound_pieces = top > 0 ? static_cast<int64_t>(n) * kMaxTop / 4 : 0;
        const int64_t want = ((pieces > bound_pieces ? pieces : bound_pieces) + 255) / 256;
        logprob_prepare_kernel<<<static_cast<unsigned>(want < 4096 ? want : 4096), 256, 0, stream>>>(
            reinterpret_cast<const uint4 *>(hidden), hidden_row_stride / 8, hidden_rows, d_row_idx, pieces, H / 8,
            reinterpret_cast<uint4 *>(dst), reinterpret_cast<uint4 *>(a.bounds), bound_pieces);
        if (cudaGetLastError() != cudaSuccess) return BLINK_CUDA_ERROR;
        if (d_row_idx) {
            rows = dst;
            row_stride = H;
        }
    }
    CUtensorMap tm_h, tm_w;
    const uint64_t e = 2;
    const uint64_t hs = static_cast<uint64_t>(row_stride) * e, wst = static_cast<uint64_t>(H) * e;
    if (!encode_tmap_3d_bf16(&tm_h, rows, H, n, 1, hs, hs * n, 64, a.a_rows, 1) ||
        !encode_tmap_3d_bf16(&tm_w, unembed, H, V, 1, wst, wst * V, 64, kVocabTile / a.plan.blocks_per_worker, 1))
        return BLINK_CUDA_ERROR;
    const bool pair = a.plan.blocks_per_worker == 2;
    cudaError_t err;
    if (top == 0)
        err = pair ? launch_logprob<2, 0>(tm_h, tm_w, a, stream) : launch_logprob<1, 0>(tm_h, tm_w, a, stream);
    else if (top <= 8)
        err = pair ? launch_logprob<2, 8>(tm_h, tm_w, a, stream) : launch_logprob<1, 8>(tm_h, tm_w, a, stream);
    else if (top <= 20)
        err = pair ? launch_logprob<2, 20>(tm_h, tm_w, a, stream) : launch_logprob<1, 20>(tm_h, tm_w, a, stream);
    else
        err = pair ? launch_logprob<2, 32>(tm_h, tm_w, a, stream) : launch_logprob<1, 32>(tm_h, tm_w, a, stream);
    if (err != cudaSuccess) return BLINK_CUDA_ERROR;

    const int lists = (a.plan.chunks > a.plan.rest_chunks ? a.plan.chunks : a.plan.rest_chunks) * kHalves;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const bool wide = lists > 64;
    cfg.gridDim = dim3(static_cast<unsigned>(wide ? n : (n + 3) / 4));
    cfg.blockDim = dim3(wide ? kWideRow : 128);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, wide ? logprob_merge_kernel<kWideRow> : logprob_merge_kernel<32>, a) != cudaSuccess)
        return BLINK_CUDA_ERROR;
    return BLINK_OK;
}

}  // namespace
}  // namespace blink

extern "C" size_t blink_token_logprobs_workspace(int32_t n, int32_t H, int32_t V, int32_t top)
{
    using namespace blink;
    return ws_sizes_ok(n, H, V, top) ? ws_bytes_needed(n, H, V, top, sm_count()) : static_cast<size_t>(kHeaderBytes);
}

extern "C" blink_status blink_token_logprobs_workspace_plan(int32_t n, int32_t H, int32_t V, int32_t top, int32_t sms,
                                                            size_t *ws_bytes, size_t *used)
{
    using namespace blink;
    if (!ws_bytes || !used) return BLINK_INVALID_ARG;
    if (sms < 2 || !ws_sizes_ok(n, H, V, top)) return BLINK_OUT_OF_RANGE;
    *ws_bytes = ws_bytes_needed(n, H, V, top, sms);
    *used = 0;
    for (int32_t r = 0; r < n; r += kLaunchRows) {
        const int32_t rows = n - r < kLaunchRows ? n - r : kLaunchRows;
        const size_t total = ws_layout(make_plan(rows, V, sms).cells(), rows, H, top).total;
        if (total > *used) *used = total;
    }
    return BLINK_OK;
}

extern "C" blink_status blink_token_logprobs(const blink_bf16 *hidden, int64_t hidden_row_stride, int32_t hidden_rows,
                                             const int32_t *d_row_idx, const blink_bf16 *unembed, int32_t V, int32_t H,
                                             const int32_t *d_targets, int32_t n, float temperature, int32_t top,
                                             float *d_logprob, float *d_entropy, float *d_lse, int32_t *d_top_ids,
                                             float *d_top_logprobs, void *d_ws, size_t ws_bytes, cudaStream_t stream)
{
    using namespace blink;
    if (!hidden || !unembed || !d_ws) return BLINK_INVALID_ARG;
    if (!d_logprob && !d_entropy && !d_lse && !d_top_ids) return BLINK_INVALID_ARG;
    if ((d_logprob && !d_targets) || (d_top_ids == nullptr) != (d_top_logprobs == nullptr)) return BLINK_INVALID_ARG;
    if (!(temperature > 0.f) || !(temperature < INFINITY) || !(kLog2e / temperature < INFINITY)) return BLINK_INVALID_ARG;
    if (H < 8 || H % 8 != 0 || V < 1 || hidden_rows < 1 || hidden_row_stride < H || hidden_row_stride % 8 != 0)
        return BLINK_INVALID_ARG;
    if (!aligned16(hidden) || !aligned16(unembed) || !aligned16(d_ws)) return BLINK_INVALID_ARG;
    if (top < 0 || top > kMaxTop || top > V || H > 32768 || V > (1 << 24)) return BLINK_OUT_OF_RANGE;
    if ((top > 0) != (d_top_ids != nullptr)) return BLINK_INVALID_ARG;
    if (n < 1 || n > BLINK_MAX_INPUT_TOKENS) return BLINK_OUT_OF_RANGE;
    if (!d_row_idx && n > hidden_rows) return BLINK_INVALID_ARG;
    if (ws_bytes < blink_token_logprobs_workspace(n, H, V, top)) return BLINK_WORKSPACE_TOO_SMALL;

    for (int32_t r = 0; r < n; r += kLaunchRows) {
        const int32_t rows = n - r < kLaunchRows ? n - r : kLaunchRows;
        const blink_bf16 *h = d_row_idx ? hidden : hidden + r * hidden_row_stride;
        auto at = [r](auto *p, int64_t width) { return p ? p + r * width : p; };
        const blink_status st = run_logprobs(h, hidden_row_stride, d_row_idx ? hidden_rows : rows, at(d_row_idx, 1), unembed, V,
                                             H, at(d_targets, 1), rows, temperature, top, at(d_logprob, 1), at(d_entropy, 1),
                                             at(d_lse, 1), at(d_top_ids, top), at(d_top_logprobs, top), d_ws, stream);
        if (st != BLINK_OK) return st;
    }
    return BLINK_OK;
}
