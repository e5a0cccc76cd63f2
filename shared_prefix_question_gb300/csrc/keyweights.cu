// keyweights.cu -- attention weight received by each prefix key (blink_prefix_key_weights): for every
// (kv head h, key p), the sum over rows and the group's query heads of exp(scale q.k_p - lse).
//
// Mathematics.  With lse known there is no running maximum: a term is 2^(c s - b), c = scale log2(e),
// b = lse log2(e), one fused multiply-add and one exp2 per score, and the result is a plain sum over
// columns, a column being a (row, query head of the group) pair.
//
// Layout.  S = Q K^T with 128 columns as the M rows of the product and 256 keys as its N.  So a thread
// holds one column: its b is a register, and it keeps one partial sum per key (64 of them, in
// registers) over all the column tiles it works through; the 128 threads of a tile are added up once, at
// the end.  (With the keys as the M rows the sum over columns stays in a thread, but every score needs
// its b from shared memory, which the tensor core's operand reads keep busy: 18k 1.37 ms.)
//
// Work.  A unit is 256 keys of one kv head.  The (unit, column tile) steps, unit-major, are cut into
// equal consecutive ranges, one per block (one block per SM): every block does the same number of
// steps whatever the shape.  A unit that one block covers is written by it; the pieces of a unit
// that a range boundary cuts go to the workspace, and a second launch adds them in block order.  So
// the order of every sum is fixed by the shapes and the number of SMs.
//
// Roles (640 threads): warps 0-15 the sums, four warps (the 128 columns) for each 64 of the keys (112
// registers a thread), warp 16 TMA producer (two buffers of 256 keys and a ring of column tiles), warp 17
// MMA issuer (32 registers).  Tensor memory: two score tiles of 256 columns.
// What bounds it: a tile is 1,024 cycles of the tensor core and 1,024 of the exp2 unit (8 lanes a clock on
// each of the SM's four partitions, measured), so the four warps of a partition have to keep one
// unit busy while others wait for scores.  Two warps with 128 keys each took 1,590 cycles a tile.  10240
// rows, 18432 keys, 32/8 heads of 128: 905 us alone, 1,400 cycles a tile, both units 73 % busy (the products
// alone, with nothing reading them, take 732 us; the sums alone, in a loop of their own, 1,034 cycles a
// tile, and 1,245 with the reads of the scores), and 1.0 ms for calls in a row, under the power limit; 1275 rows, 2048 keys: 26 us, of which the 17 tiles of a
// block are 13 and the launch, the first loads and the join the rest.  Slower, at 18432 keys: a part of
// the exponentials as a polynomial on the fused multiply-add units (6 % with an eighth of them, 30 with
// three eighths), scores read 16 at a time (11 %) or ahead of their use (14), halves of 128 keys (30), scalar
// instead of paired adds (12).
//
// Short calls.  One row and 18432 keys read 38 MB: 12 us warm, 22 with a cold L2, where the floor is 5.6;
// 60 rows and 64 keys 8 us, one launch.
//
// A column that does not count has lse -inf here and -b = -inf, so its term is 0 once its score is finite.  It need
// not be: a row owned by no question may hold NaN or infinities in q, and the zeros of a row past the last or of a
// column past g * tpt make NaN with an infinite key.  A warp with such a column clears its scores first (where g does
// not divide 128 the last warp has some in every tile: 4 % with g = 5; clearing their sums at the end of a unit
// instead takes 1.5 % there and 1 % of the time of all other shapes).
#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace blink {
namespace {

constexpr int kUnitKeys = 256;
constexpr int kThreadKeys = 64;  // keys of one thread
constexpr int kSumWarps = 16;
constexpr int kTileCols = 128;  // columns of a column tile
constexpr int kThreadsKW = 640;
constexpr int kProducer = 16, kIssuer = 17;
constexpr int kRegsNeeded = 512 * 112 + 128 * 32;
constexpr int kMaxBlocks = 256;
constexpr uint32_t kTmem = 512;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct KwLayout {
    static constexpr int kPanels = D / 64;
    static constexpr int kKPanel = kUnitKeys * 128, kQPanel = kTileCols * 128;
    static constexpr int kKBytes = kPanels * kKPanel, kQBytes = kPanels * kQPanel;
    static constexpr int kKSlots = 2, kQSlots = D == 128 ? 3 : 6;
    static constexpr int kQOff = kKSlots * kKBytes;
    static constexpr int kSumOff = kQOff + kQSlots * kQBytes;  // [4][2][64] floats
    static constexpr int kBarOff = kSumOff + 8 * kThreadKeys * 4;
    static constexpr int kBytes = kBarOff + 256;
};

struct KeyWeightArgs {
    const float *lse;
    int64_t lse_stride;
    const float *prev;
    int64_t prev_stride;
    float *w;
    int64_t w_stride;
    float *part;  // [blocks][2][kUnitKeys]
    int *err;
    int rows, P, g, tpt, n_tiles, n_units_head;  // tpt: rows per column tile; n_units_head: units of a kv head
    int64_t total;  // steps: units x column tiles
    float c, decay;
};

// Range of steps of block b: [first_step(b), first_step(b + 1)).
__host__ __device__ __forceinline__ int64_t first_step(int64_t b, int64_t total, int64_t blocks)
{
    return b * total / blocks;
}

// The steps of a block, segment by segment (a segment: consecutive column tiles of one unit).  Every
// role walks the same sequence.
template <bool kOneTile>
struct Segment {
    int64_t at, end;
    int n_tiles, n_units_head;
    int head, key0, tile0, tiles;
    bool first, new_q;  // new_q: the column tile is not the one already in shared memory
    bool last_use;      // of a single column tile that the next segment shares
    __device__ Segment(int64_t begin, int64_t e, int nt, int np) : at(begin), end(e), n_tiles(nt), n_units_head(np), first(true)
    {
        head = -1;
        load();
    }
    __device__ void load()
    {
        if (at >= end) return;
        const int64_t unit = at / n_tiles;
        const int h = static_cast<int>(unit / n_units_head);
        key0 = static_cast<int>(unit - static_cast<int64_t>(h) * n_units_head) * kUnitKeys;
        tile0 = static_cast<int>(at - unit * n_tiles);
        tiles = static_cast<int>(min(static_cast<int64_t>(n_tiles - tile0), end - at));
        new_q = n_tiles > 1 || h != head;
        last_use = n_tiles > 1 || at + 1 >= end || (unit + 1) / n_units_head != h;
        head = h;
    }
    __device__ bool more() const { return at < end; }
    __device__ void next()
    {
        at += tiles;
        first = false;
        if constexpr (kOneTile) {  // the next unit, without a division
            const int units = n_units_head * kUnitKeys;
            key0 += kUnitKeys;
            new_q = key0 == units;
            if (new_q) key0 = 0, ++head;
            last_use = at + 1 >= end || key0 + kUnitKeys == units;
        } else {
            load();
        }
    }
};

// Adds acc[0 .. 63] over the 32 threads of a warp; thread l is left with keys 2 l and 2 l + 1 in acc[0]
// and acc[1].  Each step a thread hands half of what it has to its partner.
__device__ __forceinline__ void warp_sum_scatter(float (&acc)[kThreadKeys], int lane)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < 2 * o; ++i) {
            const float give = upper ? acc[i] : acc[i + 2 * o];
            const float keep = upper ? acc[i + 2 * o] : acc[i];
            acc[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
        }
    }
}

// Forms.  kManyTiles: the columns take several tiles.  kOneTile: they fit one (a short question): a unit is one
// step, and the tile and its lse stay from unit to unit of a head.  kFewColumns: they fit 32 rows of a tile
// (a decoded token): the same 32 rows are copied to all four quarters of the tile, so that all 16
// warps have them and each sums 16 of the keys (with the one warp that would have the columns otherwise, the
// sums of a unit take 3,400 cycles against 1,700 for its keys to arrive).
constexpr int kManyTiles = 0, kOneTileForm = 1, kFewColumns = 2;

template <int D, int kForm>
__global__ void __launch_bounds__(kThreadsKW, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const KeyWeightArgs a)
{
    constexpr bool kOneTile = kForm != kManyTiles;
    constexpr bool kFew = kForm == kFewColumns;
    using L = KwLayout<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (ptx::smem_u32(smem) & 1023u) {  // the swizzled tiles need it; the whole block leaves
        if (threadIdx.x == 0) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
        return;
    }
    uint8_t *q_ring = smem + L::kQOff;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *k_full = bars, *k_empty = bars + 2, *q_full = bars + 4, *q_empty = bars + 10;
    uint64_t *s_full = bars + 16, *s_empty = bars + 18, *mma_done = bars + 20, *met = bars + 21;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(met + 4);
    int *abort_word = reinterpret_cast<int *>(tmem_holder + 1);
    volatile int *abort_flag = abort_word;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t begin = first_step(blockIdx.x, a.total, gridDim.x), end = first_step(blockIdx.x + 1, a.total, gridDim.x);
    const int cols_used = a.g * a.tpt;
    const int live_warps = kFew ? 4 : (cols_used + 31) / 32;  // of four: the others have no column in any tile

    if (warp == kProducer && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(k_full + i, 1);
            ptx::mbar_init(k_empty + i, 1);
            ptx::mbar_init(s_full + i, 1);
            ptx::mbar_init(s_empty + i, 4 * live_warps);
        }
        for (int i = 0; i < 4; ++i) ptx::mbar_init(met + i, live_warps);
        for (int i = 0; i < L::kQSlots; ++i) {
            ptx::mbar_init(q_full + i, 1);
            ptx::mbar_init(q_empty + i, 1);
        }
        ptx::mbar_init(mma_done, 1);
        ptx::fence_mbar_init();
        *abort_word = 0;
        ptx::tma_prefetch_desc(&tm_q);
        ptx::tma_prefetch_desc(&tm_k);
    }
    if (warp == 0) {
        ptx::tmem_alloc(tmem_holder, kTmem);
        ptx::tmem_relinquish();
    }
    // Columns of the last live warp past g * tpt are never copied: zero once, so that their scores are 0.
    if (warp < kSumWarps && (kFew ? cols_used < 32 : cols_used < live_warps * 32)) {
        const int pad = ((kFew ? 32 : live_warps * 32) - cols_used) * 128;
        for (int s = 0; s < L::kQSlots * L::kPanels * (kFew ? 4 : 1); ++s) {
            uint8_t *dst = q_ring + s * (kFew ? 32 * 128 : L::kQPanel) + cols_used * 128;
            for (int off = threadIdx.x * 16; off < pad; off += kSumWarps * 32 * 16)
                *reinterpret_cast<uint4 *>(dst + off) = make_uint4(0, 0, 0, 0);
        }
        ptx::fence_proxy_async_smem();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // Registers by role: 128 threads at 32 and 512 at 112 are the 640 at 96 of the launch.
    if (warp >= kSumWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");

    if (warp == kProducer) {
        if (lane == 0) {
            int nk = 0, nq = 0;
            bool ok = true;
            const uint32_t q_bytes = static_cast<uint32_t>(L::kPanels) * 128u * cols_used * (kFew ? 4u : 1u);
            for (Segment<kOneTile> sg(begin, end, a.n_tiles, a.n_units_head); ok && sg.more(); sg.next(), ++nk) {
                const int ks = nk & 1;
                // freed at the end of an earlier segment: the limit grows with a segment's length
                if (!(ok = ptx::mbar_wait(k_empty + ks, ((nk >> 1) & 1) ^ 1, abort_flag, a.err, BLINK_DEVICE_TIMEOUT,
                                          1000000000ull + 20000ull * a.n_tiles)))
                    break;
                ptx::mbar_arrive_expect_tx(k_full + ks, L::kKBytes);
                for (int p = 0; p < L::kPanels; ++p)
                    ptx::tma_load_3d(smem + ks * L::kKBytes + p * L::kKPanel, &tm_k, p * 64, sg.head, sg.key0, k_full + ks);
                for (int i = 0; ok && sg.new_q && i < sg.tiles; ++i, ++nq) {
                    const int qs = nq % L::kQSlots;
                    if (!(ok = ptx::mbar_wait(q_empty + qs, ((nq / L::kQSlots) & 1) ^ 1, abort_flag, a.err,
                                              BLINK_DEVICE_TIMEOUT)))
                        break;
                    ptx::mbar_arrive_expect_tx(q_full + qs, q_bytes);
                    for (int p = 0; p < L::kPanels; ++p)
                        for (int r = 0; r < (kFew ? 4 : 1); ++r)
                            ptx::tma_load_3d(q_ring + qs * L::kQBytes + p * L::kQPanel + r * 32 * 128, &tm_q, p * 64,
                                             sg.head * a.g, (sg.tile0 + i) * a.tpt, q_full + qs);
                }
            }
            ptx::grid_launch_dependents();
            // every copy issued must have landed before the block may exit
            volatile int no_abort = 0;
            for (int n = nk > 2 ? nk - 2 : 0; n < nk; ++n, no_abort = 0)
                ptx::mbar_wait(k_full + (n & 1), (n >> 1) & 1, &no_abort, a.err, BLINK_DEVICE_TIMEOUT);
            for (int n = nq > L::kQSlots ? nq - L::kQSlots : 0; n < nq; ++n, no_abort = 0)
                ptx::mbar_wait(q_full + n % L::kQSlots, (n / L::kQSlots) & 1, &no_abort, a.err, BLINK_DEVICE_TIMEOUT);
        }
    } else if (warp == kIssuer) {
        if (lane == 0) {
            constexpr uint32_t idesc = ptx::idesc_bf16_f32(kTileCols, kUnitKeys, false);
            const uint64_t desc0 = ptx::smem_desc_sw128(ptx::smem_u32(smem), 16, 1024);  // in units of 16 bytes
            int nk = 0, nq = -1, st = 0;
            bool ok = true;
            for (Segment<kOneTile> sg(begin, end, a.n_tiles, a.n_units_head); ok && sg.more(); sg.next(), ++nk) {
                const int ks = nk & 1;
                if (!(ok = ptx::mbar_wait(k_full + ks, (nk >> 1) & 1, abort_flag, a.err, BLINK_DEVICE_TIMEOUT))) break;
                const uint64_t kd = desc0 + (ks * L::kKBytes >> 4);
                for (int i = 0; i < sg.tiles; ++i, ++st) {
                    if (sg.new_q) ++nq;
                    const int qs = nq % L::kQSlots;
                    if (sg.new_q && !(ok = ptx::mbar_wait(q_full + qs, (nq / L::kQSlots) & 1, abort_flag, a.err,
                                                          BLINK_DEVICE_TIMEOUT)))
                        break;
                    const int buf = st & 1;
                    if (!(ok = ptx::mbar_wait(s_empty + buf, ((st >> 1) & 1) ^ 1, abort_flag, a.err, BLINK_DEVICE_TIMEOUT)))
                        break;
                    ptx::tc_fence_after();
                    const uint64_t qd = desc0 + ((L::kQOff + qs * L::kQBytes) >> 4);
#pragma unroll
                    for (int p = 0; p < L::kPanels; ++p)
                        ptx::mma_ss_x4(tmem + buf * kUnitKeys, qd + (p * L::kQPanel >> 4), kd + (p * L::kKPanel >> 4), idesc,
                                       p > 0);
                    ptx::mma_commit(s_full + buf);
                    if (sg.last_use) ptx::mma_commit(q_empty + qs);
                }
                if (ok) ptx::mma_commit(k_empty + ks);
            }
            ptx::mma_commit(mma_done);  // every product issued must be complete before tensor memory is released
            volatile int no_abort = 0;
            ptx::mbar_wait(mma_done, 0, &no_abort, a.err, BLINK_DEVICE_TIMEOUT);
        }
    } else if (warp < kSumWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
        const int quarter = warp >> 2, wq = warp & 3;  // of the unit's keys, of the tile's columns
        if constexpr (kFew) {
            // -------------------------------------------------------- sums: one column per thread, 16 keys a warp
            constexpr int kKeys = 16;
            const int offset = quarter * kThreadKeys + wq * kKeys;  // of the warp's keys in the unit
            const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16) + offset;
            const int row = lane / a.g;
            const bool has = lane < cols_used && row < a.rows;
            int st = 0;
            float b = -INFINITY;
            bool ok = true;
            for (Segment<kOneTile> sg(begin, end, a.n_tiles, a.n_units_head); ok && sg.more(); sg.next(), ++st) {
                if (sg.new_q) b = has ? __ldg(a.lse + (sg.head * a.g + lane % a.g) * a.lse_stride + row) : -INFINITY;
                const bool dead = b == -INFINITY;  // no row, or owned by no question: the score may be anything
                const float nb = dead ? -INFINITY : -b * kLog2e;
                const int key = sg.key0 + offset + (lane >> 1);  // the key this thread writes, if its lane is even
                const bool writes = (lane & 1) == 0 && key < a.P;
                const float before = writes && a.decay > 0.f ? a.prev[sg.head * a.prev_stride + key] : 0.f;
                const int buf = st & 1;
                if (!(ok = ptx::mbar_wait_warp(s_full + buf, (st >> 1) & 1, abort_flag, a.err, BLINK_DEVICE_TIMEOUT))) break;
                ptx::tc_fence_after();
                uint32_t raw[kKeys];
                ptx::tmem_ld16(trow + buf * kUnitKeys, raw);
                ptx::tmem_wait_ld();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(s_empty + buf);
                float acc[kKeys];
#pragma unroll
                for (int j = 0; j < kKeys; ++j) acc[j] = dead ? 0.f : ptx::ex2(fmaf(__uint_as_float(raw[j]), a.c, nb));
                // over the warp's threads, each step handing half of the keys to the partner
#pragma unroll
                for (int o = 16; o > 1; o >>= 1) {
                    const bool upper = (lane & o) != 0;
#pragma unroll
                    for (int j = 0; j < o / 2; ++j) {
                        const float give = upper ? acc[j] : acc[j + o / 2];
                        const float keep = upper ? acc[j + o / 2] : acc[j];
                        acc[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                    }
                }
                const float sum = acc[0] + __shfl_xor_sync(0xFFFFFFFFu, acc[0], 1);
                if (writes) a.w[sg.head * a.w_stride + key] = fmaf(a.decay, before, sum);
            }
        } else if (wq < live_warps) {
            // -------------------------------------------------------- sums: one column per thread
            const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16) + quarter * kThreadKeys;
            float *sums = reinterpret_cast<float *>(smem + L::kSumOff) + quarter * 2 * kThreadKeys;
            const int col = wq * 32 + lane;
            const int tok = col / a.g;
            const int head_off = col % a.g;
            const uint64_t cc = ptx::f32x2(a.c, a.c);
            int st = 0, meetings = 0;
            float single = 0.f;
            float2 before = make_float2(0.f, 0.f);  // previous weights of this thread's keys
            bool ok = true;
            for (Segment<kOneTile> sg(begin, end, a.n_tiles, a.n_units_head); ok && sg.more(); sg.next()) {
                const float *lse = a.lse + (sg.head * a.g + head_off) * a.lse_stride + (sg.tile0 * a.tpt + tok);
                // rows from there to the last of the segment, if the thread has a column
                int left = col < cols_used ? min(a.rows, (sg.tile0 + sg.tiles) * a.tpt) - (sg.tile0 * a.tpt + tok) : 0;
                auto lse_next = [&] {
                    const float v = left > 0 ? __ldg(lse) : -INFINITY;
                    lse += a.tpt;
                    left -= a.tpt;
                    return v;
                };
                float acc[kThreadKeys];
#pragma unroll
                for (int i = 0; i < kThreadKeys; ++i) acc[i] = 0.f;
                float next;  // a tile ahead of its use
                if constexpr (kOneTile) {
                    if (sg.new_q) single = lse_next();
                    next = single;
                    if (a.decay > 0.f && wq == 0) {  // read now, a kilocycle before its use
                        const int key = sg.key0 + quarter * kThreadKeys + 2 * lane;
                        const float *prev = a.prev + sg.head * a.prev_stride;
                        before.x = key < a.P ? prev[key] : 0.f;
                        before.y = key + 1 < a.P ? prev[key + 1] : 0.f;
                    }
                } else {
                    next = lse_next();
                }
                // two tiles a trip: 905 us instead of 940 for 18432 keys (four the same, eight 1010)
#pragma unroll(kOneTile ? 1 : 2)
                for (int i = sg.tiles; i > 0; --i, ++st) {
                    const bool dead = next == -INFINITY;  // no row, or owned by no question: the score may be anything
                    const float nb = dead ? -INFINITY : -next * kLog2e;
                    const uint64_t nb2 = ptx::f32x2(nb, nb);
                    const int buf = st & 1;
                    ok = ptx::mbar_wait(s_full + buf, (st >> 1) & 1, abort_flag, a.err, BLINK_DEVICE_TIMEOUT);
                    // one vote for both: a column that does not count, and a wait that gave up, which all lanes have to take
                    // the same way (a vote for each: 1005 us instead of 996 for 18432 keys)
                    const bool careful = !__all_sync(0xFFFFFFFFu, ok && !dead);
                    if (careful && !__all_sync(0xFFFFFFFFu, ok)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
#pragma unroll
                    for (int q = 0; q < kThreadKeys / 32; ++q) {
                        uint32_t raw[32];
                        ptx::tmem_ld32(trow + buf * kUnitKeys + q * 32, raw);
                        ptx::tmem_wait_ld();
                        if (q == kThreadKeys / 32 - 1) {  // the tile is in registers: its buffer may be written
                            ptx::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(s_empty + buf);
                            if constexpr (!kOneTile) next = lse_next();
                        }
                        if (careful) {  // such a row's scores become 0, and with -b = -inf its terms
#pragma unroll
                            for (int j = 0; j < 32; ++j) raw[j] = dead ? 0u : raw[j];
                        }
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float x0, x1;
                            ptx::f32x2_split(
                                ptx::fma_f32x2(ptx::f32x2(__uint_as_float(raw[j]), __uint_as_float(raw[j + 1])), cc, nb2), x0, x1);
                            const uint64_t s2 = ptx::add_f32x2(ptx::f32x2(acc[q * 32 + j], acc[q * 32 + j + 1]),
                                                               ptx::f32x2(ptx::ex2(x0), ptx::ex2(x1)));
                            ptx::f32x2_split(s2, acc[q * 32 + j], acc[q * 32 + j + 1]);
                        }
                    }
                }
                if (!ok) break;
                warp_sum_scatter(acc, lane);
                float2 s = make_float2(acc[0], acc[1]);  // keys 2 lane and 2 lane + 1 of this quarter
                if (live_warps > 1) {
                    // ((w0 + w2) + (w1 + w3)): the live warps of the quarter, two at a time through shared memory
                    auto meet = [&] {
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(met + quarter);
                        ok = ok && ptx::mbar_wait_warp(met + quarter, meetings & 1, abort_flag, a.err, BLINK_DEVICE_TIMEOUT);
                        ++meetings;
                    };
                    float2 *dst = reinterpret_cast<float2 *>(sums + (wq & 1) * kThreadKeys) + lane;
                    auto add = [&](const float2 &o) { s.x += o.x, s.y += o.y; };
                    if (wq >= 2) *dst = s;
                    meet();
                    if (wq < 2 && wq + 2 < live_warps) add(*dst);
                    meet();
                    if (wq == 1) *dst = s;
                    meet();
                    if (wq == 0) add(*(dst + kThreadKeys / 2));
                    meet();  // the buffers are free again
                }
                if (ok && wq == 0) {
                    const float v[2] = {s.x, s.y};
                    const int key = sg.key0 + quarter * kThreadKeys + 2 * lane;
                    if (sg.tiles == a.n_tiles) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (key + i < a.P) {
                                float *w = a.w + sg.head * a.w_stride + key + i;
                                if constexpr (kOneTile)
                                    *w = fmaf(a.decay, i ? before.y : before.x, v[i]);
                                else
                                    *w = a.decay > 0.f ? fmaf(a.decay, a.prev[sg.head * a.prev_stride + key + i], v[i]) : v[i];
                            }
                    } else {
                        float *part = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (sg.first ? 0 : 1)) * kUnitKeys;
                        *reinterpret_cast<float2 *>(part + quarter * kThreadKeys + 2 * lane) = s;
                    }
                }
            }
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 0) ptx::tmem_dealloc(tmem, kTmem);
}

constexpr int kJoinThreads = kUnitKeys / 2;

// One block per unit: adds the pieces of a unit that range boundaries cut, in block order.  128 threads of 32
// registers are what the SM has left beside a block of the sums, so these are resident before that ends
// and have their divisions and previous weights behind them.
__global__ void __launch_bounds__(kJoinThreads) key_weights_join_kernel(const KeyWeightArgs a, int blocks)
{
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.n_tiles, hi = lo + a.n_tiles;
    const int b0 = static_cast<int>(((lo + 1) * blocks - 1) / a.total);  // the block that has step lo
    const int b1 = static_cast<int>((hi * blocks - 1) / a.total);        // and step hi - 1
    const int head = blockIdx.x / a.n_units_head;
    const int key = (blockIdx.x - head * a.n_units_head) * kUnitKeys + 2 * threadIdx.x;
    const bool cut = b0 != b1;
    // the unit is the second piece of its first block, unless the block begins with it, and the first of all others
    const float2 *part = reinterpret_cast<const float2 *>(a.part) + static_cast<int64_t>(b0) * kUnitKeys + threadIdx.x;
    const int first_piece = first_step(b0, a.total, blocks) >= lo ? 0 : 1;
    float before[2] = {0.f, 0.f};
    if (cut && a.decay > 0.f) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (key + i < a.P) before[i] = a.prev[head * a.prev_stride + key + i];
    }
    ptx::grid_dep_wait();
    if (!cut) return;
    float2 sum = __ldcg(part + first_piece * kJoinThreads);
#pragma unroll 4
    for (int b = 1; b <= b1 - b0; ++b) {
        const float2 v = __ldcg(part + static_cast<int64_t>(b) * kUnitKeys);
        sum.x += v.x, sum.y += v.y;
    }
    float *w = a.w + head * a.w_stride + key;
    if (key < a.P) w[0] = a.decay > 0.f ? fmaf(a.decay, before[0], sum.x) : sum.x;
    if (key + 1 < a.P) w[1] = a.decay > 0.f ? fmaf(a.decay, before[1], sum.y) : sum.y;
}

int sm_count()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
}

template <int D, int kForm>
cudaError_t launch_key_weights(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const KeyWeightArgs &a, unsigned blocks,
                               cudaStream_t stream)
{
    auto kern = key_weights_kernel<D, kForm>;
    // The split of registers by role has to fit the registers of the launch: checked once.
    static const bool fits = [kern] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, kern) == cudaSuccess && fa.numRegs * kThreadsKW >= kRegsNeeded;
    }();
    if (!fits) return cudaErrorLaunchOutOfResources;
    // all 512 tensor-memory columns: one block per SM, which the shared memory keeps so for d = 64 too
    constexpr int kSmem = KwLayout<D>::kBytes > 120 * 1024 ? KwLayout<D>::kBytes : 120 * 1024;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    kern<<<blocks, kThreadsKW, kSmem, stream>>>(tm_q, tm_k, a);
    return cudaGetLastError();
}

}  // namespace
}  // namespace blink

extern "C" size_t blink_prefix_key_weights_workspace(int32_t rows, int32_t P, int32_t Hq, int32_t Hkv, int32_t d)
{
    using namespace blink;
    (void)rows, (void)P, (void)Hq, (void)Hkv, (void)d;
    return kHeaderBytes + static_cast<size_t>(kMaxBlocks) * 2 * kUnitKeys * sizeof(float);
}

extern "C" blink_status blink_prefix_key_weights(const blink_bf16 *q, const blink_bf16 *k_pre, int64_t pre_row_stride,
                                                 const float *lse, int64_t lse_stride, int32_t rows, int32_t P,
                                                 int32_t Hq, int32_t Hkv, int32_t d, float scale, float decay,
                                                 const float *d_prev, int64_t prev_stride, float *d_weights,
                                                 int64_t w_stride, void *d_ws, size_t ws_bytes, cudaStream_t stream)
{
    using namespace blink;
    if (!q || !k_pre || !lse || !d_weights || !d_ws || !aligned16(d_ws)) return BLINK_INVALID_ARG;
    if (rows < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > 128 || (d != 64 && d != 128))
        return BLINK_INVALID_ARG;
    if (P < 1 || P > BLINK_MAX_INPUT_TOKENS || Hkv > 65535 || rows > (1 << 30)) return BLINK_OUT_OF_RANGE;
    if (!(decay >= 0.f) || !(decay < INFINITY) || (decay > 0.f && !d_prev)) return BLINK_INVALID_ARG;
    if (scale != scale || scale == INFINITY) return BLINK_INVALID_ARG;
    if (pre_row_stride < static_cast<int64_t>(Hkv) * d || pre_row_stride % 8 != 0) return BLINK_INVALID_ARG;
    if ((lse_stride < rows && Hq > 1) || (w_stride < P && Hkv > 1)) return BLINK_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pre)) return BLINK_INVALID_ARG;
    if (decay > 0.f) {
        if (prev_stride < P && Hkv > 1) return BLINK_INVALID_ARG;
        const bool same = d_prev == d_weights && (prev_stride == w_stride || Hkv == 1);
        const float *pe = d_prev + (Hkv - 1) * prev_stride + P, *we = d_weights + (Hkv - 1) * w_stride + P;
        if (!same && !(pe <= d_weights || we <= d_prev)) return BLINK_INVALID_ARG;
    }
    if (ws_bytes < blink_prefix_key_weights_workspace(rows, P, Hq, Hkv, d)) return BLINK_WORKSPACE_TOO_SMALL;

    KeyWeightArgs a{};
    a.g = Hq / Hkv;
    a.tpt = kTileCols / a.g < rows ? kTileCols / a.g : rows;
    a.n_tiles = (rows + a.tpt - 1) / a.tpt;
    a.n_units_head = (P + kUnitKeys - 1) / kUnitKeys;
    a.total = static_cast<int64_t>(Hkv) * a.n_units_head * a.n_tiles;
    const int sms = sm_count();
    if (sms < 1) return BLINK_CUDA_ERROR;
    int64_t blocks = sms < kMaxBlocks ? sms : kMaxBlocks;
    if (blocks > a.total) blocks = a.total;
    const float sc = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(d));
    a.c = sc * kLog2e;
    a.decay = decay;
    a.lse = lse;
    a.lse_stride = lse_stride;
    a.prev = d_prev;
    a.prev_stride = prev_stride;
    a.w = d_weights;
    a.w_stride = w_stride;
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(d_ws) + kHeaderBytes);
    a.err = &static_cast<WorkspaceHeader *>(d_ws)->error;
    a.rows = rows;
    a.P = P;

    CUtensorMap tm_q, tm_k;
    const uint64_t e = 2;
    if (!encode_tmap_3d_bf16(&tm_q, q, d, Hq, rows, d * e, static_cast<uint64_t>(Hq) * d * e, 64, a.g, a.tpt) ||
        !encode_tmap_3d_bf16(&tm_k, k_pre, d, Hkv, P, d * e, static_cast<uint64_t>(pre_row_stride) * e, 64, 1,
                             kUnitKeys))
        return BLINK_CUDA_ERROR;
    const auto grid = static_cast<unsigned>(blocks);
    cudaError_t err;
    if (a.n_tiles > 1)
        err = d == 128 ? launch_key_weights<128, kManyTiles>(tm_q, tm_k, a, grid, stream)
                       : launch_key_weights<64, kManyTiles>(tm_q, tm_k, a, grid, stream);
    else if (a.g * a.tpt > 32)
        err = d == 128 ? launch_key_weights<128, kOneTileForm>(tm_q, tm_k, a, grid, stream)
                       : launch_key_weights<64, kOneTileForm>(tm_q, tm_k, a, grid, stream);
    else
        err = d == 128 ? launch_key_weights<128, kFewColumns>(tm_q, tm_k, a, grid, stream)
                       : launch_key_weights<64, kFewColumns>(tm_q, tm_k, a, grid, stream);
    if (err != cudaSuccess) return BLINK_CUDA_ERROR;
    if (a.n_tiles == 1) return BLINK_OK;  // a unit of one step is never cut
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(Hkv * a.n_units_head));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, key_weights_join_kernel, a, static_cast<int>(blocks)) != cudaSuccess)
        return BLINK_CUDA_ERROR;
    return BLINK_OK;
}
