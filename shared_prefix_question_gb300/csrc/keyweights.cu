// keyweights.cu -- attention weight received by each prefix key (blink_prefix_key_weights): for every
// (kv head h, key p), the sum over rows and the group's query heads of exp(scale q.k_p - lse).
//
// Mathematics.  With lse known there is no running maximum: a term is 2^(c s - b), c = scale log2(e),
// b = lse log2(e), one fused multiply-add and one exp2 per score, and the result is a plain sum over
// query columns.  The scores are computed transposed, S = K Q^T with the keys as the M rows, so that a
// key is a tensor-memory lane: the sum over columns stays inside one thread and needs no exchange.
//
// Work.  A unit is 256 keys (two M = 128 tiles) of one kv head; a column is (row, query head of the
// group), up to 256 of them per column tile.  The (unit, column tile) steps, unit-major, are cut into
// equal consecutive ranges, one per block (one block per SM): every block does the same number of
// steps whatever the shape.  A unit that one block covers is written by it; the pieces of a unit
// that a range boundary cuts go to the workspace, and a second launch adds them in block order.  So
// the order of every sum is fixed by the shapes and the number of SMs.
//
// Roles (352 threads): warp 8 TMA producer (K tiles and column tiles into two rings), warp 9 MMA issuer,
// warp 10 bias loader (lse of the columns, as -b, into a ring beside the column tiles), warps 0-3 /
// 4-7 the sums of key tile 0 / 1, one key per thread.
// Tensor memory (512 columns): two sets of [key tile 0, key tile 1] x 128 columns.
//
// Columns that do not count have -b = -inf, so their term is 0: columns past the last row (Q is zero
// there) and rows owned by no question.  Only the latter may hold NaN or infinities in q; column tiles
// that have any are summed with a select per column.
#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace blink {
namespace {

constexpr int kKeysPerTile = 128;
constexpr int kUnitKeys = 2 * kKeysPerTile;
constexpr int kMaxCols = 256;   // columns of a column tile
constexpr int kSubCols = 128;   // columns of one product
constexpr int kQSlots = 2;
constexpr int kMaxKSlots = 8;
constexpr int kThreadsKW = 352;
constexpr int kProducer = 8, kIssuer = 9, kBias = 10;
constexpr int kMaxBlocks = 256;
constexpr uint32_t kTmem = 512;
constexpr int kRingBytes = 224 * 1024;
constexpr int kBiasOff = kRingBytes;
constexpr int kBarOff = kBiasOff + kQSlots * kMaxCols * 4;
constexpr int kSmemBytes = kBarOff + 384;
constexpr float kLog2e = 1.4426950408889634f;

struct KeyWeightArgs {
    const float *lse;
    int64_t lse_stride;
    const float *prev;
    int64_t prev_stride;
    float *w;
    int64_t w_stride;
    float *part;  // [blocks][2][kUnitKeys]
    int *err;
    int rows, P, g, tpt, n_tiles, n_pairs, cols;  // tpt: rows per column tile; cols: columns per tile
    int k_slots, q_slot_bytes;
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
struct Segment {
    int64_t at, end;
    int n_tiles, n_pairs;
    int head, key0, tile0, tiles;
    bool first, new_q;  // new_q: the column tile is not the one already in shared memory
    bool last_use;      // of a single column tile that the next segment shares
    __device__ Segment(int64_t begin, int64_t e, int nt, int np) : at(begin), end(e), n_tiles(nt), n_pairs(np), first(true)
    {
        head = -1;
        load();
    }
    __device__ void load()
    {
        if (at >= end) return;
        const int64_t unit = at / n_tiles;
        const int h = static_cast<int>(unit / n_pairs);
        key0 = static_cast<int>(unit - static_cast<int64_t>(h) * n_pairs) * kUnitKeys;
        tile0 = static_cast<int>(at - unit * n_tiles);
        tiles = static_cast<int>(min(static_cast<int64_t>(n_tiles - tile0), end - at));
        new_q = n_tiles > 1 || h != head;
        last_use = n_tiles > 1 || at + 1 >= end || (unit + 1) / n_pairs != h;
        head = h;
    }
    __device__ bool more() const { return at < end; }
    __device__ void next()
    {
        at += tiles;
        first = false;
        load();
    }
};

template <int D>
__global__ void __launch_bounds__(kThreadsKW, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const KeyWeightArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int kPanels = D / 64;
    constexpr int kKTileBytes = kKeysPerTile * D * 2;
    constexpr int kKPanelBytes = kKeysPerTile * 128;
    uint8_t *k_ring = smem;
    uint8_t *q_ring = smem + a.k_slots * kKTileBytes;
    float *bias = reinterpret_cast<float *>(smem + kBiasOff);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kBarOff);
    uint64_t *k_full = bars, *k_empty = bars + kMaxKSlots;
    uint64_t *q_full = bars + 2 * kMaxKSlots, *q_empty = q_full + kQSlots;
    uint64_t *b_full = q_empty + kQSlots, *b_empty = b_full + kQSlots;
    uint64_t *s_full = b_empty + kQSlots, *s_empty = s_full + 4;  // [set][key tile]
    uint64_t *mma_done = s_empty + 4;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + 1);
    int *abort_word = reinterpret_cast<int *>(tmem_holder + 1);
    int *slow = abort_word + 1;  // [kQSlots]: the tile has rows owned by no question
    volatile int *abort_flag = abort_word;

    if (ptx::smem_u32(smem) & 1023u) {  // the swizzled tiles need it; the whole block leaves
        if (threadIdx.x == 0) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t begin = first_step(blockIdx.x, a.total, gridDim.x), end = first_step(blockIdx.x + 1, a.total, gridDim.x);
    const int q_panel = a.cols * 128;

    if (warp == kProducer && lane == 0) {
        for (int i = 0; i < a.k_slots; ++i) {
            ptx::mbar_init(k_full + i, 1);
            ptx::mbar_init(k_empty + i, 1);
        }
        for (int i = 0; i < kQSlots; ++i) {
            ptx::mbar_init(q_full + i, 1);
            ptx::mbar_init(q_empty + i, 1);
            ptx::mbar_init(b_full + i, 32);
            ptx::mbar_init(b_empty + i, 8);
        }
        for (int i = 0; i < 4; ++i) {
            ptx::mbar_init(s_full + i, 1);
            ptx::mbar_init(s_empty + i, 4);
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
    // Columns past g * tpt are never copied: zero once, so that their scores are 0.
    const int cols_used = a.g * a.tpt;
    if (warp < 8 && cols_used < a.cols) {
        const int pad = (a.cols - cols_used) * 128;
        for (int s = 0; s < kQSlots * kPanels; ++s) {
            uint8_t *dst = q_ring + (s / kPanels) * a.q_slot_bytes + (s % kPanels) * q_panel + cols_used * 128;
            for (int off = threadIdx.x * 16; off < pad; off += 256 * 16)
                *reinterpret_cast<uint4 *>(dst + off) = make_uint4(0, 0, 0, 0);
        }
        ptx::fence_proxy_async_smem();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    if (warp == kProducer) {
        if (lane == 0) {
            int nk = 0, nq = 0;
            bool ok = true;
            const uint32_t q_bytes = static_cast<uint32_t>(kPanels) * 64u * cols_used * 2u;
            for (Segment sg(begin, end, a.n_tiles, a.n_pairs); ok && sg.more(); sg.next()) {
                for (int t = 0; ok && t < 2; ++t, ++nk) {
                    const int slot = nk % a.k_slots;
                    // freed at the end of an earlier segment: the limit grows with a segment's length
                    if (!(ok = ptx::mbar_wait(k_empty + slot, ((nk / a.k_slots) & 1) ^ 1, abort_flag, a.err,
                                              BLINK_DEVICE_TIMEOUT, 1000000000ull + 20000ull * a.n_tiles)))
                        break;
                    ptx::mbar_arrive_expect_tx(k_full + slot, kKTileBytes);
                    for (int p = 0; p < kPanels; ++p)
                        ptx::tma_load_3d(k_ring + slot * kKTileBytes + p * kKPanelBytes, &tm_k, p * 64, sg.head,
                                         sg.key0 + t * kKeysPerTile, k_full + slot);
                }
                for (int i = 0; ok && sg.new_q && i < sg.tiles; ++i, ++nq) {
                    const int slot = nq % kQSlots;
                    if (!(ok = ptx::mbar_wait(q_empty + slot, ((nq / kQSlots) & 1) ^ 1, abort_flag, a.err,
                                              BLINK_DEVICE_TIMEOUT)))
                        break;
                    ptx::mbar_arrive_expect_tx(q_full + slot, q_bytes);
                    for (int p = 0; p < kPanels; ++p)
                        ptx::tma_load_3d(q_ring + slot * a.q_slot_bytes + p * q_panel, &tm_q, p * 64, sg.head * a.g,
                                         (sg.tile0 + i) * a.tpt, q_full + slot);
                }
            }
            ptx::grid_launch_dependents();
            // every copy issued must have landed before the block may exit
            volatile int no_abort = 0;
            for (int n = nk > a.k_slots ? nk - a.k_slots : 0; n < nk; ++n, no_abort = 0)
                ptx::mbar_wait(k_full + n % a.k_slots, (n / a.k_slots) & 1, &no_abort, a.err, BLINK_DEVICE_TIMEOUT);
            for (int n = nq > kQSlots ? nq - kQSlots : 0; n < nq; ++n, no_abort = 0)
                ptx::mbar_wait(q_full + n % kQSlots, (n / kQSlots) & 1, &no_abort, a.err, BLINK_DEVICE_TIMEOUT);
        }
    } else if (warp == kIssuer) {
        if (lane == 0) {
            const uint32_t kb = ptx::smem_u32(k_ring), qb = ptx::smem_u32(q_ring);
            const int n_sub = a.cols > kSubCols ? 2 : 1;
            const uint32_t idesc[2] = {ptx::idesc_bf16_f32(kKeysPerTile, a.cols > kSubCols ? kSubCols : a.cols, false),
                                       ptx::idesc_bf16_f32(kKeysPerTile, a.cols > kSubCols ? a.cols - kSubCols : 32, false)};
            int nk = 0, nq = -1, st = 0;
            bool ok = true;
            for (Segment sg(begin, end, a.n_tiles, a.n_pairs); ok && sg.more(); sg.next(), nk += 2) {
                const int ks[2] = {nk % a.k_slots, (nk + 1) % a.k_slots};
                uint64_t kd[2][D / 16];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        kd[t][kk] = ptx::smem_desc_sw128(kb + ks[t] * kKTileBytes + (kk >> 2) * kKPanelBytes + (kk & 3) * 32,
                                                         16, 1024);
                for (int i = 0; ok && i < sg.tiles; ++i) {
                    if (sg.new_q) ++nq;
                    const int qs = nq % kQSlots;
                    if (sg.new_q && !(ok = ptx::mbar_wait(q_full + qs, (nq / kQSlots) & 1, abort_flag, a.err,
                                                          BLINK_DEVICE_TIMEOUT)))
                        break;
                    for (int sub = 0; ok && sub < n_sub; ++sub, ++st) {
                        uint64_t qd[D / 16];
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            qd[kk] = ptx::smem_desc_sw128(qb + qs * a.q_slot_bytes + (kk >> 2) * q_panel + sub * kSubCols * 128 +
                                                              (kk & 3) * 32,
                                                          16, 1024);
                        for (int t = 0; t < 2; ++t) {
                            if (i == 0 && sub == 0 &&
                                !(ok = ptx::mbar_wait(k_full + ks[t], ((nk + t) / a.k_slots) & 1, abort_flag, a.err,
                                                      BLINK_DEVICE_TIMEOUT)))
                                break;
                            const int buf = (st & 1) * 2 + t;
                            if (!(ok = ptx::mbar_wait(s_empty + buf, ((st >> 1) & 1) ^ 1, abort_flag, a.err,
                                                      BLINK_DEVICE_TIMEOUT)))
                                break;
                            ptx::tc_fence_after();
                            if constexpr (D == 128) {
                                ptx::mma_ss_x8(tmem + buf * kSubCols, kd[t], qd, idesc[sub], 0u);
                            } else {
#pragma unroll
                                for (int kk = 0; kk < D / 16; ++kk)
                                    ptx::mma_ss(tmem + buf * kSubCols, kd[t][kk], qd[kk], idesc[sub], kk > 0 ? 1u : 0u);
                            }
                            ptx::mma_commit(s_full + buf);
                            if (i == sg.tiles - 1 && sub == n_sub - 1) ptx::mma_commit(k_empty + ks[t]);
                        }
                    }
                    if (ok && sg.last_use) ptx::mma_commit(q_empty + qs);
                }
            }
            ptx::mma_commit(mma_done);  // every product issued must be complete before tensor memory is released
            volatile int no_abort = 0;
            ptx::mbar_wait(mma_done, 0, &no_abort, a.err, BLINK_DEVICE_TIMEOUT);
        }
    } else if (warp == kBias) {
        int off_t[kMaxCols / 32], off_h[kMaxCols / 32];
#pragma unroll
        for (int j = 0; j < kMaxCols / 32; ++j) {
            const int c = lane + 32 * j;
            off_t[j] = c < cols_used ? c / a.g : 0x40000000;  // past every row
            off_h[j] = c % a.g;
        }
        int nq = 0;
        bool ok = true;
        for (Segment sg(begin, end, a.n_tiles, a.n_pairs); ok && sg.more(); sg.next()) {
            for (int i = 0; ok && sg.new_q && i < sg.tiles; ++i, ++nq) {
                const int t0 = (sg.tile0 + i) * a.tpt;
                float v[kMaxCols / 32];
                bool dead = false;
#pragma unroll
                for (int j = 0; j < kMaxCols / 32; ++j) {
                    const bool valid = off_t[j] < a.rows - t0;
                    v[j] = valid ? __ldg(a.lse + (sg.head * a.g + off_h[j]) * a.lse_stride + t0 + off_t[j]) : INFINITY;
                }
                const int slot = nq % kQSlots;
                if (!(ok = ptx::mbar_wait(b_empty + slot, ((nq / kQSlots) & 1) ^ 1, abort_flag, a.err,
                                          BLINK_DEVICE_TIMEOUT)))
                    break;
#pragma unroll
                for (int j = 0; j < kMaxCols / 32; ++j) {
                    dead = dead || v[j] == -INFINITY;
                    bias[slot * kMaxCols + lane + 32 * j] = v[j] == -INFINITY ? -INFINITY : -v[j] * kLog2e;
                }
                const bool any = __any_sync(0xFFFFFFFFu, dead);
                if (lane == 0) slow[slot] = any;
                ptx::mbar_arrive(b_full + slot);
            }
        }
    } else {
        // ------------------------------------------------------------ sums: one key per thread
        const int t = warp >> 2;
        const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const int key_off = t * kKeysPerTile + (warp & 3) * 32 + lane;
        const int n_sub = a.cols > kSubCols ? 2 : 1;
        const float c = a.c;
        int nq = -1, st = 0;
        bool ok = true;
        for (Segment sg(begin, end, a.n_tiles, a.n_pairs); ok && sg.more(); sg.next()) {
            float sum = 0.f;
            for (int i = 0; ok && i < sg.tiles; ++i) {
                if (sg.new_q) ++nq;
                const int slot = nq % kQSlots;
                if (sg.new_q && !(ok = ptx::mbar_wait(b_full + slot, (nq / kQSlots) & 1, abort_flag, a.err,
                                                      BLINK_DEVICE_TIMEOUT)))
                    break;
                const bool careful = slow[slot] != 0;
                for (int sub = 0; sub < n_sub; ++sub, ++st) {
                    const int buf = (st & 1) * 2 + t;
                    if (!(ok = ptx::mbar_wait(s_full + buf, (st >> 1) & 1, abort_flag, a.err, BLINK_DEVICE_TIMEOUT))) break;
                    ptx::tc_fence_after();
                    const float *bs = bias + slot * kMaxCols + sub * kSubCols;
                    const int cols = min(kSubCols, a.cols - sub * kSubCols);
                    float s0 = 0.f, s1 = 0.f;
                    for (int c0 = 0; c0 < cols; c0 += 32) {
                        uint32_t raw[32];
                        ptx::tmem_ld32(trow + buf * kSubCols + c0, raw);
                        ptx::tmem_wait_ld();
                        if (!careful) {
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                const float2 b = *reinterpret_cast<const float2 *>(bs + c0 + j);
                                s0 += ptx::ex2(fmaf(__uint_as_float(raw[j]), c, b.x));
                                s1 += ptx::ex2(fmaf(__uint_as_float(raw[j + 1]), c, b.y));
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const float b = bs[c0 + j];
                                s0 += b == -INFINITY ? 0.f : ptx::ex2(fmaf(__uint_as_float(raw[j]), c, b));
                            }
                        }
                    }
                    sum += s0 + s1;
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(s_empty + buf);
                }
                __syncwarp();
                if (ok && sg.last_use && lane == 0) ptx::mbar_arrive(b_empty + slot);
            }
            if (!ok) break;
            const int key = sg.key0 + key_off;
            if (sg.tiles == a.n_tiles) {
                if (key < a.P)
                    a.w[sg.head * a.w_stride + key] =
                        a.decay > 0.f ? fmaf(a.decay, a.prev[sg.head * a.prev_stride + key], sum) : sum;
            } else {
                a.part[(static_cast<int64_t>(blockIdx.x) * 2 + (sg.first ? 0 : 1)) * kUnitKeys + key_off] = sum;
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 0) ptx::tmem_dealloc(tmem, kTmem);
}

// One block per unit: adds the pieces of a unit that range boundaries cut, in block order.
__global__ void __launch_bounds__(kUnitKeys) key_weights_join_kernel(const KeyWeightArgs a, int blocks)
{
    ptx::grid_dep_wait();
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.n_tiles, hi = lo + a.n_tiles;
    const int b0 = static_cast<int>(((lo + 1) * blocks - 1) / a.total);  // the block that has step lo
    const int b1 = static_cast<int>((hi * blocks - 1) / a.total);        // and step hi - 1
    if (b0 == b1) return;
    const int head = blockIdx.x / a.n_pairs;
    const int key = (blockIdx.x - head * a.n_pairs) * kUnitKeys + threadIdx.x;
    if (key >= a.P) return;
    float sum = 0.f;
    for (int b = b0; b <= b1; ++b) {
        const int piece = first_step(b, a.total, blocks) >= lo ? 0 : 1;
        sum += __ldcg(a.part + (static_cast<int64_t>(b) * 2 + piece) * kUnitKeys + threadIdx.x);
    }
    a.w[head * a.w_stride + key] = a.decay > 0.f ? fmaf(a.decay, a.prev[head * a.prev_stride + key], sum) : sum;
}

int sm_count()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
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
    if (!q || !k_pre || !lse || !d_weights || !d_ws) return BLINK_INVALID_ARG;
    if (rows < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > 128 || (d != 64 && d != 128))
        return BLINK_INVALID_ARG;
    if (P < 1 || P > BLINK_MAX_INPUT_TOKENS || Hkv > 65535) return BLINK_OUT_OF_RANGE;
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
    a.tpt = kMaxCols / a.g < rows ? kMaxCols / a.g : rows;
    a.n_tiles = (rows + a.tpt - 1) / a.tpt;
    a.n_pairs = (P + kUnitKeys - 1) / kUnitKeys;
    a.cols = a.n_tiles > 1 ? kMaxCols : (a.g * a.tpt + 31) / 32 * 32;  // read from tensor memory 32 at a time
    a.q_slot_bytes = a.cols * d * 2;
    const int k_tile = kKeysPerTile * d * 2;
    a.k_slots = (kRingBytes - kQSlots * a.q_slot_bytes) / k_tile;
    if (a.k_slots > kMaxKSlots) a.k_slots = kMaxKSlots;
    a.total = static_cast<int64_t>(Hkv) * a.n_pairs * a.n_tiles;
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
                             kKeysPerTile))
        return BLINK_CUDA_ERROR;
    auto kern = d == 128 ? key_weights_kernel<128> : key_weights_kernel<64>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess)
        return BLINK_CUDA_ERROR;
    kern<<<static_cast<unsigned>(blocks), kThreadsKW, kSmemBytes, stream>>>(tm_q, tm_k, a);
    if (cudaGetLastError() != cudaSuccess) return BLINK_CUDA_ERROR;
    if (a.n_tiles == 1) return BLINK_OK;  // a unit of one step is never cut
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(Hkv * a.n_pairs));
    cfg.blockDim = dim3(kUnitKeys);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, key_weights_join_kernel, a, static_cast<int>(blocks)) != cudaSuccess)
        return BLINK_CUDA_ERROR;
    return BLINK_OK;
}
