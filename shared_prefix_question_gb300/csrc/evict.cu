// evict.cu -- eviction of a cached prefix's lightest keys (blink_kv_evict): per kv head the `keep` best of
// P keys are selected by accumulated attention weight, and the arena region is compacted to slots
// [0, keep).
//
// Selection.  Each weight becomes a 32-bit key whose unsigned order is the order of the keys
// (protected keys above every weight, NaN below); the keep-th largest key T is found by a radix
// select over four digits of 8 bits, which stops early when all keys of the digit found are kept.  Kept
// are the keys above T and, of those equal to T, the lowest slots.
// One thread-block cluster per head, its blocks holding consecutive pieces of the head's keys in
// shared memory: the weights are read once, the per-block histograms are summed through distributed
// shared memory, and no global counter or atomic order enters the result.  A few thousand keys take a
// block microseconds either way, so what it costs is the chain of barriers and remote reads, 3,400 cycles
// a digit with 8 blocks of 2304 keys: digits are small (with 2048 bins the blocks read 64 KB of one
// another's histograms a digit, 4 us), a thread sums a bin over the blocks, every warp finds the digit
// for itself, and there is nothing in global memory between the steps.  The blocks hand each other their
// counts by writing them before the last barrier, so that none has to wait for another's reads at its end.
//
// Compaction.  Kept keys below slot `keep` stay; the r-th evicted slot below `keep` (a hole) takes the
// r-th kept slot at `keep` or above (a survivor).  Sources are never destinations, so the moves of
// an in-place compaction need no order among themselves.  The selection writes each slot's source, or the
// rank of its survivor, and the survivors' slots; a second launch, its programmatic dependent, joins the two
// and moves keys, values, weights and positions.  (Joined in the selection, through the blocks' shared
// memory, they cost it another 5 us of 32 at 131072 keys.)
//
// 8 kv heads of width 128, warm / with a cold L2: 9216 of 18432 keys 21 / 30 us (selection 10,
// move 11), 32768 of 131072 keys 70 / 75 us (selection 25, move 42).  The move of the
// largest runs at the copy rate; the selection's chain of barriers is what is left over it.
#include <cooperative_groups.h>

#include <climits>
#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace blink {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kDigits = 4, kBins = 256;
constexpr int kMaxPiece = (BLINK_MAX_INPUT_TOKENS + kMaxCluster - 1) / kMaxCluster;  // keys of one block
// Keys per block before a head gets more blocks.  18432 x 8: 22.5 us for the call with 4096, 26.1 with 8192
// (2048 the same as 4096: the cluster is full).
constexpr int kClusterPiece = 4096;
constexpr int kLoadAhead = 8;
constexpr int kFetchAhead = 16;  // weights and positions a thread has in flight (8: 131072 keys take 1 us more)

struct EvictArgs {
    const float *w;
    const int32_t *pos;  // or nullptr: slot = position
    int64_t w_stride, pos_stride;
    int P, keep, sink, recent_from;
    int piece;                  // keys per block, a multiple of kSelThreads
    int32_t *from, *survivors;  // [Hkv][keep]: a destination slot's source, or ~r for the head's r-th survivor; their slots
};

// Larger weight = larger unsigned; NaN = 1, so that 0 is below every key and ~0 above.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w) return 1u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 becomes +0: equal weights are equal keys
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xFFFFFFFFu, v); }

// Sum of the lanes before this one.
__device__ __forceinline__ int sum_before(int v, int lane)
{
    int run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, run, o);
        if (lane >= o) run += up;
    }
    return run - v;
}

struct PieceCounts {  // of one block's or one warp's keys: above T and equal to T, slots below `keep` and not
    int gt_low, gt_high, eq_low, eq_high, n_low;
};

// Bits [0, n) of a mask, n of any size.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// With `eq_before` keys equal to T in lower slots: holes and survivors among the counted keys.
__device__ __forceinline__ int2 holes_and_survivors(const PieceCounts &c, int eq_before, int need)
{
    const int take_low = max(0, min(c.eq_low, need - eq_before));
    const int take_high = max(0, min(c.eq_high, need - eq_before - c.eq_low));
    return make_int2(c.n_low - c.gt_low - take_low, c.gt_high + take_high);
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictArgs a)
{
    extern __shared__ uint32_t keys[];  // [piece]
    __shared__ __align__(16) uint32_t hist[kDigits][kBins];
    __shared__ PieceCounts warp_cnt[kSelWarps];
    __shared__ PieceCounts block_cnt[kMaxCluster];  // written by the blocks themselves
    __shared__ int n_protected;
    __shared__ __align__(16) int total[kBins];  // a digit's histogram over the blocks
    __shared__ bool too_many;

    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int head = blockIdx.x / C;
    const int lo = rank * a.piece;
    const int n = max(0, min(a.P - lo, a.piece));  // this block's keys: slots [lo, lo + n)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int steps = a.piece / kSelThreads;
    const uint32_t below = (1u << lane) - 1u;
    // Warp w owns the consecutive keys [w * piece / warps, ...), 32 at a step, so ballots give slot order.
    const int wbase = warp * (a.piece / kSelWarps);
    auto sync_all = [&] {
        if (C > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    ptx::grid_launch_dependents();

    const float *w = a.w + head * a.w_stride;
    const int32_t *pos = a.pos ? a.pos + head * a.pos_stride : nullptr;
    const bool recent = a.recent_from < INT_MAX;
    const bool guarded = a.sink > 0 || recent;
    // Fills keys[]; returns how many of this thread's keys are protected.  `among_them`: only protected
    // keys are candidates (there are more than `keep`); otherwise protected keys come before all others.
    auto load_keys = [&](bool among_them) {
        int n_guard = 0;
        for (int s0 = 0; s0 < steps; s0 += kFetchAhead) {
            float x[kFetchAhead];
            int p[kFetchAhead];
#pragma unroll
            for (int u = 0; u < kFetchAhead; ++u) {
                const int i = wbase + (s0 + u) * 32 + lane;
                const bool in = s0 + u < steps && i < n;
                x[u] = in ? __ldg(w + lo + i) : 0.f;
                p[u] = in && guarded ? (pos ? __ldg(pos + lo + i) : lo + i) : INT_MAX;
            }
#pragma unroll
            for (int u = 0; u < kFetchAhead; ++u) {
                const int i = wbase + (s0 + u) * 32 + lane;
                if (s0 + u >= steps) break;
                const bool g = guarded && i < n && (p[u] < a.sink || (recent && p[u] >= a.recent_from));
                n_guard += g;
                uint32_t key = weight_key(x[u]);
                if (among_them)
                    key = g ? key : 0u;
                else if (g)
                    key = 0xFFFFFFFFu;
                keys[i] = i < n ? key : 0u;
            }
        }
        return n_guard;
    };
    auto zero_hists = [&] {
        for (int i = tid; i < kDigits * kBins; i += kSelThreads) (&hist[0][0])[i] = 0u;
    };

    if (tid == 0) n_protected = 0;
    zero_hists();
    __syncthreads();
    {
        const int g = warp_sum(load_keys(false));
        if (lane == 0 && g > 0) atomicAdd(&n_protected, g);
    }
    __syncthreads();

    // ---- radix select of the keep-th largest key
    uint32_t prefix = 0u, mask = 0u;
    int want = a.keep;  // rank of the key looked for among those that match the prefix
    bool among = false, all_equal = false;
    for (int pass = 0; pass < kDigits; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int s0 = 0; s0 < steps; s0 += kLoadAhead) {
            uint32_t key[kLoadAhead];
#pragma unroll
            for (int u = 0; u < kLoadAhead; ++u) key[u] = s0 + u < steps ? keys[wbase + (s0 + u) * 32 + lane] : 0u;
#pragma unroll
            for (int u = 0; u < kLoadAhead; ++u)  // no key in range is 0, and padding is
                if (key[u] != 0u && (key[u] & mask) == prefix)
                    atomicAdd(&hist[pass][(key[u] >> shift) & 255u], 1u);
        }
        sync_all();
        if (tid < kBins) {
            int sum = 0;
#pragma unroll 8
            for (int c = 0; c < C; ++c) sum += static_cast<int>(*cluster.map_shared_rank(&hist[pass][tid], c));
            total[tid] = sum;
        } else if (pass == 0 && guarded && warp == kBins / 32) {
            const int guards = warp_sum(lane < C ? *cluster.map_shared_rank(&n_protected, lane) : 0);
            if (lane == 0) too_many = !among && guards > a.keep;
        }
        __syncthreads();
        // every warp: lane l has the bins 255 - 8 l down to 248 - 8 l
        const int b0 = kBins - 8 - 8 * lane;
        const int4 t1 = *reinterpret_cast<const int4 *>(total + b0 + 4), t0 = *reinterpret_cast<const int4 *>(total + b0);
        const int cnt[8] = {t1.w, t1.z, t1.y, t1.x, t0.w, t0.z, t0.y, t0.x};
        const int mine = ((t1.w + t1.z) + (t1.y + t1.x)) + ((t0.w + t0.z) + (t0.y + t0.x));
        int above = sum_before(mine, lane);  // keys in the bins above this lane's
        const bool here = above < want && want <= above + mine;
        uint32_t digit = 0u;
        int rest = 0, count = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (above < want && want <= above + cnt[q]) {
                digit = static_cast<uint32_t>(b0 + 7 - q);
                rest = want - above;
                count = cnt[q];
            }
            above += cnt[q];
        }
        if (pass == 0 && guarded && too_many) {
            // More protected keys than `keep` (seldom): again, among them alone.
            among = true;
            sync_all();  // every block has read the histograms
            zero_hists();
            load_keys(true);
            __syncthreads();
            pass = -1;
            continue;
        }
        const int from = __ffs(static_cast<int>(__ballot_sync(0xFFFFFFFFu, here))) - 1;
        prefix |= __shfl_sync(0xFFFFFFFFu, digit, from) << shift;
        mask |= 255u << shift;
        want = __shfl_sync(0xFFFFFFFFu, rest, from);
        // every key with this prefix is kept: T is the lowest it could be
        all_equal = want == __shfl_sync(0xFFFFFFFFu, count, from);
        if (all_equal) break;
    }
    const uint32_t T = max(prefix, 1u);  // no key is 0: the padding is below T
    const int need = want;  // unless all of them are: how many of the keys equal to T are kept, the lowest slots
    auto above_T = [&](uint32_t key) { return all_equal ? key >= T : key > T; };

    // ---- counts per warp and block, then every warp's place in the slot order
    const int left_low = min(n, a.keep - lo) - wbase;  // this warp's keys below `keep`
    uint32_t seen = 0u;  // bytes: above T below `keep` and not, equal to T likewise; a thread has at most 32 keys
#pragma unroll 8
    for (int s = 0; s < steps; ++s) {
        const int i = wbase + s * 32 + lane;
        const uint32_t key = keys[i];
        const uint32_t one = above_T(key) ? 1u : key == T ? 0x10000u : 0u;
        seen += lo + i < a.keep ? one : one << 8;
    }
    static_assert(kMaxPiece / kSelThreads < 256, "a thread's counts are bytes");
    const int in_low = static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, seen & 0x00FF00FFu));
    const int in_high = static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, seen >> 8 & 0x00FF00FFu));
    const PieceCounts my = {in_low & 0xFFFF, in_high & 0xFFFF, in_low >> 16, in_high >> 16, max(0, min(left_low, steps * 32))};
    if (lane == 0) warp_cnt[warp] = my;
    __syncthreads();
    const PieceCounts none = {0, 0, 0, 0, 0};
    const PieceCounts wc = lane < kSelWarps ? warp_cnt[lane] : none;  // lane l: warp l
    if (warp == 0) {
        const PieceCounts t = {warp_sum(wc.gt_low), warp_sum(wc.gt_high), warp_sum(wc.eq_low), warp_sum(wc.eq_high),
                               warp_sum(wc.n_low)};
        if (lane < C) *cluster.map_shared_rank(&block_cnt[rank], lane) = t;
    }
    sync_all();  // the last access to another block's memory is behind it
    const PieceCounts bc = lane < C ? block_cnt[lane] : none;  // lane l: block l
    const int bc_eq_before = sum_before(bc.eq_low + bc.eq_high, lane);
    const int2 bc_hs = holes_and_survivors(bc, bc_eq_before, need);
    int eq_before = __shfl_sync(0xFFFFFFFFu, bc_eq_before, rank);
    int hole = warp_sum(lane < rank ? bc_hs.x : 0), surv = warp_sum(lane < rank ? bc_hs.y : 0);
    const int wc_eq_before = eq_before + sum_before(wc.eq_low + wc.eq_high, lane);
    const int2 wc_hs = holes_and_survivors(wc, wc_eq_before, need);
    eq_before = __shfl_sync(0xFFFFFFFFu, wc_eq_before, warp);
    hole += warp_sum(lane < warp ? wc_hs.x : 0);
    surv += warp_sum(lane < warp ? wc_hs.y : 0);

    int32_t *from = a.from + static_cast<int64_t>(head) * a.keep;
    int32_t *survivors = a.survivors + static_cast<int64_t>(head) * a.keep;
#pragma unroll 4
    for (int s = 0; s < steps; ++s) {
        const int slot = lo + wbase + s * 32 + lane;
        const uint32_t key = keys[wbase + s * 32 + lane];
        const uint32_t low = low_bits(left_low - s * 32);
        uint32_t kept = __ballot_sync(0xFFFFFFFFu, above_T(key));
        if (!all_equal) {
            const uint32_t eq = __ballot_sync(0xFFFFFFFFu, key == T);
            kept |= __ballot_sync(0xFFFFFFFFu, key == T && eq_before + __popc(eq & below) < need);
            eq_before += __popc(eq);
        }
        const uint32_t holes = low & ~kept, moves = kept & ~low;
        if (low >> lane & 1u) from[slot] = kept >> lane & 1u ? slot : ~(hole + __popc(holes & below));
        if (moves >> lane & 1u) survivors[surv + __popc(moves & below)] = slot;
        hole += __popc(holes);
        surv += __popc(moves);
    }
}

struct MoveArgs {
    const uint4 *k, *v;  // 16-byte pieces
    uint4 *k_dst, *v_dst;
    int64_t row_stride, dst_stride;  // in 16-byte pieces
    const int32_t *from, *survivors;
    int32_t *slots;
    const float *w;
    float *w_dst;  // or nullptr
    const int32_t *pos;
    int32_t *pos_dst;  // or nullptr
    int64_t w_stride, wd_stride, pos_stride, pd_stride;
    unsigned row_blocks, head_groups;
    int Hkv, keep, pieces;  // pieces: of one key (d / 8)
    int skip_k, skip_v;            // in place: a key that stays is not copied
};

// Coherent loads: the selection writes both lists while this kernel is resident already.
__device__ __forceinline__ int source_slot(const MoveArgs &a, int64_t head, int64_t j)
{
    const int f = __ldcg(a.from + head * a.keep + j);
    return f >= 0 ? f : __ldcg(a.survivors + head * a.keep + ~f);
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 16;  // destination rows of a block (32: 27 us instead of 22 for 18432 keys; 8 the same)
constexpr int kMoveHeads = 64;  // and heads
constexpr int kMoveAhead = 4;

// A thread moves 16-byte pieces of destination rows, K and V, kMoveAhead of them in flight together.  The
// blocks after those of the rows move the weights and positions, a key each thread (done by the thread of a
// key's first piece they cost 5 us of the 12 that 18k rows take, in 4-byte writes all over).
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const MoveArgs a)
{
    ptx::grid_dep_wait();
    if (blockIdx.x >= a.row_blocks) {
        const int64_t t = static_cast<int64_t>(blockIdx.x - a.row_blocks) * kMoveThreads + threadIdx.x;
        const int64_t head = t / a.keep, j = t - head * a.keep;
        if (head >= a.Hkv) return;
        const int slot = source_slot(a, head, j);
        a.slots[t] = slot;
        if (a.w_dst) a.w_dst[head * a.wd_stride + j] = a.w[head * a.w_stride + slot];
        if (a.pos_dst) a.pos_dst[head * a.pd_stride + j] = a.pos ? a.pos[head * a.pos_stride + slot] : slot;
        return;
    }
    __shared__ int slot_of[kMoveRows * kMoveHeads];  // [head][row]
    const unsigned tile = blockIdx.x / a.head_groups;
    const int h0 = static_cast<int>(blockIdx.x - tile * a.head_groups) * kMoveHeads;
    const int heads = min(kMoveHeads, a.Hkv - h0);
    const int64_t j0 = static_cast<int64_t>(tile) * kMoveRows;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kMoveRows), a.keep - j0));
    for (int i = threadIdx.x; i < heads * kMoveRows; i += kMoveThreads) {
        const int row = i % kMoveRows;
        if (row < rows) slot_of[i] = source_slot(a, h0 + i / kMoveRows, j0 + row);
    }
    __syncthreads();
    const int width = heads * a.pieces, total = rows * width;  // 16-byte pieces
    const int64_t c0 = static_cast<int64_t>(h0) * a.pieces;
    for (int t0 = threadIdx.x; t0 < total; t0 += kMoveThreads * kMoveAhead) {
        uint4 kv[kMoveAhead], vv[kMoveAhead];
        int64_t dst[kMoveAhead];
        bool do_k[kMoveAhead], do_v[kMoveAhead];
#pragma unroll
        for (int u = 0; u < kMoveAhead; ++u) {
            const int t = t0 + u * kMoveThreads;
            const int row = t / width, c = t - row * width;
            const int64_t j = j0 + row;
            const int slot = t < total ? slot_of[c / a.pieces * kMoveRows + row] : 0;
            do_k[u] = t < total && !(slot == j && a.skip_k);
            do_v[u] = t < total && !(slot == j && a.skip_v);
            dst[u] = j * a.dst_stride + c0 + c;
            const int64_t src = slot * a.row_stride + c0 + c;
            if (do_k[u]) kv[u] = __ldcs(a.k + src);
            if (do_v[u]) vv[u] = __ldcs(a.v + src);
        }
#pragma unroll
        for (int u = 0; u < kMoveAhead; ++u) {
            if (do_k[u]) a.k_dst[dst[u]] = kv[u];
            if (do_v[u]) a.v_dst[dst[u]] = vv[u];
        }
    }
}

// Whether rows of `width` bytes, `na` of them `sa` bytes apart from a, may share a byte with those of
// b.  Rows of one stride that interleave (K and V in one arena row) do not; other overlapping
// extents count as shared.
bool rows_overlap(const void *a, int64_t sa, int64_t na, const void *b, int64_t sb, int64_t nb, int64_t width)
{
    const int64_t pa = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a));
    const int64_t pb = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b));
    if (pa + (na - 1) * sa + width <= pb || pb + (nb - 1) * sb + width <= pa) return false;
    if (sa != sb || sa < 1) return true;
    const int64_t delta = ((pb - pa) % sa + sa) % sa;
    return !(delta >= width && sa - delta >= width);
}

}  // namespace
}  // namespace blink

extern "C" size_t blink_kv_evict_workspace(int32_t P, int32_t keep, int32_t Hkv)
{
    using namespace blink;
    (void)P;
    if (keep < 1 || Hkv < 1) return kHeaderBytes;
    return kHeaderBytes + 2 * sizeof(int32_t) * static_cast<size_t>(Hkv) * static_cast<size_t>(keep);
}

extern "C" blink_status blink_kv_evict(const float *d_weights, int64_t w_stride, const int32_t *d_pos,
                                       int64_t pos_stride, int32_t P, int32_t keep, int32_t sink, int32_t recent_from,
                                       int32_t Hkv, int32_t d, const blink_bf16 *k, const blink_bf16 *v,
                                       int64_t row_stride, blink_bf16 *k_dst, blink_bf16 *v_dst,
                                       int64_t dst_row_stride, int32_t *d_slots, float *d_weights_dst,
                                       int64_t wd_stride, int32_t *d_pos_dst, int64_t pd_stride, void *d_ws,
                                       size_t ws_bytes, cudaStream_t stream)
{
    using namespace blink;
    if (!d_weights || !k || !v || !k_dst || !v_dst || !d_slots || !d_ws) return BLINK_INVALID_ARG;
    if (P < 1 || P > BLINK_MAX_INPUT_TOKENS || keep < 1 || keep > P) return BLINK_OUT_OF_RANGE;
    if (Hkv < 1 || Hkv > 65535 || d < 8 || d > 1024) return BLINK_OUT_OF_RANGE;
    if (d % 8 != 0 || sink < 0 || recent_from < 0) return BLINK_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(Hkv) * d;
    if (row_stride < row || row_stride % 8 != 0 || dst_row_stride < row || dst_row_stride % 8 != 0)
        return BLINK_INVALID_ARG;
    if (w_stride < P && Hkv > 1) return BLINK_INVALID_ARG;
    if (d_pos && pos_stride < P && Hkv > 1) return BLINK_INVALID_ARG;
    if ((d_weights_dst && wd_stride < keep && Hkv > 1) || (d_pos_dst && pd_stride < keep && Hkv > 1))
        return BLINK_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_dst) || !aligned16(v_dst) || !aligned16(d_ws))
        return BLINK_INVALID_ARG;
    const bool k_in = k_dst == k && dst_row_stride == row_stride, v_in = v_dst == v && dst_row_stride == row_stride;
    const int64_t rb = row * 2, sb = row_stride * 2, db = dst_row_stride * 2;
    if ((!k_in && rows_overlap(k, sb, P, k_dst, db, keep, rb)) || (!v_in && rows_overlap(v, sb, P, v_dst, db, keep, rb)) ||
        rows_overlap(k, sb, P, v_dst, db, keep, rb) || rows_overlap(v, sb, P, k_dst, db, keep, rb) ||
        rows_overlap(k_dst, db, keep, v_dst, db, keep, rb))
        return BLINK_INVALID_ARG;
    const bool w_in = static_cast<const void *>(d_weights_dst) == d_weights && (wd_stride == w_stride || Hkv == 1);
    const bool p_in = d_pos_dst && d_pos_dst == d_pos && (pd_stride == pos_stride || Hkv == 1);
    auto lists_overlap = [&](const void *a, int64_t sa, int64_t na, const void *b, int64_t sb2, int64_t nb) {
        if (!a || !b) return false;
        const char *pa = static_cast<const char *>(a), *pb = static_cast<const char *>(b);
        return !(pa + ((Hkv - 1) * sa + na) * 4 <= pb || pb + ((Hkv - 1) * sb2 + nb) * 4 <= pa);
    };
    if ((!w_in && lists_overlap(d_weights, w_stride, P, d_weights_dst, wd_stride, keep)) ||
        (!p_in && lists_overlap(d_pos, pos_stride, P, d_pos_dst, pd_stride, keep)) ||
        lists_overlap(d_weights, w_stride, P, d_pos_dst, pd_stride, keep) ||
        lists_overlap(d_pos, pos_stride, P, d_weights_dst, wd_stride, keep) ||
        lists_overlap(d_weights_dst, wd_stride, keep, d_pos_dst, pd_stride, keep) ||
        lists_overlap(d_slots, keep, keep, d_weights, w_stride, P) ||
        lists_overlap(d_slots, keep, keep, d_pos, pos_stride, P) ||
        lists_overlap(d_slots, keep, keep, d_weights_dst, wd_stride, keep) ||
        lists_overlap(d_slots, keep, keep, d_pos_dst, pd_stride, keep))
        return BLINK_INVALID_ARG;
    if (ws_bytes < blink_kv_evict_workspace(P, keep, Hkv)) return BLINK_WORKSPACE_TOO_SMALL;

    EvictArgs e{};
    e.w = d_weights;
    e.pos = d_pos;
    e.w_stride = w_stride;
    e.pos_stride = pos_stride;
    e.P = P;
    e.keep = keep;
    e.sink = sink;
    e.recent_from = recent_from;
    int C = 1;  // blocks per head: pieces of kClusterPiece keys and more, at most kMaxCluster of them
    while (C < kMaxCluster && P > C * kClusterPiece) C *= 2;
    e.piece = (P + C * kSelThreads - 1) / (C * kSelThreads) * kSelThreads;
    e.from = reinterpret_cast<int32_t *>(static_cast<char *>(d_ws) + kHeaderBytes);
    e.survivors = e.from + static_cast<int64_t>(Hkv) * keep;

    const int smem = e.piece * static_cast<int>(sizeof(uint32_t));
    if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxPiece * static_cast<int>(sizeof(uint32_t))) != cudaSuccess)
        return BLINK_CUDA_ERROR;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(Hkv * C));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, evict_select_kernel, e) != cudaSuccess) return BLINK_CUDA_ERROR;

    MoveArgs m{};
    m.k = reinterpret_cast<const uint4 *>(k);
    m.v = reinterpret_cast<const uint4 *>(v);
    m.k_dst = reinterpret_cast<uint4 *>(k_dst);
    m.v_dst = reinterpret_cast<uint4 *>(v_dst);
    m.row_stride = row_stride / 8;
    m.dst_stride = dst_row_stride / 8;
    m.from = e.from;
    m.survivors = e.survivors;
    m.slots = d_slots;
    m.w = d_weights;
    m.w_dst = d_weights_dst;
    m.pos = d_pos;
    m.pos_dst = d_pos_dst;
    m.w_stride = w_stride;
    m.wd_stride = wd_stride;
    m.pos_stride = pos_stride;
    m.pd_stride = pd_stride;
    m.head_groups = static_cast<unsigned>((Hkv + kMoveHeads - 1) / kMoveHeads);
    m.row_blocks = m.head_groups * static_cast<unsigned>((keep + kMoveRows - 1) / kMoveRows);
    m.Hkv = Hkv;
    m.keep = keep;
    m.pieces = d / 8;
    m.skip_k = k_in;
    m.skip_v = v_in;
    cudaLaunchConfig_t mc = {};
    cudaLaunchAttribute ma[1];
    ma[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    ma[0].val.programmaticStreamSerializationAllowed = 1;
    const int64_t list_blocks = (static_cast<int64_t>(Hkv) * keep + kMoveThreads - 1) / kMoveThreads;
    mc.gridDim = dim3(m.row_blocks + static_cast<unsigned>(list_blocks));
    mc.blockDim = dim3(kMoveThreads);
    mc.stream = stream;
    mc.attrs = ma;
    mc.numAttrs = 1;
    if (cudaLaunchKernelEx(&mc, evict_move_kernel, m) != cudaSuccess) return BLINK_CUDA_ERROR;
    return BLINK_OK;
}
