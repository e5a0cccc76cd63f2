// evict.cu -- eviction of a cached prefix's lightest keys: per kv head the `keep` best of P keys are
// selected by accumulated attention weight, and the arena region is compacted to slots [0, keep).
//
// Selection.  Each weight becomes a 32-bit key whose unsigned order is the order of the keys
// (protected keys above every weight, NaN below); the keep-th largest key T is found by a radix
// select over 11 + 11 + 10 bits.  Kept are the keys above T and, of those equal to T, the lowest slots.
// One thread-block cluster per head, its blocks holding consecutive pieces of the head's keys in
// shared memory: the weights are read once, the per-block histograms are summed through distributed
// shared memory, and no global counter or atomic order enters the result.
//
// Compaction.  Kept keys below slot `keep` stay; the r-th evicted slot below `keep` (a hole) takes the
// r-th kept slot at `keep` or above (a survivor).  Sources are never destinations, so the moves of
// an in-place compaction need no order among themselves.
#include <cooperative_groups.h>

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace blink {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kMaxPiece = (BLINK_MAX_INPUT_TOKENS + kMaxCluster - 1) / kMaxCluster;  // keys of one block
constexpr int kMaxSteps = kMaxPiece / kSelThreads;                                    // 32-key steps of a warp

struct EvictArgs {
    const float *w;
    const int32_t *pos;  // or nullptr: slot = position
    int64_t w_stride, pos_stride;
    int P, keep, sink, recent_from, Hkv, piece;  // piece: keys per block, a multiple of kSelThreads
    int32_t *slots;                              // [Hkv][keep]
    int32_t *holes, *survivors;                  // [Hkv][min(keep, P - keep)]
};

// Larger weight = larger unsigned; NaN = 1, so that 0 is below every key and ~0 above.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w) return 1u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 becomes +0: equal weights are equal keys
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ bool is_protected(const EvictArgs &a, int head, int slot)
{
    const int p = a.pos ? __ldg(a.pos + head * a.pos_stride + slot) : slot;
    return p < a.sink || p >= a.recent_from;
}

// Sum over the block of one value per thread (every thread gets it).
__device__ __forceinline__ int block_sum(int v, int *warp_tot)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) warp_tot[threadIdx.x >> 5] = v;
    __syncthreads();
    int t = warp_tot[threadIdx.x & 31];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    __syncthreads();
    return t;
}

struct PieceCounts {  // of one block's or one warp's keys: above T and equal to T, slots below `keep` and not
    int gt_low, gt_high, eq_low, eq_high, n_low;
};

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictArgs a)
{
    extern __shared__ uint32_t keys[];  // [piece]
    __shared__ uint32_t hist[3][kBins];
    __shared__ int warp_tot[kSelWarps];
    __shared__ PieceCounts warp_cnt[kSelWarps];
    __shared__ PieceCounts block_cnt;
    __shared__ int n_protected;
    __shared__ uint32_t found_digit;
    __shared__ int found_rest;

    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int head = blockIdx.x / C;
    const int lo = rank * a.piece;
    const int n = max(0, min(a.P - lo, a.piece));  // this block's keys: slots [lo, lo + n)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int steps = a.piece / kSelThreads;
    // Warp w owns the consecutive keys [w * piece / 32, ...), 32 at a step, so ballots give slot order.
    const int wbase = warp * (a.piece / kSelWarps);

    for (int i = tid; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0u;
    const float *w = a.w + head * a.w_stride;
    uint32_t guard = 0u;
    int n_guard = 0;
    const bool guarded = a.sink > 0 || a.recent_from < 0x7FFFFFFF;
    for (int s = 0; s < steps; ++s) {
        const int i = wbase + s * 32 + lane;
        uint32_t key = 0u;
        if (i < n) {
            key = weight_key(__ldg(w + lo + i));
            if (guarded && is_protected(a, head, lo + i)) {
                guard |= 1u << s;
                ++n_guard;
            }
        }
        keys[i] = key;
    }
    if (guarded) {
        n_guard = block_sum(n_guard, warp_tot);
        if (tid == 0) n_protected = n_guard;
        cluster.sync();
        int total = 0;
        for (int c = 0; c < C; ++c) total += *cluster.map_shared_rank(&n_protected, c);
        // More protected keys than `keep`: the selection is among them alone.  Else they are all kept.
        for (int s = 0; s < steps; ++s) {
            const int i = wbase + s * 32 + lane;
            const bool g = (guard >> s) & 1u;
            if (total > a.keep) {
                if (!g) keys[i] = 0u;
            } else if (g) {
                keys[i] = 0xFFFFFFFFu;
            }
        }
    }
    __syncthreads();

    // ---- radix select of the keep-th largest key
    uint32_t prefix = 0u, mask = 0u;
    int want = a.keep;  // rank of the key looked for among those that match the prefix
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digit_mask = pass == 2 ? 1023u : 2047u;
        uint32_t *h = hist[pass];
        for (int s = 0; s < steps; ++s) {
            const int i = wbase + s * 32 + lane;
            const uint32_t key = keys[i];
            const bool in = i < n && (key & mask) == prefix;
            const uint32_t bin = (key >> shift) & digit_mask;
            const uint32_t act = __ballot_sync(0xFFFFFFFFu, in);
            if (act == 0u) continue;
            // a whole step in one bin (equal weights): one atomic instead of 32 on one address
            const uint32_t bin0 = __shfl_sync(0xFFFFFFFFu, bin, __ffs(act) - 1);
            if (__all_sync(0xFFFFFFFFu, !in || bin == bin0)) {
                if (lane == 0) atomicAdd(h + bin0, static_cast<uint32_t>(__popc(act)));
            } else if (in) {
                atomicAdd(h + bin, 1u);
            }
        }
        cluster.sync();
        // bins in descending order, two per thread: cluster-wide counts and their running sum
        const int b1 = kBins - 1 - 2 * tid, b0 = b1 - 1;
        int c1 = 0, c0 = 0;
        for (int c = 0; c < C; ++c) {
            const uint32_t *rh = cluster.map_shared_rank(h, c);
            const uint2 v = *reinterpret_cast<const uint2 *>(rh + b0);
            c0 += static_cast<int>(v.x);
            c1 += static_cast<int>(v.y);
        }
        int run = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, run, o);
            if (lane >= o) run += up;
        }
        if (lane == 31) warp_tot[warp] = run;
        __syncthreads();
        int before = lane < warp ? warp_tot[lane] : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
        run += before;                      // keys in bins >= b0
        const int above1 = run - c0 - c1;   // keys in bins > b1
        if (above1 < want && want <= above1 + c1) {
            found_digit = static_cast<uint32_t>(b1);
            found_rest = want - above1;
        } else if (above1 + c1 < want && want <= run) {
            found_digit = static_cast<uint32_t>(b0);
            found_rest = want - above1 - c1;
        }
        __syncthreads();
        prefix |= found_digit << shift;
        mask |= digit_mask << shift;
        want = found_rest;
        __syncthreads();
    }
    const uint32_t T = prefix;
    const int need = want;  // how many of the keys equal to T are kept: the lowest slots

    // ---- counts per warp and block, then every warp's place in the slot order
    PieceCounts my = {0, 0, 0, 0, 0};
    for (int s = 0; s < steps; ++s) {
        const int i = wbase + s * 32 + lane;
        const uint32_t key = keys[i];
        const bool in = i < n, low = lo + i < a.keep;
        my.gt_low += __popc(__ballot_sync(0xFFFFFFFFu, in && low && key > T));
        my.gt_high += __popc(__ballot_sync(0xFFFFFFFFu, in && !low && key > T));
        my.eq_low += __popc(__ballot_sync(0xFFFFFFFFu, in && low && key == T));
        my.eq_high += __popc(__ballot_sync(0xFFFFFFFFu, in && !low && key == T));
        my.n_low += __popc(__ballot_sync(0xFFFFFFFFu, in && low));
    }
    if (lane == 0) warp_cnt[warp] = my;
    __syncthreads();
    if (tid == 0) {
        PieceCounts t = {0, 0, 0, 0, 0};
        for (int i = 0; i < kSelWarps; ++i) {
            t.gt_low += warp_cnt[i].gt_low;
            t.gt_high += warp_cnt[i].gt_high;
            t.eq_low += warp_cnt[i].eq_low;
            t.eq_high += warp_cnt[i].eq_high;
            t.n_low += warp_cnt[i].n_low;
        }
        block_cnt = t;
    }
    cluster.sync();
    int eq_before = 0, hole = 0, surv = 0;  // in the slots before this warp's
    auto pass_over = [&](const PieceCounts &c) {
        const int take_low = max(0, min(c.eq_low, need - eq_before));
        const int take_high = max(0, min(c.eq_high, need - eq_before - c.eq_low));
        hole += c.n_low - c.gt_low - take_low;
        surv += c.gt_high + take_high;
        eq_before += c.eq_low + c.eq_high;
    };
    for (int c = 0; c < rank; ++c) pass_over(*cluster.map_shared_rank(&block_cnt, c));
    for (int i = 0; i < warp; ++i) pass_over(warp_cnt[i]);

    const int64_t list = static_cast<int64_t>(head) * min(a.keep, a.P - a.keep);
    int32_t *slots = a.slots + static_cast<int64_t>(head) * a.keep;
    const uint32_t below = (1u << lane) - 1u;
    for (int s = 0; s < steps; ++s) {
        const int i = wbase + s * 32 + lane;
        const int slot = lo + i;
        const uint32_t key = keys[i];
        const bool in = i < n, low = slot < a.keep;
        const uint32_t eq = __ballot_sync(0xFFFFFFFFu, in && key == T);
        const bool kept = in && (key > T || (key == T && eq_before + __popc(eq & below) < need));
        eq_before += __popc(eq);
        const uint32_t hm = __ballot_sync(0xFFFFFFFFu, in && low && !kept);
        const uint32_t sm = __ballot_sync(0xFFFFFFFFu, kept && !low);
        if (kept && low) slots[slot] = slot;
        if (in && low && !kept) a.holes[list + hole + __popc(hm & below)] = slot;
        if (kept && !low) a.survivors[list + surv + __popc(sm & below)] = slot;
        hole += __popc(hm);
        surv += __popc(sm);
    }
    // every block's lists are complete: the r-th hole takes the r-th survivor
    cluster.sync();
    int moved = 0, eqs = 0;
    for (int c = 0; c < C; ++c) {
        const PieceCounts bc = *cluster.map_shared_rank(&block_cnt, c);
        moved += bc.gt_high + max(0, min(bc.eq_high, need - eqs - bc.eq_low));
        eqs += bc.eq_low + bc.eq_high;
    }
    for (int r = rank * kSelThreads + tid; r < moved; r += C * kSelThreads)
        slots[__ldcg(a.holes + list + r)] = __ldcg(a.survivors + list + r);
    cluster.sync();  // no block leaves while another may still read its shared memory
}

struct MoveArgs {
    const uint4 *k, *v;  // 16-byte pieces
    uint4 *k_dst, *v_dst;
    int64_t row_stride, dst_stride;  // in 16-byte pieces
    const int32_t *slots;
    const float *w;
    float *w_dst;
    const int32_t *pos;
    int32_t *pos_dst;
    int64_t w_stride, wd_stride, pos_stride, pd_stride;
    int keep, Hkv, pieces;  // pieces: 16-byte pieces of one key (d / 8)
    int skip_k, skip_v, skip_w, skip_pos;  // in place: a key that stays is not copied
};

constexpr int kMoveThreads = 256;

// One thread per 16-byte piece of a destination row (pieces of a row contiguous), K and V together;
// the first piece's thread also moves the key's weight and position.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const MoveArgs a)
{
    ptx::grid_dep_wait();
    const int64_t row_pieces = static_cast<int64_t>(a.Hkv) * a.pieces;
    const int64_t total = row_pieces * a.keep;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; t < total;
         t += static_cast<int64_t>(gridDim.x) * kMoveThreads) {
        const int64_t j = t / row_pieces;
        const int64_t c = t - j * row_pieces;
        const int head = static_cast<int>(c / a.pieces);
        const int slot = __ldg(a.slots + static_cast<int64_t>(head) * a.keep + j);
        const bool stays = slot == j;
        const bool do_k = !(stays && a.skip_k), do_v = !(stays && a.skip_v);
        uint4 kv, vv;
        if (do_k) kv = __ldcs(a.k + slot * a.row_stride + c);
        if (do_v) vv = __ldcs(a.v + slot * a.row_stride + c);
        if (do_k) a.k_dst[j * a.dst_stride + c] = kv;
        if (do_v) a.v_dst[j * a.dst_stride + c] = vv;
        if (c == static_cast<int64_t>(head) * a.pieces) {
            if (a.w_dst && !(stays && a.skip_w)) a.w_dst[head * a.wd_stride + j] = a.w[head * a.w_stride + slot];
            if (a.pos_dst && !(stays && a.skip_pos))
                a.pos_dst[head * a.pd_stride + j] = a.pos ? a.pos[head * a.pos_stride + slot] : slot;
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
    if (P < 1 || keep < 1 || keep > P || Hkv < 1) return kHeaderBytes;
    const size_t list = static_cast<size_t>(keep < P - keep ? keep : P - keep) * Hkv * sizeof(int32_t);
    return kHeaderBytes + 2 * align_up(list, 256);
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
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_dst) || !aligned16(v_dst)) return BLINK_INVALID_ARG;
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
    e.Hkv = Hkv;
    int C = 1;  // blocks per head: pieces of 1024 keys and more, at most kMaxCluster of them
    while (C < kMaxCluster && P > C * kSelThreads) C *= 2;
    e.piece = (P + C * kSelThreads - 1) / (C * kSelThreads) * kSelThreads;
    e.slots = d_slots;
    const size_t list = align_up(static_cast<size_t>(keep < P - keep ? keep : P - keep) * Hkv * sizeof(int32_t), 256);
    e.holes = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(d_ws) + kHeaderBytes);
    e.survivors = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(d_ws) + kHeaderBytes + list);

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
    m.slots = d_slots;
    m.w = d_weights;
    m.w_dst = d_weights_dst;
    m.pos = d_pos;
    m.pos_dst = d_pos_dst;
    m.w_stride = w_stride;
    m.wd_stride = wd_stride;
    m.pos_stride = pos_stride;
    m.pd_stride = pd_stride;
    m.keep = keep;
    m.Hkv = Hkv;
    m.pieces = d / 8;
    m.skip_k = k_in;
    m.skip_v = v_in;
    m.skip_w = w_in;
    m.skip_pos = p_in;
    const int64_t total = static_cast<int64_t>(keep) * Hkv * m.pieces;
    const int64_t blocks = (total + kMoveThreads - 1) / kMoveThreads;
    const unsigned grid = static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20));
    evict_move_kernel<<<grid, kMoveThreads, 0, stream>>>(m);
    if (cudaGetLastError() != cudaSuccess) return BLINK_CUDA_ERROR;
    return BLINK_OK;
}
