// paged.cu -- writing the 8-bit paged cache (keys turned by their positions on the way), and the prefix-tail attention
// whose prefix is held in it.
#include <cmath>

#include "paged.cuh"
#include "ptx.cuh"
#include "rotary.cuh"

namespace blink {

blink_status check_cache(PagedCache &c, const void *k, const void *v, const void *ks, const void *vs, int64_t page_stride,
                         int64_t scale_stride, int32_t n_pages, int32_t page_tokens, int32_t Hkv, int32_t d)
{
    if (!k || !v || !ks || !vs) return BLINK_INVALID_ARG;
    if (Hkv < 1 || (d != 64 && d != 128)) return BLINK_INVALID_ARG;
    if (Hkv > BLINK_MAX_PAGED_HEADS || n_pages < 1) return BLINK_OUT_OF_RANGE;
    if (page_tokens != 16 && page_tokens != 32 && page_tokens != 64 && page_tokens != 128) return BLINK_INVALID_ARG;
    if (page_stride < static_cast<int64_t>(Hkv) * page_tokens * d || page_stride % 16 != 0 || scale_stride < Hkv)
        return BLINK_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v)) return BLINK_INVALID_ARG;
    c.k = static_cast<const uint8_t *>(k);
    c.v = static_cast<const uint8_t *>(v);
    c.k_scale = static_cast<const uint8_t *>(ks);
    c.v_scale = static_cast<const uint8_t *>(vs);
    c.page_stride = page_stride;
    c.scale_stride = scale_stride;
    c.n_pages = n_pages;
    c.log2_page = page_tokens == 16 ? 4 : page_tokens == 32 ? 5 : page_tokens == 64 ? 6 : 7;
    return BLINK_OK;
}

namespace {

// ------------------------------------------------------------------------------------------ append
struct AppendArgs {
    const uint16_t *k, *v;
    int64_t k_stride, v_stride;  // elements
    uint8_t *kc, *vc, *ks, *vs;
    int64_t page_stride, scale_stride;
    const int32_t *table;
    int64_t table_stride;
    int table_width, n_pages;
    const int32_t *cu, *start, *pos;
    int n, max_new, Hkv, heads_per_block, log2_page;
    const uint64_t *turns;
    int rot;
    float amplitude;
    int *err;
};

// The exponent of the scale of a page whose largest magnitude is m >= 0 (finite): the smallest e with m <= 448 * 2^e,
// 448 = 0.875 * 2^9 being the largest code.
__device__ __forceinline__ int scale_exponent(float m)
{
    const uint32_t b = __float_as_uint(m);
    const int e = static_cast<int>(b >> 23) - 126 - ((b & 0x7FFFFFu) <= 0x600000u ? 9 : 8);
    return m > 0.f ? min(max(e, kScaleMin), kScaleMax) : kScaleMin;
}

__device__ __forceinline__ uint2 requantised(uint2 w, float f)
{
    uint32_t *p = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float x0, x1, x2, x3;
        f16x2_split(e4m3x2_to_f16x2(p[e]), x0, x1);
        f16x2_split(e4m3x2_hi_to_f16x2(p[e]), x2, x3);
        p[e] = f32x2_to_e4m3x2(x0 * f, x1 * f) | f32x2_to_e4m3x2(x2 * f, x3 * f) << 16;
    }
    return w;
}

// The largest of the block's values, the same in all threads.  `part` has a place per warp; calls alternate between
// two of them, so that one barrier a call is enough.
__device__ __forceinline__ float block_max(float m, float *part)
{
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = part[0];
    for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) m = fmaxf(m, part[w]);
    return m;
}

// A block owns one page of a sequence and goes over some of its heads, K then V of each; a thread owns 16 values of
// one of the page's token slots, as two 16-byte pieces (a pair of halves that turn together).  The largest magnitude
// needs all of a page's new tokens before the first code is written, so the values wait in registers; those of the
// next (head, K or V) are loaded meanwhile.  Bound by HBM: 2 bytes read and 1 written a value.  The angles belong to
// the slot, so a thread computes its own once for all heads.
template <int D, int LAYOUT>
__global__ void __launch_bounds__(D * 8) append_kernel(const __grid_constant__ AppendArgs a)
{
    constexpr int kLanes = D / 16;  // threads of a token slot
    __shared__ float part[2][32];
    const int seq = blockIdx.z;
    const int c0 = __ldg(a.cu + seq) - __ldg(a.cu), n = __ldg(a.cu + seq + 1) - __ldg(a.cu + seq), start = __ldg(a.start + seq);
    if (n == 0) return;
    if (c0 < 0 || n < 0 || n > a.max_new || static_cast<int64_t>(c0) + n > a.n || start < 0) {
        if (threadIdx.x == 0) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
        return;
    }
    const int64_t index = (start >> a.log2_page) + static_cast<int64_t>(blockIdx.x), base = index << a.log2_page;
    if (base >= static_cast<int64_t>(start) + n) return;
    const int id = index < a.table_width ? __ldg(a.table + seq * a.table_stride + index) : -1;
    if (id < 0 || id >= a.n_pages) {
        if (threadIdx.x == 0) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
        return;
    }
    const int filled = static_cast<int>(max(start - base, static_cast<int64_t>(0)));  // tokens the page holds already
    const int slot = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int64_t token = base + slot - start;  // among the sequence's new ones
    const bool fresh = token >= 0 && token < n, kept = slot < filled;

    // The thread's two pieces of eight values.
    int p0 = lane, p1 = lane + kLanes;
    const int half = a.rot / 2;
    bool turn = LAYOUT != kNoRotation;
    if constexpr (LAYOUT == kHalves) {
        turn = lane < a.rot / 16;
        p0 = turn ? lane : a.rot / 8 + lane - a.rot / 16;
        p1 = p0 + (turn ? a.rot / 16 : (D - a.rot) / 16);
    }
    const int32_t pos = !fresh ? 0 : a.pos ? __ldg(a.pos + c0 + token) : static_cast<int32_t>(start + token);
    float c[8], s[8];
    if constexpr (LAYOUT == kHalves || LAYOUT == kInterleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = LAYOUT == kHalves ? p0 * 8 + e : (e < 4 ? p0 * 4 + e : p1 * 4 + e - 4);
            c[e] = 1.f;
            s[e] = 0.f;
            if (fresh && turn && i < half) turn_cos_sin(__ldg(a.turns + i), pos, a.amplitude, c[e], s[e]);
        }
    }

    const int h_begin = blockIdx.y * a.heads_per_block, h_end = min(a.Hkv, h_begin + a.heads_per_block);
    const int64_t row = c0 + token;
    uint4 next[2];
    auto load = [&](int h, int t) {
        if (!fresh) return;
        const uint16_t *x = t ? a.v + row * a.v_stride : a.k + row * a.k_stride;
        const uint4 *q = reinterpret_cast<const uint4 *>(x + static_cast<int64_t>(h) * D);
        next[0] = __ldcs(q + p0);
        next[1] = __ldcs(q + p1);
    };
    load(h_begin, 0);
    int flip = 0;
    for (int h = h_begin; h < h_end; ++h) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint8_t *scale = (t ? a.vs : a.ks) + id * a.scale_stride + h;
            uint8_t *codes = (t ? a.vc : a.kc) + id * a.page_stride + (static_cast<int64_t>(h) << a.log2_page) * D +
                             slot * D;
            int e_old = kScaleMin;
            if (filled > 0) e_old = min(static_cast<int>(*reinterpret_cast<volatile uint8_t *>(scale)) - kScaleBias, kScaleMax);
            float x[16];
            float m = 0.f;
            if (fresh) {
                const uint32_t *u = reinterpret_cast<const uint32_t *>(next);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[2 * e] = bf16_lo(u[e]);
                    x[2 * e + 1] = bf16_hi(u[e]);
                }
                if (t == 0) {
                    if constexpr (LAYOUT == kHalves) {
                        if (turn) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float y = x[e], z = x[8 + e];
                                x[e] = y * c[e] - z * s[e];
                                x[8 + e] = y * s[e] + z * c[e];
                            }
                        }
                    } else if constexpr (LAYOUT == kInterleaved) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int i = e < 4 ? p0 * 4 + e : p1 * 4 + e - 4;
                            const float y = x[2 * e], z = x[2 * e + 1];
                            if (i < half) {  // pairs past rot stay as they are, whatever they hold
                                x[2 * e] = y * c[e] - z * s[e];
                                x[2 * e + 1] = y * s[e] + z * c[e];
                            }
                        }
                    } else if constexpr (LAYOUT == kHalvesByElement) {
                        const uint16_t *k = a.k + row * a.k_stride + static_cast<int64_t>(h) * D;
#pragma unroll 1
                        for (int e = 0; e < 16; ++e) {
                            const int j = (e < 8 ? p0 : p1) * 8 + (e & 7);
                            if (j >= a.rot) continue;
                            const int i = j < half ? j : j - half;
                            float cc, ss;
                            turn_cos_sin(__ldg(a.turns + i), pos, a.amplitude, cc, ss);
                            const float y = __uint_as_float(static_cast<uint32_t>(k[i]) << 16);
                            const float z = __uint_as_float(static_cast<uint32_t>(k[i + half]) << 16);
                            const float r = j < half ? y * cc - z * ss : y * ss + z * cc;
#pragma unroll
                            for (int f = 0; f < 16; ++f)
                                if (f == e) x[f] = r;
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]));  // a NaN counts as nothing
            }
            if (t == 0)
                load(h, 1);
            else if (h + 1 < h_end)
                load(h + 1, 0);
            m = block_max(m, part[flip]);
            flip ^= 1;
            if (m == INFINITY) {  // the scale is that of the finite values; infinities take the largest code
                m = 0.f;
                if (fresh) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]) < INFINITY ? fabsf(x[e]) : 0.f);
                }
                m = block_max(m, part[flip]);
                flip ^= 1;
            }
            const int e = filled > 0 ? max(scale_exponent(m), e_old) : scale_exponent(m);
            if (fresh) {
                const float f = scale_of(-e);
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = f32x2_to_e4m3x2(x[4 * i] * f, x[4 * i + 1] * f) |
                           f32x2_to_e4m3x2(x[4 * i + 2] * f, x[4 * i + 3] * f) << 16;
                reinterpret_cast<uint2 *>(codes)[p0] = make_uint2(w[0], w[1]);
                reinterpret_cast<uint2 *>(codes)[p1] = make_uint2(w[2], w[3]);
            } else if (kept && e > e_old) {
                const float f = scale_of(e_old - e);
                uint2 *w = reinterpret_cast<uint2 *>(codes);
                w[p0] = requantised(w[p0], f);
                w[p1] = requantised(w[p1], f);
            }
            if (threadIdx.x == 0) *scale = static_cast<uint8_t>(e + kScaleBias);
        }
    }
}

// ------------------------------------------------------------------------------------------ pages to rows
constexpr int kMaxRequests = 64;
constexpr int kTile = 128;  // a region's rows are a multiple of the attention's key tile: zeros past its last token

struct GatherArgs {
    PagedCache c;
    const int32_t *table;
    int64_t table_stride;
    int Hkv;
    int64_t first[kMaxRequests];  // row of each request's region
    int len[kMaxRequests];
    uint16_t *k, *v;              // [rows][Hkv][D]
    int *err;
};

constexpr int kGatherThreads = 256;

// The prefix pages of each request as bf16 rows of a contiguous region (codes times scales are exact in bf16), so
// that the tensor-core attention reads them by its tensor maps: 2 bytes read and 4 written a key and channel, once
// per call, against hundreds of products a byte in the attention.  A thread turns 16 codes of K and of V.
template <int D>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherArgs a)
{
    constexpr int kPieces = D / 16;
    const int r = blockIdx.y;
    const int len = a.len[r], padded = (len + kTile - 1) / kTile * kTile;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kGatherThreads + threadIdx.x;
    const int piece = static_cast<int>(item % kPieces);
    const int64_t th = item / kPieces;
    const int h = static_cast<int>(th % a.Hkv);
    const int64_t token = th / a.Hkv;
    if (token >= padded) return;
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    float fk = 0.f, fv = 0.f;
    if (token < len) {
        const int id = __ldg(a.table + r * a.table_stride + (token >> a.c.log2_page));
        if (id < 0 || id >= a.c.n_pages) {
            atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
        } else {
            const int64_t at = id * a.c.page_stride +
                               ((static_cast<int64_t>(h) << a.c.log2_page) + (token & ((1 << a.c.log2_page) - 1))) * D + piece * 16;
            k = __ldg(reinterpret_cast<const uint4 *>(a.c.k + at));
            v = __ldg(reinterpret_cast<const uint4 *>(a.c.v + at));
            fk = scale_of(static_cast<int>(__ldg(a.c.k_scale + id * a.c.scale_stride + h)) - kScaleBias);
            fv = scale_of(static_cast<int>(__ldg(a.c.v_scale + id * a.c.scale_stride + h)) - kScaleBias);
        }
    }
    auto put = [&](const uint4 &codes, float f, uint16_t *dst) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&codes);
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x0, x1, x2, x3;
            f16x2_split(e4m3x2_to_f16x2(w[e]), x0, x1);
            f16x2_split(e4m3x2_hi_to_f16x2(w[e]), x2, x3);
            o[2 * e] = ptx::pack_bf16x2(x0 * f, x1 * f);
            o[2 * e + 1] = ptx::pack_bf16x2(x2 * f, x3 * f);
        }
        ptx::st_global_v8(dst, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
    };
    const int64_t to = ((a.first[r] + token) * a.Hkv + h) * D + piece * 16;
    put(k, fk, a.k + to);
    put(v, fv, a.v + to);
}

// The workspace of the prefix-tail call: the attention's own, then the regions of K, then those of V.
struct TailLayout {
    size_t k, v, total;
    int64_t rows;
};

TailLayout tail_layout(const int32_t *h_len, int n_req, int32_t rows, int32_t B, int32_t Hq, int32_t Hkv, int32_t d)
{
    TailLayout l{};
    for (int r = 0; r < n_req; ++r) l.rows += (h_len[r] + kTile - 1) / kTile * kTile;
    const size_t bytes = align_up(static_cast<size_t>(l.rows) * Hkv * d * 2, 256);
    l.k = align_up(blink_attention_workspace(rows, B, n_req == 1 ? h_len[0] : 0, Hq, Hkv, d), 256);
    l.v = l.k + bytes;
    l.total = l.v + bytes;
    return l;
}

blink_status check_requests(const int32_t *h_req_rows, const int32_t *h_len, int32_t n_req, int32_t rows)
{
    if (!h_req_rows || !h_len) return BLINK_INVALID_ARG;
    if (n_req < 1 || n_req > kMaxRequests) return BLINK_OUT_OF_RANGE;
    if (h_req_rows[0] != 0 || h_req_rows[n_req] != rows) return BLINK_INVALID_ARG;
    for (int r = 0; r < n_req; ++r) {
        if (h_req_rows[r + 1] < h_req_rows[r] || h_len[r] < 0) return BLINK_INVALID_ARG;
        if (h_len[r] > BLINK_MAX_INPUT_TOKENS) return BLINK_OUT_OF_RANGE;
    }
    return BLINK_OK;
}

}  // namespace
}  // namespace blink

extern "C" size_t blink_paged_append_workspace(void) { return blink::kHeaderBytes; }

extern "C" blink_status blink_paged_append(const blink_bf16 *k, int64_t k_stride, const blink_bf16 *v, int64_t v_stride,
                                           int32_t n, int32_t Hkv, int32_t d, uint8_t *k_codes, uint8_t *v_codes,
                                           uint8_t *k_scale, uint8_t *v_scale, int64_t page_stride, int64_t scale_stride,
                                           int32_t n_pages, int32_t page_tokens, const int32_t *d_page_table,
                                           int64_t table_stride, int32_t table_width, const int32_t *d_cu_new,
                                           const int32_t *d_start, int32_t S, int32_t max_new, const int32_t *d_positions,
                                           const uint64_t *d_turns, int32_t rot, float amplitude, int32_t interleaved,
                                           void *d_ws, size_t ws_bytes, cudaStream_t stream)
{
    using namespace blink;
    PagedCache c;
    const blink_status st = check_cache(c, k_codes, v_codes, k_scale, v_scale, page_stride, scale_stride, n_pages, page_tokens, Hkv, d);
    if (st != BLINK_OK) return st;
    if (!k || !v || !d_page_table || !d_cu_new || !d_start || !d_ws) return BLINK_INVALID_ARG;
    if (n < 0 || max_new < 0 || table_width < 1 || (S > 1 && table_stride < table_width)) return BLINK_INVALID_ARG;
    if (S < 1 || S > BLINK_MAX_PLAN_SEQUENCES || max_new > BLINK_MAX_INPUT_TOKENS) return BLINK_OUT_OF_RANGE;
    const int64_t wide = static_cast<int64_t>(Hkv) * d;
    if (k_stride < wide || v_stride < wide || k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned16(k) || !aligned16(v))
        return BLINK_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return BLINK_INVALID_ARG;
    if (rot < 0 || rot > d || rot % 2 != 0 || (rot > 0 && (!d_turns || !std::isfinite(amplitude)))) return BLINK_INVALID_ARG;
    if (ws_bytes < kHeaderBytes) return BLINK_WORKSPACE_TOO_SMALL;
    if (n == 0 || max_new == 0) return BLINK_OK;

    AppendArgs a{};
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.kc = k_codes;
    a.vc = v_codes;
    a.ks = k_scale;
    a.vs = v_scale;
    a.page_stride = page_stride;
    a.scale_stride = scale_stride;
    a.table = d_page_table;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.n_pages = n_pages;
    a.cu = d_cu_new;
    a.start = d_start;
    a.pos = d_positions;
    a.n = n;
    a.max_new = max_new;
    a.Hkv = Hkv;
    a.log2_page = c.log2_page;
    a.turns = d_turns;
    a.rot = rot;
    a.amplitude = amplitude;
    a.err = &static_cast<WorkspaceHeader *>(d_ws)->error;
    // Pages that max_new tokens can touch, and the heads of a block: as many as leave the SMs four blocks each.
    const int pages = (max_new + page_tokens - 2) / page_tokens + 1;
    const int64_t busy = (static_cast<int64_t>(n) + page_tokens - 1) / page_tokens + S;
    const int64_t groups = (4LL * current_sm_count() + busy - 1) / busy;
    a.heads_per_block = groups >= Hkv ? 1 : static_cast<int>((Hkv + groups - 1) / groups);
    const dim3 grid(static_cast<unsigned>(pages), static_cast<unsigned>((Hkv + a.heads_per_block - 1) / a.heads_per_block),
                    static_cast<unsigned>(S));
    const unsigned threads = static_cast<unsigned>(page_tokens * (d / 16));
    const int layout = rot == 0 ? kNoRotation : interleaved ? kInterleaved : rot % 16 == 0 ? kHalves : kHalvesByElement;
    auto launch = [&](auto kern) { kern<<<grid, threads, 0, stream>>>(a); };
    if (d == 128) {
        if (layout == kNoRotation) launch(append_kernel<128, kNoRotation>);
        if (layout == kHalves) launch(append_kernel<128, kHalves>);
        if (layout == kInterleaved) launch(append_kernel<128, kInterleaved>);
        if (layout == kHalvesByElement) launch(append_kernel<128, kHalvesByElement>);
    } else {
        if (layout == kNoRotation) launch(append_kernel<64, kNoRotation>);
        if (layout == kHalves) launch(append_kernel<64, kHalves>);
        if (layout == kInterleaved) launch(append_kernel<64, kInterleaved>);
        if (layout == kHalvesByElement) launch(append_kernel<64, kHalvesByElement>);
    }
    return cudaGetLastError() == cudaSuccess ? BLINK_OK : BLINK_CUDA_ERROR;
}

extern "C" size_t blink_paged_prefix_tail_workspace(const int32_t *h_req_rows, const int32_t *h_prefix_len, int32_t n_req,
                                                    int32_t B, int32_t Hq, int32_t Hkv, int32_t d)
{
    using namespace blink;
    if (!h_req_rows || n_req < 1 || n_req > kMaxRequests || Hkv < 1 || d < 1 ||
        check_requests(h_req_rows, h_prefix_len, n_req, h_req_rows[n_req]) != BLINK_OK)
        return kHeaderBytes;
    return tail_layout(h_prefix_len, n_req, h_req_rows[n_req], B, Hq, Hkv, d).total;
}

extern "C" blink_status blink_paged_prefix_tail_attention(
    const blink_bf16 *q, const uint8_t *k_codes, const uint8_t *v_codes, const uint8_t *k_scale, const uint8_t *v_scale,
    int64_t page_stride, int64_t scale_stride, int32_t n_pages, int32_t page_tokens, const int32_t *d_page_table,
    int64_t table_stride, int32_t table_width, const blink_bf16 *k_tail, const blink_bf16 *v_tail,
    const int32_t *d_cu_seqlens, const int32_t *d_seq_start, int32_t B, int32_t rows, int32_t n_req,
    const int32_t *h_req_rows, const int32_t *h_prefix_len, int32_t max_tail, int32_t Hq, int32_t Hkv, int32_t d,
    float scale, blink_bf16 *out, float *lse, void *d_ws, size_t ws_bytes, cudaStream_t stream)
{
    using namespace blink;
    GatherArgs a{};
    blink_status st = check_cache(a.c, k_codes, v_codes, k_scale, v_scale, page_stride, scale_stride, n_pages, page_tokens, Hkv, d);
    if (st != BLINK_OK) return st;
    if (!d_page_table || !d_ws || rows < 1 || Hq < 1) return BLINK_INVALID_ARG;
    st = check_requests(h_req_rows, h_prefix_len, n_req, rows);
    if (st != BLINK_OK) return st;
    if (table_width < 1 || (n_req > 1 && table_stride < table_width)) return BLINK_INVALID_ARG;
    if (!q || !k_tail || !v_tail || !d_cu_seqlens || !out || max_tail < 1 || Hq % Hkv != 0 || Hq / Hkv > 128)
        return BLINK_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_tail) || !aligned16(v_tail) || !aligned16(out)) return BLINK_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(d_ws) % 32 != 0) return BLINK_INVALID_ARG;  // rows are written 32 bytes at a time
    if (std::isnan(scale) || std::isinf(scale)) return BLINK_INVALID_ARG;
    if (B < 1 || B > BLINK_MAX_PLAN_SEQUENCES || max_tail > BLINK_MAX_INPUT_TOKENS) return BLINK_OUT_OF_RANGE;
    int longest = 0;
    for (int r = 0; r < n_req; ++r) {
        if (h_prefix_len[r] > static_cast<int64_t>(table_width) * page_tokens) return BLINK_OUT_OF_RANGE;
        longest = h_prefix_len[r] > longest ? h_prefix_len[r] : longest;
    }
    const TailLayout lay = tail_layout(h_prefix_len, n_req, rows, B, Hq, Hkv, d);
    if (lay.rows > 0x7FFFFFFF) return BLINK_OUT_OF_RANGE;
    if (ws_bytes < lay.total) return BLINK_WORKSPACE_TOO_SMALL;

    auto *ws = static_cast<uint8_t *>(d_ws);
    auto *ka = reinterpret_cast<blink_bf16 *>(ws + lay.k), *va = reinterpret_cast<blink_bf16 *>(ws + lay.v);
    int32_t first[kMaxRequests] = {};
    int64_t at = 0;
    for (int r = 0; r < n_req; ++r) {
        a.first[r] = at;
        first[r] = static_cast<int32_t>(at);
        a.len[r] = h_prefix_len[r];
        at += (h_prefix_len[r] + kTile - 1) / kTile * kTile;
    }
    if (longest > 0) {
        a.table = d_page_table;
        a.table_stride = table_stride;
        a.Hkv = Hkv;
        a.k = ka;
        a.v = va;
        a.err = &static_cast<WorkspaceHeader *>(d_ws)->error;
        const int64_t items = static_cast<int64_t>((longest + kTile - 1) / kTile * kTile) * Hkv * (d / 16);
        const dim3 grid(static_cast<unsigned>((items + kGatherThreads - 1) / kGatherThreads), static_cast<unsigned>(n_req));
        if (d == 128)
            gather_kernel<128><<<grid, kGatherThreads, 0, stream>>>(a);
        else
            gather_kernel<64><<<grid, kGatherThreads, 0, stream>>>(a);
        if (cudaGetLastError() != cudaSuccess) return BLINK_CUDA_ERROR;
    }
    const int64_t row = static_cast<int64_t>(Hkv) * d;
    if (n_req == 1)
        return blink_prefix_tail_attention(q, ka, va, row, k_tail, v_tail, d_cu_seqlens, d_seq_start, B, rows, h_prefix_len[0],
                                           max_tail, Hq, Hkv, d, scale, out, lse, d_ws, lay.k, stream);
    return blink_prefix_tail_attention_multi(q, ka, va, row, lay.rows, k_tail, v_tail, d_cu_seqlens, d_seq_start, B, rows, n_req,
                                             h_req_rows, first, h_prefix_len, max_tail, Hq, Hkv, d, scale, out, lse, d_ws,
                                             lay.k, stream);
}
