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
    int n, max_new, S, Hkv, heads_per_block, log2_page;
    bool packed;                 // the grid's x goes over the pages of all sequences, not over those of each
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

// The largest of the block's values of K and of V (none negative), the same in all threads.  `part` has a place per warp
// and value; calls alternate between two of them, so that one barrier a call is enough.
__device__ __forceinline__ void block_max(uint32_t &k, uint32_t &v, uint32_t (*part)[32])
{
    k = __reduce_max_sync(0xFFFFFFFFu, k);
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) part[0][warp] = k, part[1][warp] = v;
    __syncthreads();
    const bool on = lane < static_cast<int>(blockDim.x >> 5);
    k = __reduce_max_sync(0xFFFFFFFFu, on ? part[0][lane] : 0u);
    v = __reduce_max_sync(0xFFFFFFFFu, on ? part[1][lane] : 0u);
}

// |32-bit rotation - the exact one| <= kTurnError * (the sizes of the two rotated values).  In half steps of 32 bits, and
// relative to |x0| + |x1| <= sqrt(2) (|y0| + |y1|) / amplitude: cos and sin are off by 2, the amplitude and a product add
// one each; the sum adds one of y itself.
constexpr float kTurnError = 7.f * 5.9604645e-8f;

// A bit for each byte of w, lowest first, that is not 0.
__device__ __forceinline__ uint32_t nonzero_bytes(uint32_t w)
{
    return ((w | ((w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu)) & 0x80808080u) * 0x00204081u >> 28;
}

// Rotated values that the 32-bit rotation leaves between two codes (bit e of `mask`: value e of the thread's 16, eight
// from place j0 and eight from j1 of a head, all of them below rot): computed to some 40 bits, and the nearer code written.
// `factor`: the amplitude over the scale.
template <bool INTERLEAVED>
__device__ __noinline__ void write_nearer_codes(uint32_t mask, uint8_t *codes, const uint16_t *k, int j0, int j1, int half,
                                                const uint64_t *turns, int32_t pos, float factor)
{
    for (; mask; mask &= mask - 1) {
        const int e = __ffs(mask) - 1, j = e < 8 ? j0 + e : j1 + e - 8;
        const bool second = INTERLEAVED ? j & 1 : j >= half;
        const int i = INTERLEAVED ? j / 2 : second ? j - half : j;
        const float x0 = bf16_lo(k[INTERLEAVED ? 2 * i : i]), x1 = bf16_lo(k[INTERLEAVED ? 2 * i + 1 : i + half]);
        Two s, c;
        turn_cos_sin(__ldg(turns + i), pos, c, s);
        const Two f = {factor, 0.f};
        const Two y = mul(f, second ? add(mul({x0, 0.f}, s), mul({x1, 0.f}, c)) : add(mul({x0, 0.f}, c), mul({-x1, 0.f}, s)));
        const uint32_t two = f32x2_to_e4m3x2(y.h * (1.f - 0x1p-20f), y.h * (1.f + 0x1p-20f));
        float l, h;
        f16x2_split(e4m3x2_to_f16x2(two), l, h);
        const float middle = 0.5f * (l + h), past = (y.h - middle) + y.l;  // an exact difference, as the two are so near
        const bool up = past == 0.f ? two & 1u : (past > 0.f) == (y.h > 0.f);  // the second is the larger one
        codes[j] = static_cast<uint8_t>(up ? two >> 8 : two);
    }
}

__device__ __forceinline__ bool bad_lengths(int c0, int n, int start, int rows, int max_new)
{
    return c0 < 0 || n < 0 || n > max_new || static_cast<int64_t>(c0) + n > rows || start < 0;
}

// The sequence (x) and which of its pages that get tokens (y; < 0: none) a block has where the grid's x goes over those of all:
// sequence s has the places from cu[s] / page + 2 s on, enough for the pages that its tokens can touch (l tokens: at most
// (l + page - 2) / page + 1) wherever it starts.  One block looks at all lengths, as those of a bad sequence may have no place.
__device__ __noinline__ int2 packed_place(const int32_t *cu, const int32_t *start, int S, int rows, int max_new, int log2_page, int *err)
{
    const int64_t cu0 = __ldg(cu);
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int s = threadIdx.x; s < S; s += blockDim.x) {
            const int c = __ldg(cu + s), n = __ldg(cu + s + 1) - c;
            if (n != 0 && bad_lengths(static_cast<int>(c - cu0), n, __ldg(start + s), rows, max_new)) atomicCAS(err, 0, BLINK_DEVICE_FLAG);
        }
    auto first = [&](int s) { return ((__ldg(cu + s) - cu0) >> log2_page) + 2 * s; };
    const int seq = last_before(0, S, [&](int s) { return first(s) <= static_cast<int64_t>(blockIdx.x); });
    return make_int2(seq, static_cast<int>(max(static_cast<int64_t>(-1), blockIdx.x - first(seq))));
}

constexpr int kStages = 2;        // heads whose keys and values are in shared memory, one of them in use
constexpr int kSlots = 2;         // token slots of a thread
constexpr int kMaxBlockHeads = 8;

// A block owns one page of a sequence and goes over some of its heads; a thread owns 16 values of K and of V in each of two
// of the page's token slots, as two 16-byte pieces each (a pair of halves that turn together).  The largest magnitude needs
// all of a page's new tokens before the first code is written: one barrier a head, for K and V together.  Bound by
// HBM: 2 bytes read and 1 written a value; each thread copies its own pieces of the next heads into its own places
// in shared memory meanwhile (no registers, no barrier).  The angles belong to the slot, so a thread computes its own
// once for all heads.
// Codes are those of the exact rotation: where the 32-bit one is too near the border of two codes to tell (one value of
// some 10,000), a bit remembers it, and when the block's heads are done those values are computed to some 40 bits.  (In a page
// whose keys hold an infinity the 32-bit rotation decides.)  Values that pass and pairs of zeros are exact and never among them.
template <int D, int LAYOUT>
__global__ void __launch_bounds__(D * 4) append_kernel(const __grid_constant__ AppendArgs a)
{
    constexpr int kLanes = D / 16;  // threads of a token slot
    extern __shared__ uint4 ring[];
    __shared__ uint32_t part[2][2][32];
    __shared__ int16_t k_exponents[kMaxBlockHeads];
    ptx::grid_dep_wait();
    ptx::grid_launch_dependents();
    int seq = blockIdx.z, place = blockIdx.x;
    if (a.packed) {
        const int2 at = packed_place(a.cu, a.start, a.S, a.n, a.max_new, a.log2_page, a.err);
        seq = at.x;
        place = at.y;
    }
    const int c0 = __ldg(a.cu + seq) - __ldg(a.cu), n = __ldg(a.cu + seq + 1) - __ldg(a.cu + seq), start = __ldg(a.start + seq);
    if (n == 0 || place < 0) return;
    if (bad_lengths(c0, n, start, a.n, a.max_new)) {
        if (threadIdx.x == 0) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
        return;
    }
    const int64_t index = (start >> a.log2_page) + static_cast<int64_t>(place), base = index << a.log2_page;
    if (base >= static_cast<int64_t>(start) + n) return;
    const int id = index < a.table_width ? __ldg(a.table + seq * a.table_stride + index) : -1;
    const int filled = static_cast<int>(max(start - base, static_cast<int64_t>(0)));  // tokens the page holds already
    const int lane = threadIdx.x % kLanes;
    int slot[kSlots];
    int64_t row[kSlots];  // of k and v
    bool fresh[kSlots];
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
        slot[t] = threadIdx.x / kLanes + (t << (a.log2_page - 1));
        const int64_t token = base + slot[t] - start;  // among the sequence's new ones
        fresh[t] = token >= 0 && token < n;
        row[t] = c0 + token;
    }

    // The thread's two pieces of eight values of a slot.
    int p0 = lane, p1 = lane + kLanes;
    const int half = a.rot / 2;
    bool turn = LAYOUT != kNoRotation;
    if constexpr (LAYOUT == kHalves) {
        turn = lane < a.rot / 16;
        p0 = turn ? lane : a.rot / 8 + lane - a.rot / 16;
        p1 = p0 + (turn ? a.rot / 16 : (D - a.rot) / 16);
    }
    const int h_begin = blockIdx.y * a.heads_per_block, h_end = min(a.Hkv, h_begin + a.heads_per_block);
    const uint32_t mine = ptx::smem_u32(ring) + threadIdx.x * 16;
    const uint32_t plane = blockDim.x * 16;  // bytes of one piece of all threads; a stage is four for each slot
    uint16_t *unsure = reinterpret_cast<uint16_t *>(ring + kStages * kSlots * 4 * blockDim.x) + threadIdx.x;  // masks
    uint32_t any_unsure = 0;                                                          // a bit for each head and slot
    auto copy = [&](int h, int stage) {
        if (h < h_end) {
#pragma unroll
            for (int t = 0; t < kSlots; ++t) {
                if (!fresh[t]) continue;
                const uint16_t *k = a.k + row[t] * a.k_stride + h * D, *v = a.v + row[t] * a.v_stride + h * D;
                const uint32_t to = mine + (stage * kSlots + t) * 4 * plane;
                ptx::cp_async16(to, k + p0 * 8);
                ptx::cp_async16(to + plane, k + p1 * 8);
                ptx::cp_async16(to + 2 * plane, v + p0 * 8);
                ptx::cp_async16(to + 3 * plane, v + p1 * 8);
            }
        }
        ptx::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) copy(h_begin + i, i);
    if (id < 0 || id >= a.n_pages) {
        if (threadIdx.x == 0) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
        ptx::cp_async_wait<0>();
        return;
    }

    int32_t pos[kSlots];
    uint64_t c[kSlots][4], minus_s[kSlots][4];  // of eight pairs
    auto pair_of = [&](int e) { return LAYOUT == kHalves ? p0 * 8 + e : e < 4 ? p0 * 4 + e : p1 * 4 + e - 4; };
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
        pos[t] = !fresh[t] ? 0 : a.pos ? __ldg(a.pos + row[t]) : static_cast<int32_t>(base + slot[t]);
        if constexpr (LAYOUT == kHalves || LAYOUT == kInterleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) c[t][e] = ptx::f32x2(1.f, 1.f), minus_s[t][e] = 0;
            if (fresh[t] && turn) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float cc[2], ss[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {  // pairs past rot get any angle: they are not turned
                        const int i = LAYOUT == kHalves ? pair_of(2 * e + b) : min(pair_of(2 * e + b), half - 1);
                        turn_cos_sin(__ldg(a.turns + i), pos[t], a.amplitude, cc[b], ss[b]);
                    }
                    c[t][e] = ptx::f32x2(cc[0], cc[1]);
                    minus_s[t][e] = ptx::f32x2(-ss[0], -ss[1]);
                }
            }
        }
    }

    int flip = 0, stage = 0;
    for (int h = h_begin; h < h_end; ++h) {
        copy(h + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
        uint8_t *k_scale = a.ks + id * a.scale_stride + h, *v_scale = a.vs + id * a.scale_stride + h;
        int ek_old = kScaleMin, ev_old = kScaleMin;
        if (filled > 0) {
            ek_old = exponent_of(*reinterpret_cast<volatile uint8_t *>(k_scale));
            ev_old = exponent_of(*reinterpret_cast<volatile uint8_t *>(v_scale));
        }
        ptx::cp_async_wait<kStages - 1>();
        const uint4 *own = ring + stage * kSlots * 4 * blockDim.x + threadIdx.x;
        if (++stage == kStages) stage = 0;
        auto piece = [&](int t, int i) { return own[(t * 4 + i) * blockDim.x]; };

        // The rotated keys as pairs of 32-bit values: x[t][e] holds values 2 e and 2 e + 1 of the thread's 16 in a slot.
        uint64_t x[kSlots][8];
        float m = 0.f;
        uint32_t w = 0;
#pragma unroll
        for (int t = 0; t < kSlots; ++t) {
            if (!fresh[t]) continue;
            {
                const uint4 u0 = piece(t, 0), u1 = piece(t, 1);
                const uint32_t u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) x[t][e] = ptx::f32x2(bf16_lo(u[e]), bf16_hi(u[e]));
            }
            if constexpr (LAYOUT == kHalves) {
                if (turn) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint64_t y = x[t][e], z = x[t][4 + e];
                        x[t][e] = ptx::fma_f32x2(z, minus_s[t][e], ptx::mul_f32x2(y, c[t][e]));
                        x[t][4 + e] = ptx::fma_f32x2(z, c[t][e], ptx::mul_f32x2(y, minus_s[t][e] ^ 0x8000000080000000ull));
                    }
                }
            } else if constexpr (LAYOUT == kInterleaved) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float y, z, cc0, cc1, ss0, ss1;
                    ptx::f32x2_split(x[t][e], y, z);
                    ptx::f32x2_split(c[t][e / 2], cc0, cc1);
                    ptx::f32x2_split(minus_s[t][e / 2], ss0, ss1);
                    const float cc = e & 1 ? cc1 : cc0, ss = e & 1 ? ss1 : ss0;
                    if (pair_of(e) < half) x[t][e] = ptx::f32x2(y * cc + z * ss, z * cc - y * ss);  // others stay, whatever they hold
                }
            } else if constexpr (LAYOUT == kHalvesByElement) {
                const uint16_t *k = a.k + row[t] * a.k_stride + h * D;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = (e < 8 ? p0 : p1) * 8 + (e & 7), i = j < half ? j : j - half;
                    if (j < a.rot) {
                        float cc, ss, lo, hi;
                        turn_cos_sin(__ldg(a.turns + i), pos[t], a.amplitude, cc, ss);
                        const float y = bf16_lo(k[i]), z = bf16_lo(k[i + half]), r = j < half ? y * cc - z * ss : y * ss + z * cc;
                        ptx::f32x2_split(x[t][e / 2], lo, hi);
                        x[t][e / 2] = e & 1 ? ptx::f32x2(lo, r) : ptx::f32x2(r, hi);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float lo, hi;
                ptx::f32x2_split(x[t][e], lo, hi);
                m = ptx::max3(m, fabsf(lo), fabsf(hi));  // a NaN counts as nothing
            }
            const uint4 w0 = piece(t, 2), w1 = piece(t, 3);
            const uint32_t v[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) w = max_bf16x2(w, v[e] & 0x7FFF7FFFu);
        }
        uint32_t mk = __float_as_uint(m), mv = max(w << 16, w & 0xFFFF0000u);
        block_max(mk, mv, part[flip]);
        flip ^= 1;
        const bool infinite_key = mk == 0x7F800000u;
        if (infinite_key || mv == 0x7F800000u) {  // the scale is that of the finite values; infinities take the largest code
            mk = mv = 0;
#pragma unroll
            for (int t = 0; t < kSlots; ++t) {
                if (!fresh[t]) continue;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t b = static_cast<uint32_t>(x[t][e / 2] >> 32 * (e & 1)) & 0x7FFFFFFFu;
                    const uint4 q = piece(t, 2 + e / 8);
                    const uint32_t y = (reinterpret_cast<const uint32_t *>(&q)[e / 2 & 3] << (e & 1 ? 0 : 16)) & 0x7FFF0000u;
                    mk = b < 0x7F800000u ? max(mk, b) : mk;
                    mv = y < 0x7F800000u ? max(mv, y) : mv;
                }
            }
            block_max(mk, mv, part[flip]);
            flip ^= 1;
        }
        int ek = scale_exponent(__uint_as_float(mk)), ev = scale_exponent(__uint_as_float(mv));
        if (filled > 0) ek = max(ek, ek_old), ev = max(ev, ev_old);
        const int64_t head = id * a.page_stride + ((static_cast<int64_t>(h) << a.log2_page) * D);
        const float fk = scale_of(-ek), fv = scale_of(-ev);
        const uint64_t fk2 = ptx::f32x2(fk, fk), fv2 = ptx::f32x2(fv, fv);
#pragma unroll
        for (int t = 0; t < kSlots; ++t) {
            uint2 *kc = reinterpret_cast<uint2 *>(a.kc + head + slot[t] * D), *vc = reinterpret_cast<uint2 *>(a.vc + head + slot[t] * D);
            if (fresh[t]) {
                uint32_t q[4];
                {
                    const uint4 w0 = piece(t, 2), w1 = piece(t, 3);
                    const uint32_t v[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        q[i] = f32x4_to_e4m3x4(ptx::mul_f32x2(ptx::f32x2(bf16_lo(v[2 * i]), bf16_hi(v[2 * i])), fv2),
                                               ptx::mul_f32x2(ptx::f32x2(bf16_lo(v[2 * i + 1]), bf16_hi(v[2 * i + 1])), fv2));
                    vc[p0] = make_uint2(q[0], q[1]);
                    vc[p1] = make_uint2(q[2], q[3]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[t][e] = ptx::mul_f32x2(x[t][e], fk2);
                if (LAYOUT == kNoRotation || infinite_key || (LAYOUT == kHalves && !turn)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) q[i] = f32x4_to_e4m3x4(x[t][2 * i], x[t][2 * i + 1]);
                    kc[p0] = make_uint2(q[0], q[1]);
                    kc[p1] = make_uint2(q[2], q[3]);
                } else {
                    // Codes of the least and the most that each exact value can be.
                    const uint64_t more = ptx::f32x2(kTurnError, kTurnError), less = ptx::f32x2(-kTurnError, -kTurnError);
                    uint64_t size[8];  // what the error is relative to, for values 2 e and 2 e + 1
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float y0, y1, z0, z1;
                        ptx::f32x2_split(x[t][e], y0, y1);
                        if constexpr (LAYOUT == kHalves) {
                            ptx::f32x2_split(x[t][e ^ 4], z0, z1);
                            size[e] = e < 4 ? ptx::f32x2(fabsf(y0) + fabsf(z0), fabsf(y1) + fabsf(z1)) : size[e & 3];
                        } else if constexpr (LAYOUT == kInterleaved) {
                            const float b = pair_of(e) < half ? fabsf(y0) + fabsf(y1) : 0.f;
                            size[e] = ptx::f32x2(b, b);
                        } else {
                            const uint16_t *k = a.k + row[t] * a.k_stride + h * D;
                            float r[2];
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                const int j = (e < 4 ? p0 : p1) * 8 + (2 * e & 7) + b, i = j < half ? j : j - half;
                                r[b] = j < a.rot ? fabsf(a.amplitude) * (fabsf(bf16_lo(k[i])) + fabsf(bf16_lo(k[i + half]))) * fk : 0.f;
                            }
                            size[e] = ptx::f32x2(r[0], r[1]);
                        }
                    }
                    uint32_t differ[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        q[i] = f32x4_to_e4m3x4(ptx::fma_f32x2(size[2 * i], less, x[t][2 * i]), ptx::fma_f32x2(size[2 * i + 1], less, x[t][2 * i + 1]));
                        differ[i] = q[i] ^ f32x4_to_e4m3x4(ptx::fma_f32x2(size[2 * i], more, x[t][2 * i]),
                                                           ptx::fma_f32x2(size[2 * i + 1], more, x[t][2 * i + 1]));
                    }
                    kc[p0] = make_uint2(q[0], q[1]);
                    kc[p1] = make_uint2(q[2], q[3]);
                    if (differ[0] | differ[1] | differ[2] | differ[3]) {
                        // A pair of zeros, and a value that passes (its size is 0), is exact: its two codes differ in a zero's
                        // sign, and the first has that of x.  (All-zero keys by way of the mask: 118 us in place of 24.)
                        uint32_t exact = 0;
#pragma unroll
                        for (int e = 0; e < (LAYOUT == kHalves ? 4 : 8); ++e) {
                            if ((size[e] & 0x7FFFFFFFu) == 0) exact |= (LAYOUT == kInterleaved ? 3u : 1u) << 2 * e;
                            if (LAYOUT != kInterleaved && (size[e] >> 32 & 0x7FFFFFFFu) == 0) exact |= 2u << 2 * e;
                        }
                        if (LAYOUT == kHalves) exact |= exact << 8;
                        const uint32_t mask = (nonzero_bytes(differ[0]) | nonzero_bytes(differ[1]) << 4 | nonzero_bytes(differ[2]) << 8 |
                                               nonzero_bytes(differ[3]) << 12) & ~exact;
                        if (mask) {
                            const int which = (h - h_begin) * kSlots + t;
                            any_unsure |= 1u << which;
                            unsure[which * blockDim.x] = static_cast<uint16_t>(mask);
                        }
                    }
                }
            } else if (slot[t] < filled) {
                if (ek > ek_old) {
                    const float f = scale_of(ek_old - ek);
                    kc[p0] = requantised(kc[p0], f);
                    kc[p1] = requantised(kc[p1], f);
                }
                if (ev > ev_old) {
                    const float f = scale_of(ev_old - ev);
                    vc[p0] = requantised(vc[p0], f);
                    vc[p1] = requantised(vc[p1], f);
                }
            }
        }
        if (threadIdx.x == 0) {
            *k_scale = static_cast<uint8_t>(ek + kScaleBias);
            *v_scale = static_cast<uint8_t>(ev + kScaleBias);
            k_exponents[h - h_begin] = static_cast<int16_t>(ek);
        }
    }
    if constexpr (LAYOUT != kNoRotation) {
        if (!__syncthreads_or(static_cast<int>(any_unsure))) return;
        for (; any_unsure; any_unsure &= any_unsure - 1) {
            const int which = __ffs(any_unsure) - 1, n_head = which / kSlots, h = h_begin + n_head;
            const bool second = which % kSlots;
            write_nearer_codes<LAYOUT == kInterleaved>(
                unsure[which * blockDim.x],
                a.kc + id * a.page_stride + (((static_cast<int64_t>(h) << a.log2_page) + (second ? slot[1] : slot[0])) * D),
                a.k + (second ? row[1] : row[0]) * a.k_stride + static_cast<int64_t>(h) * D, p0 * 8, p1 * 8, half, a.turns,
                second ? pos[1] : pos[0], a.amplitude * scale_of(-k_exponents[n_head]));
        }
    }
}

// ------------------------------------------------------------------------------------------ pages to rows
constexpr int kMaxRequests = kMaxPagedRequests;
constexpr int kTile = 128;  // a region's rows are a multiple of the attention's key tile: zeros past its last token

struct GatherArgs {
    PagedCache c;
    const int32_t *table;
    int64_t table_stride;
    int Hkv, n_req;
    int64_t rows;                 // of all regions
    int64_t first[kMaxRequests];  // row of each request's region
    int len[kMaxRequests];
    uint16_t *k, *v;              // [rows][Hkv][D]
    int *err;
};

constexpr int kGatherThreads = 256;

// The prefix pages of each request as bf16 rows of a contiguous region (codes times scales are exact in bf16), so
// that the tensor-core attention reads them by its tensor maps: 2 bytes read and 4 written a key and channel, once
// per call, against hundreds of products a byte in the attention.  A thread turns 16 codes of K and of V.  The grid goes over
// the rows of all regions (a request of 131072 tokens among 63 of 1000: 1866 us a call; as many blocks for each as the longest
// takes: 2844).
template <int D>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherArgs a)
{
    constexpr int kPieces = D / 16;
    ptx::grid_dep_wait();
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kGatherThreads + threadIdx.x;
    const int piece = static_cast<int>(item % kPieces);
    const int64_t th = item / kPieces;
    const int h = static_cast<int>(th % a.Hkv);
    const int64_t row = th / a.Hkv;  // of all regions, which lie one behind the other
    if (row >= a.rows) return;
    int r = 0;                       // the last request whose region starts at or before it
    if (a.n_req > 1)
#pragma unroll
        for (int step = kMaxRequests / 2; step; step /= 2) r += r + step < a.n_req && a.first[r + step] <= row ? step : 0;
    const int64_t token = row - a.first[r];
    const int len = a.len[r];
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
            fk = scale_of(exponent_of(__ldg(a.c.k_scale + id * a.c.scale_stride + h)));
            fv = scale_of(exponent_of(__ldg(a.c.v_scale + id * a.c.scale_stride + h)));
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
    const int64_t to = (row * a.Hkv + h) * D + piece * 16;
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
    if (n == 0) return BLINK_OK;

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
    a.S = S;
    a.Hkv = Hkv;
    a.log2_page = c.log2_page;
    a.turns = d_turns;
    a.rot = rot;
    a.amplitude = amplitude;
    a.err = &static_cast<WorkspaceHeader *>(d_ws)->error;
    // Pages that max_new tokens can touch, and the heads of a block: few enough to give every SM two blocks, which is what it
    // runs at a time (18432 tokens of 8 heads: four heads 26.5 us, two 28.5, all eight 30.6).
    const int pages = (max_new + page_tokens - 2) / page_tokens + 1;
    const int64_t busy = (static_cast<int64_t>(n) + page_tokens - 1) / page_tokens + S;
    const int64_t groups = (2LL * current_sm_count() + busy - 1) / busy;
    a.heads_per_block = groups >= Hkv ? 1 : static_cast<int>((Hkv + groups - 1) / groups);
    if (a.heads_per_block > kMaxBlockHeads) a.heads_per_block = kMaxBlockHeads;
    // As many pages for each sequence as max_new tokens can touch, or (with a search in each block) places for those that n
    // tokens of S sequences can, whichever are fewer (18432 tokens and 63 single ones: 52 us with empty pages for each, 32
    // packed; 64 single ones with max_new 18432: 90, 10.5; 16 pieces of up to 511: 8.8, 8.0).  Where half of the pages are empty the
    // search can cost more than they do (16 of 100 to 3850: 42.3, 43.3).
    const int64_t places = n / page_tokens + 2LL * S;
    a.packed = places < static_cast<int64_t>(pages) * S;
    const dim3 grid(static_cast<unsigned>(a.packed ? places : pages),
                    static_cast<unsigned>((Hkv + a.heads_per_block - 1) / a.heads_per_block), static_cast<unsigned>(a.packed ? 1 : S));
    const unsigned threads = static_cast<unsigned>(page_tokens * (d / 16) / kSlots);
    const int layout = rot == 0 ? kNoRotation : interleaved ? kInterleaved : rot % 16 == 0 ? kHalves : kHalvesByElement;
    const int smem = static_cast<int>(threads) * kSlots * (64 * kStages + 2 * a.heads_per_block);
    bool set = true;
    auto launch = [&](auto kern) {
        set = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, d * 8 * (64 * kStages + 2 * kMaxBlockHeads)) == cudaSuccess;
        set = set && launch_programmatic(kern, grid, threads, smem, stream, a) == cudaSuccess;
    };
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
    return set ? BLINK_OK : BLINK_CUDA_ERROR;
}

extern "C" size_t blink_paged_prefix_tail_workspace(const int32_t *h_req_rows, const int32_t *h_prefix_len, int32_t n_req,
                                                    int32_t B, int32_t Hq, int32_t Hkv, int32_t d)
{
    using namespace blink;
    if (!h_req_rows || n_req < 1 || n_req > kMaxRequests || Hkv < 1 || d < 1 ||
        check_requests(h_req_rows, h_prefix_len, n_req, h_req_rows[n_req]) != BLINK_OK)
        return kHeaderBytes;
    if (Hq >= Hkv && few_tail_rows(h_req_rows, n_req, Hq / Hkv))
        return few_tail_workspace(h_req_rows, h_prefix_len, n_req, Hkv, Hq / Hkv, d);
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
    for (int r = 0; r < n_req; ++r)
        if (h_prefix_len[r] > static_cast<int64_t>(table_width) * page_tokens) return BLINK_OUT_OF_RANGE;
    if (few_tail_rows(h_req_rows, n_req, Hq / Hkv)) {
        if (static_cast<int64_t>(rows) * Hq > 0x7FFFFFFF) return BLINK_OUT_OF_RANGE;
        if (ws_bytes < few_tail_workspace(h_req_rows, h_prefix_len, n_req, Hkv, Hq / Hkv, d)) return BLINK_WORKSPACE_TOO_SMALL;
        return few_tail_attention(a.c, page_tokens, q, d_page_table, table_stride, table_width, k_tail, v_tail, d_cu_seqlens,
                                  d_seq_start, B, rows, n_req, h_req_rows, h_prefix_len, max_tail, Hq, Hkv, d, scale, out, lse,
                                  d_ws, stream);
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
    if (lay.rows > 0) {
        a.table = d_page_table;
        a.table_stride = table_stride;
        a.Hkv = Hkv;
        a.k = ka;
        a.v = va;
        a.err = &static_cast<WorkspaceHeader *>(d_ws)->error;
        a.n_req = n_req;
        a.rows = lay.rows;
        const int64_t blocks = (lay.rows * Hkv * (d / 16) + kGatherThreads - 1) / kGatherThreads;
        if (blocks > 0x7FFFFFFF) return BLINK_OUT_OF_RANGE;
        const dim3 grid(static_cast<unsigned>(blocks));
        const cudaError_t e = d == 128 ? launch_programmatic(gather_kernel<128>, grid, kGatherThreads, 0, stream, a)
                                       : launch_programmatic(gather_kernel<64>, grid, kGatherThreads, 0, stream, a);
        if (e != cudaSuccess) return BLINK_CUDA_ERROR;
    }
    const int64_t row = static_cast<int64_t>(Hkv) * d;
    if (n_req == 1)
        return blink_prefix_tail_attention(q, ka, va, row, k_tail, v_tail, d_cu_seqlens, d_seq_start, B, rows, h_prefix_len[0],
                                           max_tail, Hq, Hkv, d, scale, out, lse, d_ws, lay.k, stream);
    return blink_prefix_tail_attention_multi(q, ka, va, row, lay.rows, k_tail, v_tail, d_cu_seqlens, d_seq_start, B, rows, n_req,
                                             h_req_rows, first, h_prefix_len, max_tail, Hq, Hkv, d, scale, out, lse, d_ws,
                                             lay.k, stream);
}
