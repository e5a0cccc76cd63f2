// paged.cuh -- the 8-bit paged cache: its layout, and the conversions between its codes and other types.
//
// A page holds `page` tokens of every kv head, head by head: codes[page][head][token][d] in e4m3, and one scale per
// (page, head), a power of two in e8m0 (the biased exponent alone).  A value is its code times its scale, which is
// exact in 16 and in 32 bits: a scale moves no bit of a code, so it can be applied to a score or an exponent instead
// of to each value, and a page whose scale grows loses only what falls below the smallest code.
#pragma once
#include <cstdint>

#include "common.cuh"

namespace blink {

constexpr int kScaleBias = 127;
constexpr int kScaleMin = BLINK_PAGED_SCALE_MIN, kScaleMax = BLINK_PAGED_SCALE_MAX;

struct PagedCache {
    const uint8_t *k, *v;              // codes
    const uint8_t *k_scale, *v_scale;  // biased exponents
    int64_t page_stride, scale_stride; // bytes between pages
    int n_pages;
    int log2_page;
};

// Checks what every call that takes a cache checks, and fills `c`.
blink_status check_cache(PagedCache &c, const void *k, const void *v, const void *ks, const void *vs, int64_t page_stride,
                         int64_t scale_stride, int32_t n_pages, int32_t page_tokens, int32_t Hkv, int32_t d);

constexpr int kMaxPagedRequests = 64;

// Prefix-tail attention of few rows, read from the pages as they are (pagedattn.cu).  few_tail_rows: whether a call is of
// that kind; arguments as blink_paged_prefix_tail_attention has checked them.
bool few_tail_rows(const int32_t *h_req_rows, int n_req, int g);
size_t few_tail_workspace(const int32_t *h_req_rows, const int32_t *h_len, int n_req, int Hkv, int g, int d);
blink_status few_tail_attention(const PagedCache &c, int page_tokens, const uint16_t *q, const int32_t *d_page_table,
                                int64_t table_stride, int table_width, const uint16_t *k_tail, const uint16_t *v_tail,
                                const int32_t *d_cu, const int32_t *d_seq_start, int B, int rows, int n_req,
                                const int32_t *h_req_rows, const int32_t *h_len, int max_tail, int Hq, int Hkv, int d, float scale,
                                uint16_t *out, float *lse, void *d_ws, cudaStream_t stream);

#ifdef __CUDACC__

__device__ __forceinline__ float scale_of(int e) { return __uint_as_float(static_cast<uint32_t>(e + kScaleBias) << 23); }
// A scale's exponent as it is read: one outside the range (a page that was never written has 0) is the nearest in it, so
// that no difference of two exponents leaves those of a float.
__device__ __forceinline__ int exponent_of(uint8_t scale)
{
    return min(max(static_cast<int>(scale) - kScaleBias, kScaleMin), kScaleMax);
}

// By a whole warp: the last of lo + 1 .. hi - 1 for which `before` holds (it holds up to some place and not behind it), 32
// places at a time; lo if it holds for none.  Any other answers of `before` give some place of lo .. hi - 1.
template <class F>
__device__ __forceinline__ int last_before(int lo, int hi, F before)
{
    const int lane = threadIdx.x & 31;
    while (hi - lo > 1) {
        const int step = (hi - lo - 1 + 31) / 32, at = lo + (lane + 1) * step;
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && before(at)));
        if (n < 32) hi = min(hi, lo + (n + 1) * step);
        lo += n * step;
    }
    return lo;
}

// Two e4m3 codes (the lower byte first) as two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two)
{
    uint32_t r;
    asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
// The same for a word's upper two codes.
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t four)
{
    uint32_t r;
    asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}" : "=r"(r) : "r"(four));
    return r;
}
__device__ __forceinline__ void f16x2_split(uint32_t v, float &lo, float &hi)
{
    asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %2;\n\tcvt.f32.f16 %0, t;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(v));
}
// Two values as e4m3 codes: nearest, ties to even, larger ones at the largest code, NaN stays NaN.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four values, two pairs of 32-bit ones, as the codes of a word.
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(uint64_t a, uint64_t b)
{
    uint32_t r;
    asm("{\n\t.reg .b16 t, u;\n\t.reg .f32 a0, a1, b0, b1;\n\tmov.b64 {a0, a1}, %1;\n\tmov.b64 {b0, b1}, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 t, a1, a0;\n\tcvt.rn.satfinite.e4m3x2.f32 u, b1, b0;\n\tmov.b32 %0, {t, u};\n\t}"
        : "=r"(r)
        : "l"(a), "l"(b));
    return r;
}

// The larger of two bf16 values, pair by pair; a NaN counts as nothing.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

#endif
}  // namespace blink
