// rotary.cuh -- the rotation of queries and keys by their positions, shared by the kernels that apply it.
//
// Pair i of a head turns by position * theta_i.  theta_i / (2 pi) is held as a 64-bit fraction of a turn, so that
// position * fraction modulo 2^64 is the exact remainder of the angle: no digits are lost at far positions, and no
// 64-bit floating-point arithmetic is needed.  The fraction comes from a double (53 bits below 2^61): at position p
// it is off by p 2^-56 turns at most, 2^-39 at 131072.
#pragma once
#include <cstdint>

namespace blink {

// cos and sin of pos * turns, times `amplitude`: the nearest quarter turn, which only swaps and negates, and the Taylor
// series of what is left (at most pi / 4: the terms after the ninth and tenth power are below 2e-9).  The remainder's
// upper 32 bits are enough, 2^-32 turns being 1.5e-9 radians.  x is off by two half steps of 32 bits (1.6 * 2^-24 at most),
// which cos and sin take times the other's size, and adding the last term adds half a step of each: 2 * 2^-24 bounds what
// they lack (1.63 * 2^-24 was the most of a million random angles).
__device__ __forceinline__ void turn_cos_sin(uint64_t turns, int32_t pos, float amplitude, float &c, float &s)
{
    // bits 32 .. 63 of the product
    const uint32_t lo = static_cast<uint32_t>(turns), hi = static_cast<uint32_t>(turns >> 32), p = static_cast<uint32_t>(pos);
    const uint32_t phase = __umulhi(p, lo) + p * hi - (pos < 0 ? lo : 0u);
    const uint32_t quarter = phase + (1u << 29);  // its upper two bits
    const float x = static_cast<float>(static_cast<int32_t>(phase - (quarter & 0xC0000000u))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float y = x * x;
    float ss = fmaf(y, 1.f / 362880.f, -1.f / 5040.f), cc = fmaf(y, -1.f / 3628800.f, 1.f / 40320.f);
    ss = fmaf(y, ss, 1.f / 120.f);
    cc = fmaf(y, cc, -1.f / 720.f);
    ss = fmaf(y, ss, -1.f / 6.f);
    cc = fmaf(y, cc, 1.f / 24.f);
    ss = fmaf(y * x, ss, x);
    cc = fmaf(y, fmaf(y, cc, -0.5f), 1.f);
    const bool odd = quarter & 0x40000000u;
    const uint32_t cs = __float_as_uint((odd ? ss : cc) * amplitude), sc = __float_as_uint((odd ? cc : ss) * amplitude);
    c = __uint_as_float(cs ^ ((quarter + 0x40000000u) & 0x80000000u));
    s = __uint_as_float(sc ^ (quarter & 0x80000000u));
}

// Sums of two 32-bit values, the second what the first lacks: some 44 bits.  (In 64-bit arithmetic, whose rate is a small part of
// the 32-bit one, the append's undecided codes took 53 us for 18432 tokens of 8 heads in place of 27.)
struct Two {
    float h, l;
};

__device__ __forceinline__ Two two_sum(float a, float b)
{
    const float s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Two add(Two a, Two b)
{
    const Two s = two_sum(a.h, b.h);
    return two_sum(s.h, s.l + (a.l + b.l));
}
__device__ __forceinline__ Two mul(Two a, Two b)
{
    const float p = a.h * b.h;
    return two_sum(p, fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, a.l * b.h));
}

// cos(2 pi k / 64) for k = 0 .. 16.
#define BLINK_TWO(x) {static_cast<float>(x), static_cast<float>((x) - static_cast<double>(static_cast<float>(x)))}
__device__ __constant__ Two kCosine[17] = {
    BLINK_TWO(1.0),
    BLINK_TWO(0.9951847266721969),
    BLINK_TWO(0.9807852804032304),
    BLINK_TWO(0.9569403357322088),
    BLINK_TWO(0.9238795325112867),
    BLINK_TWO(0.881921264348355),
    BLINK_TWO(0.8314696123025452),
    BLINK_TWO(0.773010453362737),
    BLINK_TWO(0.7071067811865476),
    BLINK_TWO(0.6343932841636455),
    BLINK_TWO(0.5555702330196023),
    BLINK_TWO(0.4713967368259978),
    BLINK_TWO(0.38268343236508984),
    BLINK_TWO(0.29028467725446233),
    BLINK_TWO(0.19509032201612833),
    BLINK_TWO(0.09801714032956077),
    BLINK_TWO(0.0),
};
#undef BLINK_TWO

__device__ __forceinline__ Two cosine_64(uint32_t j)  // of 2 pi j / 64
{
    const uint32_t k = j & 15u, quadrant = j >> 4 & 3u;
    const Two v = kCosine[quadrant & 1u ? 16u - k : k];
    return quadrant == 1u || quadrant == 2u ? Two{-v.h, -v.l} : v;
}

// cos and sin of pos * turns to some 40 bits: the nearest 64th of a turn from the table and the Taylor series of what is
// left (at most 0.05: its terms after the seventh and eighth power are below 2e-17).
__device__ __forceinline__ void turn_cos_sin(uint64_t turns, int32_t pos, Two &c, Two &s)
{
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns;
    const uint64_t step = (phase + (1ull << 57)) >> 58;
    const int64_t rest = static_cast<int64_t>(phase - (step << 58));
    const float rh = static_cast<float>(rest), rl = static_cast<float>(rest - static_cast<int64_t>(rh));
    constexpr float uh = static_cast<float>(3.4061215800309573e-19);  // 2 pi / 2^64
    constexpr float ul = static_cast<float>(3.4061215800309573e-19 - static_cast<double>(uh));
    const Two x = mul({rh, rl}, {uh, ul}), y = mul(x, x);
    const float z = y.h;
    // sin x = x + x^3 (-1/6 + x^2/120 - x^4/5040), its second term below 2^-15 of the first; cos x likewise
    const Two sn = add(x, {x.h * z * fmaf(z, fmaf(z, -1.f / 5040.f, 1.f / 120.f), -1.f / 6.f), 0.f});
    const Two cn = add(add({1.f, 0.f}, {-0.5f * y.h, -0.5f * y.l}), {z * z * fmaf(z, fmaf(z, 1.f / 40320.f, -1.f / 720.f), 1.f / 24.f), 0.f});
    const Two ct = cosine_64(static_cast<uint32_t>(step)), st = cosine_64(static_cast<uint32_t>(step) + 48u);
    const Two a = mul(st, sn), b = mul(ct, sn);
    c = add(mul(ct, cn), {-a.h, -a.l});
    s = add(mul(st, cn), b);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// How the pairs of a head lie: (i, i + rot / 2) or (2 i, 2 i + 1).
enum RotaryLayout { kNoRotation = 0, kHalves = 1, kInterleaved = 2, kHalvesByElement = 3 };

}  // namespace blink
