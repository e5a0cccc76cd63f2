// rotary.cuh -- the rotation of queries and keys by their positions, shared by the kernels that apply it.
//
// Pair i of a head turns by position * theta_i.  theta_i / (2 pi) is held as a 64-bit fraction of a turn, so that
// position * fraction modulo 2^64 is the exact remainder of the angle: no digits are lost at far positions, and no
// 64-bit floating-point arithmetic is needed.  The fraction comes from a double (53 bits below 2^61): at position p
// it is off by p 2^-56 turns at most, 2^-39 at 131072.
#pragma once
#include <cstdint>

namespace blink {

// cos and sin of pos * turns, times `amplitude`.  The remainder's upper 32 bits are a signed part of a half turn:
// 2^-32 turns is 1.5e-9 radians, below the 6e-8 that 32-bit values of cos and sin are rounded to.
__device__ __forceinline__ void turn_cos_sin(uint64_t turns, int32_t pos, float amplitude, float &c, float &s)
{
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns;
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    c *= amplitude;
    s *= amplitude;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// How the pairs of a head lie: (i, i + rot / 2) or (2 i, 2 i + 1).
enum RotaryLayout { kNoRotation = 0, kHalves = 1, kInterleaved = 2, kHalvesByElement = 3 };

}  // namespace blink
