// rope.cu -- rotary positions: the table of frequencies (host) and the rotation of query and key rows.
//
// y[2 values of pair i] = amplitude * R(position theta_i) x[pair i]; values past `rot` pass through.  Bound by HBM:
// 4 bytes a value, three products for two values.  The angles belong to a row, not to a head, so a block computes
// the cos and sin of its rows once into shared memory, a thread keeps those of its pairs in registers and goes over
// the heads with them.
#include <cmath>

#include "common.cuh"
#include "ptx.cuh"
#include "rotary.cuh"

namespace blink {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 3;        // heads whose loads are in flight at once in a thread
constexpr int kMaxDim = 512;
constexpr int kMaxRows = 32;     // rows of a block
constexpr int kLanes = 64;       // threads over (row, item) that a block should have

struct RopeArgs {
    const uint16_t *in[2];
    uint16_t *out[2];
    int64_t in_stride[2], out_stride[2];  // elements
    int heads[2];
    bool copy[2];                         // out of place: values past rot are copied
    const int32_t *pos;
    const uint64_t *turns;
    float amplitude;
    int rows, d, rot;
    int per_block;                        // rows of a block
    int turned, passed;                   // items of a row: pieces (pairs of them in the halves' layout) that turn, pieces that pass
};

__device__ __forceinline__ void block_angles(const RopeArgs &a, int row0, int n, float2 *cs)
{
    const int half = a.rot / 2;
    for (int e = threadIdx.x; e < n * half; e += blockDim.x) {
        const int r = e / half, i = e - r * half;
        float c, s;
        turn_cos_sin(__ldg(a.turns + i), __ldg(a.pos + row0 + r), a.amplitude, c, s);
        cs[e] = make_float2(c, s);
    }
    __syncthreads();
}

template <int W>
struct Piece {
    uint32_t w[W / 2];
};
template <int W>
__device__ __forceinline__ Piece<W> load_piece(const uint16_t *p)
{
    Piece<W> x;
    if constexpr (W == 8) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        x.w[0] = v.x, x.w[1] = v.y, x.w[2] = v.z, x.w[3] = v.w;
    } else if constexpr (W == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        x.w[0] = v.x, x.w[1] = v.y;
    } else {
        x.w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
    return x;
}
template <int W>
__device__ __forceinline__ void store_piece(uint16_t *p, const Piece<W> &x)
{
    if constexpr (W == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    else if constexpr (W == 4)
        *reinterpret_cast<uint2 *>(p) = make_uint2(x.w[0], x.w[1]);
    else
        *reinterpret_cast<uint32_t *>(p) = x.w[0];
}

// Pieces of W values (16, 8 or 4 bytes).  Halves: an item is pieces i and i + rot / 2 / W of a head, W pairs.
// Interleaved: an item is one piece, W / 2 pairs.  Threads lie over (row, item), what is left of the block over heads.
template <int LAYOUT, int W>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a)
{
    extern __shared__ float2 cs[];  // [rows of the block][rot / 2]
    ptx::grid_dep_wait();
    ptx::grid_launch_dependents();
    const int row0 = blockIdx.x * a.per_block;
    const int n = min(a.per_block, a.rows - row0);
    block_angles(a, row0, n, cs);

    constexpr int kPairs = LAYOUT == kHalves ? W : W / 2;
    constexpr int kPieces = LAYOUT == kHalves ? 2 : 1;
    const int items = a.turned + a.passed, lanes = a.per_block * items;
    const int group = threadIdx.x / lanes, groups = blockDim.x / lanes;
    const int lane = threadIdx.x - group * lanes;
    const int r = lane / items, item = lane - r * items;
    if (group >= groups || r >= n) return;
    const bool turn = item < a.turned;
    const int half = a.rot / 2;
    const int first = (turn || LAYOUT != kHalves ? item : a.rot / W + item - a.turned) * W;  // value
    float c[kPairs], s[kPairs];
    if (turn) {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            const int i = item * kPairs + e;
            const float2 v = i < half ? cs[r * half + i] : make_float2(1.f, 0.f);
            c[e] = v.x;
            s[e] = v.y;
        }
    }
    const int64_t row = row0 + r;
    const int H = a.heads[0] + a.heads[1];
    for (int h0 = group; h0 < H; h0 += groups * kBatch) {
        Piece<W> x[kBatch][kPieces];
        bool on[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int hh = h0 + b * groups, t = hh >= a.heads[0];
            on[b] = hh < H && (turn || a.copy[t]);
            if (!on[b]) continue;
            const uint16_t *p = a.in[t] + row * a.in_stride[t] + static_cast<int64_t>(hh - t * a.heads[0]) * a.d + first;
            x[b][0] = load_piece<W>(p);
            if (LAYOUT == kHalves && turn) x[b][kPieces - 1] = load_piece<W>(p + half);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (!on[b]) continue;
            const int hh = h0 + b * groups, t = hh >= a.heads[0];
            uint16_t *p = a.out[t] + row * a.out_stride[t] + static_cast<int64_t>(hh - t * a.heads[0]) * a.d + first;
            if (turn) {
                uint32_t *u = x[b][0].w, *v = x[b][kPieces - 1].w;
#pragma unroll
                for (int e = 0; e < W / 2; ++e) {
                    const float u0 = bf16_lo(u[e]), u1 = bf16_hi(u[e]);
                    if constexpr (LAYOUT == kHalves) {
                        const float v0 = bf16_lo(v[e]), v1 = bf16_hi(v[e]);
                        u[e] = ptx::pack_bf16x2(u0 * c[2 * e] - v0 * s[2 * e], u1 * c[2 * e + 1] - v1 * s[2 * e + 1]);
                        v[e] = ptx::pack_bf16x2(u0 * s[2 * e] + v0 * c[2 * e], u1 * s[2 * e + 1] + v1 * c[2 * e + 1]);
                    } else if (item * kPairs + e < half) {
                        // the piece in which rot ends: pairs past it stay as they are, whatever they hold
                        u[e] = ptx::pack_bf16x2(u0 * c[e] - u1 * s[e], u0 * s[e] + u1 * c[e]);
                    }
                }
                if (LAYOUT == kHalves) store_piece<W>(p + half, x[b][kPieces - 1]);
            }
            store_piece<W>(p, x[b][0]);
        }
    }
}

__device__ __forceinline__ float bf16_value(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float x) { return static_cast<uint16_t>(ptx::pack_bf16x2(x, 0.f) & 0xFFFFu); }

// Any size, stride and alignment of rows: one row a block, one pair or passed value a thread at a time.
__global__ void __launch_bounds__(kThreads) rope_element_kernel(const __grid_constant__ RopeArgs a, bool interleaved)
{
    __shared__ float2 cs[kMaxDim / 2];
    ptx::grid_dep_wait();
    ptx::grid_launch_dependents();
    const int64_t row = blockIdx.x;
    block_angles(a, blockIdx.x, 1, cs);
    const int half = a.rot / 2, items = half + a.d - a.rot;
    for (int e = threadIdx.x; e < (a.heads[0] + a.heads[1]) * items; e += blockDim.x) {
        const int hh = e / items, i = e - hh * items, t = hh >= a.heads[0];
        const int64_t h = static_cast<int64_t>(hh - t * a.heads[0]) * a.d;
        const uint16_t *p = a.in[t] + row * a.in_stride[t] + h;
        uint16_t *o = a.out[t] + row * a.out_stride[t] + h;
        if (i < half) {
            const int j0 = interleaved ? 2 * i : i, j1 = interleaved ? 2 * i + 1 : i + half;
            const float x = bf16_value(p[j0]), y = bf16_value(p[j1]);
            o[j0] = bf16_bits(x * cs[i].x - y * cs[i].y);
            o[j1] = bf16_bits(x * cs[i].y + y * cs[i].x);
        } else if (a.copy[t]) {
            o[i + half] = p[i + half];
        }
    }
}

}  // namespace
}  // namespace blink

extern "C" blink_status blink_rope_table(int32_t rot, double base, int32_t scaling, double factor, int32_t original,
                                         double low, double high, uint64_t *h_turns, float *h_amplitude)
{
    if (!h_turns || !h_amplitude) return BLINK_INVALID_ARG;
    if (rot < 2 || rot > BLINK_MAX_ROPE_DIM) return BLINK_OUT_OF_RANGE;
    if (rot % 2 != 0 || !(base > 1.0) || !std::isfinite(base)) return BLINK_INVALID_ARG;
    if (scaling < BLINK_ROPE_PLAIN || scaling > BLINK_ROPE_BY_TURNS) return BLINK_INVALID_ARG;
    const bool ramp = scaling == BLINK_ROPE_BY_DIM || scaling == BLINK_ROPE_BY_TURNS;
    if (scaling != BLINK_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return BLINK_INVALID_ARG;
    if (scaling == BLINK_ROPE_BASE && rot < 4) return BLINK_INVALID_ARG;
    if (ramp && (original < 1 || !(low > 0.0) || !(high > low) || !std::isfinite(high))) return BLINK_INVALID_ARG;
    const double pi = 3.14159265358979323846;
    const double used = scaling == BLINK_ROPE_BASE ? base * std::pow(factor, rot / (rot - 2.0)) : base;
    if (!std::isfinite(used)) return BLINK_INVALID_ARG;
    // the pair that turns n times over the original context
    auto pair_of = [&](double n) { return rot * std::log(original / (2.0 * pi * n)) / (2.0 * std::log(base)); };
    const double lo = ramp ? std::fmax(0.0, std::floor(pair_of(high))) : 0.0;
    const double hi = ramp ? std::fmin(rot - 1.0, std::ceil(pair_of(low))) : 0.0;
    for (int i = 0; i < rot / 2; ++i) {
        double theta = std::pow(used, -2.0 * i / rot);
        if (scaling == BLINK_ROPE_LINEAR) theta /= factor;
        if (scaling == BLINK_ROPE_BY_DIM) {
            const double r = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 0.001)));
            theta *= 1.0 - r + r / factor;
        }
        if (scaling == BLINK_ROPE_BY_TURNS) {
            const double n = original * theta / (2.0 * pi);
            const double keep = std::fmin(1.0, std::fmax(0.0, (n - low) / (high - low)));
            theta *= keep + (1.0 - keep) / factor;
        }
        h_turns[i] = static_cast<uint64_t>(std::ldexp(theta / (2.0 * pi), 64));
    }
    *h_amplitude = scaling == BLINK_ROPE_BY_DIM ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return BLINK_OK;
}

extern "C" blink_status blink_rope(const blink_bf16 *q, int64_t q_stride, const blink_bf16 *k, int64_t k_stride,
                                   const int32_t *d_positions, int32_t rows, int32_t Hq, int32_t Hkv, int32_t d,
                                   int32_t rot, const uint64_t *d_turns, float amplitude, int32_t interleaved,
                                   blink_bf16 *q_out, int64_t q_out_stride, blink_bf16 *k_out, int64_t k_out_stride,
                                   cudaStream_t stream)
{
    using namespace blink;
    if (!q || !q_out || !d_positions || !d_turns || (!k != !k_out)) return BLINK_INVALID_ARG;
    if (rows < 0 || Hq < 1 || Hkv < 0 || (k && Hkv < 1)) return BLINK_INVALID_ARG;
    if (d < 2 || d > kMaxDim || rows > (1 << 30) || Hq > 65535 || Hkv > 65535) return BLINK_OUT_OF_RANGE;
    if (rot < 2 || rot > d || rot % 2 != 0 || !std::isfinite(amplitude)) return BLINK_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return BLINK_INVALID_ARG;
    if (!k) Hkv = 0;
    const blink_bf16 *in[2] = {q, k};
    blink_bf16 *out[2] = {q_out, k_out};
    const int64_t is[2] = {q_stride, k_stride}, os[2] = {q_out_stride, k_out_stride};
    const int heads[2] = {Hq, Hkv};
    // Values of a piece: as many as sizes, strides and addresses are multiples of, at most 16 bytes; 1: by element.
    int64_t fit = d | (interleaved ? 0 : rot / 2);
    RopeArgs a{};
    for (int t = 0; t < (k ? 2 : 1); ++t) {
        const int64_t wide = static_cast<int64_t>(heads[t]) * d;
        if (is[t] < wide || os[t] < wide) return BLINK_INVALID_ARG;
        const bool in_place = out[t] == in[t] && (is[t] == os[t] || rows == 1);
        for (int u = 0; u < (k ? 2 : 1); ++u)
            if (!(u == t && in_place) &&
                strided_overlap(out[t], 2 * os[t], rows, in[u], 2 * is[u], rows, 2 * wide, 2 * static_cast<int64_t>(heads[u]) * d))
                return BLINK_INVALID_ARG;
        a.in[t] = in[t];
        a.out[t] = out[t];
        a.in_stride[t] = is[t];
        a.out_stride[t] = os[t];
        a.heads[t] = heads[t];
        a.copy[t] = !in_place;
        fit |= is[t] | os[t] | static_cast<int64_t>(reinterpret_cast<uintptr_t>(in[t]) / 2) |
               static_cast<int64_t>(reinterpret_cast<uintptr_t>(out[t]) / 2);
    }
    if (k && strided_overlap(q_out, 2 * q_out_stride, rows, k_out, 2 * k_out_stride, rows, 2LL * Hq * d, 2LL * Hkv * d))
        return BLINK_INVALID_ARG;
    if (rows == 0) return BLINK_OK;
    a.pos = d_positions;
    a.turns = d_turns;
    a.amplitude = amplitude;
    a.rows = rows;
    a.d = d;
    a.rot = rot;
    const int W = fit % 8 == 0 ? 8 : fit % 4 == 0 ? 4 : fit % 2 == 0 ? 2 : 1;
    cudaError_t launched = cudaSuccess;
    if (W == 1) {
        launched = launch_programmatic(rope_element_kernel, dim3(static_cast<unsigned>(rows)), kThreads, 0, stream, a, interleaved != 0);
    } else {
        const bool copy = a.copy[0] || a.copy[1];
        a.turned = interleaved ? (rot + W - 1) / W : rot / 2 / W;
        a.passed = !copy ? 0 : interleaved ? d / W - a.turned : (d - rot) / W;
        // Rows of a block: two warps over (row, item) (one took 6 % longer on 18432 rows of 32/8 heads, four the same), more where
        // there are too few heads for the other threads, fewer where blocks would not fill the SMs twice.
        const int items = a.turned + a.passed;
        a.per_block = 1;
        while (a.per_block < kMaxRows && 2 * a.per_block * items <= kThreads && rows / (2 * a.per_block) >= 2 * current_sm_count() &&
               (a.per_block * items < kLanes || kThreads / (a.per_block * items) * kBatch > Hq + Hkv))
            a.per_block *= 2;
        const unsigned grid = static_cast<unsigned>((rows + a.per_block - 1) / a.per_block);
        const int smem = a.per_block * (rot / 2) * static_cast<int>(sizeof(float2));  // at most 32 KB
        auto launch = [&](auto kern) { launched = launch_programmatic(kern, dim3(grid), kThreads, smem, stream, a); };
        if (interleaved)
            W == 8 ? launch(rope_kernel<kInterleaved, 8>) : W == 4 ? launch(rope_kernel<kInterleaved, 4>) : launch(rope_kernel<kInterleaved, 2>);
        else
            W == 8 ? launch(rope_kernel<kHalves, 8>) : W == 4 ? launch(rope_kernel<kHalves, 4>) : launch(rope_kernel<kHalves, 2>);
    }
    return launched == cudaSuccess ? BLINK_OK : BLINK_CUDA_ERROR;
}
