// keyweights.cu -- attention weight received by each prefix key: for every (kv head, key) the sum over
// rows and the group's query heads of exp(scale q.k - lse).
//
// One thread per key, its key vector in registers; the group's query rows pass through shared memory
// 32 at a time (every thread reads the same row: a broadcast), FP32 products and sums.
#include <cstdint>

#include "common.cuh"

namespace blink {
namespace {

constexpr int kKeys = 128;
constexpr int kCols = 32;  // query columns (row, head of the group) per step
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
__global__ void __launch_bounds__(kKeys) key_weights_kernel(const uint16_t *__restrict__ q,
                                                            const uint16_t *__restrict__ k, int64_t k_stride,
                                                            const float *__restrict__ lse, int64_t lse_stride, int rows,
                                                            int P, int Hq, int g, float scale_log2, float decay,
                                                            const float *prev, int64_t prev_stride, float *w,
                                                            int64_t w_stride)
{
    __shared__ float qs[kCols][D];
    __shared__ float bias[kCols];
    const int head = blockIdx.y;
    const int p = blockIdx.x * kKeys + threadIdx.x;
    float kr[D];
#pragma unroll
    for (int i = 0; i < D; ++i)
        kr[i] = p < P ? __uint_as_float(static_cast<uint32_t>(k[p * k_stride + head * D + i]) << 16) : 0.f;
    float sum = 0.f;
    const int64_t n_col = static_cast<int64_t>(rows) * g;
    for (int64_t c0 = 0; c0 < n_col; c0 += kCols) {
        __syncthreads();
        for (int i = threadIdx.x; i < kCols * D; i += kKeys) {
            const int64_t c = c0 + i / D;
            qs[i / D][i % D] =
                c < n_col ? __uint_as_float(static_cast<uint32_t>(q[((c / g) * Hq + head * g + c % g) * D + i % D]) << 16)
                          : 0.f;
        }
        if (threadIdx.x < kCols) {
            const int64_t c = c0 + threadIdx.x;
            bias[threadIdx.x] = c < n_col ? lse[(head * g + c % g) * lse_stride + c / g] : -INFINITY;
        }
        __syncthreads();
        for (int c = 0; c < kCols; ++c) {
            if (bias[c] == -INFINITY) continue;  // a row owned by no question
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < D; ++i) s = fmaf(qs[c][i], kr[i], s);
            sum += exp2f(fmaf(s, scale_log2, -bias[c] * kLog2e));
        }
    }
    if (p < P) w[head * w_stride + p] = decay > 0.f ? fmaf(decay, prev[head * prev_stride + p], sum) : sum;
}

}  // namespace
}  // namespace blink

extern "C" size_t blink_prefix_key_weights_workspace(int32_t rows, int32_t P, int32_t Hq, int32_t Hkv, int32_t d)
{
    (void)rows, (void)P, (void)Hq, (void)Hkv, (void)d;
    return blink::kHeaderBytes;
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
    const float sc = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(d));
    const dim3 grid(static_cast<unsigned>((P + kKeys - 1) / kKeys), static_cast<unsigned>(Hkv));
    auto kern = d == 128 ? key_weights_kernel<128> : key_weights_kernel<64>;
    kern<<<grid, kKeys, 0, stream>>>(q, k_pre, pre_row_stride, lse, lse_stride, rows, P, Hq, Hq / Hkv, sc * kLog2e, decay,
                                     d_prev, prev_stride, d_weights, w_stride);
    if (cudaGetLastError() != cudaSuccess) return BLINK_CUDA_ERROR;
    return BLINK_OK;
}
