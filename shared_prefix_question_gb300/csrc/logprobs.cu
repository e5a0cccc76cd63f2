// logprobs.cu -- log probabilities of given tokens, entropy and top alternatives over the whole
// vocabulary, without writing the logits.
//
// Mathematics.  With y = z log2(e) / T for the raw product z = h . w, a part of the vocabulary is
// summarised by m = max y, s = sum 2^(y - m) and u = sum 2^(y - m) (y - m); two parts merge by
// rescaling to the larger m:  s = a s1 + b s2,  u = a (u1 + s1 (m1 - m)) + b (u2 + s2 (m2 - m)) with
// a = 2^(m1 - m), b = 2^(m2 - m).  Then lse = ln2 (m + log2 s) and entropy = ln2 (log2 s - u / s).
//
// One block per (8 hidden rows, part of the vocabulary): a warp takes a vocabulary row, its lanes
// split H, and after the reduction lane r folds the product of hidden row r into its state.
#include <cstdint>

#include "common.cuh"

namespace blink {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRows = 8;
constexpr int kWarps = 8;
constexpr int kMaxTop = BLINK_MAX_TOP_TOKENS;
constexpr int kParts = 64;

__device__ __forceinline__ float lo16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi16(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

struct LogprobArgs {
    const uint16_t *hidden;
    int64_t hidden_stride;
    int hidden_rows;
    const int32_t *row_idx;
    const uint16_t *W;
    int V, H, n, top;
    const int32_t *targets;
    float c;  // log2(e) / T
    float4 *stat;  // [parts][n]: m, s, u, target's raw product (NaN: not in this part)
    float *top_z;  // [parts][n][top] raw products, descending
    int32_t *top_id;
    float *logprob, *entropy, *lse, *top_lp;
    int32_t *top_ids;
    int *err;
};

__device__ __forceinline__ void merge_stat(float &m, float &s, float &u, float m2, float s2, float u2)
{
    if (m2 == -INFINITY) {
        s += s2;  // an empty part, or one of NaN alone
        return;
    }
    const float M = fmaxf(m, m2);
    const float d1 = m == -INFINITY ? 0.f : m - M, d2 = m2 - M;
    const float a = exp2f(d1), b = exp2f(d2);
    u = a * (u + s * d1) + b * (u2 + s2 * d2);
    s = a * s + b * s2;
    m = M;
}

// Inserts (z, id) into a descending list of n entries, equal values staying in front; NaN never enters.
__device__ __forceinline__ void insert_top(float *v, int32_t *id, int n, float z, int32_t i)
{
    if (!(z > v[n - 1]) && !(z == v[n - 1] && i < id[n - 1])) return;
    int j = n - 1;
    while (j > 0 && (v[j - 1] < z || (v[j - 1] == z && id[j - 1] > i))) {
        v[j] = v[j - 1];
        id[j] = id[j - 1];
        --j;
    }
    v[j] = z;
    id[j] = i;
}

__global__ void __launch_bounds__(kWarps * 32) logprob_part_kernel(const LogprobArgs a)
{
    extern __shared__ uint4 hs[];  // [kRows][H / 8]
    __shared__ float tv[kWarps][kRows][kMaxTop];
    __shared__ int32_t ti[kWarps][kRows][kMaxTop];
    __shared__ float4 st[kWarps][kRows];
    const int r0 = blockIdx.x * kRows, part = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nch = a.H / 8;
    for (int i = threadIdx.x; i < kRows * nch; i += kWarps * 32) {
        const int r = r0 + i / nch;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < a.n) {
            const int hr = a.row_idx ? a.row_idx[r] : r;
            if (hr >= 0 && hr < a.hidden_rows)
                x = reinterpret_cast<const uint4 *>(a.hidden + hr * a.hidden_stride)[i % nch];
        }
        hs[i] = x;
    }
    for (int i = threadIdx.x; i < kWarps * kRows * kMaxTop; i += kWarps * 32) {
        (&tv[0][0][0])[i] = -INFINITY;
        (&ti[0][0][0])[i] = 0x7FFFFFFF;
    }
    __syncthreads();
    float m = -INFINITY, s = 0.f, u = 0.f, tz = __int_as_float(0x7FC00000);
    const int target = (a.targets && lane < kRows && r0 + lane < a.n) ? a.targets[r0 + lane] : -1;
    const int64_t v0 = static_cast<int64_t>(a.V) * part / gridDim.y, v1 = static_cast<int64_t>(a.V) * (part + 1) / gridDim.y;
    for (int64_t v = v0 + warp; v < v1; v += kWarps) {
        float acc[kRows] = {};
        const uint4 *wr = reinterpret_cast<const uint4 *>(a.W + v * a.H);
        for (int c = lane; c < nch; c += 32) {
            const uint4 x = __ldg(wr + c);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const uint4 h = hs[r * nch + c];
                acc[r] = fmaf(lo16(x.x), lo16(h.x), acc[r]);
                acc[r] = fmaf(hi16(x.x), hi16(h.x), acc[r]);
                acc[r] = fmaf(lo16(x.y), lo16(h.y), acc[r]);
                acc[r] = fmaf(hi16(x.y), hi16(h.y), acc[r]);
                acc[r] = fmaf(lo16(x.z), lo16(h.z), acc[r]);
                acc[r] = fmaf(hi16(x.z), hi16(h.z), acc[r]);
                acc[r] = fmaf(lo16(x.w), lo16(h.w), acc[r]);
                acc[r] = fmaf(hi16(x.w), hi16(h.w), acc[r]);
            }
        }
        float z = 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float t = acc[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
            if (lane == r) z = t;
        }
        if (lane < kRows) {
            const float y = z * a.c;
            if (y > m) {
                const float d = m == -INFINITY ? 0.f : m - y, f = exp2f(d);
                u = f * (u + s * d);
                s *= f;
                m = y;
            }
            const float x = y - m, e = exp2f(x);
            s += e;
            u = fmaf(e, x, u);
            if (v == target) tz = z;
            if (a.top) insert_top(tv[warp][lane], ti[warp][lane], a.top, z, static_cast<int32_t>(v));
        }
        __syncwarp();
    }
    if (lane < kRows) st[warp][lane] = make_float4(m, s, u, tz);
    __syncthreads();
    if (threadIdx.x < kRows && r0 + threadIdx.x < a.n) {
        const int r = threadIdx.x;
        float4 x = st[0][r];
        for (int w = 1; w < kWarps; ++w) {
            const float4 y = st[w][r];
            merge_stat(x.x, x.y, x.z, y.x, y.y, y.z);
            if (y.w == y.w) x.w = y.w;
            for (int j = 0; j < a.top; ++j) insert_top(tv[0][r], ti[0][r], a.top, tv[w][r][j], ti[w][r][j]);
        }
        const int64_t row = static_cast<int64_t>(part) * a.n + r0 + r;
        a.stat[row] = x;
        for (int j = 0; j < a.top; ++j) {
            a.top_z[row * a.top + j] = tv[0][r][j];
            a.top_id[row * a.top + j] = ti[0][r][j];
        }
    }
}

__global__ void logprob_merge_kernel(const LogprobArgs a, int parts)
{
    const int r = blockIdx.x * blockDim.x + threadIdx.x;
    if (r >= a.n) return;
    float m = -INFINITY, s = 0.f, u = 0.f, tz = __int_as_float(0x7FC00000);
    float tv[kMaxTop];
    int32_t ti[kMaxTop];
    for (int j = 0; j < a.top; ++j) tv[j] = -INFINITY, ti[j] = 0x7FFFFFFF;
    for (int p = 0; p < parts; ++p) {
        const int64_t row = static_cast<int64_t>(p) * a.n + r;
        const float4 x = a.stat[row];
        merge_stat(m, s, u, x.x, x.y, x.z);
        if (x.w == x.w) tz = x.w;
        for (int j = 0; j < a.top; ++j) insert_top(tv, ti, a.top, a.top_z[row * a.top + j], a.top_id[row * a.top + j]);
    }
    const float nan = __int_as_float(0x7FC00000);
    const int hr = a.row_idx ? a.row_idx[r] : r;
    const bool bad = hr < 0 || hr >= a.hidden_rows;
    const int t = a.targets ? a.targets[r] : -1;
    if (bad || t < -1 || t >= a.V) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
    const float l2 = bad ? nan : m + log2f(s);
    if (a.lse) a.lse[r] = l2 * kLn2;
    if (a.entropy) a.entropy[r] = bad ? nan : (log2f(s) - u / s) * kLn2;
    if (a.logprob) a.logprob[r] = (tz * a.c - l2) * kLn2;
    for (int j = 0; j < a.top; ++j) {
        const bool none = bad || ti[j] == 0x7FFFFFFF;
        a.top_ids[static_cast<int64_t>(r) * a.top + j] = none ? -1 : ti[j];
        a.top_lp[static_cast<int64_t>(r) * a.top + j] = none ? nan : (tv[j] * a.c - l2) * kLn2;
    }
}

struct Layout {
    size_t stat, top_z, top_id, total;
};

Layout layout_of(int n, int top)
{
    Layout l{};
    const size_t cells = static_cast<size_t>(kParts) * n;
    l.stat = kHeaderBytes;
    l.top_z = l.stat + align_up(cells * sizeof(float4), 256);
    l.top_id = l.top_z + align_up(cells * top * sizeof(float), 256);
    l.total = l.top_id + align_up(cells * top * sizeof(int32_t), 256);
    return l;
}

}  // namespace
}  // namespace blink

extern "C" size_t blink_token_logprobs_workspace(int32_t n, int32_t H, int32_t V, int32_t top)
{
    using namespace blink;
    if (n < 1 || n > BLINK_MAX_INPUT_TOKENS || H < 1 || V < 1 || top < 0 || top > kMaxTop) return kHeaderBytes;
    return layout_of(n, top).total;
}

extern "C" blink_status blink_token_logprobs(const blink_bf16 *hidden, int64_t hidden_row_stride, int32_t hidden_rows,
                                             const int32_t *d_row_idx, const blink_bf16 *unembed, int32_t V, int32_t H,
                                             const int32_t *d_targets, int32_t n, float temperature, int32_t top,
                                             float *d_logprob, float *d_entropy, float *d_lse, int32_t *d_top_ids,
                                             float *d_top_logprobs, void *d_ws, size_t ws_bytes, cudaStream_t stream)
{
    using namespace blink;
    if (!hidden || !unembed || !d_ws) return BLINK_INVALID_ARG;
    if (!d_logprob && !d_entropy && !d_lse && !d_top_ids) return BLINK_INVALID_ARG;
    if ((d_logprob && !d_targets) || (d_top_ids == nullptr) != (d_top_logprobs == nullptr)) return BLINK_INVALID_ARG;
    if (!(temperature > 0.f) || !(temperature < INFINITY)) return BLINK_INVALID_ARG;
    if (H < 8 || H % 8 != 0 || V < 1 || hidden_rows < 1 || hidden_row_stride < H || hidden_row_stride % 8 != 0)
        return BLINK_INVALID_ARG;
    if (!aligned16(hidden) || !aligned16(unembed)) return BLINK_INVALID_ARG;
    if (top < 0 || top > kMaxTop || top > V || H > 32768 || V > (1 << 24)) return BLINK_OUT_OF_RANGE;
    if ((top > 0) != (d_top_ids != nullptr)) return BLINK_INVALID_ARG;
    if (n < 1 || n > BLINK_MAX_INPUT_TOKENS) return BLINK_OUT_OF_RANGE;
    if (!d_row_idx && n > hidden_rows) return BLINK_INVALID_ARG;
    if (ws_bytes < blink_token_logprobs_workspace(n, H, V, top)) return BLINK_WORKSPACE_TOO_SMALL;
    const Layout l = layout_of(n, top);
    auto *wsb = static_cast<uint8_t *>(d_ws);
    LogprobArgs a{};
    a.hidden = hidden;
    a.hidden_stride = hidden_row_stride;
    a.hidden_rows = hidden_rows;
    a.row_idx = d_row_idx;
    a.W = unembed;
    a.V = V;
    a.H = H;
    a.n = n;
    a.top = top;
    a.targets = d_targets;
    a.c = kLog2e / temperature;
    a.stat = reinterpret_cast<float4 *>(wsb + l.stat);
    a.top_z = reinterpret_cast<float *>(wsb + l.top_z);
    a.top_id = reinterpret_cast<int32_t *>(wsb + l.top_id);
    a.logprob = d_logprob;
    a.entropy = d_entropy;
    a.lse = d_lse;
    a.top_lp = d_top_logprobs;
    a.top_ids = d_top_ids;
    a.err = &static_cast<WorkspaceHeader *>(d_ws)->error;
    const int smem = kRows * H * 2;
    if (cudaFuncSetAttribute(logprob_part_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return BLINK_CUDA_ERROR;
    const dim3 grid(static_cast<unsigned>((n + kRows - 1) / kRows), kParts);
    logprob_part_kernel<<<grid, kWarps * 32, smem, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return BLINK_CUDA_ERROR;
    logprob_merge_kernel<<<(n + 127) / 128, 128, 0, stream>>>(a, kParts);
    if (cudaGetLastError() != cudaSuccess) return BLINK_CUDA_ERROR;
    return BLINK_OK;
}
