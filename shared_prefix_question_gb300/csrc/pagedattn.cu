// pagedattn.cu -- attention of a few rows over 8-bit pages: the last tokens of each sequence, or few tail rows of
// requests whose prefix the pages hold.
//
// One pass over the keys with a running maximum and sum.  A step is 16 keys of one kv head, always within a page.  Keys
// are the rows of the first product (S^T = K Q^T) and channels those of the second (O^T = V^T P^T); the columns of both
// are 8 of the (token, query head) rows that share the kv head, so that four rows waste half of the products and not
// three quarters.  Codes become fp16 values exactly, queries keep their 8 bits in fp16 too (each row moved by a power
// of two so that its largest value fits), and the scales never touch a value: K's is a factor of the step's scores,
// V's goes into the weights.
//
// Bound by HBM: 2 bytes a key, head and channel against 4 rows' products.  A lane's operands of the products are its
// own bytes of memory: both products allow any order of the summed index and of the output's channels, so a lane takes
// 16 consecutive bytes of a key for four product steps, and 16 consecutive channels of four keys for eight products.
// A step's keys and values are two tensor copies of 16 rows into the warp's own ring in shared memory, a few steps ahead;
// swizzled rows make the lanes' reads free of bank conflicts.  (The same bytes fetched by 16-byte asynchronous copies
// of each lane came at 5.2 TB/s with no arithmetic at all.)  A warp's step is a chain of products, exponentials and
// products again, so it takes warps to hide it: blocks of four, several an SM, no barrier between a block's warps.
#include <cmath>

#include "paged.cuh"
#include "ptx.cuh"

namespace blink {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 16;                        // keys
constexpr int kRound = kStep * kWarps;           // keys of a block per step of its warps
constexpr int kMaxChunk = 32 * kRound;           // a lane holds the page of one step of its warp
// (Row, query head) rows of a kv head, in any request, up to which tail rows read the pages: every 16 of them read and convert
// all codes again, while bf16 rows are written once and shared by 128.  18432 keys, one request of 16 tokens and 32/8 heads
// (64 rows): 29 us from the pages, 43 by way of bf16 rows; of 32 tokens 62 and 44; 2048 keys: 12 and 19, 18 and 19.  The limit
// does not look at the prefix: up to some 2048 keys it is too low for 128 rows, by a microsecond.
constexpr int kFewRows = 64;
// Waves of blocks from which, and sequences up to which, a grid of as many blocks as run at once takes the chunks that there are,
// one after the other, in place of a grid for all chunks that max_len allows.  A block without keys takes some 1.3 ns, but next
// chunks taken by a counter cost up to 2 % (max_len 131072, sequences of 1000 tokens, 64 of them: 72 and 39 us; 256: 257 and 112;
// 256 of 8000: 633 and 616; with max_len 18432, 11 waves, 64 of up to 18432: 187 and 191).  The lengths are on the device, so below
// the limit a call far below its max_len keeps the direct grid (eight of 1000, max_len 131072: 13.7 us, by the counter 9.8).
constexpr int kPackedWaves = 16, kMaxPacked = 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -1e37f;                 // below any score
constexpr float kHead = 6.f, kSlack = 8.f;       // weights start at 2^kHead and may grow by 2^kSlack before the maximum moves

// Tail rows: which rows of the call belong to each request, and the lengths of the prefixes.
struct TailRows {
    int row[kMaxPagedRequests + 1];
    int len[kMaxPagedRequests];
    int n_req, rows, B, max_tail;
    const uint16_t *k, *v;             // [rows][Hkv][d]
    const int32_t *cu, *seq_start;
};

struct TokenArgs {
    PagedCache c;
    const uint16_t *q;
    const int32_t *table;
    int64_t table_stride;
    int table_width;
    const int32_t *len;
    int max_len, S, T, Hq, Hkv, g, tiles;  // tiles: M tiles of a sequence and kv head
    int chunk, chunks;                     // most keys of a block, blocks of a sequence, head and tile
    int share;                             // blocks that a short sequence is cut into, if they get kRound keys each
    uint32_t one_share;                    // 2^32 / share, rounded up, of a share above 1
    float scale_log2;
    uint16_t *out;
    float *lse;
    float *part_lse, *part_o;              // [token][Hq][chunks] and the same with [D] behind
    int *err;
    int *taken;                            // items that blocks have taken past their first ones; 0 between calls
    TailRows tail;                         // with S = its requests; T and len are not used then
};

// A sequence's cached length, inside what the call allows; `bad`: it was not.
__device__ __forceinline__ int length_of(const TokenArgs &a, int seq, bool &bad)
{
    const int n = __ldg(a.len + seq);
    const int64_t room = static_cast<int64_t>(a.table_width) << a.c.log2_page;
    const int most = room < a.max_len ? static_cast<int>(room) : a.max_len;
    bad = n < 0 || n > most;
    return n < 0 ? 0 : n > most ? most : n;
}

// Keys of a block of a sequence of `len`: whole rounds of its warps, in at most a.chunks blocks.
__device__ __forceinline__ int chunk_of(const TokenArgs &a, int len)
{
    if (a.chunks == 1) return a.chunk;
    // ceil(len / share): the product is off by less than 2^-13 of a whole, a share at least 2^-11
    const int even = a.share == 1 ? len : static_cast<int>(__umulhi(static_cast<uint32_t>(len + a.share - 1), a.one_share));
    return min(max((even + kRound - 1) / kRound, 1) * kRound, a.chunk);
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t transposed(uint32_t v)  // of an 8 x 8 matrix of 16-bit values over the warp
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// NT: 8-row column tiles of a block.
template <int D, int NT>
struct Shape {
    // Blocks of an SM, and steps of a warp in shared memory (one of them in use): fewer warps with more bytes in flight
    // each.  (One tile: four blocks with three steps spill, and take 195 us instead of 186 on 64 sequences of up to 18432
    // tokens.  Two tiles: two blocks with six steps take 235 us instead of 212 on 8 sequences of up to 131072 with four
    // tokens each; three cost six registers spilled.)
    static constexpr int kResident = 3;
    static constexpr int kDepth = 4;
    static constexpr int kRows = 8 * NT;
    static constexpr int kPieces = D / 64;                 // 16-byte pieces of a key for one lane
    static constexpr int kCols = D / 8;                    // consecutive channels of a lane in the second product
    static constexpr int kTile = kStep * D;                // bytes of a step's keys, and of its values
    static constexpr int kStage = 2 * kTile;
    static constexpr int kRing = kWarps * kDepth * kStage;
    static constexpr int kPad = D + 4;                     // floats of a row where the warps' sums are joined
    static constexpr int kJoin = kWarps * kRows * kPad * 4 + 2 * kWarps * kRows * 4;
    static constexpr int kBars = kRing > kJoin ? kRing : kJoin;         // where the barriers lie
    static constexpr int kSmem = 1024 + kBars + kWarps * kDepth * 8 + 16;  // the ring is 1024-byte aligned
};

// Byte offset of a 16-byte piece of a row in a swizzled tile of D-byte rows.
template <int D>
__device__ __forceinline__ int piece_at(int row, int piece)
{
    return row * D + ((D == 128 ? piece ^ (row & 7) : piece ^ (row >> 1 & 3)) << 4);
}

// The chunks that the sequences before each have together, `first`, and all of them (returned), by a whole block.
template <bool TAIL>
__device__ __forceinline__ int count_chunks(const TokenArgs &a, int *first)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, each = (a.S + kThreads - 1) / kThreads;
    const int begin = min(threadIdx.x * each, a.S), end = min(begin + each, a.S);
    int mine = 0;
    for (int s = begin; s < end; ++s) {
        bool bad = false;
        const int len = TAIL ? a.tail.len[s] : length_of(a, s, bad), chunk = chunk_of(a, len);
        if (bad && blockIdx.x == 0) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
        first[s] = mine;
        mine += (len + chunk - 1) / chunk;
    }
    int before = mine;  // with the lanes before
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int n = __shfl_up_sync(0xFFFFFFFFu, before, d);
        before += lane >= d ? n : 0;
    }
    if (lane == 31) first[a.S + warp] = before;
    __syncthreads();
    int total = 0;
    before -= mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int n = first[a.S + w];
        before += w < warp ? n : 0;
        total += n;
    }
    for (int s = begin; s < end; ++s) first[s] += before;
    __syncthreads();
    return total;
}

// PACKED: a grid of as many blocks as run at once goes over the chunks that the sequences have, in place of a grid of those that
// the longest allowed one could have.
template <int D, int NT, bool TAIL, bool PACKED>
__global__ void __launch_bounds__(kThreads, Shape<D, NT>::kResident) token_attention_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ TokenArgs a)
{
    using Sh = Shape<D, NT>;
    constexpr int kDepth = Sh::kDepth;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-ptx::smem_u32(smem_raw) & 1023u);
    int *abort_flag = reinterpret_cast<int *>(smem + Sh::kBars + kWarps * kDepth * 8);
    int *first = abort_flag + 4;                  // [S], and the warps' sums behind them
    int *next = first + (PACKED ? a.S : 0) + kWarps;  // this block's next item, in two places by turns
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, quad = lane & 3;  // products: rows r and r + 8, columns 2 quad and 2 quad + 1
    uint8_t *ring = smem + warp * kDepth * Sh::kStage;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Sh::kBars) + warp * kDepth;
    auto init_bars = [&] {
        if (lane == 0) {
            *abort_flag = 0;
            for (int i = 0; i < kDepth; ++i) ptx::mbar_init(&bars[i], 1);
            ptx::fence_mbar_init();
        }
        __syncwarp();
    };
    int stage = 0;
    uint32_t parity = 0;

    // What is launched behind this grid starts when all its blocks are past this wait, so the join, which reads lengths,
    // queries and tails before it waits for this grid, finds what was written before this grid.
    ptx::grid_dep_wait();
    ptx::grid_launch_dependents();
    int items = 1;
    if constexpr (PACKED) {
        init_bars();
        items = count_chunks<TAIL>(a, first) * a.Hkv * a.tiles;
    }
    for (int item = PACKED ? blockIdx.x : 0, turn = 0; item < items; turn ^= 1) {
        int ticket = 0;
        if (PACKED && threadIdx.x == 0) ticket = atomicAdd(a.taken, 1) + gridDim.x;
        int seq = blockIdx.z, ht = blockIdx.y, part = blockIdx.x;  // ht: kv head and tile
        if constexpr (PACKED) {
            const int units = a.Hkv * a.tiles, c = item / units;
            ht = item - c * units;
            seq = last_before(0, a.S, [&](int s) { return first[s] <= c; });  // the last of those that start there has keys
            part = c - first[seq];
        }
        const int h = ht / a.tiles, tile = ht - h * a.tiles;
        const int T = TAIL ? a.tail.row[seq + 1] - a.tail.row[seq] : a.T;
        const int64_t token0 = TAIL ? a.tail.row[seq] : static_cast<int64_t>(seq) * a.T;
        const int Tg = T * a.g, rho0 = tile * Sh::kRows, rows = min(Sh::kRows, Tg - rho0);

        if (TAIL && rows <= 0) {  // fewer rows than another request
            if constexpr (!PACKED) return;
            if (threadIdx.x == 0) next[turn] = ticket;
            __syncthreads();
            item = next[turn];
            continue;
        }
        // The pages of this warp's steps, one a lane, read before the length is known, and again if it takes shorter chunks.
        auto page_from = [&](int k0) {
            const int64_t index = (static_cast<int64_t>(k0) + (warp + lane * kWarps) * kStep) >> a.c.log2_page;
            return index < a.table_width ? __ldg(a.table + seq * a.table_stride + index) : -1;
        };
        int page = page_from(part * a.chunk);
        bool bad = false;
        const int len = TAIL ? a.tail.len[seq] : length_of(a, seq, bad), chunk = chunk_of(a, len);
        const int k0 = part * chunk, k1 = min(len, k0 + chunk);
        if (!PACKED && bad && threadIdx.x == 0) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
        if (!PACKED && k0 >= k1 && a.chunks > 1) return;  // the join knows the length too
        if (chunk != a.chunk) page = page_from(k0);
        const int steps = max(0, (k1 - k0 + kStep - 1) / kStep);
        const int mine = steps > warp ? (steps - warp + kWarps - 1) / kWarps : 0;
        int scales = kScaleBias | kScaleBias << 8;
        if (page < 0 || page >= a.c.n_pages || lane >= mine) {
            if (lane < mine) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
            page = -1;  // past the end, or not a page: its keys are masked (TAIL: zeros, as in the rows that pages are turned to)
        } else {
            scales = (exponent_of(__ldg(a.c.k_scale + page * a.c.scale_stride + h)) + kScaleBias) |
                     (exponent_of(__ldg(a.c.v_scale + page * a.c.scale_stride + h)) + kScaleBias) << 8;
        }
        if constexpr (!PACKED) init_bars();

        // Copies of step i into its slot, which all lanes have read before.
        auto issue = [&](int i, int stage) {
            const int id = __shfl_sync(0xFFFFFFFFu, page, i & 31);
            if (i < mine && lane == 0) {
                const int key = k0 + (warp + i * kWarps) * kStep;
                uint8_t *slot = ring + stage * Sh::kStage;
                if (id >= 0) {
                    const int row = (h << a.c.log2_page) + (key & ((1 << a.c.log2_page) - 1));
                    ptx::mbar_arrive_expect_tx(&bars[stage], Sh::kStage);
                    ptx::tma_load_3d(slot, &tm_k, 0, row, id, &bars[stage]);
                    ptx::tma_load_3d(slot + Sh::kTile, &tm_v, 0, row, id, &bars[stage]);
                } else {
                    ptx::mbar_arrive(&bars[stage]);  // no page: the slot holds anything, and nothing reads it as a key
                }
            }
        };
#pragma unroll
        for (int i = 0; i < kDepth - 1; ++i) issue(i, !PACKED ? i : stage + i < kDepth ? stage + i : stage + i - kDepth);

        // Queries as the second operand, in the order of the key bytes: product step 4 p + w takes channels
        // 16 kPieces quad + 16 p + 4 w .. + 3 of this lane; the lane holds row r of each tile.
        uint32_t qb[NT][4 * Sh::kPieces][2];
        float base[NT][2];  // of rows 2 quad and 2 quad + 1: the factor of their scores
        int see[NT][2];     // keys that they see
#pragma unroll
        for (int y = 0; y < NT; ++y) {
            const int rho = rho0 + 8 * y + r, t = rho / a.g, j = rho - t * a.g;
            uint4 w[2 * Sh::kPieces];
#pragma unroll
            for (int p = 0; p < Sh::kPieces; ++p) {
                w[2 * p] = w[2 * p + 1] = make_uint4(0, 0, 0, 0);
                if (rho < Tg) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        a.q + ((token0 + t) * a.Hq + h * a.g + j) * D + quad * 16 * Sh::kPieces + p * 16);
                    w[2 * p] = __ldg(src);
                    w[2 * p + 1] = __ldg(src + 1);
                }
            }
            const uint32_t *x = reinterpret_cast<const uint32_t *>(w);
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < 8 * Sh::kPieces; ++e)
                m = fmaxf(m, fmaxf(fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xFFFF0000u))));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            // the row's largest value between 2^9 and 2^10: none overflows, and values below 2^-26 of it lose bits (fp16's last
            // step is 2^-24, a value's eight bits end 2^-7 below its first)
            int move = 9 - (static_cast<int>(__float_as_uint(m) >> 23) - 127);
            move = !(m > 0.f) || m == INFINITY ? 0 : min(move, 126);
            const float f = scale_of(move), back = a.scale_log2 * scale_of(-move);
#pragma unroll
            for (int e = 0; e < 8 * Sh::kPieces; ++e)  // word e: channels 2 e, 2 e + 1 of the lane's 16 of a piece
                qb[y][e / 2][e & 1] = pack_f16x2(__uint_as_float(x[e] << 16) * f, __uint_as_float(x[e] & 0xFFFF0000u) * f);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                base[y][c] = __shfl_sync(0xFFFFFFFFu, back, (2 * quad + c) * 4);
                see[y][c] = TAIL ? len : len - (T - 1 - min(rho0 + 8 * y + 2 * quad + c, Tg - 1) / a.g);
            }
        }
        const int t_first = TAIL ? 0 : rho0 / a.g, t_last = TAIL ? 0 : (rho0 + rows - 1) / a.g;
        const int see_least = TAIL ? len : len - (T - 1 - t_first);  // the fewest keys that a row sees

        float o[NT][Sh::kCols / 2][4];  // channels kCols r + 2 j (first two) and + 1, rows 2 quad and 2 quad + 1
#pragma unroll
        for (int y = 0; y < NT; ++y)
#pragma unroll
            for (int j = 0; j < Sh::kCols / 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[y][j][e] = 0.f;
        float most[NT][2], sum[NT][2];
#pragma unroll
        for (int y = 0; y < NT; ++y) most[y][0] = most[y][1] = kNoMax, sum[y][0] = sum[y][1] = 0.f;
        int unit = kScaleMin - 1;  // o is in units of 2^unit

        bool fine = true;
        for (int i = 0; i < mine; ++i) {
            __syncwarp();
            issue(i + kDepth - 1, stage == 0 ? kDepth - 1 : stage - 1);
            fine = ptx::mbar_wait_warp(&bars[stage], parity, abort_flag, a.err, BLINK_DEVICE_TIMEOUT);
            if (!fine) {  // the copies in flight still land in this block's memory: wait for them, again with a limit
                int other = 0;
                for (int n = i; n < min(mine, i + kDepth); ++n) {
                    ptx::mbar_wait(&bars[stage], parity, &other, a.err, BLINK_DEVICE_TIMEOUT);
                    other = 0;
                    if (++stage == kDepth) stage = 0, parity ^= 1;
                }
                break;
            }
            const int key = k0 + (warp + i * kWarps) * kStep;
            const int id = __shfl_sync(0xFFFFFFFFu, page, i), both = __shfl_sync(0xFFFFFFFFu, scales, i);
            const int ek = (both & 0xFF) - kScaleBias, ev = (both >> 8) - kScaleBias;
            const uint8_t *slot = ring + stage * Sh::kStage;
            if (++stage == kDepth) stage = 0, parity ^= 1;

            float s[NT][2][4];
#pragma unroll
            for (int y = 0; y < NT; ++y)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[y][b][e] = 0.f;
#pragma unroll
            for (int p = 0; p < Sh::kPieces; ++p) {
                const uint4 klo = *reinterpret_cast<const uint4 *>(slot + piece_at<D>(r, quad * Sh::kPieces + p));      // key r
                const uint4 khi = *reinterpret_cast<const uint4 *>(slot + piece_at<D>(r + 8, quad * Sh::kPieces + p));  // key r + 8
                const uint32_t *w = reinterpret_cast<const uint32_t *>(&klo), *x = reinterpret_cast<const uint32_t *>(&khi);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t ka[4] = {e4m3x2_to_f16x2(w[e]), e4m3x2_to_f16x2(x[e]), e4m3x2_hi_to_f16x2(w[e]),
                                            e4m3x2_hi_to_f16x2(x[e])};
#pragma unroll
                    for (int y = 0; y < NT; ++y) mma16816(s[y][e & 1], ka, qb[y][4 * p + e][0], qb[y][4 * p + e][1]);
                }
            }
            const bool edge = key + kStep > see_least || id < 0;  // warp-uniform
            const float fk = scale_of(ek);
            float x[NT][4];  // keys r (first two) and r + 8, rows 2 quad and 2 quad + 1
            bool grow = false;
#pragma unroll
            for (int y = 0; y < NT; ++y) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[y][e] = (s[y][0][e] + s[y][1][e]) * (base[y][e & 1] * fk);
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (key + r + 8 * (e >> 1) >= see[y][e & 1] || (!TAIL && id < 0)) x[y][e] = -INFINITY;
                        else if (TAIL && id < 0) x[y][e] = 0.f;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) grow = grow || fmaxf(x[y][c], x[y][c + 2]) > most[y][c] + (kSlack + kHead);
            }
            // The maximum moves only when a weight would pass 2^(kHead + kSlack), the unit when a page's V scale is above
            // it (a weight might overflow fp16) or far below (weights would lose bits).
            const bool shift = ev > unit || ev < unit - 6;
            if (__any_sync(0xFFFFFFFFu, grow) || shift) {
                const float fu = unit < kScaleMin || !shift ? 1.f : scale_of(unit - ev);
                if (shift) unit = ev;
#pragma unroll
                for (int y = 0; y < NT; ++y)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float m = fmaxf(x[y][c], x[y][c + 2]);
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
                        float f = 1.f;
                        if (m > most[y][c] + (kSlack + kHead)) {
                            const float now = m - kHead;
                            f = ptx::ex2(most[y][c] - now);
                            most[y][c] = now;
                            sum[y][c] *= f;
                        }
                        f *= fu;
#pragma unroll
                        for (int j = 0; j < Sh::kCols / 2; ++j) {
                            o[y][j][c] *= f;
                            o[y][j][c + 2] *= f;
                        }
                    }
            }
            const float fv = scale_of(ev - unit);
            uint32_t pb[NT][2];
#pragma unroll
            for (int y = 0; y < NT; ++y) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = ptx::ex2(x[y][e] - most[y][e & 1]);
                sum[y][0] += p[0] + p[2];
                sum[y][1] += p[1] + p[3];
                pb[y][0] = transposed(pack_f16x2(p[0] * fv, p[1] * fv));
                pb[y][1] = transposed(pack_f16x2(p[2] * fv, p[3] * fv));
            }
            uint32_t v[4][Sh::kCols / 4];
            const uint8_t *vs = slot + Sh::kTile;
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // keys 2 quad, 2 quad + 1, 2 quad + 8, 2 quad + 9
                const int row = 2 * quad + (e & 1) + (e >> 1) * 8;
                if constexpr (Sh::kCols == 16) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(vs + piece_at<D>(row, r));
                    v[e][0] = w.x, v[e][1] = w.y, v[e][2] = w.z, v[e][3] = w.w;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2 *>(vs + piece_at<D>(row, r >> 1) + (r & 1) * 8);
                    v[e][0] = w.x, v[e][1] = w.y;
                }
            }
            auto operand = [](uint32_t (&va)[4], uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3, uint32_t pick) {
                const uint32_t lo = __byte_perm(v0, v1, pick), hi = __byte_perm(v2, v3, pick);  // two channels of two keys each
                va[0] = e4m3x2_to_f16x2(lo);
                va[1] = e4m3x2_hi_to_f16x2(lo);
                va[2] = e4m3x2_to_f16x2(hi);
                va[3] = e4m3x2_hi_to_f16x2(hi);
            };
            if (!edge) {
#pragma unroll
                for (int j = 0; j < Sh::kCols / 2; ++j) {
                    const int w = j / 2;
                    uint32_t va[4];
                    operand(va, v[0][w], v[1][w], v[2][w], v[3][w], j & 1 ? 0x7362u : 0x5140u);
#pragma unroll
                    for (int y = 0; y < NT; ++y) mma16816(o[y][j], va, pb[y][0], pb[y][1]);
                }
            } else {
                // Keys that a row does not see may hold anything, a NaN times its zero weight too: for each token of the tile
                // the products run on the keys that it sees, and its rows take them.
                for (int t = t_first; t <= t_last; ++t) {
                    const int limit = TAIL ? len : len - (T - 1 - t);
                    uint32_t keep[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) keep[e] = id >= 0 && key + 2 * quad + (e & 1) + (e >> 1) * 8 < limit ? 0xFFFFFFFFu : 0u;
#pragma unroll
                    for (int j = 0; j < Sh::kCols / 2; ++j) {
                        const int w = j / 2;
                        uint32_t va[4];
                        operand(va, v[0][w] & keep[0], v[1][w] & keep[1], v[2][w] & keep[2], v[3][w] & keep[3], j & 1 ? 0x7362u : 0x5140u);
#pragma unroll
                        for (int y = 0; y < NT; ++y) {
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            mma16816(d, va, pb[y][0], pb[y][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[y][j][e] += TAIL || (rho0 + 8 * y + 2 * quad + (e & 1)) / a.g == t ? d[e] : 0.f;
                        }
                    }
                }
            }
        }

        // The warps' sums joined through shared memory, over the ring: every copy of this block has landed by the barrier.
        if (PACKED && threadIdx.x == 0) next[turn] = ticket;
        if (__syncthreads_or(!fine)) return;
        float *so = reinterpret_cast<float *>(smem);
        float *sm = so + kWarps * Sh::kRows * Sh::kPad, *sl = sm + kWarps * Sh::kRows;
#pragma unroll
        for (int y = 0; y < NT; ++y)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int d = 4; d < 32; d *= 2) sum[y][c] += __shfl_xor_sync(0xFFFFFFFFu, sum[y][c], d);
                if (r == 0) {
                    sm[warp * Sh::kRows + 8 * y + 2 * quad + c] = most[y][c];
                    sl[warp * Sh::kRows + 8 * y + 2 * quad + c] = sum[y][c];
                }
            }
        __syncthreads();
#pragma unroll
        for (int y = 0; y < NT; ++y)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = 8 * y + 2 * quad + c;
                if (row >= rows) continue;
                float top = kNoMax;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w * Sh::kRows + row]);
                const float f = ptx::ex2(most[y][c] - top + static_cast<float>(unit));
                float *dst = so + (warp * Sh::kRows + row) * Sh::kPad + r * Sh::kCols;
#pragma unroll
                for (int j = 0; j < Sh::kCols / 2; j += 2)
                    *reinterpret_cast<float4 *>(dst + 2 * j) =
                        make_float4(o[y][j][c] * f, o[y][j][c + 2] * f, o[y][j + 1][c] * f, o[y][j + 1][c + 2] * f);
            }
        __syncthreads();
        constexpr int kVec = D / 4;
        for (int e = threadIdx.x; e < rows * kVec; e += kThreads) {
            const int row = e / kVec, col = (e - row * kVec) * 4;
            float top = kNoMax, total = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w * Sh::kRows + row]);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                total += sl[w * Sh::kRows + row] * ptx::ex2(sm[w * Sh::kRows + row] - top);
                const float4 p = *reinterpret_cast<const float4 *>(so + (w * Sh::kRows + row) * Sh::kPad + col);
                v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
            }
            const bool none = total == 0.f;  // no key: zeros, and -inf
            const float inv = none ? 0.f : 1.f / total, l2 = none ? -INFINITY : top + log2f(total);
            v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
            const int rho = rho0 + row, t = rho / a.g, head = h * a.g + rho - t * a.g;
            const int64_t tok = token0 + t;
            if (TAIL || a.chunks > 1) {
                const int64_t at = (tok * a.Hq + head) * a.chunks + part;
                *reinterpret_cast<float4 *>(a.part_o + at * D + col) = v;
                if (col == 0) a.part_lse[at] = l2;
            } else {
                *reinterpret_cast<uint2 *>(a.out + (tok * a.Hq + head) * D + col) =
                    make_uint2(ptx::pack_bf16x2(v.x, v.y), ptx::pack_bf16x2(v.z, v.w));
                if (col == 0 && a.lse) a.lse[head * static_cast<int64_t>(a.S) * a.T + tok] = l2 * kLn2;
            }
        }
        if constexpr (PACKED) {  // the next copies land where the sums were
            ptx::fence_proxy_async_smem();
            __syncthreads();
        }
        item = PACKED ? next[turn] : 1;
    }
}

constexpr int kJoinWarps = 16;
constexpr int kJoinBatch = 8;  // chunks of a warp whose loads are in flight at once

template <int D>
__device__ __forceinline__ void load_channels(float (&x)[D / 32], const float *p)
{
    if constexpr (D == 128) {
        const float4 w = *reinterpret_cast<const float4 *>(p);
        x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
    } else {
        const float2 w = *reinterpret_cast<const float2 *>(p);
        x[0] = w.x, x[1] = w.y;
    }
}
template <int D>
__device__ __forceinline__ void load_channels(float (&x)[D / 32], const uint16_t *p)
{
    if constexpr (D == 128) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
        x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xFFFF0000u);
        x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(p));
        x[0] = __uint_as_float(w << 16), x[1] = __uint_as_float(w & 0xFFFF0000u);
    }
}

// The last question that starts at or before `row` (by a whole warp), and where it starts; -1: none.
__device__ __forceinline__ int question_of(const TailRows &t, int row, int &start)
{
    const int base = t.seq_start ? 0 : __ldg(t.cu);
    const int32_t *starts = t.seq_start ? t.seq_start : t.cu;
    const int b = last_before(-1, t.B, [&](int i) { return __ldg(starts + i) - base <= row; });
    start = b >= 0 ? __ldg(starts + b) - base : 0;
    return b;
}

// The chunks of a row joined by their log-sum-exp, a block a (token, query head): its warps share the chunks out, a lane
// holds D / 32 channels.  Bound by latency: a warp loads eight chunks at once, knows nothing of the others' maxima
// before the end, and there are warps for all chunks up to 128.  With TAIL the row's own question's keys (bf16, up to
// the row itself) are shared out to the warps as well.
template <int D, bool TAIL>
__global__ void __launch_bounds__(kJoinWarps * 32) token_join_kernel(const __grid_constant__ TokenArgs a)
{
    constexpr int kVec = D / 32;
    __shared__ float so[kJoinWarps][D], sw[kJoinWarps], st[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t row = blockIdx.x, tok = row / a.Hq;
    const int head = static_cast<int>(row - tok * a.Hq);
    int len, first = 0, keys = 0;  // keys of the question, from row `first` on
    bool owned = true;
    if constexpr (TAIL) {
        const TailRows &t = a.tail;
        int req = 0;
        while (req + 1 < t.n_req && t.row[req + 1] <= tok) ++req;
        len = t.len[req];
        const int b = question_of(t, static_cast<int>(tok), first);
        const int n = b < 0 ? 0 : __ldg(t.cu + b + 1) - __ldg(t.cu + b);
        const bool bad = b < 0 ? !t.seq_start : n < 1 || n > t.max_tail || static_cast<int64_t>(first) + n > t.rows || first < t.row[req];
        if (bad && threadIdx.x == 0) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
        owned = b >= 0 && !bad && tok < first + n;  // padding rows have no question
        keys = owned ? static_cast<int>(tok) - first + 1 : 0;
        if (row == 0)  // every question's length, also of those without a row
            for (int i = threadIdx.x; i < t.B; i += blockDim.x) {
                const int m = __ldg(t.cu + i + 1) - __ldg(t.cu + i);
                if (m < 1 || m > t.max_tail) atomicCAS(a.err, 0, BLINK_DEVICE_FLAG);
            }
    } else {
        bool bad;
        len = length_of(a, static_cast<int>(tok / a.T), bad);
    }
    const int chunk = chunk_of(a, len), n = owned ? (len + chunk - 1) / chunk : 0;
    float top = -INFINITY, total = 0.f, v[kVec] = {};
    auto take = [&](const float (&l)[kJoinBatch], const float (&x)[kJoinBatch][kVec]) {
        float now = top;
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) now = fmaxf(now, l[i]);
        const float f = top == -INFINITY ? 0.f : ptx::ex2(top - now);
        if (top != -INFINITY || total == 0.f) {  // what a NaN made stays
            total *= f;
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[e] *= f;
        }
        top = now;
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            if (l[i] == -INFINITY) continue;  // no chunk, or one without keys; a NaN counts
            const float w = ptx::ex2(l[i] - top);
            total += w;
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[e] += w * x[i][e];
        }
    };
    if constexpr (TAIL) {  // does not wait for the prefix part
        float q[kVec];
        load_channels<D>(q, a.q + row * D + lane * kVec);
        const int64_t stride = static_cast<int64_t>(a.Hkv) * D, at = first * stride + (head / a.g) * D + lane * kVec;
        for (int k0 = warp; k0 < keys; k0 += warps * kJoinBatch) {
            float l[kJoinBatch], x[kJoinBatch][kVec];
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i) {
                const int k = k0 + i * warps;
                l[i] = 0.f;
                if (k < keys) {
                    load_channels<D>(x[i], a.tail.k + at + k * stride);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) l[i] = fmaf(q[e], x[i][e], l[i]);
                    load_channels<D>(x[i], a.tail.v + at + k * stride);
                }
            }
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i) {
#pragma unroll
                for (int o = 16; o; o >>= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], o);
                l[i] = k0 + i * warps < keys ? l[i] * a.scale_log2 : -INFINITY;
            }
            take(l, x);
        }
    }
    ptx::grid_dep_wait();
    ptx::grid_launch_dependents();
    if (row == 0 && threadIdx.x == 0) *a.taken = 0;
    const float *pl = a.part_lse + row * a.chunks, *po = a.part_o + row * a.chunks * D + lane * kVec;
    for (int c0 = warp; c0 < n; c0 += warps * kJoinBatch) {
        float l[kJoinBatch], x[kJoinBatch][kVec];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            const int c = c0 + i * warps;
            l[i] = -INFINITY;
            if (c < n) {
                l[i] = pl[c];
                load_channels<D>(x[i], po + static_cast<int64_t>(c) * D);
            }
        }
        take(l, x);
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) so[warp][lane * kVec + e] = v[e];
    if (lane == 0) sw[warp] = total, st[warp] = top;
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < warps; ++w) top = fmaxf(top, st[w]);
    total = 0.f;
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = 0.f;
    for (int w = 0; w < warps; ++w) {
        if (sw[w] == 0.f) continue;
        const float f = st[w] == -INFINITY ? 1.f : ptx::ex2(st[w] - top);  // all NaN: no maximum
        total += f * sw[w];
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] += f * so[w][lane * kVec + e];
    }
    const bool none = total == 0.f;
    const float inv = none ? 0.f : 1.f / total;
    uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + row * D + lane * kVec);
#pragma unroll
    for (int e = 0; e < kVec; e += 2) dst[e / 2] = ptx::pack_bf16x2(v[e] * inv, v[e + 1] * inv);
    const int64_t tokens = TAIL ? a.tail.rows : static_cast<int64_t>(a.S) * a.T;
    if (lane == 0 && a.lse) a.lse[head * tokens + tok] = none ? -INFINITY : (top + log2f(total)) * kLn2;
}

struct TokenPlan {
    // Column tiles of a block.  Two where a head's rows need them: the codes are converted once for both (8 sequences of up
    // to 131072 with four tokens each, 32/8 heads: 212 us, with two blocks of one tile 264).  Two warps with a tile each over
    // the same ring, which convert twice, took 271.
    int wide;
    int tiles, chunk, chunks, share;
    size_t lse, o, total;  // offsets of the partial results in the workspace
};

// Keys of a block: every (sequence, head, tile) unit is cut into as many chunks as let whole waves of blocks hold all of
// them, one wave if a chunk is then no longer than the lanes can hold pages for; a chunk is whole rounds of the block's
// warps.  (320 blocks where 304 ran at a time: 39 us instead of 30 for 16 tail rows against 18432 keys.)
// T: the most rows of a sequence; `tokens` of them in all; `joined`: partial results also of a single chunk.
TokenPlan token_plan(int64_t S, int64_t T, int64_t tokens, int64_t max_len, int64_t Hkv, int64_t g, int d, bool joined)
{
    TokenPlan p{};
    p.wide = T * g > 8 ? 2 : 1;
    p.tiles = static_cast<int>((T * g + 8 * p.wide - 1) / (8 * p.wide));
    const int64_t units = S * Hkv * p.tiles;
    const int64_t at_once = static_cast<int64_t>(current_sm_count() > 0 ? current_sm_count() : 1) * Shape<128, 1>::kResident;
    // Several sequences differ in length, and blocks without keys leave the last wave uneven: shorter chunks where there are few
    // waves (8 sequences of up to 18432 tokens: 34 us, 39 otherwise; 16: 52, 57; 16 of four tokens each: 66, 69; 64, with
    // ten waves: the same).
    auto fit_of = [&](int64_t least) {  // chunks of a unit, at least `least`
        if (S > 1 && least * units < 4 * at_once) least *= 2;
        return (least * units + at_once - 1) / at_once * at_once / units;
    };
    const int64_t fit = fit_of((max_len + kMaxChunk - 1) / kMaxChunk);
    int64_t chunk = fit > 0 ? (max_len + fit - 1) / fit : 0;
    chunk = (chunk + kRound - 1) / kRound * kRound;
    if (chunk > kMaxChunk) chunk = kMaxChunk;
    if (chunk < kRound) chunk = kRound;
    p.chunk = static_cast<int>(chunk);
    p.chunks = static_cast<int>(max_len > 0 ? (max_len + chunk - 1) / chunk : 1);
    // A sequence much shorter than max_len is cut as if it were the longest (one of 1000 tokens, max_len 131072: 7.1 us, 13.4
    // in chunks for the longest; eight: 14.0, 18.7).
    p.share = static_cast<int>(fit_of(1) < p.chunks ? fit_of(1) : p.chunks);
    p.lse = kHeaderBytes;
    p.o = p.total = kHeaderBytes;
    if (p.chunks > 1 || joined) {
        const size_t parts = static_cast<size_t>(tokens) * Hkv * g * p.chunks;
        p.o = p.lse + align_up(parts * sizeof(float), 256);
        p.total = p.o + parts * d * sizeof(float);
    }
    return p;
}

template <int D, bool TAIL>
bool launch_pages(const CUtensorMap &tm_k, const CUtensorMap &tm_v, const TokenArgs &a, const TokenPlan &plan, cudaStream_t stream)
{
    dim3 grid(static_cast<unsigned>(a.chunks), static_cast<unsigned>(a.Hkv * a.tiles), static_cast<unsigned>(a.S));
    // The kernel's limit is the most that any call takes: it belongs to the function, and another thread's call may set it between
    // this one's setting and its launch.
    auto launch = [&](auto kern, int smem, int limit) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, limit) != cudaSuccess) return false;
        return launch_programmatic(kern, grid, kThreads, smem, stream, tm_k, tm_v, a) == cudaSuccess;
    };
    const int64_t blocks = static_cast<int64_t>(a.chunks) * a.Hkv * a.tiles * a.S;
    const int64_t at_once = static_cast<int64_t>(current_sm_count()) * Shape<D, 1>::kResident;
    if (a.chunks > 1 && a.S > 1 && a.S <= kMaxPacked && blocks > kPackedWaves * at_once && blocks <= 1 << 30) {
        grid = dim3(static_cast<unsigned>(at_once));
        constexpr int kInt = sizeof(int);
        const int more = (a.S + kWarps + 2) * kInt;
        constexpr int kMost = (kMaxPacked + kWarps + 2) * kInt;
        return plan.wide == 1
                   ? launch(token_attention_kernel<D, 1, TAIL, true>, Shape<D, 1>::kSmem + more, Shape<D, 1>::kSmem + kMost)
                   : launch(token_attention_kernel<D, 2, TAIL, true>, Shape<D, 2>::kSmem + more, Shape<D, 2>::kSmem + kMost);
    }
    return plan.wide == 1 ? launch(token_attention_kernel<D, 1, TAIL, false>, Shape<D, 1>::kSmem, Shape<D, 1>::kSmem)
                          : launch(token_attention_kernel<D, 2, TAIL, false>, Shape<D, 2>::kSmem, Shape<D, 2>::kSmem);
}

// The pages' part, then the join of `joined` rows as its programmatic dependent.
template <bool TAIL>
blink_status launch_token(const TokenArgs &a, const TokenPlan &plan, int page_tokens, int d, int64_t joined, cudaStream_t stream)
{
    // A page is rows of d bytes, head by head; a step's 16 keys are rows of one page.
    CUtensorMap tm_k, tm_v;
    const uint64_t page_rows = static_cast<uint64_t>(a.Hkv) * page_tokens;
    if (!encode_tmap_3d_bytes(&tm_k, a.c.k, d, page_rows, a.c.n_pages, d, a.c.page_stride, d, kStep, 1, d) ||
        !encode_tmap_3d_bytes(&tm_v, a.c.v, d, page_rows, a.c.n_pages, d, a.c.page_stride, d, kStep, 1, d))
        return BLINK_CUDA_ERROR;
    if (!(d == 128 ? launch_pages<128, TAIL>(tm_k, tm_v, a, plan, stream) : launch_pages<64, TAIL>(tm_k, tm_v, a, plan, stream)))
        return BLINK_CUDA_ERROR;
    if (!TAIL && a.chunks == 1) return BLINK_OK;
    int warps = (a.chunks + kJoinBatch - 1) / kJoinBatch;
    if (TAIL && warps < (a.tail.max_tail + kJoinBatch - 1) / kJoinBatch) warps = (a.tail.max_tail + kJoinBatch - 1) / kJoinBatch;
    const unsigned threads = static_cast<unsigned>(warps < kJoinWarps ? warps : kJoinWarps) * 32;
    const dim3 rows(static_cast<unsigned>(joined));
    const cudaError_t e = d == 128 ? launch_programmatic(token_join_kernel<128, TAIL>, rows, threads, 0, stream, a)
                                   : launch_programmatic(token_join_kernel<64, TAIL>, rows, threads, 0, stream, a);
    if (e == cudaSuccess) return BLINK_OK;
    cudaMemsetAsync(a.taken, 0, sizeof(int), stream);  // as the join would have
    return BLINK_CUDA_ERROR;
}

bool token_sizes(int32_t S, int32_t T, int32_t max_len, int32_t Hq, int32_t Hkv, int32_t d, blink_status &st)
{
    st = BLINK_INVALID_ARG;
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || (d != 64 && d != 128) || T < 1 || max_len < 0) return false;
    st = BLINK_OUT_OF_RANGE;
    if (S < 1 || S > BLINK_MAX_PLAN_SEQUENCES || T > BLINK_MAX_PAGED_TOKENS || max_len > BLINK_MAX_INPUT_TOKENS) return false;
    if (Hkv > BLINK_MAX_PAGED_HEADS || Hq / Hkv > 128) return false;
    if (static_cast<int64_t>(Hkv) * ((static_cast<int64_t>(T) * (Hq / Hkv) + 15) / 16) > 65535) return false;
    st = BLINK_OK;
    return true;
}

struct TailSizes {
    int most, longest;  // rows of a request, tokens of a prefix
};

TailSizes tail_sizes(const int32_t *h_req_rows, const int32_t *h_len, int n_req)
{
    TailSizes z{0, 0};
    for (int r = 0; r < n_req; ++r) {
        if (h_req_rows[r + 1] - h_req_rows[r] > z.most) z.most = h_req_rows[r + 1] - h_req_rows[r];
        if (h_len[r] > z.longest) z.longest = h_len[r];
    }
    return z;
}

}  // namespace

bool few_tail_rows(const int32_t *h_req_rows, int n_req, int g)
{
    int64_t most = 0;
    for (int r = 0; r < n_req; ++r) most = h_req_rows[r + 1] - h_req_rows[r] > most ? h_req_rows[r + 1] - h_req_rows[r] : most;
    return most * g <= kFewRows;
}

size_t few_tail_workspace(const int32_t *h_req_rows, const int32_t *h_len, int n_req, int Hkv, int g, int d)
{
    const TailSizes z = tail_sizes(h_req_rows, h_len, n_req);
    return token_plan(n_req, z.most, h_req_rows[n_req], z.longest, Hkv, g, d, true).total;
}

blink_status few_tail_attention(const PagedCache &c, int page_tokens, const uint16_t *q, const int32_t *d_page_table,
                                int64_t table_stride, int table_width, const uint16_t *k_tail, const uint16_t *v_tail,
                                const int32_t *d_cu, const int32_t *d_seq_start, int B, int rows, int n_req,
                                const int32_t *h_req_rows, const int32_t *h_len, int max_tail, int Hq, int Hkv, int d, float scale,
                                uint16_t *out, float *lse, void *d_ws, cudaStream_t stream)
{
    const TailSizes z = tail_sizes(h_req_rows, h_len, n_req);
    const TokenPlan plan = token_plan(n_req, z.most, rows, z.longest, Hkv, Hq / Hkv, d, true);
    TokenArgs a{};
    auto *ws = static_cast<uint8_t *>(d_ws);
    a.c = c;
    a.q = q;
    a.table = d_page_table;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.max_len = z.longest;
    a.S = n_req;
    a.T = 1;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.g = Hq / Hkv;
    a.tiles = plan.tiles;
    a.chunk = plan.chunk;
    a.chunks = plan.chunks;
    a.share = plan.share;
    a.one_share = static_cast<uint32_t>(((1ull << 32) + plan.share - 1) / plan.share);
    a.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(d))) * kLog2e;
    a.out = out;
    a.lse = lse;
    a.part_lse = reinterpret_cast<float *>(ws + plan.lse);
    a.part_o = reinterpret_cast<float *>(ws + plan.o);
    a.err = &static_cast<WorkspaceHeader *>(d_ws)->error;
    a.taken = &static_cast<WorkspaceHeader *>(d_ws)->reserved[0];
    for (int r = 0; r < n_req; ++r) a.tail.row[r] = h_req_rows[r], a.tail.len[r] = h_len[r];
    a.tail.row[n_req] = h_req_rows[n_req];
    a.tail.n_req = n_req;
    a.tail.rows = rows;
    a.tail.B = B;
    a.tail.max_tail = max_tail;
    a.tail.k = k_tail;
    a.tail.v = v_tail;
    a.tail.cu = d_cu;
    a.tail.seq_start = d_seq_start;
    return launch_token<true>(a, plan, page_tokens, d, static_cast<int64_t>(rows) * Hq, stream);
}

}  // namespace blink

extern "C" size_t blink_paged_token_attention_workspace(int32_t S, int32_t T, int32_t max_len, int32_t Hq, int32_t Hkv, int32_t d)
{
    using namespace blink;
    blink_status st;
    if (!token_sizes(S, T, max_len, Hq, Hkv, d, st)) return kHeaderBytes;
    return token_plan(S, T, static_cast<int64_t>(S) * T, max_len, Hkv, Hq / Hkv, d, false).total;
}

extern "C" blink_status blink_paged_token_attention(
    const blink_bf16 *q, const uint8_t *k_codes, const uint8_t *v_codes, const uint8_t *k_scale, const uint8_t *v_scale,
    int64_t page_stride, int64_t scale_stride, int32_t n_pages, int32_t page_tokens, const int32_t *d_page_table,
    int64_t table_stride, int32_t table_width, const int32_t *d_len, int32_t S, int32_t T, int32_t max_len, int32_t Hq,
    int32_t Hkv, int32_t d, float scale, blink_bf16 *out, float *lse, void *d_ws, size_t ws_bytes, cudaStream_t stream)
{
    using namespace blink;
    TokenArgs a{};
    blink_status st = check_cache(a.c, k_codes, v_codes, k_scale, v_scale, page_stride, scale_stride, n_pages, page_tokens, Hkv, d);
    if (st != BLINK_OK) return st;
    if (!token_sizes(S, T, max_len, Hq, Hkv, d, st)) return st;
    if (!q || !d_page_table || !d_len || !out || !d_ws) return BLINK_INVALID_ARG;
    if (table_width < 1 || (S > 1 && table_stride < table_width) || std::isnan(scale) || std::isinf(scale)) return BLINK_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(d_ws)) return BLINK_INVALID_ARG;
    const TokenPlan plan = token_plan(S, T, static_cast<int64_t>(S) * T, max_len, Hkv, Hq / Hkv, d, false);
    const int64_t joined = static_cast<int64_t>(S) * T * Hq;  // rows of the second launch
    if (joined > 0x7FFFFFFF) return BLINK_OUT_OF_RANGE;
    if (ws_bytes < plan.total) return BLINK_WORKSPACE_TOO_SMALL;
    auto *ws = static_cast<uint8_t *>(d_ws);
    a.q = q;
    a.table = d_page_table;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.len = d_len;
    a.max_len = max_len;
    a.S = S;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.g = Hq / Hkv;
    a.tiles = plan.tiles;
    a.chunk = plan.chunk;
    a.chunks = plan.chunks;
    a.share = plan.share;
    a.one_share = static_cast<uint32_t>(((1ull << 32) + plan.share - 1) / plan.share);
    a.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(d))) * kLog2e;
    a.out = out;
    a.lse = lse;
    a.part_lse = reinterpret_cast<float *>(ws + plan.lse);
    a.part_o = reinterpret_cast<float *>(ws + plan.o);
    a.err = &static_cast<WorkspaceHeader *>(d_ws)->error;
    a.taken = &static_cast<WorkspaceHeader *>(d_ws)->reserved[0];
    return launch_token<false>(a, plan, page_tokens, d, joined, stream);
}
