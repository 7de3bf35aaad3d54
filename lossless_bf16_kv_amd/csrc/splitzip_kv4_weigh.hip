// splitzip_kv4_weigh.hip -- accumulated attention weights of the 4-bit KV cache's tokens:
//
//   w_j += sum over the rows i (queries and heads of the group) that see j of 2^(x_ij - lse_i)
//
// with x and lse as powers of two.  The rows' sums are known, so each token's sum stands alone:
// a wave owns its tokens, adds over all rows in 32 bits in a fixed order, and writes each weight
// once; no atomics.  Scores are products with rows as the result's rows, so a lane holds four
// rows of one token and a sum over rows stays in the lane but for one exchange at the end.
//
// step_kernel: up to 16 rows a sequence and KV head.  The rows' operands stay in registers while
// a wave runs over groups of 16 tokens; HBM bounds it (K's 68 bytes a token at D = 128, and 8 of
// weights).  rows_kernel: more rows.  A wave keeps the operands of its groups and the workgroup
// runs over the rows through LDS; the matrix units and the exponentials bound it.
#include "splitzip_kv4_tiles.h"

namespace sz {
namespace kv4 {
namespace {

constexpr int kLanes = 256;

// Adds the lane's sum for token 16 g + r of a page to its weight.
__device__ __forceinline__ void add_weight(const Cache &c, int page, int head, int g, int len, int lane, float sum)
{
    sum = quad_sum(sum);
    if (page < 0 || lane >= 16 || 16 * g + lane >= len)
        return;
    float *w = c.weights + group_first(c, page, head, g) + lane;
    *w += sum;
}

template <int D, int T>
__global__ __launch_bounds__(kLanes, 2) void step_kernel(AttendArgs a)
{
    constexpr int kHalves = T == SPLITZIP_KV4_FP16 ? 2 : 1;
    constexpr int kSteps = D / 32;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, quad = lane >> 4;
    uint32_t b = blockIdx.x;
    const int split = b % a.splits;
    b /= a.splits;
    const int head = b % a.c.heads, s = b / a.c.heads;
    const Seq q = wave_sequence(a.c, a.b, s);
    const int rows = q.n * a.group;
    const Mask mask = {a.window, a.sinks};
    const int base = q.len - q.n;
    if (rows == 0)
        return;
    // groups that some row sees; each wave keeps its own over all rows, 16 of which go at a time
    const Groups groups(base, q.len - 1, a.window, a.sinks);
    const int per = (groups.count + a.splits - 1) / a.splits;
    const int first = min(groups.count, split * per), last = min(groups.count, first + per);
    for (int row0 = 0; row0 < rows; row0 += 16) {
        const int row = min(row0 + r, rows - 1);
        const int64_t q_row = q.row0 + row / a.group;
        const int q_head = head * a.group + row % a.group;
        const int q_lo = base + row0 / a.group, q_hi = base + min(row0 + 15, rows - 1) / a.group;
        bf16x8 qf[kHalves][kSteps];
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            const int64_t p = q_row * a.q_token + q_head * a.q_head + quad * (D / 4) + 8 * st;
            qf[0][st] = q_frag<T, 0>(a.q, p, a.wide);
            if constexpr (kHalves == 2)
                qf[1][st] = q_frag<T, 1>(a.q, p, a.wide);
        }
        // rows 4 quad + i of the result
        int query[4];
        float lse[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int y = row0 + 4 * quad + i;
            query[i] = base + min(y, rows - 1) / a.group;
            const float t = y < rows ? a.lse_in[(q.row0 + y / a.group) * (int64_t)a.q_heads + head * a.group + y % a.group]
                                     : -INFINITY;
            lse[i] = t == -INFINITY ? INFINITY : t * kLog2e;      // adds 2^-infinity
        }
        for (int v = first + wave; v < last; v += 4) {
            const int g = groups.at(v);
            const int page = page_of(a.c, a.b, s, 16 * g);
            const KRaw<D> k = load_k<D>(a.c, page, head, g, lane);
            f32x4 x = {0, 0, 0, 0};
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const bf16x8 f = k_frag<D>(k, st);
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                    x = mfma(qf[h][st], f, x);
            }
            const bool whole = mask.all(g, q_lo, q_hi);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = exp2_fast(fmaf(x[i], a.scale2, -lse[i]));
                const bool in = lse[i] != INFINITY && (whole || mask.sees(query[i], 16 * g + r));
                sum += in ? p : 0.0f;
            }
            add_weight(a.c, page, head, g, q.len, lane, sum);
        }
    }
}

// NG groups of 16 tokens a wave; rows pass 32 at a time.
template <int D, int T, int NG>
__global__ __launch_bounds__(kLanes, D == 256 && NG == 4 ? 1 : 2) void rows_kernel(AttendArgs a)
{
    constexpr int kHalves = T == SPLITZIP_KV4_FP16 ? 2 : 1;
    constexpr int kSteps = D / 32;
    constexpr int kBlock = 32;
    __shared__ uint4 sh_q[2][kHalves][kBlock / 16][kSteps][64];
    __shared__ float sh_lse[2][kBlock];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, quad = lane >> 4;
    uint32_t b = blockIdx.x;
    const int split = b % a.splits;
    b /= a.splits;
    const int head = b % a.c.heads, s = b / a.c.heads;
    const Seq q = wave_sequence(a.c, a.b, s);
    const int rows = q.n * a.group, base = q.len - q.n;
    const Mask mask = {a.window, a.sinks};
    const int all = rows > 0 ? (q.len + 15) >> 4 : 0;             // groups of the sequence

    for (int g0 = split * 4 * NG; g0 < all; g0 += a.splits * 4 * NG) {
        const int j0 = 16 * g0, j1 = min(16 * (g0 + 4 * NG), q.len) - 1;     // the workgroup's tokens
        // rows that see one of them: queries from j0, up to the window's end unless always visible
        const int64_t past = a.window > 0 && j0 >= a.sinks ? (int64_t)j1 + a.window - 1 : (int64_t)q.len;
        const int lo = max(0, j0 - base), hi = (int)min((int64_t)q.n - 1, past - base);
        if (lo > hi)
            continue;
        const int row_end = (hi + 1) * a.group;
        int page[NG], group[NG];
        bf16x8 kf[NG][kSteps];
        float sum[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            group[n] = g0 + wave * NG + n;
            page[n] = group[n] < all ? page_of(a.c, a.b, s, 16 * group[n]) : -1;
            const KRaw<D> k = load_k<D>(a.c, page[n], head, group[n], lane);
#pragma unroll
            for (int st = 0; st < kSteps; ++st)
                kf[n][st] = k_frag<D>(k, st);
            sum[n] = 0.0f;
        }
        // 32 rows to LDS as operands: piece p of a row is channels 8 p .. + 7
        auto stage = [&](int row0, int buf) {
#pragma unroll
            for (int i = threadIdx.x; i < kBlock * (D / 8); i += kLanes) {
                const int y = i % kBlock, p = i / kBlock;
                const int row = min(row0 + y, row_end - 1);
                const int64_t at = (q.row0 + row / a.group) * a.q_token + (head * a.group + row % a.group) * a.q_head + 8 * p;
                const int to = (p / kSteps) * 16 + y % 16, st = p % kSteps;
                sh_q[buf][0][y / 16][st][to] = __builtin_bit_cast(uint4, q_frag<T, 0>(a.q, at, a.wide));
                if constexpr (kHalves == 2)
                    sh_q[buf][1][y / 16][st][to] = __builtin_bit_cast(uint4, q_frag<T, 1>(a.q, at, a.wide));
            }
            if (threadIdx.x < kBlock) {
                const int row = row0 + threadIdx.x;
                const float t = row < row_end ? a.lse_in[(q.row0 + row / a.group) * (int64_t)a.q_heads + head * a.group + row % a.group]
                                              : -INFINITY;
                sh_lse[buf][threadIdx.x] = t == -INFINITY ? INFINITY : t * kLog2e;
            }
        };
        int buf = 0;
        stage(lo * a.group, 0);
        __syncthreads();
        for (int row0 = lo * a.group; row0 < row_end; row0 += kBlock, buf ^= 1) {
            if (row0 + kBlock < row_end)
                stage(row0 + kBlock, buf ^ 1);
#pragma unroll
            for (int half = 0; half < kBlock / 16; ++half) {
                const int y0 = row0 + 16 * half;
                if (y0 >= row_end)
                    break;
                const int q_lo = base + y0 / a.group, q_hi = base + min(y0 + 15, row_end - 1) / a.group;
                bf16x8 qf[kHalves][kSteps];
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
#pragma unroll
                    for (int st = 0; st < kSteps; ++st)
                        qf[h][st] = __builtin_bit_cast(bf16x8, sh_q[buf][h][half][st][lane]);
                float lse[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    lse[i] = sh_lse[buf][16 * half + 4 * quad + i];
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    f32x4 x = {0, 0, 0, 0};
#pragma unroll
                    for (int st = 0; st < kSteps; ++st)
#pragma unroll
                        for (int h = 0; h < kHalves; ++h)
                            x = mfma(qf[h][st], kf[n][st], x);
                    if (mask.all(group[n], q_lo, q_hi) && __all(lse[0] != INFINITY && lse[1] != INFINITY &&
                                                               lse[2] != INFINITY && lse[3] != INFINITY)) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sum[n] += exp2_fast(fmaf(x[i], a.scale2, -lse[i]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int query = base + min(y0 + 4 * quad + i, row_end - 1) / a.group;
                            const float p = exp2_fast(fmaf(x[i], a.scale2, -lse[i]));
                            sum[n] += lse[i] != INFINITY && mask.sees(query, 16 * group[n] + r) ? p : 0.0f;
                        }
                    }
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int n = 0; n < NG; ++n)
            add_weight(a.c, page[n], head, group[n], q.len, lane, sum[n]);
    }
}

template <int D, int T>
void weigh_dt(AttendArgs a, int max_q, int max_len, hipStream_t s)
{
    const int64_t pairs = (int64_t)a.b.n_seqs * a.c.heads;
    const int64_t groups = max_len / 16 + 1;
    auto splits = [&](int64_t unit, int64_t most) {
        const int64_t n = (groups + unit - 1) / unit;
        return (int32_t)(n < most ? n : most);
    };
    if ((int64_t)max_q * a.group <= 16) {
        a.splits = splits(16, 1 << 20);
        step_kernel<D, T><<<(unsigned)(pairs * a.splits), kLanes, 0, s>>>(a);
    } else if (pairs * groups >= 16 * 512) {
        a.splits = splits(16, 1 << 20);
        rows_kernel<D, T, 4><<<(unsigned)(pairs * a.splits), kLanes, 0, s>>>(a);
    } else {
        a.splits = splits(4, 1 << 20);
        rows_kernel<D, T, 1><<<(unsigned)(pairs * a.splits), kLanes, 0, s>>>(a);
    }
}

}  // namespace

void launch_weigh(const AttendArgs &a, int head_dim, int dtype, int max_q, int max_len, hipStream_t s)
{
    const bool b = dtype == SPLITZIP_KV4_BF16;
    if (head_dim == 64)
        b ? weigh_dt<64, SPLITZIP_KV4_BF16>(a, max_q, max_len, s) : weigh_dt<64, SPLITZIP_KV4_FP16>(a, max_q, max_len, s);
    else if (head_dim == 128)
        b ? weigh_dt<128, SPLITZIP_KV4_BF16>(a, max_q, max_len, s) : weigh_dt<128, SPLITZIP_KV4_FP16>(a, max_q, max_len, s);
    else
        b ? weigh_dt<256, SPLITZIP_KV4_BF16>(a, max_q, max_len, s) : weigh_dt<256, SPLITZIP_KV4_FP16>(a, max_q, max_len, s);
}

}  // namespace kv4
}  // namespace sz
