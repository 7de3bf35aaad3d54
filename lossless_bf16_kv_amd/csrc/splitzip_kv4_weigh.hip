// splitzip_kv4_weigh.hip -- accumulated attention weights of the 4-bit KV cache's tokens:
//
//   w_j += sum over the rows i (queries and heads of the group) that see j of 2^(x_ij - lse_i)
//
// with x and lse as powers of two.  The rows' sums are known, so each token's sum stands alone:
// a wave owns its tokens of a sequence, adds over the rows in 32 bits in a fixed order, and then adds to
// each weight by one atomic (step_kernel: one for every 16 rows, in their order).  Atomics make the sum
// right where sequences share pages, in an order that is not fixed there; elsewhere a weight has one
// adder and results do not depend on timing.  They take the time that plain stores took.  Scores are products with rows as the result's rows, so a lane holds four
// rows of one token and a sum over rows stays in the lane but for one exchange at the end.
//
// step_kernel: up to 16 rows a sequence and KV head.  The rows' operands stay in registers while
// a wave runs over 64 tokens a turn, with the codes of the next two turns on their way to
// LDS.  K's 68 bytes a token at D = 128 and 8 of weights: 64 steps of 128 .. 8192 tokens move 200 MB in
// 52 us (3.8 TB/s; 57 us with one turn ahead in registers, 74 us with 16 tokens a turn), of which the
// kernel takes 47: short sequences end before their ring is full.
//
// rows_kernel: more rows.  A wave keeps the operands of 64 tokens (32 at D = 256) and the workgroup runs
// over the rows through LDS.  1000 queries of 32 heads on two prompts of 16000 tokens: 259 GFLOP in
// 328 us, 0.79 PFLOP/s.  Neither unit bounds it (matrix 33 %, vector 53 % busy): a wave spends a quarter of
// its cycles at waits and barriers and as many waiting to issue.  Rows permuted among the LDS banks, no division in the loop, masks from LDS and parts that
// see nothing left out took it there from 572 us.
#include "splitzip_kv4_tiles.h"

namespace sz {
namespace kv4 {
namespace {

constexpr int kLanes = kWeighThreads;
// Query and head of a row, moved on without a division.
struct RowAt {
    int query, head;
    __device__ RowAt(int row, int group) : query(row / group), head(row % group) {}
    __device__ __forceinline__ bool move(int queries, int heads, int group)      // heads < group
    {
        head += heads;
        const bool over = head >= group;
        head -= over ? group : 0;
        query += queries + over;
        return over;
    }
};

template <int D>
constexpr int kWeighTokens = weigh_tokens(D);

// One turn of a wave in LDS, 64 tokens: K's codes of four groups (8 D bytes each: D >= 128 16 bytes a
// lane in lane order, D = 256 two of them; D = 64 as in the cache) and their scales (D = 64 as in the
// cache, else 4 bytes a token, D = 256 two such runs).
template <int D>
struct Turn {
    static constexpr int kCodes = 8 * D, kScales = 4 * kCodes, kBytes = kScales + 2 * D;
    static constexpr int kLoads = D == 64 ? 3 : D == 128 ? 5 : 10;       // instructions
};

// Groups g on pages `page` (-1: page 0's tokens) to a slot; t: the lane's token 16 (lane / 16) +
// lane % 16 of the turn, in the cache.
template <int D>
__device__ __forceinline__ void send_turn(const Cache &c, const int (&page)[4], int head, const int (&g)[4], int64_t t,
                                          uint32_t lane, uint8_t *slot)
{
    typedef Turn<D> L;
    const uint32_t r = lane & 15, quad = lane >> 4;
    if constexpr (D == 64) {
        int64_t first[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            first[e] = group_first(c, page[e], head, g[e]);
#pragma unroll
        for (int i = 0; i < 2; ++i)      // lanes 32 .. 63 take the second group
            to_lds16(c.k_codes + (lane < 32 ? first[2 * i] : first[2 * i + 1]) * 32 + 16 * (lane & 31), slot + 1024 * i);
        const int64_t own = lane < 8 ? first[0] : lane < 16 ? first[1] : lane < 24 ? first[2] : first[3];
        if (lane < 32)
            to_lds4(c.k_scales + own * 2 + 4 * (lane & 7), slot + L::kScales);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < D / 128; ++i)
                to_lds16(lane_at(c.k_codes + group_first(c, page[e], head, g[e]) * (D / 2), r * (D / 2) + quad * (D / 8) + 16 * i),
                         slot + e * L::kCodes + 1024 * i);
#pragma unroll
        for (int i = 0; i < D / 128; ++i)
            to_lds4(c.k_scales + t * (D / 32) + 4 * i, slot + L::kScales + 256 * i);
    }
}

// A slot's turn to registers, once its loads are done: all but the Younger instructions behind them.
template <int D, int Younger>
__device__ __forceinline__ void take_turn(const uint8_t *slot, uint32_t lane, KRaw<D> (&k)[4])
{
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const uint32_t r = lane & 15, quad = lane >> 4;
    const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr)slot;
    if constexpr (D == 64) {
        const uint32_t at = base + r * 32 + quad * 8, ks = base + r * 2 + (quad >> 1);
        u32x2 a, b, c, d;
        asm volatile("s_waitcnt vmcnt(%10)\n"
                     "ds_read_b64 %0, %8\n"
                     "ds_read_b64 %1, %8 offset:0x200\n"
                     "ds_read_b64 %2, %8 offset:0x400\n"
                     "ds_read_b64 %3, %8 offset:0x600\n"
                     "ds_read_u8 %4, %9 offset:0x800\n"
                     "ds_read_u8 %5, %9 offset:0x820\n"
                     "ds_read_u8 %6, %9 offset:0x840\n"
                     "ds_read_u8 %7, %9 offset:0x860\n"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d), "=&v"(k[0].s), "=&v"(k[1].s), "=&v"(k[2].s), "=&v"(k[3].s)
                     : "v"(at), "v"(ks), "n"(Younger)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            k[0].w[i] = a[i]; k[1].w[i] = b[i]; k[2].w[i] = c[i]; k[3].w[i] = d[i];
        }
    } else if constexpr (D == 128) {
        const uint32_t at = base + 16 * lane, ks = base + r * 4 + quad;
        u32x4 a, b, c, d;
        asm volatile("s_waitcnt vmcnt(%10)\n"
                     "ds_read_b128 %0, %8\n"
                     "ds_read_b128 %1, %8 offset:0x400\n"
                     "ds_read_b128 %2, %8 offset:0x800\n"
                     "ds_read_b128 %3, %8 offset:0xc00\n"
                     "ds_read_u8 %4, %9 offset:0x1000\n"
                     "ds_read_u8 %5, %9 offset:0x1040\n"
                     "ds_read_u8 %6, %9 offset:0x1080\n"
                     "ds_read_u8 %7, %9 offset:0x10c0\n"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d), "=&v"(k[0].s), "=&v"(k[1].s), "=&v"(k[2].s), "=&v"(k[3].s)
                     : "v"(at), "v"(ks), "n"(Younger)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k[0].w[i] = a[i]; k[1].w[i] = b[i]; k[2].w[i] = c[i]; k[3].w[i] = d[i];
        }
    } else {
        const uint32_t at = base + 16 * lane, ks = base + r * 4 + (quad >> 1) * 256 + (quad & 1) * 2;
        u32x4 a, b, c, d, e, f, g, h;
        asm volatile("s_waitcnt vmcnt(%14)\n"
                     "ds_read_b128 %0, %12\n"
                     "ds_read_b128 %1, %12 offset:0x400\n"
                     "ds_read_b128 %2, %12 offset:0x800\n"
                     "ds_read_b128 %3, %12 offset:0xc00\n"
                     "ds_read_b128 %4, %12 offset:0x1000\n"
                     "ds_read_b128 %5, %12 offset:0x1400\n"
                     "ds_read_b128 %6, %12 offset:0x1800\n"
                     "ds_read_b128 %7, %12 offset:0x1c00\n"
                     "ds_read_u16 %8, %13 offset:0x2000\n"
                     "ds_read_u16 %9, %13 offset:0x2040\n"
                     "ds_read_u16 %10, %13 offset:0x2080\n"
                     "ds_read_u16 %11, %13 offset:0x20c0\n"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d), "=&v"(e), "=&v"(f), "=&v"(g), "=&v"(h), "=&v"(k[0].s),
                       "=&v"(k[1].s), "=&v"(k[2].s), "=&v"(k[3].s)
                     : "v"(at), "v"(ks), "n"(Younger)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k[0].w[i] = a[i]; k[0].w[4 + i] = b[i]; k[1].w[i] = c[i]; k[1].w[4 + i] = d[i];
            k[2].w[i] = e[i]; k[2].w[4 + i] = f[i]; k[3].w[i] = g[i]; k[3].w[4 + i] = h[i];
        }
    }
}

template <int D, int T>
__global__ __launch_bounds__(kLanes, 2) void step_kernel(AttendArgs a)
{
    constexpr int kHalves = T == SPLITZIP_KV4_FP16 ? 2 : 1;
    constexpr int kSteps = D / 32;
    __shared__ __align__(16) uint8_t sh_turn[4][2][Turn<D>::kBytes];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, quad = lane >> 4;
    uint32_t b = blockIdx.x;
    const int head = b % a.c.heads;          // fastest: the XCDs get equal shares, and a head's rows meet in one L2
    b /= a.c.heads;
    const int s = b % a.b.n_seqs, split = b / a.b.n_seqs;
    const Seq q = wave_sequence(a.c, a.b, s);
    const int rows = q.n * a.group;
    const Mask mask = {a.window, a.sinks};
    const int base = q.len - q.n;
    if (rows == 0 || rows > a.step_rows)
        return;
    // groups that some row sees; each wave keeps its own over all rows, 16 of which go at a time
    const Groups groups(base, q.len - 1, a.window, a.sinks);
    const int per = ((groups.count + a.splits - 1) / a.splits + 15) & ~15;
    const int first = min((int64_t)groups.count, (int64_t)split * per), last = min(groups.count, first + per);
    const int turns = (last - first - 4 * wave + 15) >> 4;       // of this wave: 4 groups of every 16
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
        const bool every = __all(lse[0] != INFINITY && lse[1] != INFINITY && lse[2] != INFINITY && lse[3] != INFINITY);

        int list = -1, from = -16;       // pages of turns from .. + 15: lane 4 i + e has group e of turn i
        auto group = [&](int i, int e) {
            const int v = first + 16 * i + 4 * wave + e;
            return v < last ? groups.at(v) : -1;
        };
        // returns where the weight of the lane's token is, null: no token
        auto send = [&](int i) {
            if (i >= from + 16) {
                from = i;
                const int64_t v = first + 16 * (int64_t)(i + quad * 4 + r / 4) + 4 * wave + r % 4;
                list = v < last ? page_of(a.c, a.b, s, 16 * groups.at((int)v)) : -1;
            }
            int page[4], g[4], mine = -1, mine_g = -1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                page[e] = __builtin_amdgcn_readlane(list, 4 * (i - from) + e);
                g[e] = group(i, e);
                mine = quad == e ? page[e] : mine;
                mine_g = quad == e ? g[e] : mine_g;
            }
            const int64_t t = group_first(a.c, mine, head, mine_g) + r;
            send_turn<D>(a.c, page, head, g, t, lane, sh_turn[wave][i & 1]);
            return mine < 0 || 16 * mine_g + r >= q.len ? nullptr : a.c.weights + t;
        };
        float *at0 = nullptr, *at1 = nullptr;
        if (turns > 0)
            at0 = send(0);
        if (turns > 1)
            at1 = send(1);
        for (int i = 0; i < turns; ++i) {
            KRaw<D> k[4];
            if (i + 1 < turns)
                take_turn<D, Turn<D>::kLoads>(sh_turn[wave][i & 1], lane, k);
            else
                take_turn<D, 0>(sh_turn[wave][i & 1], lane, k);
            float *const at = at0;
            at0 = at1;
            if (i + 2 < turns)
                at1 = send(i + 2);
            float mine = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f32x4 x = {0, 0, 0, 0};
#pragma unroll
                for (int st = 0; st < kSteps; ++st) {
                    const bf16x8 f = k_frag<D>(k[e], st);
#pragma unroll
                    for (int h = 0; h < kHalves; ++h)
                        x = mfma(qf[h][st], f, x);
                }
                float sum = 0.0f;
                const int g = group(i, e);
                if (every && mask.all(g, q_lo, q_hi)) {
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        sum += exp2_fast(fmaf(x[n], a.scale2, -lse[n]));
                } else {
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float p = exp2_fast(fmaf(x[n], a.scale2, -lse[n]));
                        sum += lse[n] != INFINITY && mask.sees(query[n], 16 * g + r) ? p : 0.0f;
                    }
                }
                sum = quad_sum(sum);
                mine = quad == e ? sum : mine;
            }
            if (at)
                unsafeAtomicAdd(at, mine);
        }
    }
}

// Rows pass kBlock at a time, through two buffers in LDS: the loads of a block are on their way while
// the block before is worked on.  Products have rows as their rows, so a sum over rows stays in a lane.
template <int D, int T>
__global__ __launch_bounds__(kLanes, 2) void rows_kernel(AttendArgs a)
{
    constexpr int kHalves = T == SPLITZIP_KV4_FP16 ? 2 : 1;
    constexpr int kSteps = D / 16;
    constexpr int kTiles = kWeighTokens<D> / 128;                // of 32 tokens, a wave
    constexpr int kBlock = D * kHalves > 128 ? 32 : 64;
    constexpr int kPieces = kBlock * (D / 8) / kLanes;           // 8 channels of a row, a lane
    __shared__ uint4 sh_q[2][kHalves][kBlock / 32][kSteps][64];
    __shared__ __align__(16) float sh_lse[2][kBlock / 32][2][16];    // in the order of a result's registers
    __shared__ __align__(16) int sh_query[2][kBlock / 32][2][16];
    __shared__ int sh_every[2][kBlock / 32];                     // all of these 32 rows count
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m32 = lane & 31, half = lane >> 5;
    uint32_t b = blockIdx.x;
    const int head = b % a.c.heads;          // fastest: the XCDs get equal shares, and a head's rows meet in one L2
    b /= a.c.heads;
    const int s = b % a.b.n_seqs, split = b / a.b.n_seqs;
    const Seq q = wave_sequence(a.c, a.b, s);
    const int rows = q.n * a.group, base = q.len - q.n;
    const Mask mask = {a.window, a.sinks};
    const int len = rows > a.step_rows ? q.len : 0;

    for (int64_t j00 = (int64_t)split * kWeighTokens<D>; j00 < len; j00 += (int64_t)a.row_splits * kWeighTokens<D>) {
        const int j0 = (int)j00, j1 = (int)min(j00 + kWeighTokens<D>, (int64_t)q.len) - 1;   // the workgroup's tokens
        // rows that see one of them: queries from j0, up to the window's end unless always visible
        const int64_t past = a.window > 0 && j0 >= a.sinks ? (int64_t)j1 + a.window - 1 : (int64_t)q.len;
        const int lo = max(0, j0 - base), hi = (int)min((int64_t)q.n - 1, past - base);
        if (lo > hi)
            continue;
        const int row_end = (hi + 1) * a.group;
        // this wave's tokens; behind the last the last one again, whose sums are dropped
        int page[kTiles], token[kTiles];
        bf16x8 kf[kTiles][kSteps];
        float sum[kTiles];
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            const int j = j0 + 32 * (wave * kTiles + n) + m32;
            token[n] = min(j, q.len - 1);
            page[n] = page_of(a.c, a.b, s, token[n]);
            const int64_t at = group_first(a.c, page[n], head, token[n] >> 4) + (token[n] & 15);
            uint32_t w[D / 16];
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const uint4 c = *(const uint4 *)(a.c.k_codes + at * (D / 2) + half * (D / 4) + 16 * i);
                w[4 * i] = c.x; w[4 * i + 1] = c.y; w[4 * i + 2] = c.z; w[4 * i + 3] = c.w;
            }
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const float ks = scale_of(a.c.k_scales[at * (D / 32) + half * (D / 64) + i]);
#pragma unroll
                for (int st = 4 * i; st < 4 * i + 4; ++st)
                    kf[n][st] = frag(dequant<0>(w[st], ks), dequant<1>(w[st], ks), dequant<2>(w[st], ks), dequant<3>(w[st], ks));
            }
            if (j >= q.len)
                page[n] = -1;
            sum[n] = 0.0f;
        }
        // Piece p of a row is channels 8 p .. + 7.  Lanes of one row write pieces 1 KiB apart, so rows are
        // permuted among the 16 banks of 16 bytes, differently for each piece.
        auto spread = [](int st, int part) { return (2 * st + part) & 15; };
        struct Rows {
            bf16x8 q[kPieces][kHalves];
            float lse;
            int query;           // its token; a row behind the last has none, -1
        } next;
        const int start = lo * a.group;
        const int by_q = kBlock / a.group, by_f = kBlock % a.group;     // a block's step
        const int64_t step = by_q * a.q_token + by_f * a.q_head, step_over = step + a.q_token - a.group * a.q_head;
        int at_head[kPieces];
        int64_t at[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const RowAt x(start + (i * kLanes + (int)threadIdx.x) / (D / 8), a.group);
            at_head[i] = x.head;
            at[i] = (q.row0 + x.query) * a.q_token + (head * a.group + x.head) * a.q_head + 8 * (threadIdx.x % (D / 8));
        }
        RowAt lse_at(start + threadIdx.x % kBlock, a.group);
        // each call is for the next block
        auto fetch = [&](int row0) {
            Rows x;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const bool in = row0 + (i * kLanes + (int)threadIdx.x) / (D / 8) < row_end;
                const int64_t p = in ? at[i] : q.row0 * a.q_token + head * a.group * a.q_head;
                x.q[i][0] = q_frag<T, 0>(a.q, p, a.wide);
                if constexpr (kHalves == 2)
                    x.q[i][1] = q_frag<T, 1>(a.q, p, a.wide);
                at_head[i] += by_f;
                const bool over = at_head[i] >= a.group;
                at_head[i] -= over ? a.group : 0;
                at[i] += over ? step_over : step;
            }
            x.lse = -INFINITY;
            x.query = -1;
            if (threadIdx.x < kBlock && row0 + (int)threadIdx.x < row_end) {
                x.query = base + lse_at.query;
                x.lse = a.lse_in[(q.row0 + lse_at.query) * (int64_t)a.q_heads + head * a.group + lse_at.head];
            }
            lse_at.move(by_q, by_f, a.group);
            return x;
        };
        auto put = [&](const Rows &x, int buf) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int y = (i * kLanes + threadIdx.x) / (D / 8), p = threadIdx.x % (D / 8);
                const int st = p % kSteps, to = p / kSteps * 32 + (y % 32 ^ spread(st, p / kSteps));
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                    sh_q[buf][h][y / 32][st][to] = __builtin_bit_cast(uint4, x.q[i][h]);
            }
            if (threadIdx.x < kBlock) {
                const int y = threadIdx.x % 32;
                const uint64_t some = __ballot(x.lse != -INFINITY);
                if (y == 0)
                    sh_every[buf][threadIdx.x / 32] = (uint32_t)(some >> (lane & 32)) == 0xffffffffu;
                const int to = (y >> 3) * 4 + (y & 3);
                sh_lse[buf][threadIdx.x / 32][(y >> 2) & 1][to] = x.lse == -INFINITY ? INFINITY : x.lse * kLog2e;
                sh_query[buf][threadIdx.x / 32][(y >> 2) & 1][to] = x.lse == -INFINITY ? -1 : x.query;
            }
        };
        next = fetch(start);
        put(next, 0);
        if (start + kBlock < row_end)
            next = fetch(start + kBlock);
        __syncthreads();
        int buf = 0;
        RowAt first(start, a.group), last(start + 31, a.group);         // of 32 rows
        const int by_q32 = 32 / a.group, by_f32 = 32 % a.group;
        for (int row0 = start; row0 < row_end; row0 += kBlock, buf ^= 1) {
            if (row0 + kBlock < row_end) {
                put(next, buf ^ 1);
                if (row0 + 2 * kBlock < row_end)
                    next = fetch(row0 + 2 * kBlock);
            }
#pragma unroll 1
            for (int part = 0; part < kBlock / 32; ++part) {
                const int y0 = row0 + 32 * part;
                if (y0 >= row_end)
                    break;
                const int q_lo = base + first.query, q_hi = base + min(last.query, hi);
                first.move(by_q32, by_f32, a.group);
                last.move(by_q32, by_f32, a.group);
                f32x16 x[kTiles];
#pragma unroll
                for (int n = 0; n < kTiles; ++n)
                    x[n] = f32x16{};
                if (16 * ((j0 >> 4) + 2 * wave * kTiles) > q_hi)
                    continue;                                    // none of the wave's tokens
                const bool every = __builtin_amdgcn_readfirstlane(sh_every[buf][part]) != 0;
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    bf16x8 f[kSteps];
#pragma unroll
                    for (int st = 0; st < kSteps; ++st)
                        f[st] = __builtin_bit_cast(bf16x8, sh_q[buf][h][part][st][half * 32 + (m32 ^ spread(st, half))]);
                    __builtin_amdgcn_sched_barrier(0);           // all loads first
#pragma unroll
                    for (int st = 0; st < kSteps; ++st)
#pragma unroll
                        for (int n = 0; n < kTiles; ++n)
                            x[n] = mfma32(f[st], kf[n][st], x[n]);
                }
                float lse[16];
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const f32x4 t = *(const f32x4 *)&sh_lse[buf][part][half][e];
                    lse[e] = t[0]; lse[e + 1] = t[1]; lse[e + 2] = t[2]; lse[e + 3] = t[3];
                }
#pragma unroll
                for (int n = 0; n < kTiles; ++n) {
                    const int g = (j0 >> 4) + 2 * (wave * kTiles + n);
                    float part_sum[2] = {0.0f, 0.0f};
                    if (every && mask.all(g, q_lo, q_hi) && mask.all(g + 1, q_lo, q_hi)) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            part_sum[e & 1] += exp2_fast(fmaf(x[n][e], a.scale2, -lse[e]));
                    } else if (16 * g <= q_hi) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int query = sh_query[buf][part][half][e];
                            const float p = exp2_fast(fmaf(x[n][e], a.scale2, -lse[e]));
                            part_sum[e & 1] += mask.sees(query, token[n]) ? p : 0.0f;
                        }
                    }
                    sum[n] += part_sum[0] + part_sum[1];
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            const float all = half_sum(sum[n]);
            if (page[n] >= 0 && half == 0) {
                unsafeAtomicAdd(a.c.weights + group_first(a.c, page[n], head, token[n] >> 4) + (token[n] & 15), all);
            }
        }
    }
}

// Where both are launched, each takes the sequences that it is made for.
template <int D, int T>
hipError_t weigh_dt(const AttendArgs &a, hipStream_t s)
{
    const int64_t pairs = (int64_t)a.b.n_seqs * a.c.heads;
    if (a.splits > 0)
        step_kernel<D, T><<<(unsigned)(pairs * a.splits), kLanes, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.row_splits == 0)
        return e;
    rows_kernel<D, T><<<(unsigned)(pairs * a.row_splits), kLanes, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_weigh(const AttendArgs &a, int head_dim, int dtype, hipStream_t s)
{
    const bool b = dtype == SPLITZIP_KV4_BF16;
    if (head_dim == 64)
        return b ? weigh_dt<64, SPLITZIP_KV4_BF16>(a, s) : weigh_dt<64, SPLITZIP_KV4_FP16>(a, s);
    if (head_dim == 128)
        return b ? weigh_dt<128, SPLITZIP_KV4_BF16>(a, s) : weigh_dt<128, SPLITZIP_KV4_FP16>(a, s);
    return b ? weigh_dt<256, SPLITZIP_KV4_BF16>(a, s) : weigh_dt<256, SPLITZIP_KV4_FP16>(a, s);
}

}  // namespace kv4
}  // namespace sz
