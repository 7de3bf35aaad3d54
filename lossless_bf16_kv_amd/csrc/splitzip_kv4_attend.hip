// splitzip_kv4_attend.hip -- attention over the 4-bit KV cache.
//
//   s_ij = scale q_i . k_j over the tokens j that query i sees
//   o_i = sum_j exp(s_ij) v_j / sum_j exp(s_ij),  lse_i = log sum_j exp(s_ij)
//
// in one pass over the tokens: with x = s log2(e) and any reference m_i >= max x, keep
// l = sum 2^(x - m) and O = sum 2^(x - m) v, in 32 bits; where the reference has to grow, l and O
// are multiplied by 2^(m_old - m_new).  It grows to 8 above the score that passed it, which makes the
// multiplications rare.  No factor of v is above 1: O leaves 32 bits only where sum 2^(x - max x) |v|
// does (v goes up to 6 * 2^125).
//
// Rows are pairs of a query and a head of the group (row = query * group + head): the heads of a
// group share K and V, so they fill the 16 columns of a matrix instruction together.
//
// Two kernels.  few_rows: up to 16 or 32 rows a sequence and KV head (a decode step, a few drafts).
// Each wave takes pairs of groups of its own, has the codes of the next two pairs on their way to LDS
// while it works on this one, and waits for no other wave until their results are joined.  32 decode
// steps at 32768 tokens (64 heads on 8 of 128 channels): 1.14 GB in 218 us, 5.2 TB/s, 74 % of what
// reading alone reaches; the same loads into registers: 229 us.  Waves wait for memory 17 % of their
// time; 223 vector (96 conversions and transpositions) and 16 matrix instructions for 32 tokens keep
// those units busy 49 and 14 % of it.  More waves, priorities and 15 % fewer scalar instructions did
// not change the time.
//
// many_rows: 64, 128 or 256 rows a workgroup (long drafts, prefill chunks), which share the conversion
// of V.  4096 queries of 32 heads on 8192 tokens: 412 GFLOP in 414 us, 1.0 PFLOP/s, three quarters of
// a large bf16 matrix product's rate here; the matrix unit is busy 43 % and the vector unit 56 % of the
// time, and the rest is what two waves on a unit leave open.  Before: 16-row products with K in LDS as
// bf16, 1409 us (LDS reads as long as the products); 32-row products and K's codes in LDS, 680; two
// tiles at a time, 571; heads fastest, so that a head's tiles share an L2, 457.
//
// The scaled matrix instructions would take K's codes as they are, and a bf16 query as two e4m3 parts
// exactly, but their sums over 128 terms are off by up to 2^-13 of the terms' sizes (measured; fp32
// sums: 2^-17 allowed here), so K becomes bf16 as well.
//
// Long axes with few workgroups are split; partial results (m, l, O in 32 bits) are joined by
// join_kernel in the order of the splits, so results do not depend on timing.
//
// Probabilities enter the second product as bf16 (half a step is 2^-8 of the value, as the
// rounding of a bf16 output; the sum l takes them unrounded).  With fp16 queries, queries and
// probabilities go in as two bf16 halves each, 16 bits in all.
#include "splitzip_kv4_tiles.h"

namespace sz {
namespace kv4 {
namespace {

constexpr int kLanes = kJoinThreads;

// Workgroup b -> KV head, row tile, sequence and split, the head fastest: workgroups go to the eight
// XCDs in turn, so each gets the same share of long and short sequences (with the split fastest one
// XCD in four got the late splits that few sequences have: 310 us for 265), and tiles that read the
// same keys and values meet in one L2.
struct Place {
    int s, head, tile, split;
    __device__ Place(const AttendArgs &a)
    {
        uint32_t b = blockIdx.x;
        head = b % a.c.heads;
        b /= a.c.heads;
        tile = b % a.tiles;
        b /= a.tiles;
        s = b % a.b.n_seqs;
        split = b / a.b.n_seqs;
    }
};

__device__ __forceinline__ uint32_t to_type(float a, float b, int t)
{
    return t == SPLITZIP_KV4_BF16 ? pack_bf16(a, b) : pack_fp16(a, b);
}

// Rows before the first sequence and behind the last: out = 0, lse = -infinity.  All workgroups share them, 16
// bytes a lane: 16 single tokens and 4080 rows of 64 heads behind them 60 us, by the last sequence's workgroups
// alone 1770.  Asking for the two offsets, beside the sequence's own, takes every call with offsets 0.4 us.
template <int D>
__device__ __forceinline__ void fill_unowned(const AttendArgs &a, int64_t lead, int64_t tail)
{
    const int64_t pieces = (lead + a.b.total - tail) * a.q_heads * (D / 8);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * blockDim.x) {
        int64_t row = i / (D / 8);
        row += row < lead * a.q_heads ? 0 : (tail - lead) * a.q_heads;
        *(uint4 *)((uint16_t *)a.out + row * D + i % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
        if (i % (D / 8) == 0 && a.lse)
            a.lse[row] = -INFINITY;
    }
}

// The part of `count` groups that a split takes: [first, last).  `used` splits have one; what the
// launch did not expect goes to the last.  A split that has all of them writes the result itself.
struct Share {
    int first, last, used;
    __device__ Share(const AttendArgs &a, int count, int split)
    {
        used = max(1, min(a.splits, (int)((uint32_t)(count + a.per - 1) / (uint32_t)a.per)));
        first = min(count, split * a.per);
        last = split == used - 1 ? count : min(count, first + a.per);
    }
};

// The groups that rows row0 .. of a sequence's tile see.
__device__ __forceinline__ Groups tile_groups(const AttendArgs &a, const Seq &q, int row0, int tile_rows)
{
    const int rows = q.n * a.group, base = q.len - q.n;
    return Groups(base + row0 / a.group, base + min(row0 + tile_rows - 1, rows - 1) / a.group, a.window, a.sinks);
}

// Scores are scaled by a positive number: a negative scale's sign goes to the queries, and a scale of
// 0 makes them 0.
struct Scale {
    float by;
    uint32_t keep, flip;
    __device__ explicit Scale(float s)
    {
        by = s == 0.0f ? 1.0f : fabsf(s);
        keep = s == 0.0f ? 0u : 0xffffffffu;
        flip = s < 0.0f ? 0x80008000u : 0u;
    }
    __device__ __forceinline__ bf16x8 operator()(bf16x8 x) const
    {
        uint4 w = __builtin_bit_cast(uint4, x);
        w.x = (w.x & keep) ^ flip; w.y = (w.y & keep) ^ flip;
        w.z = (w.z & keep) ^ flip; w.w = (w.w & keep) ^ flip;
        return __builtin_bit_cast(bf16x8, w);
    }
};

// Largest of N values.
template <int N>
__device__ __forceinline__ float max_of(const float (&x)[N])
{
    float a = x[0], b = x[1];
#pragma unroll
    for (int i = 2; i < N; i += 4) {
        a = fmaxf(fmaxf(a, x[i]), x[i + 1]);
        if (i + 3 < N)
            b = fmaxf(fmaxf(b, x[i + 2]), x[i + 3]);
    }
    return fmaxf(a, b);
}

// Eight probabilities as an operand, in one or two halves.
template <int Halves>
__device__ __forceinline__ void p_frag(const float (&p)[8], bf16x8 (&f)[Halves])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = pack_bf16(p[2 * i], p[2 * i + 1]);
    f[0] = frag(w[0], w[1], w[2], w[3]);
    if constexpr (Halves == 2) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = pack_bf16(p[2 * i] - bf16_lo(w[i]), p[2 * i + 1] - bf16_hi(w[i]));
        f[1] = frag(x[0], x[1], x[2], x[3]);
    }
}

// ---- few rows -------------------------------------------------------------------------------

template <int D>
struct Pair {
    KRaw<D> ka, kb;
    VRaw<D> va, vb;
    int ga, gb;          // groups; -1: none, or on a bad page
};

// A pair's codes and scales in LDS, written there by loads that need no registers, so that two pairs
// of every wave are on their way at a time:
//   K of both groups, V of both groups, D / 32 * 256 bytes each
//     D >= 128: 16 bytes a lane in lane order (D = 256: two of them); D = 64: as in the cache
//   scales: K's of both groups (as in the cache), V's of both groups [block][token], D / 2 bytes each
template <int D>
struct Ring {
    static constexpr int kCodes = 8 * D, kScales = D / 2, kBytes = 4 * kCodes + 4 * kScales;
    static constexpr int kLoads = D == 64 ? 3 : D == 128 ? 5 : 10;       // instructions a pair
    uint8_t slot[2][kBytes];
};

// Groups ga and gb (on pages pa and pb; -1: page 0's tokens) to a slot.
template <int D>
__device__ __forceinline__ void send_pair(const Cache &c, int pa, int pb, int head, int ga, int gb, uint32_t lane, uint8_t *slot)
{
    constexpr int kCodes = Ring<D>::kCodes;
    const uint32_t r = lane & 15, quad = lane >> 4;
    const int64_t ta = group_first(c, pa, head, ga), tb = group_first(c, pb, head, gb);
    const int64_t a0 = ta >> c.page_shift << c.page_shift, b0 = tb >> c.page_shift << c.page_shift;
    const uint8_t *const va = c.v_scales + a0 * (D / 32) + (ta - a0), *const vb = c.v_scales + b0 * (D / 32) + (tb - b0);
    if constexpr (D == 64) {
        // one load for both groups: lanes 32 .. 63 take the second
        const int64_t t = lane < 32 ? ta : tb;
        to_lds16(c.k_codes + t * 32 + 16 * (lane & 31), slot);
        to_lds16(c.v_codes + t * 32 + 16 * (lane & 31), slot + 2 * kCodes);
        if (lane < 32) {
            const uint32_t x = lane & 7;
            const uint8_t *const ks = c.k_scales + (lane & 8 ? tb : ta) * 2 + 4 * x;
            const uint8_t *const vs = (lane & 8 ? vb : va) + (x >> 2 << c.page_shift) + 4 * (x & 3);
            to_lds4(lane < 16 ? ks : vs, slot + 4 * kCodes);
        }
    } else {
#pragma unroll
        for (int i = 0; i < D / 128; ++i) {
            const uint32_t k = r * (D / 2) + quad * (D / 8) + 16 * i, v = quad * (2 * D) + r * (D / 8) + 16 * i;
            to_lds16(lane_at(c.k_codes + ta * (D / 2), k), slot + 1024 * i);
            to_lds16(lane_at(c.k_codes + tb * (D / 2), k), slot + kCodes + 1024 * i);
            to_lds16(lane_at(c.v_codes + ta * (D / 2), v), slot + 2 * kCodes + 1024 * i);
            to_lds16(lane_at(c.v_codes + tb * (D / 2), v), slot + 3 * kCodes + 1024 * i);
        }
        if constexpr (D == 128) {
            const uint8_t *const ks = c.k_scales + (lane & 16 ? tb : ta) * 4 + 4 * r;
            const uint8_t *const vs = (lane & 16 ? vb : va) + (r >> 2 << c.page_shift) + 4 * (r & 3);
            to_lds4(lane < 32 ? ks : vs, slot + 4 * kCodes);
        } else {
            const uint32_t x = lane & 31;
            to_lds4(c.k_scales + (lane < 32 ? ta : tb) * 8 + 4 * x, slot + 4 * kCodes);
            to_lds4((lane < 32 ? va : vb) + (x >> 2 << c.page_shift) + 4 * (x & 3), slot + 4 * kCodes + 256);
        }
    }
}

// A slot's pair to registers, once its loads are done: all but the Younger instructions behind them.
// The compiler would wait for every load to LDS before it reads there, so waits and reads are one
// piece of assembly.
template <int D, int Younger>
__device__ __forceinline__ void take_pair(const uint8_t *slot, uint32_t lane, Pair<D> &p)
{
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const uint32_t r = lane & 15, quad = lane >> 4;
    const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr)slot;
    if constexpr (D == 64) {
        const uint32_t k = base + r * 32 + quad * 8, v = base + quad * 128 + r * 8;
        const uint32_t ks = base + r * 2 + (quad >> 1), vs = base + (r >> 3) * 16 + quad * 4;
        u32x2 a, b, c, d;
        asm volatile("s_waitcnt vmcnt(%12)\n"
                     "ds_read_b64 %0, %8\n"
                     "ds_read_b64 %1, %8 offset:0x200\n"
                     "ds_read_b64 %2, %9 offset:0x400\n"
                     "ds_read_b64 %3, %9 offset:0x600\n"
                     "ds_read_u8 %4, %10 offset:0x800\n"
                     "ds_read_u8 %5, %10 offset:0x820\n"
                     "ds_read_b32 %6, %11 offset:0x840\n"
                     "ds_read_b32 %7, %11 offset:0x860\n"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d), "=&v"(p.ka.s), "=&v"(p.kb.s), "=&v"(p.va.s), "=&v"(p.vb.s)
                     : "v"(k), "v"(v), "v"(ks), "v"(vs), "n"(Younger)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            p.ka.w[i] = a[i]; p.kb.w[i] = b[i]; p.va.w[i] = c[i]; p.vb.w[i] = d[i];
        }
    } else if constexpr (D == 128) {
        const uint32_t k = base + 16 * lane, ks = base + r * 4 + quad, vs = base + (r >> 2) * 16 + quad * 4;
        u32x4 a, b, c, d;
        asm volatile("s_waitcnt vmcnt(%11)\n"
                     "ds_read_b128 %0, %8\n"
                     "ds_read_b128 %1, %8 offset:0x400\n"
                     "ds_read_b128 %2, %8 offset:0x800\n"
                     "ds_read_b128 %3, %8 offset:0xc00\n"
                     "ds_read_u8 %4, %9 offset:0x1000\n"
                     "ds_read_u8 %5, %9 offset:0x1040\n"
                     "ds_read_b32 %6, %10 offset:0x1080\n"
                     "ds_read_b32 %7, %10 offset:0x10c0\n"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d), "=&v"(p.ka.s), "=&v"(p.kb.s), "=&v"(p.va.s), "=&v"(p.vb.s)
                     : "v"(k), "v"(ks), "v"(vs), "n"(Younger)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p.ka.w[i] = a[i]; p.kb.w[i] = b[i]; p.va.w[i] = c[i]; p.vb.w[i] = d[i];
        }
    } else {
        const uint32_t k = base + 16 * lane, ks = base + r * 8 + 2 * quad, vs = base + (r >> 1) * 16 + quad * 4;
        u32x4 a, b, c, d, e, f, g, h;
        asm volatile("s_waitcnt vmcnt(%15)\n"
                     "ds_read_b128 %0, %12\n"
                     "ds_read_b128 %1, %12 offset:0x400\n"
                     "ds_read_b128 %2, %12 offset:0x800\n"
                     "ds_read_b128 %3, %12 offset:0xc00\n"
                     "ds_read_b128 %4, %12 offset:0x1000\n"
                     "ds_read_b128 %5, %12 offset:0x1400\n"
                     "ds_read_b128 %6, %12 offset:0x1800\n"
                     "ds_read_b128 %7, %12 offset:0x1c00\n"
                     "ds_read_u16 %8, %13 offset:0x2000\n"
                     "ds_read_u16 %9, %13 offset:0x2080\n"
                     "ds_read_b32 %10, %14 offset:0x2100\n"
                     "ds_read_b32 %11, %14 offset:0x2180\n"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d), "=&v"(e), "=&v"(f), "=&v"(g), "=&v"(h), "=&v"(p.ka.s),
                       "=&v"(p.kb.s), "=&v"(p.va.s), "=&v"(p.vb.s)
                     : "v"(k), "v"(ks), "v"(vs), "n"(Younger)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p.ka.w[i] = a[i]; p.ka.w[4 + i] = b[i]; p.kb.w[i] = c[i]; p.kb.w[4 + i] = d[i];
            p.va.w[i] = e[i]; p.va.w[4 + i] = f[i]; p.vb.w[i] = g[i]; p.vb.w[4 + i] = h[i];
        }
    }
}

// 16 * Cols rows a workgroup.
template <int D, int T, int Cols>
__global__ __launch_bounds__(kLanes, D == 256 ? 1 : Cols == 2 ? 2 : T == SPLITZIP_KV4_BF16 ? 4 : 3) void few_rows(AttendArgs a)
{
    constexpr int kHalves = T == SPLITZIP_KV4_FP16 ? 2 : 1;
    constexpr int kSteps = D / 32, kTiles = D / 16;
    constexpr int kRows = 16 * Cols;
    constexpr int kPitch = D + 4;
    // a wave's ring and, behind it in time, its results
    __shared__ __align__(16) union Buffer {
        Ring<D> ring;
        float o[16][kPitch];
        __device__ Buffer() {}
    } sh[4];
    __shared__ float sh_m[4][16], sh_l[4][16];

    const Place at(a);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, quad = lane >> 4;
    const int lead = a.b.cu ? row_offset(a.b, 0) : 0, tail = a.b.cu ? row_offset(a.b, a.b.n_seqs) : (int)a.b.total;
    const Seq q = wave_sequence(a.c, a.b, at.s);
    if (lead > 0 || tail < a.b.total)
        fill_unowned<D>(a, lead, tail);
    const int rows = q.n * a.group;
    const Mask mask = {a.window, a.sinks};
    const Scale scale(a.scale2);

    for (int row0 = at.tile * kRows; row0 < rows; row0 += a.tiles * kRows) {
        const int base = q.len - q.n;
        const int q_lo = base + row0 / a.group, q_hi = base + min(row0 + kRows - 1, rows - 1) / a.group;
        int query[Cols];
        bf16x8 qf[Cols][kHalves][kSteps];
#pragma unroll
        for (int c = 0; c < Cols; ++c) {
            const int row = min(row0 + 16 * c + r, rows - 1);
            query[c] = base + row / a.group;
            const int64_t p = (q.row0 + row / a.group) * a.q_token + (at.head * a.group + row % a.group) * a.q_head +
                              quad * (D / 4);
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                qf[c][0][st] = scale(q_frag<T, 0>(a.q, p + 8 * st, a.wide));
                if constexpr (kHalves == 2)
                    qf[c][1][st] = scale(q_frag<T, 1>(a.q, p + 8 * st, a.wide));
            }
        }
        const Groups groups = tile_groups(a, q, row0, kRows);
        const Share share(a, groups.count, at.split);
        if (at.split >= share.used)
            continue;
        const int first = share.first, last = share.last;

        float m[Cols], l[Cols];
        uint32_t lost[Cols];                     // blocks whose result is a NaN
        f32x4 o[Cols][kTiles];
#pragma unroll
        for (int c = 0; c < Cols; ++c) {
            m[c] = -INFINITY;
            l[c] = 0.0f;
            lost[c] = 0;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
                o[c][t] = f32x4{0, 0, 0, 0};
        }

        Pages pages_a, pages_b;
        const int v0 = first + 2 * wave;
        auto group = [&](int v) { return v < last ? groups.at(v) : -1; };
        const int turns = v0 < last ? (last - v0 + 7) >> 3 : 0;
        // a turn's groups; -1: none, or on a bad page
        struct Two {
            int a, b;
        };
        auto send = [&](int i) {
            const int v = v0 + 8 * i;
            const int pa = pages_a.at(a.c, a.b, at.s, groups, v0, 8, last, i);
            const int pb = pages_b.at(a.c, a.b, at.s, groups, v0 + 1, 8, last, i);
            const int ga = group(v), gb = group(v + 1);
            send_pair<D>(a.c, pa, pb, at.head, ga, gb, lane, sh[wave].ring.slot[i & 1]);
            return Two{ga | pa >> 31, gb | pb >> 31};
        };
        Two now = {-1, -1}, then = {-1, -1};
        if (turns > 0)
            now = send(0);
        if (turns > 1)
            then = send(1);
        for (int n = 0; n < turns; ++n) {
            Pair<D> cur;
            if (n + 1 < turns)
                take_pair<D, Ring<D>::kLoads>(sh[wave].ring.slot[n & 1], lane, cur);
            else
                take_pair<D, 0>(sh[wave].ring.slot[n & 1], lane, cur);
            cur.ga = now.a;
            cur.gb = now.b;
            now = then;
            if (n + 2 < turns)
                then = send(n + 2);
            f32x4 sa[Cols], sb[Cols];
#pragma unroll
            for (int c = 0; c < Cols; ++c)
                sa[c] = sb[c] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const bf16x8 fa = k_frag<D>(cur.ka, st), fb = k_frag<D>(cur.kb, st);
#pragma unroll
                for (int c = 0; c < Cols; ++c)
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        sa[c] = mfma(fa, qf[c][h][st], sa[c]);
                        sb[c] = mfma(fb, qf[c][h][st], sb[c]);
                    }
            }
            const bool whole = (cur.ga >= 0) & (cur.gb >= 0) & mask.all(cur.ga, q_lo, q_hi) & mask.all(cur.gb, q_lo, q_hi);
            const int ja = 16 * cur.ga + 4 * quad, jb = 16 * cur.gb + 4 * quad;
            bf16x8 pf[Cols][kHalves];
#pragma unroll
            for (int c = 0; c < Cols; ++c) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = sa[c][i];
                    x[4 + i] = sb[c][i];
                }
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = cur.ga >= 0 && mask.sees(query[c], ja + i) ? x[i] : -INFINITY;
                        x[4 + i] = cur.gb >= 0 && mask.sees(query[c], jb + i) ? x[4 + i] : -INFINITY;
                    }
                }
                const float top = quad_max(max_of(x)) * scale.by;
                if (__any(top > m[c])) {
                    const float grown = fmaxf(m[c], top + 8.0f);
                    const float f = grown == -INFINITY ? 1.0f : exp2_fast(m[c] - grown);
                    m[c] = grown;
                    l[c] *= f;
#pragma unroll
                    for (int t = 0; t < kTiles; ++t)
                        o[c][t] *= f;
                }
                const float ref = m[c] == -INFINITY ? 0.0f : m[c];
                float p[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p[i] = exp2_fast(fmaf(x[i], scale.by, -ref));
                    l[c] += p[i];
                }
                p_frag<kHalves>(p, pf[c]);
            }
            if (!whole && __any(v_bad(cur.va.s) || v_bad(cur.vb.s))) {
                no_nan(cur.va);
                no_nan(cur.vb);
#pragma unroll
                for (int c = 0; c < Cols; ++c) {
                    lost[c] |= poison<D>(a.c, a.b, at.s, at.head, cur.ga, mask, query[c]);
                    lost[c] |= poison<D>(a.c, a.b, at.s, at.head, cur.gb, mask, query[c]);
                }
            }
#pragma unroll
            for (int t = 0; t < kTiles; t += 2) {
                uint2 a0, a1, b0, b1;
                v_half<D>(cur.va, t / 2, a0, a1);
                v_half<D>(cur.vb, t / 2, b0, b1);
                const bf16x8 f0 = frag(a0.x, a0.y, b0.x, b0.y), f1 = frag(a1.x, a1.y, b1.x, b1.y);
#pragma unroll
                for (int c = 0; c < Cols; ++c)
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        o[c][t] = mfma(f0, pf[c][h], o[c][t]);
                        o[c][t + 1] = mfma(f1, pf[c][h], o[c][t + 1]);
                    }
            }
        }

        // join the four waves
#pragma unroll
        for (int c = 0; c < Cols; ++c) {
            if (__any(lost[c] != 0)) {
                // the lane's channels (4 quad + i) * kTiles + t: of block (4 quad + i) / 2
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (lost[c] >> ((4 * quad + i) * kTiles / 32) & 1)
#pragma unroll
                        for (int t = 0; t < kTiles; ++t)
                            o[c][t][i] = NAN;
            }
            l[c] = quad_sum(l[c]);
            if (quad == 0) {
                sh_m[wave][r] = m[c];
                sh_l[wave][r] = l[c];
            }
            // channels (4 quad + i) * kTiles + t of row r
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t = 0; t < kTiles; t += 4) {
                    const f32x4 x = {o[c][t][i], o[c][t + 1][i], o[c][t + 2][i], o[c][t + 3][i]};
                    *(f32x4 *)&sh[wave].o[r][(4 * quad + i) * kTiles + t] = x;
                }
            __syncthreads();
            const int orow = threadIdx.x >> 4, part = threadIdx.x & 15;
            const int row = row0 + 16 * c + orow;
            float big = sh_m[0][orow];
#pragma unroll
            for (int w = 1; w < 4; ++w)
                big = fmaxf(big, sh_m[w][orow]);
            float f[4], sum = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                f[w] = big == -INFINITY ? 1.0f : exp2_fast(sh_m[w][orow] - big);
                sum += sh_l[w][orow] * f[w];
            }
            if (row < rows) {
                const int64_t g = (q.row0 + row / a.group) * (int64_t)a.q_heads + at.head * a.group + row % a.group;
                // thread's channels: 4 part + 64 k
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                for (int k = 0; k < D; k += 64) {
                    const int d = k + 4 * part;
                    f32x4 x = *(const f32x4 *)&sh[0].o[orow][d] * f[0];
#pragma unroll
                    for (int w = 1; w < 4; ++w)
                        x += *(const f32x4 *)&sh[w].o[orow][d] * f[w];
                    if (share.used == 1) {
                        x *= inv;
                        *(uint2 *)((uint16_t *)a.out + g * D + d) = make_uint2(to_type(x[0], x[1], T), to_type(x[2], x[3], T));
                    } else {
                        *(f32x4 *)(a.part_o + ((int64_t)at.split * a.b.total * a.q_heads + g) * D + d) = x;
                    }
                }
                if (part == 0) {
                    if (share.used == 1) {
                        if (a.lse)
                            a.lse[g] = sum == 0.0f ? -INFINITY : (big + __log2f(sum)) * kLn2;
                    } else {
                        float *ml = a.part_ml + ((int64_t)at.split * a.b.total * a.q_heads + g) * 2;
                        ml[0] = big;
                        ml[1] = sum;
                    }
                }
            }
            __syncthreads();
        }
    }
}

// ---- many rows ------------------------------------------------------------------------------

// kWaves waves, 32 rows each: `Rows` of them side by side along the rows, the others (times Rows)
// take other tokens of a turn and are joined at the end.  A turn is 16 tokens a wave: each wave puts
// the codes and scales of one group's K and the bf16 operands of its V into LDS, all in the order in
// which lanes read them, and every wave multiplies tiles of 32 tokens from there.  V's conversion
// is shared, since it takes two instructions a value pair and a transposition; K's takes one, and its
// codes are a quarter of the LDS traffic that bf16 would be.
template <int D, int kWaves>
struct Stage {
    static constexpr int kTiles = kWaves / 2;            // of 32 tokens, a turn
    static constexpr int kLaneScales = D / 64;           // K's scale bytes of a lane: of D / 2 channels
    uint4 k[kTiles][D / 64][64];                         // lane (token l % 32): channels (l / 32) D / 2 ..
    uint4 v[kWaves][D / 32][64];                         // lane (channel): tokens 8 j + 4 (l / 32) .. + 3, j < 2
    uint8_t ks[kTiles][64][kLaneScales];
    int note[kWaves];                                    // of a group; 1: no page, 2: V is not finite
};

template <int D, int T, int kWaves, int Rows>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void many_rows(AttendArgs a)
{
    constexpr int kHalves = T == SPLITZIP_KV4_FP16 ? 2 : 1;
    constexpr int kTiles = Stage<D, kWaves>::kTiles;
    constexpr int kSteps = D / 16, kOut = D / 32;
    constexpr int kParts = kWaves / Rows;                // waves that share rows
    constexpr int kRows = 32 * Rows;
    static_assert(kParts <= kTiles, "a wave without a tile");
    // tiles worked on together: their products and exponentials do not wait for each other
    constexpr int kJoin = D < 256 && kTiles / kParts >= 2 ? 2 : 1;
    __shared__ union Shared {
        Stage<D, kWaves> stage[2];
        float join[kParts > 1 ? kWaves / 2 : 1][16 * kOut + 2][64];
        __device__ Shared() {}
    } sh;

    const Place at(a);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m32 = lane & 31, half = lane >> 5;
    const int part = wave / Rows;
    const int lead = a.b.cu ? row_offset(a.b, 0) : 0, tail = a.b.cu ? row_offset(a.b, a.b.n_seqs) : (int)a.b.total;
    const Seq q = wave_sequence(a.c, a.b, at.s);
    if (lead > 0 || tail < a.b.total)
        fill_unowned<D>(a, lead, tail);
    const int rows = q.n * a.group;
    const Mask mask = {a.window, a.sinks};
    const Scale scale(a.scale2);

    // later rows see more tokens: they start first
    const int row_tiles = (rows + kRows - 1) / kRows;
    for (int n = at.tile; n < row_tiles; n += a.tiles) {
        const int row0 = (row_tiles - 1 - n) * kRows;
        const int base = q.len - q.n;
        const Groups groups = tile_groups(a, q, row0, kRows);
        const Share share(a, groups.count, at.split);
        if (at.split >= share.used)
            continue;
        const int first = share.first, last = share.last;

        // this wave's rows; a row past the end repeats the last and is not stored
        const int w_row = row0 + wave % Rows * 32;
        const int row = min(w_row + m32, rows - 1);
        const int query = base + row / a.group;
        bf16x8 qf[kHalves][kSteps];
        {
            const int64_t p0 = (q.row0 + row / a.group) * a.q_token + (at.head * a.group + row % a.group) * a.q_head +
                               half * (D / 2);
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                qf[0][st] = scale(q_frag<T, 0>(a.q, p0 + 8 * st, a.wide));
                if constexpr (kHalves == 2)
                    qf[1][st] = scale(q_frag<T, 1>(a.q, p0 + 8 * st, a.wide));
            }
        }
        const int q_lo = base + min(w_row, rows - 1) / a.group;
        const int q_hi = base + min(w_row + 31, rows - 1) / a.group;

        float m = -INFINITY, l = 0.0f;
        uint32_t lost = 0;                               // blocks whose result is a NaN
        f32x16 o[kOut];
#pragma unroll
        for (int t = 0; t < kOut; ++t)
            o[t] = f32x16{};

        struct Raw {
            KRaw<D> k;
            VRaw<D> v;
            int g;
        } raw;
        const int r = lane & 15, quad = lane >> 4;
        // the four tokens whose V a lane converts: lanes 0 .. 31 then write 256 adjacent bytes
        const int v_quad = 2 * (quad & 1) + (quad >> 1);
        Pages pages;
        auto fetch = [&](int i) {
            Raw x;
            const int v = first + wave + kWaves * i;
            const int page = pages.at(a.c, a.b, at.s, groups, first + wave, kWaves, last, i);
            x.g = v < last ? groups.at(v) : -1;
            x.k = load_k<D>(a.c, page, at.head, x.g, lane);
            x.v = load_v<D>(a.c, page, at.head, x.g, lane, v_quad);
            x.g = page < 0 ? -1 : x.g;
            return x;
        };
        auto put = [&](Raw &x, Stage<D, kWaves> &st) {
            const bool bad = __any(v_bad(x.v.s));
            if (bad)
                no_nan(x.v);
            const int to = (quad >> 1) * 32 + (wave & 1) * 16 + r;      // K's lane; its piece is of the half's second half
            if constexpr (D == 64) {
                *(uint2 *)((char *)&st.k[wave / 2][0][to] + 8 * (quad & 1)) = make_uint2(x.k.w[0], x.k.w[1]);
                if ((quad & 1) == 0)
                    st.ks[wave / 2][to][0] = (uint8_t)x.k.s;
            } else {
#pragma unroll
                for (int i = 0; i < D / 128; ++i)
                    st.k[wave / 2][(quad & 1) * (D / 128) + i][to] =
                        make_uint4(x.k.w[4 * i], x.k.w[4 * i + 1], x.k.w[4 * i + 2], x.k.w[4 * i + 3]);
                if constexpr (D == 128)
                    st.ks[wave / 2][to][quad & 1] = (uint8_t)x.k.s;
                else
                    *(uint16_t *)&st.ks[wave / 2][to][2 * (quad & 1)] = (uint16_t)x.k.s;
            }
#pragma unroll
            for (int t = 0; t < kOut; ++t) {
                uint2 lo, hi;
                v_half<D>(x.v, t, lo, hi);
                uint2 *v = (uint2 *)&st.v[wave][t][(quad >> 1) * 32 + r] + (quad & 1);
                v[0] = lo;
                v[32] = hi;                              // 16 lanes on
            }
            if (lane == 0)
                st.note[wave] = (x.g < 0 ? 1 : 0) | (bad ? 2 : 0);
        };

        if (first < last) {
            raw = fetch(0);
            put(raw, sh.stage[0]);
            raw = fetch(1);
        }
        __syncthreads();
        for (int i = 0; first + kWaves * i < last; ++i) {
            const Stage<D, kWaves> &st = sh.stage[i & 1];
            if (first + kWaves * (i + 1) < last) {
                put(raw, sh.stage[(i + 1) & 1]);
                raw = fetch(i + 2);
            }
            int notes = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                notes |= st.note[w];
            notes = __builtin_amdgcn_readfirstlane(notes);
#pragma unroll 1
            for (int tile = part * kJoin; tile < kTiles; tile += kParts * kJoin) {
                const int v = first + kWaves * i + 2 * tile;
                if (v >= last || 16 * groups.at(v) > q_hi)
                    break;
                int g[2 * kJoin];                        // -1: none, or on a bad page
                bool whole = true;
#pragma unroll
                for (int n = 0; n < 2 * kJoin; ++n) {
                    g[n] = v + n < last ? groups.at(v + n) : -1;
                    if (notes != 0 && (__builtin_amdgcn_readfirstlane(st.note[2 * tile + n]) & 1))
                        g[n] = -1;
                    whole = whole & (g[n] >= 0) & mask.all(g[n], q_lo, q_hi);
                }
                // scores of 32 tokens a tile, ahead of the other wave's exponentials: the matrix unit idles less
                // (457 -> 417 us for 4096 queries of 32 heads on 8192 tokens, with the probabilities made before the
                // second products start)
                __builtin_amdgcn_s_setprio(1);
                f32x16 x[kJoin];
                uint4 code[kJoin][D / 64];
                uint32_t ks[kJoin];
#pragma unroll
                for (int n = 0; n < kJoin; ++n) {
#pragma unroll
                    for (int p = 0; p < D / 64; ++p)
                        code[n][p] = st.k[tile + n][p][lane];
                    if constexpr (D == 64)
                        ks[n] = st.ks[tile + n][lane][0];
                    else if constexpr (D == 128)
                        ks[n] = *(const uint16_t *)st.ks[tile + n][lane];
                    else
                        ks[n] = *(const uint32_t *)st.ks[tile + n][lane];
                    x[n] = f32x16{};
                }
#pragma unroll
                for (int p = 0; p < D / 64; ++p)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int n = 0; n < kJoin; ++n) {
                            const uint4 c = code[n][p];
                            const uint32_t w = e == 0 ? c.x : e == 1 ? c.y : e == 2 ? c.z : c.w;
                            const float b = scale_of((ks[n] >> (8 * p)) & 0xff);       // 32 channels: one block
                            const bf16x8 f = frag(dequant<0>(w, b), dequant<1>(w, b), dequant<2>(w, b), dequant<3>(w, b));
#pragma unroll
                            for (int h = 0; h < kHalves; ++h)
                                x[n] = mfma32(f, qf[h][4 * p + e], x[n]);
                        }
                __builtin_amdgcn_s_setprio(0);
                if (!whole) {
#pragma unroll
                    for (int n = 0; n < kJoin; ++n)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int gr = g[2 * n + (e >> 3)];
                            const int j = 16 * gr + 8 * ((e >> 2) & 1) + 4 * half + (e & 3);
                            x[n][e] = gr >= 0 && mask.sees(query, j) ? x[n][e] : -INFINITY;
                        }
                }
                float top = -INFINITY;
#pragma unroll
                for (int n = 0; n < kJoin; ++n) {
                    float y[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        y[e] = x[n][e];
                    top = fmaxf(top, max_of(y));
                }
                top = half_max(top) * scale.by;
                if (__any(top > m)) {
                    const float grown = fmaxf(m, top + 8.0f);
                    const float f = grown == -INFINITY ? 1.0f : exp2_fast(m - grown);
                    m = grown;
                    l *= f;
#pragma unroll
                    for (int t = 0; t < kOut; ++t)
                        o[t] *= f;
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                bf16x8 pf[kJoin][2][kHalves];
#pragma unroll
                for (int n = 0; n < kJoin; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float p[8], sum[2] = {0.0f, 0.0f};
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            p[e] = exp2_fast(fmaf(x[n][8 * h + e], scale.by, -ref));
                            sum[e & 1] += p[e];
                        }
                        l += sum[0] + sum[1];
                        p_frag<kHalves>(p, pf[n][h]);
                    }
#pragma unroll
                for (int n = 0; n < kJoin; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int t = 0; t < kOut; ++t) {
                            const bf16x8 y = __builtin_bit_cast(bf16x8, st.v[2 * (tile + n) + h][t][lane]);
#pragma unroll
                            for (int k = 0; k < kHalves; ++k)
                                o[t] = mfma32(y, pf[n][h][k], o[t]);
                        }
                if (notes & 2) {
#pragma unroll
                    for (int n = 0; n < 2 * kJoin; ++n)
                        if (__builtin_amdgcn_readfirstlane(st.note[2 * tile + n]) & 2)
                            lost |= poison<D>(a.c, a.b, at.s, at.head, g[n], mask, query);
                }
            }
            __syncthreads();
        }
        l = half_sum(l);
        if (__any(lost != 0)) {
            // run 8 i + 4 half + e of D / 16 channels: block run / 2
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (lost >> ((8 * (i >> 2) + 4 * half + (i & 3)) * (D / 16) / 32) & 1)
#pragma unroll
                    for (int t = 0; t < kOut; ++t)
                        o[t][i] = o[t][8 + i] = NAN;
        }

        // join the waves of the same rows, half of the parts to the other half
        if constexpr (kParts > 1) {
#pragma unroll
            for (int d = kParts / 2; d >= 1; d /= 2) {
                float (*const x)[64] = sh.join[wave % (d * Rows)];
                if (part >= d && part < 2 * d) {
#pragma unroll
                    for (int t = 0; t < kOut; ++t)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            x[16 * t + e][lane] = o[t][e];
                    x[16 * kOut][lane] = m;
                    x[16 * kOut + 1][lane] = l;
                }
                __syncthreads();
                if (part < d) {
                    const float m2 = x[16 * kOut][lane], big = fmaxf(m, m2);
                    const float f = big == -INFINITY ? 1.0f : exp2_fast(m - big);
                    const float f2 = big == -INFINITY ? 1.0f : exp2_fast(m2 - big);
                    m = big;
                    l = l * f + x[16 * kOut + 1][lane] * f2;
#pragma unroll
                    for (int t = 0; t < kOut; ++t)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[t][e] = o[t][e] * f + x[16 * t + e][lane] * f2;
                }
                __syncthreads();
            }
        }
        if (part == 0 && w_row + m32 < rows) {
            const int64_t gr = (q.row0 + row / a.group) * (int64_t)a.q_heads + at.head * a.group + row % a.group;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            // run 8 i + 4 half + e of D / 16 channels, for this lane's row
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int d = (8 * (i >> 2) + 4 * half + (i & 3)) * (D / 16);
#pragma unroll
                for (int c = 0; c < D / 16; c += 4) {
                    f32x4 y = {o[c / 2][i], o[c / 2][8 + i], o[c / 2 + 1][i], o[c / 2 + 1][8 + i]};
                    if (share.used == 1) {
                        y *= inv;
                        *(uint2 *)((uint16_t *)a.out + gr * D + d + c) = make_uint2(to_type(y[0], y[1], T), to_type(y[2], y[3], T));
                    } else {
                        *(f32x4 *)(a.part_o + ((int64_t)at.split * a.b.total * a.q_heads + gr) * D + d + c) = y;
                    }
                }
            }
            if (half == 0) {
                if (share.used == 1) {
                    if (a.lse)
                        a.lse[gr] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
                } else {
                    float *ml = a.part_ml + ((int64_t)at.split * a.b.total * a.q_heads + gr) * 2;
                    ml[0] = m;
                    ml[1] = l;
                }
            }
        }
    }
}

// ---- joining splits -------------------------------------------------------------------------

// D / 4 lanes a row: o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, splits in order.  The factors
// are one a lane first, so that the loads of O do not wait for each other.
template <int D, int T>
__global__ __launch_bounds__(kLanes) void join_kernel(AttendArgs a)
{
    constexpr int kRow = D / 4;
    const int64_t rows = a.b.total * a.q_heads;                 // below 2^31
    const uint32_t row = blockIdx.x * (kLanes / kRow) + threadIdx.x / kRow;
    const int part = threadIdx.x % kRow, d = 4 * part;
    // Rows of no sequence fill_unowned wrote, those of one split that split did.  All lanes stay for the
    // shuffles.
    int splits = 0;
    if (row < rows) {
        const uint32_t i = row / (uint32_t)a.q_heads, f = row - i * a.q_heads;
        const int seq = sequence_of(a.b, i);
        if (seq >= 0) {
            const Seq q = sequence(a.c, a.b, seq);
            const int r = (int)(i - q.row0) * a.group + (int)(f % (uint32_t)a.group);
            splits = Share(a, tile_groups(a, q, r & ~(a.tile_rows - 1), a.tile_rows).count, 0).used;
        }
    }
    const bool mine = splits > 1;
    const int64_t from = mine ? (int64_t)row : 0;
    // O of eight splits at a time, the first on their way before the factors are known
    f32x4 y[8];
    auto load = [&](int s) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            y[e] = s + e < splits ? *(const f32x4 *)(a.part_o + ((s + e) * rows + from) * D + d) : f32x4{0, 0, 0, 0};
    };
    load(0);
    float big = -INFINITY;
    for (int s = part; s < splits; s += kRow)
        big = fmaxf(big, a.part_ml[(s * rows + from) * 2]);
#pragma unroll
    for (int x = 1; x < kRow; x *= 2)
        big = fmaxf(big, __shfl_xor(big, x));
    float sum = 0.0f;
    f32x4 x = {0, 0, 0, 0};
#pragma unroll 1
    for (int s0 = 0; __any(s0 < splits); s0 += kRow) {
        const int s = s0 + part;
        float f = 0.0f, l = 0.0f;
        if (s < splits) {
            const float m = a.part_ml[(s * rows + from) * 2];
            // m = -infinity: the split saw nothing, or NaN scores alone, which its sum holds
            f = big == -INFINITY ? 1.0f : exp2_fast(m - big);
            l = a.part_ml[(s * rows + from) * 2 + 1] * f;
        }
#pragma unroll 1
        for (int i = 0; i < kRow && __any(s0 + i < splits); i += 8) {
            if (s0 + i > 0)
                load(s0 + i);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float fe = __shfl(f, i + e, kRow);
                sum += __shfl(l, i + e, kRow);
                if (s0 + i + e < splits)
                    x += y[e] * fe;
            }
        }
    }
    if (!mine)
        return;
    x *= sum == 0.0f ? 0.0f : 1.0f / sum;
    *(uint2 *)((uint16_t *)a.out + (int64_t)row * D + d) = make_uint2(to_type(x[0], x[1], T), to_type(x[2], x[3], T));
    if (d == 0 && a.lse)
        a.lse[row] = sum == 0.0f ? -INFINITY : (big + __log2f(sum)) * kLn2;
}

template <int D, int T>
hipError_t attend_dt(const AttendArgs &a, hipStream_t s)
{
    const unsigned grid = (unsigned)((int64_t)a.b.n_seqs * a.c.heads * a.tiles * a.splits);
    constexpr int kWaves = D == 256 ? 4 : 8, kLanesMany = 64 * kWaves;
    if (a.tile_rows == 16)
        few_rows<D, T, 1><<<grid, kLanes, 0, s>>>(a);
    else if (a.tile_rows == 32) {
        if constexpr (D < 256)
            few_rows<D, T, 2><<<grid, kLanes, 0, s>>>(a);
    } else if (a.tile_rows == 64)
        many_rows<D, T, kWaves, 2><<<grid, kLanesMany, 0, s>>>(a);
    else if (a.tile_rows == 128)
        many_rows<D, T, kWaves, 4><<<grid, kLanesMany, 0, s>>>(a);
    else if constexpr (D < 256)
        many_rows<D, T, kWaves, 8><<<grid, kLanesMany, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1)
        return e;
    const int rows = join_rows(D);
    join_kernel<D, T><<<(unsigned)((a.b.total * a.q_heads + rows - 1) / rows), kLanes, 0, s>>>(a);
    return hipGetLastError();
}

template <int D>
hipError_t attend_d(const AttendArgs &a, int dtype, hipStream_t s)
{
    return dtype == SPLITZIP_KV4_BF16 ? attend_dt<D, SPLITZIP_KV4_BF16>(a, s) : attend_dt<D, SPLITZIP_KV4_FP16>(a, s);
}

}  // namespace

// Few rows wait for nobody, and waste no products on rows that are not there: drafts of 12 to 24 rows take
// 34 us by few_rows and 79 us in a tile of 64, decode steps of 8 rows 41 and 92 us.  More rows pay for a
// shared conversion: 16384 rows 672 us by 64, 511 by 128, 419 by 256; in fp16 701 by 128 and 661 by 256, though that
// one spills 5 registers at 128 channels.  At 256 channels 32 rows by few_rows
// and 256 by many_rows would not leave room for two waves' registers.
int attend_rows(int head_dim, int64_t rows)
{
    return rows <= 16 ? 16 : rows <= 32 && head_dim < 256 ? 32 : rows <= 64 ? 64 : rows <= 128 || head_dim == 256 ? 128 : 256;
}

int attend_threads(int head_dim, int tile_rows) { return tile_rows <= 32 || head_dim == 256 ? 256 : 512; }

int join_rows(int head_dim) { return kJoinThreads / (head_dim / 4); }

hipError_t launch_attend(const AttendArgs &a, int head_dim, int dtype, hipStream_t s)
{
    return head_dim == 64    ? attend_d<64>(a, dtype, s)
           : head_dim == 128 ? attend_d<128>(a, dtype, s)
                             : attend_d<256>(a, dtype, s);
}

}  // namespace kv4
}  // namespace sz
