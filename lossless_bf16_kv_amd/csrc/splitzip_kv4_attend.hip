// splitzip_kv4_attend.hip -- attention over the 4-bit KV cache.
//
//   s_ij = scale q_i . k_j over the tokens j that query i sees
//   o_i = sum_j exp(s_ij) v_j / sum_j exp(s_ij),  lse_i = log sum_j exp(s_ij)
//
// in one pass over the tokens: with x = s log2(e) and any reference m_i >= max x - 8, keep
// l = sum 2^(x - m) and O = sum 2^(x - m) v, in 32 bits; where the reference has to grow, l and O
// are multiplied by 2^(m_old - m_new).  Growing it only when a score passes it by 2^8 leaves the
// result unchanged and the multiplications rare.
//
// Rows are pairs of a query and a head of the group (row = query * group + head): the heads of a
// group share K and V, so they fill the 16 columns of a matrix instruction together.
//
// Two kernels.  few_rows: up to 16 rows a sequence and KV head (a decode step).  HBM bounds it:
// 1.06 bytes a channel pair of K and V against 64 flops.  Each wave takes pairs of groups of its
// own, holds the codes of the next pair in registers while it works on this one, and uses no LDS
// until the four waves' results are joined.  many_rows: 64 or 128 rows a workgroup (drafts,
// prefill chunks).  Each wave converts one group of every 64 tokens into matrix operands in LDS,
// which all four waves use: conversion would else cost as much as the products.
//
// Long axes with few workgroups are split; partial results (m, l, O in 32 bits) are joined by
// join_kernel in the order of the splits, so results do not depend on timing.
//
// Probabilities enter the second product as bf16 (half a step is 2^-9 of the value, as the
// rounding of a bf16 output; the sum l takes them unrounded).  With fp16 queries, queries and
// probabilities go in as two bf16 halves each, 16 bits in all.
#include "splitzip_kv4_tiles.h"

namespace sz {
namespace kv4 {
namespace {

constexpr int kLanes = 256;

// Workgroup b -> sequence, row tile, KV head and split.
struct Place {
    int s, head, tile, split;
    __device__ Place(const AttendArgs &a)
    {
        uint32_t b = blockIdx.x;
        split = b % a.splits;
        b /= a.splits;
        tile = b % a.tiles;
        b /= a.tiles;
        head = b % a.c.heads;
        s = b / a.c.heads;
    }
};

__device__ __forceinline__ uint32_t to_type(float a, float b, int t)
{
    return t == SPLITZIP_KV4_BF16 ? pack_bf16(a, b) : pack_fp16(a, b);
}

// Rows before the first sequence and behind the last: out = 0, lse = -infinity.
template <int D>
__device__ void fill_unowned(const AttendArgs &a, const Place &at)
{
    if (!a.b.cu || at.tile != 0 || at.split != 0 || (at.s != 0 && at.s != a.b.n_seqs - 1))
        return;
    for (int side = 0; side < 2; ++side) {
        if (at.s != (side ? a.b.n_seqs - 1 : 0))
            continue;
        const int64_t lo = side ? row_offset(a.b, a.b.n_seqs) : 0, hi = side ? a.b.total : row_offset(a.b, 0);
        for (int64_t i = lo; i < hi; ++i)
            for (int f = 0; f < a.group; ++f) {
                const int64_t row = i * a.q_heads + at.head * a.group + f;
                for (int d = threadIdx.x; d < D; d += kLanes)
                    ((uint16_t *)a.out)[row * D + d] = 0;
                if (threadIdx.x == 0 && a.lse)
                    a.lse[row] = -INFINITY;
            }
    }
}

// The part of `count` groups that a split takes: [first, last).
__device__ __forceinline__ void share(int count, int splits, int split, int unit, int &first, int &last)
{
    const int units = (count + unit - 1) / unit;
    const int per = (units + splits - 1) / splits;
    first = min(count, split * per * unit);
    last = min(count, first + per * unit);
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

// 1 where the query sees the token, as an operand like p_frag's.
__device__ __forceinline__ bf16x8 seen_frag(const Mask &mask, int query, int ja, int jb, bool ga, bool gb)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = (ga && mask.sees(query, ja + 2 * i) ? 0x3f80u : 0u) | (ga && mask.sees(query, ja + 2 * i + 1) ? 0x3f800000u : 0u);
        w[2 + i] = (gb && mask.sees(query, jb + 2 * i) ? 0x3f80u : 0u) | (gb && mask.sees(query, jb + 2 * i + 1) ? 0x3f800000u : 0u);
    }
    return frag(w[0], w[1], w[2], w[3]);
}

// o += V^T p over two groups for one result tile.  `odd`: some V among them is not finite and not
// every row sees all of them.  A product with a probability of 0 would be a NaN there, so such
// values are left out and the rows that do see one get a NaN.
template <int Halves>
__device__ __forceinline__ f32x4 add_pv(uint2 a, uint2 b, const bf16x8 (&p)[Halves], f32x4 o, bool odd, bf16x8 seen)
{
    if (odd) {
        uint2 ia, ib;
        split_finite(a.x, ia.x);
        split_finite(a.y, ia.y);
        split_finite(b.x, ib.x);
        split_finite(b.y, ib.y);
        const f32x4 hit = mfma(frag(ia.x, ia.y, ib.x, ib.y), seen, f32x4{0, 0, 0, 0});
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = hit[i] > 0.0f ? NAN : o[i];
    }
    const bf16x8 v = frag(a.x, a.y, b.x, b.y);
    o = mfma(v, p[0], o);
    if constexpr (Halves == 2)
        o = mfma(v, p[1], o);
    return o;
}

// ---- few rows -------------------------------------------------------------------------------

template <int D>
struct Pair {
    KRaw<D> ka, kb;
    VRaw<D> va, vb;
    int ga, gb;          // groups; -1: none, or on a bad page
};

template <int D, int T>
__global__ __launch_bounds__(kLanes, D == 256 ? 1 : 2) void few_rows(AttendArgs a)
{
    constexpr int kHalves = T == SPLITZIP_KV4_FP16 ? 2 : 1;
    constexpr int kSteps = D / 32, kTiles = D / 16;
    constexpr int kPitch = D + 4;
    __shared__ float sh_o[4][16][kPitch];
    __shared__ float sh_m[4][16], sh_l[4][16];

    const Place at(a);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, quad = lane >> 4;
    fill_unowned<D>(a, at);
    const Seq q = sequence(a.c, a.b, at.s);
    const int rows = q.n * a.group;
    const Mask mask = {a.window, a.sinks};

    for (int row0 = at.tile * 16; row0 < rows; row0 += a.tiles * 16) {
        const int base = q.len - q.n;
        const int row = min(row0 + r, rows - 1);
        const int query = base + row / a.group;
        const int q_lo = base + row0 / a.group, q_hi = base + min(row0 + 15, rows - 1) / a.group;
        const int64_t q_row = q.row0 + row / a.group;
        const int q_head = at.head * a.group + row % a.group;
        bf16x8 qf[kHalves][kSteps];
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            const int64_t p = q_row * a.q_token + q_head * a.q_head + quad * (D / 4) + 8 * st;
            qf[0][st] = q_frag<T, 0>(a.q, p, a.wide);
            if constexpr (kHalves == 2)
                qf[1][st] = q_frag<T, 1>(a.q, p, a.wide);
        }
        const Groups groups(q_lo, q_hi, a.window, a.sinks);
        int first, last;
        share(groups.count, a.splits, at.split, 8, first, last);

        float m = -INFINITY, l = 0.0f;
        f32x4 o[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            o[t] = f32x4{0, 0, 0, 0};

        auto fetch = [&](int v) {
            Pair<D> p;
            p.ga = v < last ? groups.at(v) : -1;
            p.gb = v + 1 < last ? groups.at(v + 1) : -1;
            const int pa = p.ga < 0 ? -1 : page_of(a.c, a.b, at.s, 16 * p.ga);
            const int pb = p.gb < 0 ? -1 : page_of(a.c, a.b, at.s, 16 * p.gb);
            p.ka = load_k<D>(a.c, pa, at.head, p.ga, lane);
            p.kb = load_k<D>(a.c, pb, at.head, p.gb, lane);
            p.va = load_v<D>(a.c, pa, at.head, p.ga, lane);
            p.vb = load_v<D>(a.c, pb, at.head, p.gb, lane);
            p.ga = pa < 0 ? -1 : p.ga;
            p.gb = pb < 0 ? -1 : p.gb;
            return p;
        };
        int v = first + 2 * wave;
        Pair<D> next;
        if (v < last)
            next = fetch(v);
        for (; v < last; v += 8) {
            const Pair<D> cur = next;
            if (v + 8 < last)
                next = fetch(v + 8);
            f32x4 sa = {0, 0, 0, 0}, sb = {0, 0, 0, 0};
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const bf16x8 fa = k_frag<D>(cur.ka, st), fb = k_frag<D>(cur.kb, st);
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    sa = mfma(fa, qf[h][st], sa);
                    sb = mfma(fb, qf[h][st], sb);
                }
            }
            const bool whole = cur.ga >= 0 && cur.gb >= 0 && mask.all(cur.ga, q_lo, q_hi) && mask.all(cur.gb, q_lo, q_hi);
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = sa[i] * a.scale2;
                x[4 + i] = sb[i] * a.scale2;
            }
            const int ja = 16 * cur.ga + 4 * quad, jb = 16 * cur.gb + 4 * quad;
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = cur.ga >= 0 && mask.sees(query, ja + i) ? x[i] : -INFINITY;
                    x[4 + i] = cur.gb >= 0 && mask.sees(query, jb + i) ? x[4 + i] : -INFINITY;
                }
            }
            float top = x[0];
#pragma unroll
            for (int i = 1; i < 8; ++i)
                top = fmaxf(top, x[i]);
            top = quad_max(top);
            if (__any(top > m + 8.0f)) {
                const float grown = fmaxf(m, top);
                const float f = grown == -INFINITY ? 1.0f : exp2_fast(m - grown);
                m = grown;
                l *= f;
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
                    o[t] *= f;
            }
            const float ref = m == -INFINITY ? 0.0f : m;
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = exp2_fast(x[i] - ref);
                l += p[i];
            }
            bf16x8 pf[kHalves];
            p_frag<kHalves>(p, pf);
            bf16x8 seen = {};
            const bool odd = !whole && __any(v_bad(cur.va.s) || v_bad(cur.vb.s));
            if (odd)
                seen = seen_frag(mask, query, ja, jb, cur.ga >= 0, cur.gb >= 0);
#pragma unroll
            for (int t = 0; t < kTiles; t += 2) {
                uint2 a0, a1, b0, b1;
                v_half<D>(cur.va, t / 2, a0, a1);
                v_half<D>(cur.vb, t / 2, b0, b1);
                o[t] = add_pv<kHalves>(a0, b0, pf, o[t], odd, seen);
                o[t + 1] = add_pv<kHalves>(a1, b1, pf, o[t + 1], odd, seen);
            }
        }

        // join the four waves
        l = quad_sum(l);
        if (quad == 0) {
            sh_m[wave][r] = m;
            sh_l[wave][r] = l;
        }
        // channels (4 quad + i) * kTiles + t of row r
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < kTiles; t += 4) {
                const f32x4 x = {o[t][i], o[t + 1][i], o[t + 2][i], o[t + 3][i]};
                *(f32x4 *)&sh_o[wave][r][(4 * quad + i) * kTiles + t] = x;
            }
        __syncthreads();
        const int orow = threadIdx.x >> 4, part = threadIdx.x & 15;
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
        if (row0 + orow < rows) {
            const int64_t g = (q.row0 + (row0 + orow) / a.group) * (int64_t)a.q_heads + at.head * a.group +
                              (row0 + orow) % a.group;
            // thread's channels: 4 part + 64 k
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int k = 0; k < D; k += 64) {
                const int d = k + 4 * part;
                f32x4 x = *(const f32x4 *)&sh_o[0][orow][d] * f[0];
#pragma unroll
                for (int w = 1; w < 4; ++w)
                    x += *(const f32x4 *)&sh_o[w][orow][d] * f[w];
                if (a.splits == 1) {
                    x *= inv;
                    *(uint2 *)((uint16_t *)a.out + g * D + d) = make_uint2(to_type(x[0], x[1], T), to_type(x[2], x[3], T));
                } else {
                    *(f32x4 *)(a.part_o + ((int64_t)at.split * a.b.total * a.q_heads + g) * D + d) = x;
                }
            }
            if (part == 0) {
                if (a.splits == 1) {
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

// ---- many rows ------------------------------------------------------------------------------

// A workgroup of 4 waves takes 64 * Cols rows, 16 * Cols a wave, and 64 tokens a turn.  LDS holds
// the operands of two turns, each in the order in which lanes read it, so reads need no swizzle:
//   K: [group 4][step][lane] 16 bytes;  V: [pair of groups 2][tile][half 2][lane] 8 bytes
template <int D, int T, int Cols>
__global__ __launch_bounds__(kLanes, D == 256 || Cols * (T == SPLITZIP_KV4_FP16 ? 2 : 1) > 2 ? 1 : 2) void many_rows(AttendArgs a)
{
    constexpr int kHalves = T == SPLITZIP_KV4_FP16 ? 2 : 1;
    constexpr int kSteps = D / 32, kTiles = D / 16;
    constexpr int kRows = 64 * Cols;
    __shared__ uint4 sh_k[2 * 4 * kSteps * 64];
    __shared__ uint2 sh_v[2 * 2 * kTiles * 2 * 64];
    __shared__ int sh_bad[2][4];     // a wave's group has V that is not finite
    __shared__ int sh_group[2][4];   // its group, -1: none

    const Place at(a);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, quad = lane >> 4;
    fill_unowned<D>(a, at);
    const Seq q = sequence(a.c, a.b, at.s);
    const int rows = q.n * a.group;
    const Mask mask = {a.window, a.sinks};

    // later rows see more tokens: they start first
    const int row_tiles = (rows + kRows - 1) / kRows;
    for (int n = at.tile; n < row_tiles; n += a.tiles) {
        const int row0 = (row_tiles - 1 - n) * kRows;
        const int base = q.len - q.n;
        const Groups groups(base + row0 / a.group, base + min(row0 + kRows - 1, rows - 1) / a.group, a.window, a.sinks);
        int first, last;
        share(groups.count, a.splits, at.split, 4, first, last);

        // this wave's rows; a row past the end repeats the last and is not stored
        const int w_row = row0 + wave * 16 * Cols;
        int query[Cols];
        bf16x8 qf[kHalves][Cols][kSteps];
#pragma unroll
        for (int c = 0; c < Cols; ++c) {
            const int row = min(w_row + 16 * c + r, rows - 1);
            query[c] = base + row / a.group;
            const int64_t p0 = (q.row0 + row / a.group) * a.q_token + (at.head * a.group + row % a.group) * a.q_head +
                               quad * (D / 4);
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                qf[0][c][st] = q_frag<T, 0>(a.q, p0 + 8 * st, a.wide);
                if constexpr (kHalves == 2)
                    qf[1][c][st] = q_frag<T, 1>(a.q, p0 + 8 * st, a.wide);
            }
        }
        const int q_lo = base + min(w_row, rows - 1) / a.group;
        const int q_hi = base + min(w_row + 16 * Cols - 1, rows - 1) / a.group;

        float m[Cols], l[Cols];
        f32x4 o[Cols][kTiles];
#pragma unroll
        for (int c = 0; c < Cols; ++c) {
            m[c] = -INFINITY;
            l[c] = 0.0f;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
                o[c][t] = f32x4{0, 0, 0, 0};
        }

        struct Raw {
            KRaw<D> k;
            VRaw<D> v;
            int g;
        } raw;
        auto fetch = [&](int v) {
            Raw x;
            x.g = v < last ? groups.at(v) : -1;
            const int page = x.g < 0 ? -1 : page_of(a.c, a.b, at.s, 16 * x.g);
            x.k = load_k<D>(a.c, page, at.head, x.g, lane);
            x.v = load_v<D>(a.c, page, at.head, x.g, lane);
            x.g = page < 0 ? -1 : x.g;
            return x;
        };
        auto convert = [&](const Raw &x, int buf) {
            uint4 *k = sh_k + (buf * 4 + wave) * kSteps * 64 + lane;
#pragma unroll
            for (int st = 0; st < kSteps; ++st)
                k[st * 64] = __builtin_bit_cast(uint4, k_frag<D>(x.k, st));
            uint2 *v = sh_v + ((buf * 2 + wave / 2) * kTiles * 2 + wave % 2) * 64 + lane;
#pragma unroll
            for (int t = 0; t < kTiles; t += 2) {
                uint2 lo, hi;
                v_half<D>(x.v, t / 2, lo, hi);
                v[t * 128] = lo;
                v[(t + 1) * 128] = hi;
            }
            const bool bad = __any(v_bad(x.v.s));
            if (lane == 0) {
                sh_bad[buf][wave] = bad;
                sh_group[buf][wave] = x.g;
            }
        };

        if (first < last) {
            raw = fetch(first + wave);
            convert(raw, 0);
            raw = fetch(first + 4 + wave);
        }
        __syncthreads();
        int buf = 0;
        for (int v = first; v < last; v += 4, buf ^= 1) {
            if (v + 4 < last) {
                convert(raw, buf ^ 1);
                raw = fetch(v + 8 + wave);
            }
            int g[4];
            bool whole = true, bad = false, any = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[i] = __builtin_amdgcn_readfirstlane(sh_group[buf][i]);
                whole = whole && g[i] >= 0 && mask.all(g[i], q_lo, q_hi);
                any = any || (g[i] >= 0 && 16 * g[i] <= q_hi);
                bad = bad || __builtin_amdgcn_readfirstlane(sh_bad[buf][i]) != 0;
            }
            if (any) {
                // scores of 64 tokens
                f32x4 x[Cols][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int c = 0; c < Cols; ++c)
                        x[c][i] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int st = 0; st < kSteps; ++st) {
                        const bf16x8 f = __builtin_bit_cast(bf16x8, sh_k[((buf * 4 + i) * kSteps + st) * 64 + lane]);
#pragma unroll
                        for (int c = 0; c < Cols; ++c)
#pragma unroll
                            for (int h = 0; h < kHalves; ++h)
                                x[c][i] = mfma(f, qf[h][c][st], x[c][i]);
                    }
                }
                bf16x8 pf[Cols][2][kHalves];
#pragma unroll
                for (int c = 0; c < Cols; ++c) {
                    float top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float y = x[c][i][e] * a.scale2;
                            if (!whole)
                                y = g[i] >= 0 && mask.sees(query[c], 16 * g[i] + 4 * quad + e) ? y : -INFINITY;
                            x[c][i][e] = y;
                            top = fmaxf(top, y);
                        }
                    top = quad_max(top);
                    if (__any(top > m[c] + 8.0f)) {
                        const float grown = fmaxf(m[c], top);
                        const float f = grown == -INFINITY ? 1.0f : exp2_fast(m[c] - grown);
                        m[c] = grown;
                        l[c] *= f;
#pragma unroll
                        for (int t = 0; t < kTiles; ++t)
                            o[c][t] *= f;
                    }
                    const float ref = m[c] == -INFINITY ? 0.0f : m[c];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float p[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            p[e] = exp2_fast(x[c][2 * h + e / 4][e % 4] - ref);
                            l[c] += p[e];
                        }
                        p_frag<kHalves>(p, pf[c][h]);
                    }
                }
                const bool odd = bad && !whole;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    bf16x8 seen[Cols] = {};
                    if (odd)
#pragma unroll
                        for (int c = 0; c < Cols; ++c)
                            seen[c] = seen_frag(mask, query[c], 16 * g[2 * h] + 4 * quad, 16 * g[2 * h + 1] + 4 * quad,
                                                g[2 * h] >= 0, g[2 * h + 1] >= 0);
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) {
                        const uint2 *v2 = sh_v + ((buf * 2 + h) * kTiles + t) * 128 + lane;
                        const uint2 va = v2[0], vb = v2[64];
#pragma unroll
                        for (int c = 0; c < Cols; ++c)
                            o[c][t] = add_pv<kHalves>(va, vb, pf[c][h], o[c][t], odd, seen[c]);
                    }
                }
            }
            __syncthreads();
        }

#pragma unroll
        for (int c = 0; c < Cols; ++c) {
            const int row = w_row + 16 * c + r;
            const float sum = quad_sum(l[c]);
            if (row >= rows)
                continue;
            const int64_t gr = (q.row0 + row / a.group) * (int64_t)a.q_heads + at.head * a.group + row % a.group;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t = 0; t < kTiles; t += 4) {
                    const int d = (4 * quad + i) * kTiles + t;
                    f32x4 x = {o[c][t][i], o[c][t + 1][i], o[c][t + 2][i], o[c][t + 3][i]};
                    if (a.splits == 1) {
                        x *= inv;
                        *(uint2 *)((uint16_t *)a.out + gr * D + d) = make_uint2(to_type(x[0], x[1], T), to_type(x[2], x[3], T));
                    } else {
                        *(f32x4 *)(a.part_o + ((int64_t)at.split * a.b.total * a.q_heads + gr) * D + d) = x;
                    }
                }
            if (quad == 0) {
                if (a.splits == 1) {
                    if (a.lse)
                        a.lse[gr] = sum == 0.0f ? -INFINITY : (m[c] + __log2f(sum)) * kLn2;
                } else {
                    float *ml = a.part_ml + ((int64_t)at.split * a.b.total * a.q_heads + gr) * 2;
                    ml[0] = m[c];
                    ml[1] = sum;
                }
            }
        }
    }
}

// ---- joining splits -------------------------------------------------------------------------

// D / 4 lanes a row: o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, splits in order.
template <int D, int T>
__global__ __launch_bounds__(kLanes) void join_kernel(AttendArgs a)
{
    const int64_t rows = a.b.total * a.q_heads;
    const int64_t row = (int64_t)blockIdx.x * (kLanes / (D / 4)) + threadIdx.x / (D / 4);
    const int d = threadIdx.x % (D / 4) * 4;
    if (row >= rows)
        return;
    if (sequence_of(a.b, row / a.q_heads) < 0)
        return;                                  // fill_unowned wrote it
    float big = -INFINITY;
    for (int s = 0; s < a.splits; ++s)
        big = fmaxf(big, a.part_ml[(s * rows + row) * 2]);
    float sum = 0.0f;
    f32x4 x = {0, 0, 0, 0};
    for (int s = 0; s < a.splits; ++s) {
        const float m = a.part_ml[(s * rows + row) * 2], l = a.part_ml[(s * rows + row) * 2 + 1];
        // m = -infinity: the split saw nothing, or NaN scores alone, which its sum holds
        const float f = big == -INFINITY ? 1.0f : exp2_fast(m - big);
        sum += l * f;
        x += *(const f32x4 *)(a.part_o + (s * rows + row) * D + d) * f;
    }
    x *= sum == 0.0f ? 0.0f : 1.0f / sum;
    *(uint2 *)((uint16_t *)a.out + row * D + d) = make_uint2(to_type(x[0], x[1], T), to_type(x[2], x[3], T));
    if (d == 0 && a.lse)
        a.lse[row] = sum == 0.0f ? -INFINITY : (big + __log2f(sum)) * kLn2;
}

template <int D, int T>
void attend_dt(const AttendArgs &a, int tile_rows, hipStream_t s)
{
    const unsigned grid = (unsigned)((int64_t)a.b.n_seqs * a.c.heads * a.tiles * a.splits);
    if (tile_rows == 16)
        few_rows<D, T><<<grid, kLanes, 0, s>>>(a);
    else if (tile_rows == 64)
        many_rows<D, T, 1><<<grid, kLanes, 0, s>>>(a);
    else if constexpr (D < 256 || T == SPLITZIP_KV4_BF16)
        many_rows<D, T, 2><<<grid, kLanes, 0, s>>>(a);
    if (a.splits > 1) {
        constexpr int kRows = kLanes / (D / 4);
        join_kernel<D, T><<<(unsigned)((a.b.total * a.q_heads + kRows - 1) / kRows), kLanes, 0, s>>>(a);
    }
}

template <int D>
void attend_d(const AttendArgs &a, int dtype, int tile_rows, hipStream_t s)
{
    if (dtype == SPLITZIP_KV4_BF16)
        attend_dt<D, SPLITZIP_KV4_BF16>(a, tile_rows, s);
    else
        attend_dt<D, SPLITZIP_KV4_FP16>(a, tile_rows, s);
}

}  // namespace

// 16 * Cols rows of 256 channels and two halves would take more than a lane's 512 registers.
int attend_rows(int head_dim, int dtype, int64_t rows)
{
    const int most = head_dim == 256 && dtype == SPLITZIP_KV4_FP16 ? 64 : 128;
    return rows <= 16 ? 16 : rows <= 64 ? 64 : most;
}

void launch_attend(const AttendArgs &a, int head_dim, int dtype, int tile_rows, hipStream_t s)
{
    head_dim == 64    ? attend_d<64>(a, dtype, tile_rows, s)
    : head_dim == 128 ? attend_d<128>(a, dtype, tile_rows, s)
                      : attend_d<256>(a, dtype, tile_rows, s);
}

}  // namespace kv4
}  // namespace sz
