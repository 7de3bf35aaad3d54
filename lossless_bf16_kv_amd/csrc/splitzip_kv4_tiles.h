// splitzip_kv4_tiles.h -- device code shared by the attention and weight kernels of the 4-bit KV
// cache: groups of 16 tokens, which of them a block of queries sees, and their conversion to
// matrix operands.
//
// Operands of v_mfma_f32_16x16x32_bf16, of lane l with r = l % 16 and quad = l / 16:
//   A (16 x 32): row r, columns 8 quad .. + 7;  B (32 x 16): column r, rows 8 quad .. + 7
//   result (16 x 16): rows 4 quad .. + 3, column r
// The order in which the 32 terms of a sum are given is free as long as A and B agree, and that
// makes both products readable straight from the cache:
//   scores: the sum runs over channels.  A lane holds the D / 4 adjacent channels
//     quad * D / 4 .. of token r, 8 of them a step: for D = 128 one 16-byte load and one scale.
//   values: the sum runs over 32 tokens, two groups.  The scores' result already gives a lane
//     tokens 4 quad .. + 3 of each group for one query, and V's layout gives it, for the same
//     four tokens, D / 16 adjacent channels; channel r * D / 16 + t is row r of result tile t.
//     So probabilities never leave their lane and V needs no transposition through memory.
// v_mfma_f32_32x32x16_bf16 (half = l / 32): A row and B column l % 32, terms 8 half .. + 7; result
//   rows 8 i + 4 half .. + 3 (i < 4) of column l % 32.
#pragma once

#include "splitzip_kv4_internal.h"

namespace sz {
namespace kv4 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// x of the other 16-lane rows: the largest (sum) over the four lanes l % 16 = r.
__device__ __forceinline__ float quad_max(float x)
{
    auto a = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
    x = fmaxf(as_float(a[0]), as_float(a[1]));
    auto b = __builtin_amdgcn_permlane16_swap(bits(x), bits(x), false, false);
    return fmaxf(as_float(b[0]), as_float(b[1]));
}

__device__ __forceinline__ float quad_sum(float x)
{
    auto a = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
    x = as_float(a[0]) + as_float(a[1]);
    auto b = __builtin_amdgcn_permlane16_swap(bits(x), bits(x), false, false);
    return as_float(b[0]) + as_float(b[1]);
}

__device__ __forceinline__ bf16x8 frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 v = {a, b, c, d};
    return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float half_max(float x)       // over lanes l and l ^ 32
{
    auto a = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
    return fmaxf(as_float(a[0]), as_float(a[1]));
}

__device__ __forceinline__ float half_sum(float x)
{
    auto a = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
    return as_float(a[0]) + as_float(a[1]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The groups of 16 tokens that queries at tokens lo .. hi of one sequence see, in token order:
// first those of the always visible tokens, then those from the window's start to hi.
struct Groups {
    int lead, skip, count;       // group v is v for v < lead, else v + skip

    __device__ Groups(int lo, int hi, int window, int sinks)
    {
        if (hi < 0) {
            lead = skip = count = 0;
            return;
        }
        const int from = window > 0 && lo >= window ? (lo - window + 1) >> 4 : 0;
        lead = min((sinks >> 4) + ((sinks & 15) != 0), from);
        skip = from - lead;
        count = (hi >> 4) + 1 - skip;
    }
    __device__ int at(int v) const { return v < lead ? v : v + skip; }
};

// Pages of the groups first, first + step, .. of a wave, below `last`: 64 at a time, one a lane.  A page
// looked up when its tokens are wanted would hold up the loads behind it by a load's time.
struct Pages {
    int list, from;              // lane i: page of step from + i
    __device__ Pages() : list(-1), from(-64) {}
    // Page of group first + i * step, or -1: none, or a bad page.  i grows by one from call to call.
    __device__ int at(const Cache &c, const Batch &b, int s, const Groups &groups, int first, int step, int last, int i)
    {
        if (i >= from + 64) {
            from = i;
            const int64_t v = first + (int64_t)(i + (int)(threadIdx.x & 63)) * step;
            list = v < last ? page_of(c, b, s, 16 * groups.at((int)v)) : -1;
        }
        return __builtin_amdgcn_readlane(list, i - from);
    }
};

// Which tokens queries lo .. hi see.  No short circuits: branches would cost more than the comparisons.
struct Mask {
    int window, sinks;
    __device__ bool sees(int query, int j) const
    {
        return (j <= query) & ((j < sinks) | (window == 0) | (j > query - window));
    }
    // every query of lo .. hi sees every token of group g
    __device__ int all(int g, int lo, int hi) const
    {
        const int j = 16 * g;
        return (j + 15 <= lo) & ((j + 15 < sinks) | (window == 0) | (j > hi - window));
    }
};

// One lane's part of a group's K: D / 8 bytes of codes (channels quad * D / 4 .. of token r) and
// their scales; of its V: runs r of tokens 4 quad .. + 3 and the scales of those tokens.
template <int D>
struct KRaw {
    uint32_t w[D / 32];
    uint32_t s;
};
template <int D>
struct VRaw {
    uint32_t w[D / 32];
    uint32_t s;
};

template <int D>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[D / 32])
{
    if constexpr (D == 64) {
        const uint2 t = *(const uint2 *)p;
        w[0] = t.x; w[1] = t.y;
    } else {
#pragma unroll
        for (int i = 0; i < D / 128; ++i) {
            const uint4 t = *(const uint4 *)(p + 16 * i);
            w[4 * i] = t.x; w[4 * i + 1] = t.y; w[4 * i + 2] = t.z; w[4 * i + 3] = t.w;
        }
    }
}

// Element offset (tokens) of group g of a page and head.
__device__ __forceinline__ int64_t group_first(const Cache &c, int page, int head, int g)
{
    const int64_t p = page < 0 ? 0 : page;
    return (((p * c.heads + head) << c.page_shift) | ((g << 4) & ((1 << c.page_shift) - 1)));
}

// Page and group are the wave's, so an address is a scalar base and a lane's 32-bit offset.  The empty
// asm keeps the compiler from adding the offset to the buffer's start outside of the loop, which
// would cost a 64-bit vector addition a load.
__device__ __forceinline__ const uint8_t *lane_at(const uint8_t *base, uint32_t offset)
{
    asm volatile("" : "+v"(offset));
    return base + offset;
}

template <int D>
__device__ __forceinline__ KRaw<D> load_k(const Cache &c, int page, int head, int g, int lane)
{
    const uint32_t r = lane & 15, quad = lane >> 4;
    const int64_t t = group_first(c, page, head, g);
    KRaw<D> k;
    load_words<D>(lane_at(c.k_codes + t * (D / 2), r * (D / 2) + quad * (D / 8)), k.w);
    const uint8_t *s = c.k_scales + t * (D / 32);
    if constexpr (D == 64)
        k.s = *lane_at(s, r * 2 + (quad >> 1));
    else if constexpr (D == 128)
        k.s = *lane_at(s, r * 4 + quad);
    else
        k.s = *(const uint16_t *)lane_at(s, r * 8 + 2 * quad);
    return k;
}

// quad: which four tokens of the group.
template <int D>
__device__ __forceinline__ VRaw<D> load_v(const Cache &c, int page, int head, int g, int lane, uint32_t quad)
{
    const uint32_t r = lane & 15;
    const int64_t t = group_first(c, page, head, g), page0 = t >> c.page_shift << c.page_shift;
    VRaw<D> v;
    load_words<D>(lane_at(c.v_codes + t * (D / 2), quad * (2 * D) + r * (D / 8)), v.w);
    const uint8_t *s = c.v_scales + page0 * (D / 32) + (t - page0);
    v.s = *(const uint32_t *)lane_at(s, (r * (D / 16) / 32 << c.page_shift) + 4 * quad);
    return v;
}

// ---- loads to LDS ---------------------------------------------------------------------------
// They need no registers while they are on their way.  A wave waits for them by count, in assembly
// that also reads them: the compiler would wait for all of them before any read of LDS.
typedef __attribute__((address_space(1))) const void *global_ptr;
typedef __attribute__((address_space(3))) void *lds_ptr;

// 16 or 4 bytes a lane, in lane order.
__device__ __forceinline__ void to_lds16(const uint8_t *from, uint8_t *to)
{
    __builtin_amdgcn_global_load_lds((global_ptr)from, (lds_ptr)to, 16, 0, 0);
}

__device__ __forceinline__ void to_lds4(const uint8_t *from, uint8_t *to)
{
    __builtin_amdgcn_global_load_lds((global_ptr)from, (lds_ptr)to, 4, 0, 0);
}

// K operand of step st: channels quad * D / 4 + 8 st .. + 7 of token r.
template <int D>
__device__ __forceinline__ bf16x8 k_frag(const KRaw<D> &k, int st)
{
    const float s = scale_of(D == 256 ? (st < 4 ? k.s & 0xff : k.s >> 8) : k.s);
    const uint32_t w = k.w[st];
    return frag(dequant<0>(w, s), dequant<1>(w, s), dequant<2>(w, s), dequant<3>(w, s));
}

// Channels 2 p and 2 p + 1 of lane's run, of its token i.
template <int D>
__device__ __forceinline__ uint32_t v_pair(const VRaw<D> &v, int i, int p)
{
    const float s = scale_of((v.s >> (8 * i)) & 0xff);
    if constexpr (D == 64) {
        const uint32_t w = v.w[i >> 1];
        switch ((i & 1) * 2 + p) {
        case 0: return dequant<0>(w, s);
        case 1: return dequant<1>(w, s);
        case 2: return dequant<2>(w, s);
        default: return dequant<3>(w, s);
        }
    } else {
        const uint32_t w = v.w[i * (D / 128) + (p >> 2)];
        switch (p & 3) {
        case 0: return dequant<0>(w, s);
        case 1: return dequant<1>(w, s);
        case 2: return dequant<2>(w, s);
        default: return dequant<3>(w, s);
        }
    }
}

// The lane's four tokens of channel 2 p (lo) and 2 p + 1 (hi) of its run: half of the V operands
// of tiles 2 p and 2 p + 1.
template <int D>
__device__ __forceinline__ void v_half(const VRaw<D> &v, int p, uint2 &lo, uint2 &hi)
{
    const uint32_t a = v_pair<D>(v, 0, p), b = v_pair<D>(v, 1, p), c = v_pair<D>(v, 2, p), d = v_pair<D>(v, 3, p);
    lo.x = __builtin_amdgcn_perm(b, a, 0x05040100);
    hi.x = __builtin_amdgcn_perm(b, a, 0x07060302);
    lo.y = __builtin_amdgcn_perm(d, c, 0x05040100);
    hi.y = __builtin_amdgcn_perm(d, c, 0x07060302);
}

// A product of a V that is not finite with a probability of 0 is a NaN also for queries that do not
// see it.  Where that may happen the values are taken out (no_nan), and the queries that do see one get
// their NaN from poison.  A scale byte past 252 makes its 32 channels so.
__device__ __forceinline__ bool v_bad(uint32_t s)
{
    return (s & 0xff) > 252 || ((s >> 8) & 0xff) > 252 || ((s >> 16) & 0xff) > 252 || (s >> 24) > 252;
}

template <int D>
__device__ __forceinline__ void no_nan(VRaw<D> &v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (((v.s >> (8 * i)) & 0xff) <= 252)
            continue;
        v.s &= ~(0xffu << (8 * i));
        if constexpr (D == 64) {
            v.w[i >> 1] &= i & 1 ? 0xffffu : 0xffff0000u;
        } else {
#pragma unroll
            for (int k = 0; k < D / 128; ++k)
                v.w[i * (D / 128) + k] = 0;
        }
    }
}

// Bit b: the query sees a token of group g whose block b of V is not finite.
template <int D>
__device__ __forceinline__ uint32_t poison(const Cache &c, const Batch &b, int s, int head, int g, const Mask &mask, int query)
{
    const int page = g < 0 ? -1 : page_of(c, b, s, 16 * g);
    if (page < 0)
        return 0;
    const int64_t t0 = group_first(c, page, head, g), page0 = t0 >> c.page_shift << c.page_shift;
    uint32_t bits = 0;
#pragma unroll 1
    for (int t = 0; t < 16; ++t) {
        if (!mask.sees(query, 16 * g + t))
            continue;
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k)
            bits |= (c.v_scales[page0 * (D / 32) + ((int64_t)k << c.page_shift) + (t0 - page0) + t] > 252 ? 1u : 0u) << k;
    }
    return bits;
}

// Eight channels of a query as bf16 (Half 0: the leading bits, 1: what an fp16 value has beyond
// them, exact in 3 bits).  bf16 queries have one half.
template <int T, int Half>
__device__ __forceinline__ bf16x8 q_frag(const void *q, int64_t at, bool wide)
{
    const uint16_t *h = (const uint16_t *)q + at;
    uint32_t w[4];
    if (wide) {
        const uint4 t = *(const uint4 *)h;
        w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (uint32_t)h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
    }
    if constexpr (T == SPLITZIP_KV4_FP16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = fp16_of(w[i]), b = fp16_of(w[i] >> 16);
            const uint32_t top = pack_bf16(a, b);
            // an infinity stays in the leading half alone: its difference would be a NaN
            const float x = a - bf16_lo(top), y = b - bf16_hi(top);
            w[i] = Half == 0 ? top : pack_bf16(x == x ? x : 0.0f, y == y ? y : 0.0f);
        }
    }
    return frag(w[0], w[1], w[2], w[3]);
}

}  // namespace kv4
}  // namespace sz
