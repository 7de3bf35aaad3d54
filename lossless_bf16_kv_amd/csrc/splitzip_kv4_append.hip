// splitzip_kv4_append.hip -- tokens into the 4-bit KV cache and back.
//
// Quantization of a block x[0..31] (one token, head and 32 channels):
//
//   amax = max |x| = m 2^E, 1 <= m < 2        from the bits: the largest |x| as an integer, so
//                                             a NaN or an infinity is found with it
//   e    = E - 2 + [m >= 1.75]                the smallest e with amax / 2^e < 7
//   code = nearest of 0 .5 1 1.5 2 3 4 6 to |x| / 2^e, ties to even, with x's sign
//
// Division by 2^e is exact, so each value is rounded once.  v_cvt_scalef32_pk_fp4_f32 does the
// division, the rounding and the packing of two values in one instruction.
//
// Both kernels are bound by HBM: 4 bytes of BF16 K and V to 1.06 bytes of cache and back.  A
// lane holds 8 channels (one 16-byte load) of K and of V, four lanes share a block.  A workgroup
// takes 256 * 8 / D consecutive rows of one head, so that the four tokens interleaved in V's
// layout are written by one workgroup and meet in one L2.  32768 tokens of 8 heads of 128 channels:
// append 45 us (171 MB, 3.8 TB/s: K and V are slices of a fused projection here, half of every 8 KiB),
// read 27 us (170 MB, 6.3 TB/s).  Four rows a lane, all loads first, took append 46 us.
#include "splitzip_kv4_internal.h"

namespace sz {
namespace kv4 {
namespace {

constexpr int kLanes = kRowThreads;

__device__ __forceinline__ void load8(const void *p, int64_t at, int dtype, bool wide, float (&x)[8])
{
    if (dtype == SPLITZIP_KV4_FP32) {
        const float *f = (const float *)p + at;
        if (wide) {
            const f32x4 a = *(const f32x4 *)f, b = *(const f32x4 *)(f + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = a[i];
                x[4 + i] = b[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = f[i];
        }
        return;
    }
    const uint16_t *h = (const uint16_t *)p + at;
    uint32_t w[4];
    if (wide) {
        const uint4 t = *(const uint4 *)h;
        w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (uint32_t)h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = dtype == SPLITZIP_KV4_BF16 ? bf16_lo(w[i]) : fp16_of(w[i]);
        x[2 * i + 1] = dtype == SPLITZIP_KV4_BF16 ? bf16_hi(w[i]) : fp16_of(w[i] >> 16);
    }
}

// Eight values to eight codes; `byte`: the scale of the block that four neighbouring lanes share.
__device__ __forceinline__ uint32_t quantize8(const float (&x)[8], uint32_t &byte)
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = max(top, bits(x[i]) & 0x7fffffffu);
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xb1, 0xf, 0xf, true));   // lane ^ 1
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4e, 0xf, 0xf, true));   // lane ^ 2
    const int e = (int)(top >> 23) - 2 + ((top & 0x7fffffu) >= 0x600000u ? 1 : 0);
    if (top >= 0x7f800000u) {
        byte = 255;
        return 0;
    }
    byte = (uint32_t)min(max(e, 2), 252);
    const float scale = scale_of(byte);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
    return w;
}

// Where channels 8 * lane .. + 7 of the token at place t of its page lie in a page's V codes of
// one head: runs of D / 16 channels, four tokens of each run side by side.
template <int D>
__device__ __forceinline__ uint32_t v_offset(int t, int lane)
{
    constexpr int kRun = D / 32;                 // bytes of a token's run
    const int byte = 4 * lane;                   // of the token's D / 2
    return (uint32_t)((t >> 2) * (2 * D) + byte / kRun * (4 * kRun) + (t & 3) * kRun + byte % kRun);
}

template <int D, int T>
__global__ __launch_bounds__(kLanes) void append_kernel(AppendArgs a)
{
    constexpr int kRow = D / 8;                  // lanes of a row
    constexpr int kRows = kLanes / kRow;
    const int lane = threadIdx.x % kRow;
    const int head = blockIdx.x % a.c.heads;
    const int64_t i = (int64_t)(blockIdx.x / a.c.heads) * kRows + threadIdx.x / kRow;
    if (i >= a.b.total)
        return;
    const int s = sequence_of(a.b, i);
    if (s < 0)
        return;
    float k[8], v[8];
    load8(a.k, i * a.k_token + head * a.k_head + 8 * lane, T, a.wide, k);
    load8(a.v, i * a.v_token + head * a.v_head + 8 * lane, T, a.wide, v);
    const Seq q = sequence(a.c, a.b, s);
    const int j = q.len - q.n + (int)(i - q.row0);
    if (j < 0 || j >= q.len)
        return;
    const int page = page_of(a.c, a.b, s, j);
    if (page < 0)
        return;
    const int t = j & ((1 << a.c.page_shift) - 1);
    const int64_t first = ((int64_t)page * a.c.heads + head) << a.c.page_shift;   // token 0 of this page and head
    uint32_t kb, vb;
    const uint32_t kw = quantize8(k, kb), vw = quantize8(v, vb);
    *(uint32_t *)(a.c.k_codes + (first + t) * (D / 2) + 4 * lane) = kw;
    uint8_t *vd = a.c.v_codes + first * (D / 2) + v_offset<D>(t, lane);
    if (D >= 128) {
        *(uint32_t *)vd = vw;
    } else {                                     // D = 64: two runs of 2 bytes
        *(uint16_t *)vd = (uint16_t)vw;
        *(uint16_t *)(vd + 8) = (uint16_t)(vw >> 16);
    }
    if (lane % 4 == 0) {
        a.c.k_scales[(first + t) * (D / 32) + lane / 4] = (uint8_t)kb;
        a.c.v_scales[first * (D / 32) + ((int64_t)(lane / 4) << a.c.page_shift) + t] = (uint8_t)vb;
    }
    if (lane == 0)
        a.c.weights[first + t] = 0.0f;
}

// Eight values from eight codes, in the type T.
template <int T>
__device__ __forceinline__ void store8(void *p, int64_t at, uint32_t codes, float scale)
{
    const uint32_t w[4] = {dequant<0>(codes, scale), dequant<1>(codes, scale), dequant<2>(codes, scale),
                           dequant<3>(codes, scale)};
    if (T == SPLITZIP_KV4_BF16) {
        *(uint4 *)((uint16_t *)p + at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (T == SPLITZIP_KV4_FP16) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = pack_fp16(bf16_lo(w[i]), bf16_hi(w[i]));
        *(uint4 *)((uint16_t *)p + at) = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
        f32x4 x = {bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
        f32x4 y = {bf16_lo(w[2]), bf16_hi(w[2]), bf16_lo(w[3]), bf16_hi(w[3])};
        *(f32x4 *)((float *)p + at) = x;
        *(f32x4 *)((float *)p + at + 4) = y;
    }
}

template <int D, int T>
__global__ __launch_bounds__(kLanes) void read_kernel(ReadArgs a)
{
    constexpr int kRow = D / 8;
    constexpr int kRows = kLanes / kRow;
    const int lane = threadIdx.x % kRow;
    const int head = blockIdx.x % a.c.heads;
    const int64_t i = (int64_t)(blockIdx.x / a.c.heads) * kRows + threadIdx.x / kRow;
    if (i >= a.b.total)
        return;
    uint32_t kw = 0, vw = 0, kb = 255, vb = 255;
    const int s = sequence_of(a.b, i);
    if (s >= 0) {
        const Seq q = sequence(a.c, a.b, s);
        const int j = q.len - q.n + (int)(i - q.row0);
        const int page = j < 0 || j >= q.len ? -1 : page_of(a.c, a.b, s, j);
        if (page >= 0) {
            const int t = j & ((1 << a.c.page_shift) - 1);
            const int64_t first = ((int64_t)page * a.c.heads + head) << a.c.page_shift;
            kw = *(const uint32_t *)(a.c.k_codes + (first + t) * (D / 2) + 4 * lane);
            const uint8_t *vd = a.c.v_codes + first * (D / 2) + v_offset<D>(t, lane);
            vw = D >= 128 ? *(const uint32_t *)vd
                          : (uint32_t)*(const uint16_t *)vd | (uint32_t)*(const uint16_t *)(vd + 8) << 16;
            kb = a.c.k_scales[(first + t) * (D / 32) + lane / 4];
            vb = a.c.v_scales[first * (D / 32) + ((int64_t)(lane / 4) << a.c.page_shift) + t];
        }
    }
    const int64_t at = (i * a.c.heads + head) * D + 8 * lane;
    store8<T>(a.k, at, kw, scale_of(kb));
    store8<T>(a.v, at, vw, scale_of(vb));
}

template <int D>
unsigned row_grid(const Cache &c, const Batch &b)
{
    constexpr int kRows = kLanes / (D / 8);
    return (unsigned)((b.total + kRows - 1) / kRows * c.heads);
}

template <int D>
void append_d(const AppendArgs &a, int dtype, hipStream_t s)
{
    const unsigned g = row_grid<D>(a.c, a.b);
    if (dtype == SPLITZIP_KV4_BF16)
        append_kernel<D, SPLITZIP_KV4_BF16><<<g, kLanes, 0, s>>>(a);
    else if (dtype == SPLITZIP_KV4_FP16)
        append_kernel<D, SPLITZIP_KV4_FP16><<<g, kLanes, 0, s>>>(a);
    else
        append_kernel<D, SPLITZIP_KV4_FP32><<<g, kLanes, 0, s>>>(a);
}

template <int D>
void read_d(const ReadArgs &a, int dtype, hipStream_t s)
{
    const unsigned g = row_grid<D>(a.c, a.b);
    if (dtype == SPLITZIP_KV4_BF16)
        read_kernel<D, SPLITZIP_KV4_BF16><<<g, kLanes, 0, s>>>(a);
    else if (dtype == SPLITZIP_KV4_FP16)
        read_kernel<D, SPLITZIP_KV4_FP16><<<g, kLanes, 0, s>>>(a);
    else
        read_kernel<D, SPLITZIP_KV4_FP32><<<g, kLanes, 0, s>>>(a);
}

}  // namespace

void launch_append(const AppendArgs &a, int head_dim, int dtype, hipStream_t s)
{
    head_dim == 64 ? append_d<64>(a, dtype, s) : head_dim == 128 ? append_d<128>(a, dtype, s) : append_d<256>(a, dtype, s);
}

void launch_read(const ReadArgs &a, int head_dim, int dtype, hipStream_t s)
{
    head_dim == 64 ? read_d<64>(a, dtype, s) : head_dim == 128 ? read_d<128>(a, dtype, s) : read_d<256>(a, dtype, s);
}

}  // namespace kv4
}  // namespace sz
