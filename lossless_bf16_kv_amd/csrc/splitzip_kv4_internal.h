// splitzip_kv4_internal.h -- the 4-bit KV cache's kernel arguments and device helpers: where a
// token lies, which tokens a query sees, the block format and its conversions.
#pragma once

#include "splitzip_internal.h"
#include "splitzip_kv4.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sz {
namespace kv4 {

struct Cache {
    uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    float *weights;
    uint32_t *status;
    int64_t num_pages;
    int32_t page_shift;      // log2 of the page size
    int32_t heads;
};

struct Batch {
    const int32_t *table, *lens, *cu;
    int64_t table_stride, total;
    int32_t table_width, n_seqs;
};

struct AppendArgs {
    Cache c;
    Batch b;
    const void *k, *v;
    int64_t k_token, k_head, v_token, v_head;
    int32_t wide;            // 16-byte loads fit pointers and strides
};

struct ReadArgs {
    Cache c;
    Batch b;
    void *k, *v;
};

struct AttendArgs {
    Cache c;
    Batch b;
    const void *q;
    int64_t q_token, q_head;
    int32_t q_heads, group;  // query heads, and of them to a KV head
    int32_t window, sinks;
    float scale2;            // scale * log2(e): scores are held as powers of two
    int32_t wide;
    void *out;
    float *lse;
    const float *lse_in;     // weigh
    float *part_o, *part_ml; // partial results of splits > 1: [split][row][D], [split][row][2]
    int32_t splits, tiles;   // workgroups along the tokens and along the rows of a sequence and head
    int32_t per, tile_rows;  // attend: groups of 16 tokens a split, rows a tile
    // weigh: workgroups along the tokens of rows_kernel (`splits`: of step_kernel; 0: not launched), and how many rows
    // a sequence has at most that is left to step_kernel
    int32_t row_splits, step_rows;
};

struct EvictArgs {
    Cache c;
    Batch b;
    const int32_t *out_table;
    int64_t out_stride;
    int32_t out_width;
    int32_t budget, sinks, recent;
    int32_t *out_lens, *kept;
    int32_t turns;           // workgroups of move_kernel a sequence and head
};

// HIP launches fewer than 2^32 threads at a time.
constexpr int64_t kMostThreads = UINT32_MAX;
constexpr int kRowThreads = 256, kChooseThreads = 1024, kMoveThreads = 256, kMoveTokens = 128;

void launch_append(const AppendArgs &a, int head_dim, int dtype, hipStream_t s);
void launch_read(const ReadArgs &a, int head_dim, int dtype, hipStream_t s);
int attend_rows(int head_dim, int64_t rows);   // rows of a workgroup for this many rows a sequence
int attend_threads(int head_dim, int tile_rows);
int join_rows(int head_dim);                   // rows of a workgroup of join_kernel
constexpr int kJoinThreads = 256, kWeighThreads = 256, kStepRows = 16;
constexpr int weigh_tokens(int head_dim) { return head_dim == 256 ? 128 : 256; }     // of a workgroup of rows_kernel
hipError_t launch_attend(const AttendArgs &a, int head_dim, int dtype, hipStream_t s);
hipError_t launch_weigh(const AttendArgs &a, int head_dim, int dtype, hipStream_t s);
hipError_t launch_evict(const EvictArgs &a, int head_dim, hipStream_t s);

// ---- device ---------------------------------------------------------------------------------
#ifdef __HIPCC__
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ float as_float(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ float bf16_lo(uint32_t x) { return as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return as_float(x & 0xffff0000u); }

// Two floats to bf16, nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ uint32_t pack_fp16(float a, float b)
{
    const _Float16 x = (_Float16)a, y = (_Float16)b;
    return (uint32_t)__builtin_bit_cast(uint16_t, x) | (uint32_t)__builtin_bit_cast(uint16_t, y) << 16;
}

__device__ __forceinline__ float fp16_of(uint32_t h) { return (float)__builtin_bit_cast(_Float16, (uint16_t)h); }

// Byte Sel of `codes` (two E2M1 codes) times 2^(scale byte - 127), as two bf16: exact for every
// scale the format writes; a scale byte of 255 gives NaN.
template <int Sel>
__device__ __forceinline__ uint32_t dequant(uint32_t codes, float scale)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, Sel));
}

__device__ __forceinline__ float scale_of(uint32_t byte) { return as_float(byte << 23); }

__device__ __forceinline__ void flag(const Cache &c, uint32_t bit) { atomicOr(c.status, bit); }

// A sequence's tokens and rows.
struct Seq {
    int len;         // tokens, cut to the table
    int row0, n;     // its rows in the call's tensors
};

__device__ __forceinline__ int row_offset(const Batch &b, int s)
{
    const int64_t x = b.cu[s];
    return (int)(x < 0 ? 0 : x > b.total ? b.total : x);
}

__device__ __forceinline__ Seq sequence(const Cache &c, const Batch &b, int s)
{
    Seq q;
    const int64_t cap = (int64_t)b.table_width << c.page_shift;
    const int len = b.lens[s];
    q.len = len < 0 ? 0 : len > cap ? (int)cap : len;
    if (q.len != len)
        flag(c, SPLITZIP_KV4_BAD_LENGTH);
    if (b.cu) {
        q.row0 = row_offset(b, s);
        q.n = row_offset(b, s + 1) - q.row0;
        if (q.n < 0 || b.cu[s] != q.row0 || b.cu[s + 1] != q.row0 + q.n)
            flag(c, SPLITZIP_KV4_BAD_OFFSETS);
        q.n = q.n < 0 ? 0 : q.n;
    } else {
        q.row0 = s;
        q.n = s < b.total ? 1 : 0;
    }
    return q;
}

// The same for a sequence that a whole wave shares, in scalar registers: loads behind a store go to
// vector ones, and every loop bound that follows from them would.
__device__ __forceinline__ Seq wave_sequence(const Cache &c, const Batch &b, int s)
{
    Seq q = sequence(c, b, s);
    q.len = __builtin_amdgcn_readfirstlane(q.len);
    q.row0 = __builtin_amdgcn_readfirstlane(q.row0);
    q.n = __builtin_amdgcn_readfirstlane(q.n);
    return q;
}

// Sequence of row i, or -1: the last s with cu[s] <= i, if i < cu[s + 1].
__device__ __forceinline__ int sequence_of(const Batch &b, int64_t i)
{
    if (!b.cu)
        return i < b.n_seqs ? (int)i : -1;
    int lo = 0, hi = b.n_seqs;           // cu[lo] <= i < cu[hi] if any
    if (b.n_seqs == 0 || i < b.cu[0] || i >= b.cu[b.n_seqs])
        return -1;
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        (b.cu[mid] <= i ? lo : hi) = mid;
    }
    return lo;
}

// Page of token j (of a sequence of len > j tokens), or -1.
__device__ __forceinline__ int page_of(const Cache &c, const Batch &b, int s, int j)
{
    const int p = b.table[(int64_t)s * b.table_stride + (j >> c.page_shift)];
    if (p < 0 || p >= c.num_pages) {
        flag(c, SPLITZIP_KV4_BAD_PAGE);
        return -1;
    }
    return p;
}
#endif

}  // namespace kv4
}  // namespace sz
