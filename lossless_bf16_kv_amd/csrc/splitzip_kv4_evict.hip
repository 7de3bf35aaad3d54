// splitzip_kv4_evict.hip -- cutting sequences of the 4-bit KV cache to the tokens that attention
// has used.  For each sequence longer than the budget and each KV head: its first `sinks` and last
// `recent` tokens stay, and of the others the `room` = budget - sinks - recent with the largest
// weights, equal ones in token order.
//
// choose_kernel finds the kept tokens, one workgroup a sequence and head.  Weights become 32-bit
// keys that order as the weights do; the room-th largest key is found 8 bits at a time from counts
// of the keys that share its leading bits, and one ordered pass writes the tokens: those above it
// and the first of those equal to it.  Counts are sums of integers, so nothing depends on the
// order of atomics.  move_kernel then gathers codes, scales and weights; its bytes bound it.
#include "splitzip_kv4_internal.h"

namespace sz {
namespace kv4 {
namespace {

constexpr int kChoose = 1024;
constexpr int kMove = 256;

// Larger weight, larger key; NaN 0, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float w)
{
    if (w != w)
        return 0;
    const uint32_t u = bits(w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int wave_scan(int x)         // inclusive
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(x, d);
        x += lane >= d ? y : 0;
    }
    return x;
}

__global__ __launch_bounds__(kChoose) void choose_kernel(EvictArgs a)
{
    __shared__ int sh_count[256];
    __shared__ uint32_t sh_prefix;
    __shared__ int sh_left;
    __shared__ int sh_above[16], sh_equal[16];
    const int head = blockIdx.x % a.c.heads, s = blockIdx.x / a.c.heads;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Batch b = a.b;
    b.cu = nullptr;
    const Seq q = sequence(a.c, b, s);
    const int64_t cap = (int64_t)a.out_width << a.c.page_shift;
    int *const kept = a.kept + ((int64_t)s * a.c.heads + head) * a.budget;
    const int keep = min(q.len, a.budget);
    if (head == 0 && tid == 0) {
        if (keep > cap)
            flag(a.c, SPLITZIP_KV4_BAD_LENGTH);
        a.out_lens[s] = (int)min((int64_t)keep, cap);
    }
    for (int i = keep + tid; i < a.budget; i += kChoose)
        kept[i] = -1;
    if (q.len <= a.budget) {
        for (int i = tid; i < q.len; i += kChoose)
            kept[i] = i;
        return;
    }
    auto weight_key = [&](int j) {
        const int page = page_of(a.c, a.b, s, j);
        return page < 0 ? 0u
                        : key_of(a.c.weights[(((int64_t)page * a.c.heads + head) << a.c.page_shift) +
                                             (j & ((1 << a.c.page_shift) - 1))]);
    };
    const int lo = a.sinks, hi = q.len - a.recent;          // tokens that compete
    const int room = a.budget - a.sinks - a.recent;
    // sh_prefix: leading bits of the room-th largest key; sh_left: how many of the keys with those
    // bits are kept
    if (tid == 0) {
        sh_prefix = 0;
        sh_left = room;
    }
    for (int shift = 24; shift >= 0 && room > 0; shift -= 8) {
        if (tid < 256)
            sh_count[tid] = 0;
        __syncthreads();
        const uint32_t prefix = sh_prefix;
        for (int j = lo + tid; j < hi; j += kChoose) {
            const uint32_t k = weight_key(j);
            if (shift == 24 || k >> (shift + 8) == prefix >> (shift + 8))
                atomicAdd(&sh_count[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (wave == 0) {
            // lane l holds bins 255 - 4 l .. 252 - 4 l: from the largest down
            int c[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sum += c[i] = sh_count[255 - 4 * lane - i];
            const int before = wave_scan(sum) - sum, left = sh_left;
            if (before < left && left <= before + sum) {
                int seen = before, i = 0;
                while (seen + c[i] < left)
                    seen += c[i++];
                sh_prefix = prefix | (uint32_t)(255 - 4 * lane - i) << shift;
                sh_left = left - seen;
            }
        }
        __syncthreads();
    }
    __syncthreads();
    const uint32_t border = sh_prefix;
    const int equal_room = sh_left;
    int above0 = 0, equal0 = 0;                             // kept above, and equal keys, before this turn
    for (int j0 = 0; j0 < q.len; j0 += kChoose) {
        const int j = j0 + tid;
        const bool in = j < q.len, fixed = in && (j < lo || j >= hi);
        const uint32_t k = in && !fixed && room > 0 ? weight_key(j) : 0;
        const bool above = fixed || (in && !fixed && room > 0 && k > border);
        const bool equal = in && !fixed && room > 0 && k == border;
        const uint64_t ab = __ballot(above), eq = __ballot(equal);
        __syncthreads();                                    // the turn before has read the counts
        if (lane == 0) {
            sh_above[wave] = __popcll(ab);
            sh_equal[wave] = __popcll(eq);
        }
        __syncthreads();
        int a_at = above0, e_at = equal0, a_all = 0, e_all = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            a_at += w < wave ? sh_above[w] : 0;
            e_at += w < wave ? sh_equal[w] : 0;
            a_all += sh_above[w];
            e_all += sh_equal[w];
        }
        const uint64_t below = (1ull << lane) - 1;
        a_at += __popcll(ab & below);
        e_at += __popcll(eq & below);
        if (above || (equal && e_at < equal_room))
            kept[a_at + min(e_at, equal_room)] = j;
        above0 += a_all;
        equal0 += e_all;
    }
}

// 16 tokens of one sequence and head a turn.
template <int D>
__global__ __launch_bounds__(kMove) void move_kernel(EvictArgs a)
{
    __shared__ int64_t sh_from[16];          // token's element offset in its page and head, -1: none
    __shared__ int64_t sh_page0[16];
    const int turns = (a.budget + 15) / 16;
    const int turn = blockIdx.x % turns;
    uint32_t b = blockIdx.x / turns;
    const int head = b % a.c.heads, s = b / a.c.heads;
    const int tid = threadIdx.x;
    Batch bt = a.b;
    bt.cu = nullptr;
    const int keep = min(sequence(a.c, bt, s).len, a.budget);
    const int to0 = turn * 16;
    if (to0 >= keep || to0 >= (int64_t)a.out_width << a.c.page_shift)
        return;
    const int out_page = a.out_table[(int64_t)s * a.out_stride + (to0 >> a.c.page_shift)];
    if (out_page < 0 || out_page >= a.c.num_pages) {
        if (tid == 0)
            flag(a.c, SPLITZIP_KV4_BAD_PAGE);
        return;
    }
    const int n = min(16, keep - to0);
    if (tid < n) {
        const int j = a.kept[((int64_t)s * a.c.heads + head) * a.budget + to0 + tid];
        const int page = page_of(a.c, a.b, s, j);
        const int64_t first = ((int64_t)page * a.c.heads + head) << a.c.page_shift;
        sh_page0[tid] = first;
        sh_from[tid] = page < 0 ? -1 : first + (j & ((1 << a.c.page_shift) - 1));
    }
    __syncthreads();
    const int64_t out0 = ((int64_t)out_page * a.c.heads + head) << a.c.page_shift;
    const int in = to0 & ((1 << a.c.page_shift) - 1);
    // K codes: 4 bytes a lane
    for (int i = tid; i < n * (D / 8); i += kMove) {
        const int t = i / (D / 8), w = i % (D / 8);
        const int64_t f = sh_from[t];
        ((uint32_t *)(a.c.k_codes + (out0 + in + t) * (D / 2)))[w] =
            f < 0 ? 0u : ((const uint32_t *)(a.c.k_codes + f * (D / 2)))[w];
    }
    // V codes: a run of a token (D / 32 bytes) a lane
    for (int i = tid; i < n * 16; i += kMove) {
        const int t = i % n, run = i / n;
        const int64_t f = sh_from[t], p0 = sh_page0[t];
        const int ft = (int)(f - p0), ot = in + t;
        constexpr int kRun = D / 32;
        const uint8_t *from = a.c.v_codes + p0 * (D / 2) + (ft >> 2) * (2 * D) + run * (4 * kRun) + (ft & 3) * kRun;
        uint8_t *to = a.c.v_codes + out0 * (D / 2) + (ot >> 2) * (2 * D) + run * (4 * kRun) + (ot & 3) * kRun;
        if (D == 64)
            *(uint16_t *)to = f < 0 ? 0 : *(const uint16_t *)from;
        else if (D == 128)
            *(uint32_t *)to = f < 0 ? 0 : *(const uint32_t *)from;
        else
            *(uint2 *)to = f < 0 ? make_uint2(0, 0) : *(const uint2 *)from;
    }
    for (int i = tid; i < n * (D / 32); i += kMove) {
        const int t = i % n, block = i / n;
        const int64_t f = sh_from[t], p0 = sh_page0[t];
        a.c.k_scales[(out0 + in + t) * (D / 32) + block] = f < 0 ? 0 : a.c.k_scales[f * (D / 32) + block];
        const int64_t row = (int64_t)block << a.c.page_shift;
        a.c.v_scales[out0 * (D / 32) + row + in + t] = f < 0 ? 0 : a.c.v_scales[p0 * (D / 32) + row + (f - p0)];
    }
    if (tid < n)
        a.c.weights[out0 + in + tid] = sh_from[tid] < 0 ? 0.0f : a.c.weights[sh_from[tid]];
}

}  // namespace

void launch_evict(const EvictArgs &a, int head_dim, hipStream_t s)
{
    choose_kernel<<<(unsigned)(a.b.n_seqs * a.c.heads), kChoose, 0, s>>>(a);
    const unsigned grid = (unsigned)((int64_t)a.b.n_seqs * a.c.heads * ((a.budget + 15) / 16));
    if (head_dim == 64)
        move_kernel<64><<<grid, kMove, 0, s>>>(a);
    else if (head_dim == 128)
        move_kernel<128><<<grid, kMove, 0, s>>>(a);
    else
        move_kernel<256><<<grid, kMove, 0, s>>>(a);
}

}  // namespace kv4
}  // namespace sz
