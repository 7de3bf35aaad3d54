// splitzip_kv4_evict.hip -- cutting sequences of the 4-bit KV cache to the tokens that attention
// has used.  For each sequence longer than the budget and each KV head: its first `sinks` and last
// `recent` tokens stay, and of the others the `room` = budget - sinks - recent with the largest
// weights, equal ones in token order.
//
// choose_kernel finds the kept tokens, one workgroup a sequence and head.  Weights become 32-bit
// keys that order as the weights do, up to 32 of them in a lane's registers.  The budget-th largest
// key is found 8 bits at a time from counts of the keys that share its leading bits.  Weights are
// often equal or nearly so, so each count has 32 copies, one a bank: with one copy the atomics of a
// wave queued up (97 us for 32 heads of 32768 tokens; now 21).  Counts are sums of integers, so
// nothing depends on the order of atomics.  One ordered pass writes the tokens.  A workgroup's
// instructions a key bound it (searching bit by bit with population counts took 51 us).
//
// move_kernel gathers codes, scales and weights, 128 tokens a workgroup: every load of a lane is in
// flight before its first store, since four dependent loads (length, kept token, page, codes) stand
// before each (16 tokens a workgroup took twice the time).  Memory bounds it, by lines rather than
// bytes: a token's 64 bytes of V lie in the 256 that it shares with three others, and K's rows are half
// a line.  512 heads of 128 .. 8192 tokens cut to 2048: 280 MB kept, about 370 MB of lines, in 72 us.
#include "splitzip_kv4_internal.h"

namespace sz {
namespace kv4 {
namespace {

constexpr int kChoose = kChooseThreads;
constexpr int kWaves = kChoose / 64;
constexpr int kUnits = 8;             // runs of 256 tokens a wave holds: 32 keys a lane
constexpr int kCopies = 32;           // of each count: lanes of one wave meet only in pairs
constexpr int kMove = kMoveThreads;
constexpr int kTokens = kMoveTokens;  // a workgroup of move_kernel at a time

// Larger weight, larger key; -0 as 0, NaN the smallest.  0 is left for "no token", the largest value
// for tokens that stay whatever they weigh.
constexpr uint32_t kNone = 0, kNan = 1, kStays = 0xffffffffu;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t key_of(float w)
{
    const uint32_t u = bits(w + 0.0f);
    const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return w != w ? kNan : k;
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x)
{
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xf, 0xf, true);     // lane - 1 of the row of 16
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xf, 0xf, true);     // - 2
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xf, 0xf, true);     // - 4
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xf, 0xf, true);     // - 8
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xa, 0xf, false);    // rows 1, 3: the row before's sum
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xc, 0xf, false);    // rows 2, 3: the lower half's
    return x;
}

__global__ __launch_bounds__(kChoose, 8) void choose_kernel(EvictArgs a)
{
    __shared__ __align__(16) uint32_t sh_hist[257 * kCopies];
    __shared__ __align__(16) int sh_bin[2][256];
    __shared__ int sh_above[kWaves], sh_equal[kWaves];
    const int head = blockIdx.x % a.c.heads, s = blockIdx.x / a.c.heads;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
    const int lo = a.sinks, hi = q.len - a.recent;          // tokens that compete
    // A wave takes `units` runs of 256 tokens, a lane four adjacent tokens of each; the workgroup's
    // tokens are a chunk, and only sequences of more than 32768 tokens have several.
    const int units = min(kUnits, (q.len + 4 * kChoose - 1) / (4 * kChoose));
    const int chunk = 4 * kChoose * units;
    const int chunks = (q.len + chunk - 1) / chunk;
    const int64_t row = (int64_t)s * a.b.table_stride;
    const int place = (1 << a.c.page_shift) - 1;
    u32x4 key[kUnits];
    auto token = [&](int c, int i) { return c * chunk + (wave * units + i) * 256 + 4 * lane; };
    // All loads in flight together: the empty asm keeps the compiler from moving each behind the test
    // that uses it.
    auto load = [&](int c) {
        int page[kUnits];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
            page[i] = i < units ? a.b.table[row + (min(token(c, i), q.len - 1) >> a.c.page_shift)] : 0;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            asm volatile("" : "+v"(page[i]));
            const bool none = page[i] < 0 || page[i] >= a.c.num_pages;
            const int at = min(token(c, i), q.len - 1) & place & ~3;
            key[i] = u32x4{kNone, kNone, kNone, kNone};
            if (i < units)
                key[i] = *(const u32x4 *)(a.c.weights +
                                          (((int64_t)(none ? 0 : page[i]) * a.c.heads + head) << a.c.page_shift) + at);
        }
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            if (i >= units)
                break;
            asm volatile("" : "+v"(key[i]));
            const bool none = page[i] < 0 || page[i] >= a.c.num_pages;
            bad |= none;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                key[i][e] = key_of(as_float(key[i][e]));
            const int j0 = token(c, i) - 4 * lane;          // of the wave
            if (j0 < lo || j0 + 256 > hi || __any(none)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = j0 + 4 * lane + e;
                    const uint32_t k = none ? kNan : key[i][e];
                    key[i][e] = j >= q.len ? kNone : j < lo || j >= hi ? kStays : k;
                }
            }
        }
        if (bad)
            flag(a.c, SPLITZIP_KV4_BAD_PAGE);
    };

    // border: the budget-th largest key, found 8 bits at a time from the top; of the keys equal to it
    // the first equal_room are kept.  ("No token" counts as the smallest key of all, which no border is.)
    for (int i = tid; i < 256 * kCopies / 4; i += kChoose)
        ((uint4 *)sh_hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    uint32_t *const hist = sh_hist + (lane & (kCopies - 1));
    uint32_t border = 0;
    int equal_room = a.budget;                              // keys to keep of those that share border's bits
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int c = 0; c < chunks; ++c) {
            if (chunks > 1 || shift == 24)
                load(c);
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                if (i >= units)
                    break;
#pragma unroll
                for (int e = 0; e < 4; ++e)                 // 256: another prefix than border's
                    atomicAdd(hist + min((key[i][e] ^ border) >> shift, 256u) * kCopies, 1u);
            }
        }
        __syncthreads();
        // four lanes a bin, eight copies a lane
        uint4 *const h = (uint4 *)sh_hist + 2 * tid;
        const uint4 x = h[0], y = h[1];
        h[0] = h[1] = make_uint4(0, 0, 0, 0);
        int sum = (int)(x.x + x.y + x.z + x.w + y.x + y.y + y.z + y.w);
        sum += __builtin_amdgcn_mov_dpp(sum, 0xb1, 0xf, 0xf, true);     // lane ^ 1
        sum += __builtin_amdgcn_mov_dpp(sum, 0x4e, 0xf, 0xf, true);     // lane ^ 2
        int *const bins = sh_bin[(shift >> 3) & 1];
        if ((tid & 3) == 0)
            bins[255 - (tid >> 2)] = sum;                   // from the largest down
        __syncthreads();
        // every wave for itself: lane l holds bins 4 l .. + 3
        const int4 n = *(const int4 *)&bins[4 * lane];
        const int all = n.x + n.y + n.z + n.w;
        const int upto = (int)wave_scan((uint32_t)all);
        const int at = __builtin_ctzll(__ballot(upto >= equal_room));
        int before = __builtin_amdgcn_readlane(upto - all, at), bin = 4 * at;
        const int n4[4] = {__builtin_amdgcn_readlane(n.x, at), __builtin_amdgcn_readlane(n.y, at),
                           __builtin_amdgcn_readlane(n.z, at), __builtin_amdgcn_readlane(n.w, at)};
        int in_bin = n4[0];
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            const bool next = before + in_bin < equal_room;
            before += next ? in_bin : 0;
            in_bin = next ? n4[i] : in_bin;
            bin += next;
        }
        border |= (uint32_t)(255 - bin) << shift;
        equal_room -= before;
        if (in_bin == equal_room) {                         // every key of the bin: those above what lies below it
            border -= 1;
            equal_room = 0;
            break;
        }
    }

    // Where each token goes: counts above the border (low half) and equal to it (high half), summed
    // over lanes, units, waves and chunks in token order.
    int above0 = 0, equal0 = 0;
    for (int c = 0; c < chunks; ++c) {
        if (chunks > 1)
            load(c);
        uint32_t upto[kUnits];
        int na = 0, ne = 0;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            upto[i] = 0;
            if (i < units) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    upto[i] += key[i][e] > border ? 1u : key[i][e] == border ? 0x10000u : 0u;
                upto[i] = wave_scan(upto[i]);
                const uint32_t all = (uint32_t)__builtin_amdgcn_readlane((int)upto[i], 63);
                na += all & 0xffff;
                ne += all >> 16;
            }
        }
        if (lane == 0) {
            sh_above[wave] = na;
            sh_equal[wave] = ne;
        }
        __syncthreads();
        int a_at = above0, e_at = equal0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            a_at += w < wave ? sh_above[w] : 0;
            e_at += w < wave ? sh_equal[w] : 0;
            above0 += sh_above[w];
            equal0 += sh_equal[w];
        }
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            if (i >= units)
                break;
            int pa = a_at + (int)(upto[i] & 0xffff), pe = e_at + (int)(upto[i] >> 16);      // behind the lane's four
            const uint32_t all = (uint32_t)__builtin_amdgcn_readlane((int)upto[i], 63);
            a_at += all & 0xffff;
            e_at += all >> 16;
#pragma unroll
            for (int e = 3; e >= 0; --e) {
                const bool above = key[i][e] > border, equal = key[i][e] == border;
                pa -= above;
                pe -= equal;
                if (above || (equal && pe < equal_room))
                    kept[pa + min(pe, equal_room)] = token(c, i) + e;
            }
        }
        __syncthreads();                                    // the counts are free again
    }
}

template <int Bytes>
struct Run;
template <>
struct Run<2> { typedef uint16_t type; };
template <>
struct Run<4> { typedef uint32_t type; };
template <>
struct Run<8> { typedef uint64_t type; };

template <int D>
__global__ __launch_bounds__(kMove) void move_kernel(EvictArgs a)
{
    typedef typename Run<D / 32>::type run_t;       // a token's run in V's layout
    constexpr int kPieces = D / 32;                 // 16-byte pieces of a token's K
    constexpr int kK = kTokens * kPieces / kMove, kV = kTokens / 4 * 16 / kMove;
    constexpr int kBlocks = D / 32;
    constexpr int kS = (kTokens / 4 * kBlocks + kMove - 1) / kMove;
    // token offsets in the buffers, page * heads * page_size and so on; -1: no page; and the place in the page
    __shared__ int64_t sh_from[kTokens], sh_to[kTokens];
    __shared__ int sh_from_in[kTokens], sh_to_in[kTokens];
    const uint32_t pair = blockIdx.x / a.turns;
    const int head = pair % a.c.heads, s = pair / a.c.heads;
    Batch bt = a.b;
    bt.cu = nullptr;
    const int64_t cap = (int64_t)a.out_width << a.c.page_shift;
    const int keep = (int)min((int64_t)min(wave_sequence(a.c, bt, s).len, a.budget), cap);
    for (int64_t at = (int64_t)(blockIdx.x % a.turns) * kTokens; at < keep; at += (int64_t)a.turns * kTokens) {
        const int to0 = (int)at;
        // The empty asm keeps the compiler from holding a turn's offsets over the others, which only calls with too
        // small a max_len have: 50 registers for 78 (D = 128), 512 ragged heads 4 us less.
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int n = min(kTokens, keep - to0);
        if (tid < kTokens) {
            const int mask = (1 << a.c.page_shift) - 1;
            int64_t from = -1, to = -1;
            if (tid < n) {
                const int j = a.kept[((int64_t)s * a.c.heads + head) * a.budget + to0 + tid];
                const int out_page = a.out_table[(int64_t)s * a.out_stride + ((to0 + tid) >> a.c.page_shift)];
                const int page = page_of(a.c, a.b, s, j);
                sh_from_in[tid] = j & mask;
                sh_to_in[tid] = (to0 + tid) & mask;
                if (page >= 0)
                    from = ((int64_t)page * a.c.heads + head) << a.c.page_shift;
                if (out_page >= 0 && out_page < a.c.num_pages)
                    to = ((int64_t)out_page * a.c.heads + head) << a.c.page_shift;
                else
                    flag(a.c, SPLITZIP_KV4_BAD_PAGE);
            }
            sh_from[tid] = from;
            sh_to[tid] = to;
        }
        __syncthreads();

        uint4 k[kK];
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            const int t = (i * kMove + tid) / kPieces, p = tid % kPieces;
            const int64_t f = sh_from[t];
            k[i] = f < 0 ? make_uint4(0, 0, 0, 0) : *(const uint4 *)(a.c.k_codes + (f + sh_from_in[t]) * (D / 2) + 16 * p);
        }
        run_t v[kV][4];
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = (i * kMove + tid) / 16 * 4 + e, run = tid % 16;
                const int64_t f = sh_from[t];
                const int in = sh_from_in[t];
                v[i][e] = f < 0 ? 0 : *(const run_t *)(a.c.v_codes + f * (D / 2) + (in >> 2) * (2 * D) + run * (D / 8) +
                                                       (in & 3) * (D / 32));
            }
        uint8_t vs[kS][4];
#pragma unroll
        for (int i = 0; i < kS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int u = i * kMove + tid, t = u % (kTokens / 4) * 4 + e, block = u / (kTokens / 4);
                const int64_t f = block < kBlocks ? sh_from[t] : -1;
                vs[i][e] = f < 0 ? 0 : a.c.v_scales[f * kBlocks + ((int64_t)block << a.c.page_shift) + sh_from_in[t]];
            }
        run_t ks = 0;                                   // D / 32 bytes as well
        float w = 0.0f;
        if (tid < n && sh_from[tid] >= 0) {
            ks = *(const run_t *)(a.c.k_scales + (sh_from[tid] + sh_from_in[tid]) * kBlocks);
            w = a.c.weights[sh_from[tid] + sh_from_in[tid]];
        }

#pragma unroll
        for (int i = 0; i < kK; ++i) {
            const int t = (i * kMove + tid) / kPieces, p = tid % kPieces;
            const int64_t o = sh_to[t];
            if (o >= 0)
                *(uint4 *)(a.c.k_codes + (o + sh_to_in[t]) * (D / 2) + 16 * p) = k[i];
        }
        // four tokens lie in one page on both sides of their stores: pages hold multiples of 16
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int t = (i * kMove + tid) / 16 * 4, run = tid % 16;
            const int64_t o = sh_to[t];
            if (o < 0)
                continue;
            run_t *to = (run_t *)(a.c.v_codes + o * (D / 2) + (sh_to_in[t] >> 2) * (2 * D) + run * (D / 8));
            if (t + 3 < n) {
                typedef run_t four __attribute__((ext_vector_type(4)));
                *(four *)to = four{v[i][0], v[i][1], v[i][2], v[i][3]};
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t + e < n)
                        to[e] = v[i][e];
            }
        }
#pragma unroll
        for (int i = 0; i < kS; ++i) {
            const int u = i * kMove + tid, t = u % (kTokens / 4) * 4, block = u / (kTokens / 4);
            const int64_t o = block < kBlocks ? sh_to[t] : -1;
            if (o < 0)
                continue;
            uint8_t *to = a.c.v_scales + o * kBlocks + ((int64_t)block << a.c.page_shift) + sh_to_in[t];
            if (t + 3 < n) {
                *(uint32_t *)to = vs[i][0] | (uint32_t)vs[i][1] << 8 | (uint32_t)vs[i][2] << 16 | (uint32_t)vs[i][3] << 24;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t + e < n)
                        to[e] = vs[i][e];
            }
        }
        if (tid < n && sh_to[tid] >= 0) {
            *(run_t *)(a.c.k_scales + (sh_to[tid] + sh_to_in[tid]) * kBlocks) = ks;
            a.c.weights[sh_to[tid] + sh_to_in[tid]] = w;
        }
        __syncthreads();                            // the places are free again
    }
}

}  // namespace

hipError_t launch_evict(const EvictArgs &a, int head_dim, hipStream_t s)
{
    choose_kernel<<<(unsigned)(a.b.n_seqs * a.c.heads), kChoose, 0, s>>>(a);
    if (const hipError_t e = hipGetLastError())
        return e;                               // move_kernel would read kept tokens that nobody wrote
    const unsigned grid = (unsigned)((int64_t)a.b.n_seqs * a.c.heads * a.turns);
    if (head_dim == 64)
        move_kernel<64><<<grid, kMove, 0, s>>>(a);
    else if (head_dim == 128)
        move_kernel<128><<<grid, kMove, 0, s>>>(a);
    else
        move_kernel<256><<<grid, kMove, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace kv4
}  // namespace sz
