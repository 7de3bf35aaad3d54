// splitzip_kv4_host.hip -- entry points of the 4-bit KV cache (include/splitzip_kv4.h): argument
// checks and the choice of launches.
#include "splitzip_kv4_internal.h"
#include "splitzip_tuning.h"

#include <algorithm>
#include <cmath>
#include <stdio.h>

using sz::report;
using namespace sz::kv4;

namespace {

#define KV4_REQUIRE(cond, message)                           \
    do {                                                     \
        if (!(cond))                                         \
            return report(SPLITZIP_E_INVALID, message);      \
    } while (0)

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The cache's device current for the call, and the launch error as the call's status.
struct Device {
    int before = -1, status = SPLITZIP_OK;
    explicit Device(int device)
    {
        hipError_t e = hipGetDevice(&before);
        if (e == hipSuccess && before != device)
            e = hipSetDevice(device);
        else
            before = -1;
        if (e != hipSuccess)
            status = failed(e);
    }
    ~Device()
    {
        if (before >= 0)
            (void)hipSetDevice(before);
    }
    static int failed(hipError_t e)
    {
        char text[160];
        snprintf(text, sizeof text, "4-bit cache launch: %s", hipGetErrorString(e));
        return report(e == hipErrorOutOfMemory ? SPLITZIP_E_NOMEM : SPLITZIP_E_DEVICE, text);
    }
    static int launched(hipError_t e = hipGetLastError())
    {
        return e == hipSuccess ? SPLITZIP_OK : failed(e);
    }
};

int check_cache(const splitzip_kv4_cache *c, Cache *out)
{
    KV4_REQUIRE(c, "cache is null");
    KV4_REQUIRE(c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256, "head_dim must be 64, 128 or 256");
    KV4_REQUIRE(c->kv_heads >= 1 && c->kv_heads <= 65535, "kv_heads must be in [1, 65535]");
    KV4_REQUIRE(c->page_size >= 16 && c->page_size <= 1024 && (c->page_size & (c->page_size - 1)) == 0,
                "page_size must be a power of two in [16, 1024]");
    KV4_REQUIRE(c->num_pages >= 1 && c->num_pages <= INT32_MAX, "num_pages must be in [1, 2^31)");
    KV4_REQUIRE(c->k_codes && c->k_scales && c->v_codes && c->v_scales && c->weights && c->status,
                "a cache buffer is null");
    KV4_REQUIRE(aligned16(c->k_codes) && aligned16(c->k_scales) && aligned16(c->v_codes) && aligned16(c->v_scales) &&
                    aligned16(c->weights) && (reinterpret_cast<uintptr_t>(c->status) & 3) == 0,
                "cache buffers must be 16-byte aligned");
    *out = Cache{c->k_codes, c->k_scales, c->v_codes, c->v_scales, c->weights, c->status, c->num_pages,
                 __builtin_ctz((unsigned)c->page_size), c->kv_heads};
    return SPLITZIP_OK;
}

int check_batch(const splitzip_kv4_batch *b, const Cache &c, bool rows, Batch *out)
{
    KV4_REQUIRE(b, "batch is null");
    KV4_REQUIRE(b->n_seqs >= 0 && b->total >= 0 && b->total < INT32_MAX, "negative or too large batch");
    // kernels count up to 32768 tokens past a sequence's last in 32 bits
    KV4_REQUIRE(b->table_width >= 0 && ((int64_t)b->table_width << c.page_shift) <= INT32_MAX - 65536,
                "table_width is negative or holds 2^31 - 65536 tokens or more");
    KV4_REQUIRE(b->n_seqs == 0 || (b->lens && (b->table || b->table_width == 0)), "lens or table is null");
    KV4_REQUIRE(b->n_seqs <= 1 || b->table_stride >= b->table_width, "table_stride is below table_width");
    KV4_REQUIRE(!rows || b->cu_seqlens || b->total == b->n_seqs, "without cu_seqlens there is one row a sequence");
    KV4_REQUIRE(!rows || b->total == 0 || b->n_seqs > 0, "rows without a sequence");
    KV4_REQUIRE(b->max_q >= 0 && b->max_len >= 0, "max_q or max_len is negative");
    *out = Batch{b->table, b->lens, b->cu_seqlens, b->table_stride, b->total, b->table_width, b->n_seqs};
    return SPLITZIP_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads of an append or read launch: a lane takes 8 channels, a workgroup whole rows of one head.
int64_t row_launch(const Batch &b, const Cache &c, int head_dim)
{
    return ceil_div(b.total, kRowThreads / (head_dim / 8)) * c.heads * kRowThreads;
}

int check_queries(const splitzip_kv4_queries *q, const splitzip_kv4_batch *b, const splitzip_kv4_cache *c, AttendArgs *a)
{
    KV4_REQUIRE(q, "queries is null");
    KV4_REQUIRE(q->dtype == SPLITZIP_KV4_BF16 || q->dtype == SPLITZIP_KV4_FP16, "queries must be bf16 or fp16");
    KV4_REQUIRE(q->q_heads >= c->kv_heads && q->q_heads % c->kv_heads == 0, "q_heads must be a multiple of kv_heads");
    // kernels count past a sequence's last row in 32 bits, by up to 4097 tiles of 32 rows (plan)
    KV4_REQUIRE(b->total * q->q_heads < INT32_MAX - (1 << 18), "total * q_heads must be below 2^31 - 2^18");
    KV4_REQUIRE(q->window >= 0 && q->sinks >= 0, "window or sinks is negative");
    // scores are held as powers of two
    const float scale2 = (float)((double)q->scale * 1.4426950408889634);
    KV4_REQUIRE(std::isfinite(scale2), "scale is not finite, or scale * log2(e) is not");
    KV4_REQUIRE(q->q || b->total == 0, "q is null");
    KV4_REQUIRE((reinterpret_cast<uintptr_t>(q->q) & 1) == 0, "q is not aligned to its type");
    a->q = q->q;
    a->q_token = q->token_stride;
    a->q_head = q->head_stride;
    a->q_heads = q->q_heads;
    a->group = q->q_heads / c->kv_heads;
    a->window = q->window;
    a->sinks = q->sinks;
    a->scale2 = scale2;
    a->wide = aligned16(q->q) && q->token_stride % 8 == 0 && q->head_stride % 8 == 0;
    return SPLITZIP_OK;
}

// Bytes of a split's partial results.
int64_t split_bytes(const AttendArgs &a, int head_dim) { return a.b.total * a.q_heads * (head_dim + 2) * 4; }

// Rows of a sequence and KV head that a launch is made for: the most there are, or the mean where nobody says.
int64_t expected_rows(const splitzip_kv4_batch &b, int group)
{
    const int64_t q = b.max_q > 0 ? std::min<int64_t>(b.max_q, b.total) : ceil_div(b.total, std::max(1, b.n_seqs));
    return std::max<int64_t>(1, q) * group;
}

// Launch of an attend call: rows of a workgroup, row tiles, splits along the tokens.  The lengths are
// known only to the GPU.  A split takes 4096 tokens, so that a few long sequences among short ones do
// not outlast the others (256 decode steps of 128 .. 8192 tokens: 251 us, unsplit 263, at 2048 264);
// fewer, but 256 at least, where there would be fewer workgroups than the GPU holds at a time; and more
// where there would be over 16 times as many, since a length that nobody has costs a workgroup that ends at
// once and a place in the workspace (256 steps of up to 1024 tokens on tables of 2^20: 64 us and 70 MiB
// for 1030 us and 2084 MiB).  Two steps of 2^19 tokens among 252 short ones, where that leaves parts of
// 2^17, took 1221 us for 1176.
int plan(const splitzip_kv4_cache *c, const splitzip_kv4_batch *b, const splitzip_kv4_queries *q, AttendArgs *a)
{
    const int64_t rows = expected_rows(*b, a->group);
    a->tile_rows = attend_rows(c->head_dim, rows);
    const int64_t pairs = (int64_t)b->n_seqs * c->kv_heads;
    // workgroups that a launch holds; fewer tiles and splits than there could be take rows and tokens in turn
    const int64_t most = kMostThreads / attend_threads(c->head_dim, a->tile_rows);
    KV4_REQUIRE(pairs <= most, "too many sequences and heads");
    // Without max_q a sequence may have more rows than expected, all of them at most: twice the tiles, or 8 up to 16384
    // workgroups, or what makes 4096, and rows in turn beyond.  An odd number of tiles, since the ones with
    // rows would meet on few CUs where it is a multiple of their number.  Against all rows as every
    // sequence's (us): 64 requests of 3 drafts 85 for 489, 256 single tokens 254 for 4190, 16 prompts of 64 ..
    // 4096 tokens 1040 for 1211; a prompt of 2048 among 63 single tokens 614 for 642, among 255 2090 for
    // 5400 (6030 with 4096 workgroups at most); the drafts with 16384 workgroups 107.
    const int64_t expected = ceil_div(rows, a->tile_rows);
    int64_t tiles = expected;
    if (b->max_q == 0) {
        const int64_t one = std::max<int64_t>(1, pairs);
        tiles = std::max({2 * expected, std::min<int64_t>(8, 16384 / one), 4096 / one});
        tiles = std::min(tiles, ceil_div(b->total * a->group, a->tile_rows)) | 1;
    }
    tiles = std::min(tiles, most / std::max<int64_t>(1, pairs));
    int64_t tokens = std::min<int64_t>(b->max_len, (int64_t)b->table_width * c->page_size);
    if (q->window > 0)
        tokens = std::min<int64_t>(tokens, (int64_t)q->window + q->sinks + 32 + rows / a->group);
    const int64_t blocks = std::max<int64_t>(1, pairs * expected), fill = a->tile_rows <= 32 ? 1024 : 512;
    const int64_t even = a->tile_rows <= 32 ? std::min(ceil_div(tokens, 4096), 16 * fill / blocks) : 1;
    int64_t splits = std::max(std::min(ceil_div(tokens, 256), fill / blocks), even);
    // hints that say too little do not make it larger
    splits = std::min<int64_t>(splits, (512ll << 20) / std::max<int64_t>(1, split_bytes(*a, c->head_dim)));
    if (ceil_div((int64_t)b->total * q->q_heads, join_rows(c->head_dim)) > kMostThreads / kJoinThreads)
        splits = 1;
    splits = std::min(std::max<int64_t>(1, splits), most / std::max<int64_t>(1, pairs * tiles));
    const int64_t groups = ceil_div(std::max<int64_t>(1, tokens), 16);
    a->per = (int32_t)(ceil_div(ceil_div(groups, splits), 8) * 8);
    a->tiles = (int32_t)tiles;
    a->splits = (int32_t)ceil_div(groups, a->per);
    return SPLITZIP_OK;
}

// Launch of a weigh call.
int plan_weigh(const splitzip_kv4_cache *c, const splitzip_kv4_batch *b, AttendArgs *a)
{
    const int64_t pairs = (int64_t)b->n_seqs * c->kv_heads;
    KV4_REQUIRE(pairs <= 1 << 22, "more than 2^22 sequences and heads");
    const int64_t tokens = std::min<int64_t>(b->max_len, (int64_t)b->table_width * c->page_size);
    // Up to 16 rows stay in registers: 64 decode steps of 8 rows 52 us, by rows_kernel 135.  Where the mean is up to
    // 16 and nobody says what the longest has, step_kernel takes the sequences of up to 16 and a second
    // launch of up to 8192 workgroups the others: 256 decode steps of 8 rows 187 us, all by rows_kernel 499; 255 of them
    // and a prompt of 512 queries 503, all by rows_kernel 548, by step_kernel 2474.
    const bool few = expected_rows(*b, a->group) <= kStepRows, more = !few || b->max_q == 0;
    a->splits = a->row_splits = 0;
    // 256 tokens a workgroup at least (one turn of each wave), and 2048 workgroups at most (the same at 4096;
    // 1024 took 63 us for 57)
    if (few)
        a->splits = (int32_t)std::min<int64_t>(std::max<int64_t>(1, 2048 / pairs), tokens / 256 + 1);
    // a launch that would be too large has fewer, which take tokens in turn
    const int64_t most = few ? std::max<int64_t>(1, 8192 / pairs) : kMostThreads / kWeighThreads / pairs;
    a->step_rows = !few ? 0 : more ? kStepRows : INT32_MAX;
    if (more)
        a->row_splits = (int32_t)std::min(tokens / weigh_tokens(c->head_dim) + 1, most);
    return SPLITZIP_OK;
}

uint64_t workspace_of(const AttendArgs &a, int head_dim) { return a.splits == 1 ? 0 : a.splits * split_bytes(a, head_dim); }

// Launches of an evict call: a workgroup of move_kernel for every 128 tokens that a sequence and head may
// keep.  A launch that would be too large has fewer, which take tokens in turn.
int plan_evict(const splitzip_kv4_batch *batch, int32_t budget, EvictArgs *a)
{
    const int64_t pairs = (int64_t)a->b.n_seqs * a->c.heads;
    KV4_REQUIRE(pairs <= kMostThreads / kChooseThreads, "too many sequences and heads");
    const int64_t longest = std::min<int64_t>(batch->max_len, (int64_t)a->b.table_width << a->c.page_shift);
    const int64_t turns = ceil_div(std::max<int64_t>(1, std::min<int64_t>(budget, longest)), kMoveTokens);
    a->turns = (int32_t)std::min(turns, kMostThreads / kMoveThreads / std::max<int64_t>(1, pairs));
    return SPLITZIP_OK;
}

}  // namespace

extern "C" {

int splitzip_kv4_append(const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch, const void *k,
                        int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                        int64_t v_head_stride, int32_t dtype, void *stream)
{
    AppendArgs a;
    if (int e = check_cache(cache, &a.c))
        return e;
    if (int e = check_batch(batch, a.c, true, &a.b))
        return e;
    KV4_REQUIRE(dtype >= SPLITZIP_KV4_BF16 && dtype <= SPLITZIP_KV4_FP32, "k and v must be bf16, fp16 or fp32");
    if (a.b.total == 0)
        return SPLITZIP_OK;
    KV4_REQUIRE(k && v, "k or v is null");
    const int size = dtype == SPLITZIP_KV4_FP32 ? 4 : 2;
    KV4_REQUIRE(reinterpret_cast<uintptr_t>(k) % size == 0 && reinterpret_cast<uintptr_t>(v) % size == 0,
                "k or v is not aligned to its type");
    KV4_REQUIRE(row_launch(a.b, a.c, cache->head_dim) <= kMostThreads, "more rows and heads than a launch holds");
    const int unit = 16 / size;
    a.k = k;
    a.v = v;
    a.k_token = k_token_stride;
    a.k_head = k_head_stride;
    a.v_token = v_token_stride;
    a.v_head = v_head_stride;
    a.wide = aligned16(k) && aligned16(v) && k_token_stride % unit == 0 && k_head_stride % unit == 0 &&
             v_token_stride % unit == 0 && v_head_stride % unit == 0;
    Device d(cache->device);
    if (d.status)
        return d.status;
    launch_append(a, cache->head_dim, dtype, static_cast<hipStream_t>(stream));
    return Device::launched();
}

int splitzip_kv4_read(const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch, void *k, void *v, int32_t dtype,
                      void *stream)
{
    ReadArgs a;
    if (int e = check_cache(cache, &a.c))
        return e;
    if (int e = check_batch(batch, a.c, true, &a.b))
        return e;
    KV4_REQUIRE(dtype >= SPLITZIP_KV4_BF16 && dtype <= SPLITZIP_KV4_FP32, "k and v must be bf16, fp16 or fp32");
    if (a.b.total == 0)
        return SPLITZIP_OK;
    KV4_REQUIRE(k && v && aligned16(k) && aligned16(v), "k or v is null or not 16-byte aligned");
    KV4_REQUIRE(row_launch(a.b, a.c, cache->head_dim) <= kMostThreads, "more rows and heads than a launch holds");
    a.k = k;
    a.v = v;
    Device d(cache->device);
    if (d.status)
        return d.status;
    launch_read(a, cache->head_dim, dtype, static_cast<hipStream_t>(stream));
    return Device::launched();
}

int splitzip_kv4_attend_workspace(const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch,
                                  const splitzip_kv4_queries *queries, uint64_t *bytes)
{
    AttendArgs a;
    KV4_REQUIRE(bytes, "bytes is null");
    if (int e = check_cache(cache, &a.c))
        return e;
    if (int e = check_batch(batch, a.c, true, &a.b))
        return e;
    if (int e = check_queries(queries, batch, cache, &a))
        return e;
    if (int e = plan(cache, batch, queries, &a))
        return e;
    *bytes = workspace_of(a, cache->head_dim);
    return SPLITZIP_OK;
}

int splitzip_kv4_attend(const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch,
                        const splitzip_kv4_queries *queries, void *out, float *lse, void *workspace,
                        uint64_t workspace_bytes, void *stream)
{
    AttendArgs a;
    if (int e = check_cache(cache, &a.c))
        return e;
    if (int e = check_batch(batch, a.c, true, &a.b))
        return e;
    if (int e = check_queries(queries, batch, cache, &a))
        return e;
    if (a.b.total == 0)
        return SPLITZIP_OK;
    KV4_REQUIRE(out && aligned16(out), "out is null or not 16-byte aligned");
    if (int e = plan(cache, batch, queries, &a))
        return e;
    const uint64_t need = workspace_of(a, cache->head_dim);
    KV4_REQUIRE(need == 0 || (workspace && aligned16(workspace) && workspace_bytes >= need),
                "workspace is missing, misaligned or smaller than splitzip_kv4_attend_workspace says");
    a.out = out;
    a.lse = lse;
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = a.part_o ? a.part_o + (uint64_t)a.splits * a.b.total * a.q_heads * cache->head_dim : nullptr;
    Device d(cache->device);
    if (d.status)
        return d.status;
    return Device::launched(launch_attend(a, cache->head_dim, queries->dtype, static_cast<hipStream_t>(stream)));
}

int splitzip_kv4_weigh(const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch,
                       const splitzip_kv4_queries *queries, const float *lse, void *stream)
{
    AttendArgs a;
    if (int e = check_cache(cache, &a.c))
        return e;
    if (int e = check_batch(batch, a.c, true, &a.b))
        return e;
    if (int e = check_queries(queries, batch, cache, &a))
        return e;
    if (a.b.total == 0)
        return SPLITZIP_OK;
    KV4_REQUIRE(lse, "lse is null");
    if (int e = plan_weigh(cache, batch, &a))
        return e;
    a.lse_in = lse;
    Device d(cache->device);
    if (d.status)
        return d.status;
    return Device::launched(launch_weigh(a, cache->head_dim, queries->dtype, static_cast<hipStream_t>(stream)));
}

int splitzip_kv4_evict(const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch, const int32_t *out_table,
                       int64_t out_table_stride, int32_t out_table_width, int32_t budget, int32_t sinks, int32_t recent,
                       int32_t *out_lens, int32_t *kept, void *stream)
{
    EvictArgs a;
    if (int e = check_cache(cache, &a.c))
        return e;
    if (int e = check_batch(batch, a.c, false, &a.b))
        return e;
    KV4_REQUIRE(budget >= 1 && sinks >= 0 && recent >= 0 && (int64_t)sinks + recent <= budget,
                "budget must be at least 1 and hold sinks and recent");
    if (a.b.n_seqs == 0)
        return SPLITZIP_OK;
    KV4_REQUIRE(out_table && out_lens && kept, "out_table, out_lens or kept is null");
    KV4_REQUIRE(out_table_width >= 0 && (a.b.n_seqs <= 1 || out_table_stride >= out_table_width),
                "out_table_stride is below out_table_width");
    // lengths are read while new ones are written
    KV4_REQUIRE(out_lens + a.b.n_seqs <= a.b.lens || a.b.lens + a.b.n_seqs <= out_lens, "out_lens must not overlap lens");
    // kernels count up to 1024 tokens past the budget in 32 bits
    KV4_REQUIRE(budget <= INT32_MAX - 65536 && (int64_t)a.b.n_seqs * a.c.heads * ceil_div(budget, 16) < INT32_MAX,
                "too many tokens to keep");
    if (int e = plan_evict(batch, budget, &a))
        return e;
    a.out_table = out_table;
    a.out_stride = out_table_stride;
    a.out_width = out_table_width;
    a.budget = budget;
    a.sinks = sinks;
    a.recent = recent;
    a.out_lens = out_lens;
    a.kept = kept;
    Device d(cache->device);
    if (d.status)
        return d.status;
    return Device::launched(launch_evict(a, cache->head_dim, static_cast<hipStream_t>(stream)));
}

int splitzip_kv4_launches(int32_t op, const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch,
                          const splitzip_kv4_queries *queries, int32_t budget, uint64_t workgroups[2], uint32_t threads[2])
{
    KV4_REQUIRE(workgroups && threads, "workgroups or threads is null");
    for (int i = 0; i < 2; ++i)
        workgroups[i] = threads[i] = 0;
    if (op == SPLITZIP_KV4_EVICT) {
        EvictArgs a;
        if (int e = check_cache(cache, &a.c))
            return e;
        if (int e = check_batch(batch, a.c, false, &a.b))
            return e;
        if (a.b.n_seqs == 0)
            return SPLITZIP_OK;
        if (int e = plan_evict(batch, budget, &a))
            return e;
        workgroups[0] = (uint64_t)a.b.n_seqs * a.c.heads;
        threads[0] = kChooseThreads;
        workgroups[1] = workgroups[0] * a.turns;
        threads[1] = kMoveThreads;
        return SPLITZIP_OK;
    }
    KV4_REQUIRE(op == SPLITZIP_KV4_ATTEND || op == SPLITZIP_KV4_WEIGH, "no such operator");
    AttendArgs a;
    if (int e = check_cache(cache, &a.c))
        return e;
    if (int e = check_batch(batch, a.c, true, &a.b))
        return e;
    if (int e = check_queries(queries, batch, cache, &a))
        return e;
    if (a.b.total == 0)
        return SPLITZIP_OK;
    if (op == SPLITZIP_KV4_WEIGH) {
        if (int e = plan_weigh(cache, batch, &a))
            return e;
        for (int32_t splits : {a.splits, a.row_splits})
            if (splits > 0) {
                const int i = threads[0] ? 1 : 0;
                workgroups[i] = (uint64_t)a.b.n_seqs * a.c.heads * splits;
                threads[i] = kWeighThreads;
            }
        return SPLITZIP_OK;
    }
    if (int e = plan(cache, batch, queries, &a))
        return e;
    workgroups[0] = (uint64_t)a.b.n_seqs * a.c.heads * a.tiles * a.splits;
    threads[0] = attend_threads(cache->head_dim, a.tile_rows);
    if (a.splits > 1) {
        workgroups[1] = ceil_div(a.b.total * a.q_heads, join_rows(cache->head_dim));
        threads[1] = kJoinThreads;
    }
    return SPLITZIP_OK;
}

}  // extern "C"
