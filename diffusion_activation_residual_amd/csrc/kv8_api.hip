// kv8_api.hip -- the C ABI of the 8-bit paged K/V cache: argument validation and dispatch.
// Nothing touches the device until every argument has been checked.
#include "kv8_internal.h"

#include <limits.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

namespace {

cfz_status fail(cfz_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
cfz_status fail(cfz_status st, const char *fmt, ...)
{
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return cfz::report(st, text);
}

cfz_status hip_status(hipError_t e, const char *what)
{
    if (e == hipSuccess)
        return CFZ_OK;
    return fail(CFZ_ERR_HIP, "%s: %s (%d)", what, hipGetErrorString(e), (int)e);
}

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Sizes only, so that the workspace queries can use it too.
cfz_status check_sizes(const cfz_kv8_cache *c, const cfz_kv8_batch *b, cfz::Kv8Cache *kc,
                       cfz::Kv8Batch *kb)
{
    if (!c || !b)
        return fail(CFZ_ERR_NULL, "cache and batch are required");
    if (c->format != CFZ_KV8_INT8 && c->format != CFZ_KV8_E4M3)
        return fail(CFZ_ERR_UNSUPPORTED, "format = %d", c->format);
    if (c->head_dim != 64 && c->head_dim != 128)
        return fail(CFZ_ERR_UNSUPPORTED, "head_dim = %d (supported: 64, 128)", c->head_dim);
    if (c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
        return fail(CFZ_ERR_UNSUPPORTED, "page_tokens = %d (supported: 32, 64, 128)",
                    c->page_tokens);
    if (c->kv_heads < 1 || c->kv_heads > 1024)
        return fail(CFZ_ERR_SHAPE, "kv_heads = %d", c->kv_heads);
    if (c->pages < 0 || c->pages > INT_MAX)
        return fail(CFZ_ERR_SHAPE, "pages = %lld", (long long)c->pages);
    if (b->batch < 0 || b->batch > 65535)
        return fail(CFZ_ERR_SHAPE, "batch = %d", b->batch);
    if (b->table_width < 1 || (int64_t)b->table_width * c->page_tokens > INT_MAX)
        return fail(CFZ_ERR_SHAPE, "table_width = %d", b->table_width);
    if (b->tokens < 0 || b->tokens > INT_MAX)
        return fail(CFZ_ERR_SHAPE, "tokens = %lld", (long long)b->tokens);
    if (b->max_rows < 0 || b->max_rows > INT_MAX)
        return fail(CFZ_ERR_SHAPE, "max_rows = %lld", (long long)b->max_rows);
    const int log2page = c->page_tokens == 32 ? 5 : (c->page_tokens == 64 ? 6 : 7);
    *kc = cfz::Kv8Cache{(uint8_t *)c->k, (uint8_t *)c->v, c->k_scale,     c->v_scale, c->k_mean,
                        c->pages,        c->kv_heads,     c->head_dim,    c->page_tokens,
                        log2page,        c->format};
    *kb = cfz::Kv8Batch{b->page_table, b->offsets, b->lengths, b->tokens,
                        b->max_rows,   b->batch,   b->table_width};
    return CFZ_OK;
}

// No sequence has more rows than the call.  (Not where block lists are laid out by max_rows.)
void bound_rows(cfz::Kv8Batch *b) { b->max_rows = b->max_rows < b->tokens ? b->max_rows : b->tokens; }

bool empty(const cfz::Kv8Batch &b) { return b.batch == 0 || b.max_rows == 0 || b.tokens == 0; }

cfz_status check_pointers(const cfz::Kv8Cache &c, const cfz::Kv8Batch &b)
{
    if (!b.table || !b.off || !b.len)
        return fail(CFZ_ERR_NULL, "page_table, offsets and lengths are required");
    if (!aligned(b.table, 4) || !aligned(b.off, 4) || !aligned(b.len, 4))
        return fail(CFZ_ERR_ALIGN, "page_table, offsets and lengths must be 4-byte aligned");
    if (c.pages > 0 && (!c.k || !c.v || !c.ks || !c.vs))
        return fail(CFZ_ERR_NULL, "the cache's k, v, k_scale and v_scale are required");
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.ks, 16) || !aligned(c.vs, 16) ||
        !aligned(c.km, 16))
        return fail(CFZ_ERR_ALIGN, "the cache's buffers must be 16-byte aligned");
    return CFZ_OK;
}

int width_of(int dtype) { return dtype == CFZ_KV8_F32 ? 4 : 2; }

cfz_status check_dtype(int dtype, bool f32)
{
    if (dtype == CFZ_KV8_BF16 || dtype == CFZ_KV8_F16 || (f32 && dtype == CFZ_KV8_F32))
        return CFZ_OK;
    return fail(CFZ_ERR_UNSUPPORTED, "dtype = %d", dtype);
}

cfz_status check_stride(int64_t stride, int64_t row, int dtype, const char *what)
{
    if (stride < row || stride > INT_MAX || stride * width_of(dtype) % 16 != 0)
        return fail(CFZ_ERR_SHAPE, "%s = %lld (at least %lld, a multiple of 16 bytes)", what,
                    (long long)stride, (long long)row);
    return CFZ_OK;
}

cfz_status check_groups(double groups)
{
    if (groups >= cfz::kKv8MaxGroups)
        return fail(CFZ_ERR_SHAPE, "the call needs %.0f work-groups (limit 2^23)", groups);
    return CFZ_OK;
}

cfz_status check_pages(const cfz::Kv8Cache &c, const cfz::Kv8Batch &b)
{
    // (append: keys and values each on their own)
    return check_groups(2 * ((double)((b.max_rows + c.page - 1) / c.page) + 1) * c.heads * b.batch);
}

// What attend and select share.
cfz_status check_queries(const cfz::Kv8Cache &c, const cfz::Kv8Batch &b, int32_t q_heads,
                         int64_t max_kv, const cfz_kv8_blocks *blocks)
{
    if (q_heads < c.heads || q_heads % c.heads != 0 || q_heads / c.heads > 64)
        return fail(CFZ_ERR_SHAPE, "q_heads = %d with kv_heads = %d", q_heads, c.heads);
    if (max_kv < 0 || max_kv > (int64_t)b.width * c.page || max_kv > 1 << 30)
        return fail(CFZ_ERR_SHAPE, "max_kv = %lld (table: %lld, at most 2^30)", (long long)max_kv,
                    (long long)b.width * c.page);
    if (blocks) {
        if (blocks->count < 1 || blocks->count > 4096)
            return fail(CFZ_ERR_SHAPE, "blocks: count = %d (1 .. 4096)", blocks->count);
        if (blocks->q_block < 1)
            return fail(CFZ_ERR_SHAPE, "blocks: q_block = %d", blocks->q_block);
    }
    const int64_t most = blocks ? blocks->q_block : b.tokens;
    if ((b.max_rows < most ? b.max_rows : most) * (q_heads / c.heads) > 1 << 30)
        return fail(CFZ_ERR_SHAPE, "more than 2^30 rows (queries, query heads) read a KV head");
    return CFZ_OK;
}

cfz_status check_workspace(const void *ws, size_t have, size_t need)
{
    if (need == 0)
        return CFZ_OK;
    if (!ws || have < need)
        return fail(CFZ_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? have : (size_t)0,
                    need);
    if (!aligned(ws, 256))
        return fail(CFZ_ERR_ALIGN, "workspace must be 256-byte aligned");
    return CFZ_OK;
}

}  // namespace

#define CFZ_TRY(x)                                                                                 \
    do {                                                                                           \
        const cfz_status cfz_st_ = (x);                                                            \
        if (cfz_st_ != CFZ_OK)                                                                     \
            return cfz_st_;                                                                        \
    } while (0)

extern "C" {

cfz_status cfz_kv8_append(const cfz_kv8_cache *cache, const cfz_kv8_batch *batch,
                          cfz_kv8_dtype dtype, const void *k, const void *v, int64_t k_stride,
                          int64_t v_stride, const cfz_kv8_rotation *rotation, void *hip_stream)
{
    cfz::Kv8Cache c;
    cfz::Kv8Batch b;
    CFZ_TRY(check_sizes(cache, batch, &c, &b));
    CFZ_TRY(check_dtype(dtype, true));
    const int64_t row = (int64_t)c.heads * c.dim;
    CFZ_TRY(check_stride(k_stride, row, dtype, "k_stride"));
    CFZ_TRY(check_stride(v_stride, row, dtype, "v_stride"));
    cfz::Kv8Rotation rot{nullptr, nullptr, nullptr, 0, 0, 0};
    if (rotation) {
        if (rotation->rot_dim < 8 || rotation->rot_dim > c.dim || rotation->rot_dim % 8 != 0)
            return fail(CFZ_ERR_SHAPE, "rot_dim = %d (a multiple of 8, at most %d)",
                        rotation->rot_dim, c.dim);
        if (rotation->table_rows < 1 || rotation->table_rows > INT_MAX)
            return fail(CFZ_ERR_SHAPE, "table_rows = %lld", (long long)rotation->table_rows);
        if (!rotation->cos || !rotation->sin)
            return fail(CFZ_ERR_NULL, "the rotation's cos and sin are required");
        if (!aligned(rotation->cos, 16) || !aligned(rotation->sin, 16) ||
            !aligned(rotation->positions, 4))
            return fail(CFZ_ERR_ALIGN, "cos and sin must be 16-byte, positions 4-byte aligned");
        rot = cfz::Kv8Rotation{rotation->cos,        rotation->sin,     rotation->positions,
                               rotation->table_rows, rotation->rot_dim, rotation->interleaved != 0};
    }
    bound_rows(&b);
    if (empty(b))
        return CFZ_OK;
    CFZ_TRY(check_pages(c, b));
    CFZ_TRY(check_pointers(c, b));
    if (!k || !v)
        return fail(CFZ_ERR_NULL, "k and v are required");
    if (!aligned(k, 16) || !aligned(v, 16))
        return fail(CFZ_ERR_ALIGN, "k and v must be 16-byte aligned");
    return hip_status(cfz::launch_kv8_append(c, b, dtype, k, v, k_stride, v_stride, rot,
                                             (hipStream_t)hip_stream),
                      "append launch");
}

cfz_status cfz_kv8_gather(const cfz_kv8_cache *cache, const cfz_kv8_batch *batch,
                          cfz_kv8_dtype dtype, void *k, void *v, void *hip_stream)
{
    cfz::Kv8Cache c;
    cfz::Kv8Batch b;
    CFZ_TRY(check_sizes(cache, batch, &c, &b));
    CFZ_TRY(check_dtype(dtype, true));
    bound_rows(&b);
    if (empty(b) || (!k && !v))
        return CFZ_OK;
    CFZ_TRY(check_pointers(c, b));
    if (!aligned(k, 16) || !aligned(v, 16))
        return fail(CFZ_ERR_ALIGN, "k and v must be 16-byte aligned");
    CFZ_TRY(check_pages(c, b));
    return hip_status(cfz::launch_kv8_gather(c, b, dtype, k, v, (hipStream_t)hip_stream),
                      "gather launch");
}

size_t cfz_kv8_attend_workspace_bytes(const cfz_kv8_cache *cache, const cfz_kv8_batch *batch,
                                      int32_t q_heads, int64_t max_kv,
                                      const cfz_kv8_blocks *blocks)
{
    cfz::Kv8Cache c;
    cfz::Kv8Batch b;
    if (check_sizes(cache, batch, &c, &b) != CFZ_OK ||
        check_queries(c, b, q_heads, max_kv, blocks) != CFZ_OK || empty(b))
        return 0;
    if (!blocks)
        bound_rows(&b);
    const cfz::Kv8Plan p = cfz::kv8_plan(c, b, q_heads, max_kv, blocks != nullptr,
                                         blocks ? blocks->q_block : 1, blocks ? blocks->count : 0);
    return (size_t)p.ws_bytes;
}

cfz_status cfz_kv8_attend(const cfz_kv8_cache *cache, const cfz_kv8_batch *batch,
                          cfz_kv8_dtype dtype, const void *q, int64_t q_stride, int32_t q_heads,
                          int32_t causal, float scale, int64_t max_kv,
                          const cfz_kv8_blocks *blocks, void *out, int64_t out_stride, float *lse,
                          void *workspace, size_t ws_bytes, void *hip_stream)
{
    cfz::Kv8Cache c;
    cfz::Kv8Batch b;
    CFZ_TRY(check_sizes(cache, batch, &c, &b));
    CFZ_TRY(check_dtype(dtype, false));
    CFZ_TRY(check_queries(c, b, q_heads, max_kv, blocks));
    const int64_t row = (int64_t)q_heads * c.dim;
    CFZ_TRY(check_stride(q_stride, row, dtype, "q_stride"));
    CFZ_TRY(check_stride(out_stride, row, dtype, "out_stride"));
    if (!(scale > 0.0f) || !isfinite(scale))
        return fail(CFZ_ERR_SHAPE, "scale = %g must be finite and positive", (double)scale);
    if (!blocks)
        bound_rows(&b);
    if (empty(b))
        return CFZ_OK;
    const cfz::Kv8Plan p = cfz::kv8_plan(c, b, q_heads, max_kv, blocks != nullptr,
                                         blocks ? blocks->q_block : 1, blocks ? blocks->count : 0);
    CFZ_TRY(check_groups(p.whole));
    CFZ_TRY(check_pointers(c, b));
    if (!q || !out || (blocks && !blocks->blocks))
        return fail(CFZ_ERR_NULL, "q, out and the block lists are required");
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
        (blocks && !aligned(blocks->blocks, 4)))
        return fail(CFZ_ERR_ALIGN, "q and out must be 16-byte, lse and lists 4-byte aligned");
    CFZ_TRY(check_workspace(workspace, ws_bytes, (size_t)p.ws_bytes));
    cfz::Kv8Attend a;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.ws = (float *)workspace;
    a.blocks = blocks ? blocks->blocks : nullptr;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.q_block = blocks && blocks->q_block < b.max_rows ? blocks->q_block : b.max_rows;
    a.max_kv = max_kv;
    a.q_heads = q_heads;
    a.group = q_heads / c.heads;
    a.count = blocks ? blocks->count : 0;
    a.causal = causal != 0;
    a.f16 = dtype == CFZ_KV8_F16;
    a.scale = scale;
    return hip_status(cfz::launch_kv8_attend(c, b, a, p, (hipStream_t)hip_stream),
                      "attention launch");
}

size_t cfz_kv8_select_workspace_bytes(const cfz_kv8_cache *cache, const cfz_kv8_batch *batch,
                                      int64_t max_kv, const cfz_kv8_blocks *blocks)
{
    cfz::Kv8Cache c;
    cfz::Kv8Batch b;
    if (check_sizes(cache, batch, &c, &b) != CFZ_OK || !blocks ||
        check_queries(c, b, c.heads, max_kv, blocks) != CFZ_OK || empty(b))
        return 0;
    return cfz::kv8_select_workspace_bytes(c, b, max_kv, blocks->q_block);
}

cfz_status cfz_kv8_select(const cfz_kv8_cache *cache, const cfz_kv8_batch *batch,
                          cfz_kv8_dtype dtype, const void *q, int64_t q_stride, int32_t q_heads,
                          int32_t causal, int64_t max_kv, int32_t first, int32_t last,
                          const cfz_kv8_blocks *blocks, void *workspace, size_t ws_bytes,
                          void *hip_stream)
{
    cfz::Kv8Cache c;
    cfz::Kv8Batch b;
    CFZ_TRY(check_sizes(cache, batch, &c, &b));
    CFZ_TRY(check_dtype(dtype, false));
    if (!blocks)
        return fail(CFZ_ERR_NULL, "blocks is required");
    CFZ_TRY(check_queries(c, b, q_heads, max_kv, blocks));
    CFZ_TRY(check_stride(q_stride, (int64_t)q_heads * c.dim, dtype, "q_stride"));
    if (first < 0 || last < 0 || (int64_t)first + last > blocks->count)
        return fail(CFZ_ERR_SHAPE, "first = %d, last = %d with count = %d", first, last,
                    blocks->count);
    const int64_t pages = (max_kv + c.page - 1) / c.page;
    if (pages > (1 << 20))
        return fail(CFZ_ERR_SHAPE, "%lld pages per sequence (at most 2^20)", (long long)pages);
    if (empty(b))
        return CFZ_OK;
    const double lists =
        (double)((b.max_rows + blocks->q_block - 1) / blocks->q_block) * c.heads * b.batch;
    CFZ_TRY(check_groups(lists * ((double)(pages + 63) / 64 + 1)));
    CFZ_TRY(check_pointers(c, b));
    if (!q || !blocks->blocks || (c.pages > 0 && !c.km))
        return fail(CFZ_ERR_NULL, "q, the block lists and the cache's k_mean are required");
    if (!aligned(q, 16) || !aligned(blocks->blocks, 4))
        return fail(CFZ_ERR_ALIGN, "q must be 16-byte, the block lists 4-byte aligned");
    CFZ_TRY(check_workspace(workspace, ws_bytes,
                            cfz::kv8_select_workspace_bytes(c, b, max_kv, blocks->q_block)));
    cfz::Kv8Select a;
    a.q = q;
    a.q_stride = q_stride;
    a.blocks = blocks->blocks;
    a.ws = (double *)workspace;
    a.q_block = blocks->q_block;
    a.max_kv = max_kv;
    a.q_heads = q_heads;
    a.group = q_heads / c.heads;
    a.count = blocks->count;
    a.causal = causal != 0;
    a.f16 = dtype == CFZ_KV8_F16;
    a.first = first;
    a.last = last;
    return hip_status(cfz::launch_kv8_select(c, b, a, (hipStream_t)hip_stream), "select launch");
}

}  // extern "C"
