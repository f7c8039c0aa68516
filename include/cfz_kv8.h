/*
 * cfz_kv8.h -- C ABI of libcfz's 8-bit paged K/V cache: appending keys and values
 * with the position rotation applied on the way, reading tokens back, attention
 * over the cache, attention over pages that a cheap score selects, and the
 * management of a pool's pages (cfz_kv8_free and below).
 *
 * What the codec of cfz.h rebuilds on a receiving device -- one layer's K and V of
 * another device's share -- goes into such a cache, and the device's own queries
 * attend over all shares (paper: reproducibility table, "Pseudocode", Algorithm 1:
 * project QKV, exchange K and V, attention).  The cache holds 8-bit codes with one
 * scale per page and head: the quantizer of cfz_compress at 8 bits, a page of one
 * head being the group.
 *
 * Conventions are those of cfz.h: device pointers are caller-owned and 16-byte
 * aligned, work is enqueued asynchronously on `hip_stream` of the current device,
 * arguments are validated before anything is enqueued, and a non-OK status means
 * that nothing was queued (CFZ_ERR_HIP may leave the launches before the failing
 * one queued).  Offsets, lengths, tables and block lists live on the device and
 * are not read by the host; the kernels bound every one of them: offsets are
 * clamped to [0, tokens], lengths to [0, table_width * page_tokens], and a page
 * number outside [0, pages) is a page that holds nothing -- its tokens are not
 * written, not attended to, never selected, and read back as zeros.
 */
#ifndef CFZ_KV8_H
#define CFZ_KV8_H

#include "cfz.h"

#ifdef __cplusplus
extern "C" {
#endif

/* INT8: qmax = 127, codes are the integers -127..127 (never -128).
 * E4M3: qmax = 448, codes are 8-bit floating point (1 sign, 4 exponent, 3 mantissa
 * bits; no infinities), never NaN. */
typedef enum { CFZ_KV8_INT8 = 0, CFZ_KV8_E4M3 = 1 } cfz_kv8_format;

typedef enum { CFZ_KV8_BF16 = 0, CFZ_KV8_F16 = 1, CFZ_KV8_F32 = 2 } cfz_kv8_dtype;

/* A pool of pages.  head_dim in {64, 128}, page_tokens in {32, 64, 128},
 * 1 <= kv_heads <= 1024, 0 <= pages < 2^31.
 *   k:       [pages][kv_heads][page_tokens][head_dim] codes
 *   v:       [pages][kv_heads][head_dim][page_tokens] codes (dimension-major: the
 *            order in which the product with the weights reads them)
 *   k_scale, v_scale: [pages][kv_heads] fp32, finite and >= 0 wherever tokens are held
 *   k_mean:  [pages][kv_heads][head_dim] fp32, the mean of the page's keys as held
 *            (scale times code); may be NULL if cfz_kv8_select is not used.
 * Together 2 * kv_heads * head_dim bytes a token.  Element counts may pass 2^32. */
typedef struct {
    int64_t pages;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t page_tokens;
    int32_t format;      /* cfz_kv8_format */
    void *k;
    void *v;
    float *k_scale;
    float *v_scale;
    float *k_mean;
} cfz_kv8_cache;

/* A ragged batch.  Token i of sequence b lives in page
 * page_table[b * table_width + i / page_tokens], slot i % page_tokens; no page may
 * serve two places that one call writes.
 *   offsets: [batch + 1] int32, ascending: rows offsets[b] .. offsets[b + 1] - 1 of the
 *            call's token rows (`tokens` rows in all) belong to sequence b.  Rows
 *            outside every sequence are neither read nor written.
 *   lengths: [batch] int32.  append: tokens the sequence holds before the call;
 *            gather: the first token to read; attend, select: tokens it holds.
 *   max_rows: an upper bound of the rows of one sequence, known on the host; rows
 *            past it are left out.
 * 0 <= batch <= 65535, 1 <= table_width, table_width * page_tokens < 2^31,
 * 0 <= tokens < 2^31 (0 is a no-op: nothing is written, cfz_kv8_select's lists neither).  The integer arrays need 4-byte alignment only.
 * A call that would need 2^23 or more work-groups (append: about one for the keys and
 * one for the values of each page and head) is refused. */
typedef struct {
    int32_t batch;
    int32_t table_width;
    const int32_t *page_table;
    const int32_t *offsets;
    const int32_t *lengths;
    int64_t tokens;
    int64_t max_rows;
} cfz_kv8_batch;

/* The rotation of the keys: the first rot_dim dimensions (a multiple of 8, at most
 * head_dim) of a token's key are rotated in pairs by angles given as rows of cos and
 * sin, [table_rows][rot_dim / 2] fp32 each: (a, b) -> (a cos - b sin, a sin + b cos).
 * Pair i is (i, i + rot_dim / 2), or (2 i, 2 i + 1) if interleaved.  positions[t]
 * (int32, one for each token row) is the row for token row t; NULL: the token's index
 * in its sequence.  Rows outside the table take the nearest one.  cos and sin are
 * 16-byte aligned. */
typedef struct {
    const float *cos;
    const float *sin;
    const int32_t *positions;
    int64_t table_rows;
    int32_t rot_dim;
    int32_t interleaved;
} cfz_kv8_rotation;

/* Appends each sequence's token rows behind the lengths[b] tokens that it holds.
 * k, v: rows of kv_heads * head_dim values of `dtype`, row t at k + t * k_stride (strides in
 * elements, multiples of 16 bytes, >= kv_heads * head_dim).  rotation NULL: none.
 * For each page and head that gets tokens, K and V each on its own:
 *   scale' = max(scale if older tokens stay in the page, fp32(max |x| / qmax)) over
 *   the new (rotated) values x; a new code is the one nearest to x / scale', ties to even
 *   (0 where scale' is 0); if scale' > scale, the codes c of the older tokens become
 *   the nearest to c scale / scale'; k_mean (if given) becomes scale' times the mean
 *   code of the tokens now held.
 * Rotation, quotients and means are evaluated in 64 bits, so a value next to the
 * border between two codes falls on its own side.  NaN is stored as 0 and an infinity
 * as the largest code of its sign; neither counts in max |x|.  Tokens that the pages held
 * behind the appended ones are no longer part of the sequence (their codes stay as
 * they were).  Writing whole pages again (lengths[b] back at a page border) replaces a
 * share, as each denoising step does.  Tokens past the table's end are left out.
 * Errors: CFZ_ERR_NULL, CFZ_ERR_SHAPE, CFZ_ERR_UNSUPPORTED, CFZ_ERR_ALIGN, CFZ_ERR_HIP. */
cfz_status cfz_kv8_append(const cfz_kv8_cache *cache, const cfz_kv8_batch *batch,
                          cfz_kv8_dtype dtype, const void *k, const void *v, int64_t k_stride,
                          int64_t v_stride, const cfz_kv8_rotation *rotation, void *hip_stream);

/* Reads tokens back: token row offsets[b] + i gets token lengths[b] + i of sequence b
 * as scale times code, rounded to fp32 and then to `dtype`; k, v: dense rows [tokens][kv_heads][head_dim],
 * either may be NULL.  Tokens past the table's end read as zeros.
 * Errors: as cfz_kv8_append. */
cfz_status cfz_kv8_gather(const cfz_kv8_cache *cache, const cfz_kv8_batch *batch,
                          cfz_kv8_dtype dtype, void *k, void *v, void *hip_stream);

/* Pages picked for blocks of q_block consecutive queries of a sequence (the last
 * block may be short): blocks[((b * ceil(max_rows / q_block) + i / q_block) * kv_heads + h)
 * * count + j], j < count, are logical page indices of sequence b for its query i and
 * KV head h, each at most once, padded with -1.  q_block >= 1, 1 <= count <= 4096. */
typedef struct {
    int32_t *blocks;
    int32_t count;
    int32_t q_block;
} cfz_kv8_blocks;

/* Softmax attention of the batch's query rows over the cache:
 *   out = sum_t softmax_t(scale * q . k_t) v_t,  lse = log sum_t exp(scale * q . k_t).
 * q: rows of q_heads * head_dim values of `dtype` (BF16 or F16), row t at q + t * q_stride
 * (elements; a multiple of 8); q_heads a multiple of kv_heads (at most 64 query heads to
 * one; at most 2^30 rows of queries and query heads to one KV head), query head h reads KV head h / (q_heads / kv_heads).  out: like q, row stride
 * out_stride.  lse: [tokens][q_heads] fp32 or NULL.
 * Query i of n sees the tokens t < length, and with causal != 0 only t <= length - n + i.
 * blocks (NULL: all pages) restricts it to its block's listed pages.  A row that sees
 * nothing gets out = 0 and lse = -infinity.
 * max_kv: an upper bound of the lengths, known on the host (it decides into how many
 * parts the keys are split; longer sequences are cut off there), at most 2^30.  scale is finite
 * and > 0.  The products run on the codes in fp16 (which holds every code exactly; each
 * query row is first scaled by a power of two, so that a bf16 or fp16 q is held exactly down to
 * 2^-29 of its largest entry), accumulate in fp32, and the weights enter the second
 * product rounded to fp16; the softmax statistics are fp32.  Value scales of 2^-100
 * or less count as 0; others may lie as far apart as fp32 has them (outside of 2^-32 ..
 * 2^32 the denominators are summed on their own, which takes longer).  Results do not
 * depend on the run.
 * workspace: cfz_kv8_attend_workspace_bytes(...) bytes, 256-byte aligned (may be NULL
 * if that is 0), overwritten by the call; calls that may run at the same time need one
 * each.  q, out and lse must not overlap.
 * Errors: CFZ_ERR_NULL, CFZ_ERR_SHAPE, CFZ_ERR_UNSUPPORTED, CFZ_ERR_ALIGN,
 * CFZ_ERR_WORKSPACE, CFZ_ERR_HIP. */
cfz_status cfz_kv8_attend(const cfz_kv8_cache *cache, const cfz_kv8_batch *batch,
                          cfz_kv8_dtype dtype, const void *q, int64_t q_stride, int32_t q_heads,
                          int32_t causal, float scale, int64_t max_kv,
                          const cfz_kv8_blocks *blocks, void *out, int64_t out_stride, float *lse,
                          void *workspace, size_t ws_bytes, void *hip_stream);
/* 0 if none is needed or the arguments are invalid. */
size_t cfz_kv8_attend_workspace_bytes(const cfz_kv8_cache *cache, const cfz_kv8_batch *batch,
                                      int32_t q_heads, int64_t max_kv,
                                      const cfz_kv8_blocks *blocks);

/* Picks pages: for each block of q_block queries and each KV head, page p of the
 * sequence scores s_p = (sum of the block's queries, over the query heads that share the
 * KV head) . k_mean[p], in 64 bits.  Pages that hold a token which the block's last query
 * sees can be picked; the first `first` and the last `last` of those always are
 * (first + last <= count), then the highest scores, ties going to the lower index.
 * blocks->blocks gets the indices in ascending order, -1 behind them; the lists of
 * query blocks that a sequence does not have are filled with -1.  A score that is NaN counts
 * as the lowest.  k_mean is required.  Arguments as cfz_kv8_attend; pages per sequence
 * (max_kv / page_tokens, rounded up) at most 2^20.
 * workspace: cfz_kv8_select_workspace_bytes(...) bytes, 256-byte aligned.
 * Errors: as cfz_kv8_attend. */
cfz_status cfz_kv8_select(const cfz_kv8_cache *cache, const cfz_kv8_batch *batch,
                          cfz_kv8_dtype dtype, const void *q, int64_t q_stride, int32_t q_heads,
                          int32_t causal, int64_t max_kv, int32_t first, int32_t last,
                          const cfz_kv8_blocks *blocks, void *workspace, size_t ws_bytes,
                          void *hip_stream);
size_t cfz_kv8_select_workspace_bytes(const cfz_kv8_cache *cache, const cfz_kv8_batch *batch,
                                      int64_t max_kv, const cfz_kv8_blocks *blocks);

/* ---- managing pages
 *
 * Which row of a page table holds which page of a pool.  page_table: [batch][table_width]
 * int32, -1 where a row has no page; lengths: [batch] tokens held; refs: [pages] int32, how many
 * places of the table name each page (0: free).  The arrays live on the device, and the calls keep
 * them in line with each other.  Layers whose caches have the same sizes can share
 * them: each call's page moves are then done in every layer's cache (cfz_kv8_copy).  A place that
 * names no page of 0 .. pages - 1 counts as -1; lengths count as clamped to
 * [0, table_width * page_tokens].  Limits as in cfz_kv8_cache and cfz_kv8_batch, batch >= 1.
 * The results of every call are the same whatever the order in which its parts run; calls that
 * change the same table run one after the other (on one stream, or ordered by the caller), and
 * so do a change and the attention that reads the table. */
typedef struct {
    int64_t pages;
    int32_t batch;
    int32_t table_width;
    int32_t page_tokens;
    int32_t *page_table;
    int32_t *lengths;
    int32_t *refs;
} cfz_kv8_pages;

/* Cuts rows rows[i], i < count, off behind their first keep[i] tokens (keep NULL or below 0: 0): places
 * behind ceil(keep / page_tokens) become -1 and let go of their pages, lengths become at most
 * keep.  Rows outside the table are left out; one that is listed twice keeps the least.
 * 0 <= count <= 65535.
 * Errors: CFZ_ERR_NULL, CFZ_ERR_SHAPE, CFZ_ERR_UNSUPPORTED, CFZ_ERR_ALIGN, CFZ_ERR_HIP. */
cfz_status cfz_kv8_free(const cfz_kv8_pages *pages, int32_t count, const int32_t *rows,
                        const int32_t *keep, void *hip_stream);

/* Row children[i] becomes a second holder of row parents[i]'s pages and length, i < count; what
 * it held before is let go of.  No page is copied: cfz_kv8_reserve gives a row a copy of its own of the page
 * that it is about to write.  A pair is left out if one of its rows is outside the table, if both
 * are the same, if an earlier pair has the same child, or if its child is the parent of any pair.
 * 0 <= count <= 65535; every pair is held against all others (15 us for 4096, 0.5 ms for 32,000).
 * Errors: as cfz_kv8_free. */
cfz_status cfz_kv8_fork(const cfz_kv8_pages *pages, int32_t count, const int32_t *parents,
                        const int32_t *children, void *hip_stream);

/* Makes room for counts[b] more tokens (at most max_new; below 0: 0) behind the lengths[b] of each
 * row: the places of tokens lengths[b] .. lengths[b] + counts[b] - 1 that have no page get a free one,
 * and those whose page other rows hold too get a page of their own -- except that, where all holders
 * of a page are among this call's places, the first of them keeps it.  Free pages are given out from the lowest
 * up, to the places row by row.  Where such a place already holds tokens of its row (lengths[b] inside a
 * page), source[b] and target[b] (int32 [batch] each) get the old and the new page, whose contents the
 * caller then copies (cfz_kv8_copy); otherwise they are -1.  Lengths stay as they are, so
 * calling twice gives out nothing twice.  Places past the table's end are left out
 * (cfz_kv8_reserve_rows says how many tokens that costs).
 * missing[0] gets 0 -- or, where there are not enough free pages, how many more it takes: then nothing
 * is given out.
 * One work-group: about 4 us for every 1024 places (rows times the pages that max_new tokens reach).
 * workspace: cfz_kv8_reserve_workspace_bytes(...) bytes, 256-byte aligned, overwritten.
 * Errors: as cfz_kv8_free, and CFZ_ERR_WORKSPACE. */
cfz_status cfz_kv8_reserve(const cfz_kv8_pages *pages, const int32_t *counts, int64_t max_new,
                           int32_t *source, int32_t *target, int32_t *missing, void *workspace,
                           size_t ws_bytes, void *hip_stream);
/* cfz_kv8_reserve that also says which rows are full: left_out[b] (int32 [batch]) gets how many of the
 * counts[b] tokens have no place, those past max_new or past the table's end, whatever missing[0] is.
 * The caller's lengths go on by counts[b] - left_out[b] (counts below 0 as 0): cfz_kv8_append drops the others. */
cfz_status cfz_kv8_reserve_rows(const cfz_kv8_pages *pages, const int32_t *counts, int64_t max_new,
                                int32_t *source, int32_t *target, int32_t *missing,
                                int32_t *left_out, void *workspace, size_t ws_bytes,
                                void *hip_stream);
/* 0 if none is needed or the arguments are invalid. */
size_t cfz_kv8_reserve_workspace_bytes(const cfz_kv8_pages *pages, int64_t max_new);

/* Moves the pages in use to the front of the pool: with n of them, the highest page in use goes to
 * the lowest free one until all lie in 0 .. n - 1.  live[0] gets n, moves[0] their number m, and
 * source[i], target[i], i < m, the moves (int32 [pages / 2] each); table and refs are
 * changed, the pages' contents are the caller's to copy (cfz_kv8_copy with used = moves).
 * workspace: cfz_kv8_compact_workspace_bytes(...) bytes, 256-byte aligned, overwritten.
 * Errors: as cfz_kv8_reserve. */
cfz_status cfz_kv8_compact(const cfz_kv8_pages *pages, int32_t *source, int32_t *target,
                           int32_t *live, int32_t *moves, void *workspace, size_t ws_bytes,
                           void *hip_stream);
size_t cfz_kv8_compact_workspace_bytes(const cfz_kv8_pages *pages);

/* Copies whole pages, codes, scales and mean keys: page source[i] of `from` (NULL: `to` itself) to page
 * target[i] of `to`, for i < count and, if used is given, i < used[0] (int32 on the device).  A
 * pair that names a page outside its pool is left out.  A target must not be another pair's target,
 * nor (in the same cache) its source: such pages would hold parts of either.  The caches have the same heads, head_dim,
 * page_tokens and format; from needs k_mean if to has it.  0 <= count < 2^31.
 * Errors: as cfz_kv8_free. */
cfz_status cfz_kv8_copy(const cfz_kv8_cache *to, const cfz_kv8_cache *from, int64_t count,
                        const int32_t *source, const int32_t *target, const int32_t *used,
                        void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* CFZ_KV8_H */
