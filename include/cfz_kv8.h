/*
 * cfz_kv8.h -- C ABI of libcfz's 8-bit paged K/V cache: appending keys and values
 * with the position rotation applied on the way, reading tokens back, attention
 * over the cache, and attention over pages that a cheap score selects.
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

#ifdef __cplusplus
}
#endif

#endif /* CFZ_KV8_H */
