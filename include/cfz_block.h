/*
 * cfz_block.h -- C ABI of what lies between a transformer layer's residual stream and
 * the 8-bit K/V cache of cfz_kv8.h: the norms around a block with its gate and its
 * residual sum, the rotation of queries and keys by their positions, and the low-rank
 * adapters of many requests beside a projection that they share.
 *
 * Conventions are those of cfz.h and cfz_kv8.h: device pointers are caller-owned and 16-byte
 * aligned (integer arrays 4-byte), work is enqueued asynchronously on `hip_stream` of the
 * current device, arguments are validated before anything is enqueued, and a non-OK status
 * means that nothing was queued.  Types are numbered as cfz_kv8_dtype.  Offsets, positions and
 * adapter numbers live on the device and are not read by the host; the kernels bound every
 * one of them.  Sums and statistics are fp32, results are rounded once (nearest even).
 */
#ifndef CFZ_BLOCK_H
#define CFZ_BLOCK_H

#include "cfz_kv8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A norm over the columns of a row:
 *   RMS:   v / sqrt(mean(v^2) + eps) * weight
 *   LAYER: (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) * weight + bias
 * weight and bias: [cols] of `dtype`, or NULL (1 and 0; a bias goes with LAYER only).  eps is
 * finite and >= 0.  Rows whose squares vanish in fp32 or leave its range are scaled by a power of two
 * before they are squared; what may overflow is a LAYER norm's sum of values past 2^127 / cols.  A row
 * that is 0 (or all of one value, LAYER) with eps = 0 is 0 / 0. */
typedef enum { CFZ_NORM_NONE = 0, CFZ_NORM_RMS = 1, CFZ_NORM_LAYER = 2 } cfz_norm_kind;
typedef struct {
    int32_t kind;
    float eps;
    const void *weight;
    const void *bias;
    int32_t dtype; /* F32, or the call's y_dtype */
} cfz_norm;

/* A row of `cols` values for each item of a batch, item b's at data + b * stride (elements;
 * 0: one row for all).  data NULL: none. */
typedef struct {
    const void *data;
    int64_t stride;
    int32_t dtype; /* F32, or the call's y_dtype */
} cfz_item_rows;

/* One step along the residual stream, row by row:
 *   r = x + (gate_scale * gate) * after(y)
 *   h = before(r) * (1 + scale) + shift
 * x: rows of x_dtype (the stream's type), y: rows of y_dtype (the block's output; NULL: r = x),
 * r like x, h like y.  h is computed from the sum before its rounding to x_dtype.  r NULL: the
 * sum is not stored; h NULL: no second norm (before is then not looked at).  x_dtype is
 * y_dtype or F32.  after and before may be of kind NONE.
 * cols: a multiple of 8, 8 .. 16384; row strides in elements, >= cols, multiples of 16
 * bytes.  0 <= tokens < 2^31, 1 <= batch <= 65535; 2^23 or more work-groups (of a row, or of 4 to 32
 * rows of up to 512 to 64 columns) are refused.
 * offsets: [batch + 1] int32, ascending: rows offsets[b] .. offsets[b + 1] - 1 belong to item b;
 * rows outside every item are left as they are in r and h.  NULL: batch equal runs (tokens a
 * multiple of batch).
 * r may be x, and h may be y, with the same stride; other overlaps are not allowed.
 * Errors: CFZ_ERR_NULL, CFZ_ERR_SHAPE, CFZ_ERR_UNSUPPORTED, CFZ_ERR_ALIGN, CFZ_ERR_HIP. */
typedef struct {
    int64_t tokens;
    int32_t cols;
    int32_t batch;
    const int32_t *offsets;
    int32_t x_dtype;
    int32_t y_dtype;
    const void *x;
    int64_t x_stride;
    const void *y;
    int64_t y_stride;
    void *r;
    int64_t r_stride;
    void *h;
    int64_t h_stride;
    float gate_scale;
    cfz_item_rows gate;
    cfz_item_rows scale;
    cfz_item_rows shift;
    cfz_norm after;
    cfz_norm before;
} cfz_residual;
cfz_status cfz_residual_norm(const cfz_residual *args, void *hip_stream);

/* Tables for cfz_kv8_rotation: row t of cos and sin, [rows][rot_dim / 2] fp32, holds
 * amplitude * cos(a) and amplitude * sin(a) of the angles a = position * speed, computed in
 * 64 bits.  rot_dim: a multiple of 8, 8 .. 256.  The pairs are dealt out to `axes` (1 .. 4)
 * axes in turn: axis j has axis_dim[j] / 2 of them (even, >= 2, rot_dim in all) with
 *   speed_i = base^(-2 i / axis_dim[j]),  i = 0 .. axis_dim[j] / 2 - 1,
 * and row t's position on it is positions[t * axes + j] (int32; NULL: t, with one axis).
 * scaling stretches the tables over contexts `factor` times as long:
 *   LINEAR: speed / factor;
 *   BASE:   base * factor^(d / (d - 2)) for base, d = axis_dim[j] > 2;
 *   PARTS:  speed * (k + (1 - k) / factor), k = clamp((n - slow) / (fast - slow), 0, 1), where n
 *           = trained * speed / (2 pi) is how often the pair turned over the trained length.
 * base > 1, factor > 0, amplitude finite and > 0; PARTS: trained > 0, 0 <= slow < fast.
 * Errors: CFZ_ERR_NULL, CFZ_ERR_SHAPE, CFZ_ERR_UNSUPPORTED, CFZ_ERR_ALIGN, CFZ_ERR_HIP. */
typedef enum {
    CFZ_ROTATION_PLAIN = 0,
    CFZ_ROTATION_LINEAR = 1,
    CFZ_ROTATION_BASE = 2,
    CFZ_ROTATION_PARTS = 3
} cfz_rotation_scaling;
typedef struct {
    int32_t rot_dim;
    int32_t axes;
    int32_t axis_dim[4];
    int32_t scaling;
    double base;
    double factor;
    double trained;
    double slow;
    double fast;
    double amplitude;
} cfz_rotation_angles;
cfz_status cfz_rotation_table(const cfz_rotation_angles *angles, int64_t rows,
                              const int32_t *positions, float *cos, float *sin,
                              void *hip_stream);

/* Rows of `heads` heads to be turned: row t at x + t * x_stride, its result at out + t *
 * out_stride (elements, multiples of 16 bytes, >= heads * head_dim).  weight: [head_dim] of
 * weight_dtype (F32, or the call's dtype), or NULL.  out may be x with the same stride; other
 * overlaps are not allowed. */
typedef struct {
    const void *x;
    int64_t x_stride;
    void *out;
    int64_t out_stride;
    int32_t heads;
    const void *weight;
    int32_t weight_dtype;
} cfz_rotate_rows;

/* Norm and rotation of each head, for up to 4 tensors (queries and keys) of the same tokens:
 *   v = x / sqrt(mean(x^2) + eps) * weight over a head (if `normed`, else v = x),
 * and the first rot_dim dimensions of v turned in pairs as cfz_kv8_append turns keys.
 * Heads whose squares vanish in fp32 or leave its range are scaled by a power of two before they are
 * squared; a head that is 0 with eps = 0 is 0 / 0.
 * rotation NULL: the norm alone.  Without rotation->positions, row i of sequence b is at position
 * starts[b] + i (starts NULL: i).  Positions outside the table take its nearest row.
 * head_dim in {32, 64, 128, 256}, rot_dim a multiple of 8 up to it, heads 1 .. 1024 each.
 * offsets: [batch + 1] int32 as above, rows outside are left as they are in out; NULL: one
 * sequence (batch = 1).  0 <= tokens < 2^31, 1 <= batch <= 65535; 2^23 or more work-groups (of four
 * runs of up to 2048 values of a token in a tensor) are refused.
 * Errors: as cfz_residual_norm. */
cfz_status cfz_rotate(int32_t count, const cfz_rotate_rows *tensors, cfz_kv8_dtype dtype,
                      int32_t head_dim, int64_t tokens, int32_t batch, const int32_t *offsets,
                      const int32_t *starts, const cfz_kv8_rotation *rotation, int32_t normed,
                      float eps, void *hip_stream);

/* Low-rank adapters of one projection, to be added beside it for several requests at once.
 *   a: [adapters][slices * rank][cols_in] of `dtype` (BF16 or F16), laid out by cfz_adapters_put:
 *      for each adapter [ceil(slices * rank / 16)][4 ceil(cols_in / 128)][4][16][8], row 16 i + m's
 *      column 32 k + 8 q + e at [i][k][q][m][e], zeros past either end; cfz_adapters_a_bytes bytes;
 *   b: [adapters][cols_out][rank] of `dtype`, scale: [adapters] fp32 or NULL (1).
 * The projection's columns are dealt out to 1 .. 4 slices (query, key and value of one fused
 * projection) of slice_cols[i] columns each, multiples of 16, cols_out in all; slice i's columns
 * are met by adapter rows i * rank .. (i + 1) * rank - 1 of a.  rank: a multiple of 8, 8 .. 128
 * (lower ranks: zeros).  cols_in: a multiple of 8, 8 .. 2^20;
 * cols_out at most 2^20; 1 <= adapters <= 2^20. */
typedef struct {
    int32_t adapters;
    int32_t slices;
    int32_t rank;
    int32_t cols_in;
    int32_t slice_cols[4];
    int32_t dtype;
    void *a;
    const void *b;
    const float *scale;
} cfz_adapters;

/* Bytes of the laid-out a; 0 if the arguments are invalid. */
size_t cfz_adapters_a_bytes(const cfz_adapters *adapters);
/* Lays out the rows [count][slices * rank][cols_in] of adapters first .. first + count - 1 in
 * adapters->a (b, scale are not looked at).  2^31 or more pieces of 16 bytes a call are refused.
 * Errors: CFZ_ERR_NULL, CFZ_ERR_SHAPE, CFZ_ERR_UNSUPPORTED, CFZ_ERR_ALIGN, CFZ_ERR_HIP. */
cfz_status cfz_adapters_put(const cfz_adapters *adapters, int32_t first, int32_t count,
                            const void *rows, void *hip_stream);

/* out = y + scale_a (x a^T) b^T for the token rows offsets[b] .. offsets[b + 1] - 1 of sequence b, with
 * adapter ids[b] (outside of 0 .. adapters - 1: none, out = y, every bit).  x: rows of `dtype`; y and out: rows
 * of y_dtype (dtype or F32); row strides in elements, multiples of 16 bytes.  out may be y with the same
 * stride; other overlaps are not allowed.  Rows of no sequence, and rows past a sequence's first
 * max_rows, are neither read nor written.  The products accumulate in fp32; x a^T enters the second one as the sum of
 * two numbers of `dtype` (off by 2^-16 of itself for BF16, 2^-21 of its row's largest value for F16).
 * Results do not depend on the run.  2^23 or more work-groups (of 64 tokens x 256 columns of a slice) are
 * refused.
 * workspace: cfz_adapters_workspace_bytes(...) bytes, 256-byte aligned, overwritten; calls that may
 * run at the same time need one each.
 * Errors: CFZ_ERR_NULL, CFZ_ERR_SHAPE, CFZ_ERR_UNSUPPORTED, CFZ_ERR_ALIGN, CFZ_ERR_WORKSPACE,
 * CFZ_ERR_HIP. */
cfz_status cfz_adapters_add(const cfz_adapters *adapters, int64_t tokens, int32_t batch,
                            const int32_t *offsets, const int32_t *ids, int64_t max_rows,
                            const void *x, int64_t x_stride, const void *y, int64_t y_stride,
                            void *out, int64_t out_stride, int32_t y_dtype, void *workspace,
                            size_t ws_bytes, void *hip_stream);
/* 0 if none is needed or the arguments are invalid. */
size_t cfz_adapters_workspace_bytes(const cfz_adapters *adapters, int64_t tokens, int32_t batch);

#ifdef __cplusplus
}
#endif

#endif /* CFZ_BLOCK_H */
