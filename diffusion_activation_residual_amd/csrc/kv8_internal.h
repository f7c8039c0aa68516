// kv8_internal.h -- declarations shared by the sources of the 8-bit K/V cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "cfz_kv8.h"

namespace cfz {

// The cache and the batch as the kernels take them (checked by the API).
struct Kv8Cache {
    uint8_t *k, *v;
    float *ks, *vs, *km;
    int64_t pages;
    int heads, dim, page, log2page, fmt;
};

struct Kv8Batch {
    const int32_t *table, *off, *len;
    int64_t tokens, max_rows;
    int batch, width;
};

struct Kv8Rotation {
    const float *cos, *sin;  // null: no rotation
    const int32_t *pos;
    int64_t rows;
    int dim, interleaved;
};

hipError_t launch_kv8_append(const Kv8Cache &c, const Kv8Batch &b, int dtype, const void *k,
                             const void *v, int64_t k_stride, int64_t v_stride,
                             const Kv8Rotation &rot, hipStream_t st);
hipError_t launch_kv8_gather(const Kv8Cache &c, const Kv8Batch &b, int dtype, void *k, void *v,
                             hipStream_t st);

// Work-groups of a launch stay below this: the grid in threads is a 32-bit number.
constexpr double kKv8MaxGroups = 8388608.0;

// How a call's query rows and keys are cut up; the same for the workspace query and the launch.
struct Kv8Plan {
    bool wide;         // row tiles with the keys staged in LDS, else 16-row tiles
    int joined;        // equal runs of steps, joined by a second launch; else one tile a work-group
    int rows;          // per tile
    int units;         // query blocks per sequence (1 without block lists)
    int tiles;         // row tiles per query block
    int items;         // tiles per head
    int64_t groups;    // work-groups of the launch
    int64_t ws_bytes;
    double whole;      // tiles in all; the launch is possible below kKv8MaxGroups
};

struct Kv8Attend {
    const void *q;
    void *out;
    float *lse;
    float *ws;
    const int32_t *blocks;
    int64_t q_stride, out_stride;
    int64_t q_block;  // >= max_rows without block lists
    int64_t max_kv;
    int q_heads, group, count, causal, f16;
    float scale;
};

Kv8Plan kv8_plan(const Kv8Cache &c, const Kv8Batch &b, int q_heads, int64_t max_kv, bool listed,
                 int64_t q_block, int count);
hipError_t launch_kv8_attend(const Kv8Cache &c, const Kv8Batch &b, const Kv8Attend &a,
                             const Kv8Plan &p, hipStream_t st);

struct Kv8Select {
    const void *q;
    int64_t q_stride;
    int32_t *blocks;
    double *ws;
    int64_t q_block, max_kv;
    int q_heads, group, count, causal, f16, first, last;
};
size_t kv8_select_workspace_bytes(const Kv8Cache &c, const Kv8Batch &b, int64_t max_kv,
                                  int64_t q_block);
hipError_t launch_kv8_select(const Kv8Cache &c, const Kv8Batch &b, const Kv8Select &a,
                             hipStream_t st);

// A status with its text for cfz_last_error (cfz_api.hip).
cfz_status report(cfz_status st, const char *text);

// Rows of one sequence as the kernels see them: clamped into the call's token rows.
__device__ inline void kv8_rows(const Kv8Batch &b, int seq, int &first, int &n)
{
    const int64_t t = b.tokens;
    int64_t lo = b.off[seq], hi = b.off[seq + 1];
    lo = lo < 0 ? 0 : (lo > t ? t : lo);
    hi = hi < lo ? lo : (hi > t ? t : hi);
    if (hi - lo > b.max_rows)
        hi = lo + b.max_rows;
    first = (int)lo;
    n = (int)(hi - lo);
}

__device__ inline int kv8_length(const Kv8Batch &b, int seq, int64_t most)
{
    const int64_t n = b.len[seq];
    return (int)(n < 0 ? 0 : (n > most ? most : n));
}

// The pool page of a sequence's logical page, -1 if it has none.
__device__ inline int kv8_page(const Kv8Cache &c, const Kv8Batch &b, int seq, int64_t logical)
{
    if (logical < 0 || logical >= b.width)
        return -1;
    const int p = b.table[(int64_t)seq * b.width + logical];
    return p >= 0 && p < c.pages ? p : -1;
}

}  // namespace cfz
