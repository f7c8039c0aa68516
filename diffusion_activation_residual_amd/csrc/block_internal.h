// block_internal.h -- declarations shared by the sources behind cfz_block.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "cfz_block.h"

namespace cfz {

// Work-groups of a launch stay below this: the grid in threads is a 32-bit number.
constexpr int64_t kBlockMaxGroups = 1 << 23;

// Which sequence (item) a token row belongs to.
struct BlockRows {
    const int32_t *off;  // null: equal runs of `run` rows
    int64_t tokens, run;
    int batch;
};

struct BlockVec {
    const void *p;  // null: none
    int64_t stride;
    int f32;
};

struct BlockNormOf {
    int kind;
    float eps;
    BlockVec w, b;
};

struct ResidualArgs {
    BlockRows rows;
    int cols;
    const void *x, *y;
    void *r, *h;
    int64_t xs, ys, rs, hs;
    float gate_scale;
    BlockVec gate, scale, shift;
    BlockNormOf after, before;
};
int64_t residual_groups(const ResidualArgs &a);
hipError_t launch_residual_norm(const ResidualArgs &a, int x_dtype, int y_dtype, hipStream_t st);

struct TableArgs {
    double speed[128];
    uint8_t axis[128];
    int pairs, axes;
    int64_t rows;
    const int32_t *positions;
    double amplitude;
    float *cos, *sin;
};
hipError_t launch_rotation_table(const TableArgs &a, hipStream_t st);

struct RotateRows {
    const void *x;
    void *out;
    const void *w;
    int64_t xs, os;
    int w_f32, heads;
    int first;  // waves per token of the tensors before it
};
struct RotateArgs {
    RotateRows t[4];
    int count, dim, log2lanes;
    BlockRows rows;
    const int32_t *starts;
    const float *cos, *sin;
    const int32_t *pos;
    int64_t table_rows;
    int rot, interleaved, normed;
    float eps;
    int parts;  // waves per token
};
constexpr int kRotateUnits = 4;  // units of 8 dimensions a thread
int64_t rotate_groups(const RotateArgs &a);
hipError_t launch_rotate(const RotateArgs &a, int dtype, hipStream_t st);

struct AdapterArgs {
    BlockRows rows;
    int64_t max_rows;
    const int32_t *ids;
    const void *a, *b;
    const float *scale;
    int adapters, slices, rank, cols_in, cols_out;
    int down;            // adapter rows of the first product: slices * rank
    int first_col[5];    // of each slice, and the end
    int first_tile[4];   // a slice's column tiles of the second product
    int col_tiles;
    const void *x, *y;
    void *out;
    int64_t xs, ys, os;
    uint16_t *hi, *lo;  // [tokens][down]: scale x A^T as the sum of two numbers of the type
    float *back;        // [tokens][slices]: what it was multiplied by, turned round (fp16)
    int parts, part_rows;  // work-groups a tile of the first product, adapter rows of each
    int tall;  // 16 tokens times this a tile of the first product
};
void adapter_plan(AdapterArgs &a);
int64_t adapter_tiles(const AdapterArgs &a, int rows);
int64_t adapter_groups(const AdapterArgs &a);
int64_t adapter_pieces(const AdapterArgs &a);  // of 16 bytes, of one adapter's A as it is laid out
hipError_t launch_adapters_put(const AdapterArgs &a, const void *rows, int first, int count,
                               hipStream_t st);
hipError_t launch_adapters(const AdapterArgs &a, bool f16, bool y_f32, hipStream_t st);

// ---- device helpers

template <class T> struct BlockType;
template <> struct BlockType<uint16_t> {  // bf16
    static __device__ inline float get(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
    static __device__ inline uint16_t put(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
};
template <> struct BlockType<_Float16> {
    static __device__ inline float get(_Float16 h) { return (float)h; }
    static __device__ inline _Float16 put(float f) { return (_Float16)f; }
};
template <> struct BlockType<float> {
    static __device__ inline float get(float f) { return f; }
    static __device__ inline float put(float f) { return f; }
};

// n values side by side, in vectors of at most 16 bytes.
template <class T, int N> __device__ inline void load_n(const T *p, float (&o)[N])
{
    constexpr int E = N * sizeof(T) > 16 ? 16 / (int)sizeof(T) : N;
    struct alignas(E * sizeof(T)) Piece { T v[E]; };
#pragma unroll
    for (int i = 0; i < N; i += E) {
        const Piece q = *(const Piece *)(p + i);
#pragma unroll
        for (int j = 0; j < E; ++j)
            o[i + j] = BlockType<T>::get(q.v[j]);
    }
}

template <class T, int N> __device__ inline void store_n(T *p, const float (&x)[N])
{
    constexpr int E = N * sizeof(T) > 16 ? 16 / (int)sizeof(T) : N;
    struct alignas(E * sizeof(T)) Piece { T v[E]; };
#pragma unroll
    for (int i = 0; i < N; i += E) {
        Piece q;
#pragma unroll
        for (int j = 0; j < E; ++j)
            q.v[j] = BlockType<T>::put(x[i + j]);
        *(Piece *)(p + i) = q;
    }
}

// Values of a vector of the call's 16-bit type or of fp32.
template <class T, int N> __device__ inline void load_vec(const BlockVec &v, int64_t at, float (&o)[N])
{
    if (v.f32)
        load_n((const float *)v.p + at, o);
    else
        load_n((const T *)v.p + at, o);
}

// The item of a row, by a whole wave together (every lane asks for the same row): the last one that
// starts at or before it, found 64 offsets at a time.  -1 if the row is in none.
__device__ inline int block_item(const BlockRows &rows, int64_t row, int64_t *first)
{
    if (!rows.off) {
        const int b = (int)((uint32_t)row / (uint32_t)rows.run);
        *first = (int64_t)b * rows.run;
        return b;
    }
    const int lane = threadIdx.x & 63;
    int lo = 0, n = rows.batch;  // the item is in lo .. lo + n - 1, if there is one
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int at = lo + lane * step;
        const bool before = lane * step < n && (int64_t)rows.off[at] <= row;
        const uint64_t votes = __ballot(before);
        // (lane 0 may see a start behind the row: the row is then before every item)
        const int k = votes ? 63 - __clzll(votes) : 0;
        n = n - k * step < step ? n - k * step : step;
        lo += k * step;
    }
    const int64_t a = rows.off[lo], e = rows.off[lo + 1];
    *first = a < 0 ? 0 : a;
    return row >= a && row < e ? lo : -1;
}

// x plus another lane's x, by DPP.
template <int CTRL> __device__ inline float plus_lane(float x)
{
    const int o = __builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true);
    return x + __uint_as_float((uint32_t)o);
}

// Sum over groups of `lanes` neighbouring lanes (4, 8, 16, 32 or 64), in every lane of the group:
// neighbours, pairs, then the mirrored half of 8 and of 16 lanes, then across the rows of 16.
__device__ inline float lanes_sum(float x, int lanes)
{
    x = plus_lane<0xb1>(x);  // quad_perm 1 0 3 2
    x = plus_lane<0x4e>(x);  // quad_perm 2 3 0 1
    if (lanes >= 8)
        x = plus_lane<0x141>(x);  // row_half_mirror
    if (lanes >= 16)
        x = plus_lane<0x140>(x);  // row_mirror
    if (lanes >= 32)
        x += __shfl_xor(x, 16);
    if (lanes >= 64)
        x += __shfl_xor(x, 32);
    return x;
}

// Whether a mean of squares plus eps says what it should in fp32: squares below 2^-149 vanish, and those from
// 2^128 on overflow.  Where it does not, the row is multiplied by norm_step and summed once more.
// (From 2^-96 up to infinity: the bits of numbers that are not negative are in their order, a NaN's behind.)
__device__ inline bool norm_in_range(float mean)
{
    constexpr uint32_t low = (127 - 96) << 23, high = 255u << 23;
    return __builtin_expect(__float_as_uint(mean) - low < high - low, 1);
}

// A power of two.  Means below 2^-96: a row's values, 2^-149 to 2^-41, come to 2^-45 to 2^63.  Infinite ones: the
// largest, 2^56 to 2^128, come to 2^-24 to 2^48, and 16,384 squares of them to 2^110 at most (what then falls
// below fp32's range is 2^-102 of the largest).
__device__ inline float norm_step(float mean) { return mean < 1.0f ? 0x1p104f : 0x1p-80f; }

}  // namespace cfz
