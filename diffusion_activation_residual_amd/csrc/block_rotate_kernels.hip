// block_rotate_kernels.hip -- tables of angles, and the norm and rotation of queries and keys.
#include "block_internal.h"

namespace cfz {
namespace {

constexpr int kThreads = 256;

// One angle a thread, in 64 bits: an angle past 2^16 in fp32 is only known to 2^-8 radians.  6540 rows of 32
// pairs in 3.1 us.
__global__ __launch_bounds__(kThreads) void rotation_table_kernel(TableArgs a)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t row = i / a.pairs;
    const int pair = (int)(i - row * a.pairs);
    if (row >= a.rows)
        return;
    const double place =
        a.positions ? (double)a.positions[row * a.axes + a.axis[pair]] : (double)row;
    double s, c;
    sincos(place * a.speed[pair], &s, &c);
    a.cos[i] = (float)(a.amplitude * c);
    a.sin[i] = (float)(a.amplitude * s);
}

constexpr int kStay = 0, kPairs = 1, kHalves = 2;  // how heads turn

// A wave takes kRotateUnits x 64 units of 8 dimensions of one token in one tensor; a head's units lie
// on neighbouring lanes, so that its norm is a short sum across lanes.  A unit holds whole pairs: 8
// neighbours, or 4 of each half.  All of a thread's units have the same place in their heads, so that its
// cosines and sines are loaded once.  Bound by the bytes: 2 x 4388 tokens, 30 + 30 heads of 64 with a
// norm, bf16, in 30 us (137 MB, 4.5 TB/s), 10,922 rows of 24 heads of 128 without one in 28.2 us
// (5.0 TB/s), with one in 29.0; 32 tokens, 32 + 8 heads of 128, in 5.6 us.  The tensor is the wave's, not
// the lane's: pointers looked up a lane took 46 us.
template <class T, int TURN>
__global__ __launch_bounds__(kThreads) void rotate_kernel(RotateArgs a)
{
    const int lane = threadIdx.x & 63;
    const uint32_t wave =
        __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
    const uint32_t row32 = wave / (uint32_t)a.parts;
    if (row32 >= a.rows.tokens)
        return;
    const int64_t row = row32;
    int part = (int)(wave - row32 * (uint32_t)a.parts), which = 0;
    while (which + 1 < a.count && part >= a.t[which + 1].first)
        ++which;
    const RotateRows t = a.t[which];
    const int lanes = 1 << a.log2lanes;
    const int unit = lane & (lanes - 1);
    const int head0 = ((part - t.first) * (kRotateUnits * 64) + lane) >> a.log2lanes;
    const float inv = 1.0f / (float)a.dim;  // (a power of two)
    const int half = a.rot / 2;
    const bool turn = TURN != kStay && unit * 8 < a.rot;
    const bool split = TURN == kHalves && turn;
    const int d0 = split ? 4 * unit : 8 * unit, d1 = split ? half + 4 * unit : 8 * unit + 4;

    // the values are under way while the row's sequence and position are looked up
    float v[kRotateUnits][8];
    const T *x = (const T *)t.x + row * t.xs;
#pragma unroll
    for (int i = 0; i < kRotateUnits; ++i) {
        const int head = head0 + i * (64 >> a.log2lanes);
        if (head >= t.heads) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = 0.0f;
            continue;
        }
        if (split) {
            load_n(x + head * a.dim + d0, *(float(*)[4]) & v[i][0]);
            load_n(x + head * a.dim + d1, *(float(*)[4]) & v[i][4]);
        } else {
            load_n(x + head * a.dim + d0, v[i]);
        }
    }
    int64_t first;
    const int seq = block_item(a.rows, row, &first);
    if (seq < 0)
        return;
    float w[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
    if (t.w) {
        const BlockVec wv{t.w, 0, t.w_f32};
        load_vec<T>(wv, d0, *(float(*)[4]) & w[0]);
        load_vec<T>(wv, d1, *(float(*)[4]) & w[4]);
    }
    float co[4], si[4];
    if (turn) {
        int64_t pos = a.pos ? (int64_t)a.pos[row] : (a.starts ? (int64_t)a.starts[seq] : 0) + (row - first);
        pos = pos < 0 ? 0 : (pos >= a.table_rows ? a.table_rows - 1 : pos);
        load_n(a.cos + pos * half + 4 * unit, co);
        load_n(a.sin + pos * half + 4 * unit, si);
    }
    if (a.normed) {
        // all units' sums side by side (heads past the last one hold zeros)
        float square[kRotateUnits];
        bool far = false;
#pragma unroll
        for (int i = 0; i < kRotateUnits; ++i) {
            float q = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                q = fmaf(v[i][j], v[i][j], q);
            square[i] = lanes_sum(q, lanes) * inv + a.eps;
            far |= !norm_in_range(square[i]);
        }
        if (far) {  // (the same for all lanes of a head)
#pragma unroll
            for (int i = 0; i < kRotateUnits; ++i) {
                if (norm_in_range(square[i]))
                    continue;
                const float step = norm_step(square[i]);
                float q = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[i][j] *= step;
                    q = fmaf(v[i][j], v[i][j], q);
                }
                square[i] = lanes_sum(q, lanes) * inv + a.eps * step * step;
            }
        }
#pragma unroll
        for (int i = 0; i < kRotateUnits; ++i) {
            const float f = rsqrtf(square[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] *= f * w[j];
        }
    }
#pragma unroll
    for (int i = 0; i < kRotateUnits; ++i) {
        const int head = head0 + i * (64 >> a.log2lanes);
        if (head >= t.heads)
            continue;
        if (turn) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int p0 = TURN == kHalves ? j : 2 * j, p1 = TURN == kHalves ? 4 + j : 2 * j + 1;
                const float y0 = v[i][p0], y1 = v[i][p1];
                v[i][p0] = fmaf(y0, co[j], -(y1 * si[j]));
                v[i][p1] = fmaf(y0, si[j], y1 * co[j]);
            }
        }
        T *o = (T *)t.out + row * t.os + head * a.dim;
        if (split) {
            store_n(o + d0, *(float(*)[4]) & v[i][0]);
            store_n(o + d1, *(float(*)[4]) & v[i][4]);
        } else {
            store_n(o + d0, v[i]);
        }
    }
}

template <class T> hipError_t rotate_as(const RotateArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)rotate_groups(a));
    (!a.cos          ? rotate_kernel<T, kStay>
     : a.interleaved ? rotate_kernel<T, kPairs>
                     : rotate_kernel<T, kHalves>)<<<grid, kThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotation_table(const TableArgs &a, hipStream_t st)
{
    const int64_t n = a.rows * a.pairs;
    rotation_table_kernel<<<dim3((unsigned)((n + kThreads - 1) / kThreads)), kThreads, 0, st>>>(a);
    return hipGetLastError();
}

int64_t rotate_groups(const RotateArgs &a)
{
    return (a.rows.tokens * a.parts + kThreads / 64 - 1) / (kThreads / 64);
}

hipError_t launch_rotate(const RotateArgs &a, int dtype, hipStream_t st)
{
    switch (dtype) {
    case CFZ_KV8_BF16: return rotate_as<uint16_t>(a, st);
    case CFZ_KV8_F16: return rotate_as<_Float16>(a, st);
    default: return rotate_as<float>(a, st);
    }
}

}  // namespace cfz
