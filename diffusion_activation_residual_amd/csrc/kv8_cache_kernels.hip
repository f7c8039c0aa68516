// kv8_cache_kernels.hip -- writing and reading the 8-bit paged K/V cache, and picking pages.
#include "kv8_internal.h"

#include <math.h>

#include <type_traits>

namespace cfz {
namespace {

constexpr int kThreads = 256;

__device__ inline float widen(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
__device__ inline float widen(_Float16 h) { return (float)h; }
__device__ inline float widen(float f) { return f; }

template <class T> struct alignas(4 * sizeof(T)) Four { T v[4]; };

template <class T> __device__ inline void load4(const T *p, float (&o)[4])
{
    const Four<T> f = *(const Four<T> *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = widen(f.v[i]);
}

// 8 values: two groups of 4, in one 16-byte load where they are 16 bytes side by side.
template <class T> __device__ inline void load8(const T *p0, const T *p1, bool split, float (&a)[4],
                                                float (&e)[4])
{
    if (sizeof(T) == 2 && !split) {
        struct alignas(16) Eight { T v[8]; };
        const Eight f = *(const Eight *)p0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = widen(f.v[i]);
            e[i] = widen(f.v[4 + i]);
        }
    } else {
        load4(p0, a);
        load4(p1, e);
    }
}

__device__ inline void narrow(float f, float &o) { o = f; }
__device__ inline void narrow(float f, _Float16 &o) { o = (_Float16)f; }
__device__ inline void narrow(float f, uint16_t &o)
{
    // nearest even; a cached value is never NaN
    const uint32_t u = __float_as_uint(f);
    o = (uint16_t)((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

__device__ inline double finite_or_zero(double x)
{
    return fabs(x) <= 1.7976931348623157e308 ? fabs(x) : 0.0;
}

// The 8-bit code nearest to x / s (ties to even), as its byte.  rinv = 1 / s in fp64; one
// correction by the exact remainder makes y the rounded quotient, so a tie is seen as a tie.
__device__ inline uint32_t encode(double x, double s, double rinv, int fmt)
{
    if (!(s > 0.0) || x != x)
        return 0;
    const double lim = (fmt == CFZ_KV8_INT8 ? 128.0 : 464.0) * s;
    x = x > lim ? lim : (x < -lim ? -lim : x);
    double y = x * rinv;
    y = fma(fma(-y, s, x), rinv, y);
    if (fmt == CFZ_KV8_INT8) {
        y = rint(y);
        y = y > 127.0 ? 127.0 : (y < -127.0 ? -127.0 : y);
        return (uint32_t)(int)y & 0xffu;
    }
    // (the correction of -0 is +0, but e4m3 keeps the sign of a zero)
    y = copysign(y > 448.0 ? 448.0 : (y < -448.0 ? -448.0 : y), x);
    // round to odd at 20 mantissa bits (the low word's bits are kept as one), which fp32 holds
    // exactly and which leaves every border between codes on its side
    const int hi = __double2hiint(y) | (__double2loint(y) != 0 ? 1 : 0);
    const float f = (float)__hiloint2double(hi, 0);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f, f, 0, false) & 0xffu;
}

__device__ inline float code_value(uint32_t byte, int fmt)
{
    if (fmt == CFZ_KV8_INT8)
        return (float)(int)(int8_t)(uint8_t)byte;
    return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
}

// Largest of a wave's values, which are not negative (their bits are then ordered as they are), in
// every lane: neighbours, rows of 16, then across the rows, all by DPP.
__device__ inline float wave_max(float x)
{
    uint32_t u = __float_as_uint(x);
#define CFZ_MAX_STEP(ctrl)                                                                          \
    {                                                                                              \
        const uint32_t o = __builtin_amdgcn_update_dpp(0, (int)u, ctrl, 0xf, 0xf, false);          \
        u = o > u ? o : u;                                                                         \
    }
    CFZ_MAX_STEP(0x111)  // row_shr:1
    CFZ_MAX_STEP(0x112)
    CFZ_MAX_STEP(0x114)
    CFZ_MAX_STEP(0x118)
    CFZ_MAX_STEP(0x142)  // row_bcast:15
    CFZ_MAX_STEP(0x143)  // row_bcast:31
#undef CFZ_MAX_STEP
    return __uint_as_float(__builtin_amdgcn_readlane(u, 63));
}

__device__ inline double wave_max(double x)
{
#define CFZ_MAX_STEP(ctrl)                                                                          \
    {                                                                                              \
        const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(x), ctrl, 0xf, 0xf, false);   \
        const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(x), ctrl, 0xf, 0xf, false);   \
        x = fmax(x, __hiloint2double(hi, lo));                                                     \
    }
    CFZ_MAX_STEP(0x111)
    CFZ_MAX_STEP(0x112)
    CFZ_MAX_STEP(0x114)
    CFZ_MAX_STEP(0x118)
    CFZ_MAX_STEP(0x142)
    CFZ_MAX_STEP(0x143)
#undef CFZ_MAX_STEP
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(x), 63),
                            __builtin_amdgcn_readlane(__double2loint(x), 63));
}

// Largest of a work-group's values (not negative).
template <class T> __device__ inline T block_max(T x, T *red)
{
    x = wave_max(x);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = x;
    __syncthreads();
    return fmax(fmax(red[0], red[1]), fmax(red[2], red[3]));
}

// encode() for four finite x whose magnitudes are at most a step of fp32 above the largest code
// times s, and s within 2^-100 .. 2^100: nothing to cut off, no remainder lost.
__device__ inline uint32_t encode4(const double (&x)[4], double s, double rinv, int fmt)
{
    double y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        y[j] = x[j] * rinv;
        y[j] = fma(fma(-y[j], s, x[j]), rinv, y[j]);
    }
    if (fmt == CFZ_KV8_INT8) {
        // adding 1.5 2^52 rounds to a whole number (ties to even) and leaves it in the low byte
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            b[j] = (uint32_t)__double2loint(y[j] + 6755399441055744.0);
        return __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u) |
               __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
    }
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        y[j] = copysign(y[j], x[j]);
        f[j] = (float)__hiloint2double(__double2hiint(y[j]) | (__double2loint(y[j]) != 0 ? 1 : 0), 0);
    }
    uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true);
}

// Adds the four codes' values to four sums.
__device__ inline void add_values(uint32_t w, int fmt, float *sum)
{
    if (fmt == CFZ_KV8_INT8) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sum[j] += (float)(int)(int8_t)(uint8_t)(w >> (8 * j));
    } else {
        sum[0] += __builtin_amdgcn_cvt_f32_fp8(w, 0);
        sum[1] += __builtin_amdgcn_cvt_f32_fp8(w, 1);
        sum[2] += __builtin_amdgcn_cvt_f32_fp8(w, 2);
        sum[3] += __builtin_amdgcn_cvt_f32_fp8(w, 3);
    }
}

// A page of one head that gets tokens.
struct Place {
    int page, lo, hi;  // its new slots, lo .. hi - 1
    int64_t first;     // its first token in the sequence
    int64_t src0;      // token row of slot 0
    int64_t ph;
};

template <int P>
__device__ inline bool find_place(const Kv8Cache &c, const Kv8Batch &b, int span, int64_t g,
                                  Place &p)
{
    // heads first: work-groups that run together then read whole token rows
    const int head = (int)(g % c.heads);
    g /= c.heads;
    const int at = (int)(g % span);
    const int seq = (int)(g / span);
    int row0, n;
    kv8_rows(b, seq, row0, n);
    const int64_t room = (int64_t)b.width * P;
    const int old = kv8_length(b, seq, room);
    const int64_t end = old + (int64_t)n < room ? old + (int64_t)n : room;
    p.first = ((int64_t)(old / P) + at) * P;
    if (p.first >= end || n == 0)
        return false;
    p.page = kv8_page(c, b, seq, p.first / P);
    p.lo = old > p.first ? (int)(old - p.first) : 0;
    p.hi = end - p.first < P ? (int)(end - p.first) : P;
    p.src0 = row0 + (p.first - old);
    p.ph = (int64_t)p.page * c.heads + head;
    return true;
}

// Appending: one work-group for the keys of a page of one head, another for its values.  Every new
// element is read once.  Older tokens are read only where the page keeps some (their codes enter the
// mean, and change if the scale grows).  Rotation and quotients are in fp64: a product by 1 / s alone
// loses ties (49 (1 / 49) < 1), with the remainder put right it is the rounded quotient.  What is not
// finite, and scales far from 1, take a slower way.  fp32 with a test for quotients near a border,
// and fp64 for those alone, was slower (130 against 97 us on 4 x 4388 tokens x 30 heads of 64, bf16):
// values of 8 bits lie near one time and again.  The rotated keys' fp64 values bound it: 256 threads
// hold a page of one head, which leaves 4 waves a SIMD (2 at pages of 128 tokens and head_dim 128).
// 4 x 4388 tokens from bf16 to int8, three sets of buffers in turn, rotated and not: 30 heads of 64,
// pages of 128, 85 and 55 us, 2.4 and 3.7 TB/s; 24 heads of 128 in pages of 64, 126 us rotated; in pages
// of 128, 187 and 101 us.  From fp32 (24 x 128, pages of 64) 142 and 110 us, 3.8 and 4.9 TB/s.
// Few tokens wait for dependent reads (offset, length, page, codes): 32 single tokens x 8 heads of 128 in
// 8 us.  A token that raises its page's scale has the page's older codes coded again, a byte at a time:
// then 14 (int8) and 16 us (e4m3) where every page's scale grows.
//
// Keys: units of 8 dimensions (two groups of 4 that hold whole rotation pairs).
constexpr int kStay = 0, kPairs = 1, kHalves = 2;  // how keys turn

template <class T, int D, int P, int TURN>
__device__ inline void append_keys(const Kv8Cache &c, const T *k, int64_t k_stride,
                                   const Kv8Rotation &rot, const Place &pl, int head)
{
    constexpr int U = D / 8;                // key units per token
    constexpr int NK = P * U / kThreads;    // key units per thread
    constexpr bool ROT = TURN != kStay;
    using Held = std::conditional_t<ROT, double, float>;  // what holds a key exactly
    __shared__ int sums[D];
    __shared__ Held red[4];
    const int tid = threadIdx.x, lo = pl.lo, hi = pl.hi;
    uint8_t *kp = c.k + pl.ph * (P * D);

    // (all units of a thread are of the same dimensions: U divides kThreads)
    const int half = ROT ? rot.dim / 2 : 0;
    const int u = tid % U;
    const bool turn = ROT && 8 * u < 2 * half, split = TURN == kHalves && turn;
    const int d0 = split ? 4 * u : 8 * u, d1 = split ? half + 4 * u : 8 * u + 4;
    const T *src = k + pl.src0 * k_stride + (int64_t)head * D;
    if (tid < D)
        sums[tid] = 0;
    const float prior = lo > 0 ? c.ks[pl.ph] : 0.0f;
    Held x[NK][8];
    Held big = 0;
    float bad = 0.0f;  // 0 * (NaN or infinity) shows here
    {
        float a[NK][8];
        float4 cs[ROT ? NK : 1], sn[ROT ? NK : 1];
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int slot = (tid + i * kThreads) / U;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                a[i][j] = 0.0f;
            if constexpr (ROT)
                cs[i] = sn[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (slot < lo || slot >= hi)
                continue;
            load8(src + slot * k_stride + d0, src + slot * k_stride + d1, split,
                  *(float(*)[4]) & a[i][0], *(float(*)[4]) & a[i][4]);
            if constexpr (ROT) {
                if (turn) {
                    int64_t pos = rot.pos ? (int64_t)rot.pos[pl.src0 + slot] : pl.first + slot;
                    pos = pos < 0 ? 0 : (pos >= rot.rows ? rot.rows - 1 : pos);
                    // angles 4u .. 4u + 3 in either order of the pairs
                    cs[i] = *(const float4 *)(rot.cos + pos * half + 4 * u);
                    sn[i] = *(const float4 *)(rot.sin + pos * half + 4 * u);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NK; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[i][j] = a[i][j];
                bad = fmaf(a[i][j], 0.0f, bad);
            }
            if constexpr (ROT) {
                if (turn) {
                    const float cc[4] = {cs[i].x, cs[i].y, cs[i].z, cs[i].w};
                    const float ss[4] = {sn[i].x, sn[i].y, sn[i].z, sn[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int p0 = TURN == kHalves ? j : 2 * j;
                        const int p1 = TURN == kHalves ? 4 + j : 2 * j + 1;
                        // products of two fp32 values are exact in fp64
                        const double y0 = a[i][p0], y1 = a[i][p1], co = cc[j], si = ss[j];
                        bad = fmaf(cc[j], 0.0f, fmaf(ss[j], 0.0f, bad));
                        x[i][p0] = fma(y0, co, -(y1 * si));
                        x[i][p1] = fma(y0, si, y1 * co);
                    }
                }
            }
        }
    }
    // a thread that holds something not finite looks through its values again
    const bool odd = !(bad == 0.0f);
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            big = fmax(big, (Held)fabs(x[i][j]));
    if (odd) {
        big = 0;
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                big = fmax(big, (Held)finite_or_zero(x[i][j]));
    }
    big = block_max(big, red);
    const double qmax = c.fmt == CFZ_KV8_INT8 ? 127.0 : 448.0;
    const float scale = fmaxf(prior, (float)((double)big / qmax));
    const bool grown = lo > 0 && scale > prior;
    const double rinv = 1.0 / (double)scale;
    const bool mid = scale > 0x1p-100f && scale < 0x1p100f && !odd;
    if (tid == 0)
        c.ks[pl.ph] = scale;

    float fast[8] = {};  // sums of codes (exact: at most 8 of up to 448 in steps of 2^-9)
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int slot = (tid + i * kThreads) / U;
        if (slot >= hi || (slot < lo && !grown && !c.km))
            continue;
        uint32_t w0, w1;
        if (slot >= lo) {
            if (mid) {
                const double x0[4] = {x[i][0], x[i][1], x[i][2], x[i][3]};
                const double x1[4] = {x[i][4], x[i][5], x[i][6], x[i][7]};
                w0 = encode4(x0, scale, rinv, c.fmt);
                w1 = encode4(x1, scale, rinv, c.fmt);
            } else {
                w0 = w1 = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    w0 |= encode(x[i][j], scale, rinv, c.fmt) << (8 * j);
                    w1 |= encode(x[i][4 + j], scale, rinv, c.fmt) << (8 * j);
                }
            }
        } else {
            w0 = *(const uint32_t *)(kp + slot * D + d0);
            w1 = *(const uint32_t *)(kp + slot * D + d1);
            if (grown) {
                uint32_t n0 = 0, n1 = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const double o0 = code_value((w0 >> (8 * j)) & 0xff, c.fmt);
                    const double o1 = code_value((w1 >> (8 * j)) & 0xff, c.fmt);
                    n0 |= encode(o0 * prior, scale, rinv, c.fmt) << (8 * j);
                    n1 |= encode(o1 * prior, scale, rinv, c.fmt) << (8 * j);
                }
                w0 = n0;
                w1 = n1;
            }
        }
        if (slot >= lo || grown) {
            if (split) {
                *(uint32_t *)(kp + slot * D + d0) = w0;
                *(uint32_t *)(kp + slot * D + d1) = w1;
            } else {
                *(uint2 *)(kp + slot * D + d0) = make_uint2(w0, w1);
            }
        }
        add_values(w0, c.fmt, fast);
        add_values(w1, c.fmt, fast + 4);
    }
    if (!c.km)
        return;
    // 512 times a sum of codes is a whole number: exact in any order
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        atomicAdd(&sums[d0 + j], (int)(fast[j] * 512.0f));
        atomicAdd(&sums[d1 + j], (int)(fast[4 + j] * 512.0f));
    }
    __syncthreads();
    if (tid < D)
        c.km[pl.ph * D + tid] = (float)((double)sums[tid] / 512.0 * (double)scale / (double)hi);
}

// Values: units of 4 tokens x 8 dimensions (4 in the smallest page), transposed in registers and
// merged into the page's [dim][token] bytes in LDS, so that the page is written in whole 16-byte
// vectors.
template <class T, int D, int P>
__device__ inline void append_values(const Kv8Cache &c, const T *v, int64_t v_stride,
                                     const Place &pl, int head)
{
    constexpr int W = P * D >= 32 * kThreads ? 8 : 4;  // dimensions of a unit
    constexpr int NV = P * D / (4 * W) / kThreads ? P * D / (4 * W) / kThreads : 1;
    constexpr int ROW = P / 4 + 1;          // LDS words per dimension (padded)
    __shared__ uint32_t vpage[D * ROW];
    __shared__ float red[4];
    const int tid = threadIdx.x, lo = pl.lo, hi = pl.hi;
    uint8_t *vp = c.v + pl.ph * (P * D);
    const T *src = v + pl.src0 * v_stride + (int64_t)head * D;
    float w[NV][4][W];  // [unit][token][dimension]
    float big = 0.0f, bad = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int unit = tid + i * kThreads, tq = unit / (D / W), dq = unit % (D / W);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int slot = tq * 4 + t;
            float a[4] = {}, e[4] = {};
            if (slot >= lo && slot < hi) {
                const T *p = src + slot * v_stride + dq * W;
                if (W == 8)
                    load8(p, p + 4, false, a, e);
                else
                    load4(p, a);
            }
#pragma unroll
            for (int j = 0; j < W; ++j)
                w[i][t][j] = j < 4 ? a[j & 3] : e[j & 3];
        }
    }
    // the page as it is, where bytes of it stay
    if (lo > 0 || hi < P) {
        for (int i = tid; i < D * P / 16; i += kThreads) {
            const uint4 q = ((const uint4 *)vp)[i];
            uint32_t *o = vpage + (i * 4 / (P / 4)) * ROW + i * 4 % (P / 4);
            o[0] = q.x, o[1] = q.y, o[2] = q.z, o[3] = q.w;
        }
    }
    const float prior = lo > 0 ? c.vs[pl.ph] : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < W; j += 2) {
                big = fmaxf(fmaxf(fabsf(w[i][t][j]), fabsf(w[i][t][j + 1])), big);
                bad = fmaf(w[i][t][j], 0.0f, fmaf(w[i][t][j + 1], 0.0f, bad));
            }
    // a thread that holds something not finite looks through its values again
    const bool odd = !(bad == 0.0f);
    if (odd) {
        big = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < W; ++j)
                    big = fmaxf(big,
                                   fabsf(w[i][t][j]) <= 3.4028234e38f ? fabsf(w[i][t][j]) : 0.0f);
    }
    big = block_max(big, red);
    const double qmax = c.fmt == CFZ_KV8_INT8 ? 127.0 : 448.0;
    const float scale = fmaxf(prior, (float)((double)big / qmax));
    const bool grown = lo > 0 && scale > prior;
    const double rinv = 1.0 / (double)scale;
    const bool mid = scale > 0x1p-100f && scale < 0x1p100f && !odd;
    if (tid == 0)
        c.vs[pl.ph] = scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int unit = tid + i * kThreads, tq = unit / (D / W), dq = unit % (D / W);
        if (tq >= P / 4 || (tq * 4 >= hi) || (tq * 4 + 4 <= lo && !grown))
            continue;
        uint32_t *o = vpage + dq * W * ROW + tq;
        if (mid && (tq * 4 >= lo || !grown)) {
            // the bytes of the unit's new tokens
            const int skip = lo - tq * 4, end = hi - tq * 4;
            const uint32_t fresh = (end >= 4 ? ~0u : (1u << (8 * end)) - 1u) &
                                   (skip <= 0 ? ~0u : ~0u << (8 * skip));
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const double x[4] = {w[i][0][j], w[i][1][j], w[i][2][j], w[i][3][j]};
                const uint32_t code = encode4(x, scale, rinv, c.fmt);
                o[j * ROW] = fresh == ~0u ? code : (o[j * ROW] & ~fresh) | (code & fresh);
            }
            continue;
        }
#pragma unroll 1
        for (int t = 0; t < 4; ++t) {
            const int slot = tq * 4 + t;
            if (slot >= hi || (slot < lo && !grown))
                continue;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const uint32_t was = o[j * ROW];
                double y = t == 0 ? w[i][0][j] : t == 1 ? w[i][1][j] : t == 2 ? w[i][2][j] : w[i][3][j];
                if (slot < lo)
                    y = (double)code_value(was >> (8 * t) & 0xff, c.fmt) * prior;
                o[j * ROW] = (was & ~(0xffu << (8 * t))) | encode(y, scale, rinv, c.fmt) << (8 * t);
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < D * P / 16; i += kThreads) {
        const uint32_t *o = vpage + (i * 4 / (P / 4)) * ROW + i * 4 % (P / 4);
        ((uint4 *)vp)[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <class T, int D, int P, int TURN>
__global__ __launch_bounds__(kThreads) void kv8_append_kernel(Kv8Cache c, Kv8Batch b, const T *k,
                                                              const T *v, int64_t k_stride,
                                                              int64_t v_stride, Kv8Rotation rot,
                                                              int span)
{
    Place pl;
    const int64_t g = blockIdx.x / 2;
    if (!find_place<P>(c, b, span, g, pl) || pl.page < 0)
        return;
    const int head = (int)(g % c.heads);
    if (blockIdx.x & 1)
        append_values<T, D, P>(c, v, v_stride, pl, head);
    else
        append_keys<T, D, P, TURN>(c, k, k_stride, rot, pl, head);
}

// Reads one page of one head back: keys straight, values through LDS (their codes are dimension-major),
// rows written in vectors of 4 values.  Bound by the bytes written: 4 x 4388 tokens x 30 heads of 64
// to fp32 in 64 us, 5.3 TB/s.
template <class T, int D, int P>
__global__ __launch_bounds__(kThreads) void kv8_gather_kernel(Kv8Cache c, Kv8Batch b, T *k, T *v,
                                                              int span)
{
    constexpr int ROW = P / 4 + 1;
    __shared__ uint32_t vpage[D * ROW];
    const int tid = threadIdx.x;
    int64_t g = blockIdx.x;
    const int head = (int)(g % c.heads);
    g /= c.heads;
    const int at = (int)(g % span);
    const int seq = (int)(g / span);
    int row0, n;
    kv8_rows(b, seq, row0, n);
    const int64_t room = (int64_t)b.width * P;
    const int64_t old = b.len[seq] < 0 ? 0 : b.len[seq];
    const int64_t first = (old / P + at) * P;
    if (first >= old + n || n == 0)
        return;
    const int lo = old > first ? (int)(old - first) : 0;
    const int hi = old + n - first < P ? (int)(old + n - first) : P;
    const int page = first < room ? kv8_page(c, b, seq, first / P) : -1;
    const int64_t ph = (int64_t)page * c.heads + head;
    const int64_t dst0 = row0 + (first - old);
    if (v && page >= 0) {
        const uint4 *vp = (const uint4 *)(c.v + ph * (P * D));
        for (int i = tid; i < D * P / 16; i += kThreads) {
            const uint4 q = vp[i];
            uint32_t *o = vpage + (i * 4 / (P / 4)) * ROW + i * 4 % (P / 4);
            o[0] = q.x, o[1] = q.y, o[2] = q.z, o[3] = q.w;
        }
    }
    const float ks = page >= 0 ? c.ks[ph] : 0.0f, vs = page >= 0 ? c.vs[ph] : 0.0f;
    if (k) {
        for (int i = tid; i < P * D / 4; i += kThreads) {
            const int slot = i / (D / 4), d = i % (D / 4) * 4;
            if (slot < lo || slot >= hi)
                continue;
            const uint32_t w = page >= 0 ? *(const uint32_t *)(c.k + ph * (P * D) + slot * D + d) : 0;
            Four<T> o;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                narrow(page >= 0 ? code_value((w >> (8 * j)) & 0xff, c.fmt) * ks : 0.0f, o.v[j]);
            *(Four<T> *)(k + ((dst0 + slot) * c.heads + head) * D + d) = o;
        }
    }
    if (!v)
        return;
    __syncthreads();
    for (int i = tid; i < P * D / 16; i += kThreads) {
        const int tq = i / (D / 4), d = i % (D / 4) * 4;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = page >= 0 ? vpage[(d + j) * ROW + tq] : 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int slot = tq * 4 + t;
            if (slot < lo || slot >= hi)
                continue;
            Four<T> o;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                narrow(page >= 0 ? code_value((w[j] >> (8 * t)) & 0xff, c.fmt) * vs : 0.0f, o.v[j]);
            *(Four<T> *)(v + ((dst0 + slot) * c.heads + head) * D + d) = o;
        }
    }
}

// ---- picking pages

// The order of scores as unsigned numbers; NaN below everything (a page that cannot be picked is 0).
__device__ inline uint64_t order_key(double s)
{
    if (s != s)
        return 1;
    s += 0.0;  // -0 counts as 0
    const uint64_t u = (uint64_t)__double_as_longlong(s);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// Scores of one query block and KV head against the means of up to kScorePages pages.  The block's
// queries are summed in fp64 and the products are too: 64 bits where two pages' scores may differ in
// the last bit of fp32.  A query row is read by D / 8 lanes (16 bytes each) and a page's mean by 8
// lanes, so that loads are wide and the sums across lanes short.  Bound by latency (a few dozen KB
// per work-group): 35 blocks of 128 queries x 138 pages x 30 heads of 64 in 19.7 us.
constexpr int kScorePages = 64;

template <int D>
__global__ __launch_bounds__(kThreads) void kv8_score_kernel(Kv8Cache c, Kv8Batch b, Kv8Select a,
                                                             int units, int stride, int chunks)
{
    constexpr int LANES = D / 8, ROWS = kThreads / LANES;  // lanes per row, rows at once
    constexpr int E = D / 8;                               // a lane's dimensions of a mean
    __shared__ double part[ROWS][D + 2];
    __shared__ double qs[D];
    const int tid = threadIdx.x;
    int64_t g = blockIdx.x;
    const int chunk = (int)(g % chunks);
    g /= chunks;
    const int64_t list = g;  // (seq, unit, head)
    const int head = (int)(g % c.heads);
    g /= c.heads;
    const int unit = (int)(g % units);
    const int seq = (int)(g / units);
    int row0, n;
    kv8_rows(b, seq, row0, n);
    const int len = kv8_length(b, seq, a.max_kv);
    const int64_t q0 = (int64_t)unit * a.q_block;
    if (q0 >= n)
        return;
    const int64_t q1 = q0 + a.q_block < n ? q0 + a.q_block : n;
    const int64_t end = a.causal ? (int64_t)len - n + q1 : len;
    const int seen = end <= 0 ? 0 : (int)((end + c.page - 1) >> c.log2page);
    if (chunk * kScorePages >= seen)
        return;

    // the means first: they do not wait for the queries
    constexpr int TURNS = kScorePages * 8 / kThreads;
    float4 mean[TURNS][E / 4];
    int page[TURNS];
    const int sub = tid % 8;
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int p = chunk * kScorePages + i * (kThreads / 8) + tid / 8;
        page[i] = p < seen ? kv8_page(c, b, seq, p) : -1;
#pragma unroll
        for (int j = 0; j < E / 4; ++j)
            mean[i][j] = page[i] >= 0
                             ? *(const float4 *)(c.km + ((int64_t)page[i] * c.heads + head) * D +
                                                 j * 32 + sub * 4)
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }

    double sum[8] = {};
    const int rows = (int)(q1 - q0) * a.group, d0 = tid % LANES * 8;
#pragma unroll 4
    for (int r = tid / LANES; r < rows; r += ROWS) {
        const int query = a.group == 1 ? r : r / a.group;
        const int64_t at = (row0 + q0 + query) * a.q_stride +
                           ((int64_t)(head - query) * a.group + r) * D + d0;
        const uint4 w = *(const uint4 *)((const uint16_t *)a.q + at);
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint16_t lo = (uint16_t)words[j], hi = (uint16_t)(words[j] >> 16);
            sum[2 * j] += a.f16 ? (float)__builtin_bit_cast(_Float16, lo) : widen(lo);
            sum[2 * j + 1] += a.f16 ? (float)__builtin_bit_cast(_Float16, hi) : widen(hi);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        part[tid / LANES][d0 + j] = sum[j];
    __syncthreads();
    if (tid < D) {
        double s = 0.0;
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            s += part[r][tid];
        qs[tid] = s;
    }
    __syncthreads();
    double *out = a.ws + list * stride;
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int p = chunk * kScorePages + i * (kThreads / 8) + tid / 8;
        double s = 0.0;
#pragma unroll
        for (int j = 0; j < E / 4; ++j) {
            const double *q = qs + j * 32 + sub * 4;
            s = fma(q[0], (double)mean[i][j].x, s);
            s = fma(q[1], (double)mean[i][j].y, s);
            s = fma(q[2], (double)mean[i][j].z, s);
            s = fma(q[3], (double)mean[i][j].w, s);
        }
#pragma unroll
        for (int d = 4; d >= 1; d >>= 1)
            s += __shfl_xor(s, d);
        uint64_t key = order_key(s);
        if (page[i] < 0)
            key = 0;
        else if (p < a.first || p >= seen - a.last)
            key = ~0ull;
        if (sub == 0 && p < seen)
            out[p] = __longlong_as_double((long long)key);
    }
}

// The `count` largest keys of one list: the threshold is found 8 bits at a time by counting
// (the same work whatever the keys), then the pages above it and, in index order, as many at it as
// are left are written in ascending order.  Launch, dependent reads and the passes' barriers: 10.8 us
// for 1050 lists of 138 pages, 9.9 us for 128 of up to 512; copies of the keys in LDS, and one wave a
// list counting by ballots, took 10.3 and 9.0 to 13.9.
__global__ __launch_bounds__(kThreads) void kv8_pick_kernel(Kv8Cache c, Kv8Batch b, Kv8Select a,
                                                            int units, int stride)
{
    __shared__ int hist[256];
    __shared__ int scan[4][2];
    __shared__ int pick[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int64_t g = blockIdx.x;
    const int64_t list = g;
    g /= c.heads;
    const int unit = (int)(g % units);
    const int seq = (int)(g / units);
    int row0, n;
    kv8_rows(b, seq, row0, n);
    const int len = kv8_length(b, seq, a.max_kv);
    int32_t *out = a.blocks + list * a.count;
    const int64_t q0 = (int64_t)unit * a.q_block;
    int seen = 0;
    if (q0 < n) {
        const int64_t q1 = q0 + a.q_block < n ? q0 + a.q_block : n;
        const int64_t end = a.causal ? (int64_t)len - n + q1 : len;
        seen = end <= 0 ? 0 : (int)((end + c.page - 1) >> c.log2page);
    }
    const uint64_t *keys = (const uint64_t *)(a.ws + list * stride);

    uint64_t prefix = 0;
    int need = a.count;  // how many of the keys that match the prefix so far are wanted
    if (seen > a.count) {
        for (int shift = 56; shift >= 0; shift -= 8) {
            hist[tid] = 0;
            __syncthreads();
            const uint64_t mask = shift == 56 ? 0 : ~0ull << (shift + 8);
            for (int i = tid; i < seen; i += kThreads) {
                const uint64_t key = keys[i];
                if ((key & mask) == prefix)
                    atomicAdd(&hist[(key >> shift) & 255], 1);
            }
            __syncthreads();
            // how many keys lie in the digits above this thread's
            const int digit = 255 - tid, mine = hist[digit];
            int incl = mine;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(incl, d);
                incl += lane >= d ? o : 0;
            }
            if (lane == 63)
                scan[wave][0] = incl;
            __syncthreads();
            for (int w = 0; w < wave; ++w)
                incl += scan[w][0];
            if (incl >= need && incl - mine < need) {
                pick[0] = digit;
                pick[1] = need - (incl - mine);
            }
            __syncthreads();
            prefix |= (uint64_t)pick[0] << shift;
            need = pick[1];
            __syncthreads();
        }
    }
    // threshold = prefix; pages without a key (0) are never picked
    int done = 0, ties = 0;  // written so far, ties met so far
    for (int base = 0; base < seen; base += kThreads) {
        const int i = base + tid;
        const uint64_t key = i < seen ? keys[i] : 0;
        const bool tie = key != 0 && seen > a.count && key == prefix;
        const bool over = key != 0 && (seen <= a.count || key > prefix);
        // ranks among the ties first, since only the first `need` of them are taken
        const uint64_t tb = __ballot(tie);
        if (lane == 0)
            scan[wave][0] = __popcll(tb);
        __syncthreads();
        int before = ties, all = 0;
        for (int w = 0; w < 4; ++w) {
            before += w < wave ? scan[w][0] : 0;
            all += scan[w][0];
        }
        const bool take = over || (tie && before + __popcll(tb & ((1ull << lane) - 1)) < need);
        ties += all;
        const uint64_t kb = __ballot(take);
        if (lane == 0)
            scan[wave][1] = __popcll(kb);
        __syncthreads();
        int at = done;
        all = 0;
        for (int w = 0; w < 4; ++w) {
            at += w < wave ? scan[w][1] : 0;
            all += scan[w][1];
        }
        if (take)
            out[at + __popcll(kb & ((1ull << lane) - 1))] = i;
        done += all;
        __syncthreads();
    }
    for (int i = done + tid; i < a.count; i += kThreads)
        out[i] = -1;
}

// Work-groups of a page-wise launch over `span` pages per sequence.
int64_t page_groups(const Kv8Cache &c, const Kv8Batch &b, int &span)
{
    // a run of max_rows tokens touches one page more than it fills when it starts inside a page
    const int64_t pages = (b.max_rows + c.page - 1) / c.page + 1;
    span = (int)pages;
    return pages * c.heads * b.batch;
}

template <class T>
hipError_t append_as(const Kv8Cache &c, const Kv8Batch &b, const void *k, const void *v,
                     int64_t ks, int64_t vs, const Kv8Rotation &rot, hipStream_t st)
{
    int span;
    const dim3 grid((unsigned)(2 * page_groups(c, b, span)));
#define CFZ_KV8_CASE(D, P)                                                                         \
    if (c.dim == D && c.page == P)                                                                 \
        (!rot.cos          ? kv8_append_kernel<T, D, P, kStay>                                      \
         : rot.interleaved ? kv8_append_kernel<T, D, P, kPairs>                                     \
                           : kv8_append_kernel<T, D, P, kHalves>)                                   \
            <<<grid, kThreads, 0, st>>>(c, b, (const T *)k, (const T *)v, ks, vs, rot, span);
    CFZ_KV8_CASE(64, 32)
    CFZ_KV8_CASE(64, 64)
    CFZ_KV8_CASE(64, 128)
    CFZ_KV8_CASE(128, 32)
    CFZ_KV8_CASE(128, 64)
    CFZ_KV8_CASE(128, 128)
#undef CFZ_KV8_CASE
    return hipGetLastError();
}

template <class T>
hipError_t gather_as(const Kv8Cache &c, const Kv8Batch &b, void *k, void *v, hipStream_t st)
{
    int span;
    const dim3 grid((unsigned)page_groups(c, b, span));
#define CFZ_KV8_CASE(D, P)                                                                         \
    if (c.dim == D && c.page == P)                                                                 \
        kv8_gather_kernel<T, D, P><<<grid, kThreads, 0, st>>>(c, b, (T *)k, (T *)v, span);
    CFZ_KV8_CASE(64, 32)
    CFZ_KV8_CASE(64, 64)
    CFZ_KV8_CASE(64, 128)
    CFZ_KV8_CASE(128, 32)
    CFZ_KV8_CASE(128, 64)
    CFZ_KV8_CASE(128, 128)
#undef CFZ_KV8_CASE
    return hipGetLastError();
}

int64_t select_pages(const Kv8Cache &c, int64_t max_kv) { return (max_kv + c.page - 1) / c.page; }

}  // namespace

hipError_t launch_kv8_append(const Kv8Cache &c, const Kv8Batch &b, int dtype, const void *k,
                             const void *v, int64_t k_stride, int64_t v_stride,
                             const Kv8Rotation &rot, hipStream_t st)
{
    switch (dtype) {
    case CFZ_KV8_BF16: return append_as<uint16_t>(c, b, k, v, k_stride, v_stride, rot, st);
    case CFZ_KV8_F16: return append_as<_Float16>(c, b, k, v, k_stride, v_stride, rot, st);
    default: return append_as<float>(c, b, k, v, k_stride, v_stride, rot, st);
    }
}

hipError_t launch_kv8_gather(const Kv8Cache &c, const Kv8Batch &b, int dtype, void *k, void *v,
                             hipStream_t st)
{
    switch (dtype) {
    case CFZ_KV8_BF16: return gather_as<uint16_t>(c, b, k, v, st);
    case CFZ_KV8_F16: return gather_as<_Float16>(c, b, k, v, st);
    default: return gather_as<float>(c, b, k, v, st);
    }
}

size_t kv8_select_workspace_bytes(const Kv8Cache &c, const Kv8Batch &b, int64_t max_kv,
                                  int64_t q_block)
{
    const int64_t units = (b.max_rows + q_block - 1) / q_block;
    return (size_t)(units * c.heads * b.batch * select_pages(c, max_kv)) * sizeof(double);
}

hipError_t launch_kv8_select(const Kv8Cache &c, const Kv8Batch &b, const Kv8Select &a,
                             hipStream_t st)
{
    const int units = (int)((b.max_rows + a.q_block - 1) / a.q_block);
    const int stride = (int)select_pages(c, a.max_kv);
    const int chunks = (stride + kScorePages - 1) / kScorePages;
    const int64_t lists = (int64_t)units * c.heads * b.batch;
    if (chunks > 0) {
        const dim3 grid((unsigned)(lists * chunks));
        if (c.dim == 64)
            kv8_score_kernel<64><<<grid, kThreads, 0, st>>>(c, b, a, units, stride, chunks);
        else
            kv8_score_kernel<128><<<grid, kThreads, 0, st>>>(c, b, a, units, stride, chunks);
    }
    kv8_pick_kernel<<<dim3((unsigned)lists), kThreads, 0, st>>>(c, b, a, units, stride);
    return hipGetLastError();
}

}  // namespace cfz
