// kv8_cache_kernels.hip -- writing and reading the 8-bit paged K/V cache, and picking pages.
#include "kv8_internal.h"

#include <math.h>

namespace cfz {
namespace {

constexpr int kThreads = 256;

template <int DT> struct Src;
template <> struct Src<CFZ_KV8_BF16> { using T = uint16_t; };
template <> struct Src<CFZ_KV8_F16> { using T = _Float16; };
template <> struct Src<CFZ_KV8_F32> { using T = float; };

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

// The code times 512: a whole number in both formats (e4m3 steps are 2^-9 and up), so that sums of
// codes are exact in any order.  A byte that is no code (unwritten memory) counts as 0.
__device__ inline int code_512(uint32_t byte, int fmt)
{
    const float f = code_value(byte, fmt) * 512.0f;
    return f == f ? (int)f : 0;
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

// Largest of a work-group's values, N of them at once.
template <int N> __device__ inline void block_max(float (&x)[N], float *red)
{
#pragma unroll
    for (int n = 0; n < N; ++n) {
        x[n] = wave_max(x[n]);
        if ((threadIdx.x & 63) == 0)
            red[(threadIdx.x >> 6) * N + n] = x[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n)
        x[n] = fmaxf(fmaxf(red[n], red[N + n]), fmaxf(red[2 * N + n], red[3 * N + n]));
}

// Four codes from approximate quotients y, each within e of the true one: false if one of them lies so
// near a border between codes that the true code may be another.
__device__ inline bool quick_codes(const float (&y)[4], float e, int fmt, uint32_t &word,
                                   float (&value)[4])
{
    if (fmt == CFZ_KV8_INT8) {
        // adding 1.5 2^23 rounds to a whole number (ties to even) and leaves it in the low byte
        uint32_t b[4];
        float far = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float t = y[j] + 12582912.0f;
            b[j] = __float_as_uint(t);
            value[j] = t - 12582912.0f;
            far = fmaxf(far, fabsf(y[j] - value[j]));
        }
        const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
        word = lo | hi;
        return far < 0.5f - e;
    }
    uint32_t below = 0, above = 0;
    below = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] - e, y[1] - e, below, false);
    below = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] - e, y[3] - e, below, true);
    above = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] + e, y[1] + e, above, false);
    above = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] + e, y[3] + e, above, true);
    word = above;
    value[0] = __builtin_amdgcn_cvt_f32_fp8(word, 0);
    value[1] = __builtin_amdgcn_cvt_f32_fp8(word, 1);
    value[2] = __builtin_amdgcn_cvt_f32_fp8(word, 2);
    value[3] = __builtin_amdgcn_cvt_f32_fp8(word, 3);
    // (a value that rounds to zero from both sides of it is ambiguous too: the zero has a sign)
    return below == above;
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
    const int at = (int)(g % span);
    g /= span;
    const int head = (int)(g % c.heads);
    const int seq = (int)(g / c.heads);
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
// mean, and change if the scale grows).
//
// The codes are those of 64-bit quotients, but fp64 is spent only where fp32 cannot decide: fp32
// quotients come with a bound of their error, and the few units with a quotient that near a
// border between codes, or with a value that is not finite, are done again in fp64.  Likewise
// the largest rotated key: only units whose fp32 maximum comes near the work-group's are looked at
// again.  Bound by the latency of a page's chain of reads and reductions, hence small work-groups
// with few registers, many on a CU.
//
// Keys: units of 8 dimensions (two groups of 4 that hold whole rotation pairs).
template <class T, int D, int P>
__device__ inline void append_keys(const Kv8Cache &c, const T *k, int64_t k_stride,
                                   const Kv8Rotation &rot, const Place &pl, int head)
{
    constexpr int U = D / 8;                // key units per token
    constexpr int NK = P * U / kThreads;    // key units per thread
    __shared__ int sums[D];
    __shared__ float red[8];
    __shared__ unsigned long long top64;
    const int tid = threadIdx.x, lo = pl.lo, hi = pl.hi;
    uint8_t *kp = c.k + pl.ph * (P * D);

    // (all units of a thread are of the same dimensions: U divides kThreads)
    const int half = rot.cos ? rot.dim / 2 : 0;
    const int u = tid % U;
    const bool turn = 8 * u < 2 * half, split = turn && !rot.interleaved;
    const int d0 = split ? 4 * u : 8 * u, d1 = split ? half + 4 * u : 8 * u + 4;
    auto angles = [&](int slot, float4 &cs, float4 &sn) {
        int64_t pos = rot.pos ? (int64_t)rot.pos[pl.src0 + slot] : pl.first + slot;
        pos = pos < 0 ? 0 : (pos >= rot.rows ? rot.rows - 1 : pos);
        // angles 4u .. 4u + 3 in either order of the pairs
        cs = *(const float4 *)(rot.cos + pos * half + 4 * u);
        sn = *(const float4 *)(rot.sin + pos * half + 4 * u);
    };
    const T *src = k + pl.src0 * k_stride + (int64_t)head * D;
    float x[NK][8];
    // largest key, largest product within a rotation; 0 * (NaN or infinity) shows in bad
    float big[2] = {0.0f, 0.0f}, bad = 0.0f;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int slot = (tid + i * kThreads) / U;
        float a[4] = {}, e[4] = {};
        if (slot >= lo && slot < hi) {
            load4(src + slot * k_stride + d0, a);
            load4(src + slot * k_stride + d1, e);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[i][j] = a[j];
            x[i][4 + j] = e[j];
        }
    }
    if (turn) {
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int slot = (tid + i * kThreads) / U;
            if (slot < lo || slot >= hi)
                continue;
            float4 cs, sn;
            angles(slot, cs, sn);
            const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
            float r[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float y0 = split ? x[i][j] : x[i][2 * j];
                const float y1 = split ? x[i][4 + j] : x[i][2 * j + 1];
                const float t0 = y1 * ss[j], t1 = y1 * cc[j];
                const float r0 = fmaf(y0, cc[j], -t0), r1 = fmaf(y0, ss[j], t1);
                big[1] = fmaxf(fmaxf(fabsf(t0), fabsf(t1)), big[1]);
                r[2 * j] = r0;
                r[2 * j + 1] = r1;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = split ? r[2 * j] : r[j];
                x[i][4 + j] = split ? r[2 * j + 1] : r[4 + j];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            big[0] = fmaxf(fmaxf(fabsf(x[i][j]), fabsf(x[i][j + 1])), big[0]);
            bad = fmaf(x[i][j], 0.0f, fmaf(x[i][j + 1], 0.0f, bad));
        }
    // one unit in fp64; products of two fp32 values are exact there
    auto exact_unit = [&](int slot, double (&y)[8]) {
        float a[4], e[4];
        load4(src + slot * k_stride + d0, a);
        load4(src + slot * k_stride + d1, e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[j] = a[j];
            y[4 + j] = e[j];
        }
        if (turn) {
            float4 cs, sn;
            angles(slot, cs, sn);
            const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
            double r[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const double y0 = split ? y[j] : y[2 * j], y1 = split ? y[4 + j] : y[2 * j + 1];
                const double co = cc[j], si = ss[j];
                r[2 * j] = fma(y0, co, -(y1 * si));
                r[2 * j + 1] = fma(y0, si, y1 * co);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[j] = split ? r[2 * j] : r[j];
                y[4 + j] = split ? r[2 * j + 1] : r[4 + j];
            }
        }
    };

    const bool odd = !(bad == 0.0f);
    if (odd)
        big[0] = big[1] = 0.0f;
    if (tid == 0)
        top64 = 0;
    if (tid < D)
        sums[tid] = 0;
    block_max(big, red);
    {
        // a rotated value is rounded by half a step of it and of its second product
        const float near = big[0] - 0x1p-22f * (big[0] + big[1]);
        uint32_t look = 0;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                m = fmaxf(m, fabsf(x[i][j]));
            const int slot = (tid + i * kThreads) / U;
            if ((odd || m >= near) && slot >= lo && slot < hi)
                look |= 1u << i;
        }
        while (look) {
            const int slot = (tid + __builtin_ctz(look) * kThreads) / U;
            look &= look - 1;
            double y[8], m = 0.0;
            exact_unit(slot, y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                m = fmax(m, finite_or_zero(y[j]));
            atomicMax(&top64, (unsigned long long)__double_as_longlong(m));
        }
    }
    const float prior = lo > 0 ? c.ks[pl.ph] : 0.0f;
    __syncthreads();
    const double qmax = c.fmt == CFZ_KV8_INT8 ? 127.0 : 448.0;
    const float scale = fmaxf(prior, (float)(__longlong_as_double((long long)top64) / qmax));
    const bool grown = lo > 0 && scale > prior;
    const double rinv = 1.0 / (double)scale;
    // fp32 quotients: their factor and the bound of their error; outside the middle of fp32's range
    // (and for scale 0) everything is done in fp64
    const float quick = (float)rinv;
    const bool mid = scale > 0x1p-100f && scale < 0x1p100f && !odd;
    const float err = 0x1p-23f * (big[1] * quick + 2.0f * (float)qmax);
    if (tid == 0)
        c.ks[pl.ph] = scale;

    float fast[8] = {};  // sums of codes (exact: at most 8 of up to 448 in steps of 2^-9)
    int acc[8] = {};     // the same times 512, of the units that are done below
    uint32_t again = 0;  // units for fp64, older tokens among them
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int slot = (tid + i * kThreads) / U;
        if (slot >= hi || (slot < lo && !grown && !c.km))
            continue;
        float y0[4], y1[4], v0[4], v1[4];
        uint32_t w0, w1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y0[j] = x[i][j] * quick;
            y1[j] = x[i][4 + j] * quick;
        }
        const bool sure = quick_codes(y0, err, c.fmt, w0, v0) & quick_codes(y1, err, c.fmt, w1, v1);
        if (slot >= lo && mid && sure) {
            *(uint32_t *)(kp + slot * D + d0) = w0;
            *(uint32_t *)(kp + slot * D + d1) = w1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                fast[j] += v0[j];
                fast[4 + j] += v1[j];
            }
        } else {
            again |= 1u << i;
        }
    }
    while (again) {
        const int slot = (tid + __builtin_ctz(again) * kThreads) / U;
        again &= again - 1;
        uint32_t *p0 = (uint32_t *)(kp + slot * D + d0), *p1 = (uint32_t *)(kp + slot * D + d1);
        uint32_t w0 = 0, w1 = 0;
        if (slot >= lo) {
            double y[8];
            exact_unit(slot, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w0 |= encode(y[j], scale, rinv, c.fmt) << (8 * j);
                w1 |= encode(y[4 + j], scale, rinv, c.fmt) << (8 * j);
            }
            *p0 = w0;
            *p1 = w1;
        } else {
            w0 = *p0;
            w1 = *p1;
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
                *p0 = w0;
                *p1 = w1;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[j] += code_512((w0 >> (8 * j)) & 0xff, c.fmt);
            acc[4 + j] += code_512((w1 >> (8 * j)) & 0xff, c.fmt);
        }
    }
    if (!c.km)
        return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        atomicAdd(&sums[d0 + j], acc[j] + (int)(fast[j] * 512.0f));
        atomicAdd(&sums[d1 + j], acc[4 + j] + (int)(fast[4 + j] * 512.0f));
    }
    __syncthreads();
    if (tid < D)
        c.km[pl.ph * D + tid] = (float)((double)sums[tid] / 512.0 * (double)scale / (double)hi);
}

// Values: units of 4 tokens x 4 dimensions, transposed in registers and merged into the page's
// [dim][token] bytes in LDS, so that the page is written in whole 16-byte vectors.
template <class T, int D, int P>
__device__ inline void append_values(const Kv8Cache &c, const T *v, int64_t v_stride,
                                     const Place &pl, int head)
{
    constexpr int NV = P * D / 16 / kThreads ? P * D / 16 / kThreads : 1;
    constexpr int ROW = P / 4 + 1;          // LDS words per dimension (padded)
    __shared__ uint32_t vpage[D * ROW];
    __shared__ float red[4];
    const int tid = threadIdx.x, lo = pl.lo, hi = pl.hi;
    uint8_t *vp = c.v + pl.ph * (P * D);
    const T *src = v + pl.src0 * v_stride + (int64_t)head * D;
    float w[NV][4][4];  // [unit][token][dimension]
    float big[1] = {0.0f}, bad = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int unit = tid + i * kThreads, tq = unit / (D / 4), dq = unit % (D / 4);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int slot = tq * 4 + t;
            if (slot >= lo && slot < hi) {
                load4(src + slot * v_stride + dq * 4, w[i][t]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[i][t][j] = 0.0f;
            }
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
            for (int j = 0; j < 4; j += 2) {
                big[0] = fmaxf(fmaxf(fabsf(w[i][t][j]), fabsf(w[i][t][j + 1])), big[0]);
                bad = fmaf(w[i][t][j], 0.0f, fmaf(w[i][t][j + 1], 0.0f, bad));
            }
    // a thread that holds something not finite looks through its values again
    const bool odd = !(bad == 0.0f);
    if (odd) {
        big[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    big[0] = fmaxf(big[0],
                                   fabsf(w[i][t][j]) <= 3.4028234e38f ? fabsf(w[i][t][j]) : 0.0f);
    }
    block_max(big, red);
    const double qmax = c.fmt == CFZ_KV8_INT8 ? 127.0 : 448.0;
    const float scale = fmaxf(prior, (float)((double)big[0] / qmax));
    const bool grown = lo > 0 && scale > prior;
    const double rinv = 1.0 / (double)scale;
    const float quick = (float)rinv;
    const bool mid = scale > 0x1p-100f && scale < 0x1p100f && !odd;
    const float err = 0x1p-23f * (2.0f * (float)qmax);
    if (tid == 0)
        c.vs[pl.ph] = scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int unit = tid + i * kThreads, tq = unit / (D / 4), dq = unit % (D / 4);
        if (tq >= P / 4 || (tq * 4 >= hi) || (tq * 4 + 4 <= lo && !grown))
            continue;
        const bool whole = mid && tq * 4 >= lo && tq * 4 + 4 <= hi;
        uint32_t rest = 0;  // dimensions for fp64
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float y[4] = {w[i][0][j] * quick, w[i][1][j] * quick, w[i][2][j] * quick,
                                w[i][3][j] * quick};
            float unused[4];
            uint32_t word;
            if (quick_codes(y, err, c.fmt, word, unused) && whole)
                vpage[(dq * 4 + j) * ROW + tq] = word;
            else
                rest |= 1u << j;
        }
        while (rest) {
            const int j = __builtin_ctz(rest);
            rest &= rest - 1;
            uint32_t *o = vpage + (dq * 4 + j) * ROW + tq;
            const uint32_t was = *o;
            uint32_t now = 0;
#pragma unroll 1
            for (int t = 0; t < 4; ++t) {
                const int slot = tq * 4 + t;
                const uint32_t byte = (was >> (8 * t)) & 0xff;
                uint32_t e = byte;
                if (slot >= lo && slot < hi)
                    e = encode(widen(src[slot * v_stride + dq * 4 + j]), scale, rinv, c.fmt);
                else if (slot < lo && grown)
                    e = encode((double)code_value(byte, c.fmt) * prior, scale, rinv, c.fmt);
                now |= e << (8 * t);
            }
            *o = now;
        }
    }
    __syncthreads();
    for (int i = tid; i < D * P / 16; i += kThreads) {
        const uint32_t *o = vpage + (i * 4 / (P / 4)) * ROW + i * 4 % (P / 4);
        ((uint4 *)vp)[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <class T, int D, int P>
__global__ __launch_bounds__(kThreads) void kv8_append_kernel(Kv8Cache c, Kv8Batch b, const T *k,
                                                              const T *v, int64_t k_stride,
                                                              int64_t v_stride, Kv8Rotation rot,
                                                              int span)
{
    Place pl;
    const int64_t g = blockIdx.x / 2;
    if (!find_place<P>(c, b, span, g, pl) || pl.page < 0)
        return;
    const int head = (int)(g / span % c.heads);
    if (blockIdx.x & 1)
        append_values<T, D, P>(c, v, v_stride, pl, head);
    else
        append_keys<T, D, P>(c, k, k_stride, rot, pl, head);
}

// Reads one page of one head back: keys straight, values through LDS (their codes are dimension-major),
// rows written in vectors of 4 values.
template <class T, int D, int P>
__global__ __launch_bounds__(kThreads) void kv8_gather_kernel(Kv8Cache c, Kv8Batch b, T *k, T *v,
                                                              int span)
{
    constexpr int ROW = P / 4 + 1;
    __shared__ uint32_t vpage[D * ROW];
    const int tid = threadIdx.x;
    int64_t g = blockIdx.x;
    const int at = (int)(g % span);
    g /= span;
    const int head = (int)(g % c.heads);
    const int seq = (int)(g / c.heads);
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
// per work-group).
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
// (the same work whatever the keys), then the pages above it and, in index order, as many at it as are left
// are written in ascending order.
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

// Work-groups of a page-wise launch over `span` pages per sequence, 0 if there is nothing to do.
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
        kv8_append_kernel<T, D, P><<<grid, kThreads, 0, st>>>(c, b, (const T *)k, (const T *)v, ks, \
                                                              vs, rot, span);
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
