// kv8_attend_kernels.hip -- softmax attention over the 8-bit paged K/V cache.
//
// With key codes c_t and value codes e_t, page scales s_t and z_t, and y_t = scale log2(e)
// s_t (q . c_t) + log2(z_t), the output is
//   out = sum_t 2^(y_t - m) e_t / sum_t 2^(y_t - m) / z_t
// for any m: the key scale multiplies the score, the value scale joins the exponent, and both products
// run on the codes themselves, which fp16 holds exactly (v_mfma_f32_*_f16).  One pass over the keys keeps
// the running maximum m of y; the accumulators are rescaled only where it grew by more than
// kSlack, and the weights carry 2^kLift so that the ones that fp16 flushes are under
// 2^-(24 + kLift) of the largest.
//
// Both kernels compute S^T = K Q^T: in the accumulator's layout a lane then holds scores of ONE query
// (its column), so maximum, sum and rescaling need no exchange inside the loop, and the
// weights are, as they lie, the B operand of O^T = V^T P^T.  The order of the keys inside a
// tile is free; it is chosen so that a lane's consecutive weights belong to consecutive
// tokens, which is how V's dimension-major pages store them.
#include "kv8_internal.h"

#include <limits.h>
#include <math.h>

#include <type_traits>

namespace cfz {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr float kLift = 10.0f;
constexpr float kSlack = 5.0f;  // weights reach 2^(kLift + kSlack) = 2^15 < 65504
constexpr float kNone = -3.0e38f;
constexpr float kTinyScale = 0x1p-100f;
constexpr int kBlock = 64;  // keys per step

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// 4 codes to fp16, exactly.
template <int FMT> __device__ inline void to_half4(uint32_t w, h2 &a, h2 &b)
{
    if constexpr (FMT == CFZ_KV8_INT8) {
        // 0x6400 | u is 1024 + u; u = code + 128
        const uint32_t u = w ^ 0x80808080u;
        const h2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
        a = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - bias;
        b = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - bias;
    } else {
        a = __builtin_bit_cast(h2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
        b = __builtin_bit_cast(h2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
    }
}

template <int FMT> __device__ inline h8 to_half8(uint32_t w0, uint32_t w1)
{
    h2 a, b, c, d;
    to_half4<FMT>(w0, a, b);
    to_half4<FMT>(w1, c, d);
    return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ inline h2 pack(float a, float b) { return __builtin_convertvector((f2){a, b}, h2); }

// Which rows a work-group has: rows r0 .. of the rows (query, shared head) of one query block.
struct Tile {
    int seq, head, split;
    int row0;      // token row of the sequence's first query
    int n;         // its queries
    int len;       // its keys
    int q0;        // first query of the block
    int rows;      // rows of the block, (queries in it) * group
    int r0;        // first row of the tile
    const int32_t *list;  // the block's pages or null
};

template <int BM>
__device__ inline bool find_tile(const Kv8Cache &c, const Kv8Batch &b, const Kv8Attend &a,
                                 const Kv8Plan &p, Tile &t)
{
    // Consecutive work-groups go round the 8 XCDs; give each XCD consecutive tiles, so that the
    // tiles that read the same keys share an L2.
    const unsigned total = (unsigned)p.groups, id = blockIdx.x;
    const unsigned q = total / 8, r = total % 8, x = id % 8;
    unsigned g = x * q + (x < r ? x : r) + id / 8;
    const unsigned tile = g % (unsigned)p.tiles;
    g /= (unsigned)p.tiles;
    const unsigned unit = g % (unsigned)p.units;
    g /= (unsigned)p.units;
    t.split = g % (unsigned)p.splits;
    g /= (unsigned)p.splits;
    t.head = g % (unsigned)c.heads;
    t.seq = g / (unsigned)c.heads;
    kv8_rows(b, t.seq, t.row0, t.n);
    t.len = kv8_length(b, t.seq, a.max_kv);
    const int64_t q0 = (int64_t)unit * a.q_block;
    if (q0 >= t.n)
        return false;
    t.q0 = (int)q0;
    const int64_t nq = t.n - q0 < a.q_block ? t.n - q0 : a.q_block;
    t.rows = (int)(nq * a.group);
    t.r0 = tile * BM;
    t.list = a.blocks ? a.blocks + (((int64_t)t.seq * p.units + unit) * c.heads + t.head) * a.count
                      : nullptr;
    return t.r0 < t.rows;
}

// Keys that query qi of the sequence sees: the tokens below this.
__device__ inline int reach(const Tile &t, int causal, int qi)
{
    if (!causal)
        return t.len;
    const int64_t e = (int64_t)t.len - t.n + qi + 1;
    return e < 0 ? 0 : (int)e;
}

// Half a step: 32 tokens, all in one page (or in none: page < 0).
struct Half {
    int page, tok;
    float kscale, vscale;
};

// The half that starts at position `vt` of the tile's keys: of the sequence itself, or of its listed
// pages one after the other.
__device__ inline Half find_half(const Kv8Cache &c, const Kv8Batch &b, const Kv8Attend &a,
                                 const Tile &t, int vt, int reach_max)
{
    Half h;
    int logical = vt >> c.log2page;
    if (t.list)
        logical = logical < a.count ? t.list[logical] : -1;
    if (logical >= b.width)
        logical = -1;
    h.tok = logical * c.page + (vt & (c.page - 1));
    h.page = logical >= 0 && h.tok < reach_max ? kv8_page(c, b, t.seq, logical) : -1;
    h.page = __builtin_amdgcn_readfirstlane(h.page);
    h.kscale = h.vscale = 0.0f;
    if (h.page >= 0) {
        const int64_t ph = (int64_t)h.page * c.heads + t.head;
        h.kscale = c.ks[ph];
        h.vscale = c.vs[ph];
    }
    return h;
}

// What a lane needs of a half: y = acc * mul + add, and the weight's share of the denominator.
struct Factor {
    float mul, add, back;
    bool flush;  // the value codes count as zeros
};

__device__ inline Factor factor(const Half &h, float qmul)
{
    Factor f;
    f.flush = !(h.vscale >= kTinyScale);
    const float z = f.flush ? kTinyScale : h.vscale;
    f.mul = h.kscale * qmul;
    f.add = __builtin_log2f(z);
    f.back = 1.0f / z;
    return f;
}

// Zeroes the codes of the 16 tokens from `tok` that are not live (unwritten memory may hold
// anything, and 0 * NaN is NaN).
__device__ inline u4 keep_live(u4 w, int tok, int len)
{
    const int live = len - tok;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = live - 4 * i;
        w[i] &= k >= 4 ? ~0u : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
    }
    return w;
}

// N consecutive entries of a query row as fp32.
template <int N> __device__ inline void load_q(const Kv8Attend &a, int64_t at, float (&x)[N])
{
    static_assert(N % 8 == 0, "16-byte loads");
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        const u4 w = *(const u4 *)((const uint16_t *)a.q + at + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t pair = w[j];  // (__builtin_bit_cast of a vector's element takes element 0)
            if (a.f16) {
                const h2 h = __builtin_bit_cast(h2, pair);
                x[i + 2 * j] = (float)h[0];
                x[i + 2 * j + 1] = (float)h[1];
            } else {
                x[i + 2 * j] = __uint_as_float(pair << 16);
                x[i + 2 * j + 1] = __uint_as_float(pair & 0xffff0000u);
            }
        }
    }
}

// The power of two that brings the row's largest entry to [2^14, 2^15): every bf16 or fp16
// entry down to 2^-29 of it is then a normal fp16 number.
__device__ inline float row_scale(float largest, float &inverse)
{
    if (!(largest > 0.0f && largest <= 3.4028234e38f)) {
        inverse = 1.0f;
        return 1.0f;
    }
    int e = 15 - (ilogbf(largest) + 1);
    e = e > 120 ? 120 : e;
    inverse = ldexpf(1.0f, -e);
    return ldexpf(1.0f, e);
}

__device__ inline uint32_t out_pair(float a, float b, int f16)
{
    if (f16)
        return __builtin_bit_cast(uint32_t, pack(a, b));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
}

// 4 consecutive entries of an output row.
__device__ inline void store_out(const Kv8Attend &a, int64_t at, float x0, float x1, float x2,
                                 float x3)
{
    uint2 w;
    w.x = out_pair(x0, x1, a.f16);
    w.y = out_pair(x2, x3, a.f16);
    *(uint2 *)((uint16_t *)a.out + at) = w;
}

__device__ inline float lse_of(float m, float l)
{
    return l > 0.0f ? (m - kLift + __builtin_log2f(l)) * 0.69314718055994531f
                    : (l == l ? -__builtin_inff() : l);
}

// Partial results of a split: m, l, then D sums, fp32, per (split, token row, query head).
__device__ inline float *partial(const Kv8Attend &a, const Kv8Batch &b, int D, int split,
                                 int64_t row, int head)
{
    return a.ws + (((int64_t)split * b.tokens + row) * a.q_heads + head) * (D + 4);
}

// ------------------------------------------------------------------ few rows
//
// 16 rows per work-group; its four waves take every fourth step of 64 keys, straight from memory into
// registers (each code is used by one wave only, so LDS would add a trip), and join their
// sums at the end.  Bound by the codes' bytes: at head_dim 128 a wave has 16 KB in flight.
template <int FMT, int D>
__global__ __launch_bounds__(256, 2) void kv8_attend_narrow_kernel(Kv8Cache c, Kv8Batch b,
                                                                   Kv8Attend a, Kv8Plan p)
{
    constexpr int BM = 16;
    constexpr int KS = D / 32;  // MFMA steps over the dimensions
    constexpr int KL = D / 64;  // 16-byte loads per key row and lane
    constexpr int DT = D / 16;  // tiles of output dimensions
    Tile t;
    if (!find_tile<BM>(c, b, a, p, t))
        return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;

    const int r = t.r0 + col;
    const bool have = r < t.rows;
    const int qi = t.q0 + (have ? r : t.rows - 1) / a.group;
    const int qh = t.head * a.group + (have ? r : t.rows - 1) % a.group;
    const int last_row = t.r0 + BM < t.rows ? t.r0 + BM - 1 : t.rows - 1;
    const int reach_min = reach(t, a.causal, t.q0 + t.r0 / a.group);
    const int reach_max = reach(t, a.causal, t.q0 + last_row / a.group);
    const int mine = reach(t, a.causal, qi);

    // the query row, lane group g holding dimensions g D/4 .. (the order of the dimensions in the
    // contraction is free: it follows the keys' 16-byte loads)
    h8 q[KS];
    float qmul;
    {
        float x[D / 4];
        load_q<D / 4>(a, (int64_t)(t.row0 + qi) * a.q_stride + (int64_t)qh * D + g * (D / 4), x);
        float big = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i)
            big = fmaxf(big, fabsf(x[i]));
        big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        float inv;
        const float up = row_scale(big, inv);
        qmul = inv * (a.scale * 1.4426950408889634f);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                q[s][j] = (_Float16)(x[s * 8 + j] * up);
    }

    const int keys = t.list ? a.count << c.log2page : reach_max;
    const int steps = (keys + kBlock - 1) / kBlock;
    const int s0 = (int)((int64_t)steps * t.split / p.splits);
    const int s1 = (int)((int64_t)steps * (t.split + 1) / p.splits);

    f4 o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i)
        o[i] = f4{0, 0, 0, 0};
    float m = kNone, l = 0.0f;

    // Key row `col` of tile u is token 16 (col / 4) + 4 u + col % 4: accumulator i of lane group g
    // in tile u is then token 16 g + 4 u + i.
    const int64_t page_bytes = (int64_t)c.page * D;
    const int kchunk = col >> 2, krow = (col & 3) + 16 * (kchunk & 1);

    struct Step {
        Half h[2];
        u4 k[4][KL], v[DT];
    };
    auto meta = [&](int s, Step &x) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            x.h[i] = find_half(c, b, a, t, s * kBlock + 32 * i, reach_max);
    };
    auto load = [&](Step &x) {
        const int pk = x.h[kchunk >> 1].page, pv = x.h[g >> 1].page;
        const int sk = x.h[kchunk >> 1].tok & (c.page - 1), sv = x.h[g >> 1].tok & (c.page - 1);
        if (pk >= 0) {
            const uint8_t *kp = c.k + ((int64_t)pk * c.heads + t.head) * page_bytes +
                                (sk + krow) * D + g * (D / 4);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < KL; ++j)
                    x.k[u][j] = *(const u4 *)(kp + u * 4 * D + j * 16);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < KL; ++j)
                    x.k[u][j] = u4{0, 0, 0, 0};
        }
        if (pv >= 0) {
            const uint8_t *vp = c.v + ((int64_t)pv * c.heads + t.head) * page_bytes +
                                col * c.page + sv + 16 * (g & 1);
#pragma unroll
            for (int i = 0; i < DT; ++i)
                x.v[i] = *(const u4 *)(vp + i * 16 * c.page);
        } else {
#pragma unroll
            for (int i = 0; i < DT; ++i)
                x.v[i] = u4{0, 0, 0, 0};
        }
    };

    Step x;
    int s = s0 + wave;
    if (s < s1) {
        meta(s, x);
        load(x);
    }
    for (; s < s1; s += 4) {
        // scores
        f4 acc[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            acc[u] = f4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const u4 w = x.k[u][j / 2];
                acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    to_half8<FMT>(w[j % 2 * 2], w[j % 2 * 2 + 1]), q[j], acc[u], 0, 0, 0);
            }
        }
        const Half h0 = x.h[0], h1 = x.h[1];
        u4 v[DT];
#pragma unroll
        for (int i = 0; i < DT; ++i)
            v[i] = x.v[i];
        if (s + 4 < s1) {
            meta(s + 4, x);
            load(x);
        }
        const Half h = g < 2 ? h0 : h1;
        const Factor f = factor(h, qmul);
        const int tok = h.tok + 16 * (g & 1);
        const bool plain = h0.page >= 0 && h1.page >= 0 && h0.tok + 32 <= reach_min &&
                           h1.tok + 32 <= reach_min && !(h0.vscale < kTinyScale) &&
                           !(h1.vscale < kTinyScale);
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            y[i] = fmaf(acc[i / 4][i % 4], f.mul, f.add);
        if (!plain) {
            const bool none = h.page < 0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                y[i] = none || tok + i >= mine ? -__builtin_inff() : y[i];
#pragma unroll
            for (int i = 0; i < DT; ++i)
                v[i] = f.flush ? u4{0, 0, 0, 0} : keep_live(v[i], tok, t.len);
        }
        float top = y[0];
#pragma unroll
        for (int i = 1; i < 16; ++i)
            top = fmaxf(top, y[i]);
        if (__any(top > m + kSlack)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float now = fmaxf(m, top), fall = exp2_fast(m - now);
            m = now;
            l *= fall;
#pragma unroll
            for (int i = 0; i < DT; ++i)
                o[i] *= fall;
        }
        float sum = 0.0f;
        h8 w[2];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float e0 = exp2_fast(y[i] + (kLift - m)), e1 = exp2_fast(y[i + 1] + (kLift - m));
            sum += e0 + e1;
            const h2 e = pack(e0, e1);
            w[i / 8][i % 8] = e[0];
            w[i / 8][i % 8 + 1] = e[1];
        }
        l = fmaf(sum, f.back, l);
#pragma unroll
        for (int i = 0; i < DT; ++i) {
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_half8<FMT>(v[i][0], v[i][1]), w[0],
                                                          o[i], 0, 0, 0);
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_half8<FMT>(v[i][2], v[i][3]), w[1],
                                                          o[i], 0, 0, 0);
        }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // join the four waves
    __shared__ float om[4][16], ol[4][16], oo[4][16][D + 4];
    if (g == 0) {
        om[wave][col] = m;
        ol[wave][col] = l;
    }
#pragma unroll
    for (int i = 0; i < DT; ++i)
        *(f4 *)&oo[wave][col][i * 16 + g * 4] = o[i];
    __syncthreads();
    for (int i = threadIdx.x; i < BM * (D / 4); i += 256) {
        const int row = i / (D / 4), d = i % (D / 4) * 4, rr = t.r0 + row;
        if (rr >= t.rows)
            break;
        float mm = fmaxf(fmaxf(om[0][row], om[1][row]), fmaxf(om[2][row], om[3][row]));
        // a NaN row stays one: its sums are NaN whatever the weights
        float ll = 0.0f;
        f4 s = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float e = exp2_fast(om[w][row] - mm);
            ll += ol[w][row] * e;
            s += *(const f4 *)&oo[w][row][d] * e;
        }
        const int64_t qrow = t.row0 + t.q0 + rr / a.group;
        const int head = t.head * a.group + rr % a.group;
        if (p.splits > 1) {
            float *out = partial(a, b, D, t.split, qrow, head);
            if (d == 0) {
                out[0] = mm;
                out[1] = ll;
            }
            *(f4 *)(out + 4 + d) = s;
        } else {
            const float inv = ll > 0.0f ? 1.0f / ll : (ll == ll ? 0.0f : ll);
            store_out(a, qrow * a.out_stride + (int64_t)head * D + d, s[0] * inv, s[1] * inv,
                      s[2] * inv, s[3] * inv);
            if (a.lse && d == 0)
                a.lse[qrow * a.q_heads + head] = lse_of(mm, ll);
        }
    }
}

// ------------------------------------------------------------------ many rows
//
// 128 rows per work-group, 32 per wave (v_mfma_f32_32x32x16_f16).  Each step's codes are read
// once per work-group, one step ahead, converted to fp16 on the way into LDS (each code once instead of once
// per wave) and read from there by all four waves.  16-byte chunks of a row are exchanged by an XOR of
// row bits, so that the eight lanes that LDS serves together read eight different bank groups.
template <int FMT, int D>
__global__ __launch_bounds__(256, 2) void kv8_attend_wide_kernel(Kv8Cache c, Kv8Batch b,
                                                                 Kv8Attend a, Kv8Plan p)
{
    constexpr int BM = 128;
    constexpr int KS = D / 16;       // MFMA steps over the dimensions
    constexpr int DT = D / 32;       // tiles of output dimensions
    constexpr int TPR = D / 16;      // threads per key row of codes
    constexpr int NL = D * kBlock / 16 / 256;  // 16-byte loads per thread, keys and values alike
    __shared__ h8 ks[2][kBlock][D / 8];
    __shared__ h8 vs[2][D][kBlock / 8];
    Tile t;
    if (!find_tile<BM>(c, b, a, p, t))
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 31, g = lane >> 5;

    const int r = t.r0 + wave * 32 + col;
    const bool have = r < t.rows;
    const int qi = t.q0 + (have ? r : t.rows - 1) / a.group;
    const int qh = t.head * a.group + (have ? r : t.rows - 1) % a.group;
    const int last_row = t.r0 + BM < t.rows ? t.r0 + BM - 1 : t.rows - 1;
    const int reach_min = reach(t, a.causal, t.q0 + t.r0 / a.group);
    const int reach_max = reach(t, a.causal, t.q0 + last_row / a.group);
    const int mine = reach(t, a.causal, qi);
    const int64_t row = t.row0 + qi;

    h8 q[KS];
    float qmul;
    {
        float x[KS][8];
        float big = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            load_q<8>(a, row * a.q_stride + (int64_t)qh * D + s * 16 + g * 8, x[s]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                big = fmaxf(big, fabsf(x[s][j]));
        }
        big = fmaxf(big, __shfl_xor(big, 32));
        float inv;
        const float up = row_scale(big, inv);
        qmul = inv * (a.scale * 1.4426950408889634f);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                q[s][j] = (_Float16)(x[s][j] * up);
    }

    const int keys = t.list ? a.count << c.log2page : reach_max;
    const int steps = (keys + kBlock - 1) / kBlock;
    const int s0 = (int)((int64_t)steps * t.split / p.splits);
    const int s1 = (int)((int64_t)steps * (t.split + 1) / p.splits);

    f16v o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            o[i][j] = 0.0f;
    float m = kNone, l = 0.0f;

    const int64_t page_bytes = (int64_t)c.page * D;
    u4 kr[NL], vr[NL];
    Half next[2];
    // the threads' share of a step: key rows of 16 codes, value rows of 16 tokens
    const int krow = tid / TPR, kcol = tid % TPR, vrow = tid / 4, vcol = tid % 4;
    auto load = [&](int s) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            next[i] = find_half(c, b, a, t, s * kBlock + 32 * i, reach_max);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int rr = krow + i * (256 / TPR), hk = rr >> 5;
            const int pk = hk ? next[1].page : next[0].page;
            const int sk = (hk ? next[1].tok : next[0].tok) & (c.page - 1);
            kr[i] = u4{0, 0, 0, 0};
            if (pk >= 0)
                kr[i] = *(const u4 *)(c.k + ((int64_t)pk * c.heads + t.head) * page_bytes +
                                      (sk + (rr & 31)) * D + kcol * 16);
            const int dd = vrow + i * 64, hv = vcol >> 1;
            const int pv = hv ? next[1].page : next[0].page;
            const int tv = hv ? next[1].tok : next[0].tok;
            vr[i] = u4{0, 0, 0, 0};
            if (pv >= 0)
                vr[i] = *(const u4 *)(c.v + ((int64_t)pv * c.heads + t.head) * page_bytes +
                                      dd * c.page + (tv & (c.page - 1)) + 16 * (vcol & 1));
        }
    };
    auto stage = [&](int buf) {
        const bool whole = next[0].tok + 32 <= t.len && next[1].tok + 32 <= t.len &&
                           next[0].vscale >= kTinyScale && next[1].vscale >= kTinyScale;
        if (!whole) {
            const Half h = vcol >> 1 ? next[1] : next[0];
#pragma unroll
            for (int i = 0; i < NL; ++i)
                vr[i] = h.vscale >= kTinyScale ? keep_live(vr[i], h.tok + 16 * (vcol & 1), t.len)
                                               : u4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int rr = krow + i * (256 / TPR);
            const int sw = (rr & 3) | ((rr >> 4 & 1) << 2) | ((rr >> 2 & 1) << 3);
            ks[buf][rr][(kcol * 2) ^ (sw & (D / 8 - 1))] = to_half8<FMT>(kr[i][0], kr[i][1]);
            ks[buf][rr][(kcol * 2 + 1) ^ (sw & (D / 8 - 1))] = to_half8<FMT>(kr[i][2], kr[i][3]);
            const int dd = vrow + i * 64;
            vs[buf][dd][(vcol * 2) ^ (dd & 7)] = to_half8<FMT>(vr[i][0], vr[i][1]);
            vs[buf][dd][(vcol * 2 + 1) ^ (dd & 7)] = to_half8<FMT>(vr[i][2], vr[i][3]);
        }
    };

    // key row `col` of a 32-token half is token 16 (col >> 2 & 1) + (col & 3) + 4 (col >> 3):
    // accumulator i of lane group g is then token 16 g + i
    const int ktok = 16 * (col >> 2 & 1) + (col & 3) + 4 * (col >> 3);
    const int ksw = ((ktok & 3) | ((ktok >> 4 & 1) << 2) | ((ktok >> 2 & 1) << 3)) & (D / 8 - 1);

    if (s0 < s1) {
        load(s0);
        stage(0);
    }
    __syncthreads();
    for (int s = s0; s < s1; ++s) {
        const int buf = (s - s0) & 1;
        const Half h[2] = {next[0], next[1]};
        if (s + 1 < s1)
            load(s + 1);
        f16v acc[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                acc[x][j] = 0.0f;
#pragma unroll
            for (int j = 0; j < KS; ++j)
                acc[x] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                    ks[buf][x * 32 + ktok][(2 * j + g) ^ ksw], q[j], acc[x], 0, 0, 0);
        }
        const bool plain = h[0].page >= 0 && h[1].page >= 0 && h[0].tok + 32 <= reach_min &&
                           h[1].tok + 32 <= reach_min;
        Factor f[2];
        float top = -__builtin_inff();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            f[x] = factor(h[x], qmul);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                acc[x][j] = fmaf(acc[x][j], f[x].mul, f[x].add);
            if (!plain) {
                const int tok = h[x].tok + 16 * g;
                const bool none = h[x].page < 0;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    acc[x][j] = none || tok + j >= mine ? -__builtin_inff() : acc[x][j];
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                top = fmaxf(top, acc[x][j]);
        }
        if (__any(top > m + kSlack)) {
            top = fmaxf(top, __shfl_xor(top, 32));
            const float now = fmaxf(m, top), fall = exp2_fast(m - now);
            m = now;
            l *= fall;
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    o[i][j] *= fall;
        }
        h8 w[4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const float e0 = exp2_fast(acc[x][j] + (kLift - m));
                const float e1 = exp2_fast(acc[x][j + 1] + (kLift - m));
                sum += e0 + e1;
                const h2 e = pack(e0, e1);
                w[2 * x + j / 8][j % 8] = e[0];
                w[2 * x + j / 8][j % 8 + 1] = e[1];
            }
            l = fmaf(sum, f[x].back, l);
        }
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // weights j of lane group g: tokens 32 (j / 2) + 16 g + 8 (j % 2) ..
                const int chunk = 4 * (j / 2) + 2 * g + j % 2;
                o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                    vs[buf][i * 32 + col][chunk ^ (col & 7)], w[j], o[i], 0, 0, 0);
            }
        if (s + 1 < s1)
            stage(buf ^ 1);
        __syncthreads();
    }
    l += __shfl_xor(l, 32);
    if (!have)
        return;
    if (p.splits > 1) {
        float *out = partial(a, b, D, t.split, row, qh);
        if (g == 0) {
            out[0] = m;
            out[1] = l;
        }
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *(f4 *)(out + 4 + i * 32 + j * 8 + g * 4) =
                    f4{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
    } else {
        const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                store_out(a, row * a.out_stride + (int64_t)qh * D + i * 32 + j * 8 + g * 4,
                          o[i][4 * j] * inv, o[i][4 * j + 1] * inv, o[i][4 * j + 2] * inv,
                          o[i][4 * j + 3] * inv);
        if (a.lse && g == 0)
            a.lse[row * a.q_heads + qh] = lse_of(m, l);
    }
}

// Joins the splits' partial results: D / 4 threads per row.
template <int D>
__global__ __launch_bounds__(256) void kv8_join_kernel(Kv8Cache c, Kv8Batch b, Kv8Attend a,
                                                       Kv8Plan p, int chunks)
{
    constexpr int PER = 256 / (D / 4);
    const int seq = blockIdx.x / chunks;
    int row0, n;
    kv8_rows(b, seq, row0, n);
    const int64_t i = (int64_t)(blockIdx.x % chunks) * PER + threadIdx.x / (D / 4);
    if (i >= (int64_t)n * a.q_heads)
        return;
    const int64_t row = row0 + i / a.q_heads;
    const int head = (int)(i % a.q_heads), d = threadIdx.x % (D / 4) * 4;
    float m = kNone;
    for (int s = 0; s < p.splits; ++s)
        m = fmaxf(m, partial(a, b, D, s, row, head)[0]);
    float l = 0.0f;
    f4 o = {0, 0, 0, 0};
    for (int s = 0; s < p.splits; ++s) {
        const float *x = partial(a, b, D, s, row, head);
        const float e = exp2_fast(x[0] - m);
        l += x[1] * e;
        o += *(const f4 *)(x + 4 + d) * e;
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
    store_out(a, row * a.out_stride + (int64_t)head * D + d, o[0] * inv, o[1] * inv, o[2] * inv,
              o[3] * inv);
    if (a.lse && d == 0)
        a.lse[row * a.q_heads + head] = lse_of(m, l);
}

constexpr int64_t kNarrowRows = 32;  // rows of a query block up to which the narrow kernel is taken
constexpr int64_t kFill = 512;       // work-groups that fill the chip (two on each of 256 CUs)

}  // namespace

Kv8Plan kv8_plan(const Kv8Cache &c, const Kv8Batch &b, int q_heads, int64_t max_kv, bool listed,
                 int64_t q_block, int count)
{
    Kv8Plan p;
    const int64_t group = q_heads / c.heads;
    if (!listed || q_block > b.max_rows)
        q_block = b.max_rows;
    const int64_t rows = q_block * group;
    p.wide = rows > kNarrowRows;
    p.units = q_block > 0 ? (b.max_rows + q_block - 1) / q_block : 0;
    p.tiles = p.wide ? (rows + 127) / 128 : (rows + 15) / 16;
    const int64_t whole = p.units * p.tiles * c.heads * b.batch;
    const int64_t keys = listed && (int64_t)count * c.page < max_kv ? (int64_t)count * c.page : max_kv;
    const int64_t steps = (keys + kBlock - 1) / kBlock;
    // a part should have some steps for each wave, or its joining costs more than it saves
    int64_t splits = whole > 0 ? kFill / whole : 1;
    const int64_t most = steps / (p.wide ? 4 : 8);
    splits = splits < most ? splits : most;
    p.splits = (int)(splits < 1 ? 1 : (splits > 128 ? 128 : splits));
    p.groups = whole * p.splits;
    return p;
}

hipError_t launch_kv8_attend(const Kv8Cache &c, const Kv8Batch &b, const Kv8Attend &a,
                             const Kv8Plan &p, hipStream_t st)
{
    const dim3 grid((unsigned)p.groups);
#define CFZ_KV8_CASE(F, D)                                                                         \
    if (c.fmt == F && c.dim == D) {                                                                \
        if (p.wide)                                                                                \
            kv8_attend_wide_kernel<F, D><<<grid, 256, 0, st>>>(c, b, a, p);                        \
        else                                                                                       \
            kv8_attend_narrow_kernel<F, D><<<grid, 256, 0, st>>>(c, b, a, p);                      \
    }
    CFZ_KV8_CASE(CFZ_KV8_INT8, 64)
    CFZ_KV8_CASE(CFZ_KV8_INT8, 128)
    CFZ_KV8_CASE(CFZ_KV8_E4M3, 64)
    CFZ_KV8_CASE(CFZ_KV8_E4M3, 128)
#undef CFZ_KV8_CASE
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1)
        return e;
    const int per = 256 / (c.dim / 4);
    const int64_t chunks = (b.max_rows * a.q_heads + per - 1) / per;
    const dim3 joins((unsigned)(chunks * b.batch));
    if (c.dim == 64)
        kv8_join_kernel<64><<<joins, 256, 0, st>>>(c, b, a, p, (int)chunks);
    else
        kv8_join_kernel<128><<<joins, 256, 0, st>>>(c, b, a, p, (int)chunks);
    return hipGetLastError();
}

}  // namespace cfz
