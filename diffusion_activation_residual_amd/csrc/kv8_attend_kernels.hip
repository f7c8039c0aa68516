// kv8_attend_kernels.hip -- softmax attention over the 8-bit paged K/V cache.
//
// With key codes c_t and value codes e_t, page scales s_t and z_t, and y_t = scale log2(e)
// s_t (q . c_t) + log2(z_t), the output is
//   out = sum_t 2^(y_t - m) e_t / sum_t 2^(y_t - m) / z_t
// for any m: the key scale multiplies the score, the value scale joins the exponent, and both
// products run on the codes themselves, which fp16 holds exactly (v_mfma_f32_*_f16).  One pass over
// the keys keeps m near the running maximum of y: it is moved, and the accumulators rescaled, only
// where the weights would grow out of fp16's range.  The weights carry 2^kLift, so that the ones that
// fp16 flushes are under 2^-(24 + kLift) of the one at m.  A query row is rounded to fp16 after a
// power of two has brought its largest entry to [2^14, 2^15) (exact for bf16 entries down to
// 2^-29 of it); scores, statistics and output sums are fp32.
//
// A denominator's terms are then 2^(y_t - m) / z_t, and fp32 holds the ones that count only while the z_t
// lie near each other: from 2^-32 to 2^32 the weight of a key whose score is 2^-54 of the highest is
// still a normal number, and the sum over 2^30 keys is finite (6 + 16 + 32 + 30 powers of two).  Pages
// whose values are zeros take part with z = 2^-32, at which nothing of them is lost or in the way.
// Where a page that is looked up has a z outside of that range, the run goes on with the denominator
// on its own: a second set of exponentials, of the scores alone, relative to a maximum ms of their own,
// so that out = 2^(m - ms) sum_t 2^(y_t - m) e_t / sum_t 2^(score_t - ms).  In the ordinary case ms is m.
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

constexpr float kLift = 6.0f;
constexpr float kSlack = 5.0f;      // (few rows) a row's maximum is moved where it is off by more
constexpr float kLimit = 60000.0f;  // (many rows) ... or where a lane's weights sum to more
constexpr float kNone = -3.0e38f;
constexpr float kTiny = -100.0f;  // log2 of the value scale up to which codes count as zeros
constexpr float kNear = 32.0f;    // ordinary value scales lie within 2^-kNear .. 2^kNear
constexpr float kApart = -kNear - kTiny;
constexpr float kApartPower = 0x1p68f;  // 2^kApart; sums of 2^30 weights times codes (2^55) stay finite
constexpr int kBlock = 64;  // keys per step
// Tiles per head whose steps a work-group counts.  A call with more is not cut into runs, and a long
// sequence among short ones is one work-group's: one single token over 131072 tokens beside others over
// 256, 8 heads of 128, 284 us and 16 for the join with 1000 sequences, 848 us with 1100.
constexpr int kMaxItems = 1023;
constexpr int kPrefixWords = kMaxItems + 1;
constexpr int kRowWords = 4;     // of a part, for each row: m, ms, l
constexpr int kCutWords = 4096;  // of the workspace: a Cut for each of at most 1024 work-groups

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

// A tile: rows r0 .. of the rows (query, shared head) of one query block, and one KV head.
struct Tile {
    int seq, head;
    int row0;      // token row of the sequence's first query
    int n;         // its queries
    int len;       // its keys
    int q0;        // first query of the block
    int rows;      // rows of the block, (queries in it) * group
    int r0;        // first row of the tile
    int reach_min, reach_max;  // keys that its first and its last row see
    int steps;     // of kBlock keys
    const int32_t *list;  // the block's pages or null
};

// x / d for x >= 0 where d is often 1 (and uniform): a division is some 40 instructions.
__device__ inline int quotient(int x, int d) { return d == 1 ? x : x / d; }

// Keys that query qi of the sequence sees: the tokens below this.
__device__ inline int reach(const Tile &t, int causal, int qi)
{
    if (!causal)
        return t.len;
    const int64_t e = (int64_t)t.len - t.n + qi + 1;
    return e < 0 ? 0 : (int)e;
}

// The tile `item` (query blocks and row tiles of one sequence after the other) of one KV head; false
// where the sequence has no such rows.
template <int BM>
__device__ inline bool find_tile(const Kv8Cache &c, const Kv8Batch &b, const Kv8Attend &a,
                                 const Kv8Plan &p, int item, int head, Tile &t)
{
    const int rest = quotient(item, p.tiles), tile = item - rest * p.tiles;
    t.seq = quotient(rest, p.units);
    const int unit = rest - t.seq * p.units;
    t.head = head;
    kv8_rows(b, t.seq, t.row0, t.n);
    t.len = kv8_length(b, t.seq, a.max_kv);
    const int64_t q0 = (int64_t)unit * a.q_block;
    if (q0 >= t.n)
        return false;
    t.q0 = (int)q0;
    const int64_t nq = t.n - q0 < a.q_block ? t.n - q0 : a.q_block;
    t.rows = (int)(nq * a.group);
    t.r0 = tile * BM;
    if (t.r0 >= t.rows)
        return false;
    t.list = a.blocks ? a.blocks + (((int64_t)t.seq * p.units + unit) * c.heads + head) * a.count
                      : nullptr;
    const int last = t.r0 + BM < t.rows ? t.r0 + BM - 1 : t.rows - 1;
    t.reach_min = reach(t, a.causal, t.q0 + quotient(t.r0, a.group));
    t.reach_max = reach(t, a.causal, t.q0 + quotient(last, a.group));
    const int keys = t.list ? a.count << c.log2page : t.reach_max;
    t.steps = c.pages > 0 ? (keys + kBlock - 1) / kBlock : 0;
    return true;
}

// Consecutive work-groups go round the 8 XCDs; give each XCD consecutive numbers, so that the
// tiles that read the same keys share an L2.
__device__ inline uint32_t by_xcd(uint32_t total)
{
    const uint32_t q = total / 8, r = total % 8, x = blockIdx.x % 8;
    return x * q + (x < r ? x : r) + blockIdx.x / 8;
}

// The steps of all tiles of all heads, laid end to end, are cut into p.groups equal runs, one per
// work-group: with tiles of different cost (ragged or causal sequences) or a number of tiles
// that does not fill the chip evenly, all work-groups end together.  prefix[i] is the number of
// steps before item i of one head (a tile without keys counts as one step: its rows are
// written); every work-group computes it from the lengths on the device.
template <int T, int BM>
__device__ inline void count_steps(const Kv8Cache &c, const Kv8Batch &b, const Kv8Attend &a,
                                   const Kv8Plan &p, int *prefix, int *waves)
{
    const int tid = threadIdx.x, per = (p.items + T - 1) / T;
    int sum = 0;
    for (int i = tid * per; i < (tid + 1) * per && i < p.items; ++i) {
        Tile t;
        const int n = !find_tile<BM>(c, b, a, p, i, 0, t) ? 0 : (t.steps > 0 ? t.steps : 1);
        prefix[i] = sum;
        sum += n;
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        incl += (tid & 63) >= d ? o : 0;
    }
    if ((tid & 63) == 63)
        waves[tid >> 6] = incl;
    __syncthreads();
    int before = incl - sum, all = 0;
    for (int w = 0; w < T / 64; ++w) {
        before += w < tid / 64 ? waves[w] : 0;
        all += waves[w];
    }
    for (int i = tid * per; i < (tid + 1) * per && i < p.items; ++i)
        prefix[i] += before;
    if (tid == 0)
        prefix[p.items] = all;
    __syncthreads();
}

// The last item that starts at or before step y (items without steps start where the next does).
__device__ inline int item_at(const int *prefix, int items, int y)
{
    int lo = 0, hi = items;  // prefix[lo] <= y < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (prefix[mid] <= y)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// A run of steps s0 .. s1 of one tile, and where its sums go: to the output if it is the whole tile,
// else to the work-group's first slot (the tile began in an earlier run) or second.
struct Run {
    uint32_t at, end;  // of the work-group, in steps of all tiles
    uint32_t each;     // steps of a work-group, one more for the first `extra` of them
    uint32_t extra, groups;
    int s0, s1;
    int slot;          // -1: the output
};

__device__ inline uint32_t run_start(const Run &r, uint32_t w)
{
    return r.each * w + (w < r.extra ? w : r.extra);
}

// The work-group that has step x.
__device__ inline uint32_t run_of(const Run &r, uint32_t x)
{
    const uint32_t head = (r.each + 1) * r.extra;
    return x < head ? x / (r.each + 1) : r.extra + (x - head) / r.each;
}

// A tile that a work-group begins and `more` later ones go on with (0: none), for the join.
struct Cut {
    int item, head, more, unused;
};

// The work-group's next run of steps, false when it is done.
template <int BM>
__device__ inline bool next_run(const Kv8Cache &c, const Kv8Batch &b, const Kv8Attend &a,
                                const Kv8Plan &p, const int *prefix, uint32_t w, Run &r, Tile &t)
{
    if (r.at >= r.end)
        return false;
    if (!p.joined) {  // one work-group, one tile
        r.at = r.end;
        r.slot = -1;
        r.s0 = 0;
        const uint32_t items = p.items;
        if (!find_tile<BM>(c, b, a, p, (int)(w % items), (int)(w / items), t))
            return false;
        r.s1 = t.steps;
        return true;
    }
    const uint32_t all = __builtin_amdgcn_readfirstlane(prefix[p.items]);
    const int head = (int)(r.at / all), y = (int)(r.at % all);
    const int item = __builtin_amdgcn_readfirstlane(item_at(prefix, p.items, y));
    const int from = __builtin_amdgcn_readfirstlane(prefix[item]);
    const int cost = __builtin_amdgcn_readfirstlane(prefix[item + 1]) - from;
    find_tile<BM>(c, b, a, p, item, head, t);
    r.s0 = y - from;
    r.s1 = (int)(r.end - r.at) < cost - r.s0 ? r.s0 + (int)(r.end - r.at) : cost;
    r.slot = r.s0 > 0 ? 2 * (int)w : (r.s1 < cost ? 2 * (int)w + 1 : -1);
    if (r.slot == 2 * (int)w + 1 && threadIdx.x == 0)
        ((Cut *)a.ws)[w] = Cut{item, head, (int)(run_of(r, r.at + cost - 1) - w), 0};
    r.at += r.s1 - r.s0;
    r.s1 = r.s1 < t.steps ? r.s1 : t.steps;
    return true;
}

template <int T, int BM>
__device__ inline Run first_run(const Kv8Cache &c, const Kv8Batch &b, const Kv8Attend &a,
                                const Kv8Plan &p, int *prefix, int *waves, uint32_t w)
{
    Run r = {0, 1, 1, 0, 1, 0, 0, -1};
    if (p.joined) {
        count_steps<T, BM>(c, b, a, p, prefix, waves);
        const uint32_t total = (uint32_t)prefix[p.items] * (uint32_t)c.heads;  // below 2^31
        r.groups = total < (uint32_t)p.groups ? total : (uint32_t)p.groups;
        r.at = r.end = 0;
        if (w < r.groups) {
            r.each = total / r.groups;
            r.extra = total % r.groups;
            r.at = run_start(r, w);
            r.end = run_start(r, w + 1);
        }
        if (threadIdx.x == 0)
            ((Cut *)a.ws)[w] = Cut{0, 0, 0, 0};
    }
    return r;
}

// Half a step: 32 tokens, all in one page (or in none: page < 0).
struct Half {
    int page, tok;
    float kscale, add;  // K's scale; log2 of V's
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
    if (logical < 0 || logical >= b.width)
        logical = -1;
    h.tok = logical * c.page + (vt & (c.page - 1));
    h.page = logical >= 0 && h.tok < reach_max ? kv8_page(c, b, t.seq, logical) : -1;
    h.kscale = 0.0f;
    h.add = kTiny;
    return h;
}

__device__ inline void find_scales(const Kv8Cache &c, const Tile &t, Half &h)
{
    if (h.page >= 0) {
        const int64_t ph = (int64_t)h.page * c.heads + t.head;
        h.kscale = c.ks[ph];
        const float z = c.vs[ph];
        h.add = z > 0x1p-100f ? __builtin_amdgcn_logf(z) : kTiny;  // (no subnormal gets there)
    }
}

// The value scale of a half that holds values lies outside of the ordinary range.
__device__ inline bool is_far(const Half &h)
{
    return h.add > kTiny && !(h.add > -kNear && h.add <= kNear);
}

// The half as it is used: what counts as zeros (a scale of 2^-100 or less, 0 above all) has the lowest
// z of all, and K's scale with its sign set to tell.
__device__ inline Half settled(Half h, int apart)
{
    h.kscale = h.add > kTiny ? h.kscale : -h.kscale;
    h.add = fmaxf(h.add, apart ? kTiny : -kNear);
    return h;
}

__device__ inline bool flushed(const Half &h) { return (int)__float_as_uint(h.kscale) < 0; }

// What a lane needs of a half: y = acc * mul + add, and the weight's share of the denominator, 2^-add.
struct Factor {
    float mul, add, back;
};

__device__ inline Factor factor(const Half &h, float qmul)
{
    Factor f;
    // not 0, so that the masked scores' -infinity stays one (the codes of scale 0 are zeros)
    f.mul = fmaxf(fabsf(h.kscale) * qmul, 0x1p-120f);
    f.add = h.add;
    f.back = exp2_fast(-h.add);
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

// 8 entries of a query row as fp32.
__device__ inline void widen_q(const u4 &w, int f16, float *x)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t pair = w[j];  // (__builtin_bit_cast of a vector's element takes element 0)
        if (f16) {
            const h2 h = __builtin_bit_cast(h2, pair);
            x[2 * j] = (float)h[0];
            x[2 * j + 1] = (float)h[1];
        } else {
            x[2 * j] = __uint_as_float(pair << 16);
            x[2 * j + 1] = __uint_as_float(pair & 0xffff0000u);
        }
    }
}

__device__ inline float first_lane(float x)
{
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// The power of two that brings the row's largest entry to [2^14, 2^15): every bf16 or fp16
// entry down to 2^-29 of it is then a normal fp16 number.
__device__ inline float row_scale(float largest, float &inverse)
{
    if (!(largest > 0.0f && largest <= 3.4028234e38f)) {
        inverse = 1.0f;
        return 1.0f;
    }
    int e = (int)(__float_as_uint(largest) >> 23) - 127;  // largest in [2^e, 2^(e + 1))
    e = e < -106 ? -106 : e;
    inverse = __uint_as_float((uint32_t)(127 + e - 14) << 23);
    return __uint_as_float((uint32_t)(127 - e + 14) << 23);
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

__device__ inline float lse_of(float ms, float l)
{
    return l > 0.0f ? (ms - kLift + __builtin_log2f(l)) * 0.69314718055994531f
                    : (l == l ? -__builtin_inff() : l);
}

// 2^(m - ms) as a product of two equal factors (value scales reach 2^121).
__device__ inline float half_power(float m, float ms) { return exp2_fast(0.5f * (m - ms)); }

// A run's sums of its tile, fp32: 16-byte pieces of the rows' sums in the order in which the kernel's
// lanes hold them, so that a store instruction covers one span, then m, ms, l and 0 of each row.
template <int BM, int D>
__device__ inline float *partial(const Kv8Attend &a, int64_t slot)
{
    return a.ws + kCutWords + slot * (BM * (D + kRowWords));
}

// ------------------------------------------------------------------ few rows
//
// 16 rows per work-group; its four waves take every fourth step of 64 keys, straight from memory into
// registers (each code is used by one wave only, so LDS would add a trip), and join their
// sums at the end.  The pages and scales of many steps are looked up together, and the next step's
// codes are under way while this one's weights are formed (each looked up in its own step, 147 us
// instead of 80).  Bound by the codes' bytes: 16 sequences of up to 16411 tokens, 8 KV heads of
// 128, 32 query heads, in 83 us, 4.9 TB/s, and 6 us for the join.
template <int FMT, int D>
__global__ __launch_bounds__(256, 2) void kv8_attend_narrow_kernel(Kv8Cache c, Kv8Batch b,
                                                                   Kv8Attend a, Kv8Plan p)
{
    constexpr int BM = 16;
    constexpr int KS = D / 32;  // MFMA steps over the dimensions
    constexpr int KL = D / 64;  // 16-byte loads per key row and lane
    constexpr int DT = D / 16;  // tiles of output dimensions
    __shared__ int prefix[kPrefixWords], waves[4];
    constexpr int AHEAD = 128;  // steps whose pages are looked up together
    __shared__ Half halves[2 * AHEAD];
    __shared__ int far[4];
    __shared__ float om[4][16], os[4][16], ol[4][16], oo[4][16][D + 4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const uint32_t wg = by_xcd((uint32_t)p.groups);
    Run run = first_run<256, BM>(c, b, a, p, prefix, waves, wg);
    Tile t;
    while (next_run<BM>(c, b, a, p, prefix, wg, run, t)) {
        const int r = t.r0 + col;
        const bool have = r < t.rows;
        const int qi = t.q0 + (have ? r : t.rows - 1) / a.group;
        const int qh = t.head * a.group + (have ? r : t.rows - 1) % a.group;
        const int reach_min = t.reach_min, reach_max = t.reach_max;
        const int mine = reach(t, a.causal, qi);

        // the query row, lane group g holding dimensions g D/4 .. (the order of the dimensions in the
        // contraction is free: it follows the keys' 16-byte loads)
        h8 q[KS];
        float qmul;
        {
            float x[D / 4];
            const uint16_t *at = (const uint16_t *)a.q + (int64_t)(t.row0 + qi) * a.q_stride +
                                 (int64_t)qh * D + g * (D / 4);
#pragma unroll
            for (int i = 0; i < D / 4; i += 8)
                widen_q(*(const u4 *)(at + i), a.f16, x + i);
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

        f4 o[DT];
#pragma unroll
        for (int i = 0; i < DT; ++i)
            o[i] = f4{0, 0, 0, 0};
        float m = kNone, ms = kNone, l = 0.0f;
        int apart = 0;       // the denominator is summed on its own

        // Key row `col` of tile u is token 16 (col / 4) + 4 u + col % 4: accumulator i of lane group g
        // in tile u is then token 16 g + 4 u + i.
        const int64_t page_bytes = (int64_t)c.page * D;
        const int kchunk = col >> 2, krow = (col & 3) + 16 * (kchunk & 1);

        // A lane's share of a step: 16-byte pieces of 4 key rows and of D / 16 value rows, and the
        // half that its scores and values belong to.  (Of a half without a page, page 0 is read
        // and nothing of it used.)
        u4 kr[4][KL], vr[DT];
        Half next;
        const uint32_t koff = krow * D + g * (D / 4), voff = col * c.page + 16 * (g & 1);
        auto load = [&](int i) {
            const Half hk = halves[2 * i + (kchunk >> 1)];
            next = halves[2 * i + (g >> 1)];
            const int64_t kpage = hk.page < 0 ? 0 : hk.page, vpage = next.page < 0 ? 0 : next.page;
            const uint8_t *kp = c.k + (kpage * c.heads + t.head) * page_bytes +
                                ((hk.tok & (c.page - 1)) * D + koff);
            const uint8_t *vp = c.v + (vpage * c.heads + t.head) * page_bytes +
                                ((next.tok & (c.page - 1)) + voff);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < KL; ++j)
                    kr[u][j] = *(const u4 *)(kp + u * 4 * D + j * 16);
#pragma unroll
            for (int i = 0; i < DT; ++i)
                vr[i] = *(const u4 *)(vp + i * 16 * c.page);
        };

        for (int first = run.s0; first < run.s1; first += AHEAD) {
            const int last = first + AHEAD < run.s1 ? first + AHEAD : run.s1;
            static_assert(2 * AHEAD == 256, "a half for each thread");
            const int mine_at = threadIdx.x;
            Half found = {-1, 0, 0.0f, kTiny};
            if (mine_at < 2 * (last - first)) {
                found = find_half(c, b, a, t, first * kBlock + 32 * mine_at, reach_max);
                find_scales(c, t, found);
            }
            const bool any_far = __any(is_far(found));
            if (lane == 0)
                far[wave] = any_far;
            __syncthreads();
            if (!apart && __builtin_amdgcn_readfirstlane(far[0] | far[1] | far[2] | far[3])) {
                // from the lowest z of the ordinary range to the lowest of all
                apart = 1;
                ms = m;
                m -= kApart;
#pragma unroll
                for (int i = 0; i < DT; ++i)
                    o[i] *= kApartPower;
            }
            halves[mine_at] = settled(found, apart);
            __syncthreads();
            int s = first + wave;
            if (s < last)
                load(s - first);
            for (; s < last; s += 4) {
                // scores
                f4 acc[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    acc[u] = f4{0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        const u4 w = kr[u][j / 2];
                        acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            to_half8<FMT>(w[j % 2 * 2], w[j % 2 * 2 + 1]), q[j], acc[u], 0, 0, 0);
                    }
                }
                const Half h = next;
                u4 v[DT];
#pragma unroll
                for (int i = 0; i < DT; ++i)
                    v[i] = vr[i];
                load((s + 4 < last ? s + 4 : s) - first);
                const Factor f = factor(h, qmul);
                const int tok = h.tok + 16 * (g & 1);
                float y[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    y[i] = fmaf(acc[i / 4][i % 4], f.mul, f.add);
                if (__any(h.page < 0 || h.tok + 32 > reach_min || flushed(h))) {
                    const bool none = h.page < 0;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        y[i] = none || tok + i >= mine ? -__builtin_inff() : y[i];
#pragma unroll
                    for (int i = 0; i < DT; ++i)
                        v[i] = flushed(h) ? u4{0, 0, 0, 0} : keep_live(v[i], tok, t.len);
                }
                float top = y[0];
#pragma unroll
                for (int i = 1; i < 16; ++i)
                    top = fmaxf(top, y[i]);
                if (__any(top > m + kSlack)) {
                    top = fmaxf(top, __shfl_xor(top, 16));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    // (each row on its own terms: what it gets does not depend on the rows beside it)
                    const float now = top > m + kSlack ? top : m, fall = exp2_fast(m - now);
                    m = now;
                    l *= apart ? 1.0f : fall;
#pragma unroll
                    for (int i = 0; i < DT; ++i)
                        o[i] *= fall;
                }
                float sum = 0.0f;
                h8 w[2];
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float e0 = exp2_fast(y[i] + (kLift - m));
                    const float e1 = exp2_fast(y[i + 1] + (kLift - m));
                    sum += e0 + e1;
                    const h2 e = pack(e0, e1);
                    w[i / 8][i % 8] = e[0];
                    w[i / 8][i % 8 + 1] = e[1];
                }
                if (__builtin_expect(!apart, 1)) {
                    l = fmaf(sum, f.back, l);
                } else {
                    // (the scores are y - add)
                    float peak = y[0];
#pragma unroll
                    for (int i = 1; i < 16; ++i)
                        peak = fmaxf(peak, y[i]);
                    peak -= f.add;
                    if (__any(peak > ms + kSlack)) {
                        peak = fmaxf(peak, __shfl_xor(peak, 16));
                        peak = fmaxf(peak, __shfl_xor(peak, 32));
                        const float now = peak > ms + kSlack ? peak : ms;
                        l *= exp2_fast(ms - now);
                        ms = now;
                    }
                    sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        sum += exp2_fast(y[i] - f.add + (kLift - ms));
                    l += sum;
                }
#pragma unroll
                for (int i = 0; i < DT; ++i) {
                    o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        to_half8<FMT>(v[i][0], v[i][1]), w[0], o[i], 0, 0, 0);
                    o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        to_half8<FMT>(v[i][2], v[i][3]), w[1], o[i], 0, 0, 0);
                }
            }
        }
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);

        // join the four waves
        if (g == 0) {
            om[wave][col] = m;
            os[wave][col] = apart ? ms : m;
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
            float mms = fmaxf(fmaxf(os[0][row], os[1][row]), fmaxf(os[2][row], os[3][row]));
            // a NaN row stays one: its sums are NaN whatever the weights
            float ll = 0.0f;
            f4 s = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float e = exp2_fast(om[w][row] - mm);
                ll += ol[w][row] * exp2_fast(os[w][row] - mms);
                s += *(const f4 *)&oo[w][row][d] * e;
            }
            if (run.slot >= 0) {
                float *out = partial<BM, D>(a, run.slot);
                if (d == 0)
                    *(f4 *)(out + BM * D + kRowWords * row) = f4{mm, mms, ll, 0.0f};
                *(f4 *)(out + 4 * i) = s;
            } else {
                const int64_t qrow = t.row0 + t.q0 + rr / a.group;
                const int head = t.head * a.group + rr % a.group;
                const float inv = ll > 0.0f ? 1.0f / ll : (ll == ll ? 0.0f : ll);
                const float p = half_power(mm, mms);
                s *= inv * p;
                store_out(a, qrow * a.out_stride + (int64_t)head * D + d, s[0] * p, s[1] * p,
                          s[2] * p, s[3] * p);
                if (a.lse && d == 0)
                    a.lse[qrow * a.q_heads + head] = lse_of(mms, ll);
            }
        }
        __syncthreads();  // om, os, ol and oo are read
    }
}

// ------------------------------------------------------------------ many rows
//
// 32 R rows per wave (v_mfma_f32_32x32x16_f16), NW waves, 32 H keys a step.  Each step's codes are
// read once per work-group, ahead of their use, and converted to fp16 on the way into LDS (each
// code once instead of once per wave).  At NW = 8 two waves share a SIMD and run a phase apart:
// one multiplies while the other forms weights, since a step's weights (an fp32 product, an
// exponential and half a conversion per score) take about as long as its products.  A call, the join
// included: 1024 queries over 4096 keys, 24 heads of 128, 93 us, 555 TFLOP/s; 4388 queries over 17552
// keys, 30 heads of 64, 740 to 760 us, 780 to 800 TFLOP/s.  (With the denominators on their own the
// kernels take 92 us instead of 81, and 1174 instead of 759.)  With both
// kinds of work in every wave, one step's products between the other's weights, the registers
// spilled; with products and weights one after the other it was 1141 us.
//
// The XOR of a key row's chunk number: 16 lanes that read one chunk of 16 key rows (in the order
// that the tile's rows have) must meet 16 different positions of the 256 bytes that LDS serves at
// once; a row is 256 bytes at head_dim 128, and half of that at 64, where the row's lowest bit counts.
template <int D> __device__ inline int key_swizzle(int tok)
{
    if constexpr (D == 128)
        return (tok & 3) | ((tok >> 4 & 1) << 2) | ((tok >> 2 & 1) << 3);
    else
        return (tok >> 1 & 3) | ((tok >> 4 & 1) << 2);
}

// The same for value rows of VC chunks, read by 16 lanes of consecutive rows.
template <int VC> __device__ inline int value_swizzle(int row) { return row / (16 / VC) & (VC - 1); }

constexpr int kFront = 4;  // products between an operand's read and its use

template <int FMT, int D, int NW, int R, int H>
__global__ __launch_bounds__(NW * 64, 2) void kv8_attend_wide_kernel(Kv8Cache c, Kv8Batch b,
                                                                     Kv8Attend a, Kv8Plan p)
{
    constexpr bool PAIRED = NW == 8;  // two waves of the work-group on each SIMD
    constexpr int BM = 32 * R * NW;
    constexpr int T = 64 * NW;        // threads
    constexpr int KS = D / 16;        // MFMA steps over the dimensions
    constexpr int DT = D / 32;        // tiles of output dimensions
    constexpr int BK = 32 * H;        // keys of a step
    constexpr int NK = BK * D / 16;   // 16-byte loads of a step's keys, and of its values
    constexpr int NL = 2 * NK > T ? 2 * NK / T : 1;  // loads per thread (of the first 2 NK threads)
    constexpr int VC = BK / 8;        // chunks of a value row in LDS
    constexpr int AHEAD = (PAIRED ? 1024 : 256) / H;  // steps whose pages are looked up together
    __shared__ h8 ks[2][BK][D / 8];
    __shared__ h8 vs[2][D][VC];
    __shared__ Half halves[H * AHEAD];
    __shared__ int far[NW];
    __shared__ float alone[R][T];     // ms of the rows, where it is not m (seldom: not worth registers)
    __shared__ int prefix[kPrefixWords], waves[NW];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int late = PAIRED ? wave / 4 : 0;
    const int col = lane & 31, g = lane >> 5;
    const uint32_t wg = by_xcd((uint32_t)p.groups);
    Run run = first_run<T, BM>(c, b, a, p, prefix, waves, wg);
    Tile t;
    while (next_run<BM>(c, b, a, p, prefix, wg, run, t)) {
        const int wave_row = t.r0 + wave * 32 * R;
        const bool busy = wave_row < t.rows;  // waves without rows only help to stage
        int qrow[R], qhead[R], mine[R];
        u4 raw_q[R][KS];
#pragma unroll
        for (int y = 0; y < R; ++y) {
            int r = wave_row + y * 32 + col;
            r = r < t.rows ? r : t.rows - 1;
            const int query = quotient(r, a.group);
            qrow[y] = t.q0 + query;
            qhead[y] = (t.head - query) * a.group + r;
            mine[y] = reach(t, a.causal, qrow[y]);
            const int64_t at = (int64_t)(t.row0 + qrow[y]) * a.q_stride + (int64_t)qhead[y] * D;
#pragma unroll
            for (int s = 0; s < KS; ++s)
                raw_q[y][s] = *(const u4 *)((const uint16_t *)a.q + at + s * 16 + g * 8);
        }
        h8 q[R][KS];
        float qmul[R];
        auto scale_q = [&]() {
#pragma unroll
            for (int y = 0; y < R; ++y) {
                float x[KS][8];
                float big = 0.0f;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    widen_q(raw_q[y][s], a.f16, x[s]);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        big = fmaxf(big, fabsf(x[s][j]));
                }
                big = fmaxf(big, __shfl_xor(big, 32));
                float inv;
                const float up = row_scale(big, inv);
                qmul[y] = inv * (a.scale * 1.4426950408889634f);
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        q[y][s][j] = (_Float16)(x[s][j] * up);
            }
        };

        f16v o[R][DT];
        float m[R], l[R];
        int apart = 0;       // the denominator is summed on its own
#pragma unroll
        for (int y = 0; y < R; ++y) {
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    o[y][i][j] = 0.0f;
            m[y] = kNone;
            l[y] = 0.0f;
        }

        // A thread's share of a step: loads of 16 codes, of a key row or of a value row; all of
        // a wave's in one half and of one kind, so that pages and addresses are scalar.
        const uint32_t head_off = (uint32_t)t.head * (uint32_t)(c.page * D);
        const int64_t page_bytes = (int64_t)c.heads * c.page * D;
        const int krow = tid * 16 / D, kcol = tid % (D / 16), vrow = tid / 2, vcol = tid & 1;
        u4 raw[NL];
        int first = 0, last = 0;  // the steps that `halves` holds
        // the halves of this step and the next WIN - 1
        constexpr int WIN = 3;
        Half win[WIN][H];
        auto look = [&](int s, Half (&h)[H]) {
#pragma unroll
            for (int x = 0; x < H; ++x) {
                const Half n = halves[H * (s < last ? s - first : 0) + x];
                h[x].page = s < last ? __builtin_amdgcn_readfirstlane(n.page) : -1;
                h[x].tok = __builtin_amdgcn_readfirstlane(n.tok);
                h[x].kscale = first_lane(n.kscale);
                h[x].add = first_lane(n.add);
            }
        };
        // whether load i is of keys, and of which half
        auto of_keys = [&](int i) { return T <= NK ? i * T < NK : wave * 64 < NK; };
        const bool loads = wave * 64 < 2 * NK;
        auto half_of = [&](int i) {
            const int id = wave * 64 + i * T;
            return of_keys(i) ? id * 16 / D / 32 : (id - NK) / (2 * D);
        };
        // keys of a step (its halves hk) and values of the step before it (hv)
        auto load = [&](const Half (&hk)[H], const Half (&hv)[H]) {
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int x = half_of(i);
                raw[i] = u4{0, 0, 0, 0};
                if (!loads)
                    continue;
                if (of_keys(i)) {
                    const Half h = x ? hk[H - 1] : hk[0];
                    if (h.page >= 0)
                        raw[i] = *(const u4 *)(c.k + (h.page * page_bytes + head_off +
                                                      ((h.tok & (c.page - 1)) +
                                                       (i * T * 16 / D & 31)) * D) +
                                               (uint32_t)((krow & 31) * D + kcol * 16));
                } else {
                    const Half h = x ? hv[H - 1] : hv[0];
                    if (h.page >= 0)
                        raw[i] = *(const u4 *)(c.v + (h.page * page_bytes + head_off +
                                                      (h.tok & (c.page - 1))) +
                                               (uint32_t)((vrow + (i * T - NK - x * 2 * D) / 2) *
                                                              c.page + vcol * 16));
                }
            }
        };
        // what the value rows read hold behind the live tokens becomes zeros
        auto mend = [&](const Half (&hv)[H]) {
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                if (of_keys(i))
                    continue;
                const Half h = half_of(i) ? hv[H - 1] : hv[0];
                if (h.tok + 32 > t.len || flushed(h))
                    raw[i] = flushed(h) ? u4{0, 0, 0, 0}
                                        : keep_live(raw[i], h.tok + 16 * vcol, t.len);
            }
        };
        // 8 of the read codes (part 0 .. 2 NL - 1) to fp16 in LDS: keys of step e, values of e - 1
        auto stage = [&](int e, int part) {
            if (!loads)
                return;
            const int i = part / 2, z = part & 1, x = half_of(i);
            const h8 v = to_half8<FMT>(raw[i][2 * z], raw[i][2 * z + 1]);
            if (of_keys(i)) {
                const int rr = krow + i * T * 16 / D;
                ks[(e - first) & 1][rr][(kcol * 2 + z) ^ key_swizzle<D>(rr)] = v;
            } else {
                const int dd = vrow + (i * T - NK - x * 2 * D) / 2, vc = x * 4 + vcol * 2 + z;
                vs[(e - 1 - first) & 1][dd][vc ^ value_swizzle<VC>(dd)] = v;
            }
        };

        // key row `col` of a half is token 16 (col >> 2 & 1) + (col & 3) + 4 (col >> 3):
        // accumulator i of lane group g is then token 16 g + i
        const int ktok = 16 * (col >> 2 & 1) + (col & 3) + 4 * (col >> 3);
        const int ksw = key_swizzle<D>(ktok);
        f16v acc[R][H];
        h2 w[R][8 * H];

        // The matrix products of a phase: the previous step's values, then this step's scores.  The
        // operands are read from LDS kFront products ahead (a read takes several products' time).
        constexpr int NV = 2 * H * DT, NS = H * KS;
        auto value_operand = [&](int s, int i) {
            // weights j of lane group g: tokens 32 (j / 2) + 16 g + 8 (j % 2) ..
            const int j = i / DT, chunk = 4 * (j / 2) + 2 * g + j % 2;
            return vs[(s - first) & 1][i % DT * 32 + col][chunk ^ value_swizzle<VC>(col)];
        };
        auto key_operand = [&](int s, int i) {
            return ks[(s - first) & 1][i / KS * 32 + ktok][(2 * (i % KS) + g) ^ ksw];
        };
        auto add_value = [&](const h8 &v, int i) {
            const int j = i / DT;
#pragma unroll
            for (int y = 0; y < R; ++y) {
                const h8 wj = {w[y][4 * j][0],     w[y][4 * j][1],     w[y][4 * j + 1][0],
                               w[y][4 * j + 1][1], w[y][4 * j + 2][0], w[y][4 * j + 2][1],
                               w[y][4 * j + 3][0], w[y][4 * j + 3][1]};
                o[y][i % DT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, wj, o[y][i % DT], 0, 0, 0);
            }
        };
        auto score = [&](const h8 &k, int i) {
            const int x = i / KS;
#pragma unroll
            for (int y = 0; y < R; ++y) {
                if (i % KS == 0)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        acc[y][x][j] = 0.0f;
                acc[y][x] =
                    __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[y][i % KS], acc[y][x], 0, 0, 0);
            }
        };
        // Between them goes the staging of what the next step needs: the matrix unit works on
        // while the codes are converted.
        auto multiply = [&](int s, auto scores) {
            constexpr bool MORE = decltype(scores)::value;
            constexpr int A = NV, N = A + (MORE ? NS : 0);
            __builtin_amdgcn_sched_barrier(0);
            h8 x[N];
#pragma unroll
            for (int i = 0; i < kFront; ++i)
                x[i] = i < A ? value_operand(s - 1, i) : key_operand(s, i - A);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (i + kFront < N) {
                    const int n = i + kFront;
                    x[n] = n < A ? value_operand(s - 1, n) : key_operand(s, n - A);
                }
                if (i < A)
                    add_value(x[i], i);
                else
                    score(x[i], i - A);
                if (MORE && i >= N / 2 && (i - N / 2) % (N / 4 / NL) == 0)
                    stage(s + 1, (i - N / 2) / (N / 4 / NL));
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        // The weights are formed with the maximum as it stands.  Where a lane's sum of them
        // exceeds kLimit (infinities and NaN too) the row's maximum is moved up to the true one,
        // its sums are rescaled and its weights are formed again: rare after the first steps, and one
        // comparison instead of a maximum over the scores of every step.  (Each row on its
        // own terms: what it gets does not depend on the rows beside it.)
        // (The denominator on its own, from the masked scores: in the same way.)
        auto add_alone = [&](int y, const Factor (&f)[H]) {
            float ms = alone[y][tid];
            auto weigh = [&]() {
                float sum = 0.0f;
#pragma unroll
                for (int x = 0; x < H; ++x)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        sum += exp2_fast(fmaf(acc[y][x][j], f[x].mul, kLift - ms));
                return sum;
            };
            float sum = weigh();
            const int over = !(sum <= kLimit);
            if (__any(over)) {
                float top = kNone;
#pragma unroll
                for (int x = 0; x < H; ++x) {
                    float z = acc[y][x][0];
#pragma unroll
                    for (int j = 1; j < 16; ++j)
                        z = fmaxf(z, acc[y][x][j]);
                    top = fmaxf(top, z * f[x].mul);
                }
                top = fmaxf(top, __shfl_xor(top, 32));
                const bool move = over | __shfl_xor(over, 32);
                const float now = move ? fmaxf(ms, top) : ms;
                l[y] *= exp2_fast(ms - now);
                ms = alone[y][tid] = now;
                sum = weigh();
            }
            l[y] += sum;
        };
        auto weights = [&](const Half (&h)[H]) {
#pragma unroll
            for (int x = 0; x < H; ++x)
                if (h[x].page < 0 || h[x].tok + 32 > t.reach_min) {
#pragma unroll
                    for (int y = 0; y < R; ++y) {
                        const int seen = h[x].page < 0 ? 0 : mine[y] - h[x].tok - 16 * g;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            acc[y][x][j] = j < seen ? acc[y][x][j] : -__builtin_inff();
                    }
                }
            Factor f[R][H];
            float sum[R][H];
            auto weigh = [&](int y) {
#pragma unroll
                for (int x = 0; x < H; ++x) {
                    const float base = f[y][x].add + (kLift - m[y]);
                    float part = 0.0f;
                    sum[y][x] = 0.0f;
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float e0 = exp2_fast(fmaf(acc[y][x][j], f[y][x].mul, base));
                        const float e1 = exp2_fast(fmaf(acc[y][x][j + 1], f[y][x].mul, base));
                        sum[y][x] += e0;
                        part += e1;
                        w[y][8 * x + j / 2] = pack(e0, e1);
                    }
                    sum[y][x] += part;
                }
            };
            bool any = false;
#pragma unroll
            for (int y = 0; y < R; ++y) {
#pragma unroll
                for (int x = 0; x < H; ++x)
                    f[y][x] = factor(h[x], qmul[y]);
                weigh(y);
                any |= !(sum[y][0] + sum[y][H - 1] <= kLimit);
            }
            if (__any(any)) {
#pragma unroll
                for (int y = 0; y < R; ++y) {
                    const int over = !(sum[y][0] + sum[y][H - 1] <= kLimit);
                    float top = kNone;
#pragma unroll
                    for (int x = 0; x < H; ++x) {
                        float z = acc[y][x][0];
#pragma unroll
                        for (int j = 1; j < 16; ++j)
                            z = fmaxf(z, acc[y][x][j]);
                        top = fmaxf(top, fmaf(z, f[y][x].mul, f[y][x].add));
                    }
                    top = fmaxf(top, __shfl_xor(top, 32));
                    const bool move = over | __shfl_xor(over, 32);
                    const float now = move ? fmaxf(m[y], top) : m[y], fall = exp2_fast(m[y] - now);
                    m[y] = now;
                    l[y] *= apart ? 1.0f : fall;
#pragma unroll
                    for (int i = 0; i < DT; ++i)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            o[y][i][j] *= fall;
                    weigh(y);
                }
            }
            float before[R];
#pragma unroll
            for (int y = 0; y < R; ++y) {
                before[y] = l[y];
#pragma unroll
                for (int x = 0; x < H; ++x)
                    l[y] = fmaf(sum[y][x], f[y][x].back, l[y]);
            }
            // (behind the ordinary sum and instead of it: a branch before it costs up to 2% of the kernel)
            if (__builtin_expect(apart, 0)) {
#pragma unroll
                for (int y = 0; y < R; ++y) {
                    l[y] = before[y];
                    add_alone(y, f[y]);
                }
            }
        };

        // Two phases a step, a barrier after each: the matrix products (the previous step's values,
        // this step's scores) with the staging of the next step's keys and this step's values between
        // them, then the weights.  Of the two waves on a SIMD the later one runs a phase
        // behind, so that one multiplies while the other computes weights.  The keys of step s + 1
        // and the values of step s are written in the phases of scores s (2 s and, a phase
        // behind, 2 s + 1); what their buffers held, keys s - 1 and values s - 2, was last read in the
        // late waves' phase 2 s - 1, and they are first read in the early waves' phase 2 s + 2.
        Half none[H];
#pragma unroll
        for (int x = 0; x < H; ++x)
            none[x] = Half{-1, 0, 0.0f, kTiny};
        const int begin = run.s0 * (2 / H), end = run.s1 * (2 / H);
        auto look_up = [&]() {
            constexpr int EACH = H * AHEAD / T;  // halves of a thread
            last = first + AHEAD < end ? first + AHEAD : end;
            Half found[EACH];
            bool any_far = false;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                found[i] = Half{-1, 0, 0.0f, kTiny};
                if (tid + i * T < H * (last - first)) {
                    found[i] = find_half(c, b, a, t, first * BK + 32 * (tid + i * T), t.reach_max);
                    find_scales(c, t, found[i]);
                }
                any_far |= is_far(found[i]);
            }
            any_far = __any(any_far);
            if (lane == 0)
                far[wave] = any_far;
            __syncthreads();
            int all_far = 0;
#pragma unroll
            for (int i = 0; i < NW; ++i)
                all_far |= far[i];
            if (!apart && __builtin_amdgcn_readfirstlane(all_far)) {
                // from the lowest z of the ordinary range to the lowest of all
                apart = 1;
#pragma unroll
                for (int y = 0; y < R; ++y) {
                    alone[y][tid] = m[y];
                    m[y] -= kApart;
#pragma unroll
                    for (int i = 0; i < DT; ++i)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            o[y][i][j] *= kApartPower;
                }
            }
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                halves[tid + i * T] = settled(found[i], apart);
            __syncthreads();
        };
        first = begin;
        look_up();
        scale_q();
        while (first < end) {
#pragma unroll
            for (int i = 0; i < WIN; ++i)
                look(first + i, win[i]);
            load(win[0], none);
            // the first step's product with "the previous step's values" adds zeros
#pragma unroll
            for (int i = tid; i < D * VC; i += T)
                (&vs[1][0][0])[i] = h8{};
#pragma unroll
            for (int y = 0; y < R; ++y)
#pragma unroll
                for (int j = 0; j < 8 * H; ++j)
                    w[y][j] = h2{};
#pragma unroll
            for (int i = 0; i < 2 * NL; ++i)
                if (of_keys(i / 2))
                    stage(first, i);
            load(win[1], win[0]);
            __syncthreads();
            if (late)
                __syncthreads();
            for (int s = first; s < last; ++s) {
                mend(win[0]);
                if (busy) {
                    multiply(s, std::true_type());
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * NL; ++i)
                        stage(s + 1, i);
                }
                load(win[2], win[1]);
                __syncthreads();
                if (busy)
                    weights(win[0]);
#pragma unroll
                for (int i = 0; i + 1 < WIN; ++i)
#pragma unroll
                    for (int x = 0; x < H; ++x)
                        win[i][x] = win[i + 1][x];
                look(s + WIN, win[WIN - 1]);
                __syncthreads();
            }
            if (busy)
                multiply(last, std::false_type());
            if (PAIRED && !late)
                __syncthreads();
            first = last;
            if (first < end)
                look_up();
        }

#pragma unroll
        for (int y = 0; y < R; ++y) {
            const float all = l[y] + __shfl_xor(l[y], 32);
            if (wave_row + y * 32 + col >= t.rows)
                continue;
            const int64_t row = t.row0 + qrow[y];
            const float ms = apart ? alone[y][tid] : m[y];
            if (run.slot >= 0) {
                float *out = partial<BM, D>(a, run.slot) + (wave * R + y) * 32 * D;
#pragma unroll
                for (int i = 0; i < DT * 4; ++i)
                    *(f4 *)(out + (i * 64 + lane) * 4) =
                        f4{o[y][i / 4][i % 4 * 4], o[y][i / 4][i % 4 * 4 + 1],
                           o[y][i / 4][i % 4 * 4 + 2], o[y][i / 4][i % 4 * 4 + 3]};
                if (g == 0)
                    *(f4 *)(partial<BM, D>(a, run.slot) + BM * D +
                            kRowWords * ((wave * R + y) * 32 + col)) = f4{m[y], ms, all, 0.0f};
            } else {
                const float p = half_power(m[y], ms);
                const float inv = (all > 0.0f ? 1.0f / all : (all == all ? 0.0f : all)) * p;
                const int64_t at = row * a.out_stride + (int64_t)qhead[y] * D + g * 4;
#pragma unroll
                for (int i = 0; i < DT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        store_out(a, at + i * 32 + j * 8, o[y][i][4 * j] * inv * p,
                                  o[y][i][4 * j + 1] * inv * p, o[y][i][4 * j + 2] * inv * p,
                                  o[y][i][4 * j + 3] * inv * p);
                if (a.lse && g == 0)
                    a.lse[row * a.q_heads + qhead[y]] = lse_of(ms, all);
            }
        }
    }
}

// Joins the runs of the tile that work-group blockIdx.x began and did not finish: kPieces 16-byte
// pieces per thread, read together.
constexpr int kPieces = 2;

template <int BM, int D>
__global__ __launch_bounds__(256) void kv8_join_kernel(Kv8Cache c, Kv8Batch b, Kv8Attend a,
                                                       Kv8Plan p)
{
    constexpr int ALL = BM * D / 4, N = ALL < kPieces * 256 ? ALL / 256 : kPieces;
    const uint32_t w = blockIdx.x;
    const Cut cut = ((const Cut *)a.ws)[w];
    if (cut.more == 0)
        return;
    const int i0 = blockIdx.y * (N * 256) + threadIdx.x;  // the first piece
    int row[N], d[N];
    f4 ml[N];  // m, ms, l
    f4 o[N];
    // the first part lies in the beginning work-group's second slot, the others in first ones
    const float *x = partial<BM, D>(a, 2 * w + 1);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = i0 + n * 256;
        if constexpr (BM == 16) {
            row[n] = i / (D / 4);
            d[n] = i % (D / 4) * 4;
        } else {
            row[n] = i / (8 * D) * 32 + i % 32;
            d[n] = i % (8 * D) / 64 * 8 + i % 64 / 32 * 4;
        }
        ml[n] = *(const f4 *)(x + BM * D + kRowWords * row[n]);
        o[n] = *(const f4 *)(x + 4 * i);
    }
    for (int k = 1; k <= cut.more; ++k) {
        x = partial<BM, D>(a, 2 * (w + k));
        f4 more[N];
        f4 v[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            more[n] = *(const f4 *)(x + BM * D + kRowWords * row[n]);
            v[n] = *(const f4 *)(x + 4 * (i0 + n * 256));
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float now = fmaxf(ml[n][0], more[n][0]), nows = fmaxf(ml[n][1], more[n][1]);
            o[n] = o[n] * exp2_fast(ml[n][0] - now) + v[n] * exp2_fast(more[n][0] - now);
            const float l = ml[n][2] * exp2_fast(ml[n][1] - nows) +
                            more[n][2] * exp2_fast(more[n][1] - nows);
            ml[n] = f4{now, nows, l, 0.0f};
        }
    }
    Tile t;
    if (!find_tile<BM>(c, b, a, p, cut.item, cut.head, t))
        return;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int r = t.r0 + row[n];
        if (r >= t.rows)
            continue;
        const int query = quotient(r, a.group);
        const int64_t qrow = t.row0 + t.q0 + query;
        const int qhead = (t.head - query) * a.group + r;
        const float l = ml[n][2], p = half_power(ml[n][0], ml[n][1]);
        o[n] *= (l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l)) * p;
        store_out(a, qrow * a.out_stride + (int64_t)qhead * D + d[n], o[n][0] * p, o[n][1] * p,
                  o[n][2] * p, o[n][3] * p);
        if (a.lse && d[n] == 0)
            a.lse[qrow * a.q_heads + qhead] = lse_of(ml[n][1], l);
    }
}

// Rows of a query block up to which the narrow kernel is taken, although it reads the keys again for
// every 16 rows: over 16 sequences of 8192 tokens and 8 heads, with 32 rows 70 us against 100
// at head_dim 128 and 33 against 87 at 64; with 48 rows 130 against 111 and 68 against 88; with 64
// rows 55 against 88 at 64.
inline int64_t narrow_rows(int dim) { return dim == 64 ? 64 : 32; }

// The launch's shapes: rows per tile, and work-groups that are resident at once.
struct Shape {
    int rows, slots;
};

// Taller tiles read the keys less often and need fewer LDS reads a product; lower ones waste less on
// few rows, and two or more of their work-groups share a CU.  Over 4 sequences of 8192 tokens and
// 24 heads, tiles of 128 / 256 / 512 rows take (us), at head_dim 64 with 64 rows 81 / 86 / 130, with
// 128 95 / 89 / 136, with 256 117 / 106 / 145, with 384 151 / 167 / 150, with 1000 333 / 325 / 262;
// at head_dim 128 with 128 rows 107 / 119, with 192 159 / 135, with 1000 529 / 441.
Shape shape_of(bool wide, int dim, int64_t rows)
{
    if (!wide)
        return {16, 512};
    if (rows <= 128)
        return dim == 64 ? Shape{128, 1024} : Shape{128, 512};
    return dim == 64 && rows > 256 ? Shape{512, 256} : Shape{256, 256};
}

}  // namespace

Kv8Plan kv8_plan(const Kv8Cache &c, const Kv8Batch &b, int q_heads, int64_t max_kv, bool listed,
                 int64_t q_block, int count)
{
    Kv8Plan p;
    const int64_t group = q_heads / c.heads;
    if (!listed || q_block > b.max_rows)
        q_block = b.max_rows;
    const int64_t rows = q_block * group;
    p.wide = rows > narrow_rows(c.dim);
    const Shape sh = shape_of(p.wide, c.dim, rows);
    const double units = (double)((b.max_rows + q_block - 1) / q_block);
    const double tiles = (double)((rows + sh.rows - 1) / sh.rows);
    p.whole = units * tiles * c.heads * b.batch;
    p.units = p.tiles = p.items = 1;
    p.joined = 0;
    p.groups = 1;
    p.ws_bytes = 0;
    p.rows = sh.rows;
    if (p.whole >= kKv8MaxGroups)
        return p;  // refused by the caller
    p.units = (int)units;
    p.tiles = (int)tiles;
    p.items = (int)(units * tiles) * b.batch;
    p.groups = (int64_t)p.items * c.heads;
    const int64_t keys = listed ? (int64_t)count * c.page : max_kv;  // as find_tile has it
    const int64_t steps = (keys + kBlock - 1) / kBlock;
    // Runs of equal length instead of whole tiles: only where a run is long enough to be worth
    // joining (a narrow one has 4 waves, each of which should have some steps).  Half and twice
    // as many: 18 and 25 us instead of 20 for 4 single queries x 4096 tokens x 8 heads, 55 and 37
    // instead of 36 for 4 x 256 queries x 1024 tokens.
    const int64_t least = p.wide ? 4 : 16;
    if (p.items <= kMaxItems && steps > least && p.whole * steps < 2147483648.0) {
        int64_t runs = p.groups * steps / least;
        runs = runs < sh.slots ? runs : sh.slots;
        p.joined = 1;
        p.groups = runs;
        p.ws_bytes = ((int64_t)kCutWords + 2 * runs * sh.rows * (c.dim + kRowWords)) * sizeof(float);
    }
    return p;
}

namespace {

template <int F, int D>
void attend_as(const Kv8Cache &c, const Kv8Batch &b, const Kv8Attend &a, const Kv8Plan &p,
               hipStream_t st)
{
    const dim3 grid((unsigned)p.groups);
    if (!p.wide)
        kv8_attend_narrow_kernel<F, D><<<grid, 256, 0, st>>>(c, b, a, p);
    else if (p.rows == 128 && D == 64)
        kv8_attend_wide_kernel<F, 64, 2, 2, 1><<<grid, 128, 0, st>>>(c, b, a, p);
    else if (p.rows == 128)
        kv8_attend_wide_kernel<F, 128, 4, 1, 2><<<grid, 256, 0, st>>>(c, b, a, p);
    else if (p.rows == 256)
        kv8_attend_wide_kernel<F, D, 8, 1, 2><<<grid, 512, 0, st>>>(c, b, a, p);
    else
        kv8_attend_wide_kernel<F, 64, 8, 2, 1><<<grid, 512, 0, st>>>(c, b, a, p);
}

template <int D>
void join_as(const Kv8Cache &c, const Kv8Batch &b, const Kv8Attend &a, const Kv8Plan &p,
             hipStream_t st)
{
    const int pieces = p.rows * D / 1024;  // per thread, over all
    const dim3 grid((unsigned)p.groups, (unsigned)(pieces < kPieces ? 1 : pieces / kPieces));
    if (p.rows == 512)
        kv8_join_kernel<512, D><<<grid, 256, 0, st>>>(c, b, a, p);
    else if (p.rows == 16)
        kv8_join_kernel<16, D><<<grid, 256, 0, st>>>(c, b, a, p);
    else if (p.rows == 128)
        kv8_join_kernel<128, D><<<grid, 256, 0, st>>>(c, b, a, p);
    else
        kv8_join_kernel<256, D><<<grid, 256, 0, st>>>(c, b, a, p);
}

}  // namespace

hipError_t launch_kv8_attend(const Kv8Cache &c, const Kv8Batch &b, const Kv8Attend &a,
                             const Kv8Plan &p, hipStream_t st)
{
    if (c.fmt == CFZ_KV8_INT8)
        c.dim == 64 ? attend_as<CFZ_KV8_INT8, 64>(c, b, a, p, st)
                    : attend_as<CFZ_KV8_INT8, 128>(c, b, a, p, st);
    else
        c.dim == 64 ? attend_as<CFZ_KV8_E4M3, 64>(c, b, a, p, st)
                    : attend_as<CFZ_KV8_E4M3, 128>(c, b, a, p, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.joined || p.groups == 1)
        return e;
    c.dim == 64 ? join_as<64>(c, b, a, p, st) : join_as<128>(c, b, a, p, st);
    return hipGetLastError();
}

}  // namespace cfz
