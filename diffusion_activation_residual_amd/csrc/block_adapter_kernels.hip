// block_adapter_kernels.hip -- low-rank adapters of many requests beside a shared projection.
//
//   out = y + scale (x A^T) B^T   for each sequence's own A, B and scale
//
// Two launches: h = x A^T into the workspace, then out = y + scale h B^T.  Both are bound by the rows
// that they read and write (x once, y and out once); the products are small beside them.  Row
// tiles never straddle sequences: sequence b's tiles are numbered from offsets[b] / R + b on, which
// leaves room for a short tile at its end, so that a tile finds its sequence by a search and the
// host needs no list.
#include "block_internal.h"

namespace cfz {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <class T> struct Mfma;
template <> struct Mfma<uint16_t> {
    typedef __bf16 x8 __attribute__((ext_vector_type(8)));
    static __device__ inline f32x4 mul(uint4 a, uint4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(x8, a),
                                                       __builtin_bit_cast(x8, b), c, 0, 0, 0);
    }
    static __device__ inline uint16_t bits(float f) { return BlockType<uint16_t>::put(f); }
    static __device__ inline float value(uint16_t u) { return BlockType<uint16_t>::get(u); }
};
template <> struct Mfma<_Float16> {
    typedef _Float16 x8 __attribute__((ext_vector_type(8)));
    static __device__ inline f32x4 mul(uint4 a, uint4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(x8, a),
                                                      __builtin_bit_cast(x8, b), c, 0, 0, 0);
    }
    static __device__ inline uint16_t bits(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
    static __device__ inline float value(uint16_t u) { return (float)__builtin_bit_cast(_Float16, u); }
};

// The rows of a tile: row0 .. row0 + n - 1 of the call, n <= R.  False: the tile holds nothing.
template <int R>
__device__ inline bool find_tile(const AdapterArgs &a, int tile, int &seq, int64_t &row0, int &n)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = a.rows.tokens;
    auto at = [&](int b) {
        const int64_t o = a.rows.off[b];
        return o < 0 ? 0 : (o > t ? t : o);
    };
    int lo = 0, left = a.rows.batch;  // the last sequence whose first tile is at or before this one
    while (left > 1) {
        const int step = (left + 63) / 64;
        const int b = lo + lane * step;
        const bool before = lane * step < left && at(b) / R + b <= tile;
        const uint64_t votes = __ballot(before);
        const int k = votes ? 63 - __clzll(votes) : 0;
        left = left - k * step < step ? left - k * step : step;
        lo += k * step;
    }
    seq = lo;
    const int64_t first = at(lo);
    int64_t end = at(lo + 1);
    end = end - first > a.max_rows ? first + a.max_rows : end;
    const int64_t mine = tile - (first / R + lo);
    row0 = first + mine * R;
    if (mine < 0 || row0 >= end)
        return false;
    n = (int)(end - row0 < R ? end - row0 : R);
    return true;
}

__device__ inline uint4 load16(const void *p, bool yes)
{
    return yes ? *(const uint4 *)p : make_uint4(0, 0, 0, 0);
}

// h of TM x 16 tokens for NB x 16 adapter rows, over one of a.splits runs of the columns.  The four
// waves take every fourth chunk of 64 columns, and their sums are added in LDS.  A lane holds 16
// neighbouring columns of a row, 32 bytes: the two matrix instructions of a chunk take 8 each, the
// same ones of either operand, so that four lanes read 128 bytes of a row.
template <class T, int NB, int TM>
__global__ __launch_bounds__(256) void adapter_down_kernel(AdapterArgs a)
{
    __shared__ f32x4 part[3][NB * TM][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tile = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
    int seq, n;
    int64_t row0;
    if (!find_tile<16 * TM>(a, tile, seq, row0, n))
        return;
    const int id = a.ids[seq];
    if (id < 0 || id >= a.adapters)
        return;
    const int m = lane & 15, q = lane >> 4;
    const T *x[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        // (rows past the tile's end repeat the last one: their sums are not kept)
        const int r = t * 16 + m < n ? t * 16 + m : n - 1;
        x[t] = (const T *)a.x + (row0 + r) * a.xs + q * 16;
    }
    const T *w[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int r = j * 16 + m < a.down ? j * 16 + m : a.down - 1;
        w[j] = (const T *)a.a + ((int64_t)id * a.down + r) * a.cols_in + q * 16;
    }
    f32x4 acc[TM][NB];
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int chunks = (a.cols_in + 63) / 64;
    const int c0 = (int)((int64_t)chunks * split / a.splits);
    const int c1 = (int)((int64_t)chunks * (split + 1) / a.splits);
    for (int c = c0 + wave; c < c1; c += 4) {
        const int k = c * 64;
        uint4 xv[TM][2], wv[NB][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool in = k + q * 16 + i * 8 < a.cols_in;
#pragma unroll
            for (int t = 0; t < TM; ++t)
                xv[t][i] = load16(x[t] + k + i * 8, in);
#pragma unroll
            for (int j = 0; j < NB; ++j)
                wv[j][i] = load16(w[j] + k + i * 8, in);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int t = 0; t < TM; ++t)
                    acc[t][j] = Mfma<T>::mul(wv[j][i], xv[t][i], acc[t][j]);
    }
    if (wave > 0) {
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                part[wave - 1][t * NB + j][lane] = acc[t][j];
    }
    __syncthreads();
    if (wave > 0)
        return;
    float *h = a.h + (int64_t)split * a.rows.tokens * a.down;
#pragma unroll
    for (int t = 0; t < TM; ++t) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            f32x4 s = acc[t][j];
#pragma unroll
            for (int i = 0; i < 3; ++i)
                s += part[i][t * NB + j][lane];
            // lane: token m, adapter rows 4 q .. 4 q + 3 of the block
            const int r = j * 16 + q * 4;
            if (t * 16 + m < n && r < a.down)
                *(f32x4 *)(h + (row0 + t * 16 + m) * a.down + r) = s;
        }
    }
}

// 64 columns a wave, four waves side by side, the tile's tokens 16 at a time.  Columns are the matrix
// instructions' rows, dealt out so that a lane ends up with 16 neighbouring ones of a token:
// y is read and out written in vectors of 16 bytes.  B stays in registers over the tile.
//
// h enters the second product as the sum of two 16-bit numbers, which leaves 2^-16 of it (bf16) or
// 2^-21 of its row's largest (fp16, after a power of two that brings the row into range), where
// the rounding of a result in these types leaves 2^-8 and 2^-11.
constexpr int kUpRows = 64;

template <class T, class Y, int KS>
__global__ __launch_bounds__(256) void adapter_up_kernel(AdapterArgs a)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tile = blockIdx.x / a.col_tiles;
    const int group = (int)(blockIdx.x % a.col_tiles) * 4 + wave;
    int seq, n;
    int64_t row0;
    if (!find_tile<kUpRows>(a, tile, seq, row0, n))
        return;
    const int id = a.ids[seq];
    const bool some = id >= 0 && id < a.adapters;
    if (group >= a.groups || (!some && a.y == a.out))
        return;
    int slice = 0;
    while (slice + 1 < a.slices && group >= a.first_group[slice + 1])
        ++slice;
    const int m = lane & 15, q = lane >> 4;
    const int col0 = a.first_col[slice] + (group - a.first_group[slice]) * 64;
    const int left = a.first_col[slice + 1] - col0;  // columns of the slice from here on
    const bool mine = q * 16 < left;
    uint4 w[4][KS];
    if (some) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = (m >> 2) * 16 + j * 4 + (m & 3);
            const T *b = (const T *)a.b + ((int64_t)id * a.cols_out + col0 + c) * a.rank + q * 8;
#pragma unroll
            for (int s = 0; s < KS; ++s)
                w[j][s] = load16(b + s * 32, c < left && s * 32 + q * 8 < a.rank);
        }
    }
    const float scale = some && a.scale ? a.scale[id] : 1.0f;
    const float *h = a.h + slice * a.rank + q * 8;
    for (int t = 0; t < n; t += 16) {
        const bool in = t + m < n;
        const int64_t row = row0 + (in ? t + m : n - 1);
        const Y *y = (const Y *)a.y + row * a.ys + col0 + q * 16;
        float v[16];
        if (mine)
            load_n(y, v);
        f32x4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        float back = 1.0f;
        if (some) {
            float u[KS][8];
            float top = 0.0f;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    u[s][i] = 0.0f;
                if (s * 32 + q * 8 < a.rank) {
                    for (int p = 0; p < a.splits; ++p) {
                        float f[8];
                        load_n(h + (p * a.rows.tokens + row) * a.down + s * 32, f);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            u[s][i] += f[i];
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        u[s][i] *= scale;
                        top = fmaxf(top, fabsf(u[s][i]));
                    }
                }
            }
            if (sizeof(_Float16) == sizeof(T) && __is_same(T, _Float16)) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                // a power of two that brings the row's largest into 1 .. 2 (0 and what is not finite: 1)
                const int e = (int)(__float_as_uint(top) >> 23) - 127;
                const bool ok = e > -120 && e < 120;
                const float f = __uint_as_float((uint32_t)(127 - (ok ? e : 0)) << 23);
                back = __uint_as_float((uint32_t)(127 + (ok ? e : 0)) << 23);
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        u[s][i] *= f;
            }
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint16_t a0[2], a1[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float f = u[s][2 * i + k];
                        a0[k] = Mfma<T>::bits(f);
                        const float rest = f - Mfma<T>::value(a0[k]);
                        a1[k] = Mfma<T>::bits(rest == rest ? rest : 0.0f);
                    }
                    hi[i] = (uint32_t)a0[0] | (uint32_t)a0[1] << 16;
                    lo[i] = (uint32_t)a1[0] | (uint32_t)a1[1] << 16;
                }
                const uint4 hv = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                const uint4 lv = make_uint4(lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[j] = Mfma<T>::mul(w[j][s], lv, acc[j]);
                    acc[j] = Mfma<T>::mul(w[j][s], hv, acc[j]);
                }
            }
        }
        if (mine && in) {
            // lane: token m, columns 16 q + 4 j + i
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[4 * j + i] = fmaf(acc[j][i], back, v[4 * j + i]);
            store_n((Y *)a.out + row * a.os + col0 + q * 16, v);
        }
    }
}

template <class T, int TM> hipError_t down_as(const AdapterArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)(adapter_tiles(a, 16 * TM) * a.splits));
    const int nb = (a.down + 15) / 16;
#define CFZ_DOWN_CASE(NB)                                                                          \
    if (nb <= NB) {                                                                                \
        adapter_down_kernel<T, NB, TM><<<grid, 256, 0, st>>>(a);                                    \
        return hipGetLastError();                                                                  \
    }
    CFZ_DOWN_CASE(1)
    CFZ_DOWN_CASE(2)
    CFZ_DOWN_CASE(4)
    CFZ_DOWN_CASE(6)
    CFZ_DOWN_CASE(8)
    if constexpr (TM == 1) {
        CFZ_DOWN_CASE(12)
        CFZ_DOWN_CASE(16)
    }
#undef CFZ_DOWN_CASE
    return hipErrorInvalidValue;
}

template <class T, class Y> hipError_t up_as(const AdapterArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)(adapter_tiles(a, kUpRows) * a.col_tiles));
    switch ((a.rank + 31) / 32) {
    case 1: adapter_up_kernel<T, Y, 1><<<grid, 256, 0, st>>>(a); break;
    case 2: adapter_up_kernel<T, Y, 2><<<grid, 256, 0, st>>>(a); break;
    case 3: adapter_up_kernel<T, Y, 3><<<grid, 256, 0, st>>>(a); break;
    default: adapter_up_kernel<T, Y, 4><<<grid, 256, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

template <class T> hipError_t add_as(const AdapterArgs &a, bool f32, hipStream_t st)
{
    const hipError_t e = a.tall ? down_as<T, 2>(a, st) : down_as<T, 1>(a, st);
    if (e != hipSuccess)
        return e;
    return f32 ? up_as<T, float>(a, st) : up_as<T, T>(a, st);
}

}  // namespace

int64_t adapter_tiles(const AdapterArgs &a, int rows) { return a.rows.tokens / rows + a.rows.batch; }

int64_t adapter_groups(const AdapterArgs &a)
{
    const int64_t down = adapter_tiles(a, a.tall ? 32 : 16) * a.splits;
    const int64_t up = adapter_tiles(a, kUpRows) * a.col_tiles;
    return down > up ? down : up;
}

// Tokens of a tile, and into how many runs the columns of x are cut: enough work-groups to fill the
// card twice, with no run shorter than two chunks a wave.
void adapter_plan(AdapterArgs &a)
{
    a.tall = a.rows.tokens >= 16 * (int64_t)a.rows.batch * 2 && a.down <= 128;
    const int64_t tiles = adapter_tiles(a, a.tall ? 32 : 16) + 1;  // (there may be none)
    const int64_t want = (512 + tiles - 1) / tiles, most = a.cols_in / 512;
    a.splits = (int)(want < most ? want : most);
    a.splits = a.splits < 1 ? 1 : a.splits;
}

hipError_t launch_adapters(const AdapterArgs &a, bool f16, bool y_f32, hipStream_t st)
{
    return f16 ? add_as<_Float16>(a, y_f32, st) : add_as<uint16_t>(a, y_f32, st);
}

}  // namespace cfz
