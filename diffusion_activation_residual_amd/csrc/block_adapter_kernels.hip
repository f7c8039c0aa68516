// block_adapter_kernels.hip -- low-rank adapters of many requests beside a shared projection.
//
//   out = y + scale (x A^T) B^T   for each sequence's own A, B and scale
//
// Two launches: h = scale x A^T into the workspace, then out = y + h B^T.  Both are bound by the rows
// that they read and write (x once, y and out once); the products are small beside them.  2 x 4388 rows of
// 1920 to 3 x 1920 columns at rank 32, bf16: 15.1 + 42.8 us, 237 MB at 4.1 TB/s; 12,393 ragged rows of 4096 to
// 4096 at rank 64, fp16: 29.3 + 44.2 us, 298 MB at 4.1 TB/s; 32 single tokens of 1024 to 3 x 1024 at rank 16:
// 5.7 + 4.7 us, dependent reads.
//
// Row tiles never straddle sequences: sequence b's tiles are numbered from offsets[b] / R + b on, which
// leaves room for a short tile at its end, so that a tile finds its sequence by a search and the
// host needs no list.
#include "block_internal.h"

#include <type_traits>

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

// The rows of a tile: row0 .. row0 + n - 1 of the call, n <= R, and their adapter (-1: none).  False: the tile
// holds nothing.  Up to 63 sequences are looked at together, with one load each.
template <int R>
__device__ inline bool find_tile(const AdapterArgs &a, int tile, int64_t &row0, int &n, int &id)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = a.rows.tokens;
    auto clamp = [&](int64_t o) { return o < 0 ? 0 : (o > t ? t : o); };
    int seq = 0;  // the last sequence whose first tile is at or before this one
    int64_t first, end;
    if (a.rows.batch < 64) {
        const int b = lane < a.rows.batch ? lane : a.rows.batch;
        const int o = (int)clamp(a.rows.off[b]);
        const int ids = a.ids[b < a.rows.batch ? b : 0];
        const uint64_t votes = __ballot(lane < a.rows.batch && o / R + lane <= tile);
        seq = votes ? 63 - __clzll(votes) : 0;
        first = __builtin_amdgcn_readlane(o, seq);
        end = __builtin_amdgcn_readlane(o, seq + 1);
        id = __builtin_amdgcn_readlane(ids, seq);
    } else {
        int left = a.rows.batch;
        while (left > 1) {
            const int step = (left + 63) / 64;
            const int b = seq + lane * step;
            const bool before = lane * step < left && clamp(a.rows.off[b]) / R + b <= tile;
            const uint64_t votes = __ballot(before);
            const int k = votes ? 63 - __clzll(votes) : 0;
            left = left - k * step < step ? left - k * step : step;
            seq += k * step;
        }
        first = clamp(a.rows.off[seq]);
        end = clamp(a.rows.off[seq + 1]);
        id = __builtin_amdgcn_readfirstlane(a.ids[seq]);
    }
    if (id < 0 || id >= a.adapters)
        id = -1;
    end = end - first > a.max_rows ? first + a.max_rows : end;
    const int64_t mine = tile - (first / R + seq);
    row0 = first + mine * R;
    if (mine < 0 || row0 >= end)
        return false;
    n = (int)(end - row0 < R ? end - row0 : R);
    return true;
}

// Orders a wave's own writes to LDS before its reads of what other lanes wrote, and the other way round.
__device__ inline void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Steps of 32 columns: whole groups of four, in which the first product goes.
__host__ __device__ inline int down_steps(const AdapterArgs &a) { return (a.cols_in + 127) / 128 * 4; }

// Lays out A for the matrix instructions: 16 rows x 32 columns side by side, lane 16 q + m's 8 columns 8 q ..
// 8 q + 7 of row m, zeros past either end.  A thread a piece of 16 bytes.
__global__ __launch_bounds__(256) void adapter_put_kernel(AdapterArgs a, const uint16_t *rows, int first,
                                                          int64_t pieces)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= pieces)
        return;
    const int steps = down_steps(a), blocks = (a.down + 15) / 16;
    const int lane = (int)(i % 64);
    const int64_t at = i / 64;
    const int step = (int)(at % steps), block = (int)(at / steps % blocks);
    const int64_t adapter = at / steps / blocks;
    const int row = block * 16 + (lane & 15), col = step * 32 + (lane >> 4) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < a.down && col < a.cols_in)
        v = *(const uint4 *)(rows + (adapter * a.down + row) * a.cols_in + col);
    ((uint4 *)a.a)[(int64_t)first * blocks * steps * 64 + i] = v;
}

// h = scale x A^T of TM x 16 tokens for NB x 16 adapter rows.  W waves take a run of the columns each, four
// steps of 32 at a time, and their sums are added in LDS, half of the waves at a time.  The matrix
// instructions' rows are A's and their columns the tokens.  An operand's lanes are 16 different rows: read
// so from rows in memory, each lane's 16 bytes are an access of their own, and the first-level cache gives
// 16 bytes a clock (31 us for the video shares).  So A is laid out once as the instructions take it, and of
// x eight neighbouring lanes read 128 bytes of a row, which the wave turns round in LDS, a row's eight
// pieces shifted by its number so that no bank is met twice (four lanes and 64 bytes: 34 instead of 29 us for
// the prompts).  Two or four steps are under way.  Tiles start their runs at different places, so that rows a
// power of two apart are not all read from the same channels at once.
//
// h leaves as the sum of two 16-bit numbers, the operands of the second product: that leaves 2^-16 of it
// (bf16) or 2^-21 of its row's largest in a slice (fp16, after a power of two that brings the row into
// range), where the rounding of a result in these types leaves 2^-8 and 2^-11.
template <class T, int NB, int TM, int W>
__global__ __launch_bounds__(64 * W) void adapter_down_kernel(AdapterArgs a)
{
    constexpr int kBlocks = NB * TM, kHalf = W / 2;
    constexpr int kRow = NB * 16 + 4;  // of the sums in LDS
    __shared__ union {
        uint4 turn[W][TM][128];
        f32x4 part[kHalf][kBlocks][64];
        float sum[TM * 16][kRow];
    } s;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // adapter rows first .. first + down - 1 (whole slices, from a block of 16 on)
    const int part = blockIdx.x % a.parts, tile = blockIdx.x / a.parts;
    const int first = part * a.part_rows;
    const int down = a.down - first < a.part_rows ? a.down - first : a.part_rows;
    int n, id;
    int64_t row0;
    if (!find_tile<16 * TM>(a, tile, row0, n, id) || id < 0)
        return;
    const int m = lane & 15, q = lane >> 4;
    const int r = lane >> 3, piece = lane & 7;  // of half a block: row and 16 bytes, as they are read
    const T *x[TM][2];
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // (rows past the tile's end repeat the last one: their sums are not kept)
            const int row = t * 16 + i * 8 + r;
            x[t][i] = (const T *)a.x + (row0 + (row < n ? row : n - 1)) * a.xs + piece * 8;
        }
    const int steps = down_steps(a), blocks = (down + 15) / 16;
    const uint4 *w =
        (const uint4 *)a.a + ((int64_t)id * ((a.down + 15) / 16) + first / 16) * steps * 64;
    uint4 *lds = s.turn[wave][0];
    f32x4 acc[TM][NB];
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // groups of four steps g0 .. g1 - 1, from one in their midst on and round
    const int g0 = steps / 4 * wave / W, g1 = steps / 4 * (wave + 1) / W;
    int step = 0;  // the first one of the group
    // pairs of steps of x and steps of A in registers, as many as they hold beside the sums
    constexpr int XP = TM == 4 && NB > 4 ? 1 : 2, AS = NB > 4 ? 2 : 4;
    uint4 xv[XP][TM][2], wv[AS][NB];
    auto load_x = [&](int step, auto at) {
        const int k = step * 32;
        const bool in = k + piece * 8 < a.cols_in;
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                xv[decltype(at)::value % XP][t][i] = *(const uint4 *)(x[t][i] + (in ? k : -piece * 8));
    };
    auto load_a = [&](int step, auto at) {
        // (a block past the last one repeats it: its sums are not kept)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            wv[decltype(at)::value % AS][j] =
                (w + ((int64_t)(j < blocks ? j : blocks - 1) * steps + step) * 64)[lane];
    };
    // (past the last group the loads repeat the first: no load is under a condition)
    int next = 0;
    auto ahead = [&](auto at) {
        constexpr int I = decltype(at)::value;
        return I < 4 ? step + I : next + I - 4;
    };
    auto put = [&](auto at) {
        // past the last column zeros
        constexpr int I = decltype(at)::value;
        const uint32_t keep = (step + 2 * I) * 32 + piece * 8 < a.cols_in ? ~0u : 0u;
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 v = xv[I % XP][t][i];
                const int row = i * 8 + r;
                lds[t * 128 + row * 8 + (piece ^ (row >> 1))] =
                    make_uint4(v.x & keep, v.y & keep, v.z & keep, v.w & keep);
            }
    };
    auto multiply = [&](auto at) {
        constexpr int I = decltype(at)::value;
        constexpr std::integral_constant<int, I + AS - 1> ia{};
        load_a(ahead(ia), ia);
        uint4 xo[TM];
#pragma unroll
        for (int t = 0; t < TM; ++t)
            xo[t] = lds[t * 128 + m * 8 + ((I % 2 * 4 + q) ^ (m >> 1))];
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int t = 0; t < TM; ++t)
                acc[t][j] = Mfma<T>::mul(wv[I % AS][j], xo[t], acc[t][j]);
    };
    auto pair = [&](auto at) {
        constexpr int I = decltype(at)::value;
        constexpr std::integral_constant<int, 2 * I> even{};
        constexpr std::integral_constant<int, 2 * I + 1> odd{};
        put(at);
        wave_sync();
        load_x(ahead(std::integral_constant<int, 2 * (I + XP)>()), std::integral_constant<int, I + XP>());
        multiply(even);
        multiply(odd);
        wave_sync();
    };
    constexpr std::integral_constant<int, 0> i0{};
    constexpr std::integral_constant<int, 1> i1{};
    constexpr std::integral_constant<int, 2> i2{};
    if (g0 < g1) {
        step = (g0 + tile % (g1 - g0)) * 4;
        load_x(step, i0);
        load_a(step, i0);
        if constexpr (XP == 2)
            load_x(step + 2, i1);
        if constexpr (AS == 4) {
            load_a(step + 1, i1);
            load_a(step + 2, i2);
        }
    }
    for (int g = g0; g < g1; ++g) {
        next = step + 4 < g1 * 4 ? step + 4 : g0 * 4;
        pair(i0);
        pair(i1);
        step = next;
    }
    __syncthreads();
    // the upper half's sums to the lower, then the lower half's to all
    if (wave >= kHalf) {
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                s.part[wave - kHalf][t * NB + j][lane] = acc[t][j];
    }
    __syncthreads();
    if (wave < kHalf) {
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                s.part[wave][t * NB + j][lane] = acc[t][j] + s.part[wave][t * NB + j][lane];
    }
    __syncthreads();
    constexpr int kMine = (kBlocks + W - 1) / W;
    f32x4 sum[kMine];
    const float scale = a.scale ? a.scale[id] : 1.0f;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int b = i * W + wave;
        if (b < kBlocks) {
            sum[i] = s.part[0][b][lane];
#pragma unroll
            for (int p = 1; p < kHalf; ++p)
                sum[i] += s.part[p][b][lane];
            sum[i] *= scale;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int b = i * W + wave;
        // lane: token m, adapter rows 4 q .. 4 q + 3 of the block
        if (b < kBlocks)
            *(f32x4 *)&s.sum[b / NB * 16 + m][b % NB * 16 + q * 4] = sum[i];
    }
    __syncthreads();
    const int units = down / 8;
    for (int i = threadIdx.x; i < n * units; i += 64 * W) {
        const int row = i / units, r = (i - row * units) * 8;
        const float *v = &s.sum[row][r];
        float f = 1.0f;
        if constexpr (__is_same(T, _Float16)) {
            const int slice = r / a.rank;
            float top = 0.0f;
            for (int k = slice * a.rank; k < (slice + 1) * a.rank; k += 4) {
                const f32x4 u = *(const f32x4 *)&s.sum[row][k];
                top = fmaxf(fmaxf(fmaxf(fabsf(u[0]), fabsf(u[1])), fmaxf(fabsf(u[2]), fabsf(u[3]))), top);
            }
            // a power of two that brings the largest into 1 .. 4 (0 stays; what is not finite: 1)
            int e = (int)(__float_as_uint(top) >> 23) - 127;
            e = e > 127 ? 0 : (e > 126 ? 126 : (e < -126 ? -126 : e));
            f = __uint_as_float((uint32_t)(127 - e) << 23);
            if (r == slice * a.rank)
                a.back[(row0 + row) * a.slices + first / a.rank + slice] = __uint_as_float((uint32_t)(127 + e) << 23);
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint16_t a0[2], a1[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float y = v[2 * k + u] * f;
                a0[u] = Mfma<T>::bits(y);
                const float rest = y - Mfma<T>::value(a0[u]);
                a1[u] = Mfma<T>::bits(rest == rest ? rest : 0.0f);  // (infinity has no rest)
            }
            hi[k] = (uint32_t)a0[0] | (uint32_t)a0[1] << 16;
            lo[k] = (uint32_t)a1[0] | (uint32_t)a1[1] << 16;
        }
        const int64_t at = (row0 + row) * a.down + first + r;
        *(uint4 *)(a.hi + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *(uint4 *)(a.lo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// out = y + h B^T: 64 columns a wave, four waves side by side in a slice, the tile's tokens 16 at a time,
// with the tile's y under way before the rest.  Tokens are the matrix instructions' rows and columns their
// columns, dealt out so that a lane ends up with four neighbouring ones and 16 lanes with a run of a row:
// y is read and out written in whole runs.  B stays in registers over the tile.  The tile's h
// lies in LDS, turned as x in the first product.
// Four columns a lane: eight, in half as many work-groups, take 180 registers and 46 instead of 43 us for 2 x
// 4388 rows of 5760 at rank 32, 49 instead of 45 for prompts of 4096 at rank 64.
constexpr int kUpRows = 64, CB = 4, kUpCols = 4 * 16 * CB;

// CB values of a row as they lie in memory, until they are needed as numbers.
template <class Y> struct RawRow {
    static constexpr int kBytes = CB * (int)sizeof(Y), kPiece = kBytes < 16 ? kBytes : 16;
    typedef uint32_t Words __attribute__((ext_vector_type(kPiece / 4)));
    struct alignas(kPiece) Piece { Y v[kPiece / sizeof(Y)]; } p[kBytes / kPiece];
    // (read once and for the last time: not to take the place of x, A and out in the caches)
    __device__ inline void load(const Y *y)
    {
#pragma unroll
        for (int i = 0; i < kBytes / kPiece; ++i)
            p[i] = __builtin_bit_cast(Piece, __builtin_nontemporal_load((const Words *)y + i));
    }
    __device__ inline void store(Y *o) const
    {
#pragma unroll
        for (int i = 0; i < kBytes / kPiece; ++i)
            ((Words *)o)[i] = __builtin_bit_cast(Words, p[i]);
    }
    __device__ inline void get(float (&o)[CB]) const
    {
        constexpr int E = kPiece / sizeof(Y);
#pragma unroll
        for (int i = 0; i < CB; ++i)
            o[i] = BlockType<Y>::get(p[i / E].v[i % E]);
    }
};

template <class T, class Y, int KS>
__global__ __launch_bounds__(256) void adapter_up_kernel(AdapterArgs a)
{
    // blocks of 16 tokens under way together: rank 32 in 41.7 us with two and 42.9 with four, rank 64 in 46.7 and
    // 44.6 (the sizes above)
    constexpr int kAhead = sizeof(Y) == 4 || KS == 1 ? 2 : 4;
    constexpr int RU = KS == 1 ? 4 : (KS == 2 ? 8 : 16);  // pieces of 16 bytes of a row in LDS
    __shared__ uint4 hs[2][kUpRows * RU];
    __shared__ alignas(16) float back[kUpRows];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile = blockIdx.x / a.col_tiles, part = blockIdx.x % a.col_tiles;
    int n, id;
    int64_t row0;
    if (!find_tile<kUpRows>(a, tile, row0, n, id))
        return;
    const bool some = id >= 0;
    if (!some && a.y == a.out)
        return;
    int slice = 0;
    while (slice + 1 < a.slices && part >= a.first_tile[slice + 1])
        ++slice;
    const int m = lane & 15, q = lane >> 4;
    const int col0 = a.first_col[slice] + ((part - a.first_tile[slice]) * 4 + wave) * 16 * CB;
    const int left = a.first_col[slice + 1] - col0;  // columns of the slice from here on
    const bool mine = m * CB < left;
    // Where some row or column is missing, its loads repeat another: a load under a condition of its own
    // waits for the one before.  Whole blocks, almost all of them, store without conditions.
    const Y *y = (const Y *)a.y + row0 * a.ys + (left > 0 ? col0 : 0) + (mine ? m * CB : 0);
    RawRow<Y> v[kAhead][4];
    auto load = [&](int t0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = t0 + u * 16 + q * 4 + i;
                v[u][i].load(y + (t < n ? t : n - 1) * a.ys);
            }
    };
    load(0);
    uint4 w[CB][KS];
    if (some) {
        const T *b = (const T *)a.b + ((int64_t)id * a.cols_out + (left > 0 ? col0 : 0)) * a.rank;
#pragma unroll
        for (int j = 0; j < CB; ++j)
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const bool in = mine && s * 32 + q * 8 < a.rank;
                const uint4 got = *(const uint4 *)(b + (in ? (m * CB + j) * a.rank + s * 32 + q * 8 : 0));
                const uint32_t keep = in ? ~0u : 0u;  // (a choice would become a branch around the load)
                w[j][s] = make_uint4(got.x & keep, got.y & keep, got.z & keep, got.w & keep);
            }
        constexpr int kHere = kUpRows * KS * 4 / 256;
        const int units = a.rank / 8;
        uint4 h[2][kHere];
#pragma unroll
        for (int i = 0; i < kHere; ++i) {
            const int at = threadIdx.x + i * 256, row = at / (KS * 4), u = at - row * (KS * 4);
            const int64_t from =
                (row0 + (row < n ? row : 0)) * a.down + slice * a.rank + (u < units ? u * 8 : 0);
            h[0][i] = *(const uint4 *)(a.hi + from);
            h[1][i] = *(const uint4 *)(a.lo + from);
        }
#pragma unroll
        for (int i = 0; i < kHere; ++i) {
            const int at = threadIdx.x + i * 256, row = at / (KS * 4), u = at - row * (KS * 4);
            const bool in = row < n && u < units;
            const int to = row * RU + (u ^ (row / (16 / RU) % RU));
            hs[0][to] = in ? h[0][i] : make_uint4(0, 0, 0, 0);
            hs[1][to] = in ? h[1][i] : make_uint4(0, 0, 0, 0);
        }
        if (__is_same(T, _Float16) && threadIdx.x < kUpRows)
            back[threadIdx.x] =
                (int)threadIdx.x < n ? a.back[(row0 + threadIdx.x) * a.slices + slice] : 1.0f;
        __syncthreads();
    }
    if (left <= 0)
        return;
    const bool whole = left >= 16 * CB;
    Y *out = (Y *)a.out + row0 * a.os + col0 + m * CB;
    for (int t0 = 0; t0 < n; t0 += 16 * kAhead) {
        if (t0 > 0)
            load(t0);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int t = t0 + u * 16 + q * 4;
            if (!some) {  // y as it is, to the last bit
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (mine && t + i < n)
                        v[u][i].store(out + (t + i) * a.os);
                continue;
            }
            f32x4 acc[CB];
#pragma unroll
            for (int j = 0; j < CB; ++j)
                acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            f32x4 f = {1.0f, 1.0f, 1.0f, 1.0f};
            // (rows past the last one: zeros up to the tile's end)
            const int row = t0 + u * 16 + m;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const int at = row * RU + ((s * 4 + q) ^ (row / (16 / RU) % RU));
                const uint4 hi = hs[0][at], lo = hs[1][at];
#pragma unroll
                for (int j = 0; j < CB; ++j) {
                    acc[j] = Mfma<T>::mul(lo, w[j][s], acc[j]);
                    acc[j] = Mfma<T>::mul(hi, w[j][s], acc[j]);
                }
            }
            if (__is_same(T, _Float16))
                f = *(const f32x4 *)&back[t0 + u * 16 + q * 4];
            // lane: token 4 q + i, columns CB m + j
            float o[4][CB];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[u][i].get(o[i]);
#pragma unroll
                for (int j = 0; j < CB; ++j)
                    o[i][j] = fmaf(acc[j][i], f[i], o[i][j]);
            }
            if (whole && t0 + u * 16 + 16 <= n) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    store_n(out + (t + i) * a.os, o[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (mine && t + i < n)
                        store_n(out + (t + i) * a.os, o[i]);
            }
        }
    }
}

template <class T, int TM, int W> hipError_t down_as(const AdapterArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)(adapter_tiles(a, 16 * TM) * a.parts));
    const int nb = (a.part_rows + 15) / 16;
#define CFZ_DOWN_CASE(NB)                                                                          \
    if (nb <= NB) {                                                                                \
        adapter_down_kernel<T, NB, TM, W><<<grid, 64 * W, 0, st>>>(a);                              \
        return hipGetLastError();                                                                  \
    }
    CFZ_DOWN_CASE(1)
    CFZ_DOWN_CASE(2)
    CFZ_DOWN_CASE(4)
    CFZ_DOWN_CASE(6)
    if constexpr (TM < 4) {
        CFZ_DOWN_CASE(8)
    }
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
    const hipError_t e = a.tall == 4   ? down_as<T, 4, 8>(a, st)
                         : a.tall == 2 ? down_as<T, 2, 4>(a, st)
                                       : down_as<T, 1, 8>(a, st);
    if (e != hipSuccess)
        return e;
    return f32 ? up_as<T, float>(a, st) : up_as<T, T>(a, st);
}

}  // namespace

int64_t adapter_tiles(const AdapterArgs &a, int rows) { return a.rows.tokens / rows + a.rows.batch; }

int64_t adapter_groups(const AdapterArgs &a)
{
    const int64_t down = adapter_tiles(a, 16 * a.tall) * a.parts;
    const int64_t up = adapter_tiles(a, kUpRows) * a.col_tiles;
    return down > up ? down : up;
}

// The more tokens a tile of the first product has, the less often A is read: 64, where sequences have as many on
// the average, half of the card's 256 units get a whole tile and the sums of up to 96 adapter rows fit the registers
// (2 x 4388 rows of 1920 at 96 adapter rows: 15.1 us, with 32 tokens 16.8; ragged prompts of 4096 columns at 64:
// 29.2 and 33.9; but 64 sequences of 64 tokens, 64 tiles: 15.5 and 11.6); else 32, up to 128 adapter rows; else 16
// (1000 tokens beside 63 single ones: 8.8 us, with 32 tokens a tile 11.6; 4000 beside 200: 14.2, 15.0, with 64 23.3;
// 8000 beside 300: 23.6, 22.9, 25.9).  Four waves a tile of 32, eight of the others.  More than 256 adapter rows are
// two work-groups' a tile, two slices each.
void adapter_plan(AdapterArgs &a)
{
    a.col_tiles = 0;
    for (int i = 0; i < a.slices; ++i) {
        a.first_tile[i] = a.col_tiles;
        a.col_tiles += (a.first_col[i + 1] - a.first_col[i] + kUpCols - 1) / kUpCols;
    }
    // (two slices together end with a block of 16 rows, whatever their rank)
    a.parts = a.down > 256 ? 2 : 1;
    a.part_rows = a.parts == 2 ? 2 * a.rank : a.down;
    const int64_t t = a.rows.tokens, mean = t / (a.rows.batch > 0 ? a.rows.batch : 1);
    if (a.part_rows <= 96 && mean >= 64 && t / 64 >= 128)
        a.tall = 4;
    else
        a.tall = a.part_rows <= 128 && mean >= 32 ? 2 : 1;
}

int64_t adapter_pieces(const AdapterArgs &a)
{
    return (int64_t)((a.down + 15) / 16) * down_steps(a) * 64;
}

hipError_t launch_adapters_put(const AdapterArgs &a, const void *rows, int first, int count,
                               hipStream_t st)
{
    const int64_t pieces = adapter_pieces(a) * count;
    adapter_put_kernel<<<dim3((unsigned)((pieces + 255) / 256)), 256, 0, st>>>(
        a, (const uint16_t *)rows, first, pieces);
    return hipGetLastError();
}

hipError_t launch_adapters(const AdapterArgs &a, bool f16, bool y_f32, hipStream_t st)
{
    return f16 ? add_as<_Float16>(a, y_f32, st) : add_as<uint16_t>(a, y_f32, st);
}

}  // namespace cfz
