// block_norm_kernels.hip -- the norms around a block with its gate and its residual sum.
#include "block_internal.h"

namespace cfz {
namespace {

// Threads of a work-group whose rows take G threads each: 256 / G rows of up to a wave, or one row.
constexpr int group_threads(int g) { return g <= 64 ? 256 : g; }

// Sum over the threads that hold one row: part of a wave, or up to four.
template <int G> __device__ inline float row_sum(float x, float *red)
{
    x = lanes_sum(x, G < 64 ? G : 64);
    if (G <= 64)
        return x;
    const int wave = threadIdx.x >> 6;
    __syncthreads();  // (what was read from red before)
    if ((threadIdx.x & 63) == 0)
        red[wave] = x;
    __syncthreads();
    return G == 128 ? red[0] + red[1] : (red[0] + red[1]) + (red[2] + red[3]);
}

// v becomes its norm, in two passes over registers: the mean first, so that nothing cancels in
// the squares' sum.  Vectors past the row hold zeros and are left out of the second pass.
template <class T, int V, int G>
__device__ inline void normalise(float (&v)[V][8], const BlockNormOf &n, int cols, int tid, float *red)
{
    if (n.kind == CFZ_NORM_NONE)
        return;
    const float inv = 1.0f / (float)cols;
    float mean = 0.0f;
    if (n.kind == CFZ_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s += v[i][j];
        mean = row_sum<G>(s, red) * inv;
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if ((i * G + tid) * 8 < cols) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] -= mean;
                q = fmaf(v[i][j], v[i][j], q);
            }
        }
    }
    float square = row_sum<G>(q, red) * inv + n.eps;
    if (!norm_in_range(square)) {  // (the same for all threads of the row)
        const float step = norm_step(square);
        q = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] *= step;
                q = fmaf(v[i][j], v[i][j], q);
            }
        square = row_sum<G>(q, red) * inv + n.eps * step * step;
    }
    const float f = rsqrtf(square);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = (i * G + tid) * 8;
        if (at < cols) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] *= f;
            float w[8];
            if (n.w.p) {
                load_vec<T>(n.w, at, w);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] *= w[j];
            }
            if (n.b.p) {
                load_vec<T>(n.b, at, w);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] += w[j];
            }
        }
    }
}

// A row stays in registers from its load to its stores: x and y are read once, r and h written once.
// G threads hold a row, V vectors of 8 values each.  Bound by the bytes: 2 x 4388 rows of 1920, bf16, with
// gate, scale and shift in 27.1 us (135 MB, 5.0 TB/s); 12,393 rows of 4096 between an fp32 stream and fp16 with a norm on
// either side in 115 us (609 MB, 5.3 TB/s).  Few values a thread and short work-groups keep more rows under way
// than a wave a row did (30.9 and 143 us with 4 and 8 vectors a lane), and narrow rows share a wave (131,072 rows of
// 256: 49.7 us, 5.4 TB/s, of 32 items 51.7 us and of 4096 items 59.5, as the rows of a wave look up their items one
// after the other; 524,288 rows of 64: 49.5, 64.7 and 100 us).  32 rows of 1024: 3.7 us.
template <class X, class Y, int V, int G>
__global__ __launch_bounds__(group_threads(G)) void residual_norm_kernel(ResidualArgs a)
{
    __shared__ float red[4];
    const int tid = threadIdx.x % G;
    const int64_t row = (int64_t)blockIdx.x * (group_threads(G) / G) + threadIdx.x / G;
    if (G >= 64 && row >= a.rows.tokens)
        return;
    // (a wave of several rows goes on together until their items are known: past the end, the last row)
    const int64_t near = row < a.rows.tokens ? row : a.rows.tokens - 1;
    const X *x = (const X *)a.x + near * a.xs;
    const Y *y = (const Y *)a.y + near * a.ys;
    // the rows are under way while their item is looked up
    float v[V][8], u[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = (i * G + tid) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[i][j] = u[i][j] = 0.0f;
        if (at < a.cols) {
            load_n(x + at, u[i]);
            if (a.y)
                load_n(y + at, v[i]);
        }
    }
    int64_t first;
    int item = -1;
    if (G >= 64 || !a.rows.off) {
        item = block_item(a.rows, near, &first);
    } else {
        const int64_t front = (int64_t)blockIdx.x * (256 / G) + (threadIdx.x >> 6) * (64 / G);
        for (int i = 0; i < 64 / G; ++i) {
            const int64_t r = front + i < a.rows.tokens ? front + i : a.rows.tokens - 1;
            const int found = block_item(a.rows, r, &first);
            item = (int)(threadIdx.x & 63) / G == i ? found : item;
        }
    }
    if (row >= a.rows.tokens || item < 0)
        return;
    if (a.y) {
        normalise<Y, V, G>(v, a.after, a.cols, tid, red);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = (i * G + tid) * 8;
            if (at >= a.cols)
                continue;
            float g[8];
            if (a.gate.p)
                load_vec<Y>(a.gate, item * a.gate.stride + at, g);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = fmaf(a.gate.p ? g[j] * a.gate_scale : a.gate_scale, v[i][j], u[i][j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = u[i][j];
    }
    if (a.r) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = (i * G + tid) * 8;
            if (at < a.cols)
                store_n((X *)a.r + row * a.rs + at, v[i]);
        }
    }
    if (!a.h)
        return;
    normalise<Y, V, G>(v, a.before, a.cols, tid, red);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = (i * G + tid) * 8;
        if (at >= a.cols)
            continue;
        float w[8];
        if (a.scale.p) {
            load_vec<Y>(a.scale, item * a.scale.stride + at, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] *= 1.0f + w[j];
        }
        if (a.shift.p) {
            load_vec<Y>(a.shift, item * a.shift.stride + at, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] += w[j];
        }
        store_n((Y *)a.h + row * a.hs + at, v[i]);
    }
}

template <class X, class Y> hipError_t launch_as(const ResidualArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)residual_groups(a));
#define CFZ_NORM_CASE(V, G)                                                                        \
    if (a.cols <= 8 * V * G) {                                                                     \
        residual_norm_kernel<X, Y, V, G><<<grid, group_threads(G), 0, st>>>(a);                     \
        return hipGetLastError();                                                                  \
    }
    CFZ_NORM_CASE(1, 8)
    CFZ_NORM_CASE(1, 16)
    CFZ_NORM_CASE(1, 32)
    CFZ_NORM_CASE(1, 64)
    CFZ_NORM_CASE(1, 128)
    CFZ_NORM_CASE(1, 256)
    CFZ_NORM_CASE(2, 256)
    CFZ_NORM_CASE(4, 256)
    CFZ_NORM_CASE(8, 256)
#undef CFZ_NORM_CASE
    return hipErrorInvalidValue;
}

}  // namespace

// Eight lanes a row and up: 32 rows a work-group of up to 64 columns, 16 to 4 of up to 128 to 512, else one.
int64_t residual_groups(const ResidualArgs &a)
{
    const int rows = a.cols <= 64 ? 32 : (a.cols <= 128 ? 16 : (a.cols <= 256 ? 8 : (a.cols <= 512 ? 4 : 1)));
    return (a.rows.tokens + rows - 1) / rows;
}

hipError_t launch_residual_norm(const ResidualArgs &a, int x_dtype, int y_dtype, hipStream_t st)
{
    if (y_dtype == CFZ_KV8_F32)
        return launch_as<float, float>(a, st);
    if (y_dtype == CFZ_KV8_BF16)
        return x_dtype == CFZ_KV8_F32 ? launch_as<float, uint16_t>(a, st)
                                      : launch_as<uint16_t, uint16_t>(a, st);
    return x_dtype == CFZ_KV8_F32 ? launch_as<float, _Float16>(a, st)
                                  : launch_as<_Float16, _Float16>(a, st);
}

}  // namespace cfz
