// block_api.hip -- the C ABI of cfz_block.h: argument validation and dispatch.  Nothing touches
// the device until every argument has been checked.
#include "api_checks.h"
#include "block_internal.h"

#include <limits.h>
#include <math.h>
#include <string.h>

using cfz::aligned;
using cfz::fail;
using cfz::hip_status;

namespace {

bool is_dtype(int d) { return d == CFZ_KV8_BF16 || d == CFZ_KV8_F16 || d == CFZ_KV8_F32; }
int width_of(int dtype) { return dtype == CFZ_KV8_F32 ? 4 : 2; }

cfz_status check_stride(int64_t stride, int64_t row, int dtype, const char *what)
{
    if (stride < row || stride > INT_MAX || stride * width_of(dtype) % 16 != 0)
        return fail(CFZ_ERR_SHAPE, "%s = %lld (at least %lld, a multiple of 16 bytes)", what,
                    (long long)stride, (long long)row);
    return CFZ_OK;
}

cfz_status check_rows(int64_t tokens, int32_t batch, const int32_t *offsets, cfz::BlockRows *rows)
{
    if (tokens < 0 || tokens > INT_MAX)
        return fail(CFZ_ERR_SHAPE, "tokens = %lld", (long long)tokens);
    if (batch < 1 || batch > 65535)
        return fail(CFZ_ERR_SHAPE, "batch = %d", batch);
    if (!offsets && tokens % batch != 0)
        return fail(CFZ_ERR_SHAPE, "%lld tokens do not divide into %d items", (long long)tokens,
                    batch);
    if (!aligned(offsets, 4))
        return fail(CFZ_ERR_ALIGN, "offsets must be 4-byte aligned");
    *rows = cfz::BlockRows{offsets, tokens, tokens / batch, batch};
    return CFZ_OK;
}

// A vector's type: fp32 or the call's own.
cfz_status check_vec(const void *p, int dtype, int call, const char *what)
{
    if (!p)
        return CFZ_OK;
    if (dtype != CFZ_KV8_F32 && dtype != call)
        return fail(CFZ_ERR_UNSUPPORTED, "%s: dtype = %d with rows of %d", what, dtype, call);
    if (!aligned(p, 16))
        return fail(CFZ_ERR_ALIGN, "%s must be 16-byte aligned", what);
    return CFZ_OK;
}

cfz_status check_items(const cfz_item_rows &v, int cols, int call, const char *what,
                       cfz::BlockVec *out)
{
    *out = cfz::BlockVec{v.data, v.stride, v.dtype == CFZ_KV8_F32};
    if (!v.data)
        return CFZ_OK;
    CFZ_TRY(check_vec(v.data, v.dtype, call, what));
    return v.stride == 0 ? CFZ_OK : check_stride(v.stride, cols, v.dtype, what);
}

cfz_status check_norm(const cfz_norm &n, int call, const char *what, cfz::BlockNormOf *out)
{
    if (n.kind < CFZ_NORM_NONE || n.kind > CFZ_NORM_LAYER)
        return fail(CFZ_ERR_UNSUPPORTED, "%s: kind = %d", what, n.kind);
    const bool none = n.kind == CFZ_NORM_NONE;
    if (!none && (!(n.eps >= 0.0f) || !isfinite(n.eps)))
        return fail(CFZ_ERR_SHAPE, "%s: eps = %g must be finite and not negative", what,
                    (double)n.eps);
    if (n.bias && n.kind != CFZ_NORM_LAYER)
        return fail(CFZ_ERR_UNSUPPORTED, "%s: a bias goes with the LAYER norm only", what);
    if (n.weight && none)
        return fail(CFZ_ERR_UNSUPPORTED, "%s: a weight without a norm", what);
    CFZ_TRY(check_vec(n.weight, n.dtype, call, what));
    CFZ_TRY(check_vec(n.bias, n.dtype, call, what));
    const int f32 = n.dtype == CFZ_KV8_F32;
    *out = cfz::BlockNormOf{n.kind, n.eps, {n.weight, 0, f32}, {n.bias, 0, f32}};
    return CFZ_OK;
}

// Sizes only, so that the workspace query can use it too.
cfz_status check_adapters(const cfz_adapters *w, int64_t tokens, int32_t batch, cfz::AdapterArgs *a)
{
    if (!w)
        return fail(CFZ_ERR_NULL, "adapters is required");
    memset(a, 0, sizeof *a);
    if (w->dtype != CFZ_KV8_BF16 && w->dtype != CFZ_KV8_F16)
        return fail(CFZ_ERR_UNSUPPORTED, "dtype = %d", w->dtype);
    if (w->adapters < 1 || w->adapters > 1 << 20)
        return fail(CFZ_ERR_SHAPE, "adapters = %d (1 .. 2^20)", w->adapters);
    if (w->slices < 1 || w->slices > 4)
        return fail(CFZ_ERR_SHAPE, "slices = %d (1 .. 4)", w->slices);
    if (w->rank < 8 || w->rank > 128 || w->rank % 8 != 0)
        return fail(CFZ_ERR_SHAPE, "rank = %d (a multiple of 8, 8 .. 128)", w->rank);
    if (w->cols_in < 8 || w->cols_in > 1 << 20 || w->cols_in % 8 != 0)
        return fail(CFZ_ERR_SHAPE, "cols_in = %d (a multiple of 8, 8 .. 2^20)", w->cols_in);
    int cols = 0;
    for (int i = 0; i < w->slices; ++i) {
        const int c = w->slice_cols[i];
        if (c < 16 || c > 1 << 20 || c % 16 != 0)
            return fail(CFZ_ERR_SHAPE, "slice_cols[%d] = %d (a multiple of 16, 16 .. 2^20)", i, c);
        a->first_col[i] = cols;
        cols += c;
    }
    if (cols > 1 << 20)
        return fail(CFZ_ERR_SHAPE, "%d columns (at most 2^20)", cols);
    a->first_col[w->slices] = cols;
    if (tokens < 0 || tokens > INT_MAX)
        return fail(CFZ_ERR_SHAPE, "tokens = %lld", (long long)tokens);
    if (batch < 0 || batch > 65535)
        return fail(CFZ_ERR_SHAPE, "batch = %d", batch);
    a->rows.tokens = tokens;
    a->rows.batch = batch;
    a->adapters = w->adapters;
    a->slices = w->slices;
    a->rank = w->rank;
    a->down = w->slices * w->rank;
    a->cols_in = w->cols_in;
    a->cols_out = cols;
    cfz::adapter_plan(*a);
    return CFZ_OK;
}

size_t adapters_bytes(const cfz::AdapterArgs &a)
{
    if (a.rows.tokens == 0 || a.rows.batch == 0)
        return 0;
    return (size_t)a.rows.tokens * (a.down + a.slices) * 4;
}

}  // namespace

extern "C" {

cfz_status cfz_residual_norm(const cfz_residual *r, void *hip_stream)
{
    if (!r)
        return fail(CFZ_ERR_NULL, "args is required");
    if (!is_dtype(r->x_dtype) || !is_dtype(r->y_dtype) ||
        (r->x_dtype != r->y_dtype && r->x_dtype != CFZ_KV8_F32))
        return fail(CFZ_ERR_UNSUPPORTED, "x_dtype = %d with y_dtype = %d", r->x_dtype, r->y_dtype);
    if (r->cols < 8 || r->cols > 16384 || r->cols % 8 != 0)
        return fail(CFZ_ERR_SHAPE, "cols = %d (a multiple of 8, 8 .. 16384)", r->cols);
    cfz::ResidualArgs a;
    CFZ_TRY(check_rows(r->tokens, r->batch, r->offsets, &a.rows));
    if (!isfinite(r->gate_scale))
        return fail(CFZ_ERR_SHAPE, "gate_scale = %g", (double)r->gate_scale);
    const int call = r->y_dtype;
    CFZ_TRY(check_items(r->gate, r->cols, call, "gate", &a.gate));
    CFZ_TRY(check_items(r->scale, r->cols, call, "scale", &a.scale));
    CFZ_TRY(check_items(r->shift, r->cols, call, "shift", &a.shift));
    CFZ_TRY(check_norm(r->after, call, "after", &a.after));
    CFZ_TRY(check_norm(r->before, call, "before", &a.before));
    CFZ_TRY(check_stride(r->x_stride, r->cols, r->x_dtype, "x_stride"));
    if (r->y)
        CFZ_TRY(check_stride(r->y_stride, r->cols, call, "y_stride"));
    if (r->r)
        CFZ_TRY(check_stride(r->r_stride, r->cols, r->x_dtype, "r_stride"));
    if (r->h)
        CFZ_TRY(check_stride(r->h_stride, r->cols, call, "h_stride"));
    if (r->tokens == 0)
        return CFZ_OK;
    if (!aligned(r->x, 16) || !aligned(r->y, 16) || !aligned(r->r, 16) || !aligned(r->h, 16))
        return fail(CFZ_ERR_ALIGN, "x, y, r and h must be 16-byte aligned");
    if ((r->r && r->r == r->x && r->r_stride != r->x_stride) ||
        (r->h && r->h == r->y && r->h_stride != r->y_stride))
        return fail(CFZ_ERR_SHAPE, "in place, the strides must be the same");
    a.cols = r->cols;
    if (cfz::residual_groups(a) >= cfz::kBlockMaxGroups)
        return fail(CFZ_ERR_SHAPE, "the call needs %lld work-groups (limit 2^23)",
                    (long long)cfz::residual_groups(a));
    if (!r->y && (r->gate.data || r->after.kind != CFZ_NORM_NONE))
        return fail(CFZ_ERR_NULL, "a gate and a norm of y need y");
    if (!r->r && !r->h)
        return fail(CFZ_ERR_NULL, "one of r and h is required");
    if (!r->x)
        return fail(CFZ_ERR_NULL, "x is required");
    a.x = r->x, a.y = r->y, a.r = r->r, a.h = r->h;
    a.xs = r->x_stride, a.ys = r->y_stride, a.rs = r->r_stride, a.hs = r->h_stride;
    a.gate_scale = r->gate_scale;
    return hip_status(cfz::launch_residual_norm(a, r->x_dtype, call, (hipStream_t)hip_stream),
                      "residual norm launch");
}

cfz_status cfz_rotation_table(const cfz_rotation_angles *g, int64_t rows, const int32_t *positions,
                              float *cos, float *sin, void *hip_stream)
{
    if (!g)
        return fail(CFZ_ERR_NULL, "angles is required");
    if (g->rot_dim < 8 || g->rot_dim > 256 || g->rot_dim % 8 != 0)
        return fail(CFZ_ERR_SHAPE, "rot_dim = %d (a multiple of 8, 8 .. 256)", g->rot_dim);
    if (g->axes < 1 || g->axes > 4)
        return fail(CFZ_ERR_SHAPE, "axes = %d (1 .. 4)", g->axes);
    if (g->scaling < CFZ_ROTATION_PLAIN || g->scaling > CFZ_ROTATION_PARTS)
        return fail(CFZ_ERR_UNSUPPORTED, "scaling = %d", g->scaling);
    const bool base = g->scaling == CFZ_ROTATION_BASE, parts = g->scaling == CFZ_ROTATION_PARTS;
    int sum = 0;
    for (int j = 0; j < g->axes; ++j) {
        const int d = g->axis_dim[j];
        if (d < 2 || d % 2 != 0 || d > 256 || (base && d == 2))
            return fail(CFZ_ERR_SHAPE, "axis_dim[%d] = %d", j, d);
        sum += d;
    }
    if (sum != g->rot_dim)
        return fail(CFZ_ERR_SHAPE, "the axes have %d dimensions, rot_dim is %d", sum, g->rot_dim);
    if (!(g->base > 1.0) || !isfinite(g->base) || !(g->factor > 0.0) || !isfinite(g->factor) ||
        !(g->amplitude > 0.0) || !isfinite(g->amplitude))
        return fail(CFZ_ERR_SHAPE, "base = %g, factor = %g, amplitude = %g", g->base, g->factor,
                    g->amplitude);
    if (parts && (!(g->trained > 0.0) || !isfinite(g->trained) || !(g->slow >= 0.0) ||
                  !(g->fast > g->slow) || !isfinite(g->fast)))
        return fail(CFZ_ERR_SHAPE, "trained = %g, slow = %g, fast = %g", g->trained, g->slow,
                    g->fast);
    if (rows < 0 || rows > INT_MAX)
        return fail(CFZ_ERR_SHAPE, "rows = %lld", (long long)rows);
    const int pairs = g->rot_dim / 2;
    if (rows * pairs / 256 >= cfz::kBlockMaxGroups)
        return fail(CFZ_ERR_SHAPE, "a table of %lld angles (limit 2^31)", (long long)(rows * pairs));
    if (!positions && g->axes > 1)
        return fail(CFZ_ERR_NULL, "more than one axis needs positions");
    if (!aligned(positions, 4))
        return fail(CFZ_ERR_ALIGN, "positions must be 4-byte aligned");
    cfz::TableArgs a;
    memset(&a, 0, sizeof a);
    int at = 0;
    for (int j = 0; j < g->axes; ++j) {
        const double d = g->axis_dim[j];
        const double b = base ? g->base * pow(g->factor, d / (d - 2.0)) : g->base;
        if (!(b > 0.0) || !isfinite(b))
            return fail(CFZ_ERR_SHAPE, "base = %g, stretched by factor = %g", g->base, g->factor);
        for (int i = 0; i < g->axis_dim[j] / 2; ++i, ++at) {
            double speed = pow(b, -2.0 * i / d);
            if (g->scaling == CFZ_ROTATION_LINEAR)
                speed /= g->factor;
            if (parts) {
                const double n = g->trained * speed / 6.283185307179586476925;
                double k = (n - g->slow) / (g->fast - g->slow);
                k = k < 0.0 ? 0.0 : (k > 1.0 ? 1.0 : k);
                speed *= k + (1.0 - k) / g->factor;
            }
            a.speed[at] = speed;
            a.axis[at] = (uint8_t)j;
        }
    }
    if (rows == 0)
        return CFZ_OK;
    if (!cos || !sin)
        return fail(CFZ_ERR_NULL, "cos and sin are required");
    if (!aligned(cos, 16) || !aligned(sin, 16))
        return fail(CFZ_ERR_ALIGN, "cos and sin must be 16-byte aligned");
    a.pairs = pairs;
    a.axes = g->axes;
    a.rows = rows;
    a.positions = positions;
    a.amplitude = g->amplitude;
    a.cos = cos;
    a.sin = sin;
    return hip_status(cfz::launch_rotation_table(a, (hipStream_t)hip_stream), "table launch");
}

cfz_status cfz_rotate(int32_t count, const cfz_rotate_rows *tensors, cfz_kv8_dtype dtype,
                      int32_t head_dim, int64_t tokens, int32_t batch, const int32_t *offsets,
                      const int32_t *starts, const cfz_kv8_rotation *rotation, int32_t normed,
                      float eps, void *hip_stream)
{
    if (count < 1 || count > 4)
        return fail(CFZ_ERR_SHAPE, "count = %d tensors (1 .. 4)", count);
    if (!tensors)
        return fail(CFZ_ERR_NULL, "tensors is required");
    if (!is_dtype(dtype))
        return fail(CFZ_ERR_UNSUPPORTED, "dtype = %d", dtype);
    if (head_dim != 32 && head_dim != 64 && head_dim != 128 && head_dim != 256)
        return fail(CFZ_ERR_UNSUPPORTED, "head_dim = %d (supported: 32, 64, 128, 256)", head_dim);
    cfz::RotateArgs a;
    memset(&a, 0, sizeof a);
    CFZ_TRY(check_rows(tokens, batch, offsets, &a.rows));
    if (!offsets && batch != 1)
        return fail(CFZ_ERR_NULL, "%d sequences need offsets", batch);
    if (!aligned(starts, 4))
        return fail(CFZ_ERR_ALIGN, "starts must be 4-byte aligned");
    if (!rotation && !normed)
        return fail(CFZ_ERR_NULL, "neither a rotation nor a norm");
    if (normed && (!(eps >= 0.0f) || !isfinite(eps)))
        return fail(CFZ_ERR_SHAPE, "eps = %g must be finite and not negative", (double)eps);
    if (rotation) {
        if (rotation->rot_dim < 8 || rotation->rot_dim > head_dim || rotation->rot_dim % 8 != 0)
            return fail(CFZ_ERR_SHAPE, "rot_dim = %d (a multiple of 8, at most %d)",
                        rotation->rot_dim, head_dim);
        if (rotation->table_rows < 1 || rotation->table_rows > INT_MAX)
            return fail(CFZ_ERR_SHAPE, "table_rows = %lld", (long long)rotation->table_rows);
        if (!rotation->cos || !rotation->sin)
            return fail(CFZ_ERR_NULL, "the rotation's cos and sin are required");
        if (!aligned(rotation->cos, 16) || !aligned(rotation->sin, 16) ||
            !aligned(rotation->positions, 4))
            return fail(CFZ_ERR_ALIGN, "cos and sin must be 16-byte, positions 4-byte aligned");
        a.cos = rotation->cos;
        a.sin = rotation->sin;
        a.pos = rotation->positions;
        a.table_rows = rotation->table_rows;
        a.rot = rotation->rot_dim;
        a.interleaved = rotation->interleaved != 0;
    }
    a.log2lanes = head_dim == 32 ? 2 : (head_dim == 64 ? 3 : (head_dim == 128 ? 4 : 5));
    const int heads = (cfz::kRotateUnits * 64) >> a.log2lanes;  // a wave's
    for (int i = 0; i < count; ++i) {
        const cfz_rotate_rows &t = tensors[i];
        if (t.heads < 1 || t.heads > 1024)
            return fail(CFZ_ERR_SHAPE, "tensor %d: heads = %d", i, t.heads);
        CFZ_TRY(check_stride(t.x_stride, (int64_t)t.heads * head_dim, dtype, "x_stride"));
        CFZ_TRY(check_stride(t.out_stride, (int64_t)t.heads * head_dim, dtype, "out_stride"));
        if (t.weight && !normed)
            return fail(CFZ_ERR_UNSUPPORTED, "tensor %d: a weight without a norm", i);
        CFZ_TRY(check_vec(t.weight, t.weight_dtype, dtype, "weight"));
        if (!aligned(t.x, 16) || !aligned(t.out, 16))
            return fail(CFZ_ERR_ALIGN, "tensor %d: x and out must be 16-byte aligned", i);
        if (t.x && t.x == t.out && t.x_stride != t.out_stride)
            return fail(CFZ_ERR_SHAPE, "in place, the strides must be the same");
        a.t[i] = cfz::RotateRows{t.x,      t.out, t.weight, t.x_stride, t.out_stride,
                                 t.weight_dtype == CFZ_KV8_F32, t.heads, a.parts};
        a.parts += (t.heads + heads - 1) / heads;
    }
    a.count = count;
    a.dim = head_dim;
    a.starts = starts;
    a.normed = normed != 0;
    a.eps = eps;
    if (tokens == 0)
        return CFZ_OK;
    if (cfz::rotate_groups(a) >= cfz::kBlockMaxGroups)
        return fail(CFZ_ERR_SHAPE, "the call needs %lld work-groups (limit 2^23)",
                    (long long)cfz::rotate_groups(a));
    for (int i = 0; i < count; ++i)
        if (!a.t[i].x || !a.t[i].out)
            return fail(CFZ_ERR_NULL, "tensor %d: x and out are required", i);
    return hip_status(cfz::launch_rotate(a, dtype, (hipStream_t)hip_stream), "rotation launch");
}

size_t cfz_adapters_a_bytes(const cfz_adapters *adapters)
{
    cfz::AdapterArgs a;
    if (check_adapters(adapters, 0, 0, &a) != CFZ_OK)
        return 0;
    return (size_t)cfz::adapter_pieces(a) * 16 * a.adapters;
}

cfz_status cfz_adapters_put(const cfz_adapters *w, int32_t first, int32_t count, const void *rows,
                            void *hip_stream)
{
    cfz::AdapterArgs a;
    CFZ_TRY(check_adapters(w, 0, 0, &a));
    if (first < 0 || count < 0 || (int64_t)first + count > a.adapters)
        return fail(CFZ_ERR_SHAPE, "adapters %d .. %lld of %d", first, (long long)first + count - 1,
                    a.adapters);
    if (cfz::adapter_pieces(a) * count / 256 >= cfz::kBlockMaxGroups)
        return fail(CFZ_ERR_SHAPE, "more than 2^31 pieces of 16 bytes: fewer adapters a call");
    if (count == 0)
        return CFZ_OK;
    if (!w->a || !rows)
        return fail(CFZ_ERR_NULL, "a and rows are required");
    if (!aligned(w->a, 16) || !aligned(rows, 16))
        return fail(CFZ_ERR_ALIGN, "a and rows must be 16-byte aligned");
    a.a = w->a;
    return hip_status(cfz::launch_adapters_put(a, rows, first, count, (hipStream_t)hip_stream),
                      "adapter layout launch");
}

size_t cfz_adapters_workspace_bytes(const cfz_adapters *adapters, int64_t tokens, int32_t batch)
{
    cfz::AdapterArgs a;
    return check_adapters(adapters, tokens, batch, &a) == CFZ_OK ? adapters_bytes(a) : 0;
}

cfz_status cfz_adapters_add(const cfz_adapters *w, int64_t tokens, int32_t batch,
                            const int32_t *offsets, const int32_t *ids, int64_t max_rows,
                            const void *x, int64_t x_stride, const void *y, int64_t y_stride,
                            void *out, int64_t out_stride, int32_t y_dtype, void *workspace,
                            size_t ws_bytes, void *hip_stream)
{
    cfz::AdapterArgs a;
    CFZ_TRY(check_adapters(w, tokens, batch, &a));
    if (y_dtype != w->dtype && y_dtype != CFZ_KV8_F32)
        return fail(CFZ_ERR_UNSUPPORTED, "y_dtype = %d with dtype = %d", y_dtype, w->dtype);
    if (max_rows < 0 || max_rows > INT_MAX)
        return fail(CFZ_ERR_SHAPE, "max_rows = %lld", (long long)max_rows);
    CFZ_TRY(check_stride(x_stride, a.cols_in, w->dtype, "x_stride"));
    CFZ_TRY(check_stride(y_stride, a.cols_out, y_dtype, "y_stride"));
    CFZ_TRY(check_stride(out_stride, a.cols_out, y_dtype, "out_stride"));
    if (tokens == 0 || batch == 0 || max_rows == 0)
        return CFZ_OK;
    if (cfz::adapter_groups(a) >= cfz::kBlockMaxGroups)
        return fail(CFZ_ERR_SHAPE, "the call needs %lld work-groups (limit 2^23)",
                    (long long)cfz::adapter_groups(a));
    if (!w->a || !w->b || !offsets || !ids || !x || !y || !out)
        return fail(CFZ_ERR_NULL, "a, b, offsets, ids, x, y and out are required");
    if (!aligned(w->a, 16) || !aligned(w->b, 16) || !aligned(x, 16) || !aligned(y, 16) ||
        !aligned(out, 16))
        return fail(CFZ_ERR_ALIGN, "a, b, x, y and out must be 16-byte aligned");
    if (!aligned(offsets, 4) || !aligned(ids, 4) || !aligned(w->scale, 4))
        return fail(CFZ_ERR_ALIGN, "offsets, ids and scale must be 4-byte aligned");
    if (y == out && y_stride != out_stride)
        return fail(CFZ_ERR_SHAPE, "in place, the strides must be the same");
    const size_t need = adapters_bytes(a);
    if (!workspace || ws_bytes < need)
        return fail(CFZ_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed",
                    workspace ? ws_bytes : (size_t)0, need);
    if (!aligned(workspace, 256))
        return fail(CFZ_ERR_ALIGN, "workspace must be 256-byte aligned");
    a.rows.off = offsets;
    a.max_rows = max_rows;
    a.ids = ids;
    a.a = w->a;
    a.b = w->b;
    a.scale = w->scale;
    a.x = x;
    a.y = y;
    a.out = out;
    a.xs = x_stride;
    a.ys = y_stride;
    a.os = out_stride;
    a.hi = (uint16_t *)workspace;
    a.lo = a.hi + tokens * a.down;
    a.back = (float *)(a.lo + tokens * a.down);
    return hip_status(cfz::launch_adapters(a, w->dtype == CFZ_KV8_F16, y_dtype == CFZ_KV8_F32,
                                           (hipStream_t)hip_stream),
                      "adapter launch");
}

}  // extern "C"
