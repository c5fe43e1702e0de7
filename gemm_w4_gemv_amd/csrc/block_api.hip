// C ABI of the operators around a block's products (w4_block.h): host-side
// validation and dispatch.  As in w4_api.hip, every check runs before the first
// HIP call.  An array without elements may have no address.
#include <math.h>

#include "block.hpp"
#include "w4_check.hpp"

namespace {

using w4::aligned;
using w4::any_overlap;
using w4::fail;
using w4::hip_fail;
using w4::overlap;
using w4::Range;
using w4::range;
using w4::rows_range;

constexpr int kMaxRows = 1 << 21;       // of a norm
constexpr int kMaxWide = 1 << 20;       // values of an expert's row
constexpr int64_t kMaxChoices = 1 << 23;

// Rows that are given (p) must have a stride that holds them.
bool stride_bad(const void* p, int64_t s, int64_t wide) { return p && (s < wide || s % 8 || s > (1ll << 40)); }

w4_status check_norm(const char* fn, const w4_norm_args* args) {
    if (!args) return fail(W4_ERR_NULL, "%s: args must not be NULL", fn);
    const w4_norm_args& a = *args;
    if (a.T < 0 || a.T > kMaxRows) return fail(W4_ERR_SHAPE, "%s: T = %d must lie in [0, %d]", fn, a.T, kMaxRows);
    if (a.D < 8 || a.D > W4_NORM_MAX_DIM || a.D % 8)
        return fail(W4_ERR_SHAPE, "%s: D = %d is no multiple of 8 in [8, %d]", fn, a.D, W4_NORM_MAX_DIM);
    if (!(a.eps >= 0.0f) || !isfinite(a.eps) || !isfinite(a.weight_add) || !isfinite(a.residual_scale) || !isfinite(a.branch_scale))
        return fail(W4_ERR_ARG, "%s: eps must be finite and not negative, weight_add and the scales finite", fn);
    if (a.T > 0 && !a.h) return fail(W4_ERR_NULL, "%s: h must not be NULL", fn);
    if (a.T > 0 && !a.y && (a.y_weight || a.gate)) return fail(W4_ERR_ARG, "%s: y_weight and gate go with y", fn);
    if (stride_bad(a.h, a.h_stride, a.D) || stride_bad(a.y, a.y_stride, a.D) ||
        (a.gate_stride != 0 && stride_bad(a.gate, a.gate_stride, a.D)))
        return fail(W4_ERR_ARG, "%s: row strides must be multiples of 8, at least D", fn);
    for (const void* p : {a.h, a.y, a.y_weight, a.z_weight, a.gate})
        if (!aligned(p, 16)) return fail(W4_ERR_ALIGN, "%s: arrays must be 16-byte aligned", fn);
    return W4_OK;
}

struct NormRanges {
    Range h, y, wy, wz, gate;
};
NormRanges ranges_of(const w4_norm_args& a) {
    const size_t wide = (size_t)a.D * 2;
    return {rows_range(a.h, a.T, a.h_stride, a.D, a.h_f32 ? 4 : 2), rows_range(a.y, a.T, a.y_stride, a.D),
            range(a.y_weight, a.y_weight ? wide : 0), range(a.z_weight, a.z_weight ? wide : 0),
            rows_range(a.gate, a.gate_stride ? a.T : 1, a.gate_stride, a.D)};
}

bool same(const void* x, int64_t xs, const void* y, int64_t ys) { return x && x == y && xs == ys; }

w4_status check_choices(const char* fn, int T, int top) {
    if (T < 0 || top < 1 || top > W4_MOE_MAX_TOP)
        return fail(W4_ERR_SHAPE, "%s: T = %d, top = %d (1 to %d choices)", fn, T, top, W4_MOE_MAX_TOP);
    if ((int64_t)T * top > kMaxChoices) return fail(W4_ERR_SHAPE, "%s: %d tokens of %d choices are too many for one call", fn, T, top);
    return W4_OK;
}

w4_status check_rows(const char* fn, int R, int N) {
    if (R < 0) return fail(W4_ERR_SHAPE, "%s: R = %d is negative", fn, R);
    if (N < 8 || N > kMaxWide || N % 8) return fail(W4_ERR_SHAPE, "%s: rows of %d values (a multiple of 8 in [8, %d])", fn, N, kMaxWide);
    return W4_OK;
}

}  // namespace

extern "C" {

W4_API w4_status w4_block_norm(const w4_norm_args* args, void* stream) {
    const char* fn = "w4_block_norm";
    const w4_status st = check_norm(fn, args);
    if (st != W4_OK) return st;
    const w4_norm_args& a = *args;
    if (a.T > 0 && !a.y && a.h_out) return fail(W4_ERR_ARG, "%s: h_out goes with y", fn);
    if (a.T > 0 && !a.h_out && !a.z) return fail(W4_ERR_NULL, "%s: h_out and z must not both be NULL", fn);
    if (stride_bad(a.h_out, a.h_out_stride, a.D) || stride_bad(a.z, a.z_stride, a.D))
        return fail(W4_ERR_ARG, "%s: row strides must be multiples of 8, at least D", fn);
    if (!aligned(a.h_out, 16) || !aligned(a.z, 16)) return fail(W4_ERR_ALIGN, "%s: arrays must be 16-byte aligned", fn);
    const NormRanges in = ranges_of(a);
    const Range ho = rows_range(a.h_out, a.T, a.h_out_stride, a.D, a.h_f32 ? 4 : 2), z = rows_range(a.z, a.T, a.z_stride, a.D);
    if (any_overlap({ho, z}, {in.wy, in.wz, in.gate}) || overlap(ho, z) || overlap(ho, in.y) || overlap(z, in.h) ||
        (overlap(ho, in.h) && !same(a.h, a.h_stride, a.h_out, a.h_out_stride)) ||
        (overlap(z, in.y) && !same(a.y, a.y_stride, a.z, a.z_stride)))
        return fail(W4_ERR_ALIAS, "%s: an output overlaps an input or the other output", fn);
    if (a.T == 0) return W4_OK;
    const hipError_t err = w4::launch_block_norm(a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? W4_OK : hip_fail(err, fn);
}

W4_API size_t w4_block_norm_grad_workspace_bytes(int T, int D) {
    if (T <= 0 || T > kMaxRows || D < 8 || D > W4_NORM_MAX_DIM) return 0;
    return w4::block_norm_grad_workspace_bytes(T, D);
}

W4_API w4_status w4_block_norm_grad(const w4_norm_args* args, const w4_norm_grad_args* grad, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    const char* fn = "w4_block_norm_grad";
    const w4_status st = check_norm(fn, args);
    if (st != W4_OK) return st;
    if (!grad) return fail(W4_ERR_NULL, "%s: grad must not be NULL", fn);
    const w4_norm_args& a = *args;
    const w4_norm_grad_args& g = *grad;
    if (a.T > 0 && !g.dh_out && !g.dz) return fail(W4_ERR_NULL, "%s: dh_out and dz must not both be NULL", fn);
    if (!g.dh && !g.dy && !g.d_y_weight && !g.d_z_weight && !g.d_gate && a.T > 0)
        return fail(W4_ERR_NULL, "%s: no gradient is asked for", fn);
    if ((g.d_y_weight && !a.y_weight) || (g.d_z_weight && !a.z_weight) || (g.d_gate && !a.gate) || (a.T > 0 && g.dy && !a.y))
        return fail(W4_ERR_ARG, "%s: a gradient is asked for of an input that is not given", fn);
    const bool shared_gate = a.gate && a.gate_stride == 0;
    if (stride_bad(g.dh_out, g.dh_out_stride, a.D) || stride_bad(g.dz, g.dz_stride, a.D) || stride_bad(g.dh, g.dh_stride, a.D) ||
        stride_bad(g.dy, g.dy_stride, a.D) || (!shared_gate && stride_bad(g.d_gate, g.d_gate_stride, a.D)))
        return fail(W4_ERR_ARG, "%s: row strides must be multiples of 8, at least D", fn);
    for (const void* p : {g.dh_out, g.dz, (const void*)g.dh, (const void*)g.dy, (const void*)g.d_y_weight, (const void*)g.d_z_weight,
                          (const void*)g.d_gate})
        if (!aligned(p, 16)) return fail(W4_ERR_ALIGN, "%s: arrays must be 16-byte aligned", fn);
    size_t need = 0;
    if (g.d_y_weight || g.d_z_weight || (g.d_gate && shared_gate)) need = w4_block_norm_grad_workspace_bytes(a.T, a.D);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(W4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given%s", fn, need, workspace_bytes,
                        workspace ? "" : " (NULL)");
        if (!aligned(workspace, 16)) return fail(W4_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
    }
    const size_t hb = a.h_f32 ? 4 : 2;
    const NormRanges in = ranges_of(a);
    const Range dho = rows_range(g.dh_out, a.T, g.dh_out_stride, a.D, hb), dz = rows_range(g.dz, a.T, g.dz_stride, a.D),
                dh = rows_range(g.dh, a.T, g.dh_stride, a.D, hb), dy = rows_range(g.dy, a.T, g.dy_stride, a.D),
                sy = range(g.d_y_weight, g.d_y_weight ? (size_t)a.D * 4 : 0),
                sz = range(g.d_z_weight, g.d_z_weight ? (size_t)a.D * 4 : 0),
                dg = shared_gate ? range(g.d_gate, g.d_gate ? (size_t)a.D * 4 : 0)
                                 : rows_range(g.d_gate, a.T, g.d_gate_stride, a.D),
                w = range(workspace, need);
    if (any_overlap({dh, dy, sy, sz, dg, w}, {in.h, in.y, in.wy, in.wz, in.gate}) || any_overlap({dh, dy, sy, sz, dg, w}) ||
        any_overlap({sy, sz, dg, w}, {dho, dz}) || overlap(dh, dz) || overlap(dy, dho) ||
        (overlap(dh, dho) && !same(g.dh, g.dh_stride, g.dh_out, g.dh_out_stride)) ||
        (overlap(dy, dz) && !same(g.dy, g.dy_stride, g.dz, g.dz_stride)))
        return fail(W4_ERR_ALIAS, "%s: an output or the workspace overlaps an input or another output", fn);
    const hipError_t err = w4::launch_block_norm_grad(a, g, workspace, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? W4_OK : hip_fail(err, fn);
}

W4_API size_t w4_moe_sort_workspace_bytes(int T, int top, int num_experts) {
    if (T <= 0 || top < 1 || top > W4_MOE_MAX_TOP || (int64_t)T * top > kMaxChoices || num_experts < 1 ||
        num_experts > W4_MOE_SORT_MAX_EXPERTS)
        return 0;
    return w4::moe_sort_workspace_bytes(T, top, num_experts);
}

W4_API w4_status w4_moe_sort(const w4_moe_sort_args* args, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "w4_moe_sort";
    if (!args) return fail(W4_ERR_NULL, "%s: args must not be NULL", fn);
    const w4_moe_sort_args& a = *args;
    w4_status st = check_choices(fn, a.T, a.top);
    if (st != W4_OK) return st;
    if (a.num_experts < 1 || a.num_experts > W4_MOE_SORT_MAX_EXPERTS)
        return fail(W4_ERR_SHAPE, "%s: num_experts = %d must lie in [1, %d]", fn, a.num_experts, W4_MOE_SORT_MAX_EXPERTS);
    if (a.capacity < 0) return fail(W4_ERR_ARG, "%s: capacity = %d is negative", fn, a.capacity);
    if (!a.row_start || (a.T > 0 && (!a.experts || !a.row_of)))
        return fail(W4_ERR_NULL, "%s: experts, row_start and row_of must not be NULL", fn);
    const bool moved = a.T > 0 && (a.x || a.rows);
    if (moved) {
        st = check_rows(fn, a.R, a.D);
        if (st != W4_OK) return st;
        if (!a.x || (!a.rows && a.R > 0)) return fail(W4_ERR_NULL, "%s: x and rows go together", fn);
        if (stride_bad(a.x, a.x_stride, a.D) || stride_bad(a.rows, a.rows_stride, a.D))
            return fail(W4_ERR_ARG, "%s: row strides must be multiples of 8, at least D", fn);
        if (!aligned(a.x, 16) || !aligned(a.rows, 16)) return fail(W4_ERR_ALIGN, "%s: x and rows must be 16-byte aligned", fn);
    }
    for (const int32_t* p : {a.experts, (const int32_t*)a.row_start, (const int32_t*)a.row_of, (const int32_t*)a.source})
        if (!aligned(p, 4)) return fail(W4_ERR_ALIGN, "%s: tables must be 4-byte aligned", fn);
    const size_t need = w4_moe_sort_workspace_bytes(a.T, a.top, a.num_experts);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(W4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given%s", fn, need, workspace_bytes,
                        workspace ? "" : " (NULL)");
        if (!aligned(workspace, 16)) return fail(W4_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
    }
    const size_t n4 = (size_t)a.T * a.top * 4;
    const Range ids = range(a.experts, n4), rs = range(a.row_start, ((size_t)a.num_experts + 1) * 4), ro = range(a.row_of, n4),
                so = range(a.source, a.source ? n4 : 0), w = range(workspace, need),
                x = moved ? rows_range(a.x, a.T, a.x_stride, a.D) : Range{}, r = moved ? rows_range(a.rows, a.R, a.rows_stride, a.D) : Range{};
    if (any_overlap({rs, ro, so, r, w}, {ids, x}) || any_overlap({rs, ro, so, r, w}))
        return fail(W4_ERR_ALIAS, "%s: an output or the workspace overlaps an input or another output", fn);
    const hipError_t err = w4::launch_moe_sort(a, workspace, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? W4_OK : hip_fail(err, fn);
}

W4_API w4_status w4_moe_combine(const w4_moe_combine_args* args, void* stream) {
    const char* fn = "w4_moe_combine";
    if (!args) return fail(W4_ERR_NULL, "%s: args must not be NULL", fn);
    const w4_moe_combine_args& a = *args;
    w4_status st = check_choices(fn, a.T, a.top);
    if (st == W4_OK) st = check_rows(fn, a.R, a.N);
    if (st != W4_OK) return st;
    if (a.T > 0 && (!a.out || (a.R > 0 && !a.y))) return fail(W4_ERR_NULL, "%s: y and out must not be NULL", fn);
    if (stride_bad(a.y, a.y_stride, a.N) || stride_bad(a.add, a.add_stride, a.N) || stride_bad(a.out, a.out_stride, a.N))
        return fail(W4_ERR_ARG, "%s: row strides must be multiples of 8, at least N", fn);
    if (!aligned(a.y, 16) || !aligned(a.add, 16) || !aligned(a.out, 16))
        return fail(W4_ERR_ALIGN, "%s: y, add and out must be 16-byte aligned", fn);
    if (!aligned(a.row_of, 4) || !aligned(a.weights, 4)) return fail(W4_ERR_ALIGN, "%s: row_of and weights must be 4-byte aligned", fn);
    const size_t n4 = (size_t)a.T * a.top * 4;
    const Range y = rows_range(a.y, a.R, a.y_stride, a.N), add = rows_range(a.add, a.T, a.add_stride, a.N),
                out = rows_range(a.out, a.T, a.out_stride, a.N);
    if (any_overlap({out}, {y, range(a.row_of, a.row_of ? n4 : 0), range(a.weights, a.weights ? n4 : 0)}) ||
        (overlap(out, add) && !same(a.add, a.add_stride, a.out, a.out_stride)))
        return fail(W4_ERR_ALIAS, "%s: out overlaps an input", fn);
    if (a.T == 0) return W4_OK;
    const hipError_t err = w4::launch_moe_combine(a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? W4_OK : hip_fail(err, fn);
}

W4_API w4_status w4_moe_combine_grad(const w4_moe_combine_grad_args* args, void* stream) {
    const char* fn = "w4_moe_combine_grad";
    if (!args) return fail(W4_ERR_NULL, "%s: args must not be NULL", fn);
    const w4_moe_combine_grad_args& a = *args;
    w4_status st = check_choices(fn, a.T, a.top);
    if (st == W4_OK) st = check_rows(fn, a.R, a.N);
    if (st != W4_OK) return st;
    if (a.T > 0 && (!a.dout || (a.dweights && a.R > 0 && !a.y))) return fail(W4_ERR_NULL, "%s: dout and y must not be NULL", fn);
    if (a.T > 0 && a.R > 0 && !a.dy && !a.dweights) return fail(W4_ERR_NULL, "%s: dy and dweights must not both be NULL", fn);
    if (stride_bad(a.dout, a.dout_stride, a.N) || stride_bad(a.y, a.y_stride, a.N) || stride_bad(a.dy, a.dy_stride, a.N))
        return fail(W4_ERR_ARG, "%s: row strides must be multiples of 8, at least N", fn);
    if (!aligned(a.dout, 16) || !aligned(a.y, 16) || !aligned(a.dy, 16))
        return fail(W4_ERR_ALIGN, "%s: dout, y and dy must be 16-byte aligned", fn);
    if (!aligned(a.row_of, 4) || !aligned(a.weights, 4) || !aligned(a.dweights, 4))
        return fail(W4_ERR_ALIGN, "%s: row_of, weights and dweights must be 4-byte aligned", fn);
    const size_t n4 = (size_t)a.T * a.top * 4;
    const Range g = rows_range(a.dout, a.T, a.dout_stride, a.N), y = rows_range(a.y, a.R, a.y_stride, a.N),
                dy = rows_range(a.dy, a.R, a.dy_stride, a.N), dw = range(a.dweights, a.dweights ? n4 : 0),
                ro = range(a.row_of, a.row_of ? n4 : 0), w = range(a.weights, a.weights ? n4 : 0);
    if (any_overlap({dy, dw}, {g, ro, w}) || overlap(dy, dw) || overlap(dw, y) ||
        (overlap(dy, y) && !same(a.y, a.y_stride, a.dy, a.dy_stride)))
        return fail(W4_ERR_ALIAS, "%s: an output overlaps an input or the other output", fn);
    if (a.T == 0) return W4_OK;
    const hipError_t err = w4::launch_moe_combine_grad(a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? W4_OK : hip_fail(err, fn);
}

}  // extern "C"
