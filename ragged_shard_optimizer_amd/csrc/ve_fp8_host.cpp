// ve_fp8_host.cpp -- C entry points on matrices in 8-bit floating point:
// argument checks, workspace sizing and launches (kernels in ve_fp8_pack.hip
// and ve_fp8.hip).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ve.h"
#include "ve_checks.h"
#include "ve_fp8.h"
#include "ve_fp8_pack.h"
#include "ve_fp8_product.h"

using namespace ve;

namespace {

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

ve_status check_groups(int64_t rows, int64_t cols, int32_t groups) {
    if (rows < 0 || cols < 1) return fail(VE_ERR_INVALID_ARG, "shape %lld x %lld", (long long)rows, (long long)cols);
    if (groups < 1 || groups > 65536) return fail(VE_ERR_INVALID_ARG, "groups %d outside [1, 65536]", groups);
    if (rows > kMaxDim - 128 || cols > kMaxDim - 128) return fail(VE_ERR_UNSUPPORTED, "a dimension of 2^31 or more");
    return VE_OK;
}

ve_status check_group_strides(const ve_fp8& q, int64_t rows, int64_t cols, int32_t groups, int64_t codes, int64_t scales,
                              const char* name) {
    if (groups == 1) return VE_OK;
    if (codes < (rows - 1) * q.ld_codes + cols ||
        scales < (scale_rows(cols) - 1) * q.ld_scales + (rows + q.block_rows - 1) / q.block_rows)
        return fail(VE_ERR_INVALID_ARG, "%s: group stride smaller than a group", name);
    if (codes % 16 || scales % 4) return fail(VE_ERR_INVALID_ARG, "%s: groups must start on 16 bytes, scales on 4", name);
    return VE_OK;
}

// Tiles of 128 x 128 of every launch over the matrices fit one grid.
bool tiles_fit(int64_t rows, int64_t cols, int64_t extra, int64_t times) {
    return (rows + 127) / 128 + extra <= kMaxWorkgroups / ((cols + 127) / 128) / times;
}

// E4M3 only, where the operand is the second of a product.
ve_status check_e4m3(const ve_fp8& q, const char* name) {
    return q.format == VE_E4M3 ? VE_OK : fail(VE_ERR_INVALID_ARG, "%s: must be E4M3", name);
}

ve_status check_pitch(const ve_fp8& q, const char* name) {
    if (q.ld_codes > int64_t(1) << 22 || q.ld_scales > kMaxDim)
        return fail(VE_ERR_UNSUPPORTED, "%s: rows more than 2^22 bytes apart", name);
    return VE_OK;
}

// dw's operands, whose rows are as long as the groups' runs together: the rows
// of a tile within 32-bit byte offsets of its first.
ve_status check_pitch_t(const ve_fp8& q, const char* name) {
    if (q.ld_codes >= kFp8Pitch128 || q.ld_scales > kMaxDim)
        return fail(VE_ERR_UNSUPPORTED, "%s: rows 2^24 bytes apart or more", name);
    return VE_OK;
}

ve_status check_forward(const ve_fp8_linear_forward_args& a) {
    ve_status st = check_shape(a.tokens, a.in_features, a.out_features, a.groups, a.offsets, a.activation);
    if (st != VE_OK) return st;
    const int64_t T = a.tokens, K = a.in_features, N = a.out_features;
    if ((T > 0 && (st = check_fp8(a.x, T, K, 1, "x")) != VE_OK) || (st = check_fp8(a.w, N, K, 128, "w")) != VE_OK ||
        (st = check_e4m3(a.w, "w")) != VE_OK ||
        (st = check_group_strides(a.w, N, K, a.groups, a.w_codes_group, a.w_scales_group, "w")) != VE_OK)
        return st;
    if (T > 0 && !a.y) return fail(VE_ERR_INVALID_ARG, "y is NULL");
    if (a.ldy < N || (a.residual && a.ldr < N) || (a.z && a.ldz < N))
        return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (a.groups > 1 && a.bias && a.bias_group < N) return fail(VE_ERR_INVALID_ARG, "group stride smaller than a group");
    if ((st = check_pitch(a.x, "x")) != VE_OK || (st = check_pitch(a.w, "w")) != VE_OK) return st;
    if (!launchable(T, N, a.groups, 1)) return fail(VE_ERR_UNSUPPORTED, "product too large for one launch");
    return VE_OK;
}

// C = A B^T over tokens, B grouped.
Fp8Args rows_product(const ve_fp8& A, const ve_fp8& B, int64_t codes_group, int64_t scales_group, int64_t T, int64_t N,
                     int64_t K, int32_t groups, const int64_t* offsets) {
    Fp8Args g{};
    g.A = (const uint16_t*)A.codes; g.lda = A.ld_codes / 2;
    g.B = (const uint16_t*)B.codes; g.ldb = B.ld_codes / 2; g.b_group = groups > 1 ? codes_group / 2 : 0;
    g.sa = A.scales; g.ld_sa = A.ld_scales; g.sa_rows = up(T, 4);
    g.sb = B.scales; g.ld_sb = B.ld_scales; g.sb_group = groups > 1 ? scales_group : 0; g.sb_rows = up((N + 127) / 128, 4);
    g.T = T; g.N = N; g.K = up(K, 16) / 2;
    g.E = groups; g.offsets = offsets; g.format = A.format;
    return g;
}

Fp8Args forward_product(const ve_fp8_linear_forward_args& a) {
    Fp8Args g = rows_product(a.x, a.w, a.w_codes_group, a.w_scales_group, a.tokens, a.out_features, a.in_features, a.groups,
                             a.offsets);
    g.bias = a.bias; g.bias_group = a.groups > 1 ? a.bias_group : 0;
    g.res = a.residual; g.ldr = a.ldr;
    g.y = a.y; g.ldy = a.ldy;
    g.z = a.z; g.ldz = a.ldz;
    g.act = a.activation;
    g.vec_bias = vec16(a.bias, g.bias_group);
    g.vec_res = vec16(a.residual, a.ldr);
    g.vec_y = vec16(a.y, a.ldy);
    g.vec_z = vec16(a.z, a.ldz);
    return g;
}

ve_status check_backward(const ve_fp8_linear_backward_args& a) {
    ve_status st = check_shape(a.tokens, a.in_features, a.out_features, a.groups, a.offsets, VE_ACT_NONE);
    if (st != VE_OK) return st;
    const int64_t T = a.tokens, K = a.in_features, N = a.out_features, C = ve_fp8_columns(T, a.groups);
    if (a.dx) {
        if ((T > 0 && (st = check_fp8(a.dy, T, N, 1, "dy")) != VE_OK) || (st = check_fp8(a.w_t, K, N, 128, "w_t")) != VE_OK ||
            (st = check_e4m3(a.w_t, "w_t")) != VE_OK ||
            (st = check_group_strides(a.w_t, K, N, a.groups, a.w_codes_group, a.w_scales_group, "w_t")) != VE_OK ||
            (st = check_pitch(a.dy, "dy")) != VE_OK || (st = check_pitch(a.w_t, "w_t")) != VE_OK)
            return st;
        if (a.lddx < K || (a.dx_add && a.ld_add < K))
            return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    }
    if (a.dw) {
        if (T > 0 && ((st = check_fp8(a.dy_t, N, C, 1, "dy_t")) != VE_OK || (st = check_fp8(a.x_t, K, C, 1, "x_t")) != VE_OK ||
                      (st = check_e4m3(a.x_t, "x_t")) != VE_OK || (st = check_pitch_t(a.dy_t, "dy_t")) != VE_OK ||
                      (st = check_pitch_t(a.x_t, "x_t")) != VE_OK))
            return st;
        if (a.lddw < K) return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
        if (a.groups > 1 && a.dw_group < (N - 1) * a.lddw + K)
            return fail(VE_ERR_INVALID_ARG, "group stride smaller than a group");
    }
    if ((a.dx && !launchable(T, K, a.groups, 1)) || (a.dw && !launchable(N, K, 0, a.groups)))
        return fail(VE_ERR_UNSUPPORTED, "product too large for one launch");
    return VE_OK;
}

Fp8Args dx_product(const ve_fp8_linear_backward_args& a) {
    Fp8Args g = rows_product(a.dy, a.w_t, a.w_codes_group, a.w_scales_group, a.tokens, a.in_features, a.out_features, a.groups,
                             a.offsets);
    g.res = a.dx_add; g.ldr = a.ld_add;
    g.y = a.dx; g.ldy = a.lddx;
    g.vec_res = vec16(a.dx_add, a.ld_add);
    g.vec_y = vec16(a.dx, a.lddx);
    return g;
}

Fp8Args dw_product(const ve_fp8_linear_backward_args& a) {
    Fp8Args g{};
    g.A = (const uint16_t*)a.dy_t.codes; g.lda = a.dy_t.ld_codes / 2;
    g.B = (const uint16_t*)a.x_t.codes; g.ldb = a.x_t.ld_codes / 2;
    g.sa = a.dy_t.scales; g.ld_sa = a.dy_t.ld_scales; g.sa_rows = up(a.out_features, 4);
    g.sb = a.x_t.scales; g.ld_sb = a.x_t.ld_scales; g.sb_rows = up(a.in_features, 4);
    g.T = a.offsets ? a.tokens : up(a.tokens, 128) / 2;
    g.M = a.out_features; g.N = a.in_features; g.K = ve_fp8_columns(a.tokens, a.groups) / 2;
    g.E = a.groups; g.offsets = a.offsets; g.format = a.dy_t.format;
    g.dw = a.dw; g.lddw = a.lddw; g.dw_group = a.groups > 1 ? a.dw_group : 0;
    g.wide = a.grad_fp32 != 0; g.accumulate = a.accumulate != 0;
    g.vec_dw = aligned(a.dw, 16) && a.lddw % 8 == 0 && g.dw_group % 8 == 0;
    return g;
}

struct Backward { Fp8Args dx, dw; LinPlan pdx, pdw; int64_t total; };
void plan_backward(const ve_fp8_linear_backward_args& a, Backward& b) {
    b.pdx = b.pdw = LinPlan{kPath128, 1, 0, 0};
    if (a.dx && a.tokens > 0) {
        b.dx = dx_product(a);
        b.pdx = plan_fp8(b.dx, kLinFwd);
    }
    if (a.dw) {
        b.dw = dw_product(a);
        b.pdw = plan_fp8(b.dw, kLinDw);
    }
    b.total = round256(std::max(b.pdx.partial_bytes, b.pdw.partial_bytes));
}

ve_status check_forward_apart(const ve_fp8_linear_forward_args& a, const void* ws, int64_t ws_bytes) {
    const int64_t T = a.tokens, K = a.in_features, N = a.out_features, E = a.groups;
    const bool same = a.residual == a.y && (a.ldr == a.ldy || T == 1);
    return check_apart({matrix_span("y", a.y, T, N, a.ldy, 2), matrix_span("z", a.z, T, N, a.ldz, 2),
                        matrix_span("workspace", ws_bytes ? ws : nullptr, 1, ws_bytes, ws_bytes, 1)},
                       {fp8_codes_span("x", a.x, T, K), fp8_scales_span("x's scales", a.x, T, K),
                        fp8_codes_span("w", a.w, E, N, K, a.w_codes_group),
                        fp8_scales_span("w's scales", a.w, E, N, K, a.w_scales_group),
                        group_span("bias", a.bias, E, 1, N, N, a.bias_group, 2),
                        matrix_span("residual", same ? nullptr : a.residual, T, N, a.ldr, 2),
                        matrix_span("offsets", a.offsets, 1, E + 1, E + 1, 8)});
}

ve_status check_backward_apart(const ve_fp8_linear_backward_args& a, const void* ws, int64_t ws_bytes) {
    const int64_t T = a.tokens, K = a.in_features, N = a.out_features, E = a.groups, C = ve_fp8_columns(T, a.groups);
    const bool same = a.dx_add == a.dx && (a.ld_add == a.lddx || T == 1);
    ve_fp8 none{};
    none.block_rows = 1;
    const bool some = T > 0;
    const ve_fp8 &dy = a.dx && some ? a.dy : none, &w = a.dx ? a.w_t : none, &dy_t = a.dw && some ? a.dy_t : none,
                 &x_t = a.dw && some ? a.x_t : none;
    return check_apart({matrix_span("dx", a.dx, T, K, a.lddx, 2),
                        group_span("dw", a.dw, E, N, K, a.lddw, a.dw_group, a.grad_fp32 ? 4 : 2),
                        matrix_span("workspace", ws_bytes ? ws : nullptr, 1, ws_bytes, ws_bytes, 1)},
                       {fp8_codes_span("dy", dy, T, N), fp8_scales_span("dy's scales", dy, T, N),
                        fp8_codes_span("w_t", w, E, K, N, a.w_codes_group),
                        fp8_scales_span("w_t's scales", w, E, K, N, a.w_scales_group),
                        fp8_codes_span("dy_t", dy_t, N, C), fp8_scales_span("dy_t's scales", dy_t, N, C),
                        fp8_codes_span("x_t", x_t, K, C), fp8_scales_span("x_t's scales", x_t, K, C),
                        matrix_span("dx_add", a.dx && !same ? a.dx_add : nullptr, T, K, a.ld_add, 2),
                        matrix_span("offsets", a.offsets, 1, E + 1, E + 1, 8)});
}

}  // namespace

extern "C" {

int64_t ve_fp8_columns(int64_t rows, int32_t groups) {
    if (rows <= 0 || groups <= 0) return 0;
    return (rows + 127 * std::min<int64_t>(groups, rows)) / 128 * 128;
}

ve_status ve_fp8_pack(const ve_fp8_pack_args* p, void* stream) {
    if (!p) return fail(VE_ERR_INVALID_ARG, "arguments are NULL");
    const ve_fp8_pack_args& a = *p;
    ve_status st = check_groups(a.rows, a.cols, a.groups);
    if (st != VE_OK) return st;
    if (!a.offsets && a.groups != 1) return fail(VE_ERR_INVALID_ARG, "%d groups need offsets", a.groups);
    if (a.activation < VE_ACT_NONE || a.activation > VE_ACT_SILU)
        return fail(VE_ERR_INVALID_ARG, "unknown activation %d", a.activation);
    const bool act = a.activation != VE_ACT_NONE;
    if (a.ldx < a.cols || (act && a.ldz < a.cols)) return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (a.rows == 0 || (!a.out.codes && !a.out_t.codes)) return VE_OK;
    const int64_t C = ve_fp8_columns(a.rows, a.groups);
    if (!a.x || (act && !a.z)) return fail(VE_ERR_INVALID_ARG, "x or z is NULL");
    if (a.out.codes && (st = check_fp8(a.out, a.rows, a.cols, 1, "out")) != VE_OK) return st;
    if (a.out_t.codes && (st = check_fp8(a.out_t, a.cols, C, 1, "out_t")) != VE_OK) return st;
    if (a.out.codes && a.out_t.codes && a.out.format != a.out_t.format)
        return fail(VE_ERR_INVALID_ARG, "out and out_t differ in format");
    if (!tiles_fit(a.rows, a.cols, a.groups, 1)) return fail(VE_ERR_UNSUPPORTED, "matrix too large for one launch");
    st = check_apart({fp8_codes_span("out", a.out, a.rows, a.cols), fp8_scales_span("out's scales", a.out, a.rows, a.cols),
                      fp8_codes_span("out_t", a.out_t, a.cols, C), fp8_scales_span("out_t's scales", a.out_t, a.cols, C)},
                     {matrix_span("x", a.x, a.rows, a.cols, a.ldx, 2),
                      matrix_span("z", act ? a.z : nullptr, a.rows, a.cols, a.ldz, 2),
                      matrix_span("offsets", a.offsets, 1, a.groups + 1, a.groups + 1, 8)});
    if (st != VE_OK) return st;
    Fp8PackArgs g{};
    g.rows = a.rows; g.cols = a.cols; g.groups = a.groups; g.act = a.activation; g.offsets = a.offsets;
    g.x = a.x; g.ldx = a.ldx; g.z = a.z; g.ldz = a.ldz;
    g.vec = vec16(a.x, a.ldx); g.vec_z = vec16(a.z, a.ldz);
    g.out = a.out; g.out_t = a.out_t;
    g.format = a.out.codes ? a.out.format : a.out_t.format;
    (void)hipGetLastError();
    return status_of(launch_fp8_pack(g, (hipStream_t)stream), "fp8 pack");
}

ve_status ve_fp8_pack_weight(const ve_fp8_pack_weight_args* p, void* stream) {
    if (!p) return fail(VE_ERR_INVALID_ARG, "arguments are NULL");
    const ve_fp8_pack_weight_args& a = *p;
    ve_status st = check_groups(a.rows, a.cols, a.groups);
    if (st != VE_OK) return st;
    if (a.rows < 1) return fail(VE_ERR_INVALID_ARG, "no rows");
    if (!a.w) return fail(VE_ERR_INVALID_ARG, "w is NULL");
    if (a.ldw < a.cols) return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (a.groups > 1 && a.w_group < (a.rows - 1) * a.ldw + a.cols)
        return fail(VE_ERR_INVALID_ARG, "group stride smaller than a group");
    const int64_t E = a.groups, R = a.rows, C = a.cols;
    if (a.out.codes && ((st = check_fp8(a.out, R, C, 128, "out")) != VE_OK ||
                        (st = check_group_strides(a.out, R, C, a.groups, a.out_codes_group, a.out_scales_group, "out")) != VE_OK))
        return st;
    if (a.out_t.codes &&
        ((st = check_fp8(a.out_t, C, R, 128, "out_t")) != VE_OK ||
         (st = check_group_strides(a.out_t, C, R, a.groups, a.out_t_codes_group, a.out_t_scales_group, "out_t")) != VE_OK))
        return st;
    if (!a.out.codes && !a.out_t.codes) return VE_OK;
    if (a.out.codes && a.out_t.codes && a.out.format != a.out_t.format)
        return fail(VE_ERR_INVALID_ARG, "out and out_t differ in format");
    if (!tiles_fit(R, C, 0, E)) return fail(VE_ERR_UNSUPPORTED, "matrices too large for one launch");
    st = check_apart({fp8_codes_span("out", a.out, E, R, C, a.out_codes_group),
                      fp8_scales_span("out's scales", a.out, E, R, C, a.out_scales_group),
                      fp8_codes_span("out_t", a.out_t, E, C, R, a.out_t_codes_group),
                      fp8_scales_span("out_t's scales", a.out_t, E, C, R, a.out_t_scales_group)},
                     {group_span("w", a.w, E, R, C, a.ldw, a.w_group, 2)});
    if (st != VE_OK) return st;
    Fp8PackArgs g{};
    g.rows = R; g.cols = C; g.groups = a.groups; g.weight = true;
    g.x = a.w; g.ldx = a.ldw; g.x_group = E > 1 ? a.w_group : 0;
    g.vec = vec16(a.w, a.ldw) && g.x_group % 8 == 0;
    g.out = a.out; g.out_t = a.out_t;
    if (E > 1) {
        g.out_codes_group = a.out_codes_group; g.out_scales_group = a.out_scales_group;
        g.out_t_codes_group = a.out_t_codes_group; g.out_t_scales_group = a.out_t_scales_group;
    }
    g.format = a.out.codes ? a.out.format : a.out_t.format;
    (void)hipGetLastError();
    return status_of(launch_fp8_pack(g, (hipStream_t)stream), "fp8 weight pack");
}

ve_status ve_fp8_unpack(const ve_fp8_unpack_args* p, void* stream) {
    if (!p) return fail(VE_ERR_INVALID_ARG, "arguments are NULL");
    const ve_fp8_unpack_args& a = *p;
    ve_status st = check_groups(a.rows, a.cols, a.groups);
    if (st != VE_OK) return st;
    const int64_t E = a.groups, R = a.rows, C = a.cols;
    if (a.ldx < C) return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (R == 0) return VE_OK;
    if (!a.x) return fail(VE_ERR_INVALID_ARG, "x is NULL");
    if (a.in.block_rows != 1 && a.in.block_rows != 128)
        return fail(VE_ERR_INVALID_ARG, "in: %d rows share a scale, not 1 or 128", a.in.block_rows);
    if ((st = check_fp8(a.in, R, C, a.in.block_rows, "in")) != VE_OK ||
        (st = check_group_strides(a.in, R, C, a.groups, a.in_codes_group, a.in_scales_group, "in")) != VE_OK)
        return st;
    if (E > 1 && a.x_group < (R - 1) * a.ldx + C) return fail(VE_ERR_INVALID_ARG, "group stride smaller than a group");
    if (!tiles_fit(R, C, 0, E)) return fail(VE_ERR_UNSUPPORTED, "matrices too large for one launch");
    st = check_apart({group_span("x", a.x, E, R, C, a.ldx, a.x_group, 2)},
                     {fp8_codes_span("codes", a.in, E, R, C, a.in_codes_group),
                      fp8_scales_span("scales", a.in, E, R, C, a.in_scales_group)});
    if (st != VE_OK) return st;
    ve_fp8_unpack_args g = a;
    if (E == 1) g.in_codes_group = g.in_scales_group = g.x_group = 0;
    (void)hipGetLastError();
    return status_of(launch_fp8_unpack(g, (hipStream_t)stream), "fp8 unpack");
}

ve_status ve_fp8_linear_forward_workspace(const ve_fp8_linear_forward_args* a, int64_t* bytes) {
    if (!a || !bytes) return fail(VE_ERR_INVALID_ARG, "arguments or bytes is NULL");
    if (const ve_status st = check_forward(*a); st != VE_OK) return st;
    *bytes = a->tokens == 0 ? 0 : round256(plan_fp8(forward_product(*a), kLinFwd).partial_bytes);
    return VE_OK;
}

ve_status ve_fp8_linear_forward(const ve_fp8_linear_forward_args* a, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!a) return fail(VE_ERR_INVALID_ARG, "arguments are NULL");
    ve_status st = check_forward(*a);
    if (st != VE_OK) return st;
    if (a->tokens == 0) return VE_OK;
    Fp8Args g = forward_product(*a);
    const LinPlan p = plan_fp8(g, kLinFwd);
    const int64_t need = round256(p.partial_bytes);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != VE_OK ||
        (st = check_forward_apart(*a, workspace, need)) != VE_OK)
        return st;
    g.partial = (float*)workspace;
    (void)hipGetLastError();
    return status_of(launch_fp8(g, kLinFwd, p, (hipStream_t)stream), "fp8 forward product");
}

ve_status ve_fp8_linear_backward_workspace(const ve_fp8_linear_backward_args* a, int64_t* bytes) {
    if (!a || !bytes) return fail(VE_ERR_INVALID_ARG, "arguments or bytes is NULL");
    if (const ve_status st = check_backward(*a); st != VE_OK) return st;
    Backward b;
    plan_backward(*a, b);
    *bytes = b.total;
    return VE_OK;
}

ve_status ve_fp8_linear_backward(const ve_fp8_linear_backward_args* a, void* workspace, int64_t workspace_bytes,
                                 void* stream) {
    if (!a) return fail(VE_ERR_INVALID_ARG, "arguments are NULL");
    ve_status st = check_backward(*a);
    if (st != VE_OK) return st;
    Backward b;
    plan_backward(*a, b);
    if ((st = check_workspace(workspace, workspace_bytes, b.total)) != VE_OK ||
        (st = check_backward_apart(*a, workspace, b.total)) != VE_OK)
        return st;
    b.dx.partial = b.dw.partial = (float*)workspace;
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if (a->dx && a->tokens > 0 && (st = status_of(launch_fp8(b.dx, kLinFwd, b.pdx, s), "fp8 dx product")) != VE_OK) return st;
    if (!a->dw) return VE_OK;
    return status_of(launch_fp8(b.dw, kLinDw, b.pdw, s), "fp8 dw product");
}

}  // extern "C"
