// ve_linear_host.cpp -- C entry points of the linear layer and of 8-bit saved
// activations: argument checks, workspace sizing and the launch sequences
// (kernels in ve_linear.hip and ve_act8.hip).
//
// Backward sequence:
//   1. dz = bf16(dy act'(z)) into the workspace, with the column sums by
//      token tile (no activation: the sums only, and dz is dy);
//   2. dbias from the sums;
//   3. dx = dz w;
//   4. x restored into the workspace if it comes in 8 bits, then dw = dz^T x.
// Operands that direct loads cannot take are laid out anew in the workspace
// before their product, if the time model says so (plan_copies).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ve.h"
#include "ve_checks.h"
#include "ve_linear.h"

using namespace ve;

namespace {

ve_status check_act8(const ve_act8& q, int64_t cols, const char* name) {
    if (!q.codes || !q.scales) return fail(VE_ERR_INVALID_ARG, "%s: codes or scales is NULL", name);
    if (q.block != 32 && q.block != 64 && q.block != 128)
        return fail(VE_ERR_INVALID_ARG, "%s: block %d is not 32, 64 or 128", name, q.block);
    if (q.ld_codes < cols || q.ld_scales < (cols + q.block - 1) / q.block)
        return fail(VE_ERR_INVALID_ARG, "%s: leading dimension smaller than the row", name);
    return VE_OK;
}

ve_status check_forward(const ve_linear_forward_args& a) {
    ve_status st = check_shape(a.tokens, a.in_features, a.out_features, a.groups, a.offsets, a.activation);
    if (st != VE_OK) return st;
    if (!a.w) return fail(VE_ERR_INVALID_ARG, "w is NULL");
    if (a.tokens > 0 && (!a.x || !a.y)) return fail(VE_ERR_INVALID_ARG, "x or y is NULL");
    if (a.tokens > 0 && (const uint16_t*)a.y == a.x) return fail(VE_ERR_INVALID_ARG, "y is x");
    const int64_t K = a.in_features, N = a.out_features;
    if (a.ldx < K || a.ldw < K || a.ldy < N || (a.residual && a.ldr < N) || (a.z && a.ldz < N))
        return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (a.groups > 1 && (a.w_group < (N - 1) * a.ldw + K || (a.bias && a.bias_group < N)))
        return fail(VE_ERR_INVALID_ARG, "group stride smaller than a group");
    if (a.z8.codes && (st = check_act8(a.z8, N, "z8")) != VE_OK) return st;
    if (!launchable(a.tokens, N, a.groups, 1)) return fail(VE_ERR_UNSUPPORTED, "product too large for one launch");
    return VE_OK;
}

LinArgs forward_product(const ve_linear_forward_args& a) {
    LinArgs g{};
    g.A = a.x; g.lda = a.ldx;
    g.B = a.w; g.ldb = a.ldw; g.b_group = a.groups > 1 ? a.w_group : 0;
    g.T = a.tokens; g.N = a.out_features; g.K = a.in_features;
    g.E = a.groups; g.offsets = a.offsets;
    g.bias = a.bias; g.bias_group = a.groups > 1 ? a.bias_group : 0;
    g.res = a.residual; g.ldr = a.ldr;
    g.y = a.y; g.ldy = a.ldy;
    g.z = a.z; g.ldz = a.ldz;
    g.z8 = a.z8; g.act = a.activation;
    g.vec_bias = vec16(a.bias, g.bias_group);
    g.vec_res = vec16(a.residual, a.ldr);
    g.vec_y = vec16(a.y, a.ldy);
    g.vec_z = vec16(a.z, a.ldz);
    g.vec_z8 = aligned(a.z8.codes, 8) && a.z8.ld_codes % 8 == 0;
    return g;
}

int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

// Operands of a product that direct loads cannot take are laid out anew, in
// rows of whole 16 bytes, where that and the direct form together take less
// time than the register-staged form.  A copy moves its bytes twice, at 4
// TB/s, by one launch.  8192 tokens, 8190 -> 8190: forward 2390 -> 920 us, dx
// 3030 -> 910, dw 6340 -> 915; 16 groups of 6 tokens 2046 -> 2046 forward
// keep the other form (47 us against 88: the copies are of all weights).
struct Copy {
    const uint16_t* src; int64_t ld, group, count, rows, cols;
    const int64_t* offsets; int32_t E;  // rows of tokens: of the groups' rows only
    double elems() const { return (double)count * (double)rows * (double)up8(cols); }
    int64_t bytes() const { return count * rows * up8(cols) * 2; }  // once elems() fits a launch
    double us() const { return count ? 4 + elems() * 4 / 4e6 : 0; }
};
struct Copies { Copy a, b; };

// The product g with the operands that need it laid out anew (addresses are
// set by the caller), or g itself; its plan.
// x restored from 8 bits is weighed like the same x in bf16 (without its
// padding at first, then charged like a copy), so that the choice, and with it
// every bit of dw, is the same.
LinPlan plan_copies(LinArgs& g, LinKind kind, Copies& c) {
    c = Copies{};
    const int64_t a_cols = kind == kLinDw ? g.M : g.K, b_cols = kind == kLinFwd ? g.K : g.N;
    LinArgs as_is = g;
    as_is.pad_b = g.pad_b && b_cols % 8 == 0;
    const LinPlan plain = plan_product(as_is, kind);
    const int64_t pin = option(kOptLinearPath);
    if (plain.path != kPathGeneral || pin == kPathGeneral) return plain;
    const int64_t b_rows = kind == kLinFwd ? g.N : kind == kLinDx ? g.K : g.T, b_groups = kind == kLinDw ? 1 : g.E;
    LinArgs p = g;
    if (!g.pad_a && (!vec16(g.A, g.lda) || a_cols % 8)) {
        c.a = Copy{g.A, g.lda, 0, 1, g.T, a_cols, g.offsets, g.E};
        p.A = (const uint16_t*)(uintptr_t)256; p.lda = up8(a_cols); p.pad_a = true;
    }
    double b_us = 0;
    if (g.pad_b) b_us = b_cols % 8 ? Copy{g.B, g.ldb, 0, b_groups, b_rows, b_cols, nullptr, 0}.us() : 0;
    else if (!vec16(g.B, g.ldb) || g.b_group % 8 || b_cols % 8) {
        c.b = Copy{g.B, g.ldb, g.b_group, b_groups, b_rows, b_cols, kind == kLinDw ? g.offsets : nullptr, g.E};
        b_us = c.b.us();
        p.B = (const uint16_t*)(uintptr_t)256; p.ldb = up8(b_cols); p.pad_b = true;
        if (b_groups > 1) p.b_group = b_rows * p.ldb;
    }
    const LinPlan fast = plan_product(p, kind);
    const bool pinned = pin == kPath128 || pin == kPath256;
    const double most = (double)kMaxWorkgroups * 8192;  // elements of one copying launch
    const bool fits = c.a.elems() <= most && c.b.elems() <= most;
    if (fast.path == kPathGeneral || !fits || (!pinned && fast.us + c.a.us() + b_us >= plain.us)) {
        c = Copies{};
        return plain;
    }
    g = p;
    return fast;
}

ve_status run_copy(const Copy& c, const uint16_t* to, hipStream_t s) {
    if (!c.src) return VE_OK;
    return status_of(launch_pad(c.src, c.ld, c.group, c.count, c.rows, c.cols, (uint16_t*)to, c.offsets, c.E, s),
                     "operand layout");
}

// What a forward call launches, and where its scratch lies.
struct Forward {
    LinArgs g;
    LinPlan p;
    Copies c;
    int64_t total;
};

void plan_forward(const ve_linear_forward_args& a, char* ws, Forward& f) {
    f.g = forward_product(a);
    f.p = plan_copies(f.g, kLinFwd, f.c);
    int64_t at = round256(f.p.partial_bytes);
    auto carve = [&](const Copy& c, const uint16_t*& to) {
        if (!c.src) return;
        if (ws) to = (const uint16_t*)(ws + at);
        at += round256(c.bytes());
    };
    carve(f.c.a, f.g.A);
    carve(f.c.b, f.g.B);
    f.g.partial = (float*)ws;
    f.total = at;
}

ve_status check_backward(const ve_linear_backward_args& a) {
    ve_status st = check_shape(a.tokens, a.in_features, a.out_features, a.groups, a.offsets, a.activation);
    if (st != VE_OK) return st;
    const int64_t K = a.in_features, N = a.out_features;
    const bool some = a.tokens > 0, need_z = a.activation != VE_ACT_NONE && (a.dx || a.dw || a.dbias);
    if (some && !a.dy) return fail(VE_ERR_INVALID_ARG, "dy is NULL");
    if (a.lddy < N) return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (a.dx && (a.lddx < K || (a.dx_add && a.ld_add < K)))
        return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (some && a.dx && a.dx == a.dy) return fail(VE_ERR_INVALID_ARG, "dx is dy");
    if (a.dx && !a.w) return fail(VE_ERR_INVALID_ARG, "dx needs w");
    if (a.dx && a.ldw < K) return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (a.dx && a.groups > 1 && a.w_group < (N - 1) * a.ldw + K)
        return fail(VE_ERR_INVALID_ARG, "group stride smaller than a group");
    if (a.dw) {
        if (some && (a.x != nullptr) == (a.x8.codes != nullptr))
            return fail(VE_ERR_INVALID_ARG, "dw needs exactly one of x and x8");
        if (a.lddw < K || (a.x && a.ldx < K)) return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
        if (a.x8.codes && (st = check_act8(a.x8, K, "x8")) != VE_OK) return st;
        if (a.groups > 1 && a.dw_group < (N - 1) * a.lddw + K)
            return fail(VE_ERR_INVALID_ARG, "group stride smaller than a group");
    }
    if (a.dbias && a.groups > 1 && a.dbias_group < N)
        return fail(VE_ERR_INVALID_ARG, "group stride smaller than a group");
    if (need_z) {
        if (some && (a.z != nullptr) == (a.z8.codes != nullptr))
            return fail(VE_ERR_INVALID_ARG, "the activation needs exactly one of z and z8");
        if (a.z && a.ldz < N) return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
        if (a.z8.codes && (st = check_act8(a.z8, N, "z8")) != VE_OK) return st;
    }
    if (!launchable(a.tokens, K, a.groups, 1) || !launchable(a.tokens, N, a.groups, 1) || !launchable(N, K, 0, a.groups))
        return fail(VE_ERR_UNSUPPORTED, "product too large for one launch");
    return VE_OK;
}

// What a backward call launches, and where its scratch lies.
struct Backward {
    DzArgs dz;
    LinArgs dx, dw;
    LinPlan pdx, pdw;
    Copies cdx, cdw;
    int64_t dz_at, sums_at, x_at, partial_at, total;
};

void plan_backward(const ve_linear_backward_args& a, char* ws, Backward& b) {
    const int64_t T = a.tokens, K = a.in_features, N = a.out_features;
    const bool act = a.activation != VE_ACT_NONE;
    // rows of the scratch matrices start on 16 bytes
    const int64_t ldz = (N + 7) / 8 * 8, ldx = (K + 7) / 8 * 8;
    int64_t at = 0;
    auto carve = [&](bool need, int64_t bytes) {
        const int64_t here = at;
        if (need) at += round256(bytes);
        return here;
    };
    b.dz_at = carve(act, T * ldz * 2);
    b.sums_at = carve(a.dbias != nullptr, dz_tiles(T, a.groups, a.offsets != nullptr) * N * 4);
    const bool restore = a.dw && a.x8.codes;
    b.x_at = carve(restore, T * ldx * 2);
    auto in_ws = [&](int64_t off) { return ws ? (uint16_t*)(ws + off) : (uint16_t*)(uintptr_t)256; };

    b.dz = DzArgs{};
    b.dz.dy = a.dy; b.dz.lddy = a.lddy;
    b.dz.z = a.z; b.dz.ldz = a.ldz; b.dz.z8 = a.z8;
    b.dz.dz = act ? in_ws(b.dz_at) : nullptr; b.dz.lddz = ldz;
    b.dz.sums = a.dbias ? (float*)in_ws(b.sums_at) : nullptr;
    b.dz.T = T; b.dz.N = N; b.dz.E = a.groups; b.dz.act = a.activation; b.dz.offsets = a.offsets;
    b.dz.vec = N % 8 == 0 && vec16(a.dy, a.lddy);
    if (act) b.dz.vec = b.dz.vec && (a.z8.codes ? aligned(a.z8.codes, 8) && a.z8.ld_codes % 8 == 0 : vec16(a.z, a.ldz));

    const uint16_t* dz = act ? b.dz.dz : a.dy;
    const int64_t lddz = act ? ldz : a.lddy;
    LinArgs g{};
    g.A = dz; g.lda = lddz;
    g.B = a.w; g.ldb = a.ldw; g.b_group = a.groups > 1 ? a.w_group : 0;
    g.T = T; g.N = K; g.K = N; g.E = a.groups; g.offsets = a.offsets;
    g.res = a.dx_add; g.ldr = a.ld_add;
    g.y = a.dx; g.ldy = a.lddx;
    g.vec_res = vec16(a.dx_add, a.ld_add);
    g.vec_y = vec16(a.dx, a.lddx);
    g.pad_a = act;
    b.dx = g;
    g = LinArgs{};
    g.A = dz; g.lda = lddz;
    g.B = restore ? in_ws(b.x_at) : a.x; g.ldb = restore ? ldx : a.ldx;
    g.T = T; g.M = N; g.N = K; g.E = a.groups; g.offsets = a.offsets;
    g.dw = a.dw; g.lddw = a.lddw; g.dw_group = a.groups > 1 ? a.dw_group : 0;
    g.wide = a.grad_fp32 != 0; g.accumulate = a.accumulate != 0;
    g.vec_dw = aligned(a.dw, 16) && a.lddw % 8 == 0 && g.dw_group % 8 == 0;
    g.pad_a = act;
    g.pad_b = restore;
    b.dw = g;
    b.pdx = b.pdw = LinPlan{kPathGeneral, 1, 0, 0};
    b.cdx = b.cdw = Copies{};
    if (a.dx && T > 0) b.pdx = plan_copies(b.dx, kLinDx, b.cdx);
    if (a.dw) b.pdw = T > 0 ? plan_copies(b.dw, kLinDw, b.cdw) : plan_product(b.dw, kLinDw);
    auto place = [&](const Copy& c, const uint16_t*& to) {
        if (c.src) to = in_ws(carve(true, c.bytes()));
    };
    place(b.cdx.a, b.dx.A);
    place(b.cdx.b, b.dx.B);
    // dy is laid out once for both products
    if (b.cdw.a.src && b.cdx.a.src) {
        b.dw.A = b.dx.A;
        b.cdw.a.src = nullptr;
    }
    place(b.cdw.a, b.dw.A);
    place(b.cdw.b, b.dw.B);
    const int64_t partial = std::max(b.pdx.partial_bytes, b.pdw.partial_bytes);
    b.partial_at = carve(partial > 0, partial);
    b.dx.partial = b.dw.partial = (float*)in_ws(b.partial_at);
    b.total = at;
}

Span codes_span(const ve_act8& q, int64_t rows, int64_t cols) { return matrix_span("codes", q.codes, rows, cols, q.ld_codes, 1); }
Span scales_span(const ve_act8& q, int64_t rows, int64_t cols) {
    return matrix_span("scales", q.codes ? q.scales : nullptr, rows, q.codes ? (cols + q.block - 1) / q.block : 0, q.ld_scales, 4);
}

// The residual may be y itself, dx_add may be dx itself (the same rows).
ve_status check_forward_apart(const ve_linear_forward_args& a, const void* ws, int64_t ws_bytes) {
    const int64_t T = a.tokens, K = a.in_features, N = a.out_features, E = a.groups;
    const bool same = a.residual == a.y && (a.ldr == a.ldy || T == 1);
    return check_apart({matrix_span("y", a.y, T, N, a.ldy, 2), matrix_span("z", a.z, T, N, a.ldz, 2),
                        codes_span(a.z8, T, N), scales_span(a.z8, T, N),
                        matrix_span("workspace", ws_bytes ? ws : nullptr, 1, ws_bytes, ws_bytes, 1)},
                       {matrix_span("x", a.x, T, K, a.ldx, 2), group_span("w", a.w, E, N, K, a.ldw, a.w_group, 2),
                        group_span("bias", a.bias, E, 1, N, N, a.bias_group, 2),
                        matrix_span("residual", same ? nullptr : a.residual, T, N, a.ldr, 2),
                        matrix_span("offsets", a.offsets, 1, E + 1, E + 1, 8)});
}

// What is read: w for dx, x for dw, z for an activation's slope.
ve_status check_backward_apart(const ve_linear_backward_args& a, const void* ws, int64_t ws_bytes) {
    const int64_t T = a.tokens, K = a.in_features, N = a.out_features, E = a.groups, grad = a.grad_fp32 ? 4 : 2;
    const bool same = a.dx_add == a.dx && (a.ld_add == a.lddx || T == 1), act = a.activation != VE_ACT_NONE;
    const ve_act8 none{}, x8 = a.dw ? a.x8 : none, z8 = act ? a.z8 : none;
    return check_apart({matrix_span("dx", a.dx, T, K, a.lddx, 2),
                        group_span("dw", a.dw, E, N, K, a.lddw, a.dw_group, grad),
                        group_span("dbias", a.dbias, E, 1, N, N, a.dbias_group, grad),
                        matrix_span("workspace", ws_bytes ? ws : nullptr, 1, ws_bytes, ws_bytes, 1)},
                       {matrix_span("dy", a.dy, T, N, a.lddy, 2),
                        group_span("w", a.dx ? a.w : nullptr, E, N, K, a.ldw, a.w_group, 2),
                        matrix_span("x", a.dw ? a.x : nullptr, T, K, a.ldx, 2), codes_span(x8, T, K), scales_span(x8, T, K),
                        matrix_span("z", act ? a.z : nullptr, T, N, a.ldz, 2), codes_span(z8, T, N), scales_span(z8, T, N),
                        matrix_span("dx_add", a.dx && !same ? a.dx_add : nullptr, T, K, a.ld_add, 2),
                        matrix_span("offsets", a.offsets, 1, E + 1, E + 1, 8)});
}

}  // namespace

extern "C" {

ve_status ve_act8_pack(const uint16_t* x, int64_t ldx, int64_t rows, int64_t cols, const ve_act8* out, void* stream) {
    if (!out) return fail(VE_ERR_INVALID_ARG, "out is NULL");
    if (rows < 0 || cols < 1) return fail(VE_ERR_INVALID_ARG, "shape %lld x %lld", (long long)rows, (long long)cols);
    if (ldx < cols) return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (rows == 0) return VE_OK;
    if (!x) return fail(VE_ERR_INVALID_ARG, "x is NULL");
    if (const ve_status st = check_act8(*out, cols, "out"); st != VE_OK) return st;
    if (cols > kMaxDim || rows > kMaxWorkgroups * 8192 / (cols + 128))
        return fail(VE_ERR_UNSUPPORTED, "matrix too large for one launch");
    if (const ve_status st = check_apart({codes_span(*out, rows, cols), scales_span(*out, rows, cols)},
                                         {matrix_span("x", x, rows, cols, ldx, 2)});
        st != VE_OK)
        return st;
    (void)hipGetLastError();
    return status_of(launch_act8_pack(x, ldx, rows, cols, *out, (hipStream_t)stream), "pack");
}

ve_status ve_act8_unpack(const ve_act8* in, int64_t rows, int64_t cols, uint16_t* x, int64_t ldx, void* stream) {
    if (!in) return fail(VE_ERR_INVALID_ARG, "in is NULL");
    if (rows < 0 || cols < 1) return fail(VE_ERR_INVALID_ARG, "shape %lld x %lld", (long long)rows, (long long)cols);
    if (ldx < cols) return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (rows == 0) return VE_OK;
    if (!x) return fail(VE_ERR_INVALID_ARG, "x is NULL");
    if (const ve_status st = check_act8(*in, cols, "in"); st != VE_OK) return st;
    if (cols > kMaxDim || rows > kMaxWorkgroups * 8192 / (cols + 128))
        return fail(VE_ERR_UNSUPPORTED, "matrix too large for one launch");
    if (const ve_status st = check_apart({matrix_span("x", x, rows, cols, ldx, 2)},
                                         {codes_span(*in, rows, cols), scales_span(*in, rows, cols)});
        st != VE_OK)
        return st;
    (void)hipGetLastError();
    return status_of(launch_act8_unpack(*in, rows, cols, x, ldx, nullptr, 0, (hipStream_t)stream), "unpack");
}

ve_status ve_linear_forward_workspace(const ve_linear_forward_args* a, int64_t* bytes) {
    if (!a || !bytes) return fail(VE_ERR_INVALID_ARG, "arguments or bytes is NULL");
    if (const ve_status st = check_forward(*a); st != VE_OK) return st;
    *bytes = 0;
    if (a->tokens == 0) return VE_OK;
    Forward f;
    plan_forward(*a, nullptr, f);
    *bytes = f.total;
    return VE_OK;
}

ve_status ve_linear_forward(const ve_linear_forward_args* a, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!a) return fail(VE_ERR_INVALID_ARG, "arguments are NULL");
    if (const ve_status st = check_forward(*a); st != VE_OK) return st;
    if (a->tokens == 0) return VE_OK;
    Forward f;
    plan_forward(*a, (char*)workspace, f);
    ve_status st = check_workspace(workspace, workspace_bytes, f.total);
    if (st != VE_OK || (st = check_forward_apart(*a, workspace, f.total)) != VE_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if ((st = run_copy(f.c.a, f.g.A, s)) != VE_OK || (st = run_copy(f.c.b, f.g.B, s)) != VE_OK) return st;
    return status_of(launch_product(f.g, kLinFwd, f.p, s), "forward product");
}

ve_status ve_linear_backward_workspace(const ve_linear_backward_args* a, int64_t* bytes) {
    if (!a || !bytes) return fail(VE_ERR_INVALID_ARG, "arguments or bytes is NULL");
    if (const ve_status st = check_backward(*a); st != VE_OK) return st;
    Backward b;
    plan_backward(*a, nullptr, b);
    *bytes = b.total;
    return VE_OK;
}

ve_status ve_linear_backward(const ve_linear_backward_args* a, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!a) return fail(VE_ERR_INVALID_ARG, "arguments are NULL");
    ve_status st = check_backward(*a);
    if (st != VE_OK) return st;
    Backward b;
    plan_backward(*a, (char*)workspace, b);
    if ((st = check_workspace(workspace, workspace_bytes, b.total)) != VE_OK ||
        (st = check_backward_apart(*a, workspace, b.total)) != VE_OK)
        return st;
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if (a->tokens > 0 && (a->dbias || (b.dz.dz && (a->dx || a->dw))) &&
        (st = status_of(launch_dz(b.dz, s), "dz")) != VE_OK)
        return st;
    if (a->dbias && (st = status_of(launch_dbias(b.dz, a->dbias, a->groups > 1 ? a->dbias_group : 0, a->grad_fp32 != 0,
                                                 a->accumulate != 0, s),
                                    "dbias")) != VE_OK)
        return st;
    if ((st = run_copy(b.cdx.a, b.dx.A, s)) != VE_OK || (st = run_copy(b.cdx.b, b.dx.B, s)) != VE_OK) return st;
    if (a->dx && a->tokens > 0 && (st = status_of(launch_product(b.dx, kLinDx, b.pdx, s), "dx product")) != VE_OK)
        return st;
    if (!a->dw) return VE_OK;
    if (a->tokens > 0 && a->x8.codes &&
        (st = status_of(launch_act8_unpack(a->x8, a->tokens, a->in_features, (uint16_t*)b.dw.B, b.dw.ldb, a->offsets, a->groups, s),
                        "restore")) != VE_OK)
        return st;
    if ((st = run_copy(b.cdw.a, b.dw.A, s)) != VE_OK || (st = run_copy(b.cdw.b, b.dw.B, s)) != VE_OK) return st;
    return status_of(launch_product(b.dw, kLinDw, b.pdw, s), "dw product");
}

}  // extern "C"
