// ve_expert_host.cpp -- C entry points that sort slots by expert and bring
// rows there and back: argument checks and launches (kernels in ve_expert.hip).

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ve.h"
#include "ve_checks.h"
#include "ve_expert.h"
#include "ve_fp8.h"

using namespace ve;

namespace {

ve_status check_slots(int64_t tokens, int32_t slots) {
    if (tokens < 0) return fail(VE_ERR_INVALID_ARG, "%lld tokens", (long long)tokens);
    if (slots < 1 || slots > kMaxSlots) return fail(VE_ERR_INVALID_ARG, "%d slots outside [1, %d]", slots, kMaxSlots);
    if (tokens > kMaxDim / slots) return fail(VE_ERR_UNSUPPORTED, "2^31 slots or more");
    return VE_OK;
}

ve_status check_rows(int64_t tokens, int64_t cols, int32_t slots, const int32_t* position, int64_t rows_len) {
    const ve_status st = check_slots(tokens, slots);
    if (st != VE_OK) return st;
    if (cols < 1 || rows_len < 0)
        return fail(VE_ERR_INVALID_ARG, "%lld columns, %lld rows", (long long)cols, (long long)rows_len);
    if (tokens > 0 && !position) return fail(VE_ERR_INVALID_ARG, "position is NULL");
    if (cols > kMaxDim - 4096 || rows_len > kMaxDim) return fail(VE_ERR_UNSUPPORTED, "a dimension of 2^31 or more");
    if (expert_workgroups(tokens, cols) > kMaxWorkgroups) return fail(VE_ERR_UNSUPPORTED, "too large for one launch");
    return VE_OK;
}

ve_status check_sort(int64_t tokens, int32_t slots, int32_t n_experts) {
    const ve_status st = check_slots(tokens, slots);
    if (st != VE_OK) return st;
    if (n_experts < 1 || n_experts > kMaxExperts)
        return fail(VE_ERR_INVALID_ARG, "%d experts outside [1, %d]", n_experts, kMaxExperts);
    return VE_OK;
}

SortArgs sort_args(int64_t tokens, int32_t slots, int32_t n_experts) {
    SortArgs a{};
    a.n = (uint32_t)(tokens * slots);
    a.experts_n = n_experts;
    return a;
}

Span index_span(const char* name, const void* p, int64_t tokens, int32_t slots, int64_t size) {
    return matrix_span(name, tokens ? p : nullptr, 1, tokens * slots, tokens * slots, size);
}

}  // namespace

extern "C" {

ve_status ve_expert_sort_workspace(int64_t tokens, int32_t slots, int32_t n_experts, int64_t* bytes) {
    if (!bytes) return fail(VE_ERR_INVALID_ARG, "bytes is NULL");
    if (const ve_status st = check_sort(tokens, slots, n_experts); st != VE_OK) return st;
    SortArgs a = sort_args(tokens, slots, n_experts);
    *bytes = plan_sort(a);
    return VE_OK;
}

ve_status ve_expert_sort(const void* experts, int32_t index_bytes, int64_t tokens, int32_t slots, int32_t n_experts,
                         int64_t* offsets, int32_t* position, int32_t* order, void* workspace,
                         int64_t workspace_bytes, void* stream) {
    ve_status st = check_sort(tokens, slots, n_experts);
    if (st != VE_OK) return st;
    if (index_bytes != 4 && index_bytes != 8) return fail(VE_ERR_INVALID_ARG, "index of %d bytes", index_bytes);
    if (!offsets || (tokens > 0 && (!experts || !position)))
        return fail(VE_ERR_INVALID_ARG, "experts, offsets or position is NULL");
    SortArgs a = sort_args(tokens, slots, n_experts);
    const int64_t need = plan_sort(a);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != VE_OK) return st;
    a.experts = experts; a.wide = index_bytes == 8;
    a.offsets = offsets; a.position = position; a.order = order; a.counts = (uint32_t*)workspace;
    st = check_apart({matrix_span("offsets", offsets, 1, n_experts + 1, n_experts + 1, 8),
                      index_span("position", position, tokens, slots, 4), index_span("order", order, tokens, slots, 4),
                      matrix_span("workspace", need ? workspace : nullptr, 1, need, need, 1)},
                     {index_span("experts", experts, tokens, slots, index_bytes)});
    if (st != VE_OK) return st;
    (void)hipGetLastError();
    return status_of(launch_sort(a, (hipStream_t)stream), "expert sort");
}

ve_status ve_expert_gather(const ve_expert_gather_args* a, void* stream) {
    if (!a) return fail(VE_ERR_INVALID_ARG, "arguments are NULL");
    ve_status st = check_rows(a->tokens, a->cols, a->slots, a->position, a->rows_len);
    if (st != VE_OK) return st;
    const int64_t T = a->tokens, C = a->cols, R = a->rows_len;
    const bool packed = a->rows8.codes != nullptr;
    if (a->ldx < C || (a->rows && a->ld_rows < C)) return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (packed && a->weights) return fail(VE_ERR_INVALID_ARG, "rows in 8 bits take no weights");
    if (packed && a->rows) return fail(VE_ERR_INVALID_ARG, "exactly one of rows and rows8");
    if (packed && (st = check_fp8(a->rows8, R, C, 1, "rows8")) != VE_OK) return st;
    if (T == 0 || R == 0) return VE_OK;
    if (!a->x) return fail(VE_ERR_INVALID_ARG, "x is NULL");
    if (!packed && !a->rows) return fail(VE_ERR_INVALID_ARG, "exactly one of rows and rows8");
    st = check_apart({matrix_span("rows", a->rows, R, C, a->ld_rows, 2), fp8_codes_span("codes", a->rows8, R, C),
                      fp8_scales_span("scales", a->rows8, R, C)},
                     {matrix_span("x", a->x, T, C, a->ldx, 2), index_span("position", a->position, T, a->slots, 4),
                      index_span("weights", a->weights, T, a->slots, 4)});
    if (st != VE_OK) return st;
    (void)hipGetLastError();
    return status_of(launch_gather(*a, (hipStream_t)stream), "expert gather");
}

ve_status ve_expert_combine(const ve_expert_combine_args* a, void* stream) {
    if (!a) return fail(VE_ERR_INVALID_ARG, "arguments are NULL");
    ve_status st = check_rows(a->tokens, a->cols, a->slots, a->position, a->rows_len);
    if (st != VE_OK) return st;
    const int64_t T = a->tokens, C = a->cols, R = a->rows_len;
    if ((R > 0 && a->ld_rows < C) || a->ldy < C || (a->residual && a->ldr < C))
        return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (T == 0) return VE_OK;
    if (!a->y || (R > 0 && !a->rows)) return fail(VE_ERR_INVALID_ARG, "rows or y is NULL");
    const bool same = a->residual == a->y && (a->ldr == a->ldy || T == 1);
    st = check_apart({matrix_span("y", a->y, T, C, a->ldy, 2)},
                     {matrix_span("rows", a->rows, R, C, a->ld_rows, 2),
                      matrix_span("residual", same ? nullptr : a->residual, T, C, a->ldr, 2),
                      index_span("position", a->position, T, a->slots, 4),
                      index_span("weights", a->weights, T, a->slots, 4)});
    if (st != VE_OK) return st;
    (void)hipGetLastError();
    return status_of(launch_combine(*a, (hipStream_t)stream), "expert combine");
}

ve_status ve_expert_combine_backward(const ve_expert_combine_backward_args* a, void* stream) {
    if (!a) return fail(VE_ERR_INVALID_ARG, "arguments are NULL");
    ve_status st = check_rows(a->tokens, a->cols, a->slots, a->position, a->rows_len);
    if (st != VE_OK) return st;
    const int64_t T = a->tokens, C = a->cols, R = a->rows_len;
    if (a->lddy < C || (a->dweights && R > 0 && a->ld_rows < C) || (a->drows && a->ld_drows < C))
        return fail(VE_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (T == 0 || (!a->drows && !a->dweights)) return VE_OK;
    if (!a->dy) return fail(VE_ERR_INVALID_ARG, "dy is NULL");
    if (a->dweights && R > 0 && !a->rows) return fail(VE_ERR_INVALID_ARG, "dweights needs rows");
    st = check_apart({matrix_span("drows", a->drows, R, C, a->ld_drows, 2),
                      index_span("dweights", a->dweights, T, a->slots, 4)},
                     {matrix_span("dy", a->dy, T, C, a->lddy, 2),
                      matrix_span("rows", a->dweights ? a->rows : nullptr, R, C, a->ld_rows, 2),
                      index_span("position", a->position, T, a->slots, 4),
                      index_span("weights", a->drows ? a->weights : nullptr, T, a->slots, 4)});
    if (st != VE_OK) return st;
    (void)hipGetLastError();
    return status_of(launch_combine_backward(*a, (hipStream_t)stream), "expert combine backward");
}

}  // extern "C"
