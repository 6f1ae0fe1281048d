// ve_fp8.h -- internal interface between the kernels on matrices in 8-bit
// floating point (ve_fp8_pack.hip, ve_fp8.hip) and their host side
// (ve_fp8_host.cpp), and the checks of such matrices.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ve_checks.h"
#include "ve_linear.h"

namespace ve {
namespace {

// A packed rows x cols matrix (or groups of them) that an operand may be.
ve_status check_fp8(const ve_fp8& q, int64_t rows, int64_t cols, int32_t block_rows, const char* name) {
    if (!q.codes || !q.scales) return fail(VE_ERR_INVALID_ARG, "%s: codes or scales is NULL", name);
    if (q.format != VE_E4M3 && q.format != VE_E5M2)
        return fail(VE_ERR_INVALID_ARG, "%s: unknown format %d", name, q.format);
    if (q.block_rows != block_rows)
        return fail(VE_ERR_INVALID_ARG, "%s: %d rows share a scale, not %d", name, q.block_rows, block_rows);
    if (q.ld_codes < cols || q.ld_scales < (rows + block_rows - 1) / block_rows)
        return fail(VE_ERR_INVALID_ARG, "%s: leading dimension smaller than the row", name);
    if (!aligned(q.codes, 16) || q.ld_codes % 16 || !aligned(q.scales, 4) || q.ld_scales % 4)
        return fail(VE_ERR_INVALID_ARG, "%s: codes must start on 16 bytes and scales on 4, every row", name);
    return VE_OK;
}
int64_t scale_rows(int64_t cols) { return (cols + 127) / 128; }
Span fp8_codes_span(const char* name, const ve_fp8& q, int64_t rows, int64_t cols) {
    return matrix_span(name, q.codes, rows, (cols + 15) / 16 * 16, q.ld_codes, 1);
}
Span fp8_scales_span(const char* name, const ve_fp8& q, int64_t rows, int64_t cols) {
    const int64_t n = q.codes ? (rows + q.block_rows - 1) / q.block_rows : 0;
    return matrix_span(name, q.codes && n ? q.scales : nullptr, scale_rows(cols), n, q.ld_scales, 1);
}
Span fp8_codes_span(const char* name, const ve_fp8& q, int64_t groups, int64_t rows, int64_t cols, int64_t group) {
    return group_span(name, q.codes, groups, rows, (cols + 15) / 16 * 16, q.ld_codes, group, 1);
}
Span fp8_scales_span(const char* name, const ve_fp8& q, int64_t groups, int64_t rows, int64_t cols, int64_t group) {
    const int64_t n = q.codes ? (rows + q.block_rows - 1) / q.block_rows : 0;
    return group_span(name, q.codes ? q.scales : nullptr, groups, scale_rows(cols), n, q.ld_scales, group, 1);
}

}  // namespace
}  // namespace ve
