// ve_checks.h -- argument checks shared by the host sides of the linear layer
// and of the operators around it: alignment, grid limits, overlapping buffers,
// workspaces.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "ve.h"
#include "ve_internal.h"

namespace ve {
namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxWorkgroups = kMaxGridItems / 512;  // of at most 512 threads

int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }
bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool vec16(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

ve_status status_of(hipError_t e, const char* what) {
    if (e == hipSuccess) return VE_OK;
    return fail(VE_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
}

ve_status check_shape(int64_t tokens, int64_t in, int64_t out, int32_t groups, const int64_t* offsets, int32_t act) {
    if (tokens < 0 || in < 1 || out < 1)
        return fail(VE_ERR_INVALID_ARG, "shape: %lld tokens, %lld -> %lld features", (long long)tokens, (long long)in,
                    (long long)out);
    if (groups < 1 || groups > 65536) return fail(VE_ERR_INVALID_ARG, "groups %d outside [1, 65536]", groups);
    if (!offsets && groups != 1) return fail(VE_ERR_INVALID_ARG, "%d groups need offsets", groups);
    if (act < VE_ACT_NONE || act > VE_ACT_SILU) return fail(VE_ERR_INVALID_ARG, "unknown activation %d", act);
    if (tokens > kMaxDim || in > kMaxDim || out > kMaxDim)
        return fail(VE_ERR_UNSUPPORTED, "a dimension of 2^31 or more");
    return VE_OK;
}

// The workgroups of every launch over a rows x cols matrix fit one grid.
// Tiles are at least 64 x 64 or 128 x 128; `extra` row tiles more come from
// ragged groups, and `times` matrices from grouped weights.
bool launchable(int64_t rows, int64_t cols, int64_t extra, int64_t times) {
    const int64_t tm = (rows + 63) / 64 + extra, tn = (cols + 63) / 64;
    return tm <= kMaxWorkgroups / tn / times;
}

// Device memory of a matrix, or of groups of them, in bytes.
struct Span {
    const char* name;
    const void* p;
    int64_t rows, row, pitch, groups, group;  // row: bytes of one; pitch, group: from one to the next

    // Whether the byte at q is one of the matrix's (not of what lies between
    // its rows, so that column slices of one buffer may stand side by side).
    bool holds(const void* q) const {
        if (!p || !q || (uintptr_t)q < (uintptr_t)p) return false;
        uint64_t off = (uintptr_t)q - (uintptr_t)p;
        if (off >= (uint64_t)((groups - 1) * group + (rows - 1) * pitch + row)) return false;
        if (groups > 1) off -= std::min<uint64_t>(off / group, groups - 1) * group;
        if (rows > 1) off -= std::min<uint64_t>(off / pitch, rows - 1) * pitch;
        return off < (uint64_t)row;
    }
};
Span matrix_span(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
    return Span{name, rows > 0 ? p : nullptr, rows, cols * size, ld * size, 1, 0};
}
Span group_span(const char* name, const void* p, int64_t groups, int64_t rows, int64_t cols, int64_t ld, int64_t group,
                int64_t size) {
    return Span{name, p, rows, cols * size, ld * size, groups, group * size};
}

// Refuses an output whose first element is an element of an input or of
// another output, or the other way round: outputs in place of an input, or a
// row or more into it.  Nothing that is refused could have been meant.
ve_status check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        if (!o->p) continue;
        for (const Span& i : ins)
            if (i.holds(o->p) || o->holds(i.p)) return fail(VE_ERR_INVALID_ARG, "%s overlaps %s", o->name, i.name);
        for (const Span* q = o + 1; q != outs.end(); ++q)
            if (q->holds(o->p) || o->holds(q->p)) return fail(VE_ERR_INVALID_ARG, "%s overlaps %s", o->name, q->name);
    }
    return VE_OK;
}

ve_status check_workspace(void* ws, int64_t have, int64_t need) {
    if (need == 0) return VE_OK;
    if (!ws || have < need) return fail(VE_ERR_INVALID_ARG, "workspace of %lld bytes needed", (long long)need);
    if (!aligned(ws, 256)) return fail(VE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    return VE_OK;
}

}  // namespace
}  // namespace ve
