// ve_fp8_product.h -- internal interface of the products of matrices in 8-bit
// floating point (ve_fp8.hip) and their host side (ve_fp8_host.cpp).
#pragma once

#include "ve_linear.h"

namespace ve {

// C = A B^T, both contiguous along the contraction.  Rows / columns /
// contraction:
//   kLinFwd: tokens x outputs, over inputs (x and w; dy and w_t)
//   kLinDw:  outputs x inputs, over the columns of dy_t and x_t
// Codes are taken as pairs: A, B, lda, ldb, b_group and K are in elements of 2
// bytes (K up to the rows' zeros; kLinDw: all columns), and so is T in kLinDw
// without offsets.
struct Fp8Args : LinArgs {
    const uint8_t* sa; int64_t ld_sa;            // exponents of A: [runs][rows]
    const uint8_t* sb; int64_t ld_sb, sb_group;  // ... of B (kLinFwd: one for 128 rows)
    int32_t format;                              // of A (B is E4M3)
    int64_t sa_rows, sb_rows;                    // exponents in a row, up to a multiple of 4
};
// Operands' rows are less than this many bytes apart, so that all of a tile's
// lie within 2^31 bytes of its first: of 128 x 128 and of 256 x 256 tiles.
constexpr int64_t kFp8Pitch128 = int64_t(1) << 24, kFp8Pitch256 = int64_t(1) << 23;
LinPlan plan_fp8(const Fp8Args& g, LinKind kind);
hipError_t launch_fp8(Fp8Args g, LinKind kind, const LinPlan& p, hipStream_t s);

}  // namespace ve
