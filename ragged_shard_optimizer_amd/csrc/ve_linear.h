// ve_linear.h -- internal interface between the linear layer's kernels
// (ve_linear.hip, ve_act8.hip) and their host side (ve_linear_host.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ve.h"
#include "ve_internal.h"

namespace ve {

// The three products of a layer.  Rows / columns / contraction:
//   kLinFwd: tokens x out_features, over in_features  (x w^T)
//   kLinDx:  tokens x in_features, over out_features  (dz w)
//   kLinDw:  out_features x in_features, over tokens  (dz^T x)
// In the first two the rows are ragged by group, in the third the contraction.
enum LinKind : int { kLinFwd = 0, kLinDx = 1, kLinDw = 2 };

// Tile forms of the product kernel (option "linear_path" pins one).
enum LinPath : int { kPathAuto = 0, kPathGeneral = 1, kPath128 = 2, kPath256 = 3, kPathFew = 4 };

struct LinArgs {
    const uint16_t* A; int64_t lda;           // x, dz, dz
    const uint16_t* B; int64_t ldb, b_group;  // w, w, x (b_group: elements from one group's weights to the next)
    int64_t T;                                // tokens
    int64_t M, N, K;                          // kLinDw: M output rows; N output columns; K contraction (not kLinDw)
    int32_t E;                                // groups
    const int64_t* offsets;                   // [E + 1] on the device; null: one group of all tokens
    // epilogue of kLinFwd / kLinDx: v += bias; z, z8 out; v = act(v); v += res; y out
    const uint16_t* bias; int64_t bias_group;
    const uint16_t* res; int64_t ldr;
    uint16_t* y; int64_t ldy;
    uint16_t* z; int64_t ldz;
    ve_act8 z8;
    int32_t act;
    // epilogue of kLinDw
    void* dw; int64_t lddw, dw_group;
    int32_t wide, accumulate;                 // fp32 instead of bf16; add to what dw holds
    // 16-byte accesses allowed on rows of these
    bool vec_bias, vec_res, vec_y, vec_z, vec_z8, vec_dw;
    // rows of A / B go on for whole 16 bytes (in the workspace), with zeros
    // where the contiguous dimension is the contraction
    bool pad_a, pad_b;
    // set by the launcher
    int32_t finish;                           // which epilogue
    int32_t tiles_n, ksplit;
    int64_t tiles;                            // tiles of the launch (an upper bound when the rows are ragged)
    float* partial;                           // [slice][tile][BM x BN] fp32 when ksplit > 1
};

// How a product runs: tile form and slices of the contraction.
struct LinPlan { int path; int ksplit; int64_t partial_bytes; double us; };  // us: the time model's estimate
LinPlan plan_product(const LinArgs& g, LinKind kind);
hipError_t launch_product(LinArgs g, LinKind kind, const LinPlan& p, hipStream_t s);

// dz = bf16(dy act'(z)) and the column sums of the unrounded dz by token tile
// and group; z from bf16 (z) or 8 bits (z8).  dz null: sums only (act none).
struct DzArgs {
    const uint16_t* dy; int64_t lddy;
    const uint16_t* z; int64_t ldz;
    ve_act8 z8;
    uint16_t* dz;                             // [T x N], leading dimension lddz
    int64_t lddz;
    float* sums;                              // [token tiles][N], or null
    int64_t T, N;
    int32_t E, act;
    const int64_t* offsets;
    bool vec;
};
constexpr int kDzRows = 64;                   // tokens of one tile of column sums
int64_t dz_tiles(int64_t T, int32_t E, bool ragged);
hipError_t launch_dz(const DzArgs& a, hipStream_t s);
// dbias[e][n] (+)= the sums of group e's tiles, in tile order.
hipError_t launch_dbias(const DzArgs& a, void* dbias, int64_t group, bool wide, bool accumulate, hipStream_t s);

hipError_t launch_act8_pack(const uint16_t* x, int64_t ldx, int64_t rows, int64_t cols, const ve_act8& q, hipStream_t s);
// rows x cols of each of `count` matrices (ld and group: source strides) one
// after the other into dst, whose rows of `cols` rounded up to 8 end in zeros.
// offsets (of E groups, or null): rows in no group are neither read nor written.
hipError_t launch_pad(const uint16_t* src, int64_t ld, int64_t group, int64_t count, int64_t rows, int64_t cols, uint16_t* dst,
                      const int64_t* offsets, int32_t E, hipStream_t s);
hipError_t launch_act8_unpack(const ve_act8& q, int64_t rows, int64_t cols, uint16_t* x, int64_t ldx, const int64_t* offsets,
                              int32_t E, hipStream_t s);

}  // namespace ve
