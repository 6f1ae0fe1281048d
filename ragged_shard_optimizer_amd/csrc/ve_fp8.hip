// ve_fp8.hip -- products of matrices in 8-bit floating point on the MFMA units,
// dense or grouped by expert:
//
//   forward   z[t,n]  = sum_b 2^(ex[t,b] + ew[n / 128,b]) sum_{k in b} cx[t,k] cw[n,k]
//   dx        the same of dy and the transposed weights
//   dw        dw[n,k] = sum_b 2^(edy[n,b] + ex[k,b]) sum_{t in b} cdy[n,t] cx[k,t]
//
// b runs over blocks of 128 of the contraction.  v_mfma_scale takes the
// exponents of 32 consecutive elements of both operands with the codes, so
// that the scales cost no arithmetic and the sums stay in one accumulator.
//
// Both operands are contiguous along the contraction (packing transposes what
// has to be), so that one kind of tile serves all three products: rows of 128
// codes in LDS, one block of the contraction a step.
//
// How exact the sums are: the unit aligns the products of 8 consecutive codes
// to the largest of them, cuts each 13 bits below it, and adds the sums of
// eight in fp32 (measured: 2^16 + 8 times 2^2 comes back as 2^16, with the
// products 8 apart exactly).  On normal values the error is 2^-16.2 of the
// result's rms, far below the 2^-9 of a bf16 result's rounding and the 2^-4 of
// the codes.  For dw in fp32 the codes are turned to bf16 on the way to the
// bf16 MFMAs, whose sums are exact to fp32 (2^-27.6), at half the rate; the
// unscaled 8-bit MFMA 32x32x16 cuts products the same way, and is no faster.
//
// MFMA 32x32x64, operands swapped (output columns as the first operand): the
// accumulator's layout is that of ve_linear.hip.  A lane gives 32 codes of one
// row; which ones does not matter as long as both operands agree, because the
// whole block shares its exponent.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ve_fp8_product.h"
#include "ve_linear_tiles.h"

namespace ve {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x16 mfma_fp8(i32x8 b, i32x8 a, f32x16 c, int eb, int ea, int format) {
    // (both forms are compiled into a kernel of one format each)
    return format == VE_E4M3 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, 0, 0, 0, eb, 0, ea)
                             : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, 0, 1, 0, eb, 0, ea);
}

// 32 codes times a power of two, as bf16: exact (values below 2^-126 may
// become 0).
struct Wide { bf16x8 v[4]; };
__device__ __forceinline__ Wide widen(i32x8 c, int e, int format) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const float s = __uint_as_float((uint32_t)(e & 255) << 23);
    Wide w;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bf16x2 lo = format == VE_E4M3 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c[i], s, false)
                                            : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)c[i], s, false);
        const bf16x2 hi = format == VE_E4M3 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c[i], s, true)
                                            : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)c[i], s, true);
        w.v[i >> 1][4 * (i & 1)] = lo[0];
        w.v[i >> 1][4 * (i & 1) + 1] = lo[1];
        w.v[i >> 1][4 * (i & 1) + 2] = hi[0];
        w.v[i >> 1][4 * (i & 1) + 3] = hi[1];
    }
    return w;
}

// A lane's 32 codes of row r0 + lane % 32, half kk of the block.
template <class Op>
__device__ __forceinline__ i32x8 fragment(const uint16_t* st, int r0, int kk, int lane) {
    const int row = r0 + (lane & 31), s = Op::swz(row & 15), first = 4 * kk + (lane >> 5);
    const u32x4 lo = *(const u32x4*)(st + row * BK + (first ^ s) * 8), hi = *(const u32x4*)(st + row * BK + ((first + 2) ^ s) * 8);
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// Exponents of the `rows` (at most 128) rows from r on, in one contraction
// block, whose exponents start at p: dword l of the lane l (aligned down).
__device__ __forceinline__ uint32_t load_exponents(const uint8_t* p, int64_t all, int r, int lane) {
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)all, 0x00020000);
    return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rs, lane <= 32 ? (r & ~3) + 4 * lane : (int)0x80000000, 0, 0);
}
// ... to a lane's exponent of row r + 32 a + lane % 32 (in the low byte).
__device__ __forceinline__ int spread(uint32_t raw, int r, int a, int lane) {
    const int b = (r & 3) + (lane & 31);
    return (int)((uint32_t)__builtin_amdgcn_ds_bpermute((8 * a + (b >> 2)) * 4, (int)raw) >> (8 * (b & 3)));
}

template <class CF, int KIND, int FORMAT, bool EXACT>
__global__ void __launch_bounds__(CF::THREADS, CF::PER_CU) k_fp8(Fp8Args g) {
    constexpr int TM = CF::TM, TN = CF::TN, WM = CF::WM, WN = CF::WN;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[CF::SMEM];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wr = wave / CF::WAVES_N, wc = wave % CF::WAVES_N;
    Work w;
    if (!fetch<CF, KIND, true>(g, all_tiles<CF, KIND>(g), blockIdx.x, w) || w.rows == 0) return;
    typedef Operand<false, CF::BM, CF::WAVES, true> OpA;
    typedef Operand<false, CF::BN, CF::WAVES, true> OpB;
    OpA A;
    OpB B;
    const int cols = min((int)g.N - w.col0, CF::BN);
    if (KIND == kLinDw) {
        A.init(g.A + w.row0 * g.lda + w.begin, g.lda, w.rows, w.len, lane, wave);
        B.init(g.B + w.col0 * g.ldb + w.begin, g.ldb, cols, w.len, lane, wave);
    } else {
        A.init(g.A + w.row0 * g.lda, g.lda, w.rows, (int)g.K, lane, wave);
        B.init(g.B + w.e * g.b_group + w.col0 * g.ldb, g.ldb, cols, (int)g.K, lane, wave);
    }
    const uint8_t* sa = g.sa + (KIND == kLinDw ? w.begin / BK * g.ld_sa : 0);
    const uint8_t* sb = g.sb + (KIND == kLinDw ? w.begin / BK * g.ld_sb : w.e * g.sb_group);
    const int ra = w.row0 + wr * WM, rb = KIND == kLinDw ? w.col0 + wc * WN : (w.col0 + wc * WN) >> 7;
    f32x16 acc[TM][TN];
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int b = 0; b < TN; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;
    uint16_t* st = (uint16_t*)smem;
    for (int kt = w.kbeg; kt < w.kbeg + w.nk; ++kt) {
        A.begin(kt, true);
        B.begin(kt, true);
#pragma unroll
        for (int q = 0; q < OpA::PIECES; ++q) A.piece(st, q);
#pragma unroll
        for (int q = 0; q < OpB::PIECES; ++q) B.piece(st + CF::A_ELEMS, q);
        const uint32_t raw_a = load_exponents(sa + kt * g.ld_sa, g.sa_rows, ra, lane);
        const uint32_t raw_b = load_exponents(sb + kt * g.ld_sb, g.sb_rows, rb, lane);
        __builtin_amdgcn_s_waitcnt(kWaitAll);
        __syncthreads();
        int ea[TM], eb[TN];
#pragma unroll
        for (int a = 0; a < TM; ++a) ea[a] = spread(raw_a, ra, a, lane);
#pragma unroll
        for (int b = 0; b < TN; ++b)
            eb[b] = KIND == kLinDw ? spread(raw_b, rb, b, lane) : (int)(get_lane(raw_b, 0) >> (8 * (rb & 3)));
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            i32x8 fa[TM], fb[TN];
#pragma unroll
            for (int a = 0; a < TM; ++a) fa[a] = fragment<OpA>(st, wr * WM + a * 32, kk, lane);
#pragma unroll
            for (int b = 0; b < TN; ++b) fb[b] = fragment<OpB>(st + CF::A_ELEMS, wc * WN + b * 32, kk, lane);
            if constexpr (EXACT) {
                Wide wa[TM], wb[TN];
#pragma unroll
                for (int a = 0; a < TM; ++a) wa[a] = widen(fa[a], ea[a], FORMAT);
#pragma unroll
                for (int b = 0; b < TN; ++b) wb[b] = widen(fb[b], eb[b], VE_E4M3);
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int a = 0; a < TM; ++a)
#pragma unroll
                        for (int b = 0; b < TN; ++b)
                            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[b].v[q], wa[a].v[q], acc[a][b], 0, 0, 0);
            } else {
#pragma unroll
                for (int a = 0; a < TM; ++a)
#pragma unroll
                    for (int b = 0; b < TN; ++b) acc[a][b] = mfma_fp8(fb[b], fa[a], acc[a][b], eb[b], ea[a], FORMAT);
            }
        }
        __syncthreads();
    }
    epilogue<CF, KIND>(g.finish, w, acc, smem + CF::STAGES_BYTES + wave * CF::OUT_BYTES, wr, wc, lane);
}

template <class CF, int KIND>
hipError_t launch_kind(Fp8Args g, const LinPlan& p, hipStream_t s) {
    g.tiles_n = (int)((g.N + CF::BN - 1) / CF::BN);
    g.ksplit = p.ksplit;
    g.tiles = tiles_of<CF>(g, (LinKind)KIND);
    if (g.tiles == 0) return hipSuccess;
    g.finish = finish_of(g, (LinKind)KIND);
    const dim3 grid((unsigned)items_of(g, (LinKind)KIND));
    if (KIND == kLinDw && g.wide) {
        if (g.format == VE_E4M3) hipLaunchKernelGGL((k_fp8<CF, kLinDw, VE_E4M3, true>), grid, dim3(CF::THREADS), 0, s, g);
        else hipLaunchKernelGGL((k_fp8<CF, kLinDw, VE_E5M2, true>), grid, dim3(CF::THREADS), 0, s, g);
    } else {
        if (g.format == VE_E4M3) hipLaunchKernelGGL((k_fp8<CF, KIND, VE_E4M3, false>), grid, dim3(CF::THREADS), 0, s, g);
        else hipLaunchKernelGGL((k_fp8<CF, KIND, VE_E5M2, false>), grid, dim3(CF::THREADS), 0, s, g);
    }
    return hipGetLastError();
}

}  // namespace

LinPlan plan_fp8(const Fp8Args&, LinKind) { return LinPlan{kPath128, 1, 0, 0}; }

hipError_t launch_fp8(Fp8Args g, LinKind kind, const LinPlan& p, hipStream_t s) {
    return kind == kLinDw ? launch_kind<Cfg128, kLinDw>(g, p, s) : launch_kind<Cfg128, kLinFwd>(g, p, s);
}

}  // namespace ve
