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
// eight in fp32 (measured: 2^16 + 7 times 2^2 comes back as 2^16, with the
// products 8 apart exactly), so that each of 8 loses up to 2^-13 of the largest.
// On normal values the error is 2^-16.2 of the result's rms, far below the 2^-8
// of a bf16 result's rounding and the 2^-4 of the codes, and bf16 results take
// it.  Beside what is left where large products cancel it is not small: columns
// 2^9 times the rest, in pairs that cancel, leave errors of up to 10% of the
// rms.  For dw in fp32 the codes are turned to bf16 on the way to the bf16
// MFMAs, whose sums are exact to fp32 (2^-27.6), at half the rate; tiles with
// values that bf16 cannot hold take the scaled MFMAs, one of 8 consecutive
// products at a time, which are not cut.  The unscaled 8-bit MFMA 32x32x16 cuts
// products the same way, and is no faster.
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

// 32 codes times a power of two, as bf16: exact where no value leaves bf16's
// normal numbers (bf16_exponent), which a block's largest may by rounding up to
// 2^128 when it was packed, and any may where the other operand's scale brings
// the product back.
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

// Every code under this exponent is a normal number of bf16: the smallest, 2^-9
// (E4M3) or 2^-16 (E5M2), is at least 2^-126, and the largest, below 2^9 or
// 2^16, below 2^128.
__device__ __forceinline__ bool bf16_exponent(int e, int format) {
    return (uint32_t)((e & 255) - (format == VE_E4M3 ? 10 : 17)) <= (format == VE_E4M3 ? 236u : 222u);
}

// ... under all four of a dword.
__device__ __forceinline__ bool bf16_exponents(uint32_t e, int format) {
    bool all = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) all &= bf16_exponent((int)(e >> (8 * i)), format);
    return all;
}

// A lane's 32 codes of row r0 + lane % 32, half kk of the block.
template <class Op>
__device__ __forceinline__ i32x8 fragment(const uint16_t* st, int r0, int kk, int lane) {
    const int row = r0 + (lane & 31), s = Op::swz(row & 15), first = 4 * kk + (lane >> 5);
    const u32x4 lo = *(const u32x4*)(st + row * BK + (first ^ s) * 8), hi = *(const u32x4*)(st + row * BK + ((first + 2) ^ s) * 8);
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// Exponents of an operand's rows in one contraction block after the other: a
// wave's at most 128 rows from `row` on are 33 aligned dwords, dword l in lane
// l.
struct Exponents {
    const uint8_t* p;  // the block's first
    int ld, row, all;  // to the next block; the wave's first row; rows up to a multiple of 4
    __device__ __forceinline__ void init(const uint8_t* base, int64_t ld_, int row_, int64_t all_) {
        p = (const uint8_t*)uniform64((int64_t)base);
        ld = __builtin_amdgcn_readfirstlane((int)ld_);
        row = __builtin_amdgcn_readfirstlane(row_);
        all = __builtin_amdgcn_readfirstlane((int)all_);
    }
    __device__ __forceinline__ uint32_t load(int lane, bool live) const {
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, live ? all : 0, 0x00020000);
        return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rs, lane <= 32 ? (row & ~3) + 4 * lane : (int)0x80000000, 0, 0);
    }
    // whether a lane's dword has some of the wave's first n rows
    __device__ __forceinline__ bool holds(int lane, int n) const { return 4 * lane < (row & 3) + n; }
    __device__ __forceinline__ void next() { p += ld; }
    __device__ __forceinline__ void stash(uint32_t& keep, int at) const {
        put_lane(keep, at, (uint32_t)(uintptr_t)p);
        put_lane(keep, at + 1, (uint32_t)((uintptr_t)p >> 32));
        put_lane(keep, at + 2, (uint32_t)ld);
        put_lane(keep, at + 3, (uint32_t)row);
        put_lane(keep, at + 4, (uint32_t)all);
    }
    __device__ __forceinline__ void unstash(uint32_t keep, int at) {
        const uint64_t lo = get_lane(keep, at), hi = get_lane(keep, at + 1);
        p = (const uint8_t*)(uintptr_t)((hi << 32) | lo);
        ld = (int)get_lane(keep, at + 2);
        row = (int)get_lane(keep, at + 3);
        all = (int)get_lane(keep, at + 4);
    }
};
// ... to the dword with a lane's exponent of row `row` + 32 a + lane % 32, which
// is `spread_shift` bits up.
__device__ __forceinline__ uint32_t spread_dword(uint32_t raw, int row, int a, int lane) {
    return (uint32_t)__builtin_amdgcn_ds_bpermute((8 * a + (((row & 3) + (lane & 31)) >> 2)) * 4, (int)raw);
}
__device__ __forceinline__ uint32_t spread_shift(int row, int lane) { return 8 * ((row + lane) & 3); }
__device__ __forceinline__ int spread(uint32_t raw, int row, int a, int lane) {
    return (int)(spread_dword(raw, row, a, lane) >> spread_shift(row, lane));
}

// The groups' rows (kLinFwd) or columns (kLinDw: whole runs of 128), which a
// wave keeps in registers, group l in lane l, where there are at most 64: a
// search then needs no memory (4096 rows, dw of 4096 x 2048: 64 groups 251 us,
// 65 groups 278 to 286).
template <class CF, int KIND>
struct Groups {
    int begin, len, before, tiles;  // before, tiles: row tiles (kLinFwd), runs (kLinDw)
    bool kept;
    __device__ __forceinline__ void init(const Fp8Args& g) {
        begin = len = before = tiles = 0;
        kept = g.offsets && g.E <= 64;
        if (!kept) return;
        const int lane = (int)(threadIdx.x & 63);
        int64_t b = 0, n = 0;
        if (lane < g.E) group_rows(g.offsets, lane, g.T, b, n);
        tiles = (int)((n + (KIND == kLinDw ? 127 : CF::BM - 1)) / (KIND == kLinDw ? 128 : CF::BM));
        before = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(before, d, 64);
            if (lane >= d) before += o;
        }
        before -= tiles;
        begin = (int)b;
        len = (int)n;
    }
    // tiles of the launch
    __device__ __forceinline__ uint32_t total(const Fp8Args& g) const {
        if (KIND == kLinDw || !g.offsets) return (uint32_t)g.tiles;
        const int64_t rows = kept ? (int)get_lane((uint32_t)(before + tiles), 63) : ragged_total(g.offsets, g.E, g.T, CF::BM);
        return (uint32_t)min(g.tiles, rows * g.tiles_n);
    }
    // kLinFwd: the group of tile t; false: past the last
    __device__ __forceinline__ bool find(const Fp8Args& g, uint32_t t, RaggedGroup& r) const {
        if (!kept) return ragged_find(g.offsets, g.E, g.T, CF::BM, t, g.tiles_n, r);
        const uint64_t hit = __ballot((int64_t)(before + tiles) * g.tiles_n > t);
        if (!hit) return false;
        r.e = __builtin_ctzll(hit);
        r.begin = (int)get_lane((uint32_t)begin, r.e);
        r.len = (int)get_lane((uint32_t)len, r.e);
        r.tiles = (int)get_lane((uint32_t)tiles, r.e);
        r.before = (int)get_lane((uint32_t)before, r.e);
        return true;
    }
    // kLinDw: group e's columns, in pairs
    __device__ __forceinline__ void columns(const Fp8Args& g, int e, int& first, int& pairs) const {
        first = 0;
        pairs = (int)g.T;
        if (!g.offsets) return;
        int64_t runs = 0, n = 0;
        if (kept) {
            runs = (int)get_lane((uint32_t)before, e);
            n = (int)get_lane((uint32_t)tiles, e);
        } else {
            int mine = 0;
            for (int i = (int)(threadIdx.x & 63); i < e; i += 64) {
                int64_t b, l;
                group_rows(g.offsets, i, g.T, b, l);
                mine += (int)((l + 127) / 128);
            }
#pragma unroll
            for (int d = 32; d; d >>= 1) mine += __shfl_xor(mine, d, 64);
            runs = __builtin_amdgcn_readfirstlane(mine);
            int64_t b, l;
            group_rows(g.offsets, e, g.T, b, l);
            n = __builtin_amdgcn_readfirstlane((int)((l + 127) / 128));
        }
        // (offsets that break the rules do not lead out of the matrix)
        first = (int)min(runs * 64, g.K);
        pairs = (int)min(n * 64, g.K - first);
    }
};

// Item i of the launch, as for the bf16 products (fetch in ve_linear_tiles.h):
// false if there is none, nor any later one of this workgroup.
template <class CF, int KIND>
__device__ __forceinline__ bool item_at(const Fp8Args& g, const Groups<CF, KIND>& groups, uint32_t total, uint32_t i, Work& w) {
    uint32_t t, in;
    int tm, ti, tj, K;
    w.e = 0;
    w.slice = 0;
    w.begin = 0;
    w.len = (int)g.T;
    if (g.ksplit > 1) {
        t = i / (uint32_t)g.ksplit;
        w.slice = (int)(i - t * g.ksplit);
        if (t >= total) return false;
    } else if (KIND == kLinDw) {
        const uint32_t in_e = total / (uint32_t)g.E, part = (in_e + 7) / 8, j = i / 8;
        w.e = (int)(j / part);
        if (w.e >= g.E) return false;
        t = (i % 8) * part + j - w.e * part;
        if (t >= in_e) {  // a hole: the run of this XCD is shorter
            w.rows = 0;
            w.nk = 0;
            return true;
        }
    } else {
        const uint32_t part = (total + 7) / 8, j = i / 8;
        t = (i % 8) * part + j;
        if (j >= part || t >= total) return false;
    }
    w.t = in = t;
    if constexpr (KIND == kLinDw) {
        tm = (int)((g.M + CF::BM - 1) / CF::BM);
        groups.columns(g, w.e, w.begin, w.len);
        K = w.len;
    } else {
        tm = (int)((g.T + CF::BM - 1) / CF::BM);
        if (g.offsets) {
            RaggedGroup r;
            if (!groups.find(g, t, r)) return false;
            w.e = r.e;
            w.begin = (int)r.begin;
            w.len = (int)r.len;
            tm = r.tiles;
            in = t - (uint32_t)r.before * g.tiles_n;
        }
        K = (int)g.K;
    }
    tile_in<CF>(g, in, tm, ti, tj);
    w.col0 = tj * CF::BN;
    const int i0 = ti * CF::BM;
    w.rows = min((KIND == kLinDw ? (int)g.M : w.len) - i0, CF::BM);
    w.row0 = KIND == kLinDw ? i0 : w.begin + i0;
    w.kbeg = 0;
    w.nk = (int)(((uint32_t)K + BK - 1) / BK);
    if (g.ksplit > 1) {
        const int per = (w.nk + g.ksplit - 1) / g.ksplit;
        w.kbeg = min(w.slice * per, w.nk);
        w.nk = min(per, w.nk - w.kbeg);
    }
    return true;
}

// Exchanges between the halves of a wave, and between its even and odd rows
// of 16 lanes: a's upper half (odd rows) against b's lower half (even rows).
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap_rows(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// The bf16 epilogue of dw without LDS.  In a 32 x 32 block a lane of half h
// has 4 consecutive columns 8 q + 4 h of row lane % 32 for each q.  As bf16 (2
// dwords a q), exchanging q, q + 1 between the halves gives it 8 consecutive
// ones, and exchanging the two pairs of q between the rows of 16 lanes gives
// lanes 16 bytes each of 16 rows, 64 consecutive bytes a row.  Two blocks side
// by side exchange those between lanes i and i + 8, so that a store covers 8
// rows of 128 bytes, whole lines.  The exchanges undo themselves, which is how
// what dw holds comes to the accumulators.  dw is written past the caches: its
// next reader is far away, and the operands stay in them.  A contraction of
// 512 tokens, 7168 -> 65536 (7,168 tiles of 4 steps): 345 us; 364 without the
// streaming hint, 381 through LDS as the general epilogue, 441 in rows of 64
// bytes.
// What two blocks' lanes have of rows i (i < 16), 4 dwords each, to rows i and
// i + 8 (i < 8) of both side by side, and back.
__device__ __forceinline__ void swap_eights(uint32_t& a, uint32_t& b, bool low) {
    const uint32_t give = low ? b : a;
    const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0x128, 0xf, 0xf, true);  // row_ror:8
    const uint32_t na = low ? a : got, nb = low ? got : b;
    a = na;
    b = nb;
}

// The packed values of two blocks side by side, p[block][2 q + d], as four
// stores (16 t + 8 u + lane % 8 the row, p[u][4 t + d] its dwords), and back.
__device__ __forceinline__ void turn_blocks(uint32_t (&p)[2][8], bool low, bool back) {
    auto inner = [&]() {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (back) {
#pragma unroll
                for (int d = 0; d < 4; ++d) swap_rows(p[c][d], p[c][4 + d]);
            }
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                swap_halves(p[c][d], p[c][2 + d]);
                swap_halves(p[c][4 + d], p[c][6 + d]);
            }
            if (!back) {
#pragma unroll
                for (int d = 0; d < 4; ++d) swap_rows(p[c][d], p[c][4 + d]);
            }
        }
    };
    if (!back) inner();
#pragma unroll
    for (int i = 0; i < 8; ++i) swap_eights(p[0][i], p[1][i], low);
    if (back) inner();
}

template <class CF, bool ADD>
__device__ __forceinline__ void dw_epilogue(const Work& w, f32x16 (&acc)[CF::TM][CF::TN], int wr, int wc, int lane) {
    constexpr int TM = CF::TM, TN = CF::TN;
    const LinArgs g = args_again();
    const int ld = (int)g.lddw, col0 = w.col0 + wc * CF::WN, r = lane & 7;
    const bool low = (lane & 8) == 0;
    // the lane's columns of two blocks in a store
    const int sc = 8 * (lane >> 5) + 16 * ((lane >> 4) & 1) + 32 * ((lane >> 3) & 1);
    VE_GLOBAL char* out =
        (VE_GLOBAL char*)((uint16_t*)g.dw + w.e * g.dw_group + (int64_t)(w.row0 + wr * CF::WM) * g.lddw + col0);
    const int left = w.rows - wr * CF::WM - r;  // rows from the lane's first on
    u32x4 held[ADD ? 4 : 1];                    // of the next two blocks
    auto load_held = [&](int a, int b) {
        if constexpr (ADD) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                held[t] = u32x4{0, 0, 0, 0};
                if (col0 + 64 * b + sc < (int)g.N && left > 32 * a + 8 * t)
                    held[t] = *(const VE_GLOBAL u32x4*)(out + (uint32_t)((32 * a + 8 * t + r) * ld + 64 * b + sc) * 2);
            }
        }
    };
    load_held(0, 0);
    // (not unrolled: the compiler would copy every accumulator at once)
#pragma unroll 1
    for (int b = 0; b < TN / 2; ++b) {
        const bool in = col0 + 64 * b + sc < (int)g.N;
#pragma unroll
        for (int a = 0; a < TM; ++a) {
            float v[2][16];
#pragma unroll
            for (int e = 0; e < TN / 2; ++e)
                if (b == e) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[c][i] = acc[a][2 * e + c][i];
                }
            uint32_t p[2][8];
            if constexpr (ADD) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int d = 0; d < 4; ++d) p[t & 1][4 * (t >> 1) + d] = held[t][d];
                load_held(a + 1 < TM ? a + 1 : 0, a + 1 < TM ? b : b + 1);
                turn_blocks(p, low, true);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[c][i] += i & 1 ? bf_hi(p[c][i >> 1]) : bf_lo(p[c][i >> 1]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) p[c][i] = pack_bf16x2(v[c][2 * i], v[c][2 * i + 1]);
            turn_blocks(p, low, false);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (in && left > 32 * a + 8 * t) {
                    const uint32_t* q = &p[t & 1][4 * (t >> 1)];
                    stv<true>((VE_GLOBAL u32x4*)(out + (uint32_t)((32 * a + 8 * t + r) * ld + 64 * b + sc) * 2),
                              u32x4{q[0], q[1], q[2], q[3]});
                }
        }
    }
}

// The same in fp32: exchanging q, q + 1 between the rows of 16 lanes, then both
// pairs of q between lanes i and i + 8, a store covers 8 rows of the block's
// 128 bytes.
template <class CF, bool ADD>
__device__ __forceinline__ void dw_epilogue_fp32(const Work& w, f32x16 (&acc)[CF::TM][CF::TN], int wr, int wc, int lane) {
    constexpr int TM = CF::TM, TN = CF::TN;
    const LinArgs g = args_again();
    const int ld = (int)g.lddw, col0 = w.col0 + wc * CF::WN, r = lane & 7;
    const bool low = (lane & 8) == 0;
    const int sc = 4 * (lane >> 5) + 8 * ((lane >> 4) & 1) + 16 * ((lane >> 3) & 1);  // the lane's columns of a block
    VE_GLOBAL char* out =
        (VE_GLOBAL char*)((float*)g.dw + w.e * g.dw_group + (int64_t)(w.row0 + wr * CF::WM) * g.lddw + col0);
    const int left = w.rows - wr * CF::WM - r;  // rows from the lane's first on
#pragma unroll 1
    for (int b = 0; b < TN; ++b) {
        const bool in = col0 + 32 * b + sc < (int)g.N;
        f32x4 held[ADD ? TM : 1][4];
        if constexpr (ADD) {
#pragma unroll
            for (int a = 0; a < TM; ++a)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    held[a][t] = f32x4{0.f, 0.f, 0.f, 0.f};
                    if (in && left > 32 * a + 8 * t)
                        held[a][t] = *(const VE_GLOBAL f32x4*)(out + (uint32_t)((32 * a + 8 * t + r) * ld + 32 * b + sc) * 4);
                }
        }
#pragma unroll
        for (int a = 0; a < TM; ++a) {
            uint32_t p[4][4];  // [q][column]; then the stores' rows 16 (q % 2) + 8 (q / 2)
#pragma unroll
            for (int e = 0; e < TN; ++e)
                if (b == e) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) p[i >> 2][i & 3] = __float_as_uint(acc[a][e][i]);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                swap_rows(p[0][i], p[1][i]);
                swap_rows(p[2][i], p[3][i]);
                swap_eights(p[0][i], p[2][i], low);
                swap_eights(p[1][i], p[3][i], low);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int t = 2 * (q & 1) + (q >> 1);
                if (in && left > 32 * a + 8 * t) {
                    f32x4 v = {__uint_as_float(p[q][0]), __uint_as_float(p[q][1]), __uint_as_float(p[q][2]), __uint_as_float(p[q][3])};
                    if constexpr (ADD) v += held[a][t];
                    stv<true>((VE_GLOBAL f32x4*)(out + (uint32_t)((32 * a + 8 * t + r) * ld + 32 * b + sc) * 4), v);
                }
            }
        }
    }
}

template <class CF, int KIND>
__device__ __forceinline__ void fp8_epilogue(int finish, const Work& w, f32x16 (&acc)[CF::TM][CF::TN], unsigned char* sw,
                                             int wr, int wc, int lane) {
    if constexpr (KIND == kLinDw) {
        if (finish == kFinishStore) dw_epilogue<CF, false>(w, acc, wr, wc, lane);
        else if (finish == kFinishAdd) dw_epilogue<CF, true>(w, acc, wr, wc, lane);
        else epilogue_of<CF, KIND, kFinishAll>(w, acc, sw, wr, wc, lane);
    } else {
        epilogue<CF, KIND>(finish, w, acc, sw, wr, wc, lane);
    }
}

// The arguments, read from memory again.
__device__ __forceinline__ Fp8Args fp8_args_again() {
    auto p = (const __attribute__((address_space(4))) uint32_t*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    static_assert(sizeof(Fp8Args) % 4 == 0, "whole words");
    uint32_t w[sizeof(Fp8Args) / 4];
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Fp8Args) / 4); ++i) w[i] = p[i];
    Fp8Args h;
    __builtin_memcpy(&h, w, sizeof(h));
    return h;
}

// Workgroups that stay on their CUs and run one stream of steps over their
// items, as the bf16 product's (ve_linear.hip): a step has the same bytes,
// the same LDS reads and as many cycles of MFMA, for twice the contraction.
// The exponents of a step are two loads of a dword a lane, two steps ahead,
// which the lanes exchange once the step's tile is there.
//
// 8192 tokens, 8192 -> 28672: 1,440 to 1,515 us once warm (2,540 to 2,670
// TFLOP/s; the library's product with one scale a matrix 3,000 to 3,160), with
// SiLU and z 1,560 to 1,600; dw at 8192^3 2,520 to 2,760 TFLOP/s.  By the counters the
// MFMAs are busy 66% of the cycles at 1.93 GHz: the rest of a step waits for
// its loads, which have half a step to land.  Barriers and loads at other
// places of the step were within 1%.
template <class CF, int KIND, int FORMAT>
__global__ void __launch_bounds__(CF::THREADS, CF::PER_CU) k_fp8(Fp8Args g) {
    constexpr int TM = CF::TM, TN = CF::TN, WM = CF::WM, WN = CF::WN;
    constexpr int NF = TM + TN, MM = TM * TN, H = MM / 2;  // H: MFMAs of a step's second half before its barrier
    constexpr int EB = KIND == kLinDw ? TN : 1;  // exponents of the columns: each lane's, or the wave's
    __shared__ __attribute__((aligned(1024))) unsigned char smem[CF::SMEM];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wr = wave / CF::WAVES_N, wc = wave % CF::WAVES_N;
    uint16_t* ops = (uint16_t*)smem;
    unsigned char* sw = smem + CF::STAGES_BYTES + wave * CF::OUT_BYTES;
    auto stage = [&](uint32_t s) { return ops + (s & 1) * CF::STAGE_ELEMS; };

    Groups<CF, KIND> groups;
    groups.init(g);
    const uint32_t total = groups.total(g);
    uint32_t ci = blockIdx.x, li = ci;  // items computed and loaded
    Work cw;
    bool cok = item_at<CF, KIND>(g, groups, total, ci, cw);
    if (!cok) return;
    typedef Operand<false, CF::BM, CF::WAVES, true> OpA;
    typedef Operand<false, CF::BN, CF::WAVES, true> OpB;
    OpA A;
    OpB B;
    Exponents XA, XB;
    constexpr int PA = OpA::PIECES, PB = OpB::PIECES, P = PA + PB, SPAN = MM;
    static_assert(SPAN <= MM - H + MM, "loads of a step must be issued before its barrier");

    // The loads' position: step lk of the item's steps up to lend; lok: there
    // is an item.
    int lk = 0, lend = 0;
    bool lok = true;
    uint32_t item = 0;
    auto next_loaded = [&](bool first) {  // the next item with steps
        const Fp8Args h = fp8_args_again();
        Work w;
        do {
            if (!first) li += gridDim.x;
            first = false;
            lok = __builtin_amdgcn_readfirstlane(item_at<CF, KIND>(h, groups, total, li, w)) != 0;
            w.nk = __builtin_amdgcn_readfirstlane(w.nk);
        } while (lok && w.nk == 0);
        if (!lok) return;
        // what the item's epilogue will need, in lanes of a vector register
        put_lane(item, 0, (uint32_t)w.e);
        put_lane(item, 1, (uint32_t)w.row0);
        put_lane(item, 2, (uint32_t)w.rows);
        put_lane(item, 3, (uint32_t)w.col0);
        put_lane(item, 4, (uint32_t)w.nk);
        put_lane(item, 5, (uint32_t)w.slice);
        put_lane(item, 6, w.t);
        lk = __builtin_amdgcn_readfirstlane(w.kbeg);
        lend = __builtin_amdgcn_readfirstlane(w.kbeg + w.nk);
        const int cols = min((int)h.N - w.col0, CF::BN);
        const int ra = w.row0 + wr * WM, rb = w.col0 + wc * WN;
        if constexpr (KIND == kLinDw) {
            A.init(h.A + w.row0 * h.lda + w.begin, h.lda, w.rows, w.len, lane, wave);
            B.init(h.B + w.col0 * h.ldb + w.begin, h.ldb, cols, w.len, lane, wave);
            XA.init(h.sa + (w.begin / BK + lk) * h.ld_sa, h.ld_sa, ra, h.sa_rows);
            XB.init(h.sb + (w.begin / BK + lk) * h.ld_sb, h.ld_sb, rb, h.sb_rows);
        } else {
            A.init(h.A + w.row0 * h.lda, h.lda, w.rows, (int)h.K, lane, wave);
            B.init(h.B + w.e * h.b_group + w.col0 * h.ldb, h.ldb, cols, (int)h.K, lane, wave);
            XA.init(h.sa + lk * h.ld_sa, h.ld_sa, ra, h.sa_rows);
            XB.init(h.sb + w.e * h.sb_group + lk * h.ld_sb, h.ld_sb, rb >> 7, h.sb_rows);
        }
        A.make_uniform();
        B.make_uniform();
    };
    uint32_t raw_a = 0, raw_b = 0;  // exponents of the step that the loads are at
    int at_a = 0, at_b = 0;         // and their first rows
    auto begin = [&]() {
        A.begin(lk, lok);
        B.begin(lk, lok);
    };
    auto begin_exponents = [&]() {
        raw_a = XA.load(lane, lok);
        raw_b = XB.load(lane, lok);
        at_a = XA.row;
        at_b = XB.row;
    };
    auto advance = [&]() {
        XA.next();
        XB.next();
        if (lok && ++lk >= lend) next_loaded(false);
    };
    auto advance_inside = [&]() {
        XA.next();
        XB.next();
        ++lk;
    };
    // the pieces of slot s (s MFMAs behind the barrier)
    auto pieces = [&](int slot, uint32_t s) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (p * SPAN / P == slot) {
                if (p < PA) A.piece(stage(s), p);
                else B.piece(stage(s) + CF::A_ELEMS, p - PA);
            }
    };
    auto barrier = [&]() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    f32x16 acc[TM][TN];
    i32x8 fa[2][TM], fb[2][TN];
    int ea[TM], eb[EB];             // exponents of the step
    uint32_t na[TM], nb[EB];        // of the next: dwords, and where in them
    uint32_t shift_a, shift_b;
    auto exchange = [&]() {
#pragma unroll
        for (int a = 0; a < TM; ++a) na[a] = spread_dword(raw_a, at_a, a, lane);
        shift_a = spread_shift(at_a, lane);
        if constexpr (KIND == kLinDw) {
#pragma unroll
            for (int b = 0; b < TN; ++b) nb[b] = spread_dword(raw_b, at_b, b, lane);
            shift_b = spread_shift(at_b, lane);
        } else {
            nb[0] = get_lane(raw_b, 0);
            shift_b = 8 * (at_b & 3);
        }
    };
    auto exponents = [&]() {
#pragma unroll
        for (int a = 0; a < TM; ++a) ea[a] = (int)(na[a] >> shift_a);
#pragma unroll
        for (int b = 0; b < EB; ++b) eb[b] = (int)(nb[b] >> shift_b);
    };
    // fragment f of half kk in the order the MFMAs need them: A0, all B, the other A
    auto frag1 = [&](int f, int kk, uint32_t s) {
        const uint16_t* st = stage(s);
        if (f == 0 || f > TN) {
            const int a = f == 0 ? 0 : f - TN;
            fa[kk][a] = fragment<OpA>(st, wr * WM + a * 32, kk, lane);
        } else {
            fb[kk][f - 1] = fragment<OpB>(st + CF::A_ELEMS, wc * WN + (f - 1) * 32, kk, lane);
        }
    };
    f32x16 zero;
#pragma unroll
    for (int r = 0; r < 16; ++r) zero[r] = 0.f;
    auto mfma = [&](bool first, int kk, int m) {
        const int a = m / TN, b = m % TN;
        acc[a][b] = mfma_fp8(fb[kk][b], fa[kk][a], first ? zero : acc[a][b], eb[b % EB], ea[a], FORMAT);
    };

    next_loaded(true);
    if (!lok) {  // items without steps only: their rows of dw are zeros, or kept
        A.init(g.A, g.lda, 1, 1, lane, wave);
        B.init(g.B, g.ldb, 1, 1, lane, wave);
        XA.init(g.sa, 0, 0, 0);
        XB.init(g.sb, 0, 0, 0);
    }
    begin();
    begin_exponents();
#pragma unroll
    for (int q = 0; q < PA; ++q) A.piece(stage(0), q);
#pragma unroll
    for (int q = 0; q < PB; ++q) B.piece(stage(0) + CF::A_ELEMS, q);
    __builtin_amdgcn_s_waitcnt(kWaitAll);
    exchange();
    exponents();
    advance();
    begin();
    begin_exponents();
#pragma unroll
    for (int m = 0; m < MM - H; ++m) pieces(m, 1);
    barrier();
#pragma unroll
    for (int f = 0; f < NF; ++f) frag1(f, 0, 0);

    uint32_t s = 0;  // steps computed, over all items
    while (cok) {
        // Every MFMA is followed by its share of what feeds the later ones,
        // in this order (the scheduling barriers keep it).  In the middle of a
        // step's second half all its reads are complete: the barrier there
        // frees its stage and makes the next one visible, and from there on
        // the loads of the step after the next go out into the freed stage.
        // An item's first step starts from 0 (clearing 256 registers first
        // would take 1,024 cycles, half a step).
        auto step = [&](bool first, auto&& next) {
#pragma unroll
            for (int m = 0; m < MM; ++m) {
                mfma(first, 0, m);
#pragma unroll
                for (int f = m * NF / MM; f < (m + 1) * NF / MM; ++f) frag1(f, 1, s);
                pieces(MM - H + m, s + 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            next();
#pragma unroll
            for (int m = 0; m < H; ++m) mfma(false, 1, m);
            __builtin_amdgcn_sched_barrier(0);
            // this wave's loads and LDS reads are complete, then everyone's
            __builtin_amdgcn_s_waitcnt(kWaitAll);
            barrier();
            exchange();
            begin();
            begin_exponents();
#pragma unroll
            for (int m = H; m < MM; ++m) {
                mfma(false, 1, m);
#pragma unroll
                for (int f = (m - H) * NF / (MM - H); f < (m - H + 1) * NF / (MM - H); ++f) frag1(f, 0, s + 1);
                pieces(m - H, s + 2);
                __builtin_amdgcn_sched_barrier(0);
            }
            exponents();
            ++s;
        };
        // Nothing of the previous item's epilogue may be pending for the
        // compiler here (it would wait in every step); the other workgroup of
        // the CU fills the time.
        if constexpr (CF::PER_CU > 1) __builtin_amdgcn_s_waitcnt(wait_vm(0));
        // the loads leave this item behind in its last two steps
        const int nk = __builtin_amdgcn_readfirstlane(cw.nk);
        if (nk > 0) {
            step(true, advance);
        } else {
#pragma unroll
            for (int a = 0; a < TM; ++a)
#pragma unroll
                for (int b = 0; b < TN; ++b) acc[a][b] = zero;
        }
        int kt = 1;
        for (; kt + 2 < nk; ++kt) step(false, advance_inside);
        for (; kt < nk; ++kt) step(false, advance);
        // the loads' position waits in a vector register while the epilogue
        // needs the scalar ones
        uint32_t keep = 0;
        A.stash(keep, 0);
        B.stash(keep, 5);
        XA.stash(keep, 10);
        XB.stash(keep, 15);
        put_lane(keep, 20, (uint32_t)lk);
        put_lane(keep, 21, (uint32_t)lend);
        put_lane(keep, 22, (uint32_t)lok);
        put_lane(keep, 23, li);
        put_lane(keep, 24, (uint32_t)at_a);
        put_lane(keep, 25, (uint32_t)at_b);
        if (cw.rows > 0) fp8_epilogue<CF, KIND>(fp8_args_again().finish, cw, acc, sw, wr, wc, lane);
        ci += gridDim.x;
        if (get_lane(keep, 22) != 0 && get_lane(keep, 23) == ci) {  // the item the loads are at
            cw.e = (int)get_lane(item, 0);
            cw.row0 = (int)get_lane(item, 1);
            cw.rows = (int)get_lane(item, 2);
            cw.col0 = (int)get_lane(item, 3);
            cw.nk = (int)get_lane(item, 4);
            cw.slice = (int)get_lane(item, 5);
            cw.t = get_lane(item, 6);
        } else {
            cok = item_at<CF, KIND>(fp8_args_again(), groups, total, ci, cw);
        }
        A.unstash(keep, 0);
        B.unstash(keep, 5);
        XA.unstash(keep, 10);
        XB.unstash(keep, 15);
        lk = (int)get_lane(keep, 20);
        lend = (int)get_lane(keep, 21);
        lok = get_lane(keep, 22) != 0;
        li = get_lane(keep, 23);
        at_a = (int)get_lane(keep, 24);
        at_b = (int)get_lane(keep, 25);
        begin();
    }
    // the loads past the last step (of nothing) land before the end
    __builtin_amdgcn_s_waitcnt(kWaitAll);
}

// Whether a lane's half of row 32 f + lane % 32, of `rows` from r0 on, holds what
// bf16 cannot under exponent e: a code other than 0, or a NaN scale.
template <class Op>
__device__ __forceinline__ bool leaves_bf16(const uint16_t* st, int r0, int f, int lane, int rows, int e, int format) {
    if (32 * f + (lane & 31) >= rows || bf16_exponent(e, format)) return false;
    uint32_t any = (e & 255) == 255;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
        const i32x8 c = fragment<Op>(st, r0 + 32 * f, kk, lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) any |= (uint32_t)c[i] & 0x7f7f7f7fu;
    }
    return any != 0;
}

// dw in fp32: one item a workgroup, codes turned to bf16 between LDS and the
// MFMAs.  One stage of LDS and three workgroups a CU, which load and compute in
// turn: 887 to 922 us at 8192^3 (1,190 to 1,240 TFLOP/s; with two workgroups 4%
// longer), and 16 groups of 777 rows in all, 2880 -> 2880, whose 0.53 GB of
// results bind, 113 us (4.7 TB/s; with two 122).  Looking for what bf16 cannot hold takes 3% of the first
// (860 us without), 10% where blocks of zeros make it look at codes.
template <class CF, int FORMAT>
__global__ void __launch_bounds__(CF::THREADS, 3) k_fp8_exact(Fp8Args g) {
    constexpr int KIND = kLinDw;
    constexpr int TM = CF::TM, TN = CF::TN, WM = CF::WM, WN = CF::WN;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[CF::STAGE_ELEMS * 2 + CF::WAVES * CF::OUT_BYTES];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wr = wave / CF::WAVES_N, wc = wave % CF::WAVES_N;
    Work w;
    Groups<CF, KIND> groups;
    groups.init(g);
    if (!item_at<CF, KIND>(g, groups, (uint32_t)g.tiles, blockIdx.x, w) || w.rows == 0) return;
    typedef Operand<false, CF::BM, CF::WAVES, true> OpA;
    typedef Operand<false, CF::BN, CF::WAVES, true> OpB;
    OpA A;
    OpB B;
    const int cols = min((int)g.N - w.col0, CF::BN);
    A.init(g.A + w.row0 * g.lda + w.begin, g.lda, w.rows, w.len, lane, wave);
    B.init(g.B + w.col0 * g.ldb + w.begin, g.ldb, cols, w.len, lane, wave);
    Exponents XA, XB;
    uint16_t* st = (uint16_t*)smem;
    f32x16 acc[TM][TN];
    uint32_t raw_a, raw_b;
    auto start = [&]() {
        XA.init(g.sa + (w.begin / BK + w.kbeg) * g.ld_sa, g.ld_sa, w.row0 + wr * WM, g.sa_rows);
        XB.init(g.sb + (w.begin / BK + w.kbeg) * g.ld_sb, g.ld_sb, w.col0 + wc * WN, g.sb_rows);
#pragma unroll
        for (int a = 0; a < TM; ++a)
#pragma unroll
            for (int b = 0; b < TN; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;
    };
    auto load = [&](int kt) {
        A.begin(kt, true);
        B.begin(kt, true);
#pragma unroll
        for (int q = 0; q < OpA::PIECES; ++q) A.piece(st, q);
#pragma unroll
        for (int q = 0; q < OpB::PIECES; ++q) B.piece(st + CF::A_ELEMS, q);
        raw_a = XA.load(lane, true);
        raw_b = XB.load(lane, true);
        XA.next();
        XB.next();
        __builtin_amdgcn_s_waitcnt(kWaitAll);
    };
    int ea[TM], eb[TN];
    auto exponents = [&]() {
#pragma unroll
        for (int a = 0; a < TM; ++a) ea[a] = spread(raw_a, XA.row, a, lane);
#pragma unroll
        for (int b = 0; b < TN; ++b) eb[b] = spread(raw_b, XB.row, b, lane);
    };
    start();
    const int rows_in = w.rows - wr * WM, cols_in = cols - wc * WN;  // the wave's rows and columns that exist
    const bool dword_a = XA.holds(lane, min(WM, rows_in)), dword_b = XB.holds(lane, min(WN, cols_in));
    bool past = false;
    for (int kt = w.kbeg; kt < w.kbeg + w.nk; ++kt) {
        load(kt);
        // Exponents past bf16's are seldom, but for blocks of zeros, which have
        // 0: looked for in the dwords, while the others' loads land.
        const bool seldom = __any((dword_a && !bf16_exponents(raw_a, FORMAT)) || (dword_b && !bf16_exponents(raw_b, VE_E4M3)));
        __syncthreads();
        exponents();
        if (seldom) {
#pragma unroll
            for (int a = 0; a < TM; ++a) past |= leaves_bf16<OpA>(st, wr * WM, a, lane, rows_in, ea[a], FORMAT);
#pragma unroll
            for (int b = 0; b < TN; ++b) past |= leaves_bf16<OpB>(st + CF::A_ELEMS, wc * WN, b, lane, cols_in, eb[b], VE_E4M3);
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            i32x8 fa[TM], fb[TN];
#pragma unroll
            for (int a = 0; a < TM; ++a) fa[a] = fragment<OpA>(st, wr * WM + a * 32, kk, lane);
#pragma unroll
            for (int b = 0; b < TN; ++b) fb[b] = fragment<OpB>(st + CF::A_ELEMS, wc * WN + b * 32, kk, lane);
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
        }
        __syncthreads();
    }
    // Where any wave met such values, all take the item again with the 8-bit
    // MFMAs, which take every scale and cut nothing where only one of 8
    // consecutive products is not 0: 8 passes over each half of a block.  (In
    // the loop above a second way to the sums would cost it 14%.)
    uint32_t* met = (uint32_t*)smem;
    if (lane == 0) met[wave] = 0;
    if (past) met[wave] = 1;
    __syncthreads();
    bool again = false;
#pragma unroll
    for (int v = 0; v < CF::WAVES; ++v) again |= __builtin_amdgcn_readfirstlane((int)met[v]) != 0;
    __syncthreads();
    if (again) {
        start();
        for (int kt = w.kbeg; kt < w.kbeg + w.nk; ++kt) {
            load(kt);
            __syncthreads();
            exponents();
#pragma unroll 1
            for (int pass = 0; pass < 16; ++pass) {
                const int kk = pass & 1, at = pass >> 1;
                const uint32_t keep = 255u << (8 * (at & 3));
                i32x8 fa[TM], fb[TN];
#pragma unroll
                for (int a = 0; a < TM; ++a) {
                    fa[a] = fragment<OpA>(st, wr * WM + a * 32, kk, lane);
#pragma unroll
                    for (int c = 0; c < 8; ++c) fa[a][c] &= (c & 1) == at >> 2 ? (int)keep : 0;
                }
#pragma unroll
                for (int b = 0; b < TN; ++b) fb[b] = fragment<OpB>(st + CF::A_ELEMS, wc * WN + b * 32, kk, lane);
#pragma unroll
                for (int a = 0; a < TM; ++a)
#pragma unroll
                    for (int b = 0; b < TN; ++b) acc[a][b] = mfma_fp8(fb[b], fa[a], acc[a][b], eb[b], ea[a], FORMAT);
            }
            __syncthreads();
        }
    }
    if (g.finish == kFinishWide) dw_epilogue_fp32<CF, false>(w, acc, wr, wc, lane);
    else if (g.finish == kFinishWideAdd) dw_epilogue_fp32<CF, true>(w, acc, wr, wc, lane);
    else epilogue_of<CF, KIND, kFinishAll>(w, acc, smem + CF::STAGE_ELEMS * 2 + wave * CF::OUT_BYTES, wr, wc, lane);
}

// Few rows a group (forward and dx): bound by reading the weights.  A
// workgroup takes at most 16 output columns (per) of at most 16 MT rows of one group, and its
// waves a share of the contraction each, straight from memory to the MFMAs
// (16x16x128: a lane 32 codes of one row, read as 64 consecutive bytes of 16
// rows at a time), U blocks in flight; then they join their sums.
template <int MT> struct FewRows { static constexpr int BM = 16 * MT; };
constexpr int kFewWaves = 8;
template <int MT, int U, int FORMAT>
__global__ void __launch_bounds__(64 * kFewWaves) k_fp8_few(Fp8Args g, int col_blocks, int per) {
    constexpr int BM = 16 * MT;
    __shared__ float sums[kFewWaves][BM][16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const uint32_t t = blockIdx.x / (uint32_t)col_blocks;
    const int n0 = (int)(blockIdx.x - t * col_blocks) * per;
    int e = 0, rows = (int)min(g.T - (int64_t)t * BM, (int64_t)BM);
    int64_t row0 = (int64_t)t * BM;
    if (g.offsets) {
        Groups<FewRows<MT>, kLinFwd> groups;
        groups.init(g);
        RaggedGroup r;
        if (!groups.find(g, t, r)) return;
        const int64_t in = (int64_t)(t - (uint32_t)r.before) * BM;
        e = r.e;
        row0 = r.begin + in;
        rows = (int)min(r.len - in, (int64_t)BM);
    }
    const int r = lane & 15, cols = min((int)g.N - n0, per), bytes = (int)g.K * 2;
    const int ldw = (int)g.ldb * 2, ldx = (int)g.lda * 2;
    // reads past the last row or column leave the buffers and return 0
    const __amdgpu_buffer_rsrc_t ws = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(g.B + e * g.b_group + n0 * g.ldb), (short)0, (cols - 1) * ldw + bytes, 0x00020000);
    const __amdgpu_buffer_rsrc_t xs =
        __builtin_amdgcn_make_buffer_rsrc((void*)(g.A + row0 * g.lda), (short)0, (rows - 1) * ldx + bytes, 0x00020000);
    const uint8_t* sw = g.sb + e * g.sb_group + (n0 >> 7);
    const uint8_t* sx = g.sa + row0;
    f32x4 acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int nb = (bytes + 127) / 128, first = nb * wave / kFewWaves, last = nb * (wave + 1) / kFewWaves;
    for (int k0 = first; k0 < last; k0 += U) {
        u32x4 w[U][2], x[U][MT][2];
        int ew[U], ex[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = k0 + u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = kb * 128 + 64 * h + 16 * (lane >> 4);
                const bool in = kb < last && at < bytes;
                w[u][h] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(ws, in ? r * ldw + at : (int)0x80000000, 0, 0));
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    x[u][m][h] = __builtin_bit_cast(
                        u32x4, __builtin_amdgcn_raw_buffer_load_b128(xs, in ? (16 * m + r) * ldx + at : (int)0x80000000, 0, 0));
            }
            const int kc = min(kb, nb - 1);
            ew[u] = ((const VE_GLOBAL uint8_t*)sw)[kc * g.ld_sb];
#pragma unroll
            for (int m = 0; m < MT; ++m) ex[u][m] = ((const VE_GLOBAL uint8_t*)sx)[kc * g.ld_sa + min(16 * m + r, rows - 1)];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const i32x8 b = {(int)w[u][0].x, (int)w[u][0].y, (int)w[u][0].z, (int)w[u][0].w,
                             (int)w[u][1].x, (int)w[u][1].y, (int)w[u][1].z, (int)w[u][1].w};
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const i32x8 c = {(int)x[u][m][0].x, (int)x[u][m][0].y, (int)x[u][m][0].z, (int)x[u][m][0].w,
                                 (int)x[u][m][1].x, (int)x[u][m][1].y, (int)x[u][m][1].z, (int)x[u][m][1].w};
                acc[m] = FORMAT == VE_E4M3
                             ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, c, acc[m], 0, 0, 0, ew[u], 0, ex[u][m])
                             : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, c, acc[m], 0, 1, 0, ew[u], 0, ex[u][m]);
            }
        }
    }
    // lane: columns 4 (lane / 16) .. + 3 of row lane % 16
#pragma unroll
    for (int m = 0; m < MT; ++m) *(f32x4*)&sums[wave][16 * m + r][4 * (lane >> 4)] = acc[m];
    __syncthreads();
    const int row = threadIdx.x >> 1, c8 = (threadIdx.x & 1) * 8;
    if (row >= rows || row >= BM) return;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < kFewWaves; ++q) {
        const f32x4 a = *(const f32x4*)&sums[q][row][c8], b = *(const f32x4*)&sums[q][row][c8 + 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] += a[i];
            v[4 + i] += b[i];
        }
    }
    const int cnt = min(max(cols - c8, 0), 8);
    bias8<kLinFwd>(g, e, n0 + c8, cnt, v);
    finish8<kLinFwd>(g, e, row0 + row, n0 + c8, cnt, v, 0);
}

// Workgroups of the few-row form: row tiles (with offsets the most that any
// could need) and columns of each.
struct FewGrid { int64_t tiles; int col_blocks, per; };
FewGrid few_grid(const Fp8Args& g, int mt) {
    FewGrid f;
    f.tiles = g.offsets ? std::min<int64_t>(g.T, g.T / (16 * mt) + g.E) : (g.T + 16 * mt - 1) / (16 * mt);
    // Fewer columns a workgroup where 16 leave CUs without work (one token 8192
    // -> 1024: 7.7 us, with 16 columns 8.5), but not where that reads x of many
    // rows more often (32 rows 2880 -> 2880: 10.4 against 7.8).
    f.per = mt == 1 && f.tiles * ((g.N + 15) / 16) < 2 * kCUs ? 8 : 16;
    f.col_blocks = (int)((g.N + f.per - 1) / f.per);
    return f;
}
int few_mt(const Fp8Args& g) { return g.offsets || g.T <= 16 ? 1 : 2; }

template <int MT, int U>
hipError_t launch_few(Fp8Args g, hipStream_t s) {
    const FewGrid f = few_grid(g, MT);
    g.tiles_n = 1;
    g.tiles = f.tiles;
    const dim3 grid((unsigned)(f.tiles * f.col_blocks)), block(64 * kFewWaves);
    if (g.format == VE_E4M3) hipLaunchKernelGGL((k_fp8_few<MT, U, VE_E4M3>), grid, block, 0, s, g, f.col_blocks, f.per);
    else hipLaunchKernelGGL((k_fp8_few<MT, U, VE_E5M2>), grid, block, 0, s, g, f.col_blocks, f.per);
    return hipGetLastError();
}

template <class CF, int KIND>
hipError_t launch_kind(Fp8Args g, const LinPlan& p, hipStream_t s) {
    g.tiles_n = (int)((g.N + CF::BN - 1) / CF::BN);
    g.ksplit = p.ksplit;
    g.tiles = tiles_of<CF>(g, (LinKind)KIND);
    if (g.tiles == 0) return hipSuccess;
    g.finish = finish_of(g, (LinKind)KIND);
    const int64_t items = items_of(g, (LinKind)KIND);
    const dim3 grid((unsigned)std::min<int64_t>(items, kCUs * CF::PER_CU)), block(CF::THREADS);
    if (g.format == VE_E4M3) hipLaunchKernelGGL((k_fp8<CF, KIND, VE_E4M3>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((k_fp8<CF, KIND, VE_E5M2>), grid, block, 0, s, g);
    if (p.ksplit > 1)
        hipLaunchKernelGGL((k_join<CF, KIND>), dim3((unsigned)(g.tiles * (CF::BM * (CF::BN / 8) / 256))), dim3(256), 0, s, g);
    return hipGetLastError();
}

hipError_t launch_exact(Fp8Args g, const LinPlan& p, hipStream_t s) {
    typedef Cfg128 CF;
    g.tiles_n = (int)((g.N + CF::BN - 1) / CF::BN);
    g.ksplit = p.ksplit;
    g.tiles = tiles_of<CF>(g, kLinDw);
    if (g.tiles == 0) return hipSuccess;
    g.finish = finish_of(g, kLinDw);
    const dim3 grid((unsigned)items_of(g, kLinDw)), block(CF::THREADS);
    if (g.format == VE_E4M3) hipLaunchKernelGGL((k_fp8_exact<CF, VE_E4M3>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((k_fp8_exact<CF, VE_E5M2>), grid, block, 0, s, g);
    if (p.ksplit > 1)
        hipLaunchKernelGGL((k_join<CF, kLinDw>), dim3((unsigned)(g.tiles * (CF::BM * (CF::BN / 8) / 256))), dim3(256), 0, s, g);
    return hipGetLastError();
}

// Microseconds of a product as `items` tiles (or slices) of `steps` steps, as
// for the bf16 products.  Measured: a step of 256 x 256 takes 1.48 us and its
// start and epilogue 5; of a pair of 128 x 128 tiles 1.06 and 4, of a single
// one 0.8.  dw's starts and epilogues, which whole launches of short
// contractions consist of, take 11 and 6.  Against measurements, 128^2 / 256^2
// in us: 32 groups of 4096 rows 7168 -> 2048 146 / 204 (model 126 / 176), of
// 16384 340 / 298; dw of 16 groups 4096 rows 2048 -> 4096 108 / 89, of 40
// groups 2000 rows 1000 -> 1000 46 / 60.
// The exact form's steps take 1.8 and 1.2.
double fp8_us(LinKind kind, bool exact, bool big, int64_t items, int64_t steps, int64_t bytes) {
    const double n = (double)((items + kCUs - 1) / kCUs), st = (double)steps;
    const double pair = exact ? 1.8 : 1.06, single = exact ? 1.2 : 0.8;
    const double sums = bytes ? (double)bytes * 2 / 5e6 + 4 : 0;
    const double start = kind == kLinDw ? 6 : 4, start256 = kind == kLinDw ? 11 : 5;
    if (big) return n * (1.48 * st + start256) + sums;
    const double pairs = (double)((int64_t)n / 2), one = n - 2 * pairs;
    return pairs * (pair * st + start) + one * (single * st + start) + sums;
}

}  // namespace

LinPlan plan_fp8(const Fp8Args& g, LinKind kind) {
    LinPlan p{kPath128, 1, 0, 0};
    const bool exact = kind == kLinDw && g.wide;
    const int64_t pin = option(kOptLinearPath);
    // Few rows against the tiles, us a call: dense 8192 -> 8192 of 1 / 16 / 32
    // / 64 rows 14 / 19 / 26 / 47 against 33 / 34 / 34 / 30; 64 groups 7168 ->
    // 2048 of 1 / 4 / 8 rows on average 119 / 165 / 192 against 142 / 163 / 160.
    if (kind == kLinFwd && (pin == kPathFew || (pin == kPathAuto && g.T <= (g.offsets ? 4 * (int64_t)g.E : 32)))) {
        const FewGrid f = few_grid(g, few_mt(g));
        if (f.tiles <= kMaxGridItems / (64 * kFewWaves) / f.col_blocks) {  // (else the tiles, which fit)
            p.path = kPathFew;
            return p;
        }
    }
    const int64_t K = kind != kLinDw ? g.K : g.offsets ? (g.T / g.E + 127) / 128 * 64 : g.T;
    const int64_t nk = std::max<int64_t>(1, (K + BK - 1) / BK);
    const bool may_split = !g.offsets && option(kOptLinearSplit) != 0;
    const bool far = 2 * std::max(g.lda, g.ldb) >= kFp8Pitch256;  // (lda, ldb: of 2 bytes)
    double best = 0;
    for (int path : {(int)kPath128, (int)kPath256}) {
        if (exact || far ? path != kPath128 : (pin == kPath128 || pin == kPath256) && pin != path) continue;
        int64_t tiles = path == kPath256 ? tiles_of<Cfg256>(g, kind) : tiles_of<Cfg128>(g, kind);
        // (ragged rows: two thirds of a tile more a group, not the most any offsets could need)
        if (kind == kLinFwd && g.offsets) {
            const int64_t bm = path == kPath256 ? 256 : 128;
            tiles = (g.T / bm + (2 * std::min<int64_t>(g.E, g.T) + 2) / 3) * ((g.N + bm - 1) / bm);
        }
        const int64_t slots = kCUs * (path == kPath256 ? Cfg256::PER_CU : Cfg128::PER_CU), area = path == kPath256 ? 65536 : 16384;
        for (int64_t ks = 1; ks <= 32; ++ks) {
            if (ks > 1 && (!may_split || nk / ks < 4 || tiles * ks > slots)) break;
            const double us = fp8_us(kind, exact, path == kPath256, tiles * ks, (nk + ks - 1) / ks, ks > 1 ? tiles * ks * area * 4 : 0);
            if (best == 0 || us < best) {
                best = us;
                p.us = us;
                p.path = path;
                p.ksplit = (int)ks;
                p.partial_bytes = ks > 1 ? ks * tiles * area * 4 : 0;
            }
        }
    }
    return p;
}

hipError_t launch_fp8(Fp8Args g, LinKind kind, const LinPlan& p, hipStream_t s) {
    if (kind == kLinDw && g.wide) return launch_exact(g, p, s);
    if (p.path == kPathFew) return few_mt(g) == 1 ? launch_few<1, 8>(g, s) : launch_few<2, 4>(g, s);
    if (p.path == kPath256)
        return kind == kLinDw ? launch_kind<Cfg256, kLinDw>(g, p, s) : launch_kind<Cfg256, kLinFwd>(g, p, s);
    return kind == kLinDw ? launch_kind<Cfg128, kLinDw>(g, p, s) : launch_kind<Cfg128, kLinFwd>(g, p, s);
}

}  // namespace ve
