// ve_linear_tiles.h -- what the kernels of a product share: tile
// configurations, operands in LDS, the search for a workgroup's tile among
// ragged groups, epilogues, the sum of a split contraction's slices.  The
// products themselves are in ve_linear.hip (bf16) and ve_fp8.hip (8-bit
// floating point, whose codes are taken as pairs: every size along the
// contraction is in elements of 2 bytes).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ve_linear_device.h"

namespace ve {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
#define VE_LDS __attribute__((address_space(3)))

constexpr int kCUs = 256;
constexpr int BK = 64;          // contraction step

// Workgroup tile BM x BN of four waves of WM x WN; two LDS stages of operands
// and 16 rows of output a wave.
template <int BM_, int BN_, int WM_, int WN_>
struct LinCfg {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int WAVES_M = BM / WM, WAVES_N = BN / WN, WAVES = WAVES_M * WAVES_N;
    static constexpr int THREADS = 64 * WAVES;
    static constexpr int TM = WM / 32, TN = WN / 32;
    static constexpr int A_ELEMS = BM * BK, B_ELEMS = BN * BK, STAGE_ELEMS = A_ELEMS + B_ELEMS;
    static constexpr int STAGES_BYTES = 2 * STAGE_ELEMS * 2;
    static constexpr int OUT_BYTES = 16 * WN * 4;  // a wave's 16 output rows, fp32
    static constexpr int SMEM = STAGES_BYTES + WAVES * OUT_BYTES;
    static_assert(SMEM <= 160 * 1024, "LDS");
    static constexpr int PER_CU = 160 * 1024 / SMEM;
};
using Cfg256 = LinCfg<256, 256, 128, 128>;
using Cfg128 = LinCfg<128, 128, 64, 64>;
using Cfg128W = LinCfg<128, 128, 32, 128>;  // a wave holds whole runs of 128 columns

// s_waitcnt operands: at most n vector-memory operations outstanding; every
// vector-memory and LDS operation complete.
constexpr int wait_vm(int n) { return 0x0F70 | (n & 15) | (((n >> 4) & 3) << 14); }
constexpr int kWaitAll = 0x0070;

// Transposing read.  The restricted pointer carries that no store touches
// these bytes while they are read; without it the compiler waits for every
// direct load in flight (which fill the other stage) before the read.
__device__ __forceinline__ s16x4 read_tr(const VE_LDS uint16_t* __restrict__ p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((s16x4 VE_LDS*)p);
}

// A scalar in lane `at` of a vector register.
__device__ __forceinline__ void put_lane(uint32_t& v, int at, uint32_t x) { v = (int)(threadIdx.x & 63) == at ? x : v; }

// ... and back (unsigned: the builtin's signed result would fill the upper
// half of an address with its sign).
__device__ __forceinline__ uint32_t get_lane(uint32_t v, int at) { return (uint32_t)__builtin_amdgcn_readlane((int)v, at); }

// One operand of the workgroup's tile: ROWS tile rows (KC) or columns (KS)
// over the contraction.  The tile of one step is ROWS * 128 bytes, filled in
// pieces of 1 KiB by one wave instruction each (lane l: 16 bytes at 16 l).
template <bool KS, int ROWS, int WAVES, bool DMA>
struct Operand {
    static constexpr int PIECES = ROWS * BK * 2 / 1024 / WAVES;  // per wave and step
    static constexpr int SLOTS = KS ? ROWS / 8 : 8;              // 16-byte slots of an LDS row
    static constexpr int LROWS = 64 / SLOTS;                     // LDS rows of one piece
    static_assert(PIECES * WAVES * 1024 == ROWS * BK * 2, "pieces must divide evenly");
    static_assert(WAVES % 2 == 0, "a lane's slot must not depend on the piece");
    const uint16_t* base;  // KC: row 0, contraction index 0 of the tile; KS: contraction row 0, column 0
    int64_t ld;
    int valid;             // KC: rows; KS: columns (from the tile's first on)
    int kc;                // contraction length
    int lrow, chunk, wave;
    uint32_t voff, step_off;
    __amdgpu_buffer_rsrc_t rs;
    u32x4 reg[DMA ? 1 : PIECES];

    // swizzle of KC rows: consecutive rows of one bank line get distinct slots
    __device__ static __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }
    // KS: 32-byte piece s of contraction row k lies at piece place(s) ^ (k & 3)
    // of its LDS row.  A transposing read touches pieces s, s + 1 (s even) of
    // rows k .. k + 3: eight distinct pieces modulo 256 bytes, and four
    // distinct ones modulo 128 bytes for either s alone.
    __device__ static __forceinline__ int place(int s) { return (s & ~7) | ((s & 1) << 2) | ((s >> 1) & 3); }
    __device__ static __forceinline__ int unplace(int f) { return (f & ~7) | ((f & 3) << 1) | ((f >> 2) & 1); }

    __device__ __forceinline__ void init(const uint16_t* base_, int64_t ld_, int valid_, int kc_, int lane,
                                         int wave_) {
        base = base_; ld = ld_; valid = valid_; kc = kc_; wave = wave_;
        const int slot = lane % SLOTS, row0 = wave * LROWS + lane / SLOTS;  // row of piece 0
        lrow = row0;
        if constexpr (KS) {
            const int f = (slot >> 1) ^ (row0 & 3);
            chunk = unplace(f) * 2 + (slot & 1);
        } else {
            chunk = slot ^ swz(row0);
        }
        voff = (uint32_t)((lrow * ld + chunk * 8) * 2);
    }
    // base, valid, kc and ld in five lanes of a vector register, and back
    __device__ __forceinline__ void stash(uint32_t& keep, int at) const {
        put_lane(keep, at, (uint32_t)(uintptr_t)base);
        put_lane(keep, at + 1, (uint32_t)((uintptr_t)base >> 32));
        put_lane(keep, at + 2, (uint32_t)valid);
        put_lane(keep, at + 3, (uint32_t)kc);
        put_lane(keep, at + 4, (uint32_t)ld);
    }
    __device__ __forceinline__ void unstash(uint32_t keep, int at) {
        const uint64_t lo = get_lane(keep, at), hi = get_lane(keep, at + 1);
        base = (const uint16_t*)(uintptr_t)((hi << 32) | lo);
        valid = (int)get_lane(keep, at + 2);
        kc = (int)get_lane(keep, at + 3);
        ld = (int)get_lane(keep, at + 4);
    }
    // scalars for the compiler, whatever way they were found
    __device__ __forceinline__ void make_uniform() {
        base = (const uint16_t*)uniform64((int64_t)base);
        ld = __builtin_amdgcn_readfirstlane((int)ld);
        valid = __builtin_amdgcn_readfirstlane(valid);
        kc = __builtin_amdgcn_readfirstlane(kc);
    }
    // Direct loads of step kt's tile into the LDS stage at `st`: begin() for
    // the step, then piece() for each piece.  A buffer resource from the
    // step's first element on: reads past the last valid row return 0, and so
    // do those of a KC row past the contraction (sent past the end by hand)
    // and every read of a step that does not exist (not live).
    __device__ __forceinline__ void begin(int kt, bool live) {
        const int k0 = kt * BK, l = (int)ld;
        const uint16_t* p = KS ? base + (int64_t)k0 * l : base + k0;
        const int rows = KS ? min(kc - k0, BK) : valid;
        const int bytes = live ? ((rows - 1) * l + (KS ? valid : kc - k0)) * 2 : 0;
        rs = __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, bytes, 0x00020000);
        step_off = KS || k0 + chunk * 8 < kc ? voff : 0x80000000u;
    }
    __device__ __forceinline__ void piece(uint16_t* st, int q) {
        const uint32_t v = step_off + (uint32_t)(q * WAVES * LROWS * (int)ld * 2);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (void VE_LDS*)(st + (WAVES * q + wave) * 512), 16, (int)v, 0, 0, 0);
    }
    // Step kt's tile into registers (put() then writes them to LDS).
    __device__ __forceinline__ void get(int kt) {
        const int64_t k0 = (int64_t)kt * BK;
        if constexpr (!DMA) {
            // No ragged end inside 16 bytes: plain loads, which run together.
            // KC rows past the last read it again (their outputs are not
            // stored, and the epilogue keeps them out of a run's largest
            // magnitude); KS rows past the contraction too, and become 0.
            if (KS ? valid == ROWS : k0 + BK <= kc) {
#pragma unroll
                for (int q = 0; q < PIECES; ++q) {
                    const int row = lrow + q * WAVES * LROWS;
                    const uint16_t* p = KS ? base + min(k0 + row, (int64_t)kc - 1) * ld + chunk * 8
                                           : base + min(row, valid - 1) * ld + k0 + chunk * 8;
                    reg[q] = *(const VE_GLOBAL u32x4_any*)(const VE_GLOBAL uint16_t*)p;
                }
                if constexpr (KS) {
                    if (k0 + BK > kc) {
#pragma unroll
                        for (int q = 0; q < PIECES; ++q)
                            if (k0 + lrow + q * WAVES * LROWS >= kc) reg[q] = u32x4{0, 0, 0, 0};
                    }
                }
                return;
            }
            // else element by element at the ends
#pragma unroll
            for (int q = 0; q < PIECES; ++q) {
                const int row = lrow + q * WAVES * LROWS;
                const uint16_t* p;
                int64_t cnt;
                if constexpr (KS) {
                    p = base + (k0 + row) * ld + chunk * 8;
                    cnt = k0 + row < kc ? valid - chunk * 8 : 0;
                } else {
                    p = base + row * ld + k0 + chunk * 8;
                    cnt = row < valid ? kc - (k0 + chunk * 8) : 0;
                }
                reg[q] = cnt > 0 ? load_bf16x8(p, (int)(cnt < 8 ? cnt : 8), false) : u32x4{0, 0, 0, 0};
            }
        }
    }
    __device__ __forceinline__ void put(uint16_t* st, int lane) {
        if constexpr (!DMA) {
#pragma unroll
            for (int q = 0; q < PIECES; ++q) *(u32x4*)(st + (WAVES * q + wave) * 512 + lane * 8) = reg[q];
        }
    }
    // A lane's fragment of the 32 rows (columns) from r0 on, sub-step kk.
    __device__ static __forceinline__ bf16x8 frag(const uint16_t* st, int r0, int kk, int lane) {
        if constexpr (KS) {
            const int g = lane >> 4, i = lane & 15;
            const int k = kk * 16 + (g >> 1) * 8 + (i >> 2), s = r0 / 16 + (g & 1);
            const uint16_t* p = st + k * ROWS + (place(s) ^ (i >> 2)) * 16 + (i & 3) * 4;
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(read_tr((const VE_LDS uint16_t*)p),
                                                                      read_tr((const VE_LDS uint16_t*)(p + 4 * ROWS)), 0, 1,
                                                                      2, 3, 4, 5, 6, 7));
        } else {
            const int row = r0 + (lane & 31), slot = (2 * kk + (lane >> 5)) ^ swz(row & 15);
            return __builtin_bit_cast(bf16x8, *(const u32x4*)(st + row * BK + slot * 8));
        }
    }
};

// One work item: an output tile, or a slice of one's contraction.
struct Work {
    int e;
    int row0;        // first output row (a token, or a dw row)
    int rows;        // rows of the tile that exist (0: nothing to do)
    int col0;
    int begin, len;  // the group's tokens
    int kbeg, nk;    // contraction steps of this item
    int slice;
    uint32_t t;      // tile
};

// Tile `in` of a group's tm x tiles_n tiles: bands of 8 tile rows, column by
// column, so that consecutive tiles share operand panels.
template <class CF>
__device__ __forceinline__ void tile_in(const LinArgs& g, uint32_t in, int tm, int& ti, int& tj) {
    constexpr uint32_t kBand = 8;
    const uint32_t per = kBand * g.tiles_n, band = in / per, first = band * kBand;
    const uint32_t rows = min((uint32_t)tm - first, kBand), r = in - band * per;
    tj = (int)(r / rows);
    ti = (int)(first + r - tj * rows);
}

// Tile t of a product (kLinDw: of group e): where it lies.
template <class CF, int KIND>
__device__ __forceinline__ bool tile_at(const LinArgs& g, uint32_t t, int e, Work& w) {
    int tm, ti, tj;
    uint32_t in = t;
    w.t = t;
    w.e = e;
    w.begin = 0;
    w.len = (int)g.T;
    if constexpr (KIND == kLinDw) {
        tm = (int)((g.M + CF::BM - 1) / CF::BM);
        if (g.offsets) {
            int64_t begin, len;
            group_rows(g.offsets, e, g.T, begin, len);
            w.begin = __builtin_amdgcn_readfirstlane((int)begin);
            w.len = __builtin_amdgcn_readfirstlane((int)len);
        }
    } else if (g.offsets) {
        RaggedGroup r;
        if (!ragged_find(g.offsets, g.E, g.T, CF::BM, t, g.tiles_n, r)) return false;
        w.e = r.e;
        w.begin = (int)r.begin;
        w.len = (int)r.len;
        tm = r.tiles;
        in = t - (uint32_t)r.before * g.tiles_n;
    } else {
        tm = (int)((g.T + CF::BM - 1) / CF::BM);
    }
    tile_in<CF>(g, in, tm, ti, tj);
    w.col0 = tj * CF::BN;
    const int i0 = ti * CF::BM, all = KIND == kLinDw ? (int)g.M : w.len;
    w.rows = min(all - i0, CF::BM);
    w.row0 = KIND == kLinDw ? i0 : w.begin + i0;
    return true;
}

// Item i of the launch; false: there is none, nor any later one of this
// workgroup (workgroup b takes items b, b + gridDim.x, ...).  Workgroups go
// round-robin over the 8 XCDs, each with its own L2, so item i belongs to
// XCD i % 8 and each XCD takes a contiguous run of the tile sequence; in
// kLinDw of every group's tiles, because groups differ in length.
template <class CF, int KIND>
__device__ __forceinline__ bool fetch(const LinArgs& g, uint32_t total, uint32_t i, Work& w) {
    uint32_t t;
    int e = 0;
    w.slice = 0;
    if (g.ksplit > 1) {
        t = i / (uint32_t)g.ksplit;
        w.slice = (int)(i - t * g.ksplit);
        if (t >= total) return false;
    } else if (KIND == kLinDw) {
        const uint32_t in_e = total / (uint32_t)g.E, part = (in_e + 7) / 8, j = i / 8;
        e = (int)(j / part);
        if (e >= g.E) return false;
        t = (i % 8) * part + j - e * part;
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
    if (!tile_at<CF, KIND>(g, t, e, w)) return false;
    const int K = KIND == kLinDw ? w.len : (int)g.K;
    w.kbeg = 0;
    w.nk = (int)(((uint32_t)K + BK - 1) / BK);
    if (g.ksplit > 1) {
        const int per = (w.nk + g.ksplit - 1) / g.ksplit;
        w.kbeg = min(w.slice * per, w.nk);
        w.nk = min(per, w.nk - w.kbeg);
    }
    return true;
}

// Epilogue of 8 consecutive columns of one output row: `row` the token (or
// the row of dw[e]), col the first column, cnt of the 8 that exist (0: none).
// First the bias (rows of tokens), then, where z is saved in 8 bits, the
// largest magnitude of the run the columns lie in, which the caller finds
// across its lanes, then the rest.
template <int KIND>
__device__ __forceinline__ void bias8(const LinArgs& g, int e, int64_t col, int cnt, float* v) {
    if constexpr (KIND == kLinFwd) {
        if (!g.bias || cnt <= 0) return;
        float o[8];
        widen8(load_bf16x8(g.bias + (int64_t)e * g.bias_group + col, cnt, g.vec_bias), o);
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] += o[t];
    }
}

// act of 8 values, the switch outside the loop over them
__device__ __forceinline__ void activate8(int act, float* v) {
    switch (act) {
#define VE_ACT_CASE(A)                                   \
    case A:                                              \
        _Pragma("unroll") for (int t = 0; t < 8; ++t) v[t] = activate(A, v[t]); \
        break;
        VE_ACT_CASE(VE_ACT_RELU)
        VE_ACT_CASE(VE_ACT_GELU)
        VE_ACT_CASE(VE_ACT_GELU_TANH)
        VE_ACT_CASE(VE_ACT_SILU)
#undef VE_ACT_CASE
    default: break;
    }
}

__device__ __forceinline__ uint32_t amax8(const float* v, int cnt) {
    uint32_t m = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t) m = t < cnt ? amax_of(m, v[t]) : m;
    return m;
}

template <int KIND>
__device__ __forceinline__ void finish8(const LinArgs& g, int e, int64_t row, int64_t col, int cnt, float* v, uint32_t amax) {
    if (cnt <= 0) return;
    if constexpr (KIND == kLinDw) {
        const int64_t at = (int64_t)e * g.dw_group + row * g.lddw + col;
        if (g.wide) {
            VE_GLOBAL float* p = (VE_GLOBAL float*)((float*)g.dw + at);
            typedef f32x4 __attribute__((aligned(4))) f32x4_any;
            if (cnt == 8) {
                f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
                if (g.accumulate) {
                    a += *(VE_GLOBAL f32x4_any*)p;
                    b += *(VE_GLOBAL f32x4_any*)(p + 4);
                }
                *(VE_GLOBAL f32x4_any*)p = a;
                *(VE_GLOBAL f32x4_any*)(p + 4) = b;
            } else {
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    if (t < cnt) p[t] = g.accumulate ? p[t] + v[t] : v[t];
            }
        } else {
            uint16_t* p = (uint16_t*)g.dw + at;
            if (g.accumulate) {
                float o[8];
                widen8(load_bf16x8(p, cnt, g.vec_dw), o);
#pragma unroll
                for (int t = 0; t < 8; ++t) v[t] += o[t];
            }
            store_bf16x8(p, narrow8(v), cnt, g.vec_dw);
        }
    } else {
        if constexpr (KIND == kLinFwd) {
            if (g.z) store_bf16x8(g.z + row * g.ldz + col, narrow8(v), cnt, g.vec_z);
            if (g.z8.codes) {
                const RunCode c = run_code(__uint_as_float(amax));
                store_codes8(g.z8.codes + row * g.z8.ld_codes + col, encode8(c, v), cnt, g.vec_z8);
                const uint32_t run = (uint32_t)col >> __builtin_ctz(g.z8.block);
                if (((uint32_t)col & (g.z8.block - 1)) == 0) g.z8.scales[row * g.z8.ld_scales + run] = c.scale;
            }
            activate8(g.act, v);
        }
        if (g.res) {
            float o[8];
            widen8(load_bf16x8(g.res + row * g.ldr + col, cnt, g.vec_res), o);
#pragma unroll
            for (int t = 0; t < 8; ++t) v[t] += o[t];
        }
        store_bf16x8(g.y + row * g.ldy + col, narrow8(v), cnt, g.vec_y);
    }
}

// The kernel's arguments, read from memory again.
__device__ __forceinline__ LinArgs args_again() {
    auto p = (const __attribute__((address_space(4))) uint32_t*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    static_assert(sizeof(LinArgs) % 4 == 0, "whole words");
    uint32_t w[sizeof(LinArgs) / 4];
#pragma unroll
    for (int i = 0; i < (int)(sizeof(LinArgs) / 4); ++i) w[i] = p[i];
    LinArgs h;
    __builtin_memcpy(&h, w, sizeof(h));
    return h;
}

// What the epilogue of a launch has to do, as cases that each get their own
// loop: one store of bf16, for tokens after the bias; the same after the
// residual (kLinDw: what dw holds); activation and saving too; one store of
// fp32, and the same after what dw holds (these with 16-byte rows and 32-bit
// offsets from a wave's first row); everything.  The addend is a case and
// not a condition because a load that some path does not use stays pending
// for the compiler, which then waits for all loads in every later step.
enum Finish : int { kFinishAll, kFinishStore, kFinishAdd, kFinishSave, kFinishWide, kFinishWideAdd };

// Epilogue of one item.  Each wave passes its accumulators through its own
// 16 rows of LDS (no barrier between the waves), so that a lane gets 8
// consecutive columns and WN / 8 lanes a whole row of the wave's tile:
// 16-byte accesses, and runs saved in 8 bits are neighbouring lanes.  A row's
// 16-byte chunks lie even ones first, then odd ones, permuted by the row: a
// write (16 rows of two chunks) and a read (the even, then the odd chunks of
// a row) touch distinct banks.
template <class CF, int KIND, int FIN>
__device__ __forceinline__ void epilogue_of(const Work& w, f32x16 (&acc)[CF::TM][CF::TN],
                                            unsigned char* sw, int wr, int wc, int lane) {
    constexpr int TM = CF::TM, TN = CF::TN, WM = CF::WM, WN = CF::WN, CPR = WN / 8, ROWB = WN * 4;
    constexpr int RI = 64 / CPR, IT = 16 / RI;  // rows of one iteration, iterations of 16 rows
    const LinArgs g = args_again();
    const int c8 = lane % CPR, r0 = lane / CPR, cc = wc * WN + c8 * 8;  // the lane's columns and first row
    const int cnt0 = min(max(min((int)g.N - w.col0, CF::BN) - cc, 0), 8);
    const int64_t first = (int64_t)w.row0 + wr * WM, col = w.col0 + cc;
    float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    bias8<KIND>(g, w.e, col, cnt0, bias);
    // byte offsets of the lane from the wave's first row
    constexpr bool kWide = FIN == kFinishWide || FIN == kFinishWideAdd, res = FIN == kFinishAdd || FIN == kFinishWideAdd;
    constexpr int kSize = kWide ? 4 : 2;
    const int ldo = KIND == kLinDw ? (int)g.lddw : (int)g.ldy, ldr = KIND == kLinDw ? ldo : (int)g.ldr;
    VE_GLOBAL char* out = KIND == kLinDw ? (VE_GLOBAL char*)g.dw + (w.e * g.dw_group + first * g.lddw) * kSize
                                         : (VE_GLOBAL char*)(g.y + first * g.ldy);
    uint32_t o_off = (uint32_t)(r0 * ldo + (int)col) * kSize;
    const VE_GLOBAL char* rin = KIND == kLinDw ? out : (const VE_GLOBAL char*)(res ? g.res + first * g.ldr : nullptr);
    uint32_t r_off = (uint32_t)(r0 * ldr + (int)col) * kSize;
    int ldc = 0, lds = 0, shift = 0;
    uint32_t c_off = 0, s_off = 0, z_off = 0;
    VE_GLOBAL char *codes = nullptr, *scales = nullptr, *zout = nullptr;
    if constexpr (FIN == kFinishSave) {
        if (g.z8.codes) {
            ldc = (int)g.z8.ld_codes;
            lds = (int)g.z8.ld_scales;
            shift = __builtin_ctz(g.z8.block);
            codes = (VE_GLOBAL char*)(g.z8.codes + first * ldc);
            scales = (VE_GLOBAL char*)(g.z8.scales + first * lds);
            c_off = (uint32_t)(r0 * ldc + (int)col);
            s_off = (uint32_t)(r0 * lds + ((int)col >> shift)) * 4;
        }
        if (g.z) {
            zout = (VE_GLOBAL char*)(g.z + first * g.ldz);
            z_off = (uint32_t)(r0 * (int)g.ldz + (int)col) * 2;
        }
    }
    const bool run_first = ((int)col & (g.z8.block - 1)) == 0;
#pragma unroll 1
    for (int pass = 0; pass < 2 * TM; ++pass) {
        const int left = w.rows - wr * WM - pass * 16 - r0;  // rows from the lane's first on
        u32x4 rv[IT][kWide ? 2 : 1];
        if constexpr (res) {
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int h = 0; h < (kWide ? 2 : 1); ++h) {
                    rv[i][h] = u32x4{0, 0, 0, 0};
                    if (left > RI * i && cnt0 > 0)
                        rv[i][h] = *(const VE_GLOBAL u32x4*)(rin + (r_off + (uint32_t)(RI * i * ldr * kSize) + 16 * h));
                }
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int a = 0; a < TM; ++a)
            if (a == pass >> 1 && ((lane >> 4) & 1) == (pass & 1)) {
#pragma unroll
                for (int b = 0; b < TN; ++b)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int r = lane & 15, c = ((4 * b + q) ^ (r & (CPR - 1))) + CPR * (lane >> 5);
                        *(f32x4*)(sw + r * ROWB + c * 16) =
                            f32x4{acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
                    }
            }
        __builtin_amdgcn_wave_barrier();
        float v[IT][8];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = r0 + RI * i;
            const unsigned char* src = sw + r * ROWB + (c8 ^ (r & (CPR - 1))) * 16;
            *(f32x4*)&v[i][0] = *(const f32x4*)src;
            *(f32x4*)&v[i][4] = *(const f32x4*)(src + CPR * 16);
        }
        if constexpr (FIN != kFinishAll) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const bool in = left > RI * i && cnt0 > 0;
                if constexpr (KIND == kLinFwd) {
#pragma unroll
                    for (int t = 0; t < 8; ++t) v[i][t] += bias[t];
                }
                if constexpr (FIN == kFinishSave) {
                    if (zout && in)
                        *(VE_GLOBAL u32x4*)(zout + (z_off + (uint32_t)(RI * i * (int)g.ldz * 2))) = narrow8(v[i]);
                    if (codes) {
                        // columns past the last count for nothing: w's rows for them are zeros with
                        // direct loads, but copies of the last row in the register-staged form
                        const RunCode c = run_code_quick(__uint_as_float(amax_lanes(amax8(v[i], cnt0), g.z8.block / 8)));
                        const u32x2 q = encode8(c, v[i]);
                        if (in) {
                            *(VE_GLOBAL u32x2*)(codes + (c_off + (uint32_t)(RI * i * ldc))) = q;
                            if (run_first) *(VE_GLOBAL float*)(scales + (s_off + (uint32_t)(RI * i * lds * 4))) = c.scale;
                        }
                    }
                    activate8(g.act, v[i]);
                }
                if constexpr (FIN == kFinishAdd) {
                    float o[8];
                    widen8(rv[i][0], o);
#pragma unroll
                    for (int t = 0; t < 8; ++t) v[i][t] += o[t];
                }
                if constexpr (FIN == kFinishWideAdd) {
#pragma unroll
                    for (int t = 0; t < 8; ++t) v[i][t] += __builtin_bit_cast(f32x4, rv[i][t >> 2])[t & 3];
                }
                if (in) {
                    VE_GLOBAL char* o = out + (o_off + (uint32_t)(RI * i * ldo * kSize));
                    if constexpr (kWide) {
                        *(VE_GLOBAL f32x4*)o = *(const f32x4*)&v[i][0];
                        *(VE_GLOBAL f32x4*)(o + 16) = *(const f32x4*)&v[i][4];
                    } else {
                        *(VE_GLOBAL u32x4*)o = narrow8(v[i]);
                    }
                }
            }
            o_off += (uint32_t)(16 * ldo * kSize);
            r_off += (uint32_t)(16 * ldr * kSize);
            c_off += (uint32_t)(16 * ldc);
            s_off += (uint32_t)(16 * lds * 4);
            z_off += (uint32_t)(16 * (int)g.ldz * 2);
        } else {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int rr = pass * 16 + r0 + RI * i;  // row of the wave's tile
                if (g.ksplit > 1) {
                    float* o = g.partial + ((int64_t)w.slice * g.tiles + w.t) * (CF::BM * CF::BN) + (wr * WM + rr) * CF::BN + cc;
                    *(f32x4*)o = *(const f32x4*)&v[i][0];
                    *(f32x4*)(o + 4) = *(const f32x4*)&v[i][4];
                    continue;
                }
                const int cnt = left > RI * i ? cnt0 : 0;
#pragma unroll
                for (int t = 0; t < 8; ++t) v[i][t] += bias[t];
                uint32_t m = 0;
                if (KIND == kLinFwd && g.z8.codes) m = amax_lanes(amax8(v[i], cnt), g.z8.block / 8);
                finish8<KIND>(g, w.e, first + rr, col, cnt, v[i], m);
            }
        }
    }
}

template <class CF, int KIND>
__device__ __forceinline__ void epilogue(int finish, const Work& w, f32x16 (&acc)[CF::TM][CF::TN], unsigned char* sw,
                                         int wr, int wc, int lane) {
    if (finish == kFinishStore) epilogue_of<CF, KIND, kFinishStore>(w, acc, sw, wr, wc, lane);
    else if (finish == kFinishAdd) epilogue_of<CF, KIND, kFinishAdd>(w, acc, sw, wr, wc, lane);
    else if (KIND == kLinDw && finish == kFinishWide) epilogue_of<CF, KIND, kFinishWide>(w, acc, sw, wr, wc, lane);
    else if (KIND == kLinDw && finish == kFinishWideAdd) epilogue_of<CF, KIND, kFinishWideAdd>(w, acc, sw, wr, wc, lane);
    else if (KIND == kLinFwd && finish == kFinishSave) epilogue_of<CF, KIND, kFinishSave>(w, acc, sw, wr, wc, lane);
    else epilogue_of<CF, KIND, kFinishAll>(w, acc, sw, wr, wc, lane);
}

// Tiles of the launch; of ragged rows those that the offsets give.
template <class CF, int KIND>
__device__ __forceinline__ uint32_t all_tiles(const LinArgs& g) {
    if (KIND != kLinDw && g.offsets)
        return (uint32_t)min(g.tiles, (int64_t)ragged_total(g.offsets, g.E, g.T, CF::BM) * g.tiles_n);
    return (uint32_t)g.tiles;
}

// Slices of split tiles summed in slice order, then the epilogue: one thread
// for 8 columns of a tile row.
template <class CF, int KIND>
__global__ void __launch_bounds__(256) k_join(LinArgs g) {
    constexpr int CPR = CF::BN / 8, PER = CF::BM * CPR / 256;  // workgroups of one tile
    const uint32_t t = blockIdx.x / PER;
    Work w;
    if (!tile_at<CF, KIND>(g, t, 0, w)) return;
    const int id = (int)(blockIdx.x % PER) * 256 + (int)threadIdx.x, row = id / CPR, c8 = (id % CPR) * 8;
    const float* p = g.partial + (int64_t)t * (CF::BM * CF::BN) + row * CF::BN + c8;
    float v[8];
    *(f32x4*)&v[0] = *(const f32x4*)p;
    *(f32x4*)&v[4] = *(const f32x4*)(p + 4);
    for (int s = 1; s < g.ksplit; ++s) {
        p += g.tiles * (CF::BM * CF::BN);
        const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] += a[i];
            v[4 + i] += b[i];
        }
    }
    const int cols = (int)(g.N - w.col0 < CF::BN ? g.N - w.col0 : CF::BN);
    const int cnt = row < w.rows ? min(max(cols - c8, 0), 8) : 0;
    bias8<KIND>(g, 0, w.col0 + c8, cnt, v);
    uint32_t m = 0;
    if (KIND == kLinFwd && g.z8.codes) m = amax_lanes(amax8(v, cnt), g.z8.block / 8);
    finish8<KIND>(g, 0, (int64_t)w.row0 + row, w.col0 + c8, cnt, v, m);
}

template <class CF>
int64_t tiles_of(const LinArgs& g, LinKind kind) {
    const int64_t tn = (g.N + CF::BN - 1) / CF::BN;
    if (kind == kLinDw) return (int64_t)g.E * ((g.M + CF::BM - 1) / CF::BM) * tn;
    return ((g.T + CF::BM - 1) / CF::BM + (g.offsets ? g.E : 0)) * tn;
}

// The epilogue's case: the quick ones need 16-byte rows, and 128 rows within
// 32-bit byte offsets.
inline int finish_of(const LinArgs& g, LinKind kind) {
    const int64_t kMaxLd = int64_t(1) << 21;
    if (g.ksplit > 1 || g.N % 8) return kFinishAll;
    if (kind == kLinDw) {
        if (!g.vec_dw || g.lddw > kMaxLd) return kFinishAll;
        return g.wide ? (g.accumulate ? kFinishWideAdd : kFinishWide) : (g.accumulate ? kFinishAdd : kFinishStore);
    }
    if (!g.vec_y || g.ldy > kMaxLd) return kFinishAll;
    const bool bare = kind == kLinDx || (g.act == VE_ACT_NONE && !g.z && !g.z8.codes);
    if (g.res) return bare && g.vec_res && g.ldr <= kMaxLd ? kFinishAdd : kFinishAll;
    if (bare) return kFinishStore;
    if ((!g.z || (g.vec_z && g.ldz <= kMaxLd)) &&
        (!g.z8.codes || (g.vec_z8 && g.z8.ld_codes <= kMaxLd && g.z8.ld_scales <= kMaxLd)))
        return kFinishSave;
    return kFinishAll;
}

// Items of a launch: 8 runs of equal length, one for each XCD (kLinDw: of
// every group).
inline int64_t items_of(const LinArgs& g, LinKind kind) {
    if (g.ksplit > 1) return (g.tiles * g.ksplit + 7) / 8 * 8;
    if (kind == kLinDw) return g.E * ((g.tiles / g.E + 7) / 8 * 8);
    return (g.tiles + 7) / 8 * 8;
}

}  // namespace
}  // namespace ve
