// ve_linear.hip -- the three products of a linear layer, dense or grouped by
// expert, on the MFMA units:
//
//   forward   z[t,n]  = sum_k x[t,k] w[e,n,k]     (+ bias, act, residual, saving)
//   dx        dx[t,k] = sum_n dz[t,n] w[e,n,k]    (+ addend)
//   dw        dw[e,n,k] = sum_{t in e} dz[t,n] x[t,k]   (+ what dw holds)
//
// e is the group (expert) token t belongs to: rows [offsets[e],
// offsets[e+1]).  The offsets stay on the device: a launch covers the most
// tiles that any offsets could need, and each workgroup finds its group with
// a wave-wide prefix sum over the groups' tile counts.
//
// Operands and LDS.  A contraction step is 64 deep.  An operand whose
// contraction index is contiguous in memory ("KC": x and w of the forward
// product, dz of dx) sits in LDS as rows of 64 elements; its fragments are
// 16-byte reads.  An operand whose contraction index is the row ("KS": w of
// dx, both operands of dw) sits in LDS as it lies in memory, 64 rows of the
// tile's width, and its fragments come from the transposing read
// ds_read_b64_tr_b16 (16 lanes read 4 rows x 16 columns; lane i gets column
// i), so no operand is ever transposed in memory.  Both layouts permute the
// 16- or 32-byte pieces of a row by XOR so that the lanes of one read hit
// distinct banks.
//
// MFMA 32x32x16 bf16, operands swapped (output columns as the first operand):
// accumulator register r of lane l holds row l % 32 and column
// 8 (r / 4) + 4 (l / 32) + r % 4 of a 32 x 32 block: a lane's registers run
// along a row.

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
constexpr int kFewTokens = 8;  // tokens of the few-token form, at most
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

// The operands of one work item.  With direct loads, contiguous dimensions
// are rounded up to whole 16 bytes, whose rest is 0 or whose product is not
// stored (dma_ok).
template <class CF, int KIND, bool DMA, class OpA, class OpB>
__device__ __forceinline__ void set_operands(const LinArgs& g, const Work& w, OpA& A, OpB& B, int lane, int wave) {
    const int K = KIND == kLinDw ? w.len : (int)g.K, cols = min((int)g.N - w.col0, CF::BN);
    auto up = [](int n) { return DMA ? (n + 7) & ~7 : n; };
    if constexpr (KIND == kLinDw) A.init(g.A + w.begin * g.lda + w.row0, g.lda, up(w.rows), K, lane, wave);
    else A.init(g.A + w.row0 * g.lda, g.lda, w.rows, up(K), lane, wave);
    if constexpr (KIND == kLinFwd) B.init(g.B + w.e * g.b_group + w.col0 * g.ldb, g.ldb, cols, up(K), lane, wave);
    else if constexpr (KIND == kLinDx) B.init(g.B + w.e * g.b_group + w.col0, g.ldb, up(cols), K, lane, wave);
    else B.init(g.B + w.begin * g.ldb + w.col0, g.ldb, up(cols), K, lane, wave);
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

// Work items with direct loads (16-byte operand rows, no ragged ends inside
// 16 bytes).  A workgroup stays on its CU and takes one item after the other;
// the steps of all its items are one stream, which the loads run up to two
// steps ahead of, so that an item's first loads land during the previous
// item's last step and epilogue.  (With one workgroup an item, its start and
// epilogue cost 10 us of a 256 x 256 tile, as much as 7 steps; with the
// stream, 5.)  One wave of 128 x 128 on a SIMD reads two thirds of the LDS
// bytes an MFMA of two waves of 128 x 64, which need not meet at barriers
// inside a step either: 1,375 against 1,166 TFLOP/s for dw at 8192^3, and
// 1,293 where two such waves took turns at the MFMAs.
//
// 8192 tokens, 8192 -> 28672, normal values: forward 1,384 to 1,395, dx 1,327
// to 1,332, dw 1,250 TFLOP/s (library products 1,558, 1,363, 1,176);
// values of many magnitudes cost up to 4%.  By the counters the MFMAs are busy
// 79, 76 and 72% of the cycles once the clock has settled at 1.65 to 1.7 GHz;
// the first calls after a pause run at 1.2 to 1.5 GHz and 1,040 to 1,240.
template <class CF, int KIND>
__global__ void __launch_bounds__(CF::THREADS, CF::PER_CU) k_product(LinArgs g) {
    constexpr int TM = CF::TM, TN = CF::TN, WM = CF::WM, WN = CF::WN;
    constexpr int NF = TM + TN, MM = TM * TN, H = MM / 2;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[CF::SMEM];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wr = wave / CF::WAVES_N, wc = wave % CF::WAVES_N;
    uint16_t* ops = (uint16_t*)smem;
    unsigned char* sw = smem + CF::STAGES_BYTES + wave * CF::OUT_BYTES;
    auto stage = [&](uint32_t s) { return ops + (s & 1) * CF::STAGE_ELEMS; };

    const uint32_t total = all_tiles<CF, KIND>(g);
    uint32_t ci = blockIdx.x, li = ci;  // items computed and loaded
    Work cw;
    bool cok = fetch<CF, KIND>(g, total, ci, cw);
    if (!cok) return;
    Operand<KIND == kLinDw, CF::BM, CF::WAVES, true> A;
    Operand<KIND != kLinFwd, CF::BN, CF::WAVES, true> B;
    using OpA = decltype(A);
    using OpB = decltype(B);
    constexpr int PA = OpA::PIECES, PB = OpB::PIECES, P = PA + PB, SPAN = 2 * MM;
    static_assert(SPAN <= H + 3 * MM, "loads of a step must be issued before its barrier");

    // The loads' position: step lk of the item's steps up to lend; lok: there
    // is an item.  The arguments are read anew for each item (through a
    // pointer the compiler cannot see through), so that they do not occupy
    // scalar registers in between.
    int lk = 0, lend = 0;
    bool lok = true;
    uint32_t item = 0;
    auto next_loaded = [&](bool first) {  // the next item with steps
        const LinArgs h = args_again();
        Work w;
        do {
            if (!first) li += gridDim.x;
            first = false;
            lok = __builtin_amdgcn_readfirstlane(fetch<CF, KIND>(h, total, li, w)) != 0;
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
        set_operands<CF, KIND, true>(h, w, A, B, lane, wave);
        A.make_uniform();
        B.make_uniform();
    };
    auto begin = [&]() {
        A.begin(lk, lok);
        B.begin(lk, lok);
    };
    auto advance = [&]() {
        if (lok && ++lk >= lend) next_loaded(false);
    };
    auto advance_inside = [&]() { ++lk; };
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
    bf16x8 fa[2][TM], fb[2][TN];
    // fragment f of sub-step kk in the order the MFMAs need them: A0, all B, the other A
    auto frag1 = [&](int buf, int f, int kk, uint32_t s) {
        const uint16_t* st = stage(s);
        if (f == 0 || f > TN) {
            const int a = f == 0 ? 0 : f - TN;
            fa[buf][a] = A.frag(st, wr * WM + a * 32, kk, lane);
        } else {
            fb[buf][f - 1] = B.frag(st + CF::A_ELEMS, wc * WN + (f - 1) * 32, kk, lane);
        }
    };
    auto mfma = [&](int buf, int m) {
        const int a = m / TN, b = m % TN;
        acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[buf][b], fa[buf][a], acc[a][b], 0, 0, 0);
    };

    A.init(g.A, g.lda, 1, 1, lane, wave);
    B.init(g.B, g.ldb, 1, 1, lane, wave);
    next_loaded(true);
    begin();
#pragma unroll
    for (int q = 0; q < PA; ++q) A.piece(stage(0), q);
#pragma unroll
    for (int q = 0; q < PB; ++q) B.piece(stage(0) + CF::A_ELEMS, q);
    __builtin_amdgcn_s_waitcnt(kWaitAll);
    advance();
    begin();
#pragma unroll
    for (int m = 0; m < H; ++m) pieces(m, 1);
    barrier();
#pragma unroll
    for (int f = 0; f < NF; ++f) frag1(0, f, 0, 0);

    uint32_t s = 0;  // steps computed, over all items
    while (cok) {
#pragma unroll
        for (int a = 0; a < TM; ++a)
#pragma unroll
            for (int b = 0; b < TN; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;
        // Every MFMA is followed by its share of what feeds the later ones,
        // in this order (the scheduling barriers keep it): the fragment
        // reads of the next sub-step, and direct loads.  In the middle of a
        // step's last sub-step all its reads are complete: the barrier there
        // frees its stage and makes the next one visible, and from there on
        // the loads of the step after the next go out into the freed stage,
        // spread evenly over two sub-steps: issued faster they stall the
        // wave (all within half a sub-step: 1,207 TFLOP/s forward at 8192^3,
        // one sub-step: 1,260), later they have less time to land (two and a
        // half: 1,283; two: 1,306).  Four stages of steps of 32, with the
        // loads two to three steps ahead, were slower (forward 1,249 against
        // 1,412 at 8192 x 8192 -> 28672: 64-byte pieces of a row, and twice
        // the barriers).
        auto step = [&](auto&& next) {
#pragma unroll
            for (int kk = 0; kk < BK / 16 - 1; ++kk) {
#pragma unroll
                for (int m = 0; m < MM; ++m) {
                    mfma(kk & 1, m);
#pragma unroll
                    for (int f = m * NF / MM; f < (m + 1) * NF / MM; ++f) frag1((kk + 1) & 1, f, kk + 1, s);
                    pieces(H + kk * MM + m, s + 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            next();
#pragma unroll
            for (int m = 0; m < H; ++m) mfma(1, m);
            __builtin_amdgcn_sched_barrier(0);
            // this wave's loads and LDS reads are complete, then everyone's
            __builtin_amdgcn_s_waitcnt(kWaitAll);
            barrier();
            begin();
#pragma unroll
            for (int m = H; m < MM; ++m) {
                mfma(1, m);
#pragma unroll
                for (int f = (m - H) * NF / H; f < (m - H + 1) * NF / H; ++f) frag1(0, f, 0, s + 1);
                pieces(m - H, s + 2);
                __builtin_amdgcn_sched_barrier(0);
            }
            ++s;
        };
        // Nothing of the previous item's epilogue may be pending for the
        // compiler here (it would wait in every step); the other workgroup of
        // the CU fills the time.
        if constexpr (CF::PER_CU > 1) __builtin_amdgcn_s_waitcnt(wait_vm(0));
        // the loads leave this item behind in its last two steps
        const int nk = __builtin_amdgcn_readfirstlane(cw.nk);
        int kt = 0;
        for (; kt + 2 < nk; ++kt) step(advance_inside);
        for (; kt < nk; ++kt) step(advance);
        // the loads' position waits in a vector register while the epilogue
        // needs the scalar ones (left to the compiler, it keeps them there in
        // the steps as well and fetches them back each time)
        uint32_t keep = 0;
        A.stash(keep, 0);
        B.stash(keep, 5);
        put_lane(keep, 10, (uint32_t)lk);
        put_lane(keep, 11, (uint32_t)lend);
        put_lane(keep, 12, (uint32_t)lok);
        put_lane(keep, 13, li);
        if (cw.rows > 0) epilogue<CF, KIND>(args_again().finish, cw, acc, sw, wr, wc, lane);
        ci += gridDim.x;
        if (get_lane(keep, 12) != 0 && get_lane(keep, 13) == ci) {  // the item the loads are at
            cw.e = (int)get_lane(item, 0);
            cw.row0 = (int)get_lane(item, 1);
            cw.rows = (int)get_lane(item, 2);
            cw.col0 = (int)get_lane(item, 3);
            cw.nk = (int)get_lane(item, 4);
            cw.slice = (int)get_lane(item, 5);
            cw.t = get_lane(item, 6);
        } else {
            cok = fetch<CF, KIND>(args_again(), total, ci, cw);
        }
        A.unstash(keep, 0);
        B.unstash(keep, 5);
        lk = (int)get_lane(keep, 10);
        lend = (int)get_lane(keep, 11);
        lok = get_lane(keep, 12) != 0;
        li = get_lane(keep, 13);
        begin();
    }
    // the loads past the last step (of nothing) land before the end
    __builtin_amdgcn_s_waitcnt(kWaitAll);
}

// One item a workgroup, through registers: operands of any alignment, where
// laying them out anew would take longer than it saves (calls of tens of
// microseconds, weights of many groups).
template <class CF, int KIND>
__global__ void __launch_bounds__(CF::THREADS, CF::PER_CU) k_product_any(LinArgs g) {
    constexpr int TM = CF::TM, TN = CF::TN, WM = CF::WM, WN = CF::WN;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[CF::SMEM];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wr = wave / CF::WAVES_N, wc = wave % CF::WAVES_N;
    Work w;
    if (!fetch<CF, KIND>(g, all_tiles<CF, KIND>(g), blockIdx.x, w) || w.rows == 0) return;
    Operand<KIND == kLinDw, CF::BM, CF::WAVES, false> A;
    Operand<KIND != kLinFwd, CF::BN, CF::WAVES, false> B;
    set_operands<CF, KIND, false>(g, w, A, B, lane, wave);
    f32x16 acc[TM][TN];
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int b = 0; b < TN; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;
    auto stage = [&](int kt) { return (uint16_t*)smem + (kt & 1) * CF::STAGE_ELEMS; };
    auto get = [&](int kt) {
        A.get(w.kbeg + kt);
        B.get(w.kbeg + kt);
    };
    auto put = [&](int kt) {
        A.put(stage(kt), lane);
        B.put(stage(kt) + CF::A_ELEMS, lane);
    };
    if (w.nk > 0) {
        get(0);
        put(0);
        __syncthreads();
    }
    for (int kt = 0; kt < w.nk; ++kt) {
        // the next step's registers are loaded while this one computes, and
        // written to the other stage, which everyone's reads left before the
        // last barrier
        if (kt + 1 < w.nk) get(kt + 1);
        const uint16_t* st = stage(kt);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
            bf16x8 fa[TM], fb[TN];
#pragma unroll
            for (int a = 0; a < TM; ++a) fa[a] = A.frag(st, wr * WM + a * 32, kk, lane);
#pragma unroll
            for (int b = 0; b < TN; ++b) fb[b] = B.frag(st + CF::A_ELEMS, wc * WN + b * 32, kk, lane);
#pragma unroll
            for (int a = 0; a < TM; ++a)
#pragma unroll
                for (int b = 0; b < TN; ++b) acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[b], fa[a], acc[a][b], 0, 0, 0);
        }
        if (kt + 1 < w.nk) put(kt + 1);
        __syncthreads();
    }
    epilogue<CF, KIND>(g.finish, w, acc, smem + CF::STAGES_BYTES + wave * CF::OUT_BYTES, wr, wc, lane);
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

// Few tokens (forward, one group): bound by reading the weights.  A wave takes
// R rows of w (output columns) whole: each load is 1 KiB of one row, 512
// steps of the contraction, and every lane keeps its own sums (products of
// bf16 pairs, v_dot2_f32_bf16) until the end.  x comes from the caches, once
// for the R rows.  MT: tokens, of which g.T exist.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <int MT, int R, int U>
__global__ void __launch_bounds__(256) k_few(LinArgs g) {
    __shared__ float sums[MT][4 * R];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * (4 * R);
    const int rows = (int)min(max(g.N - n0 - wave * R, (int64_t)0), (int64_t)R), toks = (int)g.T, K = (int)g.K;
    // reads past the last row, token or the contraction leave the buffers and return 0
    const uint16_t* wp = g.B + (n0 + min((int64_t)wave * R, g.N - 1 - n0)) * g.ldb;
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
        (void*)wp, (short)0, rows ? (int)(((rows - 1) * g.ldb + K) * 2) : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
        (void*)g.A, (short)0, (int)(((toks - 1) * g.lda + K) * 2), 0x00020000);
    float acc[R][MT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[r][t] = 0.f;
    for (int k0 = lane * 8; k0 < (K + 511) / 512 * 512; k0 += 512 * U) {
        u32x4 w[U][R];
        uint32_t off[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + 512 * u;
            off[u] = k < K ? (uint32_t)k * 2 : 0x80000000u;
#pragma unroll
            for (int r = 0; r < R; ++r)
                w[u][r] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, (int)(off[u] + (uint32_t)(r * (int)g.ldb * 2)), 0, 0));
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const u32x4 x = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, (int)(off[u] + (uint32_t)(t * (int)g.lda * 2)), 0, 0));
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t wq = w[u][r][q], xq = x[q];
                        acc[r][t] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, wq),
                                                                    __builtin_bit_cast(bf16x2, xq), acc[r][t], false);
                    }
            }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int d = 32; d; d >>= 1) acc[r][t] += __shfl_xor(acc[r][t], d, 64);
            if (lane == 0) sums[t][wave * R + r] = acc[r][t];
        }
    __syncthreads();
    constexpr int G = (4 * R + 7) / 8;  // groups of up to 8 columns
    const int t = threadIdx.x / G, c8 = (threadIdx.x % G) * 8;
    if (t >= toks) return;
    float v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = c8 + c < 4 * R ? sums[t][c8 + c] : 0.f;
    const int cnt = (int)min(max(g.N - n0 - c8, (int64_t)0), (int64_t)min(4 * R - c8, 8));
    bias8<kLinFwd>(g, 0, n0 + c8, cnt, v);
    finish8<kLinFwd>(g, 0, t, n0 + c8, cnt, v, 0);
}

template <int MT>
void launch_few_t(const LinArgs& g, hipStream_t s) {
    // one row a wave where four would leave CUs without work
    if (g.N < 16 * kCUs) hipLaunchKernelGGL((k_few<MT, 1, 8>), dim3((unsigned)((g.N + 3) / 4)), dim3(256), 0, s, g);
    else hipLaunchKernelGGL((k_few<MT, 4, 4>), dim3((unsigned)((g.N + 15) / 16)), dim3(256), 0, s, g);
}
hipError_t launch_few(const LinArgs& g, hipStream_t s) {
    if (g.T <= 1) launch_few_t<1>(g, s);
    else if (g.T <= 2) launch_few_t<2>(g, s);
    else if (g.T <= 4) launch_few_t<4>(g, s);
    else launch_few_t<8>(g, s);
    return hipGetLastError();
}

template <class CF>
int64_t tiles_of(const LinArgs& g, LinKind kind) {
    const int64_t tn = (g.N + CF::BN - 1) / CF::BN;
    if (kind == kLinDw) return (int64_t)g.E * ((g.M + CF::BM - 1) / CF::BM) * tn;
    return ((g.T + CF::BM - 1) / CF::BM + (g.offsets ? g.E : 0)) * tn;
}

template <class CF, int KIND, bool DMA>
hipError_t launch_kind(LinArgs g, int ksplit, hipStream_t s) {
    g.tiles_n = (int)((g.N + CF::BN - 1) / CF::BN);
    g.ksplit = ksplit;
    g.tiles = tiles_of<CF>(g, (LinKind)KIND);
    if (g.tiles == 0) return hipSuccess;
    const int64_t kMaxLd = int64_t(1) << 21;  // 128 rows within 32-bit byte offsets
    g.finish = kFinishAll;
    if (ksplit == 1 && g.N % 8 == 0) {
        if (KIND == kLinDw) {
            if (g.vec_dw && g.lddw <= kMaxLd)
                g.finish = g.wide ? (g.accumulate ? kFinishWideAdd : kFinishWide) : (g.accumulate ? kFinishAdd : kFinishStore);
        } else if (g.vec_y && g.ldy <= kMaxLd) {
            const bool bare = KIND == kLinDx || (g.act == VE_ACT_NONE && !g.z && !g.z8.codes);
            if (g.res) {
                if (bare && g.vec_res && g.ldr <= kMaxLd) g.finish = kFinishAdd;
            } else if (bare) {
                g.finish = kFinishStore;
            } else if ((!g.z || (g.vec_z && g.ldz <= kMaxLd)) &&
                       (!g.z8.codes || (g.vec_z8 && g.z8.ld_codes <= kMaxLd && g.z8.ld_scales <= kMaxLd))) {
                g.finish = kFinishSave;
            }
        }
    }
    // 8 runs of equal length, one for each XCD (kLinDw: of every group)
    int64_t items = (g.tiles + 7) / 8 * 8;
    if (KIND == kLinDw) items = g.E * ((g.tiles / g.E + 7) / 8 * 8);
    if (ksplit > 1) items = (g.tiles * ksplit + 7) / 8 * 8;
    if constexpr (DMA)
        hipLaunchKernelGGL((k_product<CF, KIND>), dim3((unsigned)std::min<int64_t>(items, kCUs * CF::PER_CU)),
                           dim3(CF::THREADS), 0, s, g);
    else
        hipLaunchKernelGGL((k_product_any<CF, KIND>), dim3((unsigned)items), dim3(CF::THREADS), 0, s, g);
    if (ksplit > 1)
        hipLaunchKernelGGL((k_join<CF, KIND>), dim3((unsigned)(g.tiles * (CF::BM * (CF::BN / 8) / 256))), dim3(256), 0, s, g);
    return hipGetLastError();
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Direct loads: 16-byte operand rows, the contiguous dimensions whole 16-byte
// groups (or padded to them), and a tile's rows within 32-bit byte offsets.
bool dma_ok(const LinArgs& g, LinKind kind) {
    const int64_t kMaxLd = int64_t(1) << 21;
    if (!aligned16(g.A) || !aligned16(g.B) || g.lda % 8 || g.ldb % 8 || g.lda > kMaxLd || g.ldb > kMaxLd) return false;
    if (kind != kLinDw && g.b_group % 8) return false;
    if (kind == kLinDw) return (g.M % 8 == 0 || g.pad_a) && (g.N % 8 == 0 || g.pad_b);
    if (kind == kLinDx) return (g.K % 8 == 0 || g.pad_a) && (g.N % 8 == 0 || g.pad_b);
    return g.K % 8 == 0 || (g.pad_a && g.pad_b);
}

template <int KIND>
hipError_t launch_path(const LinArgs& g, const LinPlan& p, hipStream_t s) {
    switch (p.path) {
    case kPathFew: return launch_few(g, s);
    case kPath256: return launch_kind<Cfg256, KIND, true>(g, p.ksplit, s);
    case kPath128:
        if constexpr (KIND == kLinFwd)
            if (g.z8.codes && g.z8.block > Cfg128::WN) return launch_kind<Cfg128W, KIND, true>(g, p.ksplit, s);
        return launch_kind<Cfg128, KIND, true>(g, p.ksplit, s);
    default: return launch_kind<Cfg128W, KIND, false>(g, p.ksplit, s);
    }
}

// Microseconds of a product as `items` tiles (or slices) of `steps` steps: a
// CU takes its share of them, 256 x 256 tiles one by one, 128 x 128 tiles two
// at a time (a last one alone).  Measured: a step of 256 x 256 takes 1.42 us
// and its start and epilogue 5; of a pair of 128 x 128 tiles 0.9 and 4, of a
// single one 0.6.  Slices' sums (bytes) are written and read at 5 TB/s, by
// one launch more (4 us).  Against measurements, 128^2 / 256^2 in us: 4001
// tokens 2880 -> 5760 dx 141 / 127 (model 143 / 133), dw 157 / 179 (163 /
// 189); 2049 tokens 4096 -> 2880 forward 59 (62).  The fit is to contractions
// of a thousand and more, and without a term for bytes: products that bytes
// bind take 2 to 2.5 times the estimate (fp32 dw of 77 tokens 7168 -> 1536 19
// us, estimated 8; of 16 groups with 500 tokens 2880 -> 2880 120, estimated
// 58; dx of the latter 91, estimated 45), and of ragged rows it counts the
// most tiles that any offsets could need.
// us: a step of two 128 x 128 tiles, of a single one, their start and
// epilogue, those of a 256 x 256 tile
struct TileCost { double pair, one, start, start256; };
constexpr TileCost kDirect{0.9, 0.6, 4, 5};
// Columns that are not whole 16 bytes take the epilogue of every case, which
// one workgroup a CU hides less than two (dw of 4099 x 4101 over one token:
// 41 us in 256 x 256 tiles, 28 in 128 x 128).
constexpr TileCost kDirectOdd{0.9, 0.6, 5.5, 14};
// The register-staged form, by kind: fitted to 13 shapes of rows that are not
// 16-byte multiples (the products' order is their cost: dw transposes both
// operands).  8192 tokens 8190 -> 8190: 2390 / 3031 / 6347 us, with operands
// laid out anew and direct loads 913 / 906 / 905; 33 tokens 4101 -> 2051
// 24 / 33 / 20 against 33 / 33 / 25.
constexpr TileCost kStaged[3] = {{2.2, 1.2, 8, 0}, {3.6, 2.4, 12, 0}, {5, 3.4, 8, 0}};

double product_us(bool big, int64_t items, int64_t steps, int64_t bytes, const TileCost& c) {
    const double n = (double)((items + kCUs - 1) / kCUs), st = (double)steps;
    const double sums = bytes ? (double)bytes * 2 / 5e6 + 4 : 0;
    if (big) return n * (1.42 * st + c.start256) + sums;
    const double pairs = (double)((int64_t)n / 2), one = n - 2 * pairs;
    return pairs * (c.pair * st + c.start) + one * (c.one * st + c.start) + sums;
}

}  // namespace

LinPlan plan_product(const LinArgs& g, LinKind kind) {
    LinPlan p{kPathGeneral, 1, 0, 0};
    const int64_t pin = option(kOptLinearPath);
    // Few tokens against the tiles split along the contraction, us a call at 1
    // / 2 / 4 / 8 tokens: 8192 -> 1024 8 / 8 / 8 / 14 against 19, 8192 -> 8192
    // 28 / 30 / 33 / 56 against 36, 8192 -> 28672 92 / 97 / 98 / 111 against
    // 120 to 130.  At 5 to 8 tokens the rule is right at the ends only: with
    // some thousand outputs the tiles are faster (2880 -> 5760 18 against 23).
    // Ragged groups stay with the tiles, unsplit, which read the weights of
    // the groups that have tokens at 5.2 to 6.0 TB/s where those are 26 or
    // more (7168 -> 2048); fewer leave CUs without work: 19 groups 4.5 TB/s, 8
    // 2.3, and one token of one group takes 46 us for 29 MB.
    const bool few = kind == kLinFwd && !g.offsets && !g.z8.codes && g.K % 8 == 0 && dma_ok(g, kind);
    if (few && g.T <= kFewTokens && (pin == kPathAuto || pin == kPathFew)) {
        p.path = kPathFew;
        return p;
    }
    const bool dma = dma_ok(g, kind) && pin != kPathGeneral;
    const int64_t K = kind == kLinDw ? g.T / g.E : g.K, nk = std::max<int64_t>(1, (K + BK - 1) / BK);
    const bool may_split = !g.offsets && option(kOptLinearSplit) != 0;
    double best = 0;
    for (int path : {(int)kPath128, (int)kPath256}) {
        if (!dma && path == kPath256) break;
        if (dma && (pin == kPath128 || pin == kPath256) && pin != path) continue;
        const int64_t tiles = path == kPath256 ? tiles_of<Cfg256>(g, kind) : tiles_of<Cfg128>(g, kind);
        const int64_t slots = kCUs * (path == kPath256 ? Cfg256::PER_CU : Cfg128::PER_CU), area = path == kPath256 ? 65536 : 16384;
        for (int64_t ks = 1; ks <= 32; ++ks) {
            if (ks > 1 && (!may_split || nk / ks < 4 || tiles * ks > slots)) break;
            double us = product_us(path == kPath256, tiles * ks, (nk + ks - 1) / ks, ks > 1 ? tiles * ks * area * 4 : 0,
                                   !dma ? kStaged[kind] : g.N % 8 ? kDirectOdd : kDirect);
            // runs of 128 columns saved from 128 x 128 tiles need waves of 32 x
            // 128, which take 1.5 times as long (16384 tokens of 32 experts
            // 7168 -> 2048: 852 us against 577)
            if (path == kPath128 && ks == 1 && kind == kLinFwd && g.z8.codes && g.z8.block > Cfg128::WN) us *= 1.5;
            if (best == 0 || us < best) {
                best = us;
                p.us = us;
                p.path = dma ? path : (int)kPathGeneral;
                p.ksplit = (int)ks;
                p.partial_bytes = ks > 1 ? ks * tiles * area * 4 : 0;
            }
        }
    }
    return p;
}

hipError_t launch_product(LinArgs g, LinKind kind, const LinPlan& p, hipStream_t s) {
    switch (kind) {
    case kLinFwd: return launch_path<kLinFwd>(g, p, s);
    case kLinDx: return launch_path<kLinDx>(g, p, s);
    default: return launch_path<kLinDw>(g, p, s);
    }
}

}  // namespace ve
