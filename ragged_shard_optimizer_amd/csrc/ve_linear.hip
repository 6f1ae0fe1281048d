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

#include "ve_linear_tiles.h"

namespace ve {
namespace {

constexpr int kFewTokens = 8;  // tokens of the few-token form, at most

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

template <class CF, int KIND, bool DMA>
hipError_t launch_kind(LinArgs g, int ksplit, hipStream_t s) {
    g.tiles_n = (int)((g.N + CF::BN - 1) / CF::BN);
    g.ksplit = ksplit;
    g.tiles = tiles_of<CF>(g, (LinKind)KIND);
    if (g.tiles == 0) return hipSuccess;
    g.finish = finish_of(g, (LinKind)KIND);
    const int64_t items = items_of(g, (LinKind)KIND);
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
