// ve_expert.hip -- slots sorted by expert, rows gathered into that order and
// combined back, with the gradients.
//
// Sort: a counting sort.  A workgroup owns consecutive slots and each of its
// waves a consecutive part of them.  A first pass counts experts per wave; the
// base of (wave, expert) is the place of the expert's first slot, plus its
// slots in the workgroups before (their counts, written by a launch of their
// own where there are several), plus those in the waves before.  The second
// pass takes 64 slots at a time: ballots over the bits of the expert find the
// lanes that share it, and a slot's rank among them is the number of lower
// ones, so that equal experts keep the order of their slots and every call
// gives the same places.  The ballots cost 0.3 us for 64 slots of a wave, so
// that chunks are short:
// 32,768 slots over 256 experts 5 + 7 us in 16 workgroups, 11 + 22 in two.
//
// Gather, combine and its gradients go by token: a token's row is read (or
// written) once, and each of its slots' rows once.  They are bound by HBM: 4096
// tokens of 7168, 8 slots, gather 99 to 116 us (4.6 to 5.3 TB/s), combine 91 to
// 106 (5.0 to 5.8), both gradients 187 to 208 (4.8 to 5.4).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ve_expert.h"
#include "ve_fp8_device.h"

namespace ve {
namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortBatch = 4;            // slots a lane holds at once
constexpr uint32_t kSortChunk = 2048;    // slots of a workgroup, unless there are more than kSortBlocks of them
constexpr uint32_t kSortBlocks = 256;
constexpr int kRowThreads = 256;        // of the row kernels: 8 columns each

// The expert of slot i, or -1.
__device__ __forceinline__ int expert_of(const SortArgs& a, uint32_t i) {
    if (a.wide) {
        const int64_t e = ((const VE_GLOBAL int64_t*)a.experts)[i];
        return e >= 0 && e < a.experts_n ? (int)e : -1;
    }
    const int32_t e = ((const VE_GLOBAL int32_t*)a.experts)[i];
    return e >= 0 && e < a.experts_n ? e : -1;
}

// A wave's slots [begin, end) in batches: lane l of round r has slot at + 64 r
// + l, and its expert or -1 (all loads of a batch in flight together).
struct SlotBatch {
    int e[kSortBatch];
    __device__ __forceinline__ void load(const SortArgs& a, uint32_t at, uint32_t end, int lane) {
#pragma unroll
        for (int r = 0; r < kSortBatch; ++r) {
            const uint32_t i = at + 64 * r + lane;
            e[r] = i < end ? expert_of(a, i) : -1;
        }
    }
};

// Slots of each expert in a workgroup's chunk.
__global__ void __launch_bounds__(kSortThreads) k_sort_count(SortArgs a) {
    extern __shared__ uint32_t hist[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < a.experts_n; e += kSortThreads) hist[e] = 0;
    __syncthreads();
    const uint32_t part = a.chunk / kSortWaves, begin = min(blockIdx.x * a.chunk + wave * part, a.n), end = min(begin + part, a.n);
    for (uint32_t at = begin; at < end; at += 64 * kSortBatch) {
        SlotBatch b;
        b.load(a, at, end, lane);
#pragma unroll
        for (int r = 0; r < kSortBatch; ++r)
            if (b.e[r] >= 0) atomicAdd(&hist[b.e[r]], 1u);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts_n; e += kSortThreads)
        a.counts[(int64_t)blockIdx.x * a.experts_n + e] = hist[e];
}

// LDS: hist[waves][experts], base[experts], slots[experts] (everywhere), one
// sum for each wave.
__global__ void __launch_bounds__(kSortThreads) k_sort_place(SortArgs a, int waves) {
    extern __shared__ uint32_t lds[];
    const int E = a.experts_n, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t* hist = lds;
    uint32_t* base = lds + waves * E;
    uint32_t* slots = base + E;
    uint32_t* sums = slots + E;
    const uint32_t part = a.chunk / waves;
    const uint32_t begin = wave < waves ? min(blockIdx.x * a.chunk + wave * part, a.n) : a.n;
    const uint32_t end = min(begin + part, a.n);
    SlotBatch b;  // the first batch stays for the second pass
    b.load(a, begin, end, lane);
    for (int i = threadIdx.x; i < waves * E; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    for (uint32_t at = begin; at < end; at += 64 * kSortBatch) {
        SlotBatch more = b;
        if (at != begin) more.load(a, at, end, lane);
#pragma unroll
        for (int r = 0; r < kSortBatch; ++r)
            if (more.e[r] >= 0) atomicAdd(&hist[wave * E + more.e[r]], 1u);
    }
    __syncthreads();
    // thread t scans experts [t per, (t + 1) per): their slots everywhere, and
    // those in the workgroups before this one
    const int per = (E + kSortThreads - 1) / kSortThreads;
    const int e0 = min((int)threadIdx.x * per, E), e1 = min(e0 + per, E);
    uint32_t mine = 0;
    for (int e = e0; e < e1; ++e) {
        uint32_t all = 0, before = 0;
        if (a.blocks > 1) {
#pragma unroll 8
            for (uint32_t c = 0; c < a.blocks; ++c) {
                const uint32_t n = a.counts[(int64_t)c * E + e];
                all += n;
                before += c < blockIdx.x ? n : 0;
            }
        } else {
            for (int w = 0; w < waves; ++w) all += hist[w * E + e];
        }
        base[e] = mine + before;  // within the thread's experts; the rest below
        mine += all;
        slots[e] = mine;
    }
    uint32_t upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(upto, d, 64);
        if (lane >= d) upto += o;
    }
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    uint32_t ahead = upto - mine;
    for (int w = 0; w < wave; ++w) ahead += sums[w];
    for (int e = e0; e < e1; ++e) {
        uint32_t at = base[e] + ahead;
        if (blockIdx.x == 0) a.offsets[e + 1] = slots[e] + ahead;
        for (int w = 0; w < waves; ++w) {  // counts become the places of the waves' first slots
            const uint32_t c = hist[w * E + e];
            hist[w * E + e] = at;
            at += c;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[0] = 0;
    __syncthreads();
    const int bits = E > 1 ? 32 - __builtin_clz((unsigned)E - 1) : 0;
    for (uint32_t at = begin; at < end; at += 64 * kSortBatch) {
        if (at != begin) b.load(a, at, end, lane);
#pragma unroll
        for (int r = 0; r < kSortBatch; ++r) {
            const uint32_t i = at + 64 * r + lane;
            const int e = b.e[r];
            uint64_t same = __ballot(e >= 0);
            if (at + 64 * r >= end) break;
            for (int k = 0; k < bits; ++k) {
                const uint64_t set = __ballot((e >> k) & 1);
                same &= (e >> k) & 1 ? set : ~set;
            }
            const uint64_t lower = same & ((1ull << lane) - 1);
            uint32_t to = 0;
            if (e >= 0) to = hist[wave * E + e];
            __builtin_amdgcn_wave_barrier();
            if (e >= 0 && lower == 0) hist[wave * E + e] = to + (uint32_t)__popcll(same);
            __builtin_amdgcn_wave_barrier();
            if (i < end) {
                const int32_t p = e >= 0 ? (int32_t)(to + (uint32_t)__popcll(lower)) : -1;
                a.position[i] = p;
                if (e >= 0 && a.order) a.order[p] = (int32_t)i;
            }
        }
    }
}

// A workgroup's token and the 8 columns of its thread.
struct RowItem { int64_t t; int col, cnt; };
__device__ __forceinline__ RowItem row_item(int cols, int per) {
    RowItem r;
    r.t = blockIdx.x / (uint32_t)per;
    r.col = ((int)(blockIdx.x - (uint32_t)r.t * per) * kRowThreads + (int)threadIdx.x) * 8;
    r.cnt = min(cols - r.col, 8);
    return r;
}

template <bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_gather(ve_expert_gather_args a, int per) {
    const RowItem r = row_item((int)a.cols, per);
    if (r.cnt <= 0) return;
    const int32_t* pos = a.position + r.t * a.slots;
    const u32x4 h = load_bf16x8(a.x + r.t * a.ldx + r.col, r.cnt, VEC);
    float v[8];
    if (a.weights) widen8(h, v);
    for (int j = 0; j < a.slots; ++j) {
        const int64_t p = pos[j];
        if (p < 0 || p >= a.rows_len) continue;
        u32x4 o = h;
        if (a.weights) {
            const float w = a.weights[r.t * a.slots + j];
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = w * v[i];
            o = narrow8(s);
        }
        store_bf16x8(a.rows + p * a.ld_rows + r.col, o, r.cnt, VEC);
    }
}

// 16 lanes hold a run of 128 columns.
template <bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_gather8(ve_expert_gather_args a, int per) {
    const RowItem r = row_item((int)a.cols, per);
    const int32_t* pos = a.position + r.t * a.slots;
    u32x4 h = {0, 0, 0, 0};
    if (r.cnt > 0) h = load_bf16x8(a.x + r.t * a.ldx + r.col, r.cnt, VEC);
    float v[8];
    widen8(h, v);
    uint32_t m = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = finite_amax(m, v[i], bad);
    m = amax_lanes(m, 16);
    const ve_fp8& q = a.rows8;
    const uint32_t e = fp8_exponent(m, q.format);
    const u32x2 c = fp8_encode8(v, fp8_inverse(e), q.format, bad);
    if (r.col >= ((int)a.cols + 15) / 16 * 16) return;  // (zeros up to there)
    for (int j = 0; j < a.slots; ++j) {
        const int64_t p = pos[j];
        if (p < 0 || p >= a.rows_len) continue;
        *(VE_GLOBAL u32x2*)(q.codes + p * q.ld_codes + r.col) = c;
        if ((r.col & 127) == 0) q.scales[(int64_t)(r.col >> 7) * q.ld_scales + p] = (uint8_t)e;
    }
}

// A token's slots are taken 8 at a time, their rows' loads in flight together.
constexpr int kSlotsAtOnce = 8;

// Rows of slots [j0, j0 + 8) of a token: the place or -1, and the weight.
struct SlotRows {
    int64_t p[kSlotsAtOnce];
    float w[kSlotsAtOnce];
    __device__ __forceinline__ void load(const int32_t* pos, const float* weights, int j0, int slots, int64_t rows_len) {
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j) {
            const int at = min(j0 + j, slots - 1);
            const int64_t q = pos[at];
            p[j] = j0 + j < slots && q >= 0 && q < rows_len ? q : -1;
            w[j] = weights ? weights[at] : 1.f;
        }
    }
};

// 8 columns of a row that is read once (4096 tokens of 7168, 8 slots: 106 us,
// without the streaming hint 141).
template <bool VEC>
__device__ __forceinline__ u32x4 load_once(const uint16_t* p, int cnt) {
    if (VEC && cnt >= 8) return ldv<true>((const VE_GLOBAL u32x4*)p);
    return load_bf16x8(p, cnt, false);
}

template <bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_combine(ve_expert_combine_args a, int per) {
    const RowItem r = row_item((int)a.cols, per);
    if (r.cnt <= 0) return;
    u32x4 add = {0, 0, 0, 0};
    if (a.residual) add = load_bf16x8(a.residual + r.t * a.ldr + r.col, r.cnt, VEC);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < a.slots; j0 += kSlotsAtOnce) {
        SlotRows s;
        s.load(a.position + r.t * a.slots, a.weights ? a.weights + r.t * a.slots : nullptr, j0, a.slots, a.rows_len);
        u32x4 h[kSlotsAtOnce];
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j)
            if (s.p[j] >= 0) h[j] = load_once<VEC>(a.rows + s.p[j] * a.ld_rows + r.col, r.cnt);
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j) {
            if (s.p[j] < 0) continue;
            float v[8];
            widen8(h[j], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(s.w[j], v[i], sum[i]);
        }
    }
    if (a.residual) {
        float v[8];
        widen8(add, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += v[i];
    }
    store_bf16x8(a.y + r.t * a.ldy + r.col, narrow8(sum), r.cnt, VEC);
}

// A workgroup a token; dy is read again for every 8 slots (from the caches).
template <bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_combine_backward(ve_expert_combine_backward_args a) {
    __shared__ float sums[kRowThreads / 64][kSlotsAtOnce];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, cols = (int)a.cols;
    for (int j0 = 0; j0 < a.slots; j0 += kSlotsAtOnce) {
        SlotRows s;
        s.load(a.position + t * a.slots, a.weights && a.drows ? a.weights + t * a.slots : nullptr, j0, a.slots, a.rows_len);
        float dot[kSlotsAtOnce];
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j) dot[j] = 0.f;
        for (int col = (int)threadIdx.x * 8; col < cols; col += kRowThreads * 8) {
            const int cnt = min(cols - col, 8);
            const u32x4 hg = load_bf16x8(a.dy + t * a.lddy + col, cnt, VEC);
            u32x4 h[kSlotsAtOnce];
            if (a.dweights) {
#pragma unroll
                for (int j = 0; j < kSlotsAtOnce; ++j)
                    if (s.p[j] >= 0) h[j] = load_bf16x8(a.rows + s.p[j] * a.ld_rows + col, cnt, VEC);
            }
            float g[8];
            widen8(hg, g);
#pragma unroll
            for (int j = 0; j < kSlotsAtOnce; ++j) {
                if (s.p[j] < 0) continue;
                if (a.drows) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = s.w[j] * g[i];
                    store_bf16x8(a.drows + s.p[j] * a.ld_drows + col, narrow8(v), cnt, VEC);
                }
                if (a.dweights) {
                    float v[8];
                    widen8(h[j], v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot[j] = __builtin_fmaf(g[i], v[i], dot[j]);
                }
            }
        }
        if (!a.dweights) continue;
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j) {
#pragma unroll
            for (int d = 32; d; d >>= 1) dot[j] += __shfl_xor(dot[j], d, 64);
            if (lane == 0) sums[wave][j] = dot[j];
        }
        __syncthreads();
        if ((int)threadIdx.x < min(kSlotsAtOnce, a.slots - j0)) {
            float v = 0.f;
            for (int w = 0; w < kRowThreads / 64; ++w) v += sums[w][threadIdx.x];
            a.dweights[t * a.slots + j0 + threadIdx.x] = v;
        }
        __syncthreads();
    }
}

bool vec_ok(const void* p, int64_t ld) { return !p || (((uintptr_t)p & 15) == 0 && ld % 8 == 0); }

}  // namespace

int64_t plan_sort(SortArgs& a) {
    constexpr uint32_t unit = 64 * kSortWaves;
    const uint32_t n = std::max(a.n, 1u);  // (no slots: one workgroup writes the offsets)
    a.blocks = std::min((n + kSortChunk - 1) / kSortChunk, kSortBlocks);
    a.chunk = ((n + a.blocks - 1) / a.blocks + unit - 1) / unit * unit;
    a.blocks = (n + a.chunk - 1) / a.chunk;
    return a.blocks > 1 ? (int64_t)a.blocks * a.experts_n * 4 : 0;
}

hipError_t launch_sort(const SortArgs& a, hipStream_t s) {
    // as many waves take part as 64 KB of LDS have counts for
    int waves = kSortWaves;
    while ((waves + 2) * a.experts_n + kSortWaves > 16 * 1024) waves /= 2;
    if (a.blocks > 1)
        hipLaunchKernelGGL(k_sort_count, dim3(a.blocks), dim3(kSortThreads), a.experts_n * 4, s, a);
    hipLaunchKernelGGL(k_sort_place, dim3(a.blocks), dim3(kSortThreads), ((waves + 2) * a.experts_n + kSortWaves) * 4, s, a,
                       waves);
    return hipGetLastError();
}

int64_t expert_workgroups(int64_t tokens, int64_t cols) { return tokens * ((cols + kRowThreads * 8 - 1) / (kRowThreads * 8)); }

hipError_t launch_gather(const ve_expert_gather_args& a, hipStream_t s) {
    const int per = (int)((a.cols + kRowThreads * 8 - 1) / (kRowThreads * 8));
    const dim3 grid((unsigned)(a.tokens * per)), block(kRowThreads);
    if (a.rows8.codes) {
        if (vec_ok(a.x, a.ldx)) hipLaunchKernelGGL(k_gather8<true>, grid, block, 0, s, a, per);
        else hipLaunchKernelGGL(k_gather8<false>, grid, block, 0, s, a, per);
    } else {
        if (vec_ok(a.x, a.ldx) && vec_ok(a.rows, a.ld_rows)) hipLaunchKernelGGL(k_gather<true>, grid, block, 0, s, a, per);
        else hipLaunchKernelGGL(k_gather<false>, grid, block, 0, s, a, per);
    }
    return hipGetLastError();
}

hipError_t launch_combine(const ve_expert_combine_args& a, hipStream_t s) {
    const int per = (int)((a.cols + kRowThreads * 8 - 1) / (kRowThreads * 8));
    const dim3 grid((unsigned)(a.tokens * per)), block(kRowThreads);
    if (vec_ok(a.rows, a.ld_rows) && vec_ok(a.residual, a.ldr) && vec_ok(a.y, a.ldy))
        hipLaunchKernelGGL(k_combine<true>, grid, block, 0, s, a, per);
    else
        hipLaunchKernelGGL(k_combine<false>, grid, block, 0, s, a, per);
    return hipGetLastError();
}

hipError_t launch_combine_backward(const ve_expert_combine_backward_args& a, hipStream_t s) {
    const dim3 grid((unsigned)a.tokens), block(kRowThreads);
    if (vec_ok(a.dy, a.lddy) && vec_ok(a.rows, a.ld_rows) && vec_ok(a.drows, a.ld_drows))
        hipLaunchKernelGGL(k_combine_backward<true>, grid, block, 0, s, a);
    else
        hipLaunchKernelGGL(k_combine_backward<false>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace ve
