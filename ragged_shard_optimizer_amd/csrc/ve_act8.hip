// ve_act8.hip -- activations saved in 8 bits (pack and unpack), and the
// elementwise half of a linear layer's backward pass: dz = dy act'(z) with
// the column sums of dz.
//
// Pack: every row is cut into runs of `block` columns; a run of 32, 64 or
// 128 columns is 4, 8 or 16 consecutive lanes of 8 columns each, so its
// largest magnitude is a few lane exchanges and the row is read once.
// All kernels are bound by HBM: 3 bytes an element for pack and unpack, 6
// (bf16 z) or 5 (8-bit z) for dz.  16384 x 8192, block 128: pack 68 us (6.0
// TB/s; 88 without the streaming hint on its loads, which leaves the caches
// to the codes), unpack 69 to 78 us (5.3 to 5.9 TB/s).  dz of 8192 x 28672 from
// 8 bits 220 to 228 us (5.2 to 5.4 TB/s).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ve_linear_device.h"

namespace ve {
namespace {

constexpr int kItems = 4;  // groups of 8 columns a thread handles, all loaded before the first is used


template <bool VEC>
__global__ void __launch_bounds__(256) k_pack(const uint16_t* x, int64_t ldx, int64_t rows, int cols, ve_act8 q, int per) {
    const int64_t first = (int64_t)blockIdx.x * (256 * kItems), row0 = first / per;
    const uint32_t rem = (uint32_t)(first - row0 * per);
    u32x4 h[kItems];
    int64_t row[kItems];
    int col[kItems], cnt[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const uint32_t i = rem + threadIdx.x + 256 * k, r = i / (uint32_t)per;
        row[k] = row0 + r;
        col[k] = (int)(i - r * per) * 8;
        cnt[k] = row[k] < rows ? min(cols - col[k], 8) : 0;
        h[k] = u32x4{0, 0, 0, 0};
        if (cnt[k] >= 8 && VEC) h[k] = ldv<true>((const VE_GLOBAL u32x4*)(x + row[k] * ldx + col[k]));
        else if (cnt[k] > 0) h[k] = load_bf16x8(x + row[k] * ldx + col[k], cnt[k], VEC);
    }
    const int shift = __builtin_ctz(q.block);
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        float v[8];
        widen8(h[k], v);
        uint32_t m = 0;
#pragma unroll
        for (int t = 0; t < 8; ++t) m = amax_of(m, v[t]);
        m = amax_lanes(m, q.block / 8);
        if (cnt[k] <= 0) continue;
        const RunCode c = run_code(__uint_as_float(m));
        store_codes8(q.codes + row[k] * q.ld_codes + col[k], encode8(c, v), cnt[k], VEC);
        if ((col[k] & (q.block - 1)) == 0) q.scales[row[k] * q.ld_scales + (col[k] >> shift)] = c.scale;
    }
}

template <bool VEC>
__global__ void __launch_bounds__(256) k_unpack(ve_act8 q, int64_t rows, int cols, uint16_t* x, int64_t ldx, int per,
                                                const int64_t* offsets, int E) {
    int64_t lo, hi;
    grouped_rows(offsets, E, rows, lo, hi);
    const int64_t first = (int64_t)blockIdx.x * (256 * kItems), row0 = first / per;
    const uint32_t rem = (uint32_t)(first - row0 * per);
    u32x2 w[kItems];
    float scale[kItems];
    int64_t row[kItems];
    int col[kItems], cnt[kItems];
    const int shift = __builtin_ctz(q.block);
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const uint32_t i = rem + threadIdx.x + 256 * k, r = i / (uint32_t)per;
        row[k] = row0 + r;
        col[k] = (int)(i - r * per) * 8;
        cnt[k] = row[k] >= lo && row[k] < hi ? min(cols - col[k], 8) : 0;
        w[k] = u32x2{0, 0};
        scale[k] = 0.f;
        if (cnt[k] > 0) {
            w[k] = load_codes8(q.codes + row[k] * q.ld_codes + col[k], cnt[k], VEC);
            scale[k] = q.scales[row[k] * q.ld_scales + (col[k] >> shift)];
        }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k)
        if (cnt[k] > 0) store_bf16x8(x + row[k] * ldx + col[k], restore8(w[k], scale[k]), cnt[k], VEC);
}

// Rows of `cols` elements, any alignment, as rows of whole 16 bytes that end
// in zeros (per: 16-byte groups of a row; rows: of one matrix; all: of all of
// them; offsets: of the E groups that the rows are cut into, or null).
// Bound by HBM, 4 bytes an element.
__global__ void __launch_bounds__(256) k_pad(const uint16_t* src, int64_t ld, int64_t group, int64_t all, int64_t rows,
                                             int cols, uint16_t* dst, int per, const int64_t* offsets, int E) {
    int64_t lo, hi;
    grouped_rows(offsets, E, all, lo, hi);
    const int64_t first = (int64_t)blockIdx.x * (256 * kItems), row0 = first / per;
    const uint32_t rem = (uint32_t)(first - row0 * per);
    const int64_t e0 = row0 / rows, in0 = row0 - e0 * rows;
    u32x4 h[kItems];
    int64_t at[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const uint32_t i = rem + threadIdx.x + 256 * k, r = i / (uint32_t)per;
        const int col = (int)(i - r * per) * 8;
        const int64_t row = row0 + r;
        int64_t e = e0, in = in0 + r;
        if (in >= rows) {
            const int64_t over = in / rows;
            e += over;
            in -= over * rows;
        }
        at[k] = row >= lo && row < hi ? row * per * 8 + col : -1;
        if (at[k] >= 0) h[k] = load_bf16x8(src + e * group + in * ld + col, min(cols - col, 8), false);
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k)
        if (at[k] >= 0) *(VE_GLOBAL u32x4*)(VE_GLOBAL uint16_t*)(dst + at[k]) = h[k];
}

// dz and column sums.  A workgroup takes a tile of kDzRows tokens of one
// group and 512 columns: 64 lanes of 8 columns, its four waves on every
// fourth row, each summing its rows in fp32; the four sums are joined in LDS.
// The sums are of dz before its rounding.  dz is rounded to bf16 once, because
// the matrix units that dx and dw run on take bf16: each term of their sums is
// off by at most 2^-8 of itself, which makes their error against exact
// gradients 1.4 times that of an fp32 dz (0.0023 against 0.0017 of the
// result's norm, most of both from the result's own rounding to bf16).  A dz
// in two bf16 parts would double the products' work.
template <int ZMODE, bool VEC>  // ZMODE 0: act none (dz = dy, sums only), 1: bf16 z, 2: 8-bit z
__global__ void __launch_bounds__(256) k_dz(DzArgs a, int col_tiles) {
    const int ct = blockIdx.x % col_tiles, rt = blockIdx.x / col_tiles;
    int64_t begin = (int64_t)rt * kDzRows, rows;
    if (a.offsets) {
        RaggedGroup r;
        if (!ragged_find(a.offsets, a.E, a.T, kDzRows, rt, 1, r)) return;
        const int64_t in = (int64_t)(rt - r.before) * kDzRows;
        begin = r.begin + in;
        rows = r.len - in;
    } else {
        rows = a.T - begin;
    }
    rows = rows < kDzRows ? rows : kDzRows;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t col = (int64_t)ct * 512 + lane * 8;
    const int cnt = a.N - col < 8 ? (int)(a.N - col) : 8;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int shift = ZMODE == 2 ? __builtin_ctz(a.z8.block) : 0;
    // n: the lane's columns, a constant for all but the row's last lane, so
    // that a lane's loads of several rows run together (8192 x 8190 with bf16
    // z: 131 us; 195 with the row's end tested at every load)
    auto rows_of = [&](auto n_of) {
#pragma unroll 4
        for (int64_t i = wave; i < rows; i += 4) {
            const int n = n_of();
            const int64_t row = begin + i;
            float d[8];
            widen8(load_bf16x8(a.dy + row * a.lddy + col, n, VEC), d);
            if constexpr (ZMODE != 0) {
                float z[8];
                if constexpr (ZMODE == 1) widen8(load_bf16x8(a.z + row * a.ldz + col, n, VEC), z);
                else
                    widen8(restore8(load_codes8(a.z8.codes + row * a.z8.ld_codes + col, n, VEC),
                                    a.z8.scales[row * a.z8.ld_scales + (col >> shift)]),
                           z);
#pragma unroll
                for (int t = 0; t < 8; ++t) d[t] = t < n ? d[t] * slope(a.act, z[t]) : 0.f;
                store_bf16x8(a.dz + row * a.lddz + col, narrow8(d), 8, true);  // rows of whole 16 bytes, zeros at the end
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) sum[t] += d[t];
        }
    };
    if (cnt >= 8) rows_of([] { return 8; });
    else if (cnt > 0) rows_of([cnt] { return cnt; });
    if (!a.sums) return;
    __shared__ float part[4][512];
#pragma unroll
    for (int t = 0; t < 8; ++t) part[wave][lane * 8 + t] = sum[t];
    __syncthreads();
    for (int c = threadIdx.x; c < 512; c += 256) {
        const int64_t n = (int64_t)ct * 512 + c;
        if (n < a.N) a.sums[(int64_t)rt * a.N + n] = (part[0][c] + part[1][c]) + (part[2][c] + part[3][c]);
    }
}

// dbias of group e, 64 columns a workgroup: its four waves sum every fourth
// tile of the group, joined in a fixed order.  all_tiles: rows of a.sums
// (offsets that break their rules could count more tiles than that).
__global__ void __launch_bounds__(256) k_dbias(DzArgs a, void* dbias, int64_t group, int wide, int accumulate,
                                               int col_tiles, int64_t all_tiles) {
    const int e = blockIdx.x / col_tiles, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = (int64_t)(blockIdx.x % col_tiles) * 64 + lane;
    int64_t before = 0, begin = 0, len = a.T;
    if (a.offsets) {
        for (int e0 = 0; e0 < e; e0 += 64) {
            int64_t b = 0, l = 0;
            if (e0 + lane < e) group_rows(a.offsets, e0 + lane, a.T, b, l);
            int64_t mt = (l + kDzRows - 1) / kDzRows;
#pragma unroll
            for (int d = 32; d; d >>= 1) mt += __shfl_xor(mt, d, 64);
            before += mt;
        }
        group_rows(a.offsets, e, a.T, begin, len);
    }
    const int64_t tiles = min((len + kDzRows - 1) / kDzRows, all_tiles - before);
    float s = 0.f;
    if (n < a.N)
#pragma unroll 8
        for (int64_t i = wave; i < tiles; i += 4) s += a.sums[(before + i) * a.N + n];
    __shared__ float part[4][64];
    part[wave][lane] = s;
    __syncthreads();
    if (wave || n >= a.N) return;
    s = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
    if (wide) {
        float* p = (float*)dbias + (int64_t)e * group + n;
        *p = accumulate ? *p + s : s;
    } else {
        uint16_t* p = (uint16_t*)dbias + (int64_t)e * group + n;
        if (accumulate) s += bf16_up(*p);
        *p = (uint16_t)pack_bf16x2(s, 0.f);
    }
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace

int64_t dz_tiles(int64_t T, int32_t E, bool ragged) { return (T + kDzRows - 1) / kDzRows + (ragged ? E : 0); }

hipError_t launch_dz(const DzArgs& a, hipStream_t s) {
    const int ct = (int)((a.N + 511) / 512);
    const int64_t grid = dz_tiles(a.T, a.E, a.offsets != nullptr) * ct;
    if (grid == 0) return hipSuccess;
    const dim3 g((unsigned)grid), b(256);
    if (a.act == VE_ACT_NONE) {
        if (a.vec) hipLaunchKernelGGL((k_dz<0, true>), g, b, 0, s, a, ct);
        else hipLaunchKernelGGL((k_dz<0, false>), g, b, 0, s, a, ct);
    } else if (!a.z8.codes) {
        if (a.vec) hipLaunchKernelGGL((k_dz<1, true>), g, b, 0, s, a, ct);
        else hipLaunchKernelGGL((k_dz<1, false>), g, b, 0, s, a, ct);
    } else {
        if (a.vec) hipLaunchKernelGGL((k_dz<2, true>), g, b, 0, s, a, ct);
        else hipLaunchKernelGGL((k_dz<2, false>), g, b, 0, s, a, ct);
    }
    return hipGetLastError();
}

hipError_t launch_pad(const uint16_t* src, int64_t ld, int64_t group, int64_t count, int64_t rows, int64_t cols, uint16_t* dst,
                      const int64_t* offsets, int32_t E, hipStream_t s) {
    const int64_t per = (cols + 7) / 8, grid = (count * rows * per + 256 * kItems - 1) / (256 * kItems);
    if (grid == 0) return hipSuccess;
    hipLaunchKernelGGL(k_pad, dim3((unsigned)grid), dim3(256), 0, s, src, ld, group, count * rows, rows, (int)cols, dst, (int)per,
                       offsets, E);
    return hipGetLastError();
}

hipError_t launch_dbias(const DzArgs& a, void* dbias, int64_t group, bool wide, bool accumulate, hipStream_t s) {
    const int ct = (int)((a.N + 63) / 64);
    hipLaunchKernelGGL(k_dbias, dim3((unsigned)((int64_t)a.E * ct)), dim3(256), 0, s, a, dbias, group, (int)wide,
                       (int)accumulate, ct, dz_tiles(a.T, a.E, a.offsets != nullptr));
    return hipGetLastError();
}

// Groups of 8 columns in a row, rounded up to whole runs, so that a run is
// always whole lanes; a workgroup covers 1,024 of them.
static int groups_per_row(int64_t cols, int block) { return (int)((cols + block - 1) / block * (block / 8)); }

hipError_t launch_act8_pack(const uint16_t* x, int64_t ldx, int64_t rows, int64_t cols, const ve_act8& q, hipStream_t s) {
    const int per = groups_per_row(cols, q.block);
    const int64_t grid = (rows * per + 256 * kItems - 1) / (256 * kItems);
    if (grid == 0) return hipSuccess;
    const bool vec = aligned(x, 16) && ldx % 8 == 0 && aligned(q.codes, 8) && q.ld_codes % 8 == 0;
    if (vec) hipLaunchKernelGGL(k_pack<true>, dim3((unsigned)grid), dim3(256), 0, s, x, ldx, rows, (int)cols, q, per);
    else hipLaunchKernelGGL(k_pack<false>, dim3((unsigned)grid), dim3(256), 0, s, x, ldx, rows, (int)cols, q, per);
    return hipGetLastError();
}

hipError_t launch_act8_unpack(const ve_act8& q, int64_t rows, int64_t cols, uint16_t* x, int64_t ldx, const int64_t* offsets,
                              int32_t E, hipStream_t s) {
    const int per = groups_per_row(cols, q.block);
    const int64_t grid = (rows * per + 256 * kItems - 1) / (256 * kItems);
    if (grid == 0) return hipSuccess;
    const bool vec = aligned(x, 16) && ldx % 8 == 0 && aligned(q.codes, 8) && q.ld_codes % 8 == 0;
    if (vec) hipLaunchKernelGGL(k_unpack<true>, dim3((unsigned)grid), dim3(256), 0, s, q, rows, (int)cols, x, ldx, per, offsets, E);
    else hipLaunchKernelGGL(k_unpack<false>, dim3((unsigned)grid), dim3(256), 0, s, q, rows, (int)cols, x, ldx, per, offsets, E);
    return hipGetLastError();
}

}  // namespace ve
