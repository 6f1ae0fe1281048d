// ve_fp8_pack.hip -- bf16 matrices packed in 8-bit floating point, for a
// product over their columns, over their rows, or both, and restored.
//
// A workgroup takes a tile of 128 x 128, which holds whole blocks of every
// kind: runs of 128 columns, runs of 128 rows, 128 x 128.  A thread holds 8
// rows x 8 columns in fp32.  A row's run is 16 lanes (lane exchanges find its
// largest magnitude), a column's 16 row blocks (4 in the wave, then through
// LDS).  The transposed codes are turned 8 x 8 in registers and go through
// 16 KB of LDS, 8-byte pieces permuted by XOR so that writes and reads touch
// distinct banks, so that memory sees whole 128-byte lines both ways.  Bound by
// HBM: 16 weights of 2048 x 7168 both ways 167 to 182 us (5.2 to 5.6 TB/s; with
// 4 rows a thread in twice the threads 173 beside 167), 16000 x 7168 rows both
// ways 91 to 98 us (4.7 to 5.1 TB/s), rows only 67 (5.1); restoring 16 x 2048 x
// 7168 137 to 141 us (5.0 to 5.1 TB/s).  Through an activation's slope (whose z
// is loaded row by row, where it is needed) 267 us with SiLU, 278 with GELU (2.5
// TB/s).  A short batch is bound by latency: 500 x 2880 in 16 groups, whose tiles
// are searched first, 11.4 to 12.4 us in a trace.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ve_fp8_device.h"
#include "ve_fp8_pack.h"

namespace ve {
namespace {

constexpr int kTile = 128;

// The tile of this workgroup: rows [row0, row0 + len) of it exist; column of
// its first row in the transposed matrix; matrix e.
struct PackTile { int64_t row0, col_t; int len, col0, e; };

__device__ __forceinline__ bool pack_tile(const Fp8PackArgs& a, PackTile& t) {
    const uint32_t r = blockIdx.x / (uint32_t)a.tiles_n;
    t.col0 = (int)(blockIdx.x - r * a.tiles_n) * kTile;
    t.e = 0;
    if (a.weight) {
        t.e = (int)(r / (uint32_t)a.tiles_m);
        t.row0 = (int64_t)(r - t.e * a.tiles_m) * kTile;
        t.col_t = t.row0;
        t.len = (int)min(a.rows - t.row0, (int64_t)kTile);
    } else if (a.offsets) {
        RaggedGroup g;
        if (!ragged_find(a.offsets, a.groups, a.rows, kTile, r, 1, g)) return false;
        const int64_t in = (int64_t)(r - g.before) * kTile;
        t.row0 = g.begin + in;
        t.col_t = (int64_t)r * kTile;
        t.len = (int)min(g.len - in, (int64_t)kTile);
    } else {
        t.row0 = t.col_t = (int64_t)r * kTile;
        t.len = (int)min(a.rows - t.row0, (int64_t)kTile);
    }
    return true;
}

// 8 x 8 bytes, rows in w[0 .. 8): out[j] holds byte j of every row.
__device__ __forceinline__ void transpose8(const u32x2* w, u32x2* out) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // columns 4 h .. 4 h + 3
        uint32_t q[2][4];
#pragma unroll
        for (int g = 0; g < 2; ++g) {  // rows 4 g .. 4 g + 3
            const uint32_t a = w[4 * g][h], b = w[4 * g + 1][h], c = w[4 * g + 2][h], d = w[4 * g + 3][h];
            const uint32_t ab_lo = __builtin_amdgcn_perm(b, a, 0x05010400u), ab_hi = __builtin_amdgcn_perm(b, a, 0x07030602u);
            const uint32_t cd_lo = __builtin_amdgcn_perm(d, c, 0x05010400u), cd_hi = __builtin_amdgcn_perm(d, c, 0x07030602u);
            q[g][0] = __builtin_amdgcn_perm(cd_lo, ab_lo, 0x05040100u);
            q[g][1] = __builtin_amdgcn_perm(cd_lo, ab_lo, 0x07060302u);
            q[g][2] = __builtin_amdgcn_perm(cd_hi, ab_hi, 0x05040100u);
            q[g][3] = __builtin_amdgcn_perm(cd_hi, ab_hi, 0x07060302u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) out[4 * h + j] = u32x2{q[0][j], q[1][j]};
    }
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <bool WEIGHT>
__global__ void __launch_bounds__(256) k_fp8_pack(Fp8PackArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t turned[kTile * kTile];
    __shared__ uint32_t amaxes[4][kTile];
    PackTile t;
    if (!pack_tile(a, t)) return;
    const int tid = threadIdx.x, c = tid & 15, rb = tid >> 4, lane = tid & 63, wave = tid >> 6;
    const int col = t.col0 + 8 * c, cnt = min((int)a.cols - col, 8);
    const bool both = a.out_t.codes != nullptr;
    const uint16_t* x = a.x + t.e * a.x_group + (t.row0 + 8 * rb) * a.ldx + col;
    u32x4 h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        h[i] = u32x4{0, 0, 0, 0};
        if (8 * rb + i < t.len && cnt > 0) {
            if (cnt == 8 && a.vec) h[i] = ldv<true>((const VE_GLOBAL u32x4*)(x + i * a.ldx));
            else h[i] = load_bf16x8(x + i * a.ldx, cnt, false);
        }
    }
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) widen8(h[i], v[i]);
    if (!WEIGHT && a.act != VE_ACT_NONE) {
        const uint16_t* z = a.z + (t.row0 + 8 * rb) * a.ldz + col;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
                const int row = 4 * half + i4;
                if (8 * rb + row >= t.len || cnt <= 0) continue;
                float s[8];
                widen8(load_bf16x8(z + row * a.ldz, cnt, a.vec_z), s);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i == row) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (k < cnt) v[i][k] *= slope(a.act, s[k]);
                    }
            }
        }
    }
    bool bad = false;
    uint32_t er[8], ec[8];
    // largest magnitudes of the rows' runs, the columns' runs, or the tile
    uint32_t mc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t f = finite_amax(0, v[i][k], bad);
            m = umax(m, f);
            mc[k] = umax(mc[k], f);
        }
        if (!WEIGHT) er[i] = fp8_exponent(amax_lanes(m, 16), a.format);
    }
    if (WEIGHT || both) {
        if (WEIGHT) {
#pragma unroll
            for (int k = 1; k < 8; ++k) mc[0] = umax(mc[0], mc[k]);
#pragma unroll
            for (int d = 32; d; d >>= 1) mc[0] = umax(mc[0], (uint32_t)__shfl_xor((int)mc[0], d, 64));
            if (lane == 0) amaxes[wave][0] = mc[0];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                mc[k] = umax(mc[k], (uint32_t)__shfl_xor((int)mc[k], 16, 64));
                mc[k] = umax(mc[k], (uint32_t)__shfl_xor((int)mc[k], 32, 64));
                if (lane < 16) amaxes[wave][8 * c + k] = mc[k];
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int at = WEIGHT ? 0 : 8 * c + k;
            ec[k] = fp8_exponent(umax(umax(amaxes[0][at], amaxes[1][at]), umax(amaxes[2][at], amaxes[3][at])), a.format);
        }
        if (WEIGHT) {
#pragma unroll
            for (int i = 0; i < 8; ++i) er[i] = ec[0];
        }
    }
    u32x2 w[8];
    if (a.out.codes || WEIGHT) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = fp8_encode8(v[i], fp8_inverse(er[i]), a.format, bad);
    }
    if (a.out.codes) {
        VE_GLOBAL uint8_t* o = (VE_GLOBAL uint8_t*)(a.out.codes + t.e * a.out_codes_group + (t.row0 + 8 * rb) * a.out.ld_codes + col);
        if (col < ((int)a.cols + 15) / 16 * 16) {  // zeros up to there
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (8 * rb + i < t.len) *(VE_GLOBAL u32x2*)(o + i * a.out.ld_codes) = w[i];
        }
        uint8_t* s = a.out.scales + t.e * a.out_scales_group + (int64_t)(t.col0 / kTile) * a.out.ld_scales;
        if (WEIGHT) {
            if (tid == 0) s[t.row0 / kTile] = (uint8_t)er[0];
        } else if (c < 8 && 8 * rb + c < t.len) {  // lane c of a run writes row c's
            uint32_t e = er[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) e = c == i ? er[i] : e;
            s[t.row0 + 8 * rb + c] = (uint8_t)e;
        }
    }
    if (!both) return;
    if (!WEIGHT) {
        float inv[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) inv[k] = fp8_inverse(ec[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = v[i][k] * inv[k];
            w[i] = fp8_encode8(s, 1.f, a.format, bad);
        }
    }
    u32x2 turn[8];
    transpose8(w, turn);
#pragma unroll
    for (int k = 0; k < 8; ++k) *(u32x2*)(turned + (8 * c + k) * kTile + ((rb ^ c) * 8)) = turn[k];
    const int64_t scales_at = t.e * a.out_t_scales_group + t.col_t / kTile * a.out_t.ld_scales;
    if (WEIGHT) {
        if (tid == 0) a.out_t.scales[scales_at + t.col0 / kTile] = (uint8_t)ec[0];
    } else if (rb == 0 && cnt > 0) {
        uint8_t* s = a.out_t.scales + scales_at + col;
        if (cnt == 8) {
            *(VE_GLOBAL uint32_t*)s = ec[0] | ec[1] << 8 | ec[2] << 16 | ec[3] << 24;
            *(VE_GLOBAL uint32_t*)(s + 4) = ec[4] | ec[5] << 8 | ec[6] << 16 | ec[7] << 24;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < cnt) s[k] = (uint8_t)ec[k];
        }
    }
    __syncthreads();
    // 16 bytes of a transposed row a thread, 8 lanes its 128
    const int piece = tid & 7;
    const int64_t ends = WEIGHT ? (a.rows - t.row0 + 15) / 16 * 16 : kTile;  // zeros up to there
    uint8_t* o = a.out_t.codes + t.e * a.out_t_codes_group + t.col_t + 16 * piece;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int tc = (tid >> 3) + 32 * i, s = tc >> 3;  // column, and what its pieces are permuted by
        const u32x4 q = *(const u32x4*)(turned + tc * kTile + ((piece ^ (s >> 1)) * 16));
        if (t.col0 + tc < a.cols && 16 * piece < ends)
            *(VE_GLOBAL u32x4*)(o + (int64_t)(t.col0 + tc) * a.out_t.ld_codes) = s & 1 ? u32x4{q.z, q.w, q.x, q.y} : q;
    }
}

constexpr int kItems = 2;  // groups of 16 columns a thread handles, all loaded before the first is used

// per: groups of 16 columns of a row; blocks: workgroups of a matrix
__global__ void __launch_bounds__(256) k_fp8_unpack(ve_fp8_unpack_args a, int per, int blocks, bool vec) {
    const uint32_t m = blockIdx.x / (uint32_t)blocks;
    const int64_t first = (int64_t)(blockIdx.x - m * blocks) * (256 * kItems), row0 = first / per;
    const uint32_t rem = (uint32_t)(first - row0 * per);
    const int shift = a.in.block_rows == 1 ? 0 : 7, cols = (int)a.cols;
    const uint8_t* codes = a.in.codes + m * a.in_codes_group;
    const uint8_t* scales = a.in.scales + m * a.in_scales_group;
    u32x4 w[kItems];
    uint32_t e[kItems];
    int64_t row[kItems];
    int col[kItems], cnt[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const uint32_t i = rem + threadIdx.x + 256 * k, r = i / (uint32_t)per;
        row[k] = row0 + r;
        col[k] = (int)(i - r * per) * 16;
        cnt[k] = row[k] < a.rows ? min(cols - col[k], 16) : 0;
        w[k] = u32x4{0, 0, 0, 0};
        e[k] = 0;
        if (cnt[k] > 0) {
            w[k] = ldv<true>((const VE_GLOBAL u32x4*)(codes + row[k] * a.in.ld_codes + col[k]));
            e[k] = ((const VE_GLOBAL uint8_t*)scales)[(int64_t)(col[k] >> 7) * a.in.ld_scales + (row[k] >> shift)];
        }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        if (cnt[k] <= 0) continue;
        uint16_t* x = a.x + m * a.x_group + row[k] * a.ldx + col[k];
        const float s = fp8_scale(e[k]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
            fp8_decode4(w[k][2 * h], a.in.format, v);
            fp8_decode4(w[k][2 * h + 1], a.in.format, v + 4);
#pragma unroll
            for (int t = 0; t < 8; ++t) v[t] *= s;
            store_bf16x8(x + 8 * h, narrow8(v), cnt[k] - 8 * h, vec);
        }
    }
}

}  // namespace

hipError_t launch_fp8_pack(Fp8PackArgs a, hipStream_t s) {
    a.tiles_n = (int)((a.cols + kTile - 1) / kTile);
    a.tiles_m = (int)((a.rows + kTile - 1) / kTile);
    int64_t tiles = a.tiles_m;
    if (a.weight) tiles *= a.groups;
    else if (a.offsets) tiles = ve_fp8_columns(a.rows, a.groups) / kTile;
    const dim3 grid((unsigned)(tiles * a.tiles_n));
    if (a.weight) hipLaunchKernelGGL(k_fp8_pack<true>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(k_fp8_pack<false>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_fp8_unpack(const ve_fp8_unpack_args& a, hipStream_t s) {
    const int64_t per = (a.cols + 15) / 16, blocks = (a.rows * per + 256 * kItems - 1) / (256 * kItems);
    const bool vec = ((uintptr_t)a.x & 15) == 0 && a.ldx % 8 == 0 && (a.groups == 1 || a.x_group % 8 == 0);
    hipLaunchKernelGGL(k_fp8_unpack, dim3((unsigned)(a.groups * blocks)), dim3(256), 0, s, a, (int)per, (int)blocks, vec);
    return hipGetLastError();
}

}  // namespace ve
