// ve_linear_device.h -- device helpers of the linear layer's kernels:
// activations and their slopes, the 8-bit code of saved activations, and the
// search for a ragged group's tile.
#pragma once

#include "ve_device.h"
#include "ve_linear.h"

namespace ve {

__device__ __forceinline__ float bf16_up(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// 16 bytes of bf16 at an address that is only 2-byte aligned, and 8 codes at
// any address, at once (the memory unit takes such addresses)
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(1))) u32x2_any;

// 8 bf16 at p (cnt of them valid, the others 0); vec: p is 16-byte aligned.
__device__ __forceinline__ u32x4 load_bf16x8(const uint16_t* p, int cnt, bool vec) {
    const VE_GLOBAL uint16_t* q = (const VE_GLOBAL uint16_t*)p;
    if (cnt >= 8) {
        if (vec) return *(const VE_GLOBAL u32x4*)q;
        return *(const VE_GLOBAL u32x4_any*)q;
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < 8; ++t)
        if (t < cnt) w[t >> 1] |= (uint32_t)q[t] << (16 * (t & 1));
    return u32x4{w[0], w[1], w[2], w[3]};
}

__device__ __forceinline__ void store_bf16x8(uint16_t* p, u32x4 h, int cnt, bool vec) {
    VE_GLOBAL uint16_t* q = (VE_GLOBAL uint16_t*)p;
    if (cnt >= 8) {
        if (vec) *(VE_GLOBAL u32x4*)q = h;
        else *(VE_GLOBAL u32x4_any*)q = h;
        return;
    }
    const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int t = 0; t < 8; ++t)
        if (t < cnt) q[t] = (uint16_t)(w[t >> 1] >> (16 * (t & 1)));
}

__device__ __forceinline__ void widen8(u32x4 h, float* v) {
    const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = (t & 1) ? bf_hi(w[t >> 1]) : bf_lo(w[t >> 1]);
}

__device__ __forceinline__ u32x4 narrow8(const float* v) {
    return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// exp (results below 2^-126 may flush to 0, above fp32's range they are infinite)
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// The upper tail of the normal distribution, Q(a) = erfc(a / sqrt 2) / 2 for
// a >= 0, as exp(-a^2 / 2) t P(t) with t = 1 / (1 + 0.33 a): erfcx falls like
// 1 / a, so t P(t) carries it with a degree-7 polynomial.  The coefficients
// are a minimax fit of the relative error over all a (1.0e-6; 1.6e-6 in fp32
// arithmetic for a < 5), far below the 2^-8 of the bf16 result.  ex returns
// exp(-a^2 / 2), which the slope needs too.
__device__ __forceinline__ float normal_tail(float a, float& ex) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.33f, a, 1.f));
    float p = 0.03328555077314377f;
    p = __builtin_fmaf(p, t, -0.10566431283950806f);
    p = __builtin_fmaf(p, t, 0.06743031740188599f);
    p = __builtin_fmaf(p, t, 0.03342943638563156f);
    p = __builtin_fmaf(p, t, 0.0910046249628067f);
    p = __builtin_fmaf(p, t, 0.1172168105840683f);
    p = __builtin_fmaf(p, t, 0.13164697587490082f);
    p = __builtin_fmaf(p, t, 0.13165107369422913f);
    ex = exp_of(-0.5f * a * a);
    return ex * (p * t);
}

constexpr float kGeluTanhC = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluTanhB = 0.044715f;

// act(z).  At the infinities the value is the limit (0 at -inf where it is
// 0 * inf by the formula); NaN stays NaN.
__device__ __forceinline__ float activate(int act, float z) {
    switch (act) {
    case VE_ACT_RELU:
        return !(z <= 0.f) ? z : 0.f;
    case VE_ACT_GELU: {
        float ex;
        const float q = normal_tail(__builtin_fabsf(z), ex);
        return __builtin_fmaxf(z, -1e4f) * (z >= 0.f ? 1.f - q : q);
    }
    case VE_ACT_GELU_TANH: {
        // 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
        const float u = z * __builtin_fmaf(kGeluTanhC * kGeluTanhB * z, z, kGeluTanhC);
        return __builtin_fmaxf(z, -1e4f) * __builtin_amdgcn_rcpf(1.f + exp_of(-2.f * u));
    }
    case VE_ACT_SILU:
        return __builtin_fmaxf(z, -1e4f) * __builtin_amdgcn_rcpf(1.f + exp_of(-z));
    default:
        return z;
    }
}

// act'(z); the factor of z in it is clamped where the other factor has
// underflowed, so that the infinities give the limits 0 and 1.
__device__ __forceinline__ float slope(int act, float z) {
    switch (act) {
    case VE_ACT_RELU:
        return z > 0.f ? 1.f : 0.f;
    case VE_ACT_GELU: {
        float ex;
        const float a = __builtin_fabsf(z), q = normal_tail(a, ex);
        const float zc = z >= 0.f ? __builtin_fminf(a, 64.f) : -__builtin_fminf(a, 64.f);
        return __builtin_fmaf(zc * 0.39894228040143268f, ex, z >= 0.f ? 1.f - q : q);
    }
    case VE_ACT_GELU_TANH: {
        const float u = kGeluTanhC * z * __builtin_fmaf(kGeluTanhB * z, z, 1.f);
        const float e = exp_of(-2.f * __builtin_fabsf(u)), r = __builtin_amdgcn_rcpf(1.f + e);
        const float a = __builtin_fminf(__builtin_fabsf(z), 64.f), zc = z >= 0.f ? a : -a;
        const float du = 2.f * kGeluTanhC * __builtin_fmaf(3.f * kGeluTanhB * zc, zc, 1.f);
        return __builtin_fmaf(zc * du, e * r * r, z >= 0.f ? r : e * r);
    }
    case VE_ACT_SILU: {
        const float e = exp_of(-__builtin_fabsf(z)), r = __builtin_amdgcn_rcpf(1.f + e);
        const float a = __builtin_fminf(__builtin_fabsf(z), 1e4f), zc = z >= 0.f ? a : -a;
        return __builtin_fmaf(zc, e * r * r, z >= 0.f ? r : e * r);
    }
    default:
        return 1.f;
    }
}

// The code of one run with largest magnitude amax: scale = amax / 127, code =
// rint(v up (127 / (amax up))), where up = 2^64 keeps the quotient finite for
// runs below 2^-100 (both products with a power of two are exact).  A run
// with an infinity or NaN has scale NaN and codes 0: it restores to NaN.
struct RunCode { float scale, up, inv; };
__device__ __forceinline__ RunCode run_code(float amax) {
    RunCode c;
    c.up = amax < 0x1p-100f ? 0x1p64f : 1.f;
    c.scale = amax / 127.f;
    c.inv = amax > 0.f ? 127.f / (amax * c.up) : 0.f;
    if (!(amax < __builtin_inff())) {
        c.scale = __builtin_nanf("");
        c.up = c.inv = 0.f;
    }
    return c;
}
// The same, bit for bit, for a product's epilogue, where two divisions for
// each 8 values show.  A quotient q = a r of a correctly rounded reciprocal r
// of b becomes the correctly rounded a / b by q + (a - b q) r, with the
// remainder exact in one fused operation (P. Markstein, IBM Journal of
// Research and Development 34, 1990); 1 / 127 is a constant, and one Newton
// step makes the hardware's reciprocal, off by a unit in the last place, the
// correctly rounded one.  Compared with the divisions for all 2^23 mantissas,
// with reciprocals up to two units off.
__device__ __forceinline__ RunCode run_code_quick(float amax) {
    if (__any(!(amax >= 0x1p-100f && amax <= 0x1p100f))) return run_code(amax);
    RunCode c;
    c.up = 1.f;
    constexpr float k = 1.f / 127.f;
    const float s = amax * k;
    c.scale = __builtin_fmaf(__builtin_fmaf(-127.f, s, amax), k, s);
    float r = __builtin_amdgcn_rcpf(amax);
    r = __builtin_fmaf(__builtin_fmaf(-amax, r, 1.f), r, r);
    const float q = 127.f * r;
    c.inv = __builtin_fmaf(__builtin_fmaf(-amax, q, 127.f), r, q);
    return c;
}
// Adding 1.5 * 2^23 rounds to a whole number (nearest even) and leaves its low
// byte, in two's complement, in the low byte of the sum.  |v inv| is at most
// 127 (1 + 2^-23), which rounds to 127, so nothing needs clamping.
__device__ __forceinline__ u32x2 encode8(const RunCode& c, const float* v) {
    uint32_t b[8];
    if (__any(c.up != 1.f)) {  // a run below 2^-100, or one that is not finite
#pragma unroll
        for (int t = 0; t < 8; ++t) b[t] = __float_as_uint(v[t] * c.up * c.inv + 12582912.f);
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) b[t] = __float_as_uint(v[t] * c.inv + 12582912.f);
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000c0cu);
        w[h] = c.inv == 0.f ? 0u : lo | hi;
    }
    return u32x2{w[0], w[1]};
}
// Largest |v|, kept as the bits of |v|: unsigned order puts infinity above
// every finite value and NaN above infinity.
__device__ __forceinline__ uint32_t amax_of(uint32_t m, float v) {
    const uint32_t a = __float_as_uint(v) & 0x7fffffffu;
    return a > m ? a : m;
}
// ... over runs of 4, 8 or 16 consecutive lanes, by exchanges inside a row of
// 16 lanes that need no LDS: neighbours, pairs, mirrored halves, mirrored row.
template <int CTRL>
__device__ __forceinline__ uint32_t amax_with(uint32_t m) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, CTRL, 0xf, 0xf, true);
    return o > m ? o : m;
}
__device__ __forceinline__ uint32_t amax_lanes(uint32_t m, int lanes) {
    m = amax_with<0xB1>(m);                    // quad_perm 1 0 3 2
    m = amax_with<0x4E>(m);                    // quad_perm 2 3 0 1
    if (lanes > 4) m = amax_with<0x141>(m);    // row_half_mirror
    if (lanes > 8) m = amax_with<0x140>(m);    // row_mirror
    return m;
}

// 8 codes at p, cnt valid; vec: p is 8-byte aligned
__device__ __forceinline__ void store_codes8(int8_t* p, u32x2 w, int cnt, bool vec) {
    VE_GLOBAL int8_t* q = (VE_GLOBAL int8_t*)p;
    if (cnt >= 8) {
        if (vec) *(VE_GLOBAL u32x2*)q = w;
        else *(VE_GLOBAL u32x2_any*)q = w;
        return;
    }
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int t = 0; t < 8; ++t)
        if (t < cnt) q[t] = (int8_t)(u[t >> 2] >> (8 * (t & 3)));
}
__device__ __forceinline__ u32x2 load_codes8(const int8_t* p, int cnt, bool vec) {
    const VE_GLOBAL int8_t* q = (const VE_GLOBAL int8_t*)p;
    if (cnt >= 8) {
        if (vec) return *(const VE_GLOBAL u32x2*)q;
        return *(const VE_GLOBAL u32x2_any*)q;
    }
    uint32_t u[2] = {0, 0};
#pragma unroll
    for (int t = 0; t < 8; ++t)
        if (t < cnt) u[t >> 2] |= ((uint32_t)q[t] & 255u) << (8 * (t & 3));
    return u32x2{u[0], u[1]};
}
// the restored values bf16(code * scale) of 8 codes, as bf16 pairs
__device__ __forceinline__ u32x4 restore8(u32x2 w, float scale) {
    const uint32_t u[2] = {w.x, w.y};
    float v[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = (float)(int8_t)(u[t >> 2] >> (8 * (t & 3))) * scale;
    return narrow8(v);
}

// Rows [begin, begin + len) of group e, its tiles of `bm` rows, and the tiles
// of the groups before it.  Offsets are clamped to [0, T] and to their
// predecessor, so no offsets array makes a kernel leave its buffers.
struct RaggedGroup { int e; int64_t begin, len; int tiles, before; };

__device__ __forceinline__ void group_rows(const int64_t* off, int e, int64_t T, int64_t& begin, int64_t& len) {
    const int64_t b = min(max(off[e], (int64_t)0), T);
    begin = b;
    len = max(min(off[e + 1], T) - b, (int64_t)0);
}

// The rows from the first group's first to the last group's last (all rows
// without offsets): what lies outside is not read.
__device__ __forceinline__ void grouped_rows(const int64_t* off, int E, int64_t T, int64_t& lo, int64_t& hi) {
    lo = off ? min(max(off[0], (int64_t)0), T) : 0;
    hi = off ? min(max(off[E], (int64_t)0), T) : T;
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Tiles of all groups (every lane of the wave takes part, lane l group l,
// l + 64, ...).
__device__ __forceinline__ int ragged_total(const int64_t* off, int E, int64_t T, int bm) {
    int total = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + (int)(threadIdx.x & 63);
        int64_t b = 0, len = 0;
        if (e < E) group_rows(off, e, T, b, len);
        int mt = (int)((len + bm - 1) / bm);
#pragma unroll
        for (int d = 32; d; d >>= 1) mt += __shfl_xor(mt, d, 64);
        total += mt;
    }
    return __builtin_amdgcn_readfirstlane(total);
}

// The group that holds row tile t / per of the sequence of all groups' tiles,
// each row tile counting `per` times; false: t is past the last tile.
__device__ __forceinline__ bool ragged_find(const int64_t* off, int E, int64_t T, int bm, int64_t t, int per,
                                            RaggedGroup& r) {
    int before = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int lane = (int)(threadIdx.x & 63), e = e0 + lane;
        int64_t b = 0, len = 0;
        if (e < E) group_rows(off, e, T, b, len);
        const int mt = (int)((len + bm - 1) / bm);
        int upto = mt;  // inclusive prefix sum over the lanes
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(upto, d, 64);
            if (lane >= d) upto += o;
        }
        const uint64_t hit = __ballot((int64_t)(before + upto) * per > t);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            r.e = e0 + src;
            r.begin = uniform64(__shfl(b, src, 64));
            r.len = uniform64(__shfl(len, src, 64));
            r.tiles = __builtin_amdgcn_readfirstlane(__shfl(mt, src, 64));
            r.before = __builtin_amdgcn_readfirstlane(before + __shfl(upto, src, 64)) - r.tiles;
            r.e = __builtin_amdgcn_readfirstlane(r.e);
            return true;
        }
        before += __shfl(upto, 63, 64);
    }
    return false;
}

}  // namespace ve
