// ve_fp8_pack.h -- launch arguments of packing in 8-bit floating point
// (ve_fp8_pack.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ve.h"

namespace ve {

struct Fp8PackArgs {
    int64_t rows, cols;
    int32_t groups, act;
    bool weight;               // `groups` matrices in blocks of 128 x 128, not one in runs
    bool vec, vec_z;           // rows of x / z start on 16 bytes
    const int64_t* offsets;
    const uint16_t* x; int64_t ldx, x_group;
    const uint16_t* z; int64_t ldz;
    int32_t format;
    ve_fp8 out; int64_t out_codes_group, out_scales_group;
    ve_fp8 out_t; int64_t out_t_codes_group, out_t_scales_group;
    int32_t tiles_n, tiles_m;  // set by the launcher
};
hipError_t launch_fp8_pack(Fp8PackArgs a, hipStream_t s);
hipError_t launch_fp8_unpack(const ve_fp8_unpack_args& a, hipStream_t s);

}  // namespace ve
