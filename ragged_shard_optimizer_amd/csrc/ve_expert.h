// ve_expert.h -- internal interface between the kernels that sort rows by
// expert and bring them back (ve_expert.hip) and their host side
// (ve_expert_host.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ve.h"
#include "ve_internal.h"

namespace ve {

constexpr int kMaxSlots = 64, kMaxExperts = 4096;

// A sort over `blocks` workgroups of consecutive slots each.
struct SortArgs {
    const void* experts; int32_t wide;  // int64 instead of int32
    uint32_t n, chunk, blocks;          // slots, slots of a workgroup (a multiple of 64 times the waves), workgroups
    int32_t experts_n;
    int64_t* offsets;
    int32_t* position;
    int32_t* order;
    uint32_t* counts;                   // [blocks][experts_n] with more than one workgroup
};
// Fills chunk and blocks; returns the bytes of counts.
int64_t plan_sort(SortArgs& a);
hipError_t launch_sort(const SortArgs& a, hipStream_t s);
hipError_t launch_gather(const ve_expert_gather_args& a, hipStream_t s);
hipError_t launch_combine(const ve_expert_combine_args& a, hipStream_t s);
hipError_t launch_combine_backward(const ve_expert_combine_backward_args& a, hipStream_t s);
// Workgroups of a launch over tokens x cols.
int64_t expert_workgroups(int64_t tokens, int64_t cols);

}  // namespace ve
