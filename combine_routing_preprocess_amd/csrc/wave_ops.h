// Reductions over the 64 lanes of a wavefront by lane permutes in the vector
// pipe (DPP), without LDS traffic.  Every lane has to be active.
#pragma once
#include "moe_internal.h"

namespace moe {
namespace ops {

constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E;               // quad_perm [1,0,3,2] and [2,3,0,1]
constexpr int kDppHalfMirror = 0x141, kDppMirror = 0x140;     // lane i <-> 7 - i of 8, 15 - i of 16

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    return __hiloint2double((int)dpp<CTRL>((uint32_t)__double2hiint(v)), (int)dpp<CTRL>((uint32_t)__double2loint(v)));
}

__device__ __forceinline__ uint32_t readlane(uint32_t v, int l) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, l);
}
__device__ __forceinline__ float readlane(float v, int l) { return __uint_as_float(readlane(__float_as_uint(v), l)); }
__device__ __forceinline__ double readlane(double v, int l) {
    return __hiloint2double((int)readlane((uint32_t)__double2hiint(v), l), (int)readlane((uint32_t)__double2loint(v), l));
}

// Sum over the 16 lanes of a row, in every one of them.
template <typename T>
__device__ __forceinline__ T row_sum(T v) {
    v += dpp<kDppXor1>(v);
    v += dpp<kDppXor2>(v);
    v += dpp<kDppHalfMirror>(v);
    v += dpp<kDppMirror>(v);
    return v;
}

// Sum over the wavefront, the same value in every lane.
template <typename T>
__device__ __forceinline__ T wave_sum_dpp(T v) {
    v = row_sum(v);
    return (readlane(v, 0) + readlane(v, 16)) + (readlane(v, 32) + readlane(v, 48));
}

__device__ __forceinline__ uint32_t wave_max_dpp(uint32_t v) {
    v = max(v, dpp<kDppXor1>(v));
    v = max(v, dpp<kDppXor2>(v));
    v = max(v, dpp<kDppHalfMirror>(v));
    v = max(v, dpp<kDppMirror>(v));
    return max(max(readlane(v, 0), readlane(v, 16)), max(readlane(v, 32), readlane(v, 48)));
}
__device__ __forceinline__ double wave_max_dpp(double v) {
    v = fmax(v, dpp<kDppXor1>(v));
    v = fmax(v, dpp<kDppXor2>(v));
    v = fmax(v, dpp<kDppHalfMirror>(v));
    v = fmax(v, dpp<kDppMirror>(v));
    return fmax(fmax(readlane(v, 0), readlane(v, 16)), fmax(readlane(v, 32), readlane(v, 48)));
}

}  // namespace ops
}  // namespace moe
