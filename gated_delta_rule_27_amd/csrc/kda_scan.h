// kda_scan.h -- 64-bit values moved between the lanes of a wavefront, and sums
// over them.
#pragma once

#include "kda_device.h"

namespace kda {

__device__ __forceinline__ double lane_value(double x, int lane) {
    union { double d; int w[2]; } v;
    v.d = x;
    v.w[0] = __builtin_amdgcn_readlane(v.w[0], lane);
    v.w[1] = __builtin_amdgcn_readlane(v.w[1], lane);
    return v.d;
}
// x of the lane that the data-parallel move `kCtrl` names, 0 where it names
// none or the lane's row of 16 is not in kRows
template <int kCtrl, int kRows>
__device__ __forceinline__ double moved(double x) {
    union { double d; int w[2]; } v;
    v.d = x;
    v.w[0] = __builtin_amdgcn_update_dpp(0, v.w[0], kCtrl, kRows, 0xf, false);
    v.w[1] = __builtin_amdgcn_update_dpp(0, v.w[1], kCtrl, kRows, 0xf, false);
    return v.d;
}
// inclusive prefix sum over the lanes: along the rows of 16 (shifts by 1, 2,
// 4, 8), then lane 15 of rows 0 and 2 to the row after, lane 31 to the upper half
__device__ __forceinline__ double wave_scan(double x) {
    x += moved<0x111, 0xf>(x);
    x += moved<0x112, 0xf>(x);
    x += moved<0x114, 0xf>(x);
    x += moved<0x118, 0xf>(x);
    x += moved<0x142, 0xa>(x);
    x += moved<0x143, 0xc>(x);
    return x;
}
__device__ __forceinline__ double wave_sum(double x) { return lane_value(wave_scan(x), 63); }

// the same for whole numbers
__device__ __forceinline__ uint64_t lane_value(uint64_t x, int lane) {
    return __builtin_bit_cast(uint64_t, lane_value(__builtin_bit_cast(double, x), lane));
}
__device__ __forceinline__ uint32_t lane_value(uint32_t x, int lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
}
template <int kCtrl, int kRows>
__device__ __forceinline__ uint64_t moved(uint64_t x) {
    return __builtin_bit_cast(uint64_t, moved<kCtrl, kRows>(__builtin_bit_cast(double, x)));
}
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t moved(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kCtrl, kRows, 0xf, false);
}
template <typename I>
__device__ __forceinline__ I wave_scan_whole(I x) {
    x += moved<0x111, 0xf>(x);
    x += moved<0x112, 0xf>(x);
    x += moved<0x114, 0xf>(x);
    x += moved<0x118, 0xf>(x);
    x += moved<0x142, 0xa>(x);
    x += moved<0x143, 0xc>(x);
    return x;
}

// 16 bytes from an address that only its elements align (rows of an odd
// vocabulary)
template <typename T>
__device__ __forceinline__ typename Vec16<T>::type load16(const T* p) {
    typename Vec16<T>::type x;
    __builtin_memcpy(&x, p, 16);
    return x;
}

}  // namespace kda
