// uzip_lanes.hpp -- sums and maxima over the lanes of a wave and the waves of a
// workgroup, by DPP moves instead of trips through LDS (internal).
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace uzip {
namespace {

// A value of another lane by DPP, zero where there is none.
template <int CTRL, int ROWS = 15, class T>
__device__ inline T moved(T v) {
    if constexpr (sizeof(T) == 8) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint64_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROWS, 15, false);
        const uint64_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 15, false);
        return __builtin_bit_cast(T, hi << 32 | lo);
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 15, false));
    }
}
constexpr int kNeighbour = 0xB1;  // lanes 0 and 1, 2 and 3, .. change places
constexpr int kRowBack = 0x100;   // + n: from the lane n above, within 16
constexpr int kRowShift = 0x110, kWaveShift1 = 0x138, kRowLast = 0x142, kHalfLast = 0x143;
template <class T>
__device__ inline T lane_of(T v, uint32_t lane) {  // (lane uniform)
    if constexpr (sizeof(T) == 8) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((int)u, lane), hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane);
        return __builtin_bit_cast(T, hi << 32 | lo);
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
    }
}
struct Sum {
    template <class T>
    __device__ static T of(T a, T b) { return a + b; }
};
struct Max {
    template <class T>
    __device__ static T of(T a, T b) { return a > b ? a : b; }
};
// Of the lanes up to this one (zero is the operation's neutral value).
template <class OP, class T>
__device__ inline T row_scan(T v) {  // within 16 lanes
    v = OP::of(moved<kRowShift + 1>(v), v);
    v = OP::of(moved<kRowShift + 2>(v), v);
    v = OP::of(moved<kRowShift + 4>(v), v);
    return OP::of(moved<kRowShift + 8>(v), v);
}
template <class OP, class T>
__device__ inline T wave_scan(T v) {
    v = row_scan<OP>(v);
    v = OP::of(moved<kRowLast, 10>(v), v);
    return OP::of(moved<kHalfLast, 12>(v), v);
}
template <class T>
__device__ inline T wave_sum(T v) { return lane_of(wave_scan<Sum>(v), 63); }
template <class T>
__device__ inline T wave_max(T v) { return lane_of(wave_scan<Max>(v), 63); }  // (of unsigned values)

// The sum over the threads before this one, in a fixed order, and over all.
// lds: WAVES (at most 16) values.
template <uint32_t WAVES, class T>
__device__ inline T scan_before(T v, T *lds, T &total) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const T x = wave_scan<Sum>(v), upto = moved<kWaveShift1>(x);
    __syncthreads();
    if (lane == 63) lds[wave] = x;
    __syncthreads();
    const T waves = row_scan<Sum>(lds[lane & (WAVES - 1)]);
    total = lane_of(waves, WAVES - 1);
    const uint32_t w = __builtin_amdgcn_readfirstlane(wave);
    return w ? lane_of(waves, w - 1) + upto : upto;
}

}  // namespace
}  // namespace uzip
