// Reductions over a wavefront without LDS: four steps inside rows of 16 lanes by
// data-parallel moves, two across rows by the swaps of gfx950. The result is the
// same in every lane, and its order of combination fixed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace specv {

template <int CTRL>
__device__ __forceinline__ uint32_t lane_move(uint32_t v) {
    return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float lane_move(float v) {
    return __uint_as_float(lane_move<CTRL>(__float_as_uint(v)));
}
template <int CTRL>
__device__ __forceinline__ int lane_move(int v) {
    return static_cast<int>(lane_move<CTRL>(static_cast<uint32_t>(v)));
}
template <int CTRL>
__device__ __forceinline__ double lane_move(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
    const uint64_t m = static_cast<uint64_t>(lane_move<CTRL>(static_cast<uint32_t>(b >> 32))) << 32 |
                       lane_move<CTRL>(static_cast<uint32_t>(b));
    return __longlong_as_double(static_cast<long long>(m));
}

// Two values of which each lane has its own and that of the lane 16 (32) away.
template <int DISTANCE>
__device__ __forceinline__ void lane_swap(uint32_t v, uint32_t& a, uint32_t& b) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 p = DISTANCE == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                                   : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = p.x;
    b = p.y;
}
template <int DISTANCE>
__device__ __forceinline__ void lane_swap(float v, float& a, float& b) {
    uint32_t x, y;
    lane_swap<DISTANCE>(__float_as_uint(v), x, y);
    a = __uint_as_float(x);
    b = __uint_as_float(y);
}
template <int DISTANCE>
__device__ __forceinline__ void lane_swap(int v, int& a, int& b) {
    uint32_t x, y;
    lane_swap<DISTANCE>(static_cast<uint32_t>(v), x, y);
    a = static_cast<int>(x);
    b = static_cast<int>(y);
}
template <int DISTANCE>
__device__ __forceinline__ void lane_swap(double v, double& a, double& b) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
    uint32_t xl, yl, xh, yh;
    lane_swap<DISTANCE>(static_cast<uint32_t>(u), xl, yl);
    lane_swap<DISTANCE>(static_cast<uint32_t>(u >> 32), xh, yh);
    a = __longlong_as_double(static_cast<long long>(static_cast<uint64_t>(xh) << 32 | xl));
    b = __longlong_as_double(static_cast<long long>(static_cast<uint64_t>(yh) << 32 | yl));
}

// f(f(..)) over all lanes, f commutative.
template <typename V, typename F>
__device__ __forceinline__ V over_lanes(V v, F&& f) {
    v = f(v, lane_move<0xB1>(v));   // quad_perm 1 0 3 2
    v = f(v, lane_move<0x4E>(v));   // quad_perm 2 3 0 1
    v = f(v, lane_move<0x141>(v));  // row_half_mirror
    v = f(v, lane_move<0x140>(v));  // row_mirror
    V a, b;
    lane_swap<16>(v, a, b);
    v = f(a, b);
    lane_swap<32>(v, a, b);
    return f(a, b);
}

}  // namespace specv
