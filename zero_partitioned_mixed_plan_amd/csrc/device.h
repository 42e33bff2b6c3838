// Device helpers of the loss and many-tensor kernels.  kernels.hip has its
// own: its committed memory-request counts name that exact source, so it is
// not edited for sharing's sake.
#pragma once

#include "internal.h"

namespace zmi {

// 16 bytes as a native vector (the non-temporal builtins take these, not
// HIP's uint4 wrapper struct).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int64_t kGridX = 65536;           // x extent of the 2-D grids

__device__ __forceinline__ int64_t block_id() {
    return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
}

inline dim3 grid_2d(int64_t blocks) {
    if (blocks < 1) blocks = 1;
    const int64_t gx = blocks < kGridX ? blocks : kGridX;
    const int64_t gy = (blocks + gx - 1) / gx;
    return dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
}

// Exponent field all ones <=> +-inf or NaN (binary16: bits 14..10,
// bfloat16: bits 14..7, binary32: bits 30..23).  x holds one element.
template <int DT>
__device__ __forceinline__ bool elem_nonfinite(uint32_t x) {
    if (DT == ZERO_F32) return (x & 0x7F800000u) == 0x7F800000u;
    return DT == ZERO_F16 ? (x & 0x7C00u) == 0x7C00u : (x & 0x7F80u) == 0x7F80u;
}

template <int DT>
__device__ __forceinline__ float grad_to_f32(uint32_t h) {
    if (DT == ZERO_F32) return __uint_as_float(h);
    if (DT == ZERO_BF16) return __uint_as_float(h << 16);
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)));
}

// fp32 -> half, IEEE round to nearest even (hardware conversion).
template <int DT>
__device__ __forceinline__ uint16_t f32_to_half(float x) {
    if (DT == ZERO_BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}

// Reductions over a wave's 64 lanes on the cross-lane data path (DPP: shifts
// within rows of 16 lanes, then two broadcasts across them), a few cycles a
// step where a permute through LDS takes tens.  The result is uniform.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp(int x, int identity) {
    return __builtin_amdgcn_update_dpp(identity, x, CTRL, ROWS, 0xF, false);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_max(float x, float identity) {
    return fmaxf(x, __int_as_float(dpp<CTRL, ROWS>(__float_as_int(x), __float_as_int(identity))));
}

// The largest value (NaNs aside).
__device__ __forceinline__ float wave_max(float x) {
    const float identity = -__builtin_inff();
    x = dpp_max<0x111, 0xF>(x, identity);
    x = dpp_max<0x112, 0xF>(x, identity);
    x = dpp_max<0x114, 0xF>(x, identity);
    x = dpp_max<0x118, 0xF>(x, identity);
    x = dpp_max<0x142, 0xA>(x, identity);
    x = dpp_max<0x143, 0xC>(x, identity);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
    return max(x, static_cast<uint32_t>(dpp<CTRL, ROWS>(static_cast<int>(x), 0)));
}

// The largest unsigned value; one instruction a step, as 0 is its identity
// (a float's needs a copy and a quieting besides).
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = dpp_max<0x111, 0xF>(x);
    x = dpp_max<0x112, 0xF>(x);
    x = dpp_max<0x114, 0xF>(x);
    x = dpp_max<0x118, 0xF>(x);
    x = dpp_max<0x142, 0xA>(x);
    x = dpp_max<0x143, 0xC>(x);
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), 63));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double x) {
    const int lo = dpp<CTRL, ROWS>(__double2loint(x), 0);
    const int hi = dpp<CTRL, ROWS>(__double2hiint(x), 0);
    return x + __hiloint2double(hi, lo);
}

__device__ __forceinline__ double wave_sum(double x) {
    x = dpp_add<0x111, 0xF>(x);
    x = dpp_add<0x112, 0xF>(x);
    x = dpp_add<0x114, 0xF>(x);
    x = dpp_add<0x118, 0xF>(x);
    x = dpp_add<0x142, 0xA>(x);
    x = dpp_add<0x143, 0xC>(x);
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(x), 63),
                            __builtin_amdgcn_readlane(__double2loint(x), 63));
}

// One element of the update, fp32, one rounding per operation.
template <bool ADAMW>
__device__ __forceinline__ void adam_elem(float g, float& p, float& m, float& v,
                                          const AdamScalars& c) {
    float gu = g * c.inv_scale;
    if (!ADAMW) gu = gu + c.wd * p;
    m = c.b1 * m + c.omb1 * gu;
    v = c.b2 * v + c.omb2 * (gu * gu);
    // __builtin_sqrtf and '/' are correctly rounded under
    // -fhip-fp32-correctly-rounded-divide-sqrt (HIP's __fsqrt_rn is not).
    const float d = __builtin_sqrtf(v) * c.rsbc2 + c.eps;
    const float u = m / d;
    p = p * c.decay - c.step * u;
}

}  // namespace zmi
