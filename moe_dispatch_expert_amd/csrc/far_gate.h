// far_gate.h -- gates of a SwiGLU for which e^g is outside fp32's range, or close to its end, while products with it are not.
#pragma once

#include "mk_device.h"
#include "route_dev.h"

namespace mk {

constexpr float kLog2eHi = 1.44268798828125f;   // log2(e) to 15 bits: its product with a bf16 value is exact
constexpr float kExpLo = 4.8884952e-06f;        // 1 - kLog2eHi ln(2): what is left of the exponent

constexpr uint32_t kFarGate = 0xC2A0u, kNegInf = 0xFF80u;   // -80 and -infinity in bf16

// Whether bf16 value g is finite and below -80.
__device__ __forceinline__ bool is_far(uint32_t g) { return g > kFarGate && g < kNegInf; }

// Whether one of 8 bf16 values is below -80 (or a NaN with a sign).
__device__ __forceinline__ bool any_far(u32x4_t x)
{
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    u16x2_t m = __builtin_bit_cast(u16x2_t, x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, x[i]));
    return max(m[0], m[1]) > kFarGate;
}

// Value j of 8.
__device__ __forceinline__ uint32_t bf16_of(u32x4_t x, int j) { return j % 2 ? x[j / 2] >> 16 : x[j / 2] & 0xFFFFu; }

// e^g = f 2^n to within 2^-22 for a far gate g (below -400 that of -400, whose products with what bf16 holds are 0):
// n + w = g kLog2eHi, 2^w e^y with y = g kExpLo.
__device__ __forceinline__ float far_exp(float g, int &n)
{
    const float a = fmaxf(g, -400.0f), r = __builtin_rintf(a * kLog2eHi), y = a * kExpLo;
    n = (int)r;
    return __builtin_amdgcn_exp2f(a * kLog2eHi - r) * __builtin_fmaf(y, __builtin_fmaf(y, 0.5f, 1.0f), 1.0f);
}

// x = (the result) 2^n with the result in [1/2, 1) (0, infinities and NaN themselves); n is added to.
__device__ __forceinline__ float apart(float x, int &n)
{
    n += __builtin_amdgcn_frexp_expf(x);
    return __builtin_amdgcn_frexp_mantf(x);
}

}  // namespace mk
