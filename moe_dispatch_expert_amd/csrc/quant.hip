// quant.hip -- rows of 8-bit integers with one scale each, from bf16 rows or from the SwiGLU of gate|up rows: what the
// 8-bit grouped product reads.
//
//   m = max |v|,   scale = m / 127,   q = round(127 v / m)   (ties to even; scale 0 and codes 0 in a row of zeros)
//
// v = x (bf16), or v = silu(g) u in fp32, not rounded in between.  127 x of a bf16 x is exact in fp32 and the quotient
// 127 x / m of two bf16 values is a tie only where it is one exactly (otherwise it is at least 2^-16 away from it,
// relative), so one correctly rounded division gives the codes of the real numbers.  A row stays in registers between its
// maximum and its codes: one pass, bound by memory.
#include <hip/hip_runtime.h>

#include "grouped_args.h"
#include "mk_device.h"
#include "mk_launch.h"
#include "route_dev.h"

namespace mk {

template <int THREADS, int NP, bool SWIGLU>
__global__ __launch_bounds__(THREADS) void k_quant_i8(QuantArgs a, int row0)
{
    const int ti = (int)threadIdx.x, r = row0 + (int)blockIdx.x;
    if (a.rows_valid && r >= *a.rows_valid) return;   // uniform
    const int pieces = a.d / 8;
    const uint16_t *x = a.x + (size_t)r * a.d * (SWIGLU ? 2 : 1);
    float v[NP][8];
    u32x4_t vx[NP], vu[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int p = min(ti + i * THREADS, pieces - 1);
        vx[i] = *(const u32x4_t *)(x + 8 * p);
        if (SWIGLU) vu[i] = *(const u32x4_t *)(x + a.d + 8 * p);
    }
    // the bits of |v| as an unsigned number: ordered like |v|, with infinities and NaN above every finite value
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        unpack8(vx[i], v[i]);
        if (SWIGLU) {
            float u[8];
            unpack8(vu[i], u);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] / (1.0f + expf(-v[i][j])) * u[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
    }
    m = wave_max_u32(m);
    __shared__ uint32_t red[THREADS / kWave];
    if (ti % kWave == 0) red[ti / kWave] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w) m = max(m, red[w]);
    const float big = __uint_as_float(m);
    const bool finite = m < 0x7F800000u;
    if (ti == 0) a.scale[r] = finite ? big / 127.0f : __uint_as_float(0x7FC00000u);
    // 127 v stays finite: rows of large values are taken 2^-8 times as large, which changes no quotient
    const float down = big > 1.0f ? 0x1p-8f : 1.0f;
    const bool live = finite && m != 0;
    const float den = live ? big * down : 1.0f;
    const float num = live ? 127.0f * down : 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int p = ti + i * THREADS;
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float t = live ? v[i][j] * num / den : 0.0f;
            w[j / 4] |= ((uint32_t)(int32_t)__builtin_rintf(t) & 0xFFu) << (8 * (j % 4));
        }
        if (p < pieces) *(uint2 *)(a.q + (size_t)r * a.d + 8 * p) = make_uint2(w[0], w[1]);
    }
}

namespace {

// A launch takes fewer than 2^32 work items, so more rows than that go to several.
template <int THREADS, int NP>
hipError_t launch_quant_as(const QuantArgs &a, bool swiglu, hipStream_t s)
{
    constexpr int kRows = 0x7FFFFFFF / THREADS;
    for (int r0 = 0; r0 < a.rows;) {
        const int n = a.rows - r0 < kRows ? a.rows - r0 : kRows;
        if (swiglu) hipLaunchKernelGGL((k_quant_i8<THREADS, NP, true>), dim3(n), dim3(THREADS), 0, s, a, r0);
        else hipLaunchKernelGGL((k_quant_i8<THREADS, NP, false>), dim3(n), dim3(THREADS), 0, s, a, r0);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        r0 += n;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_quant_i8(const QuantArgs &a, bool swiglu, hipStream_t s)
{
    const int pieces = a.d / 8;
    if (pieces <= 256) return launch_quant_as<256, 1>(a, swiglu, s);
    if (pieces <= 512) return launch_quant_as<512, 1>(a, swiglu, s);
    if (pieces <= 1024) return launch_quant_as<1024, 1>(a, swiglu, s);
    if (pieces <= 2048) return launch_quant_as<1024, 2>(a, swiglu, s);
    if (pieces <= 4096) return launch_quant_as<1024, 4>(a, swiglu, s);
    return hipErrorInvalidValue;
}

}  // namespace mk
