// quant.hip -- rows of 8-bit integers with one scale each, from bf16 rows or from the SwiGLU of gate|up rows: what the
// 8-bit grouped product reads.
//
//   m = max |v|,   scale = m / 127,   q = round(127 v / m)   (ties to even; scale 0 and codes 0 in a row of zeros)
//
// v = x (bf16), or v = silu(g) u in fp32, not rounded in between.  A row stays in registers between its maximum and its
// codes: one pass, bound by memory, as long as the arithmetic stays short:
//   - No division per element: r = v (127 / m) is within 2^-22 of 127 v / m, relative.  For bf16 rows the codes are still those of
//     the real numbers: 127 x / m of two bf16 values (significands below 2^8) is a tie only where it is one exactly, and
//     otherwise at least 2^-16 away from one, relative; so r is first rounded to 20 bits, which makes every tie a tie again and
//     carries nothing else across one.
//   - silu(g) = g / (1 + e^-g) with e^-g = 2^(-g c) e^(-g c'), c = log2(e) to 15 bits: g has 8 bits, so the product g c is exact, and
//     the second factor is 1 - g c' to within 2^-23 (|g| < 88; above, the result is g u).  Gates below -80 take a longer way that
//     keeps e^g's exponent apart (a wave without one skips it): h = g e^g u may be an ordinary number there.
// 49152 rows of 1408 from gate|up: 60 us, 5.8 TB/s (128 with expf, divisions and a workgroup a row); 8192 rows of 2048: 11 us.
#include <hip/hip_runtime.h>

#include "far_gate.h"
#include "grouped_args.h"
#include "mk_device.h"
#include "mk_launch.h"
#include "route_dev.h"

namespace mk {

namespace {

// silu(g) u for g >= -80, infinities and NaN (NaN then, of infinities too).
__device__ __forceinline__ float swiglu(float g, float u)
{
    const float e = __builtin_amdgcn_exp2f(-g * kLog2eHi) * __builtin_fmaf(-g, kExpLo, 1.0f);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// The same for a far gate, where it is g e^g u to within fp32; 2^n comes last, so that nothing leaves the range that the result
// does not leave.
__device__ __forceinline__ float swiglu_far(float g, float u)
{
    int n;
    const float e = far_exp(g, n);
    return ldexpf(fmaxf(g, -400.0f) * e * apart(u, n), n);
}

}  // namespace

// LANES threads a row (64: a wave, four rows a workgroup; else a workgroup), NP pieces of 8 columns a thread.
template <int LANES, int NP, bool SWIGLU>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void k_quant_i8(QuantArgs a, int row0)
{
    constexpr int ROWS = LANES < 256 ? 256 / LANES : 1;
    const int ti = (int)threadIdx.x % LANES;
    const uint32_t r =   // (the last workgroup's may pass 2^31)
        (uint32_t)row0 + blockIdx.x * ROWS + (ROWS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / LANES) : 0u);
    const int rows = a.rows_valid ? min(a.rows, max(0, *a.rows_valid)) : a.rows;
    if (r >= (uint32_t)rows) return;   // the same for all threads of a row
    const int pieces = a.d / 8;
    const uint16_t *x = a.x + (size_t)r * a.d * (SWIGLU ? 2 : 1);
    float v[NP][8];
    u32x4_t vx[NP], vu[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int p = min(ti + i * LANES, pieces - 1);
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
            for (int j = 0; j < 8; ++j) v[i][j] = swiglu(v[i][j], u[j]);
            if (__builtin_expect(any_far(vx[i]), 0)) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t g = bf16_of(vx[i], j);
                    if (is_far(g)) v[i][j] = swiglu_far(__uint_as_float(g << 16), u[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
    }
    m = wave_max_u32(m);
    if constexpr (LANES > kWave) {
        __shared__ uint32_t red[LANES / kWave];
        if (ti % kWave == 0) red[ti / kWave] = m;
        __syncthreads();
        m = 0;
#pragma unroll
        for (int w = 0; w < LANES / kWave; ++w) m = max(m, red[w]);
    }
    const float big = __uint_as_float(m);
    const bool finite = m < 0x7F800000u, live = finite && m != 0;
    if (ti == 0) a.scale[r] = finite ? big / 127.0f : __uint_as_float(0x7FC00000u);
    // 127 / m stays finite: rows of tiny values are taken 2^100 times as large, which changes no quotient
    const float up = big < 0x1p-100f ? 0x1p100f : 1.0f;
    const float k = 127.0f / (live ? big * up : 1.0f);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int p = ti + i * LANES;
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float t = v[i][j] * up * k;
            if (!SWIGLU) t = __uint_as_float((__float_as_uint(t) + 8u) & ~15u);   // 20 bits
            w[j / 4] |= ((uint32_t)(int32_t)__builtin_rintf(t) & 0xFFu) << (8 * (j % 4));
        }
        if (p < pieces) *(uint2 *)(a.q + (size_t)r * a.d + 8 * p) = live ? make_uint2(w[0], w[1]) : make_uint2(0u, 0u);
    }
}

namespace {

// A launch takes fewer than 2^32 work items, so more rows than that go to several.
template <int LANES, int NP>
hipError_t launch_quant_as(const QuantArgs &a, bool swiglu, hipStream_t s)
{
    constexpr int THREADS = LANES < 256 ? 256 : LANES, ROWS = THREADS / LANES;
    constexpr int64_t kRows = (int64_t)(0x7FFFFFFF / THREADS) * ROWS;
    for (int64_t r0 = 0; r0 < a.rows; r0 += kRows) {
        const int64_t n = a.rows - r0 < kRows ? a.rows - r0 : kRows;
        const dim3 grid((uint32_t)((n + ROWS - 1) / ROWS));
        if (swiglu) hipLaunchKernelGGL((k_quant_i8<LANES, NP, true>), grid, dim3(THREADS), 0, s, a, (int)r0);
        else hipLaunchKernelGGL((k_quant_i8<LANES, NP, false>), grid, dim3(THREADS), 0, s, a, (int)r0);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

// A wave holds a row of up to 2048 columns.  A few such rows of more than 1024 are spread over workgroups of their own
// instead, where all their loads are on their way at once.  Measured (us in a graph, a wave / a workgroup a row): 2048
// columns: 512 rows 2.60 / 2.23, 1024 2.70 / 2.86, 4096 4.78 / 5.39; 1024 columns: 64 rows 2.02 / 2.06, 16384 9.5 / 12.3.
hipError_t launch_quant_i8(const QuantArgs &a, bool swiglu, hipStream_t s)
{
    const int pieces = a.d / 8;
    if (pieces <= 128 || (pieces <= 256 && a.rows >= 1024)) {
        if (pieces <= 64) return launch_quant_as<64, 1>(a, swiglu, s);
        if (pieces <= 128) return launch_quant_as<64, 2>(a, swiglu, s);
        if (pieces <= 192) return launch_quant_as<64, 3>(a, swiglu, s);
        return launch_quant_as<64, 4>(a, swiglu, s);
    }
    if (pieces <= 256) return launch_quant_as<256, 1>(a, swiglu, s);
    if (pieces <= 512) return launch_quant_as<512, 1>(a, swiglu, s);
    if (pieces <= 1024) return launch_quant_as<1024, 1>(a, swiglu, s);
    if (pieces <= 2048) return launch_quant_as<1024, 2>(a, swiglu, s);
    if (pieces <= 4096) return launch_quant_as<1024, 4>(a, swiglu, s);
    return hipErrorInvalidValue;
}

}  // namespace mk
