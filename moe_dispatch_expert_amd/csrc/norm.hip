// norm.hip -- residual addition + root-mean-square norm, with outputs in bf16
// and in e4m3 with one scale per row and 128 columns: the step in front of the
// router and the experts.
//
//   h = x + r,   y = h * gamma / sqrt(mean(h^2) + eps)
//   per group of 128 columns: s = max(max |y|, 2^-40) / 448,  q = e4m3(y / s)
//
// One pass: a row's h stays in registers between the sum of squares and the
// outputs, so each input is read once and each output written once.  h, the sum
// and y are fp32; h, y and q are rounded once each, all from the fp32 values
// (the norm does not see h's bf16 rounding, q does not see y's).
//
// Bound by memory: 4 bytes in, 4 (h, y) + 1.03 (q, s) out per element.  A workgroup per row, because a row then stays in
// registers at any width with at most 32 columns a thread, and one 16-byte piece a thread keeps every load of the row on
// its way at once.  Measured: 4096 x 4096, h and y, 23 us (5.8 TB/s); 16384 x 7168, all outputs, 185 us (5.7 TB/s; a
// plain copy of 2 GiB reaches 4.9 TB/s); one token of 7168 2.7 us, the launch itself.
#include <hip/hip_runtime.h>

#include "mk_device.h"
#include "mk_launch.h"
#include "norm_args.h"
#include "route_dev.h"

namespace mk {

namespace {

constexpr float kAmaxFloor = 0x1p-40f;   // keeps 448 / amax finite in a group of zeros
constexpr float kE4m3Max = 448.0f;
// Rows of a mean square + eps below 2^-90 (only with an eps below that) are summed up again at 2^96 times their size, where
// the smallest bf16's square is 2^-74 and the largest such row's sum 2^117.
constexpr float kTinyMean = 0x1p-90f, kTinyScale = 0x1p96f;

// Maximum over the 16 lanes of a DPP row; every lane of the row receives it.
__device__ __forceinline__ float row16_max(float v)
{
    v = fmaxf(v, dpp_f32<kDppXor1>(v));
    v = fmaxf(v, dpp_f32<kDppXor2>(v));
    v = fmaxf(v, dpp_f32<kDppHalfMirror>(v));
    return fmaxf(v, dpp_f32<kDppMirror>(v));
}

__device__ __forceinline__ u32x4_t pack8(const float (&f)[8])
{
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    u32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){f[2 * i], f[2 * i + 1]}, bf16x2_t));
    return o;
}

// Sum over the workgroup; red: LDS of its own.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float *red)
{
    v = wave_sum_f32(v);
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w) v += red[w];
    return v;
}

}  // namespace

// A workgroup's row; a thread owns the 8-column pieces i THREADS + its index,
// i < NP.  A piece is one 16-byte load of x and of r, and 16 neighbouring
// threads (one DPP row) hold a group of 128 columns.
template <int THREADS, int NP>
__global__ __launch_bounds__(THREADS) void k_add_rmsnorm(NormArgs a)
{
    const int ti = (int)threadIdx.x, t = (int)blockIdx.x;
    const int pieces = a.d / 8;
    const size_t row = (size_t)t * a.d;
    float h[NP][8];
    float ss = 0.0f;
    u32x4_t vx[NP], vr[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int p = min(ti + i * THREADS, pieces - 1);
        vx[i] = *(const u32x4_t *)(a.x + row + 8 * p);
        if (a.res) vr[i] = *(const u32x4_t *)(a.res + row + 8 * p);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        unpack8(vx[i], h[i]);
        if (a.res) {
            float r[8];
            unpack8(vr[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] += r[j];
        }
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) part = __builtin_fmaf(h[i][j], h[i][j], part);
        ss += ti + i * THREADS < pieces ? part : 0.0f;
    }
    __shared__ float red[2][THREADS / kWave];
    float mean = block_sum<THREADS>(ss, red[0]) / (float)a.d + a.eps;
    if (a.res_out) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (ti + i * THREADS < pieces) *(u32x4_t *)(a.res_out + row + 8 * (ti + i * THREADS)) = pack8(h[i]);
    }
    if (mean < kTinyMean) {   // the whole row: its squares may be below fp32's range, those of 2^96 h are not
        ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float part = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[i][j] *= kTinyScale;
                part = __builtin_fmaf(h[i][j], h[i][j], part);
            }
            ss += ti + i * THREADS < pieces ? part : 0.0f;
        }
        mean = block_sum<THREADS>(ss, red[1]) / (float)a.d + a.eps * kTinyScale * kTinyScale;
    }
    const float inv = 1.0f / sqrtf(mean);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int p = ti + i * THREADS;
        const bool in = p < pieces;
        const int pc = min(p, pieces - 1);
        float g[8], y[8];
        unpack8(*(const u32x4_t *)(a.gamma + 8 * pc), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = h[i][j] * inv * g[j];
        if (a.y && in) *(u32x4_t *)(a.y + row + 8 * p) = pack8(y);
        if (a.q) {
            // d % 128 == 0: the 16 lanes of a group are all inside the row or all outside
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(y[j]));   // leaves NaN out
            const float amax = fmaxf(row16_max(m), kAmaxFloor);
            const float s = amax / kE4m3Max;
            const float rs = 1.0f / s;   // y * rs is within one fp32 step of y / s
            uint32_t lo = 0, hi = 0;
            lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * rs, y[1] * rs, lo, false);
            lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * rs, y[3] * rs, lo, true);
            hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4] * rs, y[5] * rs, hi, false);
            hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6] * rs, y[7] * rs, hi, true);
            if (in) {
                *(uint2 *)(a.q + row + 8 * p) = make_uint2(lo, hi);
                if ((ti & 15) == 0) a.qs[(size_t)t * (a.d / 128) + p / 16] = s;
            }
        }
    }
}

namespace {

// A launch takes fewer than 2^32 work items (more are not refused, their rows are left out), so more rows than that go
// to several.
template <int THREADS, int NP>
hipError_t launch_norm_as(NormArgs a, hipStream_t s)
{
    constexpr int kRows = 0x7FFFFFFF / THREADS;
    for (int left = a.T; left > 0; left -= kRows) {
        const int n = left < kRows ? left : kRows;
        const size_t e = (size_t)n * a.d;
        hipLaunchKernelGGL((k_add_rmsnorm<THREADS, NP>), dim3(n), dim3(THREADS), 0, s, a);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        a.x += e;
        if (a.res) a.res += e;
        if (a.res_out) a.res_out += e;
        if (a.y) a.y += e;
        if (a.q) a.q += e, a.qs += e / 128;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs &a, hipStream_t s)
{
    const int pieces = a.d / 8;
    if (pieces <= 256) return launch_norm_as<256, 1>(a, s);
    if (pieces <= 512) return launch_norm_as<512, 1>(a, s);
    if (pieces <= 1024) return launch_norm_as<1024, 1>(a, s);
    if (pieces <= 2048) return launch_norm_as<1024, 2>(a, s);
    if (pieces <= 4096) return launch_norm_as<1024, 4>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace mk
