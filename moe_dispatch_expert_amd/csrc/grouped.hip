// grouped.hip -- the grouped product's gradients (bf16) and the grouped product of 8-bit integers:
//   dgrad   da[r, i]    = sum_n dy[r, n] W[e, n, i]                       rows r of expert e
//   wgrad   dW[e, n, i] = sum over e's rows of dy[r, n] a[r, i]
//   8-bit   y[r, n]     = a_scale[r] w_scale[e, n] sum_i a[r, i] w[e, n, i]
// One 64 x 64 tile per workgroup; both operands go through LDS with the contraction contiguous.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gemm_dev.h"
#include "grouped_args.h"
#include "mk_device.h"
#include "mk_launch.h"

namespace mk {

namespace {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));

enum { kDgrad = 0, kWgrad = 1, kI8 = 2 };

__device__ __forceinline__ int row_lo(const GroupedArgs &a, int e) { return min(max(a.offsets[e], 0), a.rows); }
__device__ __forceinline__ int row_hi(const GroupedArgs &a, int e)
{
    return max(row_lo(a, e), min(max(a.offsets[e + 1], 0), a.rows));
}

// Row of `a` that row r of the product reads, or -1.
__device__ __forceinline__ int a_row(const GroupedArgs &a, int r)
{
    if (!a.row_token) return r;
    const int t = a.row_token[r];
    return t >= 0 && t < a.a_rows ? t : -1;
}

}  // namespace

// Tile (m0, c0) of expert blockIdx.y.  LDS row: 64 bytes of contraction (32 bf16 or 64 int8), padded to 80.
template <int KIND>
__global__ __launch_bounds__(256) void k_grouped_plain(GroupedArgs a)
{
    __shared__ __attribute__((aligned(16))) char sm[64 * 80], sc[64 * 80];
    const int e = (int)blockIdx.y;
    const int lo = row_lo(a, e), hi = row_hi(a, e), cnt = hi - lo;
    const int M = KIND == kWgrad ? a.N : cnt;          // output rows
    const int C = KIND == kI8 ? a.N : a.K;             // output columns
    const int L = KIND == kDgrad ? a.N : (KIND == kWgrad ? cnt : a.K);   // contraction
    constexpr int STEP = KIND == kI8 ? 64 : 32;
    const int nc = (C + 63) / 64, nm = (M + 63) / 64;
    const int ti = (int)threadIdx.x, lane = ti % kWave, wave = ti / kWave;
    for (int64_t q = blockIdx.x; q < (int64_t)nc * nm; q += gridDim.x) {
        const int m0 = (int)(q / nc) * 64, c0 = (int)(q % nc) * 64;
        f32x4_t acc[4];
        i32x4_t iacc[4];
        for (int j = 0; j < 4; ++j) {
            acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            iacc[j] = i32x4_t{0, 0, 0, 0};
        }
        for (int l0 = 0; l0 < L; l0 += STEP) {
            __syncthreads();
            for (int i = ti; i < 64 * STEP; i += 256) {
                const int l = l0 + i % STEP, m = m0 + i / STEP, c = c0 + i / STEP;
                if constexpr (KIND == kI8) {
                    int8_t vm = 0, vc = 0;
                    if (l < L && m < M) {
                        const int t = a_row(a, lo + m);
                        if (t >= 0) vm = ((const int8_t *)a.a)[(size_t)t * a.K + l];
                    }
                    if (l < L && c < C) vc = ((const int8_t *)a.w)[((size_t)e * a.N + c) * a.K + l];
                    sm[(i / STEP) * 80 + i % STEP] = vm;
                    sc[(i / STEP) * 80 + i % STEP] = vc;
                } else {
                    uint16_t vm = 0, vc = 0;
                    if constexpr (KIND == kDgrad) {
                        if (l < L && m < M) vm = a.dy[(size_t)(lo + m) * a.N + l];
                        if (l < L && c < C) vc = ((const uint16_t *)a.w)[((size_t)e * a.N + l) * a.K + c];
                    } else if (l < L) {
                        const int t = a_row(a, lo + l);
                        if (m < M) vm = a.dy[(size_t)(lo + l) * a.N + m];
                        if (c < C && t >= 0) vc = ((const uint16_t *)a.a)[(size_t)t * a.K + c];
                    }
                    ((uint16_t *)(sm + (i / STEP) * 80))[i % STEP] = vm;
                    ((uint16_t *)(sc + (i / STEP) * 80))[i % STEP] = vc;
                }
            }
            __syncthreads();
            const int f = (lane & 15) * 80 + (lane >> 4) * 16;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (KIND == kI8)
                    iacc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(*(i32x4_t *)(sc + j * 16 * 80 + f),
                                                                    *(i32x4_t *)(sm + wave * 16 * 80 + f), iacc[j], 0, 0, 0);
                else
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*(bf16x8_t *)(sc + j * 16 * 80 + f),
                                                                     *(bf16x8_t *)(sm + wave * 16 * 80 + f), acc[j], 0, 0, 0);
            }
        }
        const int m = m0 + wave * 16 + (lane & 15);
        if (m < M) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int c = c0 + j * 16 + 4 * (lane >> 4) + v;
                    if (c >= C) continue;
                    if constexpr (KIND == kI8) {
                        const int t = a_row(a, lo + m);
                        const float s = t >= 0 ? a.a_scale[t] : 0.0f;
                        ((uint16_t *)a.out)[(size_t)(lo + m) * a.N + c] =
                            f32_to_bf16((float)iacc[j][v] * a.w_scale[(size_t)e * a.N + c] * s);
                    } else if constexpr (KIND == kDgrad) {
                        ((uint16_t *)a.out)[(size_t)(lo + m) * a.K + c] = f32_to_bf16(acc[j][v]);
                    } else {
                        const size_t o = ((size_t)e * a.N + m) * a.K + c;
                        if (!a.out_f32) ((uint16_t *)a.out)[o] = f32_to_bf16(acc[j][v]);
                        else ((float *)a.out)[o] = a.accumulate ? ((float *)a.out)[o] + acc[j][v] : acc[j][v];
                    }
                }
        }
    }
}

namespace {

template <int KIND>
hipError_t launch_plain(const GroupedArgs &a, hipStream_t s)
{
    const int64_t m = KIND == kWgrad ? a.N : a.rows, c = KIND == kI8 ? a.N : a.K;
    const int64_t tiles = ((m + 63) / 64) * ((c + 63) / 64);
    hipLaunchKernelGGL(k_grouped_plain<KIND>, dim3((uint32_t)std::min<int64_t>(tiles, 4096), a.E), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_dgrad(const GroupedArgs &a, hipStream_t s) { return launch_plain<kDgrad>(a, s); }
hipError_t launch_grouped_wgrad(const GroupedArgs &a, hipStream_t s) { return launch_plain<kWgrad>(a, s); }
hipError_t launch_grouped_i8(const GroupedArgs &a, hipStream_t s) { return launch_plain<kI8>(a, s); }

}  // namespace mk
