// backward.hip -- gradients of the combine and of the SwiGLU: the steps around the grouped products' gradients in the
// backward pass of an MoE layer.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "far_gate.h"
#include "gemm_dev.h"
#include "grouped_args.h"
#include "mk_device.h"
#include "mk_launch.h"
#include "route_dev.h"

namespace mk {

namespace {

__device__ __forceinline__ u32x4_t pack8(const float (&f)[8])
{
    return u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

// s = 1 / (1 + e^-g) and 1 - s = 1 / (1 + e^g), both from e^-|g|, so that neither overflows nor cancels.
__device__ __forceinline__ void sigmoid_both(float g, float &s, float &t)
{
    const float z = expf(-fabsf(g));
    const float p = 1.0f / (1.0f + z), q = z * p;
    s = g < 0.0f ? q : p;
    t = g < 0.0f ? p : q;
}

}  // namespace

// Gradient of the combine  out[t] = sum_j w[t, j] y[slot(t, j)]:
//   dy[slot(t, j)] = w[t, j] dout[t],   dw[t, j] = sum_n dout[t, n] y[slot(t, j), n]
// A workgroup per token keeps the token's dout in registers (pieces of 8 columns, 2048 NP at a time) and goes through its
// choices, so dout is read once and y and dy once per choice.  A slot that a token names more than once is visited once,
// with the sum of its gates.  The dot products' partial sums (thread, wave, workgroup) are fp32 in a fixed order.  Bound by memory:
// 16384 tokens of 7168, one local choice each on the mean (0.7 GB): 138 us, 5.1 TB/s.
template <int NP>
__global__ __launch_bounds__(256) void k_combine_backward(CombineBackwardArgs a)
{
    constexpr int U = 4 / NP < 2 ? 2 : 4 / NP;
    __shared__ int32_t s_slot[kMaxK];
    __shared__ float s_w[kMaxK];
    __shared__ int32_t s_first[kMaxK];   // the token's first choice of the same slot
    __shared__ float s_dot[kMaxK][4];
    const int ti = (int)threadIdx.x, wave = ti / kWave, lane = ti % kWave;
    const int pieces = a.N / 8;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        if (wave == 0) {
            const int slot = lane < a.k ? a.slot_of[t * a.k + lane] : -1;
            const float w = lane < a.k ? a.gate[t * a.k + lane] : 0.0f;
            float sum = 0.0f;
            int first = lane;
            for (int j = a.k - 1; j >= 0; --j) {
                const int s2 = __builtin_amdgcn_readlane(slot, j);
                const float w2 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), j));
                sum += s2 == slot ? w2 : 0.0f;
                first = s2 == slot ? j : first;
            }
            if (lane < a.k) {
                s_slot[lane] = first == lane && slot >= 0 && slot < a.rows ? slot : -1;
                s_w[lane] = sum;
                s_first[lane] = first;
            }
        }
        if (ti < kMaxK * 4) ((float *)s_dot)[ti] = 0.0f;
        __syncthreads();
        for (int p0 = 0; p0 < pieces; p0 += 256 * NP) {
            u32x4_t d[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i)
                d[i] = *(const u32x4_t *)(a.dout + t * a.N + 8 * min(p0 + ti + 256 * i, pieces - 1));
            // U choices at a time: their rows are all asked for before the first is used
            for (int j0 = 0; j0 < a.k; j0 += U) {
                u32x4_t v[U][NP];
                int slot[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    slot[u] = j0 + u < a.k ? __builtin_amdgcn_readfirstlane(s_slot[min(j0 + u, kMaxK - 1)]) : -1;
                    if (a.dgate && slot[u] >= 0) {
#pragma unroll
                        for (int i = 0; i < NP; ++i)
                            v[u][i] =
                                *(const u32x4_t *)(a.y + (size_t)slot[u] * a.N + 8 * min(p0 + ti + 256 * i, pieces - 1));
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (slot[u] < 0) continue;   // uniform
                    const float w = s_w[j0 + u];
                    float dot = 0.0f;
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        const int p = p0 + ti + 256 * i;
                        const bool in = p < pieces;
                        float f[8], o[8];
                        unpack8(d[i], f);
#pragma unroll
                        for (int q = 0; q < 8; ++q) o[q] = w * f[q];
                        if (in) *(u32x4_t *)(a.dy + (size_t)slot[u] * a.N + 8 * p) = pack8(o);
                        if (a.dgate) {
                            float y[8], part = 0.0f;
                            unpack8(v[u][i], y);
#pragma unroll
                            for (int q = 0; q < 8; ++q) part = __builtin_fmaf(f[q], y[q], part);
                            dot += in ? part : 0.0f;
                        }
                    }
                    if (a.dgate) {
                        dot = wave_sum_f32(dot);
                        if (lane == 0) s_dot[j0 + u][wave] += dot;
                    }
                }
            }
        }
        __syncthreads();
        if (a.dgate && ti < a.k) {
            const float *d = s_dot[s_first[ti]];
            a.dgate[t * a.k + ti] = (d[0] + d[1]) + (d[2] + d[3]);
        }
        __syncthreads();   // the tables are free for the next token
    }
}

// Gradient of  h = silu(g) u,  silu(g) = g s,  s = 1 / (1 + e^-g):
//   dg = dh u s (1 + g (1 - s)),   du = dh g s
// in fp32, rounded once; h (if asked for) with the expression of the forward kernel, bit for bit.  Gates below -80, where s = e^g to
// within fp32, keep its exponent apart, so that dh and u may make up for it.  Item i = 8 columns of a row.
// Bound by memory: 6 bytes in, 4 (6 with h) out per feature: 8192 rows of 14336 features with h 253 us, 5.6 TB/s.
__global__ __launch_bounds__(256) void k_swiglu_backward(SwigluBackwardArgs a)
{
    const int rows = a.rows_valid ? min(a.rows, max(0, *a.rows_valid)) : a.rows;
    const int P = a.F / 8;
    const int64_t items = (int64_t)rows * P;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / P;
        const int c = (int)(i - r * P) * 8;
        float g[8], u[8], d[8], dg[8], du[8];
        const u32x4_t gates = *(const u32x4_t *)(a.gu + r * 2 * a.F + c);
        unpack8(gates, g);
        unpack8(*(const u32x4_t *)(a.gu + r * 2 * a.F + a.F + c), u);
        unpack8(*(const u32x4_t *)(a.dh + r * a.F + c), d);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float s, s1;
            sigmoid_both(g[q], s, s1);
            dg[q] = d[q] * (s * __builtin_fmaf(g[q], s1, 1.0f)) * u[q];
            du[q] = d[q] * (g[q] * s);
        }
        if (__builtin_expect(any_far(gates), 0)) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (!is_far(bf16_of(gates, q))) continue;
                int n;
                const float e = far_exp(g[q], n), f = fmaxf(g[q], -400.0f), de = apart(d[q], n) * e;
                du[q] = ldexpf(de * f, n);
                const float due = de * apart(u[q], n);
                dg[q] = ldexpf(due * (1.0f + f), n);
            }
        }
        *(u32x4_t *)(a.dgu + r * 2 * a.F + c) = pack8(dg);
        *(u32x4_t *)(a.dgu + r * 2 * a.F + a.F + c) = pack8(du);
        if (a.h) {
            float h[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) h[q] = g[q] / (1.0f + expf(-g[q])) * u[q];
            *(u32x4_t *)(a.h + r * a.F + c) = pack8(h);
        }
    }
}

hipError_t launch_combine_backward(const CombineBackwardArgs &a, hipStream_t s)
{
    const int grid = std::min(a.T, 1 << 20);
    if (a.N <= 2048) hipLaunchKernelGGL(k_combine_backward<1>, dim3(grid), dim3(256), 0, s, a);
    else if (a.N <= 4096) hipLaunchKernelGGL(k_combine_backward<2>, dim3(grid), dim3(256), 0, s, a);
    else hipLaunchKernelGGL(k_combine_backward<4>, dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_swiglu_backward(const SwigluBackwardArgs &a, hipStream_t s)
{
    const int64_t items = (int64_t)a.rows * (a.F / 8);
    const int grid = (int)std::min<int64_t>((items + 255) / 256, 65536);
    hipLaunchKernelGGL(k_swiglu_backward, dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace mk
