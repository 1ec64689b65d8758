// layer.hip -- a whole MoE layer for a few tokens (at most 128): router,
// gate|up products with SwiGLU, down product and the weighted combine.
//
//   out[t] = sum over t's local choices e of  w[t, e] * W_down[e] . ( silu(W_gate[e] . x[t]) * (W_up[e] . x[t]) )
//
// A few tokens make this a matter of streaming the chosen experts' weights once:
// 3 F d weights against 6 F d flops per row of an expert, i.e. 1 to 16 rows
// leave the matrix cores idle most of the time.  So
//   - the weights are the matrix core's A operand (16 weight rows), loaded
//     straight into registers (no LDS), 8 rows x 128 bytes per instruction, and
//     the tokens of the expert its B operand (16 columns), loaded from the L2;
//   - K is split over the waves of a workgroup, so that a workgroup's unit of
//     work is a thin slab of weights and a few experts already fill the device;
//   - the down kernel owns output columns over all experts, so the combine is a
//     sum inside one workgroup in a fixed order: no atomics, no second pass.
// Two kernels follow the router: "up" writes h = w * silu(g) * u (bf16, the
// gate folded in before the one rounding), "down" sums W_down[e] . h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "layer_args.h"
#include "mk_device.h"
#include "mk_launch.h"
#include "route_dev.h"

namespace mk {

namespace {

// ---------------------------------------------------------------- rows of the local experts

// The (token, local expert) pairs of the call, built by every workgroup in its
// LDS from the ids: a 128-bit token mask per expert (a repeated id sets the same
// bit), the experts with a bit set in ascending order, and per expert its tokens
// in ascending order.  Row r of h belongs to tok[r].
struct RowsLds {
    uint64_t *mask;     // [E_local][2]
    int32_t *start;     // [E_local] first row of the expert
    int32_t *hit;       // [<= min(E_local, T k)] experts with rows
    int32_t *n;         // [2] number of hit experts, number of rows
    uint8_t *tok;       // [T min(k, E_local)]
    float *gate;        // [T min(k, E_local)] or nullptr (down kernel)
    int32_t *ids;       // [T k]
    float *w;           // [T k] (up kernel)
};

__host__ __device__ inline int rows_cap(int T, int k, int E_local) { return T * (k < E_local ? k : E_local); }

__host__ __device__ inline size_t rows_lds_bytes(int T, int k, int E_local, bool gates)
{
    const size_t r = (size_t)rows_cap(T, k, E_local), tk = (size_t)T * k;
    const size_t hits = (size_t)E_local < tk ? (size_t)E_local : tk;
    size_t b = (size_t)E_local * 20 + hits * 4 + 8 + tk * 4 + (gates ? (tk + r) * 4 : 0) + r;
    return (b + 15) & ~(size_t)15;
}

__device__ __forceinline__ RowsLds rows_lds(char *p, const LayerArgs &a, bool gates)
{
    const int r = rows_cap(a.T, a.k, a.E_local), tk = a.T * a.k;
    RowsLds s;
    s.mask = (uint64_t *)p;
    p += (size_t)a.E_local * 16;
    s.start = (int32_t *)p;
    p += (size_t)a.E_local * 4;
    s.hit = (int32_t *)p;
    p += (size_t)min(a.E_local, tk) * 4;
    s.n = (int32_t *)p;
    p += 8;
    s.ids = (int32_t *)p;
    p += (size_t)tk * 4;
    s.w = s.gate = nullptr;
    if (gates) {
        s.w = (float *)p;
        p += (size_t)tk * 4;
        s.gate = (float *)p;
        p += (size_t)r * 4;
    }
    s.tok = (uint8_t *)p;
    return s;
}

// Rows of expert e below token t.
__device__ __forceinline__ int rank_of(const uint64_t *m, int t)
{
    return t < 64 ? __popcll(m[0] & ((1ull << t) - 1)) : __popcll(m[0]) + __popcll(m[1] & ((1ull << (t - 64)) - 1));
}

// Builds the rows from s.ids (and s.w), which the caller has filled for tokens < T; ends with a barrier.
__device__ __forceinline__ void build_rows(const RowsLds &s, const LayerArgs &a, int T)
{
    for (int i = threadIdx.x; i < 2 * a.E_local; i += blockDim.x) s.mask[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < T * a.k; i += blockDim.x) {
        const int t = i / a.k, e = s.ids[i] - a.e_begin;
        if (e >= 0 && e < a.E_local)
            atomicOr((unsigned long long *)(s.mask + 2 * e + (t >> 6)), 1ull << (t & 63));
    }
    __syncthreads();
    if (threadIdx.x < kWave) {
        const int l = threadIdx.x;
        int rows = 0, hits = 0;
        for (int c = 0; c < a.E_local; c += kWave) {
            const int e = c + l;
            const int cnt = e < a.E_local ? __popcll(s.mask[2 * e]) + __popcll(s.mask[2 * e + 1]) : 0;
            int incl = cnt;
#pragma unroll
            for (int o = 1; o < kWave; o <<= 1) {
                const int v = __shfl_up(incl, o);
                if (l >= o) incl += v;
            }
            const uint64_t b = __ballot(cnt > 0);
            if (e < a.E_local) s.start[e] = rows + incl - cnt;
            if (cnt > 0) s.hit[hits + __popcll(b & lanemask_lt())] = e;
            rows += __shfl(incl, kWave - 1);
            hits += __popcll(b);
        }
        if (l == 0) {
            s.n[0] = hits;
            s.n[1] = rows;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * a.k; i += blockDim.x) {
        const int t = i / a.k, id = s.ids[i], e = id - a.e_begin;
        if (e < 0 || e >= a.E_local) continue;
        bool first = true;
        float w = s.w ? s.w[i] : 0.0f;
        if (a.given) {   // an id given twice for a token: one row, the gates added up
            for (int j = t * a.k; j < i; ++j) first &= s.ids[j] != id;
            if (s.w)
                for (int j = i + 1; j < (t + 1) * a.k; ++j) w += s.ids[j] == id ? s.w[j] : 0.0f;
        }
        if (!first) continue;
        const int r = s.start[e] + rank_of(s.mask + 2 * e, t);
        s.tok[r] = (uint8_t)t;
        if (s.gate) s.gate[r] = w;
    }
    __syncthreads();
}

__device__ __forceinline__ int valid_tokens(const LayerArgs &a)
{
    return a.t_valid ? max(0, min(*a.t_valid, a.T)) : a.T;
}

template <int N>
struct IntC {
    static constexpr int value = N;
};

// 16 bytes at a uniform base plus the lane's 32-bit offset; load_w: weights, which no other workgroup reads.
__device__ __forceinline__ u32x4_t load_w(const char *base, uint32_t off)
{
    return __builtin_nontemporal_load((const u32x4_t *)(base + off));
}
__device__ __forceinline__ u32x4_t load_x(const char *base, uint32_t off) { return *(const u32x4_t *)(base + off); }

// Sixteen weight rows x 128 bytes come in as two loads of 8 rows x 128 bytes, so that each load reads whole cache lines:
// non-temporal loads of 16 rows x 64 bytes, which the operand layout below would give, fetch every line twice (measured
// over 2 GiB, rows 14336 bytes apart: 5.5 against 7.1 TB/s).  Lane i + 16 g of load a (rows 0 - 7) and of load b (rows
// 8 - 15) takes row i % 8, 16-byte piece g + 4 (i / 8).  Exchanging a's lanes i >= 8 with b's lanes i < 8 inside each 16
// lanes leaves the matrix core's layout, lane i + 16 g = row i: piece g in a, piece 4 + g in b.
__device__ __forceinline__ void swap_halves(u32x4_t &a, u32x4_t &b)
{
    constexpr int kRor8 = 0x128;   // DPP row_ror:8
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int x = (int)a[j], y = (int)b[j];
        a[j] = (uint32_t)__builtin_amdgcn_update_dpp(x, y, kRor8, 0xF, 0xC, false);
        b[j] = (uint32_t)__builtin_amdgcn_update_dpp(y, x, kRor8, 0xF, 0x3, false);
    }
}

__device__ __forceinline__ f32x4_t mfma_bf16(u32x4_t a, u32x4_t b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}
// Two K = 32 products of e4m3 operands: K element 16 g + i of a 64-wide step sits in lane group g, byte i, in both.
__device__ __forceinline__ f32x4_t mfma_fp8_64(u32x4_t a, u32x4_t b, f32x4_t c)
{
    const long a0 = (long)(((uint64_t)a.y << 32) | a.x), a1 = (long)(((uint64_t)a.w << 32) | a.z);
    const long b0 = (long)(((uint64_t)b.y << 32) | b.x), b1 = (long)(((uint64_t)b.w << 32) | b.z);
    c = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(a0, b0, c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(a1, b1, c, 0, 0, 0);
}

// Eight e4m3 codes as bf16 (exact).
__device__ __forceinline__ u32x4_t fp8_to_bf16(uint32_t lo, uint32_t hi)
{
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    u32x4_t o;
    o.x = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
    o.y = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
    o.z = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
    o.w = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
    return o;
}

// ---------------------------------------------------------------- gate|up

// acc[r][n] += W tile r (16 rows) x token tile n over K steps s0 .. s1 - 1 of 64.  wo[r][0], wo[r][1]: the lane's byte
// offsets from w of the tile's rows 0 - 7 and 8 - 15 (swap_halves) at K = 0; xo[n]: of its token from x, with 16 g.  U
// steps are in flight at a time.
template <int R, int NT>
__device__ __forceinline__ void up_bf16(const char *w, const uint32_t (&wo)[R][2], const char *x,
                                        const uint32_t (&xo)[NT], int s0, int s1, f32x4_t (&acc)[R][NT])
{
    int s = s0;
    auto run = [&](auto uc) {
        constexpr int U = decltype(uc)::value;
        u32x4_t wv[R][U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) wv[r][u][i] = load_w(w, wo[r][i] + (uint32_t)(s + u) * 128);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            u32x4_t xv[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) xv[u][i] = load_x(x, xo[n] + (uint32_t)(s + u) * 128 + 64 * i);
            if (n == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int r = 0; r < R; ++r) swap_halves(wv[r][u][0], wv[r][u][1]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[r][n] = mfma_bf16(wv[r][u][i], xv[u][i], acc[r][n]);
            if (NT >= 4) __builtin_amdgcn_sched_barrier(0);   // keeps later tiles' loads out of the registers
        }
        s += U;
    };
    constexpr int U = R == 1 ? 4 : NT <= 2 ? 2 : 1;
    while (s + U <= s1) run(IntC<U>());
    while (s < s1) run(IntC<1>());
}

// The same for e4m3 operands over 128-wide blocks b0 .. b1 - 1: a block's product, times the token's and the weights'
// scales of the block, joins the sum in fp32.  sw[r]: the tile's scales (this lane's rows), sx + so[n]: the lane's token's.
template <int R, int NT>
__device__ __forceinline__ void up_q8(const char *w, const uint32_t (&wo)[R][2], const char *x,
                                      const uint32_t (&xo)[NT], const float *const (&sw)[R], const float *sx,
                                      const uint32_t (&so)[NT], int b0, int b1, f32x4_t (&acc)[R][NT])
{
    int b = b0;
    auto run = [&](auto uc) {
        constexpr int U = decltype(uc)::value;
        u32x4_t wv[R][U][2];
        float fw[R][U];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < 2; ++i) wv[r][u][i] = load_w(w, wo[r][i] + (uint32_t)(b + u) * kQ8Group);
                fw[r][u] = sw[r][b + u];
            }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            u32x4_t xv[U][2];
            float fx[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int i = 0; i < 2; ++i) xv[u][i] = load_x(x, xo[n] + (uint32_t)(b + u) * kQ8Group + 64 * i);
                fx[u] = sx[so[n] + b + u];
            }
            if (n == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int r = 0; r < R; ++r) swap_halves(wv[r][u][0], wv[r][u][1]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    f32x4_t p = {0.0f, 0.0f, 0.0f, 0.0f};
                    p = mfma_fp8_64(wv[r][u][0], xv[u][0], p);
                    p = mfma_fp8_64(wv[r][u][1], xv[u][1], p);
                    const float f = fw[r][u] * fx[u];
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[r][n][q] = __builtin_fmaf(p[q], f, acc[r][n][q]);
                }
            if (NT >= 4) __builtin_amdgcn_sched_barrier(0);   // keeps later tiles' loads out of the registers
        }
        b += U;
    };
    constexpr int U = R == 1 ? 4 : NT == 1 ? 2 : 1;
    while (b + U <= b1) run(IntC<U>());
    while (b < b1) run(IntC<1>());
}

constexpr int kUpWaves = 4;

// One gate|up task: features f0 .. f0 + 8 R - 1 of local expert e, whose rows are row0 .. row0 + cnt - 1 (cnt <= 16 NT).
// R = 1: one weight tile of 8 gate and 8 up rows; R = 2: a tile of 16 gate rows and one of 16 up rows.
// red: 2 x kUpWaves x R x 256 floats; par: which half the next exchange uses.
template <bool Q8, int R, int NT>
__device__ __forceinline__ void up_task(const LayerArgs &a, const RowsLds &s, int e, int f0, int row0, int cnt,
                                        float *red, int &par)
{
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int c = lane & 15, g = lane >> 4;
    f32x4_t acc[R][NT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    // the lane's weight rows of the expert in each tile (features past F repeat the last; never stored)
    uint32_t wo[R][2], xo[NT];
    if (R == 1) {
        wo[0][0] = f0 + (c & 7);
        wo[0][1] = a.F + wo[0][0];
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            wo[0][i] = min(f0 + 8 * i + (c & 7), a.F - 1);
            wo[R - 1][i] = a.F + wo[0][i];
        }
    }
    // the lane's token in each tile (columns past cnt repeat the last; never stored)
    uint32_t tok[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) tok[n] = s.tok[row0 + min(16 * n + c, cnt - 1)];
    const size_t we = (size_t)e * 2 * a.F * a.d;
    constexpr int kBytes = Q8 ? 1 : 2;
    const char *w = (const char *)a.w_gu + we * kBytes, *x = Q8 ? (const char *)a.xq : (const char *)a.x;
    const uint32_t pitch = (uint32_t)a.d * kBytes;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) wo[r][i] = wo[r][i] * pitch + 16 * (g + 4 * (c >> 3));
#pragma unroll
    for (int n = 0; n < NT; ++n) xo[n] = tok[n] * pitch + 16 * g;
    if constexpr (Q8) {
        const int nb = a.d / kQ8Group, nf = (a.F + kQ8Group - 1) / kQ8Group;
        const float *sw[R];
        uint32_t so[NT];
        const float *se = a.s_gu + (size_t)e * 2 * nf * nb + (size_t)(f0 / kQ8Group) * nb;
        // accumulator rows 4 g .. 4 g + 3: in the mixed tile groups 0, 1 are gate rows and 2, 3 up rows
        if (R == 1) {
            sw[0] = se + (g < 2 ? 0 : (size_t)nf * nb);
        } else {
            sw[0] = se;
            sw[R - 1] = se + (size_t)nf * nb;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) so[n] = tok[n] * (uint32_t)nb;
        up_q8<R, NT>(w, wo, x, xo, sw, a.xs, so, nb * wave / kUpWaves, nb * (wave + 1) / kUpWaves, acc);
    } else {
        const int ns = a.d / 64;
        up_bf16<R, NT>(w, wo, x, xo, ns * wave / kUpWaves, ns * (wave + 1) / kUpWaves, acc);
    }
    // The waves' parts of a token tile meet in LDS ([column][row], so a lane's four rows are one 16-byte word), are
    // added in wave order, and become h.  Halves alternate: one barrier per tile.
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float *rb = red + par * kUpWaves * R * 256;
        par ^= 1;
#pragma unroll
        for (int r = 0; r < R; ++r) *(f32x4_t *)(rb + (wave * R + r) * 256 + c * 16 + 4 * g) = acc[r][n];
        __syncthreads();
        const int fi = (int)threadIdx.x % (8 * R), ci = (int)threadIdx.x / (8 * R);
        const int row = 16 * n + ci;
        if (ci < 16 && row < cnt && f0 + fi < a.F) {
            float gs = 0.0f, us = 0.0f;
#pragma unroll
            for (int w = 0; w < kUpWaves; ++w) {
                const float *q = rb + w * R * 256 + ci * 16 + fi;
                gs += q[0];
                us += q[R == 1 ? 8 : 256];
            }
            const float v = gs / (1.0f + expf(-gs)) * us * s.gate[row0 + row];
            a.h[(size_t)(row0 + row) * a.F + f0 + fi] = f32_to_bf16(v);
        }
    }
}

// SELF: the workgroup selects the experts of the few tokens itself from the router's partial sums.
template <bool Q8, int R, bool SELF>
__global__ __launch_bounds__(64 * kUpWaves, 4) void k_layer_up(LayerArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    float *red = (float *)lds;
    const RowsLds s = rows_lds(lds + 2 * kUpWaves * R * 256 * 4, a, true);
    const int T = valid_tokens(a);
    if constexpr (SELF) {
        const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
        TopkArgs ta{};
        ta.part = a.part;
        ta.bias = a.bias;
        ta.T = a.T;
        ta.E = a.E;
        ta.k = a.k;
        for (int t = wave; t < T; t += kUpWaves) {
            TopkPick p;
            if (a.E <= 64) {
                TopkPartials<1> r;
                topk_load<1>(ta, t, r);
                p = topk_pick<1>(ta, t, r);
            } else {
                TopkPartials<4> r;
                topk_load<4>(ta, t, r);
                p = topk_pick<4>(ta, t, r);
            }
            if (lane < a.k) {
                s.ids[t * a.k + lane] = p.id;
                s.w[t * a.k + lane] = p.gate();
                if (blockIdx.x == 0) a.ids_ws[t * a.k + lane] = p.id;
            }
        }
    } else {
        for (int i = threadIdx.x; i < T * a.k; i += blockDim.x) {
            s.ids[i] = a.ids[i];
            s.w[i] = a.gates[i];
        }
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < T * a.k; i += blockDim.x) {
            if (a.ids_user) a.ids_user[i] = s.ids[i];
            if (a.w_user) a.w_user[i] = s.w[i];
        }
    build_rows(s, a, T);
    const int nf = (a.F + 8 * R - 1) / (8 * R);
    const int tasks = s.n[0] * nf;
    int par = 0;
    for (int q = blockIdx.x; q < tasks; q += gridDim.x) {
        const int hi = q / nf, f0 = (q - hi * nf) * 8 * R;
        const int e = __builtin_amdgcn_readfirstlane(s.hit[hi]);
        const int row0 = __builtin_amdgcn_readfirstlane(s.start[e]);
        const int cnt = __builtin_amdgcn_readfirstlane(__popcll(s.mask[2 * e]) + __popcll(s.mask[2 * e + 1]));
        if (R == 1 || cnt <= 16) up_task<Q8, R, 1>(a, s, e, f0, row0, cnt, red, par);
        else if (cnt <= 32) up_task<Q8, R, 2>(a, s, e, f0, row0, cnt, red, par);
        else if (cnt <= 64) up_task<Q8, R, 4>(a, s, e, f0, row0, cnt, red, par);
        else up_task<Q8, R, 8>(a, s, e, f0, row0, cnt, red, par);
    }
}

// ---------------------------------------------------------------- down

constexpr int kDownWaves = 4;

// One expert's part of 16 output columns: acc[n] = sum over K of W_down rows x h rows of token tile n, for this wave's
// share of K.  wo: the lane's byte offsets from w of the rows 0 - 7 and 8 - 15 (swap_halves), ho[n]: of its h row from h
// with 16 g, all at K = 0.  kp: the lane's piece of a weight row, in elements.
template <int NT>
__device__ __forceinline__ void down_bf16(const char *w, const uint32_t (&wo)[2], int kp, const char *h,
                                          const uint32_t (&ho)[NT], int F, int wave, f32x4_t (&acc)[NT])
{
    const int ns = F / 64;
    int s = ns * wave / kDownWaves;
    const int s1 = ns * (wave + 1) / kDownWaves;
    const int kh = 8 * (int)(threadIdx.x % kWave >> 4);
    auto run = [&](auto uc, auto partial) {
        constexpr int U = decltype(uc)::value;
        // PARTIAL: the last step, with F % 64 of K left; pieces past F are zeros on both sides
        constexpr bool PARTIAL = decltype(partial)::value != 0;
        const int left = PARTIAL ? F % 64 : 64;
        const u32x4_t z = {0u, 0u, 0u, 0u};
        u32x4_t wv[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                wv[u][i] = !PARTIAL || kp < left ? load_w(w, wo[i] + (uint32_t)(s + u) * 128) : z;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            u32x4_t hv[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    hv[u][i] = !PARTIAL || kh + 32 * i < left ? load_x(h, ho[n] + (uint32_t)(s + u) * 128 + 64 * i) : z;
            if (n == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u) swap_halves(wv[u][0], wv[u][1]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) acc[n] = mfma_bf16(wv[u][i], hv[u][i], acc[n]);
            if (NT >= 4) __builtin_amdgcn_sched_barrier(0);   // keeps later tiles' loads out of the registers
        }
        s += U;
    };
    constexpr int U = NT == 1 ? 4 : 2;
    while (s + U <= s1) run(IntC<U>(), IntC<0>());
    while (s < s1) run(IntC<1>(), IntC<0>());
    if (F % 64 != 0 && wave == kDownWaves - 1) run(IntC<1>(), IntC<1>());
}

// The same with e4m3 weights, converted to bf16 (exact) in front of the matrix core; sw: the column tile's scales, one
// per 128 of K.  Lane group g holds K elements 16 g .. 16 g + 15 of a 64-wide half block in both operands.
template <int NT>
__device__ __forceinline__ void down_q8(const char *w, const uint32_t (&wo)[2], int kp, const char *h,
                                        const uint32_t (&ho)[NT], const float *sw, int F, int wave,
                                        f32x4_t (&acc)[NT])
{
    const int nb = F / kQ8Group;
    int b = nb * wave / kDownWaves;
    const int b1 = nb * (wave + 1) / kDownWaves;
    const int kh = 16 * (int)(threadIdx.x % kWave >> 4);
    auto run = [&](auto uc, auto partial) {
        constexpr int U = decltype(uc)::value;
        // PARTIAL: the last block, with F % 128 of K left; pieces past F are zeros on both sides
        constexpr bool PARTIAL = decltype(partial)::value != 0;
        const int left = PARTIAL ? F % kQ8Group : kQ8Group;
        const u32x4_t z = {0u, 0u, 0u, 0u};
        u32x4_t wv[U][2];
        float fw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                wv[u][i] = !PARTIAL || kp < left ? load_w(w, wo[i] + (uint32_t)(b + u) * kQ8Group) : z;
            fw[u] = sw[b + u];
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            u32x4_t hv[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    hv[u][i] = !PARTIAL || kh + 64 * (i / 2) < left
                                   ? load_x(h, ho[n] + (uint32_t)(b + u) * (2 * kQ8Group) + 128 * (i / 2) + 16 * (i & 1))
                                   : z;
            if (n == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u) swap_halves(wv[u][0], wv[u][1]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                f32x4_t p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const u32x4_t v = wv[u][i];
                    p = mfma_bf16(fp8_to_bf16(v.x, v.y), hv[u][2 * i], p);
                    p = mfma_bf16(fp8_to_bf16(v.z, v.w), hv[u][2 * i + 1], p);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[n][q] = __builtin_fmaf(p[q], fw[u], acc[n][q]);
            }
            if (NT >= 4) __builtin_amdgcn_sched_barrier(0);   // keeps later tiles' loads out of the registers
        }
        b += U;
    };
    constexpr int U = NT == 1 ? 2 : 1;
    while (b + U <= b1) run(IntC<U>(), IntC<0>());
    while (b < b1) run(IntC<1>(), IntC<0>());
    if (F % kQ8Group != 0 && wave == kDownWaves - 1) run(IntC<1>(), IntC<1>());
}

// Adds local expert e's part of output columns n0 .. n0 + 15 to the wave's sums ([T][16] in LDS).
template <bool Q8, int NT>
__device__ __forceinline__ void down_expert(const LayerArgs &a, const RowsLds &s, int e, int n0, int row0, int cnt,
                                            float *sum)
{
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int c = lane & 15, g = lane >> 4;
    f32x4_t acc[NT];
    uint32_t ho[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        acc[n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        ho[n] = (uint32_t)min(16 * n + c, cnt - 1) * (uint32_t)(2 * a.F) + (Q8 ? 32 : 16) * g;
    }
    const char *h = (const char *)(a.h + (size_t)row0 * a.F);
    const char *w = (const char *)a.w_dn + ((size_t)e * a.d + n0) * a.F * (Q8 ? 1 : 2);
    const int piece = g + 4 * (c >> 3);
    uint32_t wo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) wo[i] = (uint32_t)((8 * i + (c & 7)) * a.F) * (Q8 ? 1 : 2) + 16 * piece;
    if constexpr (Q8) {
        const int nf = (a.F + kQ8Group - 1) / kQ8Group;
        down_q8<NT>(w, wo, 16 * piece, h, ho, a.s_dn + ((size_t)e * (a.d / kQ8Group) + n0 / kQ8Group) * nf, a.F, wave, acc);
    } else {
        down_bf16<NT>(w, wo, 8 * piece, h, ho, a.F, wave, acc);
    }
    // tokens of an expert are distinct, so no two lanes add to one word
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (16 * n + c < cnt) {
            f32x4_t *p = (f32x4_t *)(sum + (int)s.tok[row0 + 16 * n + c] * 16 + 4 * g);
            f32x4_t v = *p;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += acc[n][q];
            *p = v;
        }
    }
}

template <bool Q8>
__global__ __launch_bounds__(64 * kDownWaves, 4) void k_layer_down(LayerArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    float *sums = (float *)lds;   // [kDownWaves][T][16]
    const RowsLds s = rows_lds(lds + (size_t)kDownWaves * a.T * 64, a, false);
    const int T = valid_tokens(a);
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    for (int i = threadIdx.x; i < T * a.k; i += blockDim.x) s.ids[i] = a.ids[i];
    __syncthreads();
    build_rows(s, a, T);
    const int hits = s.n[0];
    float *sum = sums + (size_t)wave * a.T * 16;
    for (int q = blockIdx.x; q < a.d / 16; q += gridDim.x) {
        const int n0 = 16 * q;
        for (int i = lane; i < T * 4; i += kWave) ((f32x4_t *)sum)[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        for (int hi = 0; hi < hits; ++hi) {
            const int e = __builtin_amdgcn_readfirstlane(s.hit[hi]);
            const int row0 = __builtin_amdgcn_readfirstlane(s.start[e]);
            const int cnt = __builtin_amdgcn_readfirstlane(__popcll(s.mask[2 * e]) + __popcll(s.mask[2 * e + 1]));
            if (cnt <= 16) down_expert<Q8, 1>(a, s, e, n0, row0, cnt, sum);
            else if (cnt <= 32) down_expert<Q8, 2>(a, s, e, n0, row0, cnt, sum);
            else if (cnt <= 64) down_expert<Q8, 4>(a, s, e, n0, row0, cnt, sum);
            else down_expert<Q8, 8>(a, s, e, n0, row0, cnt, sum);
        }
        __syncthreads();
        // two neighbouring columns per thread, waves in order
        for (int i = threadIdx.x; i < T * 8; i += blockDim.x) {
            const int t = i >> 3, n = 2 * (i & 7);
            float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
            for (int w = 0; w < kDownWaves; ++w) {
                const float *p = sums + ((size_t)w * a.T + t) * 16 + n;
                v0 += p[0];
                v1 += p[1];
            }
            *(uint32_t *)(a.out + (size_t)t * a.d + n0 + n) =
                (uint32_t)f32_to_bf16(v0) | (uint32_t)f32_to_bf16(v1) << 16;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- router of up to kLayerSelfT tokens

// Partial sums part[s][t][e] in the library's order (one ascending fma chain per K segment), on the vector units: with
// a few tokens the chains are few, and the time goes into fetching W_r.  A workgroup takes (segment s, 32 experts): all
// its weights are fetched at once into LDS (a segment of d = 7168 is 112 KiB), then lane l of wave w runs the chain of
// token 2 w + l / 32, expert l % 32.
constexpr int kVrThreads = 512;
constexpr int kVrExp = 32;
constexpr int kVrRows = 896;   // weight rows per staged chunk

__global__ __launch_bounds__(kVrThreads) void k_layer_router(LayerArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int seg = a.d / kRouterSegments;
    const int rows_lds_n = min(seg, kVrRows);
    float *ws = (float *)lds;                       // [rows][32]
    float *xs = ws + (size_t)rows_lds_n * kVrExp;   // [T][rows]
    const int s = (int)blockIdx.x % kRouterSegments, e0 = (int)blockIdx.x / kRouterSegments * kVrExp;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int t = 2 * wave + lane / 32, el = lane % 32;
    const bool mine = t < a.T && e0 + el < a.E;
    float acc = 0.0f;
    const bool full = a.E % 4 == 0 && e0 + kVrExp <= a.E;
    for (int r0 = 0; r0 < seg; r0 += kVrRows) {
        const int rows = min(kVrRows, seg - r0);   // a multiple of 16
        const float *w = a.wr + ((size_t)s * seg + r0) * a.E + e0;
        if (full) {
            for (int i = threadIdx.x; i < rows * 8; i += 8 * kVrThreads) {
                f32x4_t v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int j = min(i + u * kVrThreads, rows * 8 - 1);
                    v[u] = *(const f32x4_t *)(w + (size_t)(j >> 3) * a.E + 4 * (j & 7));
                }
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (i + u * kVrThreads < rows * 8) *(f32x4_t *)(ws + 4 * (i + u * kVrThreads)) = v[u];
            }
        } else {
            const int ne = min(kVrExp, a.E - e0);
            for (int i = threadIdx.x; i < rows * kVrExp; i += 8 * kVrThreads) {
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int j = min(i + u * kVrThreads, rows * kVrExp - 1);
                    v[u] = w[(size_t)(j >> 5) * a.E + min(j & 31, ne - 1)];
                }
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (i + u * kVrThreads < rows * kVrExp) ws[i + u * kVrThreads] = v[u];
            }
        }
        for (int i = threadIdx.x; i < a.T * rows / 8; i += kVrThreads) {
            const int tt = i / (rows / 8), c = i % (rows / 8);
            float f[8];
            unpack8(*(const u32x4_t *)(a.x + (size_t)tt * a.d + (size_t)s * seg + r0 + 8 * c), f);
            f32x4_t *p = (f32x4_t *)(xs + (size_t)tt * rows_lds_n + 8 * c);
            p[0] = f32x4_t{f[0], f[1], f[2], f[3]};
            p[1] = f32x4_t{f[4], f[5], f[6], f[7]};
        }
        __syncthreads();
        if (mine) {
            const float *xp = xs + (size_t)t * rows_lds_n, *wp = ws + el;
            for (int i = 0; i < rows; i += 16) {
#pragma unroll
                for (int u = 0; u < 16; ++u) acc = __builtin_fmaf(xp[i + u], wp[(i + u) * kVrExp], acc);
            }
        }
        __syncthreads();
    }
    if (mine) a.part[((size_t)s * a.T + t) * a.E + e0 + el] = acc;
}

size_t vr_lds_bytes(const LayerArgs &a)
{
    const size_t rows = std::min(a.d / kRouterSegments, kVrRows);
    return rows * kVrExp * 4 + (size_t)a.T * rows * 4;
}

int device_cus()
{
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
    return cus;
}

template <bool Q8, int R>
hipError_t launch_up(const LayerArgs &a, bool self, int grid, hipStream_t s)
{
    const size_t lds = 2 * kUpWaves * R * 256 * 4 + rows_lds_bytes(a.T, a.k, a.E_local, true);
    if constexpr (R == 1) {   // kLayerSelfT <= 16
        if (self) {
            hipLaunchKernelGGL((k_layer_up<Q8, 1, true>), dim3(grid), dim3(64 * kUpWaves), lds, s, a);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((k_layer_up<Q8, R, false>), dim3(grid), dim3(64 * kUpWaves), lds, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_router(const LayerArgs &a, hipStream_t s)
{
    const int grid = kRouterSegments * ((a.E + kVrExp - 1) / kVrExp);
    hipLaunchKernelGGL(k_layer_router, dim3(grid), dim3(kVrThreads), vr_lds_bytes(a), s, a);
    return hipGetLastError();
}

hipError_t launch_layer(const LayerArgs &a, bool q8, bool self, hipStream_t s)
{
    const int cus = device_cus();
    if (cus <= 0) return hipErrorInvalidDevice;
    const int R = a.T <= 16 ? 1 : 2;
    const long nf = (a.F + 8 * R - 1) / (8 * R);
    const long most = (long)std::min(a.E_local, a.T * a.k) * nf;   // tasks, if every choice is another local expert
    const int grid = (int)std::min<long>(most, 4L * cus);
    hipError_t e;
    if (q8) e = R == 1 ? launch_up<true, 1>(a, self, grid, s) : launch_up<true, 2>(a, self, grid, s);
    else e = R == 1 ? launch_up<false, 1>(a, self, grid, s) : launch_up<false, 2>(a, self, grid, s);
    if (e != hipSuccess) return e;
    LayerArgs b = a;
    if (self) b.ids = a.ids_ws;
    const size_t lds = (size_t)kDownWaves * a.T * 64 + rows_lds_bytes(a.T, a.k, a.E_local, false);
    const int gd = std::min(a.d / 16, 4 * cus);
    if (q8) hipLaunchKernelGGL(k_layer_down<true>, dim3(gd), dim3(64 * kDownWaves), lds, s, b);
    else hipLaunchKernelGGL(k_layer_down<false>, dim3(gd), dim3(64 * kDownWaves), lds, s, b);
    return hipGetLastError();
}

}  // namespace mk
