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

// Buffer resource of `bytes` from base (both uniform): a load is base + the lane's 32-bit offset + a scalar offset, with
// no address arithmetic in the vector registers, and a lane offset past the end reads zeros without a memory access.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, uint32_t bytes)
{
    const uint64_t b = (uint64_t)base;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)(((uint64_t)hi << 32) | lo), (short)0,
                                             (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

// load_w: weights, which no other workgroup reads (non-temporal); load_x: activations, which stay in the L2.
__device__ __forceinline__ u32x4_t load_w(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t soff)
{
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, 2));
}
__device__ __forceinline__ u32x4_t load_x(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t soff)
{
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, 0));
}
__device__ __forceinline__ float load_f32(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t soff)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, off, soff, 0));
}
// N consecutive floats (4-byte aligned) in one load.
template <int N>
__device__ __forceinline__ void load_floats(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t soff, float (&f)[N])
{
    static_assert(N == 1 || N == 2 || N == 4, "one load");
    if constexpr (N == 1) {
        f[0] = load_f32(r, off, soff);
    } else if constexpr (N == 2) {
        typedef uint32_t u32x2_v __attribute__((ext_vector_type(2)));
        const u32x2_v v = __builtin_bit_cast(u32x2_v, __builtin_amdgcn_raw_buffer_load_b64(r, off, soff, 0));
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
    } else {
        const u32x4_t v = load_x(r, off, soff);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
    }
}

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

// The tokens' operand comes in the same way: 8 tokens x 128 bytes per load, group i of 8 tokens in v[i], two neighbouring
// groups exchanged into the two halves of a 16-token tile.  A single group (8 tokens or fewer, the ordinary case of a
// decode step) needs no second load: its own lanes i >= 8 hold the other pieces, one rotation away, and what the
// columns past 8 get does not matter.  With 16 tokens x 64 bytes per load the loads of four tokens' rows slowed the
// weight stream by 5%.
template <int N8>
__device__ __forceinline__ void pair_tokens(u32x4_t (&v)[N8], u32x4_t (&first)[(N8 + 1) / 2],
                                            u32x4_t (&second)[(N8 + 1) / 2])
{
    if constexpr (N8 == 1) {
        first[0] = v[0];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            second[0][j] = (uint32_t)__builtin_amdgcn_update_dpp((int)v[0][j], (int)v[0][j], 0x128, 0xF, 0xF, false);
    } else {
#pragma unroll
        for (int n = 0; n < N8 / 2; ++n) {
            first[n] = v[2 * n];
            second[n] = v[2 * n + 1];
            swap_halves(first[n], second[n]);
        }
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

template <int N>
struct IntC {
    static constexpr int value = N;
};

constexpr int kUpWaves = 4;
constexpr int kUpRedBytes = 2 * kUpWaves * 2 * 256 * 4;   // two halves of up_task's exchange

// One gate|up task: features f0 .. f0 + 8 R - 1 of local expert e for its rows row0 .. row0 + cnt - 1 (cnt <= 8 N8).
// R = 1: one weight tile of 8 gate and 8 up rows; R = 2: a tile of 16 gate rows and one of 16 up rows.
// The wave sums its share of K in steps of 128 bytes of a weight row (64 bf16, or one 128-wide block of e4m3, whose
// product is scaled by the token's and the weights' scales before it joins the sum).
// red: 2 x kUpWaves x R x 256 floats; par: which half the next exchange uses.
template <bool Q8, int R, int N8>
__device__ __forceinline__ void up_task(const LayerArgs &a, const RowsLds &s, int e, int f0, int row0, int cnt,
                                        float *red, int &par)
{
    constexpr int NT = (N8 + 1) / 2;   // 16-column tiles
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int c = lane & 15, g = lane >> 4;
    const uint32_t pitch = (uint32_t)a.d * (Q8 ? 1 : 2);
    const int steps = (int)(pitch / 128), s0 = steps * wave / kUpWaves, s1 = steps * (wave + 1) / kUpWaves;
    const uint32_t wbytes = 2 * (uint32_t)a.F * pitch;
    const __amdgpu_buffer_rsrc_t w = buffer_of((const char *)a.w_gu + (size_t)e * wbytes, wbytes);
    const __amdgpu_buffer_rsrc_t x = buffer_of(Q8 ? (const void *)a.xq : (const void *)a.x, (uint32_t)a.T * pitch);
    // the lane's weight rows in each tile (features past F repeat the last; never stored)
    uint32_t wo[R][2], xo[N8], so[NT];
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
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) wo[r][i] = wo[r][i] * pitch + 16 * (g + 4 * (c >> 3));
    // the lane's token in each group of 8 (past cnt the last again; columns never stored)
#pragma unroll
    for (int n = 0; n < N8; ++n)
        xo[n] = s.tok[row0 + min(8 * n + (c & 7), cnt - 1)] * pitch + 16 * (g + 4 * (c >> 3));
    // 8-bit form: the scales of its column's token (a step is a block)
#pragma unroll
    for (int n = 0; n < NT; ++n) so[n] = Q8 ? s.tok[row0 + min(16 * n + c, cnt - 1)] * (uint32_t)steps * 4 : 0;
    f32x4_t acc[R][NT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    // 8-bit form: block scales of the wave's share, lane l holds block s0 + l of the gate and of the up rows (at most 64
    // blocks: d <= 32768 over four waves)
    int fg = 0, fu = 0;
    if (Q8) {
        const int nf = (a.F + kQ8Group - 1) / kQ8Group;
        const float *sg = a.s_gu + ((size_t)e * 2 * nf + f0 / kQ8Group) * steps + min(s0 + lane, steps - 1);
        fg = __float_as_int(sg[0]);
        fu = __float_as_int(sg[(size_t)nf * steps]);
    }
    const __amdgpu_buffer_rsrc_t sx = buffer_of(a.xs, (uint32_t)a.T * steps * 4);
    int k = s0;
    // U steps: all their loads, then all their products.  (Four workgroups a CU cover each other's waits; a ring of
    // single steps per wave measured no faster.)
    auto run = [&](auto uc) {
        constexpr int U = decltype(uc)::value;
        u32x4_t wv[U][R][2], xv[U][N8];
        float fx[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) wv[u][r][i] = load_w(w, wo[r][i] + 128 * u, k * 128);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int n = 0; n < N8; ++n) xv[u][n] = load_x(x, xo[n] + 128 * u, k * 128);
        if constexpr (Q8) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float f[U];
                load_floats<U>(sx, so[n], k * 4, f);
#pragma unroll
                for (int u = 0; u < U; ++u) fx[u][n] = f[u];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int r = 0; r < R; ++r) swap_halves(wv[u][r][0], wv[u][r][1]);
            u32x4_t x0[NT], x1[NT];
            pair_tokens<N8>(xv[u], x0, x1);
            if constexpr (Q8) {
                const float wg = __int_as_float(__builtin_amdgcn_readlane(fg, k - s0 + u));
                const float wu = __int_as_float(__builtin_amdgcn_readlane(fu, k - s0 + u));
                // accumulator rows 4 g .. 4 g + 3: in the mixed tile groups 0, 1 are gate rows and 2, 3 up rows
                const float fw[2] = {R == 1 ? (g < 2 ? wg : wu) : wg, wu};
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        f32x4_t p = {0.0f, 0.0f, 0.0f, 0.0f};
                        p = mfma_fp8_64(wv[u][r][0], x0[n], p);
                        p = mfma_fp8_64(wv[u][r][1], x1[n], p);
                        const float f = fw[r] * fx[u][n];
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[r][n][v] = __builtin_fmaf(p[v], f, acc[r][n][v]);
                    }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int r = 0; r < R; ++r) acc[r][n] = mfma_bf16(wv[u][r][i], i == 0 ? x0[n] : x1[n], acc[r][n]);
            }
        }
        k += U;
    };
    constexpr int U = R == 1 ? 4 : N8 == 8 ? 1 : 2;
    while (k + U <= s1) run(IntC<U>());
    while (k < s1) run(IntC<1>());
    // The waves' parts of a token tile meet in LDS ([column][row], so a lane's four rows are one 16-byte word), are
    // added in wave order, and become h, two features a thread.  Halves alternate: one barrier per tile.
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float *rb = red + par * kUpWaves * R * 256;
        par ^= 1;
#pragma unroll
        for (int r = 0; r < R; ++r) *(f32x4_t *)(rb + (wave * R + r) * 256 + c * 16 + 4 * g) = acc[r][n];
        __syncthreads();
        const int fi = 2 * ((int)threadIdx.x % (4 * R)), ci = (int)threadIdx.x / (4 * R);
        const int row = 16 * n + ci;
        if (ci < 16 && row < cnt && f0 + fi < a.F) {
            float2 gs = make_float2(0.0f, 0.0f), us = gs;
#pragma unroll
            for (int v = 0; v < kUpWaves; ++v) {
                const float *q = rb + v * R * 256 + ci * 16 + fi;
                const float2 gv = *(const float2 *)q, uv = *(const float2 *)(q + (R == 1 ? 8 : 256));
                gs.x += gv.x;
                gs.y += gv.y;
                us.x += uv.x;
                us.y += uv.y;
            }
            const float gate = s.gate[row0 + row];
            const float h0 = gs.x / (1.0f + expf(-gs.x)) * us.x * gate;
            const float h1 = gs.y / (1.0f + expf(-gs.y)) * us.y * gate;
            *(uint32_t *)(a.h + (size_t)(row0 + row) * a.F + f0 + fi) =
                (uint32_t)f32_to_bf16(h0) | (uint32_t)f32_to_bf16(h1) << 16;
        }
    }
}

// SELF: the workgroup selects the experts of the few tokens itself from the router's partial sums.
template <bool Q8, bool SELF>
__global__ __launch_bounds__(64 * kUpWaves, 4) void k_layer_up(LayerArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    float *red = (float *)lds;
    const RowsLds s = rows_lds(lds + kUpRedBytes, a, true);
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
    // Tasks of 16 features, two weight tiles beside one load of the tokens.  Where they are too few to give every CU a
    // couple (a token or two at a few experts), of 8.
    const int hits = s.n[0];
    const bool small = a.T <= 16 && (long)hits * ((a.F + 15) / 16) < a.few_tasks;
    const int fs = small ? 8 : 16;
    const int nf = (a.F + fs - 1) / fs;
    int par = 0;
    for (int q = blockIdx.x; q < hits * nf; q += gridDim.x) {
        const int hi = q / nf, f0 = (q - hi * nf) * fs;
        const int e = __builtin_amdgcn_readfirstlane(s.hit[hi]);
        const int row0 = __builtin_amdgcn_readfirstlane(s.start[e]);
        const int cnt = __builtin_amdgcn_readfirstlane(__popcll(s.mask[2 * e]) + __popcll(s.mask[2 * e + 1]));
        if (small) {
            if (cnt <= 8) up_task<Q8, 1, 1>(a, s, e, f0, row0, cnt, red, par);
            else up_task<Q8, 1, 2>(a, s, e, f0, row0, cnt, red, par);
            continue;
        }
        // up to 64 rows at once; an expert of more than 64 rows reads its weights again for the rest
        for (int r = 0; r < cnt; r += 64) {
            const int m = min(cnt - r, 64);
            if (m <= 8) up_task<Q8, 2, 1>(a, s, e, f0, row0 + r, m, red, par);
            else if (m <= 16) up_task<Q8, 2, 2>(a, s, e, f0, row0 + r, m, red, par);
            else if (m <= 32) up_task<Q8, 2, 4>(a, s, e, f0, row0 + r, m, red, par);
            else up_task<Q8, 2, 8>(a, s, e, f0, row0 + r, m, red, par);
        }
    }
}

// ---------------------------------------------------------------- down

// Steps of a stream held in registers: the loads of step s + D are issued as soon as step s has been used, so D steps
// are always on their way.  total: the steps; load(slot): the next step's loads; use(slot): the oldest step's products.
// The order is pinned, and the loop without conditions covers all but the last 2 D - 1 steps.
template <int D, class Slot, class Load, class Use>
__device__ __forceinline__ void stream(int total, Load &&load, Use &&use)
{
    Slot ring[D];
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (j < total) load(ring[j]);
    int i = 0;
    for (; i + 2 * D <= total; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            use(ring[j]);
            __builtin_amdgcn_sched_barrier(0);
            load(ring[j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int j = 0; j < D; ++j) {
        if (i + j < total) use(ring[j]);
        if (i + j + D < total) load(ring[j]);
    }
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (i + D + j < total) use(ring[j]);
}

// Registers a step takes decide how many are in flight: about 72 of the 128 a wave has.
constexpr int ring_depth(int regs) { return regs <= 18 ? 4 : regs <= 26 ? 3 : regs <= 36 ? 2 : 1; }

constexpr int kDownWaves = 8;

// Groups of 8 tokens that an expert's rows are taken in (more than 64 rows: several times 8 groups).
__device__ __forceinline__ int groups_of(int cnt) { return cnt <= 8 ? 1 : cnt <= 16 ? 2 : cnt <= 32 ? 4 : 8; }

// Adds the parts of the hit experts h0 .. h1 - 1 (all taken in N8 groups of 8 tokens) to the wave's sums of output columns
// n0 .. n0 + 15 ([T][16] in LDS): one stream of steps through all of them, over the wave's share of K of each.  A step is
// 128 bytes of a weight row: 64 of K, or 128 of K in e4m3, converted to bf16 (exact) in front of the matrix core.
// TAIL: F does not end on a step; pieces past F are zeros on both sides.
template <bool Q8, int N8, bool TAIL>
__device__ __forceinline__ void down_run(const LayerArgs &a, const RowsLds &s, int h0, int h1, int n0, float *sum)
{
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int c = lane & 15, g = lane >> 4;
    constexpr int NT = (N8 + 1) / 2;             // 16-column tiles
    constexpr int KS = Q8 ? kQ8Group : 64;       // K per step
    constexpr int KP = Q8 ? 16 : 8;              // K per 16-byte piece of a weight row
    constexpr int kBytes = Q8 ? 1 : 2;
    constexpr int HL = Q8 ? 2 : 1;               // 128-byte lines of an h row per step
    const int steps = (a.F + KS - 1) / KS, mine = (steps - wave + kDownWaves - 1) / kDownWaves;
    if (mine <= 0) return;
    const int kp = KP * (g + 4 * (c >> 3));      // the lane's piece of a weight row (swap_halves)
    // ... and of an h line (pair_tokens), 8 elements: bf16 pieces g and 4 + g, as the weights; e4m3, whose 16-byte piece
    // is two pieces of h, 2 g and 2 g + 1
    const int kh = 8 * (Q8 ? 2 * g + (c >> 3) : g + 4 * (c >> 3));
    uint32_t wo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) wo[i] = (uint32_t)((8 * i + (c & 7)) * a.F + kp) * kBytes;
    struct Slot {
        u32x4_t w[2], h[HL][N8];
        float fw;
    };
    // the loading end: hit expert lh, rows lr .. of it, step ls
    int lh = h0, lr = 0, ls = wave, lcnt = 0;
    __amdgpu_buffer_rsrc_t lw, lhp, lsw;
    uint32_t lo[N8];
    int total = 0;
    auto expert_at = [&](int hi, int &e, int &row0, int &cnt) {
        e = __builtin_amdgcn_readfirstlane(s.hit[hi]);
        row0 = __builtin_amdgcn_readfirstlane(s.start[e]);
        cnt = __builtin_amdgcn_readfirstlane(__popcll(s.mask[2 * e]) + __popcll(s.mask[2 * e + 1]));
    };
    auto load_setup = [&]() {
        int e, row0;
        expert_at(lh, e, row0, lcnt);
        lw = buffer_of((const char *)a.w_dn + ((size_t)e * a.d + n0) * a.F * kBytes, 16 * (uint32_t)a.F * kBytes);
        lhp = buffer_of(a.h + (size_t)row0 * a.F, (uint32_t)lcnt * 2 * a.F);
        if (Q8) lsw = buffer_of(a.s_dn + ((size_t)e * (a.d / kQ8Group) + n0 / kQ8Group) * steps, steps * 4);
#pragma unroll
        for (int n = 0; n < N8; ++n)
            lo[n] = (uint32_t)(min(lr + 8 * n + (c & 7), lcnt - 1) * a.F + kh) * 2;
    };
    // the using end
    int uh = h0, ur = 0, us = 0;
    f32x4_t acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int hi = h0; hi < h1; ++hi) {
        int e, row0, cnt;
        expert_at(hi, e, row0, cnt);
        total += (cnt + 8 * N8 - 1) / (8 * N8);
    }
    total *= mine;
    load_setup();
    stream<ring_depth(8 + 4 * HL * N8), Slot>(
        total,
        [&](Slot &q) {
            const uint32_t kw = (uint32_t)ls * 128;
            const int left = a.F - ls * KS;
#pragma unroll
            for (int i = 0; i < 2; ++i) q.w[i] = load_w(lw, !TAIL || kp < left ? wo[i] : kPastResource, kw);
#pragma unroll
            for (int l = 0; l < HL; ++l)
#pragma unroll
                for (int n = 0; n < N8; ++n)
                    q.h[l][n] = load_x(lhp, !TAIL || kh + 64 * l < left ? lo[n] + 128 * l : kPastResource, kw * HL);
            if (Q8) q.fw = load_f32(lsw, 0, ls * 4);
            if ((ls += kDownWaves) >= steps) {
                ls = wave;
                lr += 8 * N8;
                if (lr >= lcnt) {
                    lr = 0;
                    ++lh;
                }
                if (lh < h1) load_setup();
            }
        },
        [&](Slot &q) {
            swap_halves(q.w[0], q.w[1]);
            u32x4_t x[HL][2][NT];
#pragma unroll
            for (int l = 0; l < HL; ++l) pair_tokens<N8>(q.h[l], x[l][0], x[l][1]);
            if constexpr (Q8) {
                u32x4_t b[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    b[2 * i] = fp8_to_bf16(q.w[i].x, q.w[i].y);
                    b[2 * i + 1] = fp8_to_bf16(q.w[i].z, q.w[i].w);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    f32x4_t p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < 4; ++i) p = mfma_bf16(b[i], x[HL - 1 & i / 2][i & 1][n], p);
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[n][v] = __builtin_fmaf(p[v], q.fw, acc[n][v]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[n] = mfma_bf16(q.w[i], x[0][i][n], acc[n]);
            }
            if (++us == mine) {
                us = 0;
                int e, row0, cnt;
                expert_at(uh, e, row0, cnt);
                // tokens of an expert are distinct, so no two lanes add to one word
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int row = ur + 16 * n + c;
                    if (row < cnt) {
                        f32x4_t *p = (f32x4_t *)(sum + (int)s.tok[row0 + row] * 16 + 4 * g);
                        f32x4_t v = *p;
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] += acc[n][j];
                        *p = v;
                    }
                    acc[n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
                }
                ur += 8 * N8;
                if (ur >= cnt) {
                    ur = 0;
                    ++uh;
                }
            }
        });
}

template <bool Q8, bool TAIL>
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
        // runs of experts that take the same number of token groups, in expert order
        for (int h0 = 0; h0 < hits;) {
            auto groups = [&](int hi) {
                const int e = s.hit[hi];
                return __builtin_amdgcn_readfirstlane(groups_of(__popcll(s.mask[2 * e]) + __popcll(s.mask[2 * e + 1])));
            };
            const int n8 = groups(h0);
            int h1 = h0 + 1;
            while (h1 < hits && groups(h1) == n8) ++h1;
            if (n8 == 1) down_run<Q8, 1, TAIL>(a, s, h0, h1, n0, sum);
            else if (n8 == 2) down_run<Q8, 2, TAIL>(a, s, h0, h1, n0, sum);
            else if (n8 == 4) down_run<Q8, 4, TAIL>(a, s, h0, h1, n0, sum);
            else down_run<Q8, 8, TAIL>(a, s, h0, h1, n0, sum);
            h0 = h1;
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

template <bool Q8>
hipError_t launch_up(const LayerArgs &a, bool self, int grid, hipStream_t s)
{
    const size_t lds = kUpRedBytes + rows_lds_bytes(a.T, a.k, a.E_local, true);
    if (self) hipLaunchKernelGGL((k_layer_up<Q8, true>), dim3(grid), dim3(64 * kUpWaves), lds, s, a);
    else hipLaunchKernelGGL((k_layer_up<Q8, false>), dim3(grid), dim3(64 * kUpWaves), lds, s, a);
    return hipGetLastError();
}

template <bool Q8, bool TAIL>
hipError_t launch_down(const LayerArgs &a, int grid, size_t lds, hipStream_t s)
{
    hipLaunchKernelGGL((k_layer_down<Q8, TAIL>), dim3(grid), dim3(64 * kDownWaves), lds, s, a);
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
    LayerArgs b = a;
    b.few_tasks = 2 * cus;
    const long most = (long)std::min(a.E_local, a.T * a.k) * ((a.F + 7) / 8);   // tasks, if every choice is another local expert
    const int grid = (int)std::min<long>(most, 4L * cus);
    const hipError_t e = q8 ? launch_up<true>(b, self, grid, s) : launch_up<false>(b, self, grid, s);
    if (e != hipSuccess) return e;
    if (self) b.ids = a.ids_ws;
    const size_t lds = (size_t)kDownWaves * a.T * 64 + rows_lds_bytes(a.T, a.k, a.E_local, false);
    const int gd = std::min(a.d / 16, 4 * cus);
    const bool tail = a.F % (q8 ? kQ8Group : 64) != 0;
    if (q8 && tail) return launch_down<true, true>(b, gd, lds, s);
    if (q8) return launch_down<true, false>(b, gd, lds, s);
    return tail ? launch_down<false, true>(b, gd, lds, s) : launch_down<false, false>(b, gd, lds, s);
}

}  // namespace mk
