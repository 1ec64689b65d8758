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
//   - few waves with many registers each: a wave's loads of the next steps are
//     all on their way before it multiplies (two workgroups of four waves per CU
//     stream the weights as fast as four of them, with a quarter of the
//     instructions' register pressure).
// Launches: the router and the selection (unless the caller routed; for a few
// tokens the up kernel selects by itself), "up", which writes h = w * silu(g) * u,
// "down", which writes W_down[e] . h per row in fp32 and for few tokens adds each
// token's rows up in expert order, and "sum", which does that for more.
//
// Bound by memory; a kernel that only reads reaches 7.0 - 7.1 TB/s here.  Kernel times, bf16 / e4m3:
//   128 tokens, 32 of 256 experts, d = 7168, F = 2048:   router 18.7, selection 4.8, up 288 / 148 (6.5 / 6.3 TB/s), down
//                                                        148 / 79 (6.3 / 6.0), sum 4.9 us
//   1 token, 2 of 8 experts, d = 4096, F = 14336, bf16:  router 6.0, up 74 (6.4 TB/s), down with the sum 39 us
//   64 tokens, 2 of 8 experts, same sizes (16 rows each): up 301 / 168, down 158 / 88 us
//   128 tokens (32 rows each):                           up 354 / 211, down 221 / 168 us
// With 32 rows an expert the tokens' and h's loads weigh as much as the weights', and a wave's loads and products no
// longer overlap as well.
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
    LayerRec *rec;      // [<= min(E_local, T k)] the experts with rows
    int32_t *n;         // [1] how many
    uint64_t *mask;     // [E_local][2] (build_rows)
    int32_t *start;     // [E_local] first row of the expert (build_rows)
    uint8_t *tok;       // [T min(k, E_local)]
    float *gate;        // [T min(k, E_local)]
    int32_t *ids;       // [T k]
    float *w;           // [T k]
};

__host__ __device__ inline size_t rows_lds_bytes(int T, int k, int E_local)
{
    const size_t r = (size_t)layer_rows_cap(T, k, E_local), tk = (size_t)T * k;
    const size_t b = (size_t)layer_hits_cap(T, k, E_local) * 16 + 16 + (size_t)E_local * 20 + (2 * tk + r) * 4 + r;
    return (b + 15) & ~(size_t)15;
}

__device__ __forceinline__ RowsLds rows_lds(char *p, const LayerArgs &a)
{
    const int r = layer_rows_cap(a.T, a.k, a.E_local), tk = a.T * a.k;
    RowsLds s;
    s.rec = (LayerRec *)p;
    p += (size_t)layer_hits_cap(a.T, a.k, a.E_local) * 16;
    s.n = (int32_t *)p;
    p += 16;
    s.mask = (uint64_t *)p;
    p += (size_t)a.E_local * 16;
    s.start = (int32_t *)p;
    p += (size_t)a.E_local * 4;
    s.ids = (int32_t *)p;
    p += (size_t)tk * 4;
    s.w = (float *)p;
    p += (size_t)tk * 4;
    s.gate = (float *)p;
    p += (size_t)r * 4;
    s.tok = (uint8_t *)p;
    return s;
}

// Rows of expert e below token t.
__device__ __forceinline__ int rank_of(const uint64_t *m, int t)
{
    return t < 64 ? __popcll(m[0] & ((1ull << t) - 1)) : __popcll(m[0]) + __popcll(m[1] & ((1ull << (t - 64)) - 1));
}

// build_rows for a few choices, by one wave without the masks, a lane per choice: a row's number is the number of choices
// that come before it by (expert, token).
__device__ __forceinline__ void build_few_rows(const RowsLds &s, const LayerArgs &a, int T, bool publish)
{
    const int l = threadIdx.x, n = T * a.k;
    const int t = l / a.k;
    int e = l < n ? s.ids[l] - a.e_begin : -1;
    float w = l < n ? s.w[l] : 0.0f;
    if (e < 0 || e >= a.E_local) e = -1;
    if (a.given) {   // an id given more than once for a token: one row, the gates added up one by one as in build_rows
        bool again = false;
        const int own = __float_as_int(w);
        for (int j = 0; j < n; ++j) {
            const int ej = __builtin_amdgcn_readlane(e, j);
            const float wj = __int_as_float(__builtin_amdgcn_readlane(own, j));
            const bool same = ej == e && j / a.k == t;
            again |= same && j < l;
            w += same && j > l ? wj : 0.0f;
        }
        if (again) e = -1;
    }
    int row = 0, cnt = 0, hi = 0;
    bool first = e >= 0;
    for (int j = 0; j < n; ++j) {
        const int ej = __builtin_amdgcn_readlane(e, j);
        if (ej < 0) continue;   // uniform
        row += ej < e || (ej == e && j < l);
        cnt += ej == e;
        first &= !(ej == e && j < l);
    }
    const uint64_t firsts = __ballot(first);
    for (uint64_t m = firsts; m; m &= m - 1) hi += __builtin_amdgcn_readlane(e, __ffsll((unsigned long long)m) - 1) < e;
    if (e >= 0) {
        s.tok[row] = (uint8_t)t;
        s.gate[row] = w;
        if (first) {
            s.rec[hi] = LayerRec{e, row, cnt, 0};
            if (publish) a.plan.rec[hi] = LayerRec{e, row, cnt, 0};
        }
    }
    if (publish && l < a.T * a.k) a.plan.row_of[l] = e >= 0 ? row : -1;
    if (l == 0) {
        s.n[0] = __popcll(firsts);
        if (publish) {
            a.plan.n[0] = __popcll(firsts);
            a.plan.n[1] = T;
        }
    }
}

// Builds the rows from s.ids and s.w, which the caller has filled for tokens < T; ends with a barrier.  publish: this
// workgroup also writes what the later kernels need.
__device__ __forceinline__ void build_rows(const RowsLds &s, const LayerArgs &a, int T, bool publish)
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
            const int hi = hits + __popcll(b & lanemask_lt()), row0 = rows + incl - cnt;
            if (e < a.E_local) s.start[e] = row0;
            if (cnt > 0) {
                s.rec[hi] = LayerRec{e, row0, cnt, 0};
                if (publish) a.plan.rec[hi] = LayerRec{e, row0, cnt, 0};
            }
            rows += __shfl(incl, kWave - 1);
            hits += __popcll(b);
        }
        if (l == 0) {
            s.n[0] = hits;
            if (publish) {
                a.plan.n[0] = hits;
                a.plan.n[1] = T;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * a.k; i += blockDim.x) {
        const int t = i / a.k, id = s.ids[i], e = id - a.e_begin;
        int r = -1;
        if (e >= 0 && e < a.E_local) {
            bool first = true;
            float w = s.w[i];
            if (a.given) {   // an id given more than once for a token: one row, the gates added up in their order
                for (int j = t * a.k; j < i; ++j) first &= s.ids[j] != id;
                for (int j = i + 1; j < (t + 1) * a.k; ++j) w += s.ids[j] == id ? s.w[j] : 0.0f;
            }
            if (first) {
                r = s.start[e] + rank_of(s.mask + 2 * e, t);
                s.tok[r] = (uint8_t)t;
                s.gate[r] = w;
            }
        }
        if (publish) a.plan.row_of[i] = r;
    }
    if (publish)   // tokens past the valid ones have no rows
        for (int i = T * a.k + (int)threadIdx.x; i < a.T * a.k; i += blockDim.x) a.plan.row_of[i] = -1;
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
__device__ __forceinline__ uint32_t load_u32(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t soff)
{
    return __builtin_amdgcn_raw_buffer_load_b32(r, off, soff, 0);
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
// over 2 GiB, rows 14336 bytes apart: 5.5 against 7.1 TB/s).  Neighbouring lanes take neighbouring 16-byte pieces, since
// the address unit takes a cycle per lane otherwise (out of the L2: 9.7 TB/s, 19 with pairs, 30 with fours, which would
// need a second exchange): lane i + 16 g of load a (even rows) and of load b (odd rows) takes row i - i % 2 (+ 1), piece
// 2 g + i % 2.  Exchanging a's odd lanes with b's even ones leaves the matrix core's layout, lane i + 16 g = row i: piece
// 2 g in a, piece 2 g + 1 in b.
constexpr int kDppPairs = 0xB1;   // quad_perm:[1,0,3,2]
__device__ __forceinline__ uint32_t neighbour(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kDppPairs, 0xF, 0xF, true);
}
__device__ __forceinline__ void swap_pairs(u32x4_t &a, u32x4_t &b)
{
    const bool odd = threadIdx.x & 1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t x = a[j], y = b[j], nx = neighbour(x), ny = neighbour(y);
        a[j] = odd ? ny : x;
        b[j] = odd ? y : nx;
    }
}

// The tokens' operand comes in the same way: 8 tokens x 128 bytes per load; two neighbouring loads v[2 n], v[2 n + 1] take
// the even and the odd tokens of a 16-token tile and are exchanged.  A single group (8 tokens or fewer, the ordinary case
// of a decode step) needs no second load: token i takes column 2 i, whose lane's neighbour holds the other piece, and what
// the odd columns get does not matter.
template <int N8>
__device__ __forceinline__ int token_of(int n, int c)   // of group n, in the lane of column c
{
    return N8 == 1 ? c >> 1 : 8 * (n & ~1) + (c & 14) + (n & 1);
}
template <int N8>
__device__ __forceinline__ int column_of(int token)   // in the tile of its 16 tokens
{
    return N8 == 1 ? 2 * token : token & 15;
}
template <int N8>
__device__ __forceinline__ void pair_tokens(u32x4_t (&v)[N8], u32x4_t (&first)[(N8 + 1) / 2],
                                            u32x4_t (&second)[(N8 + 1) / 2])
{
    if constexpr (N8 == 1) {
        first[0] = v[0];
#pragma unroll
        for (int j = 0; j < 4; ++j) second[0][j] = neighbour(v[0][j]);
    } else {
#pragma unroll
        for (int n = 0; n < N8 / 2; ++n) {
            first[n] = v[2 * n];
            second[n] = v[2 * n + 1];
            swap_pairs(first[n], second[n]);
        }
    }
}

__device__ __forceinline__ f32x4_t mfma_bf16(u32x4_t a, u32x4_t b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}
// One K = 128 product of e4m3 operands: bytes 0 - 15 of both in a0, b0 and 16 - 31 in a1, b1, the same K in the same place
// of both.  The block scales are powers of two (exponent + 127 in every byte): 1.
__device__ __forceinline__ f32x4_t mfma_fp8(u32x4_t a0, u32x4_t a1, u32x4_t b0, u32x4_t b1, f32x4_t c)
{
    typedef int i32x8_v __attribute__((ext_vector_type(8)));
    const i32x8_v a = {(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
    const i32x8_v b = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
}

typedef _Float16 f16x2_v __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_v __attribute__((ext_vector_type(8)));
__device__ __forceinline__ f32x4_t mfma_f16(u32x4_t a, u32x4_t b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_v, a), __builtin_bit_cast(f16x8_v, b), c, 0, 0,
                                                  0);
}

// Eight e4m3 codes as fp16 (exact).
__device__ __forceinline__ u32x4_t fp8_to_f16(uint32_t lo, uint32_t hi)
{
    u32x4_t o;
    o.x = __builtin_bit_cast(uint32_t, (f16x2_v)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
    o.y = __builtin_bit_cast(uint32_t, (f16x2_v)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
    o.z = __builtin_bit_cast(uint32_t, (f16x2_v)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
    o.w = __builtin_bit_cast(uint32_t, (f16x2_v)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
    return o;
}

// The four groups of h in a lane, from their own binades (x4: a byte each) to the largest of the column's 16 (its four
// lanes'), which is returned.
__device__ __forceinline__ int align_groups(uint32_t x4, u32x4_t (&v)[4])
{
    int x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (x4 >> 8 * i) & 0xFF;
    int m = max(max(x[0], x[1]), max(x[2], x[3]));
    const auto far = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    m = max((int)far[0], (int)far[1]);
    const auto near = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max((int)near[0], (int)near[1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f = __builtin_amdgcn_ldexpf(1.0f, x[i] - m);   // below 2^-24: 0, and so is then h beside the largest
        const f16x2_v s = __builtin_bit_cast(f16x2_v, __builtin_amdgcn_cvt_pkrtz(f, f));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = v[i][j];
            v[i][j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_v, w) * s);
        }
    }
    return m;
}

// ---------------------------------------------------------------- gate|up
//
// A workgroup takes tasks of (expert, 8 to 32 features) in a fixed stride: tickets from an atomic counter measured slower
// (309 -> 320 us at 128 tokens), and so did each XCD working on experts of its own where their row counts differ (128 tokens
// at 64 experts with a skewed router: up 72 -> 141 us), without a gain where they do not.  Its four waves split K, so that
// a slab of 16 weight rows by 1/4 of K is one wave's, and their sums meet once per task in LDS.

template <int N>
struct IntC {
    static constexpr int value = N;
};

// Weight tiles per task.  More of them share one load of the tokens' rows, which cost as much as the weights once an
// expert has 16 rows or more; fewer make more tasks, which come out more even.  n1: tasks per expert at one tile.  Four
// tiles where the workgroups get at least four tasks each or come out nearly even (8 experts of 32 rows: up 352 us, with
// two tiles 405).  One tile (built for 16 tokens at most) where that gives a workgroup `few` tasks or fewer: up, few = 4
// (1 expert of 2048 features, d = 7168: 15 us, with two tiles 23), and down, whose tasks are shorter, few = 1 (6 experts
// of e4m3, d = 2048, 768 tasks of one tile for 512 workgroups: the whole call 28.6 us, with two tiles 25.6).
__device__ __forceinline__ int tiles_per_task(int hits, int n1, int T, int workgroups, int few)
{
    const long t4 = (long)hits * ((n1 + 3) / 4);
    const long rounds = (t4 + workgroups - 1) / workgroups;
    if (t4 >= 4L * workgroups || (t4 > 0 && 10 * t4 >= 9 * rounds * workgroups)) return 4;
    return (long)hits * n1 <= (long)few * workgroups && T <= 16 ? 1 : 2;
}

// h keeps more bits than the output, so that its rounding does not show beside the output's own (one bf16 made the layer's
// error 1.4 times a single rounding's), whatever the size of gates and activations.
// With bf16 weights it is in two parts: hi = bf16(h) and bf16(h - hi), leaving 2^-16 |h|; a rest that is not finite is left
// out.  A row: the first part, then the second.
// With 8-bit weights it is one fp16 value, 2^(14 - x) h, where 2^x is the binade of the largest of its 8 features, leaving
// 2^-11 |h| (or 2^-39 of the eight's largest); e4m3 weights are exact in fp16, so the product takes both as they are.  Eight
// features to a binade, because a task may have no more.  x + 127 is a byte of hx, 16 per block of 128 features.  The
// 16-byte pieces of every 128 values are stored as pieces 0 1 4 5 8 9 12 13, 2 3 6 7 10 11 14 15, so that the lane of weight
// piece 2 g, 2 g + 1 (elements 32 g .. 32 g + 31) finds its four in two loads of whole cache lines.
constexpr uint32_t kTopBinade = 14;                // of a stored fp16
constexpr uint32_t kLeastBinade = 27;              // 2^-100: smaller values count as that binade's

template <bool Q8>
__device__ __forceinline__ void store_h(const LayerArgs &a, int row, int f, float h0, float h1)
{
    char *p = (char *)a.h + (size_t)row * layer_h_row_bytes(Q8, a.F);
    if constexpr (Q8) {
        typedef float f32x2_t __attribute__((ext_vector_type(2)));
        typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
        // the 8 features are four neighbouring threads'
        uint32_t m = max(__float_as_uint(h0) & 0x7FFFFFFFu, __float_as_uint(h1) & 0x7FFFFFFFu);
        m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, kDppXor1, 0xF, 0xF, true));
        m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, kDppXor2, 0xF, 0xF, true));
        const uint32_t x = max(m >> 23, kLeastBinade);
        const float scale = __uint_as_float((254 + kTopBinade - x) << 23);
        const int at = (f & ~0x78) | (f & 8) | (f & 0x10) << 2 | (f & 0x60) >> 1;
        *(f16x2_t *)(p + 2 * at) = __builtin_convertvector((f32x2_t){h0 * scale, h1 * scale}, f16x2_t);
        if (f % kHGroup == 0) a.hx[(size_t)row * layer_hx_row_bytes(a.F) + f / kHGroup] = (uint8_t)x;
    } else {
        const uint32_t b0 = f32_to_bf16(h0), b1 = f32_to_bf16(h1);
        float r0 = h0 - bf16_to_f32(b0), r1 = h1 - bf16_to_f32(b1);
        r0 = fabsf(r0) < __builtin_inff() ? r0 : 0.0f;
        r1 = fabsf(r1) < __builtin_inff() ? r1 : 0.0f;
        *(uint32_t *)(p + 2 * f) = b0 | b1 << 16;
        *(uint32_t *)(p + 2 * (a.F + f)) = (uint32_t)f32_to_bf16(r0) | (uint32_t)f32_to_bf16(r1) << 16;
    }
}

constexpr int kUpWaves = kLayerWaves;

// One gate|up task: features f0 .. f0 + 8 R - 1 of local expert e for its rows row0 .. row0 + cnt - 1 (cnt <= 8 N8).
// R = 1: one weight tile of 8 gate and 8 up rows; R = 2 or 4: R / 2 tiles of 16 gate rows, then as many of up rows.
// The wave sums its share of K in steps of 128 bytes of a weight row (64 bf16, or one 128-wide block of e4m3, whose
// product is scaled by the token's and the weights' scales before it joins the sum).
// red: kExchangeBytes; par: which half the next exchange uses.
template <bool Q8, int R, int N8>
__device__ __forceinline__ void up_task(const LayerArgs &a, const RowsLds &s, int e, int f0, int row0, int cnt,
                                        float *red, int &par)
{
    constexpr int NT = (N8 + 1) / 2;   // 16-column tiles
    constexpr int NS = N8 < 4 ? N8 : 4, NST = (NS + 1) / 2;   // row groups (tiles) whose x is in registers at a time
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int c = lane & 15, g = lane >> 4;
    const uint32_t pitch = (uint32_t)a.d * (Q8 ? 1 : 2), piece = 16 * (2 * g + (c & 1));
    const int steps = (int)(pitch / 128), s0 = steps * wave / kUpWaves, s1 = steps * (wave + 1) / kUpWaves;
    const uint32_t wbytes = 2 * (uint32_t)a.F * pitch;
    const __amdgpu_buffer_rsrc_t w = buffer_of((const char *)a.w_gu + (size_t)e * wbytes, wbytes);
    const __amdgpu_buffer_rsrc_t x = buffer_of(Q8 ? (const void *)a.xq : (const void *)a.x, (uint32_t)a.T * pitch);
    // the lane's weight rows in each tile (features past F repeat the last; never stored)
    uint32_t wo[R][2], xo[N8], so[NT];
    if constexpr (R == 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) wo[0][i] = f0 + (c & 6) + i + (c < 8 ? 0 : a.F);
    } else {
#pragma unroll
        for (int r = 0; r < R / 2; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                wo[r][i] = min(f0 + 16 * r + (c & 14) + i, a.F - 1);
                wo[R / 2 + r][i] = a.F + wo[r][i];
            }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) wo[r][i] = wo[r][i] * pitch + piece;
    // the lane's token in each group of 8 (past cnt the last again; columns never stored)
#pragma unroll
    for (int n = 0; n < N8; ++n)
        xo[n] = s.tok[row0 + min(token_of<N8>(n, c), cnt - 1)] * pitch + piece;
    // 8-bit form: the scales of its column's token (a step is a block)
#pragma unroll
    for (int n = 0; n < NT; ++n)
        so[n] = Q8 ? s.tok[row0 + min(N8 == 1 ? c >> 1 : 16 * n + c, cnt - 1)] * (uint32_t)steps * 4 : 0;
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
    // U steps: all their loads, then all their products; the CU's other waves load meanwhile (a ring of single steps per
    // wave measured no faster)
    auto run = [&](auto uc) {
        constexpr int U = decltype(uc)::value;
        u32x4_t wv[U][R][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) wv[u][r][i] = load_w(w, wo[r][i] + 128 * u, k * 128);
#pragma unroll
        for (int n0 = 0; n0 < N8; n0 += NS) {
            u32x4_t xv[U][NS];
            float fx[U][NST];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int n = 0; n < NS; ++n) xv[u][n] = load_x(x, xo[n0 + n] + 128 * u, k * 128);
            if constexpr (Q8) {
#pragma unroll
                for (int n = 0; n < NST; ++n) {
                    float f[U];
                    load_floats<U>(sx, so[n0 / 2 + n], k * 4, f);
#pragma unroll
                    for (int u = 0; u < U; ++u) fx[u][n] = f[u];
                }
            }
            if (n0 == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int r = 0; r < R; ++r) swap_pairs(wv[u][r][0], wv[u][r][1]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                u32x4_t x0[NST], x1[NST];
                pair_tokens<NS>(xv[u], x0, x1);
                if constexpr (Q8) {
                    const float wg = __int_as_float(__builtin_amdgcn_readlane(fg, k - s0 + u));
                    const float wu = __int_as_float(__builtin_amdgcn_readlane(fu, k - s0 + u));
                    // accumulator rows 4 g .. 4 g + 3: in the mixed tile groups 0, 1 are gate rows and 2, 3 up rows
                    const float mixed = g < 2 ? wg : wu;
#pragma unroll
                    for (int n = 0; n < NST; ++n)
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const f32x4_t p = mfma_fp8(wv[u][r][0], wv[u][r][1], x0[n], x1[n],
                                                              f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
                            const float f = (R == 1 ? mixed : r < R / 2 ? wg : wu) * fx[u][n];
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                acc[r][n0 / 2 + n][v] = __builtin_fmaf(p[v], f, acc[r][n0 / 2 + n][v]);
                        }
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int n = 0; n < NST; ++n)
#pragma unroll
                            for (int r = 0; r < R; ++r)
                                acc[r][n0 / 2 + n] =
                                    mfma_bf16(wv[u][r][i], i == 0 ? x0[n] : x1[n], acc[r][n0 / 2 + n]);
                }
            }
            if (N8 > NS) __builtin_amdgcn_sched_barrier(0);
        }
        k += U;
    };
    constexpr int U = R == 1 ? 4 : R == 4 && N8 == 8 ? 1 : 2;
    while (k + U <= s1) run(IntC<U>());
    while (k < s1) run(IntC<1>());
    // The waves' parts of a token tile meet in LDS ([column][row], so a lane's four rows are one 16-byte word), are
    // added in wave order, and become h, two features a thread.  Halves alternate: one barrier per tile.
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float *rb = red + layer_exchange_at(par);
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
                const float *q = rb + (v * R + (fi >> 4)) * 256 + column_of<N8>(ci) * 16 + (fi & 15);
                const float2 gv = *(const float2 *)q, uv = *(const float2 *)(q + (R == 1 ? 8 : R / 2 * 256));
                gs.x += gv.x;
                gs.y += gv.y;
                us.x += uv.x;
                us.y += uv.y;
            }
            const float gate = s.gate[row0 + row];
            const float h0 = gs.x / (1.0f + expf(-gs.x)) * us.x * gate;
            const float h1 = gs.y / (1.0f + expf(-gs.y)) * us.y * gate;
            store_h<Q8>(a, row0 + row, f0 + fi, h0, h1);
        }
    }
}

// SELF: the workgroup selects the experts of the few tokens itself from the router's partial sums.
template <bool Q8, bool SELF>
__global__ __launch_bounds__(64 * kUpWaves, 2) void k_layer_up(LayerArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    float *red = (float *)lds;
    const RowsLds s = rows_lds(lds + kExchangeBytes, a);
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
    if (layer_sums_in_down(a.T, a.k) && blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.d / 16; i += blockDim.x) a.plan.done[i] = 0;
    if (a.T * a.k <= kFewChoices) {
        if (threadIdx.x < kWave) build_few_rows(s, a, T, blockIdx.x == 0);
        __syncthreads();
    } else {
        build_rows(s, a, T, blockIdx.x == 0);
    }
    const int hits = s.n[0];
    const int tiles = tiles_per_task(hits, (a.F + 7) / 8, a.T, (int)gridDim.x, 4);
    const int fs = 8 * tiles;
    const int nf = (a.F + fs - 1) / fs;
    int par = 0;
    for (int q = blockIdx.x; q < hits * nf; q += gridDim.x) {
        const int hi = q / nf, f0 = (q - hi * nf) * fs;
        const LayerRec rec = s.rec[hi];
        const int e = __builtin_amdgcn_readfirstlane(rec.e);
        const int row0 = __builtin_amdgcn_readfirstlane(rec.row0);
        const int cnt = __builtin_amdgcn_readfirstlane(rec.cnt);
        if (tiles == 1) {
            if (cnt <= 8) up_task<Q8, 1, 1>(a, s, e, f0, row0, cnt, red, par);
            else up_task<Q8, 1, 2>(a, s, e, f0, row0, cnt, red, par);
            continue;
        }
        // up to 64 rows at once; an expert of more rows reads its weights again for the rest
        for (int r = 0; r < cnt; r += 64) {
            const int m = min(cnt - r, 64);
            auto rows = [&](auto tc) {
                constexpr int R = decltype(tc)::value;
                if (m <= 8) up_task<Q8, R, 1>(a, s, e, f0, row0 + r, m, red, par);
                else if (m <= 16) up_task<Q8, R, 2>(a, s, e, f0, row0 + r, m, red, par);
                else if (m <= 32) up_task<Q8, R, 4>(a, s, e, f0, row0 + r, m, red, par);
                else up_task<Q8, R, 8>(a, s, e, f0, row0 + r, m, red, par);
            };
            if (tiles == 4) rows(IntC<4>());
            else rows(IntC<2>());
        }
    }
}

// ---------------------------------------------------------------- down

constexpr int kDownWaves = kLayerWaves;

// One down task: output columns n0 .. n0 + 16 R - 1 of expert e for its rows row0 .. row0 + cnt - 1 (cnt <= 8 N8), written
// to y in fp32.  The wave sums its share of K in steps of 128 bytes of a weight row: 64 of K, which meets both of h's parts,
// or 128 of K in e4m3, converted to fp16 (exact), its product scaled by the weights' scale and h's binade.  TAIL: F does not
// end on a step; pieces past F are zeros on both sides.  red, par: as in up_task.
template <bool Q8, int R, int N8, bool TAIL, bool SUM = false>
__device__ __forceinline__ void down_task(const LayerArgs &a, int e, int n0, int row0, int cnt, float *red, int &par)
{
    constexpr int NT = (N8 + 1) / 2;             // 16-column tiles
    constexpr int KS = Q8 ? kQ8Group : 64;       // K per step
    constexpr int KP = Q8 ? 16 : 8;              // K per 16-byte piece of a weight row
    constexpr int kBytes = Q8 ? 1 : 2;
    // row groups (tiles) whose h is in registers at a time
    constexpr int NS = N8 == 6 ? 2 : N8 < 4 ? N8 : 4, NST = (NS + 1) / 2;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int c = lane & 15, g = lane >> 4;
    // the lane's piece of a weight row (swap_pairs), in elements, and of an h row, where an 8-bit weight piece is two
    // (store_h)
    const int kp = KP * (2 * g + (c & 1)), kh = Q8 ? 8 * (4 * g + (c & 1)) : kp;
    const int steps = (a.F + KS - 1) / KS, s1 = steps * (wave + 1) / kDownWaves;
    const uint32_t wbytes = 16 * R * (uint32_t)a.F * kBytes, hrow = layer_h_row_bytes(Q8, a.F);
    const __amdgpu_buffer_rsrc_t w = buffer_of((const char *)a.w_dn + ((size_t)e * a.d + n0) * a.F * kBytes, wbytes);
    const __amdgpu_buffer_rsrc_t h = buffer_of((const char *)a.h + (size_t)row0 * hrow, (uint32_t)cnt * hrow);
    const __amdgpu_buffer_rsrc_t hx = buffer_of(a.hx + (Q8 ? (size_t)row0 * layer_hx_row_bytes(a.F) : 0),
                                                Q8 ? (uint32_t)cnt * layer_hx_row_bytes(a.F) : 0);
    const __amdgpu_buffer_rsrc_t sw =
        buffer_of(a.s_dn + (Q8 ? ((size_t)e * (a.d / kQ8Group) + n0 / kQ8Group) * steps : 0), Q8 ? steps * 4 : 0);
    uint32_t wo[R][2], ho[N8], lo[N8], xo[NT];   // lo: of the second part or line; xo: of the column's binades
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) wo[r][i] = (uint32_t)((16 * r + (c & 14) + i) * a.F + kp) * kBytes;
#pragma unroll
    for (int n = 0; n < N8; ++n) {
        ho[n] = (uint32_t)min(token_of<N8>(n, c), cnt - 1) * hrow;
        lo[n] = ho[n] + (Q8 ? 128 : 2 * a.F) + 16 * (2 * g + (c & 1));
        ho[n] += 16 * (2 * g + (c & 1));
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
        xo[n] = (uint32_t)min(N8 == 1 ? c >> 1 : 16 * n + c, cnt - 1) * layer_hx_row_bytes(a.F) + 4 * g;
    f32x4_t acc[R][NT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    int s = steps * wave / kDownWaves;
    auto run = [&](auto uc) {
        constexpr int U = decltype(uc)::value;
        u32x4_t wv[U][R][2];
        float fw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    wv[u][r][i] =
                        load_w(w, !TAIL || kp + (s + u) * KS < a.F ? wo[r][i] + 128 * u : kPastResource, s * 128);
        if constexpr (Q8) load_floats<U>(sw, 0, s * 4, fw);
#pragma unroll
        for (int n0 = 0; n0 < N8; n0 += NS) {
            u32x4_t hv[U][2][NS];   // the two parts, or the two lines of a block
            uint32_t hb[U][NST];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int l = 0; l < 2; ++l)
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        const int k = Q8 ? kh + 16 * l : kp;
                        const uint32_t off = (l == 0 ? ho[n0 + n] : lo[n0 + n]) + (Q8 ? 256 : 128) * u;
                        hv[u][l][n] = load_x(h, !TAIL || k + (s + u) * KS < a.F ? off : kPastResource,
                                             Q8 ? s * 256 : s * 128);
                    }
            if constexpr (Q8) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int n = 0; n < NST; ++n) {
                        hb[u][n] = load_u32(hx, xo[n0 / 2 + n] + 16 * u, s * 16);
                        // F % 16 == 0: a lane's four groups are all inside F, or the first two, or none
                        const int left = a.F - (s + u) * KS - 32 * g;
                        if (TAIL && left < 32) hb[u][n] = left > 0 ? hb[u][n] & 0xFFFFu : 0;
                    }
            }
            if (n0 == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int r = 0; r < R; ++r) swap_pairs(wv[u][r][0], wv[u][r][1]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                u32x4_t x[2][2][NST];
#pragma unroll
                for (int l = 0; l < 2; ++l) pair_tokens<NS>(hv[u][l], x[l][0], x[l][1]);
                if constexpr (Q8) {
                    u32x4_t xs[NST][4];
                    float f[NST];
#pragma unroll
                    for (int n = 0; n < NST; ++n) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) xs[n][i] = x[i / 2][i & 1][n];
                        const int binade = align_groups(hb[u][n], xs[n]);
                        f[n] = __builtin_amdgcn_ldexpf(fw[u], binade - 127 - (int)kTopBinade);
                    }
                    // RG tiles at a time, so that their chains of products interleave
                    constexpr int RG = NST == 1 && R > 1 ? 2 : 1;
#pragma unroll
                    for (int r0 = 0; r0 < R; r0 += RG) {
                        u32x4_t b[RG][4];
#pragma unroll
                        for (int r = 0; r < RG; ++r)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const u32x4_t v = wv[u][r0 + r][i];
                                b[r][2 * i] = fp8_to_f16(v.x, v.y);
                                b[r][2 * i + 1] = fp8_to_f16(v.z, v.w);
                            }
#pragma unroll
                        for (int n = 0; n < NST; ++n) {
                            f32x4_t p[RG];
#pragma unroll
                            for (int r = 0; r < RG; ++r) p[r] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int r = 0; r < RG; ++r) p[r] = mfma_f16(b[r][i], xs[n][i], p[r]);
#pragma unroll
                            for (int r = 0; r < RG; ++r)
#pragma unroll
                                for (int v = 0; v < 4; ++v)
                                    acc[r0 + r][n0 / 2 + n][v] =
                                        __builtin_fmaf(p[r][v], f[n], acc[r0 + r][n0 / 2 + n][v]);
                        }
                    }
                } else {
#pragma unroll
                    for (int l = 0; l < 2; ++l)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int n = 0; n < NST; ++n)
#pragma unroll
                                for (int r = 0; r < R; ++r)
                                    acc[r][n0 / 2 + n] = mfma_bf16(wv[u][r][i], x[l][i][n], acc[r][n0 / 2 + n]);
                }
            }
            if (N8 > NS) __builtin_amdgcn_sched_barrier(0);
        }
        s += U;
    };
    constexpr int U = R == 1 && N8 == 1 ? 4 : N8 >= (Q8 && R == 4 ? 2 : Q8 ? 4 : 6) ? 1 : 2;   // 256 registers
    while (s + U <= s1) run(IntC<U>());
    while (s < s1) run(IntC<1>());
    // the waves' parts meet in LDS as in up_task; two neighbouring columns a thread
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float *rb = red + layer_exchange_at(par);
        par ^= 1;
#pragma unroll
        for (int r = 0; r < R; ++r) *(f32x4_t *)(rb + (wave * R + r) * 256 + c * 16 + 4 * g) = acc[r][n];
        __syncthreads();
        for (int j = threadIdx.x; j < 8 * R * 16; j += 64 * kDownWaves) {
            const int ni = 2 * (j % (8 * R)), row = 16 * n + j / (8 * R);
            if (row >= cnt) break;
            float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int v2 = 0; v2 < kDownWaves; ++v2) {
                const float2 p = *(const float2 *)(rb + (v2 * R + (ni >> 4)) * 256 + column_of<N8>(row) * 16 + (ni & 15));
                v.x += p.x;
                v.y += p.y;
            }
            float *to = a.y + (size_t)(row0 + row) * a.d + n0 + ni;
            if constexpr (SUM) store_through((uint64_t *)to, __builtin_bit_cast(uint64_t, v));   // another XCD may add it
            else *(float2 *)to = v;
        }
    }
}

// Columns n0 .. n0 + nb - 1 of every valid token's output: the sum of its rows of y in expert order (nb even).
// mine: this thread's choice's row; sorted: LDS, one of each thread.
__device__ __forceinline__ void sum_columns(const LayerArgs &a, int valid, int n0, int nb, int mine, int *sorted)
{
    // a row's place among its token's is the number of smaller ones
    const int i = threadIdx.x, t0 = i / a.k * a.k;
    sorted[i] = mine;
    __syncthreads();
    int place = 0, rows = 0;
    if (i < a.T * a.k)
        for (int j = t0; j < t0 + a.k; ++j) {
            const int r = sorted[j];
            place += r >= 0 && r < mine;
            rows += r >= 0;
        }
    __syncthreads();
    if (i < a.T * a.k) {
        if (mine >= 0) sorted[t0 + place] = mine;
        if (i - t0 >= rows) sorted[i] = -1;
    }
    __syncthreads();
    for (int q = i; 2 * q < valid * nb; q += 64 * kDownWaves) {
        const int t = 2 * q / nb, col = n0 + 2 * q % nb;
        float2 v = make_float2(0.0f, 0.0f);
        bool more = true;
        for (int j = t * a.k; more && j < (t + 1) * a.k; j += 4) {   // four rows on their way at a time
            uint64_t p[4];
            int r[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                r[u] = j + u < (t + 1) * a.k ? sorted[j + u] : -1;
                // past the caches that may hold older values of a line another XCD has written to
                p[u] = __hip_atomic_load((const uint64_t *)(a.y + (size_t)max(r[u], 0) * a.d + col), __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float2 f = __builtin_bit_cast(float2, p[u]);
                if (r[u] >= 0) {
                    v.x += f.x;
                    v.y += f.y;
                }
            }
            more = r[3] >= 0;
        }
        *(uint32_t *)(a.out + (size_t)t * a.d + col) = (uint32_t)f32_to_bf16(v.x) | (uint32_t)f32_to_bf16(v.y) << 16;
    }
    __syncthreads();   // sorted is the next call's
}

// SUM (layer_sums_in_down): the workgroup that finishes a column block's last task adds the block's rows up, which
// saves the sum kernel's launch.
template <bool Q8, bool TAIL, bool SUM>
__global__ __launch_bounds__(64 * kDownWaves, 2) void k_layer_down(LayerArgs a)
{
    __shared__ __attribute__((aligned(16))) char lds[kExchangeBytes];
    __shared__ int sorted[SUM ? 64 * kDownWaves : 1], last;   // T k <= 32 of sorted are choices
    float *red = (float *)lds;
    const int mine = SUM && (int)threadIdx.x < a.T * a.k ? a.plan.row_of[threadIdx.x] : -1;
    const int valid = SUM ? a.plan.n[1] : 0;
    const int hits = a.plan.n[0];
    const int tiles = tiles_per_task(hits, a.d / 16, a.T, (int)gridDim.x, 1);
    const int nc = a.d / (16 * tiles);   // d % 128 == 0
    if (SUM && hits == 0) {
        for (int q = blockIdx.x; q < nc; q += gridDim.x)
            sum_columns(a, valid, q * 16 * tiles, 16 * tiles, mine, sorted);
        return;
    }
    int par = 0;
    for (int q = blockIdx.x; q < hits * nc; q += gridDim.x) {
        const int hi = q / nc, n0 = (q - hi * nc) * 16 * tiles;
        const LayerRec rec = a.plan.rec[hi];
        const int e = __builtin_amdgcn_readfirstlane(rec.e);
        const int row0 = __builtin_amdgcn_readfirstlane(rec.row0);
        const int cnt = __builtin_amdgcn_readfirstlane(rec.cnt);
        if constexpr (SUM) {
            if (tiles == 1) down_task<Q8, 1, 1, TAIL, true>(a, e, n0, row0, cnt, red, par);
            else if (tiles == 2) down_task<Q8, 2, 1, TAIL, true>(a, e, n0, row0, cnt, red, par);
            else down_task<Q8, 4, 1, TAIL, true>(a, e, n0, row0, cnt, red, par);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // every wave's part of y is in memory
            __syncthreads();
            if (threadIdx.x == 0)
                last = __hip_atomic_fetch_add(a.plan.done + n0 / (16 * tiles), 1, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT) == hits - 1;
            __syncthreads();
            if (last) sum_columns(a, valid, n0, 16 * tiles, mine, sorted);
            continue;
        }
        if (tiles == 1) {
            if (cnt <= 8) down_task<Q8, 1, 1, TAIL>(a, e, n0, row0, cnt, red, par);
            else down_task<Q8, 1, 2, TAIL>(a, e, n0, row0, cnt, red, par);
            continue;
        }
        // up to 64 rows at once; an expert of more rows reads its weights again for the rest
        for (int r = 0; r < cnt; r += 64) {
            const int m = min(cnt - r, 64);
            auto rows = [&](auto tc) {
                constexpr int R = decltype(tc)::value;
                if (m <= 8) down_task<Q8, R, 1, TAIL>(a, e, n0, row0 + r, m, red, par);
                else if (m <= 16) down_task<Q8, R, 2, TAIL>(a, e, n0, row0 + r, m, red, par);
                else if (m <= 32) down_task<Q8, R, 4, TAIL>(a, e, n0, row0 + r, m, red, par);
                else if (!Q8 && m <= 48)   // 256 choices over 8 experts, 14336 features: 221 us, without this form 247
                    down_task<Q8, R, Q8 ? 8 : 6, TAIL>(a, e, n0, row0 + r, m, red, par);
                else   // four e4m3 tiles by four token tiles would not fit the registers
                    for (int i = 0; i < (Q8 ? R / 2 : 1); ++i)
                        down_task<Q8, Q8 ? 2 : R, 8, TAIL>(a, e, n0 + 32 * i, row0 + r, m, red, par);
            };
            if (tiles == 4) rows(IntC<4>());
            else rows(IntC<2>());
        }
    }
}

// The smallest of the lanes' row numbers, -1 (none) counting as the largest.
__device__ __forceinline__ uint32_t wave_min_row(int v) { return ~wave_max_u32(~(uint32_t)v); }

// out[t] = sum of the token's rows of y in expert order.  A workgroup takes 1024 columns of a token.  4.6 us after the
// weights' stream (1.6 with y and the code still in the caches): the launch and two dependent fetches.
__global__ __launch_bounds__(256) void k_layer_sum(LayerArgs a)
{
    const int nc = (a.d + 1023) / 1024;
    const int t = (int)blockIdx.x / nc, col = ((int)blockIdx.x - t * nc) * 1024 + 4 * (int)threadIdx.x;
    const bool in = col < a.d;   // every lane stays for the reductions
    const int lane = threadIdx.x % kWave;
    // lane j of every wave holds the token's j-th row; rows of higher experts have higher numbers, so the ascending order
    // is the experts'
    int mine = lane < a.k ? a.plan.row_of[t * a.k + lane] : -1;
    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (bool more = true; more;) {   // four rows on their way at a time
        f32x4_t p[4];
        bool have[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t row = wave_min_row(mine);
            have[u] = row != 0xFFFFFFFFu;
            if ((uint32_t)mine == row) mine = -1;
            p[u] = have[u] && in ? *(const f32x4_t *)(a.y + (size_t)row * a.d + col) : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (have[u]) v += p[u];
        more = have[3];
    }
    if (!in || t >= a.plan.n[1]) return;   // valid tokens
    typedef uint32_t u32x2_v __attribute__((ext_vector_type(2)));
    *(u32x2_v *)(a.out + (size_t)t * a.d + col) =
        u32x2_v{(uint32_t)f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16,
                (uint32_t)f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16};
}

// ---------------------------------------------------------------- router of up to kLayerSelfT tokens

// Partial sums part[s][t][e] in the library's order (one ascending fma chain per K segment), on the vector units (d = 4096,
// E = 8: 5.8 us; the matrix units' router 10.5, whose dependent products follow each other in 48 cycles).  With
// a few tokens the chains are few, and the time goes into fetching W_r and into the length of a chain.  A workgroup takes
// (segment s, up to 16 experts): its weights are fetched at once into LDS (a segment of d = 7168: 56 KiB), then every
// lane runs one chain (16 experts x 4 tokens a wave, 8 x 8 where there are no more than 8 experts), its operands read 8
// steps ahead.
constexpr int kVrThreads = 512;
constexpr int kVrRows = 1024;   // weight rows per staged chunk

// LE: log2 of the experts per workgroup and of the lanes per token (3 or 4).
template <int LE>
__global__ __launch_bounds__(kVrThreads) void k_layer_router(LayerArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int S = 1 << LE;
    const int seg = a.d / kRouterSegments;
    const int cap = min(seg, kVrRows);
    const int s = (int)blockIdx.x % kRouterSegments, e0 = (int)blockIdx.x / kRouterSegments * S;
    const int ne = min(S, a.E - e0);
    float *ws = (float *)lds;                     // [cap][S]
    float *xs = ws + (size_t)cap * S;             // [T][cap]
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int t = (wave << (6 - LE)) + (lane >> LE), el = lane & (S - 1);
    const bool mine = t < a.T && el < ne;
    float acc = 0.0f;
    for (int r0 = 0; r0 < seg; r0 += kVrRows) {
        const int rows = min(kVrRows, seg - r0);   // a multiple of 16
        const float *w = a.wr + ((size_t)s * seg + r0) * a.E + e0;
        for (int i = threadIdx.x; i < a.T * rows / 8; i += kVrThreads) {
            const int tt = i / (rows / 8), c = i % (rows / 8);
            float f[8];
            unpack8(*(const u32x4_t *)(a.x + (size_t)tt * a.d + (size_t)s * seg + r0 + 8 * c), f);
            f32x4_t *p = (f32x4_t *)(xs + (size_t)tt * cap + 8 * c);
            p[0] = f32x4_t{f[0], f[1], f[2], f[3]};
            p[1] = f32x4_t{f[4], f[5], f[6], f[7]};
        }
        if (ne == S && a.E % 4 == 0) {   // 16-byte pieces
            constexpr int P = S / 4;
            for (int i = threadIdx.x; i < rows * P; i += 8 * kVrThreads) {
                f32x4_t v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int j = min(i + u * kVrThreads, rows * P - 1);
                    v[u] = *(const f32x4_t *)(w + (size_t)(j / P) * a.E + 4 * (j % P));
                }
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (i + u * kVrThreads < rows * P) *(f32x4_t *)(ws + 4 * (i + u * kVrThreads)) = v[u];
            }
        } else {   // columns past the last expert repeat it (never used)
            for (int i = threadIdx.x; i < rows * S; i += 8 * kVrThreads) {
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int j = min(i + u * kVrThreads, rows * S - 1);
                    v[u] = w[(size_t)(j / S) * a.E + min(j % S, ne - 1)];
                }
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (i + u * kVrThreads < rows * S) ws[i + u * kVrThreads] = v[u];
            }
        }
        __syncthreads();
        if (mine) {
            const float *xp = xs + (size_t)t * cap, *wp = ws + el;
            struct Ops {
                f32x4_t x[2];
                float w[8];
            };
            auto fetch = [&](int i, Ops &o) {
                o.x[0] = *(const f32x4_t *)(xp + i);
                o.x[1] = *(const f32x4_t *)(xp + i + 4);
#pragma unroll
                for (int u = 0; u < 8; ++u) o.w[u] = wp[(i + u) * S];
                __builtin_amdgcn_sched_barrier(0);
            };
            auto chain = [&](const Ops &o) {
#pragma unroll
                for (int u = 0; u < 8; ++u) acc = __builtin_fmaf(o.x[u / 4][u % 4], o.w[u], acc);
                __builtin_amdgcn_sched_barrier(0);
            };
            Ops p, q;
            fetch(0, p);
            for (int i = 0; i < rows; i += 16) {
                fetch(i + 8, q);
                chain(p);
                fetch(min(i + 16, rows - 8), p);
                chain(q);
            }
        }
        __syncthreads();
    }
    if (mine) a.part[((size_t)s * a.T + t) * a.E + e0 + el] = acc;
}

template <int LE>
hipError_t launch_vr(const LayerArgs &a, hipStream_t s)
{
    const size_t rows = std::min(a.d / kRouterSegments, kVrRows);
    const int grid = kRouterSegments * ((a.E + (1 << LE) - 1) >> LE);
    hipLaunchKernelGGL(k_layer_router<LE>, dim3(grid), dim3(kVrThreads), rows * ((1 << LE) + a.T) * 4, s, a);
    return hipGetLastError();
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
    const size_t lds = kExchangeBytes + rows_lds_bytes(a.T, a.k, a.E_local);
    if (self) hipLaunchKernelGGL((k_layer_up<Q8, true>), dim3(grid), dim3(64 * kUpWaves), lds, s, a);
    else hipLaunchKernelGGL((k_layer_up<Q8, false>), dim3(grid), dim3(64 * kUpWaves), lds, s, a);
    return hipGetLastError();
}

template <bool Q8, bool TAIL>
void launch_down(const LayerArgs &a, bool sum, int grid, hipStream_t s)
{
    if (sum) hipLaunchKernelGGL((k_layer_down<Q8, TAIL, true>), dim3(grid), dim3(64 * kDownWaves), 0, s, a);
    else hipLaunchKernelGGL((k_layer_down<Q8, TAIL, false>), dim3(grid), dim3(64 * kDownWaves), 0, s, a);
}

}  // namespace

hipError_t launch_layer_router(const LayerArgs &a, hipStream_t s)
{
    return a.E <= 8 ? launch_vr<3>(a, s) : launch_vr<4>(a, s);
}

hipError_t launch_layer(const LayerArgs &a, bool q8, bool self, hipStream_t s)
{
    const int cus = device_cus();
    if (cus <= 0) return hipErrorInvalidDevice;
    // tasks, if every choice is another local expert
    const long most = (long)layer_hits_cap(a.T, a.k, a.E_local) * ((a.F + 7) / 8);
    const int grid = (int)std::min<long>(most, 2L * cus);
    const hipError_t e = q8 ? launch_up<true>(a, self, grid, s) : launch_up<false>(a, self, grid, s);
    if (e != hipSuccess) return e;
    const bool tail = a.F % (q8 ? kQ8Group : 64) != 0;
    const int gd = (int)std::min<long>((long)layer_hits_cap(a.T, a.k, a.E_local) * (a.d / 16), 2L * cus);
    const bool sum = layer_sums_in_down(a.T, a.k);
    if (q8 && tail) launch_down<true, true>(a, sum, gd, s);
    else if (q8) launch_down<true, false>(a, sum, gd, s);
    else if (tail) launch_down<false, true>(a, sum, gd, s);
    else launch_down<false, false>(a, sum, gd, s);
    const hipError_t e2 = hipGetLastError();
    if (e2 != hipSuccess || sum) return e2;
    hipLaunchKernelGGL(k_layer_sum, dim3(a.T * ((a.d + 1023) / 1024)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace mk
