// grouped.hip -- the grouped product's gradients and its form of 8-bit integers: one persistent launch each, whose
// workgroups (one per CU) go through the tiles of all experts.  The tile itself is grouped_dev.h's.
//   dgrad   da[r, i]    = sum_n dy[r, n] W[e, n, i]                       rows r of expert e
//   wgrad   dW[e, n, i] = sum over e's rows of dy[r, n] a[r, i]
//   8-bit   y[r, n]     = a_scale[r] w_scale[e, n] sum_i a[r, i] w[e, n, i]
#include <hip/hip_runtime.h>

#include <algorithm>

#include "grouped_dev.h"
#include "grouped_few.h"
#include "mk_device.h"
#include "mk_launch.h"

namespace mk {

namespace {

struct NoTokens {
    __device__ __forceinline__ void operator()(int, int *) const {}
};

template <int BM>
__device__ __forceinline__ void dgrad_tile(const GroupedArgs &a, const GroupedJob &j, lds_char_t *lds, int wave, int lane)
{
    typedef GTile<kDgrad, BM> T;
    lane = fresh_lane(lane);
    Side<true, 256> sp;
    Side<false, BM> sq;
    side_columns(sp, (const uint16_t *)a.w + (size_t)j.e * a.N * a.K + j.col0, (uint64_t)a.K * 2, a.K - j.col0, false,
                 wave, lane);
    const uint32_t rb = (uint32_t)a.N * 2;
    side_rows(sq, make_rsrc4(a.dy + (size_t)j.row0 * a.N, (size_t)0x80000000u), wave, lane,
              [&](int m) { return m < j.rows ? (uint32_t)m * rb : kPastResource; });
    f32x16_t acc[T::NI][T::MI];
    tile_sums<T, false>(sp, sq, a.N, kPlainRecords, 0u, NoTokens{}, lds, wave, lane, acc);
    __syncthreads();
    store_bf16<T>([&](int i, int k, int v) { return acc[i][k][v]; }, (uint16_t *)a.out + (size_t)j.row0 * a.K + j.col0,
                  a.K, j.rows, a.K - j.col0, lds, wave, lane);
    __syncthreads();
}

template <int BM>
__device__ __forceinline__ void i8_tile(const GroupedArgs &a, const GroupedJob &j, lds_char_t *lds, int wave, int lane)
{
    typedef GTile<kI8, BM> T;
    lane = fresh_lane(lane);
    Side<false, 256> sp;
    Side<false, BM> sq;
    side_rows(sp, make_rsrc4((const int8_t *)a.w + ((size_t)j.e * a.N + j.col0) * a.K, (size_t)0x80000000u), wave, lane,
              [&](int n) { return j.col0 + n < a.N ? (uint32_t)n * (uint32_t)a.K : kPastResource; });
    if (a.row_token) {
        side_rows(sq, make_rsrc4(a.a, (size_t)a.a_rows * a.K), wave, lane, [&](int m) {
            if (m >= j.rows) return kPastResource;
            const int t = a.row_token[j.row0 + m];
            return t >= 0 && t < a.a_rows ? (uint32_t)t * (uint32_t)a.K : kPastResource;
        });
    } else {
        side_rows(sq, make_rsrc4((const int8_t *)a.a + (size_t)j.row0 * a.K, (size_t)0x80000000u), wave, lane,
                  [&](int m) { return m < j.rows ? (uint32_t)m * (uint32_t)a.K : kPastResource; });
    }
    i32x16_t acc[T::NI][T::MI];
    tile_sums<T, false>(sp, sq, a.K, kPlainRecords, 0u, NoTokens{}, lds, wave, lane, acc);
    // the scales of the lane's rows and of its columns, four neighbours at a time
    lane = fresh_lane(lane);
    const int wn = wave % T::WN, wm = wave / T::WN;
    float sa[T::MI];
#pragma unroll
    for (int k = 0; k < T::MI; ++k) {
        const int m = wm * (T::BM / T::WM) + 32 * k + (lane & 31);
        const int r = j.row0 + min(m, j.rows - 1);
        const int t = a.row_token ? a.row_token[r] : r;
        sa[k] = t >= 0 && t < a.a_rows ? a.a_scale[t] : 0.0f;
    }
    const float *ws = a.w_scale + (size_t)j.e * a.N;
    f32x4_t sw[T::NI][4];
#pragma unroll
    for (int i = 0; i < T::NI; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int n = j.col0 + wn * (T::BN / T::WN) + 32 * i + 8 * g + 4 * (lane >> 5);
            sw[i][g] = *(const f32x4_t *)(ws + min(n, a.N - 4));
        }
    __syncthreads();
    store_bf16<T>([&](int i, int k, int v) { return (float)acc[i][k][v] * sw[i][v / 4][v % 4] * sa[k]; },
                  (uint16_t *)a.out + (size_t)j.row0 * a.N + j.col0, a.N, j.rows, a.N - j.col0, lds, wave, lane);
    __syncthreads();
}

template <int BM, bool GATHER>
__device__ __forceinline__ void wgrad_tile(const GroupedArgs &a, const GroupedTables &t, int e, int n0, int k0,
                                           lds_char_t *lds, int wave, int lane)
{
    typedef GTile<kWgrad, BM> T;
    lane = fresh_lane(lane);
    Side<true, 256> sp;
    Side<true, BM> sq;
    const int row0 = __builtin_amdgcn_readfirstlane(t.off[e]);
    const int cnt = __builtin_amdgcn_readfirstlane(table_count(t, e));
    const uint64_t ld = (uint64_t)a.K * 2;
    side_columns(sp, (const uint16_t *)a.a + (GATHER ? 0 : (size_t)row0 * a.K) + k0, ld, a.K - k0, GATHER, wave, lane);
    side_columns(sq, a.dy + (size_t)row0 * a.N + n0, (uint64_t)a.N * 2, a.N - n0, false, wave, lane);
    f32x16_t acc[T::NI][T::MI];
    auto toks = [&](int slab, int *ids) {
        if constexpr (!GATHER) return;
#pragma unroll
        for (int i = 0; i < Side<true, 256>::SLOTS; ++i) {
            const int r = slab * 64 + sp.pos + kGroupedWaves * Side<true, 256>::RPL * i;
            const int v = a.row_token[row0 + min(r, cnt - 1)];
            ids[i] = v < a.a_rows ? v : -1;
        }
    };
    // with a gather the rows' offsets run through all of `a` (and nothing is read of no rows)
    const uint32_t records =
        GATHER ? (a.a_rows > 0 ? (uint32_t)((size_t)a.a_rows * a.K * 2 - (size_t)k0 * 2) : 0u) : (uint32_t)kPlainRecords;
    tile_sums<T, GATHER>(sp, sq, cnt, records, (uint32_t)ld, toks, lds, wave, lane, acc);
    __syncthreads();
    const size_t o = ((size_t)e * a.N + n0) * a.K + k0;
    auto value = [&](int i, int k, int v) { return acc[i][k][v]; };
    if (a.out_f32)
        store_f32<T>(value, (float *)a.out + o, a.K, a.N - n0, a.K - k0, a.accumulate, lds, wave, lane);
    else store_bf16<T>(value, (uint16_t *)a.out + o, a.K, a.N - n0, a.K - k0, lds, wave, lane);
    __syncthreads();
}

}  // namespace

// Rows' products (dgrad, 8-bit): the last rows of an expert run as a tile of 128, 64 or 32 rows.
template <int KIND>
__device__ __forceinline__ void rows_tiles(const GroupedArgs &a, const GroupedTables &t, lds_char_t *lds, int wave, int lane)
{
    const int cols = ((KIND == kI8 ? a.N : a.K) + 255) / 256;
    const int tasks = (t.tall[a.E] + t.low[a.E]) * cols;   // (outputs that fit the device have fewer than 2^31 tiles)
    for (int q = xcd_place((int)blockIdx.x, (int)gridDim.x); q < tasks; q += gridDim.x) {
        const GroupedJob j = rows_job(a, t, cols, q);
        if constexpr (KIND == kDgrad) {
            if (j.rows > 128) dgrad_tile<256>(a, j, lds, wave, lane);
            else if (j.rows > 64) dgrad_tile<128>(a, j, lds, wave, lane);
            else if (j.rows > 32) dgrad_tile<64>(a, j, lds, wave, lane);
            else dgrad_tile<32>(a, j, lds, wave, lane);
        } else {
            if (j.rows > 128) i8_tile<256>(a, j, lds, wave, lane);
            else if (j.rows > 64) i8_tile<128>(a, j, lds, wave, lane);
            else if (j.rows > 32) i8_tile<64>(a, j, lds, wave, lane);
            else i8_tile<32>(a, j, lds, wave, lane);
        }
    }
}

__global__ __launch_bounds__(kGroupedThreads, 1) void k_grouped_dgrad(GroupedArgs a)
{
    __shared__ __attribute__((aligned(1024))) char stages[kGroupedStages];
    __shared__ GroupedTables t;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave), lane = (int)threadIdx.x % kWave;
    tables_rows(a, t);
    rows_tiles<kDgrad>(a, t, (lds_char_t *)stages, wave, lane);
}

__global__ __launch_bounds__(kGroupedThreads, 1) void k_grouped_i8(GroupedArgs a)
{
    __shared__ __attribute__((aligned(1024))) union {
        struct {
            char stages[kGroupedStages];
            GroupedTables t;
        } tile;
        struct {
            char ring[kGroupedWaves * kFewRing];
            FewTables t;
        } few;
    } m;
    static_assert(sizeof(m) <= 160 * 1024 && kGroupedStages + sizeof(GroupedTables) <= kGroupedWaves * kFewRing,
                  "LDS; the few rows' tables are made from the others");
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave), lane = (int)threadIdx.x % kWave;
    const int2 hits = tables_rows(a, m.tile.t);
    const int R = __builtin_amdgcn_readfirstlane(m.tile.t.off[a.E]), H = __builtin_amdgcn_readfirstlane(hits.y);
    if (R <= kFewRows && R <= kFewGroup * H) {
        few_tables(a, m.tile.t, m.few.t, hits.x);
        // The width of a weight tile: 32, or 16 where that leaves the workgroup with the most tasks less to read.
        const int G = (int)gridDim.x;
        const int w32 = (H * ((a.N + 31) / 32) + G - 1) / G * 32, w16 = (H * ((a.N + 15) / 16) + G - 1) / G * 16;
        if (w16 < w32) few_rows<16>(a, m.few.t, H, (lds_char_t *)m.few.ring, wave, lane);
        else few_rows<32>(a, m.few.t, H, (lds_char_t *)m.few.ring, wave, lane);
    } else {
        rows_tiles<kI8>(a, m.tile.t, (lds_char_t *)m.tile.stages, wave, lane);
    }
}

// The weights' gradient: tiles of 256 x 256 (the last 128 or fewer of the N: 128 x 256), experts with the most rows
// first; every other round goes through the workgroups backwards, so that those with a long task get a short one next.
template <bool GATHER>
__global__ __launch_bounds__(kGroupedThreads, 1) void k_grouped_wgrad(GroupedArgs a)
{
    __shared__ __attribute__((aligned(1024))) char stages[kGroupedStages];
    __shared__ GroupedTables t;
    lds_char_t *lds = (lds_char_t *)stages;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave), lane = (int)threadIdx.x % kWave;
    tables_offsets(a, t);
    for (int e = (int)threadIdx.x; e < a.E; e += kGroupedThreads) {
        const int c = table_count(t, e);
        int rank = 0;
        for (int f = 0; f < a.E; ++f) {
            const int d = table_count(t, f);
            rank += d > c || (d == c && f < e);
        }
        t.low[rank] = e;
    }
    __syncthreads();
    const int nk = (a.K + 255) / 256, nn = (a.N + 255) / 256, per = nk * nn;
    const int64_t tasks = (int64_t)a.E * per;
    const int G = (int)gridDim.x, place = xcd_place((int)blockIdx.x, G);
    for (int64_t round = 0; round * G < tasks; ++round) {
        const int64_t q = round * G + ((round & 1) ? G - 1 - place : place);
        if (q >= tasks) continue;
        const int i = (int)(q / per), r = (int)(q - (int64_t)i * per);
        const int e = __builtin_amdgcn_readfirstlane(t.low[i]);
        if (a.accumulate && table_count(t, e) == 0) continue;   // nothing to add (uniform)
        const int group = r / (8 * nk), in = r - group * 8 * nk, size = min(8, nn - 8 * group);
        const int k0 = __builtin_amdgcn_readfirstlane(in / size * 256);
        const int n0 = __builtin_amdgcn_readfirstlane((8 * group + in % size) * 256);
        if (a.N - n0 > 128) wgrad_tile<256, GATHER>(a, t, e, n0, k0, lds, wave, lane);
        else wgrad_tile<128, GATHER>(a, t, e, n0, k0, lds, wave, lane);
    }
}

namespace {

// One workgroup per CU of the current device, a multiple of 8 (0 on an error).
int persistent_grid()
{
    constexpr int kMaxDevices = 64;
    static int cached[kMaxDevices] = {};
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 0;
    if (dev >= 0 && dev < kMaxDevices && cached[dev] > 0) return cached[dev];
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
    const int grid = std::max(8, cus - cus % 8);
    if (dev >= 0 && dev < kMaxDevices) cached[dev] = grid;
    return grid;
}

}  // namespace

hipError_t launch_grouped_dgrad(const GroupedArgs &a, hipStream_t s)
{
    const int grid = persistent_grid();
    if (grid <= 0) return hipErrorInvalidDevice;
    hipLaunchKernelGGL(k_grouped_dgrad, dim3(grid), dim3(kGroupedThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const GroupedArgs &a, hipStream_t s)
{
    const int grid = persistent_grid();
    if (grid <= 0) return hipErrorInvalidDevice;
    if (a.row_token) hipLaunchKernelGGL(k_grouped_wgrad<true>, dim3(grid), dim3(kGroupedThreads), 0, s, a);
    else hipLaunchKernelGGL(k_grouped_wgrad<false>, dim3(grid), dim3(kGroupedThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grouped_i8(const GroupedArgs &a, hipStream_t s)
{
    const int grid = persistent_grid();
    if (grid <= 0) return hipErrorInvalidDevice;
    hipLaunchKernelGGL(k_grouped_i8, dim3(grid), dim3(kGroupedThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace mk
