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

// A run of the row products' tiles of one shape, n of them: short ones, or tall ones from the from-th on; tiles of `width`
// columns, cols of them from column first_col.  A tall one may be cut into 2^cut tiles of BM x BN.
struct Tiles {
    int n, cols, first_col, width;
    bool low;
    int from, cut;
};

// Tiles q, q + G, ... of a run; returns the first q past it.
template <int KIND, int BM, int BN>
__device__ __forceinline__ int rows_tiles(const GroupedArgs &a, GroupedTables &t, int q, const Tiles &of, lds_char_t *lds,
                                          int wave, int lane0)
{
    typedef GTile<KIND, BM, BN> T;
    typedef TileLoads<T, false> TL;
    constexpr int STORES = 2 * T::NI * T::MI;
    const int n = of.n;
    if (q >= n) return q;
    const int G = (int)gridDim.x;
    int lane = fresh_lane(lane0);
    auto job_of = [&](int i) {
        GroupedJob j;
        if (BM <= 128 && of.low) {
            j = low_job(a, t, of.cols, BN, i);
        } else {
            constexpr int kAcross = BN == 256 ? 0 : (BN == 128 ? 1 : 2);   // of 2^kAcross parts
            j = tall_job(a, t, of.cols, of.width, of.from + (i >> of.cut));
            const int part = i & ((1 << of.cut) - 1), down = part >> kAcross;
            j.row0 += down * BM;
            j.rows = min(j.rows - down * BM, BM);
            j.col0 += of.first_col + (part & ((1 << kAcross) - 1)) * BN;
        }
        return j;
    };
    // 8-bit with a gather: the tokens of a tile's rows, into LDS (waves 0 to 3, 64 each), and token m of them, or -1.  Waves
    // that are through with a run's first begin() load the next tile's while others still read this one's: a place for each.
    const bool gather = KIND == kI8 && a.row_token;
    auto tokens = [&](const GroupedJob &j, int buf) {
        if (gather && wave < 4)
            lds_load4(make_rsrc4(a.row_token + j.row0, (size_t)j.rows * 4),
                      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char_t *)&t.tok[tile_tokens_at(buf) + 64 * wave]),
                      (uint32_t)(64 * wave + lane) * 4u);
    };
    auto token = [&](const GroupedJob &j, int m, int buf) {
        const int v = t.tok[tile_tokens_at(buf) + (m & (kTokenRows - 1))];
        return m < j.rows && v >= 0 && v < a.a_rows ? v : -1;
    };
    // The loads of a tile's scales (8-bit) and of its first slab.
    auto begin = [&](const GroupedJob &j, TL &tl, int buf) {
        if constexpr (KIND == kDgrad) {
            side_columns(tl.p, (const uint16_t *)a.w + (size_t)j.e * a.N * a.K + j.col0, (uint64_t)a.K * 2, a.K - j.col0,
                         false, wave, lane);
            const uint32_t rb = (uint32_t)a.N * 2;
            side_rows(tl.q, make_rsrc4(a.dy + (size_t)j.row0 * a.N, (size_t)0x80000000u), wave, lane,
                      [&](int m, int) { return m < j.rows ? (uint32_t)m * rb : kPastResource; });
            tl.len = a.N;
        } else {
            const uint32_t rb = (uint32_t)a.K;
            side_rows(tl.p, make_rsrc4((const int8_t *)a.w + ((size_t)j.e * a.N + j.col0) * a.K, (size_t)0x80000000u),
                      wave, lane, [&](int c, int) { return j.col0 + c < a.N ? (uint32_t)c * rb : kPastResource; });
            if (gather)
                side_rows(tl.q, make_rsrc4(a.a, (size_t)a.a_rows * a.K), wave, lane, [&](int m, int) {
                    const int v = token(j, m, buf);
                    return v >= 0 ? (uint32_t)v * rb : kPastResource;
                });
            else
                side_rows(tl.q, make_rsrc4((const int8_t *)a.a + (size_t)j.row0 * a.K, (size_t)0x80000000u), wave, lane,
                          [&](int m, int) { return m < j.rows ? (uint32_t)m * rb : kPastResource; });
            tl.len = a.K;
            // waves 0 to 3: 64 rows' scales each; the others: 64 columns'
            const int i = 64 * (wave & 3) + lane;
            const bool rows = wave < 4;
            uint32_t o = kPastResource;
            if (rows) {
                const int v = gather ? token(j, i, buf) : (i < j.rows ? i : -1);
                if (v >= 0) o = (uint32_t)v * 4u;
            } else if (i < BN && j.col0 + i < a.N) {
                o = (uint32_t)i * 4u;
            }
            const float *from = rows ? a.a_scale + (gather ? 0 : (size_t)j.row0) : a.w_scale + (size_t)j.e * a.N + j.col0;
            lds_load4(make_rsrc4(from, (size_t)0x80000000u),
                      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char_t *)&t.scale[buf][rows ? 0 : 1][64 * (wave & 3)]),
                      o);
        }
        tl.records_p = kPlainRecords;
#pragma unroll
        for (int i = 0; i < T::PRE; ++i) tl.load_slab(i);
    };
    int buf = 0;
    GroupedJob job = job_of(q);
    tokens(job, buf);
    wait_vmem_all();
    __syncthreads();
    TL tl;
    tl.dst = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds + (uint32_t)wave * 1024u);
    begin(job, tl, buf);
    for (bool first = true;; first = false) {
        const bool more = q + G < n;
        GroupedJob next = job;
        if (more) {
            next = job_of(q + G);
            tokens(next, buf ^ 1);
        }
        typename Acc<KIND>::type acc[T::NI][T::MI];
        tile_sums<T, false, STORES>(tl, !first, NoTokens{}, lds, wave, lane, acc);
        __syncthreads();   // every wave is done with the stages
        lane = fresh_lane(lane0);
        if (more) begin(next, tl, buf ^ 1);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        const int el = fresh_lane(lane0);
        if constexpr (KIND == kDgrad) {
            store_bf16<T>([&](int i, int k, int v) { return acc[i][k][v]; },
                          (uint16_t *)a.out + (size_t)job.row0 * a.K + job.col0, a.K, job.rows, a.K - job.col0, lds, wave, el);
        } else {
            const int wn = wave % T::WN, wm = wave / T::WN % T::WM;
            float sa[T::MI];
#pragma unroll
            for (int k = 0; k < T::MI; ++k) sa[k] = t.scale[buf][0][wm * (T::BM / T::WM) + 32 * k + (el & 31)];
            const float *sw = &t.scale[buf][1][wn * (T::BN / T::WN) + 4 * (el >> 5)];
            store_bf16<T>([&](int i, int k, int v) { return (float)acc[i][k][v] * sw[32 * i + 8 * (v / 4) + v % 4] * sa[k]; },
                          (uint16_t *)a.out + (size_t)job.row0 * a.N + job.col0, a.N, job.rows, a.N - job.col0, lds, wave,
                          el);
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();   // the outputs have left the stages
        q += G;
        if (!more) break;
        job = next;
        buf ^= 1;
    }
    wait_vmem_all();
    return q;
}

// The rounds that tiles take, of each of `rows` row tiles as many as cover the columns.
__device__ __forceinline__ int rounds(int rows, int columns, int width, int G)
{
    return (rows * ((columns + width - 1) / width) + G - 1) / G;
}

// What a round of tall tiles 256 x 256 takes, and of their halves, quarters and eighths, in 1 / 97 of it.
constexpr int kTallCost = 97, kTallCost2 = 56, kTallCost4 = 37, kTallCost8 = 25;

// Row products (dgrad, 8-bit): tall tiles (more than 128 rows), then the experts' last rows.
//   - Tall tiles are 256 columns wide (the last 128 or fewer: 128), but those of the last round are cut into 256 x 128,
//     128 x 128 or 128 x 64 where the workgroups suffice for all of the parts: a round of parts is shorter.  Or all are 128
//     wide, where that takes less.  Measured (us, the last round whole / halves / quarters / eighths): 528 tiles, 14336
//     deep: 985 / 945 / 855 / 843, 8-bit 542 / 503 / 458 / 452; 32 tiles, 4096 deep: 85 / 63 / 39 / 27, 8-bit 49 / 37 /
//     24 / 17.  (All of 8 x 1024 rows, 4096 x 14336, 256 / 128 wide: 752 / 1038, 8-bit 449 / 547.)
//   - The short ones read the weights for few rows.  A round of tiles 64, 128 and 256 wide takes about 5 : 8 : 15 (narrow
//     ones read the weights in shorter segments and the rows more often); the width is the one with the least.  Measured
//     (us, 64 / 128 / 256 wide): 64 experts x 20 rows, 2048 x 2816: 164 / 137 / 128, 8-bit 100 / 74 / 71; 64 x 100 rows,
//     2048 x 1408: 100 / 82 / 100, 8-bit 51 / 43 / 44; 8 x 30 rows, 2048 x 2048: 16 / 23 / 31, 8-bit 10 / 14 / 19.
template <int KIND>
__device__ __forceinline__ void rows_all(const GroupedArgs &a, GroupedTables &t, bool long_tails, lds_char_t *lds, int wave,
                                         int lane)
{
    const int G = (int)gridDim.x, C = KIND == kI8 ? a.N : a.K;
    const int tall = __builtin_amdgcn_readfirstlane(t.tall[a.E]), low = __builtin_amdgcn_readfirstlane(t.low[a.E]);
    const int full = C / 256, rest = C - full * 256, wide = full + (rest > 128);
    // (Outputs that fit the device have fewer than 2^31 tiles.)
    const int n = tall * wide, last = n % G;   // of the last round
    int cut = 0, cost = last > 0 ? kTallCost : 0;
    if (last * 8 <= G) cut = 3, cost = last > 0 ? kTallCost8 : 0;
    else if (last * 4 <= G) cut = 2, cost = kTallCost4;
    else if (last * 2 <= G) cut = 1, cost = kTallCost2;
    const int whole = n / G * kTallCost + cost + (rest > 0 && rest <= 128 ? rounds(tall, 128, 128, G) * kTallCost2 : 0);
    const bool halves = rounds(tall, C, 128, G) * kTallCost2 < whole;
    const int c256 = rounds(low, C, 256, G) * 15, c128 = rounds(low, C, 128, G) * 8, c64 = rounds(low, C, 64, G) * 5;
    const int width = c256 <= c128 && c256 <= c64 ? 256 : (c128 <= c64 ? 128 : 64);
    // The tiles of a phase are numbered on from the one before, so that workgroups without a tile in one's last round come
    // first in the next.
    int q = xcd_place((int)blockIdx.x, G);
    for (int phase = 0; phase < 4; ++phase) {
        Tiles of{0, wide, 0, 256, false, 0, 0};
        int bm = 256, bn = 256;
        if (phase == 0) {
            if (halves) of.cols = (C + 127) / 128, of.width = bn = 128, of.n = tall * of.cols;
            else of.n = n - last;
        } else if (phase == 1) {
            if (!halves) {
                of.from = n - last, of.cut = cut, of.n = last << cut;
                bm = cut >= 2 ? 128 : 256;
                bn = cut == 0 ? 256 : (cut == 3 ? 64 : 128);
            }
        } else if (phase == 2) {
            if (!halves && rest > 0 && rest <= 128) of = Tiles{tall, 1, full * 256, 128, false, 0, 0}, bn = 128;
        } else {
            of.cols = (C + width - 1) / width;
            of.n = low * of.cols;
            of.low = true;
            bm = long_tails ? 128 : 32;
            bn = width;
        }
        if (of.n == 0) continue;
        if (bm == 256) {
            if (bn == 256) q = rows_tiles<KIND, 256, 256>(a, t, q, of, lds, wave, lane);
            else q = rows_tiles<KIND, 256, 128>(a, t, q, of, lds, wave, lane);
        } else if (bm == 128) {
            if (bn == 256) q = rows_tiles<KIND, 128, 256>(a, t, q, of, lds, wave, lane);
            else if (bn == 128) q = rows_tiles<KIND, 128, 128>(a, t, q, of, lds, wave, lane);
            else q = rows_tiles<KIND, 128, 64>(a, t, q, of, lds, wave, lane);
        } else {
            if (bn == 256) q = rows_tiles<KIND, 32, 256>(a, t, q, of, lds, wave, lane);
            else if (bn == 128) q = rows_tiles<KIND, 32, 128>(a, t, q, of, lds, wave, lane);
            else q = rows_tiles<KIND, 32, 64>(a, t, q, of, lds, wave, lane);
        }
        q -= of.n;
    }
}

// The tasks of the weights' gradient: every expert's full tiles (256 x 256), then its half ones (128 x 256): of the last 128
// or fewer of N, or of all of N where one round holds all of them (8 experts x 512 rows, 1024 x 1024: 12.7 us against 19.8).  Experts with
// the most rows first; every other round goes through the workgroups backwards, so that those with a long task get a short
// one next.  The odd XCDs take their tasks from the last to the first: two places of the matrices are then under way
// (8 x 1024 rows, 4096 x 14336: 853 us against 901 with one; 64 x 768 rows, 2048 x 1408, accumulating: 417 against 437).
struct WgradTasks {
    int nk, full, half, per, n;   // tiles along K; full and half ones along N; tasks an expert, and all of them
    int G, place;
    int rounds;                   // in which this workgroup has a task
    bool backwards;

    __device__ __forceinline__ int dealt(int round) const { return round * G + ((round & 1) ? G - 1 - place : place); }
    __device__ __forceinline__ int task(int round) const { return dealt(backwards ? rounds - 1 - round : round); }
    __device__ __forceinline__ bool is_half(int q) const { return q % per >= nk * full; }
};

// The workgroup's tasks from `round` on, as long as they are tiles of BM rows; returns the first round that is not.
template <int BM, bool GATHER, bool F32>
__device__ __forceinline__ int wgrad_tiles(const GroupedArgs &a, const GroupedTables &t, const WgradTasks &w, int round,
                                           lds_char_t *lds, int wave, int lane0)
{
    typedef GTile<kWgrad, BM, 256, BM == 256 && !GATHER ? 64 : 128> T;
    typedef TileLoads<T, GATHER> TL;
    constexpr int STORES = (F32 ? 4 : 2) * T::NI * T::MI;
    const int64_t ld = (int64_t)a.K * 2;
    int lane = fresh_lane(lane0);
    struct Job {
        int e, n0, k0, row0, cnt;
    };
    auto job_of = [&](int q) {
        const int i = q / w.per, r = q - i * w.per;
        Job j;
        if constexpr (BM == 256) {
            const int group = r / (8 * w.nk), in = r - group * 8 * w.nk, size = min(8, w.full - 8 * group);
            j.k0 = __builtin_amdgcn_readfirstlane(in / size * 256);
            j.n0 = __builtin_amdgcn_readfirstlane((8 * group + in % size) * 256);
        } else {
            const int in = r - w.nk * w.full, row = in / w.nk;
            j.k0 = __builtin_amdgcn_readfirstlane((in - row * w.nk) * 256);
            j.n0 = __builtin_amdgcn_readfirstlane(w.full * 256 + row * 128);
        }
        j.e = __builtin_amdgcn_readfirstlane(t.low[i]);
        j.row0 = __builtin_amdgcn_readfirstlane(t.off[j.e]);
        j.cnt = __builtin_amdgcn_readfirstlane(table_count(t, j.e));
        return j;
    };
    // The rows of `a` of a slab (0 past the expert's: nothing is loaded for those).
    auto toks_of = [&](const Job &j, const TL &tl, int slab, int *ids) {
        if constexpr (GATHER) {
            const int rest = max(0, min(j.cnt - slab * T::L, T::L));
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.row_token + j.row0 + (size_t)slab * T::L, (size_t)rest * 4);
#pragma unroll
            for (int i = 0; i < TL::SP::SLOTS; ++i)
                ids[i] = (int)__builtin_amdgcn_raw_buffer_load_b32(
                    rs, (uint32_t)(tl.p.pos + kGroupedWaves * TL::SP::RPL * i) * 4u, 0, 0);
        }
    };
    auto begin = [&](const Job &j, TL &tl) {
        side_columns(tl.p, (const uint16_t *)a.a + (GATHER ? 0 : (size_t)j.row0 * a.K) + j.k0, (uint64_t)ld, a.K - j.k0,
                     GATHER, wave, lane);
        side_columns(tl.q, a.dy + (size_t)j.row0 * a.N + j.n0, (uint64_t)a.N * 2, a.N - j.n0, false, wave, lane);
        tl.len = j.cnt;
        // with a gather the rows' offsets run through all of `a` (and nothing is read of no rows)
        tl.records_p =
            GATHER ? (a.a_rows > 0 ? (uint32_t)((size_t)a.a_rows * a.K * 2 - (size_t)j.k0 * 2) : 0u) : (uint32_t)kPlainRecords;
        tl.row_bytes = (uint32_t)ld;
        tl.a_rows = a.a_rows;
        static_assert(!GATHER || T::PRE == 1, "the rows of slab 0 alone are known before");
#pragma unroll
        for (int i = 0; i < T::PRE; ++i) tl.load_slab(i);
        toks_of(j, tl, 1, tl.ids);
    };
    Job job = job_of(w.task(round));
    TL tl;
    tl.dst = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds + (uint32_t)wave * 1024u);
    tl.p.pos = wave * TL::SP::RPL + lane / (TL::SP::RB / 16);   // (the same for every tile)
    int ids[GATHER ? TL::SP::SLOTS : 1];
    toks_of(job, tl, 0, tl.ids);
    begin(job, tl);
    for (bool first = true;; first = false) {
        const int nq = w.task(++round);
        const bool more = round < w.rounds && w.is_half(nq) == (BM == 128);
        Job next = job;
        if (more) {
            next = job_of(nq);
            toks_of(next, tl, 0, ids);
        }
        f32x16_t acc[T::NI][T::MI];
        tile_sums<T, GATHER, STORES>(tl, !GATHER && !first, [&](int slab, int *to) { toks_of(job, tl, slab, to); }, lds, wave, lane, acc);
        __syncthreads();   // every wave is done with the stages
        lane = fresh_lane(lane0);
        if (more) {
            if constexpr (GATHER) {
#pragma unroll
                for (int i = 0; i < TL::SP::SLOTS; ++i) tl.ids[i] = ids[i];
            }
            begin(next, tl);
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        const size_t o = ((size_t)job.e * a.N + job.n0) * a.K + job.k0;
        auto value = [&](int i, int k, int v) { return acc[i][k][v]; };
        const int el = fresh_lane(lane0);
        if constexpr (F32)
            store_f32<T>(value, (float *)a.out + o, a.K, a.N - job.n0, a.K - job.k0, a.accumulate, lds, wave, el);
        else store_bf16<T>(value, (uint16_t *)a.out + o, a.K, a.N - job.n0, a.K - job.k0, lds, wave, el);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();   // the outputs have left the stages
        if (!more) break;
        job = next;
    }
    wait_vmem_all();
    return round;
}

}  // namespace

// da = dy W.  Bound by the matrix cores once an expert has some 200 rows, below by reading the weights.  8 x 1024 rows, N =
// 14336, K = 4096: 752 us (1279 TFLOP/s); 64 x 20 rows, N = 2048, K = 2816 (738 MB of weights): 129 us (5.7 TB/s).
__global__ __launch_bounds__(kGroupedThreads, 1) void k_grouped_dgrad(GroupedArgs a)
{
    __shared__ __attribute__((aligned(1024))) char stages[kGroupedStages];
    __shared__ GroupedTables t;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave), lane = (int)threadIdx.x % kWave;
    const TableTotals n = tables_rows(a, t);
    rows_all<kDgrad>(a, t, n.long_tails, (lds_char_t *)stages, wave, lane);
}

// The 8-bit product.  Few rows (512 at most, and hardly more than 16 to an expert: few_width) are a stream of the weights,
// else tiles.  Measured (us, stream / tiles): 8 experts of 4096 x 14336 (470 MB): 1 row each 73 / 110, 16 rows 77 / 111, 24 rows
// (two passes over the weights) 140 / 111.  73 us is 6.4 TB/s (68, 6.9 TB/s, on another card).
// Tiles are bound by the matrix cores: 8 x 1024 rows, K = 4096, N = 14336: 449 us (2140 TOP/s).
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
    static_assert(sizeof(m) <= 160 * 1024, "LDS");
    static_assert(kGroupedStages + offsetof(GroupedTables, scale) <= kGroupedWaves * kFewRing,
                  "the few rows' tables are made from the others");
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave), lane = (int)threadIdx.x % kWave;
    const TableTotals n = tables_rows(a, m.tile.t);
    const int R = __builtin_amdgcn_readfirstlane(m.tile.t.off[a.E]), H = __builtin_amdgcn_readfirstlane(n.hits);
    int width = 0;
    if (R <= kFewRows) {   // (every wave of the launch finds the same)
        int passes = 0, most = 1;
        if (R > kFewGroup) {
            for (int e = lane; e < a.E; e += kWave) {
                const int p = (table_count(m.tile.t, e) + kFewGroup - 1) / kFewGroup;
                passes += p;
                most = max(most, p);
            }
            most = (int)wave_max_u32((uint32_t)most);
            if (most > 1) passes = (int)wave_sum_f32((float)passes);   // (whole numbers below 2^24)
        }
        width = few_width(H, passes, most, a.N, (int)gridDim.x, a.per_grid);
    }
    if (width) {
        few_tables(a, m.tile.t, m.few.t, n.before);
        if (width == 16) few_rows<16>(a, m.few.t, H, (lds_char_t *)m.few.ring, wave, lane);
        else few_rows<32>(a, m.few.t, H, (lds_char_t *)m.few.ring, wave, lane);
    } else {
        rows_all<kI8>(a, m.tile.t, n.long_tails, (lds_char_t *)m.tile.stages, wave, lane);
    }
}

// The weights' gradient.  Bound by the matrix cores in bf16, in fp32 by what is read and written (every XCD with a task of an expert
// reads its rows: 1.4 GB of 0.3 in the shape below), and with few rows an expert by writing dW: 8 x 1024 rows, K = 4096, N =
// 14336: bf16 848 us (1134 TFLOP/s), fp32 986, accumulating 1143, with a gather too 1244; 64 x 768 rows, K = 2048, N = 1408, fp32
// accumulating (738 MB read and written): 411 us.
// Measured and not taken: every task to the workgroup with the least work so far (64 experts by Zipf's law: the longest share is
// 4% over the mean instead of 25%, but the call takes as long, and 5% longer with equal experts: it parts the tasks
// that multiply from those that write).
template <bool GATHER, bool F32>
__global__ __launch_bounds__(kGroupedThreads, 1) void k_grouped_wgrad(GroupedArgs a)
{
    __shared__ __attribute__((aligned(1024))) char stages[kGroupedStages];
    __shared__ GroupedTables t;
    lds_char_t *lds = (lds_char_t *)stages;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave), lane = (int)threadIdx.x % kWave;
    tables_offsets(a, t);
    // The experts in the order of their rows, most first.
    const int padded = (a.E + 3) & ~3;
    int experts = 0;
    for (int e0 = 0; e0 < padded; e0 += kGroupedThreads) {
        const int e = e0 + (int)threadIdx.x;
        const int c = e < a.E ? table_count(t, e) : -1;
        if (e < padded) t.tall[e] = c;
        experts += __syncthreads_count(c > 0);
    }
    for (int e = (int)threadIdx.x; e < a.E; e += kGroupedThreads) {
        const int c = t.tall[e];
        int rank = 0;
#pragma unroll 4
        for (int f = 0; f < padded; f += 4) {
            const int4 d = *(const int4 *)&t.tall[f];
            rank += (d.x > c || (d.x == c && f < e)) + (d.y > c || (d.y == c && f + 1 < e)) +
                    (d.z > c || (d.z == c && f + 2 < e)) + (d.w > c || (d.w == c && f + 3 < e));
        }
        t.low[rank] = e;
    }
    __syncthreads();
    if (!a.accumulate) experts = a.E;   // (those without rows have nothing to add)
    WgradTasks w;
    w.nk = (a.K + 255) / 256;
    w.full = a.N / 256 + (a.N % 256 > 128);
    w.half = a.N % 256 > 0 && a.N % 256 <= 128;
    w.G = (int)gridDim.x;
    if (experts * w.nk * ((a.N + 127) / 128) <= w.G) {
        w.full = 0;
        w.half = (a.N + 127) / 128;
    }
    w.per = w.nk * (w.full + w.half);
    w.n = experts * w.per;
    w.place = xcd_place((int)blockIdx.x, w.G);
    w.rounds = w.n / w.G;
    if (w.dealt(w.rounds) < w.n) ++w.rounds;
    w.backwards = blockIdx.x & 1;
    for (int round = 0; round < w.rounds;) {
        if (w.is_half(w.task(round))) round = wgrad_tiles<128, GATHER, F32>(a, t, w, round, lds, wave, lane);
        else round = wgrad_tiles<256, GATHER, F32>(a, t, w, round, lds, wave, lane);
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
    void (*k)(GroupedArgs) = a.row_token ? (a.out_f32 ? k_grouped_wgrad<true, true> : k_grouped_wgrad<true, false>)
                                         : (a.out_f32 ? k_grouped_wgrad<false, true> : k_grouped_wgrad<false, false>);
    hipLaunchKernelGGL(k, dim3(grid), dim3(kGroupedThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grouped_i8(const GroupedArgs &a, hipStream_t s)
{
    const int grid = persistent_grid();
    if (grid <= 0) return hipErrorInvalidDevice;
    GroupedArgs b = a;
    b.per_grid = inverse_of(grid);
    hipLaunchKernelGGL(k_grouped_i8, dim3(grid), dim3(kGroupedThreads), 0, s, b);
    return hipGetLastError();
}

}  // namespace mk
