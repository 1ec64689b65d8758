// grouped_few.h -- the 8-bit grouped product of a few rows an expert: a stream of the hit experts' weights.
//
// A workgroup's eight waves split the contraction: wave w takes slabs w, w + 8, ... (128 bytes of each row) of WR weight
// rows and up to 16 rows of codes.  Every wave keeps a ring of its own in LDS, three slabs deep, filled straight from memory
// (8 rows x 128 bytes a load) and waited for by the wave's own load counter, so there is no barrier in the stream and the
// stream does not stop at the end of a task: the loads run up to three slabs ahead, into the next task.  The sums are
// whole numbers, so the waves add theirs up in LDS with atomics, in any order, to the same result; one barrier a task, two
// buffers in turn.  What a task needs besides the stream lies in LDS: rows' tokens and scales from the start, its
// columns' scales loaded with its first slab.
// Bound by memory: 8 experts of 4096 x 14336 (470 MB), 1 row each: 68 to 73 us, 6.4 to 6.9 TB/s; one such matrix and one
// row: 13 us, of which the launch, the tables and the first loads' way are 5.
#pragma once

#include "grouped_dev.h"

namespace mk {

constexpr int kFewStages = 3;
constexpr int kFewStageBytes = (32 + kFewGroup) * 128;
constexpr int kFewRing = kFewStages * kFewStageBytes;       // one wave's

struct FewTables {
    uint16_t off[kGroupedMaxE + 2];
    uint16_t hit[kGroupedMaxE];        // the experts with rows
    int32_t tok[kFewRows];             // row of `a`, or -1
    float scale[kFewRows];
    int32_t sum[2][kFewGroup * 32];    // a task's sums: [row][column]
    float ws[8][64];                   // columns' scales of the next tasks
};

typedef int32_t few_acc_t __attribute__((ext_vector_type(4)));

// A place in a workgroup's stream: task q (weight tile q % tiles of the (q / tiles)-th hit expert), group g of 16 of its
// rows; item counts the groups passed.
struct FewPlace {
    int q, e, n0, r0, rows, g, item;   // r0: the expert's first row; rows: how many
};

template <int WR>
struct FewStream {
    const GroupedArgs &a;
    const FewTables &t;
    int tasks, tiles, G;

    __device__ __forceinline__ void enter(FewPlace &p) const
    {
        const int h = (int)((uint32_t)p.q / (uint32_t)tiles);
        p.e = __builtin_amdgcn_readfirstlane((int)t.hit[h]);
        p.n0 = __builtin_amdgcn_readfirstlane((p.q - h * tiles) * WR);
        p.r0 = __builtin_amdgcn_readfirstlane((int)t.off[p.e]);
        p.rows = __builtin_amdgcn_readfirstlane((int)t.off[p.e + 1]) - p.r0;
    }
    // The next group of rows, or task; false past the last one.
    __device__ __forceinline__ bool next(FewPlace &p) const
    {
        ++p.item;
        if ((p.g + 1) * kFewGroup < p.rows) {
            ++p.g;
            return true;
        }
        p.g = 0;
        p.q += G;
        if (p.q >= tasks) return false;
        enter(p);
        return true;
    }
};

template <int WR>
__device__ __forceinline__ void few_rows(const GroupedArgs &a, FewTables &t, int hits, lds_char_t *lds, int wave, int lane)
{
    constexpr int WL = WR / 8, XL = kFewGroup / 8, NL = WL + XL;   // loads a slab
    constexpr int NB = WR / 16;
    const int KK = (a.K + 127) / 128;
    const int tiles = (a.N + WR - 1) / WR;
    const FewStream<WR> st{a, t, hits * tiles, tiles,   // at most 1024 x 65536
                            (int)gridDim.x};
    FewPlace in;   // what is computed
    in.q = xcd_place((int)blockIdx.x, (int)gridDim.x);
    in.g = in.item = 0;
    if (in.q >= st.tasks) return;
    st.enter(in);
    FewPlace ld = in;   // what is loaded
    bool more = true;
    int ld_slab = wave;

    lds_char_t *ring = lds + wave * kFewRing;
    // 16-byte chunk c of LDS row r lies at c ^ ((r >> 1) & 7); load i covers rows 8 i .. 8 i + 7
    int pos[2];
#pragma unroll
    for (int par = 0; par < 2; ++par) pos[par] = ((lane & 7) ^ ((4 * par + (lane >> 4)) & 7)) * 16;
    rsrc4_t rw, rx, rs;
    uint32_t wo[WL], xo[XL], so;
    // resources and offsets of the task that is loaded next
    auto aim = [&]() {
        rw = make_rsrc4((const int8_t *)a.w + ((size_t)ld.e * a.N + ld.n0) * a.K, (size_t)0x80000000u);
#pragma unroll
        for (int i = 0; i < WL; ++i) {
            const int n = 8 * i + (lane >> 3);
            wo[i] = ld.n0 + n < a.N ? (uint32_t)n * (uint32_t)a.K + pos[i & 1] : kPastResource;
        }
        if (a.row_token) rx = make_rsrc4(a.a, (size_t)a.a_rows * a.K);
        else rx = make_rsrc4((const int8_t *)a.a + (size_t)ld.r0 * a.K, (size_t)0x80000000u);
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int m = ld.g * kFewGroup + 8 * i + (lane >> 3);
            xo[i] = kPastResource;
            if (m < ld.rows) {
                const int row = a.row_token ? t.tok[ld.r0 + m] : m;
                if (row >= 0) xo[i] = (uint32_t)row * (uint32_t)a.K + pos[i & 1];
            }
        }
        rs = make_rsrc4(a.w_scale + (size_t)ld.e * a.N + ld.n0, (size_t)0x80000000u);
        so = lane < WR && ld.n0 + lane < a.N ? (uint32_t)lane * 4u : kPastResource;
    };
    aim();
    int stage = 0;   // of the next load
    auto load = [&]() {
        const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(ring + stage * kFewStageBytes));
        if (more && ld_slab == 0)
            lds_load4(rs, __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char_t *)&t.ws[ld.item & 7][0]), so);
        const int rest = more ? a.K - ld_slab * 128 : 0;
        const uint32_t k0 = __builtin_amdgcn_readfirstlane((uint32_t)ld_slab * 128u);
#pragma unroll
        for (int i = 0; i < WL; ++i) lds_load16<true>(rw, at + i * 1024, pos[i & 1] < rest ? wo[i] : kPastResource, k0);
#pragma unroll
        for (int i = 0; i < XL; ++i)
            lds_load16(rx, at + (32 + 8 * i) * 128, pos[i & 1] < rest ? xo[i] : kPastResource, k0);
        stage = stage == kFewStages - 1 ? 0 : stage + 1;
        ld_slab += kGroupedWaves;
        if (more && ld_slab >= KK) {
            more = st.next(ld);
            ld_slab = wave;
            if (more) aim();
        }
    };
    // A wave without a slab in the tasks (KK < 8) still loads, and multiplies nothing.
    const bool idle = wave >= KK;
#pragma unroll
    for (int s = 0; s < kFewStages; ++s) load();
    int rd = 0;   // stage that is computed next
    int fo[2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) fo[kk] = (lane & 15) * 128 + (((4 * kk + (lane >> 4)) ^ (((lane & 15) >> 1) & 7)) << 4);
    for (;;) {
        few_acc_t acc[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[n] = few_acc_t{0, 0, 0, 0};
        for (int slab = wave; slab < KK; slab += kGroupedWaves) {
            __builtin_amdgcn_sched_barrier(0);
            wait_vmem<(kFewStages - 1) * NL>();
            __builtin_amdgcn_sched_barrier(0);
            const lds_char_t *b = ring + __builtin_amdgcn_readfirstlane(rd * kFewStageBytes);
            i32x4_t fw[2][NB], fx[2];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                for (int n = 0; n < NB; ++n) fw[kk][n] = *(lds_ci32x4_t *)(b + n * 16 * 128 + fo[kk]);
                fx[kk] = *(lds_ci32x4_t *)(b + 32 * 128 + fo[kk]);
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the stage has been read
            __builtin_amdgcn_sched_barrier(0);
            load();
            rd = rd == kFewStages - 1 ? 0 : rd + 1;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    acc[n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[kk][n], fx[kk], acc[n], 0, 0, 0);
        }
        // lane: row lane % 16 of the group, columns 16 n + 4 (lane / 16) + v
        int32_t *sum = t.sum[in.item & 1];
        if (!idle && in.g * kFewGroup + (lane & 15) < in.rows) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    atomicAdd(&sum[(lane & 15) * 32 + 16 * n + 4 * (lane >> 4) + v], acc[n][v]);
        }
        __syncthreads();
        const int ti = (int)threadIdx.x, m = ti / WR, n = ti % WR;
        const int r = in.g * kFewGroup + m;
        if (m < kFewGroup && r < in.rows) {
            const int32_t s = sum[m * 32 + n];
            sum[m * 32 + n] = 0;
            if (in.n0 + n < a.N)
                ((uint16_t *)a.out)[(size_t)(in.r0 + r) * a.N + in.n0 + n] =
                    f32_to_bf16((float)s * t.ws[in.item & 7][n] * t.scale[in.r0 + r]);
        }
        if (!st.next(in)) break;
    }
    wait_vmem_all();   // no load may land in this memory once the workgroup is gone
}

// The tables of this form: rows' tokens and scales, experts with rows (before: how many lie before the thread's two), sums of
// zero.  g: the offsets, whose place the tables may take.
__device__ __forceinline__ void few_tables(const GroupedArgs &a, const GroupedTables &g, FewTables &t, int before)
{
    const int ti = (int)threadIdx.x, e = 2 * ti, R = g.off[a.E];
    int off[3];
#pragma unroll
    for (int h = 0; h < 3; ++h) off[h] = g.off[min(e + h, a.E)];
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (e + h <= a.E) t.off[e + h] = (uint16_t)off[h];
        if (e + h < a.E && off[h + 1] > off[h]) t.hit[before++] = (uint16_t)(e + h);
    }
    if (e + 2 == a.E) t.off[a.E] = (uint16_t)off[2];
    for (int r = ti; r < R; r += kGroupedThreads) {
        const int v = a.row_token ? a.row_token[r] : r;
        const bool ok = v >= 0 && v < a.a_rows;
        t.tok[r] = ok ? v : -1;
        t.scale[r] = ok ? a.a_scale[v] : 0.0f;
    }
    for (int i = ti; i < 2 * kFewGroup * 32; i += kGroupedThreads) t.sum[0][i] = 0;
    __syncthreads();
}

}  // namespace mk
