// grouped_dev.h -- the tile of the grouped product's gradients (bf16) and of its 8-bit form, on gfx950 matrix cores.
//
// A workgroup of eight waves computes BM rows x BN columns of
//   out[m, n] = sum_l Q[m, l] P[n, l]
// P is the matrix instructions' A operand, so a lane ends with four neighbouring columns of a row.  The three products
// differ in which index of an operand is contiguous in memory:
//   dgrad  out = da,    P[i, n] = W[e, n, i] (rows along the contraction),  Q[r, n] = dy[r, n] (contraction contiguous)
//   wgrad  out = dW[e], P[i, r] = a[r, i] and Q[n, r] = dy[r, n] (rows along the contraction both)
//   8-bit  out = y,     P[n, i] = w[e, n, i] and Q[r, i] = a[r, i] (contraction contiguous both)
// The contraction runs in slabs of 64 bf16 or 128 int8 (wgrad's full tile with rows in place: 32), straight from memory into
// LDS (buffer_load ... lds, 1 KiB a load), into a ring of two to eight stages; four matrix instruction steps a slab (32 rows:
// two), the fragments of step s + 1 read during the products of step s, one barrier a slab, before its last step.
//   - Contraction contiguous: LDS rows of 128 bytes, 16-byte chunk c of row r at c ^ ((r >> 1) & 7); a fragment is one
//     16-byte read.
//   - Rows along the contraction: 64 LDS rows of 2 C bytes; a fragment is two transposing reads (ds_read_b64_tr_b16: 16
//     lanes hold 4 rows x 16 columns and each gets a column's 4 values).  16-byte unit u of row r lies at u ^ 4 (r & 3)
//     (C = 64: u ^ 4 ((r >> 1) & 1)), so that the 4 rows x 64 bytes that 32 lanes read lie on different banks.
// Every load is checked lane by lane against the tile's rows or columns and the slab's rest of the contraction: a lane
// outside gets an offset past the resource, which reads zeros without a memory access, so ragged ends add exact zeros
// whatever lies behind them.
// A tile's first slabs are loaded before the outputs of the tile before it are stored (these go through the upper half of
// the stages' LDS).
// Bound by the matrix cores: 256 x 256 with 8 waves is the largest tile whose sums (128 registers a lane) and fragments stay in
// registers; a slab of it takes 1.6 us (bf16), and beginning and ending a tile 5.3 us, of which the stores are 2.7.  8192^3, one
// matrix (us and rate): dgrad 808 (1360 TFLOP/s), wgrad 812 (1354), 8-bit 432 (2550 TOP/s); large library products reach 1377
// and 2083 on such a card.  Measured and not taken (the same, or 8 x 1024 rows of 4096 x 14336): four waves of 128 x 128 (no
// gain), sums in accumulation registers (8-bit 4% slower: moves and spills), 64-byte slabs for dgrad and 8-bit (3% slower),
// lines asked for 3 to 6 slabs ahead by 4-byte loads (7% slower: the address unit is what is scarce).
#pragma once

#include "gemm_dev.h"
#include "grouped_args.h"

namespace mk {

enum { kDgrad = 0, kWgrad = 1, kI8 = 2 };

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));
typedef int16_t i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
typedef __attribute__((address_space(3))) const i32x4_t lds_ci32x4_t;

constexpr int kGroupedThreads = 512, kGroupedWaves = 8;
constexpr int kGroupedStages = 131072;              // LDS of the stages; the outputs pass through its upper half
constexpr int kPlainRecords = (int)0x80000000u;     // of resources whose offsets all lie below 2 GiB

// A tile of BM rows by BN columns, the waves WN along the columns and WM along the rows (of small tiles several waves
// compute the same: they are bound by memory).
template <int KIND_, int BM_, int BN_, int KB_ = 128>
struct GTile {
    static constexpr int KIND = KIND_, BM = BM_, BN = BN_;
    static constexpr int KB = KB_, STEPS = KB / 32;                  // bytes of an operand's row in a slab, instruction steps
    static constexpr int WN = BM == 256 ? 2 : (BM == 128 ? (BN == 64 ? 2 : 4) : BN / 32);
    static constexpr int WM = BM == 32 ? 1 : kGroupedWaves / WN;
    static constexpr int NI = BN / WN / 32, MI = BM / WM / 32;
    static constexpr bool PKR = KIND != kI8, QKR = KIND == kWgrad;   // rows along the contraction
    static constexpr int ESZ = KIND == kI8 ? 1 : 2;                  // bytes of an element
    static constexpr int L = KB / ESZ;                               // contraction per slab
    static constexpr int PB = BN * KB, QB = (BM > 64 ? BM : 64) * KB, SB = PB + QB;     // bytes of a stage
    static constexpr int S = kGroupedStages / SB < 8 ? kGroupedStages / SB : 8;         // stages
    static constexpr int PRE0 = kGroupedStages / 2 / SB;                                // of them in the lower half of the LDS,
    static constexpr int PRE = PRE0 < S ? PRE0 : S;                                     // loaded before outputs are stored
    static_assert(NI >= 1 && MI >= 1 && WN * WM <= kGroupedWaves && S >= 2 && SB <= kGroupedStages / 2, "tile shape");
};

// The lane as a value of its own: what a tile computes from it stays in the tile, or in its epilogue.  (Otherwise the compiler
// keeps the offsets of every tile shape in registers throughout the task loop, and spills the tile's.)
__device__ __forceinline__ int fresh_lane(int lane)
{
    asm volatile("" : "+v"(lane));
    return lane;
}

// What the lanes of a wave hand one another through LDS: no instruction, but the compiler keeps the order, and the lanes
// together.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One operand of a tile: C rows (or columns) of it, and this lane's part of its loads.
template <bool KR, int C, int KB>
struct Side {
    static constexpr int RB = 2 * C;                         // KR: bytes of an LDS row
    static constexpr int RPL = 1024 / RB;                    // KR: rows a load
    static constexpr int SLOTS = KR ? KB / 2 / RPL / kGroupedWaves : (C / 8 + kGroupedWaves - 1) / kGroupedWaves;
    static_assert(KR ? C >= 64 && SLOTS >= 1 : KB == 128, "row swizzle");
    uint32_t off[SLOTS];   // byte offsets in the resource (kPastResource: nothing to read)
    int pos;               // place in the slab: KR the row of slot 0, else the byte
    uint64_t base;         // KR: of the next slab to load
    uint64_t step;         // KR: bytes between slabs
    rsrc4_t rs;            // not KR: the resource
};

// Contraction contiguous: LDS block b = wave + 8 slot holds rows 8 b .. 8 b + 7; row(r, i) gives the byte offset of the
// operand's row r (slot i), or kPastResource.
template <class S, class F>
__device__ __forceinline__ void side_rows(S &s, rsrc4_t rs, int wave, int lane, F &&row)
{
    const uint32_t c = dma_chunk_bytes(wave, lane);
#pragma unroll
    for (int i = 0; i < S::SLOTS; ++i) {
        const uint32_t o = row((wave + kGroupedWaves * i) * 8 + (lane >> 3), i);
        s.off[i] = o == kPastResource ? o : o + c;
    }
    s.pos = (int)c;
    s.rs = rs;
}

// Rows along the contraction: LDS block b = wave + 8 slot holds rows b RPL ..; base: the tile's first column of row 0,
// ld: bytes between rows, cols: columns there are.  (gather: off holds the column's part alone.)
template <class S>
__device__ __forceinline__ void side_columns(S &s, const void *base, uint64_t ld, int cols, bool gather, int wave, int lane)
{
    constexpr int UPR = S::RB / 16;
    const int r0 = lane / UPR;   // row of the block
    // (8 RPL is a multiple of 4, so the swizzle is the same in every slot)
    const int r4 = (S::RPL * wave + r0) & 3;
    const int u = (lane % UPR) ^ ((UPR == 8 ? r4 >> 1 : r4) << 2);
#pragma unroll
    for (int i = 0; i < S::SLOTS; ++i) {
        const int row = (wave + kGroupedWaves * i) * S::RPL + r0;
        s.off[i] = u * 8 < cols ? (gather ? 0u : (uint32_t)row * (uint32_t)ld) + (uint32_t)u * 16u : kPastResource;
    }
    s.pos = wave * S::RPL + r0;
    s.base = (uint64_t)base;
    s.step = (uint64_t)(kGroupedWaves * S::RPL * S::SLOTS) * ld;
}

__device__ __forceinline__ rsrc4_t slab_rsrc(uint64_t base, uint32_t records)
{
    return rsrc4_t{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)base),
                   (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(base >> 32) & 0xFFFFu), records, 0x00020000u};
}

// This lane's offset for load slot i of a slab; rest: what is left of the contraction from the slab's start (rows of KR, else
// bytes; <= 0: nothing).  tok (GATHER): this lane's row of `a`, which
// has a_rows of them.
template <bool GATHER, bool KR, int C, int KB>
__device__ __forceinline__ uint32_t side_offset(const Side<KR, C, KB> &s, int i, int rest, int tok, int a_rows,
                                                 uint32_t row_bytes)
{
    uint32_t o = s.off[i];
    bool ok = s.pos + (KR ? kGroupedWaves * Side<KR, C, KB>::RPL * i : 0) < rest;
    if constexpr (GATHER) {
        ok = ok & ((uint32_t)tok < (uint32_t)a_rows) & (o != kPastResource);
        o += (uint32_t)tok * row_bytes;
    }
    return ok ? o : kPastResource;
}

// One 4-byte load a lane into LDS byte lds_addr + 4 lane.
__device__ __forceinline__ void lds_load4(rsrc4_t rsrc, uint32_t lds_addr, uint32_t voff)
{
    asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "{m0}"(lds_addr));
}

// Where this lane's fragments start in a stage.  Contraction contiguous: by step of the slab; rows along it: by block of
// 32 columns (block q of the operand: q0 + index).
template <bool KR, int C, int KB, int NB>
__device__ __forceinline__ void frag_bases(lds_char_t *stage, int q0, int lane, lds_char_t *(&b)[4])
{
    b[0] = b[1] = b[2] = b[3] = stage;
    if constexpr (KR) {
        constexpr int RB = 2 * C;
        const int i = lane & 15;
        const int row = 8 * (lane >> 5) + (i >> 2);
        const int low = (2 * ((lane >> 4) & 1) + ((i & 3) >> 1)) * 16 + 8 * (i & 1);
        const int sw = C == 64 ? i >> 3 : i >> 2;   // the swizzle of rows row and row + 4
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int q = q0 + n;
            int o = row * RB + ((q & ~3) << 6) + (((q & 3) ^ sw) << 6) + low;
            asm volatile("" : "+v"(o));   // computed once, kept in a register
            b[n] = stage + o;
        }
    } else {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            int o = (lane & 31) * 128 + (((2 * kk + (lane >> 5)) ^ (((lane & 31) >> 1) & 7)) << 4);
            asm volatile("" : "+v"(o));
            b[kk] = stage + q0 * 32 * 128 + o;
        }
    }
}

// Half t of fragment n of step kk from the stage that b points into (t = 0 alone with the contraction contiguous).
template <bool KR, int C, int KB>
__device__ __forceinline__ void read_half(lds_char_t *const (&b)[4], int n, int t, int kk, i32x4_t &f)
{
    if constexpr (KR) {
        const i16x4_t v =
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(b[n] + (16 * kk + 4 * t) * 2 * C));
        const u32x2_t w = __builtin_bit_cast(u32x2_t, v);
        f[2 * t] = (int32_t)w[0];
        f[2 * t + 1] = (int32_t)w[1];
    } else {
        f = *(lds_ci32x4_t *)(b[kk] + n * 32 * 128);
    }
}

template <int KIND>
struct Acc {
    typedef f32x16_t type;
};
template <>
struct Acc<kI8> {
    typedef i32x16_t type;
};

__device__ __forceinline__ void product(i32x4_t p, i32x4_t q, f32x16_t &acc)
{
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, p), __builtin_bit_cast(bf16x8_t, q), acc,
                                                  0, 0, 0);
}
__device__ __forceinline__ void product(i32x4_t p, i32x4_t q, i32x16_t &acc)
{
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(p, q, acc, 0, 0, 0);
}

// What the loads of a tile need: its operands, the contraction's length in elements, and for a gather the rows of `a` of
// the next slab to load (ids), P's resource size and its rows' bytes.
template <class T, bool GATHER>
struct TileLoads {
    typedef Side<T::PKR, T::BN, T::KB> SP;
    typedef Side<T::QKR, T::BM, T::KB> SQ;
    static constexpr int NL = SP::SLOTS + SQ::SLOTS;   // loads a slab
    SP p;
    SQ q;
    int len;
    int ids[GATHER ? SP::SLOTS : 1];
    int a_rows;
    uint32_t records_p, row_bytes;
    rsrc4_t rp, rq;
    uint32_t dst;   // LDS address of this wave's first block of stage 0

    // The resources of the next slab (in order: 0, 1, ...).
    __device__ __forceinline__ void next_slab()
    {
        if constexpr (T::PKR) {
            rp = slab_rsrc(p.base, records_p);
            if constexpr (!GATHER) p.base += p.step;
        } else {
            rp = p.rs;
        }
        if constexpr (T::QKR) {
            rq = slab_rsrc(q.base, kPlainRecords);
            q.base += q.step;
        } else {
            rq = q.rs;
        }
    }
    // This lane's offsets for a slab, then its load i; stage: LDS address of the wave's first block of the stage.
    __device__ __forceinline__ uint32_t offset(int i, int slab) const
    {
        const int rest = len - slab * T::L;
        return i < SP::SLOTS
                   ? side_offset<GATHER>(p, i, T::PKR ? rest : rest * T::ESZ, GATHER ? ids[GATHER ? i : 0] : 0, a_rows,
                                          row_bytes)
                   : side_offset<false>(q, i - SP::SLOTS, T::QKR ? rest : rest * T::ESZ, 0, 0, 0u);
    }
    __device__ __forceinline__ void aim(int slab, uint32_t (&at)[NL]) const
    {
#pragma unroll
        for (int i = 0; i < NL; ++i) at[i] = offset(i, slab);
    }
    __device__ __forceinline__ void load(int i, const uint32_t (&at)[NL], int slab, uint32_t stage) const
    {
        const bool isp = i < SP::SLOTS;
        const uint32_t to = __builtin_amdgcn_readfirstlane(
            stage + (isp ? 0u : (uint32_t)T::PB) + (uint32_t)(kGroupedWaves * 1024 * (isp ? i : i - SP::SLOTS)));
        const uint32_t k0 = (isp ? T::PKR : T::QKR) ? 0u : __builtin_amdgcn_readfirstlane((uint32_t)(slab * T::KB));
        lds_load16(isp ? rp : rq, to, at[i], k0);
    }
    __device__ __forceinline__ void load_slab(int slab)
    {
        uint32_t at[NL], to = dst;
        // (the addresses are computed here: kept for the whole task loop they would be spilled, and a reload waits for every
        // load on its way)
        asm volatile("" : "+s"(to));
        next_slab();
        aim(slab, at);
#pragma unroll
        for (int i = 0; i < NL; ++i) load(i, at, slab, to + (uint32_t)(slab * T::SB));
    }
};

// The sums of a tile whose first PRE slabs are on their way into the stages, with STORES memory operations or more after them
// (stored: else none): acc[i][j], lane: column 32 i + 8 (v / 4) + 4 (lane / 32) + v % 4 of the wave's columns, row
// 32 j + lane % 32 of its rows.  toks(slab, ids): the rows of `a` that this lane loads of a slab (with a gather; those of
// slab PRE have been asked for).  On return every load is done, but waves may still read the stages.
template <class T, bool GATHER, int STORES, class TOK>
__device__ __forceinline__ void tile_sums(TileLoads<T, GATHER> &tl, bool stored, TOK &&toks, lds_char_t *lds, int wave,
                                          int lane, typename Acc<T::KIND>::type (&acc)[T::NI][T::MI])
{
    constexpr int NH = T::PKR ? 2 : 1, MH = T::QKR ? 2 : 1;    // reads a fragment
    constexpr int NR = T::NI * NH + T::MI * MH;                // reads a step
    constexpr int NM = T::NI * T::MI;                          // products a step
    constexpr int NL = TileLoads<T, GATHER>::NL, S = T::S, SB = T::SB;
    const int wn = wave % T::WN, wm = wave / T::WN % T::WM;
#pragma unroll
    for (int i = 0; i < T::NI; ++i)
#pragma unroll
        for (int j = 0; j < T::MI; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
    const int KK = __builtin_amdgcn_readfirstlane((tl.len + T::L - 1) / T::L);
    lds_char_t *bp[4], *bq[4];
    frag_bases<T::PKR, T::BN, T::KB, T::NI>(lds, wn * T::NI, lane, bp);
    frag_bases<T::QKR, T::BM, T::KB, T::MI>(lds + T::PB, wm * T::MI, lane, bq);
    // (the places of memory operations matter to the counts below)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = T::PRE; s < S; ++s) {
        tl.load_slab(s);
        if constexpr (GATHER) toks(s + 1, tl.ids);
    }
    // Slab 0 is here: of what came after it, (S - 1) slabs and the stores may be on their way (with a gather also tokens:
    // then less is).
    __builtin_amdgcn_sched_barrier(0);
    if (stored) wait_vmem<(S - 1) * NL + STORES>();
    else wait_vmem<(S - 1) * NL>();
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();

    i32x4_t fp0[T::NI], fq0[T::MI], fp1[T::NI], fq1[T::MI];
    // read r of a step, in the order in which the products need them: P 0, the Q, the other P
    auto rd = [&](int r, int kk, i32x4_t (&fp)[T::NI], i32x4_t (&fq)[T::MI]) {
        if (r < NH) read_half<T::PKR, T::BN, T::KB>(bp, 0, r, kk, fp[0]);
        else if (r < NH + T::MI * MH) read_half<T::QKR, T::BM, T::KB>(bq, (r - NH) / MH, (r - NH) % MH, kk, fq[(r - NH) / MH]);
        else {
            const int n = (r - T::MI * MH) / NH;
            read_half<T::PKR, T::BN, T::KB>(bp, n, (r - T::MI * MH) % NH, kk, fp[n]);
        }
    };
    // the products of a step on (fp, fq), with the reads of the next one and a slab's loads spread over them
    auto step = [&](const i32x4_t (&fp)[T::NI], const i32x4_t (&fq)[T::MI], auto &&reads, int nld, auto &&loads) {
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            product(fp[q / T::MI], fq[q % T::MI], acc[q / T::MI][q % T::MI]);
#pragma unroll
            for (int i = q * nld / NM; i < (q + 1) * nld / NM; ++i) loads(i);
#pragma unroll
            for (int r = q * NR / NM; r < (q + 1) * NR / NM; ++r) reads(r);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
#pragma unroll
    for (int r = 0; r < NR; ++r) rd(r, 0, fp0, fq0);
    auto none = [](int) {};
    // Slab j in stage j % S; slab j + S goes into the stage during the last step.  After the last slab the same steps read a
    // stage that nothing was loaded into, and their loads have nothing left to read: cheaper than forms of their own, whose
    // different exits cost copies of the sums.
    int cur = 0;   // stage
    uint32_t stage = tl.dst;
    for (int j = 0; j < KK; ++j) {
        step(fp0, fq0, [&](int r) { rd(r, 1, fp1, fq1); }, 0, none);
        if constexpr (T::STEPS == 4) {
            step(fp1, fq1, [&](int r) { rd(r, 2, fp0, fq0); }, 0, none);
            step(fp0, fq0, [&](int r) { rd(r, 3, fp1, fq1); }, 0, none);
        }
        uint32_t at[NL];
        tl.next_slab();
        // With a gather one by one among the products instead: the tokens were asked for after the loads that are waited for
        // below, and all at once after that the offsets would hold up the products.
        if constexpr (!GATHER) tl.aim(j + S, at);
        // vmcnt: slab j + 1 is here; lgkmcnt(0): so are the last step's fragments
        __builtin_amdgcn_s_waitcnt((((S - 2) * NL) & 15) | ((((S - 2) * NL) >> 4) << 14) | 0x0070);
        __syncthreads();
        const int to = __builtin_amdgcn_readfirstlane(cur == S - 1 ? -(S - 1) * SB : SB);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            bp[n] += to;
            bq[n] += to;
        }
        step(fp1, fq1, [&](int r) { rd(r, 0, fp0, fq0); }, NL, [&](int i) {
            if constexpr (GATHER) at[i] = tl.offset(i, j + S);
            tl.load(i, at, j + S, stage);
        });
        if constexpr (GATHER) toks(j + S + 1, tl.ids);
        stage = __builtin_amdgcn_readfirstlane(stage + (uint32_t)to);
        cur = cur == S - 1 ? 0 : cur + 1;
    }
    // A distance between the last product and the first read of its sums that does not depend on the schedule (see
    // gemm_tile_big); no load may still be on its way into LDS.
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7");
#pragma unroll
    for (int i = 0; i < T::NI; ++i)
#pragma unroll
        for (int k = 0; k < T::MI; ++k) asm volatile("" : "+v"(acc[i][k]));
    __builtin_amdgcn_sched_barrier(0);
    wait_vmem_all();
}

// Stores a wave's part of a tile through 8 KiB of LDS of its own, so that memory sees whole segments: 64 NI bytes of bf16 a
// row, 32 rows at a time.  2 NI MI stores a wave, whatever is outside (those are dropped by their offset).
template <class T, class F>
__device__ __forceinline__ void store_bf16(F &&value, uint16_t *out, int ldc, int rows, int cols, lds_char_t *lds, int wave,
                                           int lane)
{
    constexpr int RB = 64 * T::NI, CH = RB / 16;          // bytes and 16-byte chunks of a wave's row
    constexpr int RPI = 64 / CH;                          // rows an instruction
    lds_char_t *mine = lds + kGroupedStages / 2 + wave * 8192;
    const int wn = wave % T::WN, wm = wave / T::WN;       // (a wave past the tile's rows stores nothing)
    const int w = lane & 31, c = lane % CH, n = wn * (T::BN / T::WN) + 8 * c;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(out, (size_t)0x80000000u);
#pragma unroll
    for (int j = 0; j < T::MI; ++j) {
#pragma unroll
        for (int i = 0; i < T::NI; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                typedef __attribute__((address_space(3))) u32x2_t lds_u32x2_t;
                *(lds_u32x2_t *)(mine + w * RB + (((4 * i + g) ^ (w & (CH - 1))) << 4) + ((lane >> 5) << 3)) =
                    u32x2_t{pack_bf16x2(value(i, j, 4 * g), value(i, j, 4 * g + 1)),
                            pack_bf16x2(value(i, j, 4 * g + 2), value(i, j, 4 * g + 3))};
            }
        wave_sync();
        const int m0 = wm * (T::BM / T::WM) + 32 * j;
#pragma unroll
        for (int r = 0; r < 32; r += RPI) {
            const int m = r + lane / CH;
            const v4i_t v = *(__attribute__((address_space(3))) const v4i_t *)(mine + m * RB + ((c ^ (m & (CH - 1))) << 4));
            const uint32_t at = (uint32_t)(m0 + m) * (uint32_t)(ldc * 2) + (uint32_t)n * 2u;
            __builtin_amdgcn_raw_buffer_store_b128(v, rs, m0 + m < rows && n < cols ? at : kPastResource, 0, kStoreNT);
        }
        wave_sync();
    }
}

// (Through LDS because the width of a store matters: wgrad of 8 x 1024 rows, 4096 x 14336, in fp32 took 1194 us with 32 bytes a
// row from the registers, 1177 with 64, 1108 with 256 and 1035 with 512.)
// The same in fp32, 16 rows at a time (4 NI MI stores a wave), added to what is there where add is set.
template <class T, class F>
__device__ __forceinline__ void store_f32(F &&value, float *out, int ldc, int rows, int cols, bool add, lds_char_t *lds,
                                          int wave, int lane)
{
    constexpr int RB = 128 * T::NI, CH = RB / 16, RPI = 64 / CH, NS = 16 / RPI;
    lds_char_t *mine = lds + kGroupedStages / 2 + wave * 8192;
    const int wn = wave % T::WN, wm = wave / T::WN;
    const int w = lane & 15, c = lane % CH, n = wn * (T::BN / T::WN) + 4 * c;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(out, (size_t)0x80000000u);
#pragma unroll
    for (int j = 0; j < T::MI; ++j) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int m0 = wm * (T::BM / T::WM) + 32 * j + 16 * hf;
            uint32_t at[NS];
            f32x4_t o[NS];
#pragma unroll
            for (int b = 0; b < NS; ++b) {
                const int m = m0 + b * RPI + lane / CH;
                at[b] = m < rows && n < cols ? (uint32_t)m * (uint32_t)(ldc * 4) + (uint32_t)n * 4u : kPastResource;
            }
            if (add) {
#pragma unroll
                for (int b = 0; b < NS; ++b)
                    o[b] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, at[b], 0, kStoreNT));
            }
            if (((lane >> 4) & 1) == hf) {
#pragma unroll
                for (int i = 0; i < T::NI; ++i)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        typedef __attribute__((address_space(3))) f32x4_t lds_f32x4_t;
                        *(lds_f32x4_t *)(mine + w * RB + (((8 * i + 2 * g + (lane >> 5)) ^ w) << 4)) =
                            f32x4_t{value(i, j, 4 * g), value(i, j, 4 * g + 1), value(i, j, 4 * g + 2), value(i, j, 4 * g + 3)};
                    }
            }
            wave_sync();
#pragma unroll
            for (int b = 0; b < NS; ++b) {
                const int m = b * RPI + lane / CH;
                f32x4_t v = *(__attribute__((address_space(3))) const f32x4_t *)(mine + m * RB + ((c ^ m) << 4));
                if (add) v += o[b];
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i_t, v), rs, at[b], 0, kStoreNT);
            }
            wave_sync();
        }
    }
}

// ------------------------------------------------------------------------------------------------ which tiles there are

// Tables of a launch, in LDS behind the stages.  Every workgroup makes them from the offsets.
struct GroupedTables {
    __attribute__((aligned(16))) int32_t tall[kGroupedMaxE + 4];   // rows of tiles: how many of more than 128 rows lie before
                                       // expert e ... (wgrad: the experts' rows)
    int32_t off[kGroupedMaxE + 1];     // clamped offsets
    int32_t low[kGroupedMaxE + 1];     // ... and how many short ones (the rest of an expert, if 128 rows or fewer);
                                       // wgrad: low[i] = the expert with the i-th most rows
    uint64_t wave_sum[kGroupedWaves];
    float scale[2][2][256];            // 8-bit: scales of a tile's rows and columns, of two tiles in turn
    int32_t tok[kTokenTable];          // 8-bit: rows of `a` of two tiles in turn (tile_tokens_at)
};
static_assert(kGroupedStages + sizeof(GroupedTables) <= 160 * 1024, "LDS");

__device__ __forceinline__ void tables_offsets(const GroupedArgs &a, GroupedTables &t)
{
    // (no offset past the last one: the few rows' tables have as many places)
    const int end = min(max(a.offsets[a.E], 0), a.rows);
    for (int e = (int)threadIdx.x; e <= a.E; e += kGroupedThreads) t.off[e] = min(max(a.offsets[e], 0), end);
    __syncthreads();
}

// Rows of expert e (offsets that do not ascend, which the caller must not give, count as no rows).
__device__ __forceinline__ int table_count(const GroupedTables &t, int e) { return max(t.off[e + 1] - t.off[e], 0); }

struct TableTotals {
    int before, hits;   // experts with rows: those before the thread's two (experts 2 ti and 2 ti + 1), and all of them
    bool long_tails;    // a short tile of more than 32 rows
};

// Tall and short row tiles of every expert.
__device__ __forceinline__ TableTotals tables_rows(const GroupedArgs &a, GroupedTables &t)
{
    tables_offsets(a, t);
    const int ti = (int)threadIdx.x, lane = ti % kWave, wave = ti / kWave;
    // one scan of three sums in a word: short tiles (16 bits), experts with rows (16), tall tiles (32)
    uint64_t n[2], sum = 0;
    bool long_tail = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = 2 * ti + h;
        const int cnt = e < a.E ? table_count(t, e) : 0, rest = cnt % 256;
        n[h] = ((uint64_t)(uint32_t)(cnt / 256 + (rest > 128)) << 32) | ((uint32_t)(cnt > 0) << 16) |
               (uint32_t)(rest > 0 && rest <= 128);
        long_tail |= rest > 32 && rest <= 128;
        sum += n[h];
    }
    const bool long_tails = __syncthreads_or(long_tail);
    uint64_t inc = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const uint64_t v = __shfl_up((unsigned long long)inc, d);
        if (lane >= d) inc += v;
    }
    if (lane == kWave - 1) t.wave_sum[wave] = inc;
    __syncthreads();
    uint64_t at = inc - sum, all = 0;
    for (int w = 0; w < kGroupedWaves; ++w) {
        const uint64_t v = t.wave_sum[w];
        at += w < wave ? v : 0;
        all += v;
    }
    const int before = (int)((uint32_t)at >> 16);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = 2 * ti + h;
        if (e < a.E) {
            t.tall[e] = (int32_t)(at >> 32);
            t.low[e] = (int32_t)((uint32_t)at & 0xFFFFu);
        }
        at += n[h];
    }
    if (ti == 0) {
        t.tall[a.E] = (int32_t)(all >> 32);
        t.low[a.E] = (int32_t)((uint32_t)all & 0xFFFFu);
    }
    __syncthreads();
    return TableTotals{before, (int)((uint32_t)all >> 16), long_tails};
}

// The expert of tile row q of a prefix table (the last e with pre[e] <= q).
__device__ __forceinline__ int table_expert(const int32_t *pre, int E, int q)
{
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= q) lo = mid;
        else hi = mid;
    }
    return lo;
}

struct GroupedJob {
    int e, row0, rows, col0;
};

// Tall tile q of the rows' products, of cols column tiles of BN: expert by expert, in groups of up to 8 row tiles that go
// through the columns together (the 32 workgroups of an XCD then share 8 row tiles and 4 column tiles in its L2).
__device__ __forceinline__ GroupedJob tall_job(const GroupedArgs &a, const GroupedTables &t, int cols, int BN, int q)
{
    GroupedJob j;
    const int e = table_expert(t.tall, a.E, (int)((uint32_t)q / (uint32_t)cols));
    const int r = q - t.tall[e] * cols;
    const int n = t.tall[e + 1] - t.tall[e];
    const int group = r / (8 * cols), in = r - group * 8 * cols;
    const int size = min(8, n - 8 * group);
    const int row = (8 * group + in % size) * 256;
    j.e = __builtin_amdgcn_readfirstlane(e);
    j.col0 = __builtin_amdgcn_readfirstlane(in / size * BN);
    j.rows = __builtin_amdgcn_readfirstlane(min(table_count(t, e) - row, 256));
    j.row0 = __builtin_amdgcn_readfirstlane(t.off[e] + row);
    return j;
}

// Short tile q: the last rows of an expert.
__device__ __forceinline__ GroupedJob low_job(const GroupedArgs &a, const GroupedTables &t, int cols, int BN, int q)
{
    GroupedJob j;
    const int i = (int)((uint32_t)q / (uint32_t)cols);
    const int e = table_expert(t.low, a.E, i);
    const int row = (t.tall[e + 1] - t.tall[e]) * 256;
    j.e = __builtin_amdgcn_readfirstlane(e);
    j.col0 = __builtin_amdgcn_readfirstlane((q - i * cols) * BN);
    j.rows = __builtin_amdgcn_readfirstlane(table_count(t, e) - row);
    j.row0 = __builtin_amdgcn_readfirstlane(t.off[e] + row);
    return j;
}

// Place of workgroup w among G (a multiple of 8): the workgroups of one XCD (w % 8) take neighbouring tasks.
__device__ __forceinline__ int xcd_place(int w, int G) { return (w % 8) * (G / 8) + w / 8; }

}  // namespace mk
