// layer_args.h -- arguments and workspace of the few-token MoE layer.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "mk_args.h"

namespace mk {

constexpr int kLayerMaxT = 128;      // tokens per call (two 64-bit token masks per expert)
constexpr int kLayerSelfT = 8;       // tokens up to which the vector router runs and the up kernel selects by itself
constexpr int kLayerSelfE = 256;     // ... and experts, for the selection
constexpr int kQ8Group = 128;        // columns (and rows of weights) per scale
constexpr int kHGroup = 8;           // 8-bit form: features of h per binade

// The up and down kernels' exchange of the waves' sums in LDS: per wave at most kLayerTiles tiles of 256 floats, in halves
// that alternate.  There is one barrier per exchange and none between tasks, so a wave may write the next exchange's sums
// while others still read this one's: the two must not overlap whatever their tile counts are.  A half therefore starts in
// one place for every tile count (a 33 to 64 row expert of the 8-bit down kernel has two tiles where others have four).
constexpr int kLayerWaves = 4;       // per workgroup
constexpr int kLayerTiles = 4;       // weight tiles per task, at most
constexpr int kExchangeHalf = kLayerWaves * kLayerTiles * 256;   // floats
__host__ __device__ constexpr int layer_exchange_at(int par) { return par * kExchangeHalf; }
constexpr int kExchangeBytes = 2 * kExchangeHalf * 4;

// What the up kernel's first workgroup writes for the later ones: the experts with tokens in ascending order (per expert
// the tokens ascend, row by row), and the row of every choice.
struct LayerRec {
    int32_t e, row0, cnt, pad;       // local expert, its first row, its rows
};
struct LayerPlan {
    int32_t *n;                      // [2] experts with tokens, valid tokens
    LayerRec *rec;                   // [min(E_local, T k)]
    int32_t *row_of;                 // [T, k] row of the choice in h and y, or -1
    int32_t *done;                   // [d / 16] finished down tasks of each column block, zeroed (layer_sums_in_down)
};

struct LayerArgs {
    const uint16_t *x;               // [T, d] bf16: router input, and the experts' in the bf16 form
    const uint8_t *xq;               // [T, d] e4m3 (8-bit form)
    const float *xs;                 // [T, d / 128]
    const void *w_gu, *w_dn;         // [E_local, 2F, d], [E_local, d, F]: bf16 or e4m3
    const float *s_gu, *s_dn;        // [E_local, 2 ceil(F / 128), d / 128], [E_local, d / 128, ceil(F / 128)]
    const int32_t *ids;              // [T, k] given or selected ids (what the up kernel reads unless it selects)
    const float *gates;              // [T, k]
    LayerPlan plan;
    int32_t *ids_user;               // NULL or [T, k]: copies for the caller
    float *w_user;
    float *part;                     // [8, T, E] router partial sums
    const float *wr, *bias;          // router
    void *h;                         // gate * silu(g) * u, rows in expert order (store_h in layer.hip)
    uint8_t *hx;                     // 8-bit form: the binades of h
    float *y;                        // [T min(k, E_local), d]: the rows' products with W_down
    uint16_t *out;                   // [T, d] bf16
    const int32_t *t_valid;          // NULL or the number of tokens to compute (device)
    int32_t T, d, E, k, e_begin, E_local, F;
    int32_t given;                   // ids came from the caller: they may repeat
};

__host__ __device__ inline int layer_rows_cap(int T, int k, int E_local) { return T * (k < E_local ? k : E_local); }
__host__ __device__ inline int layer_hits_cap(int T, int k, int E_local) { return E_local < T * k ? E_local : T * k; }

// A few choices: the down kernel adds the rows up itself, one launch fewer (whole calls in a captured graph, the sum in a
// kernel of its own against in the down kernel: one token at 6 experts of e4m3 26.3 -> 25.6 us, d = F = 512 14.8 -> 14.4, a
// Mixtral-shaped token 118.8 -> 118.6).  With more the wait for other workgroups' rows costs more than the launch (8 tokens
// with 64 choices of 32 experts: 109.8 -> 111.9 us, with 48 of 64 small ones 107.7 -> 109.6, of e4m3 68.9 -> 71.1).
constexpr int kFewChoices = 32;
__host__ __device__ inline bool layer_sums_in_down(int T, int k) { return T <= kLayerSelfT && T * k <= kFewChoices; }

// Bytes of a row of h (store_h in layer.hip): bf16 weights 2 F values twice, 8-bit ones whole blocks of 128 fp16 values, with
// 16 binades per block in a row of hx.
__host__ __device__ inline uint32_t layer_h_blocks(int F) { return (uint32_t)(F + kQ8Group - 1) / kQ8Group; }
__host__ __device__ inline uint32_t layer_h_row_bytes(bool q8, int F)
{
    return q8 ? 2 * kQ8Group * layer_h_blocks(F) : 4 * (uint32_t)F;
}
__host__ __device__ inline uint32_t layer_hx_row_bytes(int F) { return kQ8Group / kHGroup * layer_h_blocks(F); }

}  // namespace mk
