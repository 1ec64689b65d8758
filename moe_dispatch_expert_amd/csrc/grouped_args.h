// grouped_args.h -- arguments of the backward and 8-bit kernels around the grouped product.
#pragma once

#include <stdint.h>

namespace mk {

constexpr int kGroupedMaxE = 1024;          // experts: their offsets are scanned in LDS
constexpr int kGroupedMaxDim = 1 << 20;     // N and K: a tile's 256 rows then stay inside 32-bit offsets
constexpr int kGroupedMaxRows = 0x7FFFFFFF - 4095;   // the ends of an expert's last tile and slabs then have 32 bits too
constexpr int kI8MaxK = 131072;             // 131072 products of -128 * -128 would pass int32
constexpr int kQuantMaxD = 32768;           // a workgroup of 1024 threads holds the row: 4 pieces of 8 columns each

// Rows of expert e: [offsets[e], offsets[e + 1]), clamped to [0, rows).  With row_token, row r of the product reads row
// row_token[r] of the a_rows rows of `a` (a value outside them reads zeros).
struct GroupedArgs {
    const int32_t *offsets;     // [E + 1]
    const int32_t *row_token;   // [rows] or nullptr
    int32_t E, rows, a_rows, N, K;
    const uint16_t *dy;         // dgrad, wgrad: [rows, N] bf16
    const void *a;              // wgrad: [rows or a_rows, K] bf16;  8-bit: the same, int8 codes
    const void *w;              // dgrad: [E, N, K] bf16;  8-bit: the same, int8 codes
    const float *a_scale;       // 8-bit: [rows or a_rows]
    const float *w_scale;       // 8-bit: [E, N]
    void *out;                  // dgrad [rows, K] bf16;  wgrad [E, N, K] fp32 or bf16;  8-bit [rows, N] bf16
    int32_t out_f32, accumulate;
};

// 8-bit product with a gather: where the tokens of a tile's rows lie in their table, by the tile's parity in a workgroup's run.
// The next tile's tokens are loaded from the start of a tile's products on, without a barrier after the reads of the first
// tile's own, so two tiles that follow one another have places of their own.
constexpr int kTokenRows = 256;                      // rows of the tallest tile
constexpr int kTokenTable = 2 * kTokenRows;
__host__ __device__ constexpr int tile_tokens_at(int parity) { return (parity & 1) * kTokenRows; }

struct CombineBackwardArgs {
    const uint16_t *dout, *y;   // [T, N], [rows, N] bf16
    const int32_t *slot_of;     // [T, k]
    const float *gate;          // [T, k]
    uint16_t *dy;               // [rows, N]
    float *dgate;               // [T, k] or nullptr
    int32_t T, k, N, rows;
};

struct SwigluBackwardArgs {
    const uint16_t *gu, *dh;    // [rows, 2F], [rows, F] bf16
    const int32_t *rows_valid;  // nullptr or one int32
    uint16_t *dgu, *h;          // [rows, 2F];  [rows, F] or nullptr
    int32_t rows, F;
};

struct QuantArgs {
    const uint16_t *x;          // [rows, d] bf16;  SwiGLU form: [rows, 2 d], gate then up
    const int32_t *rows_valid;  // nullptr or one int32
    int8_t *q;                  // [rows, d]
    float *scale;               // [rows]
    int32_t rows, d;
};

// Choices are taken in chunks (multiples of 64, at most kLayoutChunks of them), one workgroup each.
constexpr int kLayoutChunks = 128;
struct LayoutArgs {
    const int32_t *ids;         // [T, k]
    int32_t *counts;            // [chunks, E]: choices of the chunk by expert
    int32_t *offsets;           // [E + 1]
    int32_t *slot_of;           // [T, k]
    int32_t *row_token;         // [T * k] or nullptr
    int32_t n, k, e_begin, E;   // n = T * k choices
    int32_t chunk, chunks;      // choices per chunk, and how many chunks
};

}  // namespace mk
