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
    uint32_t per_grid;          // 8-bit: inverse_of the workgroups
};

// 8-bit product with a gather: where the tokens of a tile's rows lie in their table, by the tile's parity in a workgroup's run.
// The next tile's tokens are loaded from the start of a tile's products on, without a barrier after the reads of the first
// tile's own, so two tiles that follow one another have places of their own.
constexpr int kTokenRows = 256;                      // rows of the tallest tile
constexpr int kTokenTable = 2 * kTokenRows;
__host__ __device__ constexpr int tile_tokens_at(int parity) { return (parity & 1) * kTokenRows; }

// 8-bit product: the stream of the weights for few rows (grouped_few.h) against the tiles.
constexpr int kFewRows = 512;   // rows the stream takes (its tables)
constexpr int kFewGroup = 16;   // rows a pass over a weight tile

// ceil(n / G) as a product with inv = inverse_of(G): shorter than the divisions that the compiler makes, of code that runs once
// a launch.  Exact below 2^32 / G, and for every G that is a power of two; above, it may be one more.
__host__ __device__ constexpr uint32_t inverse_of(int G) { return (uint32_t)((((uint64_t)1 << 32) + G - 1) / G); }
__host__ __device__ inline int rounds_of(int n, int G, uint32_t inv)
{
    return (int)(((uint64_t)(uint32_t)(n + G - 1) * inv) >> 32);
}

// Rows of a weight tile (32, or 16 where that leaves the workgroup with the most tasks less to read) with which G workgroups
// stream the weights of H experts with rows, or 0 for the tiles.  passes: the experts' passes of kFewGroup rows together; most: of
// the expert with the most.  A workgroup goes through the passes of its weight tiles one after another, so what counts is the
// busiest one's: its share of all tiles, and beyond that the longest expert's other passes or the mean of all others, whichever is
// more.  The stream is taken for at most 10 / 7 of the passes that one a tile would be (3 for 2), or if no more weight rows are
// read one after another than the tiles' narrowest form has.  Measured (us, stream / tiles):
//   32 experts of 2816 x 2048, a row each but for one of 17: 33 / 41, of 64: 37 / 44, of 128: 45 / 44, of 256: 64 / 47, of 480:
//   98 / 48; 16 of 17 rows and 16 of 2: 45 / 41;  32 of 2048 x 1408, 16 rows each: 26 / 23 (the one case of a pass each that loses);
//   8 of 14336 x 4096, a row each but for one of 17: 82 / 110, of 64: 100 / 117, of 96: 118 / 118, of 128: 136 / 118;
//   8 of 2048 x 2048, of 17: 13 / 15, of 48: 17 / 14;  one of 4096 x 14336, 17 rows: 23 / 38, 48: 35 / 42, 64: 45 / 44, 128: 85 / 56;
//   one of 14336 x 4096, 16 rows: 17 / 20, 17: 25 / 20.
__host__ __device__ inline int few_width(int H, int passes, int most, int N, int G, uint32_t inv)
{
    const int t32 = (N + 31) / 32, t16 = (N + 15) / 16;
    const int once32 = rounds_of(H * t32, G, inv), once16 = rounds_of(H * t16, G, inv);
    const bool narrow = once16 < 2 * once32;
    const int width = narrow ? 16 : 32, tiles = narrow ? t16 : t32, once = narrow ? once16 : once32;
    if (most <= 1) return width;
    const int longest = (most - 1) * rounds_of(tiles, G, inv), mean = rounds_of((passes - H) * tiles, G, inv);
    const int busiest = once + (longest > mean ? longest : mean);
    return 7 * busiest <= 10 * once + 1 || busiest * width <= 64 ? width : 0;
}

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
