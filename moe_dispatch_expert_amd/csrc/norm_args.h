// norm_args.h -- arguments of the residual addition + RMS norm kernel.
#pragma once

#include <stdint.h>

namespace mk {

constexpr int kNormMaxD = 32768;   // a workgroup of 1024 threads holds the row: 4 pieces of 8 columns each

struct NormArgs {
    const uint16_t *x, *res, *gamma;   // [T, d] bf16, [T, d] bf16 or nullptr, [d] bf16
    uint16_t *res_out, *y;             // [T, d] bf16 or nullptr
    uint8_t *q;                        // [T, d] e4m3 or nullptr
    float *qs;                         // [T, d / 128], with q
    int32_t T, d;
    float eps;
};

}  // namespace mk
