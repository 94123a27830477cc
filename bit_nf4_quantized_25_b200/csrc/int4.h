// int4.h -- internal launchers of the 4-bit integer weights with group scales. Not part of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace qn {

// W is n x k, k % group == 0, k % 64 == 0; group is 32, 64 or 128 consecutive weights of a row.
struct Int4View {
    int64_t n, k;
    int group;
    uint8_t *codes;       // n * k / 2, low nibble first
    uint16_t *scale;      // n * k / group, bf16
    uint8_t *zero_point;  // n * k / group, or nullptr: 8 for every group
};

cudaError_t launch_int4_quantize(const uint16_t *W, const Int4View &w, cudaStream_t st);
cudaError_t launch_int4_dequantize(const Int4View &w, uint16_t *out, cudaStream_t st);

// h = dequant(W) x, kInt4Tokens tokens (8 for very large k) per launch, k <= kInt4LinearMaxK.
constexpr int kInt4Tokens = 16;
constexpr int64_t kInt4LinearMaxK = 65536;
cudaError_t launch_int4_linear(const Int4View &w, const uint16_t *x, int M, uint16_t *h, cudaStream_t st);

}  // namespace qn
