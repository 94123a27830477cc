// act8.h -- internal launchers of the 8-bit activation checkpoints. Not part of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace qn {

// An activation of `count` values (a multiple of 64) in 8 bits: int8 codes and the bf16 absmax of
// each 64 consecutive values.
cudaError_t launch_act8_quantize(const uint16_t *x, int64_t count, int8_t *codes, uint16_t *absmax, cudaStream_t st);
cudaError_t launch_act8_dequantize(const int8_t *codes, const uint16_t *absmax, int64_t count, uint16_t *x,
                                   cudaStream_t st);

// y = silu(gate) * up; gate and up also in 8 bits.
cudaError_t launch_swiglu_act8_fwd(const uint16_t *gate, const uint16_t *up, int64_t count, uint16_t *y,
                                   int8_t *gate_codes, uint16_t *gate_absmax, int8_t *up_codes, uint16_t *up_absmax,
                                   cudaStream_t st);
// The gradients of gate and up from their 8-bit forms; y again in 8 bits when y_codes is not null.
cudaError_t launch_swiglu_act8_bwd(const int8_t *gate_codes, const uint16_t *gate_absmax, const int8_t *up_codes,
                                   const uint16_t *up_absmax, const uint16_t *grad_y, int64_t count,
                                   uint16_t *grad_gate, uint16_t *grad_up, int8_t *y_codes, uint16_t *y_absmax,
                                   cudaStream_t st);

// Adapter gradients (fp32) with the input in 8 bits: grad_A (r x k), grad_B (n x r); M, n, k > 0. The workspace
// holds t = x A^T and u = grad_h B.
size_t act8_grads_workspace_bytes(int64_t M, int64_t n, int r);
cudaError_t launch_act8_grads(const int8_t *codes, const uint16_t *absmax, const uint16_t *gh, int64_t M, int64_t n,
                              int64_t k, const uint16_t *A, const uint16_t *B, int r, float s, const DropoutArgs &drop,
                              float *grad_A, float *grad_B, void *ws, cudaStream_t st);

// The same on the 5th-generation tensor cores, for long batches. The workspace also holds copies of grad_h and B with
// padded rows where TMA cannot read theirs (n % 8, r % 8). give_up (with a dropout): waits of the second kernel run out.
size_t act8_grads_tc_workspace_bytes(int64_t M, int64_t n, int r);
cudaError_t launch_act8_grads_tc(const int8_t *codes, const uint16_t *absmax, const uint16_t *gh, int64_t M, int64_t n,
                                 int64_t k, const uint16_t *A, const uint16_t *B, int r, float s,
                                 const DropoutArgs &drop, float *grad_A, float *grad_B, void *ws, cudaStream_t st,
                                 bool give_up = false);

}  // namespace qn
