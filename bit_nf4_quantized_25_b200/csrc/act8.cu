// act8.cu -- activations kept in 8 bits for the backward pass (act8.cuh has the format), and the SwiGLU
// of the MLP with gate and up kept that way:
//
//   forward   y = g sigma(g) u                           reads bf16 g, u; writes y and the 8-bit g, u
//   backward  dg = dy u sigma (1 + g (1 - sigma)), du = dy g sigma,  sigma = 1 / (1 + exp(-g))
//             from the 8-bit g, u; and y again, rounded to bf16 and then to 8 bits, which is the input
//             that the next layer's adapter gradients want
//
// Everything is elementwise but the absmax of 64 neighbours, so every kernel here is bound by HBM:
// 3.03 B per value to quantise or read back, 8.06 B for the SwiGLU forward, 9.09 B for its backward.
// A block is 8 lanes x 8 values: each lane's accesses are whole 16-byte (bf16) or 8-byte (codes) words,
// neighbouring lanes' are contiguous, and the absmax takes three shuffles. A row's length is a multiple
// of 64, so blocks never straddle rows and the tensor is walked as one flat array. Each thread takes
// kUnroll words, all loaded before the first is used.
//
// Measured at 4096 x 11008, on three sets of buffers in turn: quantise 22.7 us, read back 22.6 us (6.0 TB/s, 0.93 of the
// measured HBM rate), SwiGLU forward 60.5 us (6.0 TB/s), backward 72.7 us (5.6 TB/s, 0.87; its issue slots are 82 % busy).
#include "act8.cuh"
#include "act8.h"
#include "dependent.cuh"

namespace qn {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void decode8(const uint2 &q, float s, float (&f)[8]) {
    float a[4], b[4];
    act8::decode4(q.x, a);
    act8::decode4(q.y, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = a[i] * s;
        f[4 + i] = b[i] * s;
    }
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ float reciprocal(float v) {  // of 1 .. 2^126, by the hardware's
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// sigma(g) = e / (1 + e) below 0 and 1 / (1 + e) from 0 on, with e = exp(-|g|) <= 1, so that no gate leads out of the
// reciprocal's range. By the hardware exponential, of a rounded argument, and reciprocal it is off by at most
// (4 + 1.2 |g|) 2^-23 of itself, below 2^-16 in all of fp32's normal range and far below the bf16 rounding of the results;
// below 2^-126 it is a multiple of 2^-149.
__device__ __forceinline__ float sigmoid(float g) {
    const float e = __expf(-fabsf(g));
    return (g < 0.0f ? e : 1.0f) * reciprocal(1.0f + e);
}

// The same for |g| up to about kNear, three instructions less.
constexpr uint32_t kNear = 0x42aeu;  // 87 in bf16: exp(87.3) is 2^126
__device__ __forceinline__ float sigmoid_near(float g) { return reciprocal(1.0f + __expf(-g)); }

template <int kUnroll>
__global__ void __launch_bounds__(kThreads) k_act8_quantize(const uint16_t *x, int64_t words, int8_t *codes,
                                                            uint16_t *absmax) {
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
    begin_dependent();
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        v[u] = i < words ? ld_nc_v4(x + act8::kPer * i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        act8::store_block(v[u], i < words, i, codes, absmax);
    }
}

template <int kUnroll>
__global__ void __launch_bounds__(kThreads) k_act8_dequantize(const int8_t *codes, const uint16_t *absmax,
                                                              int64_t words, uint16_t *x) {
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
    begin_dependent();
    uint2 q[kUnroll];
    uint32_t top[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        const bool live = i < words;
        q[u] = live ? ld_nc_v2(codes + act8::kPer * i) : make_uint2(0u, 0u);
        top[u] = live ? ld_nc_u16(absmax + i / act8::kLanes) : 0u;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        if (i >= words) continue;
        float f[8];
        decode8(q[u], act8::step(top[u]), f);
        *reinterpret_cast<uint4 *>(x + act8::kPer * i) = pack8(f);
    }
}

template <int kUnroll>
__global__ void __launch_bounds__(kThreads) k_swiglu_act8_fwd(const uint16_t *gate, const uint16_t *up, int64_t words,
                                                              uint16_t *y, int8_t *gq, uint16_t *ga, int8_t *uq,
                                                              uint16_t *ua) {
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
    begin_dependent();
    uint4 g[kUnroll], w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        const bool live = i < words;
        g[u] = live ? ld_nc_v4(gate + act8::kPer * i) : make_uint4(0u, 0u, 0u, 0u);
        w[u] = live ? ld_nc_v4(up + act8::kPer * i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        const bool live = i < words;
        float a[8], b[8], f[8];
        unpack8(g[u], a);
        unpack8(w[u], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = a[e] * sigmoid(a[e]) * b[e];
        if (live) *reinterpret_cast<uint4 *>(y + act8::kPer * i) = pack8(f);
        act8::store_block(g[u], live, i, gq, ga);
        act8::store_block(w[u], live, i, uq, ua);
    }
}

template <int kUnroll>
__global__ void __launch_bounds__(kThreads) k_swiglu_act8_bwd(const int8_t *gq, const uint16_t *ga, const int8_t *uq,
                                                              const uint16_t *ua, const uint16_t *grad_y,
                                                              int64_t words, uint16_t *grad_gate, uint16_t *grad_up,
                                                              int8_t *yq, uint16_t *ya) {
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
    begin_dependent();
    uint4 d[kUnroll];
    uint2 g[kUnroll], w[kUnroll];
    uint32_t gt[kUnroll], ut[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        const bool live = i < words;
        d[u] = live ? ld_nc_v4(grad_y + act8::kPer * i) : make_uint4(0u, 0u, 0u, 0u);
        g[u] = live ? ld_nc_v2(gq + act8::kPer * i) : make_uint2(0u, 0u);
        w[u] = live ? ld_nc_v2(uq + act8::kPer * i) : make_uint2(0u, 0u);
        gt[u] = live ? ld_nc_u16(ga + i / act8::kLanes) : 0u;
        ut[u] = live ? ld_nc_u16(ua + i / act8::kLanes) : 0u;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        const bool live = i < words;
        float a[8], b[8], dy[8], dg[8], du[8], f[8];
        decode8(g[u], act8::step(gt[u]), a);
        decode8(w[u], act8::step(ut[u]), b);
        unpack8(d[u], dy);
        // Issuing instructions bounds the kernel, so blocks of ordinary gates do without sigmoid's other half: at
        // 4096 x 11008 72.7 us against 75.1.
        float sg[8];
        if (gt[u] <= kNear) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sg[e] = sigmoid_near(a[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) sg[e] = sigmoid(a[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float sig = sg[e], sl = a[e] * sig;
            dg[e] = dy[e] * b[e] * sig * (1.0f + a[e] * (1.0f - sig));
            du[e] = dy[e] * sl;
            f[e] = sl * b[e];
        }
        if (live) {
            *reinterpret_cast<uint4 *>(grad_gate + act8::kPer * i) = pack8(dg);
            *reinterpret_cast<uint4 *>(grad_up + act8::kPer * i) = pack8(du);
        }
        if (yq) act8::store_block(pack8(f), live, i, yq, ya);
    }
}

// CTAs for `words` words at kUnroll per thread; 0 when there are more than a grid holds.
unsigned grid_for(int64_t words, int unroll) {
    const int64_t per = static_cast<int64_t>(kThreads) * unroll, ctas = (words + per - 1) / per;
    return ctas > 0x7fffffffLL ? 0u : static_cast<unsigned>(ctas);
}

}  // namespace

cudaError_t launch_act8_quantize(const uint16_t *x, int64_t count, int8_t *codes, uint16_t *absmax, cudaStream_t st) {
    const int64_t words = count / act8::kPer;
    const unsigned grid = grid_for(words, 4);
    if (grid == 0) return cudaErrorInvalidConfiguration;
    return launch_dependent(k_act8_quantize<4>, grid, kThreads, st, x, words, codes, absmax);
}

cudaError_t launch_act8_dequantize(const int8_t *codes, const uint16_t *absmax, int64_t count, uint16_t *x,
                                   cudaStream_t st) {
    const int64_t words = count / act8::kPer;
    const unsigned grid = grid_for(words, 4);
    if (grid == 0) return cudaErrorInvalidConfiguration;
    return launch_dependent(k_act8_dequantize<4>, grid, kThreads, st, codes, absmax, words, x);
}

cudaError_t launch_swiglu_act8_fwd(const uint16_t *gate, const uint16_t *up, int64_t count, uint16_t *y,
                                   int8_t *gate_codes, uint16_t *gate_absmax, int8_t *up_codes, uint16_t *up_absmax,
                                   cudaStream_t st) {
    const int64_t words = count / act8::kPer;
    const unsigned grid = grid_for(words, 2);
    if (grid == 0) return cudaErrorInvalidConfiguration;
    return launch_dependent(k_swiglu_act8_fwd<2>, grid, kThreads, st, gate, up, words, y, gate_codes, gate_absmax, up_codes,
                            up_absmax);
}

cudaError_t launch_swiglu_act8_bwd(const int8_t *gate_codes, const uint16_t *gate_absmax, const int8_t *up_codes,
                                   const uint16_t *up_absmax, const uint16_t *grad_y, int64_t count,
                                   uint16_t *grad_gate, uint16_t *grad_up, int8_t *y_codes, uint16_t *y_absmax,
                                   cudaStream_t st) {
    const int64_t words = count / act8::kPer;
    const unsigned grid = grid_for(words, 2);
    if (grid == 0) return cudaErrorInvalidConfiguration;
    return launch_dependent(k_swiglu_act8_bwd<2>, grid, kThreads, st, gate_codes, gate_absmax, up_codes, up_absmax, grad_y, words,
                            grad_gate, grad_up, y_codes, y_absmax);
}

}  // namespace qn
