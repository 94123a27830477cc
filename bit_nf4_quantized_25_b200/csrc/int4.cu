// int4.cu -- weights as 4-bit integers with a scale per group of 32, 64 or 128 consecutive weights of a
// row, and back to bf16. A weight is s (q - z): s bf16, q and z integers 0..15.
//
//   with zero points: lo = min(0, min w), hi = max(0, max w), s = bf16(fl32((hi - lo) / 15)),
//                     z = clamp(round(-lo / s), 0, 15)
//   symmetric:        s = bf16(fl32(max |w| / 7)), z = 8
//   q = clamp(round(w / s) + z, 0, 15), rounding to nearest with halves away from zero; a group whose s is
//   0 has q = z.
//
// Both directions are bound by HBM: 2 B and 0.5 B + 2 or 3 B per group for each weight. A lane takes 8
// weights (one 16-byte word of W, one 4-byte word of codes); a group is 4, 8 or 16 neighbouring lanes,
// which share its minimum and maximum by shuffles. k % group == 0, so groups do not straddle rows and
// the matrix is walked as one flat array.
#include "common.cuh"
#include "dependent.cuh"
#include "int4.h"

namespace qn {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it leaves an integer in the low mantissa bits

// Scale, zero point and codes of a lane's 8 weights; all lanes of the warp call it.
//
// The quotient w / s is taken as w inv with inv = fl32((1 + 2^-17) / s): w and s have 8-bit
// significands, so a quotient that is not a half is at least 1 / 512 of a unit away from one, and one
// that is a half is raised above it by more than the rounding of inv; at up to 16 units the raise is
// below 2^-13. An fma onto 1.5 * 2^23 + z then gives round(w / s) + z with halves away from zero.
template <int kGroup, bool kZero>
__device__ __forceinline__ uint32_t encode(const uint4 &v, uint32_t &scale_bits, int &zero) {
    constexpr int kLanes = kGroup / 8;
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    float w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[2 * i] = bf16_lo(u[i]);
        w[2 * i + 1] = bf16_hi(u[i]);
    }
    float lo = 0.0f, hi = 0.0f;  // kZero: minimum and maximum with 0; else hi is max |w|
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (kZero) lo = fminf(lo, w[i]);
        hi = fmaxf(hi, kZero ? w[i] : fabsf(w[i]));
    }
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) {
        if (kZero) lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
    }
    float span = hi - lo;
    if (kZero && span > 3.4028235e38f) span = 2.0f * __fdiv_rn(0.5f * hi - 0.5f * lo, 15.0f);  // hi - lo overflowed
    else span = __fdiv_rn(span, kZero ? 15.0f : 7.0f);
    scale_bits = __bfloat16_as_ushort(__float2bfloat16_rn(span));
    float s = __uint_as_float(scale_bits << 16);
    if (s == 0.0f) {
        zero = kZero ? 0 : 8;
        return kZero ? 0u : 0x88888888u;
    }
    if (s < 0x1p-100f) {  // keep 1 / s finite: w / s of both times 2^64, exact
        s *= 0x1p64f;
        lo *= 0x1p64f;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] *= 0x1p64f;
    }
    const float inv = __fdiv_rn(0x1.0001p+0f, s);
    zero = 8;
    if (kZero) zero = min(static_cast<int>(__float_as_uint(__fmaf_rn(-lo, inv, kMagic)) - 0x4b400000u), 15);
    const float base = kMagic + static_cast<float>(zero);
    uint32_t word = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int q = static_cast<int>(__float_as_uint(__fmaf_rn(w[i], inv, base)) - 0x4b400000u);
        word |= static_cast<uint32_t>(min(max(q, 0), 15)) << (4 * i);
    }
    return word;
}

template <int kGroup, bool kZero>
__global__ void __launch_bounds__(kThreads) k_int4_quantize(const uint16_t *W, int64_t words, uint32_t *codes,
                                                            uint16_t *scale, uint8_t *zero_point) {
    constexpr int kLanes = kGroup / 8;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
    begin_dependent();
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        v[u] = i < words ? ld_nc_v4(W + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        uint32_t sb;
        int z;
        const uint32_t word = encode<kGroup, kZero>(v[u], sb, z);
        if (i >= words) continue;
        codes[i] = word;
        if ((threadIdx.x & (kLanes - 1)) == 0) {
            scale[i / kLanes] = static_cast<uint16_t>(sb);
            if (kZero) zero_point[i / kLanes] = static_cast<uint8_t>(z);
        }
    }
}

// The largest finite bf16 in place of a product above it: the step nearest to a weight near the end of the
// range may lie past it.
__device__ __forceinline__ float saturate(float v) {
    constexpr float kMax = 0x1.fep+127f;
    return v > kMax ? kMax : v < -kMax ? -kMax : v;
}

// s (q - z) is exact in fp32 (8 bits times 5); one rounding, to bf16.
__global__ void __launch_bounds__(kThreads) k_int4_dequantize(const uint32_t *codes, const uint16_t *scale,
                                                              const uint8_t *zero_point, int64_t words, int shift,
                                                              uint16_t *out) {
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
    begin_dependent();
    uint32_t c[kUnroll];
    float s[kUnroll], z[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        const bool live = i < words;
        c[u] = live ? ld_nc_u32(codes + i) : 0u;
        s[u] = __uint_as_float((live ? ld_nc_u16(scale + (i >> shift)) : 0u) << 16);
        z[u] = live && zero_point ? static_cast<float>(ld_nc_u8(zero_point + (i >> shift))) : 8.0f;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        if (i >= words) continue;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = s[u] * (static_cast<float>((c[u] >> (4 * e)) & 15u) - z[u]);
        if (s[u] > 0x1p124f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = saturate(f[e]);
        }
        *reinterpret_cast<uint4 *>(out + 8 * i) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                             pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
}

template <int kGroup>
cudaError_t quantize(const uint16_t *W, const Int4View &w, int64_t words, unsigned grid, cudaStream_t st) {
    uint32_t *codes = reinterpret_cast<uint32_t *>(w.codes);
    return launch_dependent(w.zero_point ? k_int4_quantize<kGroup, true> : k_int4_quantize<kGroup, false>, grid, kThreads, st, W,
                            words, codes, w.scale, w.zero_point);
}

bool grid_for(int64_t words, unsigned *grid) {
    const int64_t per = static_cast<int64_t>(kThreads) * kUnroll, ctas = (words + per - 1) / per;
    *grid = static_cast<unsigned>(ctas);
    return ctas <= 0x7fffffffLL;
}

}  // namespace

cudaError_t launch_int4_quantize(const uint16_t *W, const Int4View &w, cudaStream_t st) {
    const int64_t words = w.n * w.k / 8;
    unsigned grid;
    if (!grid_for(words, &grid)) return cudaErrorInvalidConfiguration;
    return w.group == 32 ? quantize<32>(W, w, words, grid, st)
                         : w.group == 64 ? quantize<64>(W, w, words, grid, st) : quantize<128>(W, w, words, grid, st);
}

cudaError_t launch_int4_dequantize(const Int4View &w, uint16_t *out, cudaStream_t st) {
    const int64_t words = w.n * w.k / 8;
    unsigned grid;
    if (!grid_for(words, &grid)) return cudaErrorInvalidConfiguration;
    const int shift = w.group == 32 ? 2 : w.group == 64 ? 3 : 4;
    return launch_dependent(k_int4_dequantize, grid, kThreads, st, reinterpret_cast<const uint32_t *>(w.codes), w.scale,
                            w.zero_point, words, shift, out);
}

}  // namespace qn
