// int4.cu -- weights as 4-bit integers with a scale per group of 32, 64 or 128 consecutive weights of a
// row, and back to bf16. A weight is s (q - z): s bf16, q and z integers 0..15.
//
//   with zero points: lo = min(0, min w), hi = max(0, max w), s = bf16(fl32((hi - lo) / 15)),
//                     z = clamp(round(-lo / s), 0, 15)
//   symmetric:        s = bf16(fl32(max |w| / 7)), z = 8
//   q = clamp(round(w / s) + z, 0, 15), rounding to nearest with halves away from zero; a group whose s is
//   0 has q = z.
//   A group with a NaN or an infinity has s = NaN, z = 0 (8 without zero points) and q = z: it reads back NaN.
//
// Both directions are bound by HBM: 2 B and 0.5 B + 2 or 3 B per group for each weight. A lane takes 8
// weights (one 16-byte word of W, one 4-byte word of codes); a group is 4, 8 or 16 neighbouring lanes,
// which share its minimum and maximum by shuffles. k % group == 0, so groups do not straddle rows and
// the matrix is walked as one flat array.
//
// Measured at 28672 x 8192, groups of 64, on three sets of buffers in turn: with zero points quantise 110 to 113 us (5.3 to
// 5.4 TB/s, 0.83 of the measured HBM rate), read back 100.5 us (6.0 TB/s, 0.92); without quantise 96.7 to 98.6 us (6.1 TB/s, 0.94),
// read back 93.3 us.
#include "common.cuh"
#include "dependent.cuh"
#include "int4.h"

namespace qn {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it leaves an integer in the low mantissa bits

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // of bf16 pairs; NaN where either is
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}

// A group's largest weight and the size of its smallest, both at least 0, or (not kZero) its largest size; NaN (both, or the
// one) when the group holds a NaN. All lanes of the warp call it. Both run through one bf16 pair: (max w, max -w).
template <int kGroup, bool kZero>
__device__ __forceinline__ void range(const uint4 &v, float &hi, float &below) {
    constexpr uint32_t kSigns = 0x80008000u;
    uint32_t m;
    if (kZero) {
        const uint32_t a = max2(max2(v.x, v.y), max2(v.z, v.w));
        const uint32_t b = max2(max2(v.x ^ kSigns, v.y ^ kSigns), max2(v.z ^ kSigns, v.w ^ kSigns));
        m = max2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    } else {
        m = max2(max2(v.x & ~kSigns, v.y & ~kSigns), max2(v.z & ~kSigns, v.w & ~kSigns));
    }
#pragma unroll
    for (int d = 1; d < kGroup / 8; d <<= 1) m = max2(m, __shfl_xor_sync(0xffffffffu, m, d));
    m = max2(m, 0u);
    if (!kZero) m = max(m & 0xffffu, m >> 16);  // as integers, which puts a NaN above all: the bits have no sign
    hi = bf16_lo(m);
    below = bf16_hi(m);
}

// Scale, zero point and codes of a lane's 8 weights in a group with this range.
//
// The quotient w / s is taken as w inv with inv = (1 + 2^-16) / s to 2^-21 of itself: w and s have 8-bit
// significands, so a quotient that is not a half is at least 1 / 512 of a unit away from one, and one
// that is a half is raised above it by more than the error of inv; at up to 16 units the raise is
// below 2^-12. An fma onto 1.5 * 2^23 + z then gives round(w / s) + z with halves away from zero.
template <bool kZero>
__device__ __noinline__ uint4 encode_any(uint4 v, float hi, float below) {  // codes, scale, zero point
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    if (!(hi <= 3.4028235e38f && below <= 3.4028235e38f)) return make_uint4(kZero ? 0u : 0x88888888u, 0x7fc0u, kZero ? 0u : 8u, 0u);
    float span = kZero ? hi + below : hi;
    if (kZero && span > 3.4028235e38f) span = 2.0f * __fdiv_rn(0.5f * hi + 0.5f * below, 15.0f);  // hi + below overflowed
    else span = __fdiv_rn(span, kZero ? 15.0f : 7.0f);
    const uint32_t scale_bits = __bfloat16_as_ushort(__float2bfloat16_rn(span));
    float s = __uint_as_float(scale_bits << 16), times = 1.0f;
    if (s == 0.0f) return kZero ? make_uint4(0u, scale_bits, 0u, 0u) : make_uint4(0x88888888u, scale_bits, 8u, 0u);
    if (s < 0x1p-80f) times = 0x1p64f;  // keep 1 / s finite: w / s of both times 2^64, exact
    const float inv = __fdiv_rn(0x1.0001p+0f, s * times);
    int z = 8;
    if (kZero) z = min(static_cast<int>(__float_as_uint(__fmaf_rn(below * times, inv, kMagic)) - 0x4b400000u), 15);
    const float base = kMagic + static_cast<float>(z);
    uint32_t word = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float w = (i & 1 ? bf16_hi(u[i / 2]) : bf16_lo(u[i / 2])) * times;
        const int q = static_cast<int>(__float_as_uint(__fmaf_rn(w, inv, base)) - 0x4b400000u);
        word |= static_cast<uint32_t>(min(max(q, 0), 15)) << (4 * i);
    }
    return make_uint4(word, scale_bits, static_cast<uint32_t>(z), 0u);
}

// The same for ordinary ranges, in a third of the instructions (with encode_any for all the kernel was bound by issuing them:
// 28672 x 8192 took 131 us instead of 104). span / 15 (7) is the product with the reciprocal and one correction by its remainder, which
// rounds as the division does (Markstein's theorem; checked for every significand). s is then span / 15 (7) to 2^-8.9 of itself, so
// w / s is above -z - 1/2 and, without zero points, within 7.1: only w / s + z with zero points can come out above 15, by 1.
template <bool kZero>
__device__ __forceinline__ uint32_t encode(const uint4 &v, float hi, float below, uint32_t &scale_bits, uint32_t &zero) {
    const float span = kZero ? hi + below : hi;
    if (!(span > 0x1p-60f && span < 0x1p120f)) {
        const uint4 r = encode_any<kZero>(v, hi, below);
        scale_bits = r.y;
        zero = r.z;
        return r.x;
    }
    constexpr float kSteps = kZero ? 15.0f : 7.0f, kOver = 1.0f / kSteps;
    const float near = span * kOver, fl = __fmaf_rn(__fmaf_rn(-kSteps, near, span), kOver, near);
    scale_bits = __bfloat16_as_ushort(__float2bfloat16_rn(fl));
    const float inv = __fdividef(0x1.0001p+0f, __uint_as_float(scale_bits << 16));
    float base = kMagic + 8.0f;
    zero = 8u;
    if (kZero) {
        base = __fmaf_rn(below, inv, kMagic);
        zero = __float_as_uint(base) & 15u;
    }
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t word = 0u - 0x4b400000u * 0x11111111u;  // the sums' leading bits, which fall out
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float q = __fmaf_rn(i & 1 ? bf16_hi(u[i / 2]) : bf16_lo(u[i / 2]), inv, base);
        if (kZero) q = fminf(q, kMagic + 15.0f);
        word += __float_as_uint(q) << (4 * i);
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
        uint32_t sb, z;
        float hi, below;
        range<kGroup, kZero>(v[u], hi, below);
        const uint32_t word = encode<kZero>(v[u], hi, below, sb, z);
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
