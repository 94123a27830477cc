// act8.cuh -- the 8-bit form of an activation, on the device.
//
// A block of 64 consecutive values keeps a = max |x| (exact: x is bf16, and so is a) and, per value,
// the int8 code q = 127 x / a rounded to the nearest integer, halves away from zero. The value read
// back is q s with s = fl32(a / 127). A block that holds a NaN or an infinity keeps a = NaN and codes
// 0, so everything read back from it is NaN; a block of zeros keeps a = 0 and codes 0.
#pragma once

#include "common.cuh"

namespace qn {
namespace act8 {

constexpr int kPer = 8;             // values per thread and step: one 16-byte load
constexpr int kLanes = kBlock / kPer;  // lanes that share a block

// Absolute maximum of the 8 values of each of the block's kLanes lanes, as bf16 bits. Comparing bits as
// integers puts infinities and NaNs above every finite value.
__device__ __forceinline__ uint32_t block_absmax(const uint4 &v) {
    uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                          __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
    return max(m & 0xffffu, m >> 16);
}

// Codes of a lane's 8 values under the block absmax `top` (bf16 bits, finite).
//
// inv = fl32(127 (1 + 2^-17) / a): 127 x / a has halves exactly where 254 |x| is an odd multiple of a,
// and any other value is at least 1 / (2 a) of a unit away from a half with a < 256 the integer
// significand. Raising the quotient by 2^-17 of itself moves it by less than half of that (the
// significands of x and a are below 256: 254 * 255 * 2^-17 < 0.5) and more than the rounding of inv, so
// it puts exact halves above the half and nothing else across. The product and the rounding to an
// integer are one fma onto 1.5 * 2^23, whose low byte is then the code. For a below 2^-100 x and a are
// first scaled by 2^64, which is exact.
__device__ __forceinline__ uint2 encode(const uint4 &v, uint32_t top) {
    if (top == 0u) return make_uint2(0u, 0u);
    float a = __uint_as_float(top << 16);
    const bool tiny = top < 0x0d80u;  // 2^-100
    if (tiny) a *= 0x1p64f;
    const float inv = __fdiv_rn(0x1.fc00fep+6f, a);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo = bf16_lo(w[i]), hi = bf16_hi(w[i]);
        if (tiny) {
            lo *= 0x1p64f;
            hi *= 0x1p64f;
        }
        c[2 * i] = __float_as_uint(__fmaf_rn(lo, inv, 12582912.0f));
        c[2 * i + 1] = __float_as_uint(__fmaf_rn(hi, inv, 12582912.0f));
    }
    uint2 q;
    q.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    q.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
    return q;
}

// A lane's 8 values as a part of their block: stores the codes (8 bytes at codes + 8 i) and, from the
// block's first lane, its absmax. Every lane of the warp calls it; `live` lanes store.
__device__ __forceinline__ void store_block(const uint4 &v, bool live, int64_t i, int8_t *codes, uint16_t *absmax) {
    const uint32_t top = block_absmax(v);
    const bool finite = top < 0x7f80u;
    const uint2 q = finite ? encode(v, top) : make_uint2(0u, 0u);
    if (!live) return;
    *reinterpret_cast<uint2 *>(codes + kPer * i) = q;
    if ((threadIdx.x & (kLanes - 1)) == 0) absmax[i / kLanes] = static_cast<uint16_t>(finite ? top : 0x7fc0u);
}

// s = a / 127 of a block absmax (bf16 bits).
__device__ __forceinline__ float step(uint32_t top) { return __fdiv_rn(__uint_as_float(top << 16), 127.0f); }

// The 4 codes of a word as fp32 integers: the byte with its sign bit flipped is q + 128, which as the low
// mantissa byte of 2^23 reads 2^23 + 128 + q.
__device__ __forceinline__ void decode4(uint32_t w, float (&f)[4]) {
    w ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540u + static_cast<uint32_t>(i))) - 8388736.0f;
}

// 8 neighbouring bf16 from column c of a row of n on, zeros past its end, of a matrix whose rows lie on any 2-byte
// boundary and that starts on a 16-byte one: cut out of the two aligned words around them. `end` is the end of the matrix,
// which no word may pass.
__device__ __forceinline__ uint4 load_row8(const uint16_t *row, int64_t c, int64_t n, const uint16_t *end) {
    if (c >= n) return make_uint4(0u, 0u, 0u, 0u);
    const uint16_t *p = row + c;
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;  // bytes, even
    const uint16_t *a = p - off / 2;
    uint32_t w[8];
    const bool low = a + 8 <= end, high = a + 16 <= end;
    const uint4 v0 = low ? ld_ro_v4(a) : make_uint4(0u, 0u, 0u, 0u), v1 = high ? ld_ro_v4(a + 8) : make_uint4(0u, 0u, 0u, 0u);
    w[0] = v0.x; w[1] = v0.y; w[2] = v0.z; w[3] = v0.w;
    w[4] = v1.x; w[5] = v1.y; w[6] = v1.z; w[7] = v1.w;
    if (!high) {  // the last words of the matrix: value by value
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t lo = a + 2 * e < end ? ld_ro_u16(a + 2 * e) : 0u, hi = a + 2 * e + 1 < end ? ld_ro_u16(a + 2 * e + 1) : 0u;
            w[e] = lo | hi << 16;
        }
    }
#pragma unroll
    for (int e = 0; e < 6; ++e) w[e] = (off & 8u) ? w[e + 2] : w[e];
#pragma unroll
    for (int e = 0; e < 5; ++e) w[e] = (off & 4u) ? w[e + 1] : w[e];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __funnelshift_r(w[e], w[e + 1], (off & 2u) * 8u);
    if (c + 8 > n) {  // the next row's values
        const uint32_t left = static_cast<uint32_t>(n - c);
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) w[e] &= (2 * e < left ? 0xffffu : 0u) | (2 * e + 1 < left ? 0xffff0000u : 0u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace act8
}  // namespace qn
