// int4_linear.cu -- h[m, i] = sum_k W[i, k] x[m, k] for 1 to 16 tokens m over 4-bit weights
// W[i, k] = s (q - z) with a scale and a zero point per group of a row (int4.h):
//
//   h[m, i] = sum over groups of s sum_{k in group} (q - z) x[m, k]
//
// The weights are read once and bound the call (0.5 B each against 2 M / n for x). The products run on
// mma.sync m16n8k16 with 16 rows of W as A and 8 tokens as B: q - z is an integer of at most 4 bits and
// sign, so exact in bf16, x is bf16, and the sum of a group is held in fp32 and scaled there; nothing is
// rounded before the one rounding of h.
//
// A warp reads its operands straight into registers. The order of k inside a group is free as long as A
// and B agree, so lane (g, t) of a warp takes a quarter t of the group of rows g and g + 8 as whole words:
// 32-bit words of 8 weights, whose nibbles p and p + 4 are a pair ((word >> 4p) & 0x000f000f | 0x43004300
// is the bf16 pair 128 + q; minus 128 + z is exact). One word of each row feeds two MMAs. The matching x
// is one 16-byte load per token, its elements paired the same way with byte permutes.
//
// The warps of a CTA share 16 rows and split the groups; their sums meet in shared memory.
#include "common.cuh"
#include "int4.h"

namespace qn {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;

struct LinArgs {
    const uint8_t *codes;
    const uint16_t *scale;
    const uint8_t *zero_point;
    int64_t n, k;
    const uint16_t *x;
    int M;
    uint16_t *h;
};

template <int kWords>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[kWords]) {
    if (kWords == 4) {
        const uint4 v = ld_nc_v4(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else if (kWords == 2) {
        const uint2 v = ld_nc_v2(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = ld_ro_u32(p);  // 4 lanes read half a sector; the next group's read finds the rest in L1
    }
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// kWords: words of a lane per row and group (group = 32 kWords); NT: token tiles of 8.
template <int kWords, int NT, bool kZero>
__global__ void __launch_bounds__(kThreads) k_int4_linear(const LinArgs p) {
    constexpr int kGroupW = 32 * kWords;
    constexpr int kUnroll = 4 / kWords * 2;  // groups loaded ahead of their use
    __shared__ float part[kWarps][kRows][8 * NT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows;
    // rows past the end read the last row and are not stored
    const int64_t ra = r0 + g < p.n ? r0 + g : p.n - 1, rb = r0 + g + 8 < p.n ? r0 + g + 8 : p.n - 1;
    const int groups = static_cast<int>(p.k / kGroupW);
    const int lo = static_cast<int>(static_cast<int64_t>(groups) * warp / kWarps);
    const int hi = static_cast<int>(static_cast<int64_t>(groups) * (warp + 1) / kWarps);
    const uint8_t *ca = p.codes + ra * (p.k / 2) + 4 * kWords * t, *cb = p.codes + rb * (p.k / 2) + 4 * kWords * t;
    const int64_t sa = ra * groups, sb = rb * groups;

    float out[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) out[nt][0] = out[nt][1] = out[nt][2] = out[nt][3] = 0.0f;

    for (int i0 = lo; i0 < hi; i0 += kUnroll) {
        uint32_t wa[kUnroll][kWords], wb[kUnroll][kWords];
        uint32_t fa[kUnroll], fb[kUnroll], za[kUnroll], zb[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u < hi ? i0 + u : hi - 1;
            load_words<kWords>(ca + static_cast<int64_t>(i) * (kGroupW / 2), wa[u]);
            load_words<kWords>(cb + static_cast<int64_t>(i) * (kGroupW / 2), wb[u]);
            fa[u] = ld_ro_u16(p.scale + sa + i);
            fb[u] = ld_ro_u16(p.scale + sb + i);
            if (kZero) {
                za[u] = __ldg(p.zero_point + sa + i);
                zb[u] = __ldg(p.zero_point + sb + i);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (i0 + u >= hi) break;
            // 128 + z as a bf16 pair
            const uint32_t oa = kZero ? 0x43004300u | (za[u] * 0x00010001u) : 0x43084308u;
            const uint32_t ob = kZero ? 0x43004300u | (zb[u] * 0x00010001u) : 0x43084308u;
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
            const int64_t kk = static_cast<int64_t>(i0 + u) * kGroupW + 8 * kWords * t;
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                uint32_t a[4], b[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a[q] = sub_bf16x2(((wa[u][w] >> (4 * q)) & 0x000f000fu) | 0x43004300u, oa);
                    b[q] = sub_bf16x2(((wb[u][w] >> (4 * q)) & 0x000f000fu) | 0x43004300u, ob);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int m = 8 * nt + g;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (m < p.M) v = ld_ro_v4(p.x + m * p.k + kk + 8 * w);
                    const uint32_t x0 = __byte_perm(v.x, v.z, 0x5410), x1 = __byte_perm(v.x, v.z, 0x7632);
                    const uint32_t x2 = __byte_perm(v.y, v.w, 0x5410), x3 = __byte_perm(v.y, v.w, 0x7632);
                    mma_16816(acc[nt], a[0], b[0], a[1], b[1], x0, x1);
                    mma_16816(acc[nt], a[2], b[2], a[3], b[3], x2, x3);
                }
            }
            const float f0 = __uint_as_float(fa[u] << 16), f1 = __uint_as_float(fb[u] << 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                out[nt][0] = __fmaf_rn(f0, acc[nt][0], out[nt][0]);
                out[nt][1] = __fmaf_rn(f0, acc[nt][1], out[nt][1]);
                out[nt][2] = __fmaf_rn(f1, acc[nt][2], out[nt][2]);
                out[nt][3] = __fmaf_rn(f1, acc[nt][3], out[nt][3]);
            }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        part[warp][g][8 * nt + 2 * t] = out[nt][0];
        part[warp][g][8 * nt + 2 * t + 1] = out[nt][1];
        part[warp][g + 8][8 * nt + 2 * t] = out[nt][2];
        part[warp][g + 8][8 * nt + 2 * t + 1] = out[nt][3];
    }
    __syncthreads();
    // the warps' sums in order; neighbouring threads store neighbouring rows
    for (int i = threadIdx.x; i < kRows * p.M; i += kThreads) {
        const int row = i & (kRows - 1), m = i / kRows;
        if (r0 + row >= p.n) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += part[w][row][m];
        p.h[m * p.n + r0 + row] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
}

template <int kWords, int NT>
void launch(const LinArgs &p, unsigned grid, cudaStream_t st) {
    if (p.zero_point)
        k_int4_linear<kWords, NT, true><<<grid, kThreads, 0, st>>>(p);
    else
        k_int4_linear<kWords, NT, false><<<grid, kThreads, 0, st>>>(p);
}

template <int kWords>
void launch_words(const LinArgs &p, unsigned grid, cudaStream_t st) {
    if (p.M <= 8)
        launch<kWords, 1>(p, grid, st);
    else
        launch<kWords, 2>(p, grid, st);
}

}  // namespace

cudaError_t launch_int4_linear(const Int4View &w, const uint16_t *x, int M, uint16_t *h, cudaStream_t st) {
    const LinArgs p{w.codes, w.scale, w.zero_point, w.n, w.k, x, M, h};
    const unsigned grid = static_cast<unsigned>((w.n + kRows - 1) / kRows);
    if (w.group == 32)
        launch_words<1>(p, grid, st);
    else if (w.group == 64)
        launch_words<2>(p, grid, st);
    else
        launch_words<4>(p, grid, st);
    count_launch();
    return cudaGetLastError();
}

}  // namespace qn
