// act8_grads.cu -- the adapter gradients of a linear layer whose input x was kept in 8 bits (act8.cuh):
//
//   t = x A^T, u = grad_h B                    (M x r)
//   grad_B[n, j] = s sum_m grad_h[m, n] t[m, j]
//   grad_A[j, k] = s sum_m u[m, j] x[m, k]
//
// with x = q a / 127, q the int8 codes and a the absmax of 64 neighbouring features, optionally under the
// forward's LoRA dropout mask. Nothing of x is written back to memory in 16 bits: an int8 code is exact in
// bf16, so the codes themselves are the tensor-core operands (mma.sync m16n8k16), and a / 127 is applied
// in fp32: to the 64-feature partial sums of t, and to u before the second product.
//
// Results are fp32 and meant to be as good: t and u are kept in fp32 between the two kernels and enter
// the second product as three bf16 terms (24 bits). All sums are fp32 in a fixed order, those of more than a few MMAs
// by fp32 additions: the tensor core cuts off what it adds to an accumulator instead of rounding it.
//
// These are the kernels for short batches; act8_grads_tc.cu has those for long ones. Two kernels, straight into registers:
//   k_down   t and u: a CTA has 32 tokens, its eight warps and a cluster's CTAs split the features.
//   k_outer  the two products over tokens: a warp has 64 columns of x or grad_h and every j, a CTA 256 columns
//            and two token streams, a cluster splits the tokens. The A operand wants neighbouring tokens of one
//            column in a register: a lane loads 8 columns of 4 tokens and pairs them with byte permutes.
//
// CTAs split the rank too, in blocks of 8 or 16 columns j.
//
// Measured: 256 x 256, 8 tokens, rank 4 5.4 us, 4096 x 4096, 16 tokens, rank 16 7.8 to 9.9 us; the latency of two kernels, each
// of loads, a few MMAs and sums across a cluster, bounds them. 28672 x 8192, 120 tokens, rank 64 41 to 47 us, for 3.4 us of
// bytes: each block of 16 columns of the rank loads and converts x and grad_h anew. With dropout 14.8 us at 16 tokens and
// 74 us at 120: the mask is drawn anew for each block of columns, too.
#include "act8.cuh"
#include "act8.h"
#include "dropout.cuh"
#include "host_cache.h"
#include "stream_common.cuh"

namespace qn {

namespace {

struct GradArgs {
    const int8_t *codes;
    const uint16_t *absmax;
    const uint16_t *gh;
    int64_t M, n, k;
    const uint16_t *A;  // r x k
    const uint16_t *B;  // n x r
    int r;
    float s;
    float *grad_A, *grad_B;
    float *t, *u;  // fragment order, see frag_index
    DropoutArgs drop;
};

// t and u lie in the order in which k_outer's lanes read them: per 16 tokens and 8 columns j 32 lanes
// x 4 values, lane (g, t) the tokens 4 t .. 4 t + 3 of column g.
__device__ __forceinline__ int64_t frag_index(int64_t m16, int jt_all, int jt, int lane) {
    return ((m16 * jt_all + jt) * 32 + lane) * 4;
}

__device__ __forceinline__ float ld_cluster(const float *p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(stream::mapa(stream::saddr(p), rank)) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// Two int8 codes, in the low bytes of the halves of p (the high bytes may hold anything), as a bf16 pair:
// 128 + (the low seven bits), less 128 for codes >= 0 and 256 for those below; every step is exact.
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t p) {
    const uint32_t a = (p & 0x007f007fu) | 0x43004300u, c = (p & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 d =
        __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&c));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// Codes of dropped elements set to 0: 8 consecutive elements from e0 on.
__device__ __forceinline__ uint2 drop_codes(uint2 v, const DropoutArgs &d, uint64_t e0) {
    const uint32_t keep = dropout_keep_bits(d, e0, 8);
    auto bytes = [](uint32_t b) {  // bit i -> byte i
        return ((b & 1u) | (b & 2u) << 7 | (b & 4u) << 14 | (b & 8u) << 21) * 0xffu;
    };
    return make_uint2(v.x & bytes(keep), v.y & bytes(keep >> 4));
}

// 8 neighbouring bf16 of a row of grad_h from column c on; zeros past its end. kAligned: rows are 16-byte aligned.
template <bool kAligned>
__device__ __forceinline__ uint4 load_gh(const uint16_t *row, int64_t c, int64_t n, const uint16_t *end) {
    if constexpr (kAligned)
        return c < n ? ld_nc_v4(row + c) : make_uint4(0u, 0u, 0u, 0u);
    else
        return act8::load_row8(row, c, n, end);
}

// ------------------------------------------------------------------------ t and u

constexpr int kDownWarps = 8;
constexpr int kDownThreads = 32 * kDownWarps;
constexpr int kDownTokens = 32;
constexpr int kPiece = 64;  // features per step of a warp

// NT neighbouring bf16 from p on, of which `count` exist, as NT / 2 pairs (NT = 1: one value).
template <int NT>
__device__ __forceinline__ void load_js(const uint16_t *p, int count, bool vec, uint32_t (&w)[(NT + 1) / 2]) {
    if (vec && count >= NT) {
        if constexpr (NT == 2) {
            w[0] = ld_ro_u32(p);
        } else {
            w[0] = ld_ro_u16(p);
        }
    } else {
#pragma unroll
        for (int i = 0; i < (NT + 1) / 2; ++i) {
            const uint32_t lo = 2 * i < count ? ld_ro_u16(p + 2 * i) : 0u;
            const uint32_t hi = NT > 1 && 2 * i + 1 < count ? ld_ro_u16(p + 2 * i + 1) : 0u;
            w[i] = lo | hi << 16;
        }
    }
}

// Everything comes straight into registers: with few tokens the factors are most of what is read, each once per 32 tokens.
// The order of the features in a step is free as long as both operands agree, and so is the order of the columns j:
//   x       lane t has the features 8 t .. 8 t + 7 of 32, two for each half of two MMAs; A's rows give the same pairs
//   grad_h  the same features; of B the lane loads those rows, NT neighbouring j, and pairs rows by byte permutes
// Column g of the MMA's tile nt is j = NT g + nt.
template <int NT, bool kX, bool kDrop, bool kAligned>
__device__ __forceinline__ void down(const GradArgs &p, float *red, int j0, int64_t tile, uint32_t rank, uint32_t ranks) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t m0 = tile * kDownTokens;
    const int64_t width = kX ? p.k : p.n, pieces = (width + kPiece - 1) / kPiece;
    int64_t row[4];  // this lane's tokens: g, g + 8, g + 16, g + 24
    bool live[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        live[h] = m0 + g + 8 * h < p.M;
        row[h] = live[h] ? m0 + g + 8 * h : 0;
    }
    const int js = p.r - j0 < 8 * NT ? p.r - j0 : 8 * NT;  // columns of this block
    const bool vec = p.r % NT == 0;

    float acc[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.0f;

    for (int64_t c = rank * kDownWarps + warp; c < pieces; c += static_cast<int64_t>(ranks) * kDownWarps) {
        float d[2][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) d[mt][nt][0] = d[mt][nt][1] = d[mt][nt][2] = d[mt][nt][3] = 0.0f;
        float sc[4];
        if (kX) {
            uint2 q[2][4];
            const int64_t c0 = c * kPiece + 8 * t;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
#pragma unroll
                for (int sub = 0; sub < 2; ++sub)
                    q[sub][h] = live[h] ? ld_nc_v2(p.codes + row[h] * p.k + c0 + 32 * sub) : make_uint2(0u, 0u);
                const uint32_t top = live[h] ? ld_ro_u16(p.absmax + row[h] * (p.k / kBlock) + c) : 0u;
                sc[h] = __uint_as_float(top << 16) * (1.0f / 127.0f);
            }
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                uint32_t a[4][4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint2 w = q[sub][h];
                    if (kDrop && live[h])
                        w = drop_codes(w, p.drop, p.drop.offset + static_cast<uint64_t>(row[h] * p.k + c0 + 32 * sub));
                    a[h][0] = codes_to_bf16(__byte_perm(w.x, 0u, 0x4140));
                    a[h][1] = codes_to_bf16(__byte_perm(w.x, 0u, 0x4342));
                    a[h][2] = codes_to_bf16(__byte_perm(w.y, 0u, 0x4140));
                    a[h][3] = codes_to_bf16(__byte_perm(w.y, 0u, 0x4342));
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int j = NT * g + nt;
                    const uint4 f = j < js ? ld_ro_v4(p.A + static_cast<int64_t>(j0 + j) * p.k + c0 + 32 * sub) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        mma_16816(d[mt][nt], a[2 * mt][0], a[2 * mt + 1][0], a[2 * mt][1], a[2 * mt + 1][1], f.x, f.y);
                        mma_16816(d[mt][nt], a[2 * mt][2], a[2 * mt + 1][2], a[2 * mt][3], a[2 * mt + 1][3], f.z, f.w);
                    }
                }
            }
        } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) sc[h] = 1.0f;
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                const int64_t c0 = c * kPiece + 32 * sub + 8 * t;
                uint4 v[4];
                uint32_t w[8][(NT + 1) / 2];
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    v[h] = live[h] ? load_gh<kAligned>(p.gh + row[h] * p.n, c0, p.n, p.gh + p.M * p.n) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    load_js<NT>(p.B + (c0 + q) * p.r + j0 + NT * g, c0 + q < p.n ? js - NT * g : 0, vec, w[q]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint32_t sel = (nt & 1) ? 0x7632 : 0x5410;
                    uint32_t b[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) b[q] = __byte_perm(w[2 * q][nt / 2], w[2 * q + 1][nt / 2], sel);
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        mma_16816(d[mt][nt], v[2 * mt].x, v[2 * mt + 1].x, v[2 * mt].y, v[2 * mt + 1].y, b[0], b[1]);
                        mma_16816(d[mt][nt], v[2 * mt].z, v[2 * mt + 1].z, v[2 * mt].w, v[2 * mt + 1].w, b[2], b[3]);
                    }
                }
            }
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mt][nt][i] = __fmaf_rn(sc[2 * mt + (i >> 1)], d[mt][nt][i], acc[mt][nt][i]);
    }

    // the warps' sums in order, then the cluster's in rank order; each rank writes its share of the tile
    constexpr int kRow = 8 * NT + 1, kTile = kDownTokens * kRow;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[warp * kTile + (16 * mt + g + 8 * (i >> 1)) * kRow + NT * (2 * t + (i & 1)) + nt] = acc[mt][nt][i];
    __syncthreads();
    for (int e = threadIdx.x; e < kTile; e += kDownThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kDownWarps; ++w) v += red[w * kTile + e];
        red[e] = v;
    }
    if (ranks > 1) {
        stream::cluster_arrive_release();
        stream::cluster_wait_acquire();
    } else {
        __syncthreads();
    }
    float *out = kX ? p.t : p.u;
    const int jt_all = (p.r + 7) / 8, jt0 = j0 / 8;
    constexpr int kAll = kDownTokens / 16 * NT * 128;
    const int e0 = static_cast<int>(kAll * rank / ranks), e1 = static_cast<int>(kAll * (rank + 1) / ranks);
    for (int e = e0 + threadIdx.x; e < e1; e += kDownThreads) {
        const int i = e & 3, l = (e >> 2) & 31, nt = (e >> 7) % NT, m16 = e / (128 * NT);
        const int64_t mg = tile * (kDownTokens / 16) + m16;
        if (mg * 16 >= p.M || jt0 + nt >= jt_all) continue;
        const float *src = red + (16 * m16 + 4 * (l & 3) + i) * kRow + 8 * nt + (l >> 2);
        float sum = 0.0f;
        if (ranks > 1)
            for (uint32_t k = 0; k < ranks; ++k) sum += ld_cluster(src, k);
        else
            sum = *src;
        out[frag_index(mg, jt_all, jt0 + nt, l) + i] = sum;
    }
    if (ranks > 1) {  // no CTA leaves while another reads its sums
        stream::cluster_arrive_release();
        stream::cluster_wait_acquire();
    }
}

// grid (ranks * token tiles, 2, blocks of 8 NT columns j): y = 0 takes u from grad_h, y = 1 t from the codes.
template <int NT, bool kDrop, bool kAligned>
__global__ void __launch_bounds__(kDownThreads) k_down(const GradArgs p) {
    extern __shared__ __align__(16) float red[];
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const int64_t tile = blockIdx.x / ranks;
    grid_dependents_launch();
    const int j0 = static_cast<int>(blockIdx.z) * 8 * NT;
    if (blockIdx.y == 0)
        down<NT, false, false, kAligned>(p, red, j0, tile, rank, ranks);
    else
        down<NT, true, kDrop, true>(p, red, j0, tile, rank, ranks);
}

// -------------------------------------------------------------- products over tokens

constexpr int kColWarps = 4;
constexpr int kTokWarps = 2;
constexpr int kOutThreads = 32 * kColWarps * kTokWarps;
constexpr int kOutCols = 64 * kColWarps;
constexpr int kOutRow = kOutCols + 4;  // floats per row j of the sums in shared memory

// v as a sum of three bf16, pairs (v0, v1) and (v2, v3) of each.
__device__ __forceinline__ void split(float (&v)[4], uint32_t (&part)[3][2]) {
#pragma unroll
    for (int term = 0; term < 3; ++term)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            part[term][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            v[2 * i] -= bf16_lo(part[term][i]);
            v[2 * i + 1] -= bf16_hi(part[term][i]);
        }
}

template <int NT, bool kX, bool kDrop, bool kAligned>
__device__ __forceinline__ void outer(const GradArgs &p, float *red, int j0, int64_t tile, uint32_t rank, uint32_t ranks) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int cw = warp % kColWarps, tw = warp / kColWarps;
    const int64_t width = kX ? p.k : p.n;
    const int64_t col0 = tile * kOutCols + 64 * cw, col = col0 + 8 * g;
    const int jt_all = (p.r + 7) / 8, jt0 = j0 / 8;
    const float *R = kX ? p.u : p.t;
    const int64_t tiles16 = (p.M + 15) / 16;

    float acc[4][NT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[i][nt][0] = acc[i][nt][1] = acc[i][nt][2] = acc[i][nt][3] = 0.0f;

    uint4 v[4];
    uint2 q[4];
    uint32_t top[4];
    auto load = [&](int64_t m16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m16 * 16 + 4 * t + i;
            if (kX) {
                q[i] = m < p.M ? ld_nc_v2(p.codes + m * p.k + col) : make_uint2(0u, 0u);
                top[i] = m < p.M ? ld_ro_u16(p.absmax + m * (p.k / kBlock) + col0 / kBlock) : 0u;
            } else {
                v[i] = m < p.M ? load_gh<kAligned>(p.gh + m * p.n, col, p.n, p.gh + p.M * p.n) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
    };

    const int64_t step = kTokWarps * static_cast<int64_t>(ranks);
    int64_t m16 = rank * kTokWarps + tw;
    const bool work = col0 < width;
    if (work && m16 < tiles16) load(m16);
    grid_dependency_wait();  // for t and u; x and grad_h were there before the first kernel
    for (; work && m16 < tiles16; m16 += step) {
        uint32_t a[4][4];  // [pair of columns 8 g + 2 i, + 1][tokens 0 1 | tokens 0 1 of the next column | 2 3 | 2 3]
        float sc[4];
        if (kX) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (kDrop && m16 * 16 + 4 * t + i < p.M)
                    q[i] = drop_codes(q[i], p.drop, p.drop.offset + static_cast<uint64_t>((m16 * 16 + 4 * t + i) * p.k + col));
                sc[i] = __uint_as_float(top[i] << 16) * (1.0f / 127.0f);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t w0 = i < 2 ? q[0].x : q[0].y, w1 = i < 2 ? q[1].x : q[1].y;
                const uint32_t w2 = i < 2 ? q[2].x : q[2].y, w3 = i < 2 ? q[3].x : q[3].y;
                const uint32_t b0 = 2u * (i & 1), b1 = b0 + 1u;
                a[i][0] = codes_to_bf16(__byte_perm(w0, w1, (4u + b0) << 8 | b0));
                a[i][1] = codes_to_bf16(__byte_perm(w0, w1, (4u + b1) << 8 | b1));
                a[i][2] = codes_to_bf16(__byte_perm(w2, w3, (4u + b0) << 8 | b0));
                a[i][3] = codes_to_bf16(__byte_perm(w2, w3, (4u + b1) << 8 | b1));
            }
        } else {
            const uint32_t w[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w},
                                      {v[1].x, v[1].y, v[1].z, v[1].w},
                                      {v[2].x, v[2].y, v[2].z, v[2].w},
                                      {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i][0] = __byte_perm(w[0][i], w[1][i], 0x5410);
                a[i][1] = __byte_perm(w[0][i], w[1][i], 0x7632);
                a[i][2] = __byte_perm(w[2][i], w[3][i], 0x5410);
                a[i][3] = __byte_perm(w[2][i], w[3][i], 0x7632);
            }
        }
        const int64_t cur = m16;
        if (m16 + step < tiles16) load(m16 + step);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (jt0 + nt >= jt_all) break;
            const float4 f = *reinterpret_cast<const float4 *>(R + frag_index(cur, jt_all, jt0 + nt, lane));
            float w[4] = {f.x, f.y, f.z, f.w};
            if (kX) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] *= sc[i];
            }
            uint32_t part[3][2];
            split(w, part);
            float d[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.0f;
#pragma unroll
            for (int term = 0; term < 3; ++term)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_16816(d[i], a[i][0], a[i][1], a[i][2], a[i][3], part[term][0], part[term][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][nt][e] += d[i][e];
        }
    }

    // the token streams of the CTA, then the cluster's CTAs in rank order
    auto at = [&](int i, int nt, int e) {
        return red + (8 * nt + 2 * t + (e & 1)) * kOutRow + 64 * cw + 8 * g + 2 * i + (e >> 1);
    };
#pragma unroll
    for (int w = 0; w < kTokWarps; ++w) {
        if (tw == w) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) *at(i, nt, e) = w == 0 ? acc[i][nt][e] : *at(i, nt, e) + acc[i][nt][e];
        }
        __syncthreads();
    }
    if (ranks > 1) {
        stream::cluster_arrive_release();
        stream::cluster_wait_acquire();
    }
    const int js = p.r - j0 < 8 * NT ? p.r - j0 : 8 * NT;
    const int all = js * kOutCols;
    const int e0 = static_cast<int>(static_cast<int64_t>(all) * rank / ranks);
    const int e1 = static_cast<int>(static_cast<int64_t>(all) * (rank + 1) / ranks);
    for (int e = e0 + threadIdx.x; e < e1; e += kOutThreads) {
        // neighbouring threads: neighbouring columns of grad_A, neighbouring j of grad_B
        const int j = kX ? e / kOutCols : e % js, c = kX ? e % kOutCols : e / js;
        const int64_t cc = tile * kOutCols + c;
        if (cc >= width) continue;
        const float *src = red + j * kOutRow + c;
        float sum = 0.0f;
        if (ranks > 1)
            for (uint32_t k = 0; k < ranks; ++k) sum += ld_cluster(src, k);
        else
            sum = *src;
        if (kX)
            p.grad_A[static_cast<int64_t>(j0 + j) * p.k + cc] = p.s * sum;
        else
            p.grad_B[cc * p.r + j0 + j] = p.s * sum;
    }
    if (ranks > 1) {
        stream::cluster_arrive_release();
        stream::cluster_wait_acquire();
    }
}

// grid (ranks * column tiles, blocks of 8 NT columns j): column tiles of grad_h first, then those of the codes.
template <int NT, bool kDrop, bool kAligned>
__global__ void __launch_bounds__(kOutThreads) k_outer(const GradArgs p) {
    extern __shared__ __align__(16) uint8_t smem[];
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const int64_t tile = blockIdx.x / ranks, tiles_gh = (p.n + kOutCols - 1) / kOutCols;
    const int j0 = static_cast<int>(blockIdx.y) * 8 * NT;
    if (tile < tiles_gh)
        outer<NT, false, false, kAligned>(p, reinterpret_cast<float *>(smem), j0, tile, rank, ranks);
    else
        outer<NT, true, kDrop, true>(p, reinterpret_cast<float *>(smem), j0, tile - tiles_gh, rank, ranks);
}

template <typename K>
cudaError_t launch_clusters(K kern, dim3 grid, int threads, size_t smem, int ranks, bool dependent, const GradArgs &p,
                            cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (dependent) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (ranks > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(ranks);
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e == cudaSuccess) count_launch();
    return e;
}

// CTAs that share a tile: doubled until the grid has `want` CTAs, at most 8 and at most `most`.
int split_ranks(int64_t tiles, int64_t want, int64_t most) {
    int s = 1;
    while (s < 8 && tiles * s < want && 2 * s <= most) s *= 2;
    return s;
}

template <int NT, bool kDrop, bool kAligned>
cudaError_t launch_pass(const GradArgs &p, int sms, cudaStream_t st) {
    const int64_t tok = (p.M + kDownTokens - 1) / kDownTokens;
    const int64_t rounds = ((p.n > p.k ? p.n : p.k) + kPiece * kDownWarps - 1) / (kPiece * kDownWarps);
    const int64_t js = (p.r + 8 * NT - 1) / (8 * NT);
    int ranks = split_ranks(2 * tok * js, 2 * sms, rounds);
    if (tok * ranks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaError_t e = launch_clusters(k_down<NT, kDrop, kAligned>, dim3(static_cast<unsigned>(tok * ranks), 2, static_cast<unsigned>(js)),
                                    kDownThreads, static_cast<size_t>(kDownWarps) * kDownTokens * (8 * NT + 1) * 4, ranks, false, p, st);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (p.n + kOutCols - 1) / kOutCols + (p.k + kOutCols - 1) / kOutCols;
    ranks = split_ranks(tiles * js, 2 * sms, (p.M + 16 * kTokWarps - 1) / (16 * kTokWarps));
    if (tiles * ranks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_clusters(k_outer<NT, kDrop, kAligned>, dim3(static_cast<unsigned>(tiles * ranks), static_cast<unsigned>(js), 1),
                           kOutThreads, static_cast<size_t>(8 * NT) * kOutRow * 4, ranks, true, p, st);
}

template <int NT>
cudaError_t launch_nt(const GradArgs &p, int sms, cudaStream_t st) {
    const bool drop = p.drop.thr != 0u;
    if (p.n % 8 == 0) return drop ? launch_pass<NT, true, true>(p, sms, st) : launch_pass<NT, false, true>(p, sms, st);
    return drop ? launch_pass<NT, true, false>(p, sms, st) : launch_pass<NT, false, false>(p, sms, st);
}

// Batches below 128 tokens, and below 1024 as long as the products are small, stay here; the others go to the tcgen05 kernels.
// Measured here and there: 4096 x 4096, rank 16 128 tokens 10.5 and 15.2 us, 256 tokens 17.1 and 15.5; 1024 x 1024, rank 8,
// 1024 tokens 11.2 and 15.8; 11008 x 4096, rank 64, 128 tokens 27.8 and 20.6.
constexpr int64_t kFewTokens = 128, kFewTokensSmall = 1024, kSmall = 24 << 20;  // tokens x features x rank (in eights)
bool few(int64_t M, int64_t n, int64_t k, int r) {
    return M < kFewTokens || (M <= kFewTokensSmall && M * (n + k) <= kSmall / ((r + 7) / 8 * 8));
}
// Workspace of these kernels: t and u.
size_t few_bytes(int64_t M, int r) {
    return 2 * sizeof(float) * static_cast<size_t>((M + 15) / 16) * 16 * static_cast<size_t>((r + 7) / 8 * 8);
}

}  // namespace

size_t act8_grads_workspace_bytes(int64_t M, int64_t n, int r) {
    const size_t here = few_bytes(M, r), there = act8_grads_tc_workspace_bytes(M, n, r);  // k decides, which is not known
    return M < kFewTokens ? here : M > kFewTokensSmall || there > here ? there : here;
}

cudaError_t launch_act8_grads(const int8_t *codes, const uint16_t *absmax, const uint16_t *gh, int64_t M, int64_t n,
                              int64_t k, const uint16_t *A, const uint16_t *B, int r, float s, const DropoutArgs &drop,
                              float *grad_A, float *grad_B, void *ws, cudaStream_t st) {
    if (!few(M, n, k, r))
        return launch_act8_grads_tc(codes, absmax, gh, M, n, k, A, B, r, s, drop, grad_A, grad_B, ws, st);
    int sms = 148;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    GradArgs p{codes, absmax, gh, M, n, k, A, B, r, s, grad_A, grad_B, static_cast<float *>(ws), nullptr, drop};
    p.u = p.t + (M + 15) / 16 * 16 * ((r + 7) / 8 * 8);
    // Blocks of 8 columns j as long as blocks of 16 would not fill the SMs twice: 4096 x 4096, 16 tokens, rank 16 8.0 us against
    // 10.1; with more CTAs blocks of 16, which read x and grad_h half as often: 28672 x 8192, 120 tokens, rank 64 39.6 us against 49.1.
    const int64_t tiles = (n + kOutCols - 1) / kOutCols + (k + kOutCols - 1) / kOutCols;
    return tiles * ((r + 15) / 16) <= 2 * sms ? launch_nt<1>(p, sms, st) : launch_nt<2>(p, sms, st);
}

}  // namespace qn
