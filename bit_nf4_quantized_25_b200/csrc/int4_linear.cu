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
// The order of k inside a group is free as long as A and B agree, so lane (g, t) of a warp takes a quarter t of
// the group of rows g and g + 8 as whole words: 32-bit words of 8 weights, whose nibbles p and p + 4 are a pair (see
// unpack). One word of each row feeds two MMAs. x is paired the same way once, when a CTA copies its part of it to shared memory.
//
// A cluster has a range of 16-row tiles, its CTAs (slices) split k. A CTA keeps its part of x, all of it, in shared
// memory, so x is read from L2 once per CTA: all SMs ask for the same lines of it at about the same time, and with x from
// L2 in the loop 8192 x 28672 at 16 tokens took 84 us (by plain loads; 107 us through a ring of asynchronous copies)
// instead of 62, now 59. The 16 warps of a CTA take a tile each, and when fewer than 16 are left, split k for them once more. A
// warp has kSlots steps of its weights in flight, in a ring of its own: asynchronous copies, since loads to registers
// that are waited for one by one end up waiting for the youngest. The parts' sums meet in shared memory.
//
// Measured, with zero points: 4096 x 4096 (group 128) 1 token 6.5 to 6.9 us; 8192 x 28672 (128) 1, 8 and 16 tokens 34.3, 41.6
// and 58.7 us (3.6, 3.0 and 2.1 TB/s), 32 and 64 tokens 117 and 233 us (a pass over the weights for each 16); 11008 x 4096 (32)
// 5 tokens 14.7 us. At 16 tokens three quarters of the warps' time goes by in the loop, 190 instructions of a warp for 16 rows x
// 128 k, and no pipe is busy for a third of it: waits between dependent instructions bound it, four warps to a scheduler. x of 16
// tokens leaves no room for more, and 120 of 148 SMs hold the clusters of 8 that it needs. One token runs under the same plan, and
// x has eight columns of shared memory for it: a choice (see plan), not a limit of its own. Small calls are start-up, the copy of x
// and the sums across CTAs.
#include "common.cuh"
#include "dependent.cuh"
#include "host_cache.h"
#include "int4.h"
#include "stream_common.cuh"

namespace qn {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;    // of a tile
constexpr int kStep = 128;   // k of a step: 4 words of a lane and row
constexpr int kSlots = 4;    // steps of a warp's ring and of a unit of its loop: 16 warps x 4 x 1 KB = 64 KB in flight on an SM
constexpr uint32_t kStepBytes = kRows * kStep / 2;
constexpr size_t kSmemMost = 224 * 1024;

struct LinArgs {
    const uint8_t *codes;
    const uint16_t *scale;
    const uint8_t *zero_point;
    int64_t n, k;
    const uint16_t *x;
    int M;
    uint16_t *h;
    int64_t tiles;  // 16-row tiles
    int slices;     // CTAs of a cluster
};

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    const __nv_bfloat162 d = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&c));
    return *reinterpret_cast<const uint32_t *>(&d);
}

template <int kWords>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t *w) {
    if constexpr (kWords == 4) {
        const uint4 v = stream::lds128(addr);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (kWords == 2) {
        const uint2 v = stream::lds64(addr);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = stream::lds32(addr);
    }
}

// A word's 8 codes less z, in pairs p and p + 4, times kUnit: as a bf16, bits 0..3 are q 2^-133 and bits 4..7 q 2^-129
// (subnormal), so a multiplication brings both to q 2^-6. nz: -z 2^-6. All exact.
constexpr float kUnit = 0x1p-6f;
constexpr uint32_t kTo6 = 0x7f007f00u, kTo6High = 0x7d007d00u;  // 2^127, 2^123
__device__ __forceinline__ void unpack(uint32_t w, uint32_t nz, uint32_t (&a)[4]) {
    const uint32_t h = w >> 8;
    a[0] = fma_bf16x2(w & 0x000f000fu, kTo6, nz);
    a[1] = fma_bf16x2(w & 0x00f000f0u, kTo6High, nz);
    a[2] = fma_bf16x2(h & 0x000f000fu, kTo6, nz);
    a[3] = fma_bf16x2(h & 0x00f000f0u, kTo6High, nz);
}
// -z 2^-6 in the lower half.
__device__ __forceinline__ uint32_t minus_zero(uint32_t z) { return fma_bf16x2(z, kTo6 | 0x80008000u, 0x80008000u); }

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// kWords: words of a lane per row and group (group = 32 kWords); NT: token tiles of 8.
template <int kWords, int NT, bool kZero>
__global__ void __launch_bounds__(kThreads, 1) k_int4_linear(const LinArgs p) {
    constexpr int kGroups = 4 / kWords;  // of a step
    constexpr int kCols = 8 * NT;
    constexpr int kSums = kWarps * kRows * kCols;  // of a batch: a tile's part for each warp
    constexpr uint32_t kWordBytes = kCols * 64, kXStep = 4 * kWordBytes;
    extern __shared__ __align__(128) uint8_t smem[];
    float *sums = reinterpret_cast<float *>(smem);  // [2][warp][row][token]
    const uint32_t xs = stream::saddr(smem) + 2 * kSums * 4 + kWarps * kSlots * kStepBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

    // Cluster c takes the tiles from tiles c / clusters on, a batch of 16 at a time, one for each warp; of the last batch's
    // `rest` tiles, each is split among kWarps / rest warps.
    const int S = p.slices, slice = static_cast<int>(blockIdx.x) % S;
    const int64_t cluster = blockIdx.x / S, clusters = gridDim.x / S;
    const int64_t tile0 = p.tiles * cluster / clusters;
    const int tiles = static_cast<int>(p.tiles * (cluster + 1) / clusters - tile0);
    const int batches = (tiles + kWarps - 1) / kWarps, rest = tiles - (batches - 1) * kWarps, splits = kWarps / rest;
    const int64_t steps = (p.k + kStep - 1) / kStep;
    const int64_t x0 = steps * slice / S;
    const int x_len = static_cast<int>(steps * (slice + 1) / S - x0);
    const int64_t groups = p.k / (32 * kWords);

    begin_dependent();

    // x of the CTA's steps: [step][word of a lane][token][t] x 16 bytes, zeros past k
    {
        const int per = x_len * (kStep / 8);  // 16-byte pieces of a token
        const int dm = per ? kThreads / per : 0, dq = per ? kThreads % per : 0;
        int m = per ? static_cast<int>(threadIdx.x) / per : p.M, q = per ? static_cast<int>(threadIdx.x) % per : 0;
        while (m < p.M) {
            const int64_t kk = x0 * kStep + 8 * static_cast<int64_t>(q);
            const int grp = q / (4 * kWords), r = q % (4 * kWords);
            const uint32_t to = xs + static_cast<uint32_t>((grp * kWords + r % kWords) * kCols + m) * 64u + static_cast<uint32_t>(r / kWords) * 16u;
            const bool in = kk < p.k;
            stream::cp_async16_zfill(to, in ? p.x + m * p.k + kk : p.x, in ? 16u : 0u);
            m += dm;
            q += dq;
            if (q >= per) {
                q -= per;
                ++m;
            }
        }
        stream::cp_async_commit();
    }

    // A step's weights lie [group][row][lane's words] in the ring: a read's lanes, and (a copy has 8 rows) a copy's, side by side.
    const uint32_t ring = stream::saddr(smem) + 2 * kSums * 4 + static_cast<uint32_t>(warp) * (kSlots * kStepBytes);
    const uint32_t c_part = lane % kWords, c_row = lane / kWords % 8, c_group = lane / (8 * kWords);
    const uint32_t c_to = ring + c_group * (256 * kWords) + c_row * (16 * kWords) + c_part * 16u;
    const uint32_t r_at = ring + static_cast<uint32_t>(g * (16 * kWords) + t * (4 * kWords));
    const uint8_t *ca = nullptr, *cb = nullptr;  // the pieces of the unit (kSlots steps) to be copied next that are this lane's
    int64_t ia = 0, ib = 0;                      // index of the scales of rows g and g + 8 there, from group t on
    int left = 0;                                // groups of the row from there on
    // This warp's steps of a batch, and none in a batch that has no tile for it.
    auto part = [&](int batch, int64_t &tile, int &lo) -> int {
        if (batch < batches - 1) {
            tile = tile0 + batch * kWarps + warp;
            lo = 0;
            return x_len;
        }
        const int i = warp / splits, j = warp - i * splits;
        tile = tile0 + batch * kWarps + i;
        lo = x_len * j / splits;
        return i < rest && batch < batches ? x_len * (j + 1) / splits - lo : 0;
    };
    // Rows past the end read the last row and are not stored.
    auto begin = [&](int64_t tile, int lo) {
        const int64_t s0 = x0 + lo, row = tile * kRows, end = p.n - 1;
        const int64_t fa = row + c_row < end ? row + c_row : end, fb = row + 8 + c_row < end ? row + 8 + c_row : end;
        ca = p.codes + fa * (p.k / 2) + s0 * (kStep / 2) + 16 * (c_group * kWords + c_part);
        cb = p.codes + fb * (p.k / 2) + s0 * (kStep / 2) + 16 * (c_group * kWords + c_part);
        const int64_t ra = row + g < end ? row + g : end, rb = row + 8 + g < end ? row + 8 + g : end;
        ia = ra * groups + s0 * kGroups + t;
        ib = rb * groups + s0 * kGroups + t;
        left = static_cast<int>(groups - s0 * kGroups);
    };
    auto next = [&] {
        ca += kSlots * (kStep / 2);
        cb += kSlots * (kStep / 2);
        ia += kSlots * kGroups;
        ib += kSlots * kGroups;
        left -= kSlots * kGroups;
    };
    // Step i of the unit to its place in the ring. k % 128 may be 64 with groups below 128: zeros for what is past the end.
    auto copy = [&](int i, bool live) {
        if (live) {
            const bool in = kWords == 4 || i * kGroups + static_cast<int>(c_group) < left;
            stream::cp_async16_zfill(c_to + i * kStepBytes, in ? ca + i * (kStep / 2) : p.codes, in ? 16u : 0u);
            stream::cp_async16_zfill(c_to + i * kStepBytes + 128 * kWords, in ? cb + i * (kStep / 2) : p.codes, in ? 16u : 0u);
        }
        stream::cp_async_commit();
    };
    // Scales and zero points of the unit: lane t of a quad has those of groups t, t + 4 and so on (0 past the end or `count`).
    uint32_t sa[kGroups], sb[kGroups], za[kGroups], zb[kGroups];
    auto load_scales = [&](int count) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            const bool in = 4 * j + t < count * kGroups && 4 * j + t < left;
            sa[j] = in ? ld_nc_u16(p.scale + ia + 4 * j) : 0u;
            sb[j] = in ? ld_nc_u16(p.scale + ib + 4 * j) : 0u;
            if (kZero) {
                za[j] = in ? ld_nc_u8(p.zero_point + ia + 4 * j) : 0u;
                zb[j] = in ? ld_nc_u8(p.zero_point + ib + 4 * j) : 0u;
            }
        }
    };

    int64_t tile;
    int lo, len = part(0, tile, lo);
    if (len) {
        begin(tile, lo);
        load_scales(len);
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) copy(i, i < len);

    // pair x as the nibbles are paired: each thread the pieces that it copied
    stream::cp_async_wait_n<kSlots>();
    {
        const int per = x_len * (kStep / 8);
        const int dm = per ? kThreads / per : 0, dq = per ? kThreads % per : 0;
        int m = per ? static_cast<int>(threadIdx.x) / per : p.M, q = per ? static_cast<int>(threadIdx.x) % per : 0;
        while (m < p.M) {
            const int grp = q / (4 * kWords), r = q % (4 * kWords);
            const uint32_t at = xs + static_cast<uint32_t>((grp * kWords + r % kWords) * kCols + m) * 64u + static_cast<uint32_t>(r / kWords) * 16u;
            const uint4 v = stream::lds128(at);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(__byte_perm(v.x, v.z, 0x5410)),
                         "r"(__byte_perm(v.x, v.z, 0x7632)), "r"(__byte_perm(v.y, v.w, 0x5410)), "r"(__byte_perm(v.y, v.w, 0x7632))
                         : "memory");
            m += dm;
            q += dq;
            if (q >= per) {
                q -= per;
                ++m;
            }
        }
    }
    __syncthreads();

    // The sums of a batch, slice by slice and split by split, and their rounding.
    auto finish = [&](int batch) {
        const bool last = batch == batches - 1;
        const int K = last ? splits : 1, rows = (last ? rest : kWarps) * kRows;
        const int r0 = rows * slice / S, own = rows * (slice + 1) / S - r0;
        const int64_t row0 = (tile0 + batch * kWarps) * kRows;
        for (int e = threadIdx.x; e < own * p.M; e += kThreads) {
            const int m = e / own, r = r0 + e - m * own;  // neighbouring threads have neighbouring rows of a token
            if (row0 + r >= p.n) continue;
            const float *from = sums + (batch & 1) * kSums + (r / kRows * K * kRows + r % kRows) * kCols + m;
            const uint32_t at = stream::saddr(from);
            float sum = 0.0f;
            int i = 0, j = 0;  // slice and split; 8 loads at a time, as another CTA's memory is about a microsecond away
            while (i < S) {
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    v[u] = i < S ? ld_cluster(stream::mapa(at + static_cast<uint32_t>(j * kRows * kCols * 4), static_cast<uint32_t>(i))) : 0.0f;
                    if (++j == K) {
                        j = 0;
                        ++i;
                    }
                }
                sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
            }
            p.h[m * p.n + row0 + r] = __bfloat16_as_ushort(__float2bfloat16_rn(sum * (1.0f / kUnit)));
        }
        __syncwarp();
    };

    // tokens past the end have whatever lies there and are not stored
    const uint32_t x_lane = xs + static_cast<uint32_t>(g * 64 + t * 16);
    for (int batch = 0; batch < batches; ++batch) {
        float out[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) out[nt][0] = out[nt][1] = out[nt][2] = out[nt][3] = 0.0f;
        uint32_t xa = x_lane + static_cast<uint32_t>(lo) * kXStep;
        int ahead_len = 0;
        for (int left_len = len; left_len > 0; left_len -= kSlots) {
            uint32_t pa[kGroups], pb[kGroups];
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                pa[j] = sa[j] << 16 | (kZero ? minus_zero(za[j]) & 0xffffu : 0u);
                pb[j] = sb[j] << 16 | (kZero ? minus_zero(zb[j]) & 0xffffu : 0u);
            }
            // what is copied next: the next unit of this part, or the first of the next batch's
            int ahead = left_len - kSlots;
            if (ahead > 0) {
                next();
            } else {
                ahead = ahead_len = part(batch + 1, tile, lo);
                if (ahead) begin(tile, lo);
            }
            if (ahead) load_scales(ahead);
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                stream::cp_async_wait_n<kSlots - 1>();
                __syncwarp();
                uint32_t wa[4], wb[4];
#pragma unroll
                for (int e = 0; e < kGroups; ++e) {
                    lds_words<kWords>(r_at + i * kStepBytes + e * (256 * kWords), &wa[e * kWords]);
                    lds_words<kWords>(r_at + i * kStepBytes + e * (256 * kWords) + 128 * kWords, &wb[e * kWords]);
                }
                __syncwarp();
                copy(i, i < ahead);
                if (i < left_len) {
#pragma unroll
                    for (int e = 0; e < kGroups; ++e) {
                        const int from = i * kGroups + e;
                        const uint32_t qa = __shfl_sync(0xffffffffu, pa[from / 4], from % 4, 4);
                        const uint32_t qb = __shfl_sync(0xffffffffu, pb[from / 4], from % 4, 4);
                        const uint32_t oa = kZero ? __byte_perm(qa, qa, 0x1010) : 0xbe00be00u;
                        const uint32_t ob = kZero ? __byte_perm(qb, qb, 0x1010) : 0xbe00be00u;
                        float acc[NT][4];
#pragma unroll
                        for (int w = 0; w < kWords; ++w) {
                            uint32_t a[4], b[4];
                            unpack(wa[e * kWords + w], oa, a);
                            unpack(wb[e * kWords + w], ob, b);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint4 v = stream::lds128(xa + i * kXStep + (e * kWords + w) * kWordBytes + nt * 512);
                                if (w == 0)
                                    stream::mma_16816_z(acc[nt], a[0], b[0], a[1], b[1], v.x, v.y);
                                else
                                    mma_16816(acc[nt], a[0], b[0], a[1], b[1], v.x, v.y);
                                mma_16816(acc[nt], a[2], b[2], a[3], b[3], v.z, v.w);
                            }
                        }
                        const float f0 = __uint_as_float(qa & 0xffff0000u), f1 = __uint_as_float(qb & 0xffff0000u);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            out[nt][0] = __fmaf_rn(f0, acc[nt][0], out[nt][0]);
                            out[nt][1] = __fmaf_rn(f0, acc[nt][1], out[nt][1]);
                            out[nt][2] = __fmaf_rn(f1, acc[nt][2], out[nt][2]);
                            out[nt][3] = __fmaf_rn(f1, acc[nt][3], out[nt][3]);
                        }
                    }
                }
            }
            xa += kSlots * kXStep;
        }
        if (len == 0) {  // a part without steps; the batch after it may have some
            ahead_len = part(batch + 1, tile, lo);
            if (ahead_len) {
                begin(tile, lo);
                load_scales(ahead_len);
            }
#pragma unroll
            for (int i = 0; i < kSlots; ++i) copy(i, i < ahead_len);
        }
        len = ahead_len;
        // The batch before is rounded only now: its sums, other CTAs' too, have arrived meanwhile. Two buffers do: a CTA
        // writes one again after a barrier at which every CTA had read it.
        if (batch > 0) {
            stream::cluster_wait_acquire();
            finish(batch - 1);
        }
        float *to = sums + (batch & 1) * kSums + warp * (kRows * kCols);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            *reinterpret_cast<float2 *>(to + g * kCols + 8 * nt + 2 * t) = make_float2(out[nt][0], out[nt][1]);
            *reinterpret_cast<float2 *>(to + (g + 8) * kCols + 8 * nt + 2 * t) = make_float2(out[nt][2], out[nt][3]);
        }
        __syncwarp();
        stream::cluster_arrive_release();
    }
    stream::cluster_wait_acquire();
    finish(batches - 1);
    stream::cluster_arrive_release();  // no CTA leaves while another reads its sums
    stream::cluster_wait_acquire();
}

size_t smem_bytes(int64_t k, int slices, int nt) {
    const int64_t steps = (k + kStep - 1) / kStep, each = (steps + slices - 1) / slices;
    return static_cast<size_t>(kWarps) * (2 * kRows * 8 * nt * 4 + kSlots * kStepBytes) + static_cast<size_t>(each) * kStep * 2 * 8 * nt;
}

// x of more than 8 tokens fits on a cluster.
bool fits16(int64_t k) { return smem_bytes(k, 8, 2) <= kSmemMost; }

static_assert((kInt4LinearMaxK / kStep + 7) / 8 * kStep * 2 * 8 + kWarps * (2 * kRows * 8 * 4 + kSlots * kStepBytes) <= kSmemMost,
              "x of 8 tokens fits on a cluster");

// CTAs of a cluster and clusters: those with the least estimated time in ns. A turn of the loop (16 warps, a step each)
// takes about 0.45 us, a batch beyond the first 1 us, or 2 us with sums across CTAs, copying x 1 us per 64 KB. Measured with
// 1, 2, 4 and 8 slices: 4096 x 4096 at 1 token 7.1, 6.7, 6.8, 11.1 us, 11008 x 4096 at 5 tokens 14.6, 14.1, 16.7, 19.8 us.
// The plan is made for 16 tokens (or the 8 that fit) whatever M, so that a token's sums are added in the same order, and come
// out the same, in any batch.
cudaError_t plan(LinArgs *p, int *clusters) {
    static thread_local uint64_t ctx = 0;
    static thread_local int dev = -1, fit[4] = {};  // resident clusters of 1, 2, 4 and 8 CTAs, for the thread's last context
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return e;
    const uint64_t c = current_context_id();
    if (d != dev || c != ctx || c == 0) {
        for (int i = 0; i < 4; ++i) {
            e = resident_clusters(reinterpret_cast<const void *>(k_int4_linear<4, 2, true>), kThreads, 1 << i, kSmemMost, &fit[i]);
            if (e != cudaSuccess) return e;
        }
        dev = d;
        ctx = c;
    }
    const int64_t steps = (p->k + kStep - 1) / kStep;
    const int nt = fits16(p->k) ? 2 : 1;
    int64_t least = 0;
    p->slices = 0;
    for (int i = 0; i < 4; ++i) {
        const int S = 1 << i;
        if (fit[i] <= 0 || smem_bytes(p->k, S, nt) > kSmemMost) continue;
        const int64_t C = p->tiles < fit[i] ? p->tiles : fit[i], most = (p->tiles + C - 1) / C;
        const int64_t full = (most - 1) / kWarps, splits = kWarps / (most - full * kWarps), len = (steps + S - 1) / S;
        const int64_t cost = 450 * (full * len + (len + splits - 1) / splits) + (S > 1 ? 2000 : 1000) * full + len * (kStep * 2 * 8 / 64) * nt;
        if (p->slices == 0 || cost < least) {
            least = cost;
            p->slices = S;
            *clusters = static_cast<int>(C);
        }
    }
    return p->slices ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int kWords, int NT, bool kZero>
cudaError_t launch(const LinArgs &p, int clusters, cudaStream_t st) {
    const size_t smem = smem_bytes(p.k, p.slices, NT);
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(k_int4_linear<kWords, NT, kZero>), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters) * static_cast<unsigned>(p.slices), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.slices);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.slices > 1 ? 2 : 1;  // a launch of clusters starts about 0.4 us later, of one CTA each too
    e = cudaLaunchKernelEx(&cfg, k_int4_linear<kWords, NT, kZero>, p);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <int kWords>
cudaError_t launch_words(const LinArgs &p, int clusters, cudaStream_t st) {
    if (p.M <= 8) return p.zero_point ? launch<kWords, 1, true>(p, clusters, st) : launch<kWords, 1, false>(p, clusters, st);
    return p.zero_point ? launch<kWords, 2, true>(p, clusters, st) : launch<kWords, 2, false>(p, clusters, st);
}

}  // namespace

cudaError_t launch_int4_linear(const Int4View &w, const uint16_t *x, int M, uint16_t *h, cudaStream_t st) {
    LinArgs p{w.codes, w.scale, w.zero_point, w.n, w.k, x, M, h, (w.n + kRows - 1) / kRows, 0};
    int clusters = 0;
    cudaError_t e = plan(&p, &clusters);
    const int most = fits16(w.k) ? kInt4Tokens : 8;
    for (int m0 = 0; m0 < M && e == cudaSuccess; m0 += most) {
        p.x = x + m0 * w.k;
        p.h = h + m0 * w.n;
        p.M = M - m0 < most ? M - m0 : most;
        e = w.group == 32 ? launch_words<1>(p, clusters, st) : w.group == 64 ? launch_words<2>(p, clusters, st) : launch_words<4>(p, clusters, st);
    }
    return e;
}

}  // namespace qn
