// act8_grads_tc.cu -- the adapter gradients of act8_grads.cu on the 5th-generation tensor cores (tcgen05, TMEM,
// TMA), for long batches:
//
//   t = x A^T, u = grad_h B;   grad_B = s grad_h^T t,  grad_A = s u^T x,   x = q a / 127
//
// Both products read each element of grad_h and of the codes once and are bound by that; the matrix work per
// byte grows with the rank and would bound the kernels on mma.sync from r = 32 on.
//
// Operands. grad_h tiles come by TMA and are used as they are. Codes come by TMA and eight or four warps turn
// them into bf16: q a / 128 has at most 15 significant bits, so it is exactly hi + lo, two bf16 (hi the rounded
// product, lo the fma of the rest), and each gets its own MMA. (a / 128 keeps the largest a in range; below
// 2^-126 it is a bf16 subnormal and loses bits that are below 2^-133 of anything.) The missing 128 / 127 goes
// into s. t and u, fp32 sums, are passed on as three bf16 terms (24 bits); their products with x or grad_h land in
// three groups of accumulator columns that the epilogue adds.
//
//   k_down_tc   one CTA: 128 tokens (the MMA's M) of x or of grad_h, N = r; a cluster splits the features and adds
//               its sums through distributed shared memory.
//   k_outer_tc  one CTA: 256 columns of x or of grad_h as two accumulators of 128 (M), N = 3 r, K = tokens; both
//               operands are read with their M or N index contiguous, as they lie. A cluster splits the
//               tokens. The second kernel walks the tokens backwards: what the first read last is still in L2.
//
// Warp 0 issues the TMA loads, warp 1 the MMAs, the others convert codes and run the epilogue. Every wait is
// bounded; a CTA whose wait runs out drains what it issued and its results are NaN.
#include <cudaTypedefs.h>

#include "act8.cuh"
#include "act8.h"
#include "dropout.cuh"
#include "host_cache.h"
#include "sm100.cuh"
#include "stream_common.cuh"

namespace qn {

namespace {

using namespace sm100;

struct TcArgs {
    const uint16_t *absmax;
    int64_t M, n, k;
    int r, j0;       // this pass: adapter columns j0 .. j0 + rp of r
    int rp;          // 16, 32, 48 or 64
    int chunks;      // 64-column pieces of a row of t or u: its three terms, rp columns each
    float s;         // already times 128 / 127
    float *grad_A, *grad_B;
    uint16_t *t, *u;  // M x 64 chunks
    DropoutArgs drop;
};

constexpr int kK = 64;                    // features or tokens per stage: a 128-byte swizzled row of bf16
constexpr uint32_t kChunk = 64 * 64 * 2;  // a 64 x 64 bf16 tile

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cta_ranks() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Four neighbouring floats at p of every CTA of the cluster, added in rank order.
__device__ __forceinline__ void cluster_sum(const float *p, uint32_t ranks, float (&v)[4]) {
    if (ranks == 1) {
        const float4 f = *reinterpret_cast<const float4 *>(p);
        v[0] = f.x;
        v[1] = f.y;
        v[2] = f.z;
        v[3] = f.w;
        return;
    }
    v[0] = v[1] = v[2] = v[3] = 0.0f;
    for (uint32_t c = 0; c < ranks; c += 2) {  // 2, 4 or 8 ranks; two loads in flight
        float f[8];
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h)
            asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(f[4 * h]), "=f"(f[4 * h + 1]), "=f"(f[4 * h + 2]), "=f"(f[4 * h + 3])
                         : "r"(stream::mapa(smem_u32(p), c + h))
                         : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (v[i] + f[i]) + f[4 + i];
    }
}

__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&v)[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

__device__ __forceinline__ uint32_t bf2(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t *>(&v); }
__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162 *>(&v); }

// A block of 64 codes, a 64-byte swizzled row of shared memory, to a 128-byte swizzled row of bf16 at `hi`. kScaled:
// times a / 128, as hi + lo, lo kLo bytes behind hi; else the codes themselves. `row` is the row's index in its tile (its
// low three bits swizzle both). A whole block per thread: with half of one, waits and addresses were half of the
// instructions, and the warps that convert are bound by issuing them.
template <bool kScaled, uint32_t kLo, bool kDrop>
__device__ __forceinline__ void convert_block(uint32_t codes, uint32_t row, float a, const DropoutArgs &drop, uint64_t e0,
                                              uint32_t hi) {
    const __nv_bfloat162 f = __float2bfloat162_rn(a * 0.0078125f);
    const uint32_t src = codes + (((row >> 1) & 3u) << 4), dst = hi + ((row & 7u) << 4);
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(src ^ (c << 4)) : "memory");
        if (kDrop) {
            const uint32_t keep = dropout_keep_bits(drop, e0 + 16 * c, 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t b = keep >> (4 * i);
                w[i] &= ((b & 1u) | (b & 2u) << 7 | (b & 4u) << 14 | (b & 8u) << 21) * 0xffu;
            }
        }
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            uint32_t oh[4], ol[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // two codes as a bf16 pair: 128 + the low seven bits, less 128 or (sign bit) 256; exact
                const uint32_t p = __byte_perm(w[2 * h + (i >> 1)], 0u, (i & 1) ? 0x4342 : 0x4140);
                const __nv_bfloat162 q =
                    __hsub2(as_bf2((p & 0x007f007fu) | 0x43004300u), as_bf2((p & 0x00800080u) | 0x43004300u));
                if (kScaled) {
                    const __nv_bfloat162 top = __hmul2(q, f);
                    oh[i] = bf2(top);
                    ol[i] = bf2(__hfma2(q, f, __hneg2(top)));
                } else {
                    oh[i] = bf2(q);
                }
            }
            const uint32_t to = dst ^ ((2 * c + h) << 4);
            sts128(to, oh);
            if (kScaled) sts128(to + kLo, ol);
        }
    }
}

// A place in a ring of n slots: the slot, and the parity of its phase in this round. (Slot and phase by division of a
// step count by n cost the one thread that issues MMAs more time than the MMAs.)
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// Waits for the last phase that `count` steps put on each of n barriers; `at` is the place behind the last step.
__device__ __forceinline__ void wait_out(uint64_t *bars, int n, int count, Ring at) {
    for (int e = count < n ? count : n; e > 0; --e) {
        if (--at.slot < 0) {
            at.slot = n - 1;
            at.phase ^= 1u;
        }
        mbar_wait(&bars[at.slot], at.phase);
    }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// Whether the phase is over; does not wait.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// The producer of the codes and of the second operand (the factor, or t or u): two rings that empty at their own
// pace. Neither waits for the other: issued in step order by one blocking thread, the second operand's load would
// go out only when the codes' slot is free, and its latency would be in every step. Issues what has room until all
// `steps` are out; gives up after about a second without progress. Returns false then.
template <typename Codes, typename Second>
__device__ __forceinline__ bool feed(int steps, int &ci, Ring &c, int slots, uint64_t *cempty, Codes &&codes, int &ri, Ring &r,
                                     int rslots, uint64_t *rempty, Second &&second, volatile uint32_t *abort_flag) {
    uint32_t idle = 0;
    while (ci < steps || ri < steps) {
        bool did = false;
        if (ri < steps && (ri < rslots || mbar_test(&rempty[r.slot], r.phase ^ 1u))) {
            second(ri, r.slot);
            ++ri;
            r.next(rslots);
            did = true;
        }
        if (ci < steps && (ci < slots || mbar_test(&cempty[c.slot], c.phase ^ 1u))) {
            codes(ci, c.slot);
            ++ci;
            c.next(slots);
            did = true;
        }
        idle = did ? 0u : idle + 1u;
        if (idle > (1u << 24) || *abort_flag) return false;
    }
    return true;
}

// A warp that brings the absmaxes of coming steps to shared memory, four steps (a batch) at a time in a ring of
// three batches of kGroups x 4 values: `at(step, group)` points at four neighbouring ones, of which `count` exist. In the
// converting warps themselves the loads' latency showed in every fourth step.
constexpr int kBatch = 4, kBatches = 3;

__device__ __forceinline__ uint64_t load4(const uint16_t *p, int count) {
    if (count >= 4 && (reinterpret_cast<uintptr_t>(p) & 7u) == 0) return __ldg(reinterpret_cast<const unsigned long long *>(p));
    uint64_t v = 0;
#pragma unroll 1
    for (int i = 0; i < count && i < 4; ++i) v |= static_cast<uint64_t>(ld_ro_u16(p + i)) << (16 * i);
    return v;
}

template <int kGroups, typename At>
__device__ __forceinline__ bool load_absmax(int steps, uint64_t *ring, uint64_t *afull, uint64_t *aempty, int lane, At &&at) {
    Ring b;
    for (int i = 0; i < steps; i += kBatch, b.next(kBatches)) {
        uint64_t v[kGroups / 32];
#pragma unroll
        for (int g = 0; g < kGroups / 32; ++g) {
            int count;
            const uint16_t *p = at(i, 32 * g + lane, count);
            v[g] = load4(p, count);
        }
        if (i >= kBatches * kBatch && !mbar_wait(&aempty[b.slot], b.phase ^ 1u)) return false;
#pragma unroll
        for (int g = 0; g < kGroups / 32; ++g) ring[b.slot * kGroups + 32 * g + lane] = v[g];
        __syncwarp();
        if (lane == 0) mbar_arrive(&afull[b.slot]);
    }
    return true;
}

// -------------------------------------------------------------------------------- t and u

constexpr int kDownTile = 128;
constexpr int kDownWarps = 8;  // converters, two groups that take steps in turn
constexpr int kDownThreads = 96 + 32 * kDownWarps;  // with the producer, the MMA and the absmax warp
constexpr uint32_t kDownTmem = 256;
constexpr int kDownStagesGh = 4, kDownStagesX = 3;
constexpr uint32_t kDownA = 2 * kChunk;  // 128 tokens x 64 features
constexpr uint32_t kDownGh = kDownA + kChunk;
constexpr uint32_t kDownRing = 104 * 1024;
// Of x: three tiles with a piece of A each (rp rows of 128 bytes), and what is left for codes, at most 4 slots.
__host__ __device__ constexpr int down_codes(int rp) {
    const uint32_t left = kDownRing - static_cast<uint32_t>(kDownStagesX) * (kDownA + static_cast<uint32_t>(rp) * 128u);
    const int n = static_cast<int>(left / (kDownA / 2));
    return n > 4 ? 4 : n;
}
static_assert(kDownStagesGh * kDownGh <= kDownRing && down_codes(64) == 4, "");
constexpr int kDownRedRow = 68;  // floats: rows start on 16 bytes, eight neighbouring ones on different banks
static_assert(2 * kDownTile * kDownRedRow * 4 <= kDownRing, "");
constexpr uint32_t kDownAbsmax = kBatches * kBatch * kDownTile * 2;
constexpr size_t kDownSmem = 1024 + kDownRing + kDownAbsmax + 512;

template <bool kX, bool kDrop>
__device__ __forceinline__ void down_tc(const CUtensorMap *act, const CUtensorMap *factor, const TcArgs &p, uint8_t *smem,
                                        uint64_t *bars, int64_t tile, uint32_t rank, uint32_t ranks) {
    constexpr int kStages = kX ? kDownStagesX : kDownStagesGh;
    uint64_t *full = bars, *empty = full + 4, *cfull = empty + 4, *cempty = cfull + 4;
    uint64_t *afull = cempty + 4, *aempty = afull + kBatches, *done = aempty + kBatches;
    uint32_t *slot = reinterpret_cast<uint32_t *>(done + 1);
    volatile uint32_t *abort_flag = slot + 1;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int64_t pieces = ((kX ? p.k : p.n) + kK - 1) / kK;
    const int64_t lo = pieces * rank / ranks;
    const int steps = static_cast<int>(pieces * (rank + 1) / ranks - lo);
    const int32_t tok0 = static_cast<int32_t>(tile * kDownTile);
    // a stage: the tile and the factor's piece; kX: the codes behind the stages
    const uint32_t piece = kX ? static_cast<uint32_t>(p.rp) * 128u : kChunk, stage = kDownA + piece;
    const int slots = down_codes(p.rp);
    uint8_t *codes = smem + kStages * stage;
    uint16_t *absmax = reinterpret_cast<uint16_t *>(smem + kDownRing);

    if (threadIdx.x == 0) {
        for (int s = 0; s < 4; ++s) {
            mbar_init(&full[s], kX ? 1 + kDownWarps / 2 : 1);  // TMA: the factor's piece and grad_h's tile; kX: the converted tile
            mbar_init(&empty[s], 1);                           // the stage's MMAs are done
            mbar_init(&cfull[s], 1);                           // TMA: codes
            mbar_init(&cempty[s], kDownWarps / 2);             // the group's warps have read them
        }
        for (int s = 0; s < kBatches; ++s) {
            mbar_init(&afull[s], 1);
            mbar_init(&aempty[s], kDownWarps);
        }
        mbar_init(done, 1);
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(slot, kDownTmem);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(act);
        tma_prefetch_desc(factor);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    grid_dependents_launch();
    // The tensor core cuts off what it adds instead of rounding it, so a long chain of MMAs drifts (448 of them: 1.6e-5
    // of the sum). grad_h: the K steps go round `accs` accumulators, which the epilogue adds. x: the codes go in as they
    // are, 64 features to a fresh accumulator, and the converting warps add it up times a / 128 in fp32.
    const int accs = p.rp <= 32 ? 8 : 4;

    // Warps 2 .. 9 have 32 lanes (tokens) of the accumulators each: of x all columns of every other step, of grad_h every
    // other accumulator.
    const uint32_t quarter = static_cast<uint32_t>(warp & 3);
    const int group = (warp - 2) >> 2;
    float sum[4][16];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int q = 0; q < 16; ++q) sum[e][q] = 0.0f;
    // adds the accumulator in columns from d on, times a
    auto add = [&](uint32_t d, float a) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (16 * e < p.rp) {
                uint32_t v[16];
                tmem_ld16(tmem + ((quarter * 32u) << 16) + d + 16 * e, v);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 16; ++q) sum[e][q] = __fmaf_rn(a, __uint_as_float(v[q]), sum[e][q]);
            }
    };

    if (warp == 0) {
        if (lane == 0) {
            if (kX) {
                int ci = 0, ri = 0;
                Ring c, r;
                if (!feed(
                        steps, ci, c, slots, cempty,
                        [&](int i, int q) {
                            mbar_arrive_expect_tx(&cfull[q], kDownA / 2);
                            for (int h = 0; h < 2; ++h)
                                tma_load_2d(codes + q * (kDownA / 2) + h * 4096, act, &cfull[q], static_cast<int32_t>((lo + i) * kK), tok0 + 64 * h);
                        },
                        ri, r, kStages, empty,
                        [&](int i, int q) {
                            mbar_arrive_expect_tx(&full[q], piece);
                            tma_load_2d(smem + q * stage + kDownA, factor, &full[q], static_cast<int32_t>((lo + i) * kK), p.j0);
                        },
                        abort_flag))
                    *abort_flag = 1u;
                // every load has landed before the CTA may leave
                wait_out(full, kStages, ri, r);
                wait_out(cfull, slots, ci, c);
            } else {
                int i = 0;
                Ring r;
                for (; i < steps && !*abort_flag; ++i, r.next(kStages)) {
                    if (i >= kStages && !mbar_wait(&empty[r.slot], r.phase ^ 1u)) {
                        *abort_flag = 1u;
                        break;
                    }
                    uint8_t *st = smem + r.slot * stage;
                    const int32_t c0 = static_cast<int32_t>((lo + i) * kK);
                    mbar_arrive_expect_tx(&full[r.slot], stage);
                    tma_load_2d(st, act, &full[r.slot], c0, tok0);
                    tma_load_2d(st + kChunk, act, &full[r.slot], c0, tok0 + 64);
                    tma_load_2d(st + kDownA, factor, &full[r.slot], p.j0, c0);  // 64 rows of B
                }
                wait_out(full, kStages, i, r);
            }
        }
    } else if (warp == 1) {
        // The whole warp keeps step and one lane issues: the descriptors stay in uniform registers. From a lane of its own,
        // an MMA took the thread 60 ns.
        const bool leader = elect();
        const uint32_t idesc = idesc_bf16(kDownTile, p.rp, 0, kX ? 0 : 1);
        // the descriptors of slot 0; a slot or a K step further is an addition to the address (in 16-byte units)
        const uint64_t a0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t b0 = kX ? smem_desc_sw128(smem_u32(smem) + kDownA, 16, 1024) : smem_desc_sw128(smem_u32(smem) + kDownA, kChunk, 1024);
        int i = 0;
        Ring r;
        for (; i < steps; ++i, r.next(kStages)) {
            if (!mbar_wait(&full[r.slot], r.phase)) break;
            __syncwarp();
            tc_fence_after();
            const uint64_t a = a0 + r.slot * (stage / 16), b = b0 + r.slot * (stage / 16);
            const uint32_t d = tmem + (kX ? static_cast<uint32_t>(r.slot) : static_cast<uint32_t>(4 * i) & static_cast<uint32_t>(accs - 1)) * p.rp;
            const uint32_t more = 4 * i >= accs ? 1u : 0u;  // the K steps of a stage start new accumulators together
            if (leader) {
#pragma unroll
                for (uint32_t kk = 0; kk < 4; ++kk)
                    mma_bf16_ss(kX ? d : d + kk * p.rp, a + 2 * kk, b + (kX ? 2 : 128) * kk, idesc, kX ? (kk > 0 ? 1u : 0u) : more);
                mma_commit(&empty[r.slot]);
            }
            __syncwarp();
        }
        if (i < steps) *abort_flag = 1u;
        if (leader) mma_commit(done);
        wait_out(empty, kStages, i, r);  // every commit has arrived before the CTA may leave
    } else if (kX && warp == kDownThreads / 32 - 1) {
        const int64_t blocks = p.k / kBlock;
        // a group: the batch's four steps of a token
        if (!load_absmax<kDownTile>(steps, reinterpret_cast<uint64_t *>(absmax), afull, aempty, lane, [&](int i, int row, int &count) {
                const int64_t m = tok0 + static_cast<int64_t>(row);
                count = m < p.M ? steps - i : 0;
                return p.absmax + (m < p.M ? m : 0) * blocks + lo + i;
            }))
            *abort_flag = 1u;
    } else if (kX) {
        const uint32_t row = (threadIdx.x - 64) & 127u;  // a token
        const int64_t m = tok0 + static_cast<int64_t>(row);
        Ring r, c, b;
        if (group == 1) {
            r.next(kStages);
            c.next(slots);
        }
        bool ok = true;
        // At step i the slot's last step, i - 3, is over: its accumulator is taken, then the slot is filled again. So MMAs
        // never run into an accumulator that is not taken. The loop goes on past the end for the last three.
        for (int i = group; ok && i < steps + kStages; i += 2) {
            const int e = i - kStages, q = e & (kBatch - 1);
            if (e >= 0) {
                ok = (q > 1 || mbar_wait(&afull[b.slot], b.phase)) && mbar_wait(&empty[r.slot], r.phase ^ 1u);
                if (!ok) break;
                tc_fence_after();
                add(static_cast<uint32_t>(r.slot * p.rp),
                    __uint_as_float(static_cast<uint32_t>(absmax[(b.slot * kDownTile + quarter * 32 + lane) * kBatch + q]) << 16) * 0.0078125f);
                tc_fence_before();
                __syncwarp();
                if (q > 1) {
                    if (lane == 0) mbar_arrive(&aempty[b.slot]);
                    b.next(kBatches);
                }
            }
            if (i < steps) {
                ok = mbar_wait(&cfull[c.slot], c.phase);
                if (!ok) break;
                convert_block<false, 0u, kDrop>(smem_u32(codes) + c.slot * (kDownA / 2) + row * 64u, row, 1.0f, p.drop,
                                                p.drop.offset + static_cast<uint64_t>(m * p.k + (lo + i) * kK),
                                                smem_u32(smem) + r.slot * stage + row * 128u);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&cempty[c.slot]);
                    mbar_arrive(&full[r.slot]);
                }
            }
            r.next(kStages);
            r.next(kStages);
            c.next(slots);
            c.next(slots);
        }
        if (!ok) *abort_flag = 1u;
    }
    __syncthreads();  // every load has landed: the ring is free for the sums

    // the CTA's sums to shared memory, a row per token; the second group's next to the first's
    float *red = reinterpret_cast<float *>(smem);
    if (warp >= 2 && warp < 2 + kDownWarps) {
        const bool ok = mbar_wait(done, 0) && !*abort_flag;
        tc_fence_after();
        if (!kX)
            for (int q = group; q < accs && q < 4 * steps; q += 2) add(static_cast<uint32_t>(q * p.rp), 1.0f);
        float4 *dst = reinterpret_cast<float4 *>(red + (group * kDownTile + quarter * 32 + lane) * kDownRedRow);
        const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (16 * e < p.rp) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    dst[4 * e + c] = ok ? make_float4(sum[e][4 * c], sum[e][4 * c + 1], sum[e][4 * c + 2], sum[e][4 * c + 3]) : make_float4(nan, nan, nan, nan);
            }
        tc_fence_before();
    }
    __syncwarp();
    if (ranks > 1) {
        stream::cluster_arrive_release();
        stream::cluster_wait_acquire();
    } else {
        __syncthreads();
    }
    // each rank adds up its share of the tokens: four columns of one token per thread, in three bf16 terms
    uint16_t *out = kX ? p.t : p.u;
    const int ld = 64 * p.chunks, quads = p.rp / 4;
    const int t0 = static_cast<int>(kDownTile * rank / ranks), t1 = static_cast<int>(kDownTile * (rank + 1) / ranks);
    for (int e = threadIdx.x; e < (t1 - t0) * quads; e += kDownThreads) {
        const int tok = t0 + e / quads, j = 4 * (e % quads);
        const int64_t m = tok0 + static_cast<int64_t>(tok);
        if (m >= p.M) continue;
        float v[4], w2[4];
        cluster_sum(red + tok * kDownRedRow + j, ranks, v);
        cluster_sum(red + (kDownTile + tok) * kDownRedRow + j, ranks, w2);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += w2[i];
        uint16_t *o = out + m * ld + j;
#pragma unroll
        for (int term = 0; term < 3; ++term) {
            uint32_t w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[h] = pack_bf16x2(v[2 * h], v[2 * h + 1]);
                v[2 * h] -= bf16_lo(w[h]);
                v[2 * h + 1] -= bf16_hi(w[h]);
            }
            *reinterpret_cast<uint2 *>(o + term * p.rp) = make_uint2(w[0], w[1]);
        }
    }
    __syncwarp();
    if (ranks > 1) {  // no CTA leaves while another reads its sums
        stream::cluster_arrive_release();
        stream::cluster_wait_acquire();
    } else {
        __syncthreads();
    }
    if (warp == 1) tmem_dealloc(tmem, kDownTmem);
}

// grid (ranks * token tiles, 2): y = 0 takes u from grad_h, y = 1 t from the codes.
template <bool kDrop>
__global__ void __launch_bounds__(kDownThreads, 2)
k_down_tc(const __grid_constant__ CUtensorMap tm_gh, const __grid_constant__ CUtensorMap tm_codes,
          const __grid_constant__ CUtensorMap tm_A, const __grid_constant__ CUtensorMap tm_B, const TcArgs p) {
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kDownRing + kDownAbsmax);
    const uint32_t rank = cta_rank(), ranks = cta_ranks();
    const int64_t tile = blockIdx.x / ranks;
    if (blockIdx.y == 0)
        down_tc<false, false>(&tm_gh, &tm_B, p, smem, bars, tile, rank, ranks);
    else
        down_tc<true, kDrop>(&tm_codes, &tm_A, p, smem, bars, tile, rank, ranks);
}

// ------------------------------------------------------------------------ products over tokens

constexpr int kOutCols = 256;
constexpr int kOutWarps = 16;  // converters, four groups with a slot each that take steps in turn
constexpr int kTokX = 32;      // tokens per step of x: with 64 and two slots a slot's round trip was the bound
constexpr int kOutThreads = 96 + 32 * kOutWarps;  // with the producer, the MMA and the absmax warp
constexpr int kDrain = 16;  // steps (4 MMAs on an accumulator each) between two drains
constexpr uint32_t kOutA = 4 * kChunk;  // 64 tokens x 256 columns
constexpr int kOutRowX = kOutCols + 4;  // floats per row j of the sums of x
constexpr int kOutRowGh = 68;           // floats per column of grad_h of its sums
constexpr uint32_t kOutAbsmax = kBatches * kBatch * kTokX * 8;
constexpr uint32_t kOutRed = kOutCols * kOutRowGh * 4;
static_assert(64 * kOutRowX * 4 <= kOutRed, "");
constexpr int kOutStagesX = 4;
constexpr uint32_t kOutTileX = kTokX * kOutCols * 2;  // bytes of hi, or of lo
constexpr uint32_t kChunkX = kTokX * 64 * 2;

// For a row of t or u of 1, 2 or 3 pieces: stages of grad_h, each with t; of x four, with u and codes.
__host__ __device__ constexpr int out_stages(int chunks) { return chunks == 1 ? 5 : chunks == 2 ? 4 : 3; }
__host__ __device__ constexpr uint32_t out_ring(int chunks) {
    const uint32_t gh = static_cast<uint32_t>(out_stages(chunks)) * (kOutA + static_cast<uint32_t>(chunks) * kChunk);
    const uint32_t x = kOutStagesX * (2 * kOutTileX + static_cast<uint32_t>(chunks) * kChunkX) + kOutStagesX * (kOutTileX / 2);
    return gh > x ? gh : x;
}
static_assert(out_ring(1) <= 216 * 1024 && out_ring(2) <= 216 * 1024 && out_ring(3) <= 216 * 1024, "");
static_assert(out_ring(1) >= kOutRed && out_ring(2) >= kOutRed && out_ring(3) >= kOutRed, "");

template <bool kX, bool kDrop>
__device__ __forceinline__ void outer_tc(const CUtensorMap *act, const CUtensorMap *mid, const TcArgs &p, uint8_t *smem,
                                         uint64_t *bars, int64_t tile, uint32_t rank, uint32_t ranks) {
    constexpr int kTok = kX ? kTokX : kK;
    const int stages = kX ? kOutStagesX : out_stages(p.chunks);
    constexpr int slots = kOutStagesX;  // of codes
    const uint32_t mid_bytes = p.chunks * (kX ? kChunkX : kChunk), stage = (kX ? 2 * kOutTileX : kOutA) + mid_bytes;
    uint64_t *full = bars, *empty = full + 5, *cfull = empty + 5, *cempty = cfull + 5;
    uint64_t *afull = cempty + 5, *aempty = afull + kBatches, *done = aempty + kBatches, *drained = done + 1;
    uint32_t *slot = reinterpret_cast<uint32_t *>(drained + 1);
    volatile uint32_t *abort_flag = slot + 1;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int64_t width = kX ? p.k : p.n;
    const int32_t col0 = static_cast<int32_t>(tile * kOutCols);
    const int64_t all = (p.M + kTok - 1) / kTok;
    const int64_t lo = all * rank / ranks;
    const int steps = static_cast<int>(all * (rank + 1) / ranks - lo);
    // a stage: the tile (kX: hi and lo), then t or u; kX: the codes behind the stages
    uint8_t *codes = smem + stages * stage;
    uint16_t *absmax = reinterpret_cast<uint16_t *>(smem + out_ring(p.chunks));
    // step i works on the tokens from tok(i) on: the last ones first
    auto tok = [&](int i) { return static_cast<int32_t>((lo + steps - 1 - i) * kTok); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < 5; ++s) {
            mbar_init(&full[s], kX ? 1 + kOutWarps / 4 : 1);  // TMA: t or u, and grad_h; kX: the group's tile
            mbar_init(&empty[s], 1);
            mbar_init(&cfull[s], 1);
            mbar_init(&cempty[s], kOutWarps / 4);
        }
        for (int s = 0; s < kBatches; ++s) {
            mbar_init(&afull[s], 1);
            mbar_init(&aempty[s], kOutWarps);
        }
        mbar_init(done, 1);             // the MMAs up to a drain are done
        mbar_init(drained, kOutWarps);  // the warps have read the accumulators
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(act);
        tma_prefetch_desc(mid);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;

    // The accumulators are emptied into registers every kDrain steps: the tensor core cuts off what it adds instead of
    // rounding it, and a chain of 256 MMAs would be off by 1e-5. Warps 2 .. 17 have 32 lanes (columns) of one of the two
    // accumulators each, and every other 16 of the columns j.
    const uint32_t quarter = static_cast<uint32_t>(warp & 3), h = (static_cast<uint32_t>(warp - 2) >> 2) & 1u;
    const int jb0 = (warp - 2) >> 3;
    float sum[2][16];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int c = 0; c < 16; ++c) sum[b][c] = 0.0f;
    auto drain = [&](uint32_t nth) -> bool {
        if (!mbar_wait(done, nth & 1u)) return false;
        tc_fence_after();
        const uint32_t d = tmem + 256 * h + ((quarter * 32u) << 16);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int j = 16 * (jb0 + 2 * b);
            if (j < p.rp) {
                uint32_t v0[16], v1[16], v2[16];
                tmem_ld16(d + j, v0);
                tmem_ld16(d + p.rp + j, v1);
                tmem_ld16(d + 2 * p.rp + j, v2);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    sum[b][c] += __uint_as_float(v0[c]) + (__uint_as_float(v1[c]) + __uint_as_float(v2[c]));
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(drained);
        return true;
    };

    if (warp == 0) {
        if (lane == 0) {
            // Up to the dependency wait only x and grad_h are read, which the preceding kernel reads too.
            if (kX) {
                int ci = 0, ri = 0;
                Ring c, r;
                auto load_codes = [&](int i, int q) {
                    mbar_arrive_expect_tx(&cfull[q], kOutTileX / 2);
                    for (int b = 0; b < 4; ++b)
                        tma_load_2d(codes + q * (kOutTileX / 2) + b * (kChunkX / 2), act, &cfull[q], col0 + 64 * b, tok(i));
                };
                for (; ci < slots && ci < steps; ++ci, c.next(slots)) load_codes(ci, c.slot);
                grid_dependency_wait();
                if (!feed(
                        steps, ci, c, slots, cempty, load_codes, ri, r, stages, empty,
                        [&](int i, int q) {
                            mbar_arrive_expect_tx(&full[q], mid_bytes);
                            for (int e = 0; e < p.chunks; ++e) tma_load_2d(smem + q * stage + 2 * kOutTileX + e * kChunkX, mid, &full[q], 64 * e, tok(i));
                        },
                        abort_flag))
                    *abort_flag = 1u;
                wait_out(full, stages, ri, r);
                wait_out(cfull, slots, ci, c);
            } else {
                int i = 0, issued = 0;  // steps whose t, and whose grad_h, is on its way
                Ring ti, gi;
                auto load_gh = [&]() {
                    mbar_arrive_expect_tx(&full[gi.slot], stage);
                    for (int b = 0; b < 4; ++b)
                        tma_load_2d(smem + gi.slot * stage + b * kChunk, act, &full[gi.slot], col0 + 64 * b, tok(issued));
                    ++issued;
                    gi.next(stages);
                };
                auto load_t = [&]() {
                    for (int e = 0; e < p.chunks; ++e)
                        tma_load_2d(smem + ti.slot * stage + kOutA + e * kChunk, mid, &full[ti.slot], 64 * e, tok(i));
                    ++i;
                    ti.next(stages);
                };
                while (issued < stages && issued < steps) load_gh();
                grid_dependency_wait();
                while (i < steps && !*abort_flag) {
                    if (i >= issued) {
                        if (!mbar_wait(&empty[gi.slot], gi.phase ^ 1u)) {
                            *abort_flag = 1u;
                            break;
                        }
                        load_gh();
                    }
                    load_t();
                }
                while (i < issued) load_t();  // a stage that the loop left without its t gets it, so that its phase ends
                wait_out(full, stages, issued, gi);
            }
        }
    } else if (warp == 1) {
        const bool leader = elect();
        const uint32_t three = idesc_bf16(128, 3 * p.rp, 1, 1), two = idesc_bf16(128, 2 * p.rp, 1, 1);
        constexpr uint32_t kPiece = kX ? kChunkX : kChunk;
        const uint64_t a0 = smem_desc_sw128(smem_u32(smem), kPiece, 1024);
        const uint64_t b0 = smem_desc_sw128(smem_u32(smem) + (kX ? 2 * kOutTileX : kOutA), kPiece, 1024);
        int i = 0;
        Ring r, d;
        for (; i < steps; ++i, r.next(stages)) {
            const bool first = i % kDrain == 0;
            if (first && i > 0) {
                if (!mbar_wait(drained, d.phase)) break;
                d.next(1);
            }
            if (!mbar_wait(&full[r.slot], r.phase)) break;
            __syncwarp();
            tc_fence_after();
            const uint64_t a = a0 + r.slot * (stage / 16), b = b0 + r.slot * (stage / 16);
            const uint32_t more = first ? 0u : 1u;
            if (leader) {
#pragma unroll
                for (uint32_t kk = 0; kk < kTok / 16; ++kk) {
                    const uint64_t bd = b + 128 * kk;
#pragma unroll
                    for (uint32_t half = 0; half < 2; ++half) {
                        const uint64_t ad = a + 2 * half * (kPiece / 16) + 128 * kk;
                        mma_bf16_ss(tmem + 256 * half, ad, bd, three, kk > 0 ? 1u : more);
                        // lo is 2^-8 of hi: its product with the third term is below the fp32 sums
                        if (kX) mma_bf16_ss(tmem + 256 * half, ad + kOutTileX / 16, bd, two, 1u);
                    }
                }
                mma_commit(&empty[r.slot]);
                if (i % kDrain == kDrain - 1 || i + 1 == steps) mma_commit(done);
            }
            __syncwarp();
        }
        if (i < steps) {  // left early: the warps wait for it all the same
            *abort_flag = 1u;
            if (leader) mma_commit(done);
        }
        wait_out(empty, stages, i, r);
    } else if (warp == kOutThreads / 32 - 1) {
        const int64_t blocks = p.k / kBlock, blk0 = col0 / kBlock;
        // a group: a token's four blocks at one of the batch's four steps
        if (kX && !load_absmax<kBatch * kTok>(steps, reinterpret_cast<uint64_t *>(absmax), afull, aempty, lane, [&](int i, int e, int &count) {
                const int64_t m = tok(i + e / kTok) + static_cast<int64_t>(e % kTok);
                const bool live = i + e / kTok < steps && m < p.M;
                count = live ? static_cast<int>(blocks - blk0 < 4 ? blocks - blk0 : 4) : 0;
                return p.absmax + (live ? m : 0) * blocks + blk0;
            }))
            *abort_flag = 1u;
    } else if (!kX) {
        for (int i = 0; i < steps; i += kDrain)
            if (*abort_flag || !drain(static_cast<uint32_t>(i / kDrain))) {
                *abort_flag = 1u;
                break;
            }
    } else {
        // token of the step, block of the tile; the group takes every fourth step, always in the same slot
        const int id = (threadIdx.x - 64) & 127, group = (warp - 2) >> 2;
        const uint32_t row = id & 31u, blk = id >> 5;
        const int64_t col = col0 + 64 * static_cast<int64_t>(blk);
        const uint32_t from = smem_u32(codes) + group * (kOutTileX / 2) + blk * (kChunkX / 2) + row * 64u;
        const uint32_t to = smem_u32(smem) + group * stage + blk * kChunkX + row * 128u;
        Ring b;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = group; i < steps; i += 4, phase ^= 1u) {
            ok = mbar_wait(&afull[b.slot], b.phase) && mbar_wait(&cfull[group], phase) && (i < 4 || mbar_wait(&empty[group], phase ^ 1u));
            if (!ok) break;
            const float a = __uint_as_float(static_cast<uint32_t>(absmax[((b.slot * kBatch + group) * kTok + row) * 4 + blk]) << 16);
            convert_block<true, kOutTileX, kDrop>(from, row, a, p.drop,
                                                  p.drop.offset + static_cast<uint64_t>((tok(i) + static_cast<int64_t>(row)) * p.k + col), to);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&cempty[group]);
                mbar_arrive(&full[group]);
                mbar_arrive(&aempty[b.slot]);
            }
            b.next(kBatches);
            // The drain of the segment before comes after the group's first step of this one: its slot is free by then, the
            // MMAs that would read it wait for the drain.
            if (i >= kDrain && i % kDrain < 4) {
                ok = drain(static_cast<uint32_t>(i / kDrain - 1));
                if (!ok) break;
            }
        }
        // drains that no step of this group followed, and the last one
        if (ok && steps > 0) {
            const int last = (steps - 1) / kDrain;
            if (last > 0 && last * kDrain + group >= steps) ok = drain(static_cast<uint32_t>(last - 1));
            ok = ok && drain(static_cast<uint32_t>(last));
        }
        if (!ok) *abort_flag = 1u;
    }
    __syncthreads();  // every load has landed: the ring is free for the sums

    // the sums to shared memory: of x a row of columns per j, of grad_h a row of j per column, as they go out
    float *red = reinterpret_cast<float *>(smem);
    if (warp >= 2 && warp < 2 + kOutWarps) {
        const bool ok = !*abort_flag;
        const int c = static_cast<int>(h * 128 + quarter * 32 + lane);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int j = 16 * (jb0 + 2 * b);
            if (j >= p.rp) break;
            if (!ok) {
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[b][e] = __uint_as_float(0x7fc00000u);
            }
            if (kX) {
#pragma unroll
                for (int e = 0; e < 16; ++e) red[(j + e) * kOutRowX + c] = sum[b][e];
            } else {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<float4 *>(red + c * kOutRowGh + j + e) =
                        make_float4(sum[b][e], sum[b][e + 1], sum[b][e + 2], sum[b][e + 3]);
            }
        }
    }
    __syncwarp();
    if (ranks > 1) {
        stream::cluster_arrive_release();
        stream::cluster_wait_acquire();
    } else {
        __syncthreads();
    }
    // each rank adds up its share, four neighbouring values of the result per thread
    const int js = p.r - p.j0 < p.rp ? p.r - p.j0 : p.rp;  // a multiple of 8
    const int inner = (kX ? kOutCols : js) / 4, items = inner * (kX ? js : kOutCols);
    const int e0 = static_cast<int>(static_cast<int64_t>(items) * rank / ranks);
    const int e1 = static_cast<int>(static_cast<int64_t>(items) * (rank + 1) / ranks);
    float *out = kX ? p.grad_A : p.grad_B;
    const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
    for (int e = e0 + threadIdx.x; e < e1; e += kOutThreads) {
        const int o = e / inner, q = 4 * (e - o * inner);
        const int j = kX ? o : q, c = kX ? q : o;
        const int64_t cc = col0 + static_cast<int64_t>(c);
        if (cc >= width) continue;  // of x: four columns lie inside or outside together
        float v[4];
        cluster_sum(red + (kX ? j * kOutRowX + c : c * kOutRowGh + j), ranks, v);
        float *dst = out + (kX ? static_cast<int64_t>(p.j0 + j) * p.k + cc : cc * p.r + p.j0 + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= p.s;
        if (vec) {
            *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = v[i];
        }
    }
    __syncwarp();
    if (ranks > 1) {  // no CTA leaves while another reads its sums
        stream::cluster_arrive_release();
        stream::cluster_wait_acquire();
    } else {
        __syncthreads();
    }
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Column tiles of grad_h first, then those of the codes.
template <bool kDrop>
__global__ void __launch_bounds__(kOutThreads, 1)
k_outer_tc(const __grid_constant__ CUtensorMap tm_gh, const __grid_constant__ CUtensorMap tm_codes,
           const __grid_constant__ CUtensorMap tm_t, const __grid_constant__ CUtensorMap tm_u, const TcArgs p) {
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + out_ring(p.chunks) + kOutAbsmax);
    const uint32_t rank = cta_rank(), ranks = cta_ranks();
    const int64_t tile = blockIdx.x / ranks, tiles_gh = (p.n + kOutCols - 1) / kOutCols;
    if (tile < tiles_gh)
        outer_tc<false, false>(&tm_gh, &tm_t, p, smem, bars, tile, rank, ranks);
    else
        outer_tc<true, kDrop>(&tm_codes, &tm_u, p, smem, bars, tile - tiles_gh, rank, ranks);
}

// ------------------------------------------------------------------------------------ host

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// A row-major rows x cols matrix in boxes of box_rows x 64, zeros outside: bf16 (128-byte swizzle) or bytes (64-byte).
bool make_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, bool bytes, uint32_t box_rows = 64) {
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * (bytes ? 1 : 2)};
    const cuuint32_t box[2] = {64, box_rows}, one[2] = {1, 1};
    return fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims,
              strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, bytes ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K>
cudaError_t launch_clusters(K kern, dim3 grid, int threads, size_t smem, int ranks, bool dependent, const CUtensorMap &a,
                            const CUtensorMap &b, const CUtensorMap &c, const CUtensorMap &d, const TcArgs &p,
                            cudaStream_t st) {
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, a, b, c, d, p);
    if (e == cudaSuccess) count_launch();
    return e;
}

int pass_rank(int r) { return r >= 64 ? 64 : (r + 15) / 16 * 16; }
int pass_chunks(int rp) { return (3 * rp + 63) / 64; }

}  // namespace

size_t act8_grads_tc_workspace_bytes(int64_t M, int r) {
    return 2 * ((static_cast<size_t>(M) * pass_chunks(pass_rank(r)) * 128 + 255) & ~size_t(255));
}

bool act8_grads_tc_supported(int64_t M, int64_t n, int r) { return n % 8 == 0 && r % 8 == 0 && M > 0; }

cudaError_t launch_act8_grads_tc(const int8_t *codes, const uint16_t *absmax, const uint16_t *gh, int64_t M, int64_t n,
                                 int64_t k, const uint16_t *A, const uint16_t *B, int r, float s,
                                 const DropoutArgs &drop, float *grad_A, float *grad_B, void *ws, cudaStream_t st) {
    int sms = 148;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    TcArgs p{absmax, M, n, k, r, 0, 0, 0, s * (128.0f / 127.0f), grad_A, grad_B, static_cast<uint16_t *>(ws), nullptr, drop};
    p.u = reinterpret_cast<uint16_t *>(static_cast<char *>(ws) + act8_grads_tc_workspace_bytes(M, r) / 2);
    CUtensorMap tm_gh, tm_codes, tm_codes32, tm_A, tm_B, tm_t, tm_u;
    if (!make_map(&tm_gh, gh, M, n, false) || !make_map(&tm_codes, codes, M, k, true) || !make_map(&tm_codes32, codes, M, k, true, kTokX) || !make_map(&tm_B, B, n, r, false))
        return cudaErrorInvalidValue;
    const int64_t tok = (M + kDownTile - 1) / kDownTile, tiles = (n + kOutCols - 1) / kOutCols + (k + kOutCols - 1) / kOutCols;
    if (tok > (int64_t(1) << 28) || tiles > (int64_t(1) << 28)) return cudaErrorInvalidConfiguration;
    const int64_t pieces = (n > k ? n : k) / kK, steps = (M + kK - 1) / kK;  // of 64; both sides of a cluster have some
    // CTAs of a cluster: as many as keep one wave (two CTAs of the first kernel fit an SM, one of the second)
    auto ranks = [](int64_t tiles, int64_t room, int64_t most) {
        int c = 1;
        while (c < 8 && 2 * c * tiles <= room && 2 * c <= most) c *= 2;
        return c;
    };
    int rd = ranks(2 * tok, 2 * sms, pieces);
    while (rd < 8 && pieces / rd > 64) rd *= 2;  // a wide side: more CTAs than one wave, evener and with shorter sums
    const int ro = ranks(tiles, sms, steps);
    for (p.j0 = 0; p.j0 < r; p.j0 += 64) {
        p.rp = pass_rank(r - p.j0);
        p.chunks = pass_chunks(p.rp);
        if (!make_map(&tm_A, A, r, k, false, static_cast<uint32_t>(p.rp)) || !make_map(&tm_t, p.t, M, 64 * p.chunks, false) || !make_map(&tm_u, p.u, M, 64 * p.chunks, false, kTokX)) return cudaErrorInvalidValue;
        const dim3 gd(static_cast<unsigned>(tok * rd), 2, 1), go(static_cast<unsigned>(tiles * ro), 1, 1);
        const size_t so = 1024 + out_ring(p.chunks) + kOutAbsmax + 512;
        if (drop.thr != 0u) {
            e = launch_clusters(k_down_tc<true>, gd, kDownThreads, kDownSmem, rd, false, tm_gh, tm_codes, tm_A, tm_B, p, st);
            if (e == cudaSuccess)
                e = launch_clusters(k_outer_tc<true>, go, kOutThreads, so, ro, true, tm_gh, tm_codes32, tm_t, tm_u, p, st);
        } else {
            e = launch_clusters(k_down_tc<false>, gd, kDownThreads, kDownSmem, rd, false, tm_gh, tm_codes, tm_A, tm_B, p, st);
            if (e == cudaSuccess)
                e = launch_clusters(k_outer_tc<false>, go, kOutThreads, so, ro, true, tm_gh, tm_codes32, tm_t, tm_u, p, st);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace qn
