// act8_grads_tc.cu -- the adapter gradients of act8_grads.cu on the 5th-generation tensor cores (tcgen05, TMEM,
// TMA), for long batches:
//
//   t = x A^T, u = grad_h B;   grad_B = s grad_h^T t,  grad_A = s u^T x,   x = q a / 127
//
// Both kernels read each element of grad_h and of the codes once; the matrix work per byte grows with the rank and would
// bound them on mma.sync from r = 32 on.
//
// Operands. grad_h tiles come by TMA and are used as they are. Codes come by TMA too. In k_down_tc they go in as
// bf16 integers, and the sum of 64 features is multiplied by a / 128 in fp32. In k_outer_tc a varies along the sum, so the
// warps form q a / 128: at most 15 significant bits, exactly hi + lo, two bf16 (hi the rounded product, lo the fma of the
// rest), each with its own MMA, as the operand in TMEM. (a / 128 keeps the largest a in range; below 2^-126 it is a bf16
// subnormal and loses bits that are below 2^-133 of anything.) The missing 128 / 127 goes into s. t and u, fp32 sums, are
// passed on as three bf16 terms (24 bits); their products with x or grad_h land in three groups of accumulator columns
// that the epilogue adds.
//
//   k_down_tc   one CTA: 128 tokens (the MMA's M) of x or of grad_h, N = r; a cluster splits the features and adds
//               its sums through distributed shared memory.
//   k_outer_tc  one CTA: 256 columns of grad_h as two accumulators of 128 (M), or 128 of x, N = 3 r, K = tokens; grad_h
//               is read with its M index contiguous, as it lies. A cluster splits the tokens. It walks them backwards:
//               what the first kernel read last is still in L2.
//
// The 23 warps of k_outer_tc leave 80 registers a thread; it spills 128 B (132 B with dropout), whose cost was not timed.
//
// Warp 0 issues the TMA loads, warp 1 the MMAs, one warp brings absmaxes, the others convert codes, drain accumulators and
// run the epilogue. Every wait on an mbarrier is bounded; a CTA whose wait runs out drains what it issued and its results are
// NaN. A warp gives up as a whole, since what follows a wait wants all its lanes, and the warps of a group that meet at
// a barrier in every step leave together (see group_all).
//
// Measured at 4096 tokens: 4096 x 4096, rank 16 39 us (the bytes once: 8 us), 28672 x 8192, rank 64 128 to 150 us (44 us; sets
// of buffers of the same sizes differ by that much, each repeats to 5 %). A step of k_outer_tc takes 0.42 us of x (conversion:
// ldmatrix, products and tcgen05.st of one step are a chain of 1.4 us, in four groups; two terms of each code, as a
// goes in with x; with u instead, scaled for each 64 columns, is not built) and of grad_h (32 KB); to that come 5 us until the first
// step of x and 5 us of epilogue. Each 64 columns of the rank are a pass of their own: rank 128 111 us and 256 to 293 us. Dropout:
// 193 us and 530 us; both kernels draw the mask, in the warps that convert.
#include <cudaTypedefs.h>

#include "act8.cuh"
#include "act8.h"
#include "dependent.cuh"
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
    int64_t tile0;   // first column tile of the launch (second kernel)
    bool codes_first;  // the second kernel's column tiles are those of the codes, then those of grad_h; else the reverse
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
    for (uint32_t c = 0; c < ranks; c += 2) {  // two loads in flight
        float f[8];
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            f[4 * h] = f[4 * h + 1] = f[4 * h + 2] = f[4 * h + 3] = 0.0f;
            if (c + h < ranks)
                asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                             : "=f"(f[4 * h]), "=f"(f[4 * h + 1]), "=f"(f[4 * h + 2]), "=f"(f[4 * h + 3])
                             : "r"(stream::mapa(smem_u32(p), c + h))
                             : "memory");
        }
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

// 16 lanes x 16 columns: thread (g, t) of the warp gives, for i = 0 .. 3, column 4 i + t of lane g (v[2 i]) and of
// lane g + 8 (v[2 i + 1]).
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem desc], bf16 inputs.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint32_t bf2(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t *>(&v); }
__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162 *>(&v); }

// Two int8 codes, in the low bytes of the halves of p (the high bytes may hold anything), as a bf16 pair: 128 + the low
// seven bits, less 128 or (sign bit) 256; exact.
__device__ __forceinline__ __nv_bfloat162 code_pair(uint32_t p) {
    return __hsub2(as_bf2((p & 0x007f007fu) | 0x43004300u), as_bf2((p & 0x00800080u) | 0x43004300u));
}

// Byte mask of four elements' keep bits.
__device__ __forceinline__ uint32_t keep_bytes(uint32_t b) {
    return ((b & 1u) | (b & 2u) << 7 | (b & 4u) << 14 | (b & 8u) << 21) * 0xffu;
}

// A block of 64 codes, a 64-byte swizzled row of shared memory, to a 128-byte swizzled row of bf16. `row` is the row's
// index in its tile (its low three bits swizzle both). A whole block per thread: with half of one, waits and addresses
// were half of the instructions, and the warps that convert are bound by issuing them.
template <bool kDrop>
__device__ __forceinline__ void convert_block(uint32_t codes, uint32_t row, const DropoutArgs &drop, uint64_t e0, uint32_t to) {
    const uint32_t src = codes + (((row >> 1) & 3u) << 4), dst = to + ((row & 7u) << 4);
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(src ^ (c << 4)) : "memory");
        if (kDrop) {
            const uint32_t keep = dropout_keep_bits(drop, e0 + 16 * c, 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] &= keep_bytes(keep >> (4 * i));
        }
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = bf2(code_pair(__byte_perm(w[2 * h + (i >> 1)], 0u, (i & 1) ? 0x4342 : 0x4140)));
            sts128(dst ^ ((2 * c + h) << 4), o);
        }
    }
}

// Barriers by their shared-window address (slot s of a ring at bar + 8 s): what the one thread that issues the MMAs
// spends on addresses shows in every step.
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes) : "memory");
}
// Bounded, as sm100::mbar_wait.
constexpr uint32_t kPolls = 1u << 24;
template <uint32_t kLimit = kPolls>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < kLimit; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
}
// One decision for the warp, whose lanes all call it and come out together: a wait that runs out in one lane may still have
// ended in another.
__device__ __forceinline__ bool warp_all(bool ok) { return __all_sync(0xffffffffu, ok); }
// One decision for four warps, 128 threads, at the named barrier `id`, which orders their memory accesses as __syncthreads does.
// A warp that has given up comes too; the named barrier itself has no limit.
__device__ __forceinline__ bool group_all(uint32_t id, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.and.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(id), "r"(static_cast<uint32_t>(ok))
        : "memory");
    return all != 0;
}
// Whether the phase is over; does not wait.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// An arrival when every MMA that this thread has issued is done.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma(uint32_t dst, const CUtensorMap *m, uint32_t bar, int32_t c0, int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
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
__device__ __forceinline__ void wait_out(uint32_t bars, int n, int count, Ring at) {
    for (int e = count < n ? count : n; e > 0; --e) {
        if (--at.slot < 0) {
            at.slot = n - 1;
            at.phase ^= 1u;
        }
        bar_wait(bars + 8 * at.slot, at.phase);
    }
}

// The producer of the codes and of the second operand (the factor, or t or u): two rings that empty at their own
// pace. Neither waits for the other: issued in step order by one blocking thread, the second operand's load would
// go out only when the codes' slot is free, and its latency would be in every step. Issues what has room until all
// `steps` are out; gives up after about a second without progress. Returns false then.
template <typename Codes, typename Second>
__device__ __forceinline__ bool feed(int steps, int &ci, Ring &c, int slots, uint32_t cempty, Codes &&codes, int &ri, Ring &r,
                                     int rslots, uint32_t rempty, Second &&second, volatile uint32_t *abort_flag) {
    uint32_t idle = 0;
    while (ci < steps || ri < steps) {
        bool did = false;
        if (ri < steps && (ri < rslots || bar_test(rempty + 8 * r.slot, r.phase ^ 1u))) {
            second(ri, r.slot);
            ++ri;
            r.next(rslots);
            did = true;
        }
        if (ci < steps && (ci < slots || bar_test(cempty + 8 * c.slot, c.phase ^ 1u))) {
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
// three batches of kGroups x kN values: `at(step, group, count)` points at kN neighbouring ones, of which `count` exist,
// and `put(batch, group, values)` stores them. In the converting warps themselves the loads' latency showed in every fourth step.
constexpr int kBatch = 4, kBatches = 3;

__device__ __forceinline__ uint64_t pair(uint2 v) { return static_cast<uint64_t>(v.y) << 32 | v.x; }

template <int kN, int kGroups, uint32_t kLimit, typename At, typename Put>
__device__ __forceinline__ bool load_absmax(int steps, uint32_t afull, uint32_t aempty, int lane, At &&at, Put &&put) {
    Ring b;
    for (int i = 0; i < steps; i += kBatch, b.next(kBatches)) {
        // All loads before the first use. Rows of an odd number of blocks put groups on any 2-byte boundary: value by value then,
        // those that do not exist from the group's first place (`at` points into the array even when none does).
        uint64_t v[kGroups / 32];
        bool rest = false;
#pragma unroll
        for (int g = 0; g < kGroups / 32; ++g) {
            int count;
            const uint16_t *p = at(i, 32 * g + lane, count);
            v[g] = 0;
            if (count >= kN && (reinterpret_cast<uintptr_t>(p) & (2u * kN - 1u)) == 0)
                v[g] = kN == 4 ? pair(ld_nc_v2(p)) : ld_nc_u32(p);
            else if (count > 0)
                rest = true;
        }
        if (rest) {
            uint32_t w[kGroups / 32][kN];
#pragma unroll
            for (int g = 0; g < kGroups / 32; ++g) {
                int count;
                const uint16_t *p = at(i, 32 * g + lane, count);
#pragma unroll
                for (int e = 0; e < kN; ++e) w[g][e] = ld_nc_u16(p + (e < count ? e : 0));
            }
#pragma unroll
            for (int g = 0; g < kGroups / 32; ++g) {
                int count;
                at(i, 32 * g + lane, count);
                v[g] = 0;
#pragma unroll
                for (int e = 0; e < kN; ++e) v[g] |= static_cast<uint64_t>(e < count ? w[g][e] : 0u) << (16 * e);
            }
        }
        if (i >= kBatches * kBatch && !warp_all(bar_wait<kLimit>(aempty + 8 * b.slot, b.phase ^ 1u))) return false;
#pragma unroll
        for (int g = 0; g < kGroups / 32; ++g) put(b.slot, 32 * g + lane, v[g]);
        __syncwarp();
        if (lane == 0) bar_arrive(afull + 8 * b.slot);
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

// kBlocks: 16-column blocks of t or u that a thread can hold, 2 (rp <= 32) or 4. With 4, 80 registers a thread (two CTAs on
// an SM) do not hold everything and some spill; at that rank grad_h, not x, sets the pace.
template <bool kX, bool kDrop, int kBlocks>
__device__ __forceinline__ void down_tc(const CUtensorMap *act, const CUtensorMap *factor, const TcArgs &p, uint8_t *smem,
                                        uint64_t *bars, int64_t tile, uint32_t rank, uint32_t ranks) {
    constexpr int kStages = kX ? kDownStagesX : kDownStagesGh;
    const uint32_t base = smem_u32(smem), full = smem_u32(bars), empty = full + 32, cfull = empty + 32, cempty = cfull + 32;
    const uint32_t afull = cempty + 32, aempty = afull + 8 * kBatches, done = aempty + 8 * kBatches;
    uint32_t *slot = reinterpret_cast<uint32_t *>(bars + 16 + 2 * kBatches + 1);
    volatile uint32_t *abort_flag = slot + 1;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int64_t pieces = ((kX ? p.k : p.n) + kK - 1) / kK;
    const int64_t lo = pieces * rank / ranks;
    const int steps = static_cast<int>(pieces * (rank + 1) / ranks - lo);
    const int32_t tok0 = static_cast<int32_t>(tile * kDownTile);
    // a stage: the tile and the factor's piece; kX: the codes behind the stages
    const uint32_t piece = kX ? static_cast<uint32_t>(p.rp) * 128u : kChunk, stage = kDownA + piece;
    const int slots = down_codes(p.rp);
    const uint32_t codes = base + kStages * stage;
    uint16_t *absmax = reinterpret_cast<uint16_t *>(smem + kDownRing);

    if (threadIdx.x == 0) {
        for (int s = 0; s < 4; ++s) {
            bar_init(full + 8 * s, kX ? 1 + kDownWarps / 2 : 1);  // TMA: the factor's piece and grad_h's tile; kX: the converted tile
            bar_init(empty + 8 * s, 1);                           // the stage's MMAs are done
            bar_init(cfull + 8 * s, 1);                // kX: TMA, codes; else an accumulator's segment is done
            bar_init(cempty + 8 * s, kDownWarps / 2);  // the group's warps have read the codes, or the accumulator
        }
        for (int s = 0; s < kBatches; ++s) {
            bar_init(afull + 8 * s, 1);
            bar_init(aempty + 8 * s, kDownWarps);
        }
        bar_init(done, 1);
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
    begin_dependent();  // the second kernel reads x and grad_h before its own wait: only once the first is past this
    // The tensor core cuts off what it adds instead of rounding it, so a long chain of MMAs drifts (448 of them: 1.6e-5
    // of the sum). So there are four accumulators, taken in turn and added up in fp32 registers by the other warps: of x,
    // whose codes go in as they are, one for each 64 features, times a / 128; of grad_h, one for each kSegment stages.
    constexpr int kSegment = 8;

    // Warps 2 .. 9 have 32 lanes (tokens) of the accumulators each, of every other one.
    const uint32_t quarter = static_cast<uint32_t>(warp & 3);
    const int group = (warp - 2) >> 2;
    float sum[kBlocks][16];
#pragma unroll
    for (int e = 0; e < kBlocks; ++e)
#pragma unroll
        for (int q = 0; q < 16; ++q) sum[e][q] = 0.0f;
    // adds the accumulator in columns from d on, times a
    auto add = [&](uint32_t d, float a) {
#pragma unroll
        for (int e = 0; e < kBlocks; ++e)
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
                            bar_expect(cfull + 8 * q, kDownA / 2);
                            for (int h = 0; h < 2; ++h)
                                tma(codes + q * (kDownA / 2) + h * 4096, act, cfull + 8 * q, static_cast<int32_t>((lo + i) * kK), tok0 + 64 * h);
                        },
                        ri, r, kStages, empty,
                        [&](int i, int q) {
                            bar_expect(full + 8 * q, piece);
                            tma(base + q * stage + kDownA, factor, full + 8 * q, static_cast<int32_t>((lo + i) * kK), p.j0);
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
                    if (i >= kStages && !bar_wait(empty + 8 * r.slot, r.phase ^ 1u)) {
                        *abort_flag = 1u;
                        break;
                    }
                    const uint32_t st = base + r.slot * stage;
                    const int32_t c0 = static_cast<int32_t>((lo + i) * kK);
                    bar_expect(full + 8 * r.slot, stage);
                    tma(st, act, full + 8 * r.slot, c0, tok0);
                    tma(st + kChunk, act, full + 8 * r.slot, c0, tok0 + 64);
                    tma(st + kDownA, factor, full + 8 * r.slot, p.j0, c0);  // 64 rows of B
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
        const uint64_t a0 = smem_desc_sw128(base, 16, 1024);
        const uint64_t b0 = kX ? smem_desc_sw128(base + kDownA, 16, 1024) : smem_desc_sw128(base + kDownA, kChunk, 1024);
        int i = 0;
        Ring r, q;  // stages; grad_h: accumulators
        for (; i < steps; ++i, r.next(kStages)) {
            if (!warp_all(bar_wait(full + 8 * r.slot, r.phase))) break;
            if (!kX && i % kSegment == 0 && i >= 4 * kSegment && !warp_all(bar_wait(cempty + 8 * q.slot, q.phase ^ 1u))) break;
            tc_fence_after();
            const uint64_t a = a0 + r.slot * (stage / 16), b = b0 + r.slot * (stage / 16);
            const uint32_t d = tmem + static_cast<uint32_t>(kX ? r.slot : q.slot) * p.rp;
            const uint32_t more = kX || i % kSegment == 0 ? 0u : 1u;
            const bool last = !kX && (i % kSegment == kSegment - 1 || i + 1 == steps);
            if (leader) {
#pragma unroll
                for (uint32_t kk = 0; kk < 4; ++kk) mma_bf16_ss(d, a + 2 * kk, b + (kX ? 2 : 128) * kk, idesc, kk > 0 ? 1u : more);
                commit(empty + 8 * r.slot);
                if (last) commit(cfull + 8 * q.slot);
            }
            __syncwarp();
            if (last) q.next(4);
        }
        if (i < steps) *abort_flag = 1u;
        if (leader) commit(done);
        // every commit has arrived before the CTA may leave
        wait_out(empty, kStages, i, r);
        if (!kX && i == steps) wait_out(cfull, 4, (steps + kSegment - 1) / kSegment, q);
    } else if (kX && warp == kDownThreads / 32 - 1) {
        const int64_t blocks = p.k / kBlock;
        // a group: the batch's four steps of a token
        if (!load_absmax<4, kDownTile, kPolls>(
                steps, afull, aempty, lane,
                [&](int i, int row, int &count) {
                    const int64_t m = tok0 + static_cast<int64_t>(row);
                    count = m < p.M ? steps - i : 0;
                    return p.absmax + (m < p.M ? m : 0) * blocks + lo + i;
                },
                [&](int batch, int row, uint64_t v) { reinterpret_cast<uint64_t *>(absmax)[batch * kDownTile + row] = v; }))
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
                ok = warp_all((q > 1 || bar_wait(afull + 8 * b.slot, b.phase)) && bar_wait(empty + 8 * r.slot, r.phase ^ 1u));
                if (!ok) break;
                tc_fence_after();
                add(static_cast<uint32_t>(r.slot * p.rp),
                    __uint_as_float(static_cast<uint32_t>(absmax[(b.slot * kDownTile + quarter * 32 + lane) * kBatch + q]) << 16) * 0.0078125f);
                tc_fence_before();
                __syncwarp();
                if (q > 1) {
                    if (lane == 0) bar_arrive(aempty + 8 * b.slot);
                    b.next(kBatches);
                }
            }
            if (i < steps) {
                ok = warp_all(bar_wait(cfull + 8 * c.slot, c.phase));
                if (!ok) break;
                convert_block<kDrop>(codes + c.slot * (kDownA / 2) + row * 64u, row, p.drop,
                                     p.drop.offset + static_cast<uint64_t>(m * p.k + (lo + i) * kK),
                                     base + r.slot * stage + row * 128u);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(cempty + 8 * c.slot);
                    bar_arrive(full + 8 * r.slot);
                }
            }
            r.next(kStages);
            r.next(kStages);
            c.next(slots);
            c.next(slots);
        }
        if (!ok) *abort_flag = 1u;
    } else if (warp < 2 + kDownWarps) {
        Ring q;
        if (group == 1) q.next(4);
        for (int i = group * kSegment; i < steps; i += 2 * kSegment) {
            if (!warp_all(bar_wait(cfull + 8 * q.slot, q.phase))) {
                *abort_flag = 1u;
                break;
            }
            tc_fence_after();
            add(static_cast<uint32_t>(q.slot * p.rp), 1.0f);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(cempty + 8 * q.slot);
            q.next(4);
            q.next(4);
        }
    }
    __syncthreads();  // every load has landed: the ring is free for the sums

    // the CTA's sums to shared memory, a row per token; the second group's next to the first's
    float *red = reinterpret_cast<float *>(smem);
    if (warp >= 2 && warp < 2 + kDownWarps) {
        const bool ok = bar_wait(done, 0) && !*abort_flag;
        tc_fence_after();
        float4 *dst = reinterpret_cast<float4 *>(red + (group * kDownTile + quarter * 32 + lane) * kDownRedRow);
        const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int e = 0; e < kBlocks; ++e)
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
template <bool kDrop, int kBlocks>
__global__ void __launch_bounds__(kDownThreads, 2)
k_down_tc(const __grid_constant__ CUtensorMap tm_gh, const __grid_constant__ CUtensorMap tm_codes,
          const __grid_constant__ CUtensorMap tm_A, const __grid_constant__ CUtensorMap tm_B, const TcArgs p) {
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kDownRing + kDownAbsmax);
    const uint32_t rank = cta_rank(), ranks = cta_ranks();
    const int64_t tile = blockIdx.x / ranks;
    if (blockIdx.y == 0)
        down_tc<false, false, kBlocks>(&tm_gh, &tm_B, p, smem, bars, tile, rank, ranks);
    else
        down_tc<true, kDrop, kBlocks>(&tm_codes, &tm_A, p, smem, bars, tile, rank, ranks);
}

// ------------------------------------------------------------------------ products over tokens

constexpr int kColsGh = 256, kColsX = 128;
constexpr int kOutWarps = 16;  // converters: four groups that take steps in turn, each with its slot of TMEM
constexpr int kDrainWarps = 4;  // of x
constexpr int kOutThreads = 96 + 32 * (kOutWarps + kDrainWarps);  // with the producer, the MMA and the absmax warp
constexpr uint32_t kTmemA = 256;  // x: columns of A, 32 hi and 32 lo for each group; the accumulator has at most 192
constexpr uint32_t kOutA = 4 * kChunk;      // 64 tokens x 256 columns of grad_h
constexpr uint32_t kOutCodes = kK * kColsX;  // bytes of codes of a step
constexpr int kMaxStages = 8;
constexpr uint32_t kOutRoom = 200 * 1024;

constexpr int kOutRowX = kColsX + 4;  // floats per row j of the sums of x, behind the stages
constexpr uint32_t kOutSums = 64 * kOutRowX * 4;

// Stages that fit for a row of t or u of `chunks` pieces: grad_h or codes, and t or u.
__host__ __device__ constexpr int out_stages(bool x, int chunks) {
    const int fit = static_cast<int>((x ? kOutRoom - kOutSums : kOutRoom) / ((x ? kOutCodes : kOutA) + static_cast<uint32_t>(chunks) * kChunk));
    return fit > kMaxStages ? kMaxStages : fit;
}
constexpr uint32_t kOutAbsmax = kBatches * kBatch * 2 * kK * 2;
constexpr int kOutRowGh = 68;         // floats per column of grad_h of its sums
static_assert(kColsGh * kOutRowGh * 4 <= kOutRoom && kOutSums % 16 == 0, "");
constexpr size_t kOutSmem = 1024 + kOutRoom + kOutAbsmax + 512;

// kGiveUp: a check of what happens when waits run out. From the middle of its steps on one warp of each group gives up, and
// the other waits that this leaves without an end have a short limit.
template <bool kX, bool kDrop, bool kGiveUp>
__device__ __forceinline__ void outer_tc(const CUtensorMap *act, const CUtensorMap *mid, const TcArgs &p, uint8_t *smem,
                                         uint64_t *bars, int64_t tile, uint32_t rank, uint32_t ranks) {
    constexpr int kCols = kX ? kColsX : kColsGh;
    constexpr uint32_t kAct = kX ? kOutCodes : kOutA, kLimit = kGiveUp ? 1u << 12 : kPolls;
    // Steps between two drains of the accumulators: the tensor core cuts off what it adds instead of rounding it, and a
    // chain of 256 MMAs would be off by 1e-5. Up to rank 32 there is TMEM for two accumulators in turn, which the MMAs do
    // not wait for, so drains are twice as frequent.
    const int turns = p.rp <= 32 ? 2 : 1;
    const int every = (kX ? 8 : 16) / turns;
    const int stages = out_stages(kX, p.chunks);
    const uint32_t stage = kAct + p.chunks * kChunk;  // codes or grad_h, then u or t
    const uint32_t base = smem_u32(smem), full = smem_u32(bars), empty = full + 8 * kMaxStages, ready = empty + 8 * kMaxStages, ufull = ready + 32;
    const uint32_t afull = ufull + 8 * kMaxStages, aempty = afull + 8 * kBatches, done = aempty + 8 * kBatches, drained = done + 16;
    uint32_t *slot = reinterpret_cast<uint32_t *>(bars + 3 * kMaxStages + 4 + 2 * kBatches + 4);
    volatile uint32_t *abort_flag = slot + 1;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int64_t width = kX ? p.k : p.n;
    const int32_t col0 = static_cast<int32_t>(tile * kCols);
    const int64_t all = (p.M + kK - 1) / kK;
    const int64_t lo = all * rank / ranks;
    const int steps = static_cast<int>(all * (rank + 1) / ranks - lo);
    uint16_t *absmax = reinterpret_cast<uint16_t *>(smem + kOutRoom);
    // step i works on the tokens from tok(i) on: the last ones first
    auto tok = [&](int i) { return static_cast<int32_t>((lo + steps - 1 - i) * kK); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            bar_init(full + 8 * s, 1);   // TMA: grad_h and t; kX: the codes
            bar_init(ufull + 8 * s, 1);  // kX: TMA, u
            bar_init(empty + 8 * s, 1);  // the stage's MMAs are done
        }
        for (int s = 0; s < 4; ++s) bar_init(ready + 8 * s, 4);  // kX: the group has put a step's A into TMEM
        for (int s = 0; s < kBatches; ++s) {
            bar_init(afull + 8 * s, 1);
            bar_init(aempty + 8 * s, kOutWarps);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(done + 8 * s, 1);                                // the MMAs up to a drain are done
            bar_init(drained + 8 * s, kX ? kDrainWarps : kOutWarps);  // the warps have read the accumulators
        }
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
    grid_dependents_launch();

    // Warps drain 32 lanes (columns) of an accumulator each: of grad_h's two, warps 2 .. 17 every other 16 of the columns j;
    // of x's, the last four warps all of them. (Were x's drained by its converters, the MMAs would wait for a conversion.)
    const uint32_t quarter = static_cast<uint32_t>(warp & 3);
    const int group = (warp - 2) >> 2;
    const uint32_t h = kX ? 0u : static_cast<uint32_t>(group & 1);
    const int jb0 = group >> 1;
    float *red = reinterpret_cast<float *>(smem + (kX ? kOutRoom - kOutSums : 0));
    float sum[2][16];  // of grad_h; those of x are in shared memory, there is no room for 64 of a thread in registers
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int c = 0; c < 16; ++c) sum[b][c] = 0.0f;
    // column of x in the warp's 32 that lies in this lane (see the converters)
    const int lane_x = (lane & 16) + ((lane & 7) << 1) + ((lane >> 3) & 1);
    Ring turn;
    auto drain = [&](bool first) -> bool {
        if (!warp_all(!*abort_flag && bar_wait<kLimit>(done + 8 * turn.slot, turn.phase))) return false;
        tc_fence_after();
        const uint32_t d = tmem + 256 * h + 128 * turn.slot + ((quarter * 32u) << 16);
#pragma unroll
        for (int b = 0; b < (kX ? 4 : 2); ++b) {
            const int j = kX ? 16 * b : 16 * (jb0 + 2 * b);
            if (j < p.rp) {
                uint32_t v0[16], v1[16], v2[16];
                tmem_ld16(d + j, v0);
                tmem_ld16(d + p.rp + j, v1);
                tmem_ld16(d + 2 * p.rp + j, v2);
                tmem_ld_wait();
                float *to = red + j * kOutRowX + static_cast<int>(quarter * 32) + lane_x;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float v = __uint_as_float(v0[c]) + (__uint_as_float(v1[c]) + __uint_as_float(v2[c]));
                    if (kX)
                        to[c * kOutRowX] = first ? v : to[c * kOutRowX] + v;
                    else
                        sum[b][c] += v;
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(drained + 8 * turn.slot);
        turn.next(turns);
        return true;
    };

    if (warp == 0) {
        if (lane == 0) {
            // Up to the dependency wait only x and grad_h are read, which the preceding kernels read too.
            int i = 0, issued = 0;  // steps whose t or u, and whose activation, is on its way
            Ring mi, ai;
            auto load_act = [&]() {
                bar_expect(full + 8 * ai.slot, kX ? kAct : stage);
                for (int b = 0; b < kCols / 64; ++b)
                    tma(base + ai.slot * stage + b * (kAct / (kCols / 64)), act, full + 8 * ai.slot, col0 + 64 * b, tok(issued));
                ++issued;
                ai.next(stages);
            };
            auto load_mid = [&]() {
                const uint32_t bar = (kX ? ufull : full) + 8 * mi.slot;
                if (kX) bar_expect(bar, stage - kAct);
                for (int e = 0; e < p.chunks; ++e) tma(base + mi.slot * stage + kAct + e * kChunk, mid, bar, 64 * e, tok(i));
                ++i;
                mi.next(stages);
            };
            while (issued < stages && issued < steps) load_act();
            grid_dependency_wait();
            while (i < steps && !*abort_flag) {
                if (i >= issued) {
                    if (!bar_wait<kLimit>(empty + 8 * ai.slot, ai.phase ^ 1u)) {
                        *abort_flag = 1u;
                        break;
                    }
                    load_act();
                }
                load_mid();
            }
            while (i < issued) load_mid();  // a stage that the loop left without its t or u gets it, so that its phase ends
            wait_out(full, stages, issued, ai);
            if (kX) wait_out(ufull, stages, i, mi);
        }
    } else if (warp == 1) {
        const bool leader = elect();
        constexpr uint32_t kMnMajor = kX ? 0 : 1;  // A: grad_h as it lies, x from TMEM
        const uint32_t three = idesc_bf16(128, 3 * p.rp, kMnMajor, 1), two = idesc_bf16(128, 2 * p.rp, kMnMajor, 1);
        uint64_t a = smem_desc_sw128(base, kChunk, 1024), b = smem_desc_sw128(base + kAct, kChunk, 1024);
        uint32_t at = tmem + kTmemA;
        Ring r, t, d;
        int i = 0;
        bool ok = true;
        while (ok && i < steps) {
            const int end = steps - i < every ? steps : i + every;
            if (i >= turns * every) {
                ok = warp_all(bar_wait<kLimit>(drained + 8 * d.slot, d.phase ^ 1u));
                if (!ok) break;
            }
            const uint32_t acc = tmem + 128 * d.slot;
            uint32_t more = 0u;
            for (; i < end; ++i) {
                ok = warp_all(kX ? bar_wait<kLimit>(ready + 8 * t.slot, t.phase) : bar_wait<kLimit>(full + 8 * r.slot, r.phase));
                if (!ok) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (uint32_t kk = 0; kk < 4; ++kk) {
                        if (kX) {
                            mma_bf16_ts(acc, at + 8 * kk, b + 128 * kk, three, kk > 0 ? 1u : more);
                            // lo is 2^-8 of hi: its product with the third term is below the fp32 sums
                            mma_bf16_ts(acc, at + 8 * kk + 32, b + 128 * kk, two, 1u);
                        } else {
#pragma unroll
                            for (uint32_t half = 0; half < 2; ++half)
                                mma_bf16_ss(acc + 256 * half, a + 2 * half * (kChunk / 16) + 128 * kk, b + 128 * kk, three, kk > 0 ? 1u : more);
                        }
                    }
                    commit(empty + 8 * r.slot);
                }
                more = 1u;
                a += stage / 16;
                b += stage / 16;
                r.next(stages);
                if (r.slot == 0) {
                    a -= stages * (stage / 16);
                    b -= stages * (stage / 16);
                }
                if (kX) {
                    t.next(4);
                    at = tmem + kTmemA + 64 * t.slot;
                }
            }
            if (leader) commit(done + 8 * d.slot);  // also when left early: the warps wait for it all the same
            d.next(turns);
        }
        if (!ok) *abort_flag = 1u;
        wait_out(empty, stages, i, r);
    } else if (warp == 2 + kOutWarps) {
        const int64_t blocks = p.k / kBlock, blk0 = col0 / kBlock;
        // a group: a token's two blocks at one of the batch's four steps; kept as [step][block][token]
        if (kX && !load_absmax<2, kBatch * kK, kLimit>(
                      steps, afull, aempty, lane,
                      [&](int i, int e, int &count) {
                          const int64_t m = tok(i + e / kK) + static_cast<int64_t>(e % kK);
                          const bool live = i + e / kK < steps && m < p.M;
                          count = live ? static_cast<int>(blocks - blk0 < 2 ? blocks - blk0 : 2) : 0;
                          return p.absmax + (live ? m : 0) * blocks + blk0;
                      },
                      [&](int batch, int e, uint64_t v) {
#pragma unroll
                          for (int q = 0; q < 2; ++q)
                              absmax[((batch * kBatch + e / kK) * 2 + q) * kK + e % kK] = static_cast<uint16_t>(v >> (16 * q));
                      }))
            *abort_flag = 1u;
    } else if (!kX || warp > 2 + kOutWarps) {
        for (int i = 0; i < steps && (kX || warp < 2 + kOutWarps); i += every)
            if (!drain(i == 0)) {
                *abort_flag = 1u;
                break;
            }
    } else {
        // The group takes every fourth step; the warp has the 32 lanes of its quarter, two segments of 16 columns of one
        // block. ldmatrix with .trans, on pairs of codes, gives thread (g, t) columns 2 g and 2 g + 1 of the tokens 2 t and
        // 2 t + 1: as bf16 pairs of tokens, the lanes g and g + 8 of a 16 x 128b store. So column 2 g (+ 1) of a segment lies
        // in lane g (g + 8). A x that goes through shared memory as hi and lo instead is written and read once more, 8 B a
        // code, and that bounds the kernel.
        const uint32_t blk = quarter >> 1, seg = 2 * (quarter & 1u);
        const uint32_t swz = ((static_cast<uint32_t>(lane) >> 1) & 3u) << 4;  // this lane points ldmatrix at tokens lane, lane + 32
        const uint32_t from = base + blk * (kOutCodes / 2) + lane * 64u;
        const uint32_t to = tmem + kTmemA + 64 * group + ((quarter * 32u) << 16);
        Ring r, b;
        for (int e = 0; e < group; ++e) r.next(stages);
        Ring last = r;  // the stage of the group's step before
        bool ok = true;
        for (int i = group; i < steps; i += 4) {
            ok = ok && bar_wait<kLimit>(afull + 8 * b.slot, b.phase) && bar_wait<kLimit>(full + 8 * r.slot, r.phase) &&
                 (i < 4 || bar_wait<kLimit>(empty + 8 * last.slot, last.phase));
            if (kGiveUp && quarter == 0 && 2 * i >= steps) ok = false;
            ok = warp_all(ok);
            if (!kDrop && !ok) break;
            tc_fence_after();
            const uint32_t here = from + r.slot * stage;
            if (kDrop) {  // the step's codes, half a row of a block (32) a thread and turn, masked in place
#pragma unroll 1
                for (uint32_t e = quarter * 32u + lane; ok && e < 256; e += 128) {
                    const uint32_t token = e & 63u, part = e >> 6;
                    const uint32_t at = base + r.slot * stage + (part >> 1) * (kOutCodes / 2) + token * 64u;
                    const uint64_t e0 = p.drop.offset + static_cast<uint64_t>((tok(i) + static_cast<int64_t>(token)) * p.k + col0 + 32 * part);
#pragma unroll
                    for (uint32_t c = 0; c < 2; ++c) {
                        const uint32_t addr = at + (((2 * (part & 1u) + c) ^ ((token >> 1) & 3u)) << 4);
                        const uint32_t keep = dropout_keep_bits(p.drop, e0 + 16 * c, 16);
                        uint32_t w[4];
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
#pragma unroll
                        for (int q = 0; q < 4; ++q) w[q] &= keep_bytes(keep >> (4 * q));
                        sts128(addr, w);
                    }
                }
                fence_proxy_async_smem();  // the stage's next load overwrites what was stored here
                __syncwarp();
                ok = group_all(1u + static_cast<uint32_t>(group), ok);
                if (!ok) break;
            }
            const uint16_t *am = absmax + ((b.slot * kBatch + group) * 2 + blk) * kK + 2 * (lane & 3);
#pragma unroll
            for (uint32_t half = 0; half < 2; ++half) {  // 32 tokens each
                __nv_bfloat162 f[4];  // a / 128 of the token pairs
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    f[e] = __hmul2(as_bf2(*reinterpret_cast<const uint32_t *>(am + 32 * half + 8 * e)), __float2bfloat162_rn(0.0078125f));
#pragma unroll
                for (uint32_t sgm = 0; sgm < 2; ++sgm) {
                    uint32_t w[4], hi[8], lw[8];
                    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                 : "r"(here + half * 2048u + (((seg + sgm) << 4) ^ swz))
                                 : "memory");
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const __nv_bfloat162 v = code_pair(c == 0 ? w[e] : w[e] >> 8);
                            const __nv_bfloat162 top = __hmul2(v, f[e]);
                            hi[2 * e + c] = bf2(top);
                            lw[2 * e + c] = bf2(__hfma2(v, f[e], __hneg2(top)));
                        }
                    tmem_st_16x128b_x4(to + ((16u * sgm) << 16) + 16 * half, hi);
                    tmem_st_16x128b_x4(to + ((16u * sgm) << 16) + 16 * half + 32, lw);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            ok = warp_all(bar_wait<kLimit>(ufull + 8 * r.slot, r.phase));  // for the MMA thread, which then waits once
            if (!kDrop && !ok) break;  // with kDrop the other warps have to hear of it, at the next step's barrier
            __syncwarp();
            if (ok && lane == 0) {
                bar_arrive(ready + 8 * group);
                bar_arrive(aempty + 8 * b.slot);
            }
            b.next(kBatches);
            last = r;
#pragma unroll
            for (int e = 0; e < 4; ++e) r.next(stages);
        }
        if (!ok) *abort_flag = 1u;
    }
    __syncthreads();  // every load has landed: the ring is free for the sums

    // the sums of grad_h to shared memory, a row of j per column, as they go out; those of x are there, a row of columns
    // per j
    const bool ok = !*abort_flag && steps > 0;
    if (!kX && ok && warp >= 2 && warp < 2 + kOutWarps) {
        const int c = static_cast<int>(h * 128 + quarter * 32) + lane;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int j = 16 * (jb0 + 2 * b);
            if (j >= p.rp) break;
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<float4 *>(red + c * kOutRowGh + j + e) =
                    make_float4(sum[b][e], sum[b][e + 1], sum[b][e + 2], sum[b][e + 3]);
        }
    }
    if (!ok) {  // no steps: zeros; a wait ran out: NaN
        const float v = *abort_flag ? __uint_as_float(0x7fc00000u) : 0.0f;
        for (int e = threadIdx.x; e < (kX ? 64 * kOutRowX : kColsGh * kOutRowGh); e += kOutThreads) red[e] = v;
    }
    __syncwarp();
    if (ranks > 1) {
        stream::cluster_arrive_release();
        stream::cluster_wait_acquire();
    } else {
        __syncthreads();
    }
    // each rank adds up its share, four neighbouring values of the result per thread
    const int js = p.r - p.j0 < p.rp ? p.r - p.j0 : p.rp;
    const int inner = (kX ? kCols : js + 3) / 4, items = inner * (kX ? js : kCols);
    const int e0 = static_cast<int>(static_cast<int64_t>(items) * rank / ranks);
    const int e1 = static_cast<int>(static_cast<int64_t>(items) * (rank + 1) / ranks);
    float *out = kX ? p.grad_A : p.grad_B;
    const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0 && (kX || p.r % 4 == 0);
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
            for (int i = 0; i < 4; ++i)
                if (kX || j + i < js) dst[i] = v[i];
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

template <bool kDrop, bool kGiveUp>
__global__ void __launch_bounds__(kOutThreads, 1)
k_outer_tc(const __grid_constant__ CUtensorMap tm_gh, const __grid_constant__ CUtensorMap tm_codes,
           const __grid_constant__ CUtensorMap tm_t, const __grid_constant__ CUtensorMap tm_u, const TcArgs p) {
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOutRoom + kOutAbsmax);
    const uint32_t rank = cta_rank(), ranks = cta_ranks();
    const int64_t tile = p.tile0 + blockIdx.x / ranks;
    const int64_t of_codes = tile - (p.codes_first ? 0 : (p.n + kColsGh - 1) / kColsGh), tiles_x = (p.k + kColsX - 1) / kColsX;
    if (of_codes >= 0 && of_codes < tiles_x)
        outer_tc<true, kDrop, kGiveUp>(&tm_codes, &tm_u, p, smem, bars, of_codes, rank, ranks);
    else
        outer_tc<false, false, false>(&tm_gh, &tm_t, p, smem, bars, p.codes_first ? tile - tiles_x : tile, rank, ranks);
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
cudaError_t launch_clusters(K kern, dim3 grid, int threads, size_t smem, int ranks, const CUtensorMap &a,
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
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, a, b, c, d, p);
    if (e == cudaSuccess) count_launch();
    return e;
}

// Copies of up to two matrices, rows x cols bf16 to rows of up8(cols), zeros behind: 8 values of a row per thread, cut out of
// the aligned words around them. A CTA has `per_cta` rows, or a row has `ctas_row` CTAs.
struct Pad {
    const uint16_t *src;
    int64_t rows, cols;
    uint16_t *to;
    unsigned chunks, per_cta, ctas_row, ctas;  // chunks: of 8 in a row
};

__global__ void __launch_bounds__(256) k_pad(const Pad a, const Pad b) {
    const bool second = blockIdx.x >= a.ctas;
    const Pad &p = second ? b : a;
    const unsigned cta = second ? blockIdx.x - a.ctas : blockIdx.x;
    const unsigned r = threadIdx.x / p.chunks;
    const int64_t row = p.ctas_row > 1 ? cta / p.ctas_row : static_cast<int64_t>(cta) * p.per_cta + r;
    const unsigned chunk = p.ctas_row > 1 ? cta % p.ctas_row * 256 + threadIdx.x : threadIdx.x - r * p.chunks;
    if ((p.ctas_row == 1 && r >= p.per_cta) || row >= p.rows || chunk >= p.chunks) return;
    const int64_t c = 8 * static_cast<int64_t>(chunk);
    *reinterpret_cast<uint4 *>(p.to + row * 8 * p.chunks + c) = act8::load_row8(p.src + row * p.cols, c, p.cols, p.src + p.rows * p.cols);
}

// False when it takes more CTAs than a grid holds.
bool pad_of(const uint16_t *src, int64_t rows, int64_t cols, uint16_t *to, Pad *p) {
    const int64_t chunks = (cols + 7) / 8, per_cta = chunks < 256 ? 256 / chunks : 1, ctas_row = (chunks + 255) / 256;
    const int64_t ctas = ctas_row > 1 ? rows * ctas_row : (rows + per_cta - 1) / per_cta;
    *p = {src, rows, cols, to, static_cast<unsigned>(chunks), static_cast<unsigned>(per_cta), static_cast<unsigned>(ctas_row),
          static_cast<unsigned>(ctas)};
    return ctas <= 0x3fffffffLL;
}

// Clusters of 1 .. 8 CTAs, one on an SM, that are resident at once: of the current context, kept per host thread.
struct Fits {
    uint64_t ctx = 0;
    int dev = -1;
    int clusters[9];
};

cudaError_t cluster_fits(const Fits **out) {
    static thread_local Fits kept;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t ctx = current_context_id();
    if (kept.dev != dev || kept.ctx != ctx || ctx == 0) {
        for (int c = 1; c <= 8; ++c) {
            e = resident_clusters(reinterpret_cast<const void *>(k_outer_tc<false, false>), kOutThreads, c, kOutSmem, &kept.clusters[c]);
            if (e != cudaSuccess) return e;
        }
        kept.dev = dev;
        kept.ctx = ctx;
    }
    *out = &kept;
    return cudaSuccess;
}

// The cluster size with the least waves x (steps of a CTA + what a CTA costs besides, in steps).
int cluster_size(const Fits &fits, int per_sm, int64_t tiles, int64_t steps, int64_t besides) {
    int best = 1;
    int64_t least = 0;
    for (int c = 1; c <= 8 && c <= steps; ++c) {
        const int64_t fit = static_cast<int64_t>(per_sm) * fits.clusters[c];
        if (fit <= 0) continue;
        const int64_t cost = (tiles + fit - 1) / fit * ((steps + c - 1) / c + besides);
        if (least == 0 || cost < least) {
            least = cost;
            best = c;
        }
    }
    return best;
}

// Column tiles of the second kernel: the first `first` ones in clusters of c CTAs, the rest in clusters of c_rest in a launch of
// their own, as the least waves x (steps + besides) in all want it (a launch costs `again` more). 112 + 64 tiles of 64 steps
// (28672 x 8192, 4096 tokens) are three waves of clusters of 2, but one of 148 CTAs and one of 28 clusters: 149 us became 132.
struct Split {
    int64_t first;
    int c, c_rest;
};

Split split_tiles(const Fits &fits, int64_t tiles, int64_t steps, int64_t besides, int64_t again) {
    auto cost = [&](int64_t n, int c) {
        const int64_t fit = fits.clusters[c];
        return (n + fit - 1) / fit * ((steps + c - 1) / c + besides);
    };
    const int whole = cluster_size(fits, 1, tiles, steps, besides);
    Split best{tiles, whole, 0};
    int64_t least = fits.clusters[whole] > 0 ? cost(tiles, whole) : 0;
    for (int c = 1; c <= 8 && c <= steps; ++c) {
        const int64_t fit = fits.clusters[c], first = fit > 0 ? tiles / fit * fit : 0;
        if (first == 0 || first == tiles) continue;
        const int rest = cluster_size(fits, 1, tiles - first, steps, besides);
        const int64_t both = cost(first, c) + cost(tiles - first, rest) + again;
        if (both < least) {
            least = both;
            best = {first, c, rest};
        }
    }
    return best;
}

int pass_rank(int r) { return r >= 64 ? 64 : (r + 15) / 16 * 16; }
int pass_chunks(int rp) { return (3 * rp + 63) / 64; }

}  // namespace

namespace {

size_t up256(size_t b) { return (b + 255) & ~size_t(255); }
size_t mid_bytes(int64_t M, int r) { return up256(static_cast<size_t>(M) * pass_chunks(pass_rank(r)) * 128); }
int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }

}  // namespace

size_t act8_grads_tc_workspace_bytes(int64_t M, int64_t n, int r) {
    return 2 * mid_bytes(M, r) + (n % 8 ? up256(2 * static_cast<size_t>(M) * static_cast<size_t>(up8(n))) : 0) +
           (r % 8 ? up256(2 * static_cast<size_t>(n) * static_cast<size_t>(up8(r))) : 0);
}

cudaError_t launch_act8_grads_tc(const int8_t *codes, const uint16_t *absmax, const uint16_t *gh, int64_t M, int64_t n,
                                 int64_t k, const uint16_t *A, const uint16_t *B, int r, float s,
                                 const DropoutArgs &drop, float *grad_A, float *grad_B, void *ws, cudaStream_t st, bool give_up) {
    cudaError_t e = cudaSuccess;
    TcArgs p{absmax, M, n, k, r, 0, 0, 0, 0, false, s * (128.0f / 127.0f), grad_A, grad_B, static_cast<uint16_t *>(ws), nullptr, drop};
    char *at = static_cast<char *>(ws) + mid_bytes(M, r);
    p.u = reinterpret_cast<uint16_t *>(at);
    at += mid_bytes(M, r);
    Pad pads[2] = {};
    int count = 0;
    if (n % 8) {
        uint16_t *to = reinterpret_cast<uint16_t *>(at);
        at += up256(2 * static_cast<size_t>(M) * static_cast<size_t>(up8(n)));
        if (!pad_of(gh, M, n, to, &pads[count++])) return cudaErrorInvalidConfiguration;
        gh = to;
    }
    if (r % 8) {
        uint16_t *to = reinterpret_cast<uint16_t *>(at);
        if (!pad_of(B, n, r, to, &pads[count++])) return cudaErrorInvalidConfiguration;
        B = to;
    }
    if (count) {
        k_pad<<<pads[0].ctas + pads[1].ctas, 256, 0, st>>>(pads[0], pads[1]);
        count_launch();
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    CUtensorMap tm_gh, tm_codes, tm_A, tm_B, tm_t, tm_u;
    if (!make_map(&tm_gh, gh, M, up8(n), false) || !make_map(&tm_codes, codes, M, k, true) || !make_map(&tm_B, B, n, up8(r), false))
        return cudaErrorInvalidValue;
    const int64_t tok = (M + kDownTile - 1) / kDownTile, tiles = (n + kColsGh - 1) / kColsGh + (k + kColsX - 1) / kColsX;
    if (tok > (int64_t(1) << 28) || tiles > (int64_t(1) << 28)) return cudaErrorInvalidConfiguration;
    const int64_t pieces = (n > k ? n : k) / kK, steps = (M + kK - 1) / kK;  // of 64; both sides of a cluster have some
    const bool masked = drop.thr != 0u;
    const Fits *fits = nullptr;
    e = cluster_fits(&fits);
    if (e != cudaSuccess) return e;
    // two CTAs of the first kernel share an SM
    const int rd = cluster_size(*fits, 2, 2 * tok, pieces, 10);
    const Split so = split_tiles(*fits, tiles, steps, 12, 4);
    // In one launch the codes' CTAs, whose first step takes longer, come first (11008 x 4096, 4096 tokens: 64.2 -> 61.9 us). In
    // two the second has only codes then: with grad_h there 28672 x 8192 took 137 us instead of 133.
    p.codes_first = so.first == tiles;
    for (p.j0 = 0; p.j0 < r; p.j0 += 64) {
        p.rp = pass_rank(r - p.j0);
        p.chunks = pass_chunks(p.rp);
        if (!make_map(&tm_A, A, r, k, false, static_cast<uint32_t>(p.rp)) ||
            !make_map(&tm_t, p.t, M, 64 * p.chunks, false) || !make_map(&tm_u, p.u, M, 64 * p.chunks, false))
            return cudaErrorInvalidValue;
        const auto down = masked ? (p.rp > 32 ? k_down_tc<true, 4> : k_down_tc<true, 2>)
                                 : (p.rp > 32 ? k_down_tc<false, 4> : k_down_tc<false, 2>);
        const auto outer = give_up ? k_outer_tc<true, true> : masked ? k_outer_tc<true, false> : k_outer_tc<false, false>;
        const auto grid = [](int64_t n, int c, unsigned y) { return dim3(static_cast<unsigned>(n * c), y, 1); };
        e = launch_clusters(down, grid(tok, rd, 2), kDownThreads, kDownSmem, rd, tm_gh, tm_codes, tm_A, tm_B, p, st);
        p.tile0 = 0;
        if (e == cudaSuccess)
            e = launch_clusters(outer, grid(so.first, so.c, 1), kOutThreads, kOutSmem, so.c, tm_gh, tm_codes, tm_t, tm_u, p, st);
        p.tile0 = so.first;
        if (e == cudaSuccess && so.first < tiles)
            e = launch_clusters(outer, grid(tiles - so.first, so.c_rest, 1), kOutThreads, kOutSmem, so.c_rest, tm_gh, tm_codes,
                                tm_t, tm_u, p, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace qn
