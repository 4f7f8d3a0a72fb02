// prompt_tiles.cuh -- the kernel of the attention of bf16 prompts over themselves on the tensor
// cores (include/spec_prompt.h); prompt_tiles.cu has it plain, prompt_tiles_options.cu
// with the score options, prompt_tiles_split.cu and prompt_tiles_split_options.cu the same for few items, split along the keys.
//
// A work item is a kv head and NQ tiles of up to 128 packed rows (TT rows of all the query heads of the
// kv head: g heads need a key once).  Over steps of KT keys
//     S = Q K^T c,  P = 2^(S - m),  O += P V,
// m a reference per row that moves only when a score passes it by 2^8: O, which lies in tensor
// memory, is rescaled then and not with every step.  P is the tensor cores' A operand from tensor memory;
// it is bf16 as V is (8 bits: the error it brings is of the size of the output's own rounding), the sums
// of weights are taken in fp32 before that rounding.
//
// Warps: eight for the softmax (a thread a row of its tile, or two that share its keys), one that issues the products,
// one that fetches (tiled TMA with the 128-byte swizzle) and hands out the items.  D = 64 and 128 keep two tiles in the CTA,
// whose products alternate: one tile's weights are made while the other's products run.  D = 256 has room for one, and S twice:
// the next step's S runs beside this step's weights; two threads share a row, half of a step's keys each, and half of the
// channels of O (one thread a row: 540 us where two take 244, 6 pieces of up to 1000 rows with a cap and a window).
//
// Bound by the tensor cores: one prompt of 20011 tokens, 32 / 8 heads of 128, takes 1944 to 2049 us from run to run (1.69 to 1.60
// PFLOP/s of visible pairs, 0.88 to 0.83 of the measured matrix rate), one of 8192 tokens and 40 / 8 heads 427 (its pipe is active
// 72 % of the time).  An item costs about 3 us beside its steps, 1.4 of them the softmax warps' own writing of the results while the
// next scores lie ready, so that 16 ragged prompts of up to 4096 tokens (35 items a CTA) are at 709 to 755 us, 0.67 to 0.63, and 65535 prompts
// of one row, 8 heads of 64, at 9.9 ms.  Elsewhere no unit is full, and the chain of a row's thread (scores from tensor memory,
// weights, weights to tensor memory) with two such warps a scheduler is the bound: at D = 64, which has half the
// products for as many weights, 301 us for 8192 tokens of 32 / 8 heads, 0.48 (tensor pipe 36 % active, special functions 33 %, issue 42 %);
// distance biases 664 us for 427 (41, 21, 48 %), caps 795 (35, 18, 45 %; the FMA pipe 50 %).  D = 64 and 128 spill some 50 bytes a
// thread at 168 registers, with options 100 to 115.
#pragma once

#include <atomic>

#include "attend.cuh"
#include "prompt.cuh"

namespace specv {

struct PromptMaps {
    CUtensorMap q, k, v;
};

namespace {

constexpr float kLazy = 8.f;               // log2 units a score may pass the reference by
// The workspace: tickets, a CTA's sums over keys, its rows' references and weights.
constexpr int kPromptSms = 152, kPromptTickets = 256;
// Tensor memory truncates what it adds up: a run of keys at most, then the sum goes to fp32 in the
// workspace.
constexpr int kRunKeys = 16384;
// Where a call has too few items for the SMs, items of many steps are split along the keys; the parts of an item are a cluster of
// CTAs, which join their sums together.  That costs as much as 8 steps (8 to 10 us): split into parts of at least 3 steps
// from 12 steps on, 128 rows over 2000 keys take 27 us for 33 (over 8000: 43 for 99, over 60000: 156 for 643); from 8 on,
// over 1000 keys, 25 to 27 for 23.
constexpr int kSplitSteps = 12, kPartSteps = 3, kMostParts = 16;

// parts of an item of n steps, of `most`
__host__ __device__ __forceinline__ int parts_of(int64_t n, int most)
{
    return n < kSplitSteps ? 1 : static_cast<int>(n / kPartSteps < most ? n / kPartSteps : most);
}

template <int D_> struct Prompt {
    static constexpr int D = D_;
    static constexpr int NQ = D == 256 ? 1 : 2;                // tiles of rows
    static constexpr int NS = 2;                               // S in tensor memory: one a tile, or two of one
    static constexpr int KT = D == 256 ? 64 : 128;             // keys of a step
    static constexpr int RUN = kRunKeys / KT;
    static constexpr int Q_TILE = 128 * D * 2, SLOT = KT * D * 2;
    static constexpr int SLOTS = D == 64 ? 8 : 4;              // of K or V
    static constexpr int STAGE = 32 * 128;                     // results on their way out: 32 rows of 64 channels a warp
    static constexpr int SMEM = NQ * Q_TILE + SLOTS * SLOT + 8 * STAGE + 1024;
    static constexpr int SHARE = 2 / NQ;                       // threads of a row
    static constexpr int KH = KT / SHARE, DH = D / SHARE;      // keys of a step, channels, of each
    // (The third warpgroup has two warps that idle: registers move between warpgroups.  384 threads launch with 168 each,
    // 64512 in all = 256 x 208 + 128 x 88.)
    static constexpr int SOFTMAX = 256, THREADS = SOFTMAX + 128, LAUNCH_REGS = 168, MORE_REGS = 208, LESS_REGS = 88;
    static_assert(SOFTMAX * MORE_REGS + 128 * LESS_REGS == THREADS * LAUNCH_REGS, "no more registers than the launch has");
    // Tensor memory: S, O, P.  Products of one shape run in their order, so that at D = 128 P can take the place of
    // its S, which the next S product then overwrites; at 64 and 256 the shapes differ, and P has columns of its own.
    static constexpr int O_COL = NS * KT;
    static constexpr int P_COL = D == 128 ? 0 : O_COL + NQ * D, P_STEP = D == 128 ? KT : KT / 2;
    static_assert((D == 128 ? O_COL + NQ * D : P_COL + NS * P_STEP) <= 512, "tensor memory");
};

// A work item.
struct Item {
    PromptTile t;
    int h, first;               // kv head (-1: there are no more); first row of the tiles
    int n[2];                   // steps that each tile sees
    int np, f0;                 // steps to visit: 0 .. np - 1, then f0, f0 + 1, ...
    int part, parts, from;      // of the item's parts; the steps before it
};

template <bool SPLIT> __device__ __forceinline__ int item_step(const Item &it, int i)
{
    if (SPLIT) i += it.from;
    return i < it.np ? i : it.f0 + i - it.np;
}

// Two values as bf16, the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Barrier of all threads of the cluster's CTAs: none of them leaves before it, whatever fails
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Barrier of the softmax warps, with a vote: whether any thread's `x` is true
__device__ __forceinline__ bool softmax_any(bool x)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x))
        : "memory");
    return r != 0;
}

// tanh(z) for |z| <= kTame as z times a polynomial in z^2 (interpolated at Chebyshev's points of [0, kTame^2]: within
// 2^-22 of the result), in packed pairs and without the special functions, which weights and quotients keep busy.
constexpr float kTame = 0.75f;
__device__ __forceinline__ uint64_t tame_tanh(uint64_t z)
{
    constexpr float co[6] = {1.0f, -0.333329529f, 0.133253396f, -0.0533411168f, 0.0195762161f, -0.00471152226f};
    const uint64_t t = f2_fma(z, z, 0);
    uint64_t y = f2_pack(co[5], co[5]);
#pragma unroll
    for (int i = 4; i >= 0; --i) y = f2_fma(y, t, f2_pack(co[i], co[i]));
    return f2_fma(y, z, 0);
}

template <int D, bool OPT, bool SPLIT>
__global__ void __launch_bounds__(Prompt<D>::THREADS, 1)
prompt_tiles_kernel(const PromptParams p, const __grid_constant__ PromptMaps maps, const int parts_most)
{
    using A = Prompt<D>;
    constexpr int NQ = A::NQ, KT = A::KT, SLOTS = A::SLOTS, SHARE = A::SHARE, KH = A::KH, DH = A::DH, kItems = 2;
    constexpr int kIssuer = A::SOFTMAX / 32, kLoader = kIssuer + 1;
    extern __shared__ uint8_t raw[];
    uint8_t *const smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    uint8_t *const qs = smem, *const slots = smem + NQ * A::Q_TILE;
    __shared__ __align__(8) uint64_t q_full[NQ], q_empty[NQ], full[SLOTS], empty[SLOTS], tail, s_full[A::NS], p_full[A::NS], o_full[A::NS],
        item_full[kItems], item_empty[kItems];
    __shared__ Item items[kItems];
    __shared__ float shared_row[SHARE == 2 ? 2 : 1][128];      // what the two threads of a row tell each other
    __shared__ uint32_t tmem_base;
    __shared__ int failed;
    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const int group = p.Hq / p.H, TT = 128 / group, split = SPLIT ? parts_most : 1;

    if (tid == 0) {
        failed = 0;
        mbar_init(&tail, 1);
        for (int i = 0; i < NQ; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < A::NS; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&o_full[i], 1);
            mbar_init(&p_full[i], 4 * SHARE);               // (a warp may be a step ahead of another where S lies twice)
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], A::SOFTMAX / 32 + 1);
        }
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&tmem_base, 512);
    __syncthreads();
    tmem_fence_after();
    const uint32_t s_t = __shfl_sync(0xFFFFFFFFu, tmem_base, 0), o_t = s_t + A::O_COL;
    bool fail = false;
    int ir = 0;
    uint32_t i_phase = 0;
    const auto next_item = [&] {
        if (++ir == kItems) {
            ir = 0;
            i_phase ^= 1;
        }
    };

    if (warp >= kIssuer) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(A::LESS_REGS));
        if (warp == kLoader) {
            uint32_t *const ticket = static_cast<uint32_t *>(p.ws);        // items taken, CTAs that are done
            if (lane == 0) {
                tma_prefetch(&maps.q);
                tma_prefetch(&maps.k);
                tma_prefetch(&maps.v);
            }
            int ring = 0, b0 = 0;
            uint32_t phase = 1, tail_phase = 0, q_phase[NQ];
            for (int q = 0; q < NQ; ++q) q_phase[q] = 1;
            int64_t base = 0, index = blockIdx.x;         // tiles of the requests before b0; the item
            // 32 requests from b0 on, a lane each, kept from item to item: their tiles up to and with this lane's
            PromptTile t = {};
            int known = -1;
            int64_t mine = 0, upto = 0;
            const auto slot = [&](bool value, const Item &it, int step) {
                const int k0 = step * KT;
                wait_or_fail(&empty[ring], phase, fail);
                uint8_t *const to = slots + ring * A::SLOT;
                // values that no row of the request sees become zeros (0 x NaN would reach every row of the tile)
                const int live = p.window > 0 ? max(it.t.m - it.t.n - p.window + 1, 0) : 0;
                const bool part = value && (k0 + KT > it.t.m || (k0 < live && k0 + KT > p.prefix));
                uint64_t *const bar = part ? &tail : &full[ring];
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, A::SLOT);
#pragma unroll
                    for (int x = 0; x < D; x += 64)
                        tma_load_3d(to + x * KT * 2, value ? &maps.v : &maps.k, x, it.h, it.t.k_lo + k0, bar);
                }
                __syncwarp();
                if (part) {
                    wait_or_fail(&tail, tail_phase, fail);
                    tail_phase ^= 1;
                    for (int e = lane; e < KT * D / 8; e += 32) {
                        const int r = e / 8 % KT, j = k0 + r;
                        if (j >= it.t.m || (j < live && j >= p.prefix))
                            *reinterpret_cast<uint4 *>(to + static_cast<int64_t>(e) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[ring]);
                }
                if (++ring == SLOTS) {
                    ring = 0;
                    phase ^= 1;
                }
            };
            for (;;) {
                Item it = {};
                it.h = -1;
                const int64_t number = index / split, line = number / p.H;
                // the request whose tiles hold `line`, its last (longest) tile first
                while (b0 < p.B && !fail) {
                    if (known != b0) {
                        mine = b0 + lane < p.B && prompt_request(p, b0 + lane, nullptr, t) ? (t.n + NQ * TT - 1) / (NQ * TT) : 0;
                        upto = mine;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                            if (lane >= o) upto += y;
                        }
                        known = b0;
                    }
                    const int64_t at = base + upto, all = __shfl_sync(0xFFFFFFFFu, upto, 31);
                    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, at - mine <= line && line < at);
                    if (hit) {
                        const int from = __ffs(hit) - 1;
                        it.t.lo = __shfl_sync(0xFFFFFFFFu, t.lo, from);
                        it.t.n = __shfl_sync(0xFFFFFFFFu, t.n, from);
                        it.t.k_lo = __shfl_sync(0xFFFFFFFFu, t.k_lo, from);
                        it.t.m = __shfl_sync(0xFFFFFFFFu, t.m, from);
                        it.first = static_cast<int>(__shfl_sync(0xFFFFFFFFu, at, from) - 1 - line) * (NQ * TT);
                        it.h = static_cast<int>(number % p.H);
                        break;
                    }
                    base += all;
                    b0 += 32;
                }
                if (it.h >= 0) {
                    const int own = it.t.m - it.t.n + it.first;            // last key of the first row
                    const int near = p.window > 0 ? max(own - p.window + 1, 0) / KT : 0;
                    it.f0 = near;
                    it.np = min((p.prefix + KT - 1) / KT, near);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int rows = min(it.t.n - it.first - q * TT, TT);
                        const int last = rows > 0 && q < NQ ? own + q * TT + rows - 1 : -1;
                        it.n[q] = last < 0 ? 0 : it.np + last / KT + 1 - near;
                    }
                    // parts of about as many steps, as many as pay for their joining
                    it.part = static_cast<int>(index % split);
                    it.parts = 1;
                    it.from = 0;
                    if (SPLIT) {
                        const int n = max(it.n[0], it.n[1]);
                        it.parts = parts_of(n, split);
                        it.from = static_cast<int>(static_cast<int64_t>(n) * it.part / it.parts);
                        const int to = static_cast<int>(static_cast<int64_t>(n) * (it.part + 1) / it.parts);
#pragma unroll
                        for (int q = 0; q < 2; ++q) it.n[q] = max(min(it.n[q], to) - it.from, 0);
                        // (a part's sums stay where they are until they are joined: its CTA takes no other)
                        if (index >= gridDim.x || it.part >= it.parts) it.h = -1;
                    }
                }
                wait_or_fail(&item_empty[ir], i_phase ^ 1, fail);
                if (fail) it.h = -1;
                if (lane == 0) {
                    items[ir] = it;
                    mbar_arrive(&item_full[ir]);
                }
                __syncwarp();
                next_item();
                if (it.h < 0) break;
                // (asked for here, looked at after the item)
                uint32_t taken = 0;
                if (lane == 0) taken = atomicAdd(ticket, 1u);
                const int n = max(it.n[0], it.n[1]);
                if (n > 0) {
                    // in the order of the products (a tile's queries as soon as its last scores are through)
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        if (it.n[q] > 0) {
                            wait_or_fail(&q_empty[q], q_phase[q], fail);
                            q_phase[q] ^= 1;
                            if (lane == 0) {
                                mbar_arrive_expect_tx(&q_full[q], TT * group * D * 2);
#pragma unroll
                                for (int x = 0; x < D; x += 64)
                                    tma_load_3d(qs + q * A::Q_TILE + x * 256, &maps.q, x, it.h * group, it.t.lo + it.first + q * TT, &q_full[q]);
                            }
                            __syncwarp();
                        }
                        if (q == 0) slot(false, it, item_step<SPLIT>(it, 0));
                    }
                    for (int i = 0; i < n; ++i) {
                        if (NQ == 2) slot(true, it, item_step<SPLIT>(it, i));
                        if (i + 1 < n) slot(false, it, item_step<SPLIT>(it, i + 1));
                        if (NQ == 1) slot(true, it, item_step<SPLIT>(it, i));
                    }
                }
                index = static_cast<int64_t>(gridDim.x) + __shfl_sync(0xFFFFFFFFu, taken, 0);
            }
            // the last CTA leaves the tickets as it found them
            if (lane == 0) {
                fence_acq_rel_gpu();
                if (atomicAdd(ticket + 1, 1u) == gridDim.x - 1) {
                    ticket[0] = 0u;
                    ticket[1] = 0u;
                }
            }
        } else if (warp == kIssuer) {
            const uint32_t q_addr = smem_addr(qs), slot_addr = smem_addr(slots);
            int ring = 0;
            uint32_t phase = 0, q_phase[NQ] = {}, p_phase[A::NS] = {};
            uint32_t steps = 0;                           // NQ = 1: steps so far, whose S alternates
            const auto arrived = [&] {                    // the next slot of the ring: its place
                wait_or_fail(&full[ring], phase, fail);
                tmem_fence_after();
                const int at = ring;
                if (++ring == SLOTS) {
                    ring = 0;
                    phase ^= 1;
                }
                return at;
            };
            const auto scores = [&](int q, int s, int at, bool last) {
                const uint32_t a = q_addr + q * A::Q_TILE, b = slot_addr + at * A::SLOT;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_f16_shared(s_t + s * KT, smem_desc_swizzled(a + k / 4 * (128 * 128) + k % 4 * 32, 16),
                                   smem_desc_swizzled(b + k / 4 * (KT * 128) + k % 4 * 32, 16), mma_f16_desc(KT, false, true), k > 0);
                mma_commit(&s_full[s]);
                if (last) mma_commit(&q_empty[q]);
            };
            const auto values = [&](int q, int s, int at, bool accumulate) {
                const uint32_t b = slot_addr + at * A::SLOT;
                wait_or_fail(&p_full[s], p_phase[s], fail);
                p_phase[s] ^= 1;
                tmem_fence_after();
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
                    mma_f16(o_t + q * D, s_t + A::P_COL + s * A::P_STEP + k * 8, smem_desc_swizzled(b + k * 2048, KT * 128),
                            mma_f16_desc(D, true, true), accumulate || k > 0);
                mma_commit(&o_full[s]);
            };
            for (;;) {
                wait_or_fail(&item_full[ir], i_phase, fail);
                const int h = *reinterpret_cast<volatile int *>(&items[ir].h);
                const int n0 = *reinterpret_cast<volatile int *>(&items[ir].n[0]), n1 = *reinterpret_cast<volatile int *>(&items[ir].n[1]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[ir]);
                next_item();
                if (__shfl_sync(0xFFFFFFFFu, h < 0 || fail, 0)) break;
                const int n = max(n0, n1);
                if (n == 0) continue;
                const auto queries = [&](int q) {
                    wait_or_fail(&q_full[q], q_phase[q], fail);
                    q_phase[q] ^= 1;
                    tmem_fence_after();
                };
                int at = arrived();
                if constexpr (NQ == 2) {
                    if (n0 > 0) {
                        queries(0);
                        scores(0, 0, at, n0 == 1);
                    }
                    if (n1 > 0) {
                        queries(1);
                        scores(1, 1, at, n1 == 1);
                    }
                } else {
                    queries(0);
                    scores(0, steps & 1, at, n == 1);
                }
                mma_commit(&empty[at]);
                for (int i = 0; i < n; ++i) {
                    const bool more = i + 1 < n, accumulate = i % A::RUN != 0;
                    if constexpr (NQ == 2) {
                        const int v = arrived();
                        if (i < n0) values(0, 0, v, accumulate);
                        if (more) at = arrived();
                        if (i + 1 < n0) scores(0, 0, at, i + 2 == n0);
                        if (i < n1) values(1, 1, v, accumulate);
                        mma_commit(&empty[v]);
                        if (i + 1 < n1) scores(1, 1, at, i + 2 == n1);
                    } else {
                        if (more) {
                            at = arrived();
                            scores(0, (steps + 1) & 1, at, i + 2 == n);
                        }
                        const int v = arrived();
                        values(0, steps & 1, v, accumulate);
                        mma_commit(&empty[v]);
                        ++steps;
                    }
                    if (more) mma_commit(&empty[at]);
                }
            }
        }
        if (SPLIT) {
            __syncwarp();
            cluster_barrier();                        // (with the softmax warps of all parts)
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(A::MORE_REGS));
        const int q = SHARE == 2 ? 0 : warp >> 2, row = tid & 127;             // tile, row of it
        const int part = SHARE == 2 ? warp >> 2 : 0;                           // which of the row's threads
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
        const uint32_t o_mine = o_t + q * D + part * DH + lanes;
        uint32_t count = 0;                           // steps of this tile so far
        const float c = p.scale * kLog2e, cap = p.cap * kLog2e, rcap = p.cap > 0.f ? cap_reciprocal(cap) : 0.f;
        // sums over the runs of keys so far, channel by channel
        float *const sums = reinterpret_cast<float *>(static_cast<uint8_t *>(p.ws) + kPromptTickets) +
                            ((static_cast<int64_t>(blockIdx.x) * NQ + q) * D + part * DH) * 128 + row;
        // reference and weight of each row of each CTA's items that are split
        float2 *const stats = reinterpret_cast<float2 *>(static_cast<uint8_t *>(p.ws) + kPromptTickets +
                                                         static_cast<int64_t>(kPromptSms) * NQ * D * 512);
        if (blockIdx.x == 0 && p.status) {
            PromptTile t;
            for (int b = tid; b < p.B; b += A::SOFTMAX) prompt_request(p, b, p.status, t);
        }
        // Wait for the products with V of the tile's step `j`.  (Where S lies twice, the step before can be under way too when
        // this is asked, and a parity tells two phases apart: the steps take turns at two barriers, as with S and P.)
        const auto values_done = [&](uint32_t j) {
            wait_or_fail(&o_full[NQ == 2 ? q : j & 1], (NQ == 2 ? j : j >> 1) & 1, fail);
            tmem_fence_after();
        };
        uint8_t *const stage = slots + SLOTS * A::SLOT + warp * A::STAGE;
        for (;;) {
            wait_or_fail(&item_full[ir], i_phase, fail);
            const Item it = items[ir];
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[ir]);
            next_item();
            // (threads that share rows, or join parts, leave together: they meet at barriers)
            const bool stop = it.h < 0 || fail;
            if (SHARE == 2 || SPLIT ? softmax_any(stop) : __any_sync(0xFFFFFFFFu, stop)) break;
            const int i_row = it.first + q * TT + row / group, head = it.h * group + row % group;
            const bool real = row < TT * group && i_row < it.t.n;
            const int own0 = it.t.m - it.t.n + it.first + q * TT;      // last key of the tile's first row
            const int own = it.t.m - it.t.n + i_row;
            const float slope = OPT && p.slopes && real ? p.slopes[head] * kLog2e : 0.f;
            const int n = it.n[q];
            float ref = -INFINITY, l = 0.f, l_low = 0.f, run_ref = 0.f;       // (l_low: what l lacks)
            for (int i = 0; i < n; ++i) {
                const int step0 = item_step<SPLIT>(it, i) * KT, k0 = step0 + part * KH;      // of the step, of this thread
                const int sb = NQ == 2 ? q : count & 1;
                wait_or_fail(&s_full[sb], (NQ == 2 ? count : count >> 1) & 1, fail);
                tmem_fence_after();
                const uint32_t s_mine = s_t + sb * KT + part * KH + lanes;
                float s[KH];
#pragma unroll
                for (int k = 0; k < KH; k += 32) tmem_ld32(s_mine + k, reinterpret_cast<uint32_t *>(s + k));
                tmem_wait_ld();
                // keys that not all of the tile's rows see: hidden ones get `x`
                const auto hide = [&](float x) {
                    if (step0 + KT - 1 > own0 || (p.window > 0 && step0 < own0 + TT - p.window)) {
                        const int last = own - k0;
                        if (p.window > 0) {
                            const int64_t least = static_cast<int64_t>(last) - p.window;
                            const int near = least < -1 ? -1 : static_cast<int>(least), always = p.prefix - k0;
#pragma unroll
                            for (int k = 0; k < KH; ++k) s[k] = k <= last && (k > near || k < always) ? s[k] : x;
                        } else {
#pragma unroll
                            for (int k = 0; k < KH; ++k) s[k] = k <= last ? s[k] : x;
                        }
                    }
                };
                if constexpr (OPT) {
                    // the scores in log2 units; the way of the tanh is chosen by what this row sees alone
                    if (p.cap > 0.f) {
                        hide(0.f);
                        float large = 0.f;
#pragma unroll
                        for (int k = 0; k < KH; ++k) large = fmaxf(large, fabsf(s[k]));
                        if (!real || large * fabsf(c * rcap) <= kTame) {
                            const uint64_t z2 = f2_pack(c * rcap, c * rcap), cap2 = f2_pack(cap, cap);
#pragma unroll
                            for (int e = 0; e < KH / 2; ++e)
                                f2_unpack(f2_fma(tame_tanh(f2_fma(f2_pack(s[2 * e], s[2 * e + 1]), z2, 0)), cap2, 0), s[2 * e], s[2 * e + 1]);
                        } else {
#pragma unroll
                            for (int k = 0; k < KH; ++k) s[k] = cap_score<false>(s[k] * c, cap, rcap);
                        }
                        __syncwarp();
                    } else {
                        const uint64_t c2 = f2_pack(c, c);
#pragma unroll
                        for (int e = 0; e < KH / 2; ++e) f2_unpack(f2_fma(f2_pack(s[2 * e], s[2 * e + 1]), c2, 0), s[2 * e], s[2 * e + 1]);
                    }
                    if (p.slopes) {
                        // (the distance first, which is exact: the row's own key has no bias, however steep the slope)
                        const float at = -static_cast<float>(own - k0);
                        const uint64_t at2 = f2_pack(at, at), slope2 = f2_pack(slope, slope);
#pragma unroll
                        for (int e = 0; e < KH / 2; ++e)
                            f2_unpack(f2_fma(slope2, f2_add(f2_pack(2.f * e, 2.f * e + 1.f), at2), f2_pack(s[2 * e], s[2 * e + 1])),
                                      s[2 * e], s[2 * e + 1]);
                    }
                }
                hide(-INFINITY);
                float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int k = 4; k < KH; ++k) top[k & 3] = fmaxf(top[k & 3], s[k]);
                float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                if (!OPT) most *= c;
                bool move = most > ref + kLazy;
                const bool fresh = i % A::RUN == 0;
                if (fresh && i > 0) {
                    // a run's products to the sums
                    values_done(count - 1);
                    const float f = i == A::RUN ? 0.f : ex2(run_ref - ref);
#pragma unroll 1
                    for (int d = 0; d < DH; d += 16) {
                        uint32_t r[16];
                        tmem_ld16(o_mine + d, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float *const to = sums + (d + e) * 128;
                            *to = __uint_as_float(r[e]) + (i == A::RUN ? 0.f : *to * f);
                        }
                    }
                    run_ref = ref;
                }
                const bool any = SHARE == 2 ? softmax_any(move) : __any_sync(0xFFFFFFFFu, move);
                if (any) {
                    if (SHARE == 2) {
                        // (both threads of a row take the same reference; the vote before keeps the places free)
                        shared_row[part][row] = most;
                        softmax_any(false);
                        most = fmaxf(most, shared_row[part ^ 1][row]);
                        move = most > ref + kLazy;
                    }
                    const float to = move ? most : ref, f = move ? ex2(ref - to) : 1.f;
                    ref = to;
                    l *= f;
                    l_low *= f;
                    if (!fresh) {
                        values_done(count - 1);
#pragma unroll 1
                        for (int d = 0; d < DH; d += 16) {
                            uint32_t r[16];
                            tmem_ld16(o_mine + d, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                            tmem_st16(o_mine + d, r);
                        }
                    }
                }
                const float down = ref == -INFINITY ? 0.f : -ref;
                const uint64_t c2 = f2_pack(c, c), down2 = f2_pack(down, down);
                uint64_t sum = 0;
#pragma unroll
                for (int k = 0; k < KH; k += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float x, y;
                        const uint64_t two = f2_pack(s[k + 2 * e], s[k + 2 * e + 1]);
                        f2_unpack(OPT ? f2_add(two, down2) : f2_fma(two, c2, down2), x, y);
                        x = ex2(x);
                        y = ex2(y);
                        sum = f2_add(sum, f2_pack(x, y));
                        w[e] = pack_bf16(x, y);
                    }
                    tmem_st16(s_t + A::P_COL + sb * A::P_STEP + part * (KH / 2) + lanes + k / 2, w);
                }
                float x, y;
                f2_unpack(sum, x, y);
                // (a step's weights to l with the error kept: up to 2^18 steps, whose roundings go one way where weights are alike)
                l_low += x + y;
                const float l_new = __fadd_rn(l, l_low);
                l_low = __fsub_rn(l_low, __fsub_rn(l_new, l));
                l = l_new;
                tmem_wait_st();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[sb]);
                ++count;
            }
            // the tile's results
            l += l_low;
            if (SHARE == 2) {
                softmax_any(false);
                shared_row[part][row] = l;
                softmax_any(false);
                l += shared_row[part ^ 1][row];
                softmax_any(false);
            }
            if (n > 0) {
                values_done(count - 1);
            }
            const int64_t at = (static_cast<int64_t>(it.t.lo) + i_row) * p.Hq + head;
            const float f = n > A::RUN ? ex2(run_ref - ref) : 0.f;
            if (SPLIT && it.parts > 1) {
                // this part's sums to the workspace, to be joined when all are through
#pragma unroll 1
                for (int d = 0; d < DH; d += 16) {
                    uint32_t r[16] = {};
                    if (n > 0) {
                        tmem_ld16(o_mine + d, r);
                        tmem_wait_ld();
                    }
                    if (real) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float *const to = sums + (d + e) * 128;
                            *to = __uint_as_float(r[e]) + (n > A::RUN ? *to * f : 0.f);
                        }
                    }
                }
                if (part == 0) stats[(static_cast<int64_t>(blockIdx.x) * NQ + q) * 128 + row] = make_float2(ref, l);
                continue;
            }
            const float inv = l > 0.f ? 1.f / l : 0.f;
            // 64 channels at a time by way of shared memory: 8 lanes then write a row's 128 bytes (a thread's own row
            // by itself meets 32 lines with every store)
            const int64_t place = real && !fail ? at * D + part * DH : -1;
#pragma unroll 1
            for (int d = 0; d < DH; d += 64) {
#pragma unroll 1
                for (int d2 = 0; d2 < 64; d2 += 32) {
                    uint32_t r[32] = {};
                    if (n > 0) {
                        tmem_ld32(o_mine + d + d2, r);
                        tmem_wait_ld();
                    }
                    if (n > A::RUN)
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) + sums[(d + d2 + e) * 128] * f);
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k] = pack_bf16(__uint_as_float(r[e + 2 * k]) * inv, __uint_as_float(r[e + 2 * k + 1]) * inv);
                        *reinterpret_cast<uint4 *>(stage + lane * 128 + (((d2 + e) / 8) ^ (lane & 7)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
#pragma unroll
                for (int k0 = 0; k0 < 8; k0 += 4) {
                    uint4 x[4];
                    int64_t to[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int from = (k0 + k) * 4 + lane / 8;
                        to[k] = __shfl_sync(0xFFFFFFFFu, place, from);
                        x[k] = *reinterpret_cast<const uint4 *>(stage + from * 128 + ((lane & 7) ^ (from & 7)) * 16);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (to[k] >= 0) *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + to[k] + d + (lane & 7) * 8) = x[k];
                }
                __syncwarp();
            }
            if (real && !fail && p.lse && part == 0) p.lse[at] = l > 0.f ? (ref + log2f(l)) * kLn2 : -INFINITY;
            tmem_fence_before();                      // (O is free with the next item's first weights)
        }
        if (SPLIT) {
            // The parts of the item, in their order: each CTA of the cluster joins its share, a warp 32 rows of 16 channels at a
            // time.  (A CTA of a split call takes one item, which still lies in the first place.)
            fence_acq_rel_gpu();
            __syncwarp();
            cluster_barrier();
            const Item &it = items[0];
            const bool join = !fail && it.h >= 0 && it.parts > 1;      // (else the item's fields say nothing)
            for (int u = join ? it.part * (A::SOFTMAX / 32) + warp : NQ * 4 * (D / 16); u < NQ * 4 * (D / 16); u += it.parts * (A::SOFTMAX / 32)) {
                const int d = u % (D / 16) * 16, q = u / (D / 16) / 4, row = u / (D / 16) % 4 * 32 + lane;
                const int i_row = it.first + q * TT + row / group, head = it.h * group + row % group;
                if (row >= TT * group || i_row >= it.t.n) continue;
                const int64_t first = (static_cast<int64_t>(blockIdx.x) - it.part) * NQ + q;     // of the parts' places, NQ apart
                const float2 *const st = stats + first * 128 + row;
                const float *const from = reinterpret_cast<const float *>(static_cast<const uint8_t *>(p.ws) + kPromptTickets) +
                                          (first * D + d) * 128 + row;
                float ref = -INFINITY, l = 0.f, o[16] = {};
                for (int s = 0; s < it.parts; ++s) ref = fmaxf(ref, __ldcg(st + s * NQ * 128).x);
#pragma unroll 2
                for (int s = 0; s < it.parts; ++s) {
                    const float2 x = __ldcg(st + s * NQ * 128);
                    const float f = x.y > 0.f ? ex2(x.x - ref) : 0.f;
                    l += x.y * f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] += __ldcg(from + (static_cast<int64_t>(s) * NQ * D + e) * 128) * f;
                }
                const float inv = l > 0.f ? 1.f / l : 0.f;
                const int64_t at = (static_cast<int64_t>(it.t.lo) + i_row) * p.Hq + head;
                uint4 *const to = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + at * D + d);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    to[k] = make_uint4(pack_bf16(o[8 * k] * inv, o[8 * k + 1] * inv), pack_bf16(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                       pack_bf16(o[8 * k + 4] * inv, o[8 * k + 5] * inv), pack_bf16(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
                if (p.lse && d == 0) p.lse[at] = l > 0.f ? (ref + log2f(l)) * kLn2 : -INFINITY;
            }
        }
    }
    if (fail) failed = 1;
    tmem_fence_before();
    __syncthreads();
    if (failed && tid == 0) {
        // a wait gave up: let the copies in flight land (bounded), then leave
        for (int i = 0; i < SLOTS; ++i)
            for (int ph = 0; ph < 2; ++ph) mbar_wait(&full[i], ph);
        for (int ph = 0; ph < 2; ++ph) {
            for (int i = 0; i < NQ; ++i) mbar_wait(&q_full[i], ph);
            mbar_wait(&tail, ph);
        }
        set_status(p.status, SPEC_STATUS_TIMEOUT);
    }
    __syncthreads();
    tmem_fence_after();
    if (warp == 0) tmem_free(s_t, 512);
}

template <int D> void split_config(cudaLaunchConfig_t &c, cudaLaunchAttribute &a, int grid, int split, cudaStream_t s)
{
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = static_cast<unsigned>(split);
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
    c = {};
    c.gridDim = dim3(static_cast<unsigned>(grid));
    c.blockDim = dim3(Prompt<D>::THREADS);
    c.dynamicSmemBytes = Prompt<D>::SMEM;
    c.stream = s;
    c.attrs = &a;
    c.numAttrs = 1;
}

// `split`: parts that the items' steps can be split into at most; as many are taken as let all clusters run at once.
// cudaErrorNotSupported: a compiler gave the kernel other registers than its warpgroups share out.
template <int D, bool OPT, bool SPLIT> cudaError_t launch_tiles_as(const PromptParams &p, const PromptMaps &maps, int grid, int split, cudaStream_t s)
{
    using A = Prompt<D>;
    // (the table decides in how many parts a call is split, and with that its bits: a thread that finds `done` finds the table too)
    static std::atomic<bool> done[64];
    static std::atomic<int> fit[SPLIT ? 64 : 1][kMostParts + 1];           // clusters of a size that run at once
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev].load(std::memory_order_acquire)) {
        // (registers that move between warpgroups have to add up to what the launch has, or their warps would wait for ever)
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, prompt_tiles_kernel<D, OPT, SPLIT>);
        if (e != cudaSuccess) return e;
        if (a.numRegs != A::LAUNCH_REGS) return cudaErrorNotSupported;
        e = cudaFuncSetAttribute(prompt_tiles_kernel<D, OPT, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, A::SMEM);
        if (e == cudaSuccess && SPLIT) e = cudaFuncSetAttribute(prompt_tiles_kernel<D, OPT, SPLIT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (SPLIT) {
            for (int n = 2; n <= kMostParts; ++n) {
                cudaLaunchConfig_t c;
                cudaLaunchAttribute a;
                split_config<D>(c, a, n, n, s);
                int most = 0;
                if (cudaOccupancyMaxActiveClusters(&most, prompt_tiles_kernel<D, OPT, SPLIT>, &c) != cudaSuccess) {
                    cudaGetLastError();               // (a size that the GPU does not have)
                    most = 0;
                }
                fit[dev][n].store(most, std::memory_order_relaxed);
            }
        }
        done[dev].store(true, std::memory_order_release);
    }
    if constexpr (SPLIT) {
        const int items = grid;
        while (split > 1 && fit[dev][split].load(std::memory_order_relaxed) < items) --split;
        grid = items * split;
        cudaLaunchConfig_t c;
        cudaLaunchAttribute a;
        split_config<D>(c, a, grid, split, s);
        return cudaLaunchKernelEx(&c, prompt_tiles_kernel<D, OPT, SPLIT>, p, maps, split);
    } else {
        prompt_tiles_kernel<D, OPT, SPLIT><<<grid, A::THREADS, A::SMEM, s>>>(p, maps, split);
        return cudaGetLastError();
    }
}

template <bool OPT, bool SPLIT> cudaError_t launch_tiles(const PromptParams &p, const PromptMaps &maps, int grid, int split, cudaStream_t s)
{
    if (p.D == 64) return launch_tiles_as<64, OPT, SPLIT>(p, maps, grid, split, s);
    return p.D == 128 ? launch_tiles_as<128, OPT, SPLIT>(p, maps, grid, split, s) : launch_tiles_as<256, OPT, SPLIT>(p, maps, grid, split, s);
}

}  // namespace

cudaError_t launch_prompt_tiles_options(const PromptParams &p, const PromptMaps &maps, int grid, cudaStream_t s);
cudaError_t launch_prompt_tiles_split(const PromptParams &p, const PromptMaps &maps, int grid, int split, cudaStream_t s);
cudaError_t launch_prompt_tiles_split_options(const PromptParams &p, const PromptMaps &maps, int grid, int split, cudaStream_t s);

}  // namespace specv
