// cache_weights.cu -- the attention weight that every cached token gets from the
// packed verify rows, added to its score (include/spec_cache.h).
//
// score_j += sum over rows and heads of exp(s_ij - lse_i): with S^T = K Q^T
// (cache_attend.cuh) a token is a lane, and its sum over the columns and heads
// stays in two threads (a half of the columns each), in a fixed order, and is added to
// the score once.  A CTA takes a few tiles of one
// request through every kv head; the keys alone are read.  The product of a step
// runs while the weights of the step before are summed and the next head's queries
// are staged; warp 8 issues the products, warp 9 fetches, and the eight warps that
// decode and sum meet them, and each other, at mbarriers only.
//
// Bound by the latency of a step: 64 requests of 2 to 5 rows and 40 query heads over
// up to 4096 tokens, ragged, take 66 us (1.2 TB/s of keys and scores), 128 x 5 rows x
// 4096 tokens 146 us (2.1 TB/s).  With a barrier a step and fetches and products by
// the decoding warps those were 109 and 237 us (84 and 174 without, all CTAs in one
// round; two rounds, which even out ragged requests, made the rest).
#include "attend.cuh"

namespace specv {

namespace {

constexpr int kMaxTiles = 8;               // tiles of a CTA at most
constexpr int kFew = 8;                    // requests whose lengths are taken as max_len

template <typename T, int D_, int NT_> struct Weights {
    static constexpr int D = D_, NT = NT_, NH = NT / 2;
    static constexpr int PIECES = sizeof(T) == 4 ? 2 : 1;
    static constexpr int K_BYTES = v_codes_at(D);              // a block's keys and their scales
    static constexpr int A_COLS = D / 2, S_COLS = PIECES * NT;
    static constexpr int COLS = tmem_cols(A_COLS + 2 * S_COLS);
    static constexpr int CTAS = COLS == 128 ? 3 : 2;           // 64 registers a thread, or 96
    static constexpr int Q_BYTES = PIECES * query_bytes(D, NT);
    static constexpr int STAGE = 4 * K_BYTES;
    static constexpr int FIXED = 1024 + 80 * NT + 2 * kMaxTiles * kTile * 4;
    static constexpr int STAGES = clamp_stages((smem_share(CTAS, FIXED) - 2 * Q_BYTES) / STAGE);
    static constexpr int NEED = 2 * Q_BYTES + STAGES * STAGE;
    static constexpr int SMEM = NEED > smem_least(CTAS) - FIXED ? NEED : smem_least(CTAS) - FIXED;
};

// Column constants of a head (shared memory).  Four sets: a warp may still read
// the one of three steps ago while the next is written.
template <int NT> struct alignas(16) Heads {          // (read by pairs)
    float mult[NT], lse[NT], slope[NT];           // (lse negated)
    int own[NT], pos[NT];
    int ncols;
};
constexpr int kSets = 4;

// Step of a CTA: tile `t` of its tiles, column tile `qt` of kv head `h`.
struct Step {
    int h, qt, t;

    __device__ __forceinline__ void next(int tiles, int qtiles)
    {
        if (++t < tiles) return;
        t = 0;
        if (++qt < qtiles) return;
        qt = 0;
        ++h;
    }
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kAttnThreads + 64, (Weights<T, D, NT>::CTAS))
weights_kernel(const CacheView c, const AttnParams p, const int tiles)
{
    using A = Weights<T, D, NT>;
    constexpr int NH = A::NH, kIssuer = 8, kLoader = 9;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *qs = smem, *stages = qs + 2 * A::Q_BYTES;
    __shared__ __align__(16) Heads<NT> sets[kSets];
    __shared__ __align__(8) uint64_t full[A::STAGES], empty[A::STAGES], k_bar, s_bar;
    __shared__ uint32_t tmem_base;
    __shared__ int nv[A::STAGES][4];
    __shared__ float acc[kMaxTiles][2][kTile];
    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const int group = p.Hq / c.H;
    Job w;
    w.b = blockIdx.y;
    if (!load_job<kTile>(c, p, w, tid == 0 ? p.status : nullptr)) return;
    const int i0 = blockIdx.x * tiles, nt = min(tiles, w.nsteps - i0);
    if (nt <= 0) return;
    const int cols = w.n * group, qt_used = (cols + NT - 1) / NT;
    const int steps = c.H * qt_used * nt;

    if (warp == kIssuer && lane == 0) {
        for (int i = 0; i < A::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 8);
        }
        mbar_init(&k_bar, 8);
        mbar_init(&s_bar, 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&tmem_base, A::COLS);
    __syncthreads();
    tmem_fence_after();
    const uint32_t a_t = __shfl_sync(0xFFFFFFFFu, tmem_base, 0), s_t = a_t + A::A_COLS;
    bool fail = false;

    if (warp == kLoader) {
        // the keys of each step into the ring, the page ids of the step after asked for
        Step at = {0, 0, 0};
        int ring = 0;
        uint32_t phase = 1;                               // (a stage is empty at first)
        Fetch next = ask_pages<true>(c, p, w, 0, step_slot<kTile>(w, i0));
        for (int i = 0; i < steps && !fail; ++i) {
            wait_or_fail(&empty[ring], phase, fail);
            load_tile<A::K_BYTES, true>(c, p, w, next, stages + ring * A::STAGE, &full[ring], nv[ring]);
            if (++ring == A::STAGES) {
                ring = 0;
                phase ^= 1;
            }
            at.next(nt, qt_used);
            if (i + 1 < steps) next = ask_pages<true>(c, p, w, at.h, step_slot<kTile>(w, i0 + at.t));
        }
        return;
    }
    if (warp == kIssuer) {
        Step at = {0, 0, 0};
        int qb = 0;
        for (int i = 0; i < steps && !fail; ++i) {
            wait_or_fail(&k_bar, i & 1, fail);
            tmem_fence_after();
            issue_scores<D, NT, A::PIECES>(s_t + (i & 1) * A::S_COLS, a_t, smem_addr(qs) + qb * A::Q_BYTES);
            mma_commit(&s_bar);
            at.next(nt, qt_used);
            if (at.t == 0) qb ^= 1;
        }
        return;
    }

    const int quarter = warp & 3, half = warp >> 2, tok = tid & 127;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const bool options = p.cap > 0.f || p.slopes || p.window > 0;
    for (int t = 0; t < nt; ++t) acc[t][half][tok] = 0.f;
    QueryStage<T, D, NT, A::PIECES> queries;
    // queries and column constants of the head that step s begins
    const auto stage_head = [&](const Step &s, Heads<NT> &set, uint8_t *q) {
        w.h = s.h;
        w.col0 = s.qt * NT;
        w.ncols = min(cols - w.col0, NT);
        if (tid < NT) {
            const int col = min(w.col0 + tid, cols - 1), j = col / group, own = w.len - w.n + j;
            const int head = s.h * group + col % group;
            set.own[tid] = own;
            set.pos[tid] = own >= 0 ? slot_position(c, p, w.b, own) : 0;
            set.slope[tid] = p.slopes ? p.slopes[head] : 0.f;
            // padded columns, and rows that saw nothing: weight exp(-inf) = 0
            const float lse = tid < w.ncols ? p.lse[static_cast<int64_t>(w.lo + j) * p.Hq + head] : -INFINITY;
            set.lse[tid] = lse == -INFINITY ? -INFINITY : -lse;
            if (tid == 0) set.ncols = w.ncols;
        }
        if ((s.h == 0 && s.qt == 0) || qt_used > 1) queries.place(p, w, group);
        queries.stage(p, static_cast<int64_t>(s.h) * group * p.q_head, fabsf(p.scale) * (c.k_scale ? c.k_scale[s.h] : 1.f), q,
                      set.mult);
        fence_proxy_async_smem();
    };
    // weights of a finished product
    const auto add_weights = [&](int i, const Step &s, const Heads<NT> &set) {
        const int real = set.ncols - half * NH;           // of this thread's columns
        if (real <= 0) return;
        const int slot0 = step_slot<kTile>(w, i0 + s.t), slot = slot0 + tok;
        const int valid = min(max(w.len - (slot - lane), 0), kTok);
        float v[NH];
        load_products<NH, NT, A::PIECES>(s_t + (i & 1) * A::S_COLS + lane_off + half * NH, v);
        const bool edge = slot0 + kTile - 1 > set.own[0] || valid < kTok;
        float sum = 0.f;
        if (edge || options) {
            const bool live = lane < valid;
            const int tpos = options && p.slot_pos && live ? slot_position(c, p, w.b, slot) : slot;
            const bool always = live && (p.window <= 0 || slot < p.prefix);
            const float rcap = p.cap > 0.f ? cap_reciprocal(p.cap) : 0.f;
#pragma unroll
            for (int k = 0; k < NH; ++k) {
                if (k >= real) break;
                const int q = half * NH + k, dist = set.pos[q] - tpos;
                float y = v[k] * set.mult[q];
                if (p.cap > 0.f) y = cap_score<true>(y, p.cap, rcap);
                y -= set.slope[q] * static_cast<float>(dist);
                const bool see = slot <= set.own[q] && (always || (live && dist < p.window));
                sum += see ? ex2((y + set.lse[q]) * kLog2e) : 0.f;
            }
        } else {
            // two columns an instruction
            uint64_t two = 0ull;
            const uint64_t log2e2 = f2_pack(kLog2e, kLog2e);
#pragma unroll
            for (int k = 0; k < NH; k += 2) {
                const uint64_t m = *reinterpret_cast<const uint64_t *>(&set.mult[half * NH + k]);
                const uint64_t ls = *reinterpret_cast<const uint64_t *>(&set.lse[half * NH + k]);
                float a, b;
                f2_unpack(f2_fma(f2_fma(f2_pack(v[k], v[k + 1]), m, ls), log2e2, 0ull), a, b);
                two = f2_add(two, f2_pack(ex2(a), ex2(b)));
            }
            float a, b;
            f2_unpack(two, a, b);
            sum = a + b;
        }
        acc[s.t][half][tok] += sum;
    };

    Step now = {0, 0, 0}, last = now;
    int cb = 0, qb = 0, ring = 0;
    uint32_t phase = 0;
    stage_head(now, sets[0], qs);
    for (int i = 0; i < steps; ++i) {
        const int cb_last = cb;
        if (i > 0) {
            wait_or_fail(&s_bar, (i - 1) & 1, fail);       // the keys' columns are used up
            tmem_fence_after();
            if (now.t == 0) {
                cb = (cb + 1) % kSets;
                qb ^= 1;
            }
        }
        wait_or_fail(&full[ring], phase, fail);
        decode_keys<D>(stages + ring * A::STAGE + quarter * A::K_BYTES, a_t + lane_off);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[ring]);
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_bar);
        if (++ring == A::STAGES) {
            ring = 0;
            phase ^= 1;
        }
        Step after = now;
        after.next(nt, qt_used);
        if (i + 1 < steps && after.t == 0) stage_head(after, sets[(cb + 1) % kSets], qs + (qb ^ 1) * A::Q_BYTES);
        if (i > 0) add_weights(i - 1, last, sets[cb_last]);
        last = now;
        now = after;
    }
    wait_or_fail(&s_bar, (steps - 1) & 1, fail);
    tmem_fence_after();
    if (csync_count(fail)) {
        if (tid == 0) {
            for (int s = 0; s < A::STAGES; ++s)
                for (int ph = 0; ph < 2; ++ph) mbar_wait(&full[s], ph);
            set_status(p.status, SPEC_STATUS_TIMEOUT);
        }
    } else {
        add_weights(steps - 1, last, sets[cb]);
        csync();
        for (int t = half; t < nt; t += 2) {
            const int slot = step_slot<kTile>(w, i0 + t) + tok;
            // (a slot that no row sees got 0, and its page may be another's by now)
            const float got = acc[t][0][tok] + acc[t][1][tok];
            const int page = slot < w.len && got != 0.f ? page_of(c, w.b, slot) : -1;
            // (requests can share a page: one addition that none of theirs falls into)
            if (page >= 0) atomicAdd(p.score + static_cast<int64_t>(page) * c.page_tokens + slot % c.page_tokens, got);
        }
    }
    tmem_fence_before();
    csync();
    if (warp == 0) tmem_free(a_t, A::COLS);
}

template <typename T, int D, int NT>
cudaError_t launch_one(const CacheView &c, const AttnParams &p, cudaStream_t s)
{
    using A = Weights<T, D, NT>;
    static bool done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev]) {
        e = cudaFuncSetAttribute(weights_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, A::SMEM);
        if (e != cudaSuccess) return e;
        done[dev] = true;
    }
    // tiles a CTA: two rounds of resident CTAs where there are many requests, whose
    // lengths differ.  (Fewer stage a head's queries for more tiles, more even out the
    // lengths: with 1, 2, 3 and 5 rounds 64 requests x 5 rows, ragged up to 4096 tokens,
    // took 84, 66, 81 and 92 us; 2 x 65533 tokens of 16
    // heads 70, and 81 with 2.)  A few requests are taken to be as long as max_len: the
    // fewest rounds, each of them a CTA's tiles and two tiles' time for the queries.  (4
    // requests x 5 rows x 16000 tokens 39 us against 56 in two rounds, 42 against 40 where
    // they are ragged; 8 x 16000 55 against 65, ragged 53 against 51; 16 x 8000 63
    // against 66, ragged 56 against 53.)
    const int tiles = (p.max_len + kTile - 1) / kTile, slots = 152 * A::CTAS * 2;
    const int64_t per = (static_cast<int64_t>(c.B) * tiles + slots - 1) / slots;
    int t = static_cast<int>(per < 1 ? 1 : (per > kMaxTiles ? kMaxTiles : per));
    if (c.B <= kFew) {
        int64_t least = INT64_MAX;
        for (int i = 1; i <= kMaxTiles; ++i) {
            const int64_t ctas = static_cast<int64_t>(c.B) * ((tiles + i - 1) / i);
            const int64_t cost = (2 * ctas + slots - 1) / slots * (i + 2);
            if (cost < least) {
                least = cost;
                t = i;
            }
        }
    }
    weights_kernel<T, D, NT><<<dim3((tiles + t - 1) / t, c.B), kAttnThreads + 64, A::SMEM, s>>>(c, p, t);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_width(const CacheView &c, const AttnParams &p, int dtype, cudaStream_t s)
{
    const int cols = (p.k_max + 1) * (p.Hq / c.H), nt = column_tile(cols, D, dtype);
    if (nt == 16) return launch_one<T, D, 16>(c, p, s);
    if constexpr (sizeof(T) == 2 && D != 256)
        if (nt == 64) return launch_one<T, D, 64>(c, p, s);
    return launch_one<T, D, 32>(c, p, s);
}

template <typename T> cudaError_t launch(const CacheView &c, const AttnParams &p, int dtype, cudaStream_t s)
{
    if (c.D == 64) return launch_width<T, 64>(c, p, dtype, s);
    if (c.D == 128) return launch_width<T, 128>(c, p, dtype, s);
    return launch_width<T, 256>(c, p, dtype, s);
}

}  // namespace

cudaError_t launch_cache_weights(const CacheView &c, const AttnParams &p, int dtype, cudaStream_t s)
{
    return dtype == SPEC_BF16 ? launch<__nv_bfloat16>(c, p, dtype, s) : launch<float>(c, p, dtype, s);
}

}  // namespace specv
