// cache_weights.cu -- the attention weight that every cached token gets from the
// packed verify rows, added to its score (include/spec_cache.h).
//
// score_j += sum over rows and heads of exp(s_ij - lse_i): with S^T = K Q^T
// (cache_attend.cu) a token is a lane and its sum over the columns and heads
// stays in one thread, in a fixed order -- no atomics, one read and one write of
// the score.  A CTA takes a few tiles of one request through every kv head, so
// that a head's queries are staged once for them; the keys alone are read.
#include "attend.cuh"

namespace specv {

namespace {

constexpr int kMaxTiles = 8;               // tiles of a CTA at most

template <typename T, int D_, int NT_> struct Weights {
    static constexpr int D = D_, NT = NT_;
    static constexpr int PIECES = sizeof(T) == 4 ? 2 : 1;
    static constexpr int K_BYTES = v_codes_at(D);              // a block's keys and their scales
    static constexpr int A_COLS = D / 2;
    static constexpr int COLS = A_COLS + 2 * NT <= 128 ? 128 : 256;
    static constexpr int CTAS = 512 / COLS;
    static constexpr int SHARE = 232448 / CTAS - 1024 - 4096 - kMaxTiles * kTile * 4;
    static constexpr int Q_BYTES = PIECES * NT * D * 2;
    static constexpr int STAGE = 4 * K_BYTES;
    static constexpr int FIT = (SHARE - Q_BYTES) / STAGE;
    static constexpr int STAGES = FIT < 2 ? 2 : (FIT > 4 ? 4 : FIT);
    static constexpr int NEED = Q_BYTES + STAGES * STAGE;
    static constexpr int LEAST = 232448 / (CTAS + 1);          // no more CTAs than tensor memory holds
    static constexpr int SMEM = NEED > LEAST ? NEED : LEAST;
};

// Step of a CTA: tile `t` of its tiles, column tile `qt` of kv head `h`.
struct Step {
    int h, qt, t;
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, (Weights<T, D, NT>::CTAS))
weights_kernel(const CacheView c, const AttnParams p, const int tiles)
{
    using A = Weights<T, D, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *qs = smem, *stages = qs + A::Q_BYTES;
    __shared__ __align__(8) uint64_t full[A::STAGES], s_bar;
    __shared__ uint32_t tmem_base;
    __shared__ int nv[A::STAGES][4], own_s[3][NT], pos_s[3][NT];
    __shared__ __align__(16) float lse_s[3][NT], slope_s[3][NT];
    __shared__ float mult_s[3], red[4], acc[kMaxTiles][kTile];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = p.Hq / c.H;
    Job w;
    w.b = blockIdx.y;
    if (!request_rows(p.cu_rows, w.b, p.R_cap, p.k_max + 1, p.status, w.lo, w.n) || w.n == 0) return;
    w.len = p.len[w.b];
    if (w.len < 0 || w.len > p.max_len) {
        if (tid == 0) set_status(p.status, SPEC_STATUS_BAD_LENGTH);
        return;
    }
    visible_tiles(p, w);
    const int i0 = blockIdx.x * tiles, nt = min(tiles, w.ntiles - i0);
    if (nt <= 0) return;

    const int cols = w.n * group, qt_used = (cols + NT - 1) / NT;
    const int steps = c.H * qt_used * nt;
    const auto step_at = [&](int i) {
        const int t = i % nt, hq = i / nt;
        return Step{hq / qt_used, hq % qt_used, t};
    };
    if (tid == 0) {
        for (int i = 0; i < A::STAGES; ++i) mbar_init(&full[i], 1);
        mbar_init(&s_bar, 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&tmem_base, A::COLS);
    for (int t = 0; t < nt; ++t) acc[t][tid] = 0.f;
    __syncthreads();
    const uint32_t a_t = tmem_base, s_t = a_t + A::A_COLS;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const auto load = [&](int i) {
        const Step s = step_at(i);
        const int tile = tile_of(w, i0 + s.t);
        load_tile<A::K_BYTES>(c, w, s.h, tile, tile_page(c, w, tile), stages + i % A::STAGES * A::STAGE,
                              &full[i % A::STAGES], nv[i % A::STAGES], p.status);
    };
    if (warp == 3)
        for (int i = 0; i < A::STAGES && i < steps; ++i) load(i);

    const bool options = p.cap > 0.f || p.slopes || p.window > 0;
    // weights of a finished product: column constants of set `cb`
    const auto add_weights = [&](int i, int cb) {
        const Step s = step_at(i);
        const int tile = tile_of(w, i0 + s.t), slot = tile * kTile + tid;
        const int valid = min(max(w.len - (slot - lane), 0), kTok);
        float v[NT];
#pragma unroll
        for (int q = 0; q < NT; q += 16)
            tmem_ld16(s_t + (i & 1) * NT + lane_off + q, reinterpret_cast<uint32_t *>(v) + q);
        tmem_wait_ld();
        const float mult = mult_s[cb];
        const bool edge = (tile + 1) * kTile - 1 > own_s[cb][0] || valid < kTok;
        float sum = 0.f;
        if (edge || options) {
            const int tpos = options && p.slot_pos && lane < valid ? slot_position(c, p, w.b, slot) : slot;
            const float twice = p.cap > 0.f ? 2.f / p.cap : 0.f;
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                float y = v[q] * mult;
                const int dist = pos_s[cb][q] - tpos;
                if (options) y = option_score(p.cap, twice, v[q], mult * kLog2e, slope_s[cb][q], dist) * kLn2;
                const bool see = slot <= own_s[cb][q] && (p.window <= 0 || dist < p.window || slot < p.prefix);
                sum += see ? ex2((y - lse_s[cb][q]) * kLog2e) : 0.f;
            }
        } else {
#pragma unroll
            for (int q = 0; q < NT; ++q) sum += ex2(fmaf(v[q], mult, -lse_s[cb][q]) * kLog2e);
        }
        acc[s.t][tid] += sum;
    };

    bool fail = false;
    int cb = 2;
    for (int i = 0; i < steps; ++i) {
        const Step s = step_at(i);
        const int st = i % A::STAGES;
        const int cb_last = cb;
        if (i > 0) {
            fail |= !mbar_wait(&s_bar, (i - 1) & 1);       // the keys' columns and the queries are used up
            tmem_fence_after();
        }
        if (s.t == 0) {
            cb = cb == 2 ? 0 : cb + 1;   // three sets: a slow warp may still read the one before last
            w.h = s.h;
            w.col0 = s.qt * NT;
            w.ncols = min(cols - w.col0, NT);
            if (tid < NT) {
                const int col = min(w.col0 + tid, cols - 1), j = col / group, own = w.len - w.n + j;
                const int head = s.h * group + col % group;
                own_s[cb][tid] = own;
                pos_s[cb][tid] = own >= 0 ? slot_position(c, p, w.b, own) : 0;
                slope_s[cb][tid] = p.slopes ? p.slopes[head] * kLog2e : 0.f;
                // padded columns, and rows that saw nothing: weight exp(-inf) = 0
                const float lse = tid < w.ncols ? p.lse[static_cast<int64_t>(w.lo + j) * p.Hq + head] : INFINITY;
                lse_s[cb][tid] = lse == -INFINITY ? INFINITY : lse;
            }
            const float down = stage_queries<T, D, NT, A::PIECES>(p, w, group, qs, red);
            if (tid == 0)
                mult_s[cb] = p.scale == 0.f ? 1.f : fabsf(p.scale) * (c.k_scale ? c.k_scale[s.h] : 1.f) * down;
        }
        fail |= !mbar_wait(&full[st], i / A::STAGES & 1);
        decode_keys<D>(stages + st * A::STAGE + warp * A::K_BYTES, a_t + lane_off);
        tmem_wait_st();
        tmem_fence_before();
        fence_proxy_async_smem();
        if (__syncthreads_or(fail)) break;
        if (tid == 0) {
            tmem_fence_after();
            issue_scores<D, NT, A::PIECES>(s_t + (i & 1) * NT, a_t, qs);
            mma_commit(&s_bar);
        }
        if (warp == 3 && i + A::STAGES < steps) load(i + A::STAGES);
        if (i > 0) add_weights(i - 1, cb_last);
    }
    if (!fail) fail = !mbar_wait(&s_bar, (steps - 1) & 1);
    tmem_fence_after();
    if (__syncthreads_or(fail)) {
        if (tid == 0) {
            for (int s = 0; s < A::STAGES; ++s)
                for (int ph = 0; ph < 2; ++ph) mbar_wait(&full[s], ph);
            set_status(p.status, SPEC_STATUS_TIMEOUT);
        }
    } else {
        add_weights(steps - 1, cb);
        for (int t = 0; t < nt; ++t) {
            const int slot = tile_of(w, i0 + t) * kTile + tid;
            const int page = slot < w.len ? page_of(c, w.b, slot) : -1;
            if (page >= 0) p.score[static_cast<int64_t>(page) * c.page_tokens + slot % c.page_tokens] += acc[t][tid];
        }
    }
    tmem_fence_before();
    __syncthreads();
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
    // as many tiles a CTA as leave two rounds of resident CTAs
    const int tiles = (p.max_len + kTile - 1) / kTile;
    const int64_t per = static_cast<int64_t>(c.B) * tiles / (152 * A::CTAS * 2);
    const int t = static_cast<int>(per < 1 ? 1 : (per > kMaxTiles ? kMaxTiles : per));
    weights_kernel<T, D, NT><<<dim3((tiles + t - 1) / t, c.B), kAttnThreads, A::SMEM, s>>>(c, p, t);
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
