// attend.cuh -- what the attention (cache_attend.cu) and the weights
// (cache_weights.cu) share: the tiles a request's rows see, their way into
// shared and tensor memory, the queries as an operand, the scores.
//
// 8 warps of a CTA decode.  Tensor memory is reached by quarter: warps w and w + 4
// hold lanes 32 (w % 4) ..., so the two share a quarter's tokens (or channels)
// and split the columns -- of K, of the scores, of the results -- in halves.
#pragma once

#include "cache.cuh"
#include "tensor.cuh"

namespace specv {

constexpr int kAttnThreads = 256;
constexpr int kTile = 128;                 // tokens of a tile: 4 blocks, the lanes of tensor memory

// What a CTA works on.
struct Job {
    int b, h, lo, n, len;       // request, kv head, first packed row, rows, tokens
    int col0, ncols;            // first column of the tile, real columns
    int nsteps, np, f0;         // steps to visit: 0 .. np - 1, then f0, f0 + 1, ...
};

// first slot of the i-th step visited, steps of STEP tokens
template <int STEP> __device__ __forceinline__ int step_slot(const Job &w, int i)
{
    return (i < w.np ? i : w.f0 + i - w.np) * STEP;
}

__device__ __forceinline__ int slot_position(const CacheView &c, const AttnParams &p, int b, int slot)
{
    if (!p.slot_pos) return slot;
    const int page = page_of(c, b, slot);
    return page < 0 ? 0 : __ldg(p.slot_pos + static_cast<int64_t>(page) * c.page_tokens + slot % c.page_tokens);
}

// The steps that some row of the request sees.  With a window the first row
// sees the prefix and what lies less than `window` positions before its own
// slot; positions do not decrease over slots, so the hidden steps in between
// are counted by an 8-way search over the steps' last slots.  A thread does it
// alone, and always by the same probes: whoever asks gets the same answer.
template <int STEP>
__device__ __forceinline__ void visible_steps(const CacheView &c, const AttnParams &p, Job &w)
{
    w.nsteps = (w.len + STEP - 1) / STEP;
    w.np = 0;
    w.f0 = 0;
    const int own = w.len - w.n;
    if (p.window <= 0 || own <= 0) return;
    int first = max(own - p.window + 1, 0) / STEP;
    if (p.slot_pos) {
        // (in 64 bits: positions can be negative, a window as wide as the type)
        const int64_t limit = static_cast<int64_t>(slot_position(c, p, w.b, own)) - p.window;
        int lo = 0, hi = own / STEP;               // steps below lo are hidden, step hi is not
        while (lo < hi) {
            const int by = (hi - lo + 6) / 7;
            uint32_t hidden = 0;
#pragma unroll
            for (int u = 0; u < 7; ++u) {
                const int t = lo + u * by, slot = t * STEP + STEP - 1;
                // (a bad page has no positions: its step counts as seen, its tokens are masked)
                if (t < hi && page_of(c, w.b, slot) >= 0 && slot_position(c, p, w.b, slot) <= limit) hidden |= 1u << u;
            }
            const int k = __ffs(~hidden) - 1;      // probes 0 .. k - 1 are hidden, probe k is not
            if (k == 0) break;
            if (k < 7) hi = min(hi, lo + k * by);
            lo += (k - 1) * by + 1;
        }
        first = lo;
    }
    w.np = min((p.prefix + STEP - 1) / STEP, first);
    w.f0 = first;
    w.nsteps = w.np + max(w.nsteps - first, 0);
}

// Rows and length of request w.b: false where it has no rows to attend with.
// `status`: where to report what is wrong with it, or null.
template <int STEP>
__device__ __forceinline__ bool load_job(const CacheView &c, const AttnParams &p, Job &w, uint32_t *status)
{
    if (!request_rows(p.cu_rows, w.b, p.R_cap, p.k_max + 1, status, w.lo, w.n) || w.n == 0) return false;
    w.len = p.len[w.b];
    if (w.len < 0 || w.len > p.max_len) {
        set_status(status, SPEC_STATUS_BAD_LENGTH);
        w.len = 0;
    }
    visible_steps<STEP>(c, p, w);
    return true;
}

// Whether the window hides the block from `slot0` on from every row of the request
// (of slots that are their own positions; where slot_pos has those, it has to be read).
__device__ __forceinline__ bool hidden_block(const AttnParams &p, const Job &w, int slot0)
{
    const int own = w.len - w.n;                       // the first row's
    return p.window > 0 && !p.slot_pos && own > 0 && slot0 >= p.prefix && slot0 + kTok - 1 <= own - p.window;
}

// The next tile to fetch, its page ids asked for ahead: a fetch does not wait for
// the page table (the ids are looked at only when the copies are issued).
struct Fetch {
    int h, slot, n, page;       // n, page: of this lane's block, its tokens and the page as the table has it
};

// (WINDOW: there can be one)
template <bool WINDOW>
__device__ __forceinline__ Fetch ask_pages(const CacheView &c, const AttnParams &p, const Job &w, int h, int slot)
{
    const int lane = threadIdx.x & 31, slot0 = slot + lane * kTok;
    Fetch f = {h, slot, 0, -1};
    if (lane < 4 && slot0 < w.len && !(WINDOW && hidden_block(p, w, slot0))) {
        f.n = min(w.len - slot0, kTok);
        f.page = __ldg(c.page_table + static_cast<int64_t>(w.b) * c.max_pages + slot0 / c.page_tokens);
    }
    return f;
}

// Report the blocks `bad` of a tile, whose page id is none.  Where the window goes by
// slot_pos, a page that it hides may have been given back, and then has no positions
// that say so: a run of bad pages counts as hidden where the good page before it ends
// hidden, or where it begins the cache and position 0 is hidden.  The pages of a run
// lead back to its first one, so looking at the 32 pages before is enough: a run that
// rows would see is reported by its first pages.
template <bool WINDOW>
__device__ __forceinline__ void report_pages(const CacheView &c, const AttnParams &p, const Job &w, int slot, uint32_t bad)
{
    const int lane = threadIdx.x & 31, own = w.len - w.n;
    bool report = !WINDOW || p.window <= 0 || !p.slot_pos || own <= 0;
    if (!report) {
        const int64_t limit = static_cast<int64_t>(slot_position(c, p, w.b, own)) - p.window;
        for (uint32_t left = bad & ~(bad << 1); left && !report; left &= left - 1) {
            const int slot0 = slot + (__ffs(left) - 1) * kTok, index = slot0 / c.page_tokens, at = index - 1 - lane;
            const int id = at >= 0 ? __ldg(c.page_table + static_cast<int64_t>(w.b) * c.max_pages + at) : -1;
            const uint32_t good = __ballot_sync(0xFFFFFFFFu, id >= 0 && id < c.n_pages);
            if (good)
                report = slot_position(c, p, w.b, (index - __ffs(good) + 1) * c.page_tokens - 1) > limit;
            else
                report = index <= 32 && limit < 0;
            report = report || slot0 < p.prefix;
        }
    }
    if (report && lane == 0) set_status(p.status, SPEC_STATUS_BAD_PAGE);
}

// Copy the first BYTES of a tile's 4 blocks into a stage (all of a block, or its
// keys); a lane of one warp per block.  nv: the tokens of each block that exist (0
// for a bad page, or a block that the window hides whole: its bytes are not fetched,
// and what the stage holds there is masked); pages, where it is asked for: their page ids.
template <int BYTES, bool WINDOW>
__device__ __forceinline__ void load_tile(const CacheView &c, const AttnParams &p, const Job &w, const Fetch &f, uint8_t *stage,
                                          uint64_t *full, int *nv, int *pages = nullptr)
{
    const int lane = threadIdx.x & 31;
    const int slot0 = f.slot + lane * kTok;
    int n = f.n;
    const uint32_t bad = __ballot_sync(0xFFFFFFFFu, n > 0 && (f.page < 0 || f.page >= c.n_pages));
    if (bad) {
        report_pages<WINDOW>(c, p, w, f.slot, bad);
        if (bad >> lane & 1u) n = 0;
    }
    const uint32_t have = __ballot_sync(0xFFFFFFFFu, n > 0);
    if (lane < 4) nv[lane] = n;
    if (pages && lane < 4) pages[lane] = f.page;
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(full, __popc(have) * BYTES);
    __syncwarp();
    if (n > 0)
        bulk_g2s(stage + lane * BYTES, block_at(c, f.page, f.h, slot0 % c.page_tokens / kTok), BYTES, full);
}

// A wait that has given up once does not wait again: the CTA runs to its end,
// stores nothing and reports the timeout.  (Most waits find their phase complete:
// one try, one branch.)
__device__ __forceinline__ void wait_or_fail(uint64_t *bar, uint32_t parity, bool &fail)
{
    if (!mbar_try(bar, parity) && !fail) fail = !mbar_wait(bar, parity);
}

__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 4 bytes of codes -> 4 f16x2
__device__ __forceinline__ void decode4(uint32_t w, uint32_t *r)
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

__device__ __forceinline__ void decode16(uint4 v, uint32_t (&r)[16])
{
    decode4(v.x, r);
    decode4(v.y, r + 4);
    decode4(v.z, r + 8);
    decode4(v.w, r + 12);
}

// This warp's half of the keys of its lane's token, D/4 columns of tensor memory
// (blk: the quarter's block)
template <int D>
__device__ __forceinline__ void decode_keys(const uint8_t *blk, uint32_t taddr)
{
    const int lane = threadIdx.x & 31, half = threadIdx.x / 128;
    constexpr int G = D / 16, CH = D / 64;           // scales of a token, 32-channel chunks of a half
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int ch = half * CH + i;
        const uint4 v = *reinterpret_cast<const uint4 *>(blk + ch * 512 + lane * 16);
        const uint32_t s2 =
            e4m3x2(*reinterpret_cast<const uint16_t *>(blk + k_scale_at(D) + lane * G + 2 * ch));
        const uint32_t s_lo = __byte_perm(s2, 0, 0x1010), s_hi = __byte_perm(s2, 0, 0x3232);
        uint32_t r[16];
        decode16(v, r);
#pragma unroll
        for (int k = 0; k < 16; ++k) r[k] = h2_mul(r[k], k < 8 ? s_lo : s_hi);
        tmem_st16(taddr + ch * 16, r);
    }
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <typename T>
__device__ __forceinline__ void load8(const T *p, bool aligned, float (&x)[8])
{
    if (aligned) {
        constexpr int N = sizeof(T) / 2;
        uint4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
        const T *e = reinterpret_cast<const T *>(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_f32<T>(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_f32<T>(p[i]);
    }
}

// The query columns of a kv head as the K-major B operand: each scaled by the
// power of two that brings its largest channel to 2^13 (and by the sign of the
// softmax scale), the second f16 term behind the first for fp32.  A thread's
// share, the same for every head, is placed once; a column belongs to D/8 lanes of
// one warp, so staging has no barrier.
//
// A core matrix (8 columns x 8 channels) starts kCore bytes after the one of the
// channels before: the lanes of a column store to different banks.
constexpr int kCore = 144;
__host__ __device__ constexpr int query_bytes(int D, int NT) { return NT / 8 * (D / 8) * kCore; }

template <typename T, int D, int NT, int PIECES> struct QueryStage {
    static constexpr int PER = D / 8;                 // 8-channel groups of a column
    static constexpr int SHARES = (NT * PER + kAttnThreads - 1) / kAttnThreads;
    const T *src[SHARES];                             // in kv head 0; null: no such column

    __device__ __forceinline__ void place(const AttnParams &p, const Job &w, int group)
    {
#pragma unroll
        for (int s = 0; s < SHARES; ++s) {
            const int i = s * kAttnThreads + threadIdx.x, col = w.col0 + i / PER;
            src[s] = i / PER < w.ncols ? static_cast<const T *>(p.q) + (w.lo + col / group) * p.q_row +
                                             col % group * p.q_head + i % PER * 8
                                       : nullptr;
        }
    }

    // kv head h; mult[col] takes a raw product to its score: unit * gk, by the
    // power of two (unit: the softmax scale's magnitude in the units wanted)
    __device__ __forceinline__ void stage(const AttnParams &p, int64_t head, float unit, uint8_t *qs, float *mult) const
    {
#pragma unroll
        for (int s = 0; s < SHARES; ++s) {
            const int i = s * kAttnThreads + threadIdx.x, cl = i / PER, k8 = i % PER;
            if (NT * PER < kAttnThreads && i >= NT * PER) break;         // (whole warps)
            float x[8] = {};
            if (src[s]) load8<T>(src[s] + head, p.q_aligned, x);
            float big = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) big = fmaxf(big, fabsf(x[k]));
#pragma unroll
            for (int o = PER / 2; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
            // exponent arithmetic on the bits; a column of zeros (or subnormals) stays as it is
            const int ex = static_cast<int>(__float_as_uint(big) >> 23) - 127;
            const int e = ex > -127 ? min(max(13 - ex, -120), 100) : 0;
            const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            const float f = p.scale == 0.f ? 0.f : (p.scale < 0.f ? -up : up);
            // never 0, so that a hidden slot's -inf stays -inf
            if (k8 == 0)
                mult[cl] = p.scale == 0.f ? 1.f
                                          : fmaxf(unit * __uint_as_float(static_cast<uint32_t>(127 - e) << 23), 1e-37f);
            uint8_t *dst = qs + (cl / 8 * PER + k8) * kCore + cl % 8 * 16;
            uint32_t hi[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) hi[k] = pack_h2(x[2 * k] * f, x[2 * k + 1] * f);
            *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (PIECES == 2) {
                uint32_t l[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 y = h2_float2(hi[k]);
                    l[k] = pack_h2(x[2 * k] * f - y.x, x[2 * k + 1] * f - y.y);
                }
                *reinterpret_cast<uint4 *>(dst + query_bytes(D, NT)) = make_uint4(l[0], l[1], l[2], l[3]);
            }
        }
    }
};

// S^T = K Q^T over all channels (one warp issues).  The terms of fp32 queries
// go to accumulators of their own, NT columns apart: the tensor cores truncate
// a sum at its last place, and adding the small products of the second term to
// the large sum would cost a bit or two in every step.
template <int D, int NT, int PIECES>
__device__ __forceinline__ void issue_scores(uint32_t s_addr, uint32_t a_addr, uint32_t q)
{
#pragma unroll
    for (int pc = 0; pc < PIECES; ++pc)
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            mma_f16(s_addr + pc * NT, a_addr + k * 8,
                    smem_desc(q + pc * query_bytes(D, NT) + k * 2 * kCore, kCore, D / 8 * kCore),
                    mma_f16_desc(NT, false), k > 0);
}

// N raw products of this thread's token, from column `addr` on
template <int N, int NT, int PIECES>
__device__ __forceinline__ void load_products(uint32_t addr, float (&v)[N])
{
    tmem_ld<N>(addr, reinterpret_cast<uint32_t *>(v));
    if constexpr (PIECES == 2) {
        float t[N];
        tmem_ld<N>(addr + NT, reinterpret_cast<uint32_t *>(t));
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] += t[q];
    } else {
        tmem_wait_ld();
    }
}

// 1 / cap, finite for the smallest cap too (scores of 0 stay 0 under it)
__device__ __forceinline__ float cap_reciprocal(float cap) { return fminf(1.f / cap, 3.4028234663852886e38f); }

// cap * tanh(s / cap), s and the result in units of `unit` (1 or log2 e).  EXACT
// (fp32 results): the library's tanh.  Else (e^2z - 1) / (e^2z + 1), and below 1/2,
// where that cancels, Lambert's continued fraction to its fifth term (9e-11 off):
// within 2^-20 of the result, relative, so that small scores under a large cap keep
// the log-sum-exp's digits; one approximate quotient for the two.
template <bool EXACT>
__device__ __forceinline__ float cap_score(float y, float cap, float rcap)
{
    const float z = y * rcap;
    if (EXACT) return cap * tanhf(z);
    const float t = ex2(fminf(2.f * kLog2e * z, 60.f)), zz = z * z;
    const bool small = fabsf(z) < 0.5f;
    const float num = small ? z * fmaf(zz, zz + 105.f, 945.f) : t - 1.f;
    const float den = small ? fmaf(zz, fmaf(zz, 15.f, 420.f), 945.f) : t + 1.f;
    return cap * __fdividef(num, den);
}

// Columns of a column tile: the fewest of 16, 32, 64 that hold a request's
// rows; 64 only for bf16 heads of up to 128 channels (tensor and shared memory).
inline int column_tile(int cols, int D, int dtype)
{
    if (cols <= 16) return 16;
    if (cols <= 32 || D == 256 || dtype == SPEC_F32) return 32;
    return 64;
}

// CTAs an SM by tensor memory (`cols` columns each), and what a CTA may then use
// of the SM's 227 KB, less `fixed` bytes of static shared memory.  No more CTAs
// than that may fit either: one more would sit waiting for tensor memory.
__host__ __device__ constexpr int tmem_cols(int used) { return used <= 128 ? 128 : (used <= 256 ? 256 : 512); }
__host__ __device__ constexpr int smem_share(int ctas, int fixed) { return 232448 / ctas - 1024 - fixed; }
__host__ __device__ constexpr int smem_least(int ctas) { return 232448 / (ctas + 1); }
__host__ __device__ constexpr int clamp_stages(int fit) { return fit < 2 ? 2 : (fit > 4 ? 4 : fit); }

}  // namespace specv
