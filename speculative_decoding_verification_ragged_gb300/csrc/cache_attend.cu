// cache_attend.cu -- attention of packed verify rows over the 4-bit paged cache
// (include/spec_cache.h).
//
// For one request and kv head the step's query rows are columns of a matrix:
// column j * group + g is row j of query head h * group + g.  Over tiles of 128
// tokens
//     S^T = K Q^T          [tokens x columns]
//     P^T = 2^(S^T c - m)  m: a running reference per column
//     O^T += V^T P^T       [channels x columns]
// so that the cache is the A operand of both products: M is always full (128
// tokens, 128 channels), N is the handful of columns, and a row of A is one
// token's key or one channel's values -- a thread decodes exactly one row,
// straight from shared memory into tensor memory (e2m1 and e4m3 convert to f16
// in one instruction a pair, their product is exact in f16).
//
// P is f16: 2^(x + 11), x the score less its reference in log2 units.  The
// reference moves only when a score passes it by 2^4 (the accumulators and sums
// are rescaled then), so that P stays below 2^15 and keeps its 11 bits down to
// x = -25.  A tile with a visible weight below that takes the product with bf16
// operands instead (values exact in bf16 too, weights as a sum of two or three
// bf16 terms): small weights keep their bits, whatever the largest is.
// Queries are scaled by a power of two to f16: 8-bit bf16 mantissas are exact
// down to 2^-31 of the tile's largest, fp32 queries are a sum of two f16 (22
// bits), and so are fp32 outputs' weights.  Products accumulate in fp32, sums
// of weights in fp32 before any rounding.
#include <climits>

#include "attend.cuh"

namespace specv {

namespace {

constexpr float kUnset = -1e30f;           // reference of a column that has seen nothing yet
constexpr float kHeadroom = 11.f;          // P = 2^(x + 11) ...
constexpr float kExceed = 15.f;            // ... stays below 2^15
// V decoded to bf16 keeps f16's exponent bits, which stand for 2^-112 of the
// value there; the weights carry the 2^112
constexpr float kWideScale = 5.192296858534828e33f;

template <typename T, int D_, int NT_> struct Attn {
    static constexpr int D = D_, NT = NT_;
    static constexpr int PIECES = sizeof(T) == 4 ? 2 : 1;      // f16 terms of a query and of a weight
    static constexpr int WIDE = sizeof(T) == 4 ? 3 : 2;        // bf16 terms of a weight in a wide tile
    // exponent of the smallest weight with its bits in f16: a normal number; for
    // two terms 15 bits above the last place, 2^-25
    static constexpr float LEAST_EXP = sizeof(T) == 4 ? -10.f : -14.f;
    // D = 64 fills the 128 lanes of V^T with two halves of the tile's tokens,
    // each with its own columns of P^T; D = 256 takes two products of 128 channels
    static constexpr int HALVES = D == 64 ? 2 : 1;
    static constexpr int VM = D == 256 ? 2 : 1;
    static constexpr int VT = kTile / HALVES;                  // tokens of a V^T row
    static constexpr int A_COLS = D == 256 ? 128 : D / 2;      // tensor memory of K, then of V^T
    static constexpr int O_COLS = NT * HALVES * VM;
    static constexpr int USED = A_COLS + NT + O_COLS;
    static constexpr int COLS = USED <= 128 ? 128 : (USED <= 256 ? 256 : 512);
    static constexpr int Q_BYTES = NT * D * 2;
    static constexpr int P_BYTES = kTile * NT * 2;
    static constexpr int STAGE = 4 * block_bytes(D);
    // As many CTAs an SM as its tensor memory holds (512 / COLS) share 227 KB:
    // what the operands leave goes to stages.  No more CTAs than that fit, so
    // that none waits for tensor memory.
    static constexpr int CTAS = 512 / COLS;
    static constexpr int SHARE = 232448 / CTAS - 1024 - 3584;  // less the system's and the static part
    static constexpr int OPERANDS = PIECES * (Q_BYTES + P_BYTES);
    static constexpr int FIT = (SHARE - OPERANDS) / STAGE;
    static constexpr int STAGES = FIT < 2 ? 2 : (FIT > 4 ? 4 : FIT);
    static constexpr int NEED = OPERANDS + STAGES * STAGE;
    static constexpr int LEAST = 232448 / (CTAS + 1);          // one CTA more would not fit
    static constexpr int SMEM = NEED > LEAST ? NEED : LEAST;
    static_assert(D != 64 || NT * D * 4 <= STAGES * STAGE, "the epilogue's exchange fits the stages");
};

// The values of one channel over the 32 tokens of a block -> 16 columns.  Tokens
// past nv get scale 0 (their bytes can be anything, NaN scales included).
template <int D, bool WIDE>
__device__ __forceinline__ void decode_values(const uint8_t *blk, int d, int nv, uint32_t taddr)
{
    const uint4 v = *reinterpret_cast<const uint4 *>(blk + v_codes_at(D) + d * 16);
    uint4 s[2];
    s[0] = *reinterpret_cast<const uint4 *>(blk + v_scale_at(D) + d / 16 * kTok);
    s[1] = *reinterpret_cast<const uint4 *>(blk + v_scale_at(D) + d / 16 * kTok + 16);
    uint32_t sw[8] = {s[0].x, s[0].y, s[0].z, s[0].w, s[1].x, s[1].y, s[1].z, s[1].w};
    if (nv < kTok) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int n = nv - 4 * i;
            sw[i] = n >= 4 ? sw[i] : (n <= 0 ? 0u : sw[i] & ((1u << 8 * n) - 1u));
        }
    }
    uint32_t r[16];
    decode4(v.x, r);
    decode4(v.y, r + 4);
    decode4(v.z, r + 8);
    decode4(v.w, r + 12);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        r[i] = h2_mul(r[i], e4m3x2(sw[i / 2] >> (i % 2 * 16)));
        // f16 (no subnormals here: the smallest product is 2^-10) to bf16 bits
        if (WIDE) r[i] = (r[i] >> 3 & 0x0FFF0FFFu) | (r[i] & 0x80008000u);
    }
    tmem_st16(taddr, r);
}

// O^T += V^T P^T over the tile's tokens, `pieces` terms of P (one thread issues)
template <typename A, bool WIDE>
__device__ __forceinline__ void issue_values(uint32_t o_addr, uint32_t a_addr, const uint8_t *ps, bool accumulate)
{
    const uint32_t pa = smem_addr(ps);
#pragma unroll
    for (int m = 0; m < A::VM; ++m)
#pragma unroll
        for (int pc = 0; pc < (WIDE ? 1 : A::PIECES); ++pc)
#pragma unroll
            for (int q = 0; q < A::VT / 16; ++q)
                mma_f16(o_addr + m * A::NT, a_addr + m * 64 + q * 8,
                        smem_desc(pa + pc * A::P_BYTES + q * 256, 128, A::VT * 16),
                        mma_f16_desc(A::NT * A::HALVES, true, WIDE), accumulate || pc > 0 || q > 0);
}

// every channel's values of the tile into tensor memory
template <typename A, bool WIDE>
__device__ __forceinline__ void decode_tile_values(const uint8_t *stage, const int *nv, uint32_t taddr)
{
    constexpr int D = A::D;
    const int tid = threadIdx.x;
#pragma unroll
    for (int m = 0; m < A::VM; ++m)
#pragma unroll
        for (int q = 0; q < 4 / A::HALVES; ++q) {
            const int blk = (D == 64 ? tid / 64 * 2 : 0) + q, d = D == 64 ? tid % 64 : m * 128 + tid;
            decode_values<D, WIDE>(stage + blk * block_bytes(D), d, nv[blk], taddr + m * 64 + q * 16);
        }
}

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Sum over the 32 lanes of each of 16 values: lane l gets the sum of value l/2
// (halving the values at each exchange: 16 shuffles).
__device__ __forceinline__ float lane_sums16(float (&v)[16])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 8; k >= 1; k >>= 1) {
        const bool up = lane & (2 * k);
#pragma unroll
        for (int i = 0; i < k; ++i) {
            const float send = up ? v[i] : v[i + k], keep = up ? v[i + k] : v[i];
            v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, 2 * k);
        }
    }
    return v[0] + __shfl_xor_sync(0xFFFFFFFFu, v[0], 1);
}

struct Split {
    int tiles, most;            // tiles of a split, splits of the longest request
    int qtiles, cols;           // column tiles, columns of a request at most
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, (Attn<T, D, NT>::CTAS))
attend_kernel(const CacheView c, const AttnParams p, const Split sp)
{
    using A = Attn<T, D, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *qs = smem, *ps = qs + A::PIECES * A::Q_BYTES, *stages = ps + A::PIECES * A::P_BYTES;
    __shared__ __align__(8) uint64_t full[A::STAGES], s_bar, o_bar;
    __shared__ uint32_t tmem_base, arrived;
    __shared__ int nv[A::STAGES][4], own_s[NT], pos_s[NT];
    __shared__ __align__(16) float ref_s[NT], f_s[NT], slope_s[NT], l_s[NT], wred[4][NT];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int group = p.Hq / c.H;
    Job w;
    const int split = blockIdx.y;
    w.h = blockIdx.x / sp.qtiles;
    w.b = blockIdx.z;
    w.col0 = static_cast<int>(blockIdx.x) % sp.qtiles * NT;
    if (!request_rows(p.cu_rows, w.b, p.R_cap, p.k_max + 1, p.status, w.lo, w.n)) return;
    w.ncols = min(w.n * group - w.col0, NT);
    if (w.ncols <= 0) return;
    w.len = p.len[w.b];
    if (w.len < 0 || w.len > p.max_len) {
        if (tid == 0) set_status(p.status, SPEC_STATUS_BAD_LENGTH);
        w.len = 0;
    }
    visible_tiles(p, w);
    const int nsplit = max((w.ntiles + sp.tiles - 1) / sp.tiles, 1);
    if (split >= nsplit) return;
    const int i0 = split * sp.tiles, i1 = min(i0 + sp.tiles, w.ntiles);

    if (tid == 0) {
        for (int i = 0; i < A::STAGES; ++i) mbar_init(&full[i], 1);
        mbar_init(&s_bar, 1);
        mbar_init(&o_bar, 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&tmem_base, A::COLS);
    int page = -1;
    if (warp == 3) {
        // the loads of the first tiles go out before the queries are staged
        __syncwarp();
        page = i0 < i1 ? tile_page(c, w, tile_of(w, i0)) : -1;
    }
    if (tid < NT) {
        const int col = w.col0 + tid, j = min(col / group, w.n - 1);
        const int own = w.len > 0 ? w.len - w.n + j : -1;
        own_s[tid] = own;
        pos_s[tid] = own >= 0 ? slot_position(c, p, w.b, own) : 0;
        slope_s[tid] = p.slopes && tid < w.ncols ? p.slopes[w.h * group + col % group] * kLog2e : 0.f;
        ref_s[tid] = tid < w.ncols ? kHeadroom - kUnset : 0.f;         // (a padded column's results are unused)
    }
    __syncthreads();
    if (warp == 3) {
#pragma unroll
        for (int i = 0; i < A::STAGES; ++i) {
            if (i0 + i < i1)
                load_tile<block_bytes(D)>(c, w, w.h, tile_of(w, i0 + i), page, stages + i * A::STAGE, &full[i], nv[i], p.status);
            page = i0 + i + 1 < i1 ? tile_page(c, w, tile_of(w, i0 + i + 1)) : -1;
        }
    }
    const float down = stage_queries<T, D, NT, A::PIECES>(p, w, group, qs, l_s);
    const float gk = c.k_scale ? c.k_scale[w.h] : 1.f, gv = c.v_scale ? c.v_scale[w.h] : 1.f;
    const bool options = p.cap > 0.f || p.slopes || p.window > 0;
    // raw product -> score: natural units before the options, log2 units without
    const float mult = p.scale == 0.f ? 1.f : fmaxf(fabsf(p.scale) * gk * down * kLog2e, 1e-37f);
    const uint32_t tm = tmem_base, a_t = tm, s_t = tm + A::A_COLS, o_t = s_t + NT;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;

    float l[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) l[i] = 0.f;
    bool fail = false;
    int o_count = 0;                                                 // completed products with V^T
    const int own_first = own_s[0];
    int i = i0;
    for (; i < i1; ++i) {
        const int k = i - i0, st = k % A::STAGES, tile = tile_of(w, i);
        uint8_t *stage = stages + st * A::STAGE;
        const int slot = tile * kTile + tid;
        int tpos = slot;
        fail |= !mbar_wait(&full[st], k / A::STAGES & 1);
        const int nv_mine = nv[st][warp];
        if (options && p.slot_pos && lane < nv_mine) tpos = slot_position(c, p, w.b, slot);
        if (k > 0) fail |= !mbar_wait(&o_bar, o_count++ & 1);        // V^T of the last tile is used up
        tmem_fence_after();
        decode_keys<D>(stage + warp * block_bytes(D), a_t + lane_off);
        tmem_wait_st();
        tmem_fence_before();
        fence_proxy_async_smem();                                    // the queries, before the first product
        if (__syncthreads_or(fail)) break;
        if (tid == 0) {
            tmem_fence_after();
            issue_scores<D, NT, A::PIECES>(s_t, a_t, qs);
            mma_commit(&s_bar);
        }
        fail |= !mbar_wait(&s_bar, k & 1);
        tmem_fence_after();
        float v[NT];
#pragma unroll
        for (int q = 0; q < NT; q += 16) tmem_ld16(s_t + lane_off + q, reinterpret_cast<uint32_t *>(v) + q);
        tmem_wait_ld();
        const bool edge = (tile + 1) * kTile - 1 > own_first || nv_mine < kTok;
        float mul = mult;
        if (options) {
            mul = 1.f;
            const float twice = p.cap > 0.f ? 2.f / p.cap : 0.f;
#pragma unroll
            for (int q = 0; q < NT; ++q) v[q] = option_score(p.cap, twice, v[q], mult, slope_s[q], pos_s[q] - tpos);
        }
        if (edge || options) {
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                const bool see = lane < nv_mine && slot <= own_s[q] &&
                                 (p.window <= 0 || pos_s[q] - tpos < p.window || slot < p.prefix);
                v[q] = see && q < w.ncols ? v[q] : -INFINITY;
            }
        }
        float most = -INFINITY, least = INFINITY;
        const auto extremes = [&] {
            least = INFINITY;
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                const float x = fmaf(v[q], mul, ref_s[q]);
                most = fmaxf(most, x);
                least = fminf(least, (edge || options) && x == -INFINITY ? INFINITY : x);
            }
        };
        extremes();
        bool wide = false;
        if (__syncthreads_or(most > kExceed || least < A::LEAST_EXP)) {
          if (__syncthreads_or(most > kExceed)) {
            // move the references to the tile's maxima
#pragma unroll
            for (int q0 = 0; q0 < NT; q0 += 16) {
                float mine = 0.f;
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const float x = warp_max_f32(v[q0 + q] * mul);
                    if (lane == q) mine = x;
                }
                if (lane < 16) wred[warp][q0 + lane] = mine;
            }
            __syncthreads();
            if (tid < NT) {
                const float old = kHeadroom - ref_s[tid];
                const float r = fmaxf(fmaxf(wred[0][tid], wred[1][tid]), fmaxf(wred[2][tid], wred[3][tid]));
                const float m = fmaxf(old, r);
                f_s[tid] = tid < w.ncols ? ex2(old - m) : 1.f;
                ref_s[tid] = tid < w.ncols ? kHeadroom - m : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int q = 0; q < NT; ++q) l[q] *= f_s[q];
            if (k > 0) {
#pragma unroll 1
                for (int q0 = 0; q0 < A::O_COLS; q0 += 16) {
                    uint32_t r[16];
                    tmem_ld16(o_t + lane_off + q0, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 16; ++q) r[q] = __float_as_uint(__uint_as_float(r[q]) * f_s[(q0 + q) % NT]);
                    tmem_st16(o_t + lane_off + q0, r);
                }
                tmem_wait_st();
            }
            extremes();
          }
          wide = __syncthreads_or(least < A::LEAST_EXP);
        }
        if (wide) {
            decode_tile_values<A, true>(stage, nv[st], a_t + lane_off);
            tmem_wait_st();
#pragma unroll
            for (int q = 0; q < NT; ++q) l[q] += ex2(fmaf(v[q], mul, ref_s[q]));
            for (int pc = 0; pc < A::WIDE; ++pc) {
                if (pc > 0) fail |= !mbar_wait(&o_bar, o_count++ & 1);
                constexpr int PN8 = A::VT * 16;
                uint8_t *dst = ps + (tid / A::VT) * (NT / 8) * PN8 + tid % A::VT * 16;
#pragma unroll
                for (int q0 = 0; q0 < NT; q0 += 8) {
                    uint32_t term[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float x = ex2(fmaf(v[q0 + 2 * q], mul, ref_s[q0 + 2 * q])) * kWideScale;
                        float y = ex2(fmaf(v[q0 + 2 * q + 1], mul, ref_s[q0 + 2 * q + 1])) * kWideScale;
                        term[q] = pack_bf2(x, y);
                        for (int k = 0; k < pc; ++k) {
                            x -= bf_lo(term[q]);
                            y -= bf_hi(term[q]);
                            term[q] = pack_bf2(x, y);
                        }
                    }
                    *reinterpret_cast<uint4 *>(dst + q0 / 8 * PN8) = make_uint4(term[0], term[1], term[2], term[3]);
                }
                tmem_fence_before();
                fence_proxy_async_smem();
                if (__syncthreads_or(fail)) break;
                if (tid == 0) {
                    tmem_fence_after();
                    issue_values<A, true>(o_t, a_t, ps, k > 0 || pc > 0);
                    mma_commit(&o_bar);
                }
            }
            if (__syncthreads_or(fail)) break;
        } else {
            // weights: sums in fp32, the operand in f16, 8 columns of this token per store
            constexpr int PN8 = A::VT * 16;
            uint8_t *dst = ps + (tid / A::VT) * (NT / 8) * PN8 + tid % A::VT * 16;
#pragma unroll
            for (int q0 = 0; q0 < NT; q0 += 8) {
                float x[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    x[q] = ex2(fmaf(v[q0 + q], mul, ref_s[q0 + q]));
                    l[q0 + q] += x[q];
                }
                uint32_t hi[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) hi[q] = pack_h2(x[2 * q], x[2 * q + 1]);
                *reinterpret_cast<uint4 *>(dst + q0 / 8 * PN8) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                if (A::PIECES == 2) {
                    uint32_t lo[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 y = h2_float2(hi[q]);
                        lo[q] = pack_h2(x[2 * q] - y.x, x[2 * q + 1] - y.y);
                    }
                    *reinterpret_cast<uint4 *>(dst + A::P_BYTES + q0 / 8 * PN8) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            // values over the keys' columns (the product that read them is complete)
            decode_tile_values<A, false>(stage, nv[st], a_t + lane_off);
            tmem_wait_st();
            tmem_fence_before();
            fence_proxy_async_smem();
            if (__syncthreads_or(fail)) break;
            if (tid == 0) {
                tmem_fence_after();
                issue_values<A, false>(o_t, a_t, ps, k > 0);
                mma_commit(&o_bar);
            }
        }
        if (warp == 3 && i + A::STAGES < i1) {
            load_tile<block_bytes(D)>(c, w, w.h, tile_of(w, i + A::STAGES), page, stage, &full[st], nv[st], p.status);
            page = i + A::STAGES + 1 < i1 ? tile_page(c, w, tile_of(w, i + A::STAGES + 1)) : -1;
        }
    }
    if (i1 > i0 && !fail) fail = !mbar_wait(&o_bar, o_count & 1);
    if (__syncthreads_or(fail)) {
        // a wait gave up: let the copies in flight land (bounded), then leave
        if (tid == 0) {
            for (int s = 0; s < A::STAGES; ++s)
                for (int ph = 0; ph < 2; ++ph) mbar_wait(&full[s], ph);
            set_status(p.status, SPEC_STATUS_TIMEOUT);
        }
        __syncthreads();
        if (warp == 0) tmem_free(tm, A::COLS);
        return;
    }
    tmem_fence_after();

    // sums over the tile's tokens (= threads)
#pragma unroll
    for (int q0 = 0; q0 < NT; q0 += 16) {
        float v[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = l[q0 + q];
        const float s = lane_sums16(v);
        // halving order: lane bits 4..1 select value bits 3..0
        if ((lane & 1) == 0) wred[warp][q0 + (lane >> 1)] = s;
    }
    __syncthreads();
    if (tid < NT) {
        // back to units of the reference: P carried 2^headroom
        l_s[tid] = (wred[0][tid] + wred[1][tid]) + (wred[2][tid] + wred[3][tid]);
    }
    __syncthreads();

    const bool seen = i1 > i0;
    const int64_t task = (static_cast<int64_t>(w.b) * c.H + w.h) * sp.qtiles + blockIdx.x % sp.qtiles;
    // partials of a task: [split][NT][D] fp32, then [split][NT] (reference, sum)
    float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(p.ws) +
                                            (static_cast<int64_t>(c.B) * c.H * sp.qtiles * 4 + 255) / 256 * 256) +
                  task * sp.most * NT * (D + 2);
    float2 *ml = reinterpret_cast<float2 *>(part + static_cast<int64_t>(sp.most) * NT * D);
    float *xch = reinterpret_cast<float *>(stages);
#pragma unroll
    for (int m = 0; m < A::VM; ++m) {
        if (D == 64 && seen) {
            // the upper lanes hold the second half of the tokens
            if (warp >= 2)
#pragma unroll
                for (int q0 = 0; q0 < NT; q0 += 16) {
                    uint32_t r[16];
                    tmem_ld16(o_t + lane_off + NT + q0, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 16; ++q) xch[(q0 + q) * 64 + tid - 64] = __uint_as_float(r[q]);
                }
            __syncthreads();
        }
        if (D != 64 || warp < 2) {
            const int d = m * 128 + tid;
#pragma unroll
            for (int q0 = 0; q0 < NT; q0 += 16) {
                uint32_t r[16] = {};
                if (seen) {
                    tmem_ld16(o_t + lane_off + m * NT + q0, r);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int col = w.col0 + q0 + q;
                    if (q0 + q >= w.ncols) continue;
                    float o = __uint_as_float(r[q]);
                    if (D == 64 && seen) o += xch[(q0 + q) * 64 + tid];
                    if (nsplit > 1) {
                        part[(static_cast<int64_t>(split) * NT + q0 + q) * D + d] = o;
                    } else {
                        const float ls = l_s[q0 + q];
                        const int64_t at = static_cast<int64_t>(w.lo + col / group) * p.Hq + w.h * group + col % group;
                        static_cast<T *>(p.out)[at * D + d] = from_f32<T>(ls > 0.f ? o * (gv / ls) : 0.f);
                    }
                }
            }
        }
    }
    if (tid < w.ncols) {
        const float m = kHeadroom - ref_s[tid], ls = l_s[tid];
        if (nsplit > 1) {
            ml[split * NT + tid] = make_float2(m, ls);
        } else if (p.lse) {
            const int col = w.col0 + tid;
            const int64_t at = static_cast<int64_t>(w.lo + col / group) * p.Hq + w.h * group + col % group;
            p.lse[at] = ls > 0.f ? (m - kHeadroom + log2f(ls)) * kLn2 : -INFINITY;
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 0) tmem_free(tm, A::COLS);
    if (nsplit == 1) return;

    // the split that arrives last joins them, in split order
    uint32_t *ticket = static_cast<uint32_t *>(p.ws) + task;
    if (tid == 0) {
        fence_acq_rel_gpu();
        arrived = atomicAdd(ticket, 1u);
        fence_acq_rel_gpu();
    }
    __syncthreads();
    if (arrived != static_cast<uint32_t>(nsplit - 1)) return;
    if (tid == 0) *ticket = 0u;
    for (int col = warp; col < w.ncols; col += 4) {
        float M = kUnset;
        for (int s = lane; s < nsplit; s += 32) {
            const float2 x = __ldcg(ml + s * NT + col);
            if (x.y > 0.f) M = fmaxf(M, x.x);
        }
        M = warp_max_f32(M);
        float L = 0.f;
        float o[D / 32] = {};
        for (int s0 = 0; s0 < nsplit; s0 += 32) {
            float2 x = make_float2(0.f, 0.f);
            if (s0 + lane < nsplit) x = __ldcg(ml + (s0 + lane) * NT + col);
            const float f = x.y > 0.f ? ex2(x.x - M) : 0.f;
            const float lf = f * x.y;
            for (int s = 0; s < min(32, nsplit - s0); ++s) {
                const float fs = __shfl_sync(0xFFFFFFFFu, f, s);
                L += __shfl_sync(0xFFFFFFFFu, lf, s);
                const float *src = part + (static_cast<int64_t>(s0 + s) * NT + col) * D;
#pragma unroll
                for (int q = 0; q < D / 32; ++q) o[q] += fs * __ldcg(src + q * 32 + lane);
            }
        }
        const int cc = w.col0 + col;
        const int64_t at = static_cast<int64_t>(w.lo + cc / group) * p.Hq + w.h * group + cc % group;
#pragma unroll
        for (int q = 0; q < D / 32; ++q)
            static_cast<T *>(p.out)[at * D + q * 32 + lane] = from_f32<T>(L > 0.f ? o[q] * (gv / L) : 0.f);
        if (p.lse && lane == 0) p.lse[at] = L > 0.f ? (M - kHeadroom + log2f(L)) * kLn2 : -INFINITY;
    }
}

// Tiles of a split: as many splits as two rounds of resident CTAs need, so that
// ragged requests even out.
Split split_of(int B, int k_max, int Hq, int H, int D, int max_len, int dtype)
{
    Split s;
    s.cols = (k_max + 1) * (Hq / H);
    const int nt = column_tile(s.cols, D, dtype);
    s.qtiles = (s.cols + nt - 1) / nt;
    const int tiles = (max_len + kTile - 1) / kTile;
    const int64_t all = static_cast<int64_t>(B) * H * s.qtiles * tiles;
    const int64_t slots = 152 * 4 * 2;
    const int64_t t = (all + slots - 1) / slots;
    s.tiles = static_cast<int>(t < 1 ? 1 : (t > tiles ? tiles : t));
    s.most = (tiles + s.tiles - 1) / s.tiles;
    return s;
}

template <typename T, int D, int NT>
cudaError_t launch_one(const CacheView &c, const AttnParams &p, const Split &sp, cudaStream_t s)
{
    using A = Attn<T, D, NT>;
    static bool done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev]) {
        e = cudaFuncSetAttribute(attend_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, A::SMEM);
        if (e != cudaSuccess) return e;
        done[dev] = true;
    }
    const dim3 grid(c.H * sp.qtiles, sp.most, c.B);
    attend_kernel<T, D, NT><<<grid, kAttnThreads, A::SMEM, s>>>(c, p, sp);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_width(const CacheView &c, const AttnParams &p, const Split &sp, int nt, cudaStream_t s)
{
    if (nt == 16) return launch_one<T, D, 16>(c, p, sp, s);
    if constexpr (sizeof(T) == 2 && D != 256)
        if (nt == 64) return launch_one<T, D, 64>(c, p, sp, s);
    return launch_one<T, D, 32>(c, p, sp, s);
}

template <typename T>
cudaError_t launch_attend(const CacheView &c, const AttnParams &p, int dtype, cudaStream_t s)
{
    const Split sp = split_of(c.B, p.k_max, p.Hq, c.H, c.D, p.max_len, dtype);
    const int nt = column_tile(sp.cols, c.D, dtype);
    if (c.D == 64) return launch_width<T, 64>(c, p, sp, nt, s);
    if (c.D == 128) return launch_width<T, 128>(c, p, sp, nt, s);
    return launch_width<T, 256>(c, p, sp, nt, s);
}

}  // namespace

// the larger of the two types' needs: the size does not depend on q's type
size_t cache_attend_workspace(int B, int k_max, int Hq, int H, int D, int max_len)
{
    size_t most = 0;
    for (int dtype : {SPEC_F32, SPEC_BF16}) {
        const Split s = split_of(B, k_max, Hq, H, D, max_len, dtype);
        const size_t tasks = static_cast<size_t>(B) * H * s.qtiles;
        size_t n = (tasks * 4 + 255) / 256 * 256;
        n += tasks * s.most * column_tile(s.cols, D, dtype) * (D + 2) * 4;
        most = n > most ? n : most;
    }
    return most;
}

cudaError_t launch_cache_attend(const CacheView &c, const AttnParams &p, int dtype, cudaStream_t s)
{
    return dtype == SPEC_BF16 ? launch_attend<__nv_bfloat16>(c, p, dtype, s) : launch_attend<float>(c, p, dtype, s);
}

}  // namespace specv
