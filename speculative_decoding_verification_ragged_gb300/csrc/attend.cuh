// attend.cuh -- what the attention (cache_attend.cu) and the weights
// (cache_weights.cu) share: the tiles a request's rows see, their way into
// shared and tensor memory, the queries as an operand, the scores.
#pragma once

#include "cache.cuh"
#include "tensor.cuh"

namespace specv {

constexpr int kAttnThreads = 128;
constexpr int kTile = 128;                 // tokens of a tile: 4 blocks
// What a CTA works on.
struct Job {
    int b, h, lo, n, len;       // request, kv head, first packed row, rows, tokens
    int col0, ncols;            // first column of the tile, real columns
    int ntiles, np, f0;         // tiles to visit: 0 .. np - 1, then f0, f0 + 1, ...
};

__device__ __forceinline__ int tile_of(const Job &w, int i) { return i < w.np ? i : w.f0 + i - w.np; }

__device__ __forceinline__ int slot_position(const CacheView &c, const AttnParams &p, int b, int slot)
{
    if (!p.slot_pos) return slot;
    const int page = page_of(c, b, slot);
    return page < 0 ? 0 : __ldg(p.slot_pos + static_cast<int64_t>(page) * c.page_tokens + slot % c.page_tokens);
}

// The tiles that some row of the request sees.
__device__ __forceinline__ void visible_tiles(const AttnParams &p, Job &w)
{
    w.ntiles = (w.len + kTile - 1) / kTile;
    w.np = 0;
    w.f0 = 0;
    if (p.window > 0 && !p.slot_pos) {
        // the first row sees from slot len - n - window + 1 on, and the prefix
        const int first = max(w.len - w.n - p.window + 1, 0) / kTile;
        w.np = min((p.prefix + kTile - 1) / kTile, first);
        w.f0 = first;
        w.ntiles = w.np + max(w.ntiles - first, 0);
    }
}

// Copy the first BYTES of the 4 blocks of a tile into a stage (all of a block,
// or its keys); lanes 0..3 of one warp, a block each.  nv: the tokens of each block that exist (0 for a bad page: its bytes
// are not fetched, and what the stage holds there is masked).
template <int BYTES>
__device__ __forceinline__ void load_tile(const CacheView &c, const Job &w, int h, int tile, int page, uint8_t *stage,
                                          uint64_t *full, int *nv, uint32_t *status)
{
    const int lane = threadIdx.x & 31;
    const int slot0 = tile * kTile + lane * kTok;
    int n = lane < 4 ? min(max(w.len - slot0, 0), kTok) : 0;
    if (n > 0 && page < 0) {
        set_status(status, SPEC_STATUS_BAD_PAGE);
        n = 0;
    }
    const uint32_t have = __ballot_sync(0xFFFFFFFFu, n > 0);
    if (lane < 4) nv[lane] = n;
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(full, __popc(have) * BYTES);
    __syncwarp();
    if (n > 0)
        bulk_g2s(stage + lane * BYTES, block_at(c, page, h, slot0 % c.page_tokens / kTok), BYTES, full);
}

__device__ __forceinline__ int tile_page(const CacheView &c, const Job &w, int tile)
{
    const int lane = threadIdx.x & 31, slot0 = tile * kTile + lane * kTok;
    return lane < 4 && slot0 < w.len ? page_of(c, w.b, slot0) : -1;
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

// The keys of this thread's token (block = warp, token = lane) -> D/2 columns
template <int D>
__device__ __forceinline__ void decode_keys(const uint8_t *blk, uint32_t taddr)
{
    const int lane = threadIdx.x & 31;
    constexpr int G = D / 16;
    uint32_t sc[G / 4];
#pragma unroll
    for (int i = 0; i < G / 4; ++i)
        sc[i] = *reinterpret_cast<const uint32_t *>(blk + k_scale_at(D) + lane * G + 4 * i);
#pragma unroll
    for (int ch = 0; ch < D / 32; ++ch) {
        const uint4 v = *reinterpret_cast<const uint4 *>(blk + ch * 512 + lane * 16);
        const uint32_t s2 = e4m3x2(sc[ch / 2] >> (ch % 2 * 16));
        const uint32_t s_lo = __byte_perm(s2, 0, 0x1010), s_hi = __byte_perm(s2, 0, 0x3232);
        uint32_t r[16];
        decode4(v.x, r);
        decode4(v.y, r + 4);
        decode4(v.z, r + 8);
        decode4(v.w, r + 12);
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = h2_mul(r[i], i < 8 ? s_lo : s_hi);
        tmem_st16(taddr + ch * 16, r);
    }
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Query columns as the K-major B operand, scaled by the power of two 2^e (and
// the sign of the softmax scale) that brings the tile's largest to 2^14; the
// second f16 term behind the first for fp32.  Returns 2^-e.
template <typename T, int D, int NT, int PIECES>
__device__ float stage_queries(const AttnParams &p, const Job &w, int group, uint8_t *qs, float *red)
{
    const int tid = threadIdx.x;
    constexpr int PER = D / 8;                        // 8-channel groups of a column
    float big = 0.f;
    for (int i = tid; i < w.ncols * PER; i += kAttnThreads) {
        const int col = w.col0 + i / PER;
        const T *src = static_cast<const T *>(p.q) + (w.lo + col / group) * p.q_row +
                       (w.h * group + col % group) * p.q_head + i % PER * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) big = fmaxf(big, fabsf(to_f32<T>(src[k])));
    }
    big = warp_max_f32(big);
    if ((tid & 31) == 0) red[tid >> 5] = big;
    __syncthreads();
    big = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    // exponent arithmetic on the bits; a tile of zeros (or subnormals) stays as it is
    const int ex = static_cast<int>(__float_as_uint(big) >> 23) - 127;
    const int e = ex > -127 ? min(max(13 - ex, -120), 100) : 0;
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    const float f = p.scale == 0.f ? 0.f : (p.scale < 0.f ? -up : up);
    for (int i = tid; i < NT * PER; i += kAttnThreads) {
        const int c = i / PER, k8 = i % PER, col = w.col0 + c;
        float x[8] = {};
        if (c < w.ncols) {
            const T *src = static_cast<const T *>(p.q) + (w.lo + col / group) * p.q_row +
                           (w.h * group + col % group) * p.q_head + k8 * 8;
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = to_f32<T>(src[k]) * f;
        }
        uint8_t *dst = qs + k8 * (NT * 16) + c / 8 * 128 + c % 8 * 16;
        uint32_t hi[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) hi[k] = pack_h2(x[2 * k], x[2 * k + 1]);
        *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (PIECES == 2) {
            uint32_t l[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 y = h2_float2(hi[k]);
                l[k] = pack_h2(x[2 * k] - y.x, x[2 * k + 1] - y.y);
            }
            *reinterpret_cast<uint4 *>(dst + NT * D * 2) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    }
    return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// S^T = K Q^T over all channels (one thread issues)
template <int D, int NT, int PIECES>
__device__ __forceinline__ void issue_scores(uint32_t s_addr, uint32_t a_addr, const uint8_t *qs)
{
    const uint32_t q = smem_addr(qs);
#pragma unroll
    for (int pc = 0; pc < PIECES; ++pc)
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            mma_f16(s_addr, a_addr + k * 8, smem_desc(q + pc * NT * D * 2 + k * 2 * NT * 16, NT * 16, 128),
                    mma_f16_desc(NT, false), pc > 0 || k > 0);
}

// the score in log2 units of a raw product, with cap and distance bias
__device__ __forceinline__ float option_score(float cap, float twice, float v, float mult, float slope2, int dist)
{
    float y = v * mult;
    if (cap > 0.f) {
        // cap tanh(s / cap) = cap - 2 cap / (1 + 2^(2 y / cap))  (y in log2 units)
        const float c2 = cap * kLog2e;
        const float t = 1.f + ex2(fminf(twice * y, 126.f));
        y = c2 - __fdividef(2.f * c2, t);
    }
    return y - slope2 * static_cast<float>(dist);
}

// Columns of a column tile: the fewest of 16, 32, 64 that hold a request's
// rows; 64 only for bf16 heads of up to 128 channels (tensor and shared memory).
inline int column_tile(int cols, int D, int dtype)
{
    if (cols <= 16) return 16;
    if (cols <= 32 || D == 256 || dtype == SPEC_F32) return 32;
    return 64;
}

}  // namespace specv
