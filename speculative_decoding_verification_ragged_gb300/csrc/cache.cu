// cache.cu -- the 4-bit paged cache itself: append (quantise and write), read,
// and eviction by accumulated attention weight (include/spec_cache.h).
#include <climits>

#include "cache.cuh"

namespace specv {

namespace {

constexpr int kRowThreads = 128;

// The slots of request b that rows touch inside its `idx`-th block: false when
// the block has none.  `start` .. `start + n - 1` are checked once per CTA.
struct BlockRows {
    int lo, n, start;       // first packed row, rows and first slot of the request
    int first, last;        // tokens of this block that are rows: first .. last - 1
    int slot0;              // slot of token 0 of the block
};

__device__ __forceinline__ bool block_rows(const CacheView &c, const CacheRows &r, int b, int idx,
                                           BlockRows &o)
{
    if (!request_rows(r.cu_rows, b, r.R_cap, r.max_rows, r.status, o.lo, o.n) || o.n == 0) return false;
    o.start = r.start[b];
    const int64_t room = static_cast<int64_t>(c.max_pages) * c.page_tokens;
    if (o.start < 0 || o.start + static_cast<int64_t>(o.n) > room) {
        if (threadIdx.x == 0) set_status(r.status, SPEC_STATUS_BAD_LENGTH);
        return false;
    }
    o.slot0 = (o.start / kTok + idx) * kTok;
    if (o.slot0 >= o.start + o.n) return false;
    o.first = max(o.start - o.slot0, 0);
    o.last = min(o.start + o.n - o.slot0, kTok);
    return true;
}

// Quantise 16 channels (spec_cache.h: s = e4m3(amax / (6 g)), code =
// e2m1(x / (s g)); IEEE divisions and round-to-nearest-even conversions, so
// the codes are those of the formula bit for bit).  Returns the scale byte;
// codes[i] holds channels 2i (low nibble) and 2i + 1.
__device__ __forceinline__ uint32_t quantise16(const float (&x)[16], float g, uint32_t (&codes)[8])
{
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
    const float t = fminf(__fdiv_rn(amax, 6.0f * g), 448.0f);
    uint16_t s8;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s8) : "f"(0.f), "f"(t));
    const float den = e4m3_value(s8) * g;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = den > 0.f ? __fdiv_rn(x[2 * i], den) : 0.f;
        const float b = den > 0.f ? __fdiv_rn(x[2 * i + 1], den) : 0.f;
        asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\t"
            "mov.b32 %0, {c, c, c, c};\n\t}"
            : "=r"(codes[i])
            : "f"(b), "f"(a));
        codes[i] &= 255u;
    }
    return s8 & 255u;
}

template <typename T>
__device__ __forceinline__ void load16(const T *p, bool aligned, float (&x)[16])
{
    if (aligned) {
        constexpr int N = 16 * sizeof(T) / 16;
        uint4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
        const T *e = reinterpret_cast<const T *>(v);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = to_f32<T>(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = to_f32<T>(p[i]);
    }
}

// One CTA per (block of 32 slots, kv head, request).  A block belongs to one
// CTA, so the value codes, two tokens to a byte, are read, merged and written
// back without atomics.
template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) append_kernel(const CacheView c, const CacheRows r)
{
    const int idx = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    BlockRows o;
    if (!block_rows(c, r, b, idx, o)) return;
    const int page = page_of(c, b, o.slot0);
    if (page < 0) {
        if (tid == 0) set_status(r.status, SPEC_STATUS_BAD_PAGE);
        return;
    }
    constexpr int G = D / 16;
    __shared__ uint8_t vcode[kTok][D];
    uint8_t *blk = block_at(c, page, h, o.slot0 % c.page_tokens / kTok);
    const float gk = c.k_scale ? c.k_scale[h] : 1.f, gv = c.v_scale ? c.v_scale[h] : 1.f;
    const int n = o.last - o.first;
    for (int i = tid; i < n * G * 2; i += kRowThreads) {
        const int g = i % G, t = o.first + i / G % n;
        const bool val = i >= n * G;
        const int64_t row = o.lo + (o.slot0 + t - o.start);
        const T *src = val ? static_cast<const T *>(r.v) + row * r.v_row + h * r.v_head
                           : static_cast<const T *>(r.k) + row * r.k_row + h * r.k_head;
        float x[16];
        uint32_t q[8];
        load16<T>(src + 16 * g, val ? r.v_aligned : r.k_aligned, x);
        const uint32_t s = quantise16(x, val ? gv : gk, q);
        const uint2 w = make_uint2(q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24,
                                   q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24);
        if (!val) {
            *reinterpret_cast<uint2 *>(blk + g / 2 * 512 + t * 16 + g % 2 * 8) = w;
            blk[k_scale_at(D) + t * G + g] = static_cast<uint8_t>(s);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                vcode[t][16 * g + 2 * j] = q[j] & 15u;
                vcode[t][16 * g + 2 * j + 1] = q[j] >> 4;
            }
            blk[v_scale_at(D) + g * kTok + t] = static_cast<uint8_t>(s);
        }
    }
    if (h == 0 && (r.score || r.slot_pos) && tid >= o.first && tid < o.last) {
        const int64_t at = static_cast<int64_t>(page) * c.page_tokens + o.slot0 % c.page_tokens + tid;
        if (r.score) r.score[at] = 0.f;
        if (r.slot_pos)
            r.slot_pos[at] = (r.pos0 ? r.pos0[b] : o.start) + (o.slot0 + tid - o.start);
    }
    __syncthreads();
    // 8 tokens of one channel per 32-bit word
    for (int i = tid; i < D * 4; i += kRowThreads) {
        const int d = i % D, t0 = i / D * 8;
        if (t0 + 8 <= o.first || t0 >= o.last) continue;
        uint32_t *p = reinterpret_cast<uint32_t *>(blk + v_codes_at(D) + d * 16 + t0 / 2);
        const bool whole = t0 >= o.first && t0 + 8 <= o.last;
        uint32_t w = whole ? 0u : *p;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (t0 + j >= o.first && t0 + j < o.last)
                w = (w & ~(15u << 4 * j)) | static_cast<uint32_t>(vcode[t0 + j][d]) << 4 * j;
        *p = w;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const CacheView c, const CacheRows r)
{
    const int idx = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    BlockRows o;
    if (!block_rows(c, r, b, idx, o)) return;
    const int page = page_of(c, b, o.slot0);
    if (page < 0 && tid == 0) set_status(r.status, SPEC_STATUS_BAD_PAGE);
    constexpr int G = D / 16;
    const uint8_t *blk = page < 0 ? nullptr : block_at(c, page, h, o.slot0 % c.page_tokens / kTok);
    const float gk = c.k_scale ? c.k_scale[h] : 1.f, gv = c.v_scale ? c.v_scale[h] : 1.f;
    const int n = o.last - o.first;
    for (int i = tid; i < n * D * 2; i += kRowThreads) {
        const int d = i % D, t = o.first + i / D % n;
        const bool val = i >= n * D;
        const int64_t row = o.lo + (o.slot0 + t - o.start);
        float x = 0.f;
        if (blk) {
            const uint32_t code = val ? blk[v_codes_at(D) + d * 16 + t / 2] >> (t % 2 * 4)
                                      : blk[d / 32 * 512 + t * 16 + d % 32 / 2] >> (d % 2 * 4);
            const uint32_t s = val ? blk[v_scale_at(D) + d / 16 * kTok + t]
                                   : blk[k_scale_at(D) + t * G + d / 16];
            x = e2m1_value(code) * e4m3_value(s) * (val ? gv : gk);
        }
        T *dst = val ? static_cast<T *>(r.v) + row * r.v_row + h * r.v_head
                     : static_cast<T *>(r.k) + row * r.k_row + h * r.k_head;
        dst[d] = from_f32<T>(x);
    }
}

// ------------------------------------------------------------- eviction ---

constexpr int kSelThreads = 1024;

// Order-preserving key of a score: NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t score_key(float x) { return x != x ? 0u : fkey(x); }

__device__ __forceinline__ float *score_at(const CacheView &c, const EvictParams &p, int b, int slot)
{
    const int64_t page = c.page_table[static_cast<int64_t>(b) * c.max_pages + slot / c.page_tokens];
    return p.score + page * c.page_tokens + slot % c.page_tokens;
}

// exclusive scan of one value per thread over the CTA, and the total
__device__ __forceinline__ int cta_scan(int v, int *warp_sum, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int s = lane < kSelThreads / 32 ? warp_sum[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += y;
    }
    total = __shfl_sync(0xFFFFFFFFu, s, 31);
    const int before = __shfl_sync(0xFFFFFFFFu, s, max(warp - 1, 0));
    return (warp ? before : 0) + incl - v;
}

// Selection: one CTA per request.  A radix search over the score keys (8 bits
// a pass) finds the key of the last score kept, then an ordered scan lists the
// kept slots: those above the key, the first few at it, and the newest.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const CacheView c, const EvictParams p)
{
    const int b = blockIdx.x, tid = threadIdx.x;
    __shared__ int hist[256], warp_sum[kSelThreads / 32], pick[2];
    const int len = p.len[b];
    int32_t *kept = p.kept + static_cast<int64_t>(b) * p.budget;
    const int64_t room = static_cast<int64_t>(c.max_pages) * c.page_tokens;
    uint32_t bad = (len < 0 || len > room) ? SPEC_STATUS_BAD_LENGTH : 0u;
    const int keep = min(len, p.budget);
    if (!bad) {
        int bad_page = 0;
        for (int i = tid; i < (len + c.page_tokens - 1) / c.page_tokens; i += kSelThreads)
            bad_page |= page_of(c, b, i * c.page_tokens) < 0;
        for (int i = tid; i < (keep + c.page_tokens - 1) / c.page_tokens; i += kSelThreads) {
            const int pg = p.dst_table[static_cast<int64_t>(b) * p.dst_pages + i];
            bad_page |= pg < 0 || pg >= c.n_pages;
        }
        if (__syncthreads_or(bad_page)) bad = SPEC_STATUS_BAD_PAGE;
    }
    if (bad) {
        if (tid == 0) {
            set_status(p.status, bad);
            p.new_len[b] = -1;
        }
        for (int i = tid; i < p.budget; i += kSelThreads) kept[i] = -1;
        return;
    }
    if (tid == 0) p.new_len[b] = keep;
    for (int i = keep + tid; i < p.budget; i += kSelThreads) kept[i] = -1;
    if (len <= p.budget) {
        for (int i = tid; i < len; i += kSelThreads) kept[i] = i;
        return;
    }
    const int old = len - p.recent;          // slots that compete for `want` places
    int want = p.budget - p.recent;
    uint32_t key = 0u;
    for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < old; i += kSelThreads) {
            const uint32_t k = score_key(*score_at(c, p, b, i));
            if (shift == 24 || (k >> (shift + 8)) == (key >> (shift + 8)))
                atomicAdd(&hist[(k >> shift) & 255u], 1);
        }
        __syncthreads();
        // the digit where the count from the top reaches `want`
        int total;
        const int mine = tid < 256 ? hist[255 - tid] : 0;
        const int above = cta_scan(mine, warp_sum, total);
        if (above < want && above + mine >= want) {
            pick[0] = 255 - tid;
            pick[1] = want - above;
        }
        __syncthreads();
        key |= static_cast<uint32_t>(pick[0]) << shift;
        want = pick[1];
        __syncthreads();
    }
    // `want` of the slots whose key equals `key` are kept, the lowest ones
    int out = 0, ties = 0;
    const bool any = p.budget > p.recent;
    for (int base = 0; base < len; base += kSelThreads) {
        const int i = base + tid;
        uint32_t k = 0u;
        if (i < old) k = score_key(*score_at(c, p, b, i));
        const int tie = any && i < old && k == key;
        int n_tie, n_out;
        const int t = ties + cta_scan(tie, warp_sum, n_tie);
        const int take = i < len && (i >= old || (any && (k > key || (tie && t < want))));
        const int at = out + cta_scan(take, warp_sum, n_out);
        if (take) kept[at] = i;
        ties += n_tie;
        out += n_out;
    }
}

constexpr int kMoveThreads = 128;

// Move: one CTA per (destination block, kv head, request).
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const CacheView c, const EvictParams p)
{
    const int blk = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int keep = p.new_len[b];
    if (blk * kTok >= keep) return;          // also a skipped request (-1)
    const int D = c.D, G = D / 16;
    __shared__ const uint8_t *src[kTok];     // source block of each token
    __shared__ int tok[kTok];
    const int32_t *kept = p.kept + static_cast<int64_t>(b) * p.budget;
    const int dpage = p.dst_table[static_cast<int64_t>(b) * p.dst_pages + blk * kTok / c.page_tokens];
    uint8_t *dst = block_at(c, dpage, h, blk * kTok % c.page_tokens / kTok);
    if (tid < kTok) {
        const int i = blk * kTok + tid;
        src[tid] = nullptr;
        tok[tid] = 0;
        float sc = 0.f;
        int pos = 0;
        if (i < keep) {
            const int slot = kept[i];
            const int page = page_of(c, b, slot), off = slot % c.page_tokens;
            src[tid] = block_at(c, page, h, off / kTok);
            tok[tid] = off % kTok;
            if (h == 0) {
                const int64_t at = static_cast<int64_t>(page) * c.page_tokens + off;
                sc = p.score[at];
                pos = p.slot_pos ? p.slot_pos[at] : 0;
            }
        }
        if (h == 0) {
            const int64_t at = static_cast<int64_t>(dpage) * c.page_tokens + i % c.page_tokens;
            p.score[at] = sc;
            if (p.slot_pos) p.slot_pos[at] = pos;
        }
    }
    __syncthreads();
    for (int i = tid; i < D; i += kMoveThreads) {          // 16 bytes of K codes each
        const int ch = i / kTok, t = i % kTok;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (src[t]) v = *reinterpret_cast<const uint4 *>(src[t] + ch * 512 + tok[t] * 16);
        *reinterpret_cast<uint4 *>(dst + ch * 512 + t * 16) = v;
    }
    for (int i = tid; i < kTok * G; i += kMoveThreads) {
        const int t = i / G, g = i % G;
        dst[k_scale_at(D) + i] = src[t] ? src[t][k_scale_at(D) + tok[t] * G + g] : 0;
        const int u = i % kTok, w = i / kTok;
        dst[v_scale_at(D) + i] = src[u] ? src[u][v_scale_at(D) + w * kTok + tok[u]] : 0;
    }
    for (int i = tid; i < D * 4; i += kMoveThreads) {      // 8 tokens of a channel
        const int d = i % D, t0 = i / D * 8;
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int t = t0 + j;
            if (src[t])
                w |= static_cast<uint32_t>(src[t][v_codes_at(D) + d * 16 + tok[t] / 2] >> (tok[t] % 2 * 4) & 15)
                     << 4 * j;
        }
        *reinterpret_cast<uint32_t *>(dst + v_codes_at(D) + d * 16 + t0 / 2) = w;
    }
}

template <typename T>
cudaError_t launch_rows(const CacheView &c, const CacheRows &r, bool append, cudaStream_t s)
{
    // a request's rows touch at most this many blocks, wherever they start
    const dim3 grid((r.max_rows + kTok - 2) / kTok + 1, c.H, c.B);
    switch (c.D) {
    case 64:
        if (append) append_kernel<T, 64><<<grid, kRowThreads, 0, s>>>(c, r);
        else read_kernel<T, 64><<<grid, kRowThreads, 0, s>>>(c, r);
        break;
    case 128:
        if (append) append_kernel<T, 128><<<grid, kRowThreads, 0, s>>>(c, r);
        else read_kernel<T, 128><<<grid, kRowThreads, 0, s>>>(c, r);
        break;
    default:
        if (append) append_kernel<T, 256><<<grid, kRowThreads, 0, s>>>(c, r);
        else read_kernel<T, 256><<<grid, kRowThreads, 0, s>>>(c, r);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_rows(const CacheView &c, const CacheRows &r, int dtype, bool append, cudaStream_t s)
{
    return dtype == SPEC_BF16 ? launch_rows<__nv_bfloat16>(c, r, append, s) : launch_rows<float>(c, r, append, s);
}

cudaError_t launch_cache_evict(const CacheView &c, const EvictParams &p, cudaStream_t s)
{
    evict_select_kernel<<<c.B, kSelThreads, 0, s>>>(c, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t most = static_cast<int64_t>(c.max_pages) * c.page_tokens;
    const int64_t keep = most < p.budget ? most : p.budget;
    const dim3 grid(static_cast<unsigned>((keep + kTok - 1) / kTok), c.H, c.B);
    evict_move_kernel<<<grid, kMoveThreads, 0, s>>>(c, p);
    return cudaGetLastError();
}

}  // namespace specv
