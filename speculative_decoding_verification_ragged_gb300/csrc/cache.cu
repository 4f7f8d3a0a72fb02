// cache.cu -- the 4-bit paged cache itself: append (quantise and write), read,
// and eviction by accumulated attention weight (include/spec_cache.h).
#include <climits>
#include <cooperative_groups.h>

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
    if (!request_rows(r.cu_rows, b, r.R_cap, r.max_rows, threadIdx.x == 0 ? r.status : nullptr, o.lo, o.n) || o.n == 0)
        return false;
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

// A thread's share of a row: 16 bytes of values (4 of fp32, 8 of bf16), so that
// a warp's loads are whole lines; LPG lanes share a group of 16 channels.
template <typename T> struct Share {
    static constexpr int N = 16 / sizeof(T), LPG = 16 / N;
};

template <typename T>
__device__ __forceinline__ void load_share(const T *p, bool aligned, float (&x)[Share<T>::N])
{
    __align__(16) T e[Share<T>::N];
    if (aligned) {
        *reinterpret_cast<uint4 *>(e) = __ldg(reinterpret_cast<const uint4 *>(p));
    } else {
#pragma unroll
        for (int i = 0; i < Share<T>::N; ++i) e[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < Share<T>::N; ++i) x[i] = to_f32<T>(e[i]);
}

// Quantise a share (spec_cache.h: s = e4m3(amax / (6 g)), code = e2m1(x / (s g));
// IEEE divisions and round-to-nearest-even conversions, so the codes are those of
// the formula bit for bit).  Returns the group's scale byte; the share's codes
// come packed, the first in the lowest nibble.
template <int N, int LPG>
__device__ __forceinline__ uint32_t quantise(const float (&x)[N], float g, uint32_t &codes)
{
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int o = 1; o < LPG; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    const float t = fminf(__fdiv_rn(amax, 6.0f * g), 448.0f);
    uint16_t s8;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s8) : "f"(0.f), "f"(t));
    const float den = e4m3_value(s8) * g;
    codes = 0;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float a = den > 0.f ? __fdiv_rn(x[i], den) : 0.f;
        const float b = den > 0.f ? __fdiv_rn(x[i + 1], den) : 0.f;
        uint32_t c;
        asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\tmov.b32 %0, {c, c, c, c};\n\t}"
            : "=r"(c)
            : "f"(b), "f"(a));
        codes |= (c & 255u) << (4 * i);
    }
    return s8 & 255u;
}

// One CTA per (block of 32 slots, kv head, request).  A block belongs to one
// CTA, so the value codes, two tokens to a byte, are read, merged and written
// back without atomics.  A warp reads 512 bytes of a row's values per load; bound by
// the instructions of the quantisation, about 1500 a warp and block: 27 k fp32 rows
// of 8 heads of 64 take 62 us (1.8 TB/s of rows), and 95 with the read of them all.
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
    constexpr int G = D / 16, N = Share<T>::N, LPG = Share<T>::LPG, PER = D / N;
    // value codes, a channel's 8 tokens to a word once transposed; a row of words
    // is padded so that the lanes of a column lie in different banks
    __shared__ uint32_t vcode[kTok][D / 8 + 1];
    uint8_t *blk = block_at(c, page, h, o.slot0 % c.page_tokens / kTok);
    const float gk = c.k_scale ? c.k_scale[h] : 1.f, gv = c.v_scale ? c.v_scale[h] : 1.f;
    const int n = o.last - o.first;
    // keys, then values: whole groups of lanes take part (PER divides the warp or
    // is a multiple of it), so the shuffles of quantise() are complete
#pragma unroll
    for (int val = 0; val < 2; ++val) {
        const T *base = val ? static_cast<const T *>(r.v) + h * r.v_head : static_cast<const T *>(r.k) + h * r.k_head;
        const int64_t stride = val ? r.v_row : r.k_row;
        const bool aligned = val ? r.v_aligned : r.k_aligned;
        for (int i0 = 0; i0 < n * PER; i0 += kRowThreads) {
            const int i = i0 + tid, t = o.first + i / PER, d = i % PER * N;
            const bool in = i < n * PER;
            float x[N] = {};
            uint32_t codes;
            if (in) load_share<T>(base + (o.lo + (o.slot0 + t - o.start)) * stride + d, aligned, x);
            const uint32_t s = quantise<N, LPG>(x, val ? gv : gk, codes);
            if (!in) continue;
            const bool lead = d % 16 == 0;
            if (!val) {
                uint8_t *at = blk + d / 32 * 512 + t * 16 + d % 32 / 2;
                if (N == 8) *reinterpret_cast<uint32_t *>(at) = codes;
                else *reinterpret_cast<uint16_t *>(at) = static_cast<uint16_t>(codes);
                if (lead) blk[k_scale_at(D) + t * G + d / 16] = static_cast<uint8_t>(s);
            } else {
                uint8_t *at = reinterpret_cast<uint8_t *>(vcode[t]) + d / 2;
                if (N == 8) *reinterpret_cast<uint32_t *>(at) = codes;
                else *reinterpret_cast<uint16_t *>(at) = static_cast<uint16_t>(codes);
                if (lead) blk[v_scale_at(D) + d / 16 * kTok + t] = static_cast<uint8_t>(s);
            }
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
        const int d = i / 4, t0 = i % 4 * 8;
        if (t0 + 8 <= o.first || t0 >= o.last) continue;
        uint32_t *p = reinterpret_cast<uint32_t *>(blk + v_codes_at(D) + d * 16 + t0 / 2);
        const bool whole = t0 >= o.first && t0 + 8 <= o.last;
        uint32_t w = whole ? 0u : *p;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (whole || (t0 + j >= o.first && t0 + j < o.last))
                w = (w & ~(15u << 4 * j)) | (vcode[t0 + j][d / 8] >> (d % 8 * 4) & 15u) << 4 * j;
        *p = w;
    }
}

// x * g rounded once to T (x: a code times its scale, exact).  For bf16 the product is
// first rounded to odd -- of the two floats around it the one whose last bit is set,
// itself where it is one -- which keeps the second rounding from a tie that is none.
// Without head scales (SCALED: there are, and T is bf16) g is 1 and nothing is lost: 27 k rows of 8
// heads of 128 read in 39 us, with them in 43.
template <typename T, bool SCALED> __device__ __forceinline__ T scaled_value(float x, float g)
{
    if constexpr (SCALED) {
        const float below = __fmul_rd(x, g), above = __fmul_ru(x, g);
        return from_f32<T>((__float_as_uint(below) & 1u) ? below : above);
    } else {
        return from_f32<T>(x * g);
    }
}

// One CTA per (block, kv head, request): a thread takes 8 channels of a token's
// key, then a channel (or two, of bf16) of every token's value, so that both
// sides move whole words.
template <typename T, int D, bool SCALED>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const CacheView c, const CacheRows r)
{
    const int idx = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    BlockRows o;
    if (!block_rows(c, r, b, idx, o)) return;
    const int page = page_of(c, b, o.slot0);
    if (page < 0 && tid == 0) set_status(r.status, SPEC_STATUS_BAD_PAGE);
    constexpr int G = D / 16, N = Share<T>::N, PER = D / N, CH = 4 / sizeof(T);
    const uint8_t *blk = page < 0 ? nullptr : block_at(c, page, h, o.slot0 % c.page_tokens / kTok);
    const float gk = c.k_scale ? c.k_scale[h] : 1.f, gv = c.v_scale ? c.v_scale[h] : 1.f;
    const int n = o.last - o.first;
    const int64_t row0 = o.lo + (o.slot0 + o.first - o.start);
    T *kp = static_cast<T *>(r.k) + row0 * r.k_row + h * r.k_head, *vp = static_cast<T *>(r.v) + row0 * r.v_row + h * r.v_head;
    for (int i = tid; i < n * PER; i += kRowThreads) {
        const int t = o.first + i / PER, d = i % PER * N;
        uint32_t w = 0;
        float s = 0.f;
        if (blk) {
            const uint8_t *at = blk + d / 32 * 512 + t * 16 + d % 32 / 2;
            w = N == 8 ? *reinterpret_cast<const uint32_t *>(at) : *reinterpret_cast<const uint16_t *>(at);
            s = e4m3_value(blk[k_scale_at(D) + t * G + d / 16]);
        }
        __align__(16) T e[N];
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 x = h2_float2(e2m1x2(w >> (4 * j)));
            e[j] = scaled_value<T, SCALED>(x.x * s, gk);
            e[j + 1] = scaled_value<T, SCALED>(x.y * s, gk);
        }
        T *to = kp + (t - o.first) * r.k_row + d;
        if (r.k_aligned) {
            *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(e);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) to[j] = e[j];
        }
    }
    for (int d = tid * CH; d < D; d += kRowThreads * CH) {
        uint4 v[CH], s[2];
#pragma unroll
        for (int k = 0; k < CH; ++k)
            v[k] = blk ? *reinterpret_cast<const uint4 *>(blk + v_codes_at(D) + (d + k) * 16) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 2; ++k)
            s[k] = blk ? *reinterpret_cast<const uint4 *>(blk + v_scale_at(D) + d / 16 * kTok + 16 * k) : make_uint4(0, 0, 0, 0);
        const uint32_t sw[8] = {s[0].x, s[0].y, s[0].z, s[0].w, s[1].x, s[1].y, s[1].z, s[1].w};
#pragma unroll
        for (int t = 0; t < kTok; t += 2) {
            const float2 sc = h2_float2(e4m3x2(sw[t / 4] >> (t % 4 * 8)));
            __align__(4) T e[2][CH];
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                const uint32_t w = t < 16 ? (t < 8 ? v[k].x : v[k].y) : (t < 24 ? v[k].z : v[k].w);
                const float2 x = h2_float2(e2m1x2(w >> (t % 8 * 4)));
                e[0][k] = scaled_value<T, SCALED>(x.x * sc.x, gv);
                e[1][k] = scaled_value<T, SCALED>(x.y * sc.y, gv);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (t + u >= o.first && t + u < o.last) {
                    T *to = vp + (t + u - o.first) * r.v_row + d;
                    if (CH == 1 || r.v_aligned) {
                        *reinterpret_cast<uint32_t *>(to) = *reinterpret_cast<const uint32_t *>(e[u]);
                    } else {
                        to[0] = e[u][0];
                        to[CH - 1] = e[u][CH - 1];
                    }
                }
        }
    }
}

// ------------------------------------------------------------- eviction ---

constexpr int kSelThreads = 1024;
constexpr int kSelCtas = 8;                // CTAs of a request's cluster at most
constexpr int kBins = 2048;                // a radix digit: 11 bits (the last: 10)
constexpr int kSelStaged = 40 * 1024;      // scores a CTA keeps in shared memory
constexpr int kRun = 16;                   // a warp's blocks of 32 slots are a multiple of this

// slots of a CTA's slice where a cluster of `ctas` shares `len`
__host__ __device__ inline int64_t sel_slice(int64_t len, int ctas)
{
    const int64_t per = static_cast<int64_t>(ctas) * kSelThreads;
    return ((len + per - 1) / per + kRun - 1) / kRun * kRun * kSelThreads;
}

// Order-preserving key of a score: NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t score_key(float x) { return x != x ? 0u : fkey(x); }

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
    int s = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += y;
    }
    total = __shfl_sync(0xFFFFFFFFu, s, 31);
    const int before = __shfl_sync(0xFFFFFFFFu, s, max(warp - 1, 0));
    return (warp ? before : 0) + incl - v;
}

// Selection: a cluster of 1, 2, 4 or 8 CTAs per request (one for every 16384
// slots: a pass costs a cluster 2 barriers and the reading of its histograms, 4 us
// in all), each with a contiguous part of the slots, its keys in shared memory
// (read again from the cache's scores where they do not fit).  A radix search, 11
// bits a pass over the cluster's summed histograms, finds the key of the last score
// kept; then a warp lists the kept slots of a contiguous run of its own by ballots:
// those above the key, the first few at it, and the newest.  2 x 131072 scores: 25 us
// (39 with a page looked up and a load waited for slot by slot, and a run a thread);
// 32 x 4096: 16 us (a cluster of 8 for each, at that step: 41).
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const CacheView c, const EvictParams p)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint32_t *keys = reinterpret_cast<uint32_t *>(smem_raw);
    __shared__ int hist[kBins], warp_sum[kSelThreads / 32], warp_over[kSelThreads / 32], pick[2], count[2];
    const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int b = blockIdx.x / ctas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    // (the same in every CTA of the cluster: none is left waiting)
    const int all = ctas * kSelThreads, me = rank * kSelThreads + tid;
    // (new_len can be len: written when the cluster has read it)
    if (bad) {
        cluster.sync();
        if (me == 0) {
            set_status(p.status, bad);
            p.new_len[b] = -1;
        }
        for (int i = me; i < p.budget; i += all) kept[i] = -1;
        return;
    }
    for (int i = keep + me; i < p.budget; i += all) kept[i] = -1;
    if (len <= p.budget) {
        cluster.sync();
        if (me == 0) p.new_len[b] = keep;
        for (int i = me; i < len; i += all) kept[i] = i;
        return;
    }

    const int old = len - p.recent;          // slots that compete for `want` places
    int want = p.budget - p.recent;
    const int slice = static_cast<int>(sel_slice(len, ctas)), run = slice / kSelThreads * 32;   // a run per warp
    const int64_t first = static_cast<int64_t>(rank) * slice;
    const bool staged = slice <= kSelStaged;
    // where the scores of a slot of this slice lie (one that competes)
    const auto score_at = [&](int i) {
        const int s = static_cast<int>(first) + i, page = s / c.page_tokens;
        const int64_t id = __ldg(c.page_table + static_cast<int64_t>(b) * c.max_pages + page);
        return id * c.page_tokens + (s - page * c.page_tokens);
    };
    const int mine = first >= old ? 0 : static_cast<int>(min(static_cast<int64_t>(slice), old - first));
    if (staged) {
        // a warp's loads are blocks of 32 slots, 16 in flight: lane u looks up the
        // page of the u-th (a block lies within a page; for one past the end, the
        // first block of the cache is loaded and not looked at)
        for (int i0 = 0; i0 < mine; i0 += kSelThreads * kRun) {
            const int i = i0 + warp * 32, look = i + lane % kRun * kSelThreads;
            const int64_t at = look < mine ? score_at(look) : 0;
            float x[kRun];            // (no condition: a warp does not wait for one load at a time)
#pragma unroll
            for (int u = 0; u < kRun; ++u) x[u] = p.score[__shfl_sync(0xFFFFFFFFu, at, u) + lane];
#pragma unroll
            for (int u = 0; u < kRun; ++u)
                if (i + u * kSelThreads + lane < mine) keys[i + u * kSelThreads + lane] = score_key(x[u]);
        }
    }
    // (a body for each of the two, so that no look-up is in the loops over keys[])
    const auto select = [&](auto key_at) {
        uint32_t key = 0u;
        const bool any = want > 0;
        for (int pass = 0; pass < 3 && any; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : kBins;
            for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < mine; i += kSelThreads) {
                const uint32_t k = key_at(i);
                if (pass == 0 || (k >> (pass == 1 ? 21 : 10)) == (key >> (pass == 1 ? 21 : 10)))
                    atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
            }
            cluster.sync();
            // bins from the top, two a thread, summed over the cluster
            int two[2] = {0, 0};
            const int at = bins - 2 - 2 * tid;
    #pragma unroll
            for (int r = 0; r < kSelCtas; ++r) {
                if (r < ctas && at >= 0) {
                    const int *h = cluster.map_shared_rank(hist, r);
                    const int2 x = *reinterpret_cast<const int2 *>(h + at);
                    two[0] += x.y;
                    two[1] += x.x;
                }
            }
            int total;
            int above = cta_scan(two[0] + two[1], warp_sum, total);
    #pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (above < want && above + two[u] >= want) {
                    pick[0] = bins - 1 - 2 * tid - u;
                    pick[1] = want - above;
                }
                above += two[u];
            }
            cluster.sync();                       // (also the CTA's barrier for `pick`)
            key |= static_cast<uint32_t>(pick[0]) << shift;
            want = pick[1];
            __syncthreads();
        }
        // `want` of the slots whose key equals `key` are kept, the lowest ones: count
        // ties and slots above the key in this warp's run, then in the warps and the
        // CTAs before
        const int r0 = min(warp * run, mine), r1 = any ? min(r0 + run, mine) : r0;
        int ties = 0, over = 0;
    #pragma unroll 4
        for (int i = r0; i < r1; i += 32) {
            const bool real = i + lane < r1;
            const uint32_t k = real ? key_at(i + lane) : 0u;
            ties += __popc(__ballot_sync(0xFFFFFFFFu, real && k == key));
            over += __popc(__ballot_sync(0xFFFFFFFFu, k > key));
        }
        if (lane == 0) {
            warp_sum[warp] = ties;
            warp_over[warp] = over;
        }
        __syncthreads();
        int n_ties = warp_sum[lane], n_over = warp_over[lane];
    #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xFFFFFFFFu, n_ties, o), v = __shfl_up_sync(0xFFFFFFFFu, n_over, o);
            if (lane >= o) {
                n_ties += t;
                n_over += v;
            }
        }
        int tie_rank = __shfl_sync(0xFFFFFFFFu, n_ties, warp) - ties;
        int over_rank = __shfl_sync(0xFFFFFFFFu, n_over, warp) - over;
        n_ties = __shfl_sync(0xFFFFFFFFu, n_ties, 31);
        n_over = __shfl_sync(0xFFFFFFFFu, n_over, 31);
        if (tid == 0) {
            count[0] = n_ties;
            count[1] = n_over;
        }
        cluster.sync();
        for (int r = 0; r < rank; ++r) {
            const int *cnt = cluster.map_shared_rank(count, r);
            tie_rank += cnt[0];
            over_rank += cnt[1];
        }
        cluster.sync();                           // no CTA leaves while its counts are read
        int at = over_rank + min(tie_rank, want);
        const uint32_t below = (1u << lane) - 1u;
    #pragma unroll 4
        for (int i = r0; i < r1; i += 32) {
            const bool real = i + lane < r1;
            const uint32_t k = real ? key_at(i + lane) : 0u;
            const uint32_t tie = __ballot_sync(0xFFFFFFFFu, real && k == key);
            const bool stays = k > key || ((tie >> lane & 1u) && tie_rank + __popc(tie & below) < want);
            const uint32_t stay = __ballot_sync(0xFFFFFFFFu, stays);
            if (stays) kept[at + __popc(stay & below)] = static_cast<int>(first) + i + lane;
            at += __popc(stay);
            tie_rank += __popc(tie);
        }
    };
    if (staged)
        select([&](int i) { return keys[i]; });
    else
        select([&](int i) { return score_key(p.score[score_at(i)]); });
    for (int i = me; i < p.recent; i += all) kept[keep - p.recent + i] = old + i;
    if (me == 0) p.new_len[b] = keep;
}

constexpr int kMoveThreads = 128;
constexpr int kWord = 1 << 16, kBlock = 1 << 17, kNone = 1 << 18;

// Move: one CTA per (destination block, kv head, request).  Keys go 16 bytes (32
// channels) a thread.  A thread takes the values of a channel: 16 bytes of a
// source block hold its 32 tokens there, read once for all the kept ones, which
// are shifted out one by one.  32 x 2048 of 4096 tokens, 8 heads of 128: 39 us (a
// word chosen and a shift for each code by itself: 47); 2 x 32768 of 131072: 65 us, 5.3 TB/s of the sectors they lie in.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const CacheView c, const EvictParams p)
{
    const int blk = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int keep = p.new_len[b];
    if (blk * kTok >= keep) return;          // also a skipped request (-1)
    constexpr int G = D / 16;
    __shared__ const uint8_t *src[kTok];     // source block of each token
    __shared__ int tok[kTok];                // its place there, -1: none
    __shared__ int step[kTok];               // how the values get to it (below)
    const int32_t *kept = p.kept + static_cast<int64_t>(b) * p.budget;
    const int dpage = p.dst_table[static_cast<int64_t>(b) * p.dst_pages + blk * kTok / c.page_tokens];
    uint8_t *dst = block_at(c, dpage, h, blk * kTok % c.page_tokens / kTok);
    if (tid < kTok) {
        const int i = blk * kTok + tid;
        src[tid] = nullptr;
        tok[tid] = -1;
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
        // shift of the token's code in its word, the word, and whether the word or
        // the block is another than the token's before
        __syncwarp();
        const int t = tok[tid], last = tid ? tok[tid - 1] : -1;
        const bool block = t >= 0 && (last < 0 || src[tid] != src[tid - 1]);
        const bool word = block || (t >= 0 && t / 8 != last / 8);
        step[tid] = t < 0 ? kNone : t % 8 * 4 | t / 8 << 8 | (word ? kWord : 0) | (block ? kBlock : 0);
        if (h == 0) {
            const int64_t at = static_cast<int64_t>(dpage) * c.page_tokens + i % c.page_tokens;
            p.score[at] = sc;
            if (p.slot_pos) p.slot_pos[at] = pos;
        }
    }
    __syncthreads();
    const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = tid; i < D; i += kMoveThreads) {          // 16 bytes of K codes each
        const int ch = i / kTok, t = i % kTok;
        const uint4 v = tok[t] >= 0 ? __ldg(reinterpret_cast<const uint4 *>(src[t] + ch * 512 + tok[t] * 16)) : none;
        *reinterpret_cast<uint4 *>(dst + ch * 512 + t * 16) = v;
    }
    if (tid < kTok) {                                      // a token's K scales
#pragma unroll
        for (int g = 0; g < G; g += 4)
            *reinterpret_cast<uint32_t *>(dst + k_scale_at(D) + tid * G + g) =
                tok[tid] >= 0 ? __ldg(reinterpret_cast<const uint32_t *>(src[tid] + k_scale_at(D) + tok[tid] * G + g)) : 0u;
    }
#pragma unroll
    for (int i = tid; i < kTok * G; i += kMoveThreads) {   // V scales
        const int u = i % kTok, w = i / kTok;
        dst[v_scale_at(D) + i] = tok[u] >= 0 ? __ldg(src[u] + v_scale_at(D) + w * kTok + tok[u]) : 0;
    }
    for (int d = tid; d < D; d += kMoveThreads) {
        uint32_t out[4], word = 0;
        uint4 v = none;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t w = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int st = step[8 * q + j];            // (uniform, as the branches)
                if (st & kBlock)
                    v = __ldg(reinterpret_cast<const uint4 *>(src[8 * q + j] + v_codes_at(D) + d * 16));
                if (st & kWord) word = (st & 0x200) ? ((st & 0x100) ? v.w : v.z) : ((st & 0x100) ? v.y : v.x);
                if (st & kNone) word = 0;
                // the code enters at the top while the ones before move down
                w = __funnelshift_r(w, word >> (st & 31), 4);
            }
            out[q] = w;
        }
        *reinterpret_cast<uint4 *>(dst + v_codes_at(D) + d * 16) = make_uint4(out[0], out[1], out[2], out[3]);
    }
}

template <typename T, int D>
void launch_rows(const CacheView &c, const CacheRows &r, bool append, cudaStream_t s)
{
    constexpr bool kTwice = sizeof(T) == 2;       // a product that takes two roundings to T
    // a request's rows touch at most this many blocks, wherever they start
    const dim3 grid((r.max_rows + kTok - 2) / kTok + 1, c.H, c.B);
    if (append) append_kernel<T, D><<<grid, kRowThreads, 0, s>>>(c, r);
    else if (kTwice && (c.k_scale || c.v_scale)) read_kernel<T, D, kTwice><<<grid, kRowThreads, 0, s>>>(c, r);
    else read_kernel<T, D, false><<<grid, kRowThreads, 0, s>>>(c, r);
}

template <typename T>
cudaError_t launch_rows(const CacheView &c, const CacheRows &r, bool append, cudaStream_t s)
{
    if (c.D == 64) launch_rows<T, 64>(c, r, append, s);
    else if (c.D == 128) launch_rows<T, 128>(c, r, append, s);
    else launch_rows<T, 256>(c, r, append, s);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_rows(const CacheView &c, const CacheRows &r, int dtype, bool append, cudaStream_t s)
{
    return dtype == SPEC_BF16 ? launch_rows<__nv_bfloat16>(c, r, append, s) : launch_rows<float>(c, r, append, s);
}

cudaError_t launch_cache_evict(const CacheView &c, const EvictParams &p, cudaStream_t s)
{
    static bool done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev]) {
        e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSelStaged * 4);
        if (e != cudaSuccess) return e;
        done[dev] = true;
    }
    const int64_t room = static_cast<int64_t>(c.max_pages) * c.page_tokens;
    int ctas = 1;
    while (ctas < kSelCtas && sel_slice(room, ctas) > kRun * kSelThreads) ctas *= 2;
    int64_t slice = sel_slice(room, ctas);
    if (slice > kSelStaged) slice = kSelStaged;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c.B * ctas, 1, 1);
    cfg.blockDim = dim3(kSelThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(slice) * 4;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, c, p);
    if (e != cudaSuccess) return e;
    const int64_t most = static_cast<int64_t>(c.max_pages) * c.page_tokens;
    const int64_t keep = most < p.budget ? most : p.budget;
    const dim3 grid(static_cast<unsigned>((keep + kTok - 1) / kTok), c.H, c.B);
    if (c.D == 64) evict_move_kernel<64><<<grid, kMoveThreads, 0, s>>>(c, p);
    else if (c.D == 128) evict_move_kernel<128><<<grid, kMoveThreads, 0, s>>>(c, p);
    else evict_move_kernel<256><<<grid, kMoveThreads, 0, s>>>(c, p);
    return cudaGetLastError();
}

}  // namespace specv
