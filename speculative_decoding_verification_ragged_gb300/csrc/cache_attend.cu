// cache_attend.cu -- attention of packed verify rows over the 4-bit paged cache,
// and the accumulation of the weights its tokens get (include/spec_cache.h).
#include <climits>

#include "cache.cuh"

namespace specv {

namespace {

constexpr int kAttnThreads = 128;

// s as a function of q.k: the cap and the distance bias
__device__ __forceinline__ float score_of(const AttnParams &p, float dot, float slope, int dist)
{
    float s = dot * p.scale;
    if (p.cap > 0.f) s = p.cap * tanhf(s / p.cap);
    return s - slope * static_cast<float>(dist);
}

__device__ __forceinline__ int slot_position(const CacheView &c, const AttnParams &p, int b, int slot)
{
    if (!p.slot_pos) return slot;
    const int page = page_of(c, b, slot);
    return page < 0 ? 0 : p.slot_pos[static_cast<int64_t>(page) * c.page_tokens + slot % c.page_tokens];
}

template <typename T>
__device__ __forceinline__ float dot_key(const uint8_t *blk, int t, int D, const float *q)
{
    float a = 0.f;
    for (int g = 0; g < D / 16; ++g) {
        float part = 0.f;
        for (int j = 0; j < 8; ++j) {
            const float2 x = h2_float2(e2m1x2(blk[g / 2 * 512 + t * 16 + g % 2 * 8 + j]));
            part += x.x * q[16 * g + 2 * j] + x.y * q[16 * g + 2 * j + 1];
        }
        a += part * e4m3_value(blk[k_scale_at(D) + t * (D / 16) + g]);
    }
    return a;
}

// One CTA per (row, query head): tiles of 128 tokens, a thread per token for
// the scores and a thread per channel for the values.
template <typename T>
__global__ void __launch_bounds__(kAttnThreads) attend_kernel(const CacheView c, const AttnParams p)
{
    const int h = blockIdx.x, j = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    int lo, n;
    if (!request_rows(p.cu_rows, b, p.R_cap, p.k_max + 1, p.status, lo, n) || j >= n) return;
    const int D = c.D, hk = h / (p.Hq / c.H);
    int len = p.len[b];
    if (len < 0 || len > p.max_len) {
        if (tid == 0) set_status(p.status, SPEC_STATUS_BAD_LENGTH);
        len = 0;
    }
    __shared__ float q[256], w[kAttnThreads], red[kAttnThreads];
    const T *qp = static_cast<const T *>(p.q) + (lo + j) * p.q_row + h * p.q_head;
    for (int d = tid; d < D; d += kAttnThreads) q[d] = to_f32<T>(qp[d]);
    __syncthreads();
    const float gk = c.k_scale ? c.k_scale[hk] : 1.f, gv = c.v_scale ? c.v_scale[hk] : 1.f;
    const float slope = p.slopes ? p.slopes[h] : 0.f;
    const int own = len > 0 ? len - n + j : -1;
    const int pos = own >= 0 ? slot_position(c, p, b, own) : 0;
    float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
    for (int base = 0; base <= own; base += kAttnThreads) {
        const int t = base + tid;
        float s = -INFINITY;
        if (t <= own) {
            const int page = page_of(c, b, t);
            const int dist = pos - slot_position(c, p, b, t);
            if (page < 0) set_status(p.status, SPEC_STATUS_BAD_PAGE);
            else if (p.window <= 0 || dist < p.window || t < p.prefix)
                s = score_of(p, gk * dot_key<T>(block_at(c, page, hk, t % c.page_tokens / kTok), t % kTok, D, q),
                             slope, dist);
        }
        red[tid] = s;
        __syncthreads();
        float mt = m;
        for (int i = 0; i < kAttnThreads; ++i) mt = fmaxf(mt, red[i]);
        __syncthreads();
        w[tid] = s == -INFINITY ? 0.f : __expf(s - mt);
        __syncthreads();
        const float f = m == -INFINITY ? 0.f : __expf(m - mt);
        l *= f;
        acc[0] *= f;
        acc[1] *= f;
        m = mt;
        for (int i = 0; i < kAttnThreads; ++i) {
            if (w[i] == 0.f) continue;
            l += w[i];
            const int u = base + i;
            const uint8_t *blk = block_at(c, page_of(c, b, u), hk, u % c.page_tokens / kTok);
            for (int k = 0, d = tid; d < D; d += kAttnThreads, ++k)
                acc[k] += w[i] * e2m1_value(blk[v_codes_at(D) + d * 16 + u % kTok / 2] >> (u % 2 * 4)) *
                          e4m3_value(blk[v_scale_at(D) + d / 16 * kTok + u % kTok]);
        }
        __syncthreads();
    }
    const int64_t o = (static_cast<int64_t>(lo + j) * p.Hq + h);
    for (int k = 0, d = tid; d < D; d += kAttnThreads, ++k)
        static_cast<T *>(p.out)[o * D + d] = from_f32<T>(l > 0.f ? acc[k] * gv / l : 0.f);
    if (p.lse && tid == 0) p.lse[o] = l > 0.f ? m + logf(l) : -INFINITY;
}

// One CTA per (tile of 128 tokens, request): a thread per token, every row and
// query head in turn.
template <typename T>
__global__ void __launch_bounds__(kAttnThreads) weights_kernel(const CacheView c, const AttnParams p)
{
    const int b = blockIdx.y, tid = threadIdx.x, t = blockIdx.x * kAttnThreads + tid;
    int lo, n;
    if (!request_rows(p.cu_rows, b, p.R_cap, p.k_max + 1, p.status, lo, n)) return;
    const int len = p.len[b], D = c.D;
    if (len < 0 || len > p.max_len) {
        if (tid == 0) set_status(p.status, SPEC_STATUS_BAD_LENGTH);
        return;
    }
    __shared__ float q[256];
    const int page = t < len ? page_of(c, b, t) : -1;
    if (t < len && page < 0) set_status(p.status, SPEC_STATUS_BAD_PAGE);
    const int tpos = page >= 0 ? slot_position(c, p, b, t) : 0;
    float sum = 0.f;
    bool seen = false;
    for (int j = 0; j < n; ++j) {
        const int own = len - n + j;
        const int pos = own >= 0 ? slot_position(c, p, b, own) : 0;
        for (int h = 0; h < p.Hq; ++h) {
            const int hk = h / (p.Hq / c.H);
            __syncthreads();
            const T *qp = static_cast<const T *>(p.q) + (lo + j) * p.q_row + h * p.q_head;
            for (int d = tid; d < D; d += kAttnThreads) q[d] = to_f32<T>(qp[d]);
            __syncthreads();
            const float lse = p.lse[static_cast<int64_t>(lo + j) * p.Hq + h];
            const int dist = pos - tpos;
            if (page >= 0 && t <= own && (p.window <= 0 || dist < p.window || t < p.prefix)) {
                seen = true;
                if (lse == -INFINITY) continue;
                const float gk = c.k_scale ? c.k_scale[hk] : 1.f;
                sum += __expf(score_of(p, gk * dot_key<T>(block_at(c, page, hk, t % c.page_tokens / kTok), t % kTok, D, q),
                                       p.slopes ? p.slopes[h] : 0.f, dist) - lse);
            }
        }
    }
    if (seen) p.score[static_cast<int64_t>(page) * c.page_tokens + t % c.page_tokens] += sum;
}

}  // namespace

cudaError_t launch_cache_attend(const CacheView &c, const AttnParams &p, int dtype, cudaStream_t s)
{
    const dim3 grid(p.Hq, p.k_max + 1, c.B);
    if (dtype == SPEC_BF16) attend_kernel<__nv_bfloat16><<<grid, kAttnThreads, 0, s>>>(c, p);
    else attend_kernel<float><<<grid, kAttnThreads, 0, s>>>(c, p);
    return cudaGetLastError();
}

cudaError_t launch_cache_weights(const CacheView &c, const AttnParams &p, int dtype, cudaStream_t s)
{
    const dim3 grid((p.max_len + kAttnThreads - 1) / kAttnThreads, c.B);
    if (dtype == SPEC_BF16) weights_kernel<__nv_bfloat16><<<grid, kAttnThreads, 0, s>>>(c, p);
    else weights_kernel<float><<<grid, kAttnThreads, 0, s>>>(c, p);
    return cudaGetLastError();
}

}  // namespace specv
