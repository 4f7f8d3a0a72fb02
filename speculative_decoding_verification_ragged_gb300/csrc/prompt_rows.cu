// prompt_rows.cu -- attention of whole prompts in fp32 arithmetic (include/spec_prompt.h):
// fp32 rows, and bf16 rows that the tensor memory accelerator cannot fetch.
//
// A CTA takes 64 packed rows of a kv head and walks over the keys, 64 at a time:
//     S = Q K^T c,  P = 2^(S - m),  O += P V,  m a reference per row that moves when a score passes it by 2.
// Sums run over up to 2^24 keys.  Added one after another they would lose up to keys x 2^-24 of themselves, and do where weights
// and values are alike (1e-2 at 2^20 keys); so a tile's sum goes to the total by a sum that keeps its error (Knuth's), and the error
// begins the next tile's sum: 64 terms' roundings are left, whatever the number of keys.  References that move by a factor of 2 or more
// keep the roundings of rescaling a geometric series.
// 16 x 16 threads hold 4 x 4 scores and 4 x D/16 results each in registers; Q, K, V and P lie
// in shared memory as fp32, rows 4 words apart in their banks, so that the 8 lanes of a 16-byte
// load meet 32 different ones.  fp32 keys and values come by asynchronous copies, a tile ahead.
// Bound by those loads (12 an SM's clock for 32 packed products: they keep their pipe busy 58 % of the time, the products theirs 52 %,
// and eight warps an SM overlap the two no further): 4 prompts of 2000 tokens, 16 / 4 heads of 128, fp32, take
// 2.02 ms, 32 TFLOP/s of visible pairs (2.15 with one sum a channel, rescaled with every tile); of 64 channels 1.06 (1.01).  As bf16 in
// rows that TMA cannot fetch 2.73 ms, where the tensor cores take 0.075.
#include "attend.cuh"
#include "prompt.cuh"

namespace specv {

namespace {

constexpr int kRows = 64, kKeys = 64, kRowThreads = 256;
constexpr float kMove = 1.f;                          // log2 units a score may pass the reference by

// total += sum; sum = what that rounded away
__device__ __forceinline__ void to_total(float &total, float &sum)
{
    const float t = __fadd_rn(total, sum), z = __fsub_rn(t, total);
    sum = __fadd_rn(__fsub_rn(total, __fsub_rn(t, z)), __fsub_rn(sum, z));
    total = t;
}

__device__ __forceinline__ void to_total(uint64_t &total, uint64_t &sum)
{
    const uint64_t minus = f2_pack(-1.f, -1.f);
    const auto sub = [&](uint64_t a, uint64_t b) { return f2_fma(b, minus, a); };
    const uint64_t t = f2_add(total, sum), z = sub(t, total);
    sum = f2_add(sub(total, sub(t, z)), sub(sum, z));
    total = t;
}

template <int D> constexpr int row_words = D + 4;
// keys and values lie twice where there is room: the next ones are fetched beside the arithmetic
template <int D> constexpr int row_buffers = D == 256 ? 1 : 2;
template <int D> constexpr int rows_smem = ((1 + 2 * row_buffers<D>) * kRows * row_words<D> + kRows * (kKeys + 4)) * 4;

// `rows` rows of D channels into shared memory; row(i): where row i starts, null for zeros
template <typename T, int D, typename F> __device__ __forceinline__ void stage_rows(float *to, bool aligned, F row)
{
    for (int i = threadIdx.x; i < kRows * (D / 8); i += kRowThreads) {
        const int r = i / (D / 8), d = i % (D / 8) * 8;
        const T *src = row(r);
        float x[8] = {};
        if (src) load8<T>(src + d, aligned, x);
        float4 *dst = reinterpret_cast<float4 *>(to + r * row_words<D> + d);
        dst[0] = make_float4(x[0], x[1], x[2], x[3]);
        dst[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// 16 bytes from global to shared memory, asynchronously; zeros where `have` is false
__device__ __forceinline__ void fetch16(float *to, const void *from, bool have)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(from), "r"(have ? 16 : 0) : "memory");
}

// the same as stage_rows for fp32 rows on 16 bytes, under way until rows_arrived
template <int D, typename F> __device__ __forceinline__ void fetch_rows(float *to, const void *any, F row)
{
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kRowThreads) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        const float *const src = row(r);
        fetch16(to + r * row_words<D> + d, src ? src + d : any, src != nullptr);
    }
}

__device__ __forceinline__ void rows_asked() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void rows_arrived() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) prompt_rows_kernel(const PromptParams p)
{
    constexpr int W = row_words<D>, PW = kKeys + 4, OC = D / 16;
    extern __shared__ __align__(16) float sm[];
    constexpr int BUF = row_buffers<D>;
    float *const qs = sm, *const kv = qs + kRows * W, *const ps = kv + 2 * BUF * kKeys * W;
    const int group = p.Hq / p.H, h = blockIdx.y;
    PromptTile t;
    int tile;
    if (!find_prompt_tile<kRowThreads>(p, blockIdx.x, blockIdx.x == 0 && h == 0,
                                       [&](int n) { return (n * group + kRows - 1) / kRows; }, t, tile))
        return;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int first = tile * kRows, count = min(t.n * group - first, kRows);
    const int own0 = t.m - t.n;                       // own key of row 0
    // 64 packed rows: (row, head) of each
    const auto row_of = [&](int r) { return (first + r) / group; };
    const auto head_of = [&](int r) { return h * group + (first + r) % group; };
    stage_rows<T, D>(qs, p.q_aligned, [&](int r) {
        return r < count ? static_cast<const T *>(p.q) + static_cast<int64_t>(t.lo + row_of(r)) * p.q_row + head_of(r) * p.q_head : nullptr;
    });
    int own[4];                                       // last key that each of this thread's rows sees
    float slope[4], m[4], l[4], l_all[4];             // l, o: of the tile, from what the totals lack on
    uint64_t o[4][OC / 2], o_all[4][OC / 2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        own[i] = r < count ? own0 + row_of(r) : -1;
        slope[i] = p.slopes && r < count ? p.slopes[head_of(r)] * kLog2e : 0.f;
        m[i] = -INFINITY;
        l[i] = l_all[i] = 0.f;
#pragma unroll
        for (int j = 0; j < OC / 2; ++j) o[i][j] = o_all[i][j] = 0;
    }
    // keys that some row of the tile sees: up to the last row's own, a window's from the first row's on
    // (those that no row of the request sees are taken as zeros, whatever they hold)
    const int end = min(own0 + row_of(count - 1) + 1, t.m);
    const int near = p.window > 0 ? max(own0 + row_of(0) - p.window + 1, 0) : 0;
    const int live = p.window > 0 ? max(own0 - p.window + 1, 0) : 0;      // of the request's first row
    const float c = p.scale * kLog2e, cap = p.cap * kLog2e, rcap = p.cap > 0.f ? cap_reciprocal(cap) : 0.f;
    const auto next = [&](int k0) {                   // the tile of keys after this one that some row sees
        do k0 += kKeys;
        while (k0 < end && k0 >= p.prefix && k0 + kKeys <= near);
        return k0;
    };
    const bool ahead = BUF == 2 && sizeof(T) == 4 && p.k_aligned && p.v_aligned;
    const auto key = [&](const void *x, int64_t row, int64_t head, int k0) {
        return [=, &p](int r) {
            const int j = k0 + r;
            return j < t.m && (j >= live || j < p.prefix)
                       ? static_cast<const T *>(x) + (t.k_lo + static_cast<int64_t>(j)) * row + h * head : nullptr;
        };
    };
    const auto fetch = [&](int k0, int buf) {
        if constexpr (sizeof(T) == 4) {
            fetch_rows<D>(kv + 2 * buf * kKeys * W, p.k, key(p.k, p.k_row, p.k_head, k0));
            fetch_rows<D>(kv + (2 * buf + 1) * kKeys * W, p.v, key(p.v, p.v_row, p.v_head, k0));
            rows_asked();
        }
    };
    int k0 = next(-kKeys), buf = 0;
    if (ahead && k0 < end) fetch(k0, 0);
    for (; k0 < end; k0 = next(k0)) {
        const float *const ks = kv + 2 * buf * kKeys * W, *const vs = ks + kKeys * W;
        if (ahead) {
            rows_arrived();
            __syncthreads();                          // (and the other buffer is read)
            const int k1 = next(k0);
            buf ^= 1;
            if (k1 < end) fetch(k1, buf);
        } else {
            __syncthreads();
            stage_rows<T, D>(kv, p.k_aligned, key(p.k, p.k_row, p.k_head, k0));
            stage_rows<T, D>(kv + kKeys * W, p.v_aligned, key(p.v, p.v_row, p.v_head, k0));
            __syncthreads();
        }
        uint64_t s2[4][4] = {};
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            ulonglong2 a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const ulonglong2 *>(qs + (ty * 4 + i) * W + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const ulonglong2 *>(ks + (tx + 16 * j) * W + d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s2[i][j] = f2_fma(a[i].y, b[j].y, f2_fma(a[i].x, b[j].x, s2[i][j]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float s[4], top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x, y;
                f2_unpack(s2[i][j], x, y);
                const int key_at = k0 + tx + 16 * j, dist = own[i] - key_at;
                s[j] = (x + y) * c;
                if (p.cap > 0.f) s[j] = cap_score<sizeof(T) == 4>(s[j], cap, rcap);
                s[j] -= slope[i] * static_cast<float>(dist);
                const bool see = dist >= 0 && (p.window <= 0 || dist < p.window || key_at < p.prefix);
                s[j] = see ? s[j] : -INFINITY;
                top = fmaxf(top, s[j]);
            }
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
            if (top > m[i] + kMove) {
                const float f = exp2f(m[i] - top);
                const uint64_t f2 = f2_pack(f, f);
                m[i] = top;
                l[i] *= f;
                l_all[i] *= f;
#pragma unroll
                for (int j = 0; j < OC / 2; ++j) {
                    o[i][j] = f2_fma(o[i][j], f2, 0);
                    o_all[i][j] = f2_fma(o_all[i][j], f2, 0);
                }
            }
            const float ref = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = exp2f(s[j] - ref);
                l[i] += w;
                ps[(ty * 4 + i) * PW + tx + 16 * j] = w;
            }
            to_total(l_all[i], l[i]);
        }
        __syncwarp();                                 // (a warp's rows are its own)
#pragma unroll 2
        for (int k = 0; k < kKeys; k += 4) {
            float4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4 *>(ps + (ty * 4 + i) * PW + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
                for (int j = 0; j < OC / 4; ++j) {
                    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(vs + (k + kk) * W + j * 64 + tx * 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = kk == 0 ? w[i].x : (kk == 1 ? w[i].y : (kk == 2 ? w[i].z : w[i].w));
                        const uint64_t x2 = f2_pack(x, x);
                        o[i][2 * j] = f2_fma(x2, v.x, o[i][2 * j]);
                        o[i][2 * j + 1] = f2_fma(x2, v.y, o[i][2 * j + 1]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < OC / 2; ++j) to_total(o_all[i][j], o[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        l[i] += l_all[i];
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], x);
        const int r = ty * 4 + i;
        if (r >= count) continue;
        const int64_t at = (t.lo + static_cast<int64_t>(row_of(r))) * p.Hq + head_of(r);
        const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
        T *const to = static_cast<T *>(p.out) + at * D;
#pragma unroll
        for (int j = 0; j < OC / 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x, y;
                f2_unpack(f2_add(o_all[i][2 * j + e], o[i][2 * j + e]), x, y);
                to[j * 64 + tx * 4 + 2 * e] = from_f32<T>(x * inv);
                to[j * 64 + tx * 4 + 2 * e + 1] = from_f32<T>(y * inv);
            }
        if (p.lse && tx == 0) p.lse[at] = l[i] > 0.f ? (m[i] + log2f(l[i])) * kLn2 : -INFINITY;
    }
}

template <typename T, int D> cudaError_t launch_rows(const PromptParams &p, cudaStream_t s)
{
    static bool done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev]) {
        e = cudaFuncSetAttribute(prompt_rows_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, rows_smem<D>);
        if (e != cudaSuccess) return e;
        done[dev] = true;
    }
    // at most this many tiles (the host checked that they are countable)
    const int64_t tiles = (static_cast<int64_t>(p.R_cap) * (p.Hq / p.H)) / kRows + p.B;
    prompt_rows_kernel<T, D><<<dim3(static_cast<unsigned>(tiles), p.H), kRowThreads, rows_smem<D>, s>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_rows_of(const PromptParams &p, cudaStream_t s)
{
    if (p.D == 64) return launch_rows<T, 64>(p, s);
    return p.D == 128 ? launch_rows<T, 128>(p, s) : launch_rows<T, 256>(p, s);
}

}  // namespace

cudaError_t launch_prompt_rows(const PromptParams &p, int dtype, cudaStream_t s)
{
    return dtype == SPEC_F32 ? launch_rows_of<float>(p, s) : launch_rows_of<__nv_bfloat16>(p, s);
}

}  // namespace specv
