// tree.cu -- acceptance of a path through a tree of drafts, and the adjustment of the
// rows' logits by penalties, biases and masks (include/spec_tree.h).
#include "cache.cuh"
#include "tree.cuh"

namespace specv {

namespace {

constexpr int kAcceptWarps = 4;

// A warp a request, a lane a node.  The walk takes a vote a node: which lanes hang on it and have its
// token.
__global__ void __launch_bounds__(kAcceptWarps * 32) tree_accept_kernel(const TreeParams p)
{
    const int b = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (b >= p.B) return;
    const int width = p.k_max + 1;
    int lo, n;
    const bool ok = request_rows(p.cu_rows, b, p.R_cap, width, nullptr, lo, n) && n > 0;
    int out = -1, path = -1, len = 0, next = -1;
    if (ok) {
        const int parent = tree_parent(p.parent, lo, n, p.status);
        const int mine = lane < n ? __ldg(p.row_token + lo + lane) : -1;
        const int token = lane > 0 && lane < n ? __ldg(p.node_token + lo + lane) : -1;
        int at = 0;
        path = 0;
        for (;;) {                                    // (a child comes after its parent: at most n steps)
            next = __shfl_sync(0xFFFFFFFFu, mine, at);
            if (lane == len) out = next;
            const uint32_t hit = __ballot_sync(0xFFFFFFFFu, lane < n && parent == at && token == next);
            if (!hit) break;
            at = __ffs(hit) - 1;
            ++len;
            if (lane >= len) path = at;
        }
        path += lo;
    } else if (lane == 0) {
        set_status(p.status, SPEC_STATUS_BAD_ROWS);
    }
    if (lane < width) {
        p.out_tokens[static_cast<int64_t>(b) * width + lane] = out;
        if (p.path_rows) p.path_rows[static_cast<int64_t>(b) * width + lane] = path;
    }
    if (lane == 0) {
        p.accepted_len[b] = len;
        p.next_token[b] = next;
    }
}

// ---- logits ----

// A CTA takes kSlice columns of a request's rows: the tokens so far are counted once, in
// shared memory, for all rows.  A column's word: how often it was generated, whether it
// was seen at all, whether one of the request's biases or nodes names it; a bit a column says
// whether the word is anything but 0, so that most columns cost a byte of shared memory each 8.
constexpr int kSlice = 8192, kLogitThreads = 256;
constexpr uint32_t kSeen = 1u << 31, kNamed = 1u << 30, kCount = kNamed - 1u;
constexpr int kNear = 256;                            // biases of a slice kept in shared memory

template <typename T> struct LogitElt;
template <> struct LogitElt<__nv_bfloat16> {
    static constexpr int VEC = 8;
    static __device__ __forceinline__ void unpack(uint4 v, float (&x)[8]) { Elt<uint16_t>::unpack(v, x); }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8])
    {
        uint4 v;
        uint32_t *w = &v.x;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        return v;
    }
};
template <> struct LogitElt<float> {
    static constexpr int VEC = 4;
    static __device__ __forceinline__ void unpack(uint4 v, float (&x)[4]) { Elt<float>::unpack(v, x); }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

struct Slice {
    uint32_t word[kSlice];
    uint32_t touched[kSlice / 32 + 1];
    int node_token[32];
    uint32_t path[32];                                // of each row: the nodes on it
    int bias_id[kNear];
    float bias_value[kNear];
    int scan[kLogitThreads / 32];
    int n_bias;
};

// N bits of a bit set from bit `i` on
__device__ __forceinline__ uint32_t bits_at(const uint32_t *set, int i, int last_word)
{
    const int w = i >> 5;
    return __funnelshift_r(set[w], w < last_word ? set[w + 1] : 0u, i & 31);
}

struct Penalty {
    float repetition, frequency, presence;
};

// one touched column (v: from the slice's first on) of a row with `path`
__device__ __forceinline__ float adjust(const LogitParams &p, const Slice &s, const Penalty &pen, int c0, int v, int n, uint32_t path,
                                        int bias0, int bias1, float z)
{
    const uint32_t w = s.word[v];
    int count = static_cast<int>(w & kCount);
    bool seen = (w & kSeen) != 0;
    if (w & kNamed) {
        for (int j = 1; j < n; ++j) count += path >> j & 1u && s.node_token[j] == c0 + v;
    }
    seen |= count > 0;
    if (seen) z = z > 0.f ? z / pen.repetition : z * pen.repetition;
    if (count > 0) z = z - pen.frequency * static_cast<float>(count) - pen.presence;
    if (w & kNamed) {
        float add = 0.f;
        if (s.n_bias <= kNear) {
            for (int i = 0; i < s.n_bias; ++i) add += s.bias_id[i] == v ? s.bias_value[i] : 0.f;
        } else {
            for (int i = bias0; i < bias1; ++i) add += __ldg(p.bias_ids + i) == c0 + v ? __ldg(p.bias_values + i) : 0.f;
        }
        z += add;
    }
    return z;
}

template <typename T>
__global__ void __launch_bounds__(kLogitThreads) adjust_logits_kernel(const LogitParams p)
{
    using E = LogitElt<T>;
    constexpr int VEC = E::VEC;
    __shared__ __align__(16) Slice s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
    const int c0 = blockIdx.x * kSlice, cols = min(p.V - c0, kSlice);
    uint32_t *const report = blockIdx.x == 0 ? p.status : nullptr;      // (one CTA of a request speaks for it)
    int lo, n;
    if (!request_rows(p.cu_rows, b, p.R_cap, p.k_max + 1, tid == 0 ? report : nullptr, lo, n) || n == 0) return;

    for (int i = tid; i < kSlice / 4; i += kLogitThreads) reinterpret_cast<uint4 *>(s.word)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < kSlice / 32 + 1; i += kLogitThreads) s.touched[i] = 0;
    const auto mark = [&](int v) { atomicOr(&s.touched[v >> 5], 1u << (v & 31)); };
    // the request's penalties
    Penalty pen = {p.repetition ? p.repetition[b] : 1.f, p.frequency ? p.frequency[b] : 0.f, p.presence ? p.presence[b] : 0.f};
    const auto finite = [](float x) { return x - x == 0.f; };
    bool bad = false;
    if (!finite(pen.repetition) || pen.repetition <= 0.f) pen.repetition = 1.f, bad = true;
    if (!finite(pen.frequency)) pen.frequency = 0.f, bad = true;
    if (!finite(pen.presence)) pen.presence = 0.f, bad = true;
    const bool penal = pen.repetition != 1.f || pen.frequency != 0.f || pen.presence != 0.f;
    int tokens = penal && p.history ? p.n_tokens[b] : 0;
    if (tokens < 0 || tokens > p.history_cap) {
        if (tid == 0) set_status(report, SPEC_STATUS_BAD_LENGTH);
        tokens = 0;
    }
    const int prompt = tokens > 0 && p.n_prompt ? p.n_prompt[b] : 0;
    int bias0 = 0, bias1 = 0;
    if (p.bias_cu) {
        bias0 = p.bias_cu[b];
        bias1 = p.bias_cu[b + 1];
        if (bias0 < 0 || bias1 < bias0 || bias1 > p.n_bias) bias0 = bias1 = 0, bad = true;
    }
    if (bad && tid == 0) set_status(report, SPEC_STATUS_BAD_PENALTY);
    __syncthreads();

    // the history
    const int32_t *hist = p.history ? p.history + static_cast<int64_t>(b) * p.history_ld : nullptr;
    const auto count = [&](int i, int t) {
        const uint32_t v = static_cast<uint32_t>(t) - static_cast<uint32_t>(c0);
        if (v < static_cast<uint32_t>(cols)) {
            if (i < prompt) atomicOr(&s.word[v], kSeen);
            else atomicAdd(&s.word[v], 1u);
            mark(v);
        }
    };
    for (int i = tid; i < tokens; i += 4 * kLogitThreads) {
        int t[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) t[u] = i + u * kLogitThreads < tokens ? __ldg(hist + i + u * kLogitThreads) : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u) count(i + u * kLogitThreads, t[u]);
    }
    // the nodes and the rows' paths
    if (warp == 0) {
        const int parent = tree_parent(p.parent, lo, n, report);
        const uint32_t hung = __ballot_sync(0xFFFFFFFFu, parent >= 0);
        const bool have = penal && p.node_token && lane < n;
        const int t = have && lane > 0 ? __ldg(p.node_token + lo + lane) : -1;
        const uint32_t anc = tree_ancestors(parent);   // (the whole warp: it exchanges them)
        s.path[lane] = have ? anc & hung : 0u;
        s.node_token[lane] = t;
        const uint32_t v = static_cast<uint32_t>(t) - static_cast<uint32_t>(c0);
        if (parent >= 0 && t >= 0 && v < static_cast<uint32_t>(cols)) {
            atomicOr(&s.word[v], kNamed);
            mark(v);
        }
    }
    // the biases of the slice, in their order
    int near = 0;
    for (int i0 = bias0; i0 < bias1; i0 += kLogitThreads) {
        const int i = i0 + tid;
        const uint32_t v = i < bias1 ? static_cast<uint32_t>(__ldg(p.bias_ids + i)) - static_cast<uint32_t>(c0) : 0xFFFFFFFFu;
        const bool mine = v < static_cast<uint32_t>(cols);
        const uint32_t vote = __ballot_sync(0xFFFFFFFFu, mine);
        if (lane == 0) s.scan[warp] = __popc(vote);
        __syncthreads();
        int at = near + __popc(vote & ((1u << lane) - 1u));
#pragma unroll
        for (int w = 0; w < kLogitThreads / 32; ++w) {
            at += w < warp ? s.scan[w] : 0;
            near += s.scan[w];
        }
        if (mine) {
            if (at < kNear) {
                s.bias_id[at] = static_cast<int>(v);
                s.bias_value[at] = __ldg(p.bias_values + i);
            }
            atomicOr(&s.word[v], kNamed);
            mark(v);
        }
        __syncthreads();
    }
    if (tid == 0) s.n_bias = near;
    __syncthreads();

    const int mask_words = (p.V + 31) / 32;
    for (int j = 0; j < n; ++j) {
        const int row = lo + j;
        const T *src = static_cast<const T *>(p.logits) + static_cast<int64_t>(row) * p.ld + c0;
        T *dst = static_cast<T *>(p.out) + static_cast<int64_t>(row) * p.out_ld + c0;
        const uint32_t path = s.path[j];
        const uint32_t *allowed = nullptr;
        if (p.allowed) {
            const int m = p.allowed_row ? __ldg(p.allowed_row + row) : row;
            if (m >= 0 && m < p.n_allowed) allowed = p.allowed + m * p.allowed_ld;
            else if ((m != -1 || !p.allowed_row) && tid == 0) set_status(report, SPEC_STATUS_BAD_MASK);
        }
        const auto one = [&](int v) {
            float z = to_f32<T>(src[v]);
            if (s.touched[v >> 5] >> (v & 31) & 1u) z = adjust(p, s, pen, c0, v, n, path, bias0, bias1, z);
            if (allowed && !(__ldg(allowed + ((c0 + v) >> 5)) >> ((c0 + v) & 31) & 1u)) z = -INFINITY;
            dst[v] = from_f32<T>(z);
        };
        // 16-byte vectors where input and output lie alike, the columns before and after one by one
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 15u);
        if (off != static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dst) & 15u)) {
            for (int v = tid; v < cols; v += kLogitThreads) one(v);
            continue;
        }
        const int head = min(static_cast<int>((16u - off) % 16u / sizeof(T)), cols);
        const int vecs = (cols - head) / VEC, tail = head + vecs * VEC;
        if (tid < head) one(tid);
        else if (tid >= 32 && tid - 32 < cols - tail) one(tail + tid - 32);
        constexpr int U = 4;
        for (int i0 = tid; i0 < vecs; i0 += U * kLogitThreads) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * kLogitThreads;
                if (i < vecs) x[u] = *reinterpret_cast<const uint4 *>(src + head + i * VEC);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * kLogitThreads, v = head + i * VEC;
                if (i >= vecs) break;
                uint32_t hit = bits_at(s.touched, v, kSlice / 32) & ((1u << VEC) - 1u);
                uint32_t may = (1u << VEC) - 1u;
                if (allowed) {
                    const int w = (c0 + v) >> 5;
                    may &= __funnelshift_r(__ldg(allowed + w), w + 1 < mask_words ? __ldg(allowed + w + 1) : 0u, (c0 + v) & 31);
                }
                if (hit == 0 && may == (1u << VEC) - 1u) {
                    *reinterpret_cast<uint4 *>(dst + v) = x[u];
                    continue;
                }
                float z[VEC];
                E::unpack(x[u], z);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    if (hit >> k & 1u) z[k] = adjust(p, s, pen, c0, v + k, n, path, bias0, bias1, z[k]);
                    if (!(may >> k & 1u)) z[k] = -INFINITY;
                }
                *reinterpret_cast<uint4 *>(dst + v) = E::pack(z);
            }
        }
    }
}

}  // namespace

cudaError_t launch_tree_accept(const TreeParams &p, cudaStream_t s)
{
    tree_accept_kernel<<<(p.B + kAcceptWarps - 1) / kAcceptWarps, kAcceptWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_adjust_logits(const LogitParams &p, int dtype, cudaStream_t s)
{
    const dim3 grid((p.V + kSlice - 1) / kSlice, p.B);
    if (dtype == SPEC_F32) adjust_logits_kernel<float><<<grid, kLogitThreads, 0, s>>>(p);
    else adjust_logits_kernel<__nv_bfloat16><<<grid, kLogitThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace specv
