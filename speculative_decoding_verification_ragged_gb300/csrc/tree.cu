// tree.cu -- acceptance of a path through a tree of drafts, and the adjustment of the
// rows' logits by penalties, biases and masks (include/spec_tree.h).
#include "cache.cuh"
#include "tensor.cuh"
#include "tree.cuh"

namespace specv {

namespace {

constexpr int kAcceptWarps = 4;

// A warp a request, a lane a node.  The walk takes a vote a node: which lanes hang on it and have its
// token.  Bound by the launch: 6 us for one tree as for 4096 of up to 32 nodes.
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

// A CTA takes kSlice columns of a request's rows (or of every few of them).  They stream by first, copied and masked; the
// tokens so far are counted once for all rows, in shared memory, and the columns that have a count, a draft of
// the paths or a bias ("touched") are written over, a thread each.  In place the touched columns come first, and only
// rows with a mask stream by (a masked column is -inf whatever it was).
//
// Bound by HBM while the rows stream by (128 x 5 rows of 152064 bf16: 64 us without rules, 6.1 TB/s, 0.90 of the measured copy
// rate), and by what a CTA does beside that (history, list, touched columns), a chain of loads that five CTAs an SM do not hide:
// 96 us with histories of 4096 tokens and every second row masked (0.61).  A slice of 8192 columns: every slice reads the
// history again, so that half of it took 120 us, and fewer CTAs have less in flight, so that twice took 105 and four times 117
// (60000 tokens, one row of 64 requests: 93, 172, 83, 81).  Each call alone over a cold L2: 117 us; in place 93, and 68
// without masks, where only touched columns are read and written.  Tried as well: four of the CTA's warps counting while the others
// stream (105), a cluster that shares the history by distributed atomics (128, frequent tokens meet there), vectors of a row
// ahead of the stores (120: registers for fewer CTAs), six CTAs an SM (119: fewer loads in flight in each).
//
// A column's word: how often it was generated, whether it was seen at all, whether one of the request's nodes names it, one of
// its biases, more than one; a bit a column says whether the word is anything but 0.
constexpr int kSlice = 8192, kLogitThreads = 256;
constexpr uint32_t kSeen = 1u << 31, kNamed = 1u << 30, kBiased = 1u << 29, kTwice = 1u << 28, kCount = kTwice - 1u;
constexpr int kNear = 256;                            // biases of a slice kept in shared memory
constexpr int kFull = 152 * 5;                        // CTAs that are resident at once
constexpr int kListed = 1024, kListedBiased = 2 * kNear;      // touched columns that are listed at a time; with more biases than kNear

template <typename T> struct LogitElt;
template <> struct LogitElt<__nv_bfloat16> {
    static constexpr int VEC = 8;
    // -inf where `may` has a bit clear
    static __device__ __forceinline__ void hide(uint4 &v, uint32_t may)
    {
        uint32_t *w = &v.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = may >> (2 * i) & 1u ? w[i] : 0xFF80u, hi = may >> (2 * i + 1) & 1u ? w[i] : 0xFF800000u;
            w[i] = __byte_perm(lo, hi, 0x7610);
        }
    }
};
template <> struct LogitElt<float> {
    static constexpr int VEC = 4;
    static __device__ __forceinline__ void hide(uint4 &v, uint32_t may)
    {
        uint32_t *w = &v.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = may >> i & 1u ? w[i] : 0xFF800000u;
    }
};

struct Slice {
    uint32_t word[kSlice];
    uint32_t touched[kSlice / 32];
    int node_token[32];
    uint32_t path[32];                                // of each row: the nodes on it
    int mask[32];                                     // of each row: its mask, -1 for none
    union {
        struct {
            int bias_id[kNear];
            float bias_value[kNear];
        };
        float bias_sum[kListedBiased];                // of each listed column, where the biases are too many
    };
    uint16_t before[kLogitThreads];                   // touched columns before each word of the bit set
    int scan[kLogitThreads / 32];
    int n_bias, twice;                                // biases of the slice; whether a column has several
    uint16_t column[kListed];
};

struct Penalty {
    float repetition, frequency, presence;
};

// one touched column (v: from the slice's first on; `at`: its place in the list) of a row with `path`
__device__ __forceinline__ float adjust(const Slice &s, const Penalty &pen, int c0, int v, int at, int n, uint32_t path, float z)
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
    if (w & kBiased) {
        float add = 0.f;
        if (s.n_bias <= kNear) {
            for (int i = 0; i < s.n_bias; ++i) add += s.bias_id[i] == v ? s.bias_value[i] : 0.f;
        } else {
            add = s.bias_sum[at];
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
    extern __shared__ __align__(16) uint8_t raw[];
    Slice &s = *reinterpret_cast<Slice *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_index(), b = blockIdx.y;
    const int c0 = blockIdx.x * kSlice, cols = min(p.V - c0, kSlice);
    uint32_t *const report = blockIdx.x == 0 && blockIdx.z == 0 ? p.status : nullptr;      // (one CTA of a request speaks for it)
    // What the request has is asked for at once, and what that leads to before the rows stream by: a CTA lives as long as
    // its chain of loads.
    Penalty pen = {p.repetition ? p.repetition[b] : 1.f, p.frequency ? p.frequency[b] : 0.f, p.presence ? p.presence[b] : 0.f};
    int tokens = p.history ? p.n_tokens[b] : 0;
    const int prompt = p.history && p.n_prompt ? p.n_prompt[b] : 0;
    int bias0 = p.bias_cu ? p.bias_cu[b] : 0, bias1 = p.bias_cu ? p.bias_cu[b + 1] : 0;
    int lo, n;
    if (!request_rows(p.cu_rows, b, p.R_cap, p.k_max + 1, tid == 0 ? report : nullptr, lo, n) || n <= static_cast<int>(blockIdx.z)) return;
    // a token's column of the slice; others, ids below 0 among them, come out beyond it
    const auto column = [&](int t) { return static_cast<uint32_t>(t) - static_cast<uint32_t>(c0); };
    const auto finite = [](float x) { return x - x == 0.f; };
    bool bad = false;
    if (!finite(pen.repetition) || pen.repetition <= 0.f) pen.repetition = 1.f, bad = true;
    if (!finite(pen.frequency)) pen.frequency = 0.f, bad = true;
    if (!finite(pen.presence)) pen.presence = 0.f, bad = true;
    if (bias0 < 0 || bias1 < bias0 || bias1 > p.n_bias) bad = bad || p.bias_cu, bias0 = bias1 = 0;
    if (bad && tid == 0) set_status(report, SPEC_STATUS_BAD_PENALTY);
    const bool penal = pen.repetition != 1.f || pen.frequency != 0.f || pen.presence != 0.f;
    if (tokens < 0 || tokens > p.history_cap) {
        if (tid == 0) set_status(report, SPEC_STATUS_BAD_LENGTH);
        tokens = 0;
    }
    if (!penal) tokens = 0;

    const bool in_place = p.out == p.logits;
    const int mask_words = (p.V + 31) / 32;
    const auto source = [&](int row) { return static_cast<const T *>(p.logits) + static_cast<int64_t>(row) * p.ld + c0; };
    const auto target = [&](int row) { return static_cast<T *>(p.out) + static_cast<int64_t>(row) * p.out_ld + c0; };
    const auto mask_of = [&](int row) {
        if (!p.allowed) return -1;
        const int m = p.allowed_row ? __ldg(p.allowed_row + row) : row;
        return m >= 0 && m < p.n_allowed ? m : (m == -1 ? -1 : -2);
    };
    const auto mask_at = [&](int m) -> const uint32_t * { return m >= 0 ? p.allowed + m * p.allowed_ld : nullptr; };
    const auto hidden = [&](const uint32_t *allowed, int v) {
        return allowed && !(__ldg(allowed + ((c0 + v) >> 5)) >> ((c0 + v) & 31) & 1u);
    };
    // a row as it streams by
    const auto stream = [&](int row) {
        const uint32_t *const allowed = mask_at(mask_of(row));
        if (in_place && !allowed) return;
        const T *const src = source(row);
        T *const dst = target(row);
        const auto one = [&](int v) { dst[v] = hidden(allowed, v) ? from_f32<T>(-INFINITY) : src[v]; };
        // 16-byte vectors where input and output lie alike, the columns before and after one by one
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 15u);
        if (off != static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dst) & 15u)) {
            for (int v = tid; v < cols; v += kLogitThreads) one(v);
            return;
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
                if (allowed) {
                    const int w = (c0 + v) >> 5;
                    E::hide(x[u], __funnelshift_r(__ldg(allowed + w), w + 1 < mask_words ? __ldg(allowed + w + 1) : 0u, (c0 + v) & 31));
                }
                *reinterpret_cast<uint4 *>(dst + v) = x[u];
            }
        }
    };

    // the first tokens, the nodes and the first biases: asked for here, looked at when the rows are through
    const int32_t *const hist = p.history ? p.history + static_cast<int64_t>(b) * p.history_ld : nullptr;
    int first_tokens[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int i = u * kLogitThreads + tid;
        first_tokens[u] = i < tokens ? __ldg(hist + i) : -1;
    }
    const int first_id = bias0 + tid < bias1 ? __ldg(p.bias_ids + bias0 + tid) : -1;
    const float first_value = bias0 + tid < bias1 ? __ldg(p.bias_values + bias0 + tid) : 0.f;
    int parent = -1, token = -1, mask = -1;
    if (warp == 0 && lane < n) {
        parent = tree_parent(p.parent, lo, n, report);
        if (penal && p.node_token && lane > 0) token = __ldg(p.node_token + lo + lane);
        mask = mask_of(lo + lane);
        if (mask == -2) set_status(report, SPEC_STATUS_BAD_MASK);
    }
    for (int i = tid; i < kSlice / 4; i += kLogitThreads) reinterpret_cast<uint4 *>(s.word)[i] = make_uint4(0, 0, 0, 0);
    s.touched[tid] = 0;
    if (tid == 0) s.twice = 0;
    const int z0 = blockIdx.z, dz = gridDim.z;        // this CTA's rows: z0, z0 + dz, ...
    if (!in_place)
        for (int j = z0; j < n; j += dz) stream(lo + j);
    __syncthreads();
    // the history
    const auto count = [&](int i, int t) {
        const uint32_t v = column(t);
        if (v >= static_cast<uint32_t>(cols)) return;
        // (most have been there before: a look instead of an atomic)
        const uint32_t word = *const_cast<volatile uint32_t *>(&s.word[v]);
        if (i >= prompt) atomicAdd(&s.word[v], 1u);
        else if (!(word & kSeen)) atomicOr(&s.word[v], kSeen);
        if (word == 0) atomicOr(&s.touched[v / 32], 1u << (v & 31));
    };
#pragma unroll
    for (int u = 0; u < 4; ++u) count(u * kLogitThreads + tid, first_tokens[u]);
    int done = 4 * kLogitThreads;
    if (reinterpret_cast<uintptr_t>(hist) % 16 == 0) {
        // (by vectors, what fills whole rounds of them)
        constexpr int U = 4, ROUND = 4 * U * kLogitThreads;
        for (; done <= tokens - ROUND; done += ROUND) {
            int4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = __ldg(reinterpret_cast<const int4 *>(hist + done) + u * kLogitThreads + tid);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = done + 4 * (u * kLogitThreads + tid);
                const uint32_t least = min(min(column(x[u].x), column(x[u].y)),
                                           min(column(x[u].z), column(x[u].w)));
                if (least >= static_cast<uint32_t>(cols)) continue;
                count(i, x[u].x);
                count(i + 1, x[u].y);
                count(i + 2, x[u].z);
                count(i + 3, x[u].w);
            }
        }
    }
    for (; done < tokens; done += 4 * kLogitThreads) {
        int t[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = done + u * kLogitThreads + tid;
            t[u] = i < tokens ? __ldg(hist + i) : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) count(done + u * kLogitThreads + tid, t[u]);
    }
    // the nodes, the rows' paths and masks
    if (warp == 0) {
        const uint32_t hung = __ballot_sync(0xFFFFFFFFu, parent >= 0), anc = tree_ancestors(parent);
        s.path[lane] = penal && p.node_token && lane < n ? anc & hung : 0u;
        s.node_token[lane] = token;
        s.mask[lane] = mask;
        const uint32_t v = column(token);
        if (parent >= 0 && token >= 0 && v < static_cast<uint32_t>(cols)) {
            atomicOr(&s.word[v], kNamed);
            atomicOr(&s.touched[v / 32], 1u << (v & 31));
        }
    }
    // the biases of the slice, in their order
    int near = 0;
    for (int64_t i0 = bias0; i0 < bias1; i0 += kLogitThreads) {
        const int64_t i = i0 + tid;
        const bool again = i0 > bias0;
        const int id = !again ? first_id : (i < bias1 ? __ldg(p.bias_ids + i) : -1);
        const uint32_t v = column(id);
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
                s.bias_value[at] = again ? __ldg(p.bias_values + i) : first_value;
            }
            if (atomicOr(&s.word[v], kBiased) & kBiased) {
                atomicOr(&s.word[v], kTwice);
                s.twice = 1;
            }
            atomicOr(&s.touched[v / 32], 1u << (v & 31));
        }
        __syncthreads();
    }
    if (tid == 0) s.n_bias = near;
    __syncthreads();

    // the touched columns in their order, some at a time; a thread has 32 columns of the set
    static_assert(kSlice == 32 * kLogitThreads && sizeof(Slice) <= 48 * 1024, "a word of the bit set a thread");
    const uint32_t set = s.touched[tid];
    int first = __popc(set), touched = 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, first, o);
        if (lane >= o) first += y;
    }
    if (lane == 31) s.scan[warp] = first;
    __syncthreads();
    first -= __popc(set);
#pragma unroll
    for (int w = 0; w < kLogitThreads / 32; ++w) {
        first += w < warp ? s.scan[w] : 0;
        touched += s.scan[w];
    }
    s.before[tid] = static_cast<uint16_t>(first);
    const bool many = near > kNear;
    const int listed = many ? kListedBiased : kListed;
    for (int e0 = 0; e0 < touched; e0 += listed) {
        const int count = min(touched - e0, listed);
        __syncthreads();
        int at = first - e0;
        for (uint32_t left = set; left; left &= left - 1, ++at)
            if (at >= 0 && at < listed) s.column[at] = static_cast<uint16_t>(tid * 32 + __ffs(left) - 1);
        if (many) {
            // Too many biases to compare every column with each: every bias goes to its column's sum, those of a column that has
            // several one after another (5 rows of 152064, a bias a column: 2.4 ms, 166 by comparing; two a column: 10 to 16).
            s.bias_sum[tid] = s.bias_sum[tid + kNear] = 0.f;
            __syncthreads();
            // the place in the list of a bias on column `id`, and whether the column has others, or -1
            const auto place_of = [&](int id, bool &again) {
                const uint32_t v = column(id);
                if (v >= static_cast<uint32_t>(cols)) return -1;
                const int to = s.before[v / 32] + __popc(s.touched[v / 32] & ((1u << (v & 31)) - 1u)) - e0;
                again = (s.word[v] & kTwice) != 0;
                return to >= 0 && to < count ? to : -1;
            };
            for (int64_t i0 = static_cast<int64_t>(bias0) + tid; i0 < bias1; i0 += 4 * kLogitThreads) {
                int id[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) id[u] = i0 + u * kLogitThreads < bias1 ? __ldg(p.bias_ids + i0 + u * kLogitThreads) : -1;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    bool again = false;
                    const int to = place_of(id[u], again);
                    if (to >= 0 && !again) s.bias_sum[to] = __ldg(p.bias_values + i0 + u * kLogitThreads);
                }
            }
            for (int64_t i0 = s.twice ? bias0 : bias1; i0 < bias1; i0 += kLogitThreads) {
                bool again = false;
                const int to = place_of(i0 + tid < bias1 ? __ldg(p.bias_ids + i0 + tid) : -1, again);
                again = again && to >= 0;
                if (!__syncthreads_or(again)) continue;
                for (int w = 0; w < kLogitThreads / 32; ++w) {
                    if (w == warp) {
                        for (uint32_t left = __ballot_sync(0xFFFFFFFFu, again); left; left &= left - 1) {
                            if (lane == __ffs(left) - 1) s.bias_sum[to] += __ldg(p.bias_values + i0 + tid);
                            __syncwarp();
                        }
                    }
                    __syncthreads();
                }
            }
        }
        __syncthreads();
        for (int e = tid; e < (n - z0 + dz - 1) / dz * count; e += kLogitThreads) {
            const int i = e / count, place = e - i * count, v = s.column[place], j = z0 + i * dz, row = lo + j;
            const float z = to_f32<T>(source(row)[v]);
            const bool gone = hidden(mask_at(s.mask[j]), v);
            target(row)[v] = from_f32<T>(gone ? -INFINITY : adjust(s, pen, c0, v, place, n, s.path[j], z));
        }
    }
    if (in_place) {
        __syncthreads();
        for (int j = z0; j < n; j += dz) stream(lo + j);
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
    // A request's rows are dealt out to several CTAs, each with counts of its own, until the SMs are full (32 requests of up to
    // 20 rows of 50257: 49 -> 27 us, one of 32 rows of 152064: 45 -> 10); a batch that fills them counts once a slice.
    const int64_t slices = (p.V + kSlice - 1) / kSlice, deals = (kFull + slices * p.B - 1) / (slices * p.B);
    const dim3 grid(static_cast<unsigned>(slices), p.B, static_cast<unsigned>(deals < p.k_max + 1 ? deals : p.k_max + 1));
    if (dtype == SPEC_F32) adjust_logits_kernel<float><<<grid, kLogitThreads, sizeof(Slice), s>>>(p);
    else adjust_logits_kernel<__nv_bfloat16><<<grid, kLogitThreads, sizeof(Slice), s>>>(p);
    return cudaGetLastError();
}

}  // namespace specv
