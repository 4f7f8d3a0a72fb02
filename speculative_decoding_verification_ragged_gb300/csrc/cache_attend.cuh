// cache_attend.cuh -- the kernel of the attention of packed verify rows over the
// 4-bit paged cache (include/spec_cache.h); cache_attend.cu has it plain,
// cache_attend_options.cu with the score options (each kernel's code stays small:
// what runs once a segment is fetched anew each time).
//
// For one request and kv head the step's query rows are columns of a matrix:
// column j * group + g is row j of query head h * group + g.  Over tiles of 128
// tokens
//     S^T = K Q^T          [tokens x columns]
//     P^T = 2^(S^T c - m)  m: a running reference per column
//     O^T += V^T P^T       [channels x columns]
// so that the cache is the A operand of both products: M is always full (128
// tokens, 128 channels), N is the handful of columns, and a row of A is one
// token's key or one channel's values -- a thread decodes a part of one row,
// straight from shared memory into tensor memory (e2m1 and e4m3 convert to f16
// in one instruction a pair, their product is exact in f16).
//
// P is f16: 2^(x + 11), x the score less its reference in log2 units.  The
// reference moves only when a score passes it by 2^4 (the accumulators and sums
// are rescaled then), so that P stays below 2^15 and keeps its 11 bits down to
// x = -25.  A tile with a visible weight below that takes the product with bf16
// operands instead (values exact in bf16 too, weights as a sum of two or three
// bf16 terms): small weights keep their bits, whatever the largest is.  (11 bits are
// enough for bf16 outputs: a second f16 term took 147 us over 128 ragged requests and
// 172 over 4 x 131071 tokens, against 139 and 163, and left the error against 64 bits
// where it is, 0.0016 to 0.0017 in norm, that of the outputs' own rounding.)
// bf16 queries are exact in f16 once scaled by a power of two; fp32 queries and
// the weights of fp32 outputs are a sum of two f16 (22 bits), and their products
// with V^T are added up tile by tile in fp32 registers (the tensor cores'
// accumulation truncates, which over a long cache would show in fp32).  Sums of
// weights are fp32, taken before any rounding.
//
// Bound by instruction issue and the latency of a tile's chain (scores, weights,
// values), not by HBM: a tile's 32 Ki codes are converted and stored to tensor
// memory against 18 KB fetched.  Four single tokens over 131071 tokens each (32 / 8
// heads of 128) take 163 us, 3.7 TB/s of cache, 55 % of the measured copy rate; 128
// requests of 2 to 5 rows over up to 4096 tokens, ragged, 139 us (2.2 TB/s).  Two CTAs
// an SM are what tensor memory holds (256 columns each); three operands of a tile in
// columns of their own (K, V^T, S) let each product run while the other operand is
// decoded (128 x 5 rows x 4096: 298 us, and 335 with one buffer for K and V^T, at
// the step that parted them).
#pragma once

#include "attend.cuh"

namespace specv {

namespace {

constexpr float kUnset = -1e30f;           // reference of a column that has seen nothing yet
constexpr float kHeadroom = 11.f;          // P = 2^(x + 11) ...
constexpr int kRun = 128;                  // tiles whose products tensor memory adds up (bf16 outputs)
constexpr int kMostMoves = 4;              // of the references for one tile
constexpr uint32_t kMostBits = 0x7800u;    // ... stays below 2^15 (f16 bits)
// V decoded to bf16 keeps f16's exponent bits, which stand for 2^-112 of the
// value there; the weights carry the 2^112
constexpr float kWideScale = 5.192296858534828e33f;

template <typename T, int D_, int NT_> struct Attn {
    using Type = T;
    static constexpr int D = D_, NT = NT_;
    static constexpr int NH = NT / 2;                          // columns of a thread
    static constexpr int PIECES = sizeof(T) == 4 ? 2 : 1;      // f16 terms of a query and of a weight
    static constexpr int WIDE = sizeof(T) == 4 ? 3 : 2;        // bf16 terms of a weight in a wide tile
    // exponent of the smallest weight with its bits in f16: a normal number; for
    // two terms 15 bits above the last place, 2^-25
    static constexpr float LEAST_EXP = sizeof(T) == 4 ? -10.f : -14.f;
    static constexpr uint32_t LEAST_BITS = sizeof(T) == 4 ? 0x1400u : 0x0400u;     // as f16 bits
    // D = 64 fills the 128 lanes of V^T with two halves of the tile's tokens,
    // each with its own columns of P^T; D = 256 takes two products of 128 channels
    static constexpr int HALVES = D == 64 ? 2 : 1;
    static constexpr int VM = D == 256 ? 2 : 1;
    static constexpr int VT = kTile / HALVES;                  // tokens of a V^T row
    static constexpr int A_COLS = D / 2;                       // tensor memory of a tile's K
    static constexpr int S_COLS = PIECES * NT;
    static constexpr int O_COLS = NT * HALVES * VM;
    static constexpr int V_COLS = D == 64 ? 32 : 64 * VM;      // tensor memory of a tile's V^T
    static constexpr int COLS = tmem_cols(A_COLS + V_COLS + S_COLS + O_COLS);
    static constexpr int CTAS = COLS <= 256 ? 2 : 1;
    static constexpr int Q_BYTES = query_bytes(D, NT);
    static constexpr int P_BYTES = kTile * NT * 2;             // a term of a tile's weights
    static constexpr int VS_BYTES = D / 16 * kTile * 2;        // a tile's scales of V as f16
    static constexpr int STAGE = 4 * block_bytes(D);
    static constexpr int OPERANDS = PIECES * Q_BYTES + WIDE * P_BYTES + 2 * VS_BYTES;
    static constexpr int STAGES = clamp_stages((smem_share(CTAS, 1024 + 60 * NT) - OPERANDS) / STAGE);
    static constexpr int NEED = OPERANDS + STAGES * STAGE;
    static constexpr int SMEM = NEED > smem_least(CTAS) ? NEED : smem_least(CTAS);
    static_assert(D != 64 || NT * D * 4 <= WIDE * P_BYTES, "the epilogue's exchange fits the weights' place");
};

// Scales of a tile's values as f16, tokens in pairs, [D/16][64]; the scale of a
// slot that does not exist is 0 (its bytes can be anything, NaN included).
template <int D>
__device__ __forceinline__ void value_scales(const uint8_t *tile, const int *nv, bool whole, uint32_t *vs)
{
    // 4 tokens a thread and group: 32 threads to a group
    const int word = threadIdx.x & 7, blk = threadIdx.x >> 3 & 3, g0 = threadIdx.x >> 5;
    if (D == 64 && g0 >= 4) return;
#pragma unroll
    for (int g = 0; g < D / 16; g += 8) {
        uint32_t s = *reinterpret_cast<const uint32_t *>(tile + blk * block_bytes(D) + v_scale_at(D) + (g0 + g) * kTok + 4 * word);
        if (!whole) {
            const int n = nv[blk] - 4 * word;
            s = n >= 4 ? s : (n <= 0 ? 0u : s & ((1u << 8 * n) - 1u));
        }
        *reinterpret_cast<uint2 *>(vs + (g0 + g) * 64 + blk * 16 + 2 * word) = make_uint2(e4m3x2(s), e4m3x2(s >> 16));
    }
}

// Scales of 0 for the tokens that the window hides from all columns (lit: a bit for
// each of a block's tokens that it does not hide).  Their weight is 0, but their bytes can be anything, NaN included.
template <int D> __device__ __forceinline__ void hide_values(const uint32_t *lit, uint32_t *vs)
{
#pragma unroll
    for (int i = threadIdx.x; i < D / 16 * 64; i += kAttnThreads) {
        const uint32_t two = lit[i % 64 / 16] >> (i % 16 * 2);
        vs[i] &= ((two & 1u) ? 0xFFFFu : 0u) | ((two & 2u) ? 0xFFFF0000u : 0u);
    }
}

// The values of one channel over the 32 tokens of a block -> 16 columns
template <int D, bool WIDE>
__device__ __forceinline__ void decode_values(const uint8_t *blk, int d, const uint32_t *vs, uint32_t taddr)
{
    const uint4 v = *reinterpret_cast<const uint4 *>(blk + v_codes_at(D) + d * 16);
    uint32_t r[16];
    decode16(v, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 s = *reinterpret_cast<const uint4 *>(vs + 4 * i);
        r[4 * i] = h2_mul(r[4 * i], s.x);
        r[4 * i + 1] = h2_mul(r[4 * i + 1], s.y);
        r[4 * i + 2] = h2_mul(r[4 * i + 2], s.z);
        r[4 * i + 3] = h2_mul(r[4 * i + 3], s.w);
    }
    if (WIDE)
#pragma unroll
        for (int i = 0; i < 16; ++i)      // f16 (no subnormals here: the smallest product is 2^-10) to bf16 bits
            r[i] = (r[i] >> 3 & 0x0FFF0FFFu) | (r[i] & 0x80008000u);
    tmem_st16(taddr, r);
}

// This warp's half of a tile's values into tensor memory
template <typename A, bool WIDE>
__device__ __forceinline__ void decode_tile_values(const uint8_t *stage, const uint32_t *vs, uint32_t taddr)
{
    constexpr int D = A::D;
    const int half = threadIdx.x / 128, row = threadIdx.x % 128;
    if constexpr (D == 64) {
        // lanes 0..63: channels over tokens 0..63, lanes 64..127: over 64..127
        const int blk = row / 64 * 2 + half, d = row % 64;
        decode_values<D, WIDE>(stage + blk * block_bytes(D), d, vs + d / 16 * 64 + blk * 16, taddr + half * 16);
    } else {
        const int m = D == 256 ? half : 0, d = m * 128 + row;
#pragma unroll
        for (int i = 0; i < (D == 256 ? 4 : 2); ++i) {
            const int blk = D == 256 ? i : half * 2 + i;
            decode_values<D, WIDE>(stage + blk * block_bytes(D), d, vs + d / 16 * 64 + blk * 16, taddr + m * 64 + blk * 16);
        }
    }
}

// O^T += V^T P^T over the tile's tokens (one warp issues); the smaller terms of
// P first, as in issue_scores
template <typename A, bool WIDE>
__device__ __forceinline__ void issue_values(uint32_t o_addr, uint32_t v_addr, uint32_t ps, bool accumulate)
{
    constexpr int PC = WIDE ? A::WIDE : A::PIECES;
#pragma unroll
    for (int m = 0; m < A::VM; ++m)
#pragma unroll
        for (int pc = PC - 1; pc >= 0; --pc)
#pragma unroll
            for (int q = 0; q < A::VT / 16; ++q)
                mma_f16(o_addr + m * A::NT, v_addr + m * 64 + q * 8,
                        smem_desc(ps + pc * A::P_BYTES + q * 256, 128, A::VT * 16),
                        mma_f16_desc(A::NT * A::HALVES, true, WIDE), accumulate || pc < PC - 1 || q > 0);
}

__device__ __forceinline__ uint32_t h2_max(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t h2_min(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Sum over the 32 lanes of each of N values: lane l gets the sum of value
// l * N / 32 (the values halve at each of the first exchanges).
template <int N> __device__ __forceinline__ float lane_sums(float (&v)[N])
{
    const int lane = threadIdx.x & 31;
    int m = 16;
#pragma unroll
    for (int k = N / 2; k >= 1; k >>= 1, m >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < k; ++i) {
            const float send = up ? v[i] : v[i + k], keep = up ? v[i + k] : v[i];
            v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, m);
        }
    }
    float s = v[0];
#pragma unroll
    for (; m >= 1; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
    return s;
}

// Column constants of a CTA (shared memory)
template <int NT> struct Columns {
    float ref[NT];              // headroom - reference: x + 11 = score + ref
    float mult[NT];             // raw product -> score (log2 units)
    float slope[NT];            // distance slope (log2 units)
    float factor[NT];           // rescale of a column whose reference moved
    float sum[NT];
    int own[NT], pos[NT];       // last slot the column sees, its position
    float run[NT];              // ref of the sums over the runs of tiles so far
    int fresh[NT];              // reference: 0 set, 1 to be set to the tile's maximum, 2 nothing seen yet
    float red[4][NT];
};

// What a thread's token of a tile is.
struct Token {
    int slot, pos;
    bool live;                  // it exists
    bool edge;                  // some row may not see some token of the quarter
};

// Scores of a token in log2 units, the column's reference added (x + headroom),
// for this thread's columns from q0 on; hidden ones -inf.
template <typename A, bool OPT>
__device__ __forceinline__ void token_scores(const AttnParams &p, const Job &w, const Columns<A::NT> &cs, uint32_t s_addr,
                                             int q0, const Token &t, float (&v)[A::NH])
{
    constexpr int N = A::NH;
    load_products<N, A::NT, A::PIECES>(s_addr + q0, v);
    if constexpr (!OPT) {
#pragma unroll
        for (int q = 0; q < N; q += 4) {
            const float4 m = *reinterpret_cast<const float4 *>(&cs.mult[q0 + q]);
            const float4 r = *reinterpret_cast<const float4 *>(&cs.ref[q0 + q]);
            v[q] = fmaf(v[q], m.x, r.x);
            v[q + 1] = fmaf(v[q + 1], m.y, r.y);
            v[q + 2] = fmaf(v[q + 2], m.z, r.z);
            v[q + 3] = fmaf(v[q + 3], m.w, r.w);
        }
        if (t.edge) {
#pragma unroll
            for (int q = 0; q < N; ++q)
                v[q] = t.live && t.slot <= cs.own[q0 + q] && q0 + q < w.ncols ? v[q] : -INFINITY;
        }
    } else {
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] *= cs.mult[q0 + q];
        if (p.cap > 0.f) {
            const float cap = p.cap * kLog2e, rcap = cap_reciprocal(cap);
#pragma unroll
            for (int q = 0; q < N; ++q) v[q] = cap_score<A::PIECES == 2>(v[q], cap, rcap);
        }
        const bool always = t.live && (p.window <= 0 || t.slot < p.prefix);
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int dist = cs.pos[q0 + q] - t.pos;
            const bool see = t.slot <= cs.own[q0 + q] && (always || (t.live && dist < p.window)) && q0 + q < w.ncols;
            v[q] = see ? v[q] - cs.slope[q0 + q] * static_cast<float>(dist) + cs.ref[q0 + q] : -INFINITY;
        }
    }
}

// Set the references to the tile's maxima where those are larger or the first, and
// the factors that take the sums and results along.  x: this thread's scores.
// Returns whether a column came to see its first slot: its scores were taken with
// no reference, and have to be taken again to set one.
template <typename A>
__device__ __forceinline__ bool move_references(const Job &w, Columns<A::NT> &cs, const float (&x)[A::NH])
{
    const int tid = threadIdx.x, lane = tid & 31, quarter = tid >> 5 & 3, half = tid >> 7;
    float mine = 0.f;
#pragma unroll
    for (int q = 0; q < A::NH; ++q) {
        const float m = warp_max_f32(x[q]);
        if (lane == q) mine = m;
    }
    if (lane < A::NH) cs.red[quarter][half * A::NH + lane] = mine;
    csync();
    bool again = false;
    if (tid < A::NT) {
        float factor = 1.f;
        if (tid < w.ncols) {
            const float r = fmaxf(fmaxf(cs.red[0][tid], cs.red[1][tid]), fmaxf(cs.red[2][tid], cs.red[3][tid]));
            const float ref = cs.ref[tid];
            const int fresh = cs.fresh[tid];
            if (fresh == 2) {
                again = r > -INFINITY;
                if (again) {
                    cs.fresh[tid] = 1;
                    cs.ref[tid] = kHeadroom;
                }
            } else if (r == -INFINITY) {
                if (fresh == 1) {
                    cs.fresh[tid] = 2;
                    cs.ref[tid] = kHeadroom - kUnset;
                }
            } else if (fresh == 1 || r > kHeadroom) {
                cs.fresh[tid] = 0;
                cs.ref[tid] = kHeadroom - (r - ref);
                if (fresh == 0) factor = ex2(kHeadroom - r);
            }
        }
        cs.factor[tid] = factor;
    }
    return csync_count(again);
}

// Rescale this thread's columns of the results in tensor memory
template <typename A>
__device__ __forceinline__ void rescale_results(const Columns<A::NT> &cs, uint32_t o_addr)
{
    const int half = threadIdx.x >> 7;
#pragma unroll 1
    for (int q0 = half * A::O_COLS / 2; q0 < (half + 1) * A::O_COLS / 2; q0 += 8) {
        uint32_t r[8];
        tmem_ld<8>(o_addr + q0, r);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 8; ++q) r[q] = __float_as_uint(__uint_as_float(r[q]) * cs.factor[(q0 + q) % A::NT]);
        tmem_st8(o_addr + q0, r);
    }
    tmem_wait_st();
}

// The work of a call, laid out in one line: request by request, kv head by kv
// head, column tile by column tile ("tasks"); a task has kTaskUnits units for what
// it costs by itself (its queries, its first references, its results), then one
// for each visible tile.  CTA i of `grid` (no more than there are units: none is
// empty) takes [i * total / grid, (i + 1) * total / grid): whatever the lengths, the
// CTAs end together, and a task is split at most where two CTAs meet.  A CTA that
// gets a task's own units only leaves it to the next one.
// (128 requests x 5 rows, ragged up to 4096 tokens, with 2, 4, 7 and 11 units a
// task: 168, 145, 139 and 144 us; 16 requests of fp32 with a window of 3000
// positions: 54, 56, 60 and 63.)
constexpr int kTaskUnits = 6;

struct Layout {
    int grid;                   // CTAs at most, all resident at once
};

// The workspace: arrivals at each split task, by the CTA where it begins, then the
// parts.  The arrivals have one place for calls of all shapes, so that calls of
// different shapes can share a workspace.
constexpr int kSms = 152, kTicketBytes = 2 * kSms * 4 + 64;
static_assert(kTicketBytes % 16 == 0, "the parts are read by vectors");

__device__ __forceinline__ int64_t range_start(int64_t total, int grid, int i) { return total * i / grid; }
// the CTA whose range holds unit t
__device__ __forceinline__ int range_of(int64_t total, int grid, int64_t t)
{
    return static_cast<int>(((t + 1) * grid - 1) / total);
}

// What a CTA does of a task: tiles first .. first + n - 1 of its visible ones (none:
// the task has none, its rows are zeros).
struct Segment {
    Job w;
    int first, n;               // n = -1: the range is done
    int64_t begin;              // the task's first unit in the line
};

// First slot of the k-th tile that a segment visits.  With options the newest come
// first, so that a distance bias sets the references once and not anew with every
// tile (16 requests with biases: 57 -> 46 us; without options the order from the
// first is the faster, 138 against 146 us over 128 ragged requests).
template <bool OPT> __device__ __forceinline__ int tile_slot(const Segment &s, int k)
{
    return step_slot<kTile>(s.w, OPT ? s.first + s.n - 1 - k : s.first + k);
}

// A place in the line: task `task` (head * column tiles + column tile) of
// request w.b, unit `unit` of it.
template <int NT> struct Cursor {
    Job w;
    int64_t at, end;            // units of the line: here, and where this CTA's range ends
    int qt, tasks, task, unit;

    __device__ __forceinline__ void start(const CacheView &c, int group)
    {
        qt = (w.n * group + NT - 1) / NT;
        tasks = c.H * qt;
    }
    __device__ __forceinline__ int units() const { return kTaskUnits + w.nsteps; }
    // The next segment of the range; false: there is none.
    __device__ __forceinline__ bool take(const CacheView &c, const AttnParams &p, int group, Segment &s)
    {
        for (;;) {
            if (at >= end) return false;
            const int have = static_cast<int>(min(static_cast<int64_t>(units() - unit), end - at));
            s.w = w;
            s.w.h = task / qt;
            s.w.col0 = task % qt * NT;
            s.w.ncols = min(w.n * group - s.w.col0, NT);
            s.first = max(unit - kTaskUnits, 0);
            s.n = max(unit + have - kTaskUnits - s.first, 0);
            s.begin = at - unit;
            // worth a segment: tiles, or the last unit of a task without any
            const bool some = s.n > 0 || (w.nsteps == 0 && unit + have == kTaskUnits);
            at += have;
            unit = 0;
            if (at < end && ++task == tasks) {
                task = 0;
                do {
                    if (++w.b >= c.B) {               // (the line ends with the last request)
                        at = end;
                        break;
                    }
                } while (!load_job<kTile>(c, p, w, nullptr));
                if (at < end) start(c, group);
            }
            if (some) return true;
        }
    }
};

// Where this CTA's range begins: every thread takes a request at a time, a scan
// of their units places them.
template <int NT>
__device__ __forceinline__ int64_t find_range(const CacheView &c, const AttnParams &p, const Layout &lay, int group,
                                              int &grid, int64_t &t0, Job &job, int64_t &off)
{
    constexpr int N = kAttnThreads + 64;
    __shared__ int64_t sums[N / 32 + 1], offset;
    __shared__ Job found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Job w;
    const auto weight = [&](int b, bool report) {
        w.b = b;
        if (b >= c.B || !load_job<kTile>(c, p, w, report && blockIdx.x == 0 ? p.status : nullptr)) return static_cast<int64_t>(0);
        return static_cast<int64_t>(c.H) * ((w.n * group + NT - 1) / NT) * (kTaskUnits + w.nsteps);
    };
    // inclusive scan over the CTA; `all`: its total
    const auto scan = [&](int64_t v, int64_t &all) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v += y;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        int64_t before = 0;
        all = 0;
#pragma unroll
        for (int i = 0; i < N / 32; ++i) {
            before += i < warp ? sums[i] : 0;
            all += sums[i];
        }
        return before + v;
    };
    int64_t total, mine = weight(tid, true), at = scan(mine, total);
    int64_t part = total;                         // of the N requests at hand
    const Job own = w;                            // of the first N requests
    for (int b = N; b < c.B; b += N) {
        int64_t v = weight(b + tid, true);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        __syncthreads();
        if (lane == 0) sums[warp] = v;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N / 32; ++i) total += sums[i];
    }
    grid = static_cast<int>(min(static_cast<int64_t>(lay.grid), total));
    if (static_cast<int>(blockIdx.x) >= grid) return total;
    t0 = range_start(total, grid, blockIdx.x);
    int64_t base = 0;
    w = own;
    for (int b = 0;; ) {
        if (at - mine + base <= t0 && t0 < at + base) {
            found = w;
            offset = t0 - (at - mine + base);
        }
        base += part;
        b += N;
        if (b >= c.B || base > t0) break;
        mine = weight(b + tid, false);
        at = scan(mine, part);
    }
    __syncthreads();
    job = found;
    off = offset;
    return total;
}

// Warps 0..7 decode, weigh and store; warp 8 issues the products, warp 9 fetches
// tiles, ahead over the whole range.  Per tile the eight warps wait for S^T, turn it
// into weights (one barrier: do the references hold?), decode the next tile's
// keys, then this tile's values; each product runs while they decode the other
// operand, and they meet the other two at mbarriers only.
template <typename T, int D, int NT, bool OPT>
__global__ void __launch_bounds__(kAttnThreads + 64, (Attn<T, D, NT>::CTAS))
attend_kernel(const CacheView c, const AttnParams p, const Layout lay)
{
    using A = Attn<T, D, NT>;
    constexpr int NH = A::NH, kIssuer = 8, kLoader = 9, kSegs = 4;
    constexpr bool kPromote = A::PIECES == 2;
    constexpr int OR = kPromote ? NH * A::VM : 1;     // fp32: results kept in registers
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *qs = smem, *ps = qs + A::PIECES * A::Q_BYTES;
    uint32_t *vs = reinterpret_cast<uint32_t *>(ps + A::WIDE * A::P_BYTES);
    uint8_t *stages = ps + A::WIDE * A::P_BYTES + 2 * A::VS_BYTES;
    __shared__ __align__(16) Columns<NT> cs;
    __shared__ __align__(8) uint64_t full[A::STAGES], empty[A::STAGES], seg_full[kSegs], seg_empty[kSegs], k_bar, p_bar,
        s_bar, o_bar;
    __shared__ Segment segs[kSegs];                   // from the loader to the eight warps
    __shared__ uint32_t tmem_base, arrived;
    // what the eight warps tell the issuer: with keys, kFirst / kLast of a segment
    // or kEnd; with weights, whether they are those of a wide tile
    constexpr int kFirst = 1, kLast = 2, kEnd = 4;
    __shared__ int keys_are, weights_wide;
    __shared__ __align__(16) int nv[A::STAGES][4], pages[A::STAGES][4];
    __shared__ __align__(16) uint32_t lit[2][4];      // tokens of a tile that the window does not hide from all columns
    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const int group = p.Hq / c.H;

    if (warp == kIssuer && lane == 0) {
        for (int i = 0; i < A::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 8);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], 8);
        }
        mbar_init(&k_bar, 8);
        mbar_init(&p_bar, 8);
        mbar_init(&s_bar, 1);
        mbar_init(&o_bar, 1);
        fence_mbar_init();
    }
    Cursor<NT> cur;
    int grid;
    int64_t off;
    const int64_t total = find_range<NT>(c, p, lay, group, grid, cur.at, cur.w, off);
    if (static_cast<int>(blockIdx.x) >= grid) return;
    if (warp == 0) tmem_alloc(&tmem_base, A::COLS);
    __syncthreads();
    tmem_fence_after();
    const uint32_t a_t = __shfl_sync(0xFFFFFFFFu, tmem_base, 0), v_t = a_t + A::A_COLS, s_t = v_t + A::V_COLS, o_t = s_t + A::S_COLS;
    bool fail = false;

    if (warp == kLoader) {
        // segments to the eight warps, their tiles into the ring, the page ids of the
        // tile after asked for
        cur.end = range_start(total, grid, blockIdx.x + 1);
        cur.start(c, group);
        cur.task = static_cast<int>(off / cur.units());
        cur.unit = static_cast<int>(off % cur.units());
        Segment seg = {};
        int ring = 0, sr = 0, k = 0;
        uint32_t phase = 1, s_phase = 1;              // (a stage is empty at first)
        bool any = true;
        Fetch next;
        const auto ask_next = [&] {
            while (any && k == seg.n) {
                any = cur.take(c, p, group, seg) && !fail;
                if (!any) seg.n = -1;
                k = 0;
                wait_or_fail(&seg_empty[sr], s_phase, fail);
                if (lane == 0) {
                    segs[sr] = seg;
                    mbar_arrive(&seg_full[sr]);
                }
                __syncwarp();
                if (++sr == kSegs) {
                    sr = 0;
                    s_phase ^= 1;
                }
            }
            if (any) next = ask_pages<OPT>(c, p, seg.w, seg.w.h, tile_slot<OPT>(seg, k++));
        };
        ask_next();
        while (any && !fail) {
            wait_or_fail(&empty[ring], phase, fail);
            load_tile<block_bytes(D), OPT>(c, p, seg.w, next, stages + ring * A::STAGE, &full[ring], nv[ring],
                                      OPT ? pages[ring] : nullptr);
            if (++ring == A::STAGES) {
                ring = 0;
                phase ^= 1;
            }
            ask_next();
        }
        return;
    }
    if (warp == kIssuer) {
        // products in the order their operands come
        const uint32_t q_addr = smem_addr(qs), p_addr = smem_addr(ps);
        int g = 0, p_count = 0, now = 0, run = 0;
        const auto scores = [&] {
            wait_or_fail(&k_bar, g++ & 1, fail);
            tmem_fence_after();
            now = __shfl_sync(0xFFFFFFFFu, fail ? kEnd : *reinterpret_cast<volatile int *>(&keys_are), 0);
            if (now == kEnd) return;
            issue_scores<D, NT, A::PIECES>(s_t, a_t, q_addr);
            mma_commit(&s_bar);
        };
        scores();
        while (now != kEnd) {
            const int here = now;
            if (!(here & kLast)) scores();
            wait_or_fail(&p_bar, p_count++ & 1, fail);
            tmem_fence_after();
            const bool wide = __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<volatile int *>(&weights_wide), 0);
            if (here & kFirst) run = 0;               // (tiles of the segment so far)
            const bool accumulate = !kPromote && run % kRun != 0;
            ++run;
            if (wide) issue_values<A, true>(o_t, v_t, p_addr, accumulate);
            else issue_values<A, false>(o_t, v_t, p_addr, accumulate);
            mma_commit(&o_bar);
            if (here & kLast) scores();
        }
        return;
    }

    const int quarter = warp & 3, half = warp >> 2, tok = tid & 127;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    // where this thread's columns of the result lie (D = 64: those of its tokens)
    const uint32_t o_mine = o_t + lane_off + half * NH + (D == 64 && quarter >= 2 ? NT : 0);
    constexpr int PN8 = A::VT * 16;
    uint8_t *const p_mine = ps + (tok / A::VT * (NT / 8) + half * (NH / 8)) * PN8 + tok % A::VT * 16;

    float l[NH], acc[OR];
    bool pending = false;                             // a product with V^T is under way
    uint32_t s_phase = 0, o_phase = 0, ring_phase = 0;
    int ring = 0, buf = 0;                            // stage, and scales' place, of the tile whose values come next
    // wait for the product with V^T under way; fp32: add its result up
    const auto finish_values = [&] {
        pending = false;
        wait_or_fail(&o_bar, o_phase, fail);
        o_phase ^= 1;
        tmem_fence_after();
        if constexpr (kPromote) {
#pragma unroll
            for (int m = 0; m < A::VM; ++m) {
                float r[NH];
                tmem_ld<NH>(o_mine + m * NT, reinterpret_cast<uint32_t *>(r));
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < NH; ++q) acc[m * NH + q] += r[q];
            }
        }
    };
    // A task that this CTA has only a part of leaves a partial result, [NT][D]
    // fp32 and [NT] (reference, sum), in slot 2 i (it began before the range) or
    // 2 i + 1 (it goes on after it); until then a segment's sums over runs of tiles lie
    // in its slot (2 i + 1 for one that is not split), each in the thread that owns it.
    float *const part_all = reinterpret_cast<float *>(static_cast<uint8_t *>(p.ws) + kTicketBytes);
    const auto sums_at = [&](const Segment &g) {
        return part_all + (2 * static_cast<int64_t>(blockIdx.x) + (g.first > 0 ? 0 : 1)) * NT * D;
    };
    // what takes a column's sums along to its present reference
    const auto run_factor = [&](int q) { return ex2(cs.ref[q] - cs.run[q]); };
    // D = 64: the upper lanes hold the second half of the tokens, which the lower ones
    // add to theirs (in P's place); false for a thread that has no result then
    const auto join_halves = [&](float (&r)[NH]) {
        if constexpr (D == 64) {
            float *const xch = reinterpret_cast<float *>(ps);
            if (quarter >= 2)
#pragma unroll
                for (int q = 0; q < NH; ++q) xch[(half * NH + q) * 64 + tok - 64] = r[q];
            csync();
            if (quarter >= 2) return false;
#pragma unroll
            for (int q = 0; q < NH; ++q) r[q] += xch[(half * NH + q) * 64 + tok];
        }
        return true;
    };
    // this thread's columns of the results in tensor memory
    const auto results = [&](int m, float (&r)[NH]) {
        tmem_ld<NH>(o_mine + m * NT, reinterpret_cast<uint32_t *>(r));
        tmem_wait_ld();
        return join_halves(r);
    };
    int pos = 0;                                      // of this thread's token of the tile whose keys came last
    // the keys of the tile in stage `st` (in phase `phase` of the ring), first slot `slot0`
    const auto keys = [&](int st, uint32_t phase, int slot0, int what) {
        wait_or_fail(&full[st], phase, fail);
        if (OPT) {
            pos = slot0 + tok;
            // (asked for here, a tile ahead of its use)
            if (p.slot_pos && lane < nv[st][quarter])
                pos = __ldg(p.slot_pos + static_cast<int64_t>(pages[st][quarter]) * c.page_tokens + pos % c.page_tokens);
        }
        decode_keys<D>(stages + st * A::STAGE + quarter * block_bytes(D), a_t + lane_off);
        if (tid == 0) keys_are = what;
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_bar);
    };

    int sr = 0;
    uint32_t seg_phase = 0;
    for (;;) {
        wait_or_fail(&seg_full[sr], seg_phase, fail);
        const Segment &seg = segs[sr];
        const Job &w = seg.w;
        const int n = seg.n;
        if (csync_count(fail || n < 0)) break;
        const float gk = c.k_scale ? c.k_scale[w.h] : 1.f, gv = c.v_scale ? c.v_scale[w.h] : 1.f;
        if (tid < NT) {
            const int col = w.col0 + tid, j = min(col / group, w.n - 1);
            const int own = w.len > 0 ? w.len - w.n + j : -1;
            cs.own[tid] = own;
            cs.pos[tid] = own >= 0 ? slot_position(c, p, w.b, own) : 0;
            cs.slope[tid] = p.slopes && tid < w.ncols ? p.slopes[w.h * group + col % group] * kLog2e : 0.f;
            cs.ref[tid] = kHeadroom;                  // (a padded column's results are unused)
            cs.fresh[tid] = 1;
        }
        QueryStage<T, D, NT, A::PIECES> queries;
        queries.place(p, w, group);
        queries.stage(p, static_cast<int64_t>(w.h) * group * p.q_head, p.scale_log2 * gk, qs, cs.mult);
        fence_proxy_async_smem();
        csync();
#pragma unroll
        for (int i = 0; i < NH; ++i) l[i] = 0.f;
#pragma unroll
        for (int i = 0; i < OR; ++i) acc[i] = 0.f;
        const int own_first = cs.own[0];
        if (n > 0) keys(ring, ring_phase, tile_slot<OPT>(seg, 0), kFirst | (n == 1 ? kLast : 0));
        // tiles in runs of kRun (fp32: all in one).  (Jumped back to: a loop around took
        // 166 us over 4 x 131071 tokens, and 140.3 over 128 ragged requests, against 163
        // and 139.0, as without runs.)
        int k = 0, stop = kPromote ? n : min(n, kRun);
    next_run:
        for (; k < stop; ++k) {
            const uint8_t *stage = stages + ring * A::STAGE;
            uint32_t *vsk = vs + buf * (A::VS_BYTES / 4);
            const int slot0 = tile_slot<OPT>(seg, k);
            Token t;
            const int4 n4 = *reinterpret_cast<const int4 *>(nv[ring]);
            const bool whole = (n4.x & n4.y & n4.z & n4.w) == kTok;      // (each at most 32)
            t.slot = slot0 + tok;
            t.pos = pos;
            t.live = whole || lane < nv[ring][quarter];
            t.edge = !whole || slot0 + kTile - 1 > own_first;
            value_scales<D>(stage, nv[ring], whole, vsk);
            uint64_t *const done = &empty[ring];
            if (++ring == A::STAGES) {
                ring = 0;
                ring_phase ^= 1;
            }
            wait_or_fail(&s_bar, s_phase, fail);
            s_phase ^= 1;
            tmem_fence_after();
            if (OPT && p.window > 0 && half == 0) {
                // (the first column's row sees no later slots than the others, and no fewer)
                const bool dark = own_first >= 0 && t.slot >= p.prefix &&
                                  t.pos <= static_cast<int64_t>(cs.pos[0]) - p.window;
                const uint32_t seen = __ballot_sync(0xFFFFFFFFu, !dark);
                if (lane == 0) lit[buf][quarter] = seen;
            }
            float v[NH], x[NH];
            uint32_t hi[NH / 2];
            // weights, and whether they are fit for f16: none beyond 2^15 (the reference
            // has to move) and no visible one without its bits (1: too large, 2: too small)
            const auto weigh = [&] {
                token_scores<A, OPT>(p, w, cs, s_t + lane_off, half * NH, t, x);
#pragma unroll
                for (int q = 0; q < NH; ++q) v[q] = ex2(x[q]);
#pragma unroll
                for (int q = 0; q < NH / 2; ++q) hi[q] = pack_h2(v[2 * q], v[2 * q + 1]);
                uint32_t most = hi[0], least = hi[0];
#pragma unroll
                for (int q = 1; q < NH / 2; ++q) {
                    most = h2_max(most, hi[q]);
                    least = h2_min(least, hi[q]);
                }
                // (weights are positive: their bits compare as they do)
                int unfit = max(most >> 16, most & 0xFFFFu) > kMostBits ? 1 : 0;
                if (t.edge || OPT) {
                    float low = INFINITY;
#pragma unroll
                    for (int q = 0; q < NH; ++q) low = fminf(low, x[q] == -INFINITY ? INFINITY : x[q]);
                    unfit |= low < A::LEAST_EXP ? 2 : 0;
                } else {
                    unfit |= min(least >> 16, least & 0xFFFFu) < A::LEAST_BITS ? 2 : 0;
                }
                return unfit;
            };
            // (a segment's first tile sets the references, whatever it holds; three moves
            // are the most that numbers need, so that NaN or infinite ones end as well)
            bool wide = false, move = k == 0;
            for (int moves = 0;; ++moves) {
                const int unfit = weigh();
                if (!move) {
                    if (!csync_count(unfit)) break;
                    wide = !csync_count(unfit & 1);
                    if (wide) break;
                }
                if (moves == kMostMoves) break;
                move = move_references<A>(w, cs, x);
                if (k == 0) continue;
                if (pending) finish_values();
#pragma unroll
                for (int q = 0; q < NH; ++q) l[q] *= cs.factor[half * NH + q];
                if (kPromote) {
#pragma unroll
                    for (int q = 0; q < OR; ++q) acc[q] *= cs.factor[half * NH + q % NH];
                } else {
                    rescale_results<A>(cs, o_t + lane_off);
                }
            }
            if (OPT && p.window > 0) {
                // (the same for all: a barrier lies between)
                const uint4 seen = *reinterpret_cast<const uint4 *>(lit[buf]);
                if ((seen.x & seen.y & seen.z & seen.w) != 0xFFFFFFFFu) {
                    hide_values<D>(lit[buf], vsk);
                    csync();
                }
            }
            // S^T is read, the keys' columns are free: on to the next tile's keys
            if (k + 1 < n) keys(ring, ring_phase, tile_slot<OPT>(seg, k + 1), k + 2 == n ? kLast : 0);
            if (pending) finish_values();             // V^T's columns and P are free
            // weights: sums in fp32, the operand 8 columns of this token per store
#pragma unroll
            for (int q = 0; q < NH; ++q) l[q] += v[q];
            if (!wide) {
#pragma unroll
                for (int q0 = 0; q0 < NH; q0 += 8) {
                    const uint32_t *h = hi + q0 / 2;
                    *reinterpret_cast<uint4 *>(p_mine + q0 / 8 * PN8) = make_uint4(h[0], h[1], h[2], h[3]);
                    if (A::PIECES == 2) {
                        uint32_t lo[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float2 y = h2_float2(h[q]);
                            lo[q] = pack_h2(v[q0 + 2 * q] - y.x, v[q0 + 2 * q + 1] - y.y);
                        }
                        *reinterpret_cast<uint4 *>(p_mine + A::P_BYTES + q0 / 8 * PN8) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
            } else {
#pragma unroll
                for (int q = 0; q < NH; ++q) v[q] *= kWideScale;
#pragma unroll 1
                for (int pc = 0; pc < A::WIDE; ++pc) {
#pragma unroll
                    for (int q0 = 0; q0 < NH; q0 += 8) {
                        uint32_t term[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float &a = v[q0 + 2 * q], &b = v[q0 + 2 * q + 1];
                            term[q] = pack_bf2(a, b);
                            a -= bf_lo(term[q]);
                            b -= bf_hi(term[q]);
                        }
                        *reinterpret_cast<uint4 *>(p_mine + pc * A::P_BYTES + q0 / 8 * PN8) =
                            make_uint4(term[0], term[1], term[2], term[3]);
                    }
                }
            }
            if (!wide) decode_tile_values<A, false>(stage, vsk, v_t + lane_off);
            else decode_tile_values<A, true>(stage, vsk, v_t + lane_off);
            if (tid == 0) weights_wide = wide;
            __syncwarp();
            if (lane == 0) mbar_arrive(done);         // the stage is read
            tmem_wait_st();
            tmem_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_bar);
            buf ^= 1;
            pending = true;
        }
        if (pending) finish_values();
        if (!kPromote && k < n) {
            // a run's products to the sums, before the next one's take their place
#pragma unroll 1
            for (int m = 0; m < A::VM; ++m) {
                float r[NH];
                if (!results(m, r)) continue;
                float *const to = sums_at(seg) + half * NH * D + m * 128 + tok;
#pragma unroll
                for (int q = 0; q < NH; ++q) to[q * D] = k == kRun ? r[q] : r[q] + to[q * D] * run_factor(half * NH + q);
            }
            csync();                                  // (P's place is free again)
            if (tid < NT) cs.run[tid] = cs.ref[tid];
            stop = min(n, k + kRun);
            goto next_run;
        }

        // sums over the tiles' tokens (= lanes and quarters)
        {
            const float s = lane_sums<NH>(l);
            if (lane % (32 / NH) == 0) cs.red[quarter][half * NH + lane / (32 / NH)] = s;
        }
        if (csync_count(fail)) break;
        if (tid < NT) cs.sum[tid] = (cs.red[0][tid] + cs.red[1][tid]) + (cs.red[2][tid] + cs.red[3][tid]);
        csync();

        const bool head = seg.first > 0, split = head || seg.first + n < w.nsteps;
        float2 *const ml_all = reinterpret_cast<float2 *>(part_all + static_cast<int64_t>(lay.grid) * 2 * NT * D);
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (head ? 0 : 1);
        const auto out_row = [&](int q) {
            const int col = w.col0 + q;
            return static_cast<int64_t>(w.lo + col / group) * p.Hq + w.h * group + col % group;
        };
#pragma unroll
        for (int m = 0; m < A::VM; ++m) {
            float r[NH] = {};
            if constexpr (kPromote) {
#pragma unroll
                for (int q = 0; q < NH; ++q) r[q] = acc[m * NH + q];
                if (!join_halves(r)) continue;
            } else {
                if (n > 0 ? !results(m, r) : D == 64 && quarter >= 2) continue;
                if (n > kRun)
#pragma unroll
                    for (int q = 0; q < NH; ++q) r[q] += sums_at(seg)[(half * NH + q) * D + m * 128 + tok] * run_factor(half * NH + q);
            }
            const int d = m * 128 + tok;
#pragma unroll
            for (int q = 0; q < NH; ++q) {
                const int col = half * NH + q;
                if (col >= w.ncols) continue;
                if (split) {
                    part_all[(slot * NT + col) * D + d] = r[q];
                } else {
                    const float ls = cs.sum[col];
                    static_cast<T *>(p.out)[out_row(col) * D + d] = from_f32<T>(ls > 0.f ? r[q] * (gv / ls) : 0.f);
                }
            }
        }
        if (tid < w.ncols) {
            const float m = kHeadroom - cs.ref[tid], ls = cs.sum[tid];
            if (split) ml_all[slot * NT + tid] = make_float2(m, ls);
            else if (p.lse) p.lse[out_row(tid)] = ls > 0.f ? (m - kHeadroom + log2f(ls)) * kLn2 : -INFINITY;
        }
        if (split) {
            // the CTA that arrives last joins the parts, in the line's order
            const int64_t tile0 = seg.begin + kTaskUnits;
            const int c0 = range_of(total, grid, tile0), c1 = range_of(total, grid, tile0 + w.nsteps - 1);
            uint32_t *ticket = static_cast<uint32_t *>(p.ws) + c0;     // (one task at most goes on after a range)
            csync();
            if (tid == 0) {
                fence_acq_rel_gpu();
                arrived = atomicAdd(ticket, 1u);
                fence_acq_rel_gpu();
            }
            csync();
            if (arrived == static_cast<uint32_t>(c1 - c0)) {
                if (tid == 0) *ticket = 0u;
                const int parts = c1 - c0 + 1;
                const auto slot_of = [&](int s) { return 2 * static_cast<int64_t>(c0 + s) + (s == 0 ? 1 : 0); };
                // a thread per column: the common reference, the sum
                if (tid < w.ncols) {
                    float M = kUnset, L = 0.f;
#pragma unroll 4
                    for (int s = 0; s < parts; ++s) {
                        const float2 x = __ldcg(ml_all + slot_of(s) * NT + tid);
                        if (x.y > 0.f) M = fmaxf(M, x.x);
                    }
#pragma unroll 4
                    for (int s = 0; s < parts; ++s) {
                        const float2 x = __ldcg(ml_all + slot_of(s) * NT + tid);
                        if (x.y > 0.f) L += ex2(x.x - M) * x.y;
                    }
                    cs.factor[tid] = M;
                    cs.sum[tid] = L > 0.f ? gv / L : 0.f;
                    if (p.lse) p.lse[out_row(tid)] = L > 0.f ? (M - kHeadroom + log2f(L)) * kLn2 : -INFINITY;
                }
                csync();
                // a thread per four channels of a column
                for (int e = tid; e < w.ncols * (D / 4); e += kAttnThreads) {
                    const int col = e / (D / 4), d = e % (D / 4) * 4;
                    const float M = cs.factor[col];
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int s = 0; s < parts; ++s) {
                        const float2 x = __ldcg(ml_all + slot_of(s) * NT + col);
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(part_all + (slot_of(s) * NT + col) * D + d));
                        const float f = x.y > 0.f ? ex2(x.x - M) : 0.f;
                        o.x += f * v.x;
                        o.y += f * v.y;
                        o.z += f * v.z;
                        o.w += f * v.w;
                    }
                    T *to = static_cast<T *>(p.out) + out_row(col) * D + d;
                    const float g = cs.sum[col];
                    to[0] = from_f32<T>(o.x * g);
                    to[1] = from_f32<T>(o.y * g);
                    to[2] = from_f32<T>(o.z * g);
                    to[3] = from_f32<T>(o.w * g);
                }
            }
        }
        tmem_fence_before();
        csync();                                      // the column constants and P are free
        if (lane == 0) mbar_arrive(&seg_empty[sr]);
        if (++sr == kSegs) {
            sr = 0;
            seg_phase ^= 1;
        }
    }
    // tell the issuer, and leave
    if (tid == 0) keys_are = kEnd;
    __syncwarp();
    if (lane == 0) mbar_arrive(&k_bar);
    if (csync_count(fail) && tid == 0) {
        // a wait gave up: let the copies in flight land (bounded), then leave
        for (int s = 0; s < A::STAGES; ++s)
            for (int ph = 0; ph < 2; ++ph) mbar_wait(&full[s], ph);
        set_status(p.status, SPEC_STATUS_TIMEOUT);
    }
    csync();
    if (warp == 0) tmem_free(a_t, A::COLS);
}

// CTAs for a call: as many as are resident, no more than there can be units.
template <typename A> Layout layout_of(int B, int k_max, int Hq, int H, int max_len)
{
    const int qtiles = ((k_max + 1) * (Hq / H) + A::NT - 1) / A::NT;
    const int64_t units = static_cast<int64_t>(B) * H * qtiles * (kTaskUnits + (max_len + kTile - 1) / kTile);
    Layout l;
    l.grid = static_cast<int>(units < kSms * A::CTAS ? units : kSms * A::CTAS);
    return l;
}

template <typename A> size_t workspace_of(int B, int k_max, int Hq, int H, int max_len)
{
    const Layout l = layout_of<A>(B, k_max, Hq, H, max_len);
    return kTicketBytes + static_cast<size_t>(l.grid) * 2 * A::NT * (A::D + 2) * 4;
}

template <typename T, int D, int NT, bool OPT>
cudaError_t launch_one(const CacheView &c, const AttnParams &p, cudaStream_t s)
{
    using A = Attn<T, D, NT>;
    static bool done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev]) {
        e = cudaFuncSetAttribute(attend_kernel<T, D, NT, OPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, A::SMEM);
        if (e != cudaSuccess) return e;
        done[dev] = true;
    }
    const Layout l = layout_of<A>(c.B, p.k_max, p.Hq, c.H, p.max_len);
    attend_kernel<T, D, NT, OPT><<<l.grid, kAttnThreads + 64, A::SMEM, s>>>(c, p, l);
    return cudaGetLastError();
}

// What to do with the kernel for a call's type, channels and columns
template <typename F> auto with_kernel(int dtype, int D, int cols, F f)
{
    const int nt = column_tile(cols, D, dtype);
    if (dtype == SPEC_F32) {
        if (D == 64) return nt == 16 ? f(Attn<float, 64, 16>()) : f(Attn<float, 64, 32>());
        if (D == 128) return nt == 16 ? f(Attn<float, 128, 16>()) : f(Attn<float, 128, 32>());
        return nt == 16 ? f(Attn<float, 256, 16>()) : f(Attn<float, 256, 32>());
    }
    using B = __nv_bfloat16;
    if (D == 64) return nt == 16 ? f(Attn<B, 64, 16>()) : (nt == 32 ? f(Attn<B, 64, 32>()) : f(Attn<B, 64, 64>()));
    if (D == 128) return nt == 16 ? f(Attn<B, 128, 16>()) : (nt == 32 ? f(Attn<B, 128, 32>()) : f(Attn<B, 128, 64>()));
    return nt == 16 ? f(Attn<B, 256, 16>()) : f(Attn<B, 256, 32>());
}

template <bool OPT> cudaError_t launch_attend(const CacheView &c, const AttnParams &p, int dtype, cudaStream_t s)
{
    return with_kernel(dtype, c.D, (p.k_max + 1) * (p.Hq / c.H), [&](auto a) {
        using A = decltype(a);
        return launch_one<typename A::Type, A::D, A::NT, OPT>(c, p, s);
    });
}

}  // namespace

}  // namespace specv
