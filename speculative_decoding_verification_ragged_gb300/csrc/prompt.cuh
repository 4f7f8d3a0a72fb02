// prompt.cuh -- what the kernels of the prompt attention (include/spec_prompt.h) share: the
// tiles of packed rows, the keys that a tile sees.
//
// The rows of a request that share a kv head are packed: row i * group + g of the tile line is
// row i of query head h * group + g.  (Rows times group stay below 2^31.)
#pragma once

#include <cstdint>

#include "cache.cuh"
#include "spec_prompt.h"

namespace specv {

// A tile of a request's packed rows.
struct PromptTile {
    int lo, n;                  // its request's first packed row and rows
    int k_lo, m;                // and its first key and keys
};

// Rows and keys of request b: false where it has no rows.  Malformed keys count as none.
__device__ __forceinline__ bool prompt_request(const PromptParams &p, int b, uint32_t *status, PromptTile &t)
{
    if (!request_rows(p.cu_rows, b, p.R_cap, p.R_cap, status, t.lo, t.n) || t.n == 0) return false;
    t.k_lo = p.cu_keys ? p.cu_keys[b] : t.lo;
    const int64_t m = p.cu_keys ? static_cast<int64_t>(p.cu_keys[b + 1]) - t.k_lo : t.n;
    t.m = static_cast<int>(m);
    if (t.k_lo < 0 || m < 0 || t.k_lo + m > p.K_cap) {
        set_status(status, SPEC_STATUS_BAD_LENGTH);
        t.k_lo = 0;
        t.m = 0;
    }
    return true;
}

// Tile `index` of the line of all requests' tiles, each request's last (longest) tile first:
// tiles(n) of a request with n rows.  THREADS threads take a request each, and a scan places them; false:
// the line ends before.  With index 0 alone the requests' errors are reported.
template <int THREADS, typename F>
__device__ __forceinline__ bool find_prompt_tile(const PromptParams &p, int64_t index, bool report, F tiles, PromptTile &t, int &tile)
{
    __shared__ int64_t sums[THREADS / 32];
    __shared__ PromptTile found;
    __shared__ int found_tile;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t base = 0;
    bool have = false;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        int64_t mine = 0;
        if (b0 + tid < p.B && prompt_request(p, b0 + tid, report ? p.status : nullptr, t)) mine = tiles(t.n);
        int64_t at = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, at, o);
            if (lane >= o) at += y;
        }
        if (lane == 31) sums[warp] = at;
        __syncthreads();
        int64_t all = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            at += w < warp ? sums[w] : 0;
            all += sums[w];
        }
        at += base;
        if (at - mine <= index && index < at) {
            found = t;
            found_tile = static_cast<int>(at - 1 - index);
        }
        base += all;
        have = index < base;
        __syncthreads();
        if (have && !report) break;
    }
    if (!have) return false;
    t = found;
    tile = found_tile;
    return true;
}

}  // namespace specv
