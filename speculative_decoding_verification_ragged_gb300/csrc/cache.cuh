// cache.cuh -- the 4-bit paged cache as the cache kernels see it: addresses of
// blocks and their parts, the masks of a packed row, and the decoding of codes
// and scales (include/spec_cache.h has the layout).
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "spec_cache.h"

namespace specv {

constexpr int kTok = SPEC_CACHE_BLOCK_TOKENS;

// byte offsets of the parts of a block with D channels
__host__ __device__ constexpr int block_bytes(int D) { return 36 * D; }
__host__ __device__ constexpr int k_scale_at(int D) { return 16 * D; }
__host__ __device__ constexpr int v_codes_at(int D) { return 18 * D; }
__host__ __device__ constexpr int v_scale_at(int D) { return 34 * D; }

// page of token slot `slot` of request b, or -1 where the table names none
__device__ __forceinline__ int page_of(const CacheView &c, int b, int slot)
{
    const int p = __ldg(c.page_table + static_cast<int64_t>(b) * c.max_pages + slot / c.page_tokens);
    return (p >= 0 && p < c.n_pages) ? p : -1;
}

// block `blk` of page `page`, kv head h (64-bit offsets: a pool can pass 4 GiB)
__device__ __forceinline__ uint8_t *block_at(const CacheView &c, int page, int h, int blk)
{
    return c.pages + ((static_cast<int64_t>(page) * c.H + h) * (c.page_tokens / kTok) + blk) *
                         block_bytes(c.D);
}

// the rows of request b: false (with the status bit) where cu_rows is malformed
__device__ __forceinline__ bool request_rows(const int32_t *cu_rows, int b, int R_cap, int max_rows,
                                             uint32_t *status, int &lo, int &n)
{
    lo = cu_rows[b];
    const int hi = cu_rows[b + 1];
    // differences in 64 bits: malformed offsets must not wrap into range
    const int64_t d = static_cast<int64_t>(hi) - lo;
    n = static_cast<int>(d);
    if (lo < 0 || hi > R_cap || d < 0 || d > max_rows) {
        set_status(status, SPEC_STATUS_BAD_ROWS);
        n = 0;
        return false;
    }
    return true;
}

// two e2m1 codes (one byte, low nibble first) as f16x2, exact
__device__ __forceinline__ uint32_t e2m1x2(uint32_t byte)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b, c0, c1, c2;\n\tmov.b32 {b, c0, c1, c2}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
        : "=r"(r)
        : "r"(byte));
    return r;
}

// two e4m3 bytes as f16x2, exact
__device__ __forceinline__ uint32_t e4m3x2(uint32_t two)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
    return r;
}

__device__ __forceinline__ float2 h2_float2(uint32_t h2)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&h2));
}

// one scale byte as a float
__device__ __forceinline__ float e4m3_value(uint32_t s) { return h2_float2(e4m3x2(s & 255u)).x; }

template <typename T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

}  // namespace specv
