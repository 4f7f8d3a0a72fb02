// cache_attend_options.cu -- the attention over the 4-bit paged cache with a cap,
// distance biases or a window (cache_attend.cuh has the kernel).
#include "cache_attend.cuh"

namespace specv {

cudaError_t launch_cache_attend_options(const CacheView &c, const AttnParams &p, int dtype, cudaStream_t s)
{
    return launch_attend<true, false>(c, p, dtype, s);
}

}  // namespace specv
