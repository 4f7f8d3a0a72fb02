// cache_attend_tree_options.cu -- the attention of trees of rows over the 4-bit paged cache
// with a cap, distance biases or a window (cache_attend.cuh has the kernel).
#include "cache_attend.cuh"

namespace specv {

cudaError_t launch_cache_attend_tree_options(const CacheView &c, const AttnParams &p, int dtype, cudaStream_t s)
{
    return launch_attend<true, true>(c, p, dtype, s);
}

}  // namespace specv
