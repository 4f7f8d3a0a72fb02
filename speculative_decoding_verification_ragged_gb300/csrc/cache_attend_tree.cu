// cache_attend_tree.cu -- the attention of trees of rows over the 4-bit paged cache
// without score options (cache_attend.cuh has the kernel).
#include "cache_attend.cuh"

namespace specv {

cudaError_t launch_cache_attend_tree(const CacheView &c, const AttnParams &p, int dtype, cudaStream_t s)
{
    return launch_attend<false, true>(c, p, dtype, s);
}

}  // namespace specv
