// cache_attend.cu -- the attention over the 4-bit paged cache without score
// options, and its workspace (cache_attend.cuh has the kernel).
#include "cache_attend.cuh"

namespace specv {

// the larger of the two types' needs: the size does not depend on q's type
size_t cache_attend_workspace(int B, int k_max, int Hq, int H, int D, int max_len)
{
    size_t most = 0;
    for (int dtype : {SPEC_F32, SPEC_BF16}) {
        const size_t n = with_kernel(dtype, D, (k_max + 1) * (Hq / H), [&](auto a) {
            return workspace_of<decltype(a)>(B, k_max, Hq, H, max_len);
        });
        most = n > most ? n : most;
    }
    return most;
}

cudaError_t launch_cache_attend(const CacheView &c, const AttnParams &p, int dtype, cudaStream_t s)
{
    const bool options = p.cap > 0.f || p.slopes || p.window > 0;
    if (p.parent) return options ? launch_cache_attend_tree_options(c, p, dtype, s) : launch_cache_attend_tree(c, p, dtype, s);
    return options ? launch_cache_attend_options(c, p, dtype, s) : launch_attend<false, false>(c, p, dtype, s);
}

}  // namespace specv
