// prompt_tiles_split.cu -- attention of a few bf16 prompts on the tensor cores whose items are
// split along the keys (prompt_tiles.cuh has the kernel).
#include "prompt_tiles.cuh"

namespace specv {

cudaError_t launch_prompt_tiles_split(const PromptParams &p, const PromptMaps &maps, int grid, int split, cudaStream_t s)
{
    return launch_tiles<false, true>(p, maps, grid, split, s);
}

}  // namespace specv
