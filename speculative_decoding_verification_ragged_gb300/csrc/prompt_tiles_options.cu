// prompt_tiles_options.cu -- attention of bf16 prompts on the tensor cores with a cap, distance
// biases or a scale that is not positive (prompt_tiles.cuh has the kernel).
#include "prompt_tiles.cuh"

namespace specv {

cudaError_t launch_prompt_tiles_options(const PromptParams &p, const PromptMaps &maps, int grid, cudaStream_t s)
{
    return launch_tiles<true, false>(p, maps, grid, 1, s);
}

}  // namespace specv
