// prompt_tiles.cu -- attention of bf16 prompts on the tensor cores without score options
// (prompt_tiles.cuh has the kernel): its tensor maps, and the choice of the kernel.
#include "prompt_tiles.cuh"

namespace specv {

namespace {

using Encode = decltype(&cuTensorMapEncodeTiled);

Encode encoder()
{
    static Encode f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<Encode>(p);
    }();
    return f;
}

// `aligned` [rows][heads][D] as boxes of 64 channels x `heads_box` heads x `rows_box` rows, each of 128-byte rows with the swizzle
// (strides positive multiples of 16 bytes below 2^40; those of one head or row do not matter)
bool map_of(CUtensorMap *m, const void *x, bool aligned, int D, int heads, int rows, int64_t head, int64_t row, int heads_box, int rows_box)
{
    if (heads == 1) head = D;
    if (rows == 1) row = D;
    if (!aligned || head <= 0 || row <= 0 || head >= (int64_t(1) << 38) || row >= (int64_t(1) << 38)) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head) * 2, static_cast<cuuint64_t>(row) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads_box), static_cast<cuuint32_t>(rows_box)}, one[3] = {1, 1, 1};
    const Encode f = encoder();
    return f && f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(x), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_prompt_tiles(const PromptParams &p, const PromptMaps &maps, cudaStream_t s)
{
    // At most this many items (of requests that do not overlap).  Where they leave SMs idle each is split, into as many parts
    // as fit and as its steps can pay for.
    const int rows = (p.D == 256 ? 1 : 2) * (128 / (p.Hq / p.H));
    const int64_t items = (p.R_cap + static_cast<int64_t>(p.B) * (rows - 1)) / rows * p.H;
    const int64_t steps = p.K_cap / (p.D == 256 ? 64 : 128) + 1;
    const int grid = static_cast<int>(items < kPromptSms ? items : kPromptSms);
    const int split = parts_of(steps, static_cast<int>(items > kPromptSms ? 1 : min(kPromptSms / items, static_cast<int64_t>(kMostParts))));
    const bool options = p.cap > 0.f || p.slopes || p.scale <= 0.f;
    if (split > 1) return options ? launch_prompt_tiles_split_options(p, maps, grid, split, s) : launch_prompt_tiles_split(p, maps, grid, split, s);
    return options ? launch_prompt_tiles_options(p, maps, grid, s) : launch_tiles<false, false>(p, maps, grid, 1, s);
}

}  // namespace

size_t prompt_workspace(int D, int dtype)
{
    if (dtype == SPEC_F32) return kPromptTickets;
    return kPromptTickets + static_cast<size_t>(kPromptSms) * (D == 256 ? 1 : 2) * 128 * (D * 4 + 8);
}

cudaError_t launch_prompt(const PromptParams &p, int dtype, cudaStream_t s)
{
    const int group = p.Hq / p.H;
    PromptMaps maps;
    // bf16 goes to the tensor cores where TMA can fetch it, a tile holds the heads of a row and the kernel was built as it has to be; else
    // to the CUDA cores
    if (dtype == SPEC_BF16 && group <= 128 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0 &&
        map_of(&maps.q, p.q, p.q_aligned, p.D, p.Hq, p.R_cap, p.q_head, p.q_row, group, 128 / group) &&
        map_of(&maps.k, p.k, p.k_aligned, p.D, p.H, p.K_cap, p.k_head, p.k_row, 1, p.D == 256 ? 64 : 128) &&
        map_of(&maps.v, p.v, p.v_aligned, p.D, p.H, p.K_cap, p.v_head, p.v_row, 1, p.D == 256 ? 64 : 128)) {
        const cudaError_t e = launch_prompt_tiles(p, maps, s);
        if (e != cudaErrorNotSupported) return e;
    }
    return launch_prompt_rows(p, dtype, s);
}

}  // namespace specv
