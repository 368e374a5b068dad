// Low-rank adapters, tiles of 128 rows: forward, BF16.
#include "lora_many.cuh"

namespace nvfp4 {
namespace lora {

cudaError_t launch_many_forward_bf16(const Params& p, int64_t tiles, bool pdl, cudaStream_t st) {
    return launch_many<__nv_bfloat16, false>(p, tiles, pdl, st);
}

}  // namespace lora
}  // namespace nvfp4
