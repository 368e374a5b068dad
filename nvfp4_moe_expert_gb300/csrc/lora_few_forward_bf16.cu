// Low-rank adapters, tiles of 16 rows: forward, BF16.
#include "lora_few.cuh"

namespace nvfp4 {
namespace lora {

cudaError_t launch_few_forward_bf16(const Params& p, int64_t tiles, bool pdl, cudaStream_t st) {
    return launch_few<__nv_bfloat16, false>(p, tiles, pdl, st);
}

}  // namespace lora
}  // namespace nvfp4
