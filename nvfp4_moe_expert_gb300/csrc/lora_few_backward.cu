// Low-rank adapters, tiles of 16 rows: backward (dx).
#include "lora_few.cuh"

namespace nvfp4 {
namespace lora {

cudaError_t launch_few_backward(const Params& p, int64_t tiles, bool pdl, cudaStream_t st) {
    return launch_few<__nv_bfloat16, true>(p, tiles, pdl, st);
}

}  // namespace lora
}  // namespace nvfp4
