// Low-rank adapters, tiles of 128 rows: backward (dx).
#include "lora_many.cuh"

namespace nvfp4 {
namespace lora {

cudaError_t launch_many_backward(const Params& p, int64_t tiles, bool pdl, cudaStream_t st) {
    return launch_many<__nv_bfloat16, true>(p, tiles, pdl, st);
}

}  // namespace lora
}  // namespace nvfp4
