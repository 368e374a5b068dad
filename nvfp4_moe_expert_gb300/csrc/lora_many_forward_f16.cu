// Low-rank adapters, tiles of 128 rows: forward, FP16.
#include "lora_many.cuh"

namespace nvfp4 {
namespace lora {

cudaError_t launch_many_forward_f16(const Params& p, int64_t tiles, bool pdl, cudaStream_t st) {
    return launch_many<__half, false>(p, tiles, pdl, st);
}

}  // namespace lora
}  // namespace nvfp4
