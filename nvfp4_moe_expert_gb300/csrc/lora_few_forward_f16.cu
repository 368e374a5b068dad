// Low-rank adapters, tiles of 16 rows: forward, FP16.
#include "lora_few.cuh"

namespace nvfp4 {
namespace lora {

cudaError_t launch_few_forward_f16(const Params& p, int64_t tiles, bool pdl, cudaStream_t st) {
    return launch_few<__half, false>(p, tiles, pdl, st);
}

}  // namespace lora
}  // namespace nvfp4
