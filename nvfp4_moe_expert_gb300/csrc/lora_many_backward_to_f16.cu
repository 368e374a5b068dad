// Low-rank adapters, tiles of 128 rows: backward (dx), outputs in F16.
#include "lora_many.cuh"

namespace nvfp4 {
namespace lora {

template cudaError_t launch_many<__nv_bfloat16, true, NVFP4_TYPE_F16>(const Params&, int64_t, bool, cudaStream_t);

}  // namespace lora
}  // namespace nvfp4
