// The layer norm's kernels on fp16 rows.
#include "mbtile_layernorm.cuh"

namespace mbt {

template cudaError_t layernorm_forward<MBT_F16>(const LayerNormArgs &, cudaStream_t);
template int layernorm_backward<MBT_F16>(const LayerNormGradArgs &, cudaStream_t);

}  // namespace mbt
