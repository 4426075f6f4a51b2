// The layer norm's kernels on fp32 rows.
#include "mbtile_layernorm.cuh"

namespace mbt {

template cudaError_t layernorm_forward<MBT_F32>(const LayerNormArgs &, cudaStream_t);
template int layernorm_backward<MBT_F32>(const LayerNormGradArgs &, cudaStream_t);

}  // namespace mbt
