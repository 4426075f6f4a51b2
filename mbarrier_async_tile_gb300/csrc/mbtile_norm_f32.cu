// The norm's kernels on fp32 rows.
#include "mbtile_norm.cuh"

namespace mbt {

template cudaError_t norm_forward<MBT_F32>(const NormArgs &, cudaStream_t);
template int norm_backward<MBT_F32>(const NormGradArgs &, cudaStream_t);

}  // namespace mbt
