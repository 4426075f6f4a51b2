// The norm's kernels on fp16 rows.
#include "mbtile_norm.cuh"

namespace mbt {

template cudaError_t norm_forward<MBT_F16>(const NormArgs &, cudaStream_t);
template int norm_backward<MBT_F16>(const NormGradArgs &, cudaStream_t);

}  // namespace mbt
