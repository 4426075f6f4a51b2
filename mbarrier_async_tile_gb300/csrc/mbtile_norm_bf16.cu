// The norm's kernels on bf16 rows.
#include "mbtile_norm.cuh"

namespace mbt {

template cudaError_t norm_forward<MBT_BF16>(const NormArgs &, cudaStream_t);
template int norm_backward<MBT_BF16>(const NormGradArgs &, cudaStream_t);

}  // namespace mbt
