// norm_rope_bwd.cu -- the backward's kernels of the norm with the position rotation
// (norm_rope_kernel.cuh).
#include "norm_rope_kernel.cuh"

namespace tsr {

namespace norm {

template tsr_status launch<true>(const NormParams&, int, const Shape&, cudaStream_t);

}  // namespace norm

}  // namespace tsr
