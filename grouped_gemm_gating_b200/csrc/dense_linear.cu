#include "dense_split.cuh"

namespace moe {

cudaError_t launch_dense_linear(const DenseProblem& p, int num_sms, cudaStream_t stream, int* launches) {
  return dense::launch_kind<kDenseLinear, kMajorKK>(&p, 1, num_sms, stream, launches);
}

}  // namespace moe
