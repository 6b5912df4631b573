#include "dense_split.cuh"

namespace moe {

cudaError_t launch_dense_grads(const DenseProblem* p, int n, int num_sms, cudaStream_t stream, int* launches) {
  if (n < 1 || n > kMaxJobs) return cudaErrorInvalidValue;
  return dense::launch_kind<kDenseLinear, kMajorAny>(p, n, num_sms, stream, launches);
}

}  // namespace moe
