// bf16 instances of the vocabulary head's kernels.
#include "zero_head.cuh"

namespace zero {
HeadKernels head_kernels_bf16() { return head_kernels<1>(); }
}  // namespace zero
