// fp16 instances of the vocabulary head's kernels.
#include "zero_head.cuh"

namespace zero {
HeadKernels head_kernels_fp16() { return head_kernels<0>(); }
}  // namespace zero
