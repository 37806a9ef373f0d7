// The block norms' forward kernels for bf16 with an fp32 stream (zero_norm.cuh).
#include "zero_norm.cuh"

namespace zero {

const void* norm_forward_bf16_fp32(int, int v, int post, int pre, bool whole)
{
    return v == 1   ? norm_forward_of<1, 2, 1>(post, pre, whole)
           : v == 2 ? norm_forward_of<1, 2, 2>(post, pre, whole)
                    : norm_forward_of<1, 2, 4>(post, pre, whole);
}

}  // namespace zero
