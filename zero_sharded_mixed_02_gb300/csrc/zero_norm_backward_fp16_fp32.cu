// The block norms' backward kernels for fp16 with an fp32 stream (zero_norm.cuh).
#include "zero_norm.cuh"

namespace zero {

const void* norm_backward_fp16_fp32(int, int v, int post, int pre, bool whole, bool copied, bool& two, int& smem)
{
    return v == 1   ? norm_backward_of<0, 2, 1>(post, pre, whole, copied, two, smem)
           : v == 2 ? norm_backward_of<0, 2, 2>(post, pre, whole, copied, two, smem)
                    : norm_backward_of<0, 2, 4>(post, pre, whole, copied, two, smem);
}

}  // namespace zero
