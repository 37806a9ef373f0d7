// The block norms' backward kernels for fp16 (zero_norm.cuh); the stream in the same type.
#include "zero_norm.cuh"

namespace zero {
const void* norm_backward_fp16_fp32(int res, int v, int post, int pre, bool whole, bool copied, bool& two, int& smem);
}

const void* zero::norm_backward_fp16(int res, int v, int post, int pre, bool whole, bool copied, bool& two, int& smem)
{
    if (res == 2) return norm_backward_fp16_fp32(res, v, post, pre, whole, copied, two, smem);
    return v == 1   ? norm_backward_of<0, 0, 1>(post, pre, whole, copied, two, smem)
           : v == 2 ? norm_backward_of<0, 0, 2>(post, pre, whole, copied, two, smem)
                    : norm_backward_of<0, 0, 4>(post, pre, whole, copied, two, smem);
}
