// The block norms' forward kernels for bf16 (zero_norm.cuh); the stream in the same type.
#include "zero_norm.cuh"

namespace zero {
const void* norm_forward_bf16_fp32(int res, int v, int post, int pre, bool whole);
}

const void* zero::norm_forward_bf16(int res, int v, int post, int pre, bool whole)
{
    if (res == 2) return norm_forward_bf16_fp32(res, v, post, pre, whole);
    return v == 1   ? norm_forward_of<1, 1, 1>(post, pre, whole)
           : v == 2 ? norm_forward_of<1, 1, 2>(post, pre, whole)
                    : norm_forward_of<1, 1, 4>(post, pre, whole);
}
