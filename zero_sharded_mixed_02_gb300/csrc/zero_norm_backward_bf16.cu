// The block norms' backward kernels for bf16 (zero_norm.cuh).
#include "zero_norm.cuh"

const void* zero::norm_backward_bf16(int res, int v, bool two, bool whole)
{
    return res == 2 ? norm_backward_of<1, 2>(v, two, whole) : norm_backward_of<1, 1>(v, two, whole);
}
