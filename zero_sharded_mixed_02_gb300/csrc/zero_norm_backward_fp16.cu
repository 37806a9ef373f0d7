// The block norms' backward kernels for fp16 (zero_norm.cuh).
#include "zero_norm.cuh"

const void* zero::norm_backward_fp16(int res, int v, bool two, bool whole)
{
    return res == 2 ? norm_backward_of<0, 2>(v, two, whole) : norm_backward_of<0, 0>(v, two, whole);
}
