// The block norms' forward kernels for fp16 (zero_norm.cuh).
#include "zero_norm.cuh"

const void* zero::norm_forward_fp16(int res, int v, bool whole)
{
    return res == 2 ? norm_forward_of<0, 2>(v, whole) : norm_forward_of<0, 0>(v, whole);
}
