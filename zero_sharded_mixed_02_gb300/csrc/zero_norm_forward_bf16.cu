// The block norms' forward kernels for bf16 (zero_norm.cuh).
#include "zero_norm.cuh"

const void* zero::norm_forward_bf16(int res, int v, bool whole)
{
    return res == 2 ? norm_forward_of<1, 2>(v, whole) : norm_forward_of<1, 1>(v, whole);
}
