// zero_wgrad.cu -- the weight gradient of a linear layer from the gradient of its
// output and the 8-bit checkpoint of its input: dw = dy^T xh, db = the column sums
// of dy (include/zero_b200.h).
//
// First form: a 64 x 64 tile of dw per block on the fp32 pipes, 16 tokens at a time
// through shared memory.
#include "zero_act.cuh"
#include "zero_b200.h"
#include "zero_trace.h"

namespace zero {

struct WgradArgs {
    const uint16_t* dy;
    const uint8_t* ckpt;
    const uint16_t *scale, *shift;
    void *dw, *db;
    int64_t tokens, n, k, ldy, ldw;
    int64_t wide, stride;
    int grad_dtype, accumulate;
};

static __device__ __forceinline__ void put_grad(void* p, int64_t i, float v, int grad_dtype, int accumulate)
{
    if (grad_dtype == 2) {
        float* o = static_cast<float*>(p) + i;
        *o = accumulate ? *o + v : v;
    } else {
        uint16_t* o = static_cast<uint16_t*>(p) + i;
        if (accumulate) v += grad_dtype == 0 ? widen1<0>(*o) : widen1<1>(*o);
        *o = grad_dtype == 0 ? narrow1<0>(v) : narrow1<1>(v);
    }
}

template <int DT>
__global__ void __launch_bounds__(256) k_wgrad(const WgradArgs a)
{
    __shared__ float sy[16][64], sx[16][64];
    const int64_t i0 = (int64_t)blockIdx.y * 64, j0 = (int64_t)blockIdx.x * 64;
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    float acc[4][4] = {}, sum[4] = {};
    for (int64_t t0 = 0; t0 < a.tokens; t0 += 16) {
        for (int e = threadIdx.x; e < 1024; e += 256) {
            const int64_t t = t0 + e / 64, i = i0 + e % 64, j = j0 + e % 64;
            const bool in = t < a.tokens;
            sy[e / 64][e % 64] = in && i < a.n ? widen1<DT>(a.dy[t * a.ldy + i]) : 0.0f;
            float v = 0.0f;
            if (in && j < a.k) {
                const uint8_t* row = a.ckpt + t * a.stride;
                uint32_t e = row[a.wide + j / 32];
                if (DT == 0 && (e < 103 || e > 136)) e = 255;      // outside fp16
                v = (float)(int8_t)row[j] * __uint_as_float(e << 23);
                if (e == 255) v = __uint_as_float(0x7FC00000u);
            }
            sx[e / 64][e % 64] = v;
        }
        __syncthreads();
#pragma unroll 4
        for (int t = 0; t < 16; t++)
            for (int p = 0; p < 4; p++) {
                const float y = sy[t][ti * 4 + p];
                sum[p] += y;
                for (int q = 0; q < 4; q++) acc[p][q] = __fmaf_rn(y, sx[t][tj * 4 + q], acc[p][q]);
            }
        __syncthreads();
    }
    for (int p = 0; p < 4; p++) {
        const int64_t i = i0 + ti * 4 + p;
        if (i >= a.n) continue;
        for (int q = 0; q < 4; q++) {
            const int64_t j = j0 + tj * 4 + q;
            if (j >= a.k) continue;
            float v = acc[p][q];
            if (a.scale) v *= widen1<DT>(a.scale[j]);
            if (a.shift) v = __fmaf_rn(sum[p], widen1<DT>(a.shift[j]), v);
            put_grad(a.dw, i * a.ldw + j, v, a.grad_dtype, a.accumulate);
        }
        if (a.db && blockIdx.x == 0 && tj == 0) put_grad(a.db, i, sum[p], a.grad_dtype, a.accumulate);
    }
}

}  // namespace zero

using namespace zero;

namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool sizes_ok(int64_t tokens, int64_t n, int64_t k)
{
    return tokens >= 0 && tokens < (1ll << 31) && n >= 1 && n <= (1ll << 24) && k >= 1 && k <= ZERO_ACT_MAX_COLS;
}

}  // namespace

extern "C" uint64_t zero_act_wgrad_workspace(int64_t tokens, int64_t n, int64_t k)
{
    return sizes_ok(tokens, n, k) ? 16 : 0;
}

extern "C" zero_status_t zero_act_wgrad(zero_dtype_t dtype, const void* dy, int64_t tokens, int64_t n,
                                        int64_t ldy, const void* ckpt, int64_t k, const void* col_scale,
                                        const void* col_shift, zero_dtype_t grad_dtype, void* dw, int64_t ldw,
                                        void* db, int accumulate, void* work, void* stream)
{
    TraceRange trace_("zero_act_wgrad");
    if ((dtype != ZERO_FP16 && dtype != ZERO_BF16) || (grad_dtype != dtype && grad_dtype != ZERO_FP32))
        return ZERO_EINVAL;
    if (!sizes_ok(tokens, n, k) || ldw < k || ldw > (1ll << 31)) return ZERO_EINVAL;
    const uintptr_t ge = grad_dtype == ZERO_FP32 ? 4 : 2;
    if (!dw || !aligned_to(dw, ge) || !aligned_to(db, ge) || !work || !aligned_to(work, 16) ||
        !aligned_to(col_scale, 2) || !aligned_to(col_shift, 2))
        return ZERO_EINVAL;
    if (tokens > 0 && (!dy || !aligned_to(dy, 2) || ldy < n || ldy > (1ll << 31) || !ckpt ||
                       !aligned_to(ckpt, 16)))
        return ZERO_EINVAL;
    WgradArgs a{};
    a.dy = static_cast<const uint16_t*>(dy);
    a.ckpt = static_cast<const uint8_t*>(ckpt);
    a.scale = static_cast<const uint16_t*>(col_scale);
    a.shift = static_cast<const uint16_t*>(col_shift);
    a.dw = dw;
    a.db = db;
    a.tokens = tokens; a.n = n; a.k = k; a.ldy = ldy; a.ldw = ldw;
    a.wide = act_wide(k);
    a.stride = act_stride(k);
    a.grad_dtype = grad_dtype;
    a.accumulate = accumulate != 0;
    const void* fn = dtype == ZERO_FP16 ? (const void*)k_wgrad<0> : (const void*)k_wgrad<1>;
    void* args[] = {&a};
    return cudaLaunchKernel(fn, dim3((unsigned)((k + 63) / 64), (unsigned)((n + 63) / 64)), dim3(256), args, 0,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ZERO_OK
               : ZERO_ECUDA;
}
