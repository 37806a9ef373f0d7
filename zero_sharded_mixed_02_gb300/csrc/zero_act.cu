// zero_act.cu -- 8-bit activation checkpoints: save and load.
//
// Both are one pass over the data and bound by HBM: save reads 2 (fp32: 4) and
// writes 1 + 1/32 bytes per element, load the reverse.  The matrix is taken as a
// flat list of 8-column chunks (a row has C/8 of them, a multiple of four, so the
// four chunks of a block are four consecutive lanes); a thread takes ZERO_ACT_UNROLL
// chunks a block apart, so every warp access is one contiguous run and several
// loads are in flight.
#include "zero_act.cuh"
#include "zero_b200.h"
#include "zero_trace.h"

namespace zero {

#define ZERO_ACT_UNROLL 4

struct ActArgs {
    const void* x;          // or the output of load
    uint8_t* ckpt;
    int64_t chunks;         // rows * per_row
    int64_t ld;
    uint32_t per_row;       // chunks of a row
    int cols, wide, stride; // columns, code bytes and bytes of a checkpoint row
    int lo, hi;
    int vec;                // rows of x are 16-byte aligned
};

// Row and first column of a thread's chunks: one 64-bit division for the block's
// first chunk, 32-bit ones (below 2^31) for the rest.
struct ActPlace {
    int64_t row0;
    uint32_t off0;
    __device__ __forceinline__ ActPlace(int64_t first, uint32_t per_row)
    {
        row0 = first / per_row;
        off0 = (uint32_t)(first - row0 * per_row);
    }
    __device__ __forceinline__ void at(uint32_t i, uint32_t per_row, int64_t& row, int& col) const
    {
        const uint32_t k = off0 + i, r = k / per_row;
        row = row0 + r;
        col = (int)(k - r * per_row) * 8;
    }
};

template <int DT>
__global__ void __launch_bounds__(ZERO_THREADS) k_act_save(const ActArgs a)
{
    const int64_t first = (int64_t)blockIdx.x * (ZERO_ACT_UNROLL * ZERO_THREADS);
    const ActPlace place(first, a.per_row);
    float v[ZERO_ACT_UNROLL][8];
    int64_t row[ZERO_ACT_UNROLL];
    int col[ZERO_ACT_UNROLL];
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++) {
        const uint32_t i = u * ZERO_THREADS + threadIdx.x;
        place.at(i, a.per_row, row[u], col[u]);
        const bool live = first + i < a.chunks;
        if (!live) row[u] = -1;
        load8<DT>(a.x, row[u] * a.ld + col[u], live ? a.cols - col[u] : 0, a.vec, v[u]);
    }
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++)
        act_store_chunk(v[u], a.ckpt + row[u] * a.stride, col[u], a.wide, a.stride, a.lo, a.hi, row[u] >= 0);
}

template <int DT>
__global__ void __launch_bounds__(ZERO_THREADS) k_act_load(const ActArgs a)
{
    const int64_t first = (int64_t)blockIdx.x * (ZERO_ACT_UNROLL * ZERO_THREADS);
    const ActPlace place(first, a.per_row);
    uint2 q[ZERO_ACT_UNROLL];
    uint32_t e[ZERO_ACT_UNROLL];
    int64_t row[ZERO_ACT_UNROLL];
    int col[ZERO_ACT_UNROLL];
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++) {
        const uint32_t i = u * ZERO_THREADS + threadIdx.x;
        place.at(i, a.per_row, row[u], col[u]);
        if (first + i >= a.chunks) col[u] = a.cols;            // nothing to write
        if (col[u] < a.cols) {
            const uint8_t* r = a.ckpt + row[u] * a.stride;
            q[u] = __ldcs(reinterpret_cast<const uint2*>(r + col[u]));
            e[u] = __ldg(r + a.wide + (col[u] >> 5));
        }
    }
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++)
        if (col[u] < a.cols) {
            float v[8];
            act_values8(q[u], e[u], v);
            store8<DT>(const_cast<void*>(a.x), row[u] * a.ld + col[u], a.cols - col[u], a.vec, v);
        }
}

}  // namespace zero

using namespace zero;

namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

zero_status_t run(bool save, zero_dtype_t dtype, const void* x, int64_t rows, int64_t cols, int64_t ld,
                  const void* ckpt, void* stream)
{
    if (dtype != ZERO_FP16 && dtype != ZERO_BF16 && dtype != ZERO_FP32) return ZERO_EINVAL;
    if (rows < 0 || rows >= (1ll << 31) || cols < 1 || cols > ZERO_ACT_MAX_COLS || ld < cols ||
        ld > (1ll << 31))
        return ZERO_EINVAL;
    if (rows == 0) return ZERO_OK;
    const int64_t size = dtype == ZERO_FP32 ? 4 : 2;
    if (!x || !ckpt || !aligned_to(x, size) || !aligned_to(ckpt, 16)) return ZERO_EINVAL;
    ActArgs a{};
    a.x = x;
    a.ckpt = static_cast<uint8_t*>(const_cast<void*>(ckpt));
    a.cols = (int)cols;
    a.wide = (int)act_wide(cols);
    a.stride = (int)act_stride(cols);
    a.per_row = (uint32_t)(a.wide / 8);
    a.chunks = rows * a.per_row;
    a.ld = ld;
    a.lo = act_lo(dtype);
    a.hi = act_hi(dtype);
    a.vec = aligned_to(x, 16) && ld * size % 16 == 0;
    const int64_t per_block = ZERO_ACT_UNROLL * ZERO_THREADS;
    const int64_t grid = (a.chunks + per_block - 1) / per_block;
    if (grid > 0x7FFFFFFF) return ZERO_EINVAL;
    const void* fn = save ? (dtype == ZERO_FP16   ? (const void*)k_act_save<0>
                             : dtype == ZERO_BF16 ? (const void*)k_act_save<1>
                                                  : (const void*)k_act_save<2>)
                          : (dtype == ZERO_FP16   ? (const void*)k_act_load<0>
                             : dtype == ZERO_BF16 ? (const void*)k_act_load<1>
                                                  : (const void*)k_act_load<2>);
    void* args[] = {&a};
    return cudaLaunchKernel(fn, dim3((unsigned)grid), dim3(ZERO_THREADS), args, 0,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ZERO_OK
               : ZERO_ECUDA;
}

}  // namespace

extern "C" uint64_t zero_act_row_bytes(int64_t cols)
{
    return cols < 1 || cols > ZERO_ACT_MAX_COLS ? 0 : (uint64_t)act_stride(cols);
}

extern "C" zero_status_t zero_act_save(zero_dtype_t dtype, const void* x, int64_t rows, int64_t cols,
                                       int64_t ld, void* ckpt, void* stream)
{
    TraceRange trace_("zero_act_save");
    return run(true, dtype, x, rows, cols, ld, ckpt, stream);
}

extern "C" zero_status_t zero_act_load(zero_dtype_t dtype, const void* ckpt, int64_t rows, int64_t cols,
                                       void* out, int64_t ld, void* stream)
{
    TraceRange trace_("zero_act_load");
    return run(false, dtype, out, rows, cols, ld, ckpt, stream);
}
