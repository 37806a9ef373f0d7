// zero_act.cu -- 8-bit activation checkpoints: save and load.
//
// Both are one pass over the data and bound by HBM: save reads 2 (fp32: 4) and
// writes 1 + 1/32 bytes per element, load the reverse.  The matrix is taken as a
// flat list of 8-column chunks (a row has C/8 of them, a multiple of four, so the
// four chunks of a block are four consecutive lanes); a thread takes ZERO_ACT_UNROLL
// chunks a block apart, so every warp access is one contiguous run and several
// loads are in flight.  At full rate an SM has about 17 instructions for an element
// read in 16 bits; the quotient by a row's chunks is a multiplication, the maximum of
// 16-bit inputs is taken on their bits two at a time, and the codes come from one
// fused multiply-add a pair.
#include "zero_act.cuh"
#include "zero_b200.h"
#include "zero_trace.h"

namespace zero {

#define ZERO_ACT_UNROLL 4

struct ActArgs {
    const void* x;          // or the output of load
    uint8_t* ckpt;
    uint32_t ld;
    uint32_t chunks;        // rows * per_row, below 2^31
    uint32_t per_row;       // chunks of a row
    uint32_t magic, shift;  // q / per_row = (q * magic) >> (32 + shift) for q < 2^31
    int cols, wide, stride; // columns, code bytes and bytes of a checkpoint row
    int lo, hi;
    int vec;                // rows of x are 16-byte aligned
};

static __device__ __forceinline__ void act_place(const ActArgs& a, uint32_t q, int64_t& row, int& col)
{
    const uint32_t r = __umulhi(q, a.magic) >> a.shift;
    row = r;
    col = (int)(q - r * a.per_row) * 8;
}

// Bits (as binary32) of a chunk's largest magnitude: those of inf or NaN if it has one.
template <int T>
static __device__ __forceinline__ uint32_t act_amax(const Raw<T>& r)
{
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
    if (T == 2) {
        const uint32_t x[4] = {r.q[T == 2].x, r.q[T == 2].y, r.q[T == 2].z, r.q[T == 2].w};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; j++) m = max(m, max(w[j] & 0x7FFFFFFFu, x[j] & 0x7FFFFFFFu));
        return m;
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    return max(m & 0xFFFFu, m >> 16);                        // still in the 16-bit type
}
template <int T>
static __device__ __forceinline__ uint32_t amax_bits(uint32_t m)
{
    return T == 2 ? m : __float_as_uint(widen1<T & 1>((uint16_t)m));
}

template <int T>
__global__ void __launch_bounds__(ZERO_THREADS) k_act_save(const __grid_constant__ ActArgs a)
{
    const uint32_t first = blockIdx.x * (ZERO_ACT_UNROLL * ZERO_THREADS) + threadIdx.x;
    Raw<T> r[ZERO_ACT_UNROLL];
    int64_t row[ZERO_ACT_UNROLL];
    int col[ZERO_ACT_UNROLL];
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++) {
        const uint32_t q = first + u * ZERO_THREADS;
        act_place(a, q, row[u], col[u]);
        if (q >= a.chunks) col[u] = a.wide;                  // nothing to read or write
        load_chunk<T>(r[u], row_of<T>(a.x, row[u], a.ld), col[u], a.cols - col[u], a.vec);
    }
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++) {
        uint32_t m = act_amax<T>(r[u]);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        if (col[u] >= a.wide) continue;
        const uint32_t e = act_exponent(amax_bits<T>(m), a.lo, a.hi);
        f32x2_t v[4];
        widen_chunk<T>(r[u], v);
        act_put(a.ckpt + row[u] * a.stride, col[u], a.wide, a.stride, act_codes(v, e, a.hi), e);
    }
}

template <int T>
__global__ void __launch_bounds__(ZERO_THREADS) k_act_load(const __grid_constant__ ActArgs a)
{
    const uint32_t first = blockIdx.x * (ZERO_ACT_UNROLL * ZERO_THREADS) + threadIdx.x;
    uint2 c[ZERO_ACT_UNROLL];
    uint32_t e[ZERO_ACT_UNROLL];
    int64_t row[ZERO_ACT_UNROLL];
    int col[ZERO_ACT_UNROLL];
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++) {
        const uint32_t q = first + u * ZERO_THREADS;
        act_place(a, q, row[u], col[u]);
        if (q >= a.chunks) col[u] = a.wide;                  // nothing to write
        if (col[u] < a.cols) {
            const uint8_t* p = a.ckpt + row[u] * a.stride;
            c[u] = __ldcs(reinterpret_cast<const uint2*>(p + col[u]));
            e[u] = __ldg(p + a.wide + (col[u] >> 5));
        }
    }
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++)
        if (col[u] < a.cols) {
            f32x2_t v[4];
            act_values(c[u], e[u], v);
            store_chunk<T>(row_of<T>(a.x, row[u], a.ld), col[u], a.cols - col[u], a.vec, v);
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
    a.cols = (int)cols;
    a.wide = (int)act_wide(cols);
    a.stride = (int)act_stride(cols);
    a.per_row = (uint32_t)(a.wide / 8);
    // ceil(log2 per_row) = l: magic = ceil(2^(31 + l) / per_row) fits 32 bits and is exact for q < 2^31
    uint32_t l = 2;
    while ((1u << l) < a.per_row) l++;
    a.magic = (uint32_t)(((1ull << (31 + l)) + a.per_row - 1) / a.per_row);
    a.shift = l - 1;
    a.ld = (uint32_t)ld;
    a.lo = act_lo(dtype);
    a.hi = act_hi(dtype);
    a.vec = aligned_to(x, 16) && ld * size % 16 == 0;
    const void* fn = save ? (dtype == ZERO_FP16   ? (const void*)k_act_save<0>
                             : dtype == ZERO_BF16 ? (const void*)k_act_save<1>
                                                  : (const void*)k_act_save<2>)
                          : (dtype == ZERO_FP16   ? (const void*)k_act_load<0>
                             : dtype == ZERO_BF16 ? (const void*)k_act_load<1>
                                                  : (const void*)k_act_load<2>);
    // as many rows a launch as keep its chunk numbers, the last block's idle ones too, below 2^31
    const int64_t per_block = ZERO_ACT_UNROLL * ZERO_THREADS;
    const int64_t most = ((1ll << 31) - per_block) / a.per_row;
    for (int64_t r = 0; r < rows; r += most) {
        const int64_t n = rows - r < most ? rows - r : most;
        a.x = static_cast<const char*>(x) + r * ld * size;
        a.ckpt = static_cast<uint8_t*>(const_cast<void*>(ckpt)) + r * a.stride;
        a.chunks = (uint32_t)(n * a.per_row);
        void* args[] = {&a};
        if (cudaLaunchKernel(fn, dim3((unsigned)((a.chunks + per_block - 1) / per_block)), dim3(ZERO_THREADS), args, 0,
                             static_cast<cudaStream_t>(stream)) != cudaSuccess)
            return ZERO_ECUDA;
    }
    return ZERO_OK;
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
