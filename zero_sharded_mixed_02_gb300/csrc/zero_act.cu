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
    const char* stop;       // end of x
    uint8_t* ckpt;
    uint32_t ld;
    uint32_t chunks;        // rows * per_row, below 2^31
    uint32_t per_row;       // chunks of a row
    uint32_t magic, shift;  // q / per_row = (q * magic) >> (32 + shift) for q < 2^31; 0: per_row is 1
    int cols, wide, stride; // columns, code bytes and bytes of a checkpoint row
    int lo, hi;
};

static __device__ __forceinline__ void act_place(const ActArgs& a, uint32_t q, int64_t& row, int& col)
{
    const uint32_t r = a.magic ? __umulhi(q, a.magic) >> a.shift : q;
    row = r;
    col = (int)(q - r * a.per_row) * 8;
}

// Bits (as binary32) of a chunk's largest magnitude: those of inf or NaN if it has one.
template <int T>
static __device__ __forceinline__ uint32_t act_amax(const Raw<T>& r)
{
    uint32_t m = 0;
    if (T == 2) {
#pragma unroll
        for (int j = 0; j < (T == 2 ? 8 : 4); j++) m = max(m, r.w[j] & 0x7FFFFFFFu);
        return m;
    }
#pragma unroll
    for (int j = 0; j < 4; j++) m = __vmaxu2(m, r.w[j] & 0x7FFF7FFFu);
    return max(m & 0xFFFFu, m >> 16);                        // still in the 16-bit type
}
template <int T>
static __device__ __forceinline__ uint32_t amax_bits(uint32_t m)
{
    return T == 2 ? m : __float_as_uint(widen1<T & 1>((uint16_t)m));
}

// Four neighbouring lanes' chunks, a block of 32 columns, to codes (col = wide: none).
template <int T>
static __device__ __forceinline__ void act_save_chunk(const ActArgs& a, int64_t row, int col, const Raw<T>& r)
{
    uint32_t m = act_amax<T>(r);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (col >= a.wide) return;
    const uint32_t e = act_exponent(amax_bits<T>(m), a.lo, a.hi);
    f32x2_t v[4];
    widen_chunk<T>(r, v);
    act_put(a.ckpt + row * a.stride, col, a.wide, a.stride, act_codes(v, e, a.hi), e);
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
        load_chunk<T>(r[u], row_of<T>(a.x, row[u], a.ld), col[u], a.cols - col[u], true);
    }
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++) {
        act_save_chunk<T>(a, row[u], col[u], r[u]);
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
            store_chunk<T>(row_of<T>(a.x, row[u], a.ld), col[u], a.cols - col[u], true, nullptr, v);
        }
}

// Rows that are not aligned to vectors.  Saving, a thread reads the aligned 16-byte words that
// its chunk lies in and shifts it out of them; words may reach into the neighbouring rows, but
// those that reach out of the matrix are read element by element.  Loading, a thread makes an
// aligned run of eight columns (`off` columns before a chunk's) out of the codes of two chunks,
// and only runs that a row's start or end cuts are written element by element.  16384 x 6401
// bf16: 88 and 76 us, where a lane for each column took 279 and 174.
template <int T>
__global__ void __launch_bounds__(ZERO_THREADS) k_act_save_any(const __grid_constant__ ActArgs a)
{
    const uint32_t first = blockIdx.x * (ZERO_ACT_UNROLL * ZERO_THREADS) + threadIdx.x;
    Words<T> w[ZERO_ACT_UNROLL];
    uint32_t sh[ZERO_ACT_UNROLL];
    int64_t row[ZERO_ACT_UNROLL];
    int col[ZERO_ACT_UNROLL];
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++) {
        const uint32_t at = first + u * ZERO_THREADS;
        act_place(a, at, row[u], col[u]);
        if (at >= a.chunks) col[u] = a.wide;                 // nothing to read or write
        load_words<T>(w[u], sh[u], row_of<T>(a.x, row[u], a.ld), col[u], a.cols - col[u], a.x, a.stop);
    }
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++) {
        Raw<T> r;
        from_words<T>(r, w[u], sh[u], a.cols - col[u]);
        act_save_chunk<T>(a, row[u], col[u], r);
    }
}

template <int T>
__global__ void __launch_bounds__(ZERO_THREADS) k_act_load_any(const __grid_constant__ ActArgs a)
{
    constexpr int SIZE = T == 2 ? 4 : 2;
    const uint32_t first = blockIdx.x * (ZERO_ACT_UNROLL * ZERO_THREADS) + threadIdx.x;
    uint2 c[ZERO_ACT_UNROLL][2];
    uint32_t e[ZERO_ACT_UNROLL][2];
    int64_t row[ZERO_ACT_UNROLL];
    int col[ZERO_ACT_UNROLL];
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++) {
        const uint32_t at = first + u * ZERO_THREADS;
        act_place(a, at, row[u], col[u]);
        const uint8_t* p = a.ckpt + row[u] * a.stride;
#pragma unroll
        for (int h = 0; h < 2; h++) {                        // the chunk before, and the chunk
            const int i = col[u] - 8 + 8 * h;
            c[u][h] = make_uint2(0, 0);
            e[u][h] = 0;
            if (at < a.chunks && i >= 0 && i < a.cols) {
                c[u][h] = __ldg(reinterpret_cast<const uint2*>(p + i));
                e[u][h] = __ldg(p + a.wide + (i >> 5));
            }
        }
    }
#pragma unroll
    for (int u = 0; u < ZERO_ACT_UNROLL; u++) {
        if (first + u * ZERO_THREADS >= a.chunks) break;
        char* line = static_cast<char*>(const_cast<void*>(row_of<T>(a.x, row[u], a.ld)));
        const int off = (int)((reinterpret_cast<uintptr_t>(line) & 15) / SIZE), i = col[u] - off;
        // the last `off` codes of the chunk before, then the chunk's first
        const uint64_t before = (uint64_t)c[u][0].y << 32 | c[u][0].x, here = (uint64_t)c[u][1].y << 32 | c[u][1].x;
        const uint64_t both_ = off ? here << 8 * off | before >> (64 - 8 * off) : here;
        const uint2 codes = make_uint2((uint32_t)both_, (uint32_t)(both_ >> 32));
        f32x2_t v[4];
        float x[8];
        act_values(codes, e[u][1], v);
#pragma unroll
        for (int j = 0; j < 4; j++) unpack2(v[j], x[2 * j], x[2 * j + 1]);
        if (off && e[u][0] != e[u][1]) {
            act_values(codes, e[u][0], v);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                float lo, hi;
                unpack2(v[j], lo, hi);
                if (2 * j < off) x[2 * j] = lo;
                if (2 * j + 1 < off) x[2 * j + 1] = hi;
            }
        }
        if (i >= 0 && i + 8 <= a.cols) {
            uint4* o = reinterpret_cast<uint4*>(line + (int64_t)i * SIZE);
            if (T == 2) {
                __stcs(o, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])));
                __stcs(o + 1, make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])));
            } else {
                __stcs(o, make_uint4(narrow2<T & 1>(x[0], x[1]), narrow2<T & 1>(x[2], x[3]), narrow2<T & 1>(x[4], x[5]),
                                     narrow2<T & 1>(x[6], x[7])));
            }
            continue;
        }
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (i + j >= 0 && i + j < a.cols) {
                if (T == 2) reinterpret_cast<float*>(line)[i + j] = x[j];
                else reinterpret_cast<uint16_t*>(line)[i + j] = narrow1<T & 1>(x[j]);
            }
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
    const bool vec = aligned_to(x, 16) && ld * size % 16 == 0;
    // chunks of a row; loading to rows that are not aligned, runs that start up to seven columns earlier
    a.per_row = (uint32_t)(vec || save ? a.wide / 8 : (cols + 14) / 8);
    // ceil(log2 per_row) = l: magic = ceil(2^(31 + l) / per_row) fits 32 bits and is exact for q < 2^31
    // (from two chunks a row; 0 says one)
    uint32_t l = 1;
    while ((1u << l) < a.per_row) l++;
    a.magic = a.per_row == 1 ? 0 : (uint32_t)(((1ull << (31 + l)) + a.per_row - 1) / a.per_row);
    a.shift = l - 1;
    a.ld = (uint32_t)ld;
    a.lo = act_lo(dtype);
    a.hi = act_hi(dtype);
    static const void* const kernels[2][2][3] = {
        {{(const void*)k_act_load_any<0>, (const void*)k_act_load_any<1>, (const void*)k_act_load_any<2>},
         {(const void*)k_act_load<0>, (const void*)k_act_load<1>, (const void*)k_act_load<2>}},
        {{(const void*)k_act_save_any<0>, (const void*)k_act_save_any<1>, (const void*)k_act_save_any<2>},
         {(const void*)k_act_save<0>, (const void*)k_act_save<1>, (const void*)k_act_save<2>}}};
    const void* fn = kernels[save][vec][dtype];
    // as many rows a launch as keep its chunk numbers, the last block's idle ones too, below 2^31
    const int64_t per_block = ZERO_ACT_UNROLL * ZERO_THREADS;
    const int64_t most = ((1ll << 31) - per_block) / a.per_row;
    for (int64_t r = 0; r < rows; r += most) {
        const int64_t n = rows - r < most ? rows - r : most;
        a.x = static_cast<const char*>(x) + r * ld * size;
        a.stop = static_cast<const char*>(a.x) + ((n - 1) * ld + cols) * size;
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
