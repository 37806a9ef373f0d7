// zero_act.cuh -- the 8-bit activation checkpoint format (include/zero_b200.h):
// row layout, block exponents, codes and their values.
//
// A block is 32 consecutive columns of a row with one exponent byte E; a code c
// stands for c * 2^(E - 127).  With max|x| = f * 2^p, f in [1, 2), the smallest
// exponent with max|x| <= 127 * 2^e is p - 6 if f <= 127/64, else p - 5: an integer
// comparison on the bits of max|x|.  Scaling by a power of two is exact, so a
// code is the correctly rounded quotient without a division.
#pragma once

#include "zero_common.cuh"
#include "zero_qwz.cuh"                  // pairs of fp32 values and their arithmetic

namespace zero {

#define ZERO_ACT_BLOCK 32
#define ZERO_ACT_BAD 255u                 // exponent byte of a block holding an inf or NaN

__host__ __device__ inline int64_t act_wide(int64_t cols)            // code bytes of a row
{
    return (cols + 31) / 32 * 32;
}
__host__ __device__ inline int64_t act_stride(int64_t cols)          // bytes of a row
{
    return (act_wide(cols) + act_wide(cols) / 32 + 31) / 32 * 32;
}

// Biased exponents a block may take: the value of every code is then exact in the
// type, subnormals included (fp16: 2^-24 is its smallest subnormal and
// 127 * 2^9 its last multiple of 2^9 that a code reaches; bf16 and fp32: 127 * 2^121).
__host__ __device__ inline int act_lo(int dtype) { return dtype == 0 ? 103 : 1; }
__host__ __device__ inline int act_hi(int dtype) { return dtype == 0 ? 136 : 248; }

// Exponent byte of a block from the bits of its largest |x| as binary32 (inf and
// NaN compare above every finite magnitude as integers).
static __device__ __forceinline__ uint32_t act_exponent(uint32_t amax_bits, int lo, int hi)
{
    const int p = (int)(amax_bits >> 23);
    if (p == 255) return ZERO_ACT_BAD;
    const int e = p - 6 + ((amax_bits & 0x7FFFFFu) > 0x7E0000u);
    return (uint32_t)(e < lo ? lo : e > hi ? hi : e);
}

// ---- chunks: eight consecutive columns, held as four pairs ---------------------------
static __device__ __forceinline__ f32x2_t fma2(f32x2_t a, f32x2_t b, f32x2_t c)
{
    f32x2_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
static __device__ __forceinline__ f32x2_t both(float a) { return pack2(a, a); }
static __device__ __forceinline__ float either(f32x2_t a)              // the pair's sum
{
    float x, y;
    unpack2(a, x, y);
    return x + y;
}

// Eight codes -> eight values.  The byte of a code, XOR 128, in the mantissa of 2^23
// is 2^23 + 128 + c exactly; one subtraction leaves c.  E = 255 gives the scale
// inf, and 0 * inf = NaN.
static __device__ __forceinline__ void act_values(uint2 q, uint32_t e, f32x2_t (&v)[4])
{
    const f32x2_t scale = both(__uint_as_float(e << 23)), bias = both(8388736.0f);
    const uint32_t w[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t a = __byte_perm(w[i / 2], 0x4B000000u, 0x7650 + (2 * i) % 4);
        const uint32_t b = __byte_perm(w[i / 2], 0x4B000000u, 0x7650 + (2 * i + 1) % 4);
        v[i] = mul2(sub2(pack2(__uint_as_float(a), __uint_as_float(b)), bias), scale);
    }
}

// Eight codes packed in two words, from eight values and their block's exponent byte.
// step = 2^(127 - E).  Adding 1.5 * 2^23 rounds to the nearest integer, ties to even,
// and leaves it in the low byte (the product is exact, so one fused operation does
// both).  Only a block whose exponent was cut at the type's largest (`hi`) can pass
// 127, so the clamp is left to that case.  A bad block's codes are 0.
static __device__ __forceinline__ uint2 act_codes(const f32x2_t (&v)[4], uint32_t e, int hi)
{
    if (e == ZERO_ACT_BAD) return make_uint2(0, 0);
    const f32x2_t step = both(__uint_as_float((254u - e) << 23)), rnd = both(12582912.0f);
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float a, b;
        if ((int)e == hi) {
            unpack2(mul2(v[i], step), a, b);
            a = __fadd_rn(fminf(fmaxf(a, -127.0f), 127.0f), 12582912.0f);
            b = __fadd_rn(fminf(fmaxf(b, -127.0f), 127.0f), 12582912.0f);
        } else {
            unpack2(fma2(v[i], step, rnd), a, b);
        }
        u[2 * i] = __float_as_uint(a);
        u[2 * i + 1] = __float_as_uint(b);
    }
    uint2 q;
    q.x = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    q.y = __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410);
    return q;
}

// Store a chunk's codes; the first lane of a block its exponent; the lanes of a row's
// last block the zeros after the exponents.  `row` is the checkpoint's row.
static __device__ __forceinline__ void act_put(uint8_t* row, uint32_t col, uint32_t wide, uint32_t stride, uint2 q, uint32_t e)
{
    *reinterpret_cast<uint2*>(row + col) = q;
    const uint32_t sub = (col >> 3) & 3;
    if (sub == 0) row[wide + (col >> 5)] = (uint8_t)e;
    if (col + 8 * (4 - sub) == wide)
        for (uint32_t i = wide + (wide >> 5) + sub; i < stride; i += 4) row[i] = 0;
}

// Largest magnitude of three, NaN if any is.
static __device__ __forceinline__ float amax3(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Quantize and store a chunk of fp32 values.  The four lanes of a block are consecutive
// and agree on the exponent by two shuffles: all lanes of the warp take part, `live` ones
// store.  Values past the row's end are 0.
static __device__ __forceinline__ void act_store(const f32x2_t (&v)[4], uint8_t* row, int col, int wide,
                                                 int stride, int lo, int hi, bool live)
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; i++) unpack2(v[i], x[2 * i], x[2 * i + 1]);
    float m = amax3(amax3(amax3(x[0], x[1], x[2]), x[3], x[4]), amax3(x[5], x[6], x[7]), 0.0f);
    m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (!live) return;
    const uint32_t e = act_exponent(__float_as_uint(m), lo, hi);
    act_put(row, col, wide, stride, act_codes(v, e, hi), e);
}

// The same for values below 2^100, as normalised rows are (at most sqrt(cols)): no exponent
// is cut at the type's largest, and the exponent needs no comparison of the fraction: adding
// 0x1FFFF to the bits carries into the exponent exactly when f > 127/64.
static __device__ __forceinline__ void act_store_small(const f32x2_t (&v)[4], uint8_t* row, int col, int wide,
                                                       int stride, int lo, bool live)
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; i++) unpack2(v[i], x[2 * i], x[2 * i + 1]);
    float m = amax3(amax3(amax3(x[0], x[1], x[2]), x[3], x[4]), amax3(x[5], x[6], x[7]), 0.0f);
    m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (!live) return;
    int e = (int)((__float_as_uint(m) + 0x1FFFFu) >> 23) - 6;
    e = e < lo ? lo : e;
    const bool bad = e > 240;
    const f32x2_t step = both(__uint_as_float((254u - (uint32_t)e) << 23)), rnd = both(12582912.0f);
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float a, b;
        unpack2(fma2(v[i], step, rnd), a, b);
        u[2 * i] = __float_as_uint(a);
        u[2 * i + 1] = __float_as_uint(b);
    }
    uint2 q;
    q.x = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    q.y = __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410);
    if (bad) {
        q = make_uint2(0, 0);
        e = ZERO_ACT_BAD;
    }
    act_put(row, col, wide, stride, q, (uint32_t)e);
}

// ---- a chunk as it lies in memory (T: 0 fp16, 1 bf16, 2 fp32) ------------------------
// Rows are read and written in 16-byte vectors where they are aligned to them.  Where they
// are not, single elements 8 columns apart in neighbouring lanes would touch as many memory
// sectors as lanes; instead the warp, whose 32 chunks are 256 consecutive columns, takes
// 32 neighbouring columns an instruction and turns them into chunks (and back) through its
// own 1 KB of shared memory (`stage`).  WHOLE: every row is aligned (an fp32 one to 32 bytes)
// and every chunk lies in the row (n >= 8) or past it (n <= 0).
template <int T> struct Raw { uint32_t w[T == 2 ? 8 : 4]; };

// The row's address is the same in all threads, so adding a column needs no arithmetic a thread.
template <int T>
static __device__ __forceinline__ const void* row_of(const void* p, int64_t row, uint32_t ld)
{
    return static_cast<const char*>(p) + row * (int64_t)((uint64_t)ld * (T == 2 ? 4 : 2));
}

template <int T>
static __device__ __forceinline__ uint32_t load_bits(const void* p, uint32_t i)
{
    return T == 2 ? __ldg(static_cast<const uint32_t*>(p) + i) : (uint32_t)__ldg(static_cast<const uint16_t*>(p) + i);
}

// Sixteen bytes from `sh` (even) of the 32 in q and n.
static __device__ __forceinline__ uint4 shifted(uint4 q, uint4 n, uint32_t sh)
{
    const uint32_t w[7] = {q.x, q.y, q.z, q.w, n.x, n.y, n.z};
    uint32_t x[6], y[5];
#pragma unroll
    for (int i = 0; i < 5; i++) x[i] = sh & 8 ? w[i + 2] : w[i];
    x[5] = sh & 8 ? n.w : w[5];
#pragma unroll
    for (int i = 0; i < 5; i++) y[i] = sh & 4 ? x[i + 1] : x[i];
    const uint32_t bits = (sh & 2) * 8;
    return make_uint4(__funnelshift_r(y[0], y[1], bits), __funnelshift_r(y[1], y[2], bits),
                      __funnelshift_r(y[2], y[3], bits), __funnelshift_r(y[3], y[4], bits));
}

// The aligned 16-byte words in which columns i .. i+8 of a row of any alignment lie, the first
// `sh` bytes before them.  Words may reach into the neighbouring rows; those that would reach
// out of the matrix [begin, stop) are put together element by element.  n as below.
template <int T> struct Words { uint4 q[T == 2 ? 3 : 2]; };
template <int T>
static __device__ __forceinline__ void load_words(Words<T>& w, uint32_t& sh, const void* row, uint32_t i, int n,
                                                  const void* begin, const char* stop)
{
    constexpr int WORDS = T == 2 ? 3 : 2;
    sh = 0;
#pragma unroll
    for (int k = 0; k < WORDS; k++) w.q[k] = make_uint4(0, 0, 0, 0);
    if (n <= 0) return;
    const char* from = static_cast<const char*>(row) + (uint64_t)i * (T == 2 ? 4 : 2);
    const uint32_t s = (uint32_t)reinterpret_cast<uintptr_t>(from) & 15;
    from -= s;
    if (from >= static_cast<const char*>(begin) && from + 16 * (WORDS - (s == 0)) <= stop) {
        sh = s;
#pragma unroll
        for (int k = 0; k < WORDS; k++)
            if (k + 1 < WORDS || s) w.q[k] = __ldg(reinterpret_cast<const uint4*>(from) + k);
        return;
    }
    uint32_t e[8];
#pragma unroll
    for (int k = 0; k < 8; k++) e[k] = k < n ? load_bits<T>(row, i + k) : 0;
    if (T == 2) {
        w.q[0] = make_uint4(e[0], e[1], e[2], e[3]);
        w.q[1] = make_uint4(e[4], e[5], e[6], e[7]);
    } else {
        w.q[0] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    }
}
template <int T>
static __device__ __forceinline__ void from_words(Raw<T>& r, const Words<T>& w, uint32_t sh, int n)
{
#pragma unroll
    for (int k = 0; k < (T == 2 ? 2 : 1); k++) {
        const uint4 x = shifted(w.q[k], w.q[k + 1], sh);
        r.w[4 * k] = x.x; r.w[4 * k + 1] = x.y; r.w[4 * k + 2] = x.z; r.w[4 * k + 3] = x.w;
    }
    if (n < 8)
#pragma unroll
        for (int k = 0; k < (T == 2 ? 8 : 4); k++)
            r.w[k] = T == 2 ? (k < n ? r.w[k] : 0u) : 2 * k + 1 < n ? r.w[k] : 2 * k < n ? r.w[k] & 0xFFFFu : 0u;
}

// Columns i .. i+8 of a row, those at or past n (of the eight) read as 0.  Unless `vec`, a
// lane has columns lane + 32 k of its warp's 256, for unstage().
template <int T, bool WHOLE = false>
static __device__ __forceinline__ void load_chunk(Raw<T>& r, const void* row, uint32_t i, int n, bool vec)
{
    if (WHOLE || vec) {
        if (WHOLE && T == 2 && n >= 8) {
            const float* s = static_cast<const float*>(row) + i;
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[T == 2 ? 4 : 0]),
                           "=r"(r.w[T == 2 ? 5 : 0]), "=r"(r.w[T == 2 ? 6 : 0]), "=r"(r.w[T == 2 ? 7 : 0])
                         : "l"(s));
            return;
        }
        if (n >= 8) {
            const uint4* s = T == 2 ? reinterpret_cast<const uint4*>(static_cast<const float*>(row) + i)
                                    : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i);
#pragma unroll
            for (int k = 0; k < (T == 2 ? 2 : 1); k++) {
                const uint4 q = __ldcs(s + k);
                r.w[4 * k] = q.x; r.w[4 * k + 1] = q.y; r.w[4 * k + 2] = q.z; r.w[4 * k + 3] = q.w;
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < (T == 2 ? 8 : 4); k++) {
            if (T == 2) r.w[k] = !WHOLE && k < n ? load_bits<T>(row, i + k) : 0u;
            else r.w[k] = (!WHOLE && 2 * k < n ? load_bits<T>(row, i + 2 * k) : 0u) |
                          (!WHOLE && 2 * k + 1 < n ? load_bits<T>(row, i + 2 * k + 1) << 16 : 0u);
        }
        return;
    }
    const int lane = threadIdx.x & 31, m = n + 7 * lane;      // lane's first of the warp's columns: i - 8 lane + lane
    const uint32_t at = i - 7 * lane;
#pragma unroll
    for (int k = 0; k < (T == 2 ? 8 : 4); k++) {
        if (T == 2) r.w[k] = 32 * k < m ? load_bits<T>(row, at + 32 * k) : 0u;
        else r.w[k] = (64 * k < m ? load_bits<T>(row, at + 64 * k) : 0u) |
                      (64 * k + 32 < m ? load_bits<T>(row, at + 64 * k + 32) << 16 : 0u);
    }
}

// What load_chunk() read without `vec`, as the lane's eight columns.
template <int T>
static __device__ __forceinline__ void unstage(Raw<T>& r, float* stage)
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
    if (T == 2) {
#pragma unroll
        for (int k = 0; k < 8; k++) stage[lane + 32 * k] = __uint_as_float(r.w[T == 2 ? k : 0]);
    } else {
        uint16_t* h = reinterpret_cast<uint16_t*>(stage);
#pragma unroll
        for (int k = 0; k < 4; k++) {
            h[lane + 64 * k] = (uint16_t)r.w[k];
            h[lane + 64 * k + 32] = (uint16_t)(r.w[k] >> 16);
        }
    }
    __syncwarp();
    const uint4* s = reinterpret_cast<const uint4*>(stage) + lane * (T == 2 ? 2 : 1);
#pragma unroll
    for (int k = 0; k < (T == 2 ? 2 : 1); k++) {
        const uint4 q = s[k];
        r.w[4 * k] = q.x; r.w[4 * k + 1] = q.y; r.w[4 * k + 2] = q.z; r.w[4 * k + 3] = q.w;
    }
}

template <int T>
static __device__ __forceinline__ void widen_chunk(const Raw<T>& r, f32x2_t (&v)[4])
{
#pragma unroll
    for (int j = 0; j < 4; j++) {
        float a, b;
        if (T == 2) {
            a = __uint_as_float(r.w[T == 2 ? 2 * j : 0]);
            b = __uint_as_float(r.w[T == 2 ? 2 * j + 1 : 0]);
        } else {
            widen2<T & 1>(r.w[j], a, b);
        }
        v[j] = pack2(a, b);
    }
}
template <int T, bool WHOLE>
static __device__ __forceinline__ void widen_chunk(Raw<T>& r, f32x2_t (&v)[4], bool vec, float* stage)
{
    if (!WHOLE && !vec) unstage<T>(r, stage);
    widen_chunk<T>(r, v);
}

template <int T, bool WHOLE = false>
static __device__ __forceinline__ void store_chunk(const void* row, uint32_t i, int n, bool vec, float* stage,
                                                   const f32x2_t (&v)[4])
{
    void* p = const_cast<void*>(row);
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; j++) unpack2(v[j], x[2 * j], x[2 * j + 1]);
    uint4 q[T == 2 ? 2 : 1];
    if (T == 2) {
        q[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        q[T == 2] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    } else {
        q[0] = make_uint4(narrow2<T & 1>(x[0], x[1]), narrow2<T & 1>(x[2], x[3]), narrow2<T & 1>(x[4], x[5]),
                          narrow2<T & 1>(x[6], x[7]));
    }
    if (WHOLE && T == 2) {
        if (n >= 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<float*>(p) + i),
                         "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                         : "memory");
        return;
    }
    if ((WHOLE || vec) && n >= 8) {
        uint4* o = T == 2 ? reinterpret_cast<uint4*>(static_cast<float*>(p) + i)
                          : reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i);
        if (T == 2 && (reinterpret_cast<uintptr_t>(o) & 31) == 0) {
            asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "f"(x[0]), "f"(x[1]),
                         "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]) : "memory");
            return;
        }
        __stcs(o, q[0]);
        if (T == 2) __stcs(o + 1, q[T == 2]);
    } else if (!WHOLE && vec) {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < n) {
                if (T == 2) static_cast<float*>(p)[i + j] = x[j];
                else static_cast<uint16_t*>(p)[i + j] = narrow1<T & 1>(x[j]);
            }
    } else if (!WHOLE) {
        const int lane = threadIdx.x & 31, m = n + 7 * lane;
        const uint32_t at = i - 7 * lane;
        __syncwarp();
        uint4* s = reinterpret_cast<uint4*>(stage) + lane * (T == 2 ? 2 : 1);
        s[0] = q[0];
        if (T == 2) s[T == 2] = q[T == 2];
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (32 * k < m) {
                if (T == 2) static_cast<float*>(p)[at + 32 * k] = stage[lane + 32 * k];
                else static_cast<uint16_t*>(p)[at + 32 * k] = reinterpret_cast<const uint16_t*>(stage)[lane + 32 * k];
            }
    }
}

}  // namespace zero
