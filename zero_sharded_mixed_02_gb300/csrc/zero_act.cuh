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

// 2^(127 - E), the factor from values to codes; 0 for a bad block.
static __device__ __forceinline__ float act_step(uint32_t e)
{
    return e == ZERO_ACT_BAD ? 0.0f : __uint_as_float((254u - e) << 23);
}

// Four codes packed in a word, from four values and their block's factor.  Adding
// 1.5 * 2^23 rounds to the nearest integer, ties to even, and leaves it in the low
// byte.  Only a block whose exponent was cut at the type's largest can pass 127,
// so the clamp is left to that case (`top`, uniform per block).  A bad block's
// codes are 0 whatever its values.
static __device__ __forceinline__ uint32_t act_codes4(float a, float b, float c, float d, float step,
                                                      bool top, bool bad)
{
    const float rnd = 12582912.0f;
    a *= step; b *= step; c *= step; d *= step;
    if (top) {
        a = fminf(fmaxf(a, -127.0f), 127.0f);
        b = fminf(fmaxf(b, -127.0f), 127.0f);
        c = fminf(fmaxf(c, -127.0f), 127.0f);
        d = fminf(fmaxf(d, -127.0f), 127.0f);
    }
    const uint32_t u0 = __float_as_uint(__fadd_rn(a, rnd)), u1 = __float_as_uint(__fadd_rn(b, rnd));
    const uint32_t u2 = __float_as_uint(__fadd_rn(c, rnd)), u3 = __float_as_uint(__fadd_rn(d, rnd));
    const uint32_t w = __byte_perm(__byte_perm(u0, u1, 0x0040), __byte_perm(u2, u3, 0x0040), 0x5410);
    return bad ? 0u : w;
}

// Eight codes (a lane's chunk) -> eight values in fp32.  Byte b of a code, XOR 128,
// in the mantissa of 2^23 is 2^23 + 128 + c exactly; one subtraction leaves c.
static __device__ __forceinline__ void act_values8(uint2 q, uint32_t e, float (&v)[8])
{
    const float scale = __uint_as_float(e << 23);          // E = 255: inf, and 0 * inf = NaN
    const uint32_t w[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t m = __byte_perm(w[i / 4], 0x4B000000u, 0x7650 + (i % 4));
        v[i] = (__uint_as_float(m) - 8388736.0f) * scale;
    }
}

// ---- rows of 8-element chunks ----------------------------------------------------
// Eight elements of a row, elements at or past n (1..8 in range) read as 0.
// VEC: the address is 16-byte aligned and all eight lie in the row.
template <int DT>
static __device__ __forceinline__ float load1(const void* p, int64_t i)
{
    if (DT == 2) return __ldg(static_cast<const float*>(p) + i);
    return widen1<DT>(__ldg(static_cast<const uint16_t*>(p) + i));
}

template <int DT>
static __device__ __forceinline__ void load8(const void* p, int64_t i, int n, bool vec, float (&v)[8])
{
    if (vec && n >= 8) {
        if (DT == 2) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
            const float4 b = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i) + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 q = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
            widen2<DT & 1>(q.x, v[0], v[1]);
            widen2<DT & 1>(q.y, v[2], v[3]);
            widen2<DT & 1>(q.z, v[4], v[5]);
            widen2<DT & 1>(q.w, v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = j < n ? load1<DT>(p, i + j) : 0.0f;
    }
}

template <int DT>
static __device__ __forceinline__ void store8(void* p, int64_t i, int n, bool vec, const float (&v)[8])
{
    if (vec && n >= 8) {
        if (DT == 2) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
            __stcs(o, make_float4(v[0], v[1], v[2], v[3]));
            __stcs(o + 1, make_float4(v[4], v[5], v[6], v[7]));
        } else {
            __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i),
                   make_uint4(narrow2<DT & 1>(v[0], v[1]), narrow2<DT & 1>(v[2], v[3]),
                              narrow2<DT & 1>(v[4], v[5]), narrow2<DT & 1>(v[6], v[7])));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < n) {
                if (DT == 2) static_cast<float*>(p)[i + j] = v[j];
                else static_cast<uint16_t*>(p)[i + j] = narrow1<DT & 1>(v[j]);
            }
    }
}

// Quantize and store one 8-column chunk: the four lanes of a block (consecutive,
// lane % 4 the chunk's place in its block) agree on the exponent by two shuffles.
// `row` is the checkpoint's row, col the chunk's first column, wide the row's code
// bytes; elements past the row's end are 0 in v.  All 32 lanes of the warp take
// part; `live` lanes store.
static __device__ __forceinline__ void act_store_chunk(const float (&v)[8], uint8_t* row, int col, int wide,
                                                       int stride, int lo, int hi, bool live)
{
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (!live) return;
    const uint32_t e = act_exponent(m, lo, hi);
    const float step = act_step(e);
    const bool top = (int)e == hi, bad = e == ZERO_ACT_BAD;
    uint2 q;
    q.x = act_codes4(v[0], v[1], v[2], v[3], step, top, bad);
    q.y = act_codes4(v[4], v[5], v[6], v[7], step, top, bad);
    *reinterpret_cast<uint2*>(row + col) = q;
    const int sub = (col >> 3) & 3;
    if (sub == 0) row[wide + (col >> 5)] = (uint8_t)e;
    if (col + 8 * (4 - sub) == wide)                        // the row's last block
        for (int i = wide + (wide >> 5) + sub; i < stride; i += 4) row[i] = 0;
}

}  // namespace zero
