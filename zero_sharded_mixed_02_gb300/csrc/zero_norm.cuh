// zero_norm.cuh -- the norms around a block fused with its gate and residual scale,
// forward and backward kernels (include/zero_b200.h gives the formulas).
//
// Both passes read every tensor once and write each output once, so HBM bounds
// them: at full rate an SM has 40 to 50 instructions for an element.  A block of
// threads holds one row at a time in registers (8-column chunks as pairs of fp32 values,
// V chunks per thread), so the row's statistics and everything after them come from
// one read; arithmetic is on pairs; the next row's loads are issued before the current
// row's reductions, which would otherwise leave the memory system idle for their latency.
//
// The backward pass keeps the sums over rows (weight, bias and gate gradients) in
// registers while a block walks its contiguous range of rows; partial sums go to
// the workspace once per block, and per gate group a block crosses, and a second
// kernel adds them in a fixed order.  With S = sum D yh and S0 = sum D over a group's
// rows, dgate = alpha (post_w S + post_b S0), and dpost_w = sum over groups of
// alpha gate S, dpost_b of alpha gate S0: one pair of sums in registers serves all three.
#pragma once

#include "zero_act.cuh"
#include "zero_b200.h"

namespace zero {

#define ZERO_NORM_THREADS 512          // most threads of a block (one row)
#define ZERO_NORM_BLOCKS 608           // most blocks of the backward pass (its partial sums)

struct NormArgs {
    const void *h, *y, *post_w, *post_b, *gate, *pre_w, *pre_b;
    void *h_out, *x;
    uint8_t *ckpt_y, *ckpt_x;
    float* stats;
    uint32_t ldh, ldy, ldho, ldx;
    uint32_t rows, group;              // group >= 1
    int cols;
    uint32_t wide, stride;
    int lo, hi;
    int post, pre;
    float eps, alpha, inv_cols;
    int vec_h, vec_y, vec_ho, vec_x, vec_w, vec_g;
    const char *stop_h, *stop_y;       // ends of h and y
};

struct NormBwdArgs {
    const void *dh_out, *dx, *post_w, *gate, *pre_w;
    const uint8_t *ckpt_y, *ckpt_x;
    const float* stats;
    void *dh, *dy;
    float* pre_part;         // [blocks][sums][wide]: dx xh (and dx)
    float* post_part;        // the same: gate D yh (and gate D)
    float* slots;            // [blocks + groups][sums][wide]: S (and S0) of a block's rows of a group
    uint32_t lddho, lddx, lddh, lddy;
    uint32_t rows, group;
    int cols;
    uint32_t wide, stride;
    int post, pre;
    float alpha, inv_cols;
    int vec_dho, vec_dx, vec_dh, vec_dy, vec_w, vec_g;
};

// Kernels by type of the stream (DT or fp32), chunks per thread (1, 2, 4), the norms' kinds,
// and whether every row and weight is read in whole aligned chunks (and y or dy is there).
const void* norm_forward_fp16(int res, int v, int post, int pre, bool whole);
const void* norm_forward_bf16(int res, int v, int post, int pre, bool whole);
const void* norm_backward_fp16(int res, int v, int post, int pre, bool whole, bool copied, bool& two, int& smem);
const void* norm_backward_bf16(int res, int v, int post, int pre, bool whole, bool copied, bool& two, int& smem);

// Rows [row0(b), row0(b + 1)) belong to block b; the block of row r is the largest b with row0(b) <= r.
__host__ __device__ inline int64_t norm_row0(int64_t b, int64_t rows, int64_t blocks) { return b * rows / blocks; }
__host__ __device__ inline int64_t norm_block_of(int64_t r, int64_t rows, int64_t blocks)
{
    return ((r + 1) * blocks - 1) / rows;
}

// Eight weights (cached: every row of a block reads the same ones).
template <int DT, bool WHOLE>
static __device__ __forceinline__ void load_weights(const void* p, uint32_t i, int n, bool vec, float* stage,
                                                    f32x2_t (&v)[4])
{
    Raw<DT> r;
    if (WHOLE) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (n >= 8) q = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
        r.w[0] = q.x; r.w[1] = q.y; r.w[2] = q.z; r.w[3] = q.w;
        widen_chunk<DT>(r, v);
    } else {
        load_chunk<DT>(r, p, i, n, vec);
        widen_chunk<DT, false>(r, v, vec, stage);
    }
}

// Sums of N values over the block, the same bits in every thread: shuffles inside a
// warp, then every warp adds the warps' sums by the same shuffles.  One barrier; two
// buffers used in turn make a second one needless.
typedef float norm_buf_t[2][8][16];
template <int N>
static __device__ __forceinline__ void block_sum(float (&v)[N], norm_buf_t& buf, int& turn)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; i++) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (warps == 1) return;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; i++) buf[turn][i][threadIdx.x >> 5] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = (lane & 15) < warps ? buf[turn][i][lane & 15] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; i++) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
    turn ^= 1;
}

// Zeros past the row's end, n elements into the chunk.
static __device__ __forceinline__ void end_of_row(f32x2_t (&v)[4], int n)
{
    if (n >= 8) return;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        float a, b;
        unpack2(v[j], a, b);
        v[j] = pack2(2 * j < n ? a : 0.0f, 2 * j + 1 < n ? b : 0.0f);
    }
}

// 1/sqrt(x), the approximation refined by one step of Newton's method (an infinite or zero x
// keeps the approximation's 0 or inf; a square root and a division by the library's
// correctly rounded functions took a tenth of the forward pass's instructions).
static __device__ __forceinline__ float inverse_sqrt(float x)
{
    const float r = rsqrtf(x), t = __fmaf_rn(-x * r, r, 1.0f);
    return fabsf(t) < 1.0f ? __fmaf_rn(0.5f * r, t, r) : r;
}

static __device__ __forceinline__ void times(f32x2_t (&v)[4], f32x2_t w)
{
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = mul2(v[j], w);
}
static __device__ __forceinline__ void times(f32x2_t (&v)[4], const f32x2_t (&w)[4])
{
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = mul2(v[j], w[j]);
}
static __device__ __forceinline__ void plus(f32x2_t (&v)[4], const f32x2_t (&w)[4])
{
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = add2(v[j], w[j]);
}

// ---- weights in shared memory ------------------------------------------------------
static __device__ __forceinline__ uint4 shared16(uint32_t at)
{
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at));
    return q;
}
static __device__ __forceinline__ void put16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
static __device__ __forceinline__ void put_chunk(uint32_t at, uint32_t step, const f32x2_t (&v)[4])
{
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; j++) unpack2(v[j], x[2 * j], x[2 * j + 1]);
    put16(at, __float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    put16(at + step, __float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
}
static __device__ __forceinline__ void get_chunk(uint32_t at, uint32_t step, f32x2_t (&v)[4])
{
    const uint4 x = shared16(at), y = shared16(at + step);
    v[0] = pack2(__uint_as_float(x.x), __uint_as_float(x.y));
    v[1] = pack2(__uint_as_float(x.z), __uint_as_float(x.w));
    v[2] = pack2(__uint_as_float(y.x), __uint_as_float(y.y));
    v[3] = pack2(__uint_as_float(y.z), __uint_as_float(y.w));
}
// Eight 16-bit values.
template <int DT>
static __device__ __forceinline__ void get16(uint32_t at, f32x2_t (&v)[4])
{
    const uint4 q = shared16(at);
    Raw<DT> r;
    r.w[0] = q.x; r.w[1] = q.y; r.w[2] = q.z; r.w[3] = q.w;
    widen_chunk<DT>(r, v);
}
template <int DT>
static __device__ __forceinline__ void put_16(uint32_t at, const f32x2_t (&v)[4])
{
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; j++) unpack2(v[j], x[2 * j], x[2 * j + 1]);
    put16(at, narrow2<DT>(x[0], x[1]), narrow2<DT>(x[2], x[3]), narrow2<DT>(x[4], x[5]), narrow2<DT>(x[6], x[7]));
}

// The weights of a thread's chunk, as the passes use them, lie in shared memory as 16-byte
// words [word][thread]: 0, 1: u = gate post_w in fp32; 2: pre_w in 16 bits; and with biases
// 3, 4: gate post_b in fp32; 5: pre_b.  They are read from there each row: fewer
// instructions than loading and widening them, and L1 need not hold them.  u (and
// words 3, 4) are made again where the gate's group changes.  A thread reads what it wrote.
#define ZERO_NORM_WORDS 3
#define ZERO_NORM_WORDS_BIAS 6
template <int DT, bool WHOLE>
static __device__ __forceinline__ void put_gate(uint32_t at, uint32_t step, const void* gate, const void* post_w,
                                                const void* post_b, uint32_t i, int n, int vec_g, int vec_w,
                                                float* stage)
{
    f32x2_t g[4], u[4], w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) g[j] = both(1.0f);
    if (gate) load_weights<DT, WHOLE>(gate, i, n, vec_g, stage, g);
#pragma unroll
    for (int j = 0; j < 4; j++) u[j] = g[j];
    if (post_w) {
        load_weights<DT, WHOLE>(post_w, i, n, vec_w, stage, w);
        times(u, w);
    }
    end_of_row(u, n);
    put_chunk(at, step, u);
    if (post_b) {
        load_weights<DT, WHOLE>(post_b, i, n, vec_w, stage, w);
        times(w, g);
        put_chunk(at + 3 * step, step, w);
    }
}
template <int DT, bool WHOLE>
static __device__ __forceinline__ void put_pre(uint32_t at, const void* p, uint32_t i, int n, int vec_w, float* stage)
{
    f32x2_t w[4];
    load_weights<DT, WHOLE>(p, i, n, vec_w, stage, w);
    put_16<DT>(at, w);
}

// ---- forward ---------------------------------------------------------------------
// A row held as v (zeros past its end) is normalised; its mean and 1/deviation returned.
template <int V>
static __device__ __forceinline__ void normalise(f32x2_t (&v)[V][4], const int (&n)[V], int kind, float eps,
                                                 float inv_cols, float& mean, float& rstd, norm_buf_t& buf, int& turn)
{
    f32x2_t t = both(0.0f);
    float s[1];
    if (kind == ZERO_NORM_LAYER) {
#pragma unroll
        for (int c = 0; c < V; c++)
#pragma unroll
            for (int j = 0; j < 4; j++) t = add2(t, v[c][j]);
        s[0] = either(t);
        block_sum<1>(s, buf, turn);
        mean = s[0] * inv_cols;
        const f32x2_t less = both(-mean);
#pragma unroll
        for (int c = 0; c < V; c++) {
#pragma unroll
            for (int j = 0; j < 4; j++) v[c][j] = add2(v[c][j], less);
            end_of_row(v[c], n[c]);
        }
        t = both(0.0f);
    }
#pragma unroll
    for (int c = 0; c < V; c++)
#pragma unroll
        for (int j = 0; j < 4; j++) t = fma2(v[c][j], v[c][j], t);
    s[0] = either(t);
    block_sum<1>(s, buf, turn);
    rstd = inverse_sqrt(__fmaf_rn(s[0], inv_cols, eps));
#pragma unroll
    for (int c = 0; c < V; c++) times(v[c], both(rstd));
}

// POST and PRE: the norms' kinds (zero_norm_kind_t) for rows of whole aligned chunks with a
// block (y) in them; -1: any kinds, sizes and alignments, by the arguments.  Knowing them
// saves a fifth of the instructions, which bound the pass next to HBM.  Two blocks of one row
// an SM (16 warps each, 64 registers) beat one block of two rows at a time, which does
// fewer instructions (weights and branches shared) but leaves half the warps to hide
// latencies: 165 against 174 us at 16384 x 4096 with an fp32 stream.
template <int DT, int RT, int V, int POST, int PRE>
__global__ void __launch_bounds__(ZERO_NORM_THREADS, V == 1 ? 2 : 1)
    k_norm_forward(const __grid_constant__ NormArgs a)
{
    constexpr bool WHOLE = POST >= 0;
    const int post = WHOLE ? POST : a.post, pre = WHOLE ? PRE : a.pre;
    const bool block = WHOLE || a.y;
    __shared__ norm_buf_t buf;
    __shared__ __align__(16) float stages[WHOLE ? 1 : ZERO_NORM_THREADS / 32][256];
    float* stage = stages[WHOLE ? 0 : threadIdx.x >> 5];
    int turn = 0, n[V];
    uint32_t col[V];
#pragma unroll
    for (int c = 0; c < V; c++) {
        col[c] = 8 * (threadIdx.x + c * blockDim.x);
        n[c] = a.cols - (int)col[c];
    }
    Raw<RT> rh[V];
    Raw<DT> ry[V];
    // rows that are not whole aligned chunks: 16-bit ones as words (16384 x 1601 bf16: 115 -> 105 us,
    // 4096 x 6001: 154 -> 99; three words of an fp32 stream gain nothing: its rows are read column
    // by column through shared memory)
    Words<RT> wh[V];
    Words<DT> wy[V];
    uint32_t sh[V], sy[V];
    const uint32_t end = (uint32_t)norm_row0(blockIdx.x + 1, a.rows, gridDim.x);
    uint32_t row = (uint32_t)norm_row0(blockIdx.x, a.rows, gridDim.x);
    uint32_t grp = row / a.group, in_group = row - grp * a.group;
    auto fetch = [&](uint32_t at) {
        const void *ph = row_of<RT>(a.h, at, a.ldh), *py = row_of<DT>(a.y, at, a.ldy);
#pragma unroll
        for (int c = 0; c < V; c++) {
            if (WHOLE) {
                load_chunk<RT, true>(rh[c], ph, col[c], n[c], true);
                load_chunk<DT, true>(ry[c], py, col[c], n[c], true);
            } else {
                if (RT == 2) load_chunk<RT>(rh[c], ph, col[c], n[c], a.vec_h);
                else load_words<RT>(wh[c], sh[c], ph, col[c], n[c], a.h, a.stop_h);
                if (block) load_words<DT>(wy[c], sy[c], py, col[c], n[c], a.y, a.stop_y);
            }
        }
    };
    extern __shared__ __align__(128) unsigned char raw[];
    const uint32_t step = 16 * blockDim.x, words = (a.post_b || a.pre_b ? ZERO_NORM_WORDS_BIAS : ZERO_NORM_WORDS) * step;
    const uint32_t weights = (uint32_t)__cvta_generic_to_shared(raw) + 16 * threadIdx.x;
    auto refresh = [&]() {
        if (!a.gate && !a.post_w && !a.post_b) return;
        const void* gate = a.gate ? row_of<DT>(a.gate, grp, a.cols) : nullptr;
#pragma unroll
        for (int c = 0; c < V; c++)
            put_gate<DT, WHOLE>(weights + c * words, step, gate, a.post_w, a.post_b, col[c], n[c], a.vec_g, a.vec_w, stage);
    };
#pragma unroll
    for (int c = 0; c < V; c++) {
        if (a.pre_w) put_pre<DT, WHOLE>(weights + c * words + 2 * step, a.pre_w, col[c], n[c], a.vec_w, stage);
        if (a.pre_b) put_pre<DT, WHOLE>(weights + c * words + 5 * step, a.pre_b, col[c], n[c], a.vec_w, stage);
    }
    refresh();
    fetch(row);
    for (; row < end; row++) {
        f32x2_t h[V][4], y[V][4], w[4];
#pragma unroll
        for (int c = 0; c < V; c++) {
            if (!WHOLE) {
                if (RT != 2) from_words<RT>(rh[c], wh[c], sh[c], n[c]);
                else if (!a.vec_h) unstage<RT>(rh[c], stage);
                if (block) from_words<DT>(ry[c], wy[c], sy[c], n[c]);
            }
            widen_chunk<RT>(rh[c], h[c]);
            if (block) widen_chunk<DT>(ry[c], y[c]);
        }
        if (row + 1 < end) fetch(row + 1);
        float mu2 = 0.0f, r2 = 1.0f, mu1 = 0.0f, r1 = 1.0f;
        if (block) {
            if (post) normalise<V>(y, n, post, a.eps, a.inv_cols, mu2, r2, buf, turn);
#pragma unroll
            for (int c = 0; c < V; c++) {
                if (a.ckpt_y) {
                    uint8_t* p = a.ckpt_y + (int64_t)row * a.stride;
                    if (post) act_store_small(y[c], p, col[c], a.wide, a.stride, a.lo, col[c] < a.wide);
                    else act_store(y[c], p, col[c], a.wide, a.stride, a.lo, a.hi, col[c] < a.wide);
                }
                if (a.gate || a.post_w) {
                    get_chunk(weights + c * words, step, w);
                    times(y[c], w);
                }
                if (a.post_b) {
                    get_chunk(weights + c * words + 3 * step, step, w);
                    plus(y[c], w);
                }
                const f32x2_t alpha = both(a.alpha);
#pragma unroll
                for (int j = 0; j < 4; j++) h[c][j] = fma2(alpha, y[c][j], h[c][j]);
            }
        }
        if (WHOLE || a.h_out) {
            const void* p = row_of<RT>(a.h_out, row, a.ldho);
#pragma unroll
            for (int c = 0; c < V; c++) store_chunk<RT, WHOLE>(p, col[c], n[c], a.vec_ho, stage, h[c]);
        }
        if (pre) {
            normalise<V>(h, n, pre, a.eps, a.inv_cols, mu1, r1, buf, turn);
            const void* px = row_of<DT>(a.x, row, a.ldx);
#pragma unroll
            for (int c = 0; c < V; c++) {
                if (a.ckpt_x)
                    act_store_small(h[c], a.ckpt_x + (int64_t)row * a.stride, col[c], a.wide, a.stride, a.lo,
                                    col[c] < a.wide);
                if (a.pre_w) {
                    get16<DT>(weights + c * words + 2 * step, w);
                    times(h[c], w);
                }
                if (a.pre_b) {
                    get16<DT>(weights + c * words + 5 * step, w);
                    plus(h[c], w);
                }
                store_chunk<DT, WHOLE>(px, col[c], n[c], a.vec_x, stage, h[c]);
            }
        }
        if (a.stats && threadIdx.x == 0)
            reinterpret_cast<float4*>(a.stats)[row] = make_float4(mu2, r2, mu1, r1);
        if (++in_group == a.group && row + 1 < end) {
            in_group = 0;
            grp++;
            if (a.gate) refresh();
        }
    }
}

// ---- backward --------------------------------------------------------------------
static __device__ __forceinline__ void put_sums(float* p, const f32x2_t (&v)[4])
{
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; j++) unpack2(v[j], x[2 * j], x[2 * j + 1]);
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

static __device__ __forceinline__ void get_sums(const float* p, f32x2_t (&v)[4])
{
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const float4 q = reinterpret_cast<const float4*>(p)[j];
        v[2 * j] = add2(pack2(q.x, q.y), v[2 * j]);
        v[2 * j + 1] = add2(pack2(q.z, q.w), v[2 * j + 1]);
    }
}

// One reduction a row serves both norms.  With g = pre_w dx, u = gate post_w and
// B = dh_out + r1 g,
//   D = B - r1 (mean(g) + mean(g xh) xh),
// so the post-norm's sums of u D and u D yh follow from sums that do not need D:
//   sum u yh D = sum u yh B - r1 (mean(g) sum u yh + mean(g xh) sum u yh xh)
// and the same without yh.  A second reduction, after D, would cost its latency once more.
//
template <int DT, int RT, int V, bool TWO>
__global__ void __launch_bounds__(ZERO_NORM_THREADS, 1) k_norm_backward(const __grid_constant__ NormBwdArgs a)
{
    // one wave of blocks: the kernel that adds their sums may be placed already
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr bool WHOLE = false;
    const int post = a.post, pre = a.pre;
    __shared__ norm_buf_t buf;
    __shared__ __align__(16) float stages[WHOLE ? 1 : ZERO_NORM_THREADS / 32][256];
    float* stage = stages[WHOLE ? 0 : threadIdx.x >> 5];
    constexpr int SUMS = TWO ? 2 : 1;
    // with more than one chunk a thread, what follows from the codes and weights is made again
    // after the reduction rather than held across it
    constexpr bool AGAIN = V > 1;
    constexpr int KEEP = AGAIN ? 1 : V;
    int turn = 0, n[V];
    uint32_t col[V];
    f32x2_t pw[V][4], sw[V][4], pb[TWO ? V : 1][4], sb[TWO ? V : 1][4];
#pragma unroll
    for (int c = 0; c < V; c++) {
        col[c] = 8 * (threadIdx.x + c * blockDim.x);
        n[c] = a.cols - (int)col[c];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            pw[c][j] = sw[c][j] = both(0.0f);
            if (TWO) pb[c][j] = sb[c][j] = both(0.0f);
        }
    }
    const uint32_t end = (uint32_t)norm_row0(blockIdx.x + 1, a.rows, gridDim.x);
    uint32_t row = (uint32_t)norm_row0(blockIdx.x, a.rows, gridDim.x);
    uint32_t grp = row / a.group, left = (grp + 1) * a.group - row;         // rows of the group to come
    Raw<RT> rd[V];
    Raw<DT> rx[V];
    uint2 qx[V], qy[V];
    uint32_t ex[V], ey[V];
    float r1 = 1.0f, r2 = 1.0f;
    auto fetch = [&](uint32_t r) {
        const uint8_t *px = a.ckpt_x + (int64_t)r * a.stride, *py = a.ckpt_y + (int64_t)r * a.stride;
        const void *pd = row_of<RT>(a.dh_out, r, a.lddho), *pdx = row_of<DT>(a.dx, r, a.lddx);
#pragma unroll
        for (int c = 0; c < V; c++) {
            if (a.dh_out) load_chunk<RT, WHOLE>(rd[c], pd, col[c], n[c], a.vec_dho);
            if (pre) load_chunk<DT, WHOLE>(rx[c], pdx, col[c], n[c], a.vec_dx);
            qx[c] = qy[c] = make_uint2(0, 0);
            ex[c] = ey[c] = 0;
            if (n[c] > 0) {
                if (pre) {
                    qx[c] = __ldcs(reinterpret_cast<const uint2*>(px + col[c]));
                    ex[c] = __ldg(px + a.wide + (col[c] >> 5));
                }
                if (a.ckpt_y) {
                    qy[c] = __ldcs(reinterpret_cast<const uint2*>(py + col[c]));
                    ey[c] = __ldg(py + a.wide + (col[c] >> 5));
                }
            }
        }
        if (a.stats) {
            const float4 st = __ldg(reinterpret_cast<const float4*>(a.stats) + r);
            r2 = st.y;
            r1 = st.w;
        }
    };
    extern __shared__ __align__(128) unsigned char raw[];
    const uint32_t step = 16 * blockDim.x, words = ZERO_NORM_WORDS * step;
    const uint32_t weights = (uint32_t)__cvta_generic_to_shared(raw) + 16 * threadIdx.x;
    auto refresh = [&]() {
        const void* gate = a.gate ? row_of<DT>(a.gate, grp, a.cols) : nullptr;
#pragma unroll
        for (int c = 0; c < V; c++)
            put_gate<DT, WHOLE>(weights + c * words, step, gate, post ? a.post_w : nullptr, nullptr, col[c], n[c], a.vec_g,
                                a.vec_w, stage);
    };
    auto scales = [&](int c, f32x2_t (&u)[4]) { get_chunk(weights + c * words, step, u); };
    if (a.pre_w)
#pragma unroll
        for (int c = 0; c < V; c++)
            put_pre<DT, WHOLE>(weights + c * words + 2 * step, a.pre_w, col[c], n[c], a.vec_w, stage);
    refresh();
    // The sums of the block's rows of group grp go to the slot block + group: along the
    // rows both only grow, so no two pairs share one.  Times the group's gate they are
    // added to the block's sums for the post-norm's weights, which stay in the workspace
    // (a group seldom ends inside a block).
    bool again = false;
    auto flush = [&]() {
#pragma unroll
        for (int c = 0; c < V; c++) {
            f32x2_t w[4];
            if (a.post_part && a.gate)                       // all lanes: a warp reads together
                load_weights<DT, WHOLE>(row_of<DT>(a.gate, grp, a.cols), col[c], n[c], a.vec_g, stage, w);
            if (col[c] >= a.wide) continue;
            if (a.slots) {
                float* p = a.slots + ((int64_t)blockIdx.x + grp) * SUMS * a.wide + col[c];
                put_sums(p, sw[c]);
                if (TWO) put_sums(p + a.wide, sb[c]);
            }
            if (a.post_part) {
                float* p = a.post_part + (int64_t)blockIdx.x * SUMS * a.wide + col[c];
                if (a.gate) {
                    times(sw[c], w);
                    if (TWO) times(sb[c], w);
                }
                if (again) {
                    get_sums(p, sw[c]);
                    if (TWO) get_sums(p + a.wide, sb[c]);
                }
                put_sums(p, sw[c]);
                if (TWO) put_sums(p + a.wide, sb[c]);
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                sw[c][j] = both(0.0f);
                if (TWO) sb[c][j] = both(0.0f);
            }
        }
        again = true;
    };
    const bool sums = a.slots || a.post_part, layer = pre == ZERO_NORM_LAYER || post == ZERO_NORM_LAYER;
    fetch(row);
    for (; row < end; row++) {
        if (left == 0) {
            if (sums) flush();
            grp++;
            left = a.group;
            if (a.gate) refresh();
        }
        left--;
        f32x2_t b[V][4], u[KEEP][4], xh[KEEP][4], yh[KEEP][4], t[8];
        const float k1 = r1, k2 = r2;
        uint2 cx[V], cy[V];                                  // the row's codes, when read again after the sums
        uint32_t fx[V], fy[V];
#pragma unroll
        for (int k = 0; k < 8; k++) t[k] = both(0.0f);
#pragma unroll
        for (int c = 0; c < V; c++) {
            const int q = AGAIN ? 0 : c;
            f32x2_t w[4];
            if (pre) {                                       // b = g
                widen_chunk<DT, WHOLE>(rx[c], b[c], a.vec_dx, stage);
                act_values(qx[c], ex[c], xh[q]);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    pw[c][j] = fma2(b[c][j], xh[q][j], pw[c][j]);
                    if (TWO) pb[c][j] = add2(pb[c][j], b[c][j]);
                }
                if (a.pre_w) {
                    get16<DT>(weights + c * words + 2 * step, w);
                    times(b[c], w);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) b[c][j] = xh[q][j] = both(0.0f);
            }
            act_values(qy[c], ey[c], yh[q]);
            scales(c, u[q]);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (pre) t[0] = fma2(b[c][j], xh[q][j], t[0]);
                if (pre == ZERO_NORM_LAYER) t[3] = add2(t[3], b[c][j]);
                w[j] = both(0.0f);
            }
            if (a.dh_out) widen_chunk<RT, WHOLE>(rd[c], w, a.vec_dho, stage);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                b[c][j] = fma2(both(k1), b[c][j], w[j]);     // b = B
                if (post) {
                    const f32x2_t uy = mul2(u[q][j], yh[q][j]);
                    t[1] = fma2(uy, b[c][j], t[1]);
                    if (pre) t[2] = fma2(uy, xh[q][j], t[2]);
                    if (pre == ZERO_NORM_LAYER) t[4] = add2(t[4], uy);
                }
                if (post == ZERO_NORM_LAYER) {
                    t[5] = fma2(u[q][j], b[c][j], t[5]);
                    if (pre == ZERO_NORM_LAYER) t[6] = add2(t[6], u[q][j]);
                    if (pre) t[7] = fma2(u[q][j], xh[q][j], t[7]);
                }
            }
            if (AGAIN) {
                cx[c] = qx[c]; cy[c] = qy[c];
                fx[c] = ex[c]; fy[c] = ey[c];
            }
        }
        if (row + 1 < end) fetch(row + 1);
        float s[8];
#pragma unroll
        for (int k = 0; k < 8; k++) s[k] = either(t[k]);
        if (layer) {
            block_sum<8>(s, buf, turn);
        } else {
            float three[3] = {s[0], s[1], s[2]};
            block_sum<3>(three, buf, turn);
            s[0] = three[0];
            s[1] = three[1];
            s[2] = three[2];
        }
        // D = b - p1 xh - p0;  dy = alpha r2 (u D - q1 yh - q0)
        const float p1 = k1 * s[0] * a.inv_cols, p0 = pre == ZERO_NORM_LAYER ? k1 * s[3] * a.inv_cols : 0.0f;
        const void *pdh = row_of<RT>(a.dh, row, a.lddh), *pdy = row_of<DT>(a.dy, row, a.lddy);
        float scale = a.alpha, q1 = 0.0f, q0 = 0.0f;
        if (post) {
            scale *= k2;
            q1 = (s[1] - p0 * s[4] - p1 * s[2]) * a.inv_cols;
            if (post == ZERO_NORM_LAYER) q0 = (s[5] - p0 * s[6] - p1 * s[7]) * a.inv_cols;
        }
#pragma unroll
        for (int c = 0; c < V; c++) {
            const int q = AGAIN ? 0 : c;
            if (AGAIN) {
                // (the empty statement keeps the compiler from holding the first reading)
                asm volatile("" : "+r"(cx[c].x), "+r"(cx[c].y), "+r"(cy[c].x), "+r"(cy[c].y));
                act_values(cx[c], fx[c], xh[q]);
                act_values(cy[c], fy[c], yh[q]);
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (pre == ZERO_NORM_LAYER) b[c][j] = sub2(b[c][j], both(p0));
                b[c][j] = fma2(both(-p1), xh[q][j], b[c][j]);
            }
            if (a.dh) store_chunk<RT, WHOLE>(pdh, col[c], n[c], a.vec_dh, stage, b[c]);
            if (!WHOLE && !a.dy) continue;
            if (sums)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    sw[c][j] = fma2(b[c][j], yh[q][j], sw[c][j]);
                    if (TWO) sb[c][j] = add2(sb[c][j], b[c][j]);
                }
            if (AGAIN) scales(c, u[q]);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                f32x2_t e = post == ZERO_NORM_LAYER ? fma2(u[q][j], b[c][j], both(-q0)) : mul2(u[q][j], b[c][j]);
                if (post) e = fma2(both(-q1), yh[q][j], e);
                b[c][j] = mul2(both(scale), e);
            }
            store_chunk<DT, WHOLE>(pdy, col[c], n[c], a.vec_dy, stage, b[c]);
        }
    }
    if (sums) flush();
    if (a.pre_part) {
        float* p = a.pre_part + (int64_t)blockIdx.x * SUMS * a.wide;
#pragma unroll
        for (int c = 0; c < V; c++)
            if (col[c] < a.wide) {
                put_sums(p + col[c], pw[c]);
                if (TWO) put_sums(p + a.wide + col[c], pb[c]);
            }
    }
}

// ---- backward, rows that are copied ahead ------------------------------------------
// The next rows' chunks are copied to shared memory asynchronously instead of being held in
// registers, and what the reduction separates, codes and weights, is read from there again.
// That leaves 64 registers enough without bias sums: two blocks of 16 warps an SM instead of
// one.
//
// A thread's part of a row is three 16-byte words [word][thread] (dx, both checkpoints' codes,
// and the stream's gradient if that is of 16 bits); it reads what it copied itself, so there
// is no barrier for the copies.  An fp32 stream's 1 KB a warp is copied 16 neighbouring bytes
// a lane and read 32 bytes a lane (copies 32 bytes apart would fetch every sector twice);
// word p lies at p ^ (p >> 3 & 1), so that eight lanes' reads fall on different banks.
//
// Rows of other sizes and alignments (ANY): a 16-bit row's words are copied from the 16-byte
// boundary at or before its start, one word more than it has chunks, and a thread shifts its
// chunk out of its own word and the next thread's; rows are copied one row earlier, so that a
// row's barrier shows the next row's words to all threads.  A word that reaches into the rows
// before or after is copied whole; only the matrix's first and last are taken element by
// element.  An fp32 stream is copied element by element (4 bytes).  2047 x 1601, fp16, two layer
// norms with biases: 35 us instead of 44 in the general kernel; 16384 x 1601, bf16: 115 instead of 221.
static __device__ __forceinline__ void copy16(uint32_t to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
static __device__ __forceinline__ void copy8(uint32_t to, const void* from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
// Sums of four values over the block, the same bits in every thread.  A warp halves the
// values a lane holds with each of the first two exchanges, so a group of eight lanes ends
// with one value's sum: half the shuffles of four sums side by side.
typedef float norm_buf4_t[2][4][16];
static __device__ __forceinline__ void block_sum4(float (&v)[4], norm_buf4_t& buf, int& turn)
{
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const bool hi = lane & 16, odd = lane & 8;
    float a = hi ? v[2] : v[0], b = hi ? v[3] : v[1];
    a += __shfl_xor_sync(0xFFFFFFFFu, hi ? v[0] : v[2], 16);
    b += __shfl_xor_sync(0xFFFFFFFFu, hi ? v[1] : v[3], 16);
    float c = (odd ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 8);   // value lane / 8
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
    if (warps > 1) {
        const int w = lane & 7;
        if (w == 0) buf[turn][lane >> 3][threadIdx.x >> 5] = c;
        __syncthreads();
        c = w < warps ? buf[turn][lane >> 3][w] : 0.0f;
        if (w + 8 < warps) c += buf[turn][lane >> 3][w + 8];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
        turn ^= 1;
    }
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = __shfl_sync(0xFFFFFFFFu, c, 8 * i);
}

#ifndef ZERO_NORM_AHEAD
#define ZERO_NORM_AHEAD 2                                    // rows in shared memory
#endif
#define ZERO_NORM_PART 48                                    // bytes of a thread's part of a chunk
// Shared memory of a thread: its parts of the rows (an fp32 stream 32 bytes more) and weights.
template <int RT, int V, bool ANY> struct NormRing {
    static constexpr int bytes = V * ((ZERO_NORM_PART + (RT == 2 ? 32 : 0)) * (ZERO_NORM_AHEAD + ANY) + ZERO_NORM_PART);
};

// With rows of any alignment: bytes of a thread and chunk.
static inline int64_t norm_ring_bytes(int res) { return res == 2 ? NormRing<2, 1, true>::bytes : NormRing<0, 1, true>::bytes; }

template <int DT, int RT, int V, int POST, int PRE, bool TWO, bool ANY>
__global__ void __launch_bounds__(ZERO_NORM_THREADS, V == 1 && !TWO && !ANY ? 2 : 1)
    k_norm_backward_whole(const __grid_constant__ NormBwdArgs a)
{
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int SUMS = TWO ? 2 : 1, PART = ZERO_NORM_PART, AHEAD = ZERO_NORM_AHEAD + ANY;
    constexpr bool LAYER = PRE == ZERO_NORM_LAYER || POST == ZERO_NORM_LAYER, WIDE = RT == 2;
    extern __shared__ __align__(128) unsigned char raw[];
    __shared__ norm_buf4_t buf, buf2;
    __shared__ __align__(16) float stages[ANY ? ZERO_NORM_THREADS / 32 : 1][256];
    float* stage = stages[ANY ? threadIdx.x >> 5 : 0];
    const uint32_t threads = blockDim.x, t = threadIdx.x, lane = t & 31;
    // [weights][AHEAD rows: parts, then an fp32 stream], each chunk c of the V after the other
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(raw);
    const uint32_t row_bytes = V * threads * (PART + (WIDE ? 32 : 0)), first = base + V * threads * PART;
    const uint32_t weights = base + 16 * t, part = first + 16 * t, T16 = 16 * threads;
    const uint32_t wide = first + V * threads * PART + (t & ~31u) * 32;                  // the warp's words
    const uint32_t mine = wide + ((2 * lane) ^ (lane >> 2 & 1)) * 16;                    // words 2 lane, 2 lane + 1
    int turn = 0, turn2 = 0;
    f32x2_t pw[V][4], sw[V][4], pb[TWO ? V : 1][4], sb[TWO ? V : 1][4];
#pragma unroll
    for (int c = 0; c < V; c++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            pw[c][j] = sw[c][j] = both(0.0f);
            if (TWO) pb[c][j] = sb[c][j] = both(0.0f);
        }
    const uint32_t end = (uint32_t)norm_row0(blockIdx.x + 1, a.rows, gridDim.x);
    uint32_t row = (uint32_t)norm_row0(blockIdx.x, a.rows, gridDim.x);
    uint32_t grp = row / a.group, left = (grp + 1) * a.group - row;         // rows of the group to come
    auto chunk = [&](int c) { return t + c * threads; };
    auto in = [&](int c) { return 8 * chunk(c) < (uint32_t)a.cols; };
    auto left_of = [&](int c) { return ANY ? a.cols - 8 * (int)chunk(c) : in(c) ? 8 : 0; };   // columns from the chunk's first
    // the next chunk's word: the next thread's, after the last thread the first's of the chunks
    // after (after all chunks there is none, and nothing that needs it)
    auto next = [&](int c) { return t + 1 < threads ? 16 : c + 1 < V ? threads * PART - 16 * t : 0; };
    // rows' addresses, the same in all threads and advanced row by row
    const char *ld = static_cast<const char*>(row_of<RT>(a.dh_out, row, a.lddho));
    const char *lx = static_cast<const char*>(row_of<DT>(a.dx, row, a.lddx));
    const uint8_t *qx = a.ckpt_x + (int64_t)row * a.stride, *qy = a.ckpt_y + (int64_t)row * a.stride;
    const int64_t ld_step = (int64_t)a.lddho * (WIDE ? 4 : 2), lx_step = (int64_t)a.lddx * 2;
    uint32_t copied = row, slot = 0;                         // the next row to copy and its place
    // ANY: the word of chunk k of a 16-bit row
    auto word = [&](uint32_t to, const char* line, uint32_t k, const void* matrix, int64_t step) {
        const uint32_t sh = (uint32_t)(uintptr_t)line & 15;
        const char* from = line + 16 * k - sh;
        const int off = 16 * (int)k - (int)sh, size = 2 * a.cols;
        if (off >= size) return;
        const char *begin = static_cast<const char*>(matrix), *stop = begin + (a.rows - 1) * step + size;
        if (from >= begin && from + 16 <= stop) {
            copy16(to, from);
            return;
        }
        for (int e = 0; e < 16; e += 2)                      // a matrix's first or last word
            if (off + e >= 0 && off + e < size) {
                const uint16_t v = __ldg(reinterpret_cast<const uint16_t*>(from + e));
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + e), "h"(v) : "memory");
            }
    };
    auto copy = [&]() {
        if (copied < end) {
#pragma unroll
            for (int c = 0; c < V; c++) {
                const uint32_t at = part + slot + c * threads * PART, k = chunk(c);
                if (in(c)) {
                    if (PRE && !ANY) copy16(at, lx + 16 * k);
                    if (PRE) copy8(at + T16, qx + 8 * k);
                    if (a.ckpt_y) copy8(at + T16 + 8, qy + 8 * k);
                    if (!ANY && !WIDE && a.dh_out) copy16(at + 2 * T16, ld + 16 * k);
                }
                if (ANY) {
                    if (PRE) word(at, lx, k, a.dx, lx_step);
                    if (!WIDE && a.dh_out) word(at + 2 * T16, ld, k, a.dh_out, ld_step);
                }
                if (ANY && WIDE && a.dh_out) {
                    const uint32_t w = (t & ~31u) + c * threads, to = wide + slot + c * threads * 32;
#pragma unroll
                    for (int h = 0; h < 8; h++) {
                        const uint32_t e = lane + 32 * h, p = e >> 2;
                        if (8 * w + e < (uint32_t)a.cols)
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                                         ::"r"(to + (p ^ (p >> 3 & 1)) * 16 + (e & 3) * 4), "l"(ld + 32 * w + 4 * e) : "memory");
                    }
                } else if (WIDE && a.dh_out) {
                    // words lane and lane + 32 of the warp's 64: columns 4 p
                    const uint32_t w = (t & ~31u) + c * threads, to = wide + slot + c * threads * 32;
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t p = lane + 32 * h;
                        if (8 * w + 4 * p < (uint32_t)a.cols) copy16(to + (p ^ (p >> 3 & 1)) * 16, ld + 32 * w + 16 * p);
                    }
                }
            }
            ld += ld_step;
            lx += lx_step;
            qx += a.stride;
            qy += a.stride;
        }
        copied++;
        slot = slot + row_bytes == AHEAD * row_bytes ? 0 : slot + row_bytes;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // exponents and statistics come by registers, a row ahead
    const uint8_t *lex = qx + a.wide, *ley = qy + a.wide;
    const float4* stats = reinterpret_cast<const float4*>(a.stats) + row;
    uint32_t ex[V], ey[V];
    float r1, r2;
    auto fetch = [&]() {
#pragma unroll
        for (int c = 0; c < V; c++) {
            ex[c] = ey[c] = 0;
            if (in(c)) {
                if (PRE) ex[c] = __ldg(lex + (chunk(c) >> 2));
                if (a.ckpt_y) ey[c] = __ldg(ley + (chunk(c) >> 2));
            }
        }
        const float4 st = __ldg(stats);
        r2 = st.y;
        r1 = st.w;
        lex += a.stride;
        ley += a.stride;
        stats++;
    };
    // zeros where no copy comes: chunks past the row's end, tensors that are not there
    for (uint32_t i = t; i < AHEAD * row_bytes / 16; i += threads) put16(first + 16 * i, 0, 0, 0, 0);
    __syncthreads();
    auto refresh = [&]() {
        const void* gate = a.gate ? row_of<DT>(a.gate, grp, a.cols) : nullptr;
#pragma unroll
        for (int c = 0; c < V; c++)
            put_gate<DT, !ANY>(weights + c * threads * PART, T16, gate, POST ? a.post_w : nullptr, nullptr, 8 * chunk(c),
                               left_of(c), ANY ? a.vec_g : 1, ANY ? a.vec_w : 1, stage);
    };
    auto scales = [&](int c, f32x2_t (&u)[4]) { get_chunk(weights + c * threads * PART, T16, u); };
    auto widen16 = [&](uint32_t at, f32x2_t (&v)[4]) { get16<DT>(at, v); };
    if (PRE && a.pre_w)
#pragma unroll
        for (int c = 0; c < V; c++)
            put_pre<DT, !ANY>(weights + c * threads * PART + 2 * T16, a.pre_w, 8 * chunk(c), left_of(c), ANY ? a.vec_w : 1, stage);
    refresh();
    // as in the general kernel: the group's sums to their slot, times the gate to the block's
    const bool sums = a.slots || a.post_part;
    bool again = false;
    auto flush = [&]() {
#pragma unroll
        for (int c = 0; c < V; c++) {
            const uint32_t k = 8 * chunk(c);
            f32x2_t w[4];
            if (ANY && a.post_part && a.gate)                // all lanes: a warp reads together
                load_weights<DT, !ANY>(row_of<DT>(a.gate, grp, a.cols), k, left_of(c), a.vec_g, stage, w);
            if (k < a.wide) {
                if (a.slots) {
                    float* p = a.slots + ((int64_t)blockIdx.x + grp) * SUMS * a.wide + k;
                    put_sums(p, sw[c]);
                    if (TWO) put_sums(p + a.wide, sb[c]);
                }
                if (a.post_part) {
                    float* p = a.post_part + (int64_t)blockIdx.x * SUMS * a.wide + k;
                    if (a.gate) {
                        if (!ANY) load_weights<DT, !ANY>(row_of<DT>(a.gate, grp, a.cols), k, left_of(c), 1, nullptr, w);
                        times(sw[c], w);
                        if (TWO) times(sb[c], w);
                    }
                    if (again) {
                        get_sums(p, sw[c]);
                        if (TWO) get_sums(p + a.wide, sb[c]);
                    }
                    put_sums(p, sw[c]);
                    if (TWO) put_sums(p + a.wide, sb[c]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                sw[c][j] = both(0.0f);
                if (TWO) sb[c][j] = both(0.0f);
            }
        }
        again = true;
    };
    char* sd = static_cast<char*>(const_cast<void*>(row_of<RT>(a.dh, row, a.lddh)));
    char* sy = static_cast<char*>(const_cast<void*>(row_of<DT>(a.dy, row, a.lddy)));
    const int64_t sd_step = (int64_t)a.lddh * (WIDE ? 4 : 2), sy_step = (int64_t)a.lddy * 2;
#pragma unroll
    for (int k = 0; k < AHEAD; k++) copy();
    fetch();
    if (ANY) {                                               // the first row's words, of all threads
        asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
        __syncthreads();
    }
    const uint32_t shift_x = (uint32_t)(uintptr_t)a.dx, shift_d = (uint32_t)(uintptr_t)a.dh_out;
    uint32_t at = 0;                                         // the row's place
    for (; row < end; row++) {
        if (left == 0) {
            if (sums) flush();
            grp++;
            left = a.group;
            if (a.gate) refresh();
        }
        left--;
        // ANY: the next row's words too, before the barrier of this row's sums
        asm volatile("cp.async.wait_group %0;" ::"n"(ZERO_NORM_AHEAD - 1) : "memory");
        if (WIDE || ANY) __syncwarp();                       // the warp's words are all there
        f32x2_t b[V][4], u[4], xh[4], yh[4], w[4], s2[8];
        const float k1 = r1, k2 = r2;
        uint32_t fx[V], fy[V];
#pragma unroll
        for (int k = 0; k < 8; k++) s2[k] = both(0.0f);
#pragma unroll
        for (int c = 0; c < V; c++) {
            const uint32_t p = part + at + c * threads * PART;
            const uint4 q = shared16(p + T16);
            fx[c] = ex[c];
            fy[c] = ey[c];
            if (PRE) {
                if (ANY) {
                    const uint4 x = shifted(shared16(p), shared16(p + next(c)), (shift_x + row * (uint32_t)lx_step) & 15);
                    Raw<DT> r;
                    r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
                    widen_chunk<DT>(r, b[c]);
                    end_of_row(b[c], left_of(c));
                } else {
                    widen16(p, b[c]);                            // dx, then g, then B
                }
                act_values(make_uint2(q.x, q.y), ex[c], xh);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    pw[c][j] = fma2(b[c][j], xh[j], pw[c][j]);
                    if (TWO) pb[c][j] = add2(pb[c][j], b[c][j]);
                }
                if (a.pre_w) {
                    widen16(weights + c * threads * PART + 2 * T16, w);
                    times(b[c], w);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) b[c][j] = xh[j] = both(0.0f);
            }
            if (WIDE) {
                const uint32_t m = mine + at + c * threads * 32;
                get_chunk(m, (m ^ 16) - m, w);
            } else if (ANY) {
                const uint4 x = shifted(shared16(p + 2 * T16), shared16(p + 2 * T16 + next(c)), (shift_d + row * (uint32_t)ld_step) & 15);
                Raw<DT> r;
                r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
                widen_chunk<DT>(r, w);
                end_of_row(w, left_of(c));
            } else {
                widen16(p + 2 * T16, w);
            }
            if (POST) {
                act_values(make_uint2(q.z, q.w), ey[c], yh);
                scales(c, u);
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (PRE) s2[0] = fma2(b[c][j], xh[j], s2[0]);
                if (PRE == ZERO_NORM_LAYER) s2[3] = add2(s2[3], b[c][j]);
                b[c][j] = PRE ? fma2(both(k1), b[c][j], w[j]) : w[j];
                if (POST) {
                    const f32x2_t uy = mul2(u[j], yh[j]);
                    s2[1] = fma2(uy, b[c][j], s2[1]);
                    if (PRE) s2[2] = fma2(uy, xh[j], s2[2]);
                    if (LAYER) s2[4] = add2(s2[4], uy);
                }
                if (POST == ZERO_NORM_LAYER) {
                    s2[5] = fma2(u[j], b[c][j], s2[5]);
                    s2[6] = add2(s2[6], u[j]);
                    s2[7] = fma2(u[j], xh[j], s2[7]);
                }
            }
        }
        if (row + 1 < end) fetch();
        float s[4] = {either(s2[0]), either(s2[1]), either(s2[2]), either(s2[3])};
        float l[4] = {either(s2[4]), either(s2[5]), either(s2[6]), either(s2[7])};
        block_sum4(s, buf, turn);
        if (LAYER && POST) block_sum4(l, buf2, turn2);
        // D = b - p1 xh - p0;  dy = alpha r2 (u D - q1 yh - q0)
        const float p1 = k1 * s[0] * a.inv_cols, p0 = PRE == ZERO_NORM_LAYER ? k1 * s[3] * a.inv_cols : 0.0f;
        float scale = a.alpha, q1 = 0.0f, q0 = 0.0f;
        if (POST) {
            scale *= k2;
            q1 = (s[1] - p0 * l[0] - p1 * s[2]) * a.inv_cols;
            if (POST == ZERO_NORM_LAYER) q0 = (l[1] - p0 * l[2] - p1 * l[3]) * a.inv_cols;
        }
#pragma unroll
        for (int c = 0; c < V; c++) {
            const uint32_t k = chunk(c);
            const uint4 q = shared16(part + at + c * threads * PART + T16);
            act_values(make_uint2(q.x, q.y), fx[c], xh);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (PRE == ZERO_NORM_LAYER) b[c][j] = sub2(b[c][j], both(p0));
                if (PRE) b[c][j] = fma2(both(-p1), xh[j], b[c][j]);
            }
            if (a.dh) store_chunk<RT, !ANY>(sd, 8 * k, left_of(c), ANY ? a.vec_dh : true, stage, b[c]);
            act_values(make_uint2(q.z, q.w), fy[c], yh);
            if (sums)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    sw[c][j] = fma2(b[c][j], yh[j], sw[c][j]);
                    if (TWO) sb[c][j] = add2(sb[c][j], b[c][j]);
                }
            scales(c, u);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                f32x2_t e = POST == ZERO_NORM_LAYER ? fma2(u[j], b[c][j], both(-q0)) : mul2(u[j], b[c][j]);
                if (POST) e = fma2(both(-q1), yh[j], e);
                b[c][j] = mul2(both(scale), e);
            }
            store_chunk<DT, !ANY>(sy, 8 * k, left_of(c), ANY ? a.vec_dy : true, stage, b[c]);
        }
        sd += sd_step;
        sy += sy_step;
        if (WIDE) __syncwarp();                              // the warp's words have all been read
        copy();
        at = at + row_bytes == AHEAD * row_bytes ? 0 : at + row_bytes;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (sums) flush();
    if (a.pre_part) {
#pragma unroll
        for (int c = 0; c < V; c++) {
            const uint32_t k = 8 * chunk(c);
            float* p = a.pre_part + (int64_t)blockIdx.x * SUMS * a.wide + k;
            if (k < a.wide) {
                put_sums(p, pw[c]);
                if (TWO) put_sums(p + a.wide, pb[c]);
            }
        }
    }
}

template <int DT, int RT, int V>
static const void* norm_forward_of(int post, int pre, bool whole)
{
    if (whole) {
        if (post == 0 && pre == 1) return (const void*)k_norm_forward<DT, RT, V, 0, 1>;
        if (post == 0 && pre == 2) return (const void*)k_norm_forward<DT, RT, V, 0, 2>;
        if (post == 1 && pre == 1) return (const void*)k_norm_forward<DT, RT, V, 1, 1>;
        if (post == 2 && pre == 2) return (const void*)k_norm_forward<DT, RT, V, 2, 2>;
    }
    return (const void*)k_norm_forward<DT, RT, V, -1, -1>;
}
// The kinds whose rows are copied ahead: the same norm on both sides, only the one before the next
// block, or only an RMS norm after this one.
static inline bool norm_kinds_copied(int post, int pre) { return pre == 0 ? post == 1 : post == 0 || post == pre; }

// `two`: both sums are wanted; set where the kernel keeps both all the same.  `smem`: bytes of
// shared memory a thread of the kernel needs.  `copied`: whether the rows can be copied ahead
// (there is dy, and with rows that are not whole a word more fits into the threads).
template <int DT, int RT, int V, bool ANY>
static const void* norm_backward_copied(int post, int pre, bool& two, int& smem)
{
    smem = NormRing<RT, V, ANY>::bytes;
    if (!norm_kinds_copied(post, pre)) return nullptr;
    if (pre == 1 && !two)
        return post == 0 ? (const void*)k_norm_backward_whole<DT, RT, V, 0, 1, false, ANY>
                         : (const void*)k_norm_backward_whole<DT, RT, V, 1, 1, false, ANY>;
    two = true;
    if (pre == 0) return (const void*)k_norm_backward_whole<DT, RT, V, 1, 0, true, ANY>;
    if (pre == 1)
        return post == 0 ? (const void*)k_norm_backward_whole<DT, RT, V, 0, 1, true, ANY>
                         : (const void*)k_norm_backward_whole<DT, RT, V, 1, 1, true, ANY>;
    return post == 0 ? (const void*)k_norm_backward_whole<DT, RT, V, 0, 2, true, ANY>
                     : (const void*)k_norm_backward_whole<DT, RT, V, 2, 2, true, ANY>;
}
template <int DT, int RT, int V>
static const void* norm_backward_of(int post, int pre, bool whole, bool copied, bool& two, int& smem)
{
    if constexpr (V <= 2) {
        const void* fn = whole    ? norm_backward_copied<DT, RT, V, false>(post, pre, two, smem)
                         : copied ? norm_backward_copied<DT, RT, V, true>(post, pre, two, smem)
                                  : nullptr;
        if (fn) return fn;
    }
    smem = 16 * ZERO_NORM_WORDS * V;
    return two ? (const void*)k_norm_backward<DT, RT, V, true> : (const void*)k_norm_backward<DT, RT, V, false>;
}

}  // namespace zero
