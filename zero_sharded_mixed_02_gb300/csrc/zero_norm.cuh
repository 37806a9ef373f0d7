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
const void* norm_backward_fp16(int res, int v, int post, int pre, bool whole, bool& two);
const void* norm_backward_bf16(int res, int v, int post, int pre, bool whole, bool& two);

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
    const uint32_t end = (uint32_t)norm_row0(blockIdx.x + 1, a.rows, gridDim.x);
    uint32_t row = (uint32_t)norm_row0(blockIdx.x, a.rows, gridDim.x);
    uint32_t grp = row / a.group, in_group = row - grp * a.group;
    auto fetch = [&](uint32_t at) {
        const void *ph = row_of<RT>(a.h, at, a.ldh), *py = row_of<DT>(a.y, at, a.ldy);
#pragma unroll
        for (int c = 0; c < V; c++) {
            load_chunk<RT, WHOLE>(rh[c], ph, col[c], n[c], a.vec_h);
            if (block) load_chunk<DT, WHOLE>(ry[c], py, col[c], n[c], a.vec_y);
        }
    };
    fetch(row);
    for (; row < end; row++) {
        f32x2_t h[V][4], y[V][4], w[4];
#pragma unroll
        for (int c = 0; c < V; c++) {
            widen_chunk<RT, WHOLE>(rh[c], h[c], a.vec_h, stage);
            if (block) widen_chunk<DT, WHOLE>(ry[c], y[c], a.vec_y, stage);
        }
        if (row + 1 < end) fetch(row + 1);
        float mu2 = 0.0f, r2 = 1.0f, mu1 = 0.0f, r1 = 1.0f;
        if (block) {
            if (post) normalise<V>(y, n, post, a.eps, a.inv_cols, mu2, r2, buf, turn);
            const void* gate = row_of<DT>(a.gate, grp, a.cols);
#pragma unroll
            for (int c = 0; c < V; c++) {
                if (a.ckpt_y) {
                    uint8_t* p = a.ckpt_y + (int64_t)row * a.stride;
                    if (post) act_store_small(y[c], p, col[c], a.wide, a.stride, a.lo, col[c] < a.wide);
                    else act_store(y[c], p, col[c], a.wide, a.stride, a.lo, a.hi, col[c] < a.wide);
                }
                if (post && a.post_w) {
                    load_weights<DT, WHOLE>(a.post_w, col[c], n[c], a.vec_w, stage, w);
                    times(y[c], w);
                }
                if (post && a.post_b) {
                    load_weights<DT, WHOLE>(a.post_b, col[c], n[c], a.vec_w, stage, w);
                    plus(y[c], w);
                }
                if (a.gate) {
                    load_weights<DT, WHOLE>(gate, col[c], n[c], a.vec_g, stage, w);
                    times(y[c], w);
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
                    load_weights<DT, WHOLE>(a.pre_w, col[c], n[c], a.vec_w, stage, w);
                    times(h[c], w);
                }
                if (a.pre_b) {
                    load_weights<DT, WHOLE>(a.pre_b, col[c], n[c], a.vec_w, stage, w);
                    plus(h[c], w);
                }
                store_chunk<DT, WHOLE>(px, col[c], n[c], a.vec_x, stage, h[c]);
            }
        }
        if (a.stats && threadIdx.x == 0)
            reinterpret_cast<float4*>(a.stats)[row] = make_float4(mu2, r2, mu1, r1);
        if (++in_group == a.group) {
            in_group = 0;
            grp++;
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
// POST and PRE as in the forward pass (known kinds: whole aligned rows with dy wanted).
template <int DT, int RT, int V, int POST, int PRE, bool TWO>
__global__ void __launch_bounds__(ZERO_NORM_THREADS, 1) k_norm_backward(const __grid_constant__ NormBwdArgs a)
{
    // one wave of blocks: the kernel that adds their sums may be placed already
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr bool WHOLE = POST >= 0;
    const int post = WHOLE ? POST : a.post, pre = WHOLE ? PRE : a.pre;
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
    auto scales = [&](int c, f32x2_t (&u)[4]) {              // gate post_w
        f32x2_t w[4];
#pragma unroll
        for (int j = 0; j < 4; j++) u[j] = both(1.0f);
        if (a.gate) load_weights<DT, WHOLE>(row_of<DT>(a.gate, grp, a.cols), col[c], n[c], a.vec_g, stage, u);
        if (post && a.post_w) {
            load_weights<DT, WHOLE>(a.post_w, col[c], n[c], a.vec_w, stage, w);
            times(u, w);
        }
        end_of_row(u, n[c]);
    };
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
                    load_weights<DT, WHOLE>(a.pre_w, col[c], n[c], a.vec_w, stage, w);
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
        if (!WHOLE || (layer && POST > 0)) {
            if (layer) {
                block_sum<8>(s, buf, turn);
            } else {
                float three[3] = {s[0], s[1], s[2]};
                block_sum<3>(three, buf, turn);
                s[0] = three[0];
                s[1] = three[1];
                s[2] = three[2];
            }
        } else if (POST > 0) {
            float three[3] = {s[0], s[1], s[2]};
            block_sum<3>(three, buf, turn);
            s[0] = three[0];
            s[1] = three[1];
            s[2] = three[2];
        } else {                                             // the pre-norm alone
            float two[2] = {s[0], s[3]};
            block_sum<2>(two, buf, turn);
            s[0] = two[0];
            s[3] = two[1];
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
// `two`: both sums are wanted; set where the kernel keeps both all the same.
template <int DT, int RT, int V>
static const void* norm_backward_of(int post, int pre, bool whole, bool& two)
{
    if (whole && (!two || pre == 2)) {
        if (post == 0 && pre == 1) return (const void*)k_norm_backward<DT, RT, V, 0, 1, false>;
        if (post == 1 && pre == 1) return (const void*)k_norm_backward<DT, RT, V, 1, 1, false>;
        if (pre == 2 && (post == 0 || post == 2)) {
            two = true;
            return post == 0 ? (const void*)k_norm_backward<DT, RT, V, 0, 2, true>
                             : (const void*)k_norm_backward<DT, RT, V, 2, 2, true>;
        }
    }
    return two ? (const void*)k_norm_backward<DT, RT, V, -1, -1, true>
               : (const void*)k_norm_backward<DT, RT, V, -1, -1, false>;
}

}  // namespace zero
