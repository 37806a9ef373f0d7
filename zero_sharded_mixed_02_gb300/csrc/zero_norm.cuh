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
    int cols, wide, stride, lo, hi;
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
    int cols, wide, stride, post, pre;
    float alpha, inv_cols;
    int vec_dho, vec_dx, vec_dh, vec_dy, vec_w, vec_g;
};

// Kernels by type of the stream (DT or fp32), chunks per thread (1, 2, 4), both sums wanted,
// and whether every row and weight is read in whole aligned chunks.
const void* norm_forward_fp16(int res, int v, bool whole);
const void* norm_forward_bf16(int res, int v, bool whole);
const void* norm_backward_fp16(int res, int v, bool two, bool whole);
const void* norm_backward_bf16(int res, int v, bool two, bool whole);

// Rows [row0(b), row0(b + 1)) belong to block b; the block of row r is the largest b with row0(b) <= r.
__host__ __device__ inline int64_t norm_row0(int64_t b, int64_t rows, int64_t blocks) { return b * rows / blocks; }
__host__ __device__ inline int64_t norm_block_of(int64_t r, int64_t rows, int64_t blocks)
{
    return ((r + 1) * blocks - 1) / rows;
}

// Eight weights (cached: every row of a block reads the same ones).
template <int DT, bool WHOLE>
static __device__ __forceinline__ void load_weights(const void* p, int64_t i, int n, bool vec, f32x2_t (&v)[4])
{
    Raw<DT> r;
    const uint16_t* w = static_cast<const uint16_t*>(p);
    if ((WHOLE || vec) && n >= 8) r.q[0] = __ldg(reinterpret_cast<const uint4*>(w + i));
    else load_chunk<DT, WHOLE>(r, p, i, n, false);
    widen_chunk<DT>(r, v);
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

// WHOLE: every chunk of every matrix and weight is whole and aligned (cols a multiple of
// 8); otherwise each tensor's flag says how it is read.  Two blocks of one row an SM
// (16 warps each, 64 registers) beat one block of two rows at a time, which does fewer
// instructions (weights and branches shared) but leaves half the warps to hide latencies:
// 165 against 174 us at 16384 x 4096 with an fp32 stream.
template <int DT, int RT, int V, bool WHOLE>
__global__ void __launch_bounds__(ZERO_NORM_THREADS, V == 1 ? 2 : 1)
    k_norm_forward(const __grid_constant__ NormArgs a)
{
    __shared__ norm_buf_t buf;
    int turn = 0, col[V], n[V];
#pragma unroll
    for (int c = 0; c < V; c++) {
        col[c] = 8 * (threadIdx.x + c * blockDim.x);
        n[c] = a.cols - col[c];
    }
    Raw<RT> rh[V];
    Raw<DT> ry[V];
    const uint32_t end = (uint32_t)norm_row0(blockIdx.x + 1, a.rows, gridDim.x);
    uint32_t row = (uint32_t)norm_row0(blockIdx.x, a.rows, gridDim.x);
    uint32_t grp = row / a.group, in_group = row - grp * a.group;
    auto fetch = [&](uint32_t at) {
#pragma unroll
        for (int c = 0; c < V; c++) {
            load_chunk<RT, WHOLE>(rh[c], a.h, (int64_t)at * a.ldh + col[c], n[c], a.vec_h);
            if (a.y) load_chunk<DT, WHOLE>(ry[c], a.y, (int64_t)at * a.ldy + col[c], n[c], a.vec_y);
        }
    };
    fetch(row);
    for (; row < end; row++) {
        f32x2_t h[V][4], y[V][4], w[4];
#pragma unroll
        for (int c = 0; c < V; c++) {
            widen_chunk<RT>(rh[c], h[c]);
            if (a.y) widen_chunk<DT>(ry[c], y[c]);
        }
        if (row + 1 < end) fetch(row + 1);
        float mu2 = 0.0f, r2 = 1.0f, mu1 = 0.0f, r1 = 1.0f;
        if (a.y) {
            if (a.post) normalise<V>(y, n, a.post, a.eps, a.inv_cols, mu2, r2, buf, turn);
#pragma unroll
            for (int c = 0; c < V; c++) {
                if (a.ckpt_y) {
                    uint8_t* p = a.ckpt_y + (int64_t)row * a.stride;
                    if (a.post) act_store_small(y[c], p, col[c], a.wide, a.stride, a.lo, col[c] < a.wide);
                    else act_store(y[c], p, col[c], a.wide, a.stride, a.lo, a.hi, col[c] < a.wide);
                }
                if (a.post_w) {
                    load_weights<DT, WHOLE>(a.post_w, col[c], n[c], a.vec_w, w);
                    times(y[c], w);
                }
                if (a.post_b) {
                    load_weights<DT, WHOLE>(a.post_b, col[c], n[c], a.vec_w, w);
                    plus(y[c], w);
                }
                if (a.gate) {
                    load_weights<DT, WHOLE>(a.gate, (int64_t)grp * a.cols + col[c], n[c], a.vec_g, w);
                    times(y[c], w);
                }
                const f32x2_t alpha = both(a.alpha);
#pragma unroll
                for (int j = 0; j < 4; j++) h[c][j] = fma2(alpha, y[c][j], h[c][j]);
            }
        }
        if (a.h_out)
#pragma unroll
            for (int c = 0; c < V; c++)
                store_chunk<RT, WHOLE>(a.h_out, (int64_t)row * a.ldho + col[c], n[c], a.vec_ho, h[c]);
        if (a.pre) {
            normalise<V>(h, n, a.pre, a.eps, a.inv_cols, mu1, r1, buf, turn);
#pragma unroll
            for (int c = 0; c < V; c++) {
                if (a.ckpt_x)
                    act_store_small(h[c], a.ckpt_x + (int64_t)row * a.stride, col[c], a.wide, a.stride, a.lo,
                                    col[c] < a.wide);
                if (a.pre_w) {
                    load_weights<DT, WHOLE>(a.pre_w, col[c], n[c], a.vec_w, w);
                    times(h[c], w);
                }
                if (a.pre_b) {
                    load_weights<DT, WHOLE>(a.pre_b, col[c], n[c], a.vec_w, w);
                    plus(h[c], w);
                }
                store_chunk<DT, WHOLE>(a.x, (int64_t)row * a.ldx + col[c], n[c], a.vec_x, h[c]);
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

// sum of a b, of a
template <int V>
static __device__ __forceinline__ float dot(const f32x2_t (&a)[V][4], const f32x2_t (&b)[V][4])
{
    f32x2_t t = both(0.0f);
#pragma unroll
    for (int c = 0; c < V; c++)
#pragma unroll
        for (int j = 0; j < 4; j++) t = fma2(a[c][j], b[c][j], t);
    return either(t);
}
template <int V>
static __device__ __forceinline__ float total(const f32x2_t (&a)[V][4])
{
    f32x2_t t = both(0.0f);
#pragma unroll
    for (int c = 0; c < V; c++)
#pragma unroll
        for (int j = 0; j < 4; j++) t = add2(t, a[c][j]);
    return either(t);
}

// One reduction a row serves both norms.  With g = pre_w dx, u = gate post_w and
// B = dh_out + r1 g,
//   D = B - r1 (mean(g) + mean(g xh) xh),
// so the post-norm's sums of u D and u D yh follow from sums that do not need D:
//   sum u yh D = sum u yh B - r1 (mean(g) sum u yh + mean(g xh) sum u yh xh)
// and the same without yh.  A second reduction, after D, would cost its latency once more.
template <int DT, int RT, int V, bool TWO, bool WHOLE>
__global__ void __launch_bounds__(ZERO_NORM_THREADS, 1) k_norm_backward(const __grid_constant__ NormBwdArgs a)
{
    // one wave of blocks: the kernel that adds their sums may be placed already
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ norm_buf_t buf;
    constexpr int SUMS = TWO ? 2 : 1;
    int turn = 0, col[V], n[V];
    f32x2_t pw[V][4], sw[V][4], pb[TWO ? V : 1][4], sb[TWO ? V : 1][4];
#pragma unroll
    for (int c = 0; c < V; c++) {
        col[c] = 8 * (threadIdx.x + c * blockDim.x);
        n[c] = a.cols - col[c];
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
#pragma unroll
        for (int c = 0; c < V; c++) {
            if (a.dh_out) load_chunk<RT, WHOLE>(rd[c], a.dh_out, (int64_t)r * a.lddho + col[c], n[c], a.vec_dho);
            if (a.pre) load_chunk<DT, WHOLE>(rx[c], a.dx, (int64_t)r * a.lddx + col[c], n[c], a.vec_dx);
            qx[c] = qy[c] = make_uint2(0, 0);
            ex[c] = ey[c] = 0;
            if (col[c] < a.cols) {
                if (a.pre) {
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
    // The sums of the block's rows of group grp go to the slot block + group: along the
    // rows both only grow, so no two pairs share one.  Times the group's gate they are
    // added to the block's sums for the post-norm's weights, which stay in the workspace
    // (a group seldom ends inside a block).
    bool again = false;
    auto flush = [&]() {
#pragma unroll
        for (int c = 0; c < V; c++) {
            if (col[c] >= a.wide) continue;
            if (a.slots) {
                float* p = a.slots + ((int64_t)blockIdx.x + grp) * SUMS * a.wide + col[c];
                put_sums(p, sw[c]);
                if (TWO) put_sums(p + a.wide, sb[c]);
            }
            if (a.post_part) {
                float* p = a.post_part + (int64_t)blockIdx.x * SUMS * a.wide + col[c];
                if (a.gate) {
                    f32x2_t w[4];
                    load_weights<DT, WHOLE>(a.gate, (int64_t)grp * a.cols + col[c], n[c], a.vec_g, w);
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
    const bool sums = a.slots || a.post_part, layer = a.pre == ZERO_NORM_LAYER || a.post == ZERO_NORM_LAYER;
    fetch(row);
    for (; row < end; row++) {
        if (left == 0) {
            if (sums) flush();
            grp++;
            left = a.group;
        }
        left--;
        f32x2_t b[V][4], u[V][4], xh[V][4], yh[V][4], w[4];
        const float k1 = r1, k2 = r2;
        float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < V; c++) {
            if (a.pre) {
                widen_chunk<DT>(rx[c], b[c]);
                act_values(qx[c], ex[c], xh[c]);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    pw[c][j] = fma2(b[c][j], xh[c][j], pw[c][j]);
                    if (TWO) pb[c][j] = add2(pb[c][j], b[c][j]);
                }
                if (a.pre_w) {
                    load_weights<DT, WHOLE>(a.pre_w, col[c], n[c], a.vec_w, w);
                    times(b[c], w);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) b[c][j] = xh[c][j] = both(0.0f);
            }
            act_values(qy[c], ey[c], yh[c]);
#pragma unroll
            for (int j = 0; j < 4; j++) u[c][j] = both(1.0f);
            if (a.gate) load_weights<DT, WHOLE>(a.gate, (int64_t)grp * a.cols + col[c], n[c], a.vec_g, u[c]);
            if (a.post_w) {
                load_weights<DT, WHOLE>(a.post_w, col[c], n[c], a.vec_w, w);
                times(u[c], w);
            }
            end_of_row(u[c], n[c]);
        }
        s[0] = dot<V>(b, xh);
        if (layer) s[3] = total<V>(b);
#pragma unroll
        for (int c = 0; c < V; c++) {                        // b = B from here, xh and yh as read
#pragma unroll
            for (int j = 0; j < 4; j++) w[j] = both(0.0f);
            if (a.dh_out) widen_chunk<RT>(rd[c], w);
#pragma unroll
            for (int j = 0; j < 4; j++) b[c][j] = fma2(both(k1), b[c][j], w[j]);
        }
        if (row + 1 < end) fetch(row + 1);
        {
            f32x2_t uy[V][4];
#pragma unroll
            for (int c = 0; c < V; c++)
#pragma unroll
                for (int j = 0; j < 4; j++) uy[c][j] = mul2(u[c][j], yh[c][j]);
            s[1] = dot<V>(uy, b);
            s[2] = dot<V>(uy, xh);
            if (layer) {
                s[4] = total<V>(uy);
                s[5] = dot<V>(u, b);
                s[6] = total<V>(u);
                s[7] = dot<V>(u, xh);
            }
        }
        if (layer) {
            block_sum<8>(s, buf, turn);
        } else {
            float t[3] = {s[0], s[1], s[2]};
            block_sum<3>(t, buf, turn);
            s[0] = t[0];
            s[1] = t[1];
            s[2] = t[2];
        }
        // D = b - p1 xh - p0;  dy = alpha r2 (u D - q1 yh - q0)
        const float p1 = k1 * s[0] * a.inv_cols, p0 = a.pre == ZERO_NORM_LAYER ? k1 * s[3] * a.inv_cols : 0.0f;
#pragma unroll
        for (int c = 0; c < V; c++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (layer) b[c][j] = sub2(b[c][j], both(p0));
                b[c][j] = fma2(both(-p1), xh[c][j], b[c][j]);
            }
        if (a.dh)
#pragma unroll
            for (int c = 0; c < V; c++)
                store_chunk<RT, WHOLE>(a.dh, (int64_t)row * a.lddh + col[c], n[c], a.vec_dh, b[c]);
        if (!a.dy) continue;
        if (sums)
#pragma unroll
            for (int c = 0; c < V; c++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    sw[c][j] = fma2(b[c][j], yh[c][j], sw[c][j]);
                    if (TWO) sb[c][j] = add2(sb[c][j], b[c][j]);
                }
        float scale = a.alpha, q1 = 0.0f, q0 = 0.0f;
        if (a.post) {
            scale *= k2;
            q1 = (s[1] - p0 * s[4] - p1 * s[2]) * a.inv_cols;
            if (a.post == ZERO_NORM_LAYER) q0 = (s[5] - p0 * s[6] - p1 * s[7]) * a.inv_cols;
        }
#pragma unroll
        for (int c = 0; c < V; c++) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const f32x2_t e = layer ? fma2(u[c][j], b[c][j], both(-q0)) : mul2(u[c][j], b[c][j]);
                b[c][j] = mul2(both(scale), fma2(both(-q1), yh[c][j], e));
            }
            store_chunk<DT, WHOLE>(a.dy, (int64_t)row * a.lddy + col[c], n[c], a.vec_dy, b[c]);
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
static const void* norm_forward_of(bool whole)
{
    return whole ? (const void*)k_norm_forward<DT, RT, V, true> : (const void*)k_norm_forward<DT, RT, V, false>;
}
template <int DT, int RT, int V>
static const void* norm_backward_of(bool two, bool whole)
{
    if (two)
        return whole ? (const void*)k_norm_backward<DT, RT, V, true, true>
                     : (const void*)k_norm_backward<DT, RT, V, true, false>;
    return whole ? (const void*)k_norm_backward<DT, RT, V, false, true>
                 : (const void*)k_norm_backward<DT, RT, V, false, false>;
}
template <int DT, int RT>
static const void* norm_forward_of(int v, bool whole)
{
    return v == 1 ? norm_forward_of<DT, RT, 1>(whole) : v == 2 ? norm_forward_of<DT, RT, 2>(whole)
                                                               : norm_forward_of<DT, RT, 4>(whole);
}
template <int DT, int RT>
static const void* norm_backward_of(int v, bool two, bool whole)
{
    return v == 1 ? norm_backward_of<DT, RT, 1>(two, whole) : v == 2 ? norm_backward_of<DT, RT, 2>(two, whole)
                                                                     : norm_backward_of<DT, RT, 4>(two, whole);
}

}  // namespace zero
