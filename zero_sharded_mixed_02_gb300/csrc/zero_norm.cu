// zero_norm.cu -- the norms around a block fused with its gate and residual scale,
// forward and backward (include/zero_b200.h gives the formulas).
//
// Both passes read every tensor once and write each output once, so HBM bounds
// them.  A block of threads holds one row at a time in registers (8-column chunks,
// V per thread), so the row's statistics and everything after them come from one
// read; the next row's loads are issued before the current row's reductions, which
// would otherwise leave the memory system idle for their latency.
//
// The backward pass keeps the sums over rows (weight, bias and gate gradients) in
// registers while a block walks its contiguous range of rows; partial sums go to
// the workspace once per block, and per gate group a block crosses, and a second
// kernel adds them in a fixed order.  With S = sum D yh and S0 = sum D over a group's
// rows, dgate = alpha (post_w S + post_b S0), and dpost_w = sum over groups of
// alpha gate S, dpost_b of alpha gate S0: one pair of sums serves all three.
#include <cmath>

#include "zero_act.cuh"
#include "zero_b200.h"
#include "zero_trace.h"

namespace zero {

#define ZERO_NORM_THREADS 512          // most threads of a block (one row)
#define ZERO_NORM_BLOCKS 608           // most blocks of the backward pass (its partial sums)

// ---- a lane's chunk of a row -----------------------------------------------------
template <int T> struct Raw { uint4 q[T == 2 ? 2 : 1]; };

template <int T>
static __device__ __forceinline__ void load_raw(Raw<T>& r, const void* p, int64_t i, int n, bool vec)
{
    if (vec && n >= 8) {
        if (T == 2) {
            const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
            r.q[0] = __ldcs(s);
            r.q[T == 2] = __ldcs(s + 1);
        } else {
            r.q[0] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
        }
        return;
    }
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; j++)
        w[j] = j >= n ? 0u
               : T == 2 ? __ldg(static_cast<const uint32_t*>(p) + i + j)
                        : (uint32_t)__ldg(static_cast<const uint16_t*>(p) + i + j);
    if (T == 2) {
        r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
        r.q[T == 2] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
        r.q[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
}

template <int T>
static __device__ __forceinline__ void widen_raw(const Raw<T>& r, float (&v)[8])
{
    if (T == 2) {
        const uint32_t w[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w,
                               r.q[T == 2].x, r.q[T == 2].y, r.q[T == 2].z, r.q[T == 2].w};
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = __uint_as_float(w[j]);
    } else {
        widen2<T & 1>(r.q[0].x, v[0], v[1]);
        widen2<T & 1>(r.q[0].y, v[2], v[3]);
        widen2<T & 1>(r.q[0].z, v[4], v[5]);
        widen2<T & 1>(r.q[0].w, v[6], v[7]);
    }
}

// Eight weights (cached: every row of a block reads the same ones).
template <int DT>
static __device__ __forceinline__ void load_w(const uint16_t* p, int64_t i, int n, bool vec, float (&v)[8])
{
    Raw<DT> r;
    if (vec && n >= 8) r.q[0] = __ldg(reinterpret_cast<const uint4*>(p + i));
    else load_raw<DT>(r, p, i, n, false);
    widen_raw<DT>(r, v);
}

// Sums of N values over the block, the same bits in every thread: shuffles inside a
// warp, then every thread adds the warps' sums in warp order.  One barrier; two
// buffers used in turn make a second one needless.
template <int N>
static __device__ __forceinline__ void block_sum(float (&v)[N], float (*buf)[ZERO_NORM_THREADS / 32][2],
                                                 int& turn)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; i++) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; i++) buf[turn][threadIdx.x >> 5][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = 0.0f;
    for (int w = 0; w < warps; w++)
#pragma unroll
        for (int i = 0; i < N; i++) v[i] += buf[turn][w][i];
    turn ^= 1;
}

struct NormArgs {
    const void *h, *y, *post_w, *post_b, *gate, *pre_w, *pre_b;
    void *h_out, *x;
    uint8_t *ckpt_y, *ckpt_x;
    float* stats;
    int64_t rows, ldh, ldy, ldho, ldx, group;    // group >= 1
    int cols, wide, stride, lo, hi;
    int post, pre;
    float eps, alpha, inv_cols;
    int vec_h, vec_y, vec_ho, vec_x, vec_w, vec_g;
};

// ---- forward ---------------------------------------------------------------------
// Statistics of a row held as v[V][8] (zeros past the row's end): the row is left
// centred (layer norm) and its mean and 1/deviation returned.
template <int V>
static __device__ __forceinline__ void row_stats(float (&v)[V][8], const int (&n)[V], int kind, float eps,
                                                 float inv_cols, float& mean, float& rstd,
                                                 float (*buf)[ZERO_NORM_THREADS / 32][2], int& turn)
{
    mean = 0.0f;
    if (kind == ZERO_NORM_LAYER) {
        float s[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < V; c++)
#pragma unroll
            for (int j = 0; j < 8; j++) s[0] += v[c][j];
        block_sum<1>(s, buf, turn);
        mean = s[0] * inv_cols;
#pragma unroll
        for (int c = 0; c < V; c++)
#pragma unroll
            for (int j = 0; j < 8; j++) v[c][j] = j < n[c] ? v[c][j] - mean : 0.0f;
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < V; c++)
#pragma unroll
        for (int j = 0; j < 8; j++) s[0] = __fmaf_rn(v[c][j], v[c][j], s[0]);
    block_sum<1>(s, buf, turn);
    rstd = 1.0f / sqrtf(s[0] * inv_cols + eps);
}

template <int DT, int RT, int V>
__global__ void __launch_bounds__(ZERO_NORM_THREADS) k_norm_forward(const __grid_constant__ NormArgs a)
{
    __shared__ float buf[2][ZERO_NORM_THREADS / 32][2];
    int turn = 0, col[V], n[V];
#pragma unroll
    for (int c = 0; c < V; c++) {
        col[c] = 8 * (threadIdx.x + c * blockDim.x);
        n[c] = a.cols - col[c];
    }
    Raw<RT> rh[V];
    Raw<DT> ry[V];
    int64_t row = blockIdx.x;
#pragma unroll
    for (int c = 0; c < V; c++) {
        load_raw<RT>(rh[c], a.h, row * a.ldh + col[c], n[c], a.vec_h);
        if (a.y) load_raw<DT>(ry[c], a.y, row * a.ldy + col[c], n[c], a.vec_y);
    }
    for (; row < a.rows; row += gridDim.x) {
        float h[V][8], y[V][8];
#pragma unroll
        for (int c = 0; c < V; c++) {
            widen_raw<RT>(rh[c], h[c]);
            if (a.y) widen_raw<DT>(ry[c], y[c]);
        }
        const int64_t next = row + gridDim.x;
        if (next < a.rows)
#pragma unroll
            for (int c = 0; c < V; c++) {
                load_raw<RT>(rh[c], a.h, next * a.ldh + col[c], n[c], a.vec_h);
                if (a.y) load_raw<DT>(ry[c], a.y, next * a.ldy + col[c], n[c], a.vec_y);
            }
        float mu2 = 0.0f, r2 = 1.0f, mu1 = 0.0f, r1 = 1.0f;
        if (a.y) {
            if (a.post) row_stats<V>(y, n, a.post, a.eps, a.inv_cols, mu2, r2, buf, turn);
            const int64_t grow = row / a.group * a.cols;
#pragma unroll
            for (int c = 0; c < V; c++) {
                if (a.post)
#pragma unroll
                    for (int j = 0; j < 8; j++) y[c][j] *= r2;
                if (a.ckpt_y)
                    act_store_chunk(y[c], a.ckpt_y + row * a.stride, col[c], a.wide, a.stride, a.lo, a.hi,
                                    col[c] < a.wide);
                float w[8];
                if (a.post_w) {
                    load_w<DT>((const uint16_t*)a.post_w, col[c], n[c], a.vec_w, w);
#pragma unroll
                    for (int j = 0; j < 8; j++) y[c][j] *= w[j];
                }
                if (a.post_b) {
                    load_w<DT>((const uint16_t*)a.post_b, col[c], n[c], a.vec_w, w);
#pragma unroll
                    for (int j = 0; j < 8; j++) y[c][j] += w[j];
                }
                if (a.gate) {
                    load_w<DT>((const uint16_t*)a.gate, grow + col[c], n[c], a.vec_g, w);
#pragma unroll
                    for (int j = 0; j < 8; j++) y[c][j] *= w[j];
                }
#pragma unroll
                for (int j = 0; j < 8; j++) h[c][j] = __fmaf_rn(a.alpha, y[c][j], h[c][j]);
            }
        }
        if (a.h_out)
#pragma unroll
            for (int c = 0; c < V; c++) store8<RT>(a.h_out, row * a.ldho + col[c], n[c], a.vec_ho, h[c]);
        if (a.pre) {
            row_stats<V>(h, n, a.pre, a.eps, a.inv_cols, mu1, r1, buf, turn);
#pragma unroll
            for (int c = 0; c < V; c++) {
#pragma unroll
                for (int j = 0; j < 8; j++) h[c][j] *= r1;
                if (a.ckpt_x)
                    act_store_chunk(h[c], a.ckpt_x + row * a.stride, col[c], a.wide, a.stride, a.lo, a.hi,
                                    col[c] < a.wide);
                float w[8];
                if (a.pre_w) {
                    load_w<DT>((const uint16_t*)a.pre_w, col[c], n[c], a.vec_w, w);
#pragma unroll
                    for (int j = 0; j < 8; j++) h[c][j] *= w[j];
                }
                if (a.pre_b) {
                    load_w<DT>((const uint16_t*)a.pre_b, col[c], n[c], a.vec_w, w);
#pragma unroll
                    for (int j = 0; j < 8; j++) h[c][j] += w[j];
                }
                store8<DT>(a.x, row * a.ldx + col[c], n[c], a.vec_x, h[c]);
            }
        }
        if (a.stats && threadIdx.x == 0)
            reinterpret_cast<float4*>(a.stats)[row] = make_float4(mu2, r2, mu1, r1);
    }
}

// ---- backward --------------------------------------------------------------------
struct NormBwdArgs {
    const void *dh_out, *dx, *post_w, *gate, *pre_w;
    const uint8_t *ckpt_y, *ckpt_x;
    const float* stats;
    void *dh, *dy;
    float* pre_part;         // [blocks][sums][cols]: dx xh (and dx)
    float* slots;            // [blocks + groups][sums][cols]: S (and S0) of a block's rows of a group
    int64_t rows, lddho, lddx, lddh, lddy, group;
    int cols, wide, stride, post, pre, sums;
    float alpha, inv_cols;
    int vec_dho, vec_dx, vec_dh, vec_dy, vec_w, vec_g;
};

// Rows [r0(b), r0(b + 1)) belong to block b; the block of row r is the largest b with r0(b) <= r.
__host__ __device__ inline int64_t norm_row0(int64_t b, int64_t rows, int64_t blocks) { return b * rows / blocks; }
__host__ __device__ inline int64_t norm_block_of(int64_t r, int64_t rows, int64_t blocks)
{
    return ((r + 1) * blocks - 1) / rows;
}

// Store a chunk of fp32 sums to the workspace (rows of `cols` floats, any alignment).
static __device__ __forceinline__ void store_sums(float* p, int n, const float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (j < n) p[j] = v[j];
}

template <int DT, int RT, int V, bool TWO>
__global__ void __launch_bounds__(ZERO_NORM_THREADS) k_norm_backward(const __grid_constant__ NormBwdArgs a)
{
    __shared__ float buf[2][ZERO_NORM_THREADS / 32][2];
    int turn = 0, col[V], n[V];
    float pw[V][8], sw[V][8], pb[TWO ? V : 1][8], sb[TWO ? V : 1][8];
#pragma unroll
    for (int c = 0; c < V; c++) {
        col[c] = 8 * (threadIdx.x + c * blockDim.x);
        n[c] = a.cols - col[c];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            pw[c][j] = sw[c][j] = 0.0f;
            if (TWO) pb[c][j] = sb[c][j] = 0.0f;
        }
    }
    const int64_t end = norm_row0(blockIdx.x + 1, a.rows, gridDim.x);
    int64_t row = norm_row0(blockIdx.x, a.rows, gridDim.x);
    int64_t grp = row / a.group, grp_end = (grp + 1) * a.group;
    Raw<RT> rd[V];
    Raw<DT> rx[V];
    uint2 qx[V], qy[V];
    uint32_t ex[V], ey[V];
    float4 st;
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int c = 0; c < V; c++) {
            if (a.dh_out) load_raw<RT>(rd[c], a.dh_out, r * a.lddho + col[c], n[c], a.vec_dho);
            if (a.pre) load_raw<DT>(rx[c], a.dx, r * a.lddx + col[c], n[c], a.vec_dx);
            qx[c] = qy[c] = make_uint2(0, 0);
            ex[c] = ey[c] = 0;
            if (col[c] < a.cols) {
                if (a.pre) {
                    const uint8_t* p = a.ckpt_x + r * a.stride;
                    qx[c] = __ldcs(reinterpret_cast<const uint2*>(p + col[c]));
                    ex[c] = __ldg(p + a.wide + (col[c] >> 5));
                }
                if (a.ckpt_y) {
                    const uint8_t* p = a.ckpt_y + r * a.stride;
                    qy[c] = __ldcs(reinterpret_cast<const uint2*>(p + col[c]));
                    ey[c] = __ldg(p + a.wide + (col[c] >> 5));
                }
            }
        }
        st = __ldg(reinterpret_cast<const float4*>(a.stats) + r);
    };
    // the sums of the block's rows of group grp go to the slot block + group: along the
    // rows both only grow, so no two pairs share one
    auto flush = [&]() {
        float* p = a.slots + (blockIdx.x + grp) * a.sums * a.cols;
#pragma unroll
        for (int c = 0; c < V; c++) {
            store_sums(p + col[c], n[c], sw[c]);
            if (TWO) store_sums(p + a.cols + col[c], n[c], sb[c]);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                sw[c][j] = 0.0f;
                if (TWO) sb[c][j] = 0.0f;
            }
        }
    };
    fetch(row);
    for (; row < end; row++) {
        if (a.slots && row == grp_end) {
            flush();
            grp++;
            grp_end += a.group;
        }
        float d[V][8], xh[V][8], yh[V][8];
        const float r2 = st.y, r1 = st.w;
        if (a.pre) {                                         // d = pre_w dx, and its two sums
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < V; c++) {
                float w[8];
                widen_raw<DT>(rx[c], d[c]);
                act_values8(qx[c], ex[c], xh[c]);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    pw[c][j] = __fmaf_rn(d[c][j], xh[c][j], pw[c][j]);
                    if (TWO) pb[c][j] += d[c][j];
                }
                if (a.pre_w) {
                    load_w<DT>((const uint16_t*)a.pre_w, col[c], n[c], a.vec_w, w);
#pragma unroll
                    for (int j = 0; j < 8; j++) d[c][j] *= w[j];
                }
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    s[0] = __fmaf_rn(d[c][j], xh[c][j], s[0]);
                    s[1] += d[c][j];
                }
            }
            float dho[V][8];
#pragma unroll
            for (int c = 0; c < V; c++) {
                act_values8(qy[c], ey[c], yh[c]);
                if (a.dh_out) widen_raw<RT>(rd[c], dho[c]);
                else
#pragma unroll
                    for (int j = 0; j < 8; j++) dho[c][j] = 0.0f;
            }
            if (row + 1 < end) fetch(row + 1);
            block_sum<2>(s, buf, turn);
            const float m1 = s[0] * a.inv_cols, m0 = a.pre == ZERO_NORM_LAYER ? s[1] * a.inv_cols : 0.0f;
#pragma unroll
            for (int c = 0; c < V; c++)
#pragma unroll
                for (int j = 0; j < 8; j++)
                    d[c][j] = __fmaf_rn(r1, __fmaf_rn(-m1, xh[c][j], d[c][j] - m0), dho[c][j]);
        } else {
#pragma unroll
            for (int c = 0; c < V; c++) {
                act_values8(qy[c], ey[c], yh[c]);
                if (a.dh_out) widen_raw<RT>(rd[c], d[c]);
                else
#pragma unroll
                    for (int j = 0; j < 8; j++) d[c][j] = 0.0f;
            }
            if (row + 1 < end) fetch(row + 1);
        }
        if (a.dh)
#pragma unroll
            for (int c = 0; c < V; c++) store8<RT>(a.dh, row * a.lddh + col[c], n[c], a.vec_dh, d[c]);
        if (!a.dy) continue;
        float s[2] = {0.0f, 0.0f};
        const int64_t grow = row / a.group * a.cols;
#pragma unroll
        for (int c = 0; c < V; c++) {
            float w[8];
            if (a.slots)
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    sw[c][j] = __fmaf_rn(d[c][j], yh[c][j], sw[c][j]);
                    if (TWO) sb[c][j] += d[c][j];
                }
            if (a.gate) {
                load_w<DT>((const uint16_t*)a.gate, grow + col[c], n[c], a.vec_g, w);
#pragma unroll
                for (int j = 0; j < 8; j++) d[c][j] *= w[j];
            }
            if (a.post_w) {
                load_w<DT>((const uint16_t*)a.post_w, col[c], n[c], a.vec_w, w);
#pragma unroll
                for (int j = 0; j < 8; j++) d[c][j] *= w[j];
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                d[c][j] = j < n[c] ? d[c][j] * a.alpha : 0.0f;
                s[0] = __fmaf_rn(d[c][j], yh[c][j], s[0]);
                s[1] += d[c][j];
            }
        }
        if (a.post) {
            block_sum<2>(s, buf, turn);
            const float m1 = s[0] * a.inv_cols, m0 = a.post == ZERO_NORM_LAYER ? s[1] * a.inv_cols : 0.0f;
#pragma unroll
            for (int c = 0; c < V; c++)
#pragma unroll
                for (int j = 0; j < 8; j++) d[c][j] = r2 * __fmaf_rn(-m1, yh[c][j], d[c][j] - m0);
        }
#pragma unroll
        for (int c = 0; c < V; c++) store8<DT>(a.dy, row * a.lddy + col[c], n[c], a.vec_dy, d[c]);
    }
    if (a.slots) flush();
    if (a.pre_part) {
        float* p = a.pre_part + (int64_t)blockIdx.x * a.sums * a.cols;
#pragma unroll
        for (int c = 0; c < V; c++) {
            store_sums(p + col[c], n[c], pw[c]);
            if (TWO) store_sums(p + a.cols + col[c], n[c], pb[c]);
        }
    }
}

struct NormSumArgs {
    const float *pre_part, *slots;
    const void *post_w, *post_b, *gate;
    void *dpost_w, *dpost_b, *dgate, *dpre_w, *dpre_b;
    int64_t rows, group, groups;
    int cols, blocks, sums, dtype, grad_dtype, accumulate;
    int col_jobs, flat_jobs, flat;
    float alpha;
};

static __device__ __forceinline__ float weight_at(const void* p, int64_t i, int dtype)
{
    if (!p) return 1.0f;
    const uint16_t u = __ldg(static_cast<const uint16_t*>(p) + i);
    return dtype == 0 ? widen1<0>(u) : widen1<1>(u);
}
static __device__ __forceinline__ void grad_out(void* p, int64_t i, float v, int grad_dtype, int accumulate)
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

// The sums of a group's rows at column c: its blocks' slots from block b0 + first by step.
static __device__ __forceinline__ void add_group(const NormSumArgs& a, int64_t g, int c, int first, int step,
                                                 float& v0, float& v1)
{
    if (a.rows == 0) return;
    const int64_t r0 = g * a.group, r1 = r0 + a.group < a.rows ? r0 + a.group : a.rows;
    const int64_t b1 = norm_block_of(r1 - 1, a.rows, a.blocks);
    for (int64_t b = norm_block_of(r0, a.rows, a.blocks) + first; b <= b1; b += step) {
        const float* p = a.slots + (b + g) * a.sums * a.cols + c;
        v0 += p[0];
        if (a.sums == 2) v1 += p[a.cols];
    }
}

static __device__ __forceinline__ void gate_out(const NormSumArgs& a, int64_t g, int c, float v0, float v1)
{
    v0 *= weight_at(a.post_w, c, a.dtype);
    if (a.post_b) v0 = __fmaf_rn(weight_at(a.post_b, c, a.dtype), v1, v0);
    grad_out(a.dgate, g * a.cols + c, a.alpha * v0, a.grad_dtype, a.accumulate);
}

// Adds the blocks' partial sums.  A job is 32 columns of the pre-norm's sums, of the
// post-norm's, or of a gate group's; its 32 strips take every 32nd block's part and
// are added in strip order.  Where there are so many groups that a group spans only
// a few blocks (flat), a gate job is 1024 columns of a group and a thread adds its column alone.
__global__ void __launch_bounds__(1024) k_norm_sums(const __grid_constant__ NormSumArgs a)
{
    __shared__ float s0[32][33], s1[32][33];
    const int strip = threadIdx.y;
    const int64_t jobs = 2ll * a.col_jobs + (a.dgate ? a.groups * (a.flat ? a.flat_jobs : a.col_jobs) : 0);
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        float v0 = 0.0f, v1 = 0.0f;
        int64_t k = job;
        if (a.flat && k >= 2 * a.col_jobs) {
            k -= 2 * a.col_jobs;
            const int64_t g = k / a.flat_jobs;
            const int c = (int)(k - g * a.flat_jobs) * 1024 + strip * 32 + threadIdx.x;
            if (c < a.cols) {
                add_group(a, g, c, 0, 1, v0, v1);
                gate_out(a, g, c, v0, v1);
            }
            continue;
        }
        const int64_t what = k / a.col_jobs;
        const int c = (int)(k - what * a.col_jobs) * 32 + threadIdx.x;
        if (c < a.cols) {
            if (what == 0) {
                if (a.dpre_w || a.dpre_b)
                    for (int b = strip; b < a.blocks; b += 32) {
                        const float* p = a.pre_part + (int64_t)b * a.sums * a.cols + c;
                        v0 += p[0];
                        if (a.sums == 2) v1 += p[a.cols];
                    }
            } else if (what == 1) {
                if (a.dpost_w || a.dpost_b)
                    for (int b = strip; b < a.blocks; b += 32) {
                        const int64_t g0 = norm_row0(b, a.rows, a.blocks) / a.group;
                        const int64_t g1 = (norm_row0(b + 1, a.rows, a.blocks) - 1) / a.group;
                        for (int64_t g = g0; g <= g1; g++) {
                            const float* p = a.slots + (b + g) * a.sums * a.cols + c;
                            const float w = a.alpha * weight_at(a.gate, g * a.cols + c, a.dtype);
                            v0 = __fmaf_rn(w, p[0], v0);
                            if (a.sums == 2) v1 = __fmaf_rn(w, p[a.cols], v1);
                        }
                    }
            } else {
                add_group(a, what - 2, c, strip, 32, v0, v1);
            }
        }
        __syncthreads();                                     // the previous job's reads are done
        s0[strip][threadIdx.x] = v0;
        s1[strip][threadIdx.x] = v1;
        __syncthreads();
        if (strip != 0 || c >= a.cols) continue;
        v0 = v1 = 0.0f;
        for (int i = 0; i < 32; i++) {
            v0 += s0[i][threadIdx.x];
            v1 += s1[i][threadIdx.x];
        }
        if (what == 0) {
            if (a.dpre_w) grad_out(a.dpre_w, c, v0, a.grad_dtype, a.accumulate);
            if (a.dpre_b) grad_out(a.dpre_b, c, v1, a.grad_dtype, a.accumulate);
        } else if (what == 1) {
            if (a.dpost_w) grad_out(a.dpost_w, c, v0, a.grad_dtype, a.accumulate);
            if (a.dpost_b) grad_out(a.dpost_b, c, v1, a.grad_dtype, a.accumulate);
        } else {
            gate_out(a, what - 2, c, v0, v1);
        }
    }
}

}  // namespace zero

using namespace zero;

namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int64_t elem(int dtype) { return dtype == ZERO_FP32 ? 4 : 2; }

// Rows of a matrix are read in 16-byte vectors if they are aligned to them.
int vec_rows(const void* p, int64_t ld, int dtype) { return p && aligned_to(p, 16) && ld * elem(dtype) % 16 == 0; }

bool matrix_ok(const void* p, int64_t ld, int64_t cols, int dtype)
{
    return p && aligned_to(p, elem(dtype)) && ld >= cols && ld <= (1ll << 31);
}

int64_t groups_of(const zero_norm_t& d)
{
    return d.group_rows == 0 || d.rows == 0 ? 1 : (d.rows + d.group_rows - 1) / d.group_rows;
}

bool description_ok(const zero_norm_t* d)
{
    if (!d) return false;
    if (d->dtype != ZERO_FP16 && d->dtype != ZERO_BF16) return false;
    if (d->res_dtype != d->dtype && d->res_dtype != ZERO_FP32) return false;
    for (int k : {d->post, d->pre})
        if (k != ZERO_NORM_NONE && k != ZERO_NORM_RMS && k != ZERO_NORM_LAYER) return false;
    if (d->rows < 0 || d->rows >= (1ll << 31) || d->cols < 1 || d->cols > ZERO_NORM_MAX_COLS ||
        d->group_rows < 0)
        return false;
    if (!std::isfinite(d->alpha) || !std::isfinite(d->eps) || d->eps < 0.0f) return false;
    if (d->post == ZERO_NORM_NONE && (d->post_w || d->post_b)) return false;
    if (d->pre == ZERO_NORM_NONE && (d->pre_w || d->pre_b)) return false;
    for (const void* p : {d->post_w, d->post_b, d->gate, d->pre_w, d->pre_b})
        if (!aligned_to(p, 2)) return false;
    return true;
}

int vec_weights(const zero_norm_t& d)
{
    for (const void* p : {d.post_w, d.post_b, d.pre_w, d.pre_b})
        if (p && !aligned_to(p, 16)) return 0;
    return 1;
}

// Chunks per thread and threads of a block for rows of `wide` columns.
void row_shape(int wide, int& v, int& threads)
{
    const int chunks = wide / 8;
    v = chunks <= ZERO_NORM_THREADS ? 1 : chunks <= 2 * ZERO_NORM_THREADS ? 2 : 4;
    threads = ((chunks + v - 1) / v + 31) / 32 * 32;
}

template <int DT, int RT>
const void* forward_kernel(int v)
{
    return v == 1 ? (const void*)k_norm_forward<DT, RT, 1>
         : v == 2 ? (const void*)k_norm_forward<DT, RT, 2>
                  : (const void*)k_norm_forward<DT, RT, 4>;
}
template <int DT, int RT, bool TWO>
const void* backward_kernel(int v)
{
    return v == 1 ? (const void*)k_norm_backward<DT, RT, 1, TWO>
         : v == 2 ? (const void*)k_norm_backward<DT, RT, 2, TWO>
                  : (const void*)k_norm_backward<DT, RT, 4, TWO>;
}
template <int DT, int RT>
const void* backward_kernel(int v, bool two)
{
    return two ? backward_kernel<DT, RT, true>(v) : backward_kernel<DT, RT, false>(v);
}

// Resident blocks of a kernel on the current device; 0: a CUDA call failed.
int64_t resident(const void* fn, int threads)
{
    int dev = 0, sms = 0, occ = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, threads, 0) != cudaSuccess)
        return 0;
    return (int64_t)sms * (occ > 0 ? occ : 1);
}

}  // namespace

extern "C" zero_status_t zero_norm_forward(const zero_norm_t* norm, const void* h, int64_t ldh, const void* y,
                                           int64_t ldy, void* h_out, int64_t ldho, void* x, int64_t ldx,
                                           void* ckpt_y, void* ckpt_x, float* stats, void* stream)
{
    TraceRange trace_("zero_norm_forward");
    if (!description_ok(norm)) return ZERO_EINVAL;
    const zero_norm_t& d = *norm;
    if (d.rows == 0) return ZERO_OK;
    if (!matrix_ok(h, ldh, d.cols, d.res_dtype)) return ZERO_EINVAL;
    if (y) {
        if (!matrix_ok(y, ldy, d.cols, d.dtype) || !matrix_ok(h_out, ldho, d.cols, d.res_dtype))
            return ZERO_EINVAL;
    } else {
        if (d.post != ZERO_NORM_NONE || d.gate || ckpt_y) return ZERO_EINVAL;
        if (h_out && !matrix_ok(h_out, ldho, d.cols, d.res_dtype)) return ZERO_EINVAL;
    }
    if (d.pre == ZERO_NORM_NONE ? (x || ckpt_x) : !matrix_ok(x, ldx, d.cols, d.dtype)) return ZERO_EINVAL;
    if (!aligned_to(ckpt_y, 16) || !aligned_to(ckpt_x, 16) || !aligned_to(stats, 16)) return ZERO_EINVAL;
    NormArgs a{};
    a.h = h; a.y = y; a.h_out = h_out; a.x = x;
    a.post_w = d.post_w; a.post_b = d.post_b; a.gate = d.gate; a.pre_w = d.pre_w; a.pre_b = d.pre_b;
    a.ckpt_y = static_cast<uint8_t*>(ckpt_y);
    a.ckpt_x = static_cast<uint8_t*>(ckpt_x);
    a.stats = stats;
    a.rows = d.rows; a.ldh = ldh; a.ldy = ldy; a.ldho = ldho; a.ldx = ldx;
    a.group = d.group_rows ? d.group_rows : d.rows;
    a.cols = (int)d.cols;
    a.wide = (int)act_wide(d.cols);
    a.stride = (int)act_stride(d.cols);
    a.lo = act_lo(d.dtype);
    a.hi = act_hi(d.dtype);
    a.post = d.post; a.pre = d.pre;
    a.eps = d.eps; a.alpha = d.alpha;
    a.inv_cols = 1.0f / (float)d.cols;
    a.vec_h = vec_rows(h, ldh, d.res_dtype);
    a.vec_y = vec_rows(y, ldy, d.dtype);
    a.vec_ho = vec_rows(h_out, ldho, d.res_dtype);
    a.vec_x = vec_rows(x, ldx, d.dtype);
    a.vec_w = vec_weights(d);
    a.vec_g = vec_rows(d.gate, d.cols, d.dtype);
    int v = 1, threads = 32;
    row_shape(a.wide, v, threads);
    const void* fn = d.res_dtype == ZERO_FP32
                         ? (d.dtype == ZERO_FP16 ? forward_kernel<0, 2>(v) : forward_kernel<1, 2>(v))
                         : (d.dtype == ZERO_FP16 ? forward_kernel<0, 0>(v) : forward_kernel<1, 1>(v));
    const int64_t most = resident(fn, threads);
    if (most == 0) return ZERO_ECUDA;
    void* args[] = {&a};
    return cudaLaunchKernel(fn, dim3((unsigned)(d.rows < most ? d.rows : most)), dim3(threads), args, 0,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ZERO_OK
               : ZERO_ECUDA;
}

extern "C" uint64_t zero_norm_workspace(const zero_norm_t* norm)
{
    if (!description_ok(norm)) return 0;
    const uint64_t blocks = norm->rows < ZERO_NORM_BLOCKS ? norm->rows : ZERO_NORM_BLOCKS;
    return 16 + (2 * blocks + (uint64_t)groups_of(*norm)) * 2 * (uint64_t)norm->cols * sizeof(float);
}

extern "C" zero_status_t zero_norm_backward(const zero_norm_t* norm, const void* dh_out, int64_t lddho,
                                            const void* dx, int64_t lddx, const void* ckpt_y,
                                            const void* ckpt_x, const float* stats, void* dh, int64_t lddh,
                                            void* dy, int64_t lddy, zero_dtype_t grad_dtype, void* dpost_w,
                                            void* dpost_b, void* dgate, void* dpre_w, void* dpre_b,
                                            int accumulate, void* work, void* stream)
{
    TraceRange trace_("zero_norm_backward");
    if (!description_ok(norm)) return ZERO_EINVAL;
    const zero_norm_t& d = *norm;
    const bool pre = d.pre != ZERO_NORM_NONE, post = d.post != ZERO_NORM_NONE;
    if ((int)grad_dtype != d.dtype && grad_dtype != ZERO_FP32) return ZERO_EINVAL;
    if ((!pre && (dpre_w || dpre_b || dx || ckpt_x)) || (!post && (dpost_w || dpost_b))) return ZERO_EINVAL;
    for (void* p : {dpost_w, dpost_b, dgate, dpre_w, dpre_b})
        if (!aligned_to(p, elem(grad_dtype))) return ZERO_EINVAL;
    if (d.rows > 0) {
        if (dh_out && !matrix_ok(dh_out, lddho, d.cols, d.res_dtype)) return ZERO_EINVAL;
        if (pre && (!matrix_ok(dx, lddx, d.cols, d.dtype) || !ckpt_x)) return ZERO_EINVAL;
        if (!dy && (!dh || post || d.gate || ckpt_y || dgate)) return ZERO_EINVAL;
        if (dh && !matrix_ok(dh, lddh, d.cols, d.res_dtype)) return ZERO_EINVAL;
        if (dy && !matrix_ok(dy, lddy, d.cols, d.dtype)) return ZERO_EINVAL;
        if ((post || dgate) && !ckpt_y) return ZERO_EINVAL;
        if ((pre || post) && !stats) return ZERO_EINVAL;
        if (!aligned_to(ckpt_y, 16) || !aligned_to(ckpt_x, 16) || !aligned_to(stats, 16)) return ZERO_EINVAL;
    }
    const bool sums = dpost_w || dpost_b || dgate || dpre_w || dpre_b;
    if (sums && (!work || !aligned_to(work, 16))) return ZERO_EINVAL;
    const bool slots = dpost_w || dpost_b || dgate;
    const bool two = dpre_b || dpost_b || (dgate && d.post_b);
    int64_t blocks = 0;
    float* const slot_sums = static_cast<float*>(work);
    float* pre_part = nullptr;
    if (d.rows > 0) {
        NormBwdArgs a{};
        a.dh_out = dh_out; a.dx = dx; a.dh = dh; a.dy = dy;
        a.post_w = d.post_w; a.gate = d.gate; a.pre_w = d.pre_w;
        a.ckpt_y = static_cast<const uint8_t*>(ckpt_y);
        a.ckpt_x = static_cast<const uint8_t*>(ckpt_x);
        a.stats = stats;
        a.rows = d.rows; a.lddho = lddho; a.lddx = lddx; a.lddh = lddh; a.lddy = lddy;
        a.group = d.group_rows ? d.group_rows : d.rows;
        a.cols = (int)d.cols;
        a.wide = (int)act_wide(d.cols);
        a.stride = (int)act_stride(d.cols);
        a.post = d.post; a.pre = d.pre;
        a.sums = two ? 2 : 1;
        a.alpha = d.alpha;
        a.inv_cols = 1.0f / (float)d.cols;
        a.vec_dho = vec_rows(dh_out, lddho, d.res_dtype);
        a.vec_dx = vec_rows(dx, lddx, d.dtype);
        a.vec_dh = vec_rows(dh, lddh, d.res_dtype);
        a.vec_dy = vec_rows(dy, lddy, d.dtype);
        a.vec_w = vec_weights(d);
        a.vec_g = vec_rows(d.gate, d.cols, d.dtype);
        int v = 1, threads = 32;
        row_shape(a.wide, v, threads);
        const void* fn = d.res_dtype == ZERO_FP32
                             ? (d.dtype == ZERO_FP16 ? backward_kernel<0, 2>(v, two) : backward_kernel<1, 2>(v, two))
                             : (d.dtype == ZERO_FP16 ? backward_kernel<0, 0>(v, two) : backward_kernel<1, 1>(v, two));
        blocks = resident(fn, threads);
        if (blocks == 0) return ZERO_ECUDA;
        if (blocks > ZERO_NORM_BLOCKS) blocks = ZERO_NORM_BLOCKS;
        if (blocks > d.rows) blocks = d.rows;
        pre_part = slot_sums + (blocks + groups_of(d)) * a.sums * d.cols;
        a.slots = slots ? slot_sums : nullptr;
        a.pre_part = dpre_w || dpre_b ? pre_part : nullptr;
        void* args[] = {&a};
        if (cudaLaunchKernel(fn, dim3((unsigned)blocks), dim3(threads), args, 0,
                             static_cast<cudaStream_t>(stream)) != cudaSuccess)
            return ZERO_ECUDA;
    }
    if (!sums) return ZERO_OK;
    NormSumArgs a{};
    a.pre_part = pre_part; a.slots = slot_sums;
    a.post_w = d.post_w; a.post_b = d.post_b; a.gate = d.gate;
    a.dpost_w = dpost_w; a.dpost_b = dpost_b; a.dgate = dgate; a.dpre_w = dpre_w; a.dpre_b = dpre_b;
    a.rows = d.rows;
    a.group = d.group_rows ? d.group_rows : d.rows > 0 ? d.rows : 1;
    a.groups = groups_of(d);
    a.cols = (int)d.cols;
    a.blocks = (int)blocks;
    a.sums = two ? 2 : 1;
    a.dtype = d.dtype; a.grad_dtype = grad_dtype; a.accumulate = accumulate != 0;
    a.alpha = d.alpha;
    a.col_jobs = (int)((d.cols + 31) / 32);
    a.flat_jobs = (int)((d.cols + 1023) / 1024);
    a.flat = a.groups * 8 > blocks;
    const int64_t jobs = 2ll * a.col_jobs + (dgate ? a.groups * (a.flat ? a.flat_jobs : a.col_jobs) : 0);
    void* args[] = {&a};
    return cudaLaunchKernel((const void*)k_norm_sums, dim3((unsigned)(jobs < (1 << 30) ? jobs : 1 << 30)),
                            dim3(32, 32), args, 0, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ZERO_OK
               : ZERO_ECUDA;
}
