// zero_norm.cu -- the norms around a block: argument checks, launches, and the kernel
// that adds the backward pass's partial sums (zero_norm.cuh has the two passes).
#include <cmath>
#include <mutex>

#include "zero_norm.cuh"
#include "zero_trace.h"

namespace zero {

struct NormSumArgs {
    const float *pre_part, *slots;
    const void *post_w, *post_b, *gate;
    void *dpost_w, *dpost_b, *dgate, *dpre_w, *dpre_b;
    int64_t rows, group, groups;
    int cols, wide, blocks, sums, dtype, grad_dtype, accumulate;
    int col_jobs;
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

static __device__ __forceinline__ void add_part(const float* p, int wide, int sums, float w, float4& v0, float4& v1)
{
    const float4 s = __ldcg(reinterpret_cast<const float4*>(p));
    v0.x = __fmaf_rn(w, s.x, v0.x); v0.y = __fmaf_rn(w, s.y, v0.y);
    v0.z = __fmaf_rn(w, s.z, v0.z); v0.w = __fmaf_rn(w, s.w, v0.w);
    if (sums == 2) {
        const float4 t = __ldcg(reinterpret_cast<const float4*>(p + wide));
        v1.x = __fmaf_rn(w, t.x, v1.x); v1.y = __fmaf_rn(w, t.y, v1.y);
        v1.z = __fmaf_rn(w, t.z, v1.z); v1.w = __fmaf_rn(w, t.w, v1.w);
    }
}

// Adds the blocks' partial sums.  A job is 128 columns (four a thread) of the pre-norm's
// sums, of the post-norm's, or of a gate group's; eight strips of threads take every
// eighth block's part, and the strips are added in order.
__global__ void __launch_bounds__(256) k_norm_sums(const __grid_constant__ NormSumArgs a)
{
    __shared__ float4 s0[8][32], s1[8][32];
    const int strip = threadIdx.y;
    const int64_t jobs = a.col_jobs * (2 + (a.dgate ? a.groups : 0));
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        float4 v0 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v1 = v0;
        const int64_t what = job / a.col_jobs;
        const int c = (int)(job - what * a.col_jobs) * 128 + 4 * threadIdx.x;
        if (c < a.wide && a.rows > 0) {
            if (what == 0) {
                if (a.dpre_w || a.dpre_b)
#pragma unroll 4
                    for (int b = strip; b < a.blocks; b += 8)
                        add_part(a.pre_part + (int64_t)b * a.sums * a.wide + c, a.wide, a.sums, 1.0f, v0, v1);
            } else if (what == 1) {
                if (a.dpost_w || a.dpost_b)
                    for (int b = strip; b < a.blocks; b += 8) {
                        const int64_t g0 = norm_row0(b, a.rows, a.blocks) / a.group;
                        const int64_t g1 = (norm_row0(b + 1, a.rows, a.blocks) - 1) / a.group;
                        for (int64_t g = g0; g <= g1; g++) {
                            float4 q0 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), q1 = q0;
                            add_part(a.slots + (b + g) * a.sums * a.wide + c, a.wide, a.sums, a.alpha, q0, q1);
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const float w = c + e < a.cols ? weight_at(a.gate, g * a.cols + c + e, a.dtype) : 0.0f;
                                (&v0.x)[e] = __fmaf_rn(w, (&q0.x)[e], (&v0.x)[e]);
                                (&v1.x)[e] = __fmaf_rn(w, (&q1.x)[e], (&v1.x)[e]);
                            }
                        }
                    }
            } else {
                const int64_t g = what - 2, r0 = g * a.group, r1 = r0 + a.group < a.rows ? r0 + a.group : a.rows;
                const int64_t b1 = norm_block_of(r1 - 1, a.rows, a.blocks);
                for (int64_t b = norm_block_of(r0, a.rows, a.blocks) + strip; b <= b1; b += 8)
                    add_part(a.slots + (b + g) * a.sums * a.wide + c, a.wide, a.sums, a.alpha, v0, v1);
            }
        }
        __syncthreads();                                     // the previous job's reads are done
        s0[strip][threadIdx.x] = v0;
        s1[strip][threadIdx.x] = v1;
        __syncthreads();
        if (strip >= 4) continue;                            // the first four finish 32 columns each
        const int own = (int)(job - what * a.col_jobs) * 128 + strip * 32 + threadIdx.x;
        if (own >= a.cols) continue;
        float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            t0 += reinterpret_cast<const float*>(s0[i])[strip * 32 + threadIdx.x];
            t1 += reinterpret_cast<const float*>(s1[i])[strip * 32 + threadIdx.x];
        }
        if (what == 0) {
            if (a.dpre_w) grad_out(a.dpre_w, own, t0, a.grad_dtype, a.accumulate);
            if (a.dpre_b) grad_out(a.dpre_b, own, t1, a.grad_dtype, a.accumulate);
        } else if (what == 1) {
            if (a.dpost_w) grad_out(a.dpost_w, own, t0, a.grad_dtype, a.accumulate);
            if (a.dpost_b) grad_out(a.dpost_b, own, t1, a.grad_dtype, a.accumulate);
        } else {
            t0 *= weight_at(a.post_w, own, a.dtype);
            if (a.post_b) t0 = __fmaf_rn(weight_at(a.post_b, own, a.dtype), t1, t0);
            grad_out(a.dgate, (what - 2) * a.cols + own, t0, a.grad_dtype, a.accumulate);
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

// Resident blocks of a kernel on the current device, looked up once for each kernel and
// block size; 0: a CUDA call failed.
int64_t resident(const void* fn, int threads)
{
    struct Known { const void* fn; int dev, threads; int64_t blocks; };
    static std::mutex lock;
    static Known known[256];
    static int count = 0;
    int dev = 0, sms = 0, occ = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> hold(lock);
    for (int i = 0; i < count; i++)
        if (known[i].fn == fn && known[i].dev == dev && known[i].threads == threads) return known[i].blocks;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, threads, 0) != cudaSuccess)
        return 0;
    const int64_t blocks = (int64_t)sms * (occ > 0 ? occ : 1);
    if (count < 256) known[count++] = {fn, dev, threads, blocks};
    return blocks;
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
    a.rows = (uint32_t)d.rows; a.ldh = ldh; a.ldy = ldy; a.ldho = ldho; a.ldx = ldx;
    a.group = (uint32_t)(d.group_rows == 0 || d.group_rows > d.rows ? d.rows : d.group_rows);
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
    const bool whole = d.cols % 8 == 0 && a.vec_h && (!y || a.vec_y) && (!h_out || a.vec_ho) && (!x || a.vec_x) &&
                       a.vec_w && (!d.gate || a.vec_g);
    const void* fn = d.dtype == ZERO_FP16 ? norm_forward_fp16(d.res_dtype, v, whole)
                                          : norm_forward_bf16(d.res_dtype, v, whole);
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
    return 16 + (2 * blocks + (uint64_t)groups_of(*norm)) * 2 * (uint64_t)act_wide(norm->cols) * sizeof(float);
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
        const bool whole = d.cols % 8 == 0 && (!dh_out || a.vec_dho) && (!dx || a.vec_dx) && (!dh || a.vec_dh) &&
                           (!dy || a.vec_dy) && a.vec_w && (!d.gate || a.vec_g);
        const void* fn = d.dtype == ZERO_FP16 ? norm_backward_fp16(d.res_dtype, v, two, whole)
                                              : norm_backward_bf16(d.res_dtype, v, two, whole);
        blocks = resident(fn, threads);
        if (blocks == 0) return ZERO_ECUDA;
        if (blocks > ZERO_NORM_BLOCKS) blocks = ZERO_NORM_BLOCKS;
        if (blocks > d.rows) blocks = d.rows;
        pre_part = slot_sums + (blocks + groups_of(d)) * (two ? 2 : 1) * a.wide;
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
    a.wide = (int)act_wide(d.cols);
    a.col_jobs = (int)((d.cols + 127) / 128);
    const int64_t jobs = a.col_jobs * (2 + (dgate ? a.groups : 0));
    void* args[] = {&a};
    return cudaLaunchKernel((const void*)k_norm_sums, dim3((unsigned)(jobs < (1 << 30) ? jobs : 1 << 30)),
                            dim3(32, 8), args, 0, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ZERO_OK
               : ZERO_ECUDA;
}
