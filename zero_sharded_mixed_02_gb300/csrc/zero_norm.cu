// zero_norm.cu -- the norms around a block: argument checks, launches, and the kernel
// that adds the backward pass's partial sums (zero_norm.cuh has the two passes).
#include <cmath>
#include <mutex>

#include "zero_norm.cuh"
#include "zero_trace.h"

namespace zero {

struct NormSumArgs {
    const float *pre_part, *post_part, *slots;
    const void *post_w, *post_b;
    void *dpost_w, *dpost_b, *dgate, *dpre_w, *dpre_b;
    int64_t rows, group, groups;
    int cols, wide, blocks, sums, dtype, grad_dtype, accumulate;
    int flat;
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

static __device__ __forceinline__ void add4(float4& v, const float* p)
{
    const float4 s = __ldcg(reinterpret_cast<const float4*>(p));
    v.x += s.x; v.y += s.y; v.z += s.z; v.w += s.w;
}

#define ZERO_NORM_SUM_THREADS 512       // of a job: strips of 32 or 8 threads

__host__ __device__ inline int64_t norm_sum_jobs(const NormSumArgs& a, int lanes)
{
    const int strips = ZERO_NORM_SUM_THREADS / lanes;
    const int64_t col_jobs = (a.cols + 4 * lanes - 1) / (4 * lanes);
    return col_jobs * (2 + (!a.dgate ? 0 : a.flat ? (a.groups + strips - 1) / strips : a.groups));
}

// The sums of a group's rows at column c: its blocks' slots from the group's block `first` by step.
static __device__ __forceinline__ void add_group(const NormSumArgs& a, int64_t g, int c, int first, int step,
                                                 float4& v0, float4& v1)
{
    if (a.rows == 0) return;
    const int64_t r0 = g * a.group, r1 = r0 + a.group < a.rows ? r0 + a.group : a.rows;
    const int64_t b1 = norm_block_of(r1 - 1, a.rows, a.blocks);
    for (int64_t b = norm_block_of(r0, a.rows, a.blocks) + first; b <= b1; b += step) {
        const float* p = a.slots + (b + g) * a.sums * a.wide + c;
        add4(v0, p);
        if (a.sums == 2) add4(v1, p + a.wide);
    }
}

static __device__ __forceinline__ void gate_out(const NormSumArgs& a, int64_t g, int64_t c, float v0, float v1)
{
    v0 *= weight_at(a.post_w, c, a.dtype);
    if (a.post_b) v0 = __fmaf_rn(weight_at(a.post_b, c, a.dtype), v1, v0);
    grad_out(a.dgate, g * a.cols + c, a.alpha * v0, a.grad_dtype, a.accumulate);
}

// Adds the blocks' partial sums.  A job is 128 or 32 columns (four a thread) of the pre-norm's
// sums, of the post-norm's, or of a gate group's; the strips of LANES threads take every 16th or
// 64th block's part, and the strips are added in order.  Where a group spans few blocks (flat), a
// gate job is these columns of as many groups instead, a strip each.  The parts lie in L2.  Few
// jobs are a matter of latency and are made narrow: 29.1 -> 24.9 us a backward pass at 8192 x 768
// (60 wide jobs), where many would come in waves: 87 -> 99 us at 8192 x 4096 (576).
template <int LANES>
__global__ void __launch_bounds__(ZERO_NORM_SUM_THREADS) k_norm_sums(const __grid_constant__ NormSumArgs a)
{
    constexpr int STRIPS = ZERO_NORM_SUM_THREADS / LANES, WIDTH = 4 * LANES, PARTS = ZERO_NORM_SUM_THREADS / WIDTH;
    __shared__ float4 s0[STRIPS][LANES], s1[STRIPS][LANES];
    __shared__ float r0[STRIPS > 16 ? PARTS : 1][WIDTH], r1[STRIPS > 16 ? PARTS : 1][WIDTH];
    asm volatile("griddepcontrol.wait;" ::: "memory");       // the pass whose sums these are
    const int strip = threadIdx.y;
    const int64_t jobs = norm_sum_jobs(a, LANES), col_jobs = (a.cols + WIDTH - 1) / WIDTH;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        float4 v0 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v1 = v0;
        const int64_t what = job / col_jobs;
        if (what >= 2 && a.flat) {
            const int64_t g = (what - 2) * STRIPS + strip;
            const int c = (int)(job - what * col_jobs) * WIDTH + 4 * threadIdx.x;
            if (g >= a.groups || c >= a.wide) continue;
            add_group(a, g, c, 0, 1, v0, v1);
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (c + e < a.cols) gate_out(a, g, c + e, (&v0.x)[e], (&v1.x)[e]);
            continue;
        }
        const int c = (int)(job - what * col_jobs) * WIDTH + 4 * threadIdx.x;
        if (what >= 2) {
            if (c < a.wide) add_group(a, what - 2, c, strip, STRIPS, v0, v1);
        } else if (const float* p = what == 0 ? a.pre_part : a.post_part; p && c < a.wide) {
#pragma unroll 8
            for (int b = strip; b < a.blocks; b += STRIPS) {
                add4(v0, p + (int64_t)b * a.sums * a.wide + c);
                if (a.sums == 2) add4(v1, p + (int64_t)b * a.sums * a.wide + a.wide + c);
            }
        }
        __syncthreads();                                     // the previous job's reads are done
        s0[strip][threadIdx.x] = v0;
        s1[strip][threadIdx.x] = v1;
        __syncthreads();
        // a thread a column; with many strips their sums by parts first
        const int at = strip * LANES + threadIdx.x, part = at / WIDTH, w = at % WIDTH;
        const float *p0 = reinterpret_cast<const float*>(s0), *p1 = reinterpret_cast<const float*>(s1);
        constexpr int LEFT = STRIPS > 16 ? PARTS : STRIPS;
        if (STRIPS > 16) {
            float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
            for (int i = 0; i < STRIPS / PARTS; i++) {
                t0 += p0[(part * (STRIPS / PARTS) + i) * WIDTH + w];
                t1 += p1[(part * (STRIPS / PARTS) + i) * WIDTH + w];
            }
            r0[part][w] = t0;
            r1[part][w] = t1;
            __syncthreads();
            p0 = r0[0];
            p1 = r1[0];
        }
        const int own = (int)(job - what * col_jobs) * WIDTH + w;
        if (part > 0 || own >= a.cols) continue;
        float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
        for (int i = 0; i < LEFT; i++) {
            t0 += p0[i * WIDTH + w];
            t1 += p1[i * WIDTH + w];
        }
        if (what == 0) {
            if (a.dpre_w) grad_out(a.dpre_w, own, t0, a.grad_dtype, a.accumulate);
            if (a.dpre_b) grad_out(a.dpre_b, own, t1, a.grad_dtype, a.accumulate);
        } else if (what == 1) {
            if (a.dpost_w) grad_out(a.dpost_w, own, a.alpha * t0, a.grad_dtype, a.accumulate);
            if (a.dpost_b) grad_out(a.dpost_b, own, a.alpha * t1, a.grad_dtype, a.accumulate);
        } else {
            gate_out(a, what - 2, own, t0, t1);
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

// ... and in whole chunks if the columns are too and an fp32 one is aligned to 32 bytes.
bool whole_rows(const void* p, int64_t ld, int dtype) { return aligned_to(p, dtype == ZERO_FP32 ? 32 : 16) && ld % 8 == 0; }

bool matrix_ok(const void* p, int64_t ld, int64_t cols, int dtype)
{
    return p && aligned_to(p, elem(dtype)) && ld >= cols && ld <= (1ll << 31);
}

// Rows of a gate group, at most all of them (and at least one), and the number of groups.
int64_t group_of(const zero_norm_t& d)
{
    const int64_t rows = d.rows > 0 ? d.rows : 1;
    return d.group_rows == 0 || d.group_rows > rows ? rows : d.group_rows;
}
int64_t groups_of(const zero_norm_t& d)
{
    return d.rows == 0 ? 1 : (d.rows + group_of(d) - 1) / group_of(d);
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

// Resident blocks of a kernel on the current device (0: a CUDA call failed) and its SMs,
// looked up once for each kernel and shape of its blocks.
int64_t resident(const void* fn, int threads, int smem, int& sms)
{
    struct Known { const void* fn; int dev, threads, smem, sms; int64_t blocks; };
    static std::mutex lock;
    static Known known[256];
    static int count = 0;
    int dev = 0, occ = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> hold(lock);
    for (int i = 0; i < count; i++)
        if (known[i].fn == fn && known[i].dev == dev && known[i].threads == threads && known[i].smem == smem) {
            sms = known[i].sms;
            return known[i].blocks;
        }
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, fn) != cudaSuccess ||
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - (int)at.sharedSizeBytes) !=
            cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, threads, smem) != cudaSuccess)
        return 0;
    const int64_t blocks = (int64_t)sms * (occ > 0 ? occ : 1);
    if (count < 256) known[count++] = {fn, dev, threads, smem, sms, blocks};
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
    a.rows = (uint32_t)d.rows;
    a.ldh = (uint32_t)ldh; a.ldy = (uint32_t)ldy; a.ldho = (uint32_t)ldho; a.ldx = (uint32_t)ldx;
    a.group = (uint32_t)group_of(d);
    a.cols = (int)d.cols;
    a.wide = (uint32_t)act_wide(d.cols);
    a.stride = (uint32_t)act_stride(d.cols);
    a.lo = act_lo(d.dtype);
    a.hi = act_hi(d.dtype);
    a.post = d.post; a.pre = d.pre;
    a.eps = d.eps; a.alpha = d.alpha;
    a.inv_cols = 1.0f / (float)d.cols;
    a.stop_h = static_cast<const char*>(h) + ((d.rows - 1) * ldh + d.cols) * elem(d.res_dtype);
    a.stop_y = static_cast<const char*>(y) + (y ? ((d.rows - 1) * ldy + d.cols) * elem(d.dtype) : 0);
    a.vec_h = vec_rows(h, ldh, d.res_dtype);
    a.vec_y = vec_rows(y, ldy, d.dtype);
    a.vec_ho = vec_rows(h_out, ldho, d.res_dtype);
    a.vec_x = vec_rows(x, ldx, d.dtype);
    a.vec_w = vec_weights(d);
    a.vec_g = vec_rows(d.gate, d.cols, d.dtype);
    int v = 1, threads = 32;
    row_shape((int)a.wide, v, threads);
    const bool whole = d.cols % 8 == 0 && y && whole_rows(h, ldh, d.res_dtype) && a.vec_y &&
                       whole_rows(h_out, ldho, d.res_dtype) && (!x || a.vec_x) && a.vec_w && (!d.gate || a.vec_g);
    const void* fn = d.dtype == ZERO_FP16 ? norm_forward_fp16(d.res_dtype, v, d.post, d.pre, whole)
                                          : norm_forward_bf16(d.res_dtype, v, d.post, d.pre, whole);
    const int smem = 16 * (d.post_b || d.pre_b ? ZERO_NORM_WORDS_BIAS : ZERO_NORM_WORDS) * v * threads;
    int sms = 0;
    const int64_t most = resident(fn, threads, smem, sms);
    if (most == 0) return ZERO_ECUDA;
    void* args[] = {&a};
    return cudaLaunchKernel(fn, dim3((unsigned)(d.rows < most ? d.rows : most)), dim3(threads), args, smem,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ZERO_OK
               : ZERO_ECUDA;
}

extern "C" uint64_t zero_norm_workspace(const zero_norm_t* norm)
{
    if (!description_ok(norm)) return 0;
    const uint64_t blocks = norm->rows < ZERO_NORM_BLOCKS ? norm->rows : ZERO_NORM_BLOCKS;
    return 16 + (3 * blocks + (uint64_t)groups_of(*norm)) * 2 * (uint64_t)act_wide(norm->cols) * sizeof(float);
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
    bool two = dpre_b || dpost_b || (dgate && d.post_b);
    int64_t blocks = 0;
    float *pre_part = nullptr, *post_part = nullptr, *slots = nullptr;
    if (d.rows > 0) {
        NormBwdArgs a{};
        a.dh_out = dh_out; a.dx = dx; a.dh = dh; a.dy = dy;
        a.post_w = d.post_w; a.gate = d.gate; a.pre_w = d.pre_w;
        a.ckpt_y = static_cast<const uint8_t*>(ckpt_y);
        a.ckpt_x = static_cast<const uint8_t*>(ckpt_x);
        a.stats = stats;
        a.rows = (uint32_t)d.rows;
        a.lddho = (uint32_t)lddho; a.lddx = (uint32_t)lddx; a.lddh = (uint32_t)lddh; a.lddy = (uint32_t)lddy;
        a.group = (uint32_t)group_of(d);
        a.cols = (int)d.cols;
        a.wide = (uint32_t)act_wide(d.cols);
        a.stride = (uint32_t)act_stride(d.cols);
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
        row_shape((int)a.wide, v, threads);
        const bool whole = d.cols % 8 == 0 && dy && (!dh_out || whole_rows(dh_out, lddho, d.res_dtype)) &&
                           (!dx || a.vec_dx) && (!dh || whole_rows(dh, lddh, d.res_dtype)) && a.vec_dy && a.vec_w &&
                           (!d.gate || a.vec_g);
        // other rows can be copied ahead too if their words, one more than chunks, have threads
        bool copied = !whole && dy && norm_kinds_copied(d.post, d.pre);
        if (copied) {
            int cv = 1, ct = 32;
            row_shape(((2 * a.cols + 13) / 16 + 1) * 8, cv, ct);
            copied = cv <= 2 && (int64_t)cv * ct * norm_ring_bytes(d.res_dtype) + 18 * 1024 <= 227 * 1024;
            if (copied) {
                v = cv;
                threads = ct;
            }
        }
        int smem = 0;
        const void* fn = d.dtype == ZERO_FP16
                             ? norm_backward_fp16(d.res_dtype, v, d.post, d.pre, whole, copied, two, smem)
                             : norm_backward_bf16(d.res_dtype, v, d.post, d.pre, whole, copied, two, smem);
        smem *= threads;
        int sms = 0;
        blocks = resident(fn, threads, smem, sms);
        if (blocks == 0) return ZERO_ECUDA;
        if (blocks > ZERO_NORM_BLOCKS) blocks = ZERO_NORM_BLOCKS;
        // At least four rows a block where that leaves a block an SM: a block's partial sums cost
        // as much as two or three rows (512 x 1600: 20.7 us with a block a row, 13 us so).
        const int64_t rows4 = (d.rows + 3) / 4, one = d.rows < sms ? d.rows : sms;
        if (blocks > (rows4 > one ? rows4 : one)) blocks = rows4 > one ? rows4 : one;
        const int64_t part = blocks * (two ? 2 : 1) * a.wide;
        float* at = static_cast<float*>(work);
        if (dpre_w || dpre_b) pre_part = at;
        if (dpost_w || dpost_b) post_part = at + part;
        if (dgate) slots = at + 2 * part;
        a.pre_part = pre_part;
        a.post_part = post_part;
        a.slots = slots;
        void* args[] = {&a};
        if (cudaLaunchKernel(fn, dim3((unsigned)blocks), dim3(threads), args, smem,
                             static_cast<cudaStream_t>(stream)) != cudaSuccess)
            return ZERO_ECUDA;
    }
    if (!sums) return ZERO_OK;
    NormSumArgs a{};
    a.pre_part = pre_part; a.post_part = post_part; a.slots = slots;
    a.post_w = d.post_w; a.post_b = d.post_b;
    a.dpost_w = dpost_w; a.dpost_b = dpost_b; a.dgate = dgate; a.dpre_w = dpre_w; a.dpre_b = dpre_b;
    a.rows = d.rows;
    a.group = group_of(d);
    a.groups = groups_of(d);
    a.cols = (int)d.cols;
    a.blocks = (int)blocks;
    a.sums = two ? 2 : 1;
    a.dtype = d.dtype; a.grad_dtype = grad_dtype; a.accumulate = accumulate != 0;
    a.alpha = d.alpha;
    a.wide = (int)act_wide(d.cols);
    a.flat = a.groups * 4 > blocks;
    const bool narrow = norm_sum_jobs(a, 32) <= 76 && blocks >= 128;
    const int64_t jobs = norm_sum_jobs(a, narrow ? 8 : 32);
    // placed while the pass drains; it waits for the pass's sums itself
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(jobs < (1 << 30) ? jobs : 1 << 30));
    c.blockDim = narrow ? dim3(8, ZERO_NORM_SUM_THREADS / 8) : dim3(32, ZERO_NORM_SUM_THREADS / 32);
    c.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, narrow ? k_norm_sums<8> : k_norm_sums<32>, a) == cudaSuccess ? ZERO_OK : ZERO_ECUDA;
}
