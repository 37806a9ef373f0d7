// zero_head.cu -- the vocabulary head's losses behind the C ABI: checks, workspace, launches.
#include "zero_head.cuh"

#include <math.h>

#include <mutex>

#include "zero_tensor_map.h"
#include "zero_trace.h"

using namespace zero;

namespace {

const int64_t MOST_PIECE = 65536;            // columns: 1024 stages of dx's accumulators

bool described(const zero_head_t* h)
{
    return h && (h->dtype == ZERO_FP16 || h->dtype == ZERO_BF16) && h->rows >= 0 && h->rows <= ZERO_HEAD_MAX_ROWS &&
           h->cols >= 1 && h->cols <= ZERO_HEAD_MAX_COLS && h->vocab >= 1 && h->vocab <= ZERO_HEAD_MAX_VOCAB &&
           h->piece >= 0 && h->top >= 0 && h->top <= ZERO_HEAD_MAX_TOP && isfinite(h->z_loss);
}
bool distill_described(const zero_head_t* h)
{
    return h->top >= 1 && h->top_dtype >= ZERO_FP16 && h->top_dtype <= ZERO_FP32 && isfinite(h->hard) && isfinite(h->soft) &&
           isfinite(h->temperature) && h->temperature > 0.0f && isfinite(1.4426950408889634f / h->temperature);
}

// Columns of a piece of the vocabulary, whole tiles: by default as many as keep dz within 1 GB, and pieces
// of about equal lengths.  Fewer where the weights are copied: within 256 MB of them.
int64_t even(int64_t vocab, int64_t most)
{
    most = up(most, ZERO_HD_TILE) * ZERO_HD_TILE;
    return up(up(vocab, up(vocab, most)), ZERO_HD_TILE) * ZERO_HD_TILE;
}
int64_t piece_of(const zero_head_t* h, int64_t npad)
{
    const int64_t room = (1ll << 29) / npad, want = h->piece > 0 ? h->piece : room < 4096 ? 4096 : room;
    return even(h->vocab, want < MOST_PIECE ? want : MOST_PIECE);
}
int64_t copied_of(int64_t piece, int64_t wide)
{
    const int64_t room = (1ll << 27) / wide;
    return room < piece ? even(piece, room) : piece;
}

// Lays the workspace out from `at`; returns its bytes.
uint64_t lay_out(const zero_head_t* h, HeadArgs& a, char* at)
{
    char* const begin = at;
    auto take = [&](auto*& p, int64_t n) {
        p = reinterpret_cast<decltype(+p)>(at);
        at += up(n * (int64_t)sizeof(*p), 256) * 256;
    };
    const int64_t rows = h->rows > 0 ? h->rows : 1, chunks = up(rows, ZERO_HD_CHUNK), tiles = up(h->vocab, ZERO_HD_TILE);
    a.npad = up(rows, ZERO_HD_TILE) * ZERO_HD_TILE;
    a.wide = (int)(up(h->cols, ZERO_HD_STEP) * ZERO_HD_STEP);
    a.pitch = piece_of(h, a.npad);
    take(a.st, 1);
    take(a.mask, chunks * 32);
    take(a.count, chunks);
    take(a.most, chunks);
    take(a.map, a.npad);
    take(a.exponent, a.npad);
    take(a.info, a.npad);
    take(a.target, rows * (h->top + 1));
    take(a.xp, a.npad * a.wide);
    take(a.wp, copied_of(a.pitch, a.wide) * a.wide);
    char* const rest = at;
    take(a.found, rows * (h->top + 1));       // forward
    take(a.partial, a.npad / 32);
    take(a.part, tiles * a.npad);
    take(a.part2, tiles * a.npad);
    char* const forward = at;
    at = rest;
    take(a.heavy, rows * ZERO_HD_HEAVY);      // backward
    take(a.heavies, rows);
    take(a.reach, a.npad);
    take(a.xs, a.npad * a.wide);
    take(a.dz, a.npad * a.pitch);
    take(a.acc, a.npad / ZERO_HD_TILE * up(h->cols, ZERO_HD_TILE) * ZERO_HD_SLOT);
    // as many parts as the largest call has
    auto parts = [&](int64_t tiles_, int64_t steps) {
        const int64_t most = (tiles_ < ZERO_HD_PAIRS ? tiles_ : ZERO_HD_PAIRS) * (steps / ZERO_HD_PART);
        return most < ZERO_HD_ROUNDS * ZERO_HD_PAIRS ? most : ZERO_HD_ROUNDS * ZERO_HD_PAIRS;
    };
    const int64_t wide = up(h->cols, ZERO_HD_TILE);
    a.slots_x = (int)parts(a.npad / ZERO_HD_TILE * wide, up(a.pitch, ZERO_HD_STEP));
    take(a.parts, (a.slots_x + parts(up(a.pitch, ZERO_HD_TILE) * wide, up(a.npad, ZERO_HD_STEP))) * ZERO_HD_SLOT);
    return (uint64_t)((at > forward ? at : forward) - begin);
}

HeadKernels kernels_of(int dtype) { return dtype == ZERO_FP16 ? head_kernels_fp16() : head_kernels_bf16(); }

// Pairs of SMs that run a launch's clusters at the same time; 0: a CUDA call failed.
int device_pairs(const HeadKernels& k)
{
    static std::mutex lock;
    static int pairs[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> hold(lock);
    if (pairs[dev] == 0) {
        for (const HeadKernels& of : {head_kernels_fp16(), head_kernels_bf16()})
            for (const void* fn : {of.logits[0], of.logits[1], of.gradient[0], of.gradient[1], of.products})
                if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, ZERO_HD_SMEM) != cudaSuccess) return 0;
        cudaLaunchConfig_t c{};
        c.gridDim = dim3(2 * ZERO_HD_PAIRS);
        c.blockDim = dim3(ZERO_HD_THREADS);
        c.dynamicSmemBytes = ZERO_HD_SMEM;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = 2;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        c.attrs = &at;
        c.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, k.products, &c) != cudaSuccess) return 0;
        pairs[dev] = n < 1 ? 1 : n > ZERO_HD_PAIRS ? ZERO_HD_PAIRS : n;
    }
    return pairs[dev];
}

// The matrices and targets of either pass; distill: of zero_distill_*.
bool inputs_ok(const zero_head_t* h, const void* x, int64_t ldx, const void* w, int64_t ldw, bool distill, const void* index,
               const void* logit, int64_t ldt, const void* labels, const void* work)
{
    if (!work || !aligned_to(work, 16) || !w || !aligned_to(w, 2) || ldw < h->cols || ldw > (1ll << 31)) return false;
    if (distill && (!distill_described(h) || ldt < h->top || ldt > (1ll << 31))) return false;
    if (!aligned_to(labels, 4) || !aligned_to(index, 4) || !aligned_to(logit, distill && h->top_dtype == ZERO_FP32 ? 4 : 2)) return false;
    if (h->rows == 0) return true;
    if (!x || !aligned_to(x, 2) || ldx < h->cols || ldx > (1ll << 31)) return false;
    return distill ? index && logit : labels != nullptr;
}

HeadArgs arguments(const zero_head_t* h, const void* x, int64_t ldx, const void* w, int64_t ldw, bool distill, const int32_t* index,
                   const void* logit, int64_t ldt, const int32_t* labels, void* work)
{
    HeadArgs a{};
    lay_out(h, a, static_cast<char*>(work));
    a.rows = h->rows; a.ldx = ldx; a.ldw = ldw; a.ldt = ldt;
    a.cols = (int)h->cols; a.vocab = (int)h->vocab;
    a.top = distill ? h->top : 0;
    a.slots = a.top + (labels ? 1 : 0);
    a.top_dtype = h->top_dtype;
    a.temperature = distill ? h->temperature : 1.0f;
    a.hard = distill ? h->hard : 1.0f;
    a.soft = distill ? h->soft : 0.0f;
    a.z_loss = h->z_loss;
    a.two = distill && labels && a.temperature != 1.0f;
    const double log2e = 1.4426950408889634;
    a.k2 = (float)(log2e / a.temperature);
    a.k1 = labels ? (float)log2e : a.k2;
    a.x = static_cast<const uint16_t*>(x);
    a.w = static_cast<const uint16_t*>(w);
    a.labels = labels;
    a.index = distill ? index : nullptr;
    a.logit = logit;
    // row tiles whose packed rows take 48 MB of L2
    const int64_t band = (48ll << 20) / (ZERO_HD_TILE * 2ll * a.wide);
    a.band = (int)(band < 1 ? 1 : band);
    return a;
}

// A launch that may begin while the kernel before it ends (which it waits for before it reads or
// writes anything): a call's kernels follow each other without the launches' latency, and with few rows the
// first one a kernel before the call that lets it (16 rows of 768 x 50257, call after call: 29.4 -> 28.1 us; blocks of
// more rows are in each other's way: 777 x 520 x 32003 backward 116 -> 118 us).
bool launch_next(const void* fn, dim3 grid, int threads, int smem, void** args, void* stream)
{
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelExC(&c, fn, args) == cudaSuccess;
}

// The passes over the rows.
bool run_rows(const HeadArgs& a, const HeadKernels& k, void* stream)
{
    void* args[] = {const_cast<HeadArgs*>(&a)};
    const dim3 grid((unsigned)up(a.rows + ZERO_HD_TILE, 8));
    const int smem = 8 * 2 * ((a.slots + 3) & ~3) * 4;
    if (a.rows <= ZERO_HD_TILE) return launch_next(k.pack, grid, 256, smem, args, stream);
    if (a.rows <= ZERO_HD_CHUNK) return launch(k.pack, grid, 256, smem, args, stream);
    return launch((const void*)k_head_rows, dim3((unsigned)up(a.rows, ZERO_HD_CHUNK)), ZERO_HD_CHUNK, 0, args, stream) &&
           launch_next(k.pack, grid, 256, smem, args, stream);
}

// Rows that leave from a writer's 32 rows of 32 columns.
bool map_out(CUtensorMap* m, const void* p, int64_t cols, int64_t rows, int64_t ld)
{
    return tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, p, cols, rows, ld * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}
bool map16(CUtensorMap* m, const void* p, int64_t cols, int64_t rows, int64_t ld, int box_rows)
{
    return tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, p, cols, rows, ld * 2, ZERO_HD_STEP, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The weights' map for a piece, which is copied first if its rows are not aligned.
bool weights(HeadArgs& a, int box_rows, bool copied, CUtensorMap* m)
{
    a.wy = copied ? 0 : a.v0;
    return copied ? map16(m, a.wp, a.wide, a.count_v, a.wide, box_rows) : map16(m, a.w, a.cols, a.vocab, a.ldw, box_rows);
}
bool copy_weights(const HeadArgs& a, int pairs, void* stream)
{
    void* args[] = {const_cast<HeadArgs*>(&a)};
    const int64_t most = 32ll * pairs, want = up(a.count_v, 8);
    return launch_next((const void*)k_head_weights, dim3((unsigned)(want < most ? want : most)), 256, 0, args, stream);
}
bool product(const void* fn, HeadArgs& a, int64_t tiles, int pairs, CUtensorMap* const (&maps)[5], void* stream)
{
    a.pairs = (int)(tiles < pairs ? tiles : pairs);
    void* args[] = {&a, maps[0], maps[1], maps[2], maps[3], maps[4]};
    return launch_next(fn, dim3(2 * a.pairs), ZERO_HD_THREADS, ZERO_HD_SMEM, args, stream);
}

zero_status_t forward(const zero_head_t* h, const void* x, int64_t ldx, const void* w, int64_t ldw, bool distill,
                      const int32_t* index, const void* logit, int64_t ldt, const int32_t* labels, float* loss, float* lse,
                      float* sums, void* work, void* stream)
{
    if (!described(h) || !inputs_ok(h, x, ldx, w, ldw, distill, index, logit, ldt, labels, work) || !aligned_to(loss, 4) ||
        !aligned_to(lse, 4) || !aligned_to(sums, 4) || (h->rows > 0 && (!loss || !lse)))
        return ZERO_EINVAL;
    if (h->rows == 0) {
        if (sums && cudaMemsetAsync(sums, 0, 8, static_cast<cudaStream_t>(stream)) != cudaSuccess) return ZERO_ECUDA;
        return ZERO_OK;
    }
    HeadArgs a = arguments(h, x, ldx, w, ldw, distill, index, logit, ldt, labels, work);
    a.loss = loss; a.lse = lse; a.sums = sums;
    a.xs = a.xp;
    const HeadKernels k = kernels_of(h->dtype);
    const int pairs = device_pairs(k);
    if (pairs == 0 || !encode() || !run_rows(a, k, stream)) return ZERO_ECUDA;
    const bool copied = !aligned_to(w, 16) || ldw % 8 != 0;
    CUtensorMap mx, mw;
    if (!map16(&mx, a.xp, a.wide, a.npad, a.wide, 128)) return ZERO_ECUDA;
    const int64_t step = copied ? copied_of(a.pitch, a.wide) : h->vocab;
    for (int64_t v = 0; v < h->vocab; v += step) {
        a.v0 = (int)v;
        a.count_v = (int)(h->vocab - v < step ? h->vocab - v : step);
        if (copied && !copy_weights(a, pairs, stream)) return ZERO_ECUDA;
        if (!weights(a, 128, copied, &mw) ||
            !product(k.logits[a.two], a, a.npad / ZERO_HD_TILE * up(a.count_v, ZERO_HD_TILE), pairs,
                     {&mx, &mw, &mx, &mw, &mx}, stream))
            return ZERO_ECUDA;
    }
    int tiles = (int)up(h->vocab, ZERO_HD_TILE);
    void* args[] = {&a, &tiles};
    const int64_t blocks = up(a.rows, 32);
    const void* loss_kernel = blocks <= 2 * pairs ? (const void*)k_head_loss<1> : (const void*)k_head_loss<2>;
    return launch_next(loss_kernel, dim3((unsigned)blocks), 1024, 0, args, stream) ? ZERO_OK : ZERO_ECUDA;
}

zero_status_t backward(const zero_head_t* h, const void* x, int64_t ldx, const void* w, int64_t ldw, bool distill,
                       const int32_t* index, const void* logit, int64_t ldt, const int32_t* labels, const float* lse,
                       const float* row_grad, float scale, const float* divisor, void* dx, int64_t lddx, void* dw, int64_t lddw,
                       int accumulate, void* work, void* stream)
{
    if (!described(h) || !inputs_ok(h, x, ldx, w, ldw, distill, index, logit, ldt, labels, work) || !aligned_to(lse, 4) ||
        !aligned_to(row_grad, 4) || !aligned_to(divisor, 4) || (!dx && !dw) || !aligned_to(dx, 2) || !aligned_to(dw, 2) ||
        (dx && (lddx < h->cols || lddx > (1ll << 31))) || (dw && (lddw < h->cols || lddw > (1ll << 31))) ||
        (h->rows > 0 && !lse))
        return ZERO_EINVAL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (h->rows == 0) {
        if (dw && !accumulate && cudaMemset2DAsync(dw, lddw * 2, 0, h->cols * 2, h->vocab, st) != cudaSuccess) return ZERO_ECUDA;
        return ZERO_OK;
    }
    HeadArgs a = arguments(h, x, ldx, w, ldw, distill, index, logit, ldt, labels, work);
    a.backward = 1;
    a.kept = lse; a.weight = row_grad; a.scale = scale; a.divisor = divisor;
    const float parts = (labels ? fabsf(a.hard) : 0.0f) + (a.index ? fabsf(a.soft) * a.temperature : 0.0f);
    a.unit = row_grad || parts == 0.0f || !isfinite(1.0f / parts) ? 1.0f : 1.0f / parts;
    a.dx = static_cast<uint16_t*>(dx);
    a.dw = static_cast<uint16_t*>(dw);
    a.lddx = lddx; a.lddw = lddw;
    a.accumulate = accumulate != 0;
    if (!row_grad && (h->z_loss == 0.0f || !labels)) a.xs = a.xp;     // all rows have one scale
    const HeadKernels k = kernels_of(h->dtype);
    const int pairs = device_pairs(k);
    if (pairs == 0 || !encode() || !run_rows(a, k, stream)) return ZERO_ECUDA;
    if (h->dtype == ZERO_FP16 && a.xs != a.xp && dw) {       // xs, which k_head_pack writes itself for bf16
        void* args[] = {&a};
        const int64_t most = 16ll * pairs, want = up(a.npad, 8);
        if (!launch_next((const void*)k_head_lift, dim3((unsigned)(want < most ? want : most)), 256, 0, args, stream)) return ZERO_ECUDA;
    }
    const bool copied = !aligned_to(w, 16) || ldw % 8 != 0;
    const int64_t rows = a.npad / ZERO_HD_TILE;
    CUtensorMap mx, ms, mz, mt, mo, md, mw, mn;
    a.vec = !copied;
    a.vec_x = aligned_to(dx, 16) && lddx % 8 == 0;
    a.vec_w = aligned_to(dw, 16) && lddw % 8 == 0;
    if (!map16(&mx, a.xp, a.wide, a.npad, a.wide, 128) || !map16(&ms, a.xs, a.wide, a.npad, a.wide, 64) ||
        !map16(&mz, a.dz, a.pitch, a.npad, a.pitch, 128) || !map16(&mt, a.dz, a.pitch, a.npad, a.pitch, 64) ||
        !map_out(&mo, a.dz, a.pitch, a.npad, a.pitch))
        return ZERO_ECUDA;
    if (!dw || !a.vec_w) md = mo;
    else if (!map_out(&md, dw, a.cols, a.vocab, lddw)) return ZERO_ECUDA;
    const int64_t step = copied ? copied_of(a.pitch, a.wide) : a.pitch;
    for (int64_t v = 0; v < h->vocab; v += step) {
        a.v0 = (int)v;
        a.count_v = (int)(h->vocab - v < step ? h->vocab - v : step);
        a.first = v == 0;
        a.last = v + step >= h->vocab;
        if (copied && !copy_weights(a, pairs, stream)) return ZERO_ECUDA;
        if (!weights(a, 128, copied, &mw) || !weights(a, 64, copied, &mn) ||
            !product(k.gradient[a.two], a, rows * up(a.count_v, ZERO_HD_TILE), pairs, {&mx, &mw, &mx, &mw, &mo}, stream) ||
            !product(k.products, a, pairs, pairs, {&mz, &mn, &mt, &ms, &md}, stream))
            return ZERO_ECUDA;
        // tiles are cut from twice a part's stages on
        void* args[] = {&a};
        const int64_t least = (2 * ZERO_HD_PART - 1) * ZERO_HD_STEP;
        if (((dx && a.count_v > least) || (dw && a.rows > least)) &&
            !launch_next(k.join, dim3(4 * pairs), 256, 0, args, stream))
            return ZERO_ECUDA;
    }
    return ZERO_OK;
}

}  // namespace

extern "C" uint64_t zero_head_workspace(const zero_head_t* head)
{
    if (!described(head)) return 0;
    HeadArgs a{};
    return lay_out(head, a, nullptr);
}

extern "C" zero_status_t zero_ce_forward(const zero_head_t* head, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                         const int32_t* labels, float* loss, float* lse, float* sums, void* work, void* stream)
{
    TraceRange trace_("zero_ce_forward");
    return forward(head, x, ldx, w, ldw, false, nullptr, nullptr, 0, labels, loss, lse, sums, work, stream);
}

extern "C" zero_status_t zero_ce_backward(const zero_head_t* head, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                          const int32_t* labels, const float* lse, const float* row_grad, float scale,
                                          const float* divisor, void* dx, int64_t lddx, void* dw, int64_t lddw, int accumulate,
                                          void* work, void* stream)
{
    TraceRange trace_("zero_ce_backward");
    return backward(head, x, ldx, w, ldw, false, nullptr, nullptr, 0, labels, lse, row_grad, scale, divisor, dx, lddx, dw, lddw,
                    accumulate, work, stream);
}

extern "C" zero_status_t zero_distill_forward(const zero_head_t* head, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                              const int32_t* top_index, const void* top_logit, int64_t ldt, const int32_t* labels,
                                              float* loss, float* lse, float* sums, void* work, void* stream)
{
    TraceRange trace_("zero_distill_forward");
    return forward(head, x, ldx, w, ldw, true, top_index, top_logit, ldt, labels, loss, lse, sums, work, stream);
}

extern "C" zero_status_t zero_distill_backward(const zero_head_t* head, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                               const int32_t* top_index, const void* top_logit, int64_t ldt, const int32_t* labels,
                                               const float* lse, const float* row_grad, float scale, const float* divisor, void* dx,
                                               int64_t lddx, void* dw, int64_t lddw, int accumulate, void* work, void* stream)
{
    TraceRange trace_("zero_distill_backward");
    return backward(head, x, ldx, w, ldw, true, top_index, top_logit, ldt, labels, lse, row_grad, scale, divisor, dx, lddx, dw,
                    lddw, accumulate, work, stream);
}
