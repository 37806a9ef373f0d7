// zero_head.cuh -- kernels of the vocabulary head's losses (include/zero_b200.h).
//
// The logits z = x w^T (rows x vocab) are never kept.  All products run on the tensor cores, a
// pair of SMs (a cluster of two) on a 256 x 256 tile, 64 steps of the contracted axis a stage:
//   LOGITS    z tile by tile; each tile leaves a row's maximum and sum of exponentials
//   GRADIENT  the same tiles again; each leaves its gradient dz (16 bits, scaled by a power of
//             two a row) in the workspace, a piece of the vocabulary at a time
//   PRODUCTS  dx += dz w of the piece, summed over pieces in fp32, and dw = dz^T x
// Rows that take no part are left out before the first product: a pass over the rows packs the
// others (aligned, padded with zeros to a whole stage), so what their x holds is not read, and
// every product's rows are the counted ones.
//
// From a thousand rows on the products are bound by the tensor cores, whose memory is busy in 96 % of an
// SM's active cycles (4096 x 4096 x 128256, bf16, settled under the power limit: forward 2395 us = 1797 TFLOP/s,
// backward 7463 = 1730; a library product 1882 at first and 1698 sustained); fewer rows by reading the weights (once
// forward, twice backward) and writing dw, and by about 7 us that a launch of k_head takes to begin and end.  A call's
// kernels follow each other by programmatic launches, which took 33 -> 29 us for 64 x 256 x 1000 backward and 109 -> 98
// us for 1999 x 771 x 32003 forward.
#pragma once

#include <cuda.h>

#include "zero_b200.h"
#include "zero_common.cuh"
#include "zero_pair.cuh"

namespace zero {

#define ZERO_HD_TILE 256                     // rows and columns of a pair's tile
#define ZERO_HD_STEP 64                      // contracted elements of a stage
#define ZERO_HD_STAGES 6                     // (five, for twice the rows on their way out: 1 to 3 % slower)
#define ZERO_HD_SIDE 16384                   // bytes of a stage's operand in one SM
#define ZERO_HD_WRITERS 16                   // warps that read the accumulators
#define ZERO_HD_THREADS (128 + 32 * ZERO_HD_WRITERS)    // warp 0 loads, 1 products, from 4 output
#define ZERO_HD_ROWS 2048                    // bytes in which a writer lays 32 rows of 32 columns
#define ZERO_HD_SMEM (ZERO_HD_STAGES * 2 * ZERO_HD_SIDE + ZERO_HD_WRITERS * ZERO_HD_ROWS + 1024)
#define ZERO_HD_PAIRS 80                     // most pairs that share a launch's work
#define ZERO_HD_PART 16                      // least stages of a part of a cut tile,
#define ZERO_HD_ROUNDS 4                     // and most parts of a pair
#define ZERO_HD_RUN 12                       // stages an accumulator adds for the loss
#define ZERO_HD_CHUNK 1024                   // rows whose counted ones are numbered by one block
#define ZERO_HD_SLOT (ZERO_HD_TILE * ZERO_HD_TILE)      // floats of a tile's sums
#define ZERO_HD_SCALE 14                     // dz is kept times 2^14 over its row's power of two
#define ZERO_HD_NONE 0x7FFFFFFF              // column of no target
#define ZERO_HD_NO_REACH (-100000)           // exponent of a row that has none
#define ZERO_HD_HEAVY 4                      // columns of a row with a quarter of its targets' weight or more
#ifndef ZERO_HD_WAIT_LIMIT                   // polls before a wait gives up
#define ZERO_HD_WAIT_LIMIT ZERO_TMA_WAIT_LIMIT
#endif

enum HeadPass { HEAD_LOGITS = 0, HEAD_GRADIENT = 1, HEAD_INPUT = 2, HEAD_WEIGHT = 3, HEAD_PRODUCTS = 4 };

// How the writers share the work.  Logits, whose runs are added in registers: all read every tile,
// 64 columns each (128 would spill: 6.4 against 4.4 ms at 8192 x 128256 x 4096; 64 at two temperatures spill 4 bytes).
// The others: two groups of eight take tiles in turn, one accumulator each, 128 columns a warp, so that one group's
// loads and stores are under way while the other computes.
__host__ __device__ constexpr int head_groups(int pass) { return pass == HEAD_LOGITS ? 1 : 2; }
__host__ __device__ constexpr int head_columns(int pass) { return 4 * ZERO_HD_TILE * head_groups(pass) / ZERO_HD_WRITERS; }

// The tensor cores cut each sum off rather than round it, so an accumulator's relative error grows by
// about 1.6e-8 a step of 16 columns.  The loss is fp32 and would show it: its logits are added in runs of 12
// stages (48 steps) and the runs in fp32.  8192 x 4096 x 128256: runs of 12 stages are off by 3.5e-7 in the
// 2-norm, of 24 by 7.4e-7, of 40 by 1.2e-6 (fp32 products without tensor cores: 6e-7), all within 2 % of the same
// time.  (At 768 columns, one run, by 6e-7, fp32 products by 2.5e-7.)  dz is rounded to 16 bits, 2^-9 or 2^-12 in the
// mean, and needs none; dx's accumulators add at most 65536 columns and dw's 65536 rows (4096 steps: 6.6e-5).

// What the passes over the rows leave for the rest, at the head of the workspace.
struct HeadState {
    int32_t err;                             // ZERO_ETIMEOUT once a wait gave up
    uint32_t ticket;
    int32_t rows;                            // counted rows
    int32_t top;                             // largest exponent of their gradients' scales
    int32_t lift;                            // of the packed rows for dw: 2^lift times what their own scales would make them
};

// A target of a row: its column (24 bits; above them its place among the row's heavy ones, from 1) and its
// weight, the teacher's share or the label's.
struct __align__(8) HeadTarget {
    int32_t column;
    float weight;
};

// A target that has much of its row's weight: its column, and what rounding dz cut off there.
struct __align__(8) HeadHeavy {
    int32_t column;
    float cut;
};

// A counted row.  Gradients: dz = c1 2^(k1 z - l1) + c2 2^(k2 z - l2) - weight at the targets.
struct __align__(16) HeadRow {
    float c1, l1, c2, l2;
};

struct HeadArgs {
    int64_t rows, ldx, ldw, ldt, lddx, lddw;
    int cols, vocab, top, slots;             // slots: targets of a row (top, and one for the label)
    int top_dtype, two, backward;            // two: both log-sum-exps are needed
    float temperature, hard, soft, z_loss, k1, k2, scale, unit;
    const uint16_t *x, *w;
    const int32_t *labels, *index;
    const void* logit;
    const float *weight, *divisor, *kept;    // the backward pass's row weights, divisor, log-sum-exps
    float *loss, *lse, *sums;
    uint16_t *dx, *dw;
    int accumulate, vec, vec_x, vec_w;       // aligned rows: of w, dx, dw
    // workspace
    HeadState* st;
    uint32_t* mask;                          // counted rows, a bit each
    int32_t *count, *most;                   // of a chunk of rows: how many; their largest exponent
    int32_t *map, *exponent;                 // counted row -> row, its scale's exponent
    int32_t* reach;                          // (backward, fp16) the exponent of its scale times its largest x
    HeadRow* info;                           // (forward: c1 is the loss's constant part, c2 the teacher's share)
    HeadTarget* target;                      // of a counted row, by columns
    float* found;                            // their logits
    HeadHeavy* heavy;                        // [ZERO_HD_HEAVY] of a counted row, and their number
    int32_t* heavies;
    double* partial;
    float2* part;                            // [tiles of the vocabulary][npad]: maximum, sum
    float* part2;                            // the sum at the temperature
    uint16_t *xp, *xs, *wp, *dz;             // packed rows, the same scaled for dw, weights where repacked, dz
    float *acc, *parts;
    int64_t npad, pitch;                     // packed rows, columns of dz
    int wide;                                // columns of packed rows
    // this launch
    int pairs, v0, count_v, wy;              // first column of the piece, columns, its first row in the weights' map
    int first, last;                         // piece
    int slots_x;                             // places of dx's parts
    int band;                                // row tiles that are taken together
};

// ---- the division of the work ------------------------------------------------------
struct HeadShape {
    uint32_t tm, tn, steps, runs, run, waves, rest;
    uint32_t ranges;                         // parts that the rest's tiles are cut into
};
struct HeadSegment {
    uint32_t tile;
    int32_t s0, s1;
    int slot;                                // of a part of a cut tile, else -1
    bool first, last;                        // run of the tile
    bool input;                              // of dx (else of dw, where there are two)
};

static __host__ __device__ __forceinline__ uint32_t head_up(uint32_t a, uint32_t b) { return (a + b - 1) / b; }

// Tiles along the left operand's rows (tm) and the right one's (tn), and how `pairs` pairs share
// them: whole waves, then the rest, whose tiles are cut along the contracted axis (INPUT, WEIGHT)
// where that is long enough to pay for joining the parts.  All are cut at the same places, and the parts of a
// range of the axis run at about the same time, so that they share their panels in L2: cut into equal shares of all
// pairs instead, 1843 rows of 4096 x 64256 took 1260 us with their dw, and take 1036.
template <int PASS>
static __host__ __device__ __forceinline__ HeadShape head_shape(const HeadArgs& a, int counted)
{
    HeadShape s;
    const uint32_t n = counted > 0 ? counted : 1, pairs = a.pairs;
    const uint32_t rows = head_up(n, ZERO_HD_TILE), words = head_up(a.count_v, ZERO_HD_TILE), wide = head_up(a.cols, ZERO_HD_TILE);
    s.tm = PASS == HEAD_WEIGHT ? words : rows;
    s.tn = PASS <= HEAD_GRADIENT ? words : wide;
    s.steps = head_up(PASS <= HEAD_GRADIENT ? a.cols : PASS == HEAD_INPUT ? a.count_v : n, ZERO_HD_STEP);
    s.runs = PASS == HEAD_LOGITS ? head_up(s.steps, ZERO_HD_RUN) : 1;
    s.run = head_up(s.steps, s.runs);
    s.runs = head_up(s.steps, s.run);
    const uint32_t tiles = s.tm * s.tn;
    s.waves = tiles / pairs;
    s.rest = tiles % pairs;
    s.ranges = 1;
    if (PASS >= HEAD_INPUT && s.rest > 0) {
        // as many parts as fill one to four rounds of all pairs: the least time, in stages, of the rounds,
        // each with its output, and the join (about 20)
        uint32_t best = s.steps + 8;
        for (uint32_t k = 1; k <= ZERO_HD_ROUNDS; k++) {
            const uint32_t fill = k * pairs / s.rest, most = s.steps / ZERO_HD_PART, r = fill < most ? fill : most;
            const uint32_t time = k * (head_up(s.steps, r > 0 ? r : 1) + 8) + 20 + r;
            if (r > 1 && time < best) {
                best = time;
                s.ranges = r;
            }
        }
    }
    return s;
}

// Segment i of a pair; false past its last.
template <int PASS>
static __host__ __device__ __forceinline__ bool head_segment(const HeadArgs& a, const HeadShape& s, uint32_t pair, uint32_t i,
                                                             HeadSegment& g)
{
    if (i < s.waves * s.runs) {
        const uint32_t w = s.runs == 1 ? i : i / s.runs, r = i - w * s.runs;
        g.tile = w * a.pairs + pair;
        g.s0 = r * s.run;
        g.last = r + 1 == s.runs;
        g.s1 = g.last ? s.steps : g.s0 + s.run;
        g.first = r == 0;
        g.slot = -1;
        return true;
    }
    i -= s.waves * s.runs;
    if (PASS <= HEAD_GRADIENT) {             // whole tiles
        if (pair >= s.rest || i >= s.runs) return false;
        g.tile = s.waves * a.pairs + pair;
        g.s0 = i * s.run;
        g.last = i + 1 == s.runs;
        g.s1 = g.last ? s.steps : g.s0 + s.run;
        g.first = i == 0;
        g.slot = -1;
        return true;
    }
    g.first = g.last = true;
    if (s.rest == 0) return false;
    const uint32_t part = i * a.pairs + pair, range = part / s.rest;
    if (range >= s.ranges) return false;
    g.tile = s.waves * a.pairs + (part - range * s.rest);
    g.s0 = range * s.steps / s.ranges;
    g.s1 = (range + 1) * s.steps / s.ranges;
    g.slot = s.ranges > 1 ? (int)part : -1;
    return true;
}

// The products' segments: dx's, then dw's, whose tiles are dealt to the pairs from the last one on, so that
// incomplete rounds of the two fall on different pairs.  `inputs`: how many a pair has of the first.
static __host__ __device__ __forceinline__ uint32_t head_inputs(const HeadArgs& a, const HeadShape& s, uint32_t pair)
{
    if (!a.dx) return 0;
    return s.waves + (s.ranges * s.rest + a.pairs - 1 - pair) / a.pairs;
}
template <int PASS>
static __host__ __device__ __forceinline__ bool head_next(const HeadArgs& a, const HeadShape& s, const HeadShape& w, uint32_t inputs,
                                                          uint32_t pair, uint32_t i, HeadSegment& g)
{
    if (PASS != HEAD_PRODUCTS) return head_segment<PASS>(a, s, pair, i, g);
    g.input = i < inputs;
    if (g.input) return head_segment<HEAD_INPUT>(a, s, pair, i, g);
    if (!a.dw || !head_segment<HEAD_WEIGHT>(a, w, a.pairs - 1 - pair, i - inputs, g)) return false;
    if (g.slot >= 0) g.slot += a.slots_x;
    return true;
}

// Tiles of the logits: bands of row tiles that stay in L2 while the weights pass by once a band;
// of the products: bands of eight, which keep a wave's panels few.
static __host__ __device__ __forceinline__ void head_place(uint32_t band, const HeadShape& s, uint32_t tile, uint32_t& i, uint32_t& j)
{
    const uint32_t b = tile / (band * s.tn), in = tile - b * band * s.tn;
    const uint32_t high = s.tm - b * band < band ? s.tm - b * band : band;
    j = in / high;
    i = b * band + (in - j * high);
}
template <int PASS>
static __host__ __device__ __forceinline__ uint32_t head_band(const HeadArgs& a) { return PASS <= HEAD_GRADIENT ? a.band : 8; }

// Columns that are multiplied of a products' tile at column tile j: half a tile at the right edge where that is
// enough (each SM's part is then one whole 64-column group of the operand's layout).
template <int PASS>
static __device__ __forceinline__ int head_width(const HeadArgs& a, uint32_t j)
{
    return PASS <= HEAD_GRADIENT || a.cols - (int)j * ZERO_HD_TILE > ZERO_HD_TILE / 2 ? ZERO_HD_TILE : ZERO_HD_TILE / 2;
}

// A call's kernels begin before the one before has ended; this waits for that one's results.  Nothing is read
// through the non-coherent path (__ldg), which is for what does not change while a kernel lives.
template <class T>
static __device__ __forceinline__ T fetch(const T* p) { return *p; }
static __device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
static __device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---- scalars -------------------------------------------------------------------------
static __device__ __forceinline__ float power2(int e)       // 2^e, 0 below the normal range
{
    return e < -126 ? 0.0f : __uint_as_float((uint32_t)(e + 127) << 23);
}
static __device__ __forceinline__ float exp2_fast(float x)  // within 2 ulp; 0 below 2^-126
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
static __device__ __forceinline__ float teacher_logit(const HeadArgs& a, int64_t row, int k)
{
    const int64_t i = row * a.ldt + k;
    if (a.top_dtype == 2) return fetch(static_cast<const float*>(a.logit) + i);
    const uint16_t u = fetch(static_cast<const uint16_t*>(a.logit) + i);
    return a.top_dtype == 0 ? widen1<0>(u) : widen1<1>(u);
}
static __device__ __forceinline__ bool has_entry(const HeadArgs& a, int64_t row, int k)
{
    return fetch(a.index + row * a.ldt + k) >= 0 && teacher_logit(a, row, k) != __uint_as_float(0xFF800000u);
}

// What all rows' gradients are multiplied with after the products: scale / divisor (0 where the divisor is), over
// `unit`; sums over no rows are 0 whatever that is.  A row's dz is kept times its weight, or where rows have none times
// `unit`, one over the sum of the parts' weights: a label's coefficient p - 1 then lies just below a power of two,
// where rounding it (which is most of dz's rounding) costs least: 0.7 of a rounding at random, in all rows.
static __device__ __forceinline__ float common_factor(const HeadArgs& a)
{
    const float d = a.divisor ? fetch(a.divisor) : 1.0f;
    return d == 0.0f ? 0.0f : a.scale / a.unit / d;
}
static __device__ __forceinline__ float row_scale(const HeadArgs& a, int64_t row)
{
    return a.weight ? fetch(a.weight + row) : a.unit;
}
// Factors of the two softmaxes in a row's gradient before the row's power of two, and a bound of |dz|.  A row of weight
// 0 has none whatever its log-sum-exp is (0 times inf or NaN would be NaN), and without z_loss that is no factor.
static __device__ __forceinline__ void row_factors(const HeadArgs& a, int64_t row, float& s, float& hard, float& soft)
{
    s = row_scale(a, row);
    hard = 0.0f;
    if (a.labels) {
        const float l = a.index ? fetch(a.kept + 2 * row + 1) : fetch(a.kept + row);
        hard = s == 0.0f ? 0.0f : s * a.hard * (a.z_loss == 0.0f ? 1.0f : 1.0f + 2.0f * a.z_loss * l);
    }
    soft = a.index ? s * a.soft * a.temperature : 0.0f;
}
static __device__ __forceinline__ float factors_bound(const HeadArgs& a, float s, float hard, float soft)
{
    return fabsf(hard) + fabsf(soft) + fabsf(s) * ((a.labels ? fabsf(a.hard) : 0.0f) + (a.index ? fabsf(a.soft) * a.temperature : 0.0f));
}
// Exponent of a bound, kept where 2^(14 - e) and its inverse are normal; of an inf or a NaN, 0.
static __device__ __forceinline__ int bound_exponent(float b)
{
    const int e = (int)(__float_as_uint(b) >> 23) - 127;
    return e == 128 ? 0 : e < -112 ? -112 : e;
}

// ---- the rows ------------------------------------------------------------------------
// What decides whether a row is counted, loaded at once (of a teacher's entries the first, mostly enough).
struct RowFirst {
    int label, index;
    float logit, s, hard, soft;
};
static __device__ __forceinline__ RowFirst row_first(const HeadArgs& a, int64_t row)
{
    RowFirst f{-1, -1, 0.0f, 0.0f, 0.0f, 0.0f};
    if (row >= a.rows) return f;
    if (a.labels) {
        f.label = fetch(a.labels + row);
    } else {
        f.index = fetch(a.index + row * a.ldt);
        f.logit = teacher_logit(a, row, 0);
    }
    if (a.backward) row_factors(a, row, f.s, f.hard, f.soft);
    return f;
}
// Whether a row is counted, and the exponent of its gradient's scale (-1000: none that is finite).
static __device__ __forceinline__ bool row_counts(const HeadArgs& a, int64_t row, const RowFirst& f, int& e)
{
    e = -1000;
    if (row >= a.rows) return false;
    if (a.labels) {
        if (f.label < 0) return false;
    } else if (f.index < 0 || f.logit == __uint_as_float(0xFF800000u)) {     // rows of which the teacher has kept something
        int k = 1;
        while (k < a.top && !has_entry(a, row, k)) k++;
        if (k >= a.top) return false;
    }
    if (!a.backward) return true;
    const float b = factors_bound(a, f.s, f.hard, f.soft);
    if (b == 0.0f || common_factor(a) == 0.0f) return false;
    if (b - b == 0.0f) e = bound_exponent(b);
    return true;
}

// Which rows are counted, and their gradients' largest power of two: a block takes a chunk of
// 1024 rows.  (With one chunk k_head_pack's blocks find this out themselves.)
static __global__ void __launch_bounds__(1024) k_head_rows(const __grid_constant__ HeadArgs a)
{
    __shared__ int32_t counts[32], tops[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * ZERO_HD_CHUNK + threadIdx.x;
    let_next_begin();
    after_previous();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.st->err = 0;
        a.st->ticket = 0;
    }
    int e;
    const bool in = row_counts(a, row, row_first(a, row), e);
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, in);
    e = __reduce_max_sync(0xFFFFFFFFu, e);
    if (lane == 0) {
        a.mask[row >> 5] = m;
        counts[warp] = __popc(m);
        tops[warp] = e;
    }
    __syncthreads();
    if (warp == 0) {
        const int c = __reduce_add_sync(0xFFFFFFFFu, counts[lane]), t = __reduce_max_sync(0xFFFFFFFFu, tops[lane]);
        if (lane == 0) {
            a.count[blockIdx.x] = c;
            a.most[blockIdx.x] = t;
        }
    }
}

// The targets of a row, the teacher's entries and the label, by columns (equal ones in their order; those that
// are none come last).  Whether targets are heavy goes by their column's weight, and the last of them stands for it.  A
// warp's; `cols` and `vals` are its shared memory, cols filled up with none to a multiple of 4.
static __device__ __forceinline__ void put_targets(const HeadArgs& a, int64_t row, const int* cols, const float* vals)
{
    const int n = a.slots, lane = threadIdx.x & 31;
    float total = 0.0f;
    for (int e = lane; e < n; e += 32) total += fabsf(vals[e]);
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    int heavies = 0;
    for (int e = lane; e < n + lane; e += 32) {              // all lanes the same number of turns
        bool heavy = false;
        int rank = 0, same = 0, col = ZERO_HD_NONE;
        if (e < n) {
            col = cols[e];
            for (int f = 0; f < n; f += 4) {
                const int4 q = *reinterpret_cast<const int4*>(cols + f);
                rank += (q.x < col || (q.x == col && f < e)) + (q.y < col || (q.y == col && f + 1 < e)) +
                        (q.z < col || (q.z == col && f + 2 < e)) + (q.w < col || (q.w == col && f + 3 < e));
                same += (q.x == col) + (q.y == col) + (q.z == col) + (q.w == col);
            }
            if (a.backward && col != ZERO_HD_NONE) {
                float weight = vals[e];
                bool last = true;
                if (same > 1)
                    for (int f = 0; f < n; f++)
                        if (f != e && cols[f] == col) {
                            weight += vals[f];
                            last = last && f < e;
                        }
                heavy = last && fabsf(weight) >= total * (1.0f / ZERO_HD_HEAVY);
            }
        }
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, heavy);
        const int at = heavies + __popc(m & ((1u << lane) - 1));
        heavy = heavy && at < ZERO_HD_HEAVY;
        if (heavy) a.heavy[row * ZERO_HD_HEAVY + at] = {col, 0.0f};
        if (e < n) a.target[row * n + rank] = {heavy ? col | (at + 1) << 24 : col, vals[e]};
        heavies += __popc(m);
    }
    if (a.backward && lane == 0) a.heavies[row] = heavies < ZERO_HD_HEAVY ? heavies : ZERO_HD_HEAVY;
}

// The `wide` columns of a row of `cols` as 16-byte vectors, zeros past its end, whatever the row's
// alignment: put(o, v) gets vector o.  A warp's.  Rows that are not aligned are read in aligned vectors, each
// lane's shifted together with the next lane's (of the vectors that reach over the row's ends only the
// row's elements are read): 49 MB of 771 columns in 19 us, 24 element by element (reading and writing them at the
// rate of HBM takes 15).
template <class Put>
static __device__ __forceinline__ void row_vectors(const uint16_t* from, int cols, int wide, Put put)
{
    const int lane = threadIdx.x & 31, s = (int)(reinterpret_cast<uintptr_t>(from) & 15) >> 1;
    // elements [8 g - s, 8 g - s + 8) of the row: an aligned vector
    auto load = [&](int g) {
        uint32_t w[4] = {0, 0, 0, 0};
        const int e = 8 * g - s;
        if (e >= 0 && e + 8 <= cols) return fetch(reinterpret_cast<const uint4*>(from + e));
        if (e < cols) {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (e + i >= 0 && e + i < cols) w[i / 2] |= (uint32_t)fetch(from + e + i) << 16 * (i & 1);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    if (s == 0) {
#pragma unroll 4
        for (int o = lane; o < wide / 8; o += 32) put(o, load(o));
        return;
    }
#pragma unroll 4
    for (int first = 0; first < wide / 8; first += 31) {
        const uint4 q = load(first + lane);
        uint32_t w[8] = {q.x, q.y, q.z, q.w, __shfl_down_sync(0xFFFFFFFFu, q.x, 1), __shfl_down_sync(0xFFFFFFFFu, q.y, 1),
                         __shfl_down_sync(0xFFFFFFFFu, q.z, 1), __shfl_down_sync(0xFFFFFFFFu, q.w, 1)};
        if (s & 4) {
#pragma unroll
            for (int i = 0; i < 6; i++) w[i] = w[i + 2];
        }
        if (s & 2) {
#pragma unroll
            for (int i = 0; i < 5; i++) w[i] = w[i + 1];
        }
        if (s & 1) {
#pragma unroll
            for (int i = 0; i < 4; i++) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        }
        if (lane < 31 && first + lane < wide / 8) put(first + lane, make_uint4(w[0], w[1], w[2], w[3]));
    }
}

// Packs the counted rows and what belongs to them: a warp a row, eight rows a block; rows past the
// last counted one are zeros up to a whole tile.  8192 rows of 4096: 26 us, at HBM's rate 20; a few rows 5 us, the
// latency of the label (for 777 rows of a teacher without labels 12 us until all that decides was loaded at once), of
// what depends on it, and of the row.
template <int DT>
__global__ void __launch_bounds__(256) k_head_pack(const __grid_constant__ HeadArgs a)
{
    extern __shared__ __align__(16) int32_t entries_of[];   // a warp's targets: columns, weights
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 8 + warp;
    const int chunks = (int)((a.rows + ZERO_HD_CHUNK - 1) / ZERO_HD_CHUNK);
    int before = 0, all = 0, top = -1000;
    __shared__ uint32_t masks[32];                          // the row's chunk's mask
    __shared__ int32_t tops[8];
    let_next_begin();
    after_previous();
    if (chunks == 1) {
        RowFirst f[4];
#pragma unroll
        for (int i = 0; i < 4; i++) f[i] = row_first(a, i * 256 + threadIdx.x);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            int e;
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, row_counts(a, i * 256 + threadIdx.x, f[i], e));
            top = max(top, __reduce_max_sync(0xFFFFFFFFu, e));
            if (lane == 0) masks[i * 8 + warp] = m;
        }
        if (lane == 0) tops[warp] = top;
        __syncthreads();
        all = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)__popc(masks[lane]));
        top = __reduce_max_sync(0xFFFFFFFFu, tops[lane & 7]);
        if (row >= a.rows) before = all;
    } else {
        const int mine = (int)(row < a.rows ? row >> 10 : chunks);
        for (int c = lane; c < chunks; c += 32) {
            const int n = a.count[c];
            all += n;
            if (c < mine) before += n;
            top = max(top, a.most[c]);
        }
        before = __reduce_add_sync(0xFFFFFFFFu, before);
        all = __reduce_add_sync(0xFFFFFFFFu, all);
        top = __reduce_max_sync(0xFFFFFFFFu, top);
    }
    if (top == -1000) top = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.st->rows = all;
        a.st->top = top;
        a.st->lift = 0;
        if (chunks == 1) {
            a.st->err = 0;
            a.st->ticket = 0;
        }
    }
    int64_t at;                                             // packed row
    bool counted = false;
    if (row < a.rows) {
        const int in = (int)(row & 1023), word = in >> 5;
        const uint32_t w = lane > word ? 0 : chunks == 1 ? masks[lane] : a.mask[(row >> 10 << 5) + lane];
        const uint32_t below = lane < word ? w : w & ((1u << (in & 31)) - 1);
        at = before + __reduce_add_sync(0xFFFFFFFFu, (uint32_t)__popc(below));
        counted = __shfl_sync(0xFFFFFFFFu, w, word) >> (in & 31) & 1;
        if (!counted) {
            if (a.backward) {
                if (a.dx)
                    for (int c = lane; c < a.cols; c += 32) a.dx[row * a.lddx + c] = 0;
            } else if (lane == 0) {
                a.loss[row] = 0.0f;
                if (a.index) a.lse[2 * row] = a.lse[2 * row + 1] = 0.0f;
                else a.lse[row] = 0.0f;
            }
            return;
        }
    } else {
        at = all + (row - a.rows);
        const int64_t end = all > 0 ? ((int64_t)all + 255) / 256 * 256 : 256;
        if (at >= end) return;
    }
    // the row
    float up = 1.0f;
    int e = 0;
    [[maybe_unused]] bool finite = true;
    float s = 0.0f, hard = 0.0f, soft = 0.0f;
    if (counted && a.backward) {
        row_factors(a, row, s, hard, soft);
        const float b = factors_bound(a, s, hard, soft);
        e = bound_exponent(b);
        finite = b - b == 0.0f;
        up = finite ? power2(e - top) : 1.0f;
        if (!finite) e = top;
    }
    uint32_t large = 0;                                     // (fp16) largest |x| of even and odd columns
    row_vectors(a.x + (counted ? row : 0) * a.ldx, counted ? a.cols : 0, a.wide, [&](int o, uint4 q) {
        reinterpret_cast<uint4*>(a.xp + at * a.wide)[o] = q;
        if (a.xs == a.xp) return;
        const uint32_t m = 0x7FFF7FFFu;
        if (DT == 0) {
            large = __vmaxu2(large, __vmaxu2(__vmaxu2(q.x & m, q.y & m), __vmaxu2(q.z & m, q.w & m)));
        } else {
            uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float lo, hi;
                widen2<DT>(w[i], lo, hi);
                w[i] = narrow2<DT>(lo * up, hi * up);
            }
            reinterpret_cast<uint4*>(a.xs + at * a.wide)[o] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    });
    if (!counted) return;
    if (DT == 0 && a.xs != a.xp) {
        // (a row that is 0 decides nothing, nor does one without a finite scale, whose dw is not finite either)
        large = __reduce_max_sync(0xFFFFFFFFu, max(large & 0xFFFFu, large >> 16));
        const int most = (int)(__float_as_uint(widen1<0>((uint16_t)large)) >> 23) - 127;
        if (lane == 0) a.reach[at] = large == 0 || !finite ? ZERO_HD_NO_REACH : e + min(most, 15);
    }
    // its targets and coefficients
    const int room = (a.slots + 3) & ~3;
    int* cols = entries_of + warp * 2 * room;
    float* vals = reinterpret_cast<float*>(cols + room);
    const float nan = __uint_as_float(0x7FC00000u);
    bool bad = false;
    float constant = 0.0f, share = 0.0f;
    const float fit = a.backward ? power2(ZERO_HD_SCALE - e) : 1.0f;
    if (a.index) {
        const float low = __uint_as_float(0xFF800000u);
        float m = low, sum = 0.0f, cross = 0.0f;
        for (int k = lane; k < a.top; k += 32) {
            const int col = fetch(a.index + row * a.ldt + k);
            float t = teacher_logit(a, row, k);
            if (col < 0) t = low;                           // (a NaN there is not read)
            const bool past = t != low && col >= a.vocab;
            cols[k] = t == low ? ZERO_HD_NONE : past ? 0 : col;
            vals[k] = t;
            bad = bad || past;
            m = fmaxf(m, t);
            if (t != low) share = 1.0f;
        }
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        share = __any_sync(0xFFFFFFFFu, share > 0.0f) ? 1.0f : 0.0f;
        for (int k = lane; k < a.top; k += 32) {
            float q = 0.0f;
            if (cols[k] != ZERO_HD_NONE) {
                const float t = (vals[k] - m) / a.temperature;
                q = expf(t);
                sum += q;
                cross += q > 0.0f ? q * t : q;              // (a NaN stays one)
            }
            vals[k] = q;
        }
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            cross += __shfl_xor_sync(0xFFFFFFFFu, cross, o);
        }
        const float each = (a.backward ? s * fit : 1.0f) * a.soft * a.temperature;
        // (none of them: sum is 0)
        for (int k = lane; k < a.top; k += 32) vals[k] = cols[k] == ZERO_HD_NONE ? 0.0f : vals[k] / sum * each;
        // sum q log q = sum q t - log(sum)
        if (share > 0.0f) constant = a.soft * a.temperature * a.temperature * (cross / sum - logf(sum));
        else soft = 0.0f;
    }
    if (a.labels && lane == 0) {
        const int label = fetch(a.labels + row);
        bad = bad || label >= a.vocab;
        cols[a.slots - 1] = label < a.vocab ? label : 0;
        vals[a.slots - 1] = (a.backward ? s * fit : 1.0f) * a.hard;
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane < room - a.slots) cols[a.slots + lane] = ZERO_HD_NONE;
    __syncwarp();
    put_targets(a, at, cols, vals);
    if (lane == 0) {
        a.map[at] = (int32_t)row;
        HeadRow h;
        if (a.backward) {
            a.exponent[at] = e;
            const float log2e = 1.4426950408889634f;
            const float soft_l = a.index ? fetch(a.kept + 2 * row) : 0.0f;
            const float hard_l = !a.labels ? 0.0f : a.index ? fetch(a.kept + 2 * row + 1) : fetch(a.kept + row);
            h.c1 = hard * fit;
            h.l1 = hard_l * log2e;
            h.c2 = soft * fit;
            h.l2 = soft_l * log2e;
            if (!a.two) {                                    // one softmax
                h.c1 += h.c2;
                if (!a.labels) h.l1 = h.l2;
            }
            if (bad) h.c1 = nan;
        } else {
            h.c1 = bad ? nan : constant;
            h.c2 = share;
            h.l1 = h.l2 = 0.0f;
        }
        a.info[at] = h;
    }
}

// The packed rows for dw of fp16 gradients whose rows have scales of their own: a row times its power of two over the
// largest row's, as k_head_pack multiplies bf16's, would fall below fp16's normal numbers (2^-14) for a row of small
// weight.  All are lifted by one power of two, so that the largest element ends in [2^15, 2^16): rounding a row then
// moves its part of dw by at most 2^-39 of the largest |g x| of all rows, two of fp16's smallest numbers where that is
// its largest.  Every block finds the power by itself; a warp a row.  A launch of its own, since the power needs all
// packed rows: 64 x 256 x 1000 with row weights 27 -> 30 us, 1023 x 771 x 32003 182 -> 186.
static __global__ void __launch_bounds__(256) k_head_lift(const __grid_constant__ HeadArgs a)
{
    __shared__ int32_t tops[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    let_next_begin();
    after_previous();
    const int counted = a.st->rows, top = a.st->top;
    int reach = ZERO_HD_NO_REACH;
    for (int r = threadIdx.x; r < counted; r += 256) reach = max(reach, a.reach[r]);
    reach = __reduce_max_sync(0xFFFFFFFFu, reach);
    if (lane == 0) tops[warp] = reach;
    __syncthreads();
    reach = __reduce_max_sync(0xFFFFFFFFu, tops[lane & 7]);
    const int lift = reach == ZERO_HD_NO_REACH ? 0 : 15 - (reach - top);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.st->lift = lift;
    const int end = counted > 0 ? (int)head_up(counted, ZERO_HD_TILE) * ZERO_HD_TILE : ZERO_HD_TILE;
    for (int64_t r = (int64_t)blockIdx.x * 8 + warp; r < end; r += (int64_t)gridDim.x * 8) {
        // (above 2^15 times 2^24 only a row of zeros is lifted)
        const int k = r < counted ? a.exponent[r] - top + lift : 0;
        const float up = power2(k < 127 ? k : 127);
#pragma unroll 4
        for (int o = lane; o < a.wide / 8; o += 32) {
            const uint4 q = reinterpret_cast<const uint4*>(a.xp + r * a.wide)[o];
            uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float lo, hi;
                widen2<0>(w[i], lo, hi);
                w[i] = narrow2<0>(lo * up, hi * up);
            }
            reinterpret_cast<uint4*>(a.xs + r * a.wide)[o] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Rows of the weights that are not aligned to 16 bytes, a piece of them, to rows that are.  Eight blocks an SM, two
// rounds of them, in 32 registers, which spills 28 bytes (five in 48 registers: 3 us more for 49 MB).
static __global__ void __launch_bounds__(256, 8) k_head_weights(const __grid_constant__ HeadArgs a)
{
    let_next_begin();
    after_previous();
    for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < a.count_v; r += (int64_t)gridDim.x * 8)
        row_vectors(a.w + (a.v0 + r) * a.ldw, a.cols, a.wide,
                    [&](int o, uint4 q) { reinterpret_cast<uint4*>(a.wp + r * a.wide)[o] = q; });
}

// ---- the pair's machinery ------------------------------------------------------------
// A box into this SM's shared memory whose bytes count on the first SM's barrier.
static __device__ __forceinline__ void box_for_first(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "{\n .reg .b32 r;\n mapa.shared::cluster.u32 r, %4, 0;\n"
        " cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [r];\n}"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
// Operand in shared memory with the contracted axis contiguous, 128-byte swizzle: rows of 64
// elements, groups of eight rows 1024 bytes apart.
static __device__ __forceinline__ uint64_t operand_rows(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
static __device__ __forceinline__ void read16(uint32_t at, float (&v)[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at) : "memory");
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}
struct HeadShared {
    uint64_t full[ZERO_HD_STAGES];          // (first SM's) both SMs' operands of a stage have come
    uint64_t empty[ZERO_HD_STAGES];         // its products are done
    uint64_t sum_full[2], sum_empty[2];     // accumulators
    uint64_t drain;
    uint32_t tmem;
    int dead;
    uint32_t issued;                        // stages this SM has loaded, and the bytes of the last ones
    uint32_t bytes[ZERO_HD_STAGES];
    uint32_t inputs;                        // (products) a pair's segments of dx
    HeadShape shape, shape_w;
};

// A word of the second SM's shared memory, at this SM's address of it.
static __device__ __forceinline__ uint32_t of_second(uint32_t at)
{
    uint32_t r;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, 1;\n ld.shared::cluster.u32 %0, [a];\n}" : "=r"(r) : "r"(at) : "memory");
    return r;
}
static __device__ __forceinline__ bool head_wait(uint32_t bar, uint32_t parity, volatile int* dead, int32_t* err)
{
    return pair_wait<ZERO_HD_WAIT_LIMIT>(bar, parity, dead, err);
}

// ---- output --------------------------------------------------------------------------
// N (a multiple of 8) columns from j of a row at `to`, in 16 bits.
template <int DT, int N>
static __device__ __forceinline__ void put_vectors(uint16_t* to, float (&v)[N], bool add)
{
    uint4* o = reinterpret_cast<uint4*>(to);
#pragma unroll
    for (int c = 0; c < N; c += 8) {
        if (add) {
            const uint4 p = o[c / 8];
            const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float lo, hi;
                widen2<DT>(w[e], lo, hi);
                v[c + 2 * e] += lo;
                v[c + 2 * e + 1] += hi;
            }
        }
        o[c / 8] = make_uint4(narrow2<DT>(v[c], v[c + 1]), narrow2<DT>(v[c + 2], v[c + 3]), narrow2<DT>(v[c + 4], v[c + 5]),
                              narrow2<DT>(v[c + 6], v[c + 7]));
    }
}

// Where row i (packed, or of the piece) of an output lies and what its sums are multiplied by;
// null if there is none.
static __device__ __forceinline__ uint16_t* out_row(const HeadArgs& a, bool input, int64_t i, int counted, int top, float common,
                                                    float& factor)
{
    if (input) {
        if (i >= counted) return nullptr;
        factor = power2(a.exponent[i] - ZERO_HD_SCALE) * common;
        return a.dx + a.map[i] * a.lddx;
    }
    if (i >= a.count_v) return nullptr;
    // (in two steps: one alone may lie below fp32's normal numbers)
    const int k = top - ZERO_HD_SCALE, half = k / 2;
    factor = power2(half) * common * power2(k - half);
    return a.dw + (a.v0 + i) * a.lddw;
}

// N columns from j of a lane's own row.
template <int DT, int N>
static __device__ __forceinline__ void put_row(const HeadArgs& a, bool input, uint16_t* to, float factor, int j, float (&v)[N])
{
    if (!to || j >= a.cols) return;
    const bool add = !input && a.accumulate;
#pragma unroll
    for (int c = 0; c < N; c++) v[c] *= factor;
    if ((input ? a.vec_x : a.vec_w) && j + N <= a.cols) {
        put_vectors<DT, N>(to + j, v, add);
        return;
    }
#pragma unroll
    for (int c = 0; c < N; c++)
        if (j + c < a.cols) {
            float x = v[c];
            if (add) x += widen1<DT>(to[j + c]);
            to[j + c] = narrow1<DT>(x);
        }
}

// Where 16-byte word q of a lane's row lies in the warp's 32 rows of 64 bytes: at q ^ (row >> 1 & 3), TMA's
// 64-byte swizzle, in which lanes that each take a row meet all banks.
static __device__ __forceinline__ uint32_t word_of(uint32_t stage, int row, int q) { return stage + row * 64 + ((q ^ (row >> 1 & 3)) << 4); }
// What rounding dz cut off at a row's heavy targets, which is most of what dx would be off by (a row's dz
// is often little else than a label's p - 1): the number of them, and their addition, times their weights, to
// N columns from j of dx's sums.
struct HeadCuts {
    int n = 0;
    int4 two, four;
    __device__ __forceinline__ void begin(const HeadArgs& a, int64_t row)
    {
        n = a.heavies[row];
        two = reinterpret_cast<const int4*>(a.heavy + row * ZERO_HD_HEAVY)[0];
        four = reinterpret_cast<const int4*>(a.heavy + row * ZERO_HD_HEAVY)[1];
    }
    template <int DT, int N>
    __device__ __forceinline__ void add_one(const HeadArgs& a, int2 h, int j, float (&v)[N]) const
    {
        const float cut = __int_as_float(h.y);
        const uint16_t* w = a.w + h.x * a.ldw + j;
        if (a.vec && j + N <= a.cols) {
#pragma unroll
            for (int c = 0; c < N; c += 8) {
                const uint4 q = fetch(reinterpret_cast<const uint4*>(w + c));
                const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    float lo, hi;
                    widen2<DT>(u[e], lo, hi);
                    v[c + 2 * e] = __fmaf_rn(cut, lo, v[c + 2 * e]);
                    v[c + 2 * e + 1] = __fmaf_rn(cut, hi, v[c + 2 * e + 1]);
                }
            }
        } else {
#pragma unroll
            for (int c = 0; c < N; c++)
                if (j + c < a.cols) v[c] = __fmaf_rn(cut, widen1<DT>(fetch(w + c)), v[c]);
        }
    }
    template <int DT, int N>
    __device__ __forceinline__ void add(const HeadArgs& a, int j, float (&v)[N]) const
    {
        if (n > 0) add_one<DT>(a, make_int2(two.x, two.y), j, v);
        if (n > 1) add_one<DT>(a, make_int2(two.z, two.w), j, v);
        if (n > 2) add_one<DT>(a, make_int2(four.x, four.y), j, v);
        if (n > 3) add_one<DT>(a, make_int2(four.z, four.w), j, v);
    }
};

// 32 columns of a lane's row in 16 bits.
template <int DT>
static __device__ __forceinline__ void lay_row(uint32_t stage, const float (&v)[32])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < 4; q++)
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(word_of(stage, lane, q)),
                     "r"(narrow2<DT>(v[8 * q], v[8 * q + 1])), "r"(narrow2<DT>(v[8 * q + 2], v[8 * q + 3])),
                     "r"(narrow2<DT>(v[8 * q + 4], v[8 * q + 5])), "r"(narrow2<DT>(v[8 * q + 6], v[8 * q + 7])) : "memory");
}
// The warp's rows on their way to column x, row y of a matrix; and the wait until they have been read.
static __device__ __forceinline__ void send_rows(uint32_t stage, const CUtensorMap* map, int x, int y)
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n"
                     "cp.async.bulk.commit_group;" ::"l"(map), "r"(x), "r"(y), "r"(stage) : "memory");
}
static __device__ __forceinline__ void rows_sent()
{
    if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}

// put_row() for rows that are not aligned to vectors: 32 columns of the warp's rows through shared
// memory, so that an access of the warp is a run of a row and not an element of each of 32 rows.
template <int DT>
static __device__ __forceinline__ void put_rows(const HeadArgs& a, bool input, uint16_t* to, float factor, int j, float (&v)[32],
                                                uint32_t stage)
{
    const int lane = threadIdx.x & 31;
    if (j >= a.cols) return;                                 // all lanes
    const uint64_t mine = reinterpret_cast<uint64_t>(to);
#pragma unroll
    for (int e = 0; e < 32; e++) v[e] *= factor;
    if (!input && a.accumulate) {
#pragma unroll 8
        for (int r = 0; r < 32; r++) {
            const uint16_t* g = reinterpret_cast<const uint16_t*>(__shfl_sync(0xFFFFFFFFu, mine, r));
            const uint16_t x = g && j + lane < a.cols ? g[j + lane] : 0;
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(word_of(stage, r, lane >> 3) + (lane & 7) * 2), "h"(x) : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; q++) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(word_of(stage, lane, q)));
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float lo, hi;
                widen2<DT>(w[e], lo, hi);
                v[8 * q + 2 * e] += lo;
                v[8 * q + 2 * e + 1] += hi;
            }
        }
    }
    lay_row<DT>(stage, v);
    __syncwarp();
#pragma unroll 16
    for (int r = 0; r < 32; r++) {
        uint16_t* g = reinterpret_cast<uint16_t*>(__shfl_sync(0xFFFFFFFFu, mine, r));
        uint16_t x;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(word_of(stage, r, lane >> 3) + (lane & 7) * 2));
        if (g && j + lane < a.cols) g[j + lane] = x;
    }
    __syncwarp();
}

// A lane's next target of its row from column `from` on; AHEAD: the one after it is loaded ahead.
template <bool AHEAD>
struct HeadGoal {
    const HeadTarget* at;
    int next, from, heavy;                                  // heavy: this one's place, or 0
    HeadTarget now, then;                                   // then as it is stored; now's column counted from `from`
    __device__ __forceinline__ HeadTarget load(const HeadArgs& a, int e) const
    {
        if (e >= a.slots) return {ZERO_HD_NONE, 0.0f};
        const int2 q = reinterpret_cast<const int2*>(at)[e];
        return {q.x, __int_as_float(q.y)};
    }
    __device__ __forceinline__ int place(int column) const { return column == ZERO_HD_NONE ? column : (column & 0xFFFFFF) - from; }
    __device__ __forceinline__ void take(const HeadTarget& t)
    {
        heavy = t.column == ZERO_HD_NONE ? 0 : t.column >> 24;
        now = {place(t.column), t.weight};
    }
    __device__ __forceinline__ void begin(const HeadArgs& a, int64_t row, int c)
    {
        at = a.target + row * a.slots;
        from = c;
        int hi = a.slots;
        next = 0;
        while (next < hi) {                                  // the first whose column is not below
            const int mid = (next + hi) >> 1;
            if ((at[mid].column & 0xFFFFFF) < c) next = mid + 1;
            else hi = mid;
        }
        take(load(a, next));
        if (AHEAD) then = load(a, next + 1);
    }
    __device__ __forceinline__ void none() { now = {ZERO_HD_NONE, 0.0f}; }
    __device__ __forceinline__ void step(const HeadArgs& a)
    {
        next++;
        take(AHEAD ? then : load(a, next));
        if (AHEAD) then = load(a, next + 1);
    }
};

// ---- the products --------------------------------------------------------------------
// A pair's two SMs hold 128 rows each of a tile and half of the other operand; one thread loads an SM's
// halves of a stage by TMA (both SMs' bytes count on the first one's barrier), one thread of the pair issues
// the products, and sixteen warps of each SM read the two accumulators in turn:
//   logits: a thread its row's 64 columns, in registers: runs added, targets picked out, maximum, sum of
//     exponentials; the four column groups meet in shared memory and leave one pair of numbers a row.
//   gradient: dz of 32 columns at a time, less the targets' weights, out by TMA through 2 KB a warp (written
//     by the lanes that have the rows, 32 sectors an access, a piece of 6144 x 25344 x 1600 took 287 us, now 246).
//   products: dw out the same way (rows that are not aligned, dx and sums that are added: by the warp or its
//     lanes), parts of cut tiles and dx's sums so far in fp32, four columns of 32 rows a run.
// map_a, map_b: the operands of the logits or of dx; map_c, map_d: of dw; map_o: where the pass's
// output goes by TMA (dz; dw where its rows are aligned).
template <int DT, int PASS, bool TWO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(ZERO_HD_THREADS, 1)
    k_head(const __grid_constant__ HeadArgs a, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
           const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_d, const __grid_constant__ CUtensorMap map_o)
{
    constexpr int GROUPS = head_groups(PASS), WIDE = head_columns(PASS);                // columns of a writer
    extern __shared__ unsigned char raw[];
    __shared__ HeadShared sh;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), pair = blockIdx.x >> 1;
    volatile int* dead = &sh.dead;
    int32_t* err = &a.st->err;
    if (threadIdx.x == 0) {
        for (int s = 0; s < ZERO_HD_STAGES; s++) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), 1);
        }
        for (int s = 0; s < 2; s++) {
            mbar_init(smem_u32(&sh.sum_full[s]), 1);
            mbar_init(smem_u32(&sh.sum_empty[s]), 2 * ZERO_HD_WRITERS / GROUPS);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        sh.dead = 0;
        sh.issued = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n"
                     "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *(volatile uint32_t*)&sh.tmem;
    let_next_begin();
    // kept in shared memory: the writers' registers hold sums.  Of all rows before their number is known, and
    // once more where not all count
    auto divide = [&](int rows) {
        sh.shape = head_shape<PASS == HEAD_PRODUCTS ? HEAD_INPUT : PASS>(a, rows);
        if (PASS == HEAD_PRODUCTS) {
            sh.shape_w = head_shape<HEAD_WEIGHT>(a, rows);
            sh.inputs = head_inputs(a, sh.shape, pair);
        }
    };
    if (threadIdx.x == 0) divide((int)a.rows);
    after_previous();
    const int counted = a.st->rows;
    if (threadIdx.x == 0 && counted != (int)a.rows) divide(counted);
    __syncthreads();
    const HeadShape &shape = sh.shape, &shape_w = sh.shape_w;
    const uint32_t& inputs = sh.inputs;
    HeadSegment g{};
    // the segment's tile, and whether it is one of dw
    auto place = [&](uint32_t& ti, uint32_t& tj) {
        const bool w = PASS == HEAD_PRODUCTS && !g.input;
        head_place(head_band<PASS>(a), w ? shape_w : shape, g.tile, ti, tj);
        return w;
    };

    if (warp == 0) {
        // ---- loads ----
        if (elected()) {
            uint32_t n = 0, s = 0, ph = 0;
            bool ok = true;
            for (int i = 0; ok && head_next<PASS>(a, shape, shape_w, inputs, pair, i, g); i++) {
                uint32_t ti, tj;
                const bool dw = place(ti, tj);
                const int half = head_width<PASS>(a, tj) / 2;
                const int ra = (int)ti * ZERO_HD_TILE + rank * 128, rb = (int)tj * ZERO_HD_TILE + rank * half;
                const uint32_t bytes = 2 * (ZERO_HD_SIDE + half * 128);
                for (int t = g.s0; t < g.s1; t++, n++) {
                    if (n >= ZERO_HD_STAGES && !head_wait(smem_u32(&sh.empty[s]), ph ^ 1u, dead, err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_u32(&sh.full[s]), at = base + s * 2 * ZERO_HD_SIDE, bt = at + ZERO_HD_SIDE;
                    const int k = t * ZERO_HD_STEP;
                    if (rank == 0) mbar_expect_tx(bar, bytes);
                    else sh.bytes[s] = bytes / 2;
                    if (dw) {
                        box_for_first(at, &map_c, ra, k, bar);
                        box_for_first(at + 8192, &map_c, ra + 64, k, bar);
                        box_for_first(bt, &map_d, rb, k, bar);
                        if (half > 64) box_for_first(bt + 8192, &map_d, rb + 64, k, bar);
                    } else {
                        box_for_first(at, &map_a, k, ra, bar);
                        if (PASS == HEAD_PRODUCTS) {
                            box_for_first(bt, &map_b, rb, a.wy + k, bar);
                            if (half > 64) box_for_first(bt + 8192, &map_b, rb + 64, a.wy + k, bar);
                        } else {
                            box_for_first(bt, &map_b, k, a.wy + rb, bar);
                        }
                    }
                    if (++s == ZERO_HD_STAGES) { s = 0; ph ^= 1u; }
                }
            }
            sh.issued = n;
            // before this SM's shared memory is given back: both SMs' copies have landed (the
            // first SM knows), and the last products are done
            for (uint32_t q = n > ZERO_HD_STAGES ? n - ZERO_HD_STAGES : 0; q < n; q++) {
                if (rank == 0)
                    for (uint32_t it = 0; it < ZERO_TMA_WAIT_LIMIT &&
                                          !mbar_try_wait(smem_u32(&sh.full[q % ZERO_HD_STAGES]), q / ZERO_HD_STAGES & 1); it++) {
                    }
                if (!*dead) head_wait(smem_u32(&sh.empty[q % ZERO_HD_STAGES]), q / ZERO_HD_STAGES & 1, dead, err);
            }
        }
    } else if (warp == 1) {
        // ---- products (the first SM's thread, for both) ----
        if (rank == 0 && elected()) {
            // fp32 sums of fp16/bf16 operands, 256 x width; the contracted axis is strided in w and x of
            // dx and dw and in dz of dw
            const uint32_t kind = 1u << 4 | (DT == 1 ? 1u << 7 | 1u << 10 : 0u) | (PASS == HEAD_PRODUCTS ? 1u << 16 : 0u) |
                                  (uint32_t)(ZERO_HD_TILE >> 4) << 24;
            constexpr uint32_t ROWS = 32 >> 4, STRIDED = 2048 >> 4, STEP_B = PASS == HEAD_PRODUCTS ? STRIDED : ROWS;
            uint32_t s = 0, ph = 0;
            bool ok = true;
            int i = 0;
            for (; ok && head_next<PASS>(a, shape, shape_w, inputs, pair, i, g); i++) {
                const int acc = i & 1;
                if (i >= 2 && !head_wait(smem_u32(&sh.sum_empty[acc]), (uint32_t)((i >> 1) - 1) & 1u, dead, err)) {
                    ok = false;
                    break;
                }
                uint32_t ti, tj;
                const bool dw = place(ti, tj);
                const uint32_t what = kind | (dw ? 1u << 15 : 0u) | (uint32_t)(head_width<PASS>(a, tj) >> 3) << 17;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int t = g.s0; t < g.s1; t++) {
                    if (!head_wait(smem_u32(&sh.full[s]), ph, dead, err)) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t at = base + s * 2 * ZERO_HD_SIDE, bt = at + ZERO_HD_SIDE;
                    const uint64_t da = dw ? operand(at) : operand_rows(at), db = PASS == HEAD_PRODUCTS ? operand(bt) : operand_rows(bt);
                    const uint32_t step_a = dw ? STRIDED : ROWS;
#pragma unroll
                    for (int q = 0; q < ZERO_HD_STEP / 16; q++)
                        product(tmem + acc * ZERO_HD_TILE, da + q * step_a, db + q * STEP_B, what, t > g.s0 || q > 0);
                    commit_both(smem_u32(&sh.empty[s]));
                    if (++s == ZERO_HD_STAGES) { s = 0; ph ^= 1u; }
                }
                if (ok) commit_both(smem_u32(&sh.sum_full[acc]));
            }
            // the other SM's last arrivals are here before this SM can exit
            for (int q = i > 2 ? i - 2 : 0; ok && q < i; q++)
                ok = head_wait(smem_u32(&sh.sum_empty[q & 1]), (uint32_t)(q >> 1) & 1u, dead, err);
            if (*dead) {                                     // let the products in flight finish
                commit_both(smem_u32(&sh.drain), 1);
                for (uint32_t it = 0; it < ZERO_TMA_WAIT_LIMIT && !mbar_try_wait(smem_u32(&sh.drain), 0); it++) {
                }
            }
        }
    } else if (warp >= 4) {
        // ---- output: warp w reads rows 32 (w mod 4) + lane of this SM's half, WIDE columns ----
        const int quad = warp & 3, side = ((warp - 4) >> 2) % (4 / GROUPS), group = (warp - 4) / (ZERO_HD_WRITERS / GROUPS);
        const float nan = __uint_as_float(0x7FC00000u), low = __uint_as_float(0xFF800000u);
        [[maybe_unused]] const uint32_t stage = base + ZERO_HD_STAGES * 2 * ZERO_HD_SIDE + (warp - 4) * ZERO_HD_ROWS;
        [[maybe_unused]] const int top = a.st->top - a.st->lift;
        [[maybe_unused]] const float common = PASS == HEAD_PRODUCTS && counted > 0 ? common_factor(a) : 0.0f;
        [[maybe_unused]] float z[PASS == HEAD_LOGITS ? WIDE : 1];
        // maxima and sums of a tile's column groups but the first: [group][which][lane] of this quad
        [[maybe_unused]] const auto merge = reinterpret_cast<float(*)[3][32]>(
            raw + (base - smem_u32(raw)) + ZERO_HD_STAGES * 2 * ZERO_HD_SIDE + quad * (9 * 32 * 4));
        for (int i = group; head_next<PASS>(a, shape, shape_w, inputs, pair, i, g); i += GROUPS) {
            const int acc = i & 1;
            uint32_t ti, tj;
            const bool dw = place(ti, tj);
            const int64_t r = (int64_t)ti * ZERO_HD_TILE + rank * 128 + quad * 32 + lane;
            const uint32_t from = tmem + acc * ZERO_HD_TILE + side * WIDE + ((uint32_t)quad << 21);
            const bool live = r < counted;
            // what does not depend on the sums, while they are made
            [[maybe_unused]] const int c0 = (int)tj * ZERO_HD_TILE + side * WIDE;     // first column, of the piece
            [[maybe_unused]] const int end = a.count_v - c0;                          // columns there are from it
            [[maybe_unused]] HeadGoal<PASS == HEAD_GRADIENT> goal;
            [[maybe_unused]] HeadRow row{};
            [[maybe_unused]] uint16_t* to = nullptr;
            [[maybe_unused]] HeadCuts cuts;
            [[maybe_unused]] float factor = 0.0f;
            if (PASS <= HEAD_GRADIENT) {
                goal.none();
                if (live && g.last) {
                    if (PASS == HEAD_GRADIENT) row = a.info[r];
                    goal.begin(a, r, a.v0 + c0);
                }
            } else if (g.slot < 0 && (dw || a.last)) {
                to = out_row(a, !dw, r, counted, top, common, factor);
                if (!dw && to) cuts.begin(a, r);
            }
            const bool have = __all_sync(0xFFFFFFFFu, head_wait(smem_u32(&sh.sum_full[acc]), (uint32_t)(i >> 1) & 1u, dead, err));
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if constexpr (PASS == HEAD_LOGITS) {
                // z: the tile's sums, runs of it added in fp32
#pragma unroll
                for (int c = 0; c < WIDE; c += 16) {
                    float v[16];
                    read16(from + c, v);
#pragma unroll
                    for (int e = 0; e < 16; e++) z[c + e] = v[e] + (g.first ? 0.0f : z[c + e]);
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive_first(smem_u32(&sh.sum_empty[acc]));
                if (!g.last) continue;
                // logits of targets in these columns, every lane's next one at a time
                while (__any_sync(0xFFFFFFFFu, goal.now.column < WIDE)) {
                    float x = z[0];
#pragma unroll
                    for (int c = 1; c < WIDE; c++) x = goal.now.column == c ? z[c] : x;
                    if (goal.now.column < WIDE) {
                        a.found[r * a.slots + goal.next] = have ? x : nan;
                        goal.step(a);
                    }
                }
                if (end < WIDE) {
#pragma unroll
                    for (int c = 0; c < WIDE; c++)
                        if (c >= end) z[c] = low;
                }
                float m[4], s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int e = 0; e < 4; e++) m[e] = z[e];
#pragma unroll
                for (int c = 4; c < WIDE; c++) m[c & 3] = fmaxf(m[c & 3], z[c]);
                float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
                if (end > 0) {
                    const float b1 = -most * a.k1, b2 = -most * a.k2;
#pragma unroll
                    for (int c = 0; c < WIDE; c++) {
                        s[c & 3] += exp2_fast(__fmaf_rn(z[c], a.k1, b1));
                        if (TWO) s2[c & 3] += exp2_fast(__fmaf_rn(z[c], a.k2, b2));
                    }
                }
                float sum = (s[0] + s[1]) + (s[2] + s[3]), sum2 = (s2[0] + s2[1]) + (s2[2] + s2[3]);
                if (!have) sum = sum2 = nan;
                // the tile's column groups
                if (side > 0) {
                    merge[side - 1][0][lane] = most;
                    merge[side - 1][1][lane] = sum;
                    if (TWO) merge[side - 1][2][lane] = sum2;
                }
                asm volatile("bar.sync %0, 128;" ::"r"(1 + quad) : "memory");
                if (side == 0) {
                    float o[3], all = most;
#pragma unroll
                    for (int e = 0; e < 3; e++) {
                        o[e] = merge[e][0][lane];
                        all = fmaxf(all, o[e]);
                    }
                    sum *= exp2_fast((most - all) * a.k1);
                    if (TWO) sum2 *= exp2_fast((most - all) * a.k2);
#pragma unroll
                    for (int e = 0; e < 3; e++) {
                        sum += merge[e][1][lane] * exp2_fast((o[e] - all) * a.k1);
                        if (TWO) sum2 += merge[e][2][lane] * exp2_fast((o[e] - all) * a.k2);
                    }
                    if (live) {
                        const int64_t at = (int64_t)(a.v0 / ZERO_HD_TILE + tj) * a.npad + r;
                        a.part[at] = make_float2(all, sum);
                        if (TWO) a.part2[at] = sum2;
                    }
                }
                asm volatile("bar.sync %0, 128;" ::"r"(1 + quad) : "memory");
            } else if constexpr (PASS == HEAD_GRADIENT) {
                const int rows = counted > 0 ? (int)head_up(counted, ZERO_HD_STEP) * ZERO_HD_STEP : ZERO_HD_STEP;
                for (int c = 0; c < WIDE; c += 32) {
                    float v[32];
                    __syncwarp();
                    read_accumulator(from + c, v);
#pragma unroll
                    for (int e = 0; e < 32; e++) {
                        float d = row.c1 * exp2_fast(__fmaf_rn(v[e], a.k1, -row.l1));
                        if (TWO) d = __fmaf_rn(row.c2, exp2_fast(__fmaf_rn(v[e], a.k2, -row.l2)), d);
                        v[e] = d;
                    }
                    if (!live || c + 32 > end) {
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            if (!live || c + e >= end) v[e] = 0.0f;
                    }
                    if (!have) {
#pragma unroll
                        for (int e = 0; e < 32; e++) v[e] = nan;
                    }
                    // less the targets' weights, every lane's next target at a time
                    while (__any_sync(0xFFFFFFFFu, goal.now.column < c + 32)) {
                        float x = 0.0f;
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            if (goal.now.column == c + e) x = v[e] -= goal.now.weight;
                        if (goal.now.column < c + 32) {
                            // (of targets in one column that is the last, which has it all)
                            if (goal.heavy)
                                a.heavy[r * ZERO_HD_HEAVY + goal.heavy - 1].cut = x - widen1<DT>(narrow1<DT>(x));
                            goal.step(a);
                        }
                    }
                    // rows past the last counted one are read up to a whole stage
                    if (r - lane >= rows) continue;
                    rows_sent();
                    lay_row<DT>(stage, v);
                    send_rows(stage, &map_o, c0 + c, (int)(r - lane));
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive_first(smem_u32(&sh.sum_empty[acc]));
            } else {
                const int j = (int)tj * ZERO_HD_TILE, width = head_width<PASS>(a, tj);
                // four columns of 32 rows are one run of 512 bytes
                const int64_t own = (int64_t)((rank * 4 + quad) * 64) * 32 + lane;
                float4* part = g.slot < 0 ? nullptr : reinterpret_cast<float4*>(a.parts + (int64_t)g.slot * ZERO_HD_SLOT) + own;
                float4* kept = dw ? nullptr : reinterpret_cast<float4*>(a.acc + (int64_t)(ti * shape.tn + tj) * ZERO_HD_SLOT) + own;
                // (TMA writes whole 16-byte vectors past a matrix's right edge)
                const int sent = dw && !part && a.vec_w && !a.accumulate ? (a.cols % 8 == 0 ? 1 << 30 : a.cols) : 0;
                // (dx: rows past the last counted one are neither kept nor joined)
                for (int c = side * WIDE; (dw || r - lane < counted) && c < (side + 1) * WIDE && c < width; c += 32) {
                    float v[32];
                    __syncwarp();
                    read_accumulator(tmem + acc * ZERO_HD_TILE + c + ((uint32_t)quad << 21), v);
                    if (!have) {
#pragma unroll
                        for (int e = 0; e < 32; e++) v[e] = nan;
                    }
                    if (!part && !dw && !a.first) {
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const float4 p = kept[(c / 4 + e) * 32];
                            v[4 * e] += p.x;
                            v[4 * e + 1] += p.y;
                            v[4 * e + 2] += p.z;
                            v[4 * e + 3] += p.w;
                        }
                    }
                    if (part || (!dw && !a.last)) {
                        float4* o = part ? part : kept;
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            o[(c / 4 + e) * 32] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                        continue;
                    }
                    if (!dw && to) cuts.add<DT>(a, j + c, v);
                    if (j + c + 32 <= sent) {
#pragma unroll
                        for (int e = 0; e < 32; e++) v[e] *= factor;
                        rows_sent();
                        lay_row<DT>(stage, v);
                        send_rows(stage, &map_o, j + c, a.v0 + (int)(r - lane));
                    } else if (dw ? a.vec_w : a.vec_x) {
                        put_row<DT, 32>(a, !dw, to, factor, j + c, v);
                    } else {
                        put_rows<DT>(a, !dw, to, factor, j + c, v, stage);
                    }
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive_first(smem_u32(&sh.sum_empty[acc]));
            }
        }
        // rows on their way have been written before the kernel ends
        if (PASS != HEAD_LOGITS && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    cluster_sync();
    // after a wait that gave up, the second SM may have loaded stages that the first has not: those land too
    if (rank == 0 && threadIdx.x == 0) {
        const uint32_t mine = sh.issued, other = of_second(smem_u32(&sh.issued));
        for (uint32_t q = mine; q < other; q++) {
            const uint32_t bar = smem_u32(&sh.full[q % ZERO_HD_STAGES]);
            mbar_expect_tx(bar, of_second(smem_u32(&sh.bytes[q % ZERO_HD_STAGES])));
            for (uint32_t it = 0; it < ZERO_TMA_WAIT_LIMIT && !mbar_try_wait(bar, q / ZERO_HD_STAGES & 1); it++) {
            }
        }
    }
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    cluster_sync();
}

// Adds the parts of cut tiles of one pass in the contracted axis's order: a warp takes 32 rows and 16
// columns of a tile, or (DEEP) the eight warps of a block share their parts, add them and the eight sums
// in order: for few tiles, of many parts (16 rows of 768 x 50257, 25 parts a tile: 29 us by warps, 9 by blocks).
template <int DT, int PASS, bool DEEP>
static __device__ __forceinline__ void join(const HeadArgs& a, const HeadShape& shape, uint32_t unit, int counted, int top, float common,
                                            float (*turns)[32][17])
{
    constexpr bool INPUT = PASS == HEAD_INPUT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float (*const turn)[17] = turns[warp];
    const uint32_t q = unit >> 7;
    const int strip = (unit >> 4) & 7, c = unit & 15;
    uint32_t ti, tj;
    head_place(head_band<PASS>(a), shape, shape.waves * a.pairs + q, ti, tj);
    const int j = (int)tj * ZERO_HD_TILE + c * 16;
    if (j >= a.cols || (INPUT && (int)ti * ZERO_HD_TILE + strip * 32 >= counted)) return;     // (of a block, all warps)
    const float* parts = a.parts + (INPUT ? 0 : (int64_t)a.slots_x * ZERO_HD_SLOT);
    const int64_t r = (int64_t)ti * ZERO_HD_TILE + strip * 32 + lane;
    float factor = 0.0f;
    uint16_t* to = !INPUT || a.last ? out_row(a, INPUT, r, counted, top, common, factor) : nullptr;
    HeadCuts cuts;
    if (INPUT && to) cuts.begin(a, r);
    float v[16];
#pragma unroll
    for (int e = 0; e < 16; e++) v[e] = 0.0f;
    const int64_t own = (int64_t)(strip * 64 + c * 4) * 32 + lane;
#pragma unroll 4
    for (uint32_t p = DEEP ? warp : 0; p < shape.ranges; p += DEEP ? 8 : 1) {
        const float4* s = reinterpret_cast<const float4*>(parts + (int64_t)(p * shape.rest + q) * ZERO_HD_SLOT) + own;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float4 f = __ldcg(s + e * 32);
            v[4 * e] += f.x;
            v[4 * e + 1] += f.y;
            v[4 * e + 2] += f.z;
            v[4 * e + 3] += f.w;
        }
    }
    if (DEEP) {
        __syncthreads();                                     // (the sums of the unit before have been read)
#pragma unroll
        for (int e = 0; e < 16; e++) turn[lane][e] = v[e];
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int e = 0; e < 16; e++) {
            v[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; w++) v[e] += turns[w][lane][e];
        }
        __syncwarp();
    }
    if (INPUT) {
        float4* kept = reinterpret_cast<float4*>(a.acc + (int64_t)(ti * shape.tn + tj) * ZERO_HD_SLOT) + own;
        if (!a.first) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float4 f = kept[e * 32];
                v[4 * e] += f.x;
                v[4 * e + 1] += f.y;
                v[4 * e + 2] += f.z;
                v[4 * e + 3] += f.w;
            }
        }
        if (!a.last) {
#pragma unroll
            for (int e = 0; e < 4; e++) kept[e * 32] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            return;
        }
    }
    if (INPUT && to) cuts.add<DT>(a, j, v);
    if (INPUT ? a.vec_x : a.vec_w) {
        put_row<DT, 16>(a, INPUT, to, factor, j, v);
        return;
    }
    // two rows' runs of 16 columns an access
#pragma unroll
    for (int e = 0; e < 16; e++) turn[lane][e] = v[e] * factor;
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; e++) {
        const int row = 2 * e + (lane >> 4), col = lane & 15;
        uint16_t* g = reinterpret_cast<uint16_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(to), row));
        if (!g || j + col >= a.cols) continue;
        float x = turn[row][col];
        if (!INPUT && a.accumulate) x += widen1<DT>(g[j + col]);
        g[j + col] = narrow1<DT>(x);
    }
    __syncwarp();
}
template <int DT>
__global__ void __launch_bounds__(256) k_head_join(const __grid_constant__ HeadArgs a)
{
    __shared__ float turn[8][32][17];
    let_next_begin();
    after_previous();
    const int counted = a.st->rows, top = a.st->top - a.st->lift;
    const float common = counted > 0 ? common_factor(a) : 0.0f;
    const HeadShape x = head_shape<HEAD_INPUT>(a, counted), w = head_shape<HEAD_WEIGHT>(a, counted);
    const uint32_t of_x = a.dx && x.ranges > 1 ? x.rest * 128 : 0, of_w = a.dw && w.ranges > 1 ? w.rest * 128 : 0;
    // by blocks if there are too few units for warps, two a block at most.  dw of 4096 rows of 64, whole calls: 4 tiles
    // of 256 tokens 35.4 us by blocks and 36.2 by warps, 6 tiles 37.0 and 36.9, 8 tiles 38.9 and 37.2; dx of 16 rows
    // over 50257 tokens, where seven units of eight have no rows: 4 tiles 66 and 72, 8 tiles 100 and 102.
    if (of_x + of_w <= 2 * gridDim.x) {
        for (uint32_t unit = blockIdx.x; unit < of_x + of_w; unit += gridDim.x) {
            if (unit < of_x) join<DT, HEAD_INPUT, true>(a, x, unit, counted, top, common, turn);
            else join<DT, HEAD_WEIGHT, true>(a, w, unit - of_x, counted, top, common, turn);
        }
        return;
    }
    for (uint32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5); unit < of_x + of_w; unit += gridDim.x * 8) {
        if (unit < of_x) join<DT, HEAD_INPUT, false>(a, x, unit, counted, top, common, turn);
        else join<DT, HEAD_WEIGHT, false>(a, w, unit - of_x, counted, top, common, turn);
    }
}

// ---- the loss ------------------------------------------------------------------------
// 32 counted rows a block: first a lane a row, the 32 warps sharing the tiles' maxima and sums, then a
// warp a row.  The last block to finish adds the blocks' sums in order.  Bound by latency: 7 us for 16 rows of 197
// tiles, 15 for 8192 of 501 (33 MB).
// Blocks that have an SM to themselves take eight tiles at a time, others two (two blocks an SM have 32 registers a
// thread, and that spills 56 bytes).
template <int BLOCKS>
static __global__ void __launch_bounds__(1024, BLOCKS) k_head_loss(const __grid_constant__ HeadArgs a, int tiles)
{
    constexpr int EACH = BLOCKS > 1 ? 2 : 8;
    __shared__ float ms[32][33], ss[32][33], ts[32][33];
    __shared__ double losses[32];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    let_next_begin();
    after_previous();
    const int counted = a.st->rows;
    const int64_t r = (int64_t)blockIdx.x * 32 + lane;
    const float low = __uint_as_float(0xFF800000u), nan = __uint_as_float(0x7FC00000u);
    float m = low, s = 0.0f, t = 0.0f;
    if (r < counted) {
        const float2* part = a.part + r;
        const float* part2 = a.part2 + r;
        for (int v = warp; v < tiles; v += 32 * EACH) {
            float2 p[EACH];
            float p2[EACH];
            float most = m;
#pragma unroll
            for (int e = 0; e < EACH; e++) {
                const bool in = v + 32 * e < tiles;
                p[e] = in ? part[(v + 32 * e) * a.npad] : make_float2(low, 0.0f);
                p2[e] = in && a.two ? part2[(v + 32 * e) * a.npad] : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < EACH; e++) most = fmaxf(most, p[e].x);
            const float base = most == low ? 0.0f : most;   // (a NaN sum of a lowest maximum is kept)
            s *= exp2_fast((m - base) * a.k1);
            if (a.two) t *= exp2_fast((m - base) * a.k2);
#pragma unroll
            for (int e = 0; e < EACH; e++) {
                s += p[e].y * exp2_fast((p[e].x - base) * a.k1);
                if (a.two) t += p2[e] * exp2_fast((p[e].x - base) * a.k2);
            }
            m = most;
        }
    }
    ms[warp][lane] = m;
    ss[warp][lane] = s;
    ts[warp][lane] = t;
    // a warp a row: its targets' logits times their weights
    const int64_t w = (int64_t)blockIdx.x * 32 + warp;
    float dot = 0.0f;
    if (w < counted)
        for (int e = lane; e < a.slots; e += 32) {
            const HeadTarget g = a.target[w * a.slots + e];
            if (g.column < a.vocab) dot += g.weight * a.found[w * a.slots + e];
        }
    __syncthreads();
    float most = m = ms[lane][warp];
    s = ss[lane][warp];
    t = ts[lane][warp];
    for (int o = 16; o > 0; o >>= 1) {
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
        dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
    }
    const float base = most == low ? 0.0f : most;
    s *= exp2_fast((m - base) * a.k1);
    t *= exp2_fast((m - base) * a.k2);
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    }
    if (lane == 0) {
        double loss = 0.0;
        if (w < counted) {
            // k1 is 1/T only where there is no other log-sum-exp
            const HeadRow h = a.info[w];
            const float scale1 = a.labels ? 1.0f : 1.0f / a.temperature;
            float l1 = base * scale1 + logf(s), l2 = a.two ? base / a.temperature + logf(t) : l1;
            if (h.c1 != h.c1) l1 = l2 = nan;
            float x = h.c1 - dot;
            if (a.index) x = __fmaf_rn(h.c2 * a.soft * a.temperature * a.temperature, l2, x);
            if (a.labels) x = __fmaf_rn(a.hard, __fmaf_rn(a.z_loss * l1, l1, l1), x);
            const int64_t row = a.map[w];
            a.loss[row] = x;
            if (a.index) {
                a.lse[2 * row] = l2;
                a.lse[2 * row + 1] = a.labels ? l1 : 0.0f;
            } else {
                a.lse[row] = l1;
            }
            loss = x;
        }
        losses[warp] = loss;
    }
    __syncthreads();
    if (warp > 0 || !a.sums) return;
    double loss = losses[lane];
    for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(0xFFFFFFFFu, loss, o);
    if (gridDim.x > 1) {
        if (lane == 0) {
            __stcg(a.partial + blockIdx.x, loss);
            __threadfence();
            last = atomicAdd(&a.st->ticket, 1u) == gridDim.x - 1;
        }
        __syncwarp();
        if (!last) return;
        __threadfence();
        loss = 0.0;
        for (unsigned b = lane; b < gridDim.x; b += 32) loss += __ldcg(a.partial + b);
        for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(0xFFFFFFFFu, loss, o);
    }
    if (lane == 0) {
        a.sums[0] = (float)loss;
        a.sums[1] = (float)counted;
    }
}

// The kernels of a 16-bit type.
struct HeadKernels {
    const void *pack, *logits[2], *gradient[2], *products, *join;
};
HeadKernels head_kernels_fp16();
HeadKernels head_kernels_bf16();

template <int DT>
HeadKernels head_kernels()
{
    return {(const void*)k_head_pack<DT>,
            {(const void*)k_head<DT, HEAD_LOGITS, false>, (const void*)k_head<DT, HEAD_LOGITS, true>},
            {(const void*)k_head<DT, HEAD_GRADIENT, false>, (const void*)k_head<DT, HEAD_GRADIENT, true>},
            (const void*)k_head<DT, HEAD_PRODUCTS, false>,
            (const void*)k_head_join<DT>};
}

}  // namespace zero
