// zero_wgrad.cu -- the weight gradient of a linear layer from the gradient of its
// output and the 8-bit checkpoint of its input: dw = dy^T xh, db = the column sums
// of dy (include/zero_b200.h).
//
// dw is a matrix product whose contraction runs over tokens, bound by the 16-bit
// tensor cores (2 tokens n k operations) once there are more than a few hundred
// tokens.  The checkpoint's values are exact in the 16-bit type, so they are widened
// into the tensor cores' shared-memory operand and multiplied as they are.
//
// A pair of SMs (a cluster of two) computes a 256 x 256 tile of dw, 64 tokens at a
// time: each SM's 128 rows of dy^T come by TMA in the layout the tensor cores read
// (both operands have the non-contracted axis contiguous, so nothing is transposed),
// its 128 columns of codes and their exponents come by TMA as bytes, eight warps
// widen the codes into the second operand, and one thread of the pair issues the
// products, which accumulate in tensor memory.  With two accumulators, four other
// warps write one tile out while the next is summed.
//
// Tiles are dealt to the pairs in whole waves, where all pairs work on the same
// tokens at the same time and share their panels in L2; the tiles of an incomplete
// last wave are cut along the token axis into equal parts, one for each pair.  Parts
// go to the workspace and a second kernel adds them in token order, so the sums do
// not depend on timing.
#include <cuda.h>

#include <mutex>

#include "zero_act.cuh"
#include "zero_b200.h"
#include "zero_tma.cuh"
#include "zero_trace.h"

namespace zero {

#define ZERO_WG_TILE 256                    // rows and columns of a pair's tile
#define ZERO_WG_TOK 64                      // tokens of a stage
#define ZERO_WG_STAGES 6                    // stages of dy rows
#define ZERO_WG_CODES 4                     // stages of codes
#define ZERO_WG_WIDE 5                      // widened stages
#define ZERO_WG_GROUPS 4                    // groups of widening warps, a stage each
#define ZERO_WG_WIDENERS 256                // threads that widen codes
#define ZERO_WG_THREADS (256 + ZERO_WG_WIDENERS)    // warps 0 and 2 TMA, 1 products, 4-7 output, from 8 widening
#define ZERO_WG_PAIRS 80                    // most pairs that share a launch's work
#define ZERO_WG_PART 8                      // least stages of a part of a cut tile
#define ZERO_WG_RUN 12                      // stages an accumulator adds for an fp32 gradient (from 16 stages),
#define ZERO_WG_RUN_16 1024                 // and for a 16-bit one
#define ZERO_WG_DEEP 4                      // parts a tile from which eight warps share them
#define ZERO_WG_FEW 64                      // most tokens that k_wgrad_few takes,
#define ZERO_WG_FEW_WORK (60ll << 20)       // and most products
#define ZERO_WG_FEW_TOK 32                  // tokens it adds at a time
#define ZERO_WG_RANGES 32                   // most token ranges that k_wgrad_columns adds
#ifndef ZERO_WG_WAIT_LIMIT                  // polls before a wait gives up (not those for what is in flight)
#define ZERO_WG_WAIT_LIMIT ZERO_TMA_WAIT_LIMIT
#endif

// bytes of a stage in one SM: dy rows, codes, exponents; and of widened codes (as dy rows); the
// column sums of a tile (a row of 128 from each widening warp)
#define ZERO_WG_A 16384
#define ZERO_WG_C 8192
#define ZERO_WG_E 1024
#define ZERO_WG_SUMS (ZERO_WG_WIDENERS / 32 * 512)
#define ZERO_WG_OUT 2048                    // rows that an output warp writes
#define ZERO_WG_SMEM \
    (ZERO_WG_STAGES * ZERO_WG_A + ZERO_WG_CODES * (ZERO_WG_C + ZERO_WG_E) + ZERO_WG_WIDE * ZERO_WG_A + ZERO_WG_SUMS + 4 * ZERO_WG_OUT + 1024)
// Slots of the workspace for sums: two for each pair's parts of cut tiles, one for its runs.
#define ZERO_WG_SLOTS (3 * ZERO_WG_PAIRS)
#define ZERO_WG_SLOT (ZERO_WG_TILE * (ZERO_WG_TILE + 1))  // floats of one: a tile's sums, its rows' sums of dy

struct WgradArgs {
    const uint16_t* dy;
    const uint8_t* ckpt;
    const uint16_t *scale, *shift;
    void *dw, *db;
    int32_t* err;
    float *sums, *slots;                    // dy's columns added [ZERO_WG_RANGES][n] (null: not); parts of cut tiles, runs' sums
    int64_t tokens, n, k, ldy, ldw;
    int64_t wide;
    int steps;                              // stages of a tile
    uint32_t tiles_n, tiles_k, share, extra, run;
    int pairs, waves, rest, rest_pairs;
    int grad_dtype, accumulate, vec, vec_s;
    int ranges;                             // the sums' token ranges
};

// ---- the division of the work ------------------------------------------------------
// A run of stages whose products one accumulator adds.  The tensor cores cut each sum off
// rather than round it, so an accumulator's relative error grows by about 1.6e-8 a step of
// 16 tokens (6.4e-6 after 400, at random inputs): fp32 gradients, whose type would show it,
// are summed in runs of 12 stages (48 steps; from 16 stages) that are added in fp32.  At 30011 tokens,
// 776 x 771, runs of 64 stages take 59.6 us and are off by 3.8e-6, runs of 12 take 77.9 us and
// are off by 7.4e-7 (an fp32 product without tensor cores: 2.9e-7).  16-bit gradients are rounded
// to 2.1e-4 (fp16) or 1.7e-3 of their 2-norm; runs of 1024 stages (65536 tokens) keep the sums'
// error below a third of that: 1 M tokens, 2560 x 2048 in fp16 were off by 1.23e-3 in one run.
struct WgradSegment {
    uint32_t tile;
    int32_t s0, s1;                         // stages [s0, s1) of a tile
    int slot;                               // -1: the whole tile's, else the place of its part
    bool first, last;                       // run of its tile or part
};

// First unit (stage of a tile of the last wave) of a pair's share.
static __host__ __device__ __forceinline__ uint32_t wgrad_share(const WgradArgs& a, uint32_t pair)
{
    return pair * a.share + (pair < a.extra ? pair : a.extra);
}

// Run `c` of stages [b, e) of a tile.
static __host__ __device__ __forceinline__ void wgrad_run(const WgradArgs& a, uint32_t b, uint32_t e, uint32_t c, WgradSegment& g)
{
    g.s0 = (int32_t)(b + c * a.run);
    g.first = c == 0;
    g.last = e - g.s0 <= a.run;
    g.s1 = g.last ? (int32_t)e : (int32_t)(g.s0 + a.run);
}

// Segment i of a pair; false past its last.
static __host__ __device__ __forceinline__ bool wgrad_segment(const WgradArgs& a, uint32_t pair, uint32_t i, WgradSegment& g)
{
    const uint32_t steps = a.steps, runs = (steps + a.run - 1) / a.run;
    if (i < a.waves * runs) {
        const uint32_t w = runs == 1 ? i : i / runs;
        g.tile = w * a.pairs + pair;
        g.slot = -1;
        wgrad_run(a, 0, steps, i - w * runs, g);
        return true;
    }
    if (pair >= (uint32_t)a.rest_pairs) return false;
    i -= a.waves * runs;
    const uint32_t u0 = wgrad_share(a, pair), u1 = wgrad_share(a, pair + 1), t0 = u0 / steps;
    for (uint32_t part = 0; part < 2; part++) {             // a share lies in two tiles at most
        const uint32_t t = t0 + part;
        uint32_t b = t * steps, e = b + steps;
        if (b >= u1) return false;
        b = b > u0 ? b : u0;
        e = e < u1 ? e : u1;
        const uint32_t n = (e - b + a.run - 1) / a.run;
        if (i < n) {
            g.tile = (uint32_t)a.waves * a.pairs + t;
            g.slot = e - b == steps ? -1 : (int)(2 * pair + part);
            wgrad_run(a, b - t * steps, e - t * steps, i, g);
            return true;
        }
        i -= n;
    }
    return false;
}

// The slot that a segment's sums go to where they are kept, and whether they are: those of a
// part, and of a whole tile's run that others come before or after.
static __host__ __device__ __forceinline__ int wgrad_slot(const WgradSegment& g, uint32_t pair)
{
    return g.slot >= 0 ? g.slot : 2 * ZERO_WG_PAIRS + (int)pair;
}
static __host__ __device__ __forceinline__ bool wgrad_kept(const WgradSegment& g)
{
    return g.slot >= 0 || !g.first || !g.last;
}

// Tiles in an order that keeps a wave's panels few: bands of eight tiles along n.
static __host__ __device__ __forceinline__ void wgrad_place(const WgradArgs& a, uint32_t tile, int64_t& i0, int64_t& j0)
{
    const uint32_t band = tile / (8u * a.tiles_k), in = tile - band * 8u * a.tiles_k;
    const uint32_t high = a.tiles_n - band * 8 < 8 ? a.tiles_n - band * 8 : 8;
    j0 = (int64_t)(in / high) * ZERO_WG_TILE;
    i0 = (int64_t)(band * 8 + in % high) * ZERO_WG_TILE;
}

// For each tile of the last wave: the pairs that have parts of it, and whether the first of
// them has it as its second tile.
struct WgradJoin {
    uint8_t p0[ZERO_WG_PAIRS], p1[ZERO_WG_PAIRS], second[ZERO_WG_PAIRS];
};

// Columns of the tile at j0 that are multiplied: half a tile at the right edge where that is
// enough (each SM's part of the operand is then one whole 64-column group of its layout; a
// smaller part is not a documented form).
static __device__ __forceinline__ int wgrad_width(const WgradArgs& a, int64_t j0)
{
    return a.k - j0 > ZERO_WG_TILE / 2 ? ZERO_WG_TILE : ZERO_WG_TILE / 2;
}

// ---- output ------------------------------------------------------------------------
static __device__ __forceinline__ float grad_in(const void* p, int64_t i, int grad_dtype)
{
    if (grad_dtype == 2) return static_cast<const float*>(p)[i];
    const uint16_t u = static_cast<const uint16_t*>(p)[i];
    return grad_dtype == 0 ? widen1<0>(u) : widen1<1>(u);
}
static __device__ __forceinline__ void put_grad(void* p, int64_t i, float v, int grad_dtype, int accumulate)
{
    if (accumulate) v += grad_in(p, i, grad_dtype);
    if (grad_dtype == 2) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = grad_dtype == 0 ? narrow1<0>(v) : narrow1<1>(v);
}

template <int DT>
static __device__ __forceinline__ void eight(const uint16_t* p, float (&w)[8])
{
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
    widen2<DT>(q.x, w[0], w[1]);
    widen2<DT>(q.y, w[2], w[3]);
    widen2<DT>(q.z, w[4], w[5]);
    widen2<DT>(q.w, w[6], w[7]);
}

// N columns from j of a row: times the norm's weight, plus its bias times s, the row's column
// sum of dy.
template <int DT, int N>
static __device__ __forceinline__ void affine(const WgradArgs& a, int64_t j, float (&v)[N], float s)
{
    const int m = a.k - j < N ? (int)(a.k - j) : N;
    if ((a.scale || a.shift) && a.vec_s && m == N) {
#pragma unroll
        for (int c = 0; c < N; c += 8) {
            float w[8];
            if (a.scale) {
                eight<DT>(a.scale + j + c, w);
#pragma unroll
                for (int e = 0; e < 8; e++) v[c + e] *= w[e];
            }
            if (a.shift) {
                eight<DT>(a.shift + j + c, w);
#pragma unroll
                for (int e = 0; e < 8; e++) v[c + e] = __fmaf_rn(s, w[e], v[c + e]);
            }
        }
    } else if (a.scale || a.shift) {
#pragma unroll
        for (int c = 0; c < N; c++)
            if (c < m) {
                if (a.scale) v[c] *= widen1<DT>(__ldg(a.scale + j + c));
                if (a.shift) v[c] = __fmaf_rn(s, widen1<DT>(__ldg(a.shift + j + c)), v[c]);
            }
    }
}

// N columns from j of row i, a lane its own row.
template <int DT, int N>
static __device__ __forceinline__ void put_row(const WgradArgs& a, int64_t i, int64_t j, float (&v)[N], float s)
{
    if (i >= a.n || j >= a.k) return;
    const int m = a.k - j < N ? (int)(a.k - j) : N;
    affine<DT, N>(a, j, v, s);
    const int64_t at = i * a.ldw + j;
    if (a.vec && m == N) {
        if (a.grad_dtype == 2) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.dw) + at);
#pragma unroll
            for (int c = 0; c < N; c += 4) {
                float4 q = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
                if (a.accumulate) {
                    const float4 p = o[c / 4];
                    q = make_float4(q.x + p.x, q.y + p.y, q.z + p.z, q.w + p.w);
                }
                o[c / 4] = q;
            }
        } else {
            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dw) + at);
#pragma unroll
            for (int c = 0; c < N; c += 8) {
                if (a.accumulate) {
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
                o[c / 8] = make_uint4(narrow2<DT>(v[c], v[c + 1]), narrow2<DT>(v[c + 2], v[c + 3]),
                                      narrow2<DT>(v[c + 4], v[c + 5]), narrow2<DT>(v[c + 6], v[c + 7]));
            }
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < N; c++)
        if (c < m) put_grad(a.dw, at + c, v[c], a.grad_dtype, a.accumulate);
}

// A warp's 32 rows of 64 bytes (of 16 or 32 columns from j) between dw and shared memory, a lane
// a column.  16-byte word q of row r lies at q ^ (r >> 1 & 3), so that lanes that each take a row
// meet all banks too.
template <bool IN>
static __device__ __forceinline__ void move_rows(const WgradArgs& a, int64_t i0, int64_t j, uint32_t stage)
{
    const int lane = threadIdx.x & 31, half = lane >> 4;
    if (a.grad_dtype == 2) {
#pragma unroll 8
        for (int p = 0; p < 16; p++) {
            const int r = 2 * p + half, c = lane & 15;
            const uint32_t s = stage + r * 64 + ((c >> 2) ^ (r >> 1 & 3)) * 16 + (c & 3) * 4;
            float* g = static_cast<float*>(a.dw) + (i0 + r) * a.ldw + j + c;
            if (i0 + r >= a.n || j + c >= a.k) continue;
            if (IN) {
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(s), "f"(*g) : "memory");
            } else {
                float x;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(s));
                *g = x;
            }
        }
        return;
    }
#pragma unroll 8
    for (int r = 0; r < 32; r++) {
        const uint32_t s = stage + r * 64 + ((lane >> 3) ^ (r >> 1 & 3)) * 16 + (lane & 7) * 2;
        uint16_t* g = static_cast<uint16_t*>(a.dw) + (i0 + r) * a.ldw + j + lane;
        if (i0 + r >= a.n || j + lane >= a.k) continue;
        if (IN) {
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(s), "h"(*g) : "memory");
        } else {
            uint16_t x;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(s));
            *g = x;
        }
    }
}

// put_row() for rows of dw that are not aligned to vectors: 32 columns from j of the warp's rows
// from i0, through 2 KB of shared memory, so that an access of the warp is a run of a row and not
// an element of each of 32 rows (4095 x 4095 over 128 tokens: 171 -> 40 us, 440 -> 134 us when
// added to what is there).  Aligned rows are faster written by the lanes that have them: 21
// against 31 us at 4096 x 4096.
template <int DT>
static __device__ __forceinline__ void put_rows(const WgradArgs& a, int64_t i0, int64_t j, float (&v)[32], float s, uint32_t stage)
{
    const int lane = threadIdx.x & 31;
    if (j >= a.k || i0 >= a.n) return;                       // all lanes
    if (i0 + lane < a.n) affine<DT, 32>(a, j, v, s);
    const uint32_t own = stage + lane * 64;
    auto word = [&](int q) { return own + (q ^ (lane >> 1 & 3)) * 16; };
    auto get = [&](int q) {
        uint4 x;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(word(q)));
        return x;
    };
    auto put = [&](int q, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(word(q)), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
    };
    if (a.grad_dtype == 2) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            if (j + 16 * h >= a.k) break;
            if (a.accumulate) {
                move_rows<true>(a, i0, j + 16 * h, stage);
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const uint4 x = get(q);
                    v[16 * h + 4 * q] += __uint_as_float(x.x);
                    v[16 * h + 4 * q + 1] += __uint_as_float(x.y);
                    v[16 * h + 4 * q + 2] += __uint_as_float(x.z);
                    v[16 * h + 4 * q + 3] += __uint_as_float(x.w);
                }
            }
#pragma unroll
            for (int q = 0; q < 4; q++)
                put(q, __float_as_uint(v[16 * h + 4 * q]), __float_as_uint(v[16 * h + 4 * q + 1]),
                    __float_as_uint(v[16 * h + 4 * q + 2]), __float_as_uint(v[16 * h + 4 * q + 3]));
            __syncwarp();
            move_rows<false>(a, i0, j + 16 * h, stage);
            __syncwarp();
        }
        return;
    }
    if (a.accumulate) {
        move_rows<true>(a, i0, j, stage);
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const uint4 x = get(q);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float lo, hi;
                widen2<DT>(w[e], lo, hi);
                v[8 * q + 2 * e] += lo;
                v[8 * q + 2 * e + 1] += hi;
            }
        }
    }
#pragma unroll
    for (int q = 0; q < 4; q++)
        put(q, narrow2<DT>(v[8 * q], v[8 * q + 1]), narrow2<DT>(v[8 * q + 2], v[8 * q + 3]),
            narrow2<DT>(v[8 * q + 4], v[8 * q + 5]), narrow2<DT>(v[8 * q + 6], v[8 * q + 7]));
    __syncwarp();
    move_rows<false>(a, i0, j, stage);
    __syncwarp();
}

// Whether a tile adds its rows' sums of dy: for db (and for the norm's bias if there are no
// other columns of tiles), in the first column, unless k_wgrad_columns has added them all.
static __device__ __forceinline__ bool adds_sums(const WgradArgs& a, int64_t j0)
{
    return (a.db || a.shift) && j0 == 0 && !a.sums;
}

// Row i's sum of dy from k_wgrad_columns.
static __device__ __forceinline__ float column_sum(const WgradArgs& a, int64_t i)
{
    float s = 0.0f;
    if (a.sums && i < a.n)
        for (int p = 0; p < a.ranges; p++) s += __ldg(a.sums + p * a.n + i);
    return s;
}

// ---- the pair's machinery ------------------------------------------------------------
static __device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// True in one lane of a whole warp.  Code under it is known to run in one thread, so that the
// operands of the copies and products it issues stay in the warp's uniform registers: issuing a
// stage's four products or its copies took about 800 cycles with `lane == 0`, longer than the
// products themselves (1161 -> 1048 us at 16384 x 4096 x 14336).
static __device__ __forceinline__ bool elected()
{
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}
// Every thread of both SMs; the warp is together again after it (what follows may be a
// whole-warp instruction).
static __device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
    __syncwarp();
}
// Arrive on the barrier of the pair's first SM that lies at this SM's address `bar`.  What
// the arrival announces lies in this SM's own shared or tensor memory and is ordered for the
// tensor cores by the proxy fence or the tcgen05 fence before it, so the arrival itself
// carries no cluster-wide release (which, with the matching acquire in the wait, cost a third of
// the rate: 1089 against 1504 TFLOP/s at 8192 x 4096 x 4096).
static __device__ __forceinline__ void arrive_first(uint32_t bar)
{
    asm volatile("{\n .reg .b32 r;\n mapa.shared::cluster.u32 r, %0, 0;\n"
                 " mbarrier.arrive.shared::cluster.b64 _, [r];\n}" ::"r"(bar) : "memory");
}
// A lane to arrive for the warp, known once every lane has its x.  An arrival that hands a
// buffer back must not be made while loads from it are under way, and the barrier unit does not
// wait for loads before it: x is made of the loaded values.
static __device__ __forceinline__ int lane_with(uint32_t x) { return __any_sync(0xFFFFFFFFu, x == 0) ? 0 : 1; }
// Bounded wait of a lane: false when it gave up (here or in another warp of this SM).
static __device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity, volatile int* dead, int32_t* err)
{
    for (uint32_t it = 0; it < ZERO_WG_WAIT_LIMIT; it++) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*dead) return false;
    }
    *dead = 1;
    atomicExch(err, ZERO_ETIMEOUT);
    return false;
}
// The same for a whole warp, whose lanes go on or stop together (votes and shuffles of all lanes
// follow), so every poll is voted on.  A vote after lanes that polled by themselves took 154 us
// instead of 146 at 8192 x 6400 x 1600, a loop without a first poll of its own 151.
static __device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* dead, int32_t* err)
{
    if (ZERO_WG_WAIT_LIMIT > 0 && __all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
#pragma unroll 1
    for (uint32_t it = 0; it < ZERO_WG_WAIT_LIMIT; it++) {
        if (__any_sync(0xFFFFFFFFu, *dead)) return false;
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    }
    *dead = 1;
    atomicExch(err, ZERO_ETIMEOUT);
    __syncwarp();
    return false;
}
static __device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
// Completion of every product issued so far arrives on `bar` in both SMs (or in those of a mask).
static __device__ __forceinline__ void commit_both(uint32_t bar, uint16_t sms = 3)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"(sms) : "memory");
}
// Operand in shared memory with the non-contracted axis contiguous, 128-byte swizzle:
// groups of 64 columns are 8192 bytes apart, groups of 8 tokens 1024.
static __device__ __forceinline__ uint64_t operand(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)(8192 >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
static __device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t what, bool add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(what), "r"((uint32_t)add) : "memory");
}
static __device__ __forceinline__ void read_accumulator(uint32_t at, float (&v)[32])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at) : "memory");
#pragma unroll
    for (int i = 0; i < 32; i++) v[i] = __uint_as_float(r[i]);
}

// Two codes (bytes 0 and 1, or 2 and 3, of w) times their block's 2^e, as a 16-bit pair.
// bf16: with l the code's low seven bits, 0x4300 | l is 128 + l, and 0x4300 with the
// code's sign bit in place 7 is 128 or 256; the difference is the code.  fp16: 1024 plus
// the code XOR 128 in the mantissa, less 1152.  Difference and product are exact.
template <int DT>
static __device__ __forceinline__ uint32_t widen_codes(uint32_t w, uint32_t select, uint32_t scale)
{
    if (DT == 1) {
        const uint32_t x = __byte_perm(w, 0x43434343u, select);
        const uint32_t t = x & 0xFF7FFF7Fu, u = x & 0xFF80FF80u;
        const __nv_bfloat162 c = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&t),
                                         *reinterpret_cast<const __nv_bfloat162*>(&u));
        const __nv_bfloat162 r = __hmul2(c, *reinterpret_cast<const __nv_bfloat162*>(&scale));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    const uint32_t x = __byte_perm(w, 0x64646464u, select), bias = 0x64806480u;     // 1152
    const __half2 c = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&bias));
    const __half2 r = __hmul2(c, *reinterpret_cast<const __half2*>(&scale));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// 2^(E - 127) twice in the 16-bit type.  E = 0 is no block's (a row past the last token):
// 0.  255 gives inf, and 0 * inf = NaN; exponents that fp16 does not have give NaN.
template <int DT>
static __device__ __forceinline__ uint32_t code_scale(uint32_t e)
{
    uint32_t s;
    if (DT == 1) {
        s = e << 7;
    } else {
        s = __half_as_ushort(__float2half_rn(__uint_as_float(e << 23)));
        if (e != 0 && e != ZERO_ACT_BAD && (e < 103 || e > 136)) s = 0x7FFF;
    }
    return s | s << 16;
}

// Three rings, as stage g of a pair (counted over all its segments) goes through them: codes
// (slot g mod CODES, free when a group of warps has read them), dy rows (slot g mod STAGES) and
// widened codes (place g mod WIDE), both free when the products are done.
// A parity wait does not tell a barrier's use from the one after next, so a thread may only wait
// for a use when it knows the one before to be over.  Threads that take every stage in turn know
// it.  A group of widening warps takes every fourth stage, and meets a ring's barriers only now
// and then; each barrier it waits on is therefore one of (slots x GROUPS), of which it alone
// meets every fourth, at every use.
// The rings' depths: six, four and five fill the 227 KB and were the fastest at 16384 x 4096 x
// 14336 and 8192 x 4096 x 4096 (one ring of six for both loads and four places: 2 to 5 % slower,
// of five stages 13 %).  A stage's way through them takes about 2300 cycles (850 for the loads,
// 1100 to widen, the arrivals), its products 512.
static_assert((ZERO_WG_WIDENERS / ZERO_WG_GROUPS / 4) % 8 == 0, "a thread's tokens keep their swizzle");
static_assert(ZERO_WG_GROUPS <= ZERO_WG_CODES && ZERO_WG_GROUPS <= ZERO_WG_STAGES && ZERO_WG_GROUPS <= ZERO_WG_WIDE,
              "every group's stage has a place in each ring");

struct WgradShared {
    uint64_t rows[ZERO_WG_STAGES * ZERO_WG_GROUPS];     // a stage's dy rows have come
    uint64_t codes[ZERO_WG_CODES * ZERO_WG_GROUPS];     // its codes and exponents have come
    uint64_t done[ZERO_WG_WIDE * ZERO_WG_GROUPS];       // its products are done: the place is free
    uint64_t empty[ZERO_WG_STAGES];         // the same, for the dy rows' slot
    uint64_t read[ZERO_WG_CODES];           // its codes have been read
    uint64_t ready[ZERO_WG_WIDE];           // both SMs' operands are in place (first SM's)
    uint64_t sum_full[2], sum_empty[2];     // accumulators
    uint64_t col_full, col_empty;           // column sums
    uint64_t drain;                         // products in flight after a wait gave up
    uint32_t tmem;
    int dead;
};

template <int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(ZERO_WG_THREADS, 1)
    k_wgrad(const __grid_constant__ WgradArgs a, const __grid_constant__ CUtensorMap map_y,
            const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_e)
{
    extern __shared__ unsigned char raw[];
    __shared__ WgradShared sh;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t base_c = base + ZERO_WG_STAGES * ZERO_WG_A, wide = base_c + ZERO_WG_CODES * (ZERO_WG_C + ZERO_WG_E);
    const uint32_t cols = wide + ZERO_WG_WIDE * ZERO_WG_A;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t pair = blockIdx.x >> 1;
    volatile int* dead = &sh.dead;
    if (threadIdx.x == 0) {
        for (int s = 0; s < ZERO_WG_STAGES * ZERO_WG_GROUPS; s++) mbar_init(smem_u32(&sh.rows[s]), 1);
        for (int s = 0; s < ZERO_WG_CODES * ZERO_WG_GROUPS; s++) mbar_init(smem_u32(&sh.codes[s]), 1);
        for (int s = 0; s < ZERO_WG_CODES; s++) mbar_init(smem_u32(&sh.read[s]), ZERO_WG_WIDENERS / 32 / ZERO_WG_GROUPS);
        for (int s = 0; s < ZERO_WG_STAGES; s++) mbar_init(smem_u32(&sh.empty[s]), 1);
        for (int s = 0; s < ZERO_WG_WIDE; s++) mbar_init(smem_u32(&sh.ready[s]), 2 * ZERO_WG_WIDENERS / 32 / ZERO_WG_GROUPS);
        for (int s = 0; s < ZERO_WG_WIDE * ZERO_WG_GROUPS; s++) mbar_init(smem_u32(&sh.done[s]), 1);
        for (int s = 0; s < 2; s++) {
            mbar_init(smem_u32(&sh.sum_full[s]), 1);
            mbar_init(smem_u32(&sh.sum_empty[s]), 8);
        }
        mbar_init(smem_u32(&sh.col_full), ZERO_WG_WIDENERS / 32);
        mbar_init(smem_u32(&sh.col_empty), 4);
        mbar_init(smem_u32(&sh.drain), 1);
        sh.dead = 0;
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
    WgradSegment g;

    if (warp == 0 || warp == 2) {
        // ---- loads: warp 0 dy rows, warp 2 codes and exponents ----
        if (elected()) {
            const bool codes = warp == 2;
            const uint32_t ring = codes ? ZERO_WG_CODES : ZERO_WG_STAGES, bars = ring * ZERO_WG_GROUPS;
            const uint32_t loads = smem_u32(codes ? sh.codes : sh.rows), frees = smem_u32(codes ? sh.read : sh.empty);
            uint32_t n = 0, s = 0, l = 0, ph = 0;            // stages issued; slot, barrier, the slot's turn
            bool ok = true;
            for (int i = 0; ok && wgrad_segment(a, pair, i, g); i++) {
                int64_t i0, j0;
                wgrad_place(a, g.tile, i0, j0);
                const int x = (int)(i0 + rank * 128), c = (int)j0 + rank * (wgrad_width(a, j0) / 2);
                const int e = (int)a.wide + (c / 32 & ~15);
                for (int t = g.s0; t < g.s1; t++, n++) {
                    if (n >= ring && !pair_wait(frees + 8 * s, ph ^ 1u, dead, a.err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = loads + 8 * l;
                    const int y = t * ZERO_WG_TOK;           // below 2^31
                    if (codes) {
                        const uint32_t at = base_c + s * (ZERO_WG_C + ZERO_WG_E);
                        mbar_expect_tx(bar, ZERO_WG_C + ZERO_WG_E);
                        tma_box(at, &map_c, c, y, bar);
                        tma_box(at + ZERO_WG_C, &map_e, e, y, bar);
                    } else {
                        const uint32_t at = base + s * ZERO_WG_A;
                        mbar_expect_tx(bar, ZERO_WG_A);
                        tma_box(at, &map_y, x, y, bar);
                        tma_box(at + 8192, &map_y, x + 64, y, bar);
                    }
                    if (++s == ring) { s = 0; ph ^= 1u; }
                    if (++l == bars) l = 0;
                }
            }
            // before this SM's shared memory is given back: the last copies have landed, and the
            // last products are done, as all barriers that they arrive on say
            for (uint32_t q = n > ring ? n - ring : 0; q < n; q++) {
                for (uint32_t it = 0; it < ZERO_TMA_WAIT_LIMIT && !mbar_try_wait(loads + 8 * (q % bars), q / bars & 1); it++) {
                }
                if (!codes && !*dead) pair_wait(frees + 8 * (q % ring), q / ring & 1, dead, a.err);
            }
            const uint32_t places = ZERO_WG_WIDE * ZERO_WG_GROUPS;
            for (uint32_t q = n > ZERO_WG_WIDE ? n - ZERO_WG_WIDE : 0; codes && q < n; q++)
                if (!*dead) pair_wait(smem_u32(&sh.done[q % places]), q / places & 1, dead, a.err);
        }
    } else if (warp == 1) {
        // ---- products (the first SM's thread, for both) ----
        if (rank == 0 && elected()) {
            // fp32 sums of fp16/bf16 operands, both with the contracted axis strided, 256 x width
            const uint32_t kind = 1u << 4 | (DT == 1 ? 1u << 7 | 1u << 10 : 0u) | 1u << 15 | 1u << 16 |
                                  (uint32_t)(ZERO_WG_TILE >> 4) << 24;
            uint32_t s = 0, b = 0, f = 0, ph = 0;            // slot, place, the place's barrier, turn
            bool ok = true;
            int i = 0;
            for (; ok && wgrad_segment(a, pair, i, g); i++) {
                const int acc = i & 1;
                if (i >= 2 && !pair_wait(smem_u32(&sh.sum_empty[acc]), (uint32_t)((i >> 1) - 1) & 1u, dead, a.err)) {
                    ok = false;
                    break;
                }
                int64_t i0, j0;
                wgrad_place(a, g.tile, i0, j0);
                const uint32_t what = kind | (uint32_t)(wgrad_width(a, j0) >> 3) << 17;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int t = g.s0; t < g.s1; t++) {
                    if (!pair_wait(smem_u32(&sh.ready[b]), ph, dead, a.err)) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint64_t da = operand(base + s * ZERO_WG_A), db = operand(wide + b * ZERO_WG_A);
#pragma unroll
                    for (int q = 0; q < ZERO_WG_TOK / 16; q++)
                        product(tmem + acc * ZERO_WG_TILE, da + q * (2048 >> 4), db + q * (2048 >> 4), what,
                                t > g.s0 || q > 0);
                    commit_both(smem_u32(&sh.done[f]));
                    commit_both(smem_u32(&sh.empty[s]));
                    if (++s == ZERO_WG_STAGES) s = 0;
                    if (++b == ZERO_WG_WIDE) { b = 0; ph ^= 1u; }
                    if (++f == ZERO_WG_WIDE * ZERO_WG_GROUPS) f = 0;
                }
                if (ok) commit_both(smem_u32(&sh.sum_full[acc]));
            }
            // the other SM's last arrivals are here before this SM can exit: one that came
            // after would find no barrier
            for (int q = i > 2 ? i - 2 : 0; ok && q < i; q++)
                ok = pair_wait(smem_u32(&sh.sum_empty[q & 1]), (uint32_t)(q >> 1) & 1u, dead, a.err);
            if (*dead) {                                     // let the products in flight finish
                commit_both(smem_u32(&sh.drain), 1);
                for (uint32_t it = 0; it < ZERO_TMA_WAIT_LIMIT && !mbar_try_wait(smem_u32(&sh.drain), 0); it++) {
                }
            }
        }
    } else if (warp >= 8) {
        // ---- codes to 16-bit values ----
        // Groups of warps take stages in turn, so a stage's latencies (its barrier, shared
        // memory, the fence before the tensor cores read) overlap the other groups' work.  A
        // thread takes a token's block of 32 columns, and further tokens of the stage.  The
        // order in which it takes a block's halves (h) makes the eight lanes of each shared-
        // memory access fall on different 16-byte columns, reading and writing.
        constexpr int GROUPS = ZERO_WG_GROUPS, GROUP = ZERO_WG_WIDENERS / GROUPS, TOKENS = GROUP / 4, EACH = ZERO_WG_TOK / TOKENS;
        const int w = (threadIdx.x - 256) % GROUP, group = (threadIdx.x - 256) / GROUP;
        const int blk = w & 3, tok = w >> 2, h = (blk >> 1) ^ (tok & 1);
        const uint32_t from = tok * 128 + blk * 32 + 16 * h, row = (blk >> 1) * 8192 + tok * 128;
        const uint32_t col = (uint32_t)(((blk & 1) * 4 + 2 * h) ^ (tok & 7)) * 16;
        // this group's stage: its place, slots and barriers, and their turns; the stage whose
        // products free the place
        uint32_t b = group % ZERO_WG_WIDE, cs = group % ZERO_WG_CODES, cl = group, rs = group % ZERO_WG_STAGES, rl = group;
        uint32_t cph = 0, rph = 0, fph = 0;
        int f = group - ZERO_WG_WIDE;                       // below 0: the place is new
        int skip = group;
        // column sums of dy, for the tiles that need them: eight columns (chunk) of every few tokens
        const int chunk = w & 15, tok0 = w >> 4;
        int summed = 0;
        bool ok = true;
        for (int i = 0; ok && wgrad_segment(a, pair, i, g); i++) {
            int64_t i0, j0;
            wgrad_place(a, g.tile, i0, j0);
            const bool sums = adds_sums(a, j0);
            f32x2_t total[4];
#pragma unroll
            for (int c = 0; c < 4; c++) total[c] = pack2(0.0f, 0.0f);
            const int half = wgrad_width(a, j0) / 2;          // this SM's columns
            const uint32_t eat = tok * 16 + (uint32_t)((j0 + rank * half) / 32 & 15) + blk;
            const bool mine = blk * 32 < half;
            const int len = g.s1 - g.s0;
            int t = skip;
            for (; t < len; t += GROUPS) {
                if (!warp_wait(smem_u32(&sh.codes[cl]), cph, dead, a.err)) {
                    ok = false;
                    break;
                }
                const uint32_t codes = base_c + cs * (ZERO_WG_C + ZERO_WG_E), to = wide + b * ZERO_WG_A + row;
                uint32_t e[EACH], q[EACH][2][4], all = 0;
                if (mine) {
#pragma unroll
                    for (int u = 0; u < EACH; u++) {
                        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(e[u]) : "r"(codes + ZERO_WG_C + eat + u * TOKENS * 16));
#pragma unroll
                        for (int c = 0; c < 2; c++)
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(q[u][c][0]), "=r"(q[u][c][1]), "=r"(q[u][c][2]), "=r"(q[u][c][3])
                                         : "r"(codes + u * TOKENS * 128 + (from ^ 16 * c)));
                    }
                }
                if (mine)
#pragma unroll
                    for (int u = 0; u < EACH; u++) all |= e[u] | q[u][0][0] | q[u][1][0];
                if (lane == lane_with(all)) mbar_arrive(smem_u32(&sh.read[cs]));
                if (f >= 0 && !warp_wait(smem_u32(&sh.done[f]), fph, dead, a.err)) {
                    ok = false;
                    break;
                }
                if (mine) {
#pragma unroll
                    for (int u = 0; u < EACH; u++) {
                        const uint32_t sc = code_scale<DT>(e[u]);
#pragma unroll
                        for (int c = 0; c < 2; c++)
#pragma unroll
                            for (int p = 0; p < 2; p++) {          // eight codes -> 16 bytes
                                uint32_t r[4];
#pragma unroll
                                for (int d = 0; d < 4; d++) {
                                    const uint32_t x = q[u][c][2 * p + d / 2];
                                    r[d] = widen_codes<DT>(DT == 1 ? x : x ^ 0x80808080u, d & 1 ? 0x4342 : 0x4140, sc);
                                }
                                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                                             ::"r"(to + u * TOKENS * 128 + (col ^ (2 * c + p) * 16)), "r"(r[0]), "r"(r[1]),
                                             "r"(r[2]), "r"(r[3]) : "memory");
                            }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                if (!warp_wait(smem_u32(&sh.rows[rl]), rph, dead, a.err)) {
                    ok = false;
                    break;
                }
                if (sums) {
                    const uint32_t at = base + rs * ZERO_WG_A + (chunk >> 3) * 8192;
#pragma unroll 4
                    for (int k = tok0; k < ZERO_WG_TOK; k += GROUP / 16) {
                        uint32_t v[4];
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                     : "r"(at + k * 128 + (((chunk & 7) ^ (k & 7)) << 4)));
#pragma unroll
                        for (int c = 0; c < 4; c++) {
                            float lo, hi;
                            widen2<DT>(v[c], lo, hi);
                            total[c] = add2(total[c], pack2(lo, hi));
                        }
                    }
                }
                int one = 0;
                if (sums) {
                    uint32_t last = 0;
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        float lo, hi;
                        unpack2(total[c], lo, hi);
                        last |= __float_as_uint(lo);
                    }
                    one = lane_with(last);
                }
                // one lane arrives for all: their stores and proxy fences come before (a vote orders
                // no memory)
                __syncwarp();
                if (lane == one) arrive_first(smem_u32(&sh.ready[b]));
                b = (b + GROUPS) % ZERO_WG_WIDE;
                f += GROUPS;
                if (f >= ZERO_WG_WIDE * GROUPS) { f -= ZERO_WG_WIDE * GROUPS; fph ^= 1u; }
                cs = (cs + GROUPS) % ZERO_WG_CODES;
                cl += GROUPS;
                if (cl >= ZERO_WG_CODES * ZERO_WG_GROUPS) { cl -= ZERO_WG_CODES * ZERO_WG_GROUPS; cph ^= 1u; }
                rs = (rs + GROUPS) % ZERO_WG_STAGES;
                rl += GROUPS;
                if (rl >= ZERO_WG_STAGES * ZERO_WG_GROUPS) { rl -= ZERO_WG_STAGES * ZERO_WG_GROUPS; rph ^= 1u; }
            }
            skip = t - len;
            if (sums && ok) {
                // the two lanes of a warp with the same columns, then a row of 128 from each warp
                if (summed >= 1 && !warp_wait(smem_u32(&sh.col_empty), (uint32_t)(summed - 1) & 1u, dead, a.err)) break;
                float v[8];
#pragma unroll
                for (int c = 0; c < 4; c++) unpack2(total[c], v[2 * c], v[2 * c + 1]);
#pragma unroll
                for (int c = 0; c < 8; c++) v[c] += __shfl_xor_sync(0xFFFFFFFFu, v[c], 16);
                if (lane < 16) {
                    const uint32_t to = cols + (warp - 8) * 512 + chunk * 32;
#pragma unroll
                    for (int c = 0; c < 8; c += 4)
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to + 4 * c), "f"(v[c]), "f"(v[c + 1]),
                                     "f"(v[c + 2]), "f"(v[c + 3]) : "memory");
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.col_full));
                summed++;
            }
        }
    } else if (warp >= 4) {
        // ---- output: warp w has rows 32 (w - 4) + lane of this SM's half ----
        int summed = 0;
        float sum = 0.0f;
        for (int i = 0; wgrad_segment(a, pair, i, g); i++) {
            const int acc = i & 1;
            int64_t i0, j0;
            wgrad_place(a, g.tile, i0, j0);
            const int64_t r = i0 + rank * 128 + (warp - 4) * 32 + lane;
            // a wait that gave up in any lane leaves the whole warp without the sums
            bool have = __all_sync(0xFFFFFFFFu, pair_wait(smem_u32(&sh.sum_full[acc]), (uint32_t)(i >> 1) & 1u, dead, a.err));
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            float* part = g.slot < 0 ? nullptr : a.slots + (int64_t)g.slot * ZERO_WG_SLOT;
            // where the sums of a tile's or part's earlier runs are kept
            float* kept = wgrad_kept(g) ? a.slots + (int64_t)wgrad_slot(g, pair) * ZERO_WG_SLOT : nullptr;
            if (g.first) sum = part ? 0.0f : column_sum(a, r);
            if (adds_sums(a, j0)) {
                have = __all_sync(0xFFFFFFFFu, pair_wait(smem_u32(&sh.col_full), (uint32_t)summed & 1u, dead, a.err)) && have;
#pragma unroll
                for (int w = 0; w < ZERO_WG_WIDENERS / 32; w++) {
                    float x;
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x)
                                 : "r"(cols + w * 512 + ((warp - 4) * 32 + lane) * 4));
                    sum += x;
                }
                if (!have) sum = __uint_as_float(0x7FC00000u);
                if (lane == lane_with(__float_as_uint(sum))) mbar_arrive(smem_u32(&sh.col_empty));
                summed++;
            }
            if (g.last && part && adds_sums(a, j0))
                part[ZERO_WG_TILE * ZERO_WG_TILE + rank * 128 + (warp - 4) * 32 + lane] = sum;
            if (g.last && !part && a.db && j0 == 0 && r < a.n) put_grad(a.db, r, sum, a.grad_dtype, a.accumulate);
            const int width = wgrad_width(a, j0);
            for (int c = 0; c < width / 32; c++) {
                float v[32];
                __syncwarp();                                // a whole-warp instruction follows
                if (have) {
                    read_accumulator(tmem + acc * ZERO_WG_TILE + c * 32 + ((uint32_t)(warp - 4) << 21), v);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e++) v[e] = __uint_as_float(0x7FC00000u);
                }
                // four columns of 32 rows are one run of 512 bytes
                float4* o = reinterpret_cast<float4*>(kept) + ((rank * 4 + warp - 4) * 64 + c * 8) * 32 + lane;
                if (!g.first)
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const float4 p = __ldcg(o + e * 32);
                        v[4 * e] += p.x;
                        v[4 * e + 1] += p.y;
                        v[4 * e + 2] += p.z;
                        v[4 * e + 3] += p.w;
                    }
                if (g.last && !part) {
                    if (a.vec) put_row<DT, 32>(a, r, j0 + c * 32, v, sum);
                    else put_rows<DT>(a, r - lane, j0 + c * 32, v, sum, cols + ZERO_WG_SUMS + (warp - 4) * ZERO_WG_OUT);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++) o[e * 32] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) arrive_first(smem_u32(&sh.sum_empty[acc]));
        }
    }
    cluster_sync();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    cluster_sync();                          // the two SMs give the tensor memory back together
}

// Adds the parts of the cut tiles in token order and writes them out: a warp takes 32 rows and 16
// columns of a tile, or (DEEP) the eight warps of a block share their parts, add them and the
// eight sums in order.  That is for tiles of many parts, where a warp alone would wait for one
// load after another (a call on 41245 tokens, 64 x 128, 76 parts: 23 us instead of 41; with two
// parts a tile it costs 6 us at 8192 x 6400 x 1600).
template <int DT, bool DEEP>
__global__ void __launch_bounds__(256) k_wgrad_join(const __grid_constant__ WgradArgs a, const __grid_constant__ WgradJoin of)
{
    __shared__ __align__(16) float4 sums_of[DEEP ? 8 : 1][4][32];
    __shared__ float rows_of[DEEP ? 8 : 1][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t unit = DEEP ? blockIdx.x : blockIdx.x * 8 + warp;
    const int q = unit >> 7;
    const int strip = (unit >> 4) & 7, c = unit & 15;               // (SM, warp) of the rows; 16 columns
    const int first = of.second[q];
    int p0 = of.p0[q], p1 = of.p1[q];
    int64_t i0, j0;
    wgrad_place(a, (uint32_t)(a.waves * a.pairs + q), i0, j0);
    const int64_t r = i0 + strip * 32 + lane;
    if (p0 == p1 || j0 + c * 16 >= a.k) return;                     // not cut, or past the right edge
    const bool sums = adds_sums(a, j0);
    const int begin = p0;
    if (DEEP) {
        const int each = (p1 - p0 + 8) / 8;
        p0 += warp * each;
        p1 = p1 < p0 + each - 1 ? p1 : p0 + each - 1;
    }
    float v[16], sum = DEEP ? 0.0f : column_sum(a, r);
#pragma unroll
    for (int e = 0; e < 16; e++) v[e] = 0.0f;
#pragma unroll 4
    for (int p = p0; p <= p1; p++) {
        const float* part = a.slots + (int64_t)(2 * p + (p == begin ? first : 0)) * ZERO_WG_SLOT;
        const float4* s = reinterpret_cast<const float4*>(part) + (strip * 64 + c * 4) * 32 + lane;
        if (sums) sum += __ldcg(part + ZERO_WG_TILE * ZERO_WG_TILE + strip * 32 + lane);
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
#pragma unroll
        for (int e = 0; e < 4; e++) sums_of[warp][e][lane] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        rows_of[warp][lane] = sum;
        __syncthreads();
        if (warp > 0) return;
        sum = column_sum(a, r);
#pragma unroll
        for (int e = 0; e < 16; e++) v[e] = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; w++) {
            sum += rows_of[w][lane];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float4 f = sums_of[w][e][lane];
                v[4 * e] += f.x;
                v[4 * e + 1] += f.y;
                v[4 * e + 2] += f.z;
                v[4 * e + 3] += f.w;
            }
        }
    }
    if (a.db && j0 == 0 && c == 0 && r < a.n) put_grad(a.db, r, sum, a.grad_dtype, a.accumulate);
    put_row<DT, 16>(a, r, j0 + c * 16, v, sum);
}

// A first pass over dy where one is needed: its columns added over ZERO_WG_RANGES token
// ranges (blockIdx.y) for the norm's bias, which every tile's output needs (adding them in
// every tile would read each dy operand from shared memory once more, the product kernel's
// bound: 23 us more at 8192 x 6400 x 1600, this pass 18 us), and rows that are not aligned to
// 16 bytes copied to rows that are, so that TMA can read them.  A warp takes 256 columns.
template <int DT, bool COPY>
__global__ void __launch_bounds__(256) k_wgrad_columns(const __grid_constant__ WgradArgs a, uint16_t* out, int64_t pitch)
{
    __shared__ float part[8][256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t i0 = (int64_t)blockIdx.x * 256;
    const int64_t t0 = blockIdx.y * a.tokens / gridDim.y, t1 = (blockIdx.y + 1) * a.tokens / gridDim.y;
    float s[8];
#pragma unroll
    for (int c = 0; c < 8; c++) s[c] = 0.0f;
    // a lane's columns: eight neighbours, or where rows are not aligned four pairs 64 apart
    const int64_t i = i0 + (COPY ? 2 : 8) * lane;
#pragma unroll (COPY ? 4 : 8)
    for (int64_t t = t0 + warp; t < t1; t += 8) {
        const uint16_t* p = a.dy + t * a.ldy;
        uint32_t w[4] = {0, 0, 0, 0};
        if (COPY) {
#pragma unroll
            for (int c = 0; c < 4; c++) {
                if (i + 64 * c < a.n) w[c] = __ldg(p + i + 64 * c);
                if (i + 64 * c + 1 < a.n) w[c] |= (uint32_t)__ldg(p + i + 64 * c + 1) << 16;
                if (i + 64 * c < pitch) *reinterpret_cast<uint32_t*>(out + t * pitch + i + 64 * c) = w[c];
            }
        } else if (i + 8 <= a.n) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(p + i));
            w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
        } else {
#pragma unroll
            for (int c = 0; c < 8; c++)
                if (i + c < a.n) w[c / 2] |= (uint32_t)__ldg(p + i + c) << 16 * (c & 1);
        }
#pragma unroll
        for (int c = 0; c < 4; c++) {
            float lo, hi;
            widen2<DT>(w[c], lo, hi);
            s[2 * c] += lo;
            s[2 * c + 1] += hi;
        }
    }
    if (!a.sums) return;
#pragma unroll
    for (int c = 0; c < 8; c++) part[warp][COPY ? 64 * (c / 2) + 2 * lane + (c & 1) : 8 * lane + c] = s[c];
    __syncthreads();
    float v = 0.0f;
    for (int w = 0; w < 8; w++) v += part[w][threadIdx.x];
    if (i0 + threadIdx.x < a.n) a.sums[blockIdx.y * a.n + i0 + threadIdx.x] = v;
}

// ---- few tokens ----------------------------------------------------------------------
// A small product of few tokens is a matter of latency, of which the machinery above has 10 us:
// here a block takes 64 rows and 128 columns of dw, widens the tokens' codes and gradients to
// fp32 in shared memory, and each thread adds 8 rows of 4 columns in registers.  dy is read
// element by element, in any alignment.  768 x 768: 4.1 us for 16 tokens and 8.8 for 64, against
// 10.2; 1600 x 1600: 7.9 for 16 and 17.7 for 64, against 10; 4096 x 4096: 18 for one and 28 for
// 16, against 20.  So it is taken for up to ZERO_WG_FEW tokens and ZERO_WG_FEW_WORK products, and
// for up to four tokens and 32 M elements of dw.
template <int DT>
__global__ void __launch_bounds__(256) k_wgrad_few(const __grid_constant__ WgradArgs a)
{
    __shared__ __align__(16) float ys[ZERO_WG_FEW_TOK][64], xs[ZERO_WG_FEW_TOK][128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i0 = (int64_t)blockIdx.x * 64, stride = act_stride(a.k);
    for (int64_t j0 = (int64_t)blockIdx.y * 128; j0 < a.k; j0 += (int64_t)gridDim.y * 128) {
        f32x2_t v[8][2];
        float sum = 0.0f;                                   // lane r (of eight): row r's sum of dy
#pragma unroll
        for (int r = 0; r < 8; r++) v[r][0] = v[r][1] = pack2(0.0f, 0.0f);
        for (int t0 = 0; t0 < (int)a.tokens; t0 += ZERO_WG_FEW_TOK) {
            const int m = (int)a.tokens - t0 < ZERO_WG_FEW_TOK ? (int)a.tokens - t0 : ZERO_WG_FEW_TOK;
            __syncthreads();                                // the previous tokens' reads are done
            for (int e = threadIdx.x; e < m * 64; e += 256) {
                const int t = e >> 6, c = e & 63;
                ys[t][c] = i0 + c < a.n ? widen1<DT>(__ldg(a.dy + (t0 + t) * a.ldy + i0 + c)) : 0.0f;
            }
            for (int e = threadIdx.x; e < m * 16; e += 256) {
                const int t = e >> 4;
                const int64_t j = j0 + (e & 15) * 8;
                f32x2_t x[4];
#pragma unroll
                for (int c = 0; c < 4; c++) x[c] = pack2(0.0f, 0.0f);
                if (j < a.wide) {
                    const uint8_t* p = a.ckpt + (t0 + t) * stride;
                    const uint32_t b = __ldg(p + a.wide + (j >> 5));
                    act_values(__ldg(reinterpret_cast<const uint2*>(p + j)), b, x);
                    if (DT == 0 && (b < 103 || b > 136))    // fp16 has no such block
                        for (int c = 0; c < 4; c++) x[c] = both(__uint_as_float(0x7FC00000u));
                }
                float4* o = reinterpret_cast<float4*>(&xs[t][(e & 15) * 8]);
                float w[8];
#pragma unroll
                for (int c = 0; c < 4; c++) unpack2(x[c], w[2 * c], w[2 * c + 1]);
                o[0] = make_float4(w[0], w[1], w[2], w[3]);
                o[1] = make_float4(w[4], w[5], w[6], w[7]);
            }
            __syncthreads();
#pragma unroll 4
            for (int t = 0; t < m; t++) {
                const float4 x = *reinterpret_cast<const float4*>(&xs[t][4 * lane]);
                const f32x2_t x0 = pack2(x.x, x.y), x1 = pack2(x.z, x.w);
                const float4 y0 = *reinterpret_cast<const float4*>(&ys[t][8 * warp]);
                const float4 y1 = *reinterpret_cast<const float4*>(&ys[t][8 * warp + 4]);
                const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                for (int r = 0; r < 8; r++) {
                    v[r][0] = fma2(both(y[r]), x0, v[r][0]);
                    v[r][1] = fma2(both(y[r]), x1, v[r][1]);
                }
            }
            for (int t = 0; t < m; t++) sum += ys[t][8 * warp + (lane & 7)];
        }
        const int64_t j = j0 + 4 * lane;
        if (a.db && j0 == 0 && lane < 8 && i0 + 8 * warp + lane < a.n)
            put_grad(a.db, i0 + 8 * warp + lane, sum, a.grad_dtype, a.accumulate);
        float scale[4], shift[4];
#pragma unroll
        for (int c = 0; c < 4; c++) {
            scale[c] = a.scale && j + c < a.k ? widen1<DT>(__ldg(a.scale + j + c)) : 1.0f;
            shift[c] = a.shift && j + c < a.k ? widen1<DT>(__ldg(a.shift + j + c)) : 0.0f;
        }
#pragma unroll
        for (int r = 0; r < 8; r++) {
            const float s = __shfl_sync(0xFFFFFFFFu, sum, r);
            const int64_t i = i0 + 8 * warp + r;
            if (i >= a.n || j >= a.k) continue;
            float w[4];
            unpack2(v[r][0], w[0], w[1]);
            unpack2(v[r][1], w[2], w[3]);
#pragma unroll
            for (int c = 0; c < 4; c++) {
                if (a.scale) w[c] *= scale[c];
                if (a.shift) w[c] = __fmaf_rn(s, shift[c], w[c]);
            }
            const int64_t at = i * a.ldw + j;
            if (!a.vec || j + 4 > a.k) {
#pragma unroll
                for (int c = 0; c < 4; c++)
                    if (j + c < a.k) put_grad(a.dw, at + c, w[c], a.grad_dtype, a.accumulate);
            } else if (a.grad_dtype == 2) {
                float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.dw) + at);
                if (a.accumulate) {
                    const float4 p = *o;
                    w[0] += p.x; w[1] += p.y; w[2] += p.z; w[3] += p.w;
                }
                *o = make_float4(w[0], w[1], w[2], w[3]);
            } else {
                uint2* o = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dw) + at);
                if (a.accumulate) {
                    const uint2 p = *o;
                    float lo, hi;
                    widen2<DT>(p.x, lo, hi);
                    w[0] += lo; w[1] += hi;
                    widen2<DT>(p.y, lo, hi);
                    w[2] += lo; w[3] += hi;
                }
                *o = make_uint2(narrow2<DT>(w[0], w[1]), narrow2<DT>(w[2], w[3]));
            }
        }
    }
}

}  // namespace zero

using namespace zero;

namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool sizes_ok(int64_t tokens, int64_t n, int64_t k)
{
    return tokens >= 0 && tokens < (1ll << 31) && n >= 1 && n <= (1ll << 24) && k >= 1 && k <= ZERO_ACT_MAX_COLS &&
           n * k < (1ll << 46);              // tiles are counted in 32 bits
}

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t steps_of(int64_t tokens) { return up(tokens, ZERO_WG_TOK); }

// Whether a call on so many stages keeps sums in the workspace: only then are tiles cut into parts,
// or their stages into runs, and only then does the workspace have slots.  Below, one run of at
// most 15 stages (60 steps) is off by about 1e-6 where runs of 12 would be by 8e-7.
bool keeps_sums(int64_t steps) { return steps >= 2 * ZERO_WG_PART; }

// Workspace: the status word (256 bytes), the columns' sums, the parts and runs' sums, dy's copy.
int64_t round_bytes(int64_t b) { return up(b, 256) * 256; }
int64_t sums_bytes(int64_t n) { return round_bytes(ZERO_WG_RANGES * n * 4); }
int64_t parts_bytes(int64_t tokens)
{
    return keeps_sums(steps_of(tokens)) ? round_bytes((int64_t)ZERO_WG_SLOTS * ZERO_WG_SLOT * 4) : 0;
}
int64_t copy_bytes(int64_t tokens, int64_t n) { return round_bytes(tokens * up(n, 8) * 16); }

// The division of a.tokens, a.n and a.k among `pairs` pairs of SMs (units of the last wave: below
// 80 * 2^25).
void divide(WgradArgs& a, int pairs)
{
    a.pairs = pairs;
    a.steps = (int)steps_of(a.tokens);
    a.run = !keeps_sums(a.steps) ? (uint32_t)a.steps : a.grad_dtype == ZERO_FP32 ? ZERO_WG_RUN : ZERO_WG_RUN_16;
    a.tiles_n = (uint32_t)up(a.n, ZERO_WG_TILE);
    a.tiles_k = (uint32_t)up(a.k, ZERO_WG_TILE);
    const int64_t tiles = (int64_t)a.tiles_n * a.tiles_k;
    a.waves = (int)(tiles / a.pairs);
    a.rest = (int)(tiles % a.pairs);
    a.rest_pairs = a.rest;
    const int64_t units = (int64_t)a.rest * a.steps;
    if (a.rest > 0 && keeps_sums(a.steps)) {
        const int64_t parts = units / ZERO_WG_PART;
        a.rest_pairs = (int)(parts < a.rest ? a.rest : parts < a.pairs ? parts : a.pairs);
    }
    if (a.rest > 0) {
        a.share = (uint32_t)(units / a.rest_pairs);
        a.extra = (uint32_t)(units % a.rest_pairs);
    }
}

decltype(&cuTensorMapEncodeTiled) encode()
{
    static decltype(&cuTensorMapEncodeTiled) fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(p);
    }();
    return fn;
}

bool tensor_map(CUtensorMap* m, CUtensorMapDataType type, const void* p, int64_t cols, int64_t rows, int64_t pitch,
                int box_cols, int box_rows, CUtensorMapSwizzle swizzle)
{
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return encode()(m, type, 2, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of SMs that run a launch's clusters at the same time; 0: a CUDA call failed.
int device_pairs()
{
    static std::mutex lock;
    static int pairs[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> hold(lock);
    if (pairs[dev] == 0) {
        for (const void* fn : {(const void*)k_wgrad<0>, (const void*)k_wgrad<1>})
            if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, ZERO_WG_SMEM) != cudaSuccess)
                return 0;
        cudaLaunchConfig_t c{};
        c.gridDim = dim3(2 * ZERO_WG_PAIRS);
        c.blockDim = dim3(ZERO_WG_THREADS);
        c.dynamicSmemBytes = ZERO_WG_SMEM;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = 2;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        c.attrs = &at;
        c.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, (const void*)k_wgrad<1>, &c) != cudaSuccess) return 0;
        pairs[dev] = n < 1 ? 1 : n > ZERO_WG_PAIRS ? ZERO_WG_PAIRS : n;
    }
    return pairs[dev];
}

bool launch(const void* fn, dim3 grid, int threads, int smem, void** args, void* stream)
{
    return cudaLaunchKernel(fn, grid, dim3(threads), args, smem, static_cast<cudaStream_t>(stream)) == cudaSuccess;
}

}  // namespace

extern "C" uint64_t zero_act_wgrad_workspace(int64_t tokens, int64_t n, int64_t k)
{
    if (!sizes_ok(tokens, n, k)) return 0;
    return (uint64_t)(256 + sums_bytes(n) + parts_bytes(tokens) + copy_bytes(tokens, n));
}

extern "C" zero_status_t zero_act_wgrad(zero_dtype_t dtype, const void* dy, int64_t tokens, int64_t n,
                                        int64_t ldy, const void* ckpt, int64_t k, const void* col_scale,
                                        const void* col_shift, zero_dtype_t grad_dtype, void* dw, int64_t ldw,
                                        void* db, int accumulate, void* work, void* stream)
{
    TraceRange trace_("zero_act_wgrad");
    if ((dtype != ZERO_FP16 && dtype != ZERO_BF16) || (grad_dtype != dtype && grad_dtype != ZERO_FP32))
        return ZERO_EINVAL;
    if (!sizes_ok(tokens, n, k) || ldw < k || ldw > (1ll << 31)) return ZERO_EINVAL;
    const int64_t ge = grad_dtype == ZERO_FP32 ? 4 : 2;
    if (!dw || !aligned_to(dw, ge) || !aligned_to(db, ge) || !work || !aligned_to(work, 16) ||
        !aligned_to(col_scale, 2) || !aligned_to(col_shift, 2))
        return ZERO_EINVAL;
    if (tokens > 0 && (!dy || !aligned_to(dy, 2) || ldy < n || ldy > (1ll << 31) || !ckpt ||
                       !aligned_to(ckpt, 16)))
        return ZERO_EINVAL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (tokens == 0) {
        if (accumulate) return ZERO_OK;
        if (cudaMemset2DAsync(dw, ldw * ge, 0, k * ge, n, st) != cudaSuccess) return ZERO_ECUDA;
        if (db && cudaMemsetAsync(db, 0, n * ge, st) != cudaSuccess) return ZERO_ECUDA;
        return ZERO_OK;
    }
    WgradArgs a{};
    a.dy = static_cast<const uint16_t*>(dy);
    a.ckpt = static_cast<const uint8_t*>(ckpt);
    a.scale = static_cast<const uint16_t*>(col_scale);
    a.shift = static_cast<const uint16_t*>(col_shift);
    a.dw = dw;
    a.db = db;
    a.err = static_cast<int32_t*>(work);
    char* at = static_cast<char*>(work) + 256;
    if (col_shift && k > ZERO_WG_TILE) a.sums = reinterpret_cast<float*>(at);
    at += sums_bytes(n);
    a.slots = reinterpret_cast<float*>(at);
    at += parts_bytes(tokens);
    a.tokens = tokens; a.n = n; a.k = k; a.ldy = ldy; a.ldw = ldw;
    a.wide = act_wide(k);
    a.grad_dtype = grad_dtype;
    a.accumulate = accumulate != 0;
    a.vec = aligned_to(dw, 16) && ldw * ge % 16 == 0;
    a.vec_s = aligned_to(col_scale, 16) && aligned_to(col_shift, 16);
    const bool half = dtype == ZERO_FP16;
    void* args[] = {&a, nullptr, nullptr, nullptr};
    if ((tokens <= ZERO_WG_FEW && tokens * n * k <= ZERO_WG_FEW_WORK) || (tokens <= 4 && n * k <= 32 << 20)) {
        const int64_t wide = up(k, 128);
        return launch(half ? (const void*)k_wgrad_few<0> : (const void*)k_wgrad_few<1>,
                      dim3((unsigned)up(n, 64), (unsigned)(wide < 32768 ? wide : 32768)), 256, 0, args, stream)
                   ? ZERO_OK
                   : ZERO_ECUDA;
    }
    const int pairs = device_pairs();
    if (pairs == 0 || !encode()) return ZERO_ECUDA;
    divide(a, pairs);
    WgradJoin join{};
    if (a.rest > 0) {
        for (int p = a.rest_pairs - 1; p >= 0; p--) {       // backwards: a tile's first pair is written last
            const uint32_t t0 = wgrad_share(a, p) / a.steps, t1 = (wgrad_share(a, p + 1) - 1) / a.steps;
            for (uint32_t t = t0; t <= t1; t++) {
                if (join.p1[t] == 0) join.p1[t] = (uint8_t)p;
                join.p0[t] = (uint8_t)p;
                join.second[t] = t > t0;
            }
        }
    }
    CUtensorMap my, mc, me;
    const int64_t stride = act_stride(k);
    const bool copy = !aligned_to(dy, 16) || ldy % 8 != 0;
    if (copy || a.sums) {
        uint16_t* out = reinterpret_cast<uint16_t*>(at);
        int64_t pitch = up(n, 8) * 8;
        const void* fn = copy ? (half ? (const void*)k_wgrad_columns<0, true> : (const void*)k_wgrad_columns<1, true>)
                              : (half ? (const void*)k_wgrad_columns<0, false> : (const void*)k_wgrad_columns<1, false>);
        void* first[] = {&a, &out, &pitch};
        // sums: one wave of blocks (three an SM); a copy: four (195 -> 182 us for a call on 8192 x
        // 6401 x 1600); at least 32 tokens a block
        const int64_t wide = up(n, 256), most = up(tokens, 32), fill = (copy ? 24ll : 6ll) * a.pairs / wide;
        a.ranges = (int)(fill < 1 ? 1 : fill < most ? fill : most);
        if (a.sums && a.ranges > ZERO_WG_RANGES) a.ranges = ZERO_WG_RANGES;
        if (!launch(fn, dim3((unsigned)wide, (unsigned)a.ranges), 256, 0, first, stream)) return ZERO_ECUDA;
        if (copy) {
            dy = out;
            ldy = pitch;
        }
    }
    if (!tensor_map(&my, CU_TENSOR_MAP_DATA_TYPE_UINT16, dy, n, tokens, ldy * 2, 64, ZERO_WG_TOK, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !tensor_map(&mc, CU_TENSOR_MAP_DATA_TYPE_UINT8, ckpt, stride, tokens, stride, 128, ZERO_WG_TOK, CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !tensor_map(&me, CU_TENSOR_MAP_DATA_TYPE_UINT8, ckpt, stride, tokens, stride, 16, ZERO_WG_TOK, CU_TENSOR_MAP_SWIZZLE_NONE))
        return ZERO_ECUDA;
    args[1] = &my;
    args[2] = &mc;
    args[3] = &me;
    const int run = a.waves > 0 ? a.pairs : a.rest_pairs;
    if (!launch(half ? (const void*)k_wgrad<0> : (const void*)k_wgrad<1>, dim3(2 * run), ZERO_WG_THREADS, ZERO_WG_SMEM, args,
                stream))
        return ZERO_ECUDA;
    if (a.rest_pairs > a.rest) {
        const bool deep = a.rest_pairs >= ZERO_WG_DEEP * a.rest;
        const void* const joins[2][2] = {{(const void*)k_wgrad_join<1, false>, (const void*)k_wgrad_join<1, true>},
                                         {(const void*)k_wgrad_join<0, false>, (const void*)k_wgrad_join<0, true>}};
        void* last[] = {&a, &join};
        if (!launch(joins[half][deep], dim3(a.rest * (deep ? 128 : 16)), 256, 0, last, stream)) return ZERO_ECUDA;
    }
    return ZERO_OK;
}
