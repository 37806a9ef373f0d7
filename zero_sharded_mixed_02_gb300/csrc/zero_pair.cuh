// zero_pair.cuh -- what kernels on pairs of SMs (clusters of two blocks) share: barriers of the
// pair, TMA boxes, products into tensor memory and the way back.
#pragma once

#include <cuda.h>

#include "zero_b200.h"
#include "zero_tma.cuh"

namespace zero {

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
template <uint32_t LIMIT>
static __device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity, volatile int* dead, int32_t* err)
{
    for (uint32_t it = 0; it < LIMIT; it++) {
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
template <uint32_t LIMIT>
static __device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* dead, int32_t* err)
{
    if (LIMIT > 0 && __all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
#pragma unroll 1
    for (uint32_t it = 0; it < LIMIT; it++) {
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

}  // namespace zero
