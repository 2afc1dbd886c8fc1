// Pieces shared by the tcgen05 kernels of the gated delta rule and of causal attention: bounded
// waits, MMA descriptors of 128-byte swizzled tiles, issue by an elected lane, packed arithmetic.
#pragma once

#include "mixers.h"
#include "sm100.cuh"

namespace kda {
namespace tc {

using namespace sm100;

constexpr uint64_t kWaitNs = 2000000000ull;   // a wait that lasts longer is reported and given up
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---- waits ------------------------------------------------------------------------------
// The first wait that runs out raises the CTA's flag and records DEV_TIMEOUT; from then on no
// wait waits, no copy is issued, and every role runs to its end (MMAs still issued work on whatever
// is there).  Warps that use warp-wide instructions or barriers keep their loops whole: the flag
// is seen by lanes at different times.  Nothing may be in flight when the CTA leaves, and a wait may run out
// after a role has ended: so whoever issues copies or MMAs waits for its last ones at its end, whether
// the flag is up or not (they need nothing from anyone, so the wait is short).
//
// Test hook (the kernels' `drop`): one barrier of a kernel expects the arrivals of a warp more than there are, so the
// wait for it runs out.  A whole warp's where all lanes of a warp arrive at once: a phase must not turn within such an
// arrival (128 + 1 ended in a launch failure; without the hook every count is a multiple of what arrives together).
struct Guard {
    volatile int* flag;
    int* status;
    __device__ __forceinline__ bool up() const { return *flag != 0; }
};
static __device__ __noinline__ void wait_slow(uint64_t* bar, uint32_t parity, Guard g)
{
    const uint64_t t0 = globaltimer_ns();
    while (!g.up()) {
        if (mbar_try_wait_sleep(bar, parity, 20000u)) return;
        if (globaltimer_ns() - t0 > kWaitNs) {
            *g.flag = 1;
            atomicCAS(g.status, DEV_OK, DEV_TIMEOUT);
        }
    }
}
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, const Guard& g)
{
    if (!mbar_try_wait(bar, parity)) wait_slow(bar, parity, g);
}

// Whole-warp form for code with warp-wide instructions: the same answer in every lane.
__device__ __forceinline__ bool warp_up(const Guard& g) { return __any_sync(~0u, g.up()); }
// The copies issued into a ring (the last STAGES of `issued`) have landed.
__device__ __forceinline__ void drain_ring(uint64_t* full, int stages, int issued)
{
    for (int j = issued > stages ? issued - stages : 0; j < issued; ++j)
        mbar_wait_bounded(full + j % stages, (j / stages) & 1, kWaitNs);
}

// ---- tiles ------------------------------------------------------------------------------
// A tile of R rows x D values (bf16): D / 64 panels of R x 64, a row of a panel 128 bytes, its
// eight 16-byte pieces permuted by the row's low three bits (the 128-byte swizzle of the
// copy engine and of the MMA's descriptors).  Panels start on 1024-byte boundaries.
__device__ __forceinline__ uint32_t piece_at(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }

// rows as M or N, values as K ("K-major"): 8 rows x 128 bytes is one unit, 1024 bytes apart
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr)
{
    return sdesc(addr, 16, 1024) | (2ull << 61);
}
// values as M or N, rows as K ("MN-major"): 64 values x 8 rows is one unit; units 1024 bytes apart
// along the rows, a panel apart along the values
__device__ __forceinline__ uint64_t desc_cols(uint32_t addr, uint32_t panel)
{
    return sdesc(addr, panel, 1024) | (2ull << 61);
}

// One lane of a converged warp, the same each time.  The issuing warps run their loops whole and
// let one lane issue: the descriptors then stay in uniform registers, where an MMA takes them
// from (inside a one-lane branch each would be moved there first, about 100 cycles an MMA).
__device__ __forceinline__ bool elect()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(~0u, (int)(threadIdx.x >> 5), 0); }
// The MMAs that the warp has issued have ended; bar: used for nothing else.
__device__ __forceinline__ void drain_mma(uint64_t* bar)
{
    __syncwarp();
    if (elect()) umma_commit(bar);
    mbar_wait_bounded(bar, 0, kWaitNs);
}
// K-step x (16 values) of an operand whose values are K, and of one whose rows are K
__device__ __forceinline__ uint64_t step_rows(uint64_t desc, int x, uint32_t panel)
{
    return desc + (((x >> 2) * panel + (x & 3) * 32) >> 4);
}
__device__ __forceinline__ uint64_t step_cols(uint64_t desc, int x) { return desc + ((x * 2048) >> 4); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Pairs of fp32 in one instruction, and a maximum of three.
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(smem_addr(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

}  // namespace tc
}  // namespace kda
