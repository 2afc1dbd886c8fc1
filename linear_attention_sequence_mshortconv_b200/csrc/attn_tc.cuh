// Pieces shared by the tensor-core kernels of causal attention: tensor maps of 128-byte
// swizzled tiles, their MMA descriptors, bounded waits.
#pragma once

#include <algorithm>

#include "mixers.h"
#include "sm100.cuh"

namespace kda {
namespace attn {

using namespace sm100;

constexpr uint64_t kWaitNs = 2000000000ull;   // a wait that lasts longer is reported and given up
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---- waits ------------------------------------------------------------------------------
// The first wait that runs out raises the CTA's flag and records DEV_TIMEOUT; from then on no
// wait waits, no copy is issued, and every role runs to its end (MMAs still issued work on whatever
// is there).  Warps that use warp-wide instructions or barriers keep their loops whole: the flag
// is seen by lanes at different times.
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
// After a timeout: the copies issued into a ring (the last STAGES of `issued`) land before the
// CTA leaves.
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
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

// ---- tiles of a launch --------------------------------------------------------------------
// The query heads that share a key/value head are rows of one matrix: row i is token i / r, head
// i % r of the group (r = H / Hkv).  A launch has one CTA per tile of R rows (or keys, r = 1) and
// key/value head.  Tiles of one sequence differ in work from none to the whole sequence, so they
// start in order of it, or a heavy one that comes last runs alone: equal rows tile by tile, packed
// samples from the longest on, all heads of a tile together.
struct Tiles {
    int n, heads;
    int per;                       // >= 0: equal rows of `per` tiles; < 0: packed
    uint8_t seq[kMaxSeqs];         // samples by length
    int32_t first[kMaxSeqs + 1];   // their first tiles
    // CTA -> head, sequence and how many tiles of the sequence start before this one
    __device__ __forceinline__ void locate(int block, int& head, int& s, int& rank) const
    {
        head = block % heads;
        const int b = block / heads;
        if (per >= 0) {
            s = b % n;
            rank = b / n;
            return;
        }
        int lo = 0, hi = n - 1;   // the last sample whose first tile is <= b
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= b) lo = mid; else hi = mid - 1;
        }
        s = seq[lo];
        rank = b - first[lo];
    }
};
inline int tiles_of(int len, int r, int R) { return (int)(((int64_t)len * r + R - 1) / R); }
// returns the number of CTAs
inline int64_t make_tiles(Tiles& t, const Seqs& s, int heads, int r, int R)
{
    t.n = s.n;
    t.heads = heads;
    if (s.T >= 0) {
        t.per = tiles_of(s.T, r, R);
        return (int64_t)t.per * s.n * heads;
    }
    t.per = -1;
    for (int i = 0; i < s.n; ++i) t.seq[i] = (uint8_t)i;
    std::sort(t.seq, t.seq + s.n, [&](uint8_t x, uint8_t y) { return s.len(x) != s.len(y) ? s.len(x) > s.len(y) : x < y; });
    t.first[0] = 0;
    for (int i = 0; i < s.n; ++i) t.first[i + 1] = t.first[i] + tiles_of(s.len(t.seq[i]), r, R);
    return (int64_t)t.first[s.n] * heads;
}
// Rows of one sequence and group: the offset of row i in a [tokens, H, D] tensor.  A tensor that
// fits the device has fewer than 2^32 rows of 64 values, so rows count in 32 bits.
struct RowAt {
    int64_t t0;       // first token
    int H, h0, r, D;  // heads, the group's first, the group's
    __device__ __forceinline__ int64_t operator()(uint32_t i) const { return ((t0 + i / r) * H + h0 + i % r) * D; }
};
// A thread's row (of 128, to a warp 32) of a finished D-column accumulator, scaled, to memory: 16-byte
// pieces through a tile of shared memory, so that a warp writes whole rows.  off: the row's offset,
// negative for a row that is not written.
template <int D>
__device__ __forceinline__ void store_rows(uint32_t taddr, float f, char* tile, __nv_bfloat16* dst, int64_t off, int row)
{
    constexpr int P = D / 8;
    const int lane = threadIdx.x & 31;
    auto at = [&](int r, int piece) { return tile + r * (2 * D) + (((piece & ~7) | ((piece ^ r) & 7)) << 4); };
#pragma unroll
    for (int x = 0; x < D; x += 32) {
        float v[32];
        tmem_ld32(taddr + x, v);
#pragma unroll
        for (int y = 0; y < 32; y += 8)
            *(uint4*)at(row, (x + y) / 8) = make_uint4(pack_bf16(v[y] * f, v[y + 1] * f), pack_bf16(v[y + 2] * f, v[y + 3] * f),
                                                       pack_bf16(v[y + 4] * f, v[y + 5] * f), pack_bf16(v[y + 6] * f, v[y + 7] * f));
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const int r = k * (32 / P) + lane / P;   // of the warp's 32
        const int64_t o = __shfl_sync(~0u, off, r);
        if (o >= 0) *(uint4*)(dst + o + (lane % P) * 8) = *(const uint4*)at((row & ~31) + r, lane % P);
    }
}

}  // namespace attn
}  // namespace kda
