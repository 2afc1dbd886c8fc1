// Pieces shared by the whole-head scans of the gated delta rule (gdn_chain.cu, gdn_rchain.cu): a thread has 32
// values of one value column (a lane of tensor memory).
#pragma once

#include "gdn_tc.cuh"
#include "tc.cuh"

namespace kda {
namespace gdn {

using namespace tc;

constexpr int PANEL = C * 128;            // 64 tokens x 64 values, bf16
constexpr uint32_t NEG = 1u << 13;        // in an MMA's descriptor: minus A

// 32 fp32 values of a thread as N bf16 planes, x = p0 - p1 (+ p2): the second has the opposite sign (its
// MMAs negate it)
template <int N>
__device__ __forceinline__ void planes_of(const float (&x)[32], uint32_t (&p)[N][16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            p[n][i] = pack(a, b);
            if (n + 1 < N) {
                a = less((uint16_t)p[n][i], a);
                b = less((uint16_t)(p[n][i] >> 16), b);
            }
        }
    }
}
__device__ __forceinline__ void store32(uint32_t taddr, const float (&x)[32])
{
    uint32_t m[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) m[i] = __float_as_uint(x[i]);
    tmem_st32u_nowait(taddr, m);
}
// x *= 32 factors in shared memory
__device__ __forceinline__ void scale32(float (&x)[32], const float* f)
{
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const float4 v = *(const float4*)(f + i);
        x[i] *= v.x; x[i + 1] *= v.y; x[i + 2] *= v.z; x[i + 3] *= v.w;
    }
}
// 32 bf16 values of a row, to a tile of ROWS rows (sign: 0x80008000 to negate them)
template <int ROWS>
__device__ __forceinline__ void to_tile(char* tile, int row, int piece, const uint32_t (&p)[16], uint32_t sign = 0)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *(uint4*)(tile + state_at(row, piece + i, ROWS)) =
            make_uint4(p[4 * i] ^ sign, p[4 * i + 1] ^ sign, p[4 * i + 2] ^ sign, p[4 * i + 3] ^ sign);
}
// COLS columns of planes that the thread has put into tensor memory, to a tile of ROWS rows
template <int ROWS, int COLS>
__device__ __forceinline__ void planes_to_tile(uint32_t taddr, char* tile, int row, int piece, bool real, uint32_t sign)
{
#pragma unroll
    for (int i = 0; i < COLS / 16; ++i) {
        float x[16];
        uint32_t p[16];
        tmem_ld16(taddr + i * 16, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) p[j] = __float_as_uint(x[j]);
        if (real) to_tile<ROWS>(tile, row, piece + i * 4, p, sign);
    }
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void prefetch_3d(const CUtensorMap* map, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(c0),
                 "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void prefetch(const void* src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

}  // namespace gdn
}  // namespace kda
