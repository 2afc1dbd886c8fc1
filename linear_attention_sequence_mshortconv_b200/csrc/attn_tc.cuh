// Pieces shared by the tensor-core kernels of causal attention: the order of their tiles, and rows
// of a query group.
#pragma once

#include <algorithm>

#include "tc.cuh"

namespace kda {
namespace attn {

using namespace tc;

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

// Whether 128 rows (token x head of the group) are whole tokens, so that they are a box of the [tokens, H, D]
// tensor: such tiles come and go by the copy engine.  (By the threads a 64 KB tile took 2.6 us to ask for, and 1.5 to
// store, of a CTA with 8 blocks of keys.  Forward by the threads, then by boxes: 512 tokens 15.5 and 14.1 us, 4 rows of 4352
// 270 and 261, 16384 tokens 810 and 816, where it hardly counts; the backward's rows at 4 x 4352 422 and 405.)
inline bool box_rows(int r) { return r <= 128 && 128 % r == 0; }

// As store_rows, of a tile of 128 whole rows, by the copy engine: 128 threads, barrier `bar`; token: the tile's first.
template <int D>
__device__ __forceinline__ void store_box(uint32_t taddr, float f, char* tile, const CUtensorMap* map, int head, int token, int row, int bar)
{
#pragma unroll
    for (int x = 0; x < D; x += 32) {
        float v[32];
        tmem_ld32(taddr + x, v);
#pragma unroll
        for (int y = 0; y < 32; y += 8)
            *(uint4*)(tile + (x >> 6) * 128 * 128 + piece_at(row, ((x + y) & 63) / 8)) =
                make_uint4(pack_bf16(v[y] * f, v[y + 1] * f), pack_bf16(v[y + 2] * f, v[y + 3] * f),
                           pack_bf16(v[y + 4] * f, v[y + 5] * f), pack_bf16(v[y + 6] * f, v[y + 7] * f));
    }
    fence_async_smem();
    asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");
    if (row == 0) {
        for (int p = 0; p < D / 64; ++p) store_3d(map, tile + p * 128 * 128, p * 64, head, token);
        bulk_commit();
        bulk_wait_read0();
    }
}

}  // namespace attn
}  // namespace kda
