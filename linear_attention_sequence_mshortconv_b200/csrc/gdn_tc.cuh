// Pieces shared by the tensor-core kernels of the gated delta rule: bf16 warp MMAs, values
// split over bf16 planes, swizzled tiles, and the record of a chunk's factors.
#pragma once

#include "mixers.h"
#include "sm100.cuh"

namespace kda {
namespace gdn {

using namespace sm100;

constexpr int C = 64;          // tokens per chunk
// bf16 planes of the MMA operands that are not inputs.  Three carry fp32's 24 bits, two 16 to 17.
// What enters the state directly (Y = beta o R and U) has three.  Two are enough for S in K S and
// for T: their rounding (2^-18) reaches U only through K S, a fraction of V, and through T's
// off-diagonal entries, beta k_i.k_j.
// P and U in P U have two as well: the sum over a chunk's tokens may cancel (with keys that repeat, U
// holds the differences of successive values).
constexpr int PLANES = 3, SPL = 2, TPL = 2, PPL = 2;

// D(16x8, fp32) += A(16x16, bf16, rows) * B(16x8, bf16, columns)
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi)   // bf16 pair, round to nearest even
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float low(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float high(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }
// A pair of fp32 values as N bf16 planes: x = p0 + p1 + ..., each plane the rounded rest of
// the ones before, so N planes leave 2^-(9N) of x (N = 3: less than fp32's own half step).
__device__ __forceinline__ float less(uint16_t a, float b)   // a - b, in one instruction
{
    float r;
    asm("sub.rn.f32.bf16 %0, %1, %2;" : "=f"(r) : "h"(a), "f"(b));
    return r;
}
template <int N>
__device__ __forceinline__ void split(float a, float b, uint32_t (&p)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p[i] = pack(a, b);
        if (i + 1 < N) {   // minus the rest
            a = less((uint16_t)p[i], a);
            b = less((uint16_t)(p[i] >> 16), b);
        }
    }
    if (N > 1) p[1] ^= 0x80008000u;
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) { ldsm_x4(r, addr); }
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) { ldsm_x4_t(r, addr); }
// transposing store of four 8x8 blocks: lane l gives the address of one 16-byte row
__device__ __forceinline__ void stsm_t(uint32_t addr, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
// 16 bytes global -> shared, or 16 zero bytes
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Tiles of rows of W values (bf16, W = 32, 64 or 128): the 16-byte pieces of a row are
// permuted by the row's low bits, so 8 rows of one piece lie in 8 different bank groups
// for ldmatrix.
template <int W>
__device__ __forceinline__ uint32_t tile_at(int row, int piece)
{
    return row * (2 * W) + ((piece ^ (W == 32 ? (row >> 1) & 3 : row & 7)) << 4);
}
// A tile of a state, `rows` rows of W values: panels of 64 values, a row of a panel 128 bytes, its pieces
// permuted as above (the 128-byte swizzle of the copy engine and of tcgen05's operands).
__device__ __forceinline__ uint32_t state_at(int row, int piece, int rows)
{
    return ((piece >> 3) * rows + row) * 128 + (((piece & 7) ^ (row & 7)) << 4);
}
template <int W, int THREADS, int ROWS = C>
__device__ __forceinline__ void load_tile(uint32_t dst, const __nv_bfloat16* src, int64_t row_stride, int valid, int tid)
{
    constexpr int P = W / 8;
#pragma unroll
    for (int i = 0; i < ROWS * P / THREADS; ++i) {
        const int e = i * THREADS + tid, row = e / P, piece = e % P;
        const bool in = row < valid;
        cp16(dst + tile_at<W>(row, piece), src + (in ? row : 0) * row_stride + piece * 8, in);
    }
}

// A chunk's factors for one value head, written by the prologue kernel and read by the scans:
// T = (I + A)^-1 in TPL planes and P = lower(e^{cum_i - cum_j} q_i.k_j) in PPL planes, each
// the ten 16x16 blocks on and below the diagonal, a block as four 8x8 core matrices of 128
// contiguous bytes, and two of zeros; then e^cum, e^{cum_C - cum}, beta, and cum log2(e) as a sum of two floats.
constexpr int BLK = 512;
constexpr int TRI = 12 * BLK;
constexpr int REC_P = TPL * TRI, REC_SCAL = (TPL + PPL) * TRI, REC_BYTES = REC_SCAL + 5 * C * 4;
// Blocks column by column, with zeros before (1, 1) and (3, 3), that is, as (0, 1) and (2, 3): the two
// blocks that any column has in one half of the rows lie side by side, as an MMA needs.
__host__ __device__ constexpr int blk(int ib, int jb) { return (ib + (jb ? 2 + 2 * jb : 0)) * BLK; }

// What the backward keeps of each chunk and value head, bf16: the entry state S^T and the
// gradient D^T of the exit state, [Dv][Dk] in two planes each; U^T, [Dv][64] in two planes, R^T,
// [Dv][64], and dY^T, [Dv][64] in two planes; every plane as the tile (state_at; of 64 values tile_at, which is
// the same) that the gradients' kernel reads.
struct Kept {
    int Dk, Dv;
    __host__ __device__ size_t state() const { return (size_t)Dv * Dk * 2; }     // bytes of a plane
    __host__ __device__ size_t rows() const { return (size_t)Dv * C * 2; }
    __host__ __device__ size_t s() const { return 0; }
    __host__ __device__ size_t d() const { return 2 * state(); }
    __host__ __device__ size_t u() const { return 4 * state(); }
    __host__ __device__ size_t r() const { return u() + 2 * rows(); }
    __host__ __device__ size_t y() const { return r() + rows(); }
    __host__ __device__ size_t bytes() const { return y() + 2 * rows(); }
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

// The same scan with all value columns of a head in one CTA (Dv = 64 or 128)
cudaError_t launch_chain(const GdnArgs& a, const Seqs& s, const void* records, void* kept, int* status, cudaStream_t st);
// and the reverse scan (D and dY kept)
cudaError_t launch_rchain(const GdnBwdArgs& b, const Seqs& s, const void* records, void* kept, int* status, cudaStream_t st);
// the gradients of q, k, g and beta (Dv = 64 or 128)
cudaError_t launch_grads(const GdnBwdArgs& b, const Seqs& s, const void* records, void* kept, int sms, int* status, cudaStream_t st);
bool whole_heads(const GdnArgs& a, const Seqs& s, int sms);   // which of the two
// The forward over pieces of long samples: chunks to a piece (0: not worth it), bytes, launch
int piece_chunks(const Seqs& s, int Hv, int Dk, int Dv, int sms);
size_t pieces_workspace(const Seqs& s, int Hv, int Dk, int Dv, int per);
cudaError_t launch_pieces(const GdnArgs& a, const Seqs& s, void* ws, int per, int* status, cudaStream_t st);
// launch of the forward scan: o and S_T (kept null), or what the backward needs (kept and, if
// not null, S_T; o unused)
cudaError_t launch_scan(const GdnArgs& a, const Seqs& s, const void* records, void* kept, int sms, cudaStream_t st);
// launch of the prologue kernel: one record per (slot, value head)
cudaError_t launch_prologue(const GdnArgs& a, const Seqs& s, void* records, cudaStream_t st);

}  // namespace gdn
}  // namespace kda
