// Gradients of the gated delta rule on the tensor cores (bf16; Dk = 64 or 128).
//
// Four launches: the prologue (T, P, gates) and the forward scan again, which keeps every
// chunk's entry state S, U and R; a reverse scan, a chain like the forward's (here by columns of heads, in
// gdn_rchain.cu by whole heads; the forward scan's rule says which),
//   dU = P^T dO + e^{cum_C - cum} o (K D),  dY = T^T dU,  dV = beta o dY,
//   D' = e^{cum_C} D + Q^T (e^cum o dO) - K^T (e^cum o dV)
// with D the gradient of the chunk's exit state and D' that of its entry state, which keeps D and
// dY; and a kernel without a chain, one CTA per chunk and key head, for the sums over the value
// columns:
//   N = e^{cum_i - cum_j} o lower(dO U^T),  M = -e^{cum_i - cum_j} o strict_lower(dY U^T)
//   dQ = e^cum o (dO S^T) + N K
//   dK = row + col,  row = beta o (M K - e^cum o (dY S^T)),
//                    col = (beta M)^T K + N^T Q + e^{cum_C - cum} o (U D^T)
//   dbeta_i = dY_i . R_i + sum_j M_ij k_i.k_j
//   dcum_i = q_i.dQ_i + k_i.row_i - k_i.col_i,  dg_i = sum_{j >= i} dcum_j + <S', D>
// where S' is the chunk's exit state: scaling it is what a gate of the chunk does to all that
// follows, so <S', D> is the later chunks' share, and no sum of gates' gradients runs over more
// than one chunk.  It is e^{cum_C} <S, D> + sum_t k_t . (e^{cum_C - cum} o (U D^T))_t.
//
// Precision: sums and chains are fp32; operands that are not inputs are two bf16 planes (16 to 17
// bits), R one.  Every gradient is rounded once, at the end.

#include "gdn_tc.cuh"

namespace kda {
namespace gdn {
namespace {

// ---- reverse scan -------------------------------------------------------------------------
// The forward scan's layout: MT groups of 16 value columns, four chain warps and four helpers
// each.  The helpers load the next chunk, compute the two products that do not wait for the chain
// (P^T dO and Q^T (e^cum o dO)), and write out what is kept.
template <int DK, int MT>
struct RScan {
    static constexpr int THREADS = 256 * MT;
    static constexpr int VROW = 32 * MT + 16, SROW = 2 * DK + 16, TROW = 2 * C + 16;
    static constexpr int WROW = DK + 4, PROW = C + 4;                  // floats
    static constexpr int K_ = 0, Q_ = K_ + C * DK * 2, REC = Q_ + C * DK * 2;
    static constexpr int G_ = REC + REC_BYTES, STAGE = G_ + C * VROW;
    static constexpr int DP = 2 * STAGE;                               // planes of D [2][16 MT][SROW]
    static constexpr int UP = DP + 2 * 16 * MT * SROW;                 // of dU [2][16 MT][TROW]
    static constexpr int YP = UP + 2 * 16 * MT * TROW;                 // of dY
    static constexpr int VP = YP + 2 * 16 * MT * TROW;                 // of -e^cum o dV
    static constexpr int OS = VP + 2 * 16 * MT * TROW;                 // dV, 512 bytes a chain warp
    static constexpr int WS = OS + 4 * MT * 512;                       // Q^T (e^cum o dO), fp32 [16 MT][WROW]
    static constexpr int PS = WS + 16 * MT * WROW * 4;                 // P^T dO, fp32 [16 MT][PROW]
    static constexpr int SMEM = PS + 16 * MT * PROW * 4;
};

template <int DK, int MT>
__global__ void __launch_bounds__(256 * MT) gdn_rscan_kernel(GdnBwdArgs b, const __grid_constant__ Seqs seqs, const char* records,
                                                             char* kept)
{
    using L = RScan<DK, MT>;
    const GdnArgs& a = b.f;
    constexpr int NS = DK / 32;
    constexpr int LOADERS = 128 * MT;
    extern __shared__ __align__(128) char sm[];
    const uint32_t base = smem_addr(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool chain = warp < 4 * MT;
    const int m = (warp >> 2) % MT;
    const int f = ((warp >> 2) & 1) ? 3 - (warp & 3) : (warp & 3);
    const int h = blockIdx.y, seq = blockIdx.z, hk = h / (a.Hv / a.Hk);
    const int v0 = blockIdx.x * 16 * MT, row0 = m * 16;
    const int len = seqs.len(seq), nch = (len + C - 1) / C;
    const int64_t t0 = seqs.start(seq);
    const int g4 = lane >> 2, t2 = (lane & 3) * 2;
    const uint32_t a_row = row0 + (lane & 15), a_piece = (lane >> 4) * 16;
    const int b_row = f * 16 + (lane & 7) + ((lane >> 4) << 3), b_piece = (lane >> 3) & 1;
    // lane's core matrix row of a transposed 16x16 block of T or P as a B operand
    const int t_off = (((lane >> 3) & 1) * 2 + (lane >> 4)) * 128 + (lane & 7) * 16;
    const Kept keep{DK, a.Dv};
    char* mine = kept + ((int64_t)seqs.slot0(seq, C) * a.Hv + h) * keep.bytes();   // chunk 0
    const int64_t next = (int64_t)a.Hv * keep.bytes();

    if (chain) {
        float D[NS][4];
        const int64_t soff = ((int64_t)seq * a.Hv + h) * DK * a.Dv + v0 + row0 + g4;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                D[n][e] = b.dST ? b.dST[soff + (int64_t)(f * (DK / 4) + n * 8 + t2 + (e & 1)) * a.Dv + (e >> 1) * 8] : 0.f;
        auto put_state = [&] {
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t p[2];
                    split<2>(D[n][2 * e], D[n][2 * e + 1], p);
                    const uint32_t dst = base + L::DP + (row0 + g4 + 8 * e) * L::SROW + (f * (DK / 4) + n * 8 + t2) * 2;
                    st_shared_b32(dst, p[0]);
                    st_shared_b32(dst + 16 * MT * L::SROW, p[1]);
                }
        };
        put_state();
        for (int c = nch - 1; c >= 0; --c) {
            __syncthreads();   // chunk c has landed and D is in place
            const uint32_t st = base + (c & 1) * L::STAGE;
            const float* scal = (const float*)(sm + (c & 1) * L::STAGE + L::REC + REC_SCAL);
            float kd[2][2][4] = {};
#pragma unroll
            for (int s = 0; s < DK / 16; ++s) {
                uint32_t bk[4], x[2][4];
                ldsm(bk, st + L::K_ + tile_at<DK>(b_row, 2 * s + b_piece));
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    ldsm(x[p], base + L::DP + p * 16 * MT * L::SROW + a_row * L::SROW + s * 32 + a_piece);
                    mma(kd[0][p], x[p], bk[0], bk[1]);
                    mma(kd[1][p], x[p], bk[2], bk[3]);
                }
            }
            bar_sync(1 + MT + m, 256);   // P^T dO is in place
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int t = f * 16 + n * 8 + t2;
                const float2 en = *(const float2*)&scal[C + t];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 w = *(const float2*)(sm + L::PS + ((row0 + g4 + 8 * e) * L::PROW + t) * 4);
                    uint32_t p[2];
                    split<2>(fmaf(en.x, kd[n][0][2 * e] + kd[n][1][2 * e], w.x),
                             fmaf(en.y, kd[n][0][2 * e + 1] + kd[n][1][2 * e + 1], w.y), p);
                    const uint32_t off = (row0 + g4 + 8 * e) * L::TROW + t * 2;
                    st_shared_b32(base + L::UP + off, p[0]);
                    st_shared_b32(base + L::UP + 16 * MT * L::TROW + off, p[1]);
                }
            }
            bar_sync(1 + m, 128);
            // dY = T^T dU for the warp's tokens: rows ib >= f of T
            float y[2][2][4] = {};
#pragma unroll
            for (int ib = 0; ib < 4; ++ib) {
                if (ib < f) continue;
                uint32_t x[2][4], t[2][4];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    ldsm(x[p], base + L::UP + p * 16 * MT * L::TROW + a_row * L::TROW + ib * 32 + a_piece);
                    ldsm_t(t[p], st + L::REC + p * TRI + blk(ib, f) + t_off);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    mma(y[n][0], x[0], t[0][2 * n], t[0][2 * n + 1]);
                    mma(y[n][1], x[1], t[0][2 * n], t[0][2 * n + 1]);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) mma(y[n][1], x[0], t[1][2 * n], t[1][2 * n + 1]);
            }
            uint32_t w4[4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int t = f * 16 + n * 8 + t2;
                const float2 gr = *(const float2*)&scal[t], be = *(const float2*)&scal[2 * C + t];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float y0 = y[n][0][2 * e] + y[n][1][2 * e], y1 = y[n][0][2 * e + 1] + y[n][1][2 * e + 1];
                    const float d0 = be.x * y0, d1 = be.y * y1;
                    uint32_t p[2], q[2];
                    split<2>(-gr.x * d0, -gr.y * d1, p);
                    split<2>(y0, y1, q);
                    const uint32_t off = (row0 + g4 + 8 * e) * L::TROW + t * 2;
                    st_shared_b32(base + L::VP + off, p[0]);
                    st_shared_b32(base + L::VP + 16 * MT * L::TROW + off, p[1]);
                    st_shared_b32(base + L::YP + off, q[0]);
                    st_shared_b32(base + L::YP + 16 * MT * L::TROW + off, q[1]);
                    w4[2 * n + e] = pack(d0, d1);
                }
            }
            stsm_t(base + L::OS + warp * 512 + ((lane >> 4) * 8 + (lane & 7)) * 32 + ((lane >> 3) & 1) * 16, w4);
            // dV and dY are in place, and Q^T (e^cum o dO); no one reads the planes of D any more
            bar_sync(1 + 2 * MT + m, 128 + LOADERS);
            const float gam = scal[C - 1];
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 w = *(const float2*)(sm + L::WS + ((row0 + g4 + 8 * e) * L::WROW + f * (DK / 4) + n * 8 + t2) * 4);
                    D[n][2 * e] = fmaf(gam, D[n][2 * e], w.x);
                    D[n][2 * e + 1] = fmaf(gam, D[n][2 * e + 1], w.y);
                }
#pragma unroll
            for (int jb = 0; jb < 4; ++jb) {
                uint32_t x[2][4], k4[NS / 2][4];
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    ldsm(x[p], base + L::VP + p * 16 * MT * L::TROW + a_row * L::TROW + jb * 32 + a_piece);
#pragma unroll
                for (int n = 0; n < NS; n += 2)
                    ldsm_t(k4[n / 2], st + L::K_ + tile_at<DK>(jb * 16 + (lane & 15), f * (DK / 32) + n + (lane >> 4)));
#pragma unroll
                for (int p = 1; p >= 0; --p)
#pragma unroll
                    for (int n = 0; n < NS; ++n) mma(D[n], x[p], k4[n / 2][(n & 1) * 2], k4[n / 2][(n & 1) * 2 + 1]);
            }
            put_state();
        }
        if (b.dS0)
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    b.dS0[soff + (int64_t)(f * (DK / 4) + n * 8 + t2 + (e & 1)) * a.Dv + (e >> 1) * 8] = D[n][e];
    } else {
        const int lt = tid - LOADERS;
        const __nv_bfloat16* kp = (const __nv_bfloat16*)a.k + (t0 * a.Hk + hk) * DK;
        const __nv_bfloat16* qp = (const __nv_bfloat16*)a.q + (t0 * a.Hk + hk) * DK;
        const __nv_bfloat16* gp = (const __nv_bfloat16*)b.dout + (t0 * a.Hv + h) * a.Dv + v0;
        __nv_bfloat16* vp = (__nv_bfloat16*)b.dv + (t0 * a.Hv + h) * a.Dv + v0;
        const char* rec = records + ((int64_t)seqs.slot0(seq, C) * a.Hv + h) * REC_BYTES;
        auto load = [&](int c) {
            const uint32_t st = base + (c & 1) * L::STAGE;
            const int valid = min(C, len - c * C);
            load_tile<DK, LOADERS>(st + L::K_, kp + (int64_t)c * C * a.Hk * DK, (int64_t)a.Hk * DK, valid, lt);
            load_tile<DK, LOADERS>(st + L::Q_, qp + (int64_t)c * C * a.Hk * DK, (int64_t)a.Hk * DK, valid, lt);
            for (int e = lt; e < C * 2 * MT; e += LOADERS) {
                const int row = e / (2 * MT), piece = e % (2 * MT);
                const bool in = row < valid;
                cp16(st + L::G_ + row * L::VROW + piece * 16, gp + ((int64_t)c * C + (in ? row : 0)) * a.Hv * a.Dv + piece * 8, in);
            }
            const char* src = rec + (int64_t)c * a.Hv * REC_BYTES;
            for (int e = lt; e < REC_BYTES / 16; e += LOADERS) cp16(st + L::REC + e * 16, src + e * 16, true);
            cp_async_commit();
        };
        if (nch > 0) load(nch - 1);
        for (int c = nch - 1; c >= 0; --c) {
            cp_async_wait_all();
            __syncthreads();
            const uint32_t st = base + (c & 1) * L::STAGE;
            const float* scal = (const float*)(sm + (c & 1) * L::STAGE + L::REC + REC_SCAL);
            char* dst = mine + c * next;
            // dO^T, 16 columns x 64 tokens, as A operands
            uint32_t g[4][4];
#pragma unroll
            for (int ib = 0; ib < 4; ++ib)
                ldsm_t(g[ib], st + L::G_ + (ib * 16 + (lane & 7) + ((lane >> 4) << 3)) * L::VROW + (row0 + ((lane >> 3) & 1) * 8) * 2);
            {
                float o[2][2][4] = {};
#pragma unroll
                for (int ib = 0; ib < 4; ++ib) {
                    if (ib < f) continue;
                    uint32_t p[2][4];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        ldsm_t(p[q], st + L::REC + REC_P + q * TRI + blk(ib, f) + t_off);
                        mma(o[0][q], g[ib], p[q][0], p[q][1]);
                        mma(o[1][q], g[ib], p[q][2], p[q][3]);
                    }
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *(float2*)(sm + L::PS + ((row0 + g4 + 8 * e) * L::PROW + f * 16 + n * 8 + t2) * 4) =
                            make_float2(o[n][0][2 * e] + o[n][1][2 * e], o[n][0][2 * e + 1] + o[n][1][2 * e + 1]);
            }
            bar_sync(1 + MT + m, 256);
            if (c > 0) load(c - 1);
            {
                float w[NS][4] = {};
#pragma unroll
                for (int ib = 0; ib < 4; ++ib) {
                    uint32_t x[2][4], q4[NS / 2][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 gr = *(const float2*)&scal[ib * 16 + (e >> 1) * 8 + t2];
                        uint32_t p[2];
                        split<2>(gr.x * low(g[ib][e]), gr.y * high(g[ib][e]), p);
                        x[0][e] = p[0];
                        x[1][e] = p[1];
                    }
#pragma unroll
                    for (int n = 0; n < NS; n += 2)
                        ldsm_t(q4[n / 2], st + L::Q_ + tile_at<DK>(ib * 16 + (lane & 15), f * (DK / 32) + n + (lane >> 4)));
#pragma unroll
                    for (int p = 1; p >= 0; --p)
#pragma unroll
                        for (int n = 0; n < NS; ++n) mma(w[n], x[p], q4[n / 2][(n & 1) * 2], q4[n / 2][(n & 1) * 2 + 1]);
                }
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *(float2*)(sm + L::WS + ((row0 + g4 + 8 * e) * L::WROW + f * (DK / 4) + n * 8 + t2) * 4) =
                            make_float2(w[n][2 * e], w[n][2 * e + 1]);
            }
            for (int e = lt; e < 16 * MT * DK / 8; e += LOADERS) {   // the planes of D
                const int piece = e % (DK / 8), row = e / (DK / 8);
                const uint32_t off = state_at(v0 + row, piece, a.Dv);
                *(uint4*)(dst + keep.d() + off) = *(const uint4*)(sm + L::DP + row * L::SROW + piece * 16);
                *(uint4*)(dst + keep.d() + keep.state() + off) = *(const uint4*)(sm + L::DP + (16 * MT + row) * L::SROW + piece * 16);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) bar_sync(1 + 2 * MT + i, 128 + LOADERS);
            for (int e = lt; e < 2 * 16 * MT * 8; e += LOADERS) {
                const int piece = e & 7, row = e / 8 % (16 * MT), p = e / 8 / (16 * MT);
                *(uint4*)(dst + keep.y() + p * keep.rows() + tile_at<C>(v0 + row, piece)) =
                    *(const uint4*)(sm + L::YP + (p * 16 * MT + row) * L::TROW + piece * 16);
            }
            // dV: 16 tokens x 16 columns of the chain warp of the same place
            const int cw = warp - 4 * MT, cf = ((cw >> 2) & 1) ? 3 - (cw & 3) : (cw & 3), cm = cw >> 2;
            const int tok = c * C + cf * 16 + (lane >> 1);
            if (tok < len)
                *(uint4*)(vp + (int64_t)tok * a.Hv * a.Dv + cm * 16 + (lane & 1) * 8) =
                    *(const uint4*)(sm + L::OS + cw * 512 + lane * 16);
        }
    }
}

// ---- gradients of q, k, g and beta ----------------------------------------------------------
// Dv = 32 (gdn_grads.cu has the others: half of an MMA's K = 64 panels would be empty).  One CTA per chunk and key
// head: 16 warps, warp (mt, qt) owns 16 tokens and a quarter of the columns of every product; the value heads of
// the group follow one another and are summed in registers.  D comes in where S was while the pair products
// are taken.  Bound by the rate and latency of warp MMAs (at Dv = 128 it took 0.50 ms for 4352 chunks and heads, of which
// their rate alone is 0.37; 8 warps took 0.56).
template <int DK, int DV>
struct Grads {
    static constexpr int THREADS = 512;
    static constexpr int NROW = 2 * C + 16;
    static constexpr int K_ = 0, Q_ = K_ + C * DK * 2;
    static constexpr int SB = Q_ + C * DK * 2;              // planes of S^T, then of D^T [2][DV][DK]
    static constexpr int G_ = SB + 2 * DV * DK * 2;         // dO [64][DV]
    static constexpr int U_ = G_ + C * DV * 2;              // planes of U^T [2][DV][64]
    static constexpr int Y_ = U_ + 2 * DV * C * 2;          // of dY^T
    static constexpr int N_ = Y_ + 2 * DV * C * 2;          // of N [2][64][NROW], then of beta M
    static constexpr int M_ = N_ + 2 * C * NROW;
    static constexpr int SC = M_ + 2 * C * NROW;            // grow, end, beta, cum
    static constexpr int RED = SC + 5 * C * 4;              // fp32 [20][64]
    static constexpr int SMEM = RED + 20 * C * 4;
};

template <int DK, int DV>
__global__ void __launch_bounds__(512) gdn_grads_kernel(GdnBwdArgs b, const __grid_constant__ Seqs seqs, const char* records,
                                                        const char* kept)
{
    using L = Grads<DK, DV>;
    const GdnArgs& a = b.f;
    constexpr int NT = L::THREADS, NK = DK / 32;   // 8-column tiles of a quarter of the key channels
    extern __shared__ __align__(128) char sm[];
    const uint32_t base = smem_addr(sm);
    int seq, c;
    if (!seqs.locate(blockIdx.x, C, seq, c)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the triangular products have mt + 1 steps (or 4 - mt): the quarters put the tokens on different
    // SM partitions
    const int qt = warp >> 2, mt = (warp + qt) & 3;
    const int hk = blockIdx.y, r = a.Hv / a.Hk;
    const int valid = min(C, seqs.len(seq) - c * C);
    const int64_t t0 = (int64_t)seqs.start(seq) + c * C;
    const int g4 = lane >> 2, t2 = (lane & 3) * 2, i0 = mt * 16 + g4;
    const Kept keep{DK, DV};
    const float* scal = (const float*)(sm + L::SC);
    float* red = (float*)(sm + L::RED);
    const int arow = mt * 16 + (lane & 15), apc = lane >> 4;                              // A, stored [row][k]
    const int krow = (lane & 7) + ((lane >> 4) << 3), tpc = (lane >> 3) & 1;              // A, stored [k][row]
    const int brow = lane & 15, bpc = lane >> 4;                                          // B, stored [k][column]

    load_tile<DK, NT>(base + L::K_, (const __nv_bfloat16*)a.k + (t0 * a.Hk + hk) * DK, (int64_t)a.Hk * DK, valid, tid);
    load_tile<DK, NT>(base + L::Q_, (const __nv_bfloat16*)a.q + (t0 * a.Hk + hk) * DK, (int64_t)a.Hk * DK, valid, tid);
    float sq[NK][4] = {}, sk[NK][4] = {};
    for (int h = hk * r; h < hk * r + r; ++h) {
        const char* mine = kept + ((int64_t)blockIdx.x * a.Hv + h) * keep.bytes();
        const char* rec = records + ((int64_t)blockIdx.x * a.Hv + h) * REC_BYTES;
        auto take = [&](uint32_t dst, size_t off, int bytes) {   // kept tiles are laid out as they are read
            for (int e = tid; e < bytes / 16; e += NT) cp16(dst + e * 16, mine + off + e * 16, true);
        };
        for (int e = tid; e < C * DV / 8; e += NT) {
            const int row = e / (DV / 8), piece = e % (DV / 8);
            const bool in = row < valid;
            cp16(base + L::G_ + tile_at<DV>(row, piece), (const __nv_bfloat16*)b.dout + ((t0 + (in ? row : 0)) * a.Hv + h) * DV + piece * 8, in);
        }
        take(base + L::SB, keep.s(), 2 * DV * DK * 2);
        take(base + L::Y_, keep.y(), 2 * DV * C * 2);
        cp_async_commit();
        take(base + L::U_, keep.u(), 2 * DV * C * 2);
        for (int e = tid; e < 5 * C / 4; e += NT) cp16(base + L::SC + e * 16, rec + REC_SCAL + e * 16, true);
        cp_async_commit();
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        // dO S^T and dY S^T, the warp's 16 tokens and quarter of the channels
        float xq[NK][4] = {}, xr[NK][4] = {};
#pragma unroll
        for (int s = 0; s < DV / 16; ++s) {
            uint32_t g[4], y[2][4];
            ldsm(g, base + L::G_ + tile_at<DV>(arow, 2 * s + apc));
#pragma unroll
            for (int p = 0; p < 2; ++p) ldsm_t(y[p], base + L::Y_ + p * DV * C * 2 + tile_at<C>(s * 16 + krow, mt * 2 + tpc));
#pragma unroll
            for (int n = 0; n < NK; n += 2) {
                uint32_t t[2][4];
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    ldsm_t(t[p], base + L::SB + p * DV * DK * 2 + state_at(s * 16 + brow, qt * NK + n + bpc, DV));
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mma(xq[n + e], g, t[0][2 * e], t[0][2 * e + 1]);
                    mma(xr[n + e], y[0], t[0][2 * e], t[0][2 * e + 1]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mma(xq[n + e], g, t[1][2 * e], t[1][2 * e + 1]);
                    mma(xr[n + e], y[1], t[0][2 * e], t[0][2 * e + 1]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) mma(xr[n + e], y[0], t[1][2 * e], t[1][2 * e + 1]);
            }
        }
        cp_async_wait_all();
        __syncthreads();   // S has been read; U and the gates are in
        take(base + L::SB, keep.d(), 2 * DV * DK * 2);
        cp_async_commit();
        // dO U^T, dY U^T and K K^T, the warp's 16 rows and 16 columns, on and below the diagonal
        float db[2] = {0.f, 0.f};   // sum_j M_ij k_i.k_j, rows i0 and i0 + 8
        if (qt <= mt) {
            float n4[2][4] = {}, m4[2][2][4] = {}, kk[2][4] = {};
#pragma unroll
            for (int s = 0; s < DV / 16; ++s) {
                uint32_t g[4], y[2][4], u[2][4];
                ldsm(g, base + L::G_ + tile_at<DV>(arow, 2 * s + apc));
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    ldsm_t(y[p], base + L::Y_ + p * DV * C * 2 + tile_at<C>(s * 16 + krow, mt * 2 + tpc));
                    ldsm_t(u[p], base + L::U_ + p * DV * C * 2 + tile_at<C>(s * 16 + brow, qt * 2 + bpc));
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    mma(n4[n], g, u[0][2 * n], u[0][2 * n + 1]);
                    mma(m4[n][0], y[0], u[0][2 * n], u[0][2 * n + 1]);
                    mma(m4[n][1], y[1], u[0][2 * n], u[0][2 * n + 1]);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    mma(n4[n], g, u[1][2 * n], u[1][2 * n + 1]);
                    mma(m4[n][1], y[0], u[1][2 * n], u[1][2 * n + 1]);
                }
            }
#pragma unroll
            for (int s = 0; s < DK / 16; ++s) {
                uint32_t x[4], k4[4];
                ldsm(x, base + L::K_ + tile_at<DK>(arow, 2 * s + apc));
                ldsm(k4, base + L::K_ + tile_at<DK>(qt * 16 + krow, 2 * s + tpc));
                mma(kk[0], x, k4[0], k4[1]);
                mma(kk[1], x, k4[2], k4[3]);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int j = qt * 16 + n * 8 + t2;
                const float2 hj = *(const float2*)&scal[3 * C + j], lj = *(const float2*)&scal[4 * C + j];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = i0 + 8 * e;
                    const float hi = scal[3 * C + i], li = scal[4 * C + i], be = scal[2 * C + i];
                    const float d0 = j <= i ? ex2_approx((hi - hj.x) + (li - lj.x)) : 0.f;
                    const float d1 = j + 1 <= i ? ex2_approx((hi - hj.y) + (li - lj.y)) : 0.f;
                    const float m0 = j < i ? -d0 * (m4[n][0][2 * e] + m4[n][1][2 * e]) : 0.f;
                    const float m1 = j + 1 < i ? -d1 * (m4[n][0][2 * e + 1] + m4[n][1][2 * e + 1]) : 0.f;
                    db[e] = fmaf(m0, kk[n][2 * e], fmaf(m1, kk[n][2 * e + 1], db[e]));
                    uint32_t p[2];
                    const uint32_t off = i * L::NROW + j * 2;
                    split<2>(d0 * n4[n][2 * e], d1 * n4[n][2 * e + 1], p);
                    st_shared_b32(base + L::N_ + off, p[0]);
                    st_shared_b32(base + L::N_ + C * L::NROW + off, p[1]);
                    split<2>(be * m0, be * m1, p);
                    st_shared_b32(base + L::M_ + off, p[0]);
                    st_shared_b32(base + L::M_ + C * L::NROW + off, p[1]);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            db[e] += __shfl_xor_sync(~0u, db[e], 1);
            db[e] += __shfl_xor_sync(~0u, db[e], 2);
            if ((lane & 3) == 0) red[qt * C + i0 + 8 * e] = db[e];
        }
        // dY . R: 8 tokens a thread, its rows strided by 64
        {
            const int pc = tid & 7;
            float acc[8] = {};
            for (int row = tid >> 3; row < DV; row += NT / 8) {
                const uint4 rr = *(const uint4*)(mine + keep.r() + tile_at<C>(row, pc));
                const uint4 y0 = *(const uint4*)(sm + L::Y_ + tile_at<C>(row, pc));
                const uint4 y1 = *(const uint4*)(sm + L::Y_ + DV * C * 2 + tile_at<C>(row, pc));
                const uint32_t rv[4] = {rr.x, rr.y, rr.z, rr.w}, a0[4] = {y0.x, y0.y, y0.z, y0.w}, a1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[2 * i] = fmaf(low(a0[i]) + low(a1[i]), low(rv[i]), acc[2 * i]);
                    acc[2 * i + 1] = fmaf(high(a0[i]) + high(a1[i]), high(rv[i]), acc[2 * i + 1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[i] += __shfl_xor_sync(~0u, acc[i], 8);
                acc[i] += __shfl_xor_sync(~0u, acc[i], 16);
                if (lane < 8) red[(4 + warp) * C + pc * 8 + i] = acc[i];
            }
        }
        __syncthreads();
        if (tid < valid) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < 20; ++w) s += red[w * C + tid];
            ((__nv_bfloat16*)b.dbeta)[(t0 + tid) * a.Hv + h] = __float2bfloat16_rn(s);
        }
        float dc[2] = {0.f, 0.f};   // the warp's part of dcum, rows i0 and i0 + 8
        auto dot = [&](uint32_t tile, const float (&x)[NK][4], float sign) {
#pragma unroll
            for (int n = 0; n < NK; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t v = *(const uint32_t*)(sm + tile + tile_at<DK>(i0 + 8 * e, qt * NK + n) + t2 * 2);
                    dc[e] += sign * fmaf(low(v), x[n][2 * e], high(v) * x[n][2 * e + 1]);
                }
        };
        auto scale = [&](float (&x)[NK][4], float f0, float f1) {
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                x[n][0] *= f0; x[n][1] *= f0; x[n][2] *= f1; x[n][3] *= f1;
            }
        };
        // dQ = e^cum o (dO S^T) + N K;  row part of dK: -beta e^cum o (dY S^T) + (beta M) K
        scale(xq, scal[i0], scal[i0 + 8]);
        scale(xr, -scal[i0] * scal[2 * C + i0], -scal[i0 + 8] * scal[2 * C + i0 + 8]);
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
            if (jb > mt) break;
            uint32_t w[2][2][4];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t off = p * C * L::NROW + arow * L::NROW + jb * 32 + apc * 16;
                ldsm(w[0][p], base + L::N_ + off);
                ldsm(w[1][p], base + L::M_ + off);
            }
#pragma unroll
            for (int n = 0; n < NK; n += 2) {
                uint32_t t[4];
                ldsm_t(t, base + L::K_ + tile_at<DK>(jb * 16 + brow, qt * NK + n + bpc));
#pragma unroll
                for (int p = 1; p >= 0; --p)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mma(xq[n + e], w[0][p], t[2 * e], t[2 * e + 1]);
                        mma(xr[n + e], w[1][p], t[2 * e], t[2 * e + 1]);
                    }
            }
        }
        dot(L::Q_, xq, 1.f);
        dot(L::K_, xr, 1.f);
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sq[n][e] += xq[n][e];
                sk[n][e] += xr[n][e];
            }
        // column part of dK: e^{cum_C - cum} o (U D^T) + (beta M)^T K + N^T Q
        float x[NK][4] = {}, ex = 0.f;
        cp_async_wait_all();
        __syncthreads();
        // S once more, 16 bytes of each plane a thread and round, while the product runs
        constexpr int NP = (DV * DK + 4095) / 4096;
        const bool has = DV * DK >= 4096 || tid < DV * DK / 8;
        uint4 sp[2][NP];
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p)
                sp[p][i] = has ? __ldcg((const uint4*)(mine + keep.s() + p * keep.state() + tid * 16 + i * 8192)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int s = 0; s < DV / 16; ++s) {
            uint32_t u[2][4];
#pragma unroll
            for (int p = 0; p < 2; ++p) ldsm_t(u[p], base + L::U_ + p * DV * C * 2 + tile_at<C>(s * 16 + krow, mt * 2 + tpc));
#pragma unroll
            for (int n = 0; n < NK; n += 2) {
                uint32_t t[2][4];
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    ldsm_t(t[p], base + L::SB + p * DV * DK * 2 + state_at(s * 16 + brow, qt * NK + n + bpc, DV));
#pragma unroll
                for (int p = 0; p < 3; ++p)   // U0 D0, U1 D0, U0 D1
#pragma unroll
                    for (int e = 0; e < 2; ++e) mma(x[n + e], u[p & 1], t[p >> 1][2 * e], t[p >> 1][2 * e + 1]);
            }
        }
        scale(x, scal[C + i0], scal[C + i0 + 8]);
        // <S', D> = e^cum_C <S, D> + sum_t k_t . (e^{cum_C - cum_t} (U D^T)_t)
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if (!has) break;
            const uint4 d0 = *(const uint4*)(sm + L::SB + tid * 16 + i * 8192), d1 = *(const uint4*)(sm + L::SB + DV * DK * 2 + tid * 16 + i * 8192);
            const uint32_t ss[2][4] = {{sp[0][i].x, sp[0][i].y, sp[0][i].z, sp[0][i].w}, {sp[1][i].x, sp[1][i].y, sp[1][i].z, sp[1][i].w}};
            const uint32_t dd[2][4] = {{d0.x, d0.y, d0.z, d0.w}, {d1.x, d1.y, d1.z, d1.w}};
#pragma unroll
            for (int z = 0; z < 4; ++z)
                ex = fmaf(low(dd[0][z]) + low(dd[1][z]), low(ss[0][z]) + low(ss[1][z]),
                          fmaf(high(dd[0][z]) + high(dd[1][z]), high(ss[0][z]) + high(ss[1][z]), ex));
        }
        ex *= scal[C - 1];
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t v = *(const uint32_t*)(sm + L::K_ + tile_at<DK>(i0 + 8 * e, qt * NK + n) + t2 * 2);
                ex = fmaf(low(v), x[n][2 * e], fmaf(high(v), x[n][2 * e + 1], ex));
            }
#pragma unroll
        for (int ib = 0; ib < 4; ++ib) {
            if (ib < mt) continue;
            uint32_t w[2][2][4];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t off = p * C * L::NROW + (ib * 16 + krow) * L::NROW + mt * 32 + tpc * 16;
                ldsm_t(w[0][p], base + L::M_ + off);
                ldsm_t(w[1][p], base + L::N_ + off);
            }
#pragma unroll
            for (int n = 0; n < NK; n += 2)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    uint32_t t[4];
                    ldsm_t(t, base + (z ? L::Q_ : L::K_) + tile_at<DK>(ib * 16 + brow, qt * NK + n + bpc));
#pragma unroll
                    for (int p = 1; p >= 0; --p) {
                        mma(x[n], w[z][p], t[0], t[1]);
                        mma(x[n + 1], w[z][p], t[2], t[3]);
                    }
                }
        }
        dot(L::K_, x, -1.f);
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sk[n][e] += x[n][e];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            dc[e] += __shfl_xor_sync(~0u, dc[e], 1);
            dc[e] += __shfl_xor_sync(~0u, dc[e], 2);
            if ((lane & 3) == 0) red[qt * C + i0 + 8 * e] = dc[e];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ex += __shfl_xor_sync(~0u, ex, o);
        if (lane == 0) red[4 * C + warp] = ex;
        __syncthreads();
        if (warp == 0) {   // dg: suffix sums of dcum, two tokens a lane, and the exit term
            float all = lane < 16 ? red[4 * C + lane] : 0.f;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) all += __shfl_xor_sync(~0u, all, o);
            all = __shfl_sync(~0u, all, 0);
            float d0 = 0.f, d1 = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                d0 += red[w * C + 2 * lane];
                d1 += red[w * C + 2 * lane + 1];
            }
            float s = d0 + d1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float y = __shfl_down_sync(~0u, s, o);
                if (lane + o < 32) s += y;
            }
            __nv_bfloat16* dg = (__nv_bfloat16*)b.dg + t0 * a.Hv + h;
            if (2 * lane < valid) dg[(int64_t)(2 * lane) * a.Hv] = __float2bfloat16_rn(s + all);
            if (2 * lane + 1 < valid) dg[(int64_t)(2 * lane + 1) * a.Hv] = __float2bfloat16_rn(s - d0 + all);
        }
        __syncthreads();   // the next head's tiles overwrite these
    }
    // dq and dk: 4-byte stores, 16 bytes a row and tile
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = i0 + 8 * e;
            if (i >= valid) continue;
            const int64_t off = ((t0 + i) * a.Hk + hk) * DK + qt * (DK / 4) + n * 8 + t2;
            *(uint32_t*)((__nv_bfloat16*)b.dq + off) = pack(sq[n][2 * e], sq[n][2 * e + 1]);
            *(uint32_t*)((__nv_bfloat16*)b.dk + off) = pack(sk[n][2 * e], sk[n][2 * e + 1]);
        }
}

template <int DK, int MT>
cudaError_t rscan(const GdnBwdArgs& a, const Seqs& s, const void* records, void* kept, cudaStream_t st)
{
    using L = RScan<DK, MT>;
    auto kern = gdn_rscan_kernel<DK, MT>;
    const cudaError_t e = allow_smem<gdn_rscan_kernel<DK, MT>>(L::SMEM);
    if (e != cudaSuccess) return e;
    ProfileScope prof("gdn_rscan", st);
    count_launch();
    kern<<<dim3(a.f.Dv / (16 * MT), a.f.Hv, s.n), L::THREADS, L::SMEM, st>>>(a, s, (const char*)records, (char*)kept);
    return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t grads(const GdnBwdArgs& a, const Seqs& s, const void* records, const void* kept, cudaStream_t st)
{
    using L = Grads<DK, DV>;
    auto kern = gdn_grads_kernel<DK, DV>;
    const cudaError_t e = allow_smem<gdn_grads_kernel<DK, DV>>(L::SMEM);
    if (e != cudaSuccess) return e;
    ProfileScope prof("gdn_grads_narrow", st);
    count_launch();
    kern<<<dim3(s.slots(C), a.f.Hk), L::THREADS, L::SMEM, st>>>(a, s, (const char*)records, (const char*)kept);
    return cudaGetLastError();
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
size_t rec_part(const Seqs& s, int Hv) { return up256((size_t)s.slots(C) * Hv * REC_BYTES); }
size_t kept_part(const Seqs& s, int Hv, int Dk, int Dv) { return (size_t)s.slots(C) * Hv * Kept{Dk, Dv}.bytes(); }
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
}  // namespace
}  // namespace gdn

bool gdn_tc_bwd_supported(const GdnBwdArgs& a)
{
    return gdn_tc_supported(a.f) && gdn::aligned16(a.dout) && gdn::aligned16(a.dq) && gdn::aligned16(a.dk) && gdn::aligned16(a.dv);
}

size_t gdn_tc_bwd_workspace(const Seqs& s, int Hv, int Dk, int Dv)
{
    return gdn::rec_part(s, Hv) + gdn::kept_part(s, Hv, Dk, Dv);
}

cudaError_t launch_gdn_tc_bwd(const GdnBwdArgs& b, const Seqs& s, void* ws, int sms, int* status, cudaStream_t st)
{
    using namespace gdn;
    char* records = (char*)ws;
    char* kept = records + rec_part(s, b.f.Hv);
    const bool whole = whole_heads(b.f, s, sms);
    cudaError_t e = cudaSuccess;
    if (s.tokens() > 0) {
        e = launch_prologue(b.f, s, records, st);
        if (e == cudaSuccess) e = whole ? launch_chain(b.f, s, records, kept, status, st) : launch_scan(b.f, s, records, kept, sms, st);
    }
    const bool wide = (int64_t)s.n * b.f.Hv * (b.f.Dv / 32) >= sms;   // as in the forward scan
    if (e == cudaSuccess)
        e = whole          ? launch_rchain(b, s, records, kept, status, st)
            : b.f.Dk == 64 ? (wide ? rscan<64, 2>(b, s, records, kept, st) : rscan<64, 1>(b, s, records, kept, st))
                           : (wide ? rscan<128, 2>(b, s, records, kept, st) : rscan<128, 1>(b, s, records, kept, st));
    if (e != cudaSuccess || s.tokens() == 0) return e;
    if (b.f.Dv != 32) return launch_grads(b, s, records, kept, sms, status, st);
    return b.f.Dk == 64 ? grads<64, 32>(b, s, records, kept, st) : grads<128, 32>(b, s, records, kept, st);
}

}  // namespace kda
