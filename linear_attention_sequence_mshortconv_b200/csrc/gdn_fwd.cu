// Gated delta rule over whole sequences on the tensor cores (bf16; Dk = 64 or 128).
//
// Chunks of C = 64 tokens; with cum the inclusive sum of g in the chunk and S its entry state
//   A = strict_lower(beta_i e^{cum_i - cum_j} k_i.k_j),  T = (I + A)^-1,
//   P = lower(e^{cum_i - cum_j} q_i.k_j)                                (prologue kernel)
//   R = V - e^cum o (K S),  U = T (beta o R),  O = e^cum o (Q S) + P U,
//   S' = e^{cum_C} S + K^T (e^{cum_C - cum} o U)                        (scan kernel)
// Every exponent is a sum of gates, so no factor exceeds 1 and any decay is safe.
//
// The prologue has no chain: one CTA per chunk and key head, all of them at once.  The scan is
// a chain over the chunks of a sequence, and its value columns are independent: a CTA owns
// 16 or 32 of them.  It keeps S transposed in the accumulators of its warps (rows: value
// columns), so K S, T Y and K^T U are three products whose left operands are the
// transposes of S, Y and U.
//
// Precision.  The state and every sum are fp32.  MMA operands that are not inputs (S, Y, U, T)
// are split over bf16 planes: three planes carry 24 bits and keep bf16's range (fp16 would need
// fewer, but overflows at 65504), two 16 to 17; gdn_tc.cuh says which take how many.  The state that
// is handed on is within 1e-6 of the recurrence's.

#include <algorithm>

#include "gdn_tc.cuh"

namespace kda {
namespace gdn {

// ---- prologue: T, P and the gates of each chunk -----------------------------------------
// KK^T and QK^T are bf16 MMAs (exact products, fp32 sums), shared by the value heads of a key
// head.  The unit lower triangular I + A is inverted in fp32: the four 16x16 diagonal blocks by
// forward substitution, a warp each, a column to a lane; then twice T21 = -T22 (A21 T11), on
// the two 32x32 and on the one 64x64 block.  Nothing here waits for another chunk, so what bounds
// it is the latency of these steps against the warps an SM holds: A and T take the place of K and
// Q, and 96 registers a thread (12 to 20 bytes spilled) let five CTAs share an SM.  (4352 chunks and heads, Dk = 128: 84 us, 0.25 GB of
// factors and inputs; the shared-memory pipe is busy 72% of it.)
constexpr int ALD = 68;   // row of A and T in floats: rows of a warp's reads fall in different banks
template <int DK>
constexpr int pro_smem()
{
    constexpr int tiles = 2 * C * DK * 2, at = 2 * C * ALD * 4;
    return (tiles > at ? tiles : at) + 4 * 3 * C * 4;
}

// One thread's share of X = A B (fp32, row-major with ALD): rows i and, if TWO, i + 16, columns
// c .. c + 3, K terms.
template <int K, bool TWO>
__device__ __forceinline__ void small_mm(const float (*A)[ALD], const float (*B)[ALD], int i, int c, float (&x)[2][4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) x[0][e] = x[1][e] = 0.f;
#pragma unroll
    for (int m = 0; m < K; m += 4) {
        float a[2][4];
#pragma unroll
        for (int q = 0; q < (TWO ? 2 : 1); ++q) {
            const float4 v = *(const float4*)&A[i + 16 * q][m];
            a[q][0] = v.x; a[q][1] = v.y; a[q][2] = v.z; a[q][3] = v.w;
        }
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const float4 v = *(const float4*)&B[m + z][c];
#pragma unroll
            for (int q = 0; q < (TWO ? 2 : 1); ++q) {
                x[q][0] = fmaf(a[q][z], v.x, x[q][0]); x[q][1] = fmaf(a[q][z], v.y, x[q][1]);
                x[q][2] = fmaf(a[q][z], v.z, x[q][2]); x[q][3] = fmaf(a[q][z], v.w, x[q][3]);
            }
        }
    }
}

template <int DK>
__global__ void __launch_bounds__(128, 5) gdn_prologue_kernel(GdnArgs a, const __grid_constant__ Seqs seqs, char* records)
{
    extern __shared__ __align__(128) char sm[];
    float (*A)[ALD] = (float (*)[ALD])sm;
    float (*T)[ALD] = A + C;
    // of up to four heads: cum log2(e), as a sum of two floats, and beta
    float* gates = (float*)(sm + pro_smem<DK>() - 4 * 3 * C * 4);
    int seq, c;
    if (!seqs.locate(blockIdx.x, C, seq, c)) return;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, hk = blockIdx.y, r = a.Hv / a.Hk;
    const int valid = min(C, seqs.len(seq) - c * C);
    const int64_t t0 = (int64_t)seqs.start(seq) + c * C;
    const uint32_t uK = smem_addr(sm), uQ = uK + C * DK * 2;
    load_tile<DK, 128>(uK, (const __nv_bfloat16*)a.k + (t0 * a.Hk + hk) * DK, (int64_t)a.Hk * DK, valid, tid);
    load_tile<DK, 128>(uQ, (const __nv_bfloat16*)a.q + (t0 * a.Hk + hk) * DK, (int64_t)a.Hk * DK, valid, tid);
    cp_async_commit();

    // a warp per head: inclusive sum of the gates in 64 bits, two tokens a lane
    auto sum_gates = [&](int h) {
        float* scal = (float*)(records + ((int64_t)blockIdx.x * a.Hv + h) * REC_BYTES + REC_SCAL);
        double s[2];
        float b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const int64_t off = (t0 + t) * a.Hv + h;
            s[i] = t < valid ? (double)finite_gate(to_f32(((const __nv_bfloat16*)a.g)[off])) : 0.0;
            b[i] = t < valid ? to_f32(((const __nv_bfloat16*)a.beta)[off]) : 0.f;
        }
        double sum = s[0] + s[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double x = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += x;
        }
        const double c1 = sum * 1.4426950408889634, c0 = (sum - s[1]) * 1.4426950408889634;
        const double last = __shfl_sync(~0u, c1, 31);
        const double cum[2] = {c0, c1};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const float hi = (float)cum[i], lo = (float)(cum[i] - (double)hi);
            float* g = gates + (h & 3) * 3 * C;
            g[t] = hi;
            g[C + t] = lo;
            g[2 * C + t] = b[i];
            scal[t] = exp2f(hi);
            scal[C + t] = exp2f((float)(last - cum[i]));
            scal[2 * C + t] = b[i];
            scal[3 * C + t] = hi;
            scal[4 * C + t] = lo;
        }
    };
    // heads hk r .. hk r + r - 1 in groups that share h / 4: slot h & 3 of `gates`, warp h & 3
    auto gates_from = [&](int h) {
        const int mine = (h & ~3) + w;
        if (mine >= h && mine < hk * r + r) sum_gates(mine);
    };
    gates_from(hk * r);
    cp_async_wait_all();
    __syncthreads();

    // rows 16 w .. 16 w + 15 of KK^T and QK^T, columns up to the diagonal block
    float kk[8][4] = {}, qk[8][4] = {};
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
        uint32_t ak[4], aq[4];
        const int arow = w * 16 + (lane & 15), apiece = 2 * s + (lane >> 4);
        ldsm(ak, uK + tile_at<DK>(arow, apiece));
        ldsm(aq, uQ + tile_at<DK>(arow, apiece));
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
            if (jb > w) break;
            uint32_t b[4];
            ldsm(b, uK + tile_at<DK>(jb * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * s + ((lane >> 3) & 1)));
            mma(kk[2 * jb], ak, b[0], b[1]);
            mma(kk[2 * jb + 1], ak, b[2], b[3]);
            mma(qk[2 * jb], aq, b[0], b[1]);
            mma(qk[2 * jb + 1], aq, b[2], b[3]);
        }
    }
    __syncthreads();   // K and Q have been read: A and T take their place
    const int g4 = lane >> 2, t2 = (lane & 3) * 2;
    for (int h = hk * r; h < hk * r + r; ++h) {
        char* rec = records + ((int64_t)blockIdx.x * a.Hv + h) * REC_BYTES;
        if (h > hk * r && (h & 3) == 0) {
            gates_from(h);
            __syncthreads();
        }
        const float* ch = gates + (h & 3) * 3 * C;
        const float *cl = ch + C, *bet = cl + C;
        // A to shared memory, P to the record
        const int i0 = w * 16 + g4, i1 = i0 + 8;
        const float h0 = ch[i0], h1 = ch[i1], l0 = cl[i0], l1 = cl[i1], b0 = bet[i0], b1 = bet[i1];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            if (n > 2 * w + 1) break;
            const int j = n * 8 + t2;
            const float2 hj = *(const float2*)&ch[j], lj = *(const float2*)&cl[j];
            float d[4] = {ex2_approx((h0 - hj.x) + (l0 - lj.x)), ex2_approx((h0 - hj.y) + (l0 - lj.y)),
                          ex2_approx((h1 - hj.x) + (l1 - lj.x)), ex2_approx((h1 - hj.y) + (l1 - lj.y))};
            if (n >= 2 * w) {   // the diagonal block
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + (e & 1) > (e < 2 ? i0 : i1)) d[e] = 0.f;
                *(float2*)&A[i0][j] = make_float2(j < i0 ? b0 * d[0] * kk[n][0] : 0.f, j + 1 < i0 ? b0 * d[1] * kk[n][1] : 0.f);
                *(float2*)&A[i1][j] = make_float2(j < i1 ? b1 * d[2] * kk[n][2] : 0.f, j + 1 < i1 ? b1 * d[3] * kk[n][3] : 0.f);
            } else {
                *(float2*)&A[i0][j] = make_float2(b0 * d[0] * kk[n][0], b0 * d[1] * kk[n][1]);
                *(float2*)&A[i1][j] = make_float2(b1 * d[2] * kk[n][2], b1 * d[3] * kk[n][3]);
            }
            uint32_t lo[PPL], hi[PPL];
            split<PPL>(d[0] * qk[n][0], d[1] * qk[n][1], lo);
            split<PPL>(d[2] * qk[n][2], d[3] * qk[n][3], hi);
            char* dst = rec + REC_P + blk(w, n >> 1) + (n & 1) * 128 + g4 * 16 + t2 * 2;
#pragma unroll
            for (int q = 0; q < PPL; ++q) {
                *(uint32_t*)(dst + q * TRI) = lo[q];
                *(uint32_t*)(dst + q * TRI + 256) = hi[q];
            }
        }
        __syncwarp();   // a warp's diagonal block is its own
        if (lane < 16) {
            const int base = 16 * w;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s0 = i == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                for (int m = 0; m < i; m += 4) {   // entries at and right of the diagonal are 0
                    const float4 v = *(const float4*)&A[base + i][base + m];
                    s0 = fmaf(-v.x, x[m], s0);
                    if (m + 1 < i) s1 = fmaf(-v.y, x[m + 1], s1);
                    if (m + 2 < i) s0 = fmaf(-v.z, x[m + 2], s0);
                    if (m + 3 < i) s1 = fmaf(-v.w, x[m + 3], s1);
                }
                x[i] = s0 + s1;
                T[base + i][base + lane] = x[i];
            }
        }
        __syncthreads();
        // the products A21 T11 go to blocks above A's diagonal, which nothing else uses
        float x[2][4];
        {
            const int p = (tid >> 6) * 32, i = (tid >> 2) & 15, cc = (tid & 3) * 4;   // two 32x32 blocks
            auto at = [&](float (*M)[ALD], int ro, int co) { return (float (*)[ALD])&M[ro][co]; };
            small_mm<16, false>(at(A, p + 16, p), at(T, p, p), i, cc, x);
            *(float4*)&A[p + i][p + 16 + cc] = make_float4(x[0][0], x[0][1], x[0][2], x[0][3]);
            __syncthreads();
            small_mm<16, false>(at(T, p + 16, p + 16), at(A, p, p + 16), i, cc, x);
            *(float4*)&T[p + 16 + i][p + cc] = make_float4(-x[0][0], -x[0][1], -x[0][2], -x[0][3]);
            __syncthreads();
            const int i2 = (tid >> 3) & 15, c2 = (tid & 7) * 4;   // the 64x64 block: rows i2, i2 + 16
            // T's 32x32 diagonal blocks are 0 above their own 16x16 ones
            if (tid < 64) *(float4*)&T[(tid >> 5) * 32 + (tid & 15)][(tid >> 5) * 32 + 16 + ((tid >> 4) & 1) * 8] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (tid < 64) *(float4*)&T[(tid >> 5) * 32 + (tid & 15)][(tid >> 5) * 32 + 20 + ((tid >> 4) & 1) * 8] = make_float4(0.f, 0.f, 0.f, 0.f);
            __syncthreads();
            small_mm<32, true>(at(A, 32, 0), at(T, 0, 0), i2, c2, x);
            *(float4*)&A[i2][32 + c2] = make_float4(x[0][0], x[0][1], x[0][2], x[0][3]);
            *(float4*)&A[i2 + 16][32 + c2] = make_float4(x[1][0], x[1][1], x[1][2], x[1][3]);
            __syncthreads();
            small_mm<32, true>(at(T, 32, 32), at(A, 0, 32), i2, c2, x);
            *(float4*)&T[32 + i2][c2] = make_float4(-x[0][0], -x[0][1], -x[0][2], -x[0][3]);
            *(float4*)&T[48 + i2][c2] = make_float4(-x[1][0], -x[1][1], -x[1][2], -x[1][3]);
        }
        __syncthreads();
        // the ten blocks, 128 pairs each, as planes; and the zeros
        for (int e = tid; e < 2 * (TPL + PPL) * BLK / 16; e += 128)
            *(uint4*)(rec + e / (2 * BLK / 16) * TRI + (e & (BLK / 16) ? blk(2, 3) : blk(0, 1)) + e % (BLK / 16) * 16) = make_uint4(0, 0, 0, 0);
        const int ii = ((tid >> 6) << 3) + ((tid >> 2) & 7), jj = (((tid >> 5) & 1) << 3) + (tid & 3) * 2;
#pragma unroll
        for (int ib = 0; ib < 4; ++ib)
#pragma unroll
            for (int jb = 0; jb <= ib; ++jb) {
                const float2 v = *(const float2*)&T[ib * 16 + ii][jb * 16 + jj];
                uint32_t p[TPL];
                split<TPL>(v.x, v.y, p);
#pragma unroll
                for (int q = 0; q < TPL; ++q) *(uint32_t*)(rec + q * TRI + blk(ib, jb) + tid * 4) = p[q];
            }
        __syncthreads();
    }
}

cudaError_t launch_prologue(const GdnArgs& a, const Seqs& s, void* records, cudaStream_t st)
{
    const dim3 grid(s.slots(C), a.Hk);
    ProfileScope prof("gdn_prologue", st);
    count_launch();
    auto go = [&](auto kern, cudaError_t allowed, int smem) {
        if (allowed != cudaSuccess) return allowed;
        kern<<<grid, 128, smem, st>>>(a, s, (char*)records);
        return cudaGetLastError();
    };
    if (a.Dk == 64) return go(gdn_prologue_kernel<64>, allow_smem<gdn_prologue_kernel<64>>(pro_smem<64>()), pro_smem<64>());
    return go(gdn_prologue_kernel<128>, allow_smem<gdn_prologue_kernel<128>>(pro_smem<128>()), pro_smem<128>());
}

// ---- scan ---------------------------------------------------------------------------------
// MT groups of eight warps; group m owns value columns 16 m .. 16 m + 15 of the CTA.  Four
// warps run the chain, four the output.  The warp of quarter f owns tokens 16 f .. of every
// product over tokens, and a chain warp key channels DK / 4 f .. of the state.  Per chunk:
//   chain:  K S -> Y | U = T Y | S' = e^{cum_C} S + K^T U'
//   output: next chunk's loads (cp.async, two stages), Q S | O = e^cum o (Q S) + P U
// with a barrier at each bar, where Y, U and S pass through shared memory as planes.  The
// chain is bound by latency (one warp a scheduler issues every fourth cycle), which the
// output warps fill: 1.5 us a chunk where a CTA has its SM to itself (16 heads of 512 chunks, 16 columns a CTA:
// 0.77 ms), 88 us for 12 ragged samples of 33 chunks at most with 8 heads (Dk = Dv = 128).
//
// KEEP: the scan of the backward.  The output warps then write what the gradients need of each
// chunk (the planes of S and U and R) in place of the output.
template <int DK, int MT, bool KEEP>
struct Scan {
    static constexpr int THREADS = 256 * MT;
    static constexpr int VROW = 32 * MT + 16;        // bytes of a staged row of V: odd multiple of 16
    static constexpr int SROW = 2 * DK + 16;         // of a row of the S planes
    static constexpr int TROW = 2 * C + 16;          // of a row of the Y and U planes
    static constexpr int K_ = 0, Q_ = K_ + C * DK * 2, REC = Q_ + (KEEP ? 0 : C * DK * 2);
    static constexpr int V_ = REC + REC_BYTES, STAGE = V_ + C * VROW;
    static constexpr int SP = 2 * STAGE;                               // [plane][16 MT][SROW]
    static constexpr int YP = SP + SPL * 16 * MT * SROW;            // [plane][16 MT][TROW]
    static constexpr int UP = YP + PLANES * 16 * MT * TROW;            // decayed U
    static constexpr int WP = UP + PLANES * 16 * MT * TROW;            // U, two planes
    static constexpr int OS = WP + 2 * 16 * MT * TROW;                 // 512 bytes an output warp, or R
    static constexpr int SMEM = OS + (KEEP ? 16 * MT * TROW : 4 * MT * 512);
};

template <int DK, int MT, bool KEEP>
__global__ void __launch_bounds__(256 * MT) gdn_scan_kernel(GdnArgs a, const __grid_constant__ Seqs seqs, const char* records,
                                                            char* kept)
{
    using L = Scan<DK, MT, KEEP>;
    constexpr int NS = DK / 32;   // 8-column tiles of the state a warp holds
    constexpr int LOADERS = 128 * MT;
    extern __shared__ __align__(128) char sm[];
    const uint32_t base = smem_addr(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool chain = warp < 4 * MT;
    const int m = (warp >> 2) % MT;
    // quarter 3 has the most work in the triangular products: groups and roles put it on
    // different SM partitions (warp % 4)
    const int f = ((warp >> 2) & 1) ? 3 - (warp & 3) : (warp & 3);
    const int h = blockIdx.y, seq = blockIdx.z, hk = h / (a.Hv / a.Hk);
    const int v0 = blockIdx.x * 16 * MT, row0 = m * 16;
    const int len = seqs.len(seq), nch = (len + C - 1) / C;
    const int64_t t0 = seqs.start(seq);
    const int g4 = lane >> 2, t2 = (lane & 3) * 2;
    // lane's address in a plane of [16 rows][columns] for a 16x16 A operand
    const uint32_t a_row = row0 + (lane & 15), a_piece = (lane >> 4) * 16;
    // lane's row and piece of 16 tokens x 16 channels as a B operand
    const int b_row = f * 16 + (lane & 7) + ((lane >> 4) << 3), b_piece = (lane >> 3) & 1;

    if (chain) {
        // S^T: row = value column, column = key channel
        float S[NS][4];
        const int64_t soff = ((int64_t)seq * a.Hv + h) * DK * a.Dv + v0 + row0 + g4;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[n][e] = a.S0 ? a.S0[soff + (int64_t)(f * (DK / 4) + n * 8 + t2 + (e & 1)) * a.Dv + (e >> 1) * 8] : 0.f;
        auto put_state = [&] {
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t p[SPL];
                    split<SPL>(S[n][2 * e], S[n][2 * e + 1], p);
                    const uint32_t dst = base + L::SP + (row0 + g4 + 8 * e) * L::SROW + (f * (DK / 4) + n * 8 + t2) * 2;
#pragma unroll
                    for (int q = 0; q < SPL; ++q) st_shared_b32(dst + q * 16 * MT * L::SROW, p[q]);
                }
        };
        put_state();
        for (int c = 0; c < nch; ++c) {
            __syncthreads();   // chunk c has landed and S is in place
            const uint32_t st = base + (c & 1) * L::STAGE;
            const float* scal = (const float*)(sm + (c & 1) * L::STAGE + L::REC + REC_SCAL);
            // K S of the warp's 16 tokens (two 8-token tiles), transposed
            float ks[2][SPL][4] = {};
#pragma unroll
            for (int s = 0; s < DK / 16; ++s) {
                uint32_t bk[4], x[SPL][4];
                ldsm(bk, st + L::K_ + tile_at<DK>(b_row, 2 * s + b_piece));
#pragma unroll
                for (int p = 0; p < SPL; ++p)
                    ldsm(x[p], base + L::SP + p * 16 * MT * L::SROW + a_row * L::SROW + s * 32 + a_piece);
#pragma unroll
                for (int p = 0; p < SPL; ++p) {
                    mma(ks[0][p], x[p], bk[0], bk[1]);
                    mma(ks[1][p], x[p], bk[2], bk[3]);
                }
            }
            // Y = beta o (V - e^cum o (K S))
            {
                uint32_t v[4];   // tiles (token half 0, 1) x (column half 0, 1)
                ldsm_t(v, st + L::V_ + (f * 16 + (lane & 15)) * L::VROW + (row0 + (lane >> 4) * 8) * 2);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int t = f * 16 + n * 8 + t2;
                    const float2 gr = *(const float2*)&scal[t], be = *(const float2*)&scal[2 * C + t];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t vv = v[n + 2 * e];
                        const float r0 = low(vv) - gr.x * (ks[n][0][2 * e] + ks[n][1][2 * e]);
                        const float r1 = high(vv) - gr.y * (ks[n][0][2 * e + 1] + ks[n][1][2 * e + 1]);
                        uint32_t p[PLANES];
                        split<PLANES>(be.x * r0, be.y * r1, p);
                        const uint32_t dst = base + L::YP + (row0 + g4 + 8 * e) * L::TROW + t * 2;
                        if (KEEP) st_shared_b32(base + L::OS + (row0 + g4 + 8 * e) * L::TROW + t * 2, pack(r0, r1));
#pragma unroll
                        for (int q = 0; q < PLANES; ++q) st_shared_b32(dst + q * 16 * MT * L::TROW, p[q]);
                    }
                }
            }
            bar_sync(1 + m, 128);
            // U = T Y for the warp's tokens: every product of planes but T1 Y2 (2^-27 of the result)
            float u[2][PLANES][4] = {};
#pragma unroll
            for (int jb = 0; jb < 4; ++jb) {
                if (jb > f) break;
                uint32_t y[PLANES][4], t[TPL][4];
#pragma unroll
                for (int p = 0; p < PLANES; ++p) ldsm(y[p], base + L::YP + p * 16 * MT * L::TROW + a_row * L::TROW + jb * 32 + a_piece);
#pragma unroll
                for (int p = 0; p < TPL; ++p) ldsm(t[p], st + L::REC + p * TRI + blk(f, jb) + lane * 16);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    mma(u[n][0], y[0], t[0][2 * n], t[0][2 * n + 1]);
                    mma(u[n][1], y[1], t[0][2 * n], t[0][2 * n + 1]);
                    mma(u[n][2], y[2], t[0][2 * n], t[0][2 * n + 1]);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    mma(u[n][1], y[0], t[1][2 * n], t[1][2 * n + 1]);
                    mma(u[n][2], y[1], t[1][2 * n], t[1][2 * n + 1]);
                }
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int t = f * 16 + n * 8 + t2;
                const float2 en = *(const float2*)&scal[C + t];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float u0 = u[n][0][2 * e] + (u[n][1][2 * e] + u[n][2][2 * e]);
                    const float u1 = u[n][0][2 * e + 1] + (u[n][1][2 * e + 1] + u[n][2][2 * e + 1]);
                    uint32_t p[PLANES], q2[2];
                    split<PLANES>(en.x * u0, en.y * u1, p);
                    split<2>(u0, u1, q2);
                    const uint32_t off = (row0 + g4 + 8 * e) * L::TROW + t * 2;
#pragma unroll
                    for (int q = 0; q < PLANES; ++q) st_shared_b32(base + L::UP + q * 16 * MT * L::TROW + off, p[q]);
                    st_shared_b32(base + L::WP + off, q2[0]);
                    st_shared_b32(base + L::WP + 16 * MT * L::TROW + off, q2[1]);
                }
            }
            // U is in place; no warp of the group reads the planes of S any more
            bar_sync(1 + MT + m, KEEP ? 128 + LOADERS : 256);
            // S' = e^{cum_C} S + K^T (decayed U), the warp's key channels
            const float gam = scal[C - 1];
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[n][e] *= gam;
#pragma unroll
            for (int jb = 0; jb < 4; ++jb) {
                uint32_t x[PLANES][4], b[NS / 2][4];
#pragma unroll
                for (int p = 0; p < PLANES; ++p)
                    ldsm(x[p], base + L::UP + p * 16 * MT * L::TROW + a_row * L::TROW + jb * 32 + a_piece);
#pragma unroll
                for (int n = 0; n < NS; n += 2)
                    ldsm_t(b[n / 2], st + L::K_ + tile_at<DK>(jb * 16 + (lane & 15), f * (DK / 32) + n + (lane >> 4)));
#pragma unroll
                for (int p = PLANES - 1; p >= 0; --p)
#pragma unroll
                    for (int n = 0; n < NS; ++n) mma(S[n], x[p], b[n / 2][(n & 1) * 2], b[n / 2][(n & 1) * 2 + 1]);
            }
            put_state();
        }
        if (a.ST)
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    a.ST[soff + (int64_t)(f * (DK / 4) + n * 8 + t2 + (e & 1)) * a.Dv + (e >> 1) * 8] = S[n][e];
    } else {
        const int lt = tid - LOADERS;
        const __nv_bfloat16* kp = (const __nv_bfloat16*)a.k + (t0 * a.Hk + hk) * DK;
        const __nv_bfloat16* qp = (const __nv_bfloat16*)a.q + (t0 * a.Hk + hk) * DK;
        const __nv_bfloat16* vp = (const __nv_bfloat16*)a.v + (t0 * a.Hv + h) * a.Dv + v0;
        __nv_bfloat16* op = (__nv_bfloat16*)a.o + (t0 * a.Hv + h) * a.Dv + v0;
        const char* rec = records + ((int64_t)seqs.slot0(seq, C) * a.Hv + h) * REC_BYTES;
        const Kept keep{DK, a.Dv};
        auto load = [&](int c) {
            const uint32_t st = base + (c & 1) * L::STAGE;
            const int valid = min(C, len - c * C);
            load_tile<DK, LOADERS>(st + L::K_, kp + (int64_t)c * C * a.Hk * DK, (int64_t)a.Hk * DK, valid, lt);
            if (!KEEP) load_tile<DK, LOADERS>(st + L::Q_, qp + (int64_t)c * C * a.Hk * DK, (int64_t)a.Hk * DK, valid, lt);
            for (int e = lt; e < C * 2 * MT; e += LOADERS) {
                const int row = e / (2 * MT), piece = e % (2 * MT);
                const bool in = row < valid;
                cp16(st + L::V_ + row * L::VROW + piece * 16, vp + ((int64_t)c * C + (in ? row : 0)) * a.Hv * a.Dv + piece * 8, in);
            }
            const char* src = rec + (int64_t)c * a.Hv * REC_BYTES;
            for (int e = lt; e < REC_BYTES / 16; e += LOADERS) cp16(st + L::REC + e * 16, src + e * 16, true);
            cp_async_commit();
        };
        if (nch > 0) load(0);
        for (int c = 0; c < nch; ++c) {
            cp_async_wait_all();
            __syncthreads();   // chunk c has landed; no one reads stage (c + 1) % 2
            if (c + 1 < nch) load(c + 1);
            const uint32_t st = base + (c & 1) * L::STAGE;
            if (KEEP) {
                char* dst = kept + ((int64_t)(seqs.slot0(seq, C) + c) * a.Hv + h) * keep.bytes();
                for (int e = lt; e < SPL * 16 * MT * DK / 8; e += LOADERS) {
                    const int piece = e % (DK / 8), row = e / (DK / 8) % (16 * MT), p = e / (DK / 8) / (16 * MT);
                    *(uint4*)(dst + keep.s() + p * keep.state() + state_at(v0 + row, piece, a.Dv)) =
                        *(const uint4*)(sm + L::SP + (p * 16 * MT + row) * L::SROW + piece * 16);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) bar_sync(1 + MT + i, 128 + LOADERS);
                for (int e = lt; e < 3 * 16 * MT * 8; e += LOADERS) {
                    const int piece = e & 7, row = e / 8 % (16 * MT), p = e / 8 / (16 * MT);
                    const uint4 x = *(const uint4*)(sm + (p < 2 ? L::WP + (p * 16 * MT + row) * L::TROW : L::OS + row * L::TROW) + piece * 16);
                    *(uint4*)(dst + (p < 2 ? keep.u() + p * keep.rows() : keep.r()) + tile_at<C>(v0 + row, piece)) = x;
                }
                continue;
            }
            const float* scal = (const float*)(sm + (c & 1) * L::STAGE + L::REC + REC_SCAL);
            float qs[2][2][4] = {};
#pragma unroll
            for (int s = 0; s < DK / 16; ++s) {
                uint32_t bq[4], x[2][4];
                ldsm(bq, st + L::Q_ + tile_at<DK>(b_row, 2 * s + b_piece));
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    ldsm(x[p], base + L::SP + p * 16 * MT * L::SROW + a_row * L::SROW + s * 32 + a_piece);
                    mma(qs[0][p], x[p], bq[0], bq[1]);
                    mma(qs[1][p], x[p], bq[2], bq[3]);
                }
            }
            float o[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float2 gr = *(const float2*)&scal[f * 16 + n * 8 + t2];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] = ((e & 1) ? gr.y : gr.x) * (qs[n][0][e] + qs[n][1][e]);
            }
            bar_sync(1 + MT + m, 256);
#pragma unroll
            for (int jb = 0; jb < 4; ++jb) {
                if (jb > f) break;
                uint32_t x[2][4], b[PPL][4];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    ldsm(b[p], st + L::REC + REC_P + p * TRI + blk(f, jb) + lane * 16);
                    ldsm(x[p], base + L::WP + p * 16 * MT * L::TROW + a_row * L::TROW + jb * 32 + a_piece);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p) {   // P0 U0, P0 U1, P1 U0
                    mma(o[0], x[p & 1], b[p >> 1][0], b[p >> 1][1]);
                    mma(o[1], x[p & 1], b[p >> 1][2], b[p >> 1][3]);
                }
            }
            // 16 tokens x 16 columns, turned over in the warp's own 512 bytes
            const int mine = L::OS + (warp - 4 * MT) * 512;
            const uint32_t w4[4] = {pack(o[0][0], o[0][1]), pack(o[0][2], o[0][3]), pack(o[1][0], o[1][1]), pack(o[1][2], o[1][3])};
            stsm_t(base + mine + ((lane >> 4) * 8 + (lane & 7)) * 32 + ((lane >> 3) & 1) * 16, w4);
            __syncwarp();
            const int tok = c * C + f * 16 + (lane >> 1);
            const uint4 out = *(const uint4*)(sm + mine + lane * 16);
            if (tok < len) *(uint4*)(op + (int64_t)tok * a.Hv * a.Dv + row0 + (lane & 1) * 8) = out;
            __syncwarp();
        }
    }
}

namespace {
template <int DK, int MT, bool KEEP>
cudaError_t scan(const GdnArgs& a, const Seqs& s, const void* records, void* kept, cudaStream_t st)
{
    using L = Scan<DK, MT, KEEP>;
    auto kern = gdn_scan_kernel<DK, MT, KEEP>;
    const cudaError_t e = allow_smem<gdn_scan_kernel<DK, MT, KEEP>>(L::SMEM);
    if (e != cudaSuccess) return e;
    ProfileScope prof(KEEP ? "gdn_scan_keep" : "gdn_scan", st);
    count_launch();
    kern<<<dim3(a.Dv / (16 * MT), a.Hv, s.n), L::THREADS, L::SMEM, st>>>(a, s, (const char*)records, (char*)kept);
    return cudaGetLastError();
}
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
}  // namespace

cudaError_t launch_scan(const GdnArgs& a, const Seqs& s, const void* records, void* kept, int sms, cudaStream_t st)
{
    // 32 columns a CTA re-read K, Q and the factors half as often; 16 put twice as many SMs to
    // work where the heads alone do not fill them.
    const bool wide = (int64_t)s.n * a.Hv * (a.Dv / 32) >= sms;
    if (kept) {
        if (a.Dk == 64) return wide ? scan<64, 2, true>(a, s, records, kept, st) : scan<64, 1, true>(a, s, records, kept, st);
        return wide ? scan<128, 2, true>(a, s, records, kept, st) : scan<128, 1, true>(a, s, records, kept, st);
    }
    if (a.Dk == 64) return wide ? scan<64, 2, false>(a, s, records, kept, st) : scan<64, 1, false>(a, s, records, kept, st);
    return wide ? scan<128, 2, false>(a, s, records, kept, st) : scan<128, 1, false>(a, s, records, kept, st);
}
}  // namespace gdn

namespace gdn {
// Which scan: whole heads (gdn_chain.cu) or columns of heads.  Columns make Dv / 32 times as many CTAs, whose
// steps are shorter (1.5 us alone on an SM against 2.6) but read the head's chunk records once each.  So they are
// for calls whose time is set by the longest sample's steps in a row, and whole heads for those where
// the columns' steps, shared out over the SMs, are more than that.
// Measured (Dk = Dv = 128): 4 x 68 chunks, 16 heads (117 steps of work an SM against 68 in a row): columns
// 333 us, whole heads 179; 108 chunks in 12 ragged samples, 8 heads (23 against 33): 86 and 94.
bool whole_heads(const GdnArgs& a, const Seqs& s, int sms)
{
    int64_t longest = 0, all = 0;
    for (int i = 0; i < s.n; ++i) {
        const int chunks = (s.len(i) + C - 1) / C;
        longest = max(longest, (int64_t)chunks);
        all += chunks;
    }
    return a.Dv != 32 && all * a.Hv * (a.Dv / 32) > sms * longest;
}
}  // namespace gdn

// The tensor-core path copies rows in 16-byte pieces.
bool gdn_tc_supported(const GdnArgs& a)
{
    return a.t == ET_BF16 && (a.Dk == 64 || a.Dk == 128) && gdn::aligned16(a.q) && gdn::aligned16(a.k) &&
           gdn::aligned16(a.v) && gdn::aligned16(a.o);
}

size_t gdn_tc_workspace(const GdnArgs& a, const Seqs& s, int sms)
{
    // (enough for either way: which one is taken depends on the states' alignment as well)
    const int per = gdn::piece_chunks(s, a.Hv, a.Dk, a.Dv, sms);
    const size_t records = (size_t)s.slots(gdn::C) * a.Hv * gdn::REC_BYTES;
    return per ? std::max(records, gdn::pieces_workspace(s, a.Hv, a.Dk, a.Dv, per)) : records;
}

cudaError_t launch_gdn_tc(const GdnArgs& a, const Seqs& s, void* ws, int sms, int* status, cudaStream_t st)
{
    // (states are carried from piece to piece 16 bytes at a time)
    const int per = gdn::aligned16(a.S0) && gdn::aligned16(a.ST) ? gdn::piece_chunks(s, a.Hv, a.Dk, a.Dv, sms) : 0;
    if (per) return gdn::launch_pieces(a, s, ws, per, status, st);
    cudaError_t e = cudaSuccess;
    const bool whole = gdn::whole_heads(a, s, sms);
    if (s.tokens() > 0) e = gdn::launch_prologue(a, s, ws, st);
    if (e != cudaSuccess) return e;
    return whole ? gdn::launch_chain(a, s, ws, nullptr, status, st) : gdn::launch_scan(a, s, ws, nullptr, sms, st);
}

}  // namespace kda
