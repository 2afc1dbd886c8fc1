// Gradients of q, k, g and beta of the gated delta rule on tcgen05 tensor cores (bf16; Dk and Dv 64 or 128).
//
// The mathematics is that of gdn_bwd.cu.  Every product has the key channels, or pairs of tokens, as its 128 rows:
//   E1 = U dO^T, E2 = U dY^T      rows: the tokens of U's two planes, one after the other, so that one product
//                                 takes both; their sum comes about when the threads read it
//   XQ = S dO^T, XR = S dY^T, XC = D U^T, NK = K^T N^T, MK = K^T (beta M)^T, CC = K^T (beta M) + Q^T N
//                                 rows: key channels; columns: tokens
// and all operands lie as the copy engine brought them: what is kept of a chunk (S, D, U, dY) has its rows (value
// columns) as K.  Only N and beta M are written by the threads, two planes each.
//
// The other part of dbeta, sum_j M_ij k_i.k_j, is k_i . (beta M K)_i / beta_i; so that this holds for beta = 0 as well,
// betas below 2^-24 count as 2^-24 in beta M (less than the planes' rounding), and as themselves in dK's row part.
//
// One CTA per SM takes chunks of key heads in turn, and the value heads of each one after another.
//
//   warps 0-3   E1 -> N, E2 -> beta M; then dY . R
//   warps 4-19  (four warpgroups) <S, D>, and the sums over the key channels, a channel a lane, 16 tokens a
//               warpgroup; these and the first four warps are a head apart
//   warp 20     issues the MMAs
//   warp 21     the loads: S and then D share a buffer; each goes on as soon as its buffer is free, into the
//               next head and chunk
//
// The tiles of a chunk and value head are 208 KB at Dk = Dv = 128, 0.14 ms of HBM for 4 rows of 68 chunks, 16 heads; the
// kernel takes 0.26 ms there (warp MMAs, as gdn_bwd.cu has them for Dv = 32, 0.50).  What bounds it is the circle from one head
// to the next, 7.7 us: U's load and E 2, the threads' N and M 3.4, the products that wait for them 2.3.
//
// Every wait is bounded; after one runs out all roles run to their end on whatever is there.

#include "gdn_whole.cuh"

namespace kda {
namespace gdn {
namespace {

template <int DK, int DV>
struct TGrads {
    static constexpr int THREADS = 704;
    static constexpr int Q_ = 0, K_ = Q_ + DK / 64 * PANEL;
    static constexpr int SD = K_ + DK / 64 * PANEL;          // planes of S^T, then of D^T [2][DK / 64][DV][64]
    static constexpr int U_ = SD + 2 * DV * DK * 2;          // planes of U^T [2][DV][64]
    static constexpr int Y_ = U_ + 2 * DV * C * 2;           // of dY^T
    static constexpr int G_ = Y_ + 2 * DV * C * 2;           // dO
    static constexpr int N_ = G_ + DV / 64 * PANEL;          // planes of N^T [2][64][64], then of beta M^T
    static constexpr int SC = N_ + 4 * PANEL;                // grow, end, beta, cum, of three heads: the loads are two ahead of the last reader
    static constexpr int RED = SC + 3 * 5 * C * 4;               // fp32: of two heads dY.R [4][64]; dbeta [4][64], dcum [4][64], exit [16]
    static constexpr int RY = 4 * C, DB = 2 * RY, DC = DB + 4 * C, EX = DC + 4 * C;
    static constexpr int BAR = RED + (EX + 16) * 4;
    static constexpr int SMEM = BAR + 256 + 1024 > 116 * 1024 ? BAR + 256 + 1024 : 116 * 1024;   // one CTA to an SM
    static constexpr int XQ = 0, XR = 64, XC = 128, CC = 192, NK = 256, MK = 320, E1 = 384, E2 = 448;   // tensor memory
};

// v[c], c = 0 .. 7, summed over the warp: lane l gets the sum of v[l & 7]
__device__ __forceinline__ float transpose_sum(float (&v)[8], int lane)
{
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int k = 0; k < o; ++k) {
            const float give = up ? v[k] : v[k + o], keep = up ? v[k + o] : v[k];
            v[k] = keep + __shfl_xor_sync(~0u, give, o);
        }
    }
    v[0] += __shfl_xor_sync(~0u, v[0], 8);
    return v[0] + __shfl_xor_sync(~0u, v[0], 16);
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8])
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ float at_least(float beta) { return fabsf(beta) < 5.9604644775390625e-8f ? 5.9604644775390625e-8f : beta; }

template <int DK, int DV>
__global__ void __launch_bounds__(704, 1)
gdn_tgrads_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                  GdnBwdArgs b, const __grid_constant__ Seqs seqs, const char* records, char* kept, int* status, int drop)
{
    using L = TGrads<DK, DV>;
    const GdnArgs& a = b.f;
    extern __shared__ char raw[];
    char* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t base = smem_addr(sm);
    uint64_t* bars = (uint64_t*)(sm + L::BAR);
    uint64_t *kq_full = bars, *kq_empty = bars + 1, *y_full = bars + 2, *y_empty = bars + 3, *s_full = bars + 4, *s_done = bars + 5;
    uint64_t *d_full = bars + 6, *d_empty = bars + 7, *landed = bars + 8, *e_done = bars + 9, *ry_ready = bars + 10, *sum_free = bars + 11;
    uint64_t *nm_ready = bars + 12, *out_done = bars + 13, *acc_free = bars + 14, *drain = bars + 15, *u_full = bars + 16, *u_empty = bars + 17;
    uint32_t* tm_ptr = (uint32_t*)(bars + 18);
    const Guard guard{(volatile int*)(tm_ptr + 1), status};

    const int tid = threadIdx.x, lane = tid & 31, warp = uniform_warp();
    const int r = a.Hv / a.Hk, items = seqs.slots(C) * a.Hk;
    const Kept keep{DK, DV};

    if (warp == 21) {
        if (lane == 0) {
            for (uint64_t* x : {kq_full, y_full, u_full, u_empty, s_full, s_done, d_full, landed, e_done, drain}) mbar_init(x, 1);
            for (uint64_t* x : {y_empty, out_done}) mbar_init(x, 5);            // the MMAs and warps 0-3
            for (uint64_t* x : {d_empty, kq_empty}) mbar_init(x, 17);           // the MMAs and warps 4-19
            mbar_init(nm_ready, 4 + drop);
            mbar_init(ry_ready, 4);
            for (uint64_t* x : {acc_free, sum_free}) mbar_init(x, 16);
            *guard.flag = 0;
            fence_mbar_init();
            fence_async_smem();
        }
    } else if (warp == 20) {
        tmem_alloc(tm_ptr, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm_ptr;
    int n = 0, hd = 0;   // chunks and value heads so far

    if (warp == 21) {
        int ragged = 0, kq_in = 0, y_in = 0, u_in = 0, s_in = 0, d_in = 0;   // copies issued
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            int seq, c;
            if (!seqs.locate(item / a.Hk, C, seq, c)) continue;
            if (warp_up(guard)) break;
            const int hk = item % a.Hk, valid = min(C, seqs.len(seq) - c * C), y = seqs.start(seq) + c * C;
            // rows behind the sequence belong to another one, or to none: they are zeros here
            auto clear = [&](int tile, int panels, uint64_t* full) {
                wait(landed, ragged & 1, guard);
                ++ragged;
                for (int p = 0; p < panels; ++p)
                    for (int e = lane; e < (C - valid) * 8; e += 32)
                        *(uint4*)(sm + tile + p * PANEL + (valid + e / 8) * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                warp_arrive(full);
                __syncwarp();
            };
            if (lane == 0)   // K and Q come late: as far as L2 meanwhile
                for (int p = 0; p < DK / 64; ++p) {
                    prefetch_3d(&mk, p * 64, hk, y);
                    prefetch_3d(&mq, p * 64, hk, y);
                }
            for (int h = hk * r; h < hk * r + r; ++h, ++hd) {
                const char* mine = kept + ((int64_t)(item / a.Hk) * a.Hv + h) * keep.bytes();
                const char* rec = records + ((int64_t)(item / a.Hk) * a.Hv + h) * REC_BYTES;
                if (hd > 0) wait(y_empty, (hd - 1) & 1, guard);
                if (warp_up(guard)) break;
                if (lane == 0) {
                    uint64_t* bar = valid < C ? landed : y_full;
                    mbar_arrive_expect_tx(bar, C * DV * 2 + 2 * DV * C * 2 + 5 * C * 4);
                    bulk_load(sm + L::Y_, mine + keep.y(), 2 * DV * C * 2, bar);
                    for (int p = 0; p < DV / 64; ++p) tma_load_3d(sm + L::G_ + p * PANEL, &mg, bar, p * 64, h, y);
                    bulk_load(sm + L::SC + hd % 3 * 5 * C * 4, rec + REC_SCAL, 5 * C * 4, bar);
                    prefetch(mine + keep.u(), 3 * DV * C * 2);   // and R
                    prefetch(mine + keep.s(), 2 * DV * DK * 2);
                }
                ++y_in;
                __syncwarp();
                if (valid < C) clear(L::G_, DV / 64, y_full);
                if (hd > 0) wait(u_empty, (hd - 1) & 1, guard);
                if (warp_up(guard)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(u_full, 2 * DV * C * 2);
                    bulk_load(sm + L::U_, mine + keep.u(), 2 * DV * C * 2, u_full);
                }
                ++u_in;
                __syncwarp();
                if (hd > 0) wait(d_empty, (hd - 1) & 1, guard);
                if (warp_up(guard)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(s_full, 2 * DV * DK * 2);
                    bulk_load(sm + L::SD, mine + keep.s(), 2 * DV * DK * 2, s_full);
                    prefetch(mine + keep.d(), 2 * DV * DK * 2);
                }
                ++s_in;
                __syncwarp();
                if (h == hk * r) {
                    if (n > 0) wait(kq_empty, (n - 1) & 1, guard);
                    if (warp_up(guard)) break;
                    if (lane == 0) {
                        uint64_t* bar = valid < C ? landed : kq_full;
                        mbar_arrive_expect_tx(bar, 2 * C * DK * 2);
                        for (int p = 0; p < DK / 64; ++p) {
                            tma_load_3d(sm + L::K_ + p * PANEL, &mk, bar, p * 64, hk, y);
                            tma_load_3d(sm + L::Q_ + p * PANEL, &mq, bar, p * 64, hk, y);
                        }
                    }
                    ++kq_in;
                    __syncwarp();
                    if (valid < C) clear(L::Q_, 2 * (DK / 64), kq_full);
                }
                wait(s_done, hd & 1, guard);
                if (warp_up(guard)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(d_full, 2 * DV * DK * 2);
                    bulk_load(sm + L::SD, mine + keep.d(), 2 * DV * DK * 2, d_full);
                }
                ++d_in;
                __syncwarp();
            }
            ++n;
        }
        drain_ring(landed, 1, ragged);   // (those of ragged chunks land there)
        drain_ring(kq_full, 1, kq_in);
        drain_ring(y_full, 1, y_in);
        drain_ring(u_full, 1, u_in);
        drain_ring(s_full, 1, s_in);
        drain_ring(d_full, 1, d_in);
    } else if (warp == 20) {
        constexpr uint32_t id_rows = idesc_f16(128, C, true, false, false, true);    // right operand: its values are K
        constexpr uint32_t id_cols = idesc_f16(128, C, true, true, false, true);     // its rows are K
        constexpr int ST = DV * 128, KV = DV / 16;   // bytes of a panel of S, k-steps of the value columns
        const uint64_t ds = desc_cols(base + L::SD, ST), du = desc_cols(base + L::U_, ST), dy = desc_cols(base + L::Y_, ST);
        const uint64_t dg = desc_rows(base + L::G_), dkc = desc_cols(base + L::K_, PANEL), dqc = desc_cols(base + L::Q_, PANEL);
        const uint64_t dnc = desc_cols(base + L::N_, PANEL), dnr = desc_rows(base + L::N_);
        constexpr int S1 = DV * DK * 2 >> 4, U1 = DV * C * 2 >> 4, P1 = PANEL >> 4;   // second planes
        // products of planes 0 0, 0 1 and (all) 1 0, their rows as K; `left1` and U1: the second planes
        auto planes = [&](uint32_t to, uint64_t left, uint64_t right, int left1, bool all) {
#pragma unroll 1
            for (int p = 0; p < (all ? 3 : 2); ++p) {
                const uint64_t l = left + (p == 2 ? left1 : 0), w = right + (p == 1 ? U1 : 0);
#pragma unroll
                for (int x = 0; x < KV; ++x) umma_f16(to, step_cols(l, x), step_cols(w, x), id_cols, p + x > 0);
            }
        };
        auto by_dout = [&](uint32_t to, uint64_t left, int count) {
#pragma unroll 1
            for (int p = 0; p < count; ++p)
#pragma unroll
                for (int x = 0; x < KV; ++x) umma_f16(to, step_cols(left + p * S1, x), step_rows(dg, x, PANEL), id_rows, p + x > 0);
        };
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            int seq, c;
            if (!seqs.locate(item / a.Hk, C, seq, c)) continue;
            for (int i = 0; i < r; ++i, ++hd) {
                wait(y_full, hd & 1, guard);
                wait(u_full, hd & 1, guard);
                tc_fence_after();
                if (elect()) {
                    by_dout(tmem + L::E1, du, 1);
                    planes(tmem + L::E2, du, dy, 0, false);
                    umma_commit(e_done);
                }
                if (hd > 0) wait(acc_free, (hd - 1) & 1, guard);
                wait(s_full, hd & 1, guard);
                tc_fence_after();
                if (elect()) {
                    planes(tmem + L::XR, ds, dy, S1, true);
                    by_dout(tmem + L::XQ, ds, 2);
                    umma_commit(s_done);
                    umma_commit(y_empty);
                }
                if (i == 0) wait(kq_full, n & 1, guard);
                wait(nm_ready, hd & 1, guard);
                tc_fence_after();
                if (elect()) {
#pragma unroll 1
                    for (int m = 0; m < 2; ++m)   // NK, MK
#pragma unroll
                        for (int p = 0; p < 2; ++p)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                umma_f16(tmem + L::NK + 64 * m, step_cols(dkc, x), step_cols(dnc + (2 * m + p) * P1, x), id_cols, p + x > 0);
#pragma unroll 1
                    for (int m = 1; m >= 0; --m)   // CC: K by beta M, Q by N
#pragma unroll
                        for (int p = 0; p < 2; ++p)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                umma_f16(tmem + L::CC, step_cols(m ? dkc : dqc, x), step_rows(dnr + (2 * m + p) * P1, x, PANEL), id_rows, (1 - m) + p + x > 0);
                }
                wait(d_full, hd & 1, guard);
                tc_fence_after();
                if (elect()) {
                    planes(tmem + L::XC, ds, du, S1, true);
                    umma_commit(d_empty);
                    umma_commit(u_empty);
                    if (i + 1 == r) umma_commit(kq_empty);
                    umma_commit(out_done);
                }
            }
            ++n;
        }
        drain_mma(drain);
    } else if (warp < 4) {
        const int j = tid & 63, own = 32 * (warp >> 1);   // token of U, and 32 of the others
        const uint32_t at = tmem + ((uint32_t)warp * 32u << 16);
        char *sums = sm + L::N_ + tid * 128, *theirs = sm + L::N_ + (tid ^ 64) * 128;   // 128 rows of 32 sums, twice
        float* red = (float*)(sm + L::RED);
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            int seq, c;
            if (!seqs.locate(item / a.Hk, C, seq, c)) continue;
            const int hk = item % a.Hk;
            for (int i = 0; i < r; ++i, ++hd) {
                const float* scal = (const float*)(sm + L::SC + hd % 3 * 5 * C * 4);
                const char* mine = kept + ((int64_t)(item / a.Hk) * a.Hv + hk * r + i) * keep.bytes();
                if (hd > 0) wait(out_done, (hd - 1) & 1, guard);   // the planes have been read
                wait(y_full, hd & 1, guard);
                wait(e_done, hd & 1, guard);
                tc_fence_after();
                // The planes' sums: each of the two threads of a token hands over the columns that are not its own.
#pragma unroll 1
                for (int m = 0; m < 2; ++m) {
                    float x[32];
                    tmem_ld32(at + L::E1 + 64 * m + (own ^ 32), x);
#pragma unroll
                    for (int z = 0; z < 8; ++z)
                        *(float4*)(sums + m * 2 * PANEL + ((z ^ (tid & 7)) << 4)) = make_float4(x[4 * z], x[4 * z + 1], x[4 * z + 2], x[4 * z + 3]);
                }
                bar_sync(1, 128);
                const float hj = scal[3 * C + j], lj = scal[4 * C + j];
#pragma unroll 1
                for (int m = 0; m < 2; ++m) {   // N, beta M
                    uint32_t p[2][16];
#pragma unroll
                    for (int w = 0; w < 32; w += 16) {
                        float y[16];
                        tmem_ld16(at + L::E1 + 64 * m + own + w, y);
#pragma unroll
                        for (int z = 0; z < 16; z += 4) {
                            const int i0 = own + w + z;
                            const float4 v = *(const float4*)(theirs + m * 2 * PANEL + ((((w + z) >> 2) ^ (tid & 7)) << 4));
                            const float4 hi = *(const float4*)&scal[3 * C + i0], li = *(const float4*)&scal[4 * C + i0], be = *(const float4*)&scal[2 * C + i0];
                            const float vv[4] = {v.x, v.y, v.z, v.w}, hh[4] = {hi.x, hi.y, hi.z, hi.w}, ll[4] = {li.x, li.y, li.z, li.w}, bb[4] = {be.x, be.y, be.z, be.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float d = ex2_approx((hh[e] - hj) + (ll[e] - lj));
                                y[z + e] = j + m <= i0 + e ? (m ? -at_least(bb[e]) : 1.f) * (d * (y[z + e] + vv[e])) : 0.f;
                            }
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                uint32_t q[2];
                                split<2>(y[z + e], y[z + e + 1], q);
                                p[0][(w + z + e) / 2] = q[0];
                                p[1][(w + z + e) / 2] = q[1];
                            }
                        }
                    }
                    bar_sync(1, 128);   // the sums have been read: the planes take their place
                    to_tile<C>(sm + L::N_ + m * 2 * PANEL, j, own / 8, p[0]);
                    to_tile<C>(sm + L::N_ + m * 2 * PANEL + PANEL, j, own / 8, p[1]);
                }
                tc_fence_before();
                fence_async_smem();
                warp_arrive(nm_ready);
                warp_arrive(out_done);   // (whoever waits for it sees the gates as well)
                // dY . R: 8 tokens a thread, its rows strided by 16
                {
                    const int row = tid >> 3, piece = tid & 7;
                    float acc[8] = {};
#pragma unroll 1
                    for (int z0 = 0; z0 < DV / 16; z0 += 4) {
                        uint4 rr[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) rr[z] = __ldcg((const uint4*)(mine + keep.r() + tile_at<C>(row + 16 * (z0 + z), piece)));
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const uint32_t off = L::Y_ + tile_at<C>(row + 16 * (z0 + z), piece);
                            const uint4 y0 = *(const uint4*)(sm + off), y1 = *(const uint4*)(sm + DV * C * 2 + off);
                            const uint32_t rv[4] = {rr[z].x, rr[z].y, rr[z].z, rr[z].w}, a0[4] = {y0.x, y0.y, y0.z, y0.w}, a1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                acc[2 * e] = fmaf(low(a0[e]) + low(a1[e]), low(rv[e]), acc[2 * e]);
                                acc[2 * e + 1] = fmaf(high(a0[e]) + high(a1[e]), high(rv[e]), acc[2 * e + 1]);
                            }
                        }
                    }
                    warp_arrive(y_empty);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        acc[e] += __shfl_xor_sync(~0u, acc[e], 8);
                        acc[e] += __shfl_xor_sync(~0u, acc[e], 16);
                        if (lane < 8) red[(hd & 1) * L::RY + warp * C + piece * 8 + e] = acc[e];
                    }
                }
                if (hd > 0) wait(sum_free, (hd - 1) & 1, guard);   // two heads' sums at most are on their way
                warp_arrive(ry_ready);
            }
            ++n;
        }
    } else {
        const int tok = 16 * ((warp - 4) >> 2), w4 = warp & 3, row = tid & 127;   // 16 tokens from tok on, channel
        const uint32_t at = tmem + ((uint32_t)w4 * 32u << 16) + tok;
        float* red = (float*)(sm + L::RED);
        const bool real = DK == 128 || row < DK;
        const char* ch = sm + (DK > 64 ? row >> 6 : 0) * PANEL + (row & 7) * 2;   // the channel's column of Q and K
        const int pc = (row & 63) >> 3;
        auto value = [&](int tile, int t) { return __uint_as_float((uint32_t)*(const uint16_t*)(ch + tile + piece_at(tok + t, pc)) << 16); };
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            int seq, c;
            if (!seqs.locate(item / a.Hk, C, seq, c)) continue;
            const int hk = item % a.Hk, valid = min(C, seqs.len(seq) - c * C);
            const int64_t t0 = (int64_t)seqs.start(seq) + c * C;
            // the sums over the value heads so far, fp32 [2][64][Dk], in the place of the first one's S and D
            float* so_far = (float*)(kept + ((int64_t)(item / a.Hk) * a.Hv + hk * r) * keep.bytes()) + tok * DK + row;
            for (int i = 0; i < r; ++i, ++hd) {
                const int h = hk * r + i;
                const float* scal = (const float*)(sm + L::SC + hd % 3 * 5 * C * 4) + tok;
                const char* mine = kept + ((int64_t)(item / a.Hk) * a.Hv + h) * keep.bytes();
                float ex = 0.f;
                {   // <S, D>, 16 bytes of each plane a thread and round; S once more from L2
                    constexpr int PIECES = DV * DK * 2 / (512 * 16);
                    const char *s = mine + keep.s() + (tid - 128) * 16, *d = sm + L::SD + (tid - 128) * 16;
                    uint4 sp[2][PIECES];
#pragma unroll
                    for (int z = 0; z < PIECES; ++z)
#pragma unroll
                        for (int q = 0; q < 2; ++q) sp[q][z] = __ldcg((const uint4*)(s + q * keep.state() + z * 8192));
                    wait(d_full, hd & 1, guard);
#pragma unroll
                    for (int z = 0; z < PIECES; ++z) {
                        const uint4 d0 = *(const uint4*)(d + z * 8192), d1 = *(const uint4*)(d + DV * DK * 2 + z * 8192);
                        const uint32_t ss[2][4] = {{sp[0][z].x, sp[0][z].y, sp[0][z].z, sp[0][z].w}, {sp[1][z].x, sp[1][z].y, sp[1][z].z, sp[1][z].w}};
                        const uint32_t dd[2][4] = {{d0.x, d0.y, d0.z, d0.w}, {d1.x, d1.y, d1.z, d1.w}};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            ex = fmaf(low(dd[0][e]) + low(dd[1][e]), low(ss[0][e]) + low(ss[1][e]),
                                      fmaf(high(dd[0][e]) + high(dd[1][e]), high(ss[0][e]) + high(ss[1][e]), ex));
                    }
                    warp_arrive(d_empty);
                    if (i == 0 && r > 1) bar_sync(2, 512);   // every warp has read S: the sums so far take its place
                }
                if (i == 0) wait(kq_full, n & 1, guard);
                wait(out_done, hd & 1, guard);
                ex *= scal[C - 1 - tok];
                tc_fence_after();
#pragma unroll 1
                for (int z = 0; z < 16; z += 8) {   // (a loop: see the scans)
                    float u[8], v[8], k[8], dq[8], dk[8], dc[8], db[8];
                    // row part of dK: (beta M) K - beta e^cum o (dY S^T), and k . (beta M K)
                    tmem_ld8(at + L::XR + z, u);
                    tmem_ld8(at + L::MK + z, v);
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        const float be = scal[2 * C + z + t], mk = real ? v[t] : 0.f;
                        k[t] = real ? value(L::K_, z + t) : 0.f;
                        dk[t] = real ? fmaf(-be * scal[z + t], u[t], at_least(be) == be ? mk : mk * (be * 16777216.f)) : 0.f;   // (2^24)
                        dc[t] = k[t] * dk[t];
                        db[t] = k[t] * mk;
                    }
                    // dQ = e^cum o (dO S^T) + N K
                    tmem_ld8(at + L::XQ + z, u);
                    tmem_ld8(at + L::NK + z, v);
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        dq[t] = real ? fmaf(scal[z + t], u[t], v[t]) : 0.f;
                        if (real) dc[t] = fmaf(value(L::Q_, z + t), dq[t], dc[t]);
                    }
                    // column part: e^{cum_C - cum} o (U D^T) + (beta M)^T K + N^T Q
                    tmem_ld8(at + L::XC + z, u);
                    tmem_ld8(at + L::CC + z, v);
                    if (z == 8) {
                        tc_fence_before();
                        warp_arrive(acc_free);
                        if (i + 1 == r) warp_arrive(kq_empty);
                    }
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        const float g = real ? scal[C + z + t] * u[t] : 0.f, f = real ? g + v[t] : 0.f;
                        dk[t] += f;
                        ex = fmaf(k[t], g, ex);
                        dc[t] = fmaf(-k[t], f, dc[t]);
                    }
                    const float s0 = transpose_sum(db, lane), s1 = transpose_sum(dc, lane);
                    if (lane < 8) {
                        red[L::DB + w4 * C + tok + z + lane] = s0 / at_least(scal[2 * C + z + lane]);
                        red[L::DC + w4 * C + tok + z + lane] = s1;
                    }
                    if (i > 0 && real)
#pragma unroll
                        for (int t = 0; t < 8; ++t) {
                            dq[t] += so_far[(z + t) * DK];
                            dk[t] += so_far[(C + z + t) * DK];
                        }
                    if (i + 1 < r) {
                        if (real)
#pragma unroll
                            for (int t = 0; t < 8; ++t) {
                                so_far[(z + t) * DK] = dq[t];
                                so_far[(C + z + t) * DK] = dk[t];
                            }
                    } else {
                        // even lanes take the even tokens of their channel and the next, odd lanes the odd ones
                        const bool odd = lane & 1;
                        const int64_t off = ((t0 + tok + z + odd) * a.Hk + hk) * DK + row - odd, step = 2 * (int64_t)a.Hk * DK;
#pragma unroll
                        for (int t = 0; t < 8; t += 2) {
                            const float q1 = __shfl_xor_sync(~0u, odd ? dq[t] : dq[t + 1], 1), k1 = __shfl_xor_sync(~0u, odd ? dk[t] : dk[t + 1], 1);
                            if (real && tok + z + t + odd < valid) {
                                *(uint32_t*)((__nv_bfloat16*)b.dq + off + t / 2 * step) = odd ? pack(q1, dq[t + 1]) : pack(dq[t], q1);
                                *(uint32_t*)((__nv_bfloat16*)b.dk + off + t / 2 * step) = odd ? pack(k1, dk[t + 1]) : pack(dk[t], k1);
                            }
                        }
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) ex += __shfl_xor_sync(~0u, ex, o);
                if (lane == 0) red[L::EX + warp - 4] = ex;
                wait(ry_ready, hd & 1, guard);
                bar_sync(2, 512);
                if (warp == 4) {   // dg: suffix sums of dcum, two tokens a lane, and the exit term
                    float all = lane < 16 ? red[L::EX + lane] : 0.f;
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) all += __shfl_xor_sync(~0u, all, o);
                    all = __shfl_sync(~0u, all, 0);
                    float d0 = 0.f, d1 = 0.f;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        d0 += red[L::DC + w * C + 2 * lane];
                        d1 += red[L::DC + w * C + 2 * lane + 1];
                    }
                    float sum = d0 + d1;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const float y = __shfl_down_sync(~0u, sum, o);
                        if (lane + o < 32) sum += y;
                    }
                    __nv_bfloat16* dst = (__nv_bfloat16*)b.dg + t0 * a.Hv + h;
                    if (2 * lane < valid) dst[(int64_t)(2 * lane) * a.Hv] = __float2bfloat16_rn(sum + all);
                    if (2 * lane + 1 < valid) dst[(int64_t)(2 * lane + 1) * a.Hv] = __float2bfloat16_rn(sum - d0 + all);
                } else if (warp >= 8 && warp < 10) {
                    const int t = tid & 63;
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < 4; ++w) sum += red[(hd & 1) * L::RY + w * C + t] + red[L::DB + w * C + t];
                    if (t < valid) ((__nv_bfloat16*)b.dbeta)[(t0 + t) * a.Hv + h] = __float2bfloat16_rn(sum);
                }
                warp_arrive(sum_free);
                bar_sync(2, 512);   // the next head's sums take these' place
            }
            ++n;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 20) tmem_dealloc(tmem, 512);
}

template <int DK, int DV>
cudaError_t tgrads(const GdnBwdArgs& b, const Seqs& s, const void* records, void* kept, int sms, int* status, cudaStream_t st)
{
    using L = TGrads<DK, DV>;
    CUtensorMap k{}, q{}, g{};
    const GdnArgs& a = b.f;
    const int64_t T = s.tokens(), items = (int64_t)s.slots(C) * a.Hk;
    if (!make_map(&k, a.k, T, a.Hk, DK, 64, 1, C) || !make_map(&q, a.q, T, a.Hk, DK, 64, 1, C) || !make_map(&g, b.dout, T, a.Hv, DV, 64, 1, C))
        return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<gdn_tgrads_kernel<DK, DV>>(L::SMEM);
    if (e != cudaSuccess) return e;
    ProfileScope prof("gdn_grads", st);
    count_launch();
    gdn_tgrads_kernel<DK, DV><<<(unsigned)min(items, (int64_t)sms), L::THREADS, L::SMEM, st>>>(k, q, g, b, s, (const char*)records, (char*)kept, status, debug_drop_handoff());
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_grads(const GdnBwdArgs& b, const Seqs& s, const void* records, void* kept, int sms, int* status, cudaStream_t st)
{
    if (b.f.Dk == 64) return b.f.Dv == 64 ? tgrads<64, 64>(b, s, records, kept, sms, status, st) : tgrads<64, 128>(b, s, records, kept, sms, status, st);
    return b.f.Dv == 64 ? tgrads<128, 64>(b, s, records, kept, sms, status, st) : tgrads<128, 128>(b, s, records, kept, sms, status, st);
}

}  // namespace gdn
}  // namespace kda
