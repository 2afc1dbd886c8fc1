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
// One CTA per SM takes chunks of key heads in turn, and the value heads of each one after another.
//
//   warps 0-15 (four warpgroups) E1 -> N, E2 -> beta M and its part of dbeta; dY . R; <S, D>; then all
//              sums over the key channels, a channel a lane, 16 tokens a warpgroup
//   warp 16    issues the MMAs
//   warp 17    the loads: S and then D share a buffer; each goes on as soon as its buffer is free, into the next
//              head and chunk
//
// What bounds it: the tiles of a chunk and value head are 208 KB at Dk = Dv = 128, 0.14 ms of HBM at the image stream.
//
// Every wait is bounded; after one runs out all roles run to their end on whatever is there.

#include "gdn_whole.cuh"

namespace kda {
namespace gdn {
namespace {

template <int DK, int DV>
struct TGrads {
    static constexpr int THREADS = 576;
    // (Q before K: with the rows of K as the lower half of a product's, the upper half reads Q's panels)
    static constexpr int Q_ = 0, K_ = Q_ + DK / 64 * PANEL;
    static constexpr int SD = K_ + DK / 64 * PANEL;          // planes of S^T, then of D^T [2][DK / 64][DV][64]
    static constexpr int U_ = SD + 2 * DV * DK * 2;          // planes of U^T [2][DV][64]
    static constexpr int Y_ = U_ + 2 * DV * C * 2;           // of dY^T
    static constexpr int G_ = Y_ + 2 * DV * C * 2;           // dO
    static constexpr int N_ = G_ + DV / 64 * PANEL;          // planes of N^T [2][64][64], then of beta M^T
    static constexpr int SC = N_ + 4 * PANEL;                // grow, end, beta, cum, of two heads
    static constexpr int RED = SC + 2 * 5 * C * 4;               // fp32: dY.R [16][64], dbeta [2][64], dcum [4][64], exit [16]
    static constexpr int BAR = RED + 22 * C * 4 + 64;
    static constexpr int SMEM = BAR + 256 + 1024 > 116 * 1024 ? BAR + 256 + 1024 : 116 * 1024;   // one CTA to an SM
    static constexpr int XQ = 0, XR = 64, XC = 128, CC = 192, NK = 256, MK = 320, E1 = 384, E2 = 448;   // tensor memory
};

// v[c], c = 0 .. 15, summed over the warp: lanes c and c + 16 get the sum of v[c]
__device__ __forceinline__ float transpose_sum(float (&v)[16], int lane)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int k = 0; k < o; ++k) {
            const float give = up ? v[k] : v[k + o], keep = up ? v[k + o] : v[k];
            v[k] = keep + __shfl_xor_sync(~0u, give, o);
        }
    }
    return v[0] + __shfl_xor_sync(~0u, v[0], 16);
}
__device__ __forceinline__ void load16(float (&x)[16], const float* f)
{
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        const float4 v = *(const float4*)(f + i);
        x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
}

template <int DK, int DV>
__global__ void __launch_bounds__(576, 1)
gdn_tgrads_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                  const __grid_constant__ CUtensorMap mdq, const __grid_constant__ CUtensorMap mdk, GdnBwdArgs b, const __grid_constant__ Seqs seqs, const char* records, const char* kept, int* status)
{
    using L = TGrads<DK, DV>;
    const GdnArgs& a = b.f;
    extern __shared__ char raw[];
    char* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t base = smem_addr(sm);
    uint64_t* bars = (uint64_t*)(sm + L::BAR);
    uint64_t *kq_full = bars, *kq_empty = bars + 1, *y_full = bars + 2, *y_empty = bars + 3, *s_full = bars + 4, *s_done = bars + 5;
    uint64_t *d_full = bars + 6, *d_empty = bars + 7, *landed = bars + 8, *e_done = bars + 9, *kk_done = bars + 10, *kk_read = bars + 11;
    uint64_t *nm_ready = bars + 12, *out_done = bars + 13, *acc_free = bars + 14, *drain = bars + 15, *u_full = bars + 16, *u_empty = bars + 17;
    uint32_t* tm_ptr = (uint32_t*)(bars + 18);
    const Guard guard{(volatile int*)(tm_ptr + 1), status};

    const int tid = threadIdx.x, lane = tid & 31, warp = uniform_warp();
    const int r = a.Hv / a.Hk, items = seqs.slots(C) * a.Hk;
    const Kept keep{DK, DV};

    if (warp == 17) {
        if (lane == 0) {
            for (uint64_t* x : {kq_full, y_full, u_full, u_empty, s_full, s_done, d_full, landed, e_done, kk_done, out_done, drain}) mbar_init(x, 1);
            for (uint64_t* x : {kq_empty, y_empty, d_empty}) mbar_init(x, 17);   // the MMAs and warps 0-15
            for (uint64_t* x : {nm_ready, acc_free}) mbar_init(x, 16);
            mbar_init(kk_read, 8);
            *guard.flag = 0;
            fence_mbar_init();
            fence_async_smem();
        }
    } else if (warp == 16) {
        tmem_alloc(tm_ptr, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm_ptr;
    int n = 0, hd = 0;   // chunks and value heads so far

    if (warp == 17) {
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
                    bulk_load(sm + L::SC + (hd & 1) * 5 * C * 4, rec + REC_SCAL, 5 * C * 4, bar);
                }
                ++y_in;
                __syncwarp();
                if (valid < C) clear(L::G_, DV / 64, y_full);
                if (hd > 0) wait(u_empty, (hd - 1) & 1, guard);
                if (warp_up(guard)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(u_full, 2 * DV * C * 2);
                    bulk_load(sm + L::U_, mine + keep.u(), 2 * DV * C * 2, u_full);
                    prefetch(mine + keep.r(), DV * C * 2);
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
        if (warp_up(guard)) {   // copies still on their way (those of ragged chunks land on `landed`)
            if (ragged > 0) mbar_wait_bounded(landed, (ragged - 1) & 1, kWaitNs);
            if (kq_in > 0) mbar_wait_bounded(kq_full, (kq_in - 1) & 1, kWaitNs);
            if (y_in > 0) mbar_wait_bounded(y_full, (y_in - 1) & 1, kWaitNs);
            if (u_in > 0) mbar_wait_bounded(u_full, (u_in - 1) & 1, kWaitNs);
            if (s_in > 0) mbar_wait_bounded(s_full, (s_in - 1) & 1, kWaitNs);
            if (d_in > 0) mbar_wait_bounded(d_full, (d_in - 1) & 1, kWaitNs);
        }
    } else if (warp == 16) {
        constexpr uint32_t id_rows = idesc_f16(128, C, true, false, false, true);    // right operand: its values are K
        constexpr uint32_t id_cols = idesc_f16(128, C, true, true, false, true);     // its rows are K
        constexpr uint32_t id_kk = idesc_f16(128, 32, false, false, false, true);
        constexpr int ST = DV * 128, KV = DV / 16;   // bytes of a panel of S, k-steps of the value columns
        const uint64_t ds = desc_cols(base + L::SD, ST), du = desc_cols(base + L::U_, ST), dy = desc_cols(base + L::Y_, ST);
        const uint64_t dg = desc_rows(base + L::G_), dkc = desc_cols(base + L::K_, PANEL), dqc = desc_cols(base + L::Q_, PANEL);
        const uint64_t dnc = desc_cols(base + L::N_, PANEL), dnr = desc_rows(base + L::N_), dk = desc_rows(base + L::K_);
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
                }
                if (i == 0) {   // K K^T: columns 0-31 for rows 0-63, 32-63 for rows 64-127, where the threads want them
                    wait(kq_full, n & 1, guard);
                    tc_fence_after();
                    if (elect()) {
#pragma unroll 1
                        for (int z = 0; z < 2; ++z)
#pragma unroll
                            for (int x = 0; x < DK / 16; ++x)
                                umma_f16(tmem + L::XQ + 32 * z, step_rows(dk - z * P1, x, PANEL), step_rows(dk + (z * 4096 >> 4), x, PANEL), id_kk, x > 0);
                        umma_commit(kk_done);
                    }
                    wait(kk_read, n & 1, guard);
                    tc_fence_after();
                }
                if (elect()) {
                    by_dout(tmem + L::XQ, ds, 2);
                    umma_commit(s_done);
                    umma_commit(y_empty);
                }
                wait(nm_ready, hd & 1, guard);
                tc_fence_after();
                if (elect()) {
#pragma unroll 1
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            umma_f16(tmem + L::NK, step_cols(dkc, x), step_cols(dnc + p * P1, x), id_cols, p + x > 0);
                            umma_f16(tmem + L::MK, step_cols(dkc, x), step_cols(dnc + (2 + p) * P1, x), id_cols, p + x > 0);
                        }
#pragma unroll 1
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            umma_f16(tmem + L::CC, step_cols(dkc, x), step_rows(dnr + (2 + p) * P1, x, PANEL), id_rows, p + x > 0);
                            umma_f16(tmem + L::CC, step_cols(dqc, x), step_rows(dnr + p * P1, x, PANEL), id_rows, 1);
                        }
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
        if (warp_up(guard)) {
            if (elect()) umma_commit(drain);
            mbar_wait_bounded(drain, 0, kWaitNs);
        }
    } else {
        // Warpgroup g: of the pairs, N (0, 1) or M (2, 3), columns 16 z .. of either half of the tokens; of the
        // sums over the channels, tokens 16 g ..
        const int g = warp >> 2, m = g >> 1, w4 = warp & 3, row = tid & 127, j = row & 63, own = 32 * (w4 >> 1) + 16 * (g & 1), other = own ^ 32;
        const uint32_t at = tmem + ((uint32_t)w4 * 32u << 16);
        float* red = (float*)(sm + L::RED);
        const bool real = row < DK;
        const int ch = (DK > 64 ? row >> 6 : 0) * PANEL + (row & 7) * 2, pc = (row & 63) >> 3;   // a channel's column of K and Q
        char* planes = sm + L::N_ + m * 2 * PANEL;            // N's or beta M's
        char* sums = sm + L::N_ + g * PANEL;                  // before them, 128 x 16 sums
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            int seq, c;
            if (!seqs.locate(item / a.Hk, C, seq, c)) continue;
            const int hk = item % a.Hk, valid = min(C, seqs.len(seq) - c * C);
            const int64_t t0 = (int64_t)seqs.start(seq) + c * C;
            float sq[16] = {}, sk[16] = {}, kk[16] = {};
            for (int i = 0; i < r; ++i, ++hd) {
                const int h = hk * r + i;
                const float* scal = (const float*)(sm + L::SC + (hd & 1) * 5 * C * 4);
                const char* mine = kept + ((int64_t)(item / a.Hk) * a.Hv + h) * keep.bytes();
                // dY . R: 8 tokens a thread, its rows strided by 64
                {
                    uint4 rr[DV / 64];
                    const int at_row = tid >> 3, piece = tid & 7;
#pragma unroll
                    for (int z = 0; z < DV / 64; ++z) rr[z] = __ldcg((const uint4*)(mine + keep.r() + tile_at<C>(at_row + 64 * z, piece)));
                    wait(y_full, hd & 1, guard);
                    float acc[8] = {};
#pragma unroll
                    for (int z = 0; z < DV / 64; ++z) {
                        const uint4 y0 = *(const uint4*)(sm + L::Y_ + tile_at<C>(at_row + 64 * z, piece));
                        const uint4 y1 = *(const uint4*)(sm + L::Y_ + DV * C * 2 + tile_at<C>(at_row + 64 * z, piece));
                        const uint32_t rv[4] = {rr[z].x, rr[z].y, rr[z].z, rr[z].w}, a0[4] = {y0.x, y0.y, y0.z, y0.w}, a1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            acc[2 * e] = fmaf(low(a0[e]) + low(a1[e]), low(rv[e]), acc[2 * e]);
                            acc[2 * e + 1] = fmaf(high(a0[e]) + high(a1[e]), high(rv[e]), acc[2 * e + 1]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        acc[e] += __shfl_xor_sync(~0u, acc[e], 8);
                        acc[e] += __shfl_xor_sync(~0u, acc[e], 16);
                        if (lane < 8) red[warp * C + piece * 8 + e] = acc[e];
                    }
                    warp_arrive(y_empty);
                }
                if (i == 0 && m) {
                    wait(kk_done, n & 1, guard);
                    tc_fence_after();
                    tmem_ld16(at + L::XQ + own, kk);
                    tc_fence_before();
                    warp_arrive(kk_read);
                }
                if (i == 0) {   // dq and dk of the chunk before have been read from where the sums go
                    if (tid == 0) bulk_wait_read0();
                    bar_sync(3, 512);
                }
                // E: token j of U, 16 of the other tokens.  The planes' sums: each of the two threads of a token hands
                // over the columns that are not its own.
                wait(e_done, hd & 1, guard);
                tc_fence_after();
                float x[16];
                const uint32_t e = at + (m ? L::E2 : L::E1);
                tmem_ld16(e + other, x);
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    *(float4*)(sums + row * 64 + ((z ^ ((row >> 1) & 3)) << 4)) = make_float4(x[4 * z], x[4 * z + 1], x[4 * z + 2], x[4 * z + 3]);
                tmem_ld16(e + own, x);
                bar_sync(1 + m, 256);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const float4 v = *(const float4*)(sums + (row ^ 64) * 64 + ((z ^ ((row >> 1) & 3)) << 4));
                    x[4 * z] += v.x; x[4 * z + 1] += v.y; x[4 * z + 2] += v.z; x[4 * z + 3] += v.w;
                }
                {
                    float hi[16], li[16];
                    load16(hi, scal + 3 * C + own);
                    load16(li, scal + 4 * C + own);
                    const float hj = scal[3 * C + j], lj = scal[4 * C + j];
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        const float d = ex2_approx((hi[t] - hj) + (li[t] - lj));
                        x[t] = m ? (j < own + t ? -d * x[t] : 0.f) : (j <= own + t ? d * x[t] : 0.f);
                    }
                }
                if (m) {   // M: its part of dbeta, then beta M
                    float v[16];
#pragma unroll
                    for (int t = 0; t < 16; ++t) v[t] = j < own + t ? x[t] * kk[t] : 0.f;
                    const float s = transpose_sum(v, lane);
                    if (lane < 16) red[(16 + (w4 & 1)) * C + own + lane] = s;
                    load16(v, scal + 2 * C + own);
#pragma unroll
                    for (int t = 0; t < 16; ++t) x[t] *= v[t];
                }
                bar_sync(1 + m, 256);   // the sums have been read: the planes take their place
                {
                    uint32_t p[2][8];
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        uint32_t w[2];
                        split<2>(x[2 * t], x[2 * t + 1], w);
                        p[0][t] = w[0];
                        p[1][t] = w[1];
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int z = 0; z < 2; ++z)
                            *(uint4*)(planes + q * PANEL + piece_at(j, (own >> 3) + z)) = make_uint4(p[q][4 * z], p[q][4 * z + 1], p[q][4 * z + 2], p[q][4 * z + 3]);
                }
                tc_fence_before();
                fence_async_smem();
                warp_arrive(nm_ready);
                // <S, D>, 16 bytes of each plane a thread and round; S once more from L2
                float ex = 0.f;
                {
                    constexpr int PIECES = DV * DK * 2 / (512 * 16);
                    const char *s = mine + keep.s() + tid * 16, *d = sm + L::SD + tid * 16;
                    uint4 sp[2][PIECES];
#pragma unroll
                    for (int z = 0; z < PIECES; ++z) {
                        sp[0][z] = __ldcg((const uint4*)(s + z * 8192));
                        sp[1][z] = __ldcg((const uint4*)(s + keep.state() + z * 8192));
                    }
                    wait(d_full, hd & 1, guard);
#pragma unroll
                    for (int z = 0; z < PIECES; ++z) {
                        const uint4 d0 = *(const uint4*)(d + z * 8192), d1 = *(const uint4*)(d + DV * DK * 2 + z * 8192);
                        const uint32_t ss[2][4] = {{sp[0][z].x, sp[0][z].y, sp[0][z].z, sp[0][z].w}, {sp[1][z].x, sp[1][z].y, sp[1][z].z, sp[1][z].w}};
                        const uint32_t dd[2][4] = {{d0.x, d0.y, d0.z, d0.w}, {d1.x, d1.y, d1.z, d1.w}};
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            ex = fmaf(low(dd[0][y]) + low(dd[1][y]), low(ss[0][y]) + low(ss[1][y]),
                                      fmaf(high(dd[0][y]) + high(dd[1][y]), high(ss[0][y]) + high(ss[1][y]), ex));
                    }
                    ex *= scal[C - 1];
                }
                warp_arrive(d_empty);
                // channel `row`, 16 tokens
                if (i == 0) wait(kq_full, n & 1, guard);
                wait(out_done, hd & 1, guard);
                tc_fence_after();
                const int tok = 16 * g;
                float dc[16];
                {
                    float u[16], v[16], f[16], k[16];
                    auto value = [&](int tile, int t) { return __uint_as_float((uint32_t)*(const uint16_t*)(sm + tile + ch + piece_at(tok + t, pc)) << 16); };
                    // dQ = e^cum o (dO S^T) + N K
                    tmem_ld16(at + L::XQ + tok, u);
                    tmem_ld16(at + L::NK + tok, v);
                    load16(f, scal + tok);
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        const float w = fmaf(f[t], u[t], v[t]);
                        sq[t] += w;
                        dc[t] = real ? value(L::Q_, t) * w : 0.f;
                    }
                    // row part of dK: (beta M) K - beta e^cum o (dY S^T)
                    load16(k, scal + 2 * C + tok);
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        f[t] *= -k[t];
                        k[t] = value(L::K_, t);
                    }
                    tmem_ld16(at + L::XR + tok, u);
                    tmem_ld16(at + L::MK + tok, v);
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        const float w = fmaf(f[t], u[t], v[t]);
                        sk[t] += w;
                        if (real) dc[t] = fmaf(k[t], w, dc[t]);
                    }
                    // column part: e^{cum_C - cum} o (U D^T) + (beta M)^T K + N^T Q
                    tmem_ld16(at + L::XC + tok, u);
                    tmem_ld16(at + L::CC + tok, v);
                    tc_fence_before();
                    warp_arrive(acc_free);
                    load16(f, scal + C + tok);
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        const float y = f[t] * u[t], w = y + v[t];
                        sk[t] += w;
                        if (real) {
                            ex = fmaf(k[t], y, ex);
                            dc[t] = fmaf(-k[t], w, dc[t]);
                        }
                    }
                }
                if (i + 1 == r) warp_arrive(kq_empty);
                const float s = transpose_sum(dc, lane);
                if (lane < 16) red[(18 + w4) * C + tok + lane] = s;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) ex += __shfl_xor_sync(~0u, ex, o);
                if (lane == 0) red[22 * C + warp] = ex;
                if (i + 1 == r && real) {   // dq and dk, as tiles in the place of N and M
                    const int col = (DK > 64 ? row >> 6 : 0) * PANEL + (row & 7) * 2;
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        *(__nv_bfloat16*)(sm + L::N_ + col + piece_at(tok + t, pc)) = __float2bfloat16_rn(sq[t]);
                        *(__nv_bfloat16*)(sm + L::N_ + 2 * PANEL + col + piece_at(tok + t, pc)) = __float2bfloat16_rn(sk[t]);
                    }
                    fence_async_smem();
                }
                bar_sync(3, 512);
                if (warp == 0) {   // dg: suffix sums of dcum, two tokens a lane, and the exit term
                    float all = lane < 16 ? red[22 * C + lane] : 0.f;
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) all += __shfl_xor_sync(~0u, all, o);
                    all = __shfl_sync(~0u, all, 0);
                    float d0 = 0.f, d1 = 0.f;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        d0 += red[(18 + w) * C + 2 * lane];
                        d1 += red[(18 + w) * C + 2 * lane + 1];
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
                } else if (warp >= 4 && warp < 6) {
                    const int t = tid & 63;
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < 18; ++w) sum += red[w * C + t];
                    if (t < valid) ((__nv_bfloat16*)b.dbeta)[(t0 + t) * a.Hv + h] = __float2bfloat16_rn(sum);
                }
                if (i + 1 == r) {
                    if (valid == C) {
                        if (tid == 0) {
                            for (int p = 0; p < DK / 64; ++p) {
                                store_3d(&mdq, sm + L::N_ + p * PANEL, p * 64, hk, (int)t0);
                                store_3d(&mdk, sm + L::N_ + (2 + p) * PANEL, p * 64, hk, (int)t0);
                            }
                            bulk_commit();
                        }
                    } else {   // the rows behind the sequence are not its own
                        for (int z = tid; z < 2 * valid * (DK / 8); z += 512) {
                            const int which = z & 1, piece = (z >> 1) % (DK / 8), t = (z >> 1) / (DK / 8);
                            *(uint4*)((__nv_bfloat16*)(which ? b.dk : b.dq) + ((t0 + t) * a.Hk + hk) * DK + piece * 8) =
                                *(const uint4*)(sm + L::N_ + which * 2 * PANEL + piece / 8 * PANEL + piece_at(t, piece & 7));
                        }
                    }
                }
                bar_sync(3, 512);   // the next head's sums take these' place
            }
            ++n;
        }
        if (tid == 0) bulk_wait0();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 16) tmem_dealloc(tmem, 512);
}

template <int DK, int DV>
cudaError_t tgrads(const GdnBwdArgs& b, const Seqs& s, const void* records, const void* kept, int sms, int* status, cudaStream_t st)
{
    using L = TGrads<DK, DV>;
    CUtensorMap k{}, q{}, g{}, dq{}, dk{};
    const GdnArgs& a = b.f;
    const int64_t T = s.tokens(), items = (int64_t)s.slots(C) * a.Hk;
    if (!make_map(&k, a.k, T, a.Hk, DK, 64, 1, C) || !make_map(&q, a.q, T, a.Hk, DK, 64, 1, C) || !make_map(&g, b.dout, T, a.Hv, DV, 64, 1, C) ||
        !make_map(&dq, b.dq, T, a.Hk, DK, 64, 1, C) || !make_map(&dk, b.dk, T, a.Hk, DK, 64, 1, C))
        return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<gdn_tgrads_kernel<DK, DV>>(L::SMEM);
    if (e != cudaSuccess) return e;
    ProfileScope prof("gdn_grads", st);
    count_launch();
    gdn_tgrads_kernel<DK, DV><<<(unsigned)min(items, (int64_t)sms), L::THREADS, L::SMEM, st>>>(k, q, g, dq, dk, b, s, (const char*)records, (const char*)kept, status);
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_grads(const GdnBwdArgs& b, const Seqs& s, const void* records, const void* kept, int sms, int* status, cudaStream_t st)
{
    if (b.f.Dk == 64) return b.f.Dv == 64 ? tgrads<64, 64>(b, s, records, kept, sms, status, st) : tgrads<64, 128>(b, s, records, kept, sms, status, st);
    return b.f.Dv == 64 ? tgrads<128, 64>(b, s, records, kept, sms, status, st) : tgrads<128, 128>(b, s, records, kept, sms, status, st);
}

}  // namespace gdn
}  // namespace kda
