// The reverse scan of the gated delta rule's backward on tcgen05 tensor cores (bf16; Dk and Dv 64 or 128),
// one CTA per sequence and value head.
//
// The mathematics is that of gdn_bwd.cu's reverse scan, the division of work that of gdn_chain.cu: all
// value columns are the 128 rows of every product.  D (the gradient of a chunk's exit state), dU and dV are
// left operands in tensor memory, K, Q, T and P right ones in shared memory.
//
//   warps 0-7  (two warpgroups, each with half of the columns of every operand) what the chain computes
//              between its products: K D -> dU, T^T dU -> dY and dV, D -> planes
//   warps 8-11 dO^T, turned over and split into planes, for the two products that do not wait for the chain
//   warp 12    issues the MMAs: P^T dO, K D, half of Q^T (e^cum o dO), T^T dU, the other half,
//              -K^T (e^cum o dV)
//   warp 13    the loads.  K, T and the gates are double-buffered; Q, dO and P, which only the products aside
//              from the chain read, come in when those of the chunk before are done.
//   warp 14    D, dY and dV out to memory, by the copy engine
//
// Bound by the latency of that chain, 3.2 us a chunk (4 rows of 68 chunks, 16 heads, Dk = Dv = 128: 217 us; columns of
// heads on warp MMAs take 608).  What made the difference here was code, not data: with every loop unrolled the
// roles' 85 KB of instructions were fetched anew each chunk (370 us), and spilled registers came back from L2, since the tiles
// leave the L1 cache little.
//
// Tensor memory (512 columns): D (fp32, Dk), its two planes (Dk), X (64: K D, then the planes of dU),
// Y (64: dO^T, then T^T dU, then the planes of e^cum o dV), W (64: P^T dO), G (64: planes of e^cum o dO).  A
// warpgroup writes planes only where its own half of a product was.
//
// Every wait is bounded; after one runs out the chain runs to its end on whatever is there.

#include "gdn_whole.cuh"

namespace kda {
namespace gdn {
namespace {

template <int DK, int DV>
struct RChain {
    static constexpr int THREADS = 480;
    static constexpr int K_ = 0, T_ = K_ + DK / 64 * PANEL, SCAL = T_ + TPL * TRI;
    static constexpr int STAGE = (SCAL + REC_BYTES - REC_SCAL + 1023) / 1024 * 1024;
    static constexpr int Q_ = 2 * STAGE, G_ = Q_ + DK / 64 * PANEL, P_ = G_ + DV / 64 * PANEL;
    static constexpr int OUT_D = P_ + PPL * TRI;               // planes of D, two tiles
    static constexpr int OUT_Y = OUT_D + 2 * DV * DK * 2;      // of dY
    static constexpr int OUT_V = OUT_Y + 2 * DV * C * 2;       // dV, panels of 64 columns
    static constexpr int BAR = OUT_V + C * DV * 2;
    // the base is aligned up to 1024 bytes; more than half of an SM's, since each CTA takes all of its
    // tensor memory
    static constexpr int SMEM = BAR + 256 + 1024 > 116 * 1024 ? BAR + 256 + 1024 : 116 * 1024;
    static constexpr int M_ = 0, DP = DK, X_ = 2 * DK, Y_ = X_ + 64, W_ = Y_ + 64, GE = W_ + 64;   // tensor memory columns
};
// plane p of dU (or e^cum o dV), k-step x of 16 tokens: where its half of the product was
__host__ __device__ constexpr int half_at(int p, int x) { return (x >> 1) * 32 + p * 16 + (x & 1) * 8; }

template <int DK, int DV>
__global__ void __launch_bounds__(480, 1)
gdn_rchain_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                  const __grid_constant__ CUtensorMap mv, GdnBwdArgs b, const __grid_constant__ Seqs seqs, const char* records, char* kept, int* status, int drop)
{
    using L = RChain<DK, DV>;
    const GdnArgs& a = b.f;
    extern __shared__ char raw[];
    char* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t base = smem_addr(sm);
    uint64_t* bars = (uint64_t*)(sm + L::BAR);
    // [2]: by stage (full, empty), or of the two warpgroups
    uint64_t *full = bars, *empty = full + 2, *kd_done = empty + 2, *ty_done = kd_done + 2, *d_done = ty_done + 2;
    uint64_t *u_ready = d_done + 2, *v_ready = u_ready + 2, *d_ready = v_ready + 2;
    uint64_t *g_full = d_ready + 2, *g_empty = g_full + 1, *landed = g_empty + 1, *g_ready = landed + 1, *w_done = g_ready + 1;
    uint64_t *d_kept = w_done + 1, *d_free = d_kept + 1, *y_kept = d_free + 1, *y_free = y_kept + 1, *drain = y_free + 1;
    uint32_t* tm_ptr = (uint32_t*)(drain + 1);
    const Guard guard{(volatile int*)(tm_ptr + 1), status};

    const int tid = threadIdx.x, lane = tid & 31, warp = uniform_warp();
    const int h = blockIdx.x, seq = blockIdx.y, hk = h / (a.Hv / a.Hk);
    const int len = seqs.len(seq), nch = (len + C - 1) / C;   // step it: chunk nch - 1 - it
    const int64_t t0 = seqs.start(seq);
    const Kept keep{DK, DV};
    char* mine = kept + ((int64_t)seqs.slot0(seq, C) * a.Hv + h) * keep.bytes();   // chunk 0
    const int64_t next = (int64_t)a.Hv * keep.bytes();

    if (warp == 13) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(full + i, 1);
                mbar_init(empty + i, 13);   // the MMAs, and each warp that reads the gates
                for (uint64_t* x : {kd_done, ty_done, d_done}) mbar_init(x + i, 1);
                mbar_init(u_ready + i, 4 + drop);
                for (uint64_t* x : {v_ready, d_ready}) mbar_init(x + i, 4);
            }
            for (uint64_t* x : {g_full, landed, w_done, d_free, y_free, drain}) mbar_init(x, 1);
            mbar_init(g_ready, 4);
            mbar_init(g_empty, 5);   // warps 8-11 and the MMAs
            for (uint64_t* x : {d_kept, y_kept}) mbar_init(x, 8);
            *guard.flag = 0;
            fence_mbar_init();
            fence_async_smem();
        }
    } else if (warp == 12) {
        tmem_alloc(tm_ptr, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm_ptr;

    if (warp == 13) {
        const char* rec = records + ((int64_t)seqs.slot0(seq, C) * a.Hv + h) * REC_BYTES;
        constexpr int SCAL_BYTES = REC_BYTES - REC_SCAL;
        int in = 0, g_in = 0;   // issued
        for (int it = 0; it < nch; ++it) {
            const int c = nch - 1 - it, valid = min(C, len - c * C), y = (int)t0 + c * C;
            char* st = sm + (it & 1) * L::STAGE;
            const char* src = rec + (int64_t)c * a.Hv * REC_BYTES;
            if (it >= 2) wait(empty + (it & 1), ((it >> 1) & 1) ^ 1, guard);
            if (warp_up(guard)) break;
            if (lane == 0) {
                uint64_t* bar = valid < C ? landed : full + (it & 1);
                mbar_arrive_expect_tx(bar, C * DK * 2 + REC_P + SCAL_BYTES + (valid < C ? C * DK * 2 + C * DV * 2 + REC_SCAL - REC_P : 0));
                for (int p = 0; p < DK / 64; ++p) tma_load_3d(st + L::K_ + p * PANEL, &mk, bar, p * 64, hk, y);
                bulk_load(st + L::T_, src, REC_P, bar);
                bulk_load(st + L::SCAL, src + REC_SCAL, SCAL_BYTES, bar);
            }
            ++in;
            __syncwarp();
            if (it >= 1) {   // (the first step's copies go out whole: a ragged chunk's land on one barrier)
                wait(g_empty, (it - 1) & 1, guard);
                if (warp_up(guard)) break;
            }
            if (lane == 0) {
                uint64_t* bar = valid < C ? landed : g_full;
                if (valid == C) mbar_arrive_expect_tx(bar, C * DK * 2 + C * DV * 2 + REC_SCAL - REC_P);
                for (int p = 0; p < DV / 64; ++p) tma_load_3d(sm + L::G_ + p * PANEL, &mg, bar, p * 64, h, y);
                bulk_load(sm + L::P_, src + REC_P, REC_SCAL - REC_P, bar);
                for (int p = 0; p < DK / 64; ++p) tma_load_3d(sm + L::Q_ + p * PANEL, &mq, bar, p * 64, hk, y);
                // The data of the step after come as far as L2 meanwhile, or the chain would wait for memory
                // once a chunk.
                if (c >= 2) {
                    for (int p = 0; p < DK / 64; ++p) {
                        prefetch_3d(&mk, p * 64, hk, y - 2 * C);
                        prefetch_3d(&mq, p * 64, hk, y - 2 * C);
                    }
                    for (int p = 0; p < DV / 64; ++p) prefetch_3d(&mg, p * 64, h, y - 2 * C);
                    prefetch(src - 2 * (int64_t)a.Hv * REC_BYTES, REC_BYTES);
                }
            }
            ++g_in;
            __syncwarp();
            if (valid < C) {
                // the rows behind the sequence belong to another one, or to none: they are zeros here
                wait(landed, 0, guard);
                for (int e = lane; e < (C - valid) * 8; e += 32) {
                    const int off = (valid + e / 8) * 128 + (e & 7) * 16;
                    for (int p = 0; p < DK / 64; ++p) {
                        *(uint4*)(st + L::K_ + p * PANEL + off) = make_uint4(0, 0, 0, 0);
                        *(uint4*)(sm + L::Q_ + p * PANEL + off) = make_uint4(0, 0, 0, 0);
                    }
                    for (int p = 0; p < DV / 64; ++p) *(uint4*)(sm + L::G_ + p * PANEL + off) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(full + (it & 1));
                    mbar_arrive(g_full);
                }
                __syncwarp();
            }
        }
        drain_ring(full, 2, in);
        drain_ring(g_full, 1, g_in);
        if (in > 0 && len % C != 0) mbar_wait_bounded(landed, 0, kWaitNs);
    } else if (warp == 12) {
        const uint64_t dk = desc_rows(base + L::K_), dkc = desc_cols(base + L::K_, PANEL), dqc = desc_cols(base + L::Q_, PANEL);
        // T and P as they stand have the rows as K: core matrices 256 bytes apart along it, 128 along the columns
        const uint64_t dt = sdesc(base + L::T_, 256, 128), dp = sdesc(base + L::P_, 256, 128);
        // MMAs that follow one another on the same columns have the same shape, which is what orders them.
        constexpr uint32_t id_kd = idesc_f16(128, 32, false, false, false, true);
        constexpr uint32_t id_t = idesc_f16(128, 16, false, true, false, true);
        constexpr uint32_t id_s = idesc_f16(128, 64, false, true, false, true);
        constexpr int KH = DK / 32;   // k-steps of half of the key channels
        auto kd = [&](int th, uint64_t desc, int kh) {   // 32 tokens, half of the key channels
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int x = kh * KH; x < kh * KH + KH; ++x)
                    umma_f16_ts(tmem + L::X_ + 32 * th, tmem + L::DP + p * (DK / 2) + x * 8, step_rows(desc + (th * 4096 >> 4), x, PANEL),
                                id_kd ^ (p ? NEG : 0), kh + p + (x - kh * KH) > 0);
        };
        auto qg = [&](int n) {   // 64 key channels of Q^T (e^cum o dO)
#pragma unroll
            for (int p = 1; p >= 0; --p)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    umma_f16_ts(tmem + L::M_ + 64 * n, tmem + L::GE + p * 32 + x * 8, step_cols(dqc, x) + (n * PANEL >> 4), id_s ^ (p ? NEG : 0), 1);
        };
        for (int it = 0; it < nch; ++it) {
            const uint32_t so = (it & 1) * (L::STAGE >> 4);
            wait(g_full, it & 1, guard);
            wait(g_ready, it & 1, guard);
            tc_fence_after();
            if (elect()) {
#pragma unroll
                for (int jb = 0; jb < 4; ++jb)
#pragma unroll
                    for (int q = 0; q < PPL; ++q)
#pragma unroll
                        for (int x = jb; x < 4; ++x)
                            umma_f16_ts(tmem + L::W_ + 16 * jb, tmem + L::Y_ + x * 8, dp + ((q * TRI + blk(x, jb)) >> 4), id_t, q + x > jb);
                umma_commit(w_done);
            }
            wait(full + (it & 1), (it >> 1) & 1, guard);
            wait(d_ready, it & 1, guard);
            tc_fence_after();
            if (elect()) {
                kd(1, dk + so, 0);
                kd(0, dk + so, 0);
            }
            wait(d_ready + 1, it & 1, guard);
            tc_fence_after();
            if (elect()) {
                kd(1, dk + so, 1);
                umma_commit(kd_done + 1);
                kd(0, dk + so, 1);
                umma_commit(kd_done);
                qg(0);   // while the threads turn K D into dU
                if (DK == 64) umma_commit(g_empty);
            }
#pragma unroll
            for (int th = 1; th >= 0; --th) {   // T^T dU: the later tokens first, the others wait for both
                wait(u_ready + th, it & 1, guard);
                tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int jb = 2 * th + 1; jb >= 2 * th; --jb)
#pragma unroll
                        for (int q = 0; q < TPL; ++q)
#pragma unroll
                            for (int p = 0; p < 2 - q; ++p)
#pragma unroll
                                for (int x = jb; x < 4; ++x)
                                    umma_f16_ts(tmem + L::Y_ + 16 * jb, tmem + L::X_ + half_at(p, x), dt + so + ((q * TRI + blk(x, jb)) >> 4),
                                                id_t ^ (p ? NEG : 0), p + q + x > jb);
                    umma_commit(ty_done + th);
                }
            }
            if (DK == 128 && elect()) {
                qg(1);
                umma_commit(g_empty);
            }
#pragma unroll
            for (int th = 1; th >= 0; --th) {
                wait(v_ready + th, it & 1, guard);
                tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int n = 0; n < DK / 64; ++n) {   // 64 key channels
#pragma unroll
                        for (int p = 1; p >= 0; --p)
#pragma unroll
                            for (int x = 2 * th; x < 2 * th + 2; ++x)
                                umma_f16_ts(tmem + L::M_ + 64 * n, tmem + L::Y_ + half_at(p, x), step_cols(dkc + so, x) + (n * PANEL >> 4),
                                            id_s ^ (p ? NEG : 0), 1);
                        if (!th) umma_commit(d_done + n);
                    }
                    if (!th && DK == 64) umma_commit(d_done + 1);
                }
            }
            if (elect()) umma_commit(empty + (it & 1));
        }
        drain_mma(drain);
    } else if (warp < 8) {
        constexpr int HK = DK / 2, NI = HK / 32;   // key channels of a warpgroup's half of the state
        const int hf = warp >> 2, row = tid & 127;   // row: value column
        const uint32_t at = tmem + ((uint32_t)(warp & 3) * 32u << 16);
        const bool real = row < DV;
        const int64_t soff = ((int64_t)seq * a.Hv + h) * DK * DV + (int64_t)hf * HK * DV + row;
        char* out = sm + L::OUT_V + (DV > 64 ? row >> 6 : 0) * PANEL + (row & 7) * 2;
        if (nch > 0) wait(full, 0, guard);
        // (Loops over 32 channels stay loops here: unrolled, the kernel's roles fetched instructions for longer than
        // they took to issue.)
        for (int it = 0;; ++it) {
            // D for step it: to the planes, and decayed; at the end, out
            const float* scal = (const float*)(sm + (it & 1) * L::STAGE + L::SCAL);
#pragma unroll 1
            for (int i = 0; i < NI; ++i) {
                float x[32];
                if (it == 0) {
#pragma unroll
                    for (int z = 0; z < 32; ++z) {
                        const int64_t off = soff + (int64_t)(i * 32 + z) * DV;
                        x[z] = b.dST && real ? b.dST[off] : 0.f;
                    }
                } else {
                    tmem_ld32(at + L::M_ + hf * HK + i * 32, x);
                }
                if (it < nch) {
                    uint32_t p[2][16];
                    planes_of<2>(x, p);
                    tmem_st16u_nowait(at + L::DP + hf * (HK / 2) + i * 16, p[0]);
                    tmem_st16u_nowait(at + L::DP + DK / 2 + hf * (HK / 2) + i * 16, p[1]);
                    const float gam = scal[C - 1];
#pragma unroll
                    for (int z = 0; z < 32; ++z) x[z] *= gam;
                    store32(at + L::M_ + hf * HK + i * 32, x);
                } else if (b.dS0 && real) {
#pragma unroll
                    for (int z = 0; z < 32; ++z) b.dS0[soff + (int64_t)(i * 32 + z) * DV] = x[z];
                }
            }
            if (it == nch) break;
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(d_ready + hf);
            if (it > 0) wait(d_free, (it - 1) & 1, guard);
            // while K D runs, the planes to where they are copied from
#pragma unroll 1
            for (int p = 0; p < 2; ++p)
                planes_to_tile<DV, HK / 2>(at + L::DP + p * (DK / 2) + hf * (HK / 2), sm + L::OUT_D + p * DV * DK * 2, row, hf * (HK / 8), real,
                                           p ? 0x80008000u : 0u);
            fence_async_smem();
            warp_arrive(d_kept);
            float x[32];
            uint32_t p[2][16];
            // dU = P^T dO + e^{cum_C - cum} o (K D), 32 tokens
            wait(w_done, it & 1, guard);
            wait(kd_done + hf, it & 1, guard);
            tc_fence_after();
            {
                float w[32];
                tmem_ld32(at + L::X_ + hf * 32, x);
                tmem_ld32(at + L::W_ + hf * 32, w);
                scale32(x, scal + C + hf * 32);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] += w[i];
            }
            planes_of<2>(x, p);
            tmem_st16u_nowait(at + L::X_ + hf * 32, p[0]);
            tmem_st16u_nowait(at + L::X_ + hf * 32 + 16, p[1]);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(u_ready + hf);
            // dY, and -e^cum o dV = -e^cum o beta o dY
            if (it + 1 < nch) wait(full + ((it + 1) & 1), ((it + 1) >> 1) & 1, guard);
            if (it > 0) wait(y_free, (it - 1) & 1, guard);
            wait(ty_done + hf, it & 1, guard);
            tc_fence_after();
            tmem_ld32(at + L::Y_ + hf * 32, x);
            {
                float z[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = -x[i];
                scale32(z, scal + 2 * C + hf * 32);
                scale32(z, scal + hf * 32);
                planes_of<2>(z, p);
            }
            tmem_st16u_nowait(at + L::Y_ + hf * 32, p[0]);
            tmem_st16u_nowait(at + L::Y_ + hf * 32 + 16, p[1]);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(v_ready + hf);
            // while K^T (e^cum o dV) runs: dY and dV to where they are copied from
            planes_of<2>(x, p);
            scale32(x, scal + 2 * C + hf * 32);
            warp_arrive(empty + (it & 1));
            if (real) {
                to_tile<DV>(sm + L::OUT_Y, row, hf * 4, p[0]);
                to_tile<DV>(sm + L::OUT_Y + DV * C * 2, row, hf * 4, p[1], 0x80008000u);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t v = pack(x[2 * i], x[2 * i + 1]);
                    *(uint16_t*)(out + piece_at(hf * 32 + 2 * i, (row & 63) >> 3)) = (uint16_t)v;
                    *(uint16_t*)(out + piece_at(hf * 32 + 2 * i + 1, (row & 63) >> 3)) = (uint16_t)(v >> 16);
                }
            }
            fence_async_smem();
            warp_arrive(y_kept);
            wait(d_done + hf, it & 1, guard);
            tc_fence_after();
        }
    } else if (warp == 14) {
        __nv_bfloat16* vp = (__nv_bfloat16*)b.dv + (t0 * a.Hv + h) * DV;
        for (int it = 0; it < nch; ++it) {
            const int c = nch - 1 - it, valid = min(C, len - c * C);
            char* dst = mine + c * next;
            wait(d_kept, it & 1, guard);
            __syncwarp();
            if (lane == 0) {
                bulk_store(dst + keep.d(), sm + L::OUT_D, 2 * DV * DK * 2);
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(d_free);
            }
            wait(y_kept, it & 1, guard);
            if (valid < C)   // the rows behind the sequence are not its own
                for (int i = lane; i < valid * (DV / 8); i += 32) {
                    const int tok = i / (DV / 8), piece = i % (DV / 8);
                    *(uint4*)(vp + ((int64_t)c * C + tok) * a.Hv * DV + piece * 8) =
                        *(const uint4*)(sm + L::OUT_V + piece / 8 * PANEL + piece_at(tok, piece & 7));
                }
            __syncwarp();
            if (lane == 0) {
                bulk_store(dst + keep.y(), sm + L::OUT_Y, 2 * DV * C * 2);
                if (valid == C)
                    for (int p = 0; p < DV / 64; ++p) store_3d(&mv, sm + L::OUT_V + p * PANEL, p * 64, h, (int)t0 + c * C);
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(y_free);
            }
        }
        if (lane == 0) bulk_wait0();
    } else {
        const int row = tid & 127;
        const uint32_t at = tmem + ((uint32_t)(warp & 3) * 32u << 16);
        const char* col = sm + L::G_ + (DV > 64 ? row >> 6 : 0) * PANEL + (row & 7) * 2;
        for (int it = 0; it < nch; ++it) {
            const float* scal = (const float*)(sm + (it & 1) * L::STAGE + L::SCAL);
            wait(full + (it & 1), (it >> 1) & 1, guard);
            wait(g_full, it & 1, guard);
            if (it > 0) {   // dV's planes and the last of e^cum o dO have been read
                wait(d_done, (it - 1) & 1, guard);
                wait(d_done + 1, (it - 1) & 1, guard);
                tc_fence_after();
            }
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
                float x[32];
                uint32_t g[16], e[2][16];   // dO^T, planes of e^cum o dO^T
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    // (with Dv = 64, rows 64 on repeat the others; they are not used)
                    const uint32_t lo = *(const uint16_t*)(col + hf * 4096 + piece_at(2 * i, (row & 63) >> 3));
                    const uint32_t hi = *(const uint16_t*)(col + hf * 4096 + piece_at(2 * i + 1, (row & 63) >> 3));
                    g[i] = lo | hi << 16;
                    x[2 * i] = low(g[i]);
                    x[2 * i + 1] = high(g[i]);
                }
                tmem_st16u_nowait(at + L::Y_ + hf * 16, g);
                scale32(x, scal + hf * 32);
                planes_of<2>(x, e);
                tmem_st16u_nowait(at + L::GE + hf * 16, e[0]);
                tmem_st16u_nowait(at + L::GE + 32 + hf * 16, e[1]);
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(g_ready);
            warp_arrive(g_empty);
            warp_arrive(empty + (it & 1));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int DK, int DV>
cudaError_t rchain(const GdnBwdArgs& b, const Seqs& s, const void* records, void* kept, int* status, cudaStream_t st)
{
    using L = RChain<DK, DV>;
    CUtensorMap k{}, q{}, g{}, v{};
    const GdnArgs& a = b.f;
    const int64_t T = s.tokens();
    if (T > 0 && (!make_map(&k, a.k, T, a.Hk, DK, 64, 1, C) || !make_map(&q, a.q, T, a.Hk, DK, 64, 1, C) ||
                  !make_map(&g, b.dout, T, a.Hv, DV, 64, 1, C) || !make_map(&v, b.dv, T, a.Hv, DV, 64, 1, C)))
        return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<gdn_rchain_kernel<DK, DV>>(L::SMEM);
    if (e != cudaSuccess) return e;
    ProfileScope prof("gdn_rchain", st);
    count_launch();
    gdn_rchain_kernel<DK, DV><<<dim3(a.Hv, s.n), L::THREADS, L::SMEM, st>>>(k, q, g, v, b, s, (const char*)records, (char*)kept, status, debug_drop_handoff());
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_rchain(const GdnBwdArgs& b, const Seqs& s, const void* records, void* kept, int* status, cudaStream_t st)
{
    if (b.f.Dk == 64) return b.f.Dv == 64 ? rchain<64, 64>(b, s, records, kept, status, st) : rchain<64, 128>(b, s, records, kept, status, st);
    return b.f.Dv == 64 ? rchain<128, 64>(b, s, records, kept, status, st) : rchain<128, 128>(b, s, records, kept, status, st);
}

}  // namespace gdn
}  // namespace kda
