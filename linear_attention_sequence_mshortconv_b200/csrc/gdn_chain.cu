// The forward scan of the gated delta rule on tcgen05 tensor cores (bf16; Dk and Dv 64 or 128), one
// CTA per sequence and value head.
//
// The mathematics, the prologue and the planes are those of gdn_fwd.cu.  There a CTA owns 16 or 32
// value columns, so a head's K, Q and factors are read once per 16 or 32 columns, and shared
// memory bounds it as soon as the heads fill the SMs.  Here all Dv columns are the 128 rows of every
// product: S, Y and U are left operands in tensor memory (lane = value column), and K, Q, T and P
// are read from shared memory once per chunk and plane.  A chunk takes 2.6 us against 1.5 there, for 4 to 8
// times the columns (4 rows of 68 chunks, 16 heads, Dk = Dv = 128: 181 us, columns 333; what the backward keeps,
// 208 KB a chunk less D and dY, comes out in 190).  Bound by the latency of the chain: three products in a row and
// what the threads do between them, about 0.4 us each time.
//
//   warps 0-7  (two warpgroups, each with half of the columns of every operand): K S -> Y,
//              U -> decayed U, S -> planes: what lies between the products, in fp32
//   warps 8-11 the output: O = e^cum o (Q S), to which P U is added, and its store
//   warp 12    issues the MMAs: K S, Q S | T Y | K^T U, P U
//   warp 13    the loads of the next chunk
//
// Tensor memory (512 columns): S (fp32, Dk), its two planes (Dk), R (128: V^T and K S, then the planes of
// Y, then of decayed U), U (64: the product, then its planes), O (64).  A warpgroup writes planes only
// where its own half of a product was, so the two need no barrier between them.  V comes in by a
// product with the identity (exact), which turns it over: two-byte reads of its columns took the
// threads longer than K S takes.
//
// Every wait is bounded; after one runs out the chain runs to its end on whatever is there.

#include "gdn_whole.cuh"

namespace kda {
namespace gdn {
namespace {

// What a launch gives: o (and S_T); what the backward keeps; S_T alone; or the transition of the whole
// sequence, that is, S_T with S_0 = 1 and V = 0 (Dv = Dk).
enum { CHAIN_OUT, CHAIN_KEEP, CHAIN_STATE, CHAIN_TRANSITION };

template <int DK, int DV, int MODE>
struct Chain {
    static constexpr bool KEEP = MODE == CHAIN_KEEP, READ = MODE == CHAIN_OUT, HAS_V = MODE != CHAIN_TRANSITION;
    static constexpr int THREADS = 448;
    static constexpr int K_ = 0, Q_ = K_ + DK / 64 * PANEL, V_ = Q_ + (READ ? DK / 64 * PANEL : 0);
    // the record; only o needs P
    static constexpr int REC = V_ + (HAS_V ? DV / 64 * PANEL : 0), SCAL = REC + (READ ? REC_SCAL : REC_P);
    static constexpr int STAGE = (SCAL + REC_BYTES - REC_SCAL + 1023) / 1024 * 1024;
    static constexpr int OUT = 2 * STAGE;                     // the output [64][DV] bf16; or what is kept: two planes
    static constexpr int OUT_U = OUT + 2 * DV * DK * 2;       // of S, of U, and R, as tiles
    static constexpr int OUT_R = OUT_U + 2 * DV * C * 2;
    static constexpr int EYE = KEEP ? OUT_R + DV * C * 2 : OUT + (READ ? C * DV * 2 : 0);   // 64x64 identity, bf16, a panel
    static constexpr int BAR = EYE + PANEL;
    // the base is aligned up to 1024 bytes; more than half of an SM's, since each CTA takes all of its
    // tensor memory
    static constexpr int SMEM = BAR + 256 + 1024 > 116 * 1024 ? BAR + 256 + 1024 : 116 * 1024;
    // tensor memory columns
    static constexpr int M_ = 0, SP_ = DK, R_ = 2 * DK, U_ = R_ + 128, O_ = U_ + 64;
};
// plane p of Y (or decayed U), k-step x of 16 tokens: planes 0 and 1 where the warpgroup's half of V was,
// plane 2 where its half of K S was
__host__ __device__ constexpr int y_at(int p, int x) { return (p < 2 ? p * 16 : 64) + (x >> 1) * 32 + (x & 1) * 8; }

template <int DK, int DV, int MODE>
__global__ void __launch_bounds__(448, 1)
gdn_chain_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mv,
                 GdnArgs a, const __grid_constant__ Seqs seqs, const char* records, char* kept, int* status, int drop)
{
    using L = Chain<DK, DV, MODE>;
    constexpr bool KEEP = L::KEEP, READ = L::READ, HAS_V = L::HAS_V;
    extern __shared__ char raw[];
    char* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t base = smem_addr(sm);
    uint64_t* bars = (uint64_t*)(sm + L::BAR);
    // [2]: by stage (full, empty), or of the two warpgroups
    uint64_t *full = bars, *empty = full + 2, *ks_done = empty + 2, *ty_done = ks_done + 2, *s_done = ty_done + 2;
    uint64_t *y_ready = s_done + 2, *u_ready = y_ready + 2, *s_ready = u_ready + 2;
    uint64_t *landed = s_ready + 2, *qs_done = landed + 1;
    uint64_t *o_done = qs_done + 1, *o_scaled = o_done + 1, *o_read = o_scaled + 1;
    uint64_t *s_kept = o_read + 1, *u_kept = s_kept + 1, *s_free = u_kept + 1, *u_free = s_free + 1, *drain = u_free + 1;
    uint32_t* tm_ptr = (uint32_t*)(drain + 1);
    const Guard guard{(volatile int*)(tm_ptr + 1), status};

    const int tid = threadIdx.x, lane = tid & 31, warp = uniform_warp();
    const int h = blockIdx.x, seq = blockIdx.y, hk = h / (a.Hv / a.Hk);
    const int len = seqs.len(seq), nch = (len + C - 1) / C;
    const int64_t t0 = seqs.start(seq);
    const char* rec = records + ((int64_t)seqs.slot0(seq, C) * a.Hv + h) * REC_BYTES;

    if (warp == 13) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(full + i, 1);
                mbar_init(empty + i, READ ? 13 : 9);   // the MMAs, and each warp that reads the stage
                for (uint64_t* b : {ks_done, ty_done, s_done}) mbar_init(b + i, 1);
                mbar_init(y_ready + i, 4 + drop);
                for (uint64_t* b : {u_ready, s_ready}) mbar_init(b + i, 4);
            }
            for (uint64_t* b : {landed, qs_done, o_done, s_free, u_free, drain}) mbar_init(b, 1);
            for (uint64_t* b : {o_scaled, o_read}) mbar_init(b, 4);
            for (uint64_t* b : {s_kept, u_kept}) mbar_init(b, 8);
            *guard.flag = 0;
            fence_mbar_init();
            fence_async_smem();
        }
    } else if (warp == 12) {
        tmem_alloc(tm_ptr, 512);
        tmem_relinquish();
    } else if (tid < 64) {
        for (int i = 0; i < 8; ++i) *(uint4*)(sm + L::EYE + tid * 128 + i * 16) = make_uint4(0, 0, 0, 0);
        *(uint16_t*)(sm + L::EYE + piece_at(tid, tid >> 3) + (tid & 7) * 2) = 0x3f80;
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm_ptr;

    if (warp == 13) {
        int issued = 0;
        for (int c = 0; c < nch; ++c) {
            char* st = sm + (c & 1) * L::STAGE;
            const int valid = min(C, len - c * C);
            if (c >= 2) wait(empty + (c & 1), ((c >> 1) & 1) ^ 1, guard);
            if (warp_up(guard)) break;
            uint64_t* bar = valid < C ? landed : full + (c & 1);
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, (READ ? 2 : 1) * C * DK * 2 + (HAS_V ? C * DV * 2 : 0) + REC_BYTES - (READ ? 0 : REC_SCAL - REC_P));
                for (int p = 0; p < DK / 64; ++p) {
                    tma_load_3d(st + L::K_ + p * PANEL, &mk, bar, p * 64, hk, (int)t0 + c * C);
                    if (READ) tma_load_3d(st + L::Q_ + p * PANEL, &mq, bar, p * 64, hk, (int)t0 + c * C);
                }
                for (int p = 0; HAS_V && p < DV / 64; ++p) tma_load_3d(st + L::V_ + p * PANEL, &mv, bar, p * 64, h, (int)t0 + c * C);
                const char* src = rec + (int64_t)c * a.Hv * REC_BYTES;
                if (READ) {
                    bulk_load(st + L::REC, src, REC_BYTES, bar);
                } else {
                    bulk_load(st + L::REC, src, REC_P, bar);
                    bulk_load(st + L::SCAL, src + REC_SCAL, REC_BYTES - REC_SCAL, bar);
                }
                // The stage after next is still in use: its data come as far as L2 meanwhile, or the
                // chain would wait for memory once a chunk.
                if (c + 2 < nch) {
                    const int y = (int)t0 + (c + 2) * C;
                    for (int p = 0; p < DK / 64; ++p) {
                        prefetch_3d(&mk, p * 64, hk, y);
                        if (READ) prefetch_3d(&mq, p * 64, hk, y);
                    }
                    for (int p = 0; HAS_V && p < DV / 64; ++p) prefetch_3d(&mv, p * 64, h, y);
                    prefetch(src + 2 * (int64_t)a.Hv * REC_BYTES, REC_BYTES);
                }
            }
            ++issued;
            if (valid < C) {
                // the rows behind the sequence belong to another one, or to none: they are zeros here
                __syncwarp();
                wait(landed, 0, guard);
                constexpr int TILES = (L::REC - L::K_) / PANEL;
                for (int e = lane; e < TILES * (C - valid) * 8; e += 32)
                    *(uint4*)(st + e / (8 * (C - valid)) * PANEL + (valid + e / 8 % (C - valid)) * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                warp_arrive(full + (c & 1));
            }
        }
        drain_ring(full, 2, issued);
        if (issued == nch && len % C != 0) mbar_wait_bounded(landed, 0, kWaitNs);
    } else if (warp == 12) {
        const uint64_t dk = desc_rows(base + L::K_), dq = desc_rows(base + L::Q_), dkc = desc_cols(base + L::K_, PANEL);
        const uint64_t dv = desc_cols(base + L::V_, PANEL), de = desc_rows(base + L::EYE);
        const uint64_t dt = sdesc(base + L::REC, 128, 256);   // core matrices: halves 128 bytes apart along K, rows 256
        // MMAs that follow one another on the same columns have the same shape, which is what orders
        // them.  The halves of the tokens (32 columns of a product) and of the key channels are the
        // warpgroups': each starts on its half while the other's is computed.
        constexpr uint32_t id_t = idesc_f16(128, 32, false, false, false, true);
        constexpr uint32_t id_ks = idesc_f16(128, 32, false, false, true, true);     // -K S
        constexpr uint32_t id_qs = idesc_f16(128, C, false, false, false, true);
        // (with Dv = 64 rows 64 on read what is behind V; they are not used)
        constexpr uint32_t id_v = idesc_f16(128, C, true, false, false, true);
        constexpr uint32_t id_s = idesc_f16(128, 64, false, true, false, true);
        constexpr int KH = DK / 32;          // k-steps of half of the key channels
        auto by_s = [&](uint32_t to, uint64_t desc, uint32_t id, int kh) {
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int x = kh * KH; x < kh * KH + KH; ++x)
                    umma_f16_ts(to, tmem + L::SP_ + p * (DK / 2) + x * 8, step_rows(desc, x, PANEL), id ^ (p ? NEG : 0), kh + p + (x - kh * KH) > 0);
        };
        // rows 32 th .. 32 th + 31 of a plane of T or P, times the tokens of k-step x
        auto tri = [&](uint32_t so, int plane, int th, int x) { return dt + so + ((plane * TRI + blk(2 * th, x)) >> 4); };
        for (int c = 0; c < nch; ++c) {
            const uint32_t so = (c & 1) * (L::STAGE >> 4);
            wait(full + (c & 1), (c >> 1) & 1, guard);
            if (c > 0) wait(s_done + 1, (c - 1) & 1, guard);   // decayed U is where K S goes
            wait(s_ready, c & 1, guard);
            tc_fence_after();
            if (elect()) {
                by_s(tmem + L::R_ + 64, dk + so, id_ks, 0);
                by_s(tmem + L::R_ + 96, dk + so + (4096 >> 4), id_ks, 0);
#pragma unroll
                for (int x = 0; HAS_V && x < 4; ++x) umma_f16(tmem + L::R_, step_cols(dv + so, x), step_rows(de, x, PANEL), id_v, x > 0);
            }
            wait(s_ready + 1, c & 1, guard);
            tc_fence_after();
            if (elect()) {
                by_s(tmem + L::R_ + 64, dk + so, id_ks, 1);
                umma_commit(ks_done);
                by_s(tmem + L::R_ + 96, dk + so + (4096 >> 4), id_ks, 1);
                umma_commit(ks_done + 1);
            }
            if (READ && c > 0) wait(o_done, (c - 1) & 1, guard);   // the planes of U are where T Y goes
#pragma unroll
            for (int th = 0; th < 2; ++th) {   // T Y: every product of planes but T1 Y2
                wait(y_ready + th, c & 1, guard);
                tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int q = 0; q < TPL; ++q)
#pragma unroll
                        for (int p = 0; p < PLANES - q; ++p)
#pragma unroll
                            for (int x = 0; x < 2 * th + 2; ++x)
                                umma_f16_ts(tmem + L::U_ + 32 * th, tmem + L::R_ + y_at(p, x), tri(so, q, th, x), id_t ^ (p == 1 ? NEG : 0), p + q + x > 0);
                    umma_commit(ty_done + th);
                }
            }
            if (READ) {   // while U is turned into its planes
                if (c > 0) wait(o_read, (c - 1) & 1, guard);
                tc_fence_after();
                if (elect()) {
                    by_s(tmem + L::O_, dq + so, id_qs, 0);
                    by_s(tmem + L::O_, dq + so, id_qs, 1);
                    umma_commit(qs_done);
                }
            }
#pragma unroll
            for (int th = 0; th < 2; ++th) {
                wait(u_ready + th, c & 1, guard);
                tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int n = 0; n < DK / 64; ++n) {   // 64 key channels
#pragma unroll
                        for (int p = PLANES - 1; p >= 0; --p)
#pragma unroll
                            for (int x = 2 * th; x < 2 * th + 2; ++x)
                                umma_f16_ts(tmem + L::M_ + 64 * n, tmem + L::R_ + y_at(p, x), step_cols(dkc + so, x) + (n * PANEL >> 4),
                                            id_s ^ (p == 1 ? NEG : 0), 1);
                        if (th) umma_commit(s_done + n);
                    }
                    if (th && DK == 64) umma_commit(s_done + 1);
                }
            }
            if (READ) {
                wait(o_scaled, c & 1, guard);
                tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int th = 0; th < 2; ++th)
#pragma unroll
                        for (int q = 0; q < PPL; ++q)
#pragma unroll
                            for (int p = 0; p < 2 - q; ++p)
#pragma unroll
                                for (int x = 0; x < 2 * th + 2; ++x)
                                    umma_f16_ts(tmem + L::O_ + 32 * th, tmem + L::U_ + (x >> 1) * 32 + p * 16 + (x & 1) * 8, tri(so, TPL + q, th, x),
                                                id_t ^ (p ? NEG : 0), 1);
                    umma_commit(o_done);
                }
            }
            if (elect()) umma_commit(empty + (c & 1));
        }
        drain_mma(drain);
    } else if (warp < 8) {
        constexpr int HK = DK / 2;   // key channels of a warpgroup's half of the state
        const int hf = warp >> 2, row = tid & 127;   // row: value column
        const uint32_t at = tmem + ((uint32_t)(warp & 3) * 32u << 16);
        const bool real = row < DV;
        const int64_t soff = ((int64_t)seq * a.Hv + h) * DK * DV + (int64_t)hf * HK * DV + row;
        if (nch > 0) wait(full, 0, guard);
        // (Loops over 32 channels stay loops here: unrolled, the kernel's roles fetched instructions for longer than
        // they took to issue.)
        for (int c = 0;; ++c) {
            // S for chunk c: to the planes, and decayed; at the end, out
            const float* scal = (const float*)(sm + (c & 1) * L::STAGE + L::SCAL);
#pragma unroll 1
            for (int i = 0; i < HK / 32; ++i) {
                float s[32];
                if (c == 0) {
#pragma unroll
                    for (int z = 0; z < 32; ++z) {
                        if (HAS_V) s[z] = a.S0 && real ? a.S0[soff + (int64_t)(i * 32 + z) * DV] : 0.f;
                        else s[z] = hf * HK + i * 32 + z == row ? 1.f : 0.f;
                    }
                } else {
                    tmem_ld32(at + L::M_ + hf * HK + i * 32, s);
                }
                if (c < nch) {
                    uint32_t p[2][16];
                    planes_of<2>(s, p);
                    tmem_st16u_nowait(at + L::SP_ + hf * (HK / 2) + i * 16, p[0]);
                    tmem_st16u_nowait(at + L::SP_ + DK / 2 + hf * (HK / 2) + i * 16, p[1]);
                    const float gam = scal[C - 1];
#pragma unroll
                    for (int z = 0; z < 32; ++z) s[z] *= gam;
                    store32(at + L::M_ + hf * HK + i * 32, s);
                } else if (a.ST && real) {
#pragma unroll
                    for (int z = 0; z < 32; ++z) a.ST[soff + (int64_t)(i * 32 + z) * DV] = s[z];
                }
            }
            if (c == nch) break;
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(s_ready + hf);
            if (KEEP) {   // while K S runs, the planes to where they are copied from
                if (c > 0) wait(s_free, (c - 1) & 1, guard);
#pragma unroll 1
                for (int p = 0; p < 2; ++p)
                    planes_to_tile<DV, HK / 2>(at + L::SP_ + p * (DK / 2) + hf * (HK / 2), sm + L::OUT + p * DV * DK * 2, row, hf * (HK / 8), real,
                                               p ? 0x80008000u : 0u);
                fence_async_smem();
                warp_arrive(s_kept);
            }
            float x[32];
            uint32_t p[3][16];
            auto put_y = [&] {
                planes_of<3>(x, p);
#pragma unroll
                for (int q = 0; q < 3; ++q) tmem_st16u_nowait(at + L::R_ + y_at(q, 2 * hf), p[q]);
            };
            // Y = beta o (V - e^cum o (K S)), 32 tokens
            wait(ks_done + hf, c & 1, guard);
            tc_fence_after();
            {
                float ks[32];
                if (HAS_V) {
                    tmem_ld32(at + L::R_ + hf * 32, x);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = 0.f;
                }
                tmem_ld32(at + L::R_ + 64 + hf * 32, ks);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 g = *(const float4*)&scal[hf * 32 + i];
                    x[i] = fmaf(g.x, ks[i], x[i]);
                    x[i + 1] = fmaf(g.y, ks[i + 1], x[i + 1]);
                    x[i + 2] = fmaf(g.z, ks[i + 2], x[i + 2]);
                    x[i + 3] = fmaf(g.w, ks[i + 3], x[i + 3]);
                }
            }
            if (DV < 128 && !real) {   // rows that no column of V fills
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = 0.f;
            }
            uint32_t r[1][16];
            if (KEEP) planes_of<1>(x, r);
            scale32(x, scal + 2 * C + hf * 32);
            put_y();
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(y_ready + hf);
            if (KEEP) {   // R, and later U, while the next product runs
                if (c > 0) wait(u_free, (c - 1) & 1, guard);
                if (real) to_tile<DV>(sm + L::OUT_R, row, hf * 4, r[0]);
            }
            // U, its planes, and decayed
            if (c + 1 < nch) wait(full + ((c + 1) & 1), ((c + 1) >> 1) & 1, guard);
            wait(ty_done + hf, c & 1, guard);
            tc_fence_after();
            tmem_ld32(at + L::U_ + hf * 32, x);
            uint32_t u[2][16];
            planes_of<2>(x, u);
            if (READ) {
                tmem_st16u_nowait(at + L::U_ + hf * 32, u[0]);
                tmem_st16u_nowait(at + L::U_ + hf * 32 + 16, u[1]);
            }
            scale32(x, scal + C + hf * 32);
            wait(ty_done + 1, c & 1, guard);   // the second half of T Y reads both halves' planes of Y
            tc_fence_after();
            put_y();
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(u_ready + hf);
            if (KEEP) {
                if (real) {
                    to_tile<DV>(sm + L::OUT_U, row, hf * 4, u[0]);
                    to_tile<DV>(sm + L::OUT_U + DV * C * 2, row, hf * 4, u[1], 0x80008000u);
                }
                fence_async_smem();
                warp_arrive(u_kept);
            }
            warp_arrive(empty + (c & 1));
            if (READ) wait(qs_done, c & 1, guard);   // its planes of S
            wait(s_done + hf, c & 1, guard);
            tc_fence_after();
        }
    } else if (KEEP) {
        if (warp == 8 && lane == 0) {   // what the gradients need goes out by the copy engine
            const Kept keep{DK, DV};
            char* dst = kept + ((int64_t)seqs.slot0(seq, C) * a.Hv + h) * keep.bytes();
            for (int c = 0; c < nch; ++c, dst += (int64_t)a.Hv * keep.bytes()) {
                wait(s_kept, c & 1, guard);
                bulk_store(dst + keep.s(), sm + L::OUT, 2 * DV * DK * 2);
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(s_free);
                wait(u_kept, c & 1, guard);
                bulk_store(dst + keep.u(), sm + L::OUT_U, 3 * DV * C * 2);   // U and, behind it, R
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(u_free);
            }
            bulk_wait0();
        }
    } else if (READ) {
        const int row = tid & 127, t = tid - 256;
        const uint32_t at = tmem + ((uint32_t)(warp & 3) * 32u << 16) + L::O_;
        __nv_bfloat16* op = (__nv_bfloat16*)a.o + (t0 * a.Hv + h) * DV;
        __nv_bfloat16* out = (__nv_bfloat16*)(sm + L::OUT);
        for (int c = 0; c < nch; ++c) {
            const float* scal = (const float*)(sm + (c & 1) * L::STAGE + L::SCAL);
            wait(full + (c & 1), (c >> 1) & 1, guard);
            wait(qs_done, c & 1, guard);
            tc_fence_after();
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float x[32];
                tmem_ld32(at + hf * 32, x);
                scale32(x, scal + hf * 32);
                store32(at + hf * 32, x);
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(o_scaled);
            warp_arrive(empty + (c & 1));
            wait(o_done, c & 1, guard);
            tc_fence_after();
            asm volatile("bar.sync 1, 128;" ::: "memory");   // the last chunk's rows have been stored
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float x[32];
                tmem_ld32(at + hf * 32, x);
                if (row < DV)
#pragma unroll
                    for (int i = 0; i < 32; ++i) out[(hf * 32 + i) * DV + row] = __float2bfloat16_rn(x[i]);
            }
            tc_fence_before();
            warp_arrive(o_read);
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const int valid = min(C, len - c * C);
            for (int e = t; e < valid * (DV / 8); e += 128)
                *(uint4*)(op + ((int64_t)c * C + e / (DV / 8)) * a.Hv * DV + e % (DV / 8) * 8) = *(const uint4*)(out + e * 8);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int DK, int DV, int MODE>
cudaError_t chain(const GdnArgs& a, const Seqs& s, const void* records, void* kept, int* status, cudaStream_t st)
{
    using L = Chain<DK, DV, MODE>;
    CUtensorMap k{}, q{}, v{};
    const int64_t T = s.tokens();
    if (T > 0 && (!make_map(&k, a.k, T, a.Hk, DK, 64, 1, C) || (L::READ && !make_map(&q, a.q, T, a.Hk, DK, 64, 1, C)) ||
                  (L::HAS_V && !make_map(&v, a.v, T, a.Hv, DV, 64, 1, C))))
        return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<gdn_chain_kernel<DK, DV, MODE>>(L::SMEM);
    if (e != cudaSuccess) return e;
    ProfileScope prof(MODE == CHAIN_OUT ? "gdn_chain" : MODE == CHAIN_KEEP ? "gdn_chain_keep" : MODE == CHAIN_STATE ? "gdn_chain_state" : "gdn_chain_transition", st);
    count_launch();
    gdn_chain_kernel<DK, DV, MODE><<<dim3(a.Hv, s.n), L::THREADS, L::SMEM, st>>>(k, q, v, a, s, (const char*)records, (char*)kept, status, debug_drop_handoff());
    return cudaGetLastError();
}
template <int MODE>
cudaError_t chain(const GdnArgs& a, const Seqs& s, const void* records, void* kept, int* status, cudaStream_t st)
{
    if (a.Dk == 64) return a.Dv == 64 ? chain<64, 64, MODE>(a, s, records, kept, status, st) : chain<64, 128, MODE>(a, s, records, kept, status, st);
    return a.Dv == 64 ? chain<128, 64, MODE>(a, s, records, kept, status, st) : chain<128, 128, MODE>(a, s, records, kept, status, st);
}

// ---- pieces of long samples ---------------------------------------------------------------------
// Where few heads have many chunks in a row, the samples are cut into pieces of equal length that run at
// once.  The state is linear in the one before, S_out = M S_in + B: one launch gives every piece's B (from
// a state of zero), one its M (from the identity, without V), this kernel carries the states from piece
// to piece, and a last launch runs every piece from the right state: three times the work, on more SMs than
// that.  (16 heads of 512 chunks in 9 pieces: 139, 129, 38 and 171 us; one chain of columns takes 770.)
//
// A CTA has 16 columns of a head's states; thread (i, j) has rows i, i + 32, ... and columns 4j .. 4j + 3.  The next
// piece's M is on its way while one is used.
template <int DK>
struct Carry {
    static constexpr int THREADS = 128, COLS = 16, MROW = DK + 4;   // floats; rows 16 bytes apart in banks
    static constexpr int S_ = 2 * DK * MROW, SMEM = (S_ + DK * COLS) * 4;
};
struct Pieces {
    int16_t first[kMaxSeqs + 1];   // a sample's first piece
};
template <int DK>
__global__ void __launch_bounds__(128) gdn_carry_kernel(const __grid_constant__ Pieces pieces, const float* M, const float* B, const float* S0, float* in,
                                                        float* ST, int Hv, int Dv)
{
    using L = Carry<DK>;
    extern __shared__ float fm[];
    float* S = fm + L::S_;
    const int tid = threadIdx.x, ri = tid >> 2, j = (tid & 3) * 4;
    const int h = blockIdx.x, seq = blockIdx.y, col = blockIdx.z * L::COLS + j;
    const int p0 = pieces.first[seq], p1 = pieces.first[seq + 1];
    constexpr int R = DK / 32;
    auto fetch = [&](int p) {
        const float* src = M + ((int64_t)p * Hv + h) * DK * DK;
        const uint32_t dst = smem_addr(fm + (p & 1) * DK * L::MROW);
        for (int e = tid; e < DK * DK / 4; e += L::THREADS)
            cp16(dst + (e / (DK / 4) * L::MROW + e % (DK / 4) * 4) * 4, src + e * 4, true);
        cp_async_commit();
    };
    float4 s[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        s[i] = S0 ? *(const float4*)(S0 + (((int64_t)seq * Hv + h) * DK + ri + 32 * i) * Dv + col) : make_float4(0.f, 0.f, 0.f, 0.f);
    // (the last piece's is for S_T alone)
    if (p0 + (ST ? 0 : 1) < p1) fetch(p0);
    for (int p = p0; p < p1; ++p) {
        const int64_t off = ((int64_t)p * Hv + h) * DK * Dv + col;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            *(float4*)(in + off + (int64_t)(ri + 32 * i) * Dv) = s[i];
            *(float4*)(S + (ri + 32 * i) * L::COLS + j) = s[i];
        }
        if (p + 1 == p1 && !ST) break;
        cp_async_wait_all();
        __syncthreads();
        if (p + (ST ? 1 : 2) < p1) fetch(p + 1);
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] = *(const float4*)(B + off + (int64_t)(ri + 32 * i) * Dv);
        const float* m = fm + (p & 1) * DK * L::MROW + ri * L::MROW;
#pragma unroll 4
        for (int k = 0; k < DK; k += 4) {
            float4 x[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) x[z] = *(const float4*)(S + (k + z) * L::COLS + j);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float4 w = *(const float4*)(m + 32 * i * L::MROW + k);
                const float ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    s[i].x = fmaf(ww[z], x[z].x, s[i].x);
                    s[i].y = fmaf(ww[z], x[z].y, s[i].y);
                    s[i].z = fmaf(ww[z], x[z].z, s[i].z);
                    s[i].w = fmaf(ww[z], x[z].w, s[i].w);
                }
            }
        }
        __syncthreads();
    }
    if (ST)
#pragma unroll
        for (int i = 0; i < R; ++i) *(float4*)(ST + (((int64_t)seq * Hv + h) * DK + ri + 32 * i) * Dv + col) = s[i];
}
template <int DK>
cudaError_t carry(const GdnArgs& a, const Seqs& s, const Pieces& pieces, const float* M, const float* B, float* in, cudaStream_t st)
{
    using L = Carry<DK>;
    const cudaError_t e = allow_smem<gdn_carry_kernel<DK>>(L::SMEM);
    if (e != cudaSuccess) return e;
    ProfileScope prof("gdn_carry", st);
    count_launch();
    gdn_carry_kernel<DK><<<dim3(a.Hv, s.n, a.Dv / L::COLS), L::THREADS, L::SMEM, st>>>(pieces, M, B, a.S0, in, a.ST, a.Hv, a.Dv);
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_chain(const GdnArgs& a, const Seqs& s, const void* records, void* kept, int* status, cudaStream_t st)
{
    return kept ? chain<CHAIN_KEEP>(a, s, records, kept, status, st) : chain<CHAIN_OUT>(a, s, records, nullptr, status, st);
}

int piece_chunks(const Seqs& s, int Hv, int Dk, int Dv, int sms)
{
    if (Dv == 32 || Dk == 32) return 0;
    int64_t longest = 0;
    for (int i = 0; i < s.n; ++i) longest = max(longest, ((int64_t)s.len(i) + C - 1) / C);
    auto pieces = [&](int64_t per) {
        int64_t n = 0;
        for (int i = 0; i < s.n; ++i) n += ((s.len(i) + C - 1) / C + per - 1) / per;
        return n;
    };
    // the shortest pieces that the SMs take at once
    int64_t lo = 1, hi = longest;
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (pieces(mid) * Hv <= sms && pieces(mid) <= kMaxSeqs) hi = mid; else lo = mid + 1;
    }
    const int64_t per = max(lo, (int64_t)8);
    if (pieces(per) * Hv > sms || pieces(per) > kMaxSeqs) return 0;
    // Steps in a row, in units of 0.1 us: 15 a chunk with columns of heads; 26 a chunk and launch, 40 a piece
    // carried, 150 for the launches.  Measured (columns, then pieces): one head pair of 6016 tokens 154 and 128 us, of
    // 12288 301 and 168; 16 heads of 8192 239 and 217, of 32768 913 and 614 (Dk = Dv = 128; 64 x 128 and 128 x 64 go by Dk);
    // Dk = Dv = 64: 138 and 91, 269 and 110, 213 and 163, 812 and 502.  (4096 tokens are not cut at any width.)
    const int64_t steps = (longest + per - 1) / per;
    return 3 * 26 * per + 40 * steps + 150 < 15 * longest ? (int)per : 0;
}
size_t pieces_workspace(const Seqs& s, int Hv, int Dk, int Dv, int per)
{
    int64_t n = 0;
    for (int i = 0; i < s.n; ++i) n += ((s.len(i) + C - 1) / C + per - 1) / per;
    return (size_t)(s.tokens() / C + n) * Hv * REC_BYTES + (size_t)n * Hv * Dk * (Dk + 2 * Dv) * sizeof(float);
}
cudaError_t launch_pieces(const GdnArgs& a, const Seqs& s, void* ws, int per, int* status, cudaStream_t st)
{
    Seqs cut;
    Pieces pieces;
    cut.n = 0;
    cut.T = -1;
    for (int i = 0; i < s.n; ++i) {
        pieces.first[i] = (int16_t)cut.n;
        for (int at = 0; at < s.len(i); at += per * C) cut.cu[cut.n++] = s.start(i) + at;
    }
    pieces.first[s.n] = (int16_t)cut.n;
    cut.cu[cut.n] = s.tokens();
    const size_t states = (size_t)cut.n * a.Hv * a.Dk;
    float* M = (float*)((char*)ws + (size_t)cut.slots(C) * a.Hv * REC_BYTES);
    float *B = M + states * a.Dk, *in = B + states * a.Dv;
    cudaError_t e = launch_prologue(a, cut, ws, st);
    GdnArgs x = a;
    x.S0 = nullptr;
    x.ST = B;
    if (e == cudaSuccess) e = chain<CHAIN_STATE>(x, cut, ws, nullptr, status, st);
    x.ST = M;
    if (e == cudaSuccess) e = a.Dk == 64 ? chain<64, 64, CHAIN_TRANSITION>(x, cut, ws, nullptr, status, st) : chain<128, 128, CHAIN_TRANSITION>(x, cut, ws, nullptr, status, st);
    if (e == cudaSuccess) e = a.Dk == 64 ? carry<64>(a, s, pieces, M, B, in, st) : carry<128>(a, s, pieces, M, B, in, st);
    x.S0 = in;
    x.ST = nullptr;
    if (e == cudaSuccess) e = chain<CHAIN_OUT>(x, cut, ws, nullptr, status, st);
    return e;
}

}  // namespace gdn
}  // namespace kda
