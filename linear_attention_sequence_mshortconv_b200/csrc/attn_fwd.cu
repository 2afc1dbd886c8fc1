// Causal attention with grouped heads on tcgen05 tensor cores (bf16, head width 64 or 128).
//
//   s_ij = scale q_i.k_j,  m_i = max_j s_ij,  p_ij = e^{s_ij - m_i},  o_i = sum_j p_ij v_j / sum_j p_ij,
// over the keys in blocks of 64 from the first, with a running m and sum.
//
// A CTA owns 256 rows of one key/value head's query group (row = token x query head of the
// group, so the group shares every K and V tile, and a tile's keys end soon after its first
// token) as two tiles of 128 rows:
//   warps 0-3 and 4-7: the softmax of tile 0 and 1, one row to a thread, so maxima and sums need
//                      no exchange;
//   warps 8 and 9:     issue the MMAs of tile 0 and 1, S = Q K^T and O += P V (P from tensor
//                      memory, where it takes the place of S);
//   warp 10:           TMA loads of K and V into rings.
// Each tile has two buffers of scores: while one block's softmax runs, P V of the block before
// and the scores of the block after are computed, so neither waits for the other.  With blocks
// of 128 keys there is room for one buffer a tile only; the chain S -> softmax -> P V -> S then
// left the tensor cores idle half of the time (16384 tokens, 16 heads, width 128: 0.93 ms).
// Tensor memory (512 columns): 2 x 2 x S (64 each), O0, O1 (D each).
//
// (16384 tokens, 16 heads to 4, width 128: 0.81 ms, 1.35 PFLOP/s or 82% of a large product's burst rate, at
// the power limit 0.95 ms, 83% of its sustained one; the exponentials and the tensor cores are both nearly full.)
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since the reference of
// its exponents was set (sums and weights then stay below 2^8 times their size, far from
// overflow), which after the first blocks is rare; the result does not depend on the reference.

#include "attn_tc.cuh"

namespace kda {
namespace attn {

namespace {

constexpr int QR = 128;   // rows of a tile
constexpr int KB = 64;    // keys of a block

template <int D>
struct Fwd {
    static constexpr int QPANEL = QR * 128, QTILE = D / 64 * QPANEL;   // bytes of 128 rows x 64 values, of a tile
    static constexpr int PANEL = KB * 128, TILE = D / 64 * PANEL;
    static constexpr int STAGES = D == 64 ? 6 : 4;          // K and V tiles in flight, each
    static constexpr int Q_ = 0, K_ = Q_ + 2 * QTILE, V_ = K_ + STAGES * TILE, BAR = V_ + STAGES * TILE;
    static constexpr int SMEM = BAR + 512 + 1024;           // the base is aligned up to 1024 bytes
    static constexpr int THREADS = 384;
    // tensor memory columns
    static constexpr int S_ = 0, O_ = 4 * KB;
};

__device__ __forceinline__ float max_of(const float (&s)[64])
{
    float m0 = s[0], m1 = s[1], m2 = s[2], m3 = s[3];
#pragma unroll
    for (int x = 4; x < 60; x += 8) {
        m0 = max3(m0, s[x], s[x + 1]);
        m1 = max3(m1, s[x + 2], s[x + 3]);
        m2 = max3(m2, s[x + 4], s[x + 5]);
        m3 = max3(m3, s[x + 6], s[x + 7]);
    }
    return max3(max3(m0, s[60], s[61]), max3(m1, s[62], s[63]), fmaxf(m2, m3));
}

template <int D>
__global__ void __launch_bounds__(384, 1)
attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_q,
                const __grid_constant__ CUtensorMap tm_o, bool boxes, AttnArgs a,
                const __grid_constant__ Seqs seqs, const __grid_constant__ Tiles tiles, int* status, int drop)
{
    using L = Fwd<D>;
    extern __shared__ char raw[];
    char* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t base = smem_addr(sm);
    uint64_t* bars = (uint64_t*)(sm + L::BAR);
    uint64_t *kfull = bars, *kempty = kfull + L::STAGES, *vfull = kempty + L::STAGES, *vempty = vfull + L::STAGES;
    uint64_t *sfull = vempty + L::STAGES, *pready = sfull + 4, *pvdone = pready + 4, *vfix = pvdone + 4, *drain = vfix + 1;
    uint64_t* qfull = drain + 2;   // by tile, where Q comes in boxes
    uint32_t* tm_ptr = (uint32_t*)(qfull + 2);
    const Guard guard{(volatile int*)(tm_ptr + 1), status};

    const int tid = threadIdx.x, lane = tid & 31, warp = uniform_warp();
    int hk, seq, rank;
    tiles.locate(blockIdx.x, hk, seq, rank);
    const int64_t t0 = seqs.start(seq);
    const int len = seqs.len(seq);
    // a sequence's last tile has the most keys
    const uint32_t r = a.H / a.Hkv, all = (uint32_t)len * r, first = ((all + 2 * QR - 1) / (2 * QR) - 1 - rank) * 2 * QR;
    auto blocks = [&](int t) {   // key blocks tile t sees
        const uint32_t r0 = first + t * QR;
        return r0 >= all ? 0 : (int)((min(r0 + QR, all) - 1) / r / KB + 1);
    };
    const int n0 = blocks(0), n1 = blocks(1), n = max(n0, n1);

    const RowAt row_at{t0, a.H, hk * (int)r, (int)r, D};

    auto load_k = [&](int j) {
        const int s = j % L::STAGES;
        mbar_arrive_expect_tx(kfull + s, L::TILE);
        for (int p = 0; p < D / 64; ++p)
            tma_load_3d(sm + L::K_ + s * L::TILE + p * L::PANEL, &tm_k, kfull + s, p * 64, hk, (int)t0 + j * KB);
    };
    auto load_v = [&](int j) {
        const int s = j % L::STAGES;
        mbar_arrive_expect_tx(vfull + s, L::TILE);
        for (int p = 0; p < D / 64; ++p)
            tma_load_3d(sm + L::V_ + s * L::TILE + p * L::PANEL, &tm_v, vfull + s, p * 64, hk, (int)t0 + j * KB);
    };
    if (warp == 10) {
        if (lane == 0) {
            for (int i = 0; i < L::STAGES; ++i) {
                mbar_init(kfull + i, 1);
                mbar_init(kempty + i, 2);
                mbar_init(vfull + i, 1);
                mbar_init(vempty + i, 2);
            }
            for (int i = 0; i < 4; ++i) {   // 2 x tile + buffer
                mbar_init(sfull + i, 1);
                mbar_init(pready + i, QR + 32 * drop);
                mbar_init(pvdone + i, 1);
            }
            mbar_init(vfix, 32);
            mbar_init(drain, 1);
            mbar_init(drain + 1, 1);
            mbar_init(qfull, 1);
            mbar_init(qfull + 1, 1);
            *guard.flag = 0;
            fence_mbar_init();
            fence_async_smem();
            // (rows past the sequence's end are another one's, or zeros: no other row sees them)
            for (int t = 0; boxes && t < 2 && first + t * QR < all; ++t) {
                mbar_arrive_expect_tx(qfull + t, L::QTILE);
                for (int p = 0; p < D / 64; ++p)
                    tma_load_3d(sm + L::Q_ + t * L::QTILE + p * L::QPANEL, &tm_q, qfull + t, p * 64, hk * r, (int)t0 + (first + t * QR) / r);
            }
            for (int j = 0; j < n && j < L::STAGES; ++j) {
                load_k(j);
                load_v(j);
            }
        }
    } else if (warp == 8) {
        tmem_alloc(tm_ptr, 512);
        tmem_relinquish();
    } else if (warp < 8 && !boxes) {
        // Q: rows past the sequence's end are zeros
        for (int e = tid; e < 2 * QR * (D / 8); e += 256) {
            const int piece = e % (D / 8), row = e / (D / 8);
            const bool in = first + row < all;
            cp16(base + L::Q_ + (row / QR) * L::QTILE + (piece >> 3) * L::QPANEL + piece_at(row % QR, piece & 7),
                 (const __nv_bfloat16*)a.q + (in ? row_at(first + row) + piece * 8 : 0), in);
        }
        cp_async_commit();
        cp_async_wait_all();
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm_ptr;

    if (warp >= 10) {
        if (warp == 10 && lane == 0) {
            int k_issued = min(n, L::STAGES), v_issued = k_issued;
            for (int j = k_issued; j < n; ++j) {
                const int s = j % L::STAGES, u = j / L::STAGES;
                wait(kempty + s, (u & 1) ^ 1, guard);
                if (guard.up()) break;
                load_k(j);
                ++k_issued;
                wait(vempty + s, (u & 1) ^ 1, guard);
                if (guard.up()) break;
                load_v(j);
                ++v_issued;
            }
            for (int t = 0; boxes && t < 2 && first + t * QR < all; ++t) mbar_wait_bounded(qfull + t, 0, kWaitNs);
            drain_ring(kfull, L::STAGES, k_issued);
            drain_ring(vfull, L::STAGES, v_issued);
        }
        __syncwarp();
        // The last block's rows past the end hold the next sequence, or nothing: their weights are
        // 0, but 0 times a value that is not finite is not.  The whole warp clears them.
        const int tail = len - (n - 1) * KB;
        if (warp == 10 && tail < KB && !guard.up()) {
            const int s = (n - 1) % L::STAGES;
            wait(vfull + s, ((n - 1) / L::STAGES) & 1, guard);
            for (int e = lane; e < (KB - tail) * (D / 8); e += 32) {
                const int row = tail + e / (D / 8), piece = e % (D / 8);
                *(uint4*)(sm + L::V_ + s * L::TILE + (piece >> 3) * L::PANEL + piece_at(row, piece & 7)) = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            mbar_arrive(vfix);
        }
    } else if (warp >= 8) {
        const int t = warp - 8, nt = t ? n1 : n0;
        const uint32_t id_s = idesc_f16(QR, KB, false, false, a.scale < 0.f, true);
        const uint32_t id_o = idesc_f16(QR, D, false, true, false, true);
        const uint32_t ts = tmem + L::S_ + t * 2 * KB, to = tmem + L::O_ + t * D;
        const uint64_t dq = desc_rows(base + L::Q_ + t * L::QTILE), dk = desc_rows(base + L::K_), dv = desc_cols(base + L::V_, L::PANEL);
        auto scores = [&](int j) {
            const int s = j % L::STAGES;
            tc_fence_after();
            if (elect()) {
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
                    umma_f16(ts + (j & 1) * KB, step_rows(dq, x, L::QPANEL), step_rows(dk + (s * L::TILE >> 4), x, L::PANEL), id_s, x > 0);
                umma_commit(sfull + 2 * t + (j & 1));
                umma_commit(kempty + s);
            }
        };
        // Each wait costs some 85 cycles even when there is nothing to wait for: those for the copies
        // are made while MMAs already issued run.
        if (boxes && nt > 0) wait(qfull + t, 0, guard);
        for (int j = 0; j < 2 && j < nt; ++j) {
            wait(kfull + j, 0, guard);
            scores(j);
        }
        for (int j = 0; j < nt; ++j) {
            const int s = j % L::STAGES, w = 2 * t + (j & 1), u = (j >> 1) & 1;
            wait(vfull + s, (j / L::STAGES) & 1, guard);
            if (j == n - 1 && len - j * KB < KB) wait(vfix, 0, guard);
            wait(pready + w, u, guard);
            tc_fence_after();
            if (elect()) {
#pragma unroll
                for (int x = 0; x < KB / 16; ++x)
                    umma_f16_ts(to, ts + (j & 1) * KB + x * 8, step_cols(dv + (s * L::TILE >> 4), x), id_o, j > 0 || x > 0);
                umma_commit(vempty + s);
                umma_commit(pvdone + w);
            }
            if (j + 2 < nt) {
                wait(kfull + (j + 2) % L::STAGES, ((j + 2) / L::STAGES) & 1, guard);
                wait(pvdone + w, u, guard);   // P is in S's place: it must have been read
                scores(j + 2);
            }
        }
        if (lane == 0) {
            // blocks that only the other tile sees: this one is done with them, once the stage's
            // use before has ended (an arrival counts for the phase that is open)
            for (int j = nt; j < n && !guard.up(); ++j) {
                const int s = j % L::STAGES, u = j / L::STAGES;
                wait(kempty + s, (u & 1) ^ 1, guard);
                mbar_arrive(kempty + s);
                wait(vempty + s, (u & 1) ^ 1, guard);
                mbar_arrive(vempty + s);
            }
        }
        __syncwarp();
        drain_mma(drain + t);
    } else {
        const int t = warp >> 2, nt = t ? n1 : n0;
        const uint32_t i = first + t * QR + (tid & 127);
        const bool real = i < all;
        const int token = (int)(min(i, all - 1) / r);
        const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
        const uint32_t ts = tmem + L::S_ + t * 2 * KB + lanes, to = tmem + L::O_ + t * D + lanes;
        // scores come with the sign of scale applied by the MMA; never 0, so that a masked -inf stays one
        const float sl = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
        // the warp's first row sees the fewest keys
        const int least = (int)(min(first + t * QR + (warp & 3) * 32, all - 1) / r);
        float ref = 0.f, sum = 0.f;
        for (int j = 0; j < nt; ++j) {
            const int w = 2 * t + (j & 1), u = (j >> 1) & 1;
            wait(sfull + w, u, guard);
            tc_fence_after();
            float s[64];
            tmem_ld64(ts + (j & 1) * KB, s);
            if (j * KB + KB - 1 > least) {
                const int seen = token - j * KB;   // keys 0 .. seen of the block
#pragma unroll
                for (int x = 0; x < 64; ++x)
                    if (x > seen) s[x] = -INFINITY;
            }
            const float top = max_of(s);
            if (j == 0) ref = top;
            float off = -ref * sl;
            if (__any_sync(~0u, (top - ref) * sl > 8.f || fabsf(off) > 1048576.f)) {
                const bool grown = (top - ref) * sl > 8.f;
                if (__any_sync(~0u, grown)) {
                    const float f = grown ? ex2_approx((ref - top) * sl) : 1.f;
                    if (grown) ref = top;
                    off = -ref * sl;
                    sum *= f;
                    wait(pvdone + (w ^ 1), ((j - 1) >> 1) & 1, guard);
                    tc_fence_after();
#pragma unroll
                    for (int x = 0; x < D; x += 32) {
                        float o[32];
                        tmem_ld32(to + x, o);
#pragma unroll
                        for (int y = 0; y < 32; ++y) o[y] *= f;
                        tmem_st32(to + x, o);
                    }
                }
                // Far from 0 the product's rounding would be more than the exponent itself (and -inf less -inf is no
                // number): such a reference is taken off the scores, and a row that has seen only -inf has none.
                if (__any_sync(~0u, fabsf(off) > 1048576.f)) {
                    const float from = ref == -INFINITY ? 0.f : ref;
#pragma unroll
                    for (int x = 0; x < 64; ++x) s[x] -= from;
                    off = 0.f;
                }
            }
            const uint64_t sl2 = pair(sl, sl), off2 = pair(off, off);
            uint64_t z = 0, y = 0;
            uint32_t p[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                float e0, e1;
                unpair(fma2(pair(s[2 * x], s[2 * x + 1]), sl2, off2), e0, e1);
                e0 = ex2_approx(e0);
                e1 = ex2_approx(e1);
                if (x & 1) y = add2(y, pair(e0, e1)); else z = add2(z, pair(e0, e1));
                p[x] = pack_bf16(e0, e1);
            }
            tmem_st32u_nowait(ts + (j & 1) * KB, p);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(pready + w);
            float z0, z1;
            unpair(add2(z, y), z0, z1);
            sum += z0 + z1;
        }
        if (nt > 0) {
            wait(pvdone + 2 * t + ((nt - 1) & 1), ((nt - 1) >> 1) & 1, guard);
            tc_fence_after();
            // every product that read Q has ended: its tile takes the output
            const bool whole = boxes && first + t * QR + QR <= all;
            if (whole)   // (after a timeout too: the four warps meet in it, and may see the flag at different times)
                store_box<D>(to, 1.f / sum, sm + L::Q_ + t * L::QTILE, &tm_o, hk * r, (int)t0 + (first + t * QR) / r, tid & 127, 1 + t);
            if (!warp_up(guard)) {
                const int64_t off = real ? row_at(i) : -1;
                if (!whole) store_rows<D>(to, 1.f / sum, sm + L::Q_ + t * L::QTILE, (__nv_bfloat16*)a.o, off, tid & 127);
                if (real && a.lse) a.lse[off / D] = (ref * sl + log2f(sum)) * kLn2;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t forward(const AttnArgs& a, const Seqs& s, int* status, cudaStream_t st)
{
    using L = Fwd<D>;
    CUtensorMap k, v, q{}, o{};
    const int r = a.H / a.Hkv;
    const bool boxes = box_rows(r);
    if (!make_map(&k, a.k, s.tokens(), a.Hkv, D, 64, 1, KB) || !make_map(&v, a.v, s.tokens(), a.Hkv, D, 64, 1, KB) ||
        (boxes && (!make_map(&q, a.q, s.tokens(), a.H, D, 64, r, QR / r) || !make_map(&o, a.o, s.tokens(), a.H, D, 64, r, QR / r))))
        return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<attn_fwd_kernel<D>>(L::SMEM);
    if (e != cudaSuccess) return e;
    Tiles tiles;
    const int64_t ctas = make_tiles(tiles, s, a.Hkv, r, 2 * QR);
    ProfileScope prof("attn_fwd", st);
    count_launch();
    attn_fwd_kernel<D><<<(unsigned)ctas, L::THREADS, L::SMEM, st>>>(k, v, q, o, boxes, a, s, tiles, status, debug_drop_handoff());
    return cudaGetLastError();
}
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
}  // namespace
}  // namespace attn

bool attn_tc_supported(const AttnArgs& a)
{
    return a.t == ET_BF16 && (a.D == 64 || a.D == 128) && attn::aligned16(a.q) && attn::aligned16(a.k) &&
           attn::aligned16(a.v) && attn::aligned16(a.o);
}

cudaError_t launch_attn_tc(const AttnArgs& a, const Seqs& s, int* status, cudaStream_t st)
{
    return a.D == 64 ? attn::forward<64>(a, s, status, st) : attn::forward<128>(a, s, status, st);
}

}  // namespace kda
