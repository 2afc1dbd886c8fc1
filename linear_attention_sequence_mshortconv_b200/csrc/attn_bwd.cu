// Gradients of causal attention with grouped heads on tcgen05 tensor cores (bf16, head width 64
// or 128):
//   p_ij = e^{s_ij - lse_i},  dv_j = sum_i p_ij do_i,
//   ds_ij = p_ij (do_i.v_j - delta_i),  delta_i = do_i.o_i,
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i.
//
// Two kernels, so that every sum has one owner and no atomics are needed: one owns 128 keys and
// goes over the rows (token x query head of the group) that see them, so dk and dv are summed
// over the group where they are accumulated; the other owns 256 rows and goes over the keys.
// That computes s and do.v twice (7 products instead of 5), but results do not depend on an
// order of arrival and no fp32 gradient passes through memory.  A first kernel computes delta and
// lays it and lse out row by row.
//
// 4 rows of 4352 tokens, 16 heads to 4, width 128: delta 40 us, rows 405, keys 475; the 7 products run at 1.23 PFLOP/s.
//
// Both kernels have the forward's roles: warps 0-3 and 4-7 turn scores into the operands of the
// next product, warps 8 and 9 issue the MMAs, warp 10 the loads.

#include "attn_tc.cuh"

namespace kda {
namespace attn {
namespace {

// ---- delta ----------------------------------------------------------------------------------
// -lse log2(e) and -delta of every row, [key/value head][token][head of the group] each.  Bound by
// the bytes of o and do: D / 8 lanes to a row, 16 bytes of each a lane, four rows in flight.
template <int D>
__global__ void __launch_bounds__(256) attn_delta_kernel(AttnArgs a, const __nv_bfloat16* dout, float* nlse, float* ndelta, int64_t tokens)
{
    constexpr int P = D / 8, PER = 256 / P, U = 4;   // lanes to a row, rows of a block at once
    const int piece = threadIdx.x % P;
    const int64_t row0 = (int64_t)blockIdx.x * PER * U + threadIdx.x / P, n = tokens * a.H;
    uint4 x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + u * PER;
        const bool in = row < n;
        x[u] = in ? *(const uint4*)((const __nv_bfloat16*)a.o + row * D + piece * 8) : make_uint4(0, 0, 0, 0);
        y[u] = in ? *(const uint4*)(dout + row * D + piece * 8) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t p[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, q[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s = fmaf(__uint_as_float(p[i] << 16), __uint_as_float(q[i] << 16),
                     fmaf(__uint_as_float(p[i] & 0xffff0000u), __uint_as_float(q[i] & 0xffff0000u), s));
#pragma unroll
        for (int o = 1; o < P; o <<= 1) s += __shfl_xor_sync(~0u, s, o);
        const int64_t row = row0 + u * PER;
        if (piece == 0 && row < n) {
            const int h = (int)(row % a.H), r = a.H / a.Hkv;
            const int64_t at = ((int64_t)(h / r) * tokens + row / a.H) * r + h % r;
            nlse[at] = -a.lse[row] * kLog2e;
            ndelta[at] = -s;
        }
    }
}

// ---- dk and dv ------------------------------------------------------------------------------
// Keys are rows of every product: S^T = K Q^T and dP^T = V dO^T for 64 rows at a time, then
// dV += P^T dO and dK += dS^T Q with P^T and dS^T read from tensor memory.  Two buffers of
// (S^T, dP^T), one to each softmax warpgroup: while one is turned into P and dS, the tensor cores
// fill or read the other.  Tensor memory: dV, dK (D columns each), 2 x (64 + 64).
// A tile holds 64 / r tokens, all heads of the group, as one TMA box; rows left over where r does
// not divide 64 stay zero.
template <int D>
struct Keys {
    static constexpr int KEYS = 128, RB = 64;
    static constexpr int KPANEL = KEYS * 128, KTILE = D / 64 * KPANEL;
    static constexpr int RPANEL = RB * 128, RTILE = D / 64 * RPANEL;
    static constexpr int STAGES = D == 64 ? 6 : 4;          // (Q, dO) tiles in flight
    static constexpr int K_ = 0, V_ = K_ + KTILE, Q_ = V_ + KTILE, G_ = Q_ + STAGES * RTILE;
    static constexpr int LD = G_ + STAGES * RTILE;          // [2 warpgroups][2][-lse, -delta][64]
    static constexpr int BAR = LD + 8 * RB * 4;
    static constexpr int SMEM = BAR + 512 + 1024;
    static constexpr int DV_ = 0, DK_ = D, S_ = 2 * D, P_ = 2 * D + RB, BUF = 2 * RB;
};

template <int D>
__global__ void __launch_bounds__(384, 1)
attn_bwd_keys_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_g, AttnBwdArgs b,
                     const __grid_constant__ Seqs seqs, const __grid_constant__ Tiles tiles, const float* nlse, const float* ndelta, int* status, int drop)
{
    using L = Keys<D>;
    const AttnArgs& a = b.f;
    extern __shared__ char raw[];
    char* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t base = smem_addr(sm);
    uint64_t* bars = (uint64_t*)(sm + L::BAR);
    uint64_t *kvfull = bars, *full = kvfull + 1, *empty = full + L::STAGES, *sfull = empty + L::STAGES, *gfull = sfull + 2;
    uint64_t *pready = gfull + 2, *dready = pready + 2, *done = dready + 2, *fix = done + 2, *all_done = fix + 1, *drain = all_done + 1;
    uint32_t* tm_ptr = (uint32_t*)(drain + 2);
    const Guard guard{(volatile int*)(tm_ptr + 1), status};

    const int tid = threadIdx.x, lane = tid & 31, warp = uniform_warp();
    const int r = a.H / a.Hkv;
    int hk, seq, rank;
    tiles.locate(blockIdx.x, hk, seq, rank);
    const int64_t t0 = seqs.start(seq);
    const int len = seqs.len(seq), key0 = rank * L::KEYS;   // a sequence's first tile has the most rows
    const int tq = L::RB / r;                                // tokens of a tile of rows
    const int n = (len - key0 + tq - 1) / tq;
    const int tail = (len - key0 - (n - 1) * tq) * r;        // rows of the last tile

    auto load = [&](int j) {
        const int s = j % L::STAGES;
        mbar_arrive_expect_tx(full + s, (uint32_t)(2 * tq * r * D * 2));
        for (int p = 0; p < D / 64; ++p) {
            tma_load_3d(sm + L::Q_ + s * L::RTILE + p * L::RPANEL, &tm_q, full + s, p * 64, hk * r, (int)t0 + key0 + j * tq);
            tma_load_3d(sm + L::G_ + s * L::RTILE + p * L::RPANEL, &tm_g, full + s, p * 64, hk * r, (int)t0 + key0 + j * tq);
        }
    };
    if (warp == 10) {
        if (lane == 0) {
            mbar_init(kvfull, 1);
            for (int i = 0; i < L::STAGES; ++i) {
                mbar_init(full + i, 1);
                mbar_init(empty + i, 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(sfull + i, 1);
                mbar_init(gfull + i, 1);
                mbar_init(pready + i, 128 + 32 * drop);
                mbar_init(dready + i, 128);
                mbar_init(done + i, 1);
                mbar_init(drain + i, 1);
            }
            mbar_init(fix, 32);
            mbar_init(all_done, 1);
            *guard.flag = 0;
            fence_mbar_init();
            fence_async_smem();
            mbar_arrive_expect_tx(kvfull, 2 * L::KTILE);
            for (int p = 0; p < D / 64; ++p) {
                tma_load_3d(sm + L::K_ + p * L::KPANEL, &tm_k, kvfull, p * 64, hk, (int)t0 + key0);
                tma_load_3d(sm + L::V_ + p * L::KPANEL, &tm_v, kvfull, p * 64, hk, (int)t0 + key0);
            }
            for (int j = 0; j < n && j < L::STAGES; ++j) load(j);
        }
    } else if (warp == 8) {
        tmem_alloc(tm_ptr, 512);
        tmem_relinquish();
    } else if (tq * r < L::RB && warp < 8) {   // rows that no copy writes
        for (int e = tid; e < 2 * L::STAGES * (L::RB - tq * r) * (D / 8); e += 256) {
            const int piece = e % (D / 8), row = tq * r + e / (D / 8) % (L::RB - tq * r), st = e / (D / 8) / (L::RB - tq * r);
            *(uint4*)(sm + L::Q_ + st * L::RTILE + (piece >> 3) * L::RPANEL + piece_at(row, piece & 7)) = make_uint4(0, 0, 0, 0);
        }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm_ptr;

    if (warp >= 10) {
        if (warp == 10 && lane == 0) {
            int issued = min(n, L::STAGES);
            for (; issued < n; ++issued) {
                wait(empty + issued % L::STAGES, ((issued / L::STAGES) & 1) ^ 1, guard);
                if (guard.up()) break;
                load(issued);
            }
            mbar_wait_bounded(kvfull, 0, kWaitNs);
            drain_ring(full, L::STAGES, issued);
        }
        __syncwarp();
        // rows of the last tile past the end: their weights are 0, but 0 times a value that is not
        // finite (the next sequence's) is not
        if (warp == 10 && tail < tq * r && !guard.up()) {
            const int s = (n - 1) % L::STAGES;
            wait(full + s, ((n - 1) / L::STAGES) & 1, guard);
            for (int e = lane; e < 2 * (tq * r - tail) * (D / 8); e += 32) {
                const int piece = e % (D / 8), row = tail + e / (D / 8) % (tq * r - tail), g = e / (D / 8) / (tq * r - tail);
                *(uint4*)(sm + (g ? L::G_ : L::Q_) + s * L::RTILE + (piece >> 3) * L::RPANEL + piece_at(row, piece & 7)) = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            mbar_arrive(fix);
        }
    } else if (warp == 9) {   // scores and dP
        const uint32_t id_s = idesc_f16(L::KEYS, L::RB, false, false, a.scale < 0.f, true);
        const uint32_t id_g = idesc_f16(L::KEYS, L::RB, false, false, false, true);
        const uint64_t dk = desc_rows(base + L::K_), dv = desc_rows(base + L::V_), dq = desc_rows(base + L::Q_), dg = desc_rows(base + L::G_);
        wait(kvfull, 0, guard);
        for (int j = 0; j < n; ++j) {
            const int s = j % L::STAGES, w = j & 1;
            wait(full + s, (j / L::STAGES) & 1, guard);
            if (j == n - 1 && tail < tq * r) wait(fix, 0, guard);
            if (j >= 2) wait(done + w, ((j - 2) >> 1) & 1, guard);   // P and dS are in the places of S and dP
            tc_fence_after();
            if (elect()) {
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
                    umma_f16(tmem + L::S_ + w * L::BUF, step_rows(dk, x, L::KPANEL), step_rows(dq + (s * L::RTILE >> 4), x, L::RPANEL), id_s, x > 0);
                umma_commit(sfull + w);
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
                    umma_f16(tmem + L::P_ + w * L::BUF, step_rows(dv, x, L::KPANEL), step_rows(dg + (s * L::RTILE >> 4), x, L::RPANEL), id_g, x > 0);
                umma_commit(gfull + w);
            }
        }
        drain_mma(drain + 1);
    } else if (warp == 8) {   // dV and dK
        const uint32_t id_o = idesc_f16(L::KEYS, D, false, true, false, true);
        const uint64_t dq = desc_cols(base + L::Q_, L::RPANEL), dg = desc_cols(base + L::G_, L::RPANEL);
        for (int j = 0; j < n; ++j) {
            const int s = j % L::STAGES, w = j & 1, u = (j >> 1) & 1;
            wait(pready + w, u, guard);
            tc_fence_after();
            if (elect()) {
#pragma unroll
                for (int x = 0; x < L::RB / 16; ++x)
                    umma_f16_ts(tmem + L::DV_, tmem + L::S_ + w * L::BUF + x * 8, step_cols(dg + (s * L::RTILE >> 4), x), id_o, j > 0 || x > 0);
            }
            wait(dready + w, u, guard);
            tc_fence_after();
            if (elect()) {
#pragma unroll
                for (int x = 0; x < L::RB / 16; ++x)
                    umma_f16_ts(tmem + L::DK_, tmem + L::P_ + w * L::BUF + x * 8, step_cols(dq + (s * L::RTILE >> 4), x), id_o, j > 0 || x > 0);
                umma_commit(empty + s);
                umma_commit(done + w);
                if (j == n - 1) umma_commit(all_done);
            }
        }
        drain_mma(drain);
    } else {
        const int w = warp >> 2, key = key0 + (tid & 127);
        const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
        const uint32_t ts = tmem + L::S_ + w * L::BUF + lanes, tp = tmem + L::P_ + w * L::BUF + lanes;
        const float sl = fabsf(a.scale) * kLog2e;
        const uint64_t sl2 = pair(sl, sl);
        // threads 0-63 fetch -lse of the tile's rows, 64-127 -delta: one tile ahead, in registers
        const float* src = ((tid & 64) ? ndelta : nlse) + ((int64_t)hk * seqs.tokens() + t0 + key0) * r + (tid & 63);
        auto fetch = [&](int j) { return j < n && (tid & 63) < (j == n - 1 ? tail : tq * r) ? src[(int64_t)j * tq * r] : 0.f; };
        float* ld = (float*)(sm + L::LD) + w * 4 * L::RB;
        float ahead = fetch(w);
        for (int j = w; j < n; j += 2) {
            const int u = (j >> 1) & 1;
            const int live = j == n - 1 ? tail : tq * r;   // rows of this tile
            ld[u * 2 * L::RB + (tid & 127)] = ahead;
            asm volatile("bar.sync %0, 128;" ::"r"(1 + w) : "memory");
            ahead = fetch(j + 2);
            const ulonglong2* col = (const ulonglong2*)(ld + u * 2 * L::RB);   // -lse of four rows; -delta 16 further
            // the first row (column) that sees this key
            const int lo = (key - key0 - j * tq) * r;
            wait(sfull + w, u, guard);
            tc_fence_after();
            float p[64];
            tmem_ld64(ts, p);
#pragma unroll
            for (int x = 0; x < 64; x += 4) {
                const ulonglong2 c = col[x / 4];
                unpair(fma2(pair(p[x], p[x + 1]), sl2, c.x), p[x], p[x + 1]);
                unpair(fma2(pair(p[x + 2], p[x + 3]), sl2, c.y), p[x + 2], p[x + 3]);
            }
#pragma unroll
            for (int x = 0; x < 64; ++x) p[x] = ex2_approx(p[x]);
            const bool edge = j * tq < L::KEYS || live < L::RB;   // warp-uniform
            if (edge)
#pragma unroll
                for (int x = 0; x < 64; ++x)
                    if (x < lo || x >= live) p[x] = 0.f;
            uint32_t q[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) q[x] = pack_bf16(p[2 * x], p[2 * x + 1]);
            tmem_st32u_nowait(ts, q);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(pready + w);
            wait(gfull + w, u, guard);
            tc_fence_after();
#pragma unroll
            for (int hlf = 0; hlf < 2; ++hlf) {
                float g[32];
                tmem_ld32(tp + hlf * 32, g);
#pragma unroll
                for (int x = 0; x < 32; x += 4) {
                    const ulonglong2 c = col[16 + hlf * 8 + x / 4];
                    unpair(mul2(pair(p[hlf * 32 + x], p[hlf * 32 + x + 1]), add2(pair(g[x], g[x + 1]), c.x)), g[x], g[x + 1]);
                    unpair(mul2(pair(p[hlf * 32 + x + 2], p[hlf * 32 + x + 3]), add2(pair(g[x + 2], g[x + 3]), c.y)), g[x + 2], g[x + 3]);
                }
                if (edge)   // what a masked dP held may not be finite
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (hlf * 32 + x < lo || hlf * 32 + x >= live) g[x] = 0.f;
#pragma unroll
                for (int x = 0; x < 16; ++x) q[hlf * 16 + x] = pack_bf16(g[2 * x], g[2 * x + 1]);
            }
            tmem_st32u_nowait(tp, q);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(dready + w);
        }
        wait(all_done, 0, guard);
        tc_fence_after();
        if (!warp_up(guard)) {
            const int64_t off = key < len ? ((t0 + key) * a.Hkv + hk) * D : -1;
            // K and V have been read: dV and dK go out through their places
            if (w == 0)
                store_rows<D>(tmem + L::DV_ + lanes, 1.f, sm + L::V_, (__nv_bfloat16*)b.dv, off, tid & 127);
            else
                store_rows<D>(tmem + L::DK_ + lanes, a.scale, sm + L::K_, (__nv_bfloat16*)b.dk, off, tid & 127);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// ---- dq -------------------------------------------------------------------------------------
// The forward's layout: two tiles of 128 rows in turn over blocks of 64 keys, S = Q K^T and
// dP = dO V^T, then dQ += dS K.  Tensor memory: dQ0, dQ1 (D each), 2 x (S 64, dP 64).
//
// delta = do.o is as exact as the rounded o.  For a row that sees few keys o is as large as a value, and
// its rounding (2^-8) weighs as much in dS as dS's own: rows of the first SHORT blocks take
// delta = sum_j p_ij (do_i.v_j) from a pass of their own over their keys (a few blocks), and leave it
// for the keys' kernel, which runs after this one.  For longer rows o is an average, and smaller.
template <int D>
struct Dq {
    static constexpr int QR = 128, KB = 64, SHORT = 4;
    static constexpr int QPANEL = QR * 128, QTILE = D / 64 * QPANEL;
    static constexpr int KPANEL = KB * 128, KTILE = D / 64 * KPANEL;
    static constexpr int STAGES = D == 64 ? 6 : 2;
    static constexpr int Q_ = 0, G_ = Q_ + 2 * QTILE, K_ = G_ + 2 * QTILE, V_ = K_ + STAGES * KTILE;
    static constexpr int BAR = V_ + STAGES * KTILE, SMEM = BAR + 512 + 1024;
    static constexpr int DQ_ = 0, S_ = 2 * D, P_ = 2 * D + KB, BUF = 2 * KB;
};

template <int D>
__global__ void __launch_bounds__(384, 1)
attn_bwd_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_g, const __grid_constant__ CUtensorMap tm_dq, bool boxes, AttnBwdArgs b,
                     const __grid_constant__ Seqs seqs, const __grid_constant__ Tiles tiles, const float* nlse, float* ndelta, int* status, int drop)
{
    using L = Dq<D>;
    const AttnArgs& a = b.f;
    extern __shared__ char raw[];
    char* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t base = smem_addr(sm);
    uint64_t* bars = (uint64_t*)(sm + L::BAR);
    uint64_t *full = bars, *empty = full + L::STAGES, *sfull = empty + L::STAGES, *gfull = sfull + 2, *dready = gfull + 2;
    uint64_t *done = dready + 2, *fix = done + 2, *drain = fix + 1;
    uint64_t* qfull = drain + 2;   // by tile, where Q and dO come in boxes
    uint32_t* tm_ptr = (uint32_t*)(qfull + 2);
    const Guard guard{(volatile int*)(tm_ptr + 1), status};

    const int tid = threadIdx.x, lane = tid & 31, warp = uniform_warp();
    int hk, seq, rank;
    tiles.locate(blockIdx.x, hk, seq, rank);
    const int64_t t0 = seqs.start(seq);
    const int len = seqs.len(seq);
    const uint32_t r = a.H / a.Hkv, all = (uint32_t)len * r, first = ((all + 2 * L::QR - 1) / (2 * L::QR) - 1 - rank) * 2 * L::QR;
    auto blocks = [&](int t) {
        const uint32_t r0 = first + t * L::QR;
        return r0 >= all ? 0 : (int)((min(r0 + L::QR, all) - 1) / r / L::KB + 1);
    };
    const int n0 = blocks(0), n1 = blocks(1), n = max(n0, n1);
    const int tail = len - (n - 1) * L::KB;   // keys of the last block
    const int passes = n <= L::SHORT ? 2 : 1, total = passes * n;   // blocks that go through the ring

    const RowAt row_at{t0, a.H, hk * (int)r, (int)r, D};
    auto load = [&](int j) {
        const int s = j % L::STAGES, y = (int)t0 + j % n * L::KB;
        mbar_arrive_expect_tx(full + s, 2 * L::KTILE);
        for (int p = 0; p < D / 64; ++p) {
            tma_load_3d(sm + L::K_ + s * L::KTILE + p * L::KPANEL, &tm_k, full + s, p * 64, hk, y);
            tma_load_3d(sm + L::V_ + s * L::KTILE + p * L::KPANEL, &tm_v, full + s, p * 64, hk, y);
        }
    };
    if (warp == 10) {
        if (lane == 0) {
            for (int i = 0; i < L::STAGES; ++i) {
                mbar_init(full + i, 1);
                mbar_init(empty + i, 2);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(sfull + i, 1);
                mbar_init(gfull + i, 1);
                mbar_init(dready + i, 128 + 32 * drop);
                mbar_init(done + i, 1);
                mbar_init(drain + i, 1);
                mbar_init(qfull + i, 1);
            }
            mbar_init(fix, 32);
            *guard.flag = 0;
            fence_mbar_init();
            fence_async_smem();
            // (rows past the sequence's end are another one's, or zeros: no other row sees them)
            for (int t = 0; boxes && t < 2 && first + t * L::QR < all; ++t) {
                mbar_arrive_expect_tx(qfull + t, 2 * L::QTILE);
                for (int p = 0; p < D / 64; ++p) {
                    const int at = t * L::QTILE + p * L::QPANEL, y = (int)t0 + (first + t * L::QR) / r;
                    tma_load_3d(sm + L::Q_ + at, &tm_q, qfull + t, p * 64, hk * r, y);
                    tma_load_3d(sm + L::G_ + at, &tm_g, qfull + t, p * 64, hk * r, y);
                }
            }
            for (int j = 0; j < total && j < L::STAGES; ++j) load(j);
        }
    } else if (warp == 8) {
        tmem_alloc(tm_ptr, 512);
        tmem_relinquish();
    } else if (warp < 8 && !boxes) {
        for (int e = tid; e < 2 * L::QR * (D / 8); e += 256) {
            const int piece = e % (D / 8), row = e / (D / 8);
            const bool in = first + row < all;
            const int64_t off = in ? row_at(first + row) + piece * 8 : 0;
            const uint32_t at = (row / L::QR) * L::QTILE + (piece >> 3) * L::QPANEL + piece_at(row % L::QR, piece & 7);
            cp16(base + L::Q_ + at, (const __nv_bfloat16*)a.q + off, in);
            cp16(base + L::G_ + at, (const __nv_bfloat16*)b.dout + off, in);
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
            int issued = min(total, L::STAGES);
            for (; issued < total; ++issued) {
                wait(empty + issued % L::STAGES, ((issued / L::STAGES) & 1) ^ 1, guard);
                if (guard.up()) break;
                load(issued);
            }
            for (int t = 0; boxes && t < 2 && first + t * L::QR < all; ++t) mbar_wait_bounded(qfull + t, 0, kWaitNs);
            drain_ring(full, L::STAGES, issued);
        }
        __syncwarp();
        if (warp == 10 && tail < L::KB && !guard.up()) {   // keys past the end (dS is 0 there): K must be finite
            const int s = (total - 1) % L::STAGES;
            wait(full + s, ((total - 1) / L::STAGES) & 1, guard);
            for (int e = lane; e < (L::KB - tail) * (D / 8); e += 32) {
                const int row = tail + e / (D / 8), piece = e % (D / 8);
                *(uint4*)(sm + L::K_ + s * L::KTILE + (piece >> 3) * L::KPANEL + piece_at(row, piece & 7)) = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            mbar_arrive(fix);
        }
    } else if (warp >= 8) {
        const int t = warp - 8, nt = t ? n1 : n0;
        const uint32_t id_s = idesc_f16(L::QR, L::KB, false, false, a.scale < 0.f, true);
        const uint32_t id_g = idesc_f16(L::QR, L::KB, false, false, false, true);
        const uint32_t id_o = idesc_f16(L::QR, D, false, true, false, true);
        const uint32_t ts = tmem + L::S_ + t * L::BUF, tp = tmem + L::P_ + t * L::BUF, to = tmem + L::DQ_ + t * D;
        const uint64_t dq = desc_rows(base + L::Q_ + t * L::QTILE), dg = desc_rows(base + L::G_ + t * L::QTILE);
        const uint64_t dk = desc_rows(base + L::K_), dv = desc_rows(base + L::V_), dkc = desc_cols(base + L::K_, L::KPANEL);
        if (boxes && nt > 0) wait(qfull + t, 0, guard);
        for (int g = 0, it = 0, j = 0; g < total; ++g, j = j + 1 == n ? 0 : j + 1) {   // g: block of the ring, it: of this tile
            const int s = g % L::STAGES;
            if (j >= nt) {   // a block that only the other tile sees (as in the forward)
                if (lane == 0) {
                    wait(empty + s, ((g / L::STAGES) & 1) ^ 1, guard);
                    mbar_arrive(empty + s);
                }
                __syncwarp();
                continue;
            }
            wait(full + s, (g / L::STAGES) & 1, guard);
            if (it > 0) wait(done + t, (it - 1) & 1, guard);   // dS is in dP's place
            tc_fence_after();
            if (elect()) {
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
                    umma_f16(ts, step_rows(dq, x, L::QPANEL), step_rows(dk + (s * L::KTILE >> 4), x, L::KPANEL), id_s, x > 0);
                umma_commit(sfull + t);
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
                    umma_f16(tp, step_rows(dg, x, L::QPANEL), step_rows(dv + (s * L::KTILE >> 4), x, L::KPANEL), id_g, x > 0);
                umma_commit(gfull + t);
            }
            if (g == total - 1 && tail < L::KB) wait(fix, 0, guard);
            wait(dready + t, it & 1, guard);
            tc_fence_after();
            if (elect()) {
                if (g >= total - n)   // (the pass for delta has no dS)
#pragma unroll
                    for (int x = 0; x < L::KB / 16; ++x)
                        umma_f16_ts(to, tp + x * 8, step_cols(dkc + (s * L::KTILE >> 4), x), id_o, j > 0 || x > 0);
                umma_commit(empty + s);
                umma_commit(done + t);
            }
            ++it;
        }
        __syncwarp();
        drain_mma(drain + t);
    } else {
        const int t = warp >> 2, nt = t ? n1 : n0;
        const uint32_t i = first + t * L::QR + (tid & 127);
        const bool real = i < all;
        const int token = (int)(min(i, all - 1) / r);
        const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
        const uint32_t ts = tmem + L::S_ + t * L::BUF + lanes, tp = tmem + L::P_ + t * L::BUF + lanes;
        const float sl = fabsf(a.scale) * kLog2e;
        const int least = (int)(min(first + t * L::QR + (warp & 3) * 32, all - 1) / r);
        const int64_t rd = ((int64_t)hk * seqs.tokens() + t0) * r + i;
        const float nl = real ? nlse[rd] : 0.f, nd = real ? ndelta[rd] : 0.f;
        const uint64_t sl2 = pair(sl, sl), nl2 = pair(nl, nl);
        uint64_t nd2 = pair(nd, nd), sum = 0;
        for (int it = 0, j = 0; it < passes * nt; ++it, j = j + 1 == nt ? 0 : j + 1) {
            const bool last = it >= (passes - 1) * nt;
            wait(sfull + t, it & 1, guard);
            tc_fence_after();
            float p[64];
            tmem_ld64(ts, p);
#pragma unroll
            for (int x = 0; x < 64; x += 2) {
                unpair(fma2(pair(p[x], p[x + 1]), sl2, nl2), p[x], p[x + 1]);
                p[x] = ex2_approx(p[x]);
                p[x + 1] = ex2_approx(p[x + 1]);
            }
            wait(gfull + t, it & 1, guard);
            tc_fence_after();
            const bool edge = j * L::KB + L::KB - 1 > least;
            const int seen = token - j * L::KB;
            uint32_t q[32];
#pragma unroll
            for (int hlf = 0; hlf < 2; ++hlf) {
                float g[32];
                tmem_ld32(tp + hlf * 32, g);
                const uint64_t off = last ? nd2 : 0;
#pragma unroll
                for (int x = 0; x < 32; x += 2)
                    unpair(mul2(pair(p[hlf * 32 + x], p[hlf * 32 + x + 1]), add2(pair(g[x], g[x + 1]), off)), g[x], g[x + 1]);
                if (edge)
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (hlf * 32 + x > seen) g[x] = 0.f;
                if (!last)
#pragma unroll
                    for (int x = 0; x < 32; x += 2) sum = add2(sum, pair(g[x], g[x + 1]));
#pragma unroll
                for (int x = 0; x < 16; ++x) q[hlf * 16 + x] = pack_bf16(g[2 * x], g[2 * x + 1]);
            }
            if (last) {
                tmem_st32u_nowait(tp, q);
                tmem_wait_st();
            }
            tc_fence_before();
            mbar_arrive(dready + t);
            if (!last && j == nt - 1) {
                float lo, hi;
                unpair(sum, lo, hi);
                nd2 = pair(-(lo + hi), -(lo + hi));
                if (real) ndelta[rd] = -(lo + hi);
            }
        }
        if (nt > 0) {
            wait(done + t, (passes * nt - 1) & 1, guard);
            tc_fence_after();
            if (boxes && first + t * L::QR + L::QR <= all) {   // (after a timeout too, as in the forward)
                store_box<D>(tmem + L::DQ_ + t * D + lanes, a.scale, sm + L::Q_ + t * L::QTILE, &tm_dq, hk * r,
                             (int)t0 + (first + t * L::QR) / r, tid & 127, 1 + t);
            } else if (!warp_up(guard)) {
                store_rows<D>(tmem + L::DQ_ + t * D + lanes, a.scale, sm + L::Q_ + t * L::QTILE, (__nv_bfloat16*)b.dq,
                                  real ? row_at(i) : -1, tid & 127);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t backward(const AttnBwdArgs& b, const Seqs& s, float* nlse, int* status, cudaStream_t st)
{
    const AttnArgs& a = b.f;
    const int64_t T = s.tokens();
    const int r = a.H / a.Hkv;
    float* ndelta = nlse + T * a.H;
    CUtensorMap k128, v128, k64, v64, q, g, q128{}, g128{}, dq{};
    const bool boxes = box_rows(r);
    if (!make_map(&k128, a.k, T, a.Hkv, D, 64, 1, 128) || !make_map(&v128, a.v, T, a.Hkv, D, 64, 1, 128) ||
        !make_map(&k64, a.k, T, a.Hkv, D, 64, 1, 64) || !make_map(&v64, a.v, T, a.Hkv, D, 64, 1, 64) ||
        !make_map(&q, a.q, T, a.H, D, 64, r, 64 / r) || !make_map(&g, b.dout, T, a.H, D, 64, r, 64 / r) ||
        (boxes && (!make_map(&q128, a.q, T, a.H, D, 64, r, 128 / r) || !make_map(&g128, b.dout, T, a.H, D, 64, r, 128 / r) ||
                   !make_map(&dq, b.dq, T, a.H, D, 64, r, 128 / r))))
        return cudaErrorInvalidValue;
    cudaError_t e = allow_smem<attn_bwd_keys_kernel<D>>(Keys<D>::SMEM);
    if (e == cudaSuccess) e = allow_smem<attn_bwd_rows_kernel<D>>(Dq<D>::SMEM);
    if (e != cudaSuccess) return e;
    Tiles tiles;
    {
        ProfileScope prof("attn_delta", st);
        count_launch();
        constexpr int PER = 256 / (D / 8) * 4;
        attn_delta_kernel<D><<<(unsigned)((T * a.H + PER - 1) / PER), 256, 0, st>>>(a, (const __nv_bfloat16*)b.dout, nlse, ndelta, T);
    }
    {
        ProfileScope prof("attn_bwd_rows", st);
        count_launch();
        const int64_t ctas = make_tiles(tiles, s, a.Hkv, r, 256);
        attn_bwd_rows_kernel<D><<<(unsigned)ctas, 384, Dq<D>::SMEM, st>>>(k64, v64, q128, g128, dq, boxes, b, s, tiles, nlse, ndelta, status, debug_drop_handoff());
    }
    {
        ProfileScope prof("attn_bwd_keys", st);
        count_launch();
        const int64_t ctas = make_tiles(tiles, s, a.Hkv, 1, 128);
        attn_bwd_keys_kernel<D><<<(unsigned)ctas, 384, Keys<D>::SMEM, st>>>(k128, v128, q, g, b, s, tiles, nlse, ndelta, status, debug_drop_handoff());
    }
    return cudaGetLastError();
}
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
}  // namespace
}  // namespace attn

// A group of more than 64 query heads does not fit the tile of rows of the dk/dv kernel.
bool attn_tc_bwd_supported(const AttnBwdArgs& b)
{
    return attn_tc_supported(b.f) && b.f.H / b.f.Hkv <= 64 && attn::aligned16(b.dout) && attn::aligned16(b.dq) &&
           attn::aligned16(b.dk) && attn::aligned16(b.dv);
}

size_t attn_tc_bwd_workspace(int64_t tokens, int H) { return (size_t)tokens * H * 2 * sizeof(float); }

cudaError_t launch_attn_tc_bwd(const AttnBwdArgs& b, const Seqs& s, void* ws, int* status, cudaStream_t st)
{
    return b.f.D == 64 ? attn::backward<64>(b, s, (float*)ws, status, st) : attn::backward<128>(b, s, (float*)ws, status, st);
}

}  // namespace kda
