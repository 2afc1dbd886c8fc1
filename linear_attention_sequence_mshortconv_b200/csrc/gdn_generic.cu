// The gated delta rule in fp32 on CUDA cores, for every type and head width: the recurrence
// token by token (forward), and its gradients by chunks of 16 tokens (backward).
//
//   S_t = a_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,  o_t = S_t^T q_t,  a_t = e^{g_t}
//
// These are the permanent path of fp32 tensors and of tensors that are not 16-byte aligned.

#include "mixers.h"

namespace kda {
namespace {

__device__ __forceinline__ double gate_of(float g) { return (double)finite_gate(g); }

// ---- forward: one warp per 4 value columns, 8 lanes to a column ------------------------
// A lane holds Dk / 8 entries of its column of S in registers.  Four tokens at a time: their products with the
// S before them, k_t^T S and q_t^T S, are summed over the 8 lanes together, and then go from token to
// token without S, since after token s
//   k_t^T S_s = a_s k_t^T S_{s-1} + (k_t.k_s) u_s   (and so for q_t),   u_s = beta_s (v_s - a_s k_s^T S_{s-1}).
// So only three dependent operations a token are left in the chain, and the shuffles are once in four.  Tokens
// are staged 16 to 64 at a time in shared memory, with the products k.k and q.k of each four; the next ones are
// read into registers while these are computed.  Bound by the latency of the chain, not by bytes.
constexpr int RB = 4;        // tokens at a time
constexpr int RCOLS = 16;    // value columns per CTA (4 warps)

template <typename T, int DK>
__global__ void __launch_bounds__(128) gdn_recurrent_kernel(GdnArgs a, const __grid_constant__ Seqs seqs)
{
    constexpr int NR = DK / 8;
    constexpr int RT = 2048 / DK;        // tokens per stage
    constexpr int PER = RT * DK / 128;   // staged k (and q) values per thread
    __shared__ __align__(16) float sk[RT][DK], sq[RT][DK];
    __shared__ float sv[RT][RCOLS], sa[RT], sb[RT];
    __shared__ __align__(16) float sqk[RT][RB], skk[RT][RB];   // q_t.k_s and k_t.k_s with the tokens s of t's four
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int seq = blockIdx.z, h = blockIdx.y, c0 = blockIdx.x * RCOLS;
    const int col = wid * 4 + (lane >> 3), l8 = lane & 7;
    const int len = seqs.len(seq), hk = h / (a.Hv / a.Hk);
    const int64_t t0 = seqs.start(seq);
    const T* q = (const T*)a.q;
    const T* k = (const T*)a.k;
    const T* v = (const T*)a.v;
    const T* g = (const T*)a.g;
    const T* beta = (const T*)a.beta;
    const int64_t s_off = ((int64_t)seq * a.Hv + h) * DK * a.Dv + c0 + col;

    // entry r of a lane is key channel (r / 4) * 32 + l8 * 4 + r % 4
    float S[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int i = (r >> 2) * 32 + l8 * 4 + (r & 3);
        S[r] = a.S0 ? a.S0[s_off + (int64_t)i * a.Dv] : 0.f;
    }
    float pk[PER], pq[PER], pv[RT * RCOLS / 128], pg = 0.f, pb = 0.f;
    auto fetch = [&](int base) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = j * 128 + tid, t = base + e / DK;
            const bool in = t < len;
            const int64_t off = ((t0 + t) * a.Hk + hk) * DK + e % DK;
            pk[j] = in ? to_f32(k[off]) : 0.f;
            pq[j] = in ? to_f32(q[off]) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < RT * RCOLS / 128; ++j) {
            const int e = j * 128 + tid, t = base + e / RCOLS;
            pv[j] = t < len ? to_f32(v[((t0 + t) * a.Hv + h) * a.Dv + c0 + e % RCOLS]) : 0.f;
        }
        if (tid < RT) {   // (tokens behind the sequence change nothing: alpha = 1, beta = 0)
            const bool in = base + tid < len;
            pg = in ? to_f32(g[(t0 + base + tid) * a.Hv + h]) : 0.f;
            pb = in ? to_f32(beta[(t0 + base + tid) * a.Hv + h]) : 0.f;
        }
    };
    if (len > 0) fetch(0);
    for (int base = 0; base < len; base += RT) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = j * 128 + tid;
            sk[e / DK][e % DK] = pk[j];
            sq[e / DK][e % DK] = pq[j];
        }
#pragma unroll
        for (int j = 0; j < RT * RCOLS / 128; ++j) {
            const int e = j * 128 + tid;
            sv[e / RCOLS][e % RCOLS] = pv[j];
        }
        if (tid < RT) {
            sa[tid] = expf((float)gate_of(pg));
            sb[tid] = pb;
        }
        __syncthreads();
        if (base + RT < len) fetch(base + RT);
        const int n = min(RT, len - base);
        // two threads to a pair of tokens, each with one of the products
        for (int z = tid; z < RT * 8; z += 128) {
            const int t = z >> 3, j = (z >> 1) & 3, other = (t & ~3) + j;
            const float* x = (tid & 1) ? sk[t] : sq[t];
            float s = 0.f;
#pragma unroll 4
            for (int i0 = 0; i0 < DK; i0 += 4) {
                const int i = (i0 + (tid >> 1) * 4) % DK;   // the threads of a warp in different banks
                const float4 u = *(const float4*)&x[i], w = *(const float4*)&sk[other][i];
                s = fmaf(u.x, w.x, fmaf(u.y, w.y, fmaf(u.z, w.z, fmaf(u.w, w.w, s))));
            }
            ((tid & 1) ? skk : sqk)[t][j] = s;
        }
        __syncthreads();
        for (int t = 0; t < n; t += RB) {
            float ks[RB] = {}, qs[RB] = {};
#pragma unroll
            for (int r = 0; r < NR; r += 4)
#pragma unroll
                for (int j = 0; j < RB; ++j) {
                    const float4 kv = *(const float4*)&sk[t + j][r * 8 + l8 * 4];
                    const float4 qv = *(const float4*)&sq[t + j][r * 8 + l8 * 4];
                    ks[j] = fmaf(kv.x, S[r], fmaf(kv.y, S[r + 1], fmaf(kv.z, S[r + 2], fmaf(kv.w, S[r + 3], ks[j]))));
                    qs[j] = fmaf(qv.x, S[r], fmaf(qv.y, S[r + 1], fmaf(qv.z, S[r + 2], fmaf(qv.w, S[r + 3], qs[j]))));
                }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
#pragma unroll
                for (int j = 0; j < RB; ++j) {
                    ks[j] += __shfl_xor_sync(~0u, ks[j], o);
                    qs[j] += __shfl_xor_sync(~0u, qs[j], o);
                }
            float al[RB], u[RB];
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                al[i] = sa[t + i];
                u[i] = sb[t + i] * (sv[t + i][col] - al[i] * ks[i]);
#pragma unroll
                for (int j = i; j < RB; ++j) {
                    ks[j] = fmaf(skk[t + j][i], u[i], al[i] * ks[j]);
                    qs[j] = fmaf(sqk[t + j][i], u[i], al[i] * qs[j]);
                }
            }
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const float4 kv = *(const float4*)&sk[t + i][r * 8 + l8 * 4];
                    S[r] = fmaf(kv.x, u[i], al[i] * S[r]);
                    S[r + 1] = fmaf(kv.y, u[i], al[i] * S[r + 1]);
                    S[r + 2] = fmaf(kv.z, u[i], al[i] * S[r + 2]);
                    S[r + 3] = fmaf(kv.w, u[i], al[i] * S[r + 3]);
                }
            const float out = l8 == 0 ? qs[0] : l8 == 1 ? qs[1] : l8 == 2 ? qs[2] : qs[3];   // (qs[j] is that of S_j by now)
            if (l8 < RB && t + l8 < n) ((T*)a.o)[((t0 + base + t + l8) * a.Hv + h) * a.Dv + c0 + col] = from_f32<T>(out);
        }
    }
    if (a.ST) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int i = (r >> 2) * 32 + l8 * 4 + (r & 3);
            a.ST[s_off + (int64_t)i * a.Dv] = S[r];
        }
    }
}

// ---- backward: one CTA per (sequence, value head), chunks of 16 tokens ------------------
// Chunk form, with cum the inclusive sum of g inside the chunk, K, Q, V, dO its rows, S its
// entry state and D the gradient of its exit state:
//   A = strict_lower(beta_i e^{cum_i - cum_j} k_i.k_j), T = (I + A)^-1,
//   P = lower(e^{cum_i - cum_j} q_i.k_j), R = V - e^cum o (K S), U = T (beta o R)
//   dU = P^T dO + e^{cum_C - cum} o (K D),  dY = T^T dU,  dV = beta o dY
//   dQ = e^cum o (dO S^T) + N K,            N = e^{cum_i - cum_j} o lower(dO U^T)
//   dK = rowpart + colpart: rowpart = -e^cum o (dV S^T) + M K,
//        colpart = M^T K + N^T Q + e^{cum_C - cum} o (U D^T),
//        M = -beta_i e^{cum_i - cum_j} o strict_lower(dY U^T)
//   dbeta_i = dY_i . R_i + (M K)_i . k_i / beta_i   (computed without the division)
//   dcum_i = q_i . dQ_i + k_i . rowpart_i - k_i . colpart_i, and for the last row also
//        e^{cum_C} <S, D> + sum_j e^{cum_C - cum_j} k_j . (U_j D^T);  dg = reverse sum of dcum
//   D <- e^{cum_C} D + Q^T (e^cum o dO) - K^T (e^cum o dV)
// Per value head dQ and dK go to fp32 buffers; a second kernel sums the heads of a group.
constexpr int BC = 16;


template <typename T>
__global__ void __launch_bounds__(256) gdn_generic_bwd_kernel(GdnBwdArgs b, const __grid_constant__ Seqs seqs,
                                                              float* states, float* dq_part, float* dk_part)
{
    extern __shared__ float sm[];
    const GdnArgs& a = b.f;
    const int DK = a.Dk, DV = a.Dv, tid = threadIdx.x;
    const int h = blockIdx.x, seq = blockIdx.y, hk = h / (a.Hv / a.Hk), len = seqs.len(seq);
    const int64_t t0 = seqs.start(seq);
    float* S = sm;
    float* D = S + DK * DV;
    float* k = D + DK * DV;
    float* q = k + BC * DK;
    float* x1 = q + BC * DK;       // dQ, then scratch
    float* x2 = x1 + BC * DK;      // rowpart of dK
    float* x3 = x2 + BC * DK;      // colpart of dK
    float* R = x3 + BC * DK;
    float* dO = R + BC * DV;
    float* U = dO + BC * DV;
    float* dU = U + BC * DV;
    float* dY = dU + BC * DV;
    float* KK = dY + BC * DV;      // decayed k_i . k_j (all pairs i >= j)
    float* P = KK + BC * BC;
    float* Tm = P + BC * BC;
    float* N = Tm + BC * BC;
    float* M = N + BC * BC;
    float* dec = M + BC * BC;      // e^{cum_i - cum_j}, i >= j, else 0
    float* grow = dec + BC * BC;
    float* end = grow + BC;
    float* bet = end + BC;
    float* red = bet + BC;         // [256]
    double* cum = (double*)(red + 256);

    const int nch = (len + BC - 1) / BC;
    const int64_t st0 = (int64_t)seqs.slot0(seq, BC);
    auto load = [&](int c, bool with_do) {
        __syncthreads();
        for (int e = tid; e < BC * DK; e += 256) {
            const int t = c * BC + e / DK;
            const int64_t off = ((t0 + t) * a.Hk + hk) * DK + e % DK;
            k[e] = t < len ? to_f32(((const T*)a.k)[off]) : 0.f;
            q[e] = t < len ? to_f32(((const T*)a.q)[off]) : 0.f;
        }
        for (int e = tid; e < BC * DV; e += 256) {
            const int t = c * BC + e / DV;
            const int64_t off = ((t0 + t) * a.Hv + h) * DV + e % DV;
            R[e] = t < len ? to_f32(((const T*)a.v)[off]) : 0.f;
            if (with_do) dO[e] = t < len ? to_f32(((const T*)b.dout)[off]) : 0.f;
        }
        if (tid == 0) {
            double s = 0.0;
            for (int i = 0; i < BC; ++i) {
                const int t = c * BC + i;
                if (t < len) s += gate_of(to_f32(((const T*)a.g)[(t0 + t) * a.Hv + h]));
                cum[i] = s;
                bet[i] = t < len ? to_f32(((const T*)a.beta)[(t0 + t) * a.Hv + h]) : 0.f;
            }
        }
        __syncthreads();
        {
            const int i = tid / BC, j = tid % BC;
            dec[tid] = i >= j ? expf((float)(cum[i] - cum[j])) : 0.f;
            float s = 0.f, p = 0.f;
            for (int d = 0; d < DK; ++d) {
                s = fmaf(k[i * DK + d], k[j * DK + d], s);
                p = fmaf(q[i * DK + d], k[j * DK + d], p);
            }
            KK[tid] = dec[tid] * s;
            P[tid] = dec[tid] * p;
        }
        if (tid < BC) {
            grow[tid] = expf((float)cum[tid]);
            end[tid] = expf((float)(cum[BC - 1] - cum[tid]));
        }
        __syncthreads();
        if (tid < BC) {   // T = (I + A)^-1, one column per thread
            for (int i = 0; i < BC; ++i) {
                float s = i == tid ? 1.f : 0.f;
                for (int m = tid; m < i; ++m) s = fmaf(-bet[i] * KK[i * BC + m], Tm[m * BC + tid], s);
                Tm[i * BC + tid] = i < tid ? 0.f : s;
            }
        }
        for (int e = tid; e < BC * DV; e += 256) {   // R = V - e^cum o (K S)
            const int i = e / DV, j = e % DV;
            float s = 0.f;
            for (int d = 0; d < DK; ++d) s = fmaf(k[i * DK + d], S[d * DV + j], s);
            R[e] -= grow[i] * s;
        }
        __syncthreads();
        for (int e = tid; e < BC * DV; e += 256) {   // U = T (beta o R)
            const int i = e / DV, j = e % DV;
            float s = 0.f;
            for (int m = 0; m <= i; ++m) s = fmaf(Tm[i * BC + m] * bet[m], R[m * DV + j], s);
            U[e] = s;
        }
        __syncthreads();
    };

    const int64_t sidx = ((int64_t)seq * a.Hv + h) * DK * DV;
    for (int e = tid; e < DK * DV; e += 256) S[e] = a.S0 ? a.S0[sidx + e] : 0.f;
    for (int c = 0; c < nch; ++c) {   // entry states of the chunks
        float* dst = states + ((st0 + c) * a.Hv + h) * DK * DV;
        load(c, false);
        for (int e = tid; e < DK * DV; e += 256) {
            const int i = e / DV, j = e % DV;
            dst[e] = S[e];
            float s = grow[BC - 1] * S[e];
            for (int m = 0; m < BC; ++m) s = fmaf(k[m * DK + i] * end[m], U[m * DV + j], s);
            S[e] = s;
        }
    }
    __syncthreads();
    for (int e = tid; e < DK * DV; e += 256) D[e] = b.dST ? b.dST[sidx + e] : 0.f;
    for (int c = nch - 1; c >= 0; --c) {
        const float* src = states + ((st0 + c) * a.Hv + h) * DK * DV;
        __syncthreads();
        for (int e = tid; e < DK * DV; e += 256) S[e] = src[e];
        load(c, true);
        for (int e = tid; e < BC * DV; e += 256) {   // dU = P^T dO + end o (K D)
            const int i = e / DV, j = e % DV;
            float s = 0.f, d = 0.f;
            for (int m = i; m < BC; ++m) s = fmaf(P[m * BC + i], dO[m * DV + j], s);
            for (int x = 0; x < DK; ++x) d = fmaf(k[i * DK + x], D[x * DV + j], d);
            dU[e] = fmaf(end[i], d, s);
        }
        __syncthreads();
        for (int e = tid; e < BC * DV; e += 256) {   // dY = T^T dU
            const int i = e / DV, j = e % DV;
            float s = 0.f;
            for (int m = i; m < BC; ++m) s = fmaf(Tm[m * BC + i], dU[m * DV + j], s);
            dY[e] = s;
        }
        __syncthreads();
        {
            const int i = tid / BC, j = tid % BC;
            float n = 0.f, m = 0.f;
            for (int x = 0; x < DV; ++x) {
                n = fmaf(dO[i * DV + x], U[j * DV + x], n);
                m = fmaf(dY[i * DV + x], U[j * DV + x], m);
            }
            N[tid] = dec[tid] * n;                            // dec is 0 above the diagonal
            M[tid] = i > j ? -dec[tid] * m : 0.f;             // without beta_i
        }
        __syncthreads();
        for (int e = tid; e < BC * DK; e += 256) {
            const int i = e / DK, d = e % DK;
            float s = 0.f, w = 0.f, u = 0.f, nk = 0.f, mk = 0.f, col = 0.f;
            for (int x = 0; x < DV; ++x) {
                s = fmaf(dO[i * DV + x], S[d * DV + x], s);
                w = fmaf(dY[i * DV + x], S[d * DV + x], w);
                u = fmaf(U[i * DV + x], D[d * DV + x], u);
            }
            for (int m = 0; m < BC; ++m) {
                nk = fmaf(N[i * BC + m], k[m * DK + d], nk);
                mk = fmaf(M[i * BC + m], k[m * DK + d], mk);
                col = fmaf(N[m * BC + i], q[m * DK + d], col);
                col = fmaf(bet[m] * M[m * BC + i], k[m * DK + d], col);
            }
            x1[e] = fmaf(grow[i], s, nk);
            x2[e] = bet[i] * (mk - grow[i] * w);
            x3[e] = fmaf(end[i], u, col);
            const int t = c * BC + i;
            if (t < len) {
                const int64_t off = ((t0 + t) * a.Hv + h) * DK + d;
                dq_part[off] = x1[e];
                dk_part[off] = x2[e] + x3[e];
            }
        }
        float sd = 0.f;   // <S, D> and the exit terms, summed over the block
        for (int e = tid; e < DK * DV; e += 256) sd = fmaf(S[e], D[e], sd);
        sd *= grow[BC - 1];
        for (int e = tid; e < BC * DK; e += 256) {
            const int i = e / DK, d = e % DK;
            float u = 0.f;
            for (int x = 0; x < DV; ++x) u = fmaf(U[i * DV + x], D[d * DV + x], u);
            sd = fmaf(end[i] * k[e], u, sd);
        }
        red[tid] = sd;
        __syncthreads();
        for (int w = 128; w > 0; w >>= 1) {
            if (tid < w) red[tid] += red[tid + w];
            __syncthreads();
        }
        const float exit_sum = red[0];
        __syncthreads();
        if (tid < BC) {
            float dc = 0.f, db = 0.f;
            for (int d = 0; d < DK; ++d)
                dc = fmaf(q[tid * DK + d], x1[tid * DK + d],
                          fmaf(k[tid * DK + d], x2[tid * DK + d] - x3[tid * DK + d], dc));
            for (int x = 0; x < DV; ++x) db = fmaf(dY[tid * DV + x], R[tid * DV + x], db);
            for (int m = 0; m < tid; ++m) {
                float kk = 0.f;
                for (int d = 0; d < DK; ++d) kk = fmaf(k[tid * DK + d], k[m * DK + d], kk);
                db = fmaf(M[tid * BC + m], kk, db);
            }
            red[tid] = dc + (tid == BC - 1 ? exit_sum : 0.f);
            const int t = c * BC + tid;
            if (t < len) ((T*)b.dbeta)[(t0 + t) * a.Hv + h] = from_f32<T>(db);
        }
        __syncthreads();
        if (tid == 0) {
            float s = 0.f;
            for (int i = BC - 1; i >= 0; --i) {
                s += red[i];
                const int t = c * BC + i;
                if (t < len) ((T*)b.dg)[(t0 + t) * a.Hv + h] = from_f32<T>(s);
            }
        }
        for (int e = tid; e < BC * DV; e += 256) {
            const int t = c * BC + e / DV;
            dY[e] *= bet[e / DV];
            if (t < len) ((T*)b.dv)[((t0 + t) * a.Hv + h) * DV + e % DV] = from_f32<T>(dY[e]);
        }
        __syncthreads();
        for (int e = tid; e < DK * DV; e += 256) {
            const int d = e / DV, x = e % DV;
            float s = grow[BC - 1] * D[e];
            for (int m = 0; m < BC; ++m)
                s = fmaf(grow[m], fmaf(q[m * DK + d], dO[m * DV + x], -k[m * DK + d] * dY[m * DV + x]), s);
            D[e] = s;
        }
    }
    __syncthreads();
    if (b.dS0)
        for (int e = tid; e < DK * DV; e += 256) b.dS0[sidx + e] = D[e];
}

// dq and dk: the sum over the value heads of each key head, in head order
template <typename T>
__global__ void gdn_sum_heads_kernel(const float* dq_part, const float* dk_part, T* dq, T* dk, int64_t n, int r, int Dk)
{
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = e / Dk;   // (token, key head)
        float sq = 0.f, sk = 0.f;
        for (int j = 0; j < r; ++j) {
            const int64_t off = (row * r + j) * Dk + e % Dk;
            sq += dq_part[off];
            sk += dk_part[off];
        }
        dq[e] = from_f32<T>(sq);
        dk[e] = from_f32<T>(sk);
    }
}

template <typename T>
cudaError_t recurrent(const GdnArgs& a, const Seqs& s, cudaStream_t st)
{
    const dim3 grid(a.Dv / RCOLS, a.Hv, s.n);
    ProfileScope prof("gdn_recurrent", st);
    count_launch();
    switch (a.Dk) {
        case 32: gdn_recurrent_kernel<T, 32><<<grid, 128, 0, st>>>(a, s); break;
        case 64: gdn_recurrent_kernel<T, 64><<<grid, 128, 0, st>>>(a, s); break;
        default: gdn_recurrent_kernel<T, 128><<<grid, 128, 0, st>>>(a, s); break;
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t generic_bwd(const GdnBwdArgs& a, const Seqs& s, void* ws, cudaStream_t st)
{
    const int DK = a.f.Dk, DV = a.f.Dv;
    const size_t smem = (2 * DK * DV + BC * (5 * DK + 5 * DV) + 6 * BC * BC + 3 * BC + 256) * sizeof(float) + BC * sizeof(double);
    cudaError_t e = cudaFuncSetAttribute(gdn_generic_bwd_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    float* states = (float*)ws;
    float* dqp = states + (size_t)s.slots(BC) * a.f.Hv * DK * DV;
    float* dkp = dqp + (size_t)s.tokens() * a.f.Hv * DK;
    ProfileScope prof("gdn_bwd_generic", st);
    count_launch();
    gdn_generic_bwd_kernel<T><<<dim3(a.f.Hv, s.n), 256, smem, st>>>(a, s, states, dqp, dkp);
    const int64_t n = (int64_t)s.tokens() * a.f.Hk * DK;
    if (n > 0) {
        count_launch();
        gdn_sum_heads_kernel<T><<<(int)((n + 255) / 256 < 8192 ? (n + 255) / 256 : 8192), 256, 0, st>>>(
            dqp, dkp, (T*)a.dq, (T*)a.dk, n, a.f.Hv / a.f.Hk, DK);
    }
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_gdn_recurrent(const GdnArgs& a, const Seqs& s, cudaStream_t st)
{
    return a.t == ET_F32 ? recurrent<float>(a, s, st) : recurrent<__nv_bfloat16>(a, s, st);
}

size_t gdn_generic_bwd_workspace(int slots16, int tokens, int Hv, int Dk, int Dv)
{
    return ((size_t)slots16 * Hv * Dk * Dv + 2 * (size_t)tokens * Hv * Dk) * sizeof(float);
}

cudaError_t launch_gdn_generic_bwd(const GdnBwdArgs& a, const Seqs& s, void* ws, cudaStream_t st)
{
    return a.f.t == ET_F32 ? generic_bwd<float>(a, s, ws, st) : generic_bwd<__nv_bfloat16>(a, s, ws, st);
}

}  // namespace kda
