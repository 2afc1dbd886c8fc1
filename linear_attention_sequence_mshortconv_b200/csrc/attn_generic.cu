// Causal attention with grouped heads in fp32 on CUDA cores, any type and head width: the
// permanent path of fp32 tensors, of width 32 and of tensors that are not 16-byte aligned.
//   s_ij = scale q_i.k_j (j <= i), p_ij = e^{s_ij - lse_i}, o_i = sum_j p_ij v_j
//   dv_j = sum_i p_ij do_i, ds_ij = scale p_ij (do_i.v_j - do_i.o_i), dq_i = sum_j ds_ij k_j,
//   dk_j = sum_i ds_ij q_i, the sums of dk and dv running over the query heads of the group.
// One warp owns a row (a query, or a key for dk and dv) and goes over the others 32 at a
// time, one to a lane; the block's 8 rows share the staged tile.  Bound by the shared-memory reads of the staged tile.

#include "mixers.h"

namespace kda {
namespace {

constexpr int W = 8;     // rows (warps) per block
constexpr int TT = 32;   // rows of the staged tile

template <typename T, int D>
__device__ __forceinline__ void stage(float (*dst)[D + 1], const T* src, int64_t row_stride, int first, int count)
{
    for (int e = threadIdx.x; e < TT * D; e += W * 32) {
        const int r = first + e / D;
        dst[e / D][e % D] = r < count ? to_f32(src[r * row_stride + e % D]) : 0.f;
    }
}

// MODE 0: o and lse.  MODE 1: dq.
template <typename T, int D, int MODE>
__global__ void __launch_bounds__(W * 32) attn_rows_kernel(AttnArgs a, const T* dout, T* dq, const __grid_constant__ Seqs seqs)
{
    constexpr int N = D / 32;
    extern __shared__ float sm[];
    float (*K)[D + 1] = (float (*)[D + 1])sm;
    float (*V)[D + 1] = K + TT;
    float (*Q)[D + 1] = V + TT;
    float (*G)[D + 1] = Q + W;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, h = blockIdx.y, hk = h / (a.H / a.Hkv);
    int seq, tile;
    if (!seqs.locate(blockIdx.x, W, seq, tile)) return;
    const int len = seqs.len(seq), i = tile * W + w;
    const int64_t t0 = seqs.start(seq);
    const int64_t row = ((t0 + i) * a.H + h) * D;
    const int64_t ks = (int64_t)a.Hkv * D;
    const T* kp = (const T*)a.k + (t0 * a.Hkv + hk) * D;
    const T* vp = (const T*)a.v + (t0 * a.Hkv + hk) * D;
    float delta = 0.f, lse = 0.f;
    if (i < len) {
        for (int d = lane; d < D; d += 32) {
            Q[w][d] = to_f32(((const T*)a.q)[row + d]) * a.scale;
            if (MODE) {
                const float g = to_f32(dout[row + d]);
                G[w][d] = g;
                delta = fmaf(g, to_f32(((const T*)a.o)[row + d]), delta);
            }
        }
        if (MODE) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) delta += __shfl_xor_sync(~0u, delta, o);
            lse = a.lse[(t0 + i) * a.H + h];
        }
    }
    float acc[N] = {}, m = -INFINITY, z = 0.f;
    const int last = min(len, tile * W + W);   // keys the block's last row sees
    for (int j0 = 0; j0 < last; j0 += TT) {
        __syncthreads();
        stage<T, D>(K, kp, ks, j0, len);
        stage<T, D>(V, vp, ks, j0, len);
        __syncthreads();
        if (i >= len || j0 > i) continue;
        float s = 0.f;
        for (int d = 0; d < D; ++d) s = fmaf(Q[w][d], K[lane][d], s);
        const bool seen = j0 + lane <= i;
        float p;
        if (MODE == 0) {
            float top = seen ? s : -INFINITY;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            const float m2 = fmaxf(m, top), base = m2 == -INFINITY ? 0.f : m2;
            const float f = expf(m - base);
            p = seen ? expf(s - base) : 0.f;
            z = z * f + p;   // each lane sums its own keys
            m = m2;
#pragma unroll
            for (int n = 0; n < N; ++n) acc[n] *= f;
        } else {
            float gp = 0.f;
            for (int d = 0; d < D; ++d) gp = fmaf(G[w][d], V[lane][d], gp);
            p = seen ? expf(s - lse) * (gp - delta) : 0.f;
        }
        const int n_seen = min(TT, i - j0 + 1);
        for (int j = 0; j < n_seen; ++j) {
            const float pj = __shfl_sync(~0u, p, j);
#pragma unroll
            for (int n = 0; n < N; ++n) acc[n] = fmaf(pj, (MODE ? K : V)[j][n * 32 + lane], acc[n]);
        }
    }
    if (i >= len) return;
    if (MODE == 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(~0u, z, o);
        for (int n = 0; n < N; ++n) ((T*)a.o)[row + n * 32 + lane] = from_f32<T>(acc[n] / z);
        if (lane == 0 && a.lse) a.lse[(t0 + i) * a.H + h] = m + logf(z);
    } else {
        for (int n = 0; n < N; ++n) dq[row + n * 32 + lane] = from_f32<T>(acc[n] * a.scale);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(W * 32) attn_keys_kernel(AttnArgs a, const T* dout, T* dk, T* dv, const __grid_constant__ Seqs seqs)
{
    constexpr int N = D / 32;
    extern __shared__ float sm[];
    float (*Q)[D + 1] = (float (*)[D + 1])sm;
    float (*G)[D + 1] = Q + TT;
    float (*K)[D + 1] = G + TT;
    float (*V)[D + 1] = K + W;
    float* dl = (float*)(V + W);   // [2][TT]: delta, lse
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, hk = blockIdx.y, r = a.H / a.Hkv;
    int seq, tile;
    if (!seqs.locate(blockIdx.x, W, seq, tile)) return;
    const int len = seqs.len(seq), j = tile * W + w;
    const int64_t t0 = seqs.start(seq);
    const int64_t row = ((t0 + j) * a.Hkv + hk) * D, qs = (int64_t)a.H * D;
    if (j < len)
        for (int d = lane; d < D; d += 32) {
            K[w][d] = to_f32(((const T*)a.k)[row + d]) * a.scale;
            V[w][d] = to_f32(((const T*)a.v)[row + d]);
        }
    float gk[N] = {}, gv[N] = {};
    for (int h = hk * r; h < hk * r + r; ++h) {
        const int64_t base = (t0 * a.H + h) * D;
        for (int i0 = (tile * W) / TT * TT; i0 < len; i0 += TT) {
            __syncthreads();
            stage<T, D>(Q, (const T*)a.q + base, qs, i0, len);
            stage<T, D>(G, dout + base, qs, i0, len);
            for (int i = w; i < TT; i += W) {
                float x = 0.f;
                if (i0 + i < len)
                    for (int d = lane; d < D; d += 32)
                        x = fmaf(to_f32(dout[base + (i0 + i) * qs + d]), to_f32(((const T*)a.o)[base + (i0 + i) * qs + d]), x);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
                if (lane == 0) {
                    dl[i] = x;
                    dl[TT + i] = i0 + i < len ? a.lse[(t0 + i0 + i) * a.H + h] : 0.f;
                }
            }
            __syncthreads();
            if (j >= len) continue;
            float s = 0.f, gp = 0.f;
            for (int d = 0; d < D; ++d) {
                s = fmaf(K[w][d], Q[lane][d], s);
                gp = fmaf(V[w][d], G[lane][d], gp);
            }
            const bool seen = i0 + lane >= j && i0 + lane < len;
            const float p = seen ? expf(s - dl[TT + lane]) : 0.f;
            const float ds = seen ? p * (gp - dl[lane]) : 0.f;
            for (int i = max(0, j - i0); i < TT; ++i) {
                const float pi = __shfl_sync(~0u, p, i), di = __shfl_sync(~0u, ds, i);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    gv[n] = fmaf(pi, G[i][n * 32 + lane], gv[n]);
                    gk[n] = fmaf(di, Q[i][n * 32 + lane], gk[n]);
                }
            }
        }
    }
    if (j >= len) return;
    for (int n = 0; n < N; ++n) {
        dk[row + n * 32 + lane] = from_f32<T>(gk[n] * a.scale);
        dv[row + n * 32 + lane] = from_f32<T>(gv[n]);
    }
}

template <typename T, int D>
cudaError_t forward(const AttnArgs& a, const Seqs& s, cudaStream_t st)
{
    const size_t smem = (2 * TT + 2 * W) * (D + 1) * sizeof(float);
    auto kern = attn_rows_kernel<T, D, 0>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ProfileScope prof("attn_generic", st);
    count_launch();
    kern<<<dim3(s.slots(W), a.H), W * 32, smem, st>>>(a, (const T*)nullptr, (T*)nullptr, s);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t backward(const AttnBwdArgs& b, const Seqs& s, cudaStream_t st)
{
    const size_t rows = (2 * TT + 2 * W) * (D + 1) * sizeof(float), keys = rows + 2 * TT * sizeof(float);
    auto kq = attn_rows_kernel<T, D, 1>;
    auto kk = attn_keys_kernel<T, D>;
    cudaError_t e = cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)rows);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kk, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)keys);
    if (e != cudaSuccess) return e;
    ProfileScope prof("attn_bwd_generic", st);
    count_launch();
    count_launch();
    kq<<<dim3(s.slots(W), b.f.H), W * 32, rows, st>>>(b.f, (const T*)b.dout, (T*)b.dq, s);
    kk<<<dim3(s.slots(W), b.f.Hkv), W * 32, keys, st>>>(b.f, (const T*)b.dout, (T*)b.dk, (T*)b.dv, s);
    return cudaGetLastError();
}
}  // namespace

#define KDA_BY_TYPE_AND_WIDTH(fn, args, D, t, ...)                                             \
    (t == ET_F32 ? (D == 32 ? fn<float, 32>(args, __VA_ARGS__)                                 \
                    : D == 64 ? fn<float, 64>(args, __VA_ARGS__) : fn<float, 128>(args, __VA_ARGS__)) \
                 : (D == 32 ? fn<__nv_bfloat16, 32>(args, __VA_ARGS__)                         \
                    : D == 64 ? fn<__nv_bfloat16, 64>(args, __VA_ARGS__) : fn<__nv_bfloat16, 128>(args, __VA_ARGS__)))

cudaError_t launch_attn_generic(const AttnArgs& a, const Seqs& s, cudaStream_t st)
{
    return KDA_BY_TYPE_AND_WIDTH(forward, a, a.D, a.t, s, st);
}

cudaError_t launch_attn_generic_bwd(const AttnBwdArgs& b, const Seqs& s, cudaStream_t st)
{
    return KDA_BY_TYPE_AND_WIDTH(backward, b, b.f.D, b.f.t, s, st);
}

}  // namespace kda
