// One token of the gated delta rule per request (serving), on states kept in a pool:
//   u = beta (v - a k^T S),  S' = a S + k u^T,  o = a q^T S + (q.k) u,   a = e^g.
// o needs only the old S, so one pass over the state feeds both sums, and the state is read
// once and written once: 8 bytes for 7 operations an entry, bound by HBM.
//
// A CTA owns 32 value columns of one (request, value head): 128-byte rows of the state,
// loaded as float4 by 8 lanes, Dk / 32 of them held in registers by each of 256 threads
// between the sums and the update.  16 KB a CTA and 8 CTAs an SM keep 128 KB in flight per
// SM; one request alone still spreads over Dv / 32 CTAs per head.  (256 requests, 32 heads, 128 x 128: 194 to 204 us,
// 5.3 to 5.5 TB/s or 81 to 85% of a copy's rate; one request of 16 heads: 4.6 us, a launch's latency.)

#include "mixers.h"

namespace kda {
namespace {

constexpr int SC = 32;   // value columns per CTA

template <typename T, int DK>
__global__ void __launch_bounds__(256) gdn_step_kernel(GdnStepArgs a)
{
    constexpr int NR = DK / 32;
    __shared__ float sq[DK], sk[DK];
    __shared__ float4 pk[8][8], pq[8][8];
    __shared__ float sqk;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int c0 = blockIdx.x * SC, h = blockIdx.y, req = blockIdx.z;
    const int hk = h / (a.Hv / a.Hk);
    const int c4 = tid & 7, row = tid >> 3;   // float4 column, first state row
    const int64_t vo = ((int64_t)req * a.Hv + h) * a.Dv + c0;
    const int slot = a.slots ? a.slots[req] : req;
    if (slot < 0 || slot >= a.n_slots) {   // a padding request, or a slot outside the pool
        if (tid < SC) ((T*)a.o)[vo + tid] = from_f32<T>(0.f);
        if (slot >= 0 && tid == 0) atomicCAS(a.status, DEV_OK, DEV_SLOT);
        return;
    }
    float4* S = (float4*)(a.state + (((int64_t)slot * a.Hv + h) * DK + row) * a.Dv + c0) + c4;
    const int64_t step = (int64_t)32 * a.Dv / 4;
    float4 s[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) s[r] = __ldcs(S + r * step);
    // A slot named twice would be updated by two CTAs at once: the first request has it.  (Every CTA reads the slots
    // before its own, quadratic in the requests: with states of 32 x 32, one head, it costs 14.1 us against 12.8 without
    // slots at 256 requests, 17.4 against 14.6 at 4096, 68 against 45 at 16384; with 16 heads 202 against 172 at 4096.)
    bool taken = false;
    if (a.slots)
        for (int i = tid; i < req; i += 256) taken |= a.slots[i] == slot;
    if (tid < DK) {
        const int64_t off = ((int64_t)req * a.Hk + hk) * DK + tid;
        sq[tid] = to_f32(((const T*)a.q)[off]);
        sk[tid] = to_f32(((const T*)a.k)[off]);
    }
    const float al = expf(to_f32(((const T*)a.g)[(int64_t)req * a.Hv + h]));
    const float be = to_f32(((const T*)a.beta)[(int64_t)req * a.Hv + h]);
    float4 v4;
    {
        const T* v = (const T*)a.v + vo + c4 * 4;
        v4 = make_float4(to_f32(v[0]), to_f32(v[1]), to_f32(v[2]), to_f32(v[3]));
    }
    if (__syncthreads_or(taken)) {
        if (tid < SC) ((T*)a.o)[vo + tid] = from_f32<T>(0.f);
        if (tid == 0) atomicCAS(a.status, DEV_OK, DEV_SLOT);
        return;
    }
    float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), qs = ks;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const float kr = sk[row + 32 * r], qr = sq[row + 32 * r];
        ks.x = fmaf(kr, s[r].x, ks.x); ks.y = fmaf(kr, s[r].y, ks.y);
        ks.z = fmaf(kr, s[r].z, ks.z); ks.w = fmaf(kr, s[r].w, ks.w);
        qs.x = fmaf(qr, s[r].x, qs.x); qs.y = fmaf(qr, s[r].y, qs.y);
        qs.z = fmaf(qr, s[r].z, qs.z); qs.w = fmaf(qr, s[r].w, qs.w);
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {   // over the warp's 4 rows
        ks.x += __shfl_xor_sync(~0u, ks.x, o); ks.y += __shfl_xor_sync(~0u, ks.y, o);
        ks.z += __shfl_xor_sync(~0u, ks.z, o); ks.w += __shfl_xor_sync(~0u, ks.w, o);
        qs.x += __shfl_xor_sync(~0u, qs.x, o); qs.y += __shfl_xor_sync(~0u, qs.y, o);
        qs.z += __shfl_xor_sync(~0u, qs.z, o); qs.w += __shfl_xor_sync(~0u, qs.w, o);
    }
    if (lane < 8) {
        pk[wid][lane] = ks;
        pq[wid][lane] = qs;
    }
    if (wid == 0) {
        float x = 0.f;
        for (int i = lane; i < DK; i += 32) x = fmaf(sq[i], sk[i], x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
        if (lane == 0) sqk = x;
    }
    __syncthreads();
    ks = pk[0][c4];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
        const float4 x = pk[w][c4];
        ks.x += x.x; ks.y += x.y; ks.z += x.z; ks.w += x.w;
    }
    const float4 u = make_float4(be * (v4.x - al * ks.x), be * (v4.y - al * ks.y), be * (v4.z - al * ks.z),
                                 be * (v4.w - al * ks.w));
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const float kr = sk[row + 32 * r];
        __stcs(S + r * step, make_float4(fmaf(kr, u.x, al * s[r].x), fmaf(kr, u.y, al * s[r].y),
                                         fmaf(kr, u.z, al * s[r].z), fmaf(kr, u.w, al * s[r].w)));
    }
    if (tid < 8) {
        qs = pq[0][c4];
#pragma unroll
        for (int w = 1; w < 8; ++w) {
            const float4 x = pq[w][c4];
            qs.x += x.x; qs.y += x.y; qs.z += x.z; qs.w += x.w;
        }
        T* o = (T*)a.o + vo + c4 * 4;
        o[0] = from_f32<T>(fmaf(sqk, u.x, al * qs.x));
        o[1] = from_f32<T>(fmaf(sqk, u.y, al * qs.y));
        o[2] = from_f32<T>(fmaf(sqk, u.z, al * qs.z));
        o[3] = from_f32<T>(fmaf(sqk, u.w, al * qs.w));
    }
}

template <typename T>
cudaError_t step(const GdnStepArgs& a, cudaStream_t st)
{
    const dim3 grid(a.Dv / SC, a.Hv, a.n);
    ProfileScope prof("gdn_step", st);
    count_launch();
    switch (a.Dk) {
        case 32: gdn_step_kernel<T, 32><<<grid, 256, 0, st>>>(a); break;
        case 64: gdn_step_kernel<T, 64><<<grid, 256, 0, st>>>(a); break;
        default: gdn_step_kernel<T, 128><<<grid, 256, 0, st>>>(a); break;
    }
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_gdn_step(const GdnStepArgs& a, cudaStream_t st)
{
    return a.t == ET_F32 ? step<float>(a, st) : step<__nv_bfloat16>(a, st);
}

}  // namespace kda
