// Internal declarations of the gated delta rule and of causal attention (not installed).
#pragma once

#include <cuda.h>
#include <stddef.h>

#include <atomic>

#include "internal.h"

namespace kda {

// The sequences of one launch, passed by value: B rows of T tokens, or up to kMaxSeqs
// packed samples with the token offset of each.  A call with more samples is cut into
// groups of launches.  Kernel parameters instead of a device table: no copy per call, and a
// captured graph holds its own offsets.
constexpr int kMaxSeqs = 255;
struct Seqs {
    int n;                       // sequences
    int T;                       // >= 0: n rows of T tokens; < 0: cu[] holds the offsets
    int32_t cu[kMaxSeqs + 1];    // relative to the group's first token
    __host__ __device__ int start(int i) const { return T >= 0 ? i * T : cu[i]; }
    __host__ __device__ int len(int i) const { return T >= 0 ? T : cu[i + 1] - cu[i]; }
    __host__ __device__ int tokens() const { return start(n); }
    // Tiles of C tokens are numbered so that no table is needed: tile c of sequence i is
    // slot start(i) / C + i + c.  Slots never overlap (a sequence of l tokens from token s has
    // ceil(l / C) <= (s + l) / C - s / C + 1 tiles); the few left over belong to no tile.
    __host__ __device__ int slot0(int i, int C) const { return start(i) / C + i; }
    __host__ __device__ int slots(int C) const { return tokens() / C + n; }
    // sequence and tile of a slot; false if the slot holds none
    __device__ bool locate(int slot, int C, int& seq, int& tile) const
    {
        int lo = 0, hi = n - 1;   // the last sequence whose first slot is <= slot
        if (T >= 0) {
            // first slots are i * T / C + i: a guess from the mean spacing, corrected
            lo = min(hi, (int)((float)slot * (float)C / (float)(T + C)));
            while (lo > 0 && slot0(lo, C) > slot) --lo;
            while (lo < hi && slot0(lo + 1, C) <= slot) ++lo;
        } else {
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (slot0(mid, C) <= slot) lo = mid; else hi = mid - 1;
            }
        }
        seq = lo;
        tile = slot - slot0(lo, C);
        return tile * (long long)C < len(lo);
    }
};

// Tensor map of a [tokens, heads, D] bf16 tensor (16-byte aligned), box = rows tokens x box_heads heads
// x cols values.  cols = 64 lands as rows of 128 bytes whose eight 16-byte pieces are permuted by
// the row's low three bits (the 128-byte swizzle); other widths land as they are.
bool make_map(CUtensorMap* m, const void* base, int64_t tokens, int heads, int D, int cols, int box_heads, int rows);

// Lets a kernel use `bytes` of dynamic shared memory; asked of the driver once per device.
template <auto Kernel>
cudaError_t allow_smem(int bytes)
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t{1} << dev, std::memory_order_relaxed);
    return e;
}

// ---- gated delta rule ---------------------------------------------------------------
// e^g is 0 in fp32 below about -104: the clamp keeps sums of gates finite for g = -inf.  (Not by fmaxf, which
// would take a gate that is not a number for the bound: its state and all that follows are not numbers either.)
__device__ __forceinline__ float finite_gate(float g) { return g < -1000.f ? -1000.f : g; }

struct GdnArgs {
    const void *q, *k, *v, *g, *beta;   // [tokens, Hk, Dk] x 2, [tokens, Hv, Dv], [tokens, Hv] x 2
    const float* S0;                    // [sequences, Hv, Dk, Dv] or null
    void* o;
    float* ST;                          // or null
    int Hk, Hv, Dk, Dv;
    ElemType t;
};
struct GdnBwdArgs {
    GdnArgs f;                          // o and ST unused
    const void* dout;                   // [tokens, Hv, Dv]
    const float* dST;                   // or null
    void *dq, *dk, *dv, *dg, *dbeta;    // shapes and type of q, k, v, g, beta
    float* dS0;                         // or null
};
// fp32 arithmetic on CUDA cores, any type and head width
cudaError_t launch_gdn_recurrent(const GdnArgs& a, const Seqs& s, cudaStream_t st);
// tensor cores (bf16, Dk = 64 or 128, 16-byte aligned tensors)
bool gdn_tc_supported(const GdnArgs& a);
size_t gdn_tc_workspace(const GdnArgs& a, const Seqs& s, int sms);
cudaError_t launch_gdn_tc(const GdnArgs& a, const Seqs& s, void* ws, int sms, int* status, cudaStream_t st);
bool gdn_tc_bwd_supported(const GdnBwdArgs& a);
size_t gdn_tc_bwd_workspace(const Seqs& s, int Hv, int Dk, int Dv);
cudaError_t launch_gdn_tc_bwd(const GdnBwdArgs& a, const Seqs& s, void* ws, int sms, int* status, cudaStream_t st);
size_t gdn_generic_bwd_workspace(int slots16, int tokens, int Hv, int Dk, int Dv);
cudaError_t launch_gdn_generic_bwd(const GdnBwdArgs& a, const Seqs& s, void* ws, cudaStream_t st);

struct GdnStepArgs {
    const void *q, *k, *v, *g, *beta;
    float* state;                       // [n_slots, Hv, Dk, Dv]
    const int32_t* slots;               // [n] or null (request i uses slot i)
    void* o;
    int n, n_slots, Hk, Hv, Dk, Dv;
    ElemType t;
    int* status;
};
cudaError_t launch_gdn_step(const GdnStepArgs& a, cudaStream_t st);

// ---- causal attention ---------------------------------------------------------------
struct AttnArgs {
    const void *q, *k, *v;              // [tokens, H, D], [tokens, Hkv, D] x 2
    void* o;
    float* lse;                         // [tokens, H]; the forward may leave it out (null)
    int H, Hkv, D;
    float scale;
    ElemType t;
};
struct AttnBwdArgs {
    AttnArgs f;                         // o and lse are inputs here
    const void* dout;
    void *dq, *dk, *dv;
};
// tcgen05 (bf16, D = 64 or 128, 16-byte aligned tensors)
bool attn_tc_supported(const AttnArgs& a);
cudaError_t launch_attn_tc(const AttnArgs& a, const Seqs& s, int* status, cudaStream_t st);
cudaError_t launch_attn_generic(const AttnArgs& a, const Seqs& s, cudaStream_t st);
bool attn_tc_bwd_supported(const AttnBwdArgs& b);
size_t attn_tc_bwd_workspace(int64_t tokens, int H);
cudaError_t launch_attn_tc_bwd(const AttnBwdArgs& b, const Seqs& s, void* ws, int* status, cudaStream_t st);
cudaError_t launch_attn_generic_bwd(const AttnBwdArgs& a, const Seqs& s, cudaStream_t st);

}  // namespace kda
