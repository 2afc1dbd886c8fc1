// C ABI of the gated delta rule and of causal attention: argument validation, workspaces,
// groups of packed samples and dispatch.  The operations are documented in include/kda.h.

#include <cmath>

#include "mixers.h"

using namespace kda;

namespace {

kda_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }
bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
ElemType et_of(kda_dtype d) { return d == KDA_F32 ? ET_F32 : ET_BF16; }
size_t elem(ElemType t) { return t == ET_F32 ? 4 : 2; }
int num_sms()
{
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}
size_t max_of(size_t a, size_t b) { return a > b ? a : b; }

// The sequences of a call: B rows of T tokens (cu null), or n samples with host offsets.
struct Batch {
    const int32_t* cu;
    int n, T;
    int per = 0;   // rows to a group of launches (0: all of them)
    int64_t tokens() const { return cu ? (n ? cu[n] : 0) : (int64_t)n * T; }
};

kda_status check_batch(const Batch& b, bool packed)
{
    if (packed) {
        if (b.n < 0 || !b.cu || b.cu[0] != 0) return KDA_ERR_INVALID_ARG;
        for (int i = 0; i < b.n; ++i)
            if (b.cu[i + 1] < b.cu[i]) return KDA_ERR_INVALID_ARG;
    } else {
        if (b.n < 0 || b.T < 0) return KDA_ERR_INVALID_ARG;
        if (b.n > 65535) return KDA_ERR_UNSUPPORTED;
    }
    // token indexes and tile numbers are 32-bit
    if (b.tokens() > 0x7fff0000LL) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// Calls fn(seqs, first sequence, first token) for each group of launches.
template <typename F>
kda_status each_group(const Batch& b, F fn)
{
    Seqs s;
    if (!b.cu) {
        const int per = b.per ? b.per : b.n;
        for (int i = 0; i < b.n; i += per) {
            s.n = b.n - i < per ? b.n - i : per;
            s.T = b.T;
            const kda_status st = fn(s, i, (int64_t)i * b.T);
            if (st != KDA_OK) return st;
        }
        return KDA_OK;
    }
    for (int i = 0; i < b.n; i += kMaxSeqs) {
        s.n = b.n - i < kMaxSeqs ? b.n - i : kMaxSeqs;
        s.T = -1;
        for (int j = 0; j <= s.n; ++j) s.cu[j] = b.cu[i + j] - b.cu[i];
        const kda_status st = fn(s, i, b.cu[i]);
        if (st != KDA_OK) return st;
    }
    return KDA_OK;
}

Seqs rows64(const Batch& b)
{
    Seqs s;
    s.n = 64;
    s.T = b.T;
    return s;
}

// Rows shorter than a chunk of 64 tokens take the workspace of a whole one each (16 heads of 128 x 128: 0.4 MB in the
// forward, 3.8 in the backward).  So they go in groups, as packed samples do: of 4 GiB of workspace or of kMaxSeqs rows,
// and all of nearly one size.  (4096 rows of 16 tokens, 8 heads of 128 x 128: the backward took 6.21 ms with 9.8 GB, and
// takes 6.28 in three groups; of 1 GiB, nine groups, 6.59.)  need: of 64 rows.
Batch in_groups(Batch b, size_t need)
{
    if (b.cu || b.T >= 64 || b.n <= kMaxSeqs || need == 0) return b;
    const int64_t fit = (int64_t)max_of(kMaxSeqs, ((size_t)4 << 30) / need * 64), groups = (b.n + fit - 1) / fit;
    b.per = (int)((b.n + groups - 1) / groups);
    return b;
}

// The caller's workspace, or a stream-ordered allocation of `need` bytes.
struct Scratch {
    void* ptr = nullptr;
    bool owned = false;
    cudaStream_t stream = nullptr;
    kda_status acquire(void* user, size_t user_bytes, size_t need, cudaStream_t s)
    {
        stream = s;
        if (need == 0) return KDA_OK;
        if (user) {
            if (user_bytes < need) return KDA_ERR_WORKSPACE;
            if (((uintptr_t)user & 255) != 0) return KDA_ERR_INVALID_ARG;
            ptr = user;
            return KDA_OK;
        }
        if (cudaMallocAsync(&ptr, need, s) != cudaSuccess) return KDA_ERR_CUDA;
        owned = true;
        return KDA_OK;
    }
    ~Scratch() { if (owned) cudaFreeAsync(ptr, stream); }
};

template <typename T>
T* at(T* p, int64_t n) { return p ? p + n : p; }
const void* at(const void* p, int64_t n, ElemType t) { return p ? (const char*)p + n * elem(t) : p; }
void* at(void* p, int64_t n, ElemType t) { return p ? (char*)p + n * elem(t) : p; }

// ---- gated delta rule ---------------------------------------------------------------
kda_status check_gdn(int Hk, int Hv, int Dk, int Dv, kda_dtype dtype)
{
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (Hk <= 0 || Hv <= 0 || Hv % Hk != 0) return KDA_ERR_INVALID_ARG;
    if (!dim_ok(Dk) || !dim_ok(Dv) || Hv > 65535) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

GdnArgs gdn_sizes(int Hk, int Hv, int Dk, int Dv, kda_dtype dtype)
{
    GdnArgs a{};
    a.Hk = Hk; a.Hv = Hv; a.Dk = Dk; a.Dv = Dv; a.t = et_of(dtype);
    return a;
}

GdnArgs moved(GdnArgs a, int seq, int64_t token)
{
    a.q = at(a.q, token * a.Hk * a.Dk, a.t);
    a.k = at(a.k, token * a.Hk * a.Dk, a.t);
    a.v = at(a.v, token * a.Hv * a.Dv, a.t);
    a.g = at(a.g, token * a.Hv, a.t);
    a.beta = at(a.beta, token * a.Hv, a.t);
    a.o = at(a.o, token * a.Hv * a.Dv, a.t);
    a.S0 = at(a.S0, (int64_t)seq * a.Hv * a.Dk * a.Dv);
    a.ST = at(a.ST, (int64_t)seq * a.Hv * a.Dk * a.Dv);
    return a;
}

// Workspace of the tensor-core path; asked for whenever the sizes allow that path, so the
// answer does not depend on the tensors' alignment.  Cuts short rows into groups.
size_t gdn_fwd_need(const GdnArgs& a, Batch& b)
{
    GdnArgs x = a;
    x.q = x.k = x.v = x.o = nullptr;
    if (!gdn_tc_supported(x)) return 0;
    const int sms = num_sms();
    if (!b.cu) b = in_groups(b, gdn_tc_workspace(a, rows64(b), sms));
    size_t need = 0;
    each_group(b, [&](const Seqs& s, int, int64_t) {
        if (s.tokens() > 0) need = max_of(need, gdn_tc_workspace(a, s, sms));
        return KDA_OK;
    });
    return need;
}

kda_status run_gdn_forward(const GdnArgs& a, Batch b, void* workspace, size_t workspace_bytes,
                           kda_stream_t stream)
{
    if (b.n == 0) return KDA_OK;
    Scratch ws;
    const size_t need = gdn_fwd_need(a, b);
    const kda_status st = ws.acquire(workspace, workspace_bytes, need, (cudaStream_t)stream);
    if (st != KDA_OK) return st;
    const bool tc = gdn_tc_supported(a);
    const int sms = num_sms();
    int* status = tc ? device_status_ptr() : nullptr;
    if (tc && !status) return KDA_ERR_CUDA;
    return each_group(b, [&](const Seqs& s, int seq, int64_t token) {
        const GdnArgs x = moved(a, seq, token);
        return from_cuda(tc ? launch_gdn_tc(x, s, ws.ptr, sms, status, (cudaStream_t)stream)
                            : launch_gdn_recurrent(x, s, (cudaStream_t)stream));
    });
}

size_t gdn_bwd_need(const GdnArgs& a, Batch& b, bool tc)
{
    auto of = [&](const Seqs& s) {
        return tc ? gdn_tc_bwd_workspace(s, a.Hv, a.Dk, a.Dv) : gdn_generic_bwd_workspace(s.slots(16), s.tokens(), a.Hv, a.Dk, a.Dv);
    };
    if (!b.cu) b = in_groups(b, of(rows64(b)));
    size_t need = 0;
    each_group(b, [&](const Seqs& s, int, int64_t) {
        need = max_of(need, of(s));
        return KDA_OK;
    });
    return need;
}
// What is stated goes by the sizes alone; a call whose tensors are not aligned, and whose kernel then needs more,
// allocates for itself.
size_t gdn_bwd_stated(const GdnArgs& a, Batch b)
{
    GdnArgs x = a;
    x.q = x.k = x.v = x.o = nullptr;
    return gdn_bwd_need(a, b, gdn_tc_supported(x));
}

kda_status run_gdn_backward(const GdnBwdArgs& a, Batch b, void* workspace, size_t workspace_bytes,
                            kda_stream_t stream)
{
    if (b.n == 0) return KDA_OK;
    const bool tc = gdn_tc_bwd_supported(a);
    const size_t stated = gdn_bwd_stated(a.f, b), need = gdn_bwd_need(a.f, b, tc);
    Scratch ws;
    kda_status st = ws.acquire(workspace, workspace_bytes, workspace ? stated : need, (cudaStream_t)stream);
    if (st == KDA_OK && workspace && need > stated) st = ws.acquire(nullptr, 0, need, (cudaStream_t)stream);
    if (st != KDA_OK) return st;
    const int sms = num_sms();
    int* status = tc ? device_status_ptr() : nullptr;
    if (tc && !status) return KDA_ERR_CUDA;
    return each_group(b, [&](const Seqs& s, int seq, int64_t token) {
        GdnBwdArgs x = a;
        x.f = moved(a.f, seq, token);
        x.dout = at(a.dout, token * a.f.Hv * a.f.Dv, a.f.t);
        x.dST = at(a.dST, (int64_t)seq * a.f.Hv * a.f.Dk * a.f.Dv);
        x.dS0 = at(a.dS0, (int64_t)seq * a.f.Hv * a.f.Dk * a.f.Dv);
        x.dq = at(a.dq, token * a.f.Hk * a.f.Dk, a.f.t);
        x.dk = at(a.dk, token * a.f.Hk * a.f.Dk, a.f.t);
        x.dv = at(a.dv, token * a.f.Hv * a.f.Dv, a.f.t);
        x.dg = at(a.dg, token * a.f.Hv, a.f.t);
        x.dbeta = at(a.dbeta, token * a.f.Hv, a.f.t);
        return from_cuda(tc ? launch_gdn_tc_bwd(x, s, ws.ptr, sms, status, (cudaStream_t)stream)
                            : launch_gdn_generic_bwd(x, s, ws.ptr, (cudaStream_t)stream));
    });
}

kda_status gdn_forward_any(GdnArgs a, const Batch& b, bool packed, kda_dtype dtype, void* workspace,
                           size_t workspace_bytes, kda_stream_t stream)
{
    kda_status st = check_batch(b, packed);
    if (st == KDA_OK) st = check_gdn(a.Hk, a.Hv, a.Dk, a.Dv, dtype);
    if (st != KDA_OK) return st;
    if (b.tokens() > 0 && (!a.q || !a.k || !a.v || !a.g || !a.beta || !a.o)) return KDA_ERR_INVALID_ARG;
    a.t = et_of(dtype);
    return run_gdn_forward(a, b, workspace, workspace_bytes, stream);
}

kda_status gdn_backward_any(GdnBwdArgs a, const Batch& b, bool packed, kda_dtype dtype, void* workspace,
                            size_t workspace_bytes, kda_stream_t stream)
{
    kda_status st = check_batch(b, packed);
    if (st == KDA_OK) st = check_gdn(a.f.Hk, a.f.Hv, a.f.Dk, a.f.Dv, dtype);
    if (st != KDA_OK) return st;
    if (b.tokens() > 0 && (!a.f.q || !a.f.k || !a.f.v || !a.f.g || !a.f.beta || !a.dout || !a.dq || !a.dk || !a.dv ||
                           !a.dg || !a.dbeta))
        return KDA_ERR_INVALID_ARG;
    a.f.t = et_of(dtype);
    return run_gdn_backward(a, b, workspace, workspace_bytes, stream);
}

// ---- attention ----------------------------------------------------------------------
kda_status check_attn(int H, int Hkv, int D, float scale, kda_dtype dtype)
{
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (H <= 0 || Hkv <= 0 || H % Hkv != 0 || !std::isfinite(scale)) return KDA_ERR_INVALID_ARG;
    if (!dim_ok(D) || H > 65535) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

AttnArgs moved(AttnArgs a, int64_t token)
{
    a.q = at(a.q, token * a.H * a.D, a.t);
    a.k = at(a.k, token * a.Hkv * a.D, a.t);
    a.v = at(a.v, token * a.Hkv * a.D, a.t);
    a.o = at(a.o, token * a.H * a.D, a.t);
    a.lse = at(a.lse, token * a.H);
    return a;
}

kda_status attn_forward_any(AttnArgs a, const Batch& b, bool packed, kda_dtype dtype, kda_stream_t stream)
{
    kda_status st = check_batch(b, packed);
    if (st == KDA_OK) st = check_attn(a.H, a.Hkv, a.D, a.scale, dtype);
    if (st != KDA_OK) return st;
    if (b.tokens() == 0) return KDA_OK;
    if (!a.q || !a.k || !a.v || !a.o) return KDA_ERR_INVALID_ARG;
    a.t = et_of(dtype);
    const bool tc = attn_tc_supported(a);
    int* status = tc ? device_status_ptr() : nullptr;
    if (tc && !status) return KDA_ERR_CUDA;
    return each_group(b, [&](const Seqs& s, int, int64_t token) {
        if (s.tokens() == 0) return KDA_OK;
        const AttnArgs x = moved(a, token);
        return from_cuda(tc ? launch_attn_tc(x, s, status, (cudaStream_t)stream) : launch_attn_generic(x, s, (cudaStream_t)stream));
    });
}

size_t attn_bwd_need(int64_t tokens, int H, int D, kda_dtype dtype)
{
    return dtype == KDA_BF16 && D != 32 ? attn_tc_bwd_workspace(tokens, H) : 0;
}

kda_status attn_backward_any(AttnBwdArgs a, const Batch& b, bool packed, kda_dtype dtype, void* workspace,
                             size_t workspace_bytes, kda_stream_t stream)
{
    kda_status st = check_batch(b, packed);
    if (st == KDA_OK) st = check_attn(a.f.H, a.f.Hkv, a.f.D, a.f.scale, dtype);
    if (st != KDA_OK) return st;
    if (b.tokens() == 0) return KDA_OK;
    if (!a.f.q || !a.f.k || !a.f.v || !a.f.o || !a.f.lse || !a.dout || !a.dq || !a.dk || !a.dv)
        return KDA_ERR_INVALID_ARG;
    a.f.t = et_of(dtype);
    Scratch ws;
    st = ws.acquire(workspace, workspace_bytes, attn_bwd_need(b.tokens(), a.f.H, a.f.D, dtype), (cudaStream_t)stream);
    if (st != KDA_OK) return st;
    const bool tc = attn_tc_bwd_supported(a);
    int* status = tc ? device_status_ptr() : nullptr;
    if (tc && !status) return KDA_ERR_CUDA;
    return each_group(b, [&](const Seqs& s, int, int64_t token) {
        if (s.tokens() == 0) return KDA_OK;
        AttnBwdArgs x = a;
        x.f = moved(a.f, token);
        x.dout = at(a.dout, token * a.f.H * a.f.D, a.f.t);
        x.dq = at(a.dq, token * a.f.H * a.f.D, a.f.t);
        x.dk = at(a.dk, token * a.f.Hkv * a.f.D, a.f.t);
        x.dv = at(a.dv, token * a.f.Hkv * a.f.D, a.f.t);
        return from_cuda(tc ? launch_attn_tc_bwd(x, s, ws.ptr, status, (cudaStream_t)stream)
                            : launch_attn_generic_bwd(x, s, (cudaStream_t)stream));
    });
}

}  // namespace

extern "C" {

size_t gdn_forward_workspace_size(int B, int T, int Hk, int Hv, int Dk, int Dv, kda_dtype dtype)
{
    Batch b{nullptr, B, T};
    if (check_batch(b, false) != KDA_OK || check_gdn(Hk, Hv, Dk, Dv, dtype) != KDA_OK) return 0;
    return gdn_fwd_need(gdn_sizes(Hk, Hv, Dk, Dv, dtype), b);
}

size_t gdn_forward_varlen_workspace_size(const int32_t* cu_seqlens, int n_seqs, int Hk, int Hv, int Dk, int Dv,
                                         kda_dtype dtype)
{
    Batch b{cu_seqlens, n_seqs, 0};
    if (check_batch(b, true) != KDA_OK || check_gdn(Hk, Hv, Dk, Dv, dtype) != KDA_OK) return 0;
    return gdn_fwd_need(gdn_sizes(Hk, Hv, Dk, Dv, dtype), b);
}

kda_status gdn_forward(const void* q, const void* k, const void* v, const void* g, const void* beta, const float* S0,
                       void* o, float* S_T, int B, int T, int Hk, int Hv, int Dk, int Dv, kda_dtype dtype,
                       void* workspace, size_t workspace_bytes, kda_stream_t stream)
{
    const GdnArgs a{q, k, v, g, beta, S0, o, S_T, Hk, Hv, Dk, Dv, ET_F32};
    return gdn_forward_any(a, Batch{nullptr, B, T}, false, dtype, workspace, workspace_bytes, stream);
}

kda_status gdn_forward_varlen(const void* q, const void* k, const void* v, const void* g, const void* beta,
                              const float* S0, void* o, float* S_T, const int32_t* cu_seqlens, int n_seqs, int Hk,
                              int Hv, int Dk, int Dv, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                              kda_stream_t stream)
{
    const GdnArgs a{q, k, v, g, beta, S0, o, S_T, Hk, Hv, Dk, Dv, ET_F32};
    return gdn_forward_any(a, Batch{cu_seqlens, n_seqs, 0}, true, dtype, workspace, workspace_bytes, stream);
}

size_t gdn_backward_workspace_size(int B, int T, int Hk, int Hv, int Dk, int Dv, kda_dtype dtype)
{
    Batch b{nullptr, B, T};
    if (check_batch(b, false) != KDA_OK || check_gdn(Hk, Hv, Dk, Dv, dtype) != KDA_OK) return 0;
    return gdn_bwd_stated(gdn_sizes(Hk, Hv, Dk, Dv, dtype), b);
}

size_t gdn_backward_varlen_workspace_size(const int32_t* cu_seqlens, int n_seqs, int Hk, int Hv, int Dk, int Dv,
                                          kda_dtype dtype)
{
    Batch b{cu_seqlens, n_seqs, 0};
    if (check_batch(b, true) != KDA_OK || check_gdn(Hk, Hv, Dk, Dv, dtype) != KDA_OK) return 0;
    return gdn_bwd_stated(gdn_sizes(Hk, Hv, Dk, Dv, dtype), b);
}

kda_status gdn_backward(const void* q, const void* k, const void* v, const void* g, const void* beta, const float* S0,
                        const void* d_o, const float* dS_T, void* dq, void* dk, void* dv, void* dg, void* dbeta,
                        float* dS0, int B, int T, int Hk, int Hv, int Dk, int Dv, kda_dtype dtype, void* workspace,
                        size_t workspace_bytes, kda_stream_t stream)
{
    const GdnArgs f{q, k, v, g, beta, S0, nullptr, nullptr, Hk, Hv, Dk, Dv, ET_F32};
    return gdn_backward_any(GdnBwdArgs{f, d_o, dS_T, dq, dk, dv, dg, dbeta, dS0}, Batch{nullptr, B, T}, false, dtype,
                            workspace, workspace_bytes, stream);
}

kda_status gdn_backward_varlen(const void* q, const void* k, const void* v, const void* g, const void* beta,
                               const float* S0, const void* d_o, const float* dS_T, void* dq, void* dk, void* dv,
                               void* dg, void* dbeta, float* dS0, const int32_t* cu_seqlens, int n_seqs, int Hk,
                               int Hv, int Dk, int Dv, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                               kda_stream_t stream)
{
    const GdnArgs f{q, k, v, g, beta, S0, nullptr, nullptr, Hk, Hv, Dk, Dv, ET_F32};
    return gdn_backward_any(GdnBwdArgs{f, d_o, dS_T, dq, dk, dv, dg, dbeta, dS0}, Batch{cu_seqlens, n_seqs, 0}, true,
                            dtype, workspace, workspace_bytes, stream);
}

kda_status gdn_step(const void* q, const void* k, const void* v, const void* g, const void* beta, float* state,
                    const int32_t* slots, void* o, int n, int n_slots, int Hk, int Hv, int Dk, int Dv,
                    kda_dtype dtype, kda_stream_t stream)
{
    if (n < 0 || n_slots < 0) return KDA_ERR_INVALID_ARG;
    if (n > 65535) return KDA_ERR_UNSUPPORTED;
    const kda_status st = check_gdn(Hk, Hv, Dk, Dv, dtype);
    if (st != KDA_OK) return st;
    if (n == 0) return KDA_OK;
    if (!q || !k || !v || !g || !beta || !o || (!state && n_slots > 0)) return KDA_ERR_INVALID_ARG;
    if (!slots && n > n_slots) return KDA_ERR_INVALID_ARG;
    if (((uintptr_t)state & 15) != 0) return KDA_ERR_INVALID_ARG;
    int* status = device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    const GdnStepArgs a{q, k, v, g, beta, state, slots, o, n, n_slots, Hk, Hv, Dk, Dv, et_of(dtype), status};
    return from_cuda(launch_gdn_step(a, (cudaStream_t)stream));
}

kda_status attn_forward(const void* q, const void* k, const void* v, void* o, float* lse, int B, int T, int H, int Hkv,
                        int D, float scale, kda_dtype dtype, kda_stream_t stream)
{
    return attn_forward_any(AttnArgs{q, k, v, o, lse, H, Hkv, D, scale, ET_F32}, Batch{nullptr, B, T}, false, dtype,
                            stream);
}

kda_status attn_forward_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                               const int32_t* cu_seqlens, int n_seqs, int H, int Hkv, int D, float scale,
                               kda_dtype dtype, kda_stream_t stream)
{
    return attn_forward_any(AttnArgs{q, k, v, o, lse, H, Hkv, D, scale, ET_F32}, Batch{cu_seqlens, n_seqs, 0}, true,
                            dtype, stream);
}

size_t attn_backward_workspace_size(int64_t tokens, int H, int Hkv, int D, kda_dtype dtype)
{
    if (tokens < 0 || check_attn(H, Hkv, D, 1.f, dtype) != KDA_OK) return 0;
    return attn_bwd_need(tokens, H, D, dtype);
}

kda_status attn_backward(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* d_o,
                         void* dq, void* dk, void* dv, int B, int T, int H, int Hkv, int D, float scale,
                         kda_dtype dtype, void* workspace, size_t workspace_bytes, kda_stream_t stream)
{
    const AttnArgs f{q, k, v, (void*)o, (float*)lse, H, Hkv, D, scale, ET_F32};
    return attn_backward_any(AttnBwdArgs{f, d_o, dq, dk, dv}, Batch{nullptr, B, T}, false, dtype, workspace,
                             workspace_bytes, stream);
}

kda_status attn_backward_varlen(const void* q, const void* k, const void* v, const void* o, const float* lse,
                                const void* d_o, void* dq, void* dk, void* dv, const int32_t* cu_seqlens, int n_seqs,
                                int H, int Hkv, int D, float scale, kda_dtype dtype, void* workspace,
                                size_t workspace_bytes, kda_stream_t stream)
{
    const AttnArgs f{q, k, v, (void*)o, (float*)lse, H, Hkv, D, scale, ET_F32};
    return attn_backward_any(AttnBwdArgs{f, d_o, dq, dk, dv}, Batch{cu_seqlens, n_seqs, 0}, true, dtype, workspace,
                             workspace_bytes, stream);
}

}  // extern "C"
