// lin_abi.cpp -- the extern "C" boundary of linear attention with a decay per head:
// argument checks and workspace sizing. The contract is in include/kda.h.
#include "../../include/kda.h"

#include <climits>

#include "kda_launch.h"

using kda::Dt;

namespace {

bool dtype_ok(int d) { return d == KDA_F32 || d == KDA_BF16; }
bool width_ok(int D) { return D == 64 || D == 128; }
bool gate_ok(int gate) { return gate == KDA_GATE_HEAD || gate == KDA_GATE_FIXED; }
bool misaligned(const void *p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

// Whether an output is one of the n buffers.
bool among(const void *out, const void *const *buffers, int n) {
    for (int i = 0; out && i < n; ++i)
        if (out == buffers[i]) return true;
    return false;
}

// Sizes of a chunked call: 0, or the status it is refused with.
int check_sizes(int N, int B, int T, int H, int Hk, int Dk, int Dv, const int32_t *cu, int gate) {
    if (N < 1 || B < 1 || T < 0 || H < 1 || Hk < 1 || H % Hk != 0 || Dk < 1 || Dv < 1) return KDA_ERR_INVALID_ARG;
    if (!gate_ok(gate) || (cu ? B != 1 : N != B)) return KDA_ERR_INVALID_ARG;
    if ((long long)B * T > INT_MAX / 2 || (long long)N * H > INT_MAX / 2) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t lin_prefill_workspace_size(int N, int T_total, int H, int Dk, int Dv) {
    if (N < 1 || T_total < 0 || H < 1 || !width_ok(Dk) || !width_ok(Dv) || T_total > INT_MAX / 2) return 0;
    if (!kda::lin_chunk_fits(N, T_total, H)) return 0;
    return kda::lin_prefill_workspace(N, T_total, H, Dk, Dv);
}

int lin_prefill(const void *q, const void *k, const void *v, const float *g, const float *S0, void *out, float *S_out,
                const int32_t *cu_seqlens, int N, int B, int T, int H, int Hk, int Dk, int Dv, kda_dtype io_dtype,
                kda_dtype out_dtype, int gate, int zero_rows, void *workspace, size_t workspace_bytes, void *stream) {
    const int bad = check_sizes(N, B, T, H, Hk, Dk, Dv, cu_seqlens, gate);
    if (bad != KDA_OK) return bad;
    if (!dtype_ok(io_dtype) || !dtype_ok(out_dtype) || (zero_rows != 0 && zero_rows != 1)) return KDA_ERR_INVALID_ARG;
    const long long T_total = (long long)B * T;
    if (T_total > 0 && (!q || !k || !v || !out)) return KDA_ERR_INVALID_ARG;
    const void *vectors[] = {q, k, v, out, S0, S_out};
    for (const void *x : vectors)
        if (misaligned(x, 15)) return KDA_ERR_INVALID_ARG;
    if (misaligned(g, 3)) return KDA_ERR_INVALID_ARG;
    const void *ins[] = {q, k, v, g, S0, S_out};
    if (among(out, ins, 6) || among(S_out, ins, 4)) return KDA_ERR_INVALID_ARG;
    if (!width_ok(Dk) || !width_ok(Dv) || (io_dtype == KDA_F32 && out_dtype != KDA_F32)) return KDA_ERR_UNSUPPORTED;
    if (!kda::lin_chunk_fits(N, T_total, H)) return KDA_ERR_UNSUPPORTED;
    const size_t need = kda::lin_prefill_workspace(N, T_total, H, Dk, Dv);
    if ((need > 0 && (!workspace || workspace_bytes < need)) || misaligned(workspace, 255)) return KDA_ERR_WORKSPACE;
    kda::LinPrefillArgs a;
    a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0; a.out = out; a.S_out = S_out; a.cu_seqlens = cu_seqlens;
    a.N = N; a.B = B; a.T = T; a.H = H; a.Hk = Hk; a.Dk = Dk; a.Dv = Dv;
    a.io = static_cast<Dt>(io_dtype); a.out_dt = static_cast<Dt>(out_dtype);
    a.fixed = gate == KDA_GATE_FIXED;
    a.zero_rows = zero_rows != 0;
    a.ws = workspace;
    a.stream = static_cast<hipStream_t>(stream);
    return kda::launch_lin_prefill(a) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t lin_prefill_backward_workspace_size(int N, int T_total, int H, int Hk, int Dk, int Dv) {
    if (N < 1 || T_total < 0 || H < 1 || Hk < 1 || H % Hk != 0 || !width_ok(Dk) || !width_ok(Dv)) return 0;
    if (T_total > INT_MAX / 2 || !kda::lin_chunk_fits(N, T_total, H)) return 0;
    return kda::lin_backward_workspace(N, T_total, H, Hk, Dk, Dv);
}

int lin_prefill_backward(const void *q, const void *k, const void *v, const float *g, const void *dout, const float *S0,
                         const float *dS_out, void *dq, void *dk, void *dv, float *dg, float *dS0,
                         const int32_t *cu_seqlens, int N, int B, int T, int H, int Hk, int Dk, int Dv,
                         kda_dtype io_dtype, int gate, int zero_rows, void *workspace, size_t workspace_bytes,
                         void *stream) {
    const int bad = check_sizes(N, B, T, H, Hk, Dk, Dv, cu_seqlens, gate);
    if (bad != KDA_OK) return bad;
    if (!dtype_ok(io_dtype) || (zero_rows & ~(KDA_ZERO_DQ | KDA_ZERO_DK | KDA_ZERO_DV | KDA_ZERO_DG))) return KDA_ERR_INVALID_ARG;
    const long long T_total = (long long)B * T;
    if (T_total > 0 && (!q || !k || !v || !dout || !dq || !dk || !dv)) return KDA_ERR_INVALID_ARG;
    if (!g != !dg && (T_total > 0 || gate == KDA_GATE_FIXED)) return KDA_ERR_INVALID_ARG;    // a gate has a gradient, no gate has none
    const void *vectors[] = {q, k, v, dout, dq, dk, dv, S0, dS_out, dS0};
    for (const void *x : vectors)
        if (misaligned(x, 15)) return KDA_ERR_INVALID_ARG;
    if (misaligned(g, 3) || misaligned(dg, 3)) return KDA_ERR_INVALID_ARG;
    // every gradient is a buffer of its own: other workgroups still read the inputs
    const void *all[] = {q, k, v, g, dout, S0, dS_out, dq, dk, dv, dg, dS0};
    for (int i = 7; i < 12; ++i)
        if (among(all[i], all, i)) return KDA_ERR_INVALID_ARG;
    if (!width_ok(Dk) || !width_ok(Dv) || !kda::lin_chunk_fits(N, T_total, H)) return KDA_ERR_UNSUPPORTED;
    const size_t need = kda::lin_backward_workspace(N, T_total, H, Hk, Dk, Dv);
    if ((need > 0 && (!workspace || workspace_bytes < need)) || misaligned(workspace, 255)) return KDA_ERR_WORKSPACE;
    kda::LinBackwardArgs a;
    a.q = q; a.k = k; a.v = v; a.g = g; a.dout = dout; a.S0 = S0; a.dS_out = dS_out;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dS0 = dS0; a.cu_seqlens = cu_seqlens;
    a.N = N; a.B = B; a.T = T; a.H = H; a.Hk = Hk; a.Dk = Dk; a.Dv = Dv;
    a.io = static_cast<Dt>(io_dtype);
    a.fixed = gate == KDA_GATE_FIXED;
    a.zero_rows = zero_rows;
    a.ws = workspace;
    a.stream = static_cast<hipStream_t>(stream);
    return kda::launch_lin_backward(a) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"

namespace {

int recurrent_impl(const void *q, const void *k, const void *v, const float *g, float *S, void *out, const int32_t *cu,
                   const int32_t *slot_in, const int32_t *slot_out, int N, int T, int H, int Hk, int Dk, int Dv, int slots,
                   kda_dtype io_dtype, kda_dtype out_dtype, int gate, int zero_rows, void *stream) {
    if (N < 1 || T < 0 || H < 1 || Hk < 1 || H % Hk != 0 || Dk < 1 || Dv < 1 || slots < 1) return KDA_ERR_INVALID_ARG;
    if (!gate_ok(gate) || (zero_rows != 0 && zero_rows != 1)) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(io_dtype) || !dtype_ok(out_dtype) || T > INT_MAX / 2 || !S) return KDA_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !out)) return KDA_ERR_INVALID_ARG;
    const void *vectors[] = {q, k, v, S, out};
    for (const void *x : vectors)
        if (misaligned(x, 15)) return KDA_ERR_INVALID_ARG;
    if (misaligned(g, 3)) return KDA_ERR_INVALID_ARG;
    const void *ins[] = {q, k, v, g, S};
    if (among(out, ins, 5) || among(S, ins, 4)) return KDA_ERR_INVALID_ARG;
    if (!width_ok(Dk) || !width_ok(Dv) || !kda::lin_recurrent_fits(N, H, Dk, Dv)) return KDA_ERR_UNSUPPORTED;
    if (T == 0) return KDA_OK;
    kda::LinRecurrentArgs a;
    a.q = q; a.k = k; a.v = v; a.g = g; a.S = S; a.out = out; a.cu = cu; a.slot_in = slot_in; a.slot_out = slot_out;
    a.N = N; a.T = T; a.H = H; a.Hk = Hk; a.Dk = Dk; a.Dv = Dv; a.slots = slots;
    a.io = static_cast<Dt>(io_dtype); a.out_dt = static_cast<Dt>(out_dtype);
    a.fixed = gate == KDA_GATE_FIXED;
    a.zero_rows = zero_rows != 0;
    a.stream = static_cast<hipStream_t>(stream);
    return kda::launch_lin_recurrent(a) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // namespace

extern "C" {

int lin_decode(const void *q, const void *k, const void *v, const float *g, float *S, void *out, int N, int H, int Hk,
               int Dk, int Dv, kda_dtype io_dtype, kda_dtype out_dtype, int gate, void *stream) {
    return recurrent_impl(q, k, v, g, S, out, nullptr, nullptr, nullptr, N, N, H, Hk, Dk, Dv, N, io_dtype, out_dtype, gate, 0,
                          stream);
}

int lin_recurrent(const void *q, const void *k, const void *v, const float *g, float *S, void *out,
                  const int32_t *cu_seqlens, const int32_t *slot_in, const int32_t *slot_out, int N, int T_total, int H,
                  int Hk, int Dk, int Dv, int slots, kda_dtype io_dtype, kda_dtype out_dtype, int gate, int zero_rows,
                  void *stream) {
    if (!cu_seqlens) return KDA_ERR_INVALID_ARG;
    return recurrent_impl(q, k, v, g, S, out, cu_seqlens, slot_in, slot_out, N, T_total, H, Hk, Dk, Dv, slots, io_dtype,
                          out_dtype, gate, zero_rows, stream);
}

}  // extern "C"
