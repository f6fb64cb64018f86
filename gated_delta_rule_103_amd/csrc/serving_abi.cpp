// serving_abi.cpp -- the extern "C" boundary of trees of drafted tokens and of the state
// pool's slots: argument checks. The contract is in include/kda.h.
#include "../../include/kda.h"

#include <climits>

#include "kda_launch.h"

using kda::Dt;

static_assert(KDA_TREE_NODES == kda::kMaxTreeNodes, "one limit");

namespace {

bool dtype_ok(int d) { return d == KDA_F32 || d == KDA_BF16; }
bool width_ok(int D) { return D == 64 || D == 128; }
bool misaligned(const void *p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

// The delta-rule forms' options; false: refused.
bool options_ok(const kda_options *o) {
    if (!o) return true;
    if (o->gate != KDA_GATE_CHANNEL && o->gate != KDA_GATE_HEAD) return false;
    if (o->qk_l2norm && !(o->l2norm_eps > 0.f)) return false;      // also rejects NaN
    return !o->snapshots;
}

// What outputs and accepted states share; a.slot_in and a.slot_out may be NULL only where the caller says so.
int check(const kda::TreeArgs &a, kda_dtype io, int beta_dtype, bool delta) {
    if (a.N < 1 || a.T < 1 || a.H < 1 || a.Hk < 1 || a.H % a.Hk != 0 || a.Dk < 1 || a.Dv < 1 || a.slots < 1)
        return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(io) || !dtype_ok(beta_dtype)) return KDA_ERR_INVALID_ARG;
    if (!a.k || !a.v || !a.S || !a.parent || (delta && !a.beta)) return KDA_ERR_INVALID_ARG;
    if (a.gate == KDA_GATE_CHANNEL && !a.g) return KDA_ERR_INVALID_ARG;
    if ((long long)a.N * a.T > INT_MAX / 2) return KDA_ERR_INVALID_ARG;
    if (misaligned(a.q, 15) || misaligned(a.k, 15) || misaligned(a.v, 15) || misaligned(a.S, 15) || misaligned(a.out, 15) ||
        misaligned(a.g, a.gate == KDA_GATE_CHANNEL ? 15 : 3))
        return KDA_ERR_INVALID_ARG;
    if (!width_ok(a.Dk) || !width_ok(a.Dv) || (delta && a.Dk != a.Dv)) return KDA_ERR_UNSUPPORTED;
    if (a.T > KDA_TREE_NODES || !kda::tree_fits(a.N, a.H)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

int tree_impl(kda::TreeArgs &a, kda_dtype io, int beta_dtype, int out_dtype, int zero_rows, bool delta) {
    if (!dtype_ok(out_dtype) || (zero_rows != 0 && zero_rows != 1) || !a.q || !a.out) return KDA_ERR_INVALID_ARG;
    const void *ins[] = {a.q, a.k, a.v, a.g, a.beta, a.S, a.slot_in, a.parent};
    for (const void *x : ins)
        if (x == a.out) return KDA_ERR_INVALID_ARG;
    const int bad = check(a, io, beta_dtype, delta);
    if (bad != KDA_OK) return bad;
    a.out_dt = static_cast<Dt>(out_dtype);
    a.zero_rows = zero_rows != 0;
    return kda::launch_tree(a) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

int accept_impl(kda::TreeArgs &a, kda_dtype io, int beta_dtype, bool delta) {
    if (!a.node || !a.slot_out) return KDA_ERR_INVALID_ARG;
    // the pool is written while other workgroups still read the tokens and the indexes
    const void *ins[] = {a.k, a.v, a.g, a.beta, a.slot_in, a.slot_out, a.parent, a.node};
    for (const void *x : ins)
        if (x && x == a.S) return KDA_ERR_INVALID_ARG;
    const int bad = check(a, io, beta_dtype, delta);
    if (bad != KDA_OK) return bad;
    return kda::launch_tree_accept(a) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda::TreeArgs args(const void *q, const void *k, const void *v, const float *g, const void *beta, const float *S, void *out,
                   const int32_t *slot_in, const int32_t *slot_out, const int32_t *parent, const int32_t *node, int N, int T,
                   int H, int Hk, int Dk, int Dv, int slots, kda_dtype io, int beta_dtype, int gate, void *stream) {
    kda::TreeArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S = const_cast<float *>(S); a.out = out;
    a.slot_in = slot_in; a.slot_out = slot_out; a.parent = parent; a.node = node;
    a.N = N; a.T = T; a.H = H; a.Hk = Hk; a.Dk = Dk; a.Dv = Dv; a.slots = slots;
    a.io = static_cast<Dt>(io); a.beta_dt = static_cast<Dt>(beta_dtype);
    a.gate = gate;
    a.stream = static_cast<hipStream_t>(stream);
    return a;
}

}  // namespace

extern "C" {

int kda_tree(const void *q, const void *k, const void *v, const float *g, const void *beta, const float *S, void *out,
             const int32_t *slot_in, const int32_t *parent, int N, int T, int H, int Dk, int Dv, int slots,
             kda_dtype io_dtype, kda_dtype beta_dtype, kda_dtype out_dtype, int zero_rows, const kda_options *opt,
             void *stream) {
    if (!options_ok(opt)) return KDA_ERR_INVALID_ARG;
    const kda_options o = opt ? *opt : kda_options{};
    kda::TreeArgs a = args(q, k, v, g, beta, S, out, slot_in, nullptr, parent, nullptr, N, T, H, H, Dk, Dv, slots, io_dtype,
                           beta_dtype, o.gate, stream);
    a.qk_norm = o.qk_l2norm != 0;
    a.norm_eps = o.l2norm_eps;
    return tree_impl(a, io_dtype, beta_dtype, out_dtype, zero_rows, true);
}

int kda_tree_accept(const void *k, const void *v, const float *g, const void *beta, float *S, const int32_t *slot_in,
                    const int32_t *slot_out, const int32_t *parent, const int32_t *node, int N, int T, int H, int Dk,
                    int Dv, int slots, kda_dtype io_dtype, kda_dtype beta_dtype, const kda_options *opt, void *stream) {
    if (!options_ok(opt)) return KDA_ERR_INVALID_ARG;
    const kda_options o = opt ? *opt : kda_options{};
    kda::TreeArgs a = args(nullptr, k, v, g, beta, S, nullptr, slot_in, slot_out, parent, node, N, T, H, H, Dk, Dv, slots,
                           io_dtype, beta_dtype, o.gate, stream);
    a.qk_norm = o.qk_l2norm != 0;
    a.norm_eps = o.l2norm_eps;
    return accept_impl(a, io_dtype, beta_dtype, true);
}

int lin_tree(const void *q, const void *k, const void *v, const float *g, const float *S, void *out,
             const int32_t *slot_in, const int32_t *parent, int N, int T, int H, int Hk, int Dk, int Dv, int slots,
             kda_dtype io_dtype, kda_dtype out_dtype, int gate, int zero_rows, void *stream) {
    if (gate != KDA_GATE_HEAD && gate != KDA_GATE_FIXED) return KDA_ERR_INVALID_ARG;
    kda::TreeArgs a = args(q, k, v, g, nullptr, S, out, slot_in, nullptr, parent, nullptr, N, T, H, Hk, Dk, Dv, slots,
                           io_dtype, KDA_F32, gate, stream);
    return tree_impl(a, io_dtype, KDA_F32, out_dtype, zero_rows, false);
}

int lin_tree_accept(const void *k, const void *v, const float *g, float *S, const int32_t *slot_in,
                    const int32_t *slot_out, const int32_t *parent, const int32_t *node, int N, int T, int H, int Hk,
                    int Dk, int Dv, int slots, kda_dtype io_dtype, int gate, void *stream) {
    if (gate != KDA_GATE_HEAD && gate != KDA_GATE_FIXED) return KDA_ERR_INVALID_ARG;
    kda::TreeArgs a = args(nullptr, k, v, g, nullptr, S, nullptr, slot_in, slot_out, parent, node, N, T, H, Hk, Dk, Dv, slots,
                           io_dtype, KDA_F32, gate, stream);
    return accept_impl(a, io_dtype, KDA_F32, false);
}

int kda_slots_copy(const void *from, void *to, const int32_t *src, const int32_t *dst, int n, int layers, int from_slots,
                   int to_slots, size_t slot_bytes, void *stream) {
    if (n < 0 || layers < 1 || from_slots < 1 || to_slots < 1 || slot_bytes == 0 || slot_bytes % 16 != 0) return KDA_ERR_INVALID_ARG;
    if (!from || !to || (n > 0 && (!src || !dst)) || misaligned(from, 15) || misaligned(to, 15)) return KDA_ERR_INVALID_ARG;
    if (from == to && from_slots != to_slots) return KDA_ERR_INVALID_ARG;
    if (!kda::slots_copy_fits(n, layers, slot_bytes)) return KDA_ERR_UNSUPPORTED;
    if (n == 0) return KDA_OK;
    kda::SlotsCopyArgs a;
    a.from = static_cast<const char *>(from); a.to = static_cast<char *>(to); a.src = src; a.dst = dst;
    a.n = n; a.layers = layers; a.from_slots = from_slots; a.to_slots = to_slots; a.slot_bytes = slot_bytes;
    a.stream = static_cast<hipStream_t>(stream);
    return kda::launch_slots_copy(a) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"

namespace {

int count_impl(int32_t *uses, const int32_t *which, int n, int slots, int add, void *stream) {
    if (n < 0 || n > INT_MAX / 2 || slots < 1 || slots > INT_MAX / 2 || !uses || (n > 0 && !which) || uses == which) return KDA_ERR_INVALID_ARG;
    if (n == 0) return KDA_OK;
    return kda::launch_slots_count(uses, which, n, slots, add, static_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK
                                                                                                              : KDA_ERR_HIP;
}

}  // namespace

extern "C" {

int kda_slots_share(int32_t *uses, const int32_t *which, int n, int slots, void *stream) {
    return count_impl(uses, which, n, slots, 1, stream);
}
int kda_slots_release(int32_t *uses, const int32_t *which, int n, int slots, void *stream) {
    return count_impl(uses, which, n, slots, -1, stream);
}

int kda_slots_acquire(int32_t *uses, int32_t *taken, int n, int slots, void *stream) {
    if (n < 0 || n > INT_MAX / 2 || slots < 1 || slots > INT_MAX / 2 || !uses || (n > 0 && !taken) || uses == taken) return KDA_ERR_INVALID_ARG;
    if (n == 0) return KDA_OK;
    return kda::launch_slots_acquire(uses, slots, taken, n, static_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK
                                                                                                           : KDA_ERR_HIP;
}

// a new place for every slot, and a pair for every move of at most half of them
size_t kda_slots_compact_workspace_size(int slots) {
    return slots < 1 || slots > INT_MAX / 8 ? 0 : ((size_t)slots * 2 + 2) * sizeof(int32_t);
}

int kda_slots_compact(void *pool, int32_t *uses, int32_t *table, int32_t *count, int table_n, int layers, int slots,
                      size_t slot_bytes, void *workspace, size_t workspace_bytes, void *stream) {
    if (layers < 1 || slots < 1 || table_n < 0 || table_n > INT_MAX / 2 || slot_bytes == 0 || slot_bytes % 16 != 0)
        return KDA_ERR_INVALID_ARG;
    if (!pool || !uses || !count || (table_n > 0 && !table) || misaligned(pool, 15)) return KDA_ERR_INVALID_ARG;
    if (uses == count || (table && (table == uses || table == count))) return KDA_ERR_INVALID_ARG;
    if (!kda::slots_compact_fits(slots, slot_bytes)) return KDA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < kda_slots_compact_workspace_size(slots) || misaligned(workspace, 255))
        return KDA_ERR_WORKSPACE;
    kda::SlotsCompactArgs a;
    a.pool = static_cast<char *>(pool); a.uses = uses; a.count = count; a.table = table;
    a.slots = slots; a.layers = layers; a.table_n = table_n; a.slot_bytes = slot_bytes;
    a.moved = static_cast<int32_t *>(workspace);
    a.stream = static_cast<hipStream_t>(stream);
    return kda::launch_slots_compact(a) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
