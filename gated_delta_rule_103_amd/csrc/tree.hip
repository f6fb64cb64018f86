// tree.hip -- trees of drafted tokens: the outputs of every node of a tree that continues a
// sequence's state, and the state behind the node that was accepted.
//
// Node t continues the state of its parent (an earlier node, or the sequence's own state S):
//     S_t = S_p Diag(a_t) + u_t k_t^T,  u_t = b_t (v_t - S_p Diag(a_t) k_t),  o_t = S_t q_t
// (u_t = v_t in linear attention). This is the chunk form with "ancestor" in place of
// "earlier": with r_ts the product of the decays of the nodes below s down to t, r_t that of
// the whole path,
//     L[t][s] = b_t k_t . (r_ts k_s),  M[t][s] = q_t . (r_ts k_s)   (s an ancestor; M[t][t] = q_t . k_t)
//     (I + L) U = b (V - Kd S^T),  O = Qd S^T + M U,   Kd_t = r_t k_t, Qd_t = r_t q_t
// so the state is read once for the whole tree, whatever its shape, and no node's state is
// formed: memory bounds the kernel, 4 Dk Dv bytes a (sequence, head). The decays only ever
// multiply down a path, so no exponent is cut or inverted.
//
// A workgroup takes one (sequence, head), or half of its value channels where there are few.
// D/4 lanes walk from a node to its root, a group of lanes a node; the products with the state
// are fp32 matrix instructions (16 x 16 x 4), whose operands are the state as it lies in memory
// and rows of Kd and Qd in LDS, four steps of one 16-byte load each. U stays in accumulator
// layout, which is the operand layout of the products that follow, and (I + L) is inverted in
// its 16 x 16 diagonal blocks only.
#include "kda_device.h"
#include "kda_launch.h"

namespace kda {
namespace {

template <int W>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = 1; o < W; o <<= 1) x += __shfl_xor(x, o, W);
    return x;
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) { return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w; }

template <typename T> __device__ __forceinline__ f32x4 load4(const T *p);
template <> __device__ __forceinline__ f32x4 load4<float>(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
template <> __device__ __forceinline__ f32x4 load4<bf16_t>(const bf16_t *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                 __uint_as_float(u.y & 0xffff0000u)};
}

// a scalar tensor of either type
__device__ __forceinline__ float scalar_at(const void *p, bool bf16, size_t i) {
    return bf16 ? bf16_to_f32(static_cast<const bf16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

// Log-decays of nodes: per key channel, or one a head, `step` values from a node to the next (0: one for all nodes).
struct Decays {
    const float *g;         // nullptr: none
    bool channels;
    size_t step, at;        // values a node, and this head's first
    __device__ Decays(const TreeArgs &p, int h, int DK)
        : g(p.g), channels(p.gate == 0), step(p.gate == 2 ? 0 : channels ? (size_t)p.H * DK : p.H),
          at(channels ? (size_t)h * DK : h) {}
    // the decays of node (row) for four key channels
    __device__ __forceinline__ f32x4 at4(size_t row, int c) const {
        if (!g) return f32x4{1.f, 1.f, 1.f, 1.f};
        const float *p = g + row * step + at;
        if (channels) {
            const f32x4 x = *reinterpret_cast<const f32x4 *>(p + c);
            return f32x4{expf(x.x), expf(x.y), expf(x.z), expf(x.w)};
        }
        const float x = expf(*p);
        return f32x4{x, x, x, x};
    }
};

__device__ __forceinline__ f32x4 mfma(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

constexpr int kPad = 4, kTile = 20;      // floats of padding a row; floats a row of a 16 x 16 tile
__device__ __forceinline__ constexpr int tile_of(int a, int b) { return a * (a + 1) / 2 + b; }

// TT: tiles of 16 nodes; CT: tiles of 16 value channels a wavefront
template <int DK, int DV, typename T, bool DELTA, int TT, int CT>
__global__ __launch_bounds__(256) void tree_kernel(TreeArgs p) {
    constexpr int NODES = 16 * TT, LPR = DK / 4, GROUPS = 256 / LPR, SPLIT = DV / (64 * CT), KM = DK / 16;
    __shared__ f32x4 Ks[NODES][LPR], As[NODES][LPR];             // keys, decays
    __shared__ float Kd[DELTA ? NODES : 1][DK + kPad], Qd[NODES][DK + kPad];
    __shared__ float Lt[DELTA ? tile_of(TT, 0) : 1][16 * kTile], Mt[tile_of(TT, 0)][16 * kTile];
    __shared__ float beta[NODES];
    __shared__ int up[NODES];
    const int chain = blockIdx.x / SPLIT, n = chain / p.H, h = chain % p.H, group = p.H / p.Hk, hs = h / group;
    const int t = threadIdx.x, lane = t & 63, w = t >> 6, r16 = lane & 15, q4 = lane >> 4, nodes = p.T;
    const T *qp = static_cast<const T *>(p.q), *kp = static_cast<const T *>(p.k), *vp = static_cast<const T *>(p.v);

    // the state's rows of this lane's value channels, 16 bytes of key channels each
    const int from = p.slot_in ? p.slot_in[n] : -1;
    const bool live = from >= 0 && from < p.slots;
    const float *S = p.S + ((size_t)(live ? from : 0) * p.H + h) * DK * DV;
    const int dv0 = ((blockIdx.x % SPLIT) * 4 + w) * 16 * CT + r16;
    f32x4 s[CT][KM];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int m = 0; m < KM; ++m)
            s[c][m] = live ? *reinterpret_cast<const f32x4 *>(S + (size_t)(dv0 + 16 * c) * DK + 16 * m + 4 * q4)
                           : f32x4{0.f, 0.f, 0.f, 0.f};

    // nodes, keys and decays into LDS
    const size_t row0 = (size_t)n * nodes;
    if (t < NODES) {
        up[t] = t < nodes ? p.parent[row0 + t] : -2;
        beta[t] = DELTA && t < nodes ? scalar_at(p.beta, p.beta_dt == Dt::BF16, (row0 + t) * p.H + h) : 0.f;
    }
    for (int i = t; i < tile_of(TT, 0) * 16 * kTile; i += 256) {
        if (DELTA) Lt[0][i] = 0.f;
        Mt[0][i] = 0.f;
    }
    const int g0 = t / LPR, c4 = t % LPR;
    const Decays decays(p, h, DK);
    for (int i = g0; i < nodes; i += GROUPS) {
        f32x4 k = load4(kp + ((row0 + i) * p.Hk + hs) * DK + 4 * c4);
        if (p.qk_norm) k *= 1.f / sqrtf(group_sum<LPR>(dot4(k, k)) + p.norm_eps);
        Ks[i][c4] = k;
        As[i][c4] = decays.at4(row0 + i, 4 * c4);
    }
    __syncthreads();

    // from every node to its root; a node whose path does not end there is absent
    for (int i = g0; i < NODES; i += GROUPS) {
        int a = i, b = i < nodes ? up[i] : -2;
        bool there = true;
        while (b != -1) {                                  // parents come earlier: at most 64 steps
            if (b < 0 || b >= a) { there = false; break; }
            a = b;
            b = up[a];
        }
        f32x4 kd = {0.f, 0.f, 0.f, 0.f}, qd = kd;
        if (there) {
            f32x4 q = load4(qp + ((row0 + i) * p.Hk + hs) * DK + 4 * c4);
            if (p.qk_norm) q *= 1.f / sqrtf(group_sum<LPR>(dot4(q, q)) + p.norm_eps);
            const f32x4 k = Ks[i][c4];
            f32x4 r = As[i][c4];
            const float own = group_sum<LPR>(dot4(q, k)), bt = beta[i];
            if (c4 == 0) Mt[tile_of(i / 16, i / 16)][(i % 16) * (kTile + 1)] = own;
            for (int x = up[i]; x >= 0; x = up[x]) {
                const f32x4 rk = r * Ks[x][c4];
                const float m = group_sum<LPR>(dot4(q, rk));
                const float l = DELTA ? group_sum<LPR>(dot4(k, rk)) : 0.f;
                if (c4 == 0) {
                    Mt[tile_of(i / 16, x / 16)][(i % 16) * kTile + x % 16] = m;
                    if (DELTA) Lt[tile_of(i / 16, x / 16)][(i % 16) * kTile + x % 16] = bt * l;
                }
                r *= As[x][c4];
            }
            kd = k * r;
            qd = q * r;
        } else if (c4 == 0) {
            beta[i] = 0.f;
        }
        if (DELTA) *reinterpret_cast<f32x4 *>(&Kd[i][4 * c4]) = kd;
        *reinterpret_cast<f32x4 *>(&Qd[i][4 * c4]) = qd;
        // up[] is still read by other walkers: whether a node is there is kept beside it
        if (c4 == 0) reinterpret_cast<int *>(&Qd[i][DK])[0] = there;
    }
    __syncthreads();

    // (I + L)^-1 of the diagonal blocks, a column a lane, in place
    if (DELTA && w < TT && lane < 16) {
        float *L = Lt[tile_of(w, w)], x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float y = i == lane ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) y -= L[i * kTile + j] * x[j];
            x[i] = y;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) L[i * kTile + lane] = x[i];
    }
    if (DELTA) __syncthreads();

    f32x4 U[TT][CT];
#pragma unroll
    for (int a = 0; a < TT; ++a) {
        if (16 * a >= nodes) break;                        // uniform
        // Kd S^T and Qd S^T of 16 nodes
        f32x4 X[CT], Y[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) X[c] = Y[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < KM; ++m) {
            const f32x4 y = *reinterpret_cast<const f32x4 *>(&Qd[16 * a + r16][16 * m + 4 * q4]);
            f32x4 x = y;
            if (DELTA) x = *reinterpret_cast<const f32x4 *>(&Kd[16 * a + r16][16 * m + 4 * q4]);
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (DELTA) X[c] = mfma(x[e], s[c][m][e], X[c]);
                    Y[c] = mfma(y[e], s[c][m][e], Y[c]);
                }
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * a + 4 * q4 + e;
                const bool there = reinterpret_cast<const int *>(&Qd[i][DK])[0] != 0;
                v[e] = there ? io<T>::load(vp, ((row0 + i) * p.H + h) * DV + dv0 + 16 * c) : 0.f;
                if (DELTA) v[e] = beta[i] * (v[e] - X[c][e]);
            }
            if constexpr (DELTA) {
#pragma unroll
                for (int b = 0; b < a; ++b) {
                    const f32x4 l = *reinterpret_cast<const f32x4 *>(&Lt[tile_of(a, b)][r16 * kTile + 4 * q4]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v = mfma(-l[e], U[b][c][e], v);
                }
                const f32x4 inv = *reinterpret_cast<const f32x4 *>(&Lt[tile_of(a, a)][r16 * kTile + 4 * q4]);
                U[a][c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 4; ++e) U[a][c] = mfma(inv[e], v[e], U[a][c]);
            } else {
                U[a][c] = v;
            }
#pragma unroll
            for (int b = 0; b <= a; ++b) {
                const f32x4 m = *reinterpret_cast<const f32x4 *>(&Mt[tile_of(a, b)][r16 * kTile + 4 * q4]);
#pragma unroll
                for (int e = 0; e < 4; ++e) Y[c] = mfma(m[e], U[b][c][e], Y[c]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * a + 4 * q4 + e;
                if (i >= nodes) continue;
                const bool there = reinterpret_cast<const int *>(&Qd[i][DK])[0] != 0;
                if (!there && !p.zero_rows) continue;
                const size_t o = ((row0 + i) * p.H + h) * DV + dv0 + 16 * c;
                const float y = there ? Y[c][e] : 0.f;
                if (p.out_dt == Dt::F32) static_cast<float *>(p.out)[o] = y;
                else static_cast<bf16_t *>(p.out)[o] = f32_to_bf16(y);
            }
        }
    }
}

// ---- the accepted state ---------------------------------------------------------
// The path from the root to the node, then its tokens one by one: 64 rows (value channels) of a
// state a workgroup, Dk / 4 lanes a row, as the recurrent form does; each state is read and
// written once, 8 Dk Dv bytes a (sequence, head).
template <int DK, int DV, typename T, bool DELTA>
__global__ __launch_bounds__(DK * 4) void accept_kernel(TreeArgs p) {
    constexpr int LPR = DK / 4, R = 4, ROWS = 64, PASS = ROWS / R, SPLIT = DV / ROWS;
    __shared__ int up[kMaxTreeNodes], path[kMaxTreeNodes], steps;
    const int chain = blockIdx.x / SPLIT, n = chain / p.H, h = chain % p.H, hs = h / (p.H / p.Hk);
    const int t = threadIdx.x, kq = t % LPR, row0 = (blockIdx.x % SPLIT) * ROWS + t / LPR;
    const int to = p.slot_out[n], node = p.node[n];
    if (to < 0 || to >= p.slots || node < -1 || node >= p.T) return;      // uniform
    const int from = p.slot_in ? p.slot_in[n] : -1;
    const bool live = from >= 0 && from < p.slots;
    const size_t DD = (size_t)DK * DV, tok0 = (size_t)n * p.T;
    const f32x4 *Sp = reinterpret_cast<const f32x4 *>(p.S + ((size_t)(live ? from : 0) * p.H + h) * DD);
    f32x4 s[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        s[i] = live ? __builtin_nontemporal_load(&Sp[(row0 + PASS * i) * LPR + kq]) : f32x4{0.f, 0.f, 0.f, 0.f};
    if (t < p.T) up[t] = p.parent[tok0 + t];
    __syncthreads();
    if (t == 0) {
        int d = 0, x = node;
        while (x >= 0) {                                   // parents come earlier: at most 64 steps
            path[d++] = x;
            const int y = up[x];
            x = y < x && y >= -1 ? y : -2;                 // the node is absent
        }
        steps = x == -1 ? d : -1;
    }
    __syncthreads();
    if (steps < 0) return;

    struct Token { f32x4 k, a; float v[R], b; };
    const Decays decays(p, h, DK);
    const T *kp = static_cast<const T *>(p.k), *vp = static_cast<const T *>(p.v);
    auto load = [&](int i) {
        Token x;
        const size_t tok = tok0 + path[i];
        x.k = load4(kp + (tok * p.Hk + hs) * DK + 4 * kq);
        x.a = decays.at4(tok, 4 * kq);
#pragma unroll
        for (int r = 0; r < R; ++r) x.v[r] = io<T>::load(vp, (tok * p.H + h) * DV + row0 + PASS * r);
        x.b = DELTA ? scalar_at(p.beta, p.beta_dt == Dt::BF16, tok * p.H + h) : 0.f;
        return x;
    };
    Token next{};
    if (steps > 0) next = load(steps - 1);
    for (int i = steps - 1; i >= 0; --i) {
        Token x = next;
        if (i > 0) next = load(i - 1);
        if (p.qk_norm) x.k *= 1.f / sqrtf(group_sum<LPR>(dot4(x.k, x.k)) + p.norm_eps);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const f32x4 d = s[r] * x.a;
            const float u = DELTA ? x.b * (x.v[r] - group_sum<LPR>(dot4(d, x.k))) : x.v[r];
            s[r] = d + x.k * u;
        }
    }
    f32x4 *To = reinterpret_cast<f32x4 *>(p.S + ((size_t)to * p.H + h) * DD);
#pragma unroll
    for (int i = 0; i < R; ++i) __builtin_nontemporal_store(s[i], &To[(row0 + PASS * i) * LPR + kq]);
}

// ---- host -----------------------------------------------------------------------
template <int DK, int DV, typename T, bool DELTA, int CT> hipError_t tree_ct(const TreeArgs &a) {
    const dim3 grid((unsigned)(a.N * a.H * (DV / (64 * CT))));
    if (a.T <= 16) hipLaunchKernelGGL((tree_kernel<DK, DV, T, DELTA, 1, CT>), grid, dim3(256), 0, a.stream, a);
    else if (a.T <= 32) hipLaunchKernelGGL((tree_kernel<DK, DV, T, DELTA, 2, CT>), grid, dim3(256), 0, a.stream, a);
    else hipLaunchKernelGGL((tree_kernel<DK, DV, T, DELTA, 4, CT>), grid, dim3(256), 0, a.stream, a);
    return hipGetLastError();
}
template <int DK, int DV, typename T, bool DELTA> hipError_t tree_t(const TreeArgs &a) {
    // a half state a workgroup until there is a whole one for every CU
    if constexpr (DV == 128)
        if ((long long)a.N * a.H >= 256) return tree_ct<DK, DV, T, DELTA, 2>(a);
    return tree_ct<DK, DV, T, DELTA, 1>(a);
}
template <int DK, int DV, typename T, bool DELTA> hipError_t accept_t(const TreeArgs &a) {
    hipLaunchKernelGGL((accept_kernel<DK, DV, T, DELTA>), dim3((unsigned)(a.N * a.H * (DV / 64))), dim3(DK * 4), 0, a.stream, a);
    return hipGetLastError();
}

template <bool ACCEPT, typename T> hipError_t by_width(const TreeArgs &a) {
#define KDA_TREE(DK, DV, DELTA) (ACCEPT ? accept_t<DK, DV, T, DELTA>(a) : tree_t<DK, DV, T, DELTA>(a))
    if (a.beta) return a.Dk == 64 ? KDA_TREE(64, 64, true) : KDA_TREE(128, 128, true);
    if (a.Dk == 64) return a.Dv == 64 ? KDA_TREE(64, 64, false) : KDA_TREE(64, 128, false);
    return a.Dv == 64 ? KDA_TREE(128, 64, false) : KDA_TREE(128, 128, false);
#undef KDA_TREE
}

}  // namespace

bool tree_fits(int N, int H) { return (unsigned long long)N * H * 1024 < (1ull << 32); }     // threads of a launch

hipError_t launch_tree(const TreeArgs &a) {
    return a.io == Dt::F32 ? by_width<false, float>(a) : by_width<false, bf16_t>(a);
}
hipError_t launch_tree_accept(const TreeArgs &a) {
    return a.io == Dt::F32 ? by_width<true, float>(a) : by_width<true, bf16_t>(a);
}

}  // namespace kda
