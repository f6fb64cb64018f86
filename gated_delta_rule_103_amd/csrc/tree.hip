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
// A workgroup takes one (sequence, head). Sixteen lanes, whose sums
// need no LDS, walk from a node to its root. The products with the state run on the bf16 matrix
// instructions with all operands cut in three (2^-25, the six products that matter): the fp32 ones
// would take five times as long, which is more than the state's way from memory for more than 16 nodes.
// The state is an operand as it lies in memory, 16 bytes a load; Kd and Qd lie in LDS in the order that
// this asks for, in the place of the keys and decays that the walks read. U stays in accumulator layout,
// which is the operand layout of the fp32 products that follow, and (I + L) is inverted in its 16 x 16
// diagonal blocks only.
//
// 128 trees of 16 nodes x 32 heads x 128 channels: 83-88 us, 369 MB, 4.2-4.4 TB/s, against 72 at a copy's rate (fp32 matrix
// instructions 89); linear attention's 68 against 61. More nodes bring more walks, a step a pair of node and ancestor on the
// vector units: 64 trees of 32 nodes 75-78 us against 46, 32 of 64 91-98 against 33 (all their Kd and Qd in LDS at once: 104
// and 110, for want of workgroups a CU), linear attention's 56 against 34 and 64 against 21. One tree of 61 nodes x 16 heads:
// 21 us, latency.
#include "kda_device.h"
#include "kda_launch.h"

#include <type_traits>

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

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The bf16 values next to x, which keeps the rest: three times, and the parts' sum is x to 2^-25.
__device__ __forceinline__ uint32_t cut_off(float &a, float &b) {
    const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
    a -= __uint_as_float(w << 16);
    b -= __uint_as_float(w & 0xffff0000u);
    return w;
}
__device__ __forceinline__ u32x2 cut_off(f32x4 &x) {
    float a = x.x, b = x.y, c = x.z, d = x.w;
    const u32x2 w = {cut_off(a, b), cut_off(c, d)};
    x = f32x4{a, b, c, d};
    return w;
}
__device__ __forceinline__ void cut3(f32x4 x, f32x4 y, bf16x8 (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const u32x2 a = cut_off(x), b = cut_off(y);
        p[i] = __builtin_bit_cast(bf16x8, u32x4{a.x, a.y, b.x, b.y});
    }
}

// four values as they lie
template <typename T> struct quad;
template <> struct quad<float> {
    typedef f32x4 raw;
    __device__ __forceinline__ static f32x4 wide(raw x) { return x; }
};
template <> struct quad<bf16_t> {
    typedef uint32_t raw __attribute__((ext_vector_type(2)));
    __device__ __forceinline__ static f32x4 wide(raw u) {
        return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u)};
    }
};

// a scalar tensor of either type
__device__ __forceinline__ float scalar_at(const void *p, bool bf16, size_t i) {
    return bf16 ? bf16_to_f32(static_cast<const bf16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

// Log-decays of a sequence's nodes (row0: its first): per key channel, or one a head, `step` values from a node to
// the next (0: one for all nodes).
struct Decays {
    const float *g;         // this head's, of the first node; nullptr: none
    bool channels;
    unsigned step;
    __device__ Decays(const TreeArgs &p, size_t row0, int h, int DK) : channels(p.gate == 0) {
        step = p.gate == 2 ? 0u : channels ? (unsigned)(p.H * DK) : (unsigned)p.H;
        g = p.g ? p.g + row0 * step + (channels ? (size_t)h * DK : h) : nullptr;
    }
    // the decays of node i for four key channels
    __device__ __forceinline__ f32x4 at4(unsigned i, unsigned c) const {
        if (!g) return f32x4{1.f, 1.f, 1.f, 1.f};
        if (channels) {
            const f32x4 x = *reinterpret_cast<const f32x4 *>(g + (i * step + c));
            return f32x4{expf(x.x), expf(x.y), expf(x.z), expf(x.w)};
        }
        const float x = expf(g[i * step]);
        return f32x4{x, x, x, x};
    }
};

__device__ __forceinline__ f32x4 mfma(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// the sum over 16 neighbouring lanes, in all of them
__device__ __forceinline__ float row_sum(float x) {
    auto turned = [](float y, auto by) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(y), 0x120 + decltype(by)::value, 0xf, 0xf, false));
    };
    x += turned(x, std::integral_constant<int, 8>{});
    x += turned(x, std::integral_constant<int, 4>{});
    x += turned(x, std::integral_constant<int, 2>{});
    return x + turned(x, std::integral_constant<int, 1>{});
}

constexpr int kPad = 8, kTile = 20;      // values of padding a row; floats a row of a 16 x 16 tile
__device__ __forceinline__ constexpr int tile_of(int a, int b) { return a * (a + 1) / 2 + b; }

// TT: tiles of 16 nodes; NW wavefronts
template <int DK, int DV, typename T, bool DELTA, int TT, int NW>
__global__ __launch_bounds__(64 * NW, TT == 1 || NW == 8 ? 4 : 2) void tree_kernel(TreeArgs p) {
    constexpr int NODES = 16 * TT, KM = DK / 16, CH = DK / 64, NT = 64 * NW;
    constexpr int GROUPS = NT / 16, NP = (NODES + GROUPS - 1) / GROUPS;      // 16 lanes a node, NP nodes a group
    constexpr int CT = DV / (16 * NW), PART = 16;           // tiles of value channels a wavefront; nodes whose Kd and Qd are in LDS at a time
    static_assert(NW * CT * 16 == DV && (PART % GROUPS == 0 || GROUPS % PART == 0), "tree tiling");
    // keys (as they came) and decays for the walk; then, in their place, Kd and Qd
    struct Walk { T k[NODES][DK]; f32x4 a[NODES][DK / 4]; };
    struct Products { bf16_t k[DELTA ? 3 : 1][DELTA ? PART : 1][DK + kPad], q[3][PART][DK + kPad]; };
    __shared__ union { Walk walk; Products prod; } u;
    __shared__ float Lt[DELTA ? tile_of(TT, 0) : 1][16 * kTile], Mt[tile_of(TT, 0)][16 * kTile];
    __shared__ float beta[NODES], kn[NODES];                     // kn: the normalisation's factor
    __shared__ int up[NODES], there[NODES];
    const int n = blockIdx.x / p.H, h = blockIdx.x % p.H, hs = h / (p.H / p.Hk);
    const int t = threadIdx.x, lane = t & 63, w = t >> 6, r16 = lane & 15, q4 = lane >> 4, nodes = p.T;
    // this head's first values of the sequence's first node; offsets from them stay below 2^31
    const size_t row0 = (size_t)n * nodes, kv0 = (row0 * p.Hk + hs) * DK, vo0 = (row0 * p.H + h) * DV;
    const T *qp = static_cast<const T *>(p.q) + kv0, *kp = static_cast<const T *>(p.k) + kv0,
            *vp = static_cast<const T *>(p.v) + vo0;
    const unsigned vs = (unsigned)p.H * DV;

    // nodes: 16 lanes each, a lane's channels 64j + 4 r16 .. + 3
    const int i0 = t / 16;
    const Decays decays(p, row0, h, DK);
    f32x4 k[NP][CH], q[NP][CH], r[NP][CH];
    typename quad<T>::raw raw[NP][CH];
#pragma unroll
    for (int a = 0; a < NP; ++a)
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const unsigned i = min(GROUPS * a + i0, nodes - 1), c = 64 * j + 4 * r16, at = i * (unsigned)(p.Hk * DK) + c;
            raw[a][j] = *reinterpret_cast<const typename quad<T>::raw *>(kp + at);
            q[a][j] = load4(qp + at);
            r[a][j] = decays.at4(i, c);
        }
    // the state's rows of this lane's value channels, 16 bytes of key channels each
    const int from = p.slot_in ? p.slot_in[n] : -1;
    const bool live = from >= 0 && from < p.slots;
    const float *S = p.S + ((size_t)(live ? from : 0) * p.H + h) * DK * DV;
    const unsigned dv0 = 16 * CT * w + r16, s0 = dv0 * DK + 4 * q4;
    f32x4 s[CT][KM];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int m = 0; m < KM; ++m)
            s[c][m] = live ? __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(S + (s0 + 16 * c * DK + 16 * m)))
                           : f32x4{0.f, 0.f, 0.f, 0.f};
    if (w == 0) {
        // a node whose path does not end at the sequence is absent; parents come earlier, so paths are at most 64 long
        const int parent = lane < nodes ? p.parent[row0 + lane] : -2;
        bool ok = true;
        int x = lane, y = parent;
        while (__any(y != -1)) {
            if (y != -1 && (y < 0 || y >= x)) {
                ok = false;
                y = -1;
            }
            const int next = __shfl(parent, y < 0 ? 0 : y, 64);
            if (y != -1) {
                x = y;
                y = next;
            }
        }
        if (lane < NODES) {
            up[lane] = parent;
            there[lane] = ok;
            beta[lane] = DELTA && ok ? scalar_at(p.beta, p.beta_dt == Dt::BF16, (row0 + lane) * p.H + h) : 0.f;
        }
    }
    for (int i = t; i < tile_of(TT, 0) * 16 * kTile; i += NT) {
        if (DELTA) Lt[0][i] = 0.f;
        Mt[0][i] = 0.f;
    }
#pragma unroll
    for (int a = 0; a < NP; ++a) {
        const int i = GROUPS * a + i0;
        float nk = 1.f;
#pragma unroll
        for (int j = 0; j < CH; ++j) k[a][j] = quad<T>::wide(raw[a][j]);
        if (p.qk_norm) {                                   // uniform
            float kk = 0.f, qq = 0.f;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                kk += dot4(k[a][j], k[a][j]);
                qq += dot4(q[a][j], q[a][j]);
            }
            nk = 1.f / sqrtf(row_sum(kk) + p.norm_eps);
            qq = 1.f / sqrtf(row_sum(qq) + p.norm_eps);
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                k[a][j] *= nk;
                q[a][j] *= qq;
            }
        }
        if (i < NODES) {
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                *reinterpret_cast<typename quad<T>::raw *>(&u.walk.k[i][64 * j + 4 * r16]) = raw[a][j];
                u.walk.a[i][16 * j + r16] = r[a][j];
            }
            if (r16 == 0) kn[i] = nk;
        }
    }
    __syncthreads();

    // from every node to its root, a group's nodes in step
    int x[NP];
    bool on[NP];
    float bt[NP];
#pragma unroll
    for (int a = 0; a < NP; ++a) {
        const int i = min(GROUPS * a + i0, NODES - 1);
        on[a] = GROUPS * a + i0 < NODES && there[i];
        x[a] = on[a] ? up[i] : -1;
        bt[a] = beta[i];
        float own = 0.f;
#pragma unroll
        for (int j = 0; j < CH; ++j) own += dot4(q[a][j], k[a][j]);
        own = row_sum(own);
        if (on[a] && r16 == 0) Mt[tile_of(i / 16, i / 16)][i % 16 * (kTile + 1)] = own;
    }
    for (;;) {
        bool more = false;
#pragma unroll
        for (int a = 0; a < NP; ++a) more |= x[a] >= 0;
        if (!more) break;
        int y[NP];
        float m[NP], l[NP];
        f32x4 ra[NP][CH];
#pragma unroll
        for (int a = 0; a < NP; ++a) {
            const int z = max(x[a], 0);
            y[a] = up[z];
            m[a] = l[a] = 0.f;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const f32x4 rk = r[a][j] * load4(&u.walk.k[z][64 * j + 4 * r16]);
                m[a] += dot4(q[a][j], rk);
                if (DELTA) l[a] += dot4(k[a][j], rk);
                ra[a][j] = r[a][j] * u.walk.a[z][16 * j + r16];
            }
        }
#pragma unroll
        for (int a = 0; a < NP; ++a) {
            m[a] = row_sum(m[a]);
            if (DELTA) l[a] = row_sum(l[a]);
            if (x[a] >= 0) {
                const int i = GROUPS * a + i0, tile = tile_of(i / 16, 0) + x[a] / 16, at = i % 16 * kTile + x[a] % 16;
                if (r16 == 0) {
                    Mt[tile][at] = kn[x[a]] * m[a];
                    if (DELTA) Lt[tile][at] = bt[a] * (kn[x[a]] * l[a]);
                }
#pragma unroll
                for (int j = 0; j < CH; ++j) r[a][j] = ra[a][j];
                x[a] = y[a];
            }
        }
    }
#pragma unroll
    for (int a = 0; a < NP; ++a)
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
            k[a][j] = on[a] ? k[a][j] * r[a][j] : zero;
            q[a][j] = on[a] ? q[a][j] * r[a][j] : zero;
        }
    __syncthreads();                                       // the walks are done
    // rows of Kd and Qd of PART nodes from `first` on
    auto publish = [&](int first) {
#pragma unroll
        for (int a = 0; a < NP; ++a) {
            const int i = GROUPS * a + i0 - first;
            if (i < 0 || i >= PART) continue;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                // channel 32m + 16b + 4g + e lies at 32m + 8g + 4b + e: as lane group g of the state holds its channels
                const int at = 64 * j + 32 * (r16 >> 3) + 8 * (r16 & 3) + 4 * ((r16 >> 2) & 1);
                f32x4 x = k[a][j], y = q[a][j];
#pragma unroll
                for (int part = 0; part < 3; ++part) {
                    if (DELTA) *reinterpret_cast<u32x2 *>(&u.prod.k[part][i][at]) = cut_off(x);
                    *reinterpret_cast<u32x2 *>(&u.prod.q[part][i][at]) = cut_off(y);
                }
            }
        }
        __syncthreads();
    };
    publish(0);

    // (I + L)^-1 of the diagonal blocks, a column a lane, in place, while the others start on the products
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

    f32x4 U[TT][CT];
#pragma unroll
    for (int a = 0; a < TT; ++a) {
        if (16 * a >= nodes) break;                        // uniform; never at a == 0
        if (a > 0 && 16 * a % PART == 0) {
            __syncthreads();
            publish(16 * a);
        }
        f32x4 v[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * a + 4 * q4 + e;
                const float y = io<T>::load(vp, min(i, nodes - 1) * vs + dv0 + 16 * c);
                v[c][e] = there[i] ? y : 0.f;
            }
        // Kd S^T and Qd S^T of 16 nodes
        f32x4 X[CT], Y[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) X[c] = Y[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < KM / 2; ++m) {
            bf16x8 x[3], y[3];
#pragma unroll
            for (int part = 0; part < 3; ++part) {
                if (DELTA) x[part] = *reinterpret_cast<const bf16x8 *>(&u.prod.k[DELTA ? part : 0][16 * a % PART + r16][32 * m + 8 * q4]);
                y[part] = *reinterpret_cast<const bf16x8 *>(&u.prod.q[part][16 * a % PART + r16][32 * m + 8 * q4]);
            }
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                bf16x8 z[3];
                cut3(s[c][2 * m], s[c][2 * m + 1], z);
#pragma unroll
                for (int i = 2; i >= 0; --i)
#pragma unroll
                    for (int j = 2 - i; j >= 0; --j) {
                        if (DELTA) X[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], z[j], X[c], 0, 0, 0);
                        Y[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y[i], z[j], Y[c], 0, 0, 0);
                    }
            }
        }
        if (DELTA && a == 0) __syncthreads();              // the inverses are there
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            if (DELTA) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[c][e] = beta[16 * a + 4 * q4 + e] * (v[c][e] - X[c][e]);
            }
            if constexpr (DELTA) {
#pragma unroll
                for (int b = 0; b < a; ++b) {
                    const f32x4 l = *reinterpret_cast<const f32x4 *>(&Lt[tile_of(a, b)][r16 * kTile + 4 * q4]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[c] = mfma(-l[e], U[b][c][e], v[c]);
                }
                const f32x4 inv = *reinterpret_cast<const f32x4 *>(&Lt[tile_of(a, a)][r16 * kTile + 4 * q4]);
                U[a][c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 4; ++e) U[a][c] = mfma(inv[e], v[c][e], U[a][c]);
            } else {
                U[a][c] = v[c];
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
                if (i < nodes && (there[i] || p.zero_rows)) {
                    const float y = there[i] ? Y[c][e] : 0.f;
                    const size_t o = vo0 + (i * vs + dv0 + 16 * c);
                    if (p.out_dt == Dt::F32) static_cast<float *>(p.out)[o] = y;
                    else static_cast<__bf16 *>(p.out)[o] = (__bf16)y;
                }
            }
        }
    }
}

// ---- the accepted state ---------------------------------------------------------
// The path from the root to the node, then its tokens one by one: 64 rows (value channels) of a
// state a workgroup, Dk / 4 lanes a row, as the recurrent form does; each state is read and
// written once, 8 Dk Dv bytes a (sequence, head), which bounds it: 128 trees of 16 nodes x 32 heads x 128
// channels in 113 us, 4.9 TB/s.
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
    const Decays decays(p, tok0, h, DK);
    const T *kp = static_cast<const T *>(p.k), *vp = static_cast<const T *>(p.v);
    auto load = [&](int i) {
        Token x;
        const size_t tok = tok0 + path[i];
        x.k = load4(kp + (tok * p.Hk + hs) * DK + 4 * kq);
        x.a = decays.at4(path[i], 4 * kq);
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
template <int DK, int DV, typename T, bool DELTA, int TT, int NW> hipError_t tree_nodes(const TreeArgs &a) {
    hipLaunchKernelGGL((tree_kernel<DK, DV, T, DELTA, TT, NW>), dim3((unsigned)(a.N * a.H)), dim3(64 * NW), 0, a.stream, a);
    return hipGetLastError();
}
// Four wavefronts for 16 nodes; for more, whose LDS leaves two workgroups a CU and whose walks want the wavefronts, one
// for each 16 value channels. The other way round, at 128 channels: 128 x 16 nodes 83 -> 103 us, 64 x 32 75 -> 91, 32 x 64
// 91 -> 109. Half of a state a workgroup gains nothing for few trees either (8 heads x 64 nodes 29 -> 33 us).
template <int DK, int DV, typename T, bool DELTA> hipError_t tree_t(const TreeArgs &a) {
    return a.T <= 16   ? tree_nodes<DK, DV, T, DELTA, 1, 4>(a)
           : a.T <= 32 ? tree_nodes<DK, DV, T, DELTA, 2, DV / 16>(a)
                       : tree_nodes<DK, DV, T, DELTA, 4, DV / 16>(a);
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

bool tree_fits(int N, int H) {
    // threads of a launch, and a sequence's values
    return (unsigned long long)N * H * 1024 < (1ull << 32) && H <= 65536;
}

hipError_t launch_tree(const TreeArgs &a) {
    return a.io == Dt::F32 ? by_width<false, float>(a) : by_width<false, bf16_t>(a);
}
hipError_t launch_tree_accept(const TreeArgs &a) {
    return a.io == Dt::F32 ? by_width<true, float>(a) : by_width<true, bf16_t>(a);
}

}  // namespace kda
