// recurrent.hip -- the recurrent form: a few tokens of each sequence, one by
// one, over states that live in the slots of a pool.
//
//     S' = S Diag(exp g),  u = beta (v - S' k),  S = S' + u k^T,  o = S q
//
// A sequence starts from the slot slot_in names and the state after token t
// goes to the slot slot_out[t] names (none where that is negative), so a
// serving loop can check several draft tokens in one call and go on from
// whichever state it accepts, and a shared prefix is read without a copy.
//
// Rows of S (value channels) do not meet in the recurrence: every row has its
// own u. A workgroup therefore owns some rows of one (sequence, head) for all
// of its tokens, holds them in registers and reads and writes each state once,
// which is what bounds the kernel: memory, at 4 D^2 bytes for each state read
// and each state kept. D/4 consecutive lanes own a row (four key channels
// each), as in the single-token kernel, so both dot products of a row are
// sums inside those lanes. The next token's vectors are loaded while the
// current one is computed. 128 sequences x 4 tokens x 32 heads x 128 channels with every
// state kept: 1.38 GB in 276 us (255-303 over 60 launches under the profiler), 5.0 TB/s, the
// rate of a large copy, 5.1. One sequence x 3 tokens: 8 us, the latency of three dependent
// tokens behind that of loading a state.
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

// One token's vectors as a lane holds them.
template <int R> struct Token {
    f32x4 q, k, g;
    float v[R], beta;
    int slot;
};

template <int D, int NT, int R, typename TI, typename TB, typename TO>
__global__ __launch_bounds__(NT) void recurrent_kernel(const TI *__restrict__ q, const TI *__restrict__ k,
                                                       const TI *__restrict__ v, const float *__restrict__ g,
                                                       const TB *__restrict__ beta, float *__restrict__ S,
                                                       TO *__restrict__ out, const int32_t *__restrict__ cu,
                                                       const int32_t *__restrict__ slot_in,
                                                       const int32_t *__restrict__ slot_out, int N, int T, int H, int slots,
                                                       bool g_head, bool qk_norm, float norm_eps, bool zero_rows) {
    constexpr int LPR = D / 4, SLOTS = NT / LPR, ROWS = R * SLOTS, SPLIT = D / ROWS;
    static_assert(NT % LPR == 0 && D % ROWS == 0, "recurrent tiling");
    const int chain = blockIdx.x / SPLIT, n = chain / H, h = chain % H;
    const int t = threadIdx.x, kq = t % LPR;
    const int row0 = (blockIdx.x % SPLIT) * ROWS + t / LPR;
    // offsets outside the packed rows are cut to them
    const int begin = min(max(cu[n], 0), T), end = min(max(cu[n + 1], begin), T);
    if (zero_rows) {                                     // uniform
        // rows of no sequence lie before the first one and behind the last one, whose
        // workgroups clear them, each its head's value channels
        constexpr int TOKENS = NT / ROWS;
        const int col = (blockIdx.x % SPLIT) * ROWS + t % ROWS;
        auto clear = [&](int from, int to) {
            for (int tok = from + t / ROWS; tok < to; tok += TOKENS) out[((size_t)tok * H + h) * D + col] = TO(0);
        };
        if (n == 0) clear(0, begin);
        if (n == N - 1) clear(end, T);
    }
    if (begin == end) return;

    const size_t DD = (size_t)D * D;
    f32x4 s[R];
    const int from = slot_in ? slot_in[n] : -1;
    const bool live = from >= 0 && from < slots;
    const f32x4 *Sp = reinterpret_cast<const f32x4 *>(S + ((size_t)(live ? from : 0) * H + h) * DD);
#pragma unroll
    for (int i = 0; i < R; ++i) s[i] = live ? Sp[(row0 + SLOTS * i) * (D / 4) + kq] : f32x4{0.f, 0.f, 0.f, 0.f};

    auto load = [&](int tok) {
        Token<R> x;
        const size_t th = (size_t)tok * H + h;
        x.q = load4(q + th * D + 4 * kq);
        x.k = load4(k + th * D + 4 * kq);
        x.g = f32x4{0.f, 0.f, 0.f, 0.f};
        if (g) {
            if (g_head) {
                const float y = g[th];
                x.g = f32x4{y, y, y, y};
            } else {
                x.g = load4(g + th * D + 4 * kq);
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) x.v[i] = io<TI>::load(v, th * D + row0 + SLOTS * i);
        x.beta = io<TB>::load(beta, th);
        x.slot = slot_out ? slot_out[tok] : -1;
        return x;
    };

    Token<R> next = load(begin);
    for (int tok = begin; tok < end; ++tok) {
        Token<R> x = next;
        if (tok + 1 < end) next = load(tok + 1);
        f32x4 a;
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = expf(x.g[e]);
        if (qk_norm) {
            x.q *= 1.f / sqrtf(group_sum<LPR>(dot4(x.q, x.q)) + norm_eps);
            x.k *= 1.f / sqrtf(group_sum<LPR>(dot4(x.k, x.k)) + norm_eps);
        }
        const float qk = group_sum<LPR>(dot4(x.q, x.k));
        const bool keep = x.slot >= 0 && x.slot < slots;
        f32x4 *Kp = reinterpret_cast<f32x4 *>(S + ((size_t)(keep ? x.slot : 0) * H + h) * DD);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const f32x4 d = s[i] * a;                        // S' = S Diag(exp g)
            const float pk = group_sum<LPR>(dot4(d, x.k));   // (S' k)_row
            const float pq = group_sum<LPR>(dot4(d, x.q));   // (S' q)_row
            const float u = x.beta * (x.v[i] - pk);
            s[i] = d + x.k * u;
            const int row = row0 + SLOTS * i;
            if (keep) __builtin_nontemporal_store(s[i], &Kp[row * (D / 4) + kq]);
            if (kq == 0) io<TO>::store(out, ((size_t)tok * H + h) * D + row, pq + qk * u);
        }
    }
}

template <int D, typename TI, typename TB, typename TO>
hipError_t launch_t(const RecurrentArgs &a) {
    constexpr int NT = D == 128 ? 512 : 256, R = 4, SPLIT = D / (R * NT / (D / 4));
    hipLaunchKernelGGL((recurrent_kernel<D, NT, R, TI, TB, TO>), dim3((unsigned)(a.N * a.H * SPLIT)), dim3(NT), 0,
                       a.stream, static_cast<const TI *>(a.q), static_cast<const TI *>(a.k),
                       static_cast<const TI *>(a.v), a.g, static_cast<const TB *>(a.beta), a.S,
                       static_cast<TO *>(a.out), a.cu, a.slot_in, a.slot_out, a.N, a.T, a.H, a.slots, a.g_head,
                       a.qk_norm, a.norm_eps, a.zero_rows);
    return hipGetLastError();
}

template <int D, typename TI, typename TB>
hipError_t launch_o(const RecurrentArgs &a) {
    return a.out_dt == Dt::F32 ? launch_t<D, TI, TB, float>(a) : launch_t<D, TI, TB, bf16_t>(a);
}

template <int D, typename TI>
hipError_t launch_b(const RecurrentArgs &a) {
    return a.beta_dt == Dt::F32 ? launch_o<D, TI, float>(a) : launch_o<D, TI, bf16_t>(a);
}

template <int D>
hipError_t launch_i(const RecurrentArgs &a) {
    return a.io == Dt::F32 ? launch_b<D, float>(a) : launch_b<D, bf16_t>(a);
}

}  // namespace

bool recurrent_fits(int N, int H, int Dk) {
    return (unsigned long long)N * H * (Dk * Dk / 16) < (1ull << 32);    // sixteen values of a state per thread
}

hipError_t launch_recurrent(const RecurrentArgs &a) { return a.Dk == 64 ? launch_i<64>(a) : launch_i<128>(a); }

}  // namespace kda
