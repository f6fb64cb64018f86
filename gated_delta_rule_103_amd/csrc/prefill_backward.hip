// prefill_backward.hip -- the gradient of the chunked gated delta rule.
//
// Forward, per chunk of C = 64 tokens with start state M = S^T, a the
// cumulative log-decay inside the chunk, b = beta and
//     A[t,s] = sum_c k_t k_s exp(a_t - a_s) (s < t),  P[t,s] = sum_c q_t k_s exp(a_t - a_s) (s <= t)
//     Qd = q exp(a),  Kd = k exp(a),  Kr = k exp(a_last - a),  gam = exp(a_last):
//     E = (I + A Diag(b))^-1 (V - Kd M),  U = b E,  O = Qd M + P U,  M' = gam M + Kr^T U
// (E is the error v - S' k of every token). Reverse mode, with dM' the gradient
// of the state behind the chunk:
//     Y  = (I + Diag(b) A)^-T (P^T dO + Kr dM'),  dV = b Y,  dbeta = rowsum(Y E)
//     dM = gam dM' + Qd^T dO - Kd^T dV
//     dP = tril(dO U^T),  dA = -stril(dV U^T)
//     dq_t = exp(a_t) (dO M^T)_t + sum_s dP[t,s] exp(a_t - a_s) k_s
//     dk_t = -exp(a_t) (dV M^T)_t + exp(a_last - a_t) (U dM'^T)_t
//            + sum_s dA[t,s] exp(a_t - a_s) k_s + sum_s exp(a_s - a_t) (dA[s,t] k_s + dP[s,t] q_s)
// A decay g_i is passed by everything that joins a token before i to one at or
// behind it. With row_t = what token t receives (q dq + k dk of the terms that
// carry +a_t) less what it sends inside the chunk, and out_t = k_t times the
// Kr term,
//     dg_i = sum_{t >= i} row_t + sum_{t < i} out_t + gam sum_j M dM'
// where the s = t terms of P, which no decay touches, stay out of row.
//
// With TE and TY the inverses of I + A Diag(b) and I + Diag(b) A, the recurrences are
//     E = TE V - (TE Kd) M,   Y = (P TY)^T dO + (TY^T Kr) dM',
// every matrix but the state known beforehand: the state passes through one product
// before U (dV) and one after it. That took the scans from 572 to 510 us for 45 us more
// in prep (a second product through TE or TY costs the scan a barrier and 24 matrix
// instructions a chunk).
//
// Three kernels (times: 8192 tokens x 32 heads x 128 channels, bf16; average and range of
// 60 launches under the profiler, where they take a little longer than in a call of
// 1.17-1.23 ms among others):
//   prep    every (chunk, head): P, A, both inverses and the matrices above to a
//           record. 274 us (261-358); 0.27 GB in, 0.76 GB out (3.8 TB/s), matrix units busy
//           34%, vector units 43% of the time, between barriers that two workgroups a CU
//           cover for each other
//   scan    every (sequence, head, 16 or 32 value channels), once forwards for M
//           and E and once backwards for dM' and Y. Value channels never meet in
//           either recurrence, and neither needs the other, so both run in one
//           launch. 500 us (468-653); 0.92 GB in, 0.81 GB out (3.5 TB/s), matrix units 23%,
//           vector units 30%, one wavefront a SIMD: a chain's chunks wait for one another
//   finish  every (chunk, head, 64 key channels): all gradients but dS0 from M,
//           dM', E and Y. 494 us (468-641); bound by instruction issue: vector instructions
//           43% and matrix instructions 40% of the cycles at two wavefronts a SIMD;
//           1.15 GB in, 0.34 GB out (3.0 TB/s)
//
// The call's floor is 145 us for inputs and outputs (739 MB at 5.1 TB/s); chunks of 64
// tokens leave 0.8 GB of states beside them, each written and read once.
//
// All products have fp32 operands and accumulation (fp32 MFMA, or the bf16 matrix
// cores with operands cut in three): gradients arrive in any magnitude, dg is a
// difference of sums that nearly cancel inside a chunk, and dg and dS0 leave in
// fp32.
//
// Exponents. exp(a_t - a_s) is split where the tokens part in a binary tree over
// the chunk: blocks of 16, halves of 8, groups of 4. With the border between
// t's and s's subtrees it is exp(sum from the border to t) exp(sum from s to the
// border), both summed directly (never as a difference of long sums), so
// every exponent is <= 0 and good to its own rounding: what is not negligible has
// a short exponent. Inside a group the three single decays and their products
// serve. Decays are cut at -104, below which exp is 0 in fp32 (g = -inf wipes a
// channel).
//
// MFMA 16x16x4 operands. Lane l holds A[l % 16][l / 16], B[l / 16][l % 16] and
// accumulator rows 4 (l / 16) + r of column l % 16. The order of the inner
// index is free, so four MFMAs take one float4 from each side: MFMA e sums the
// inner indices 4 (l / 16) + e. An accumulator is then at once a B operand of
// the next product along its rows, which finish and prep use, and the states
// and E, Y go to memory as whole accumulators (1 KB per wavefront store) in the
// order in which finish reads them as operands.
#include "../../include/kda.h"

#include "kda_chunks.h"
#include "kda_device.h"
#include "kda_launch.h"

#include <cstddef>
#include <type_traits>

namespace kda {
namespace {

typedef uint32_t u32v2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32v4 __attribute__((ext_vector_type(4)));

constexpr int C = 64, BT = 16, NB = C / BT;   // chunk, block of tokens, blocks
constexpr int LP = C + 4;                     // LDS row stride of a C x C matrix
constexpr float MIN_G = -104.f;
// the block tiles on and below the diagonal of a lower triangular C x C matrix
constexpr int TILES = NB * (NB + 1) / 2;
__device__ __forceinline__ constexpr int tile_of(int bi, int bj) { return bi * (bi + 1) / 2 + bj; }

__device__ __forceinline__ f32x4 mfma16(f32x4 a, f32x4 b, f32x4 acc) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], acc, 0, 0, 0);
    return acc;
}

// Round to nearest even by the conversion instruction (f32_to_bf16 tests for NaN with a
// branch, which 48 stores per lane feel).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ uint16_t round_bf16(float a) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(a)); }

// x of another lane of the same 16: lane 15 - i, 7 - i (in its eight), i ^ 2, i ^ 1
template <int M> __device__ __forceinline__ float lane_across(float x) {
    constexpr int ctrl = M == 8 ? 0x140 : M == 4 ? 0x141 : M == 2 ? 0x4e : 0xb1;
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), ctrl, 0xf, 0xf, true));
}
// fp32 products on the bf16 matrix cores. A value x is cut into three bf16 parts of
// eight significand bits each, x = h + m + l, exactly. Of the nine products of two values
// the three smallest (m l, l m, l l) are left out. On one side of every product h and m are
// rounded to nearest, so |m| <= 2^-8 |x| and |l| <= 2^-17 |x| and both have either sign; on
// the other they may be truncated, |m| < 2^-7 |x| and |l| < 2^-15 |x|, which takes less. What
// is left out is then at most 2^-23 + 2^-24 of the whole and 0 on average, an fp32
// product's own rounding twice or so; six of nine products take 6 / 16 of fp32 MFMA's time
// (3 / 16 where one side is bf16 already). With both sides truncated it would be up to
// 8 x 2^-24, always downwards; with both rounded 2^-24, for 4% of the packed gradient's
// time (265 -> 274 us). (A value that rounds beyond bf16's largest, 3.39e38, is not cut.)
// MFMA 16x16x32: a lane holds row (column) l % 16 and eight inner indices of its
// lane group l / 16; two float4 of neighbouring 16-wide tiles make one operand.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ uint32_t high_halves(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float high_value(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// The first bf16 part of a and of b, rounded with NEAR and truncated without; a and b keep
// what it leaves. With DOT, x - h is one
// instruction, h still packed: a dot product of the pair with (-1, 0) or (0, -1) onto
// x, exact like the subtraction. It is used where operands of many products are cut
// at once (8k gradient 1284 -> 1259 us); where few values are cut and used at once,
// in the scan of 16 channels, its latency costs more (packed gradient 266 -> 272 us).
template <bool NEAR, bool DOT> __device__ __forceinline__ uint32_t cut_pair(float &a, float &b) {
#pragma clang fp contract(off)                         // x is the product's rounded value in every variant
    const uint32_t h = NEAR ? pack_bf16(a, b) : high_halves(a, b);
    if constexpr (DOT) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        uint32_t first = 0xbf80u, second = 0xbf800000u;
        asm("" : "+s"(first), "+s"(second));           // as an immediate the first would reach the wrong half
        const bf16x2 hv = __builtin_bit_cast(bf16x2, h);
        a = __builtin_amdgcn_fdot2_f32_bf16(hv, __builtin_bit_cast(bf16x2, first), a, false);
        b = __builtin_amdgcn_fdot2_f32_bf16(hv, __builtin_bit_cast(bf16x2, second), b, false);
    } else {
        a -= NEAR ? __uint_as_float(h << 16) : high_value(__float_as_uint(a));
        b -= high_value(NEAR ? h : __float_as_uint(b));
    }
    return h;
}
// Part z of a pair, taken in turn: what two parts leave has eight bits.
template <bool NEAR, bool DOT> __device__ __forceinline__ uint32_t part_of(int z, float &a, float &b) {
    return z < 2 ? cut_pair<NEAR, DOT>(a, b) : high_halves(a, b);
}
template <bool NEAR, bool DOT> __device__ __forceinline__ void split3(f32x4 a, f32x4 b, u32v4 (&p)[3]) {
    float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int z = 0; z < 3; ++z)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[z][i] = part_of<NEAR, DOT>(z, x[2 * i], x[2 * i + 1]);
}
__device__ __forceinline__ f32x4 mfma32(u32v4 a, u32v4 b, f32x4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}
template <int PA> __device__ __forceinline__ f32x4 product(const u32v4 (&a)[PA], const u32v4 (&b)[3], f32x4 acc) {
    acc = mfma32(a[0], b[2], acc);                     // small terms first
    if constexpr (PA == 3) {
        acc = mfma32(a[2], b[0], acc);
        acc = mfma32(a[1], b[1], acc);
    }
    acc = mfma32(a[0], b[1], acc);
    if constexpr (PA == 3) acc = mfma32(a[1], b[0], acc);
    return mfma32(a[0], b[0], acc);
}

// One step of summing 2 M values over 16 lanes: each lane keeps M of them, those
// of its bit M, and adds what the lane across kept for it.
template <int M> __device__ __forceinline__ void halve(float *v, int lane) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const bool up = lane & M;
        const float keep = up ? v[i + M] : v[i], give = up ? v[i] : v[i + M];
        v[i] = keep + lane_across<M>(give);
    }
}

// The sums of v[0..15] over the 16 lanes of a row: lane l of them gets that of v[l]. Fifteen
// exchanges instead of 64 (and in prep no second reading of q and k for their norms): the
// gradient of 4 x 1000 tokens x 16 heads x 64 with normalised q and k 184 -> 159 us,
// 8192 tokens x 32 heads x 128 1573 -> 1468 us.
__device__ __forceinline__ float sums16(float (&v)[16], int lane) {
    halve<8>(v, lane);
    halve<4>(v, lane);
    halve<2>(v, lane);
    halve<1>(v, lane);
    return v[0];
}

// Keeps the computation of x before what follows: without it the compiler sinks
// whole chains of products towards their uses and holds all their operands.
__device__ __forceinline__ void settle(f32x4 &x) { asm volatile("" : "+v"(x)); }
__device__ __forceinline__ void settle(float &x) { asm volatile("" : "+v"(x)); }

__device__ __forceinline__ void store4(float *p, f32x4 x) { *reinterpret_cast<f32x4 *>(p) = x; }
// what a later kernel reads, from memory by then
__device__ __forceinline__ void store4_far(float *p, f32x4 x) { __builtin_nontemporal_store(x, reinterpret_cast<f32x4 *>(p)); }
__device__ __forceinline__ f32x4 ld4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
// four values `stride` apart
__device__ __forceinline__ f32x4 ld4s(const float *p, int stride) {
    return f32x4{p[0], p[stride], p[2 * stride], p[3 * stride]};
}

// What prep leaves for a (chunk, head), in floats. Operands lie in the order in
// which the scans load them, 1 KB per wavefront and instruction:
//   R (rows):    float4 l of (token block, 16 channels): token l % 16, channels 4 (l / 16) + 0..3
//   T (columns): float4 l of (16 channels, token block): channel l % 16, tokens 4 (l / 16) + 0..3
//   lower triangular C x C matrices: the ten tiles on and below the diagonal,
//   float4 l: row l % 16, columns 4 (l / 16) + 0..3, or transposed the reverse
template <int D> struct Rec {
    static constexpr size_t WR = 0, KRT = WR + C * D, TE = KRT + C * D,      // the forward scan's: -TE Kd, Kr, TE
        XR = TE + TILES * 256, KDT = XR + C * D, QDT = KDT + C * D,          // the backward scan's: TY^T Kr, Kd, Qd
        ZT = QDT + C * D,                                                    // and (P TY)^T
        GAM = ZT + TILES * 256,                                         // [D]
        RQ = GAM + D, RK = RQ + C,                                      // 1 / norms of q and k [C]
        SIZE = RK + C;
};

// block row and column of tile i
__device__ __forceinline__ void tile_at(int i, int &bi, int &bj) {
    i = min(i, TILES - 1);
    bi = i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3;
    bj = i - bi * (bi + 1) / 2;
}

struct Ws {
    int32_t *cut, *chunk_off;
    float *rec, *M, *dM, *E, *Y;
};

struct Common {
    SeqView sv;
    Ws ws;
    const float *g;
    int H, slots;             // heads; workspace slots of a head, one per chunk
    bool g_head, qk_norm;
    float norm_eps;
    int zero_rows;            // KDA_ZERO_*: gradients whose rows of no sequence are set to zero
};

// A (chunk, head) and its tokens: the first one's row of [T_total][H] tensors,
// rows p.H apart; offsets inside a chunk fit 32 bits.
struct Item {
    int Lc;
    size_t row0;
    size_t slot;              // in the workspace: chunks of a head lie one behind the other, which
                              // keeps a scan inside few memory pages
    __device__ bool find(const Common &p, size_t item) {
        const int ci = (int)(item / p.H), h = (int)(item % p.H);
        if (ci >= p.sv.total_chunks()) return false;
        const int n = p.sv.seq_of_chunk(ci);
        const int s0 = p.sv.seq_start(n) + (ci - p.sv.first_chunk(n)) * C;
        Lc = min(C, p.sv.seq_end(n) - s0);
        row0 = (size_t)s0 * p.H + h;
        slot = (size_t)h * p.slots + ci;
        return true;
    }
};

// The rows of one (chunk, head) in a [T_total][H][width] tensor, through a buffer
// descriptor whose range ends with the chunk's last row: elements of later rows
// read as 0 and are not written, without a branch. Indices are in elements.
template <typename T> struct Rows {
    __amdgpu_buffer_rsrc_t r;
    int row;
    __device__ Rows(const T *base, const Item &it, int H, int width)
        : r(buf_rsrc(base ? base + it.row0 * width : nullptr,
                     base ? ((it.Lc - 1) * H * width + width) * (int)sizeof(T) : 0)),
          row(H * width) {}
    // one element and four as they are in memory, for a load that is used later
    typedef std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t> Raw;
    typedef std::conditional_t<sizeof(T) == 4, u32v4, u32v2> Raw4;
    __device__ Raw raw(int tau, int c) const {
        const int off = (tau * row + c) * (int)sizeof(T);
        if constexpr (sizeof(T) == 4) return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
        else return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    }
    __device__ Raw4 raw4(int tau, int c) const {
        const int off = (tau * row + c) * (int)sizeof(T);
        if constexpr (sizeof(T) == 4) return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
        else return __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
    }
    __device__ static float value(Raw u) {
        if constexpr (sizeof(T) == 4) return __uint_as_float(u);
        else return bf16_to_f32(u);
    }
    __device__ static f32x4 value4(Raw4 u) {
        if constexpr (sizeof(T) == 4) {
            return __builtin_bit_cast(f32x4, u);
        } else {
            return f32x4{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xffff0000u),
                         __uint_as_float(u[1] << 16), __uint_as_float(u[1] & 0xffff0000u)};
        }
    }
    __device__ float at(int tau, int c) const { return value(raw(tau, c)); }
    __device__ void put(int tau, int c, float x) const {
        const int off = (tau * row + c) * (int)sizeof(T);
        if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), r, off, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b16(round_bf16(x), r, off, 0, 0);
    }
    __device__ void put16(int tau, int c, u32v4 x) const {      // 16 bytes as they are
        __builtin_amdgcn_raw_buffer_store_b128(x, r, (tau * row + c) * (int)sizeof(T), 0, 0);
    }
    __device__ void put4(int tau, int c, f32x4 x) const {
        const int off = (tau * row + c) * (int)sizeof(T);
        if constexpr (sizeof(T) == 4) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32v4, x), r, off, 0, 0);
        } else {
            __builtin_amdgcn_raw_buffer_store_b64(u32v2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])}, r, off, 0, 0);
        }
    }
};

// Log-decays of a chunk's tokens (0 without a gate and behind the last token).
struct Decay {
    Rows<float> g;
    int col;                  // 1, or 0 for a gate per head
    __device__ Decay(const Common &p, const Item &it, int D)
        : g(p.g, it, p.H, p.g_head ? 1 : D), col(p.g_head ? 0 : 1) {}
    __device__ float at(int tau, int c) const { return cut(g.at(tau, c * col)); }
    __device__ static float cut(float x) { return x < MIN_G ? MIN_G : x; }      // NaN stays
};

// ---- plan -----------------------------------------------------------------

// Packed offsets, cut so that they rise and stay inside the T rows, and how many
// chunks lie before each sequence. The device's own copy: no offset that a caller
// leaves there can lead a kernel outside its buffers.
__global__ __launch_bounds__(256) void plan_kernel(const int32_t *__restrict__ cu, int N, int T, int32_t *cut,
                                                   int32_t *chunk_off) {
    __shared__ int32_t part[4];
    const int t = threadIdx.x, per = N / 256 + 1;
    const int lo = min(N + 1, t * per), hi = min(N + 1, lo + per);
    // what `op` makes of the threads' x before this one (0 for none)
    auto before = [&](int32_t x, auto op) {
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int32_t y = __shfl_up(x, o, 64);
            if ((t & 63) >= o) x = op(x, y);
        }
        __syncthreads();
        if ((t & 63) == 63) part[t >> 6] = x;
        __syncthreads();
        x = __shfl_up(x, 1, 64);
        if ((t & 63) == 0) x = 0;
        for (int i = 0; i < t >> 6; ++i) x = op(x, part[i]);
        return x;
    };
    auto larger = [](int32_t a, int32_t b) { return max(a, b); };
    int32_t top = 0;
    for (int n = lo; n < hi; ++n) top = max(top, min(cu[n], T));
    top = before(top, larger);
    for (int n = lo; n < hi; ++n) cut[n] = top = max(top, min(cu[n], T));
    __syncthreads();
    // chunks of sequence n, which ends at offset n + 1
    auto chunks = [&](int n) { return n < N ? (cut[n + 1] - cut[n] + C - 1) / C : 0; };
    int32_t sum = 0;
    for (int n = lo; n < hi; ++n) sum += chunks(n);
    sum = before(sum, [](int32_t a, int32_t b) { return a + b; });
    for (int n = lo; n < hi; ++n) {
        chunk_off[n] = sum;
        sum += chunks(n);
    }
}

// ---- prep -----------------------------------------------------------------

constexpr int TP = 20;                        // LDS row stride of a block tile
typedef float Tile[BT][TP];

// Thread (blk, c) owns channel c of the 16 tokens of block blk and forms every
// decay there by itself. The products over channels run half a head (64
// channels) at a time through the three staging tiles, which keeps two
// workgroups on a CU.
template <int D>
struct PrepLds {
    float X[3][C][64 + 4];
    Tile A[TILES], P[TILES];
    float dec[NB][D];                 // decay over a whole block
    float b[C], rq[C], rk[C];
};

template <int D, typename TI, typename TB>
__global__ __launch_bounds__(4 * D, D == 128 ? 4 : 2) void prep_kernel(Common p, const TI *__restrict__ q,
                                                                      const TI *__restrict__ k,
                                                                      const TB *__restrict__ beta) {
    using R = Rec<D>;
    constexpr int THREADS = 4 * D, NW = D / 16, HALVES = D / 64;
    extern __shared__ char lds_raw[];
    PrepLds<D> &s = *reinterpret_cast<PrepLds<D> *>(lds_raw);
    Item it;
    if (!it.find(p, blockIdx.x)) return;
    float *rec = p.ws.rec + it.slot * R::SIZE;
    const int t = threadIdx.x, w = t / 64, l = t % 64, lr = l % 16, lg = l / 16;
    const int c = t % D, blk = t / D, ch = c % 64;
    const Rows<TI> qr(q, it, p.H, D), kr(k, it, p.H, D);
    const Decay decay(p, it, D);

    float kv[BT], qv[BT], gv[BT];
#pragma unroll
    for (int i = 0; i < BT; ++i) {
        kv[i] = kr.at(blk * BT + i, c);
        qv[i] = qr.at(blk * BT + i, c);
        gv[i] = decay.at(blk * BT + i, c);
    }
    if (t < C) s.b[t] = Rows<TB>(beta, it, p.H, 1).at(t, 0);
    for (int i = t; i < TILES * BT * TP; i += THREADS) (&s.A[0][0][0])[i] = (&s.P[0][0][0])[i] = 0.f;
    if (p.qk_norm) {
        // squares summed over the wavefront's 64 channels, then over the wavefronts of the block
        float(*sums)[2][BT] = reinterpret_cast<float(*)[2][BT]>(&s.X[0][0][0]);
        auto squares = [&](const float(&x)[BT], int which) {
            float y[BT];
#pragma unroll
            for (int i = 0; i < BT; ++i) y[i] = x[i] * x[i];
            float z = sums16(y, l);
            z += __shfl_xor(z, 16, 64);
            z += __shfl_xor(z, 32, 64);
            if (l < BT) sums[w][which][l] = z;
        };
        squares(qv, 0);
        squares(kv, 1);
        __syncthreads();
        if (t < 2 * C) {
            const int which = t / C, tau = t % C, b = tau / BT;
            float x = sums[b * HALVES][which][tau % BT];
            if (HALVES == 2) x += sums[b * HALVES + HALVES - 1][which][tau % BT];
            x = 1.f / sqrtf(x + p.norm_eps);
            (which ? s.rk : s.rq)[tau] = x;
            rec[(which ? R::RK : R::RQ) + tau] = x;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < BT; ++i) {
            kv[i] *= s.rk[blk * BT + i];
            qv[i] *= s.rq[blk * BT + i];
        }
    }
    float G[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) G[j] = (gv[4 * j] + gv[4 * j + 1]) + (gv[4 * j + 2] + gv[4 * j + 3]);
    s.dec[blk][c] = __expf((G[0] + G[1]) + (G[2] + G[3]));

    float(*part)[64] = reinterpret_cast<float(*)[64]>(&s.X[0][0][0]);    // one row per wavefront
    // Pairs inside groups of four: ten products for P, six for A, summed over the
    // wavefront's channels. The 16 values of a group are halved lane by lane, so
    // that lane l ends with the sum of value l % 16.
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int o = 4 * j;
        const float e10 = __expf(gv[o + 1]), e21 = __expf(gv[o + 2]), e32 = __expf(gv[o + 3]);
        const float e20 = e21 * e10, e31 = e32 * e21, e30 = e32 * e20;
        const float k0 = kv[o], k1 = kv[o + 1], k2 = kv[o + 2], k3 = kv[o + 3];
        const float q1 = qv[o + 1], q2 = qv[o + 2], q3 = qv[o + 3];
        float v[16] = {qv[o] * k0,      q1 * (e10 * k0), q1 * k1,         q2 * (e20 * k0), q2 * (e21 * k1), q2 * k2,
                       q3 * (e30 * k0), q3 * (e31 * k1), q3 * (e32 * k2), q3 * k3,         k1 * (e10 * k0), k2 * (e20 * k0),
                       k2 * (e21 * k1), k3 * (e30 * k0), k3 * (e31 * k1), k3 * (e32 * k2)};
        float x = sums16(v, l);
        x += __shfl_xor(x, 16, 64);
        x += __shfl_xor(x, 32, 64);
        settle(x);
        if (l < 16) part[w][16 * j + l] = x;
    }
    __syncthreads();

    if (t < 64 * NB) {                                  // in-group products into the diagonal tiles
        const int b = t / 64, e = t % 16, o = 4 * (l / 16);
        float x = part[b * HALVES][l];
        if (HALVES == 2) x += part[b * HALVES + HALVES - 1][l];
        const int pr = e < 1 ? 0 : e < 3 ? 1 : e < 6 ? 2 : 3, ar = e < 11 ? 1 : e < 13 ? 2 : 3;
        if (e < 10) s.P[tile_of(b, b)][o + pr][o + e - pr * (pr + 1) / 2] = x;
        else s.A[tile_of(b, b)][o + ar][o + e - 10 - ar * (ar - 1) / 2] = x;
    }

    // Pairs of different blocks: row factor exp(sum from the block's start),
    // column factor exp(sum to the block's end), whole blocks between on the rows.
    constexpr int JOBS = (12 + NW - 1) / NW;
    f32x4 acc[JOBS];
#pragma unroll
    for (int i = 0; i < JOBS; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int hf = 0; hf < HALVES; ++hf) {
        __syncthreads();
        if (c / 64 == hf) {
            float run = 0.f;
            settle(run);                                // or both halves' decays are formed ahead of the loop
#pragma unroll
            for (int i = 0; i < BT; ++i) {
                run += gv[i];
                const float e = __expf(run);
                s.X[0][blk * BT + i][ch] = kv[i] * e;
                s.X[2][blk * BT + i][ch] = qv[i] * e;
            }
            run = 0.f;
#pragma unroll
            for (int i = BT - 1; i >= 0; --i) {
                s.X[1][blk * BT + i][ch] = kv[i] * __expf(run);
                run += gv[i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < JOBS; ++i) {
            const int job = w + i * NW, pr = job >> 1;
            if (job < 12) {
                const int bi = pr < 1 ? 1 : pr < 3 ? 2 : 3, bj = pr - bi * (bi - 1) / 2;
                const float(*rows)[64 + 4] = s.X[job & 1 ? 2 : 0] + 16 * bi, (*cols)[64 + 4] = s.X[1] + 16 * bj;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const int x = 16 * kk + 4 * lg;
                    f32x4 a = ld4(&rows[lr][x]);
                    if (bi - bj > 1) a *= ld4(&s.dec[bj + 1][64 * hf + x]);
                    if (bi - bj > 2) a *= ld4(&s.dec[bj + 2][64 * hf + x]);
                    acc[i] = mfma16(a, ld4(&cols[lr][x]), acc[i]);
                }
            }
        }
        // Qd from its staging tile, the decay of whole blocks before comes in
        const int tt = w % NB;                          // this wavefront's token block
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) {
            if (NW == 8 && (ct & 1) != w / NB) continue;
            const int x = 16 * ct + lr, at = (((4 * hf + ct) * NB + tt) * 64 + l) * 4;
            const float d0 = s.dec[0][64 * hf + x], d1 = s.dec[1][64 * hf + x], d2 = s.dec[2][64 * hf + x];
            const float f0 = tt == 0 ? 1.f : tt == 1 ? d0 : tt == 2 ? d0 * d1 : d0 * d1 * d2;
            store4_far(rec + R::QDT + at, ld4s(&s.X[2][16 * tt + 4 * lg][x], 64 + 4) * f0);
        }
    }
#pragma unroll
    for (int i = 0; i < JOBS; ++i) {
        const int job = w + i * NW, pr = job >> 1;
        if (job < 12) {
            const int bi = pr < 1 ? 1 : pr < 3 ? 2 : 3, bj = pr - bi * (bi - 1) / 2;
            Tile &out = job & 1 ? s.P[tile_of(bi, bj)] : s.A[tile_of(bi, bj)];
#pragma unroll
            for (int r = 0; r < 4; ++r) out[4 * lg + r][lr] = acc[i][r];
        }
    }

    // Pairs of the halves of a block (staging tile 0) and of the group pairs of a
    // half (tile 1): rows of the later part carry exp(sum from its start), rows
    // of the earlier exp(sum to its end). One MFMA tile gives A (rows 0-7) and P
    // (rows 8-15, q in tile 2: later halves, then later groups).
    constexpr int JOBS2 = 8 / NW;
    f32x4 acc2[JOBS2];
#pragma unroll
    for (int i = 0; i < JOBS2; ++i) acc2[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int hf = 0; hf < HALVES; ++hf) {
        __syncthreads();
        if (c / 64 == hf) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float pre[4], suf[4];
                pre[0] = gv[4 * j];
                suf[3] = 0.f;
                settle(pre[0]);
                settle(suf[3]);
#pragma unroll
                for (int i = 1; i < 4; ++i) pre[i] = pre[i - 1] + gv[4 * j + i];
#pragma unroll
                for (int i = 2; i >= 0; --i) suf[i] = suf[i + 1] + gv[4 * j + i + 1];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int x = 4 * j + i, tau = blk * BT + x;
                    // within the half: from its start (later half) or to its end (earlier half)
                    const float e8 = __expf(j == 3 ? G[2] + pre[i] : j == 2 ? pre[i] : j == 1 ? suf[i] : suf[i] + G[1]);
                    const float e4 = __expf(j & 1 ? pre[i] : suf[i]);
                    s.X[0][tau][ch] = kv[x] * e8;
                    s.X[1][tau][ch] = kv[x] * e4;
                    if (j >= 2) s.X[2][8 * blk + x - 8][ch] = qv[x] * e8;
                    if (j & 1) s.X[2][32 + 8 * blk + (j >> 1) * 4 + i][ch] = qv[x] * e4;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < JOBS2; ++i) {
            const int job = w + i * NW, b = job >> 1, four = job & 1, r8 = lr & 7;
            const int row = four ? (r8 < 4 ? 4 + r8 : 8 + r8) : 8 + r8, col = four ? (r8 < 4 ? r8 : 4 + r8) : r8;
            const float *rp = lr < 8 ? s.X[four][16 * b + row] : s.X[2][32 * four + 8 * b + r8];
            const float *cp = s.X[four][16 * b + col];
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                acc2[i] = mfma16(ld4(rp + 16 * kk + 4 * lg), ld4(cp + 16 * kk + 4 * lg), acc2[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < JOBS2; ++i) {
        const int job = w + i * NW, b = job >> 1, four = job & 1;
        Tile &out = lg < 2 ? s.A[tile_of(b, b)] : s.P[tile_of(b, b)];
        const int part = lg & 1;                        // rows 0-3 or 4-7 of the later part
        if (lr < 8 && (!four || (lr >> 2) == part)) {
            const int row = four ? 4 + 8 * part : 8 + 4 * part, col = four ? (lr < 4 ? lr : 4 + lr) : lr;
#pragma unroll
            for (int r = 0; r < 4; ++r) out[row + r][col] = acc2[i][r];
        }
    }
    __syncthreads();

    // (I + A Diag(b))^-1 in the staging tiles' place: the diagonal blocks by
    // substitution, one column per lane
    Tile *X = reinterpret_cast<Tile *>(&s.X[0][0][0]);
    if (w < NB && l < 16) {
        const Tile &a = s.A[tile_of(w, w)];
        Tile &xt = X[tile_of(w, w)];
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i == l ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) v -= a[i][j] * x[j];
            xt[i][l] = v;
            x[i] = v * s.b[16 * w + i];
        }
    }
    __syncthreads();
    // block row bi, column bj: -X_ii sum_k (A Diag(b))_ik X_kj, by distance from the diagonal
#pragma unroll 1
    for (int d = 1; d < NB; ++d) {
        if (w < NB - d) {
            const int bj = w, bi = w + d;
            f32x4 sum = {0.f, 0.f, 0.f, 0.f}, res = sum;
            for (int bk = bj; bk < bi; ++bk)
                sum = mfma16(ld4(&s.A[tile_of(bi, bk)][lr][4 * lg]) * ld4(&s.b[16 * bk + 4 * lg]),
                             ld4s(&X[tile_of(bk, bj)][4 * lg][lr], TP), sum);
            res = mfma16(ld4(&X[tile_of(bi, bi)][lr][4 * lg]), -sum, res);
#pragma unroll
            for (int r = 0; r < 4; ++r) X[tile_of(bi, bj)][4 * lg + r][lr] = res[r];
        }
        __syncthreads();
    }
    // TY = (I + Diag(b) A)^-1 = I - Diag(b) X A, in A's place, its tiles transposed
    constexpr int OWN = (TILES + NW - 1) / NW;
    f32x4 ty[OWN];
#pragma unroll
    for (int n = 0; n < OWN; ++n) {
        int bi, bj;
        tile_at(w + n * NW, bi, bj);
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int bk = bj; bk <= bi; ++bk)
            sum = mfma16(ld4(&X[tile_of(bi, bk)][lr][4 * lg]), ld4s(&s.A[tile_of(bk, bj)][4 * lg][lr], TP), sum);
        const int row = 16 * bi + 4 * lg, col = 16 * bj + lr;
#pragma unroll
        for (int r = 0; r < 4; ++r) ty[n][r] = (row + r == col ? 1.f : 0.f) - s.b[row + r] * sum[r];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < OWN; ++n)
        if (w + n * NW < TILES) store4(&s.A[w + n * NW][lr][4 * lg], ty[n]);
    // Kd and Kr again, 64 channels at a time: out by columns, and times X and TY
#pragma unroll 1
    for (int hf = 0; hf < HALVES; ++hf) {
        if (hf) __syncthreads();
        if (c / 64 == hf) {
            const float d0 = s.dec[0][c], d1 = s.dec[1][c], d2 = s.dec[2][c], d3 = s.dec[3][c];
            const float f0 = blk == 0 ? 1.f : blk == 1 ? d0 : blk == 2 ? d0 * d1 : d0 * d1 * d2;
            const float f1 = blk == 3 ? 1.f : blk == 2 ? d3 : blk == 1 ? d2 * d3 : d1 * d2 * d3;
            float run = 0.f;
            settle(run);
#pragma unroll
            for (int i = 0; i < BT; ++i) {
                run += gv[i];
                s.X[1][blk * BT + i][ch] = kv[i] * (__expf(run) * f0);
            }
            run = 0.f;
#pragma unroll
            for (int i = BT - 1; i >= 0; --i) {
                s.X[2][blk * BT + i][ch] = kv[i] * (__expf(run) * f1);
                run += gv[i];
            }
        }
        __syncthreads();
        if (hf == 0) {
            for (int i = w; i < TILES; i += NW) {
                int bi, bj;
                tile_at(i, bi, bj);
                f32x4 z = {0.f, 0.f, 0.f, 0.f};
                for (int bk = bj; bk <= bi; ++bk)
                    z = mfma16(ld4(&s.P[tile_of(bi, bk)][lr][4 * lg]), ld4(&s.A[tile_of(bk, bj)][lr][4 * lg]), z);
                store4_far(rec + R::ZT + (i * 64 + l) * 4, z);
                store4_far(rec + R::TE + (i * 64 + l) * 4, ld4(&X[i][lr][4 * lg]));
            }
        }
        // a wavefront has 16 channels, and with eight of them two token blocks of four:
        // the first and last or the middle ones, which are the same work
        const int x = 16 * (w % 4) + lr, at = 4 * hf + w % 4;
        f32x4 kd[NB], kr[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            kd[b] = ld4s(&s.X[1][16 * b + 4 * lg][x], 64 + 4);
            kr[b] = ld4s(&s.X[2][16 * b + 4 * lg][x], 64 + 4);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (NW == 8 && (b == 0 || b == NB - 1) != (w < 4)) continue;
            store4_far(rec + R::KDT + ((at * NB + b) * 64 + l) * 4, kd[b]);
            store4_far(rec + R::KRT + ((at * NB + b) * 64 + l) * 4, kr[b]);
            f32x4 y = {0.f, 0.f, 0.f, 0.f}, z = y;
#pragma unroll
            for (int i = 0; i <= b; ++i) y = mfma16(kd[i], -ld4(&X[tile_of(b, i)][lr][4 * lg]), y);
#pragma unroll
            for (int i = b; i < NB; ++i) z = mfma16(kr[i], ld4(&s.A[tile_of(i, b)][lr][4 * lg]), z);
            store4_far(rec + R::WR + ((b * (D / 16) + at) * 64 + l) * 4, y);
            store4_far(rec + R::XR + ((b * (D / 16) + at) * 64 + l) * 4, z);
        }
    }
    if (t < D) rec[R::GAM + t] = (s.dec[0][t] * s.dec[1][t]) * (s.dec[2][t] * s.dec[3][t]);
}

// ---- scan -----------------------------------------------------------------

// A workgroup of four wavefronts carries TV = 16 JT value channels (rows j of S,
// the accumulators' rows) of one chain; wavefront w owns D / 4 key channels of S
// and the w-th 16 tokens of a chunk. Left operands pass through LDS cut in three
// rounded bf16 parts; right operands come from the record and are cut in registers by
// truncation, once for the JT tiles.
template <int D, int TV, int PO>
struct ScanLds {
    uint16_t S[3][TV][D + 8];         // the state
    uint16_t U[3][TV][C + 8];         // U or -dV
    uint16_t O[PO][TV][C + 8];        // V^T or dO^T
};
// Column of inner index k in those: the eight that a lane multiplies (of two
// neighbouring 16-wide tiles, four each) lie together.
__device__ __forceinline__ int inner(int k) { return (k & ~31) | (k & 12) << 1 | (k & 16) >> 2 | (k & 3); }

template <int D, int TV, typename TI, typename TB, typename TG>
__global__ __launch_bounds__(256, 2) void scan_kernel(Common p, const TI *__restrict__ v, const TB *__restrict__ beta,
                                                      const TG *__restrict__ dout, const float *__restrict__ S0,
                                                      const float *__restrict__ dS_out, float *__restrict__ dS0) {
    using R = Rec<D>;
    constexpr int PO = sizeof(TG) == 2 ? 1 : 3, JT = TV / 16;
    constexpr int NT = D / 16, CT = D / 64;      // value tiles of a chain, key tiles of a wavefront
    __shared__ __align__(16) ScanLds<D, TV, PO> s;
    // The tiles of a chain, which read the same records, run on one XCD (workgroups
    // go to the eight XCDs in turn); the backward scans, which are longer, come first.
    const int per_dir = gridDim.x / 16, slot = blockIdx.x / 8;
    const bool back = slot < per_dir;
    const int chain = (back ? slot : slot - per_dir) / (D / TV) * 8 + blockIdx.x % 8;
    if (chain >= p.sv.N * p.H) return;
    const int n = chain / p.H, h = chain % p.H;
    const int t = threadIdx.x, w = t / 64, l = t % 64, lr = l % 16, lg = l / 16;
    const int j0 = slot % (D / TV) * TV, jt = j0 / 16;   // the workgroup's first value channel and tile
    const int jr = j0 + 4 * lg;                          // this lane's first accumulator row
    const int begin = p.sv.seq_start(n), len = p.sv.seq_end(n) - begin, chunks = (len + C - 1) / C;
    const size_t item0 = (size_t)h * p.slots + p.sv.first_chunk(n);
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    auto key = [&](int i) { return (w * CT + i) * 16 + lr; };

    f32x4 st[JT][CT];
    const float *init = back ? dS_out : S0;
    const size_t state0 = ((size_t)n * p.H + h) * D;
#pragma unroll
    for (int y = 0; y < JT; ++y)
#pragma unroll
        for (int i = 0; i < CT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) st[y][i][r] = init ? init[(state0 + jr + 16 * y + r) * D + key(i)] : 0.f;

    // Operands of a chunk stay in registers from a chunk ahead: each set is
    // loaded again as soon as its products are done, and the other phases of the
    // chunk cover the latency.
    const int tau = 16 * w + lr, tau_col = inner(tau);   // this lane's token where tokens are columns
    auto item_of = [&](int step) { return item0 + (back ? chunks - 1 - step : step); };
    // an accumulator (rows 4 lg + r of tile y) into column `col` of an LDS matrix, cut in
    // three rounded parts: in pairs where two tiles' work covers the latency, one by one
    // with the same rounding by an addition else (packed gradient 267 us against 270)
    auto put = [&](auto &m, int y, int col, f32x4 x) {
#pragma clang fp contract(off)
        if constexpr (TV == 32) {
#pragma unroll
            for (int r = 0; r < 4; r += 2) {
                float f0 = x[r], f1 = x[r + 1];
#pragma unroll
                for (int z = 0; z < 3; ++z) {
                    const uint32_t u = part_of<true, true>(z, f0, f1);
                    m[z][16 * y + 4 * lg + r][col] = static_cast<uint16_t>(u);
                    m[z][16 * y + 4 * lg + r + 1][col] = static_cast<uint16_t>(u >> 16);
                }
            }
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float f = x[r];
#pragma unroll
                for (int z = 0; z < 3; ++z) {
                    uint32_t u = __float_as_uint(f);
                    if (z < 2) u += 0x7fffu + __builtin_amdgcn_ubfe(u, 16, 1);     // to nearest, ties to even
                    m[z][16 * y + 4 * lg + r][col] = static_cast<uint16_t>(u >> 16);
                    f -= high_value(u);
                }
            }
        }
    };
    // rows of tile y as a left operand over the inner indices 32 m ..
    auto left = [&](auto &m, int y, int at, auto &a) {
#pragma unroll
        for (int z = 0; z < (int)(sizeof(a) / sizeof(a[0])); ++z)
            a[z] = *reinterpret_cast<const u32v4 *>(&m[z][16 * y + lr][32 * at + 8 * lg]);
    };
    auto put_state = [&](size_t item) {
        float *Mw = (back ? p.ws.dM : p.ws.M) + item * D * D;
#pragma unroll
        for (int y = 0; y < JT; ++y)
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                store4_far(Mw + (((w * CT + i) * NT + jt + y) * 64 + l) * 4, st[y][i]);
                put(s.S, y, inner(key(i)), st[y][i]);
            }
    };
    auto rows_of = [&](f32x4(&x)[D / 16], const float *m) {           // this wavefront's tokens, all channels
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) x[kk] = ld4(m + ((w * (D / 16) + kk) * 64 + l) * 4);
    };
    auto cols_of = [&](f32x4(&x)[CT][NB], const float *m) {           // its channels, all tokens
#pragma unroll
        for (int i = 0; i < CT; ++i)
#pragma unroll
            for (int kk = 0; kk < NB; ++kk) x[i][kk] = ld4(m + (((w * CT + i) * NB + kk) * 64 + l) * 4);
    };
    auto gam_of = [&](float(&x)[CT], const float *rec) {
#pragma unroll
        for (int i = 0; i < CT; ++i) x[i] = rec[R::GAM + key(i)];
    };
    auto chunk_of = [&](int step) {
        const int ci = back ? chunks - 1 - step : step;
        return Item{min(C, len - ci * C), (size_t)(begin + ci * C) * p.H + h, item0 + ci};
    };
    auto beta_of = [&](const Item &it) { return Rows<TB>(beta, it, p.H, 1).raw(tau, 0); };
    // state times rows: S Kd^T or dS Kr^T, for this wavefront's tokens
    auto times_rows = [&](const f32x4(&x)[D / 16], f32x4(&acc)[JT]) {
#pragma unroll
        for (int m = 0; m < D / 32; ++m) {
            u32v4 b[3];
            split3<false, TV == 32>(x[2 * m], x[2 * m + 1], b);
#pragma unroll
            for (int y = 0; y < JT; ++y) {
                u32v4 a[3];
                left(s.S, y, m, a);
                acc[y] = product(a, b, acc[y]);
            }
        }
    };
    // a matrix over tokens times a triangular one: the pairs of token blocks that
    // have a block at or before (behind) this wavefront's
    auto times_tri = [&](auto &mat, const f32x4(&x)[NB], f32x4(&acc)[JT], auto parts) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
            if (back ? 2 * m + 1 >= w : 2 * m <= w) {
                u32v4 b[3];
                split3<false, TV == 32>(x[2 * m], x[2 * m + 1], b);
#pragma unroll
                for (int y = 0; y < JT; ++y) {
                    u32v4 a[decltype(parts)::value];
                    left(mat, y, m, a);
                    acc[y] = product(a, b, acc[y]);
                }
            }
    };
    // its product over the tokens with this wavefront's channels, onto the state
    auto onto_state = [&](auto &mat, const f32x4(&x)[CT][NB], auto parts) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            u32v4 a[JT][decltype(parts)::value];
#pragma unroll
            for (int y = 0; y < JT; ++y) left(mat, y, m, a[y]);
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                u32v4 b[3];
                split3<false, TV == 32>(x[i][2 * m], x[i][2 * m + 1], b);
#pragma unroll
                for (int y = 0; y < JT; ++y) st[y][i] = product(a[y], b, st[y][i]);
            }
        }
    };
    // The chain's workgroups together touch every 128-byte line of the record two
    // chunks ahead, so that it is in L2 when their operand loads are issued (8k
    // gradient 1297 -> 1278 us).
    const size_t region = back ? R::XR : 0, lines = ((back ? R::GAM : R::XR) - region) / 32;
    const size_t line = region + 32 * min((size_t)(((slot % (D / TV)) * 4 + w) * 64 + l), lines - 1);
    float touched = 0.f;
    auto touch = [&](int step) {
        settle(touched);
        touched = p.ws.rec[item_of(min(step, chunks - 1)) * R::SIZE + line];
    };
    auto tri_of = [&](f32x4(&x)[NB], const float *rec) {     // the other blocks stay zero
#pragma unroll
        for (int kk = 0; kk < NB; ++kk)
            if (back ? kk >= w : kk <= w)
                x[kk] = ld4(rec + (back ? R::ZT + (tile_of(kk, w) * 64 + l) * 4 : R::TE + (tile_of(w, kk) * 64 + l) * 4));
    };
    typedef std::integral_constant<int, 3> Three;
    // `in`: V or dO, T its type
    auto run = [&](auto direction, const auto *in) {
        constexpr bool BACK = decltype(direction)::value;
        typedef std::decay_t<decltype(*in)> T;
        typedef std::integral_constant<int, sizeof(T) == 2 ? 1 : 3> Parts;
        f32x4 rows[D / 16], tri[NB] = {zero, zero, zero, zero}, qd[CT][NB], kt[CT][NB];
        float gam[CT];
        typename Rows<T>::Raw4 ov[JT];
        typename Rows<TB>::Raw b;
        const int ot = t / 4, oj = t % 4 * 4;
        auto in_of = [&](const Item &it) {
            const Rows<T> r(in, it, p.H, D);
#pragma unroll
            for (int y = 0; y < JT; ++y) ov[y] = r.raw4(ot, j0 + 16 * y + oj);
        };
        {
            const float *rec = p.ws.rec + item_of(0) * R::SIZE;
            const Item it = chunk_of(0);
            in_of(it);
            tri_of(tri, rec);
            rows_of(rows, rec + (BACK ? R::XR : R::WR));
            if constexpr (BACK) cols_of(qd, rec + R::QDT);
            gam_of(gam, rec);
            b = beta_of(it);
            cols_of(kt, rec + (BACK ? R::KDT : R::KRT));
        }
        for (int step = 0; step < chunks; ++step) {
            const int next = min(step + 1, chunks - 1);
            const Item it = chunk_of(next);
            const size_t item = item_of(step);
            const float *rec = p.ws.rec + item_of(next) * R::SIZE;
            put_state(item);
            touch(step + 2);
#pragma unroll
            for (int y = 0; y < JT; ++y)
#pragma unroll
                for (int r = 0; r < 4; r += 2) {
                    float f0 = 0.f, f1 = 0.f;
                    if constexpr (Parts::value == 3) f0 = Rows<T>::value4(ov[y])[r], f1 = Rows<T>::value4(ov[y])[r + 1];
#pragma unroll
                    for (int z = 0; z < Parts::value; ++z) {
                        uint32_t u = ov[y][r / 2];
                        if constexpr (Parts::value == 3) u = part_of<true, false>(z, f0, f1);
                        s.O[z][16 * y + oj + r][inner(ot)] = static_cast<uint16_t>(u);
                        s.O[z][16 * y + oj + r + 1][inner(ot)] = static_cast<uint16_t>(u >> 16);
                    }
                }
            in_of(it);
            __syncthreads();
            f32x4 e[JT];
#pragma unroll
            for (int y = 0; y < JT; ++y) e[y] = zero;
            times_tri(s.O, tri, e, Parts{});
            tri_of(tri, rec);
            times_rows(rows, e);
            rows_of(rows, rec + (BACK ? R::XR : R::WR));
            const float be = BACK ? -Rows<TB>::value(b) : Rows<TB>::value(b);
            b = beta_of(it);
#pragma unroll
            for (int y = 0; y < JT; ++y) {
                put(s.U, y, tau_col, e[y] * be);
                store4_far((BACK ? p.ws.Y : p.ws.E) + item * C * D + ((w * NT + jt + y) * 64 + l) * 4, e[y]);
            }
#pragma unroll
            for (int i = 0; i < CT; ++i)
#pragma unroll
                for (int y = 0; y < JT; ++y) st[y][i] *= gam[i];
            gam_of(gam, rec);
            if constexpr (BACK) {                          // dO's share of the new state waits for nothing
                onto_state(s.O, qd, Parts{});
                cols_of(qd, rec + R::QDT);
            }
            __syncthreads();
            onto_state(s.U, kt, Three{});
            cols_of(kt, rec + (BACK ? R::KDT : R::KRT));
        }
    };
    if (chunks > 0) {
        if (back) run(std::true_type{}, dout);
        else run(std::false_type{}, v);
    }
    if (back && dS0)
#pragma unroll
        for (int y = 0; y < JT; ++y)
#pragma unroll
            for (int i = 0; i < CT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) dS0[(state0 + jr + 16 * y + r) * D + key(i)] = st[y][i][r];
}

// ---- finish ---------------------------------------------------------------

// Zeros into rows of tokens in no sequence, all of which lie before the first sequence or
// behind the last one: of those, in order, the 64 that start with 64 `behind`, channels
// c0 .. c0 + CH of one head. `behind` counts the workgroups behind the last chunk: the grid
// is for ceil(T / 64) + N chunks and a sequence of n tokens takes at most (n + 63) / 64, so
// 64 tokens each reach every row that the sequences leave.
template <int D, int CH, typename TI, typename TB>
__device__ void clear_rows(const Common &p, size_t item, int part, TI *dq, TI *dk, TI *dv, float *dg, TB *dbeta) {
    const int h = (int)(item % p.H), before = p.sv.cu[0], end = p.sv.cu[p.sv.N];
    const long long first = 64ll * ((long long)(item / p.H) - p.sv.total_chunks());
    const u32v4 zero = {0, 0, 0, 0};
    for (int i = threadIdx.x / (CH / 4); i < C; i += 4 * CH / (CH / 4)) {
        const long long n = first + i, token = n < before ? n : n - before + end;
        if (token >= p.sv.T) return;
        const size_t row = (size_t)token * p.H + h, x = row * D + part * CH + threadIdx.x % (CH / 4) * 4;
        auto clear4 = [&](auto *to) {
            if constexpr (sizeof(*to) == 4) *reinterpret_cast<u32v4 *>(to) = zero;
            else *reinterpret_cast<u32v2 *>(to) = u32v2{0, 0};
        };
        if (p.zero_rows & KDA_ZERO_DQ) clear4(dq + x);
        if (p.zero_rows & KDA_ZERO_DK) clear4(dk + x);
        if (p.zero_rows & KDA_ZERO_DV) clear4(dv + x);
        const bool gate = dg && (p.zero_rows & KDA_ZERO_DG);
        if (gate && !p.g_head) clear4(dg + x);
        if (part == 0 && threadIdx.x % (CH / 4) == 0) {
            if (gate && p.g_head) dg[row] = 0.f;
            if (p.zero_rows & KDA_ZERO_DBETA) dbeta[row] = TB(0);
        }
    }
}

// A workgroup takes CH key channels of a (chunk, head), one wavefront for each 16.
// CH = 64 leaves room for two workgroups on a CU, which cover each other's loads
// and barriers (dP and dA are then formed twice at D = 128); where rows are summed
// over all channels (normalised q and k, a gate per head) CH = D.
// O, U and V hold dO, U = b E and dV = b Y as split operands over 32 SM value
// channels at a time: [part][32 channels][token block], lane l's 16 bytes.
template <int CH, int PO>
struct FinishLds {
    static constexpr int NW = CH / 16, SM = NW / 4;
    union {
        struct {
            u32v4 O[PO][SM][NB][64], U[3][SM][NB][64], V[3][SM][NB][64];
        };
        f32x4 wait[2][NB][4 * CH];    // each thread's own values, while the pairs need its registers
    };
    float dP[C][LP], dA[C][LP];       // tiles on and below the diagonal; above it nothing is used
    float db[C][4];
    float rows[2][NW][C];             // sums over a wavefront's channels
};

template <int D, int CH, typename TI, typename TB, typename TG>
__global__ __launch_bounds__(4 * CH, 2) void finish_kernel(Common p, const TI *__restrict__ q, const TI *__restrict__ k,
                                                          const TB *__restrict__ beta, const TG *__restrict__ dout,
                                                          TI *__restrict__ dq, TI *__restrict__ dk,
                                                          TI *__restrict__ dv, float *__restrict__ dg,
                                                          TB *__restrict__ dbeta) {
    constexpr int NT = D / 16, NW = CH / 16, SM = NW / 4, STAGES = NT / (2 * SM), PO = sizeof(TG) == 2 ? 1 : 3;
    using R = Rec<D>;
    extern __shared__ char lds_raw[];
    typedef FinishLds<CH, PO> FinishLds_t;
    FinishLds_t &s = *reinterpret_cast<FinishLds_t *>(lds_raw);
    Item it;
    // the parts of an item, which read the same rows, run on one XCD (workgroups go
    // to the eight XCDs in turn)
    constexpr unsigned PARTS = D / CH;
    const int part = blockIdx.x / 8 % PARTS;
    const size_t nth = blockIdx.x / (8 * PARTS) * 8 + blockIdx.x % 8;
    if (!it.find(p, nth)) {
        if (p.sv.cu && p.zero_rows) clear_rows<D, CH>(p, nth, part, dq, dk, dv, dg, dbeta);
        return;
    }
    const size_t item = it.slot;
    const float *rec = p.ws.rec + item * R::SIZE, *M = p.ws.M + item * D * D, *dM = p.ws.dM + item * D * D;
    const float *E = p.ws.E + item * C * D, *Y = p.ws.Y + item * C * D;
    const int t = threadIdx.x, w = t / 64, l = t % 64, lr = l % 16, lg = l / 16;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const Rows<TI> qr(q, it, p.H, D), kr(k, it, p.H, D), dqr(dq, it, p.H, D), dkr(dk, it, p.H, D), dvr(dv, it, p.H, D);
    const Rows<TG> dor(dout, it, p.H, D);
    const Rows<TB> br(beta, it, p.H, 1), dbr(dbeta, it, p.H, 1);
    const Decay decay(p, it, D);
    const int ct = part * NW + w, c = 16 * ct + lr;    // this wavefront's channel tile, this lane's channel

    // Through the states (rows 16 b + 4 lg + r of channel c): dO M^T, dV M^T and
    // U dM^T; and dP and dA, of each the ten tiles on and below the diagonal. The
    // next stage's data are on their way while a stage is computed.
    // every second wavefront has the tiles tile_first, + NW / 2, ..; one behind the
    // last is the last again
    constexpr int JOBS = (2 * TILES + NW - 1) / NW;
    const int tile_first = w / 2;
    f32x4 aq[NB], ak[NB], ar[NB], ap[JOBS];
#pragma unroll
    for (int b = 0; b < NB; ++b) aq[b] = ak[b] = ar[b] = zero;
#pragma unroll
    for (int i = 0; i < JOBS; ++i) ap[i] = zero;
    float mdm = 0.f;
    const int sb = w % NB, sm = w / NB, stau = 16 * sb + lr;   // staging: token block, 32 value channels, token
    const float be = br.at(stau, 0);
    f32x4 e0, e1, y0, y1, m0[SM], m1[SM], d0[SM], d1[SM];
    typename Rows<TG>::Raw4 o0, o1;
    auto load_rows = [&](int stage) {
        const int jt = 2 * (stage * SM + sm), f = ((sb * NT + jt) * 64 + l) * 4, j = 16 * jt + 4 * lg;
        e0 = ld4(E + f);
        e1 = ld4(E + f + 256);
        y0 = ld4(Y + f);
        y1 = ld4(Y + f + 256);
        o0 = dor.raw4(stau, j);
        o1 = dor.raw4(stau, j + 16);
    };
    auto load_states = [&](int stage, int m) {
        const int f = ((ct * NT + 2 * (stage * SM + m)) * 64 + l) * 4;
        m0[m] = ld4(M + f);
        m1[m] = ld4(M + f + 256);
        d0[m] = ld4(dM + f);
        d1[m] = ld4(dM + f + 256);
    };
    load_rows(0);
#pragma unroll
    for (int m = 0; m < SM; ++m) load_states(0, m);
    const bool first = part == 0;                      // dv and dbeta are the first workgroup's
#pragma unroll 1
    for (int stage = 0; stage < STAGES; ++stage) {
        const int next = min(stage + 1, STAGES - 1);
        if (stage) __syncthreads();
        {
            const int j = 32 * (stage * SM + sm) + 4 * lg;
            u32v4 o[PO], u[3], v[3];                   // u and the states M are the rounded sides
            if constexpr (PO == 1) o[0] = u32v4{o0[0], o0[1], o1[0], o1[1]};
            else split3<false, true>(Rows<TG>::value4(o0), Rows<TG>::value4(o1), o);
            split3<true, true>(e0 * be, e1 * be, u);
            split3<false, true>(y0 * be, y1 * be, v);
            if (first) {
                dvr.put4(stau, j, y0 * be);
                dvr.put4(stau, j + 16, y1 * be);
            }
#pragma unroll
            for (int x = 0; x < PO; ++x) s.O[x][sm][sb][l] = o[x];
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                s.U[x][sm][sb][l] = u[x];
                s.V[x][sm][sb][l] = v[x];
            }
            const f32x4 ye = e0 * y0 + e1 * y1;
            float x = (ye[0] + ye[1]) + (ye[2] + ye[3]);
            x += __shfl_xor(x, 16, 64);
            x += __shfl_xor(x, 32, 64);
            if (lg == 0) s.db[stau][stage * SM + sm] = x;
        }
        load_rows(next);
        __syncthreads();
#pragma unroll
        for (int m = 0; m < SM; ++m) {
            u32v4 ms[3], ds[3];
            const f32x4 x = m0[m] * d0[m] + m1[m] * d1[m];
            mdm += (x[0] + x[1]) + (x[2] + x[3]);
            split3<true, true>(m0[m], m1[m], ms);
            split3<false, true>(d0[m], d1[m], ds);
            load_states(next, m);
            // operands of the next block are read while this one's products run
            u32v4 o[2][PO], u[2][3], v[2][3];
            auto read = [&](int b) {
#pragma unroll
                for (int x = 0; x < PO; ++x) o[b & 1][x] = s.O[x][m][b][l];
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    v[b & 1][x] = s.V[x][m][b][l];
                    u[b & 1][x] = s.U[x][m][b][l];
                }
            };
            read(0);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (b + 1 < NB) read(b + 1);
                __builtin_amdgcn_sched_barrier(0);
                aq[b] = product(o[b & 1], ms, aq[b]);
                ak[b] = product(v[b & 1], ms, ak[b]);
                ar[b] = product(u[b & 1], ds, ar[b]);
                settle(aq[b]);
                settle(ak[b]);
                settle(ar[b]);
            }
            // even wavefronts have tiles of dP, odd ones of dA
            auto tiles = [&](auto &left, auto np) {
                constexpr int PL = decltype(np)::value;
                u32v4 x[2][PL], y[2][3];
                auto read_tile = [&](int i) {
                    int bi, bj;
                    tile_at(tile_first + i * (NW / 2), bi, bj);
#pragma unroll
                    for (int z = 0; z < PL; ++z) x[i & 1][z] = left[z][m][bi][l];
#pragma unroll
                    for (int z = 0; z < 3; ++z) y[i & 1][z] = s.U[z][m][bj][l];
                };
                read_tile(0);
#pragma unroll
                for (int i = 0; i < JOBS; ++i) {
                    if (i + 1 < JOBS) read_tile(i + 1);
                    __builtin_amdgcn_sched_barrier(0);
                    ap[i] = product(x[i & 1], y[i & 1], ap[i]);
                    settle(ap[i]);
                }
            };
            if (w & 1) tiles(s.V, std::integral_constant<int, 3>{});
            else tiles(s.O, std::integral_constant<int, PO>{});
        }
    }
    // q, k and the log-decays on their way: a lane holds the group lg
    // of four tokens of each block, for its channel
    typename Rows<TI>::Raw qraw[NB][4], kraw[NB][4];
    f32x4 gv[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int tau = 16 * b + 4 * lg + r;
            qraw[b][r] = qr.raw(tau, c);
            kraw[b][r] = kr.raw(tau, c);
            gv[b][r] = decay.g.at(tau, c * decay.col);
        }
#pragma unroll
    for (int i = 0; i < JOBS; ++i) {
        int bi, bj;
        tile_at(tile_first + i * (NW / 2), bi, bj);
        float(*out)[LP] = w & 1 ? s.dA : s.dP;
#pragma unroll
        for (int r = 0; r < 4; ++r) out[16 * bi + 4 * lg + r][16 * bj + lr] = w & 1 ? -ap[i][r] : ap[i][r];
    }
    mdm += __shfl_xor(mdm, 16, 64);
    mdm += __shfl_xor(mdm, 32, 64);
    if (first && t < C) {
        float x = 0.f;
        for (int i = 0; i < NT / 2; ++i) x += s.db[t][i];
        dbr.put(t, 0, x);
    }

    f32x4 qv[NB], kv[NB], ein[NB], eout[NB];
    float end[NB], grp[NB];                            // the block's and the other group's sum
    uint32_t wiped = 0;                                // tokens whose decay is 0, of gradient 0
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            qv[b][r] = Rows<TI>::value(qraw[b][r]);
            kv[b][r] = Rows<TI>::value(kraw[b][r]);
            gv[b][r] = Decay::cut(gv[b][r]);
            wiped |= (gv[b][r] <= MIN_G ? 1u : 0u) << (4 * b + r);
        }
    }
    if (p.qk_norm) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            qv[b] *= ld4(rec + R::RQ + 16 * b + 4 * lg);
            kv[b] *= ld4(rec + R::RK + 16 * b + 4 * lg);
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const f32x4 g = gv[b];
        const float own = (g[0] + g[1]) + (g[2] + g[3]);
        grp[b] = __shfl_xor(own, 16, 64);
        const float half = own + grp[b], other = __shfl_xor(half, 32, 64);
        end[b] = half + other;
        const float in0 = (lg & 1 ? grp[b] : 0.f) + (lg & 2 ? other : 0.f),
                    out0 = (lg & 1 ? 0.f : grp[b]) + (lg & 2 ? 0.f : other);
        const f32x4 pre = {g[0], g[0] + g[1], (g[0] + g[1]) + g[2], own};
        const f32x4 suf = {(g[1] + g[2]) + g[3], g[2] + g[3], g[3], 0.f};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            ein[b][r] = __expf(in0 + pre[r]);          // from the block's start, the token included
            eout[b][r] = __expf(out0 + suf[r]);        // behind the token to the block's end
        }
    }
    // what came through the states gets its decay from the chunk's start or to its
    // end: aq and ak become dq's and dk's share, ar what a token sends behind the chunk
    float all;
    {
        float before[NB], behind[NB];
        before[0] = behind[NB - 1] = 0.f;
#pragma unroll
        for (int b = 1; b < NB; ++b) {
            before[b] = before[b - 1] + end[b - 1];
            behind[NB - 1 - b] = behind[NB - b] + end[NB - b];
        }
        all = __expf(before[NB - 1] + end[NB - 1]) * mdm;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const f32x4 fi = ein[b] * __expf(before[b]);
            aq[b] *= fi;
            ak[b] *= -fi;
            ar[b] *= eout[b] * __expf(behind[b]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        s.wait[0][b][t] = ak[b];
        s.wait[1][b][t] = ar[b];
    }

    // pairs of tokens of different blocks: what a token receives is scaled by
    // ein, what it sends by eout, whole blocks between on the operand
    f32x4 pq[NB], pk[NB], pc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) pq[b] = pk[b] = pc[b] = zero;
    // tiles of dP and dA in the order of use, each read as left operands (by rows and
    // by columns) while the one before it is multiplied
    constexpr int ORDER[TILES][2] = {{1, 0}, {2, 1}, {2, 0}, {3, 2}, {3, 1}, {3, 0}, {0, 0}, {1, 1}, {2, 2}, {3, 3}};
    struct Operands {
        f32x4 prow, arow, pcol, acol;
    } op[2];
    auto read = [&](int n) {
        const int bi = ORDER[n][0], bj = ORDER[n][1];
        op[n & 1] = Operands{ld4(&s.dP[16 * bi + lr][16 * bj + 4 * lg]), ld4(&s.dA[16 * bi + lr][16 * bj + 4 * lg]),
                             ld4s(&s.dP[16 * bi + 4 * lg][16 * bj + lr], LP),
                             ld4s(&s.dA[16 * bi + 4 * lg][16 * bj + lr], LP)};
    };
    read(0);
#pragma unroll
    for (int n = 0; n < TILES - NB; ++n) {
        const int bi = ORDER[n][0], bj = ORDER[n][1];
        read(n + 1);
        __builtin_amdgcn_sched_barrier(0);
        const Operands &x = op[n & 1];
        const float f = bi - bj == 1 ? 1.f : __expf(bi - bj == 2 ? end[bj + 1] : end[1] + end[2]);
        const f32x4 key = kv[bj] * eout[bj] * f, fe = ein[bi] * f;
        pq[bi] = mfma16(x.prow, key, pq[bi]);
        pk[bi] = mfma16(x.arow, key, pk[bi]);
        pc[bj] = mfma16(x.pcol, qv[bi] * fe, pc[bj]);
        pc[bj] = mfma16(x.acol, kv[bi] * fe, pc[bj]);
        settle(pq[bi]);
        settle(pk[bi]);
        settle(pc[bj]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        pq[b] *= ein[b];
        pk[b] *= ein[b];
        pc[b] *= eout[b];
        settle(pq[b]);
        settle(pk[b]);
        settle(pc[b]);
    }
    // in-block pairs, and the pair terms put together: pq and pk become dq's and
    // dk's share, pc row's
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (b + 1 < NB) read(TILES - NB + b + 1);
        const Operands &x = op[b & 1];                 // TILES - NB is even
        const f32x4 g = gv[b];
        const f32x4 pre = {g[0], g[0] + g[1], (g[0] + g[1]) + g[2], (g[0] + g[1]) + (g[2] + g[3])};
        const f32x4 suf = {(g[1] + g[2]) + g[3], g[2] + g[3], g[3], 0.f};
        // the halves of the block, then the groups of a half: the left operand keeps
        // only pairs of its level
#pragma unroll
        for (int level = 8; level >= 4; level -= 4) {
            const bool row = level == 8 ? lr >= 8 && lg < 2 : (lr >> 2) == lg + 1 && !(lg & 1);
            const bool col = level == 8 ? lr < 8 && lg >= 2 : (lr >> 2) + 1 == lg && (lg & 1);
            const float in0 = level == 8 && (lg & 1) ? grp[b] : 0.f, out0 = level == 8 && !(lg & 1) ? grp[b] : 0.f;
            f32x4 ei, eo;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                ei[r] = __expf(in0 + pre[r]);
                eo[r] = __expf(out0 + suf[r]);
            }
            const f32x4 key = kv[b] * eo;
            pq[b] += mfma16(row ? x.prow : zero, key, zero) * ei;
            pk[b] += mfma16(row ? x.arow : zero, key, zero) * ei;
            pc[b] += mfma16(col ? x.acol : zero, kv[b] * ei, mfma16(col ? x.pcol : zero, qv[b] * ei, zero)) * eo;
        }
        // inside the group: all in this lane
        f32x4 dp[3], da[3];                            // the group's rows
#pragma unroll
        for (int r = 1; r < 4; ++r) {
            dp[r - 1] = ld4(&s.dP[16 * b + 4 * lg + r][16 * b + 4 * lg]);
            da[r - 1] = ld4(&s.dA[16 * b + 4 * lg + r][16 * b + 4 * lg]);
        }
        const float diag0 = s.dP[16 * b + 4 * lg][16 * b + 4 * lg];
        const float e10 = __expf(g[1]), e21 = __expf(g[2]), e32 = __expf(g[3]);
        const f32x4 ex[3] = {{e10, 0.f, 0.f, 0.f}, {e21 * e10, e21, 0.f, 0.f}, {e32 * e21 * e10, e32 * e21, e32, 0.f}};
#pragma unroll
        for (int r = 1; r < 4; ++r) {
#pragma unroll
            for (int y = 0; y < r; ++y) {
                const float e = ex[r - 1][y], ek = e * kv[b][y];
                pq[b][r] += dp[r - 1][y] * ek;
                pk[b][r] += da[r - 1][y] * ek;
                pc[b][y] += e * (dp[r - 1][y] * qv[b][r] + da[r - 1][y] * kv[b][r]);
            }
        }
        const f32x4 dg4 = {diag0, dp[0][1], dp[1][2], dp[2][3]}, send = pc[b];
        pq[b] += aq[b];
        pk[b] += s.wait[0][b][t];
        pc[b] = qv[b] * pq[b] + kv[b] * (pk[b] - send);
        pq[b] += dg4 * kv[b];
        const f32x4 sent = s.wait[1][b][t];
        pk[b] += send + dg4 * qv[b] + sent;
        ar[b] = sent * kv[b];
        settle(pq[b]);
        settle(pk[b]);
        settle(pc[b]);
    }

    if (p.qk_norm) {                                   // dx = (dx^ - x^ (x^ . dx^)) / |x|
        float v[16];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) v[4 * b + r] = which ? kv[b][r] * pk[b][r] : qv[b][r] * pq[b][r];
            s.rows[which][w][16 * (lr / 4) + 4 * lg + lr % 4] = sums16(v, lr);
        }
        __syncthreads();
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            f32x4 x = zero, y = zero;
            for (int i = 0; i < NW; ++i) {
                x += ld4(&s.rows[0][i][16 * b + 4 * lg]);
                y += ld4(&s.rows[1][i][16 * b + 4 * lg]);
            }
            pq[b] = (pq[b] - qv[b] * x) * ld4(rec + R::RQ + 16 * b + 4 * lg);
            pk[b] = (pk[b] - kv[b] * y) * ld4(rec + R::RK + 16 * b + 4 * lg);
        }
        __syncthreads();
    }
    // dg_i = sum_{t >= i} row_t + sum_{t < i} out_t + all
    float after = 0.f, past = 0.f;
#pragma unroll
    for (int b = NB - 1; b >= 0; --b) {                // suffix sums of row
        f32x4 x = pc[b];
        x[2] += x[3];
        x[1] += x[2];
        x[0] += x[1];
        const float x0 = __shfl(x[0], lr, 64), x1 = __shfl(x[0], lr + 16, 64), x2 = __shfl(x[0], lr + 32, 64),
                    x3 = __shfl(x[0], lr + 48, 64);
        pc[b] = x + (after + (lg == 3 ? 0.f : lg == 2 ? x3 : lg == 1 ? x3 + x2 : (x3 + x2) + x1));
        after += (x0 + x1) + (x2 + x3);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {                     // prefix sums of out (ar), without the token itself
        const f32x4 y = ar[b];
        f32x4 x = {0.f, y[0], y[0] + y[1], (y[0] + y[1]) + y[2]};
        const float tot = x[3] + y[3];
        const float x0 = __shfl(tot, lr, 64), x1 = __shfl(tot, lr + 16, 64), x2 = __shfl(tot, lr + 32, 64),
                    x3 = __shfl(tot, lr + 48, 64);
        pc[b] += x + (past + (lg == 0 ? 0.f : lg == 1 ? x0 : lg == 2 ? x0 + x1 : (x0 + x1) + x2)) + all;
        past += (x0 + x1) + (x2 + x3);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) pc[b][r] = wiped >> (4 * b + r) & 1 ? 0.f : pc[b][r];

    // out through LDS, in whole rows of 16-byte stores
    constexpr int SI = CH + 16 / (int)sizeof(TI), SG = CH + 4;
    TI *sq = reinterpret_cast<TI *>(lds_raw), *sk = sq + C * SI;
    float *sg = reinterpret_cast<float *>(sk + C * SI);
    static_assert(2 * C * SI * sizeof(TI) + C * SG * sizeof(float) <= offsetof(FinishLds_t, rows), "staging");
    __syncthreads();                                   // dP, dA and wait are done with
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int tau = 16 * b + 4 * lg + r, x = 16 * w + lr;
            if constexpr (sizeof(TI) == 4) {
                sq[tau * SI + x] = pq[b][r];
                sk[tau * SI + x] = pk[b][r];
            } else {
                sq[tau * SI + x] = round_bf16(pq[b][r]);
                sk[tau * SI + x] = round_bf16(pk[b][r]);
            }
            if (!p.g_head) sg[tau * SG + x] = pc[b][r];
        }
    if (p.g_head) {
        float v[16];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[4 * b + r] = pc[b][r];
        s.rows[0][w][16 * (lr / 4) + 4 * lg + lr % 4] = sums16(v, lr);
    }
    __syncthreads();
    constexpr int PER = 16 / sizeof(TI), CHUNKS = CH / PER;         // elements of a store, stores of a row
#pragma unroll
    for (int i = 0; i < C * CHUNKS / (4 * CH); ++i) {
        const int n = t + i * 4 * CH, tau = n / CHUNKS, x = (n % CHUNKS) * PER;
        dqr.put16(tau, part * CH + x, *reinterpret_cast<const u32v4 *>(sq + tau * SI + x));
        dkr.put16(tau, part * CH + x, *reinterpret_cast<const u32v4 *>(sk + tau * SI + x));
    }
    if (!dg) return;
    const Rows<float> dgr(dg, it, p.H, p.g_head ? 1 : D);
    if (p.g_head) {
        if (t < C) {
            float x = 0.f;
            for (int i = 0; i < NW; ++i) x += s.rows[0][i][t];
            dgr.put(t, 0, x);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = t + i * 4 * CH, tau = n / (CH / 4), x = (n % (CH / 4)) * 4;
        dgr.put16(tau, part * CH + x, *reinterpret_cast<const u32v4 *>(sg + tau * SG + x));
    }
}

// ---- host -----------------------------------------------------------------

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

template <int D>
size_t carve(int N, long long T_total, int H, char *base, Ws *ws) {
    const size_t items = (size_t)max_chunks(N, T_total, C) * H;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *at = base ? base + off : nullptr;
        off += round256(bytes);
        return at;
    };
    int32_t *plan[2];
    for (int i = 0; i < 2; ++i) plan[i] = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * (size_t)(N + 1)));
    float *a[5];
    const size_t sizes[5] = {Rec<D>::SIZE, (size_t)D * D, (size_t)D * D, (size_t)C * D, (size_t)C * D};
    for (int i = 0; i < 5; ++i) a[i] = reinterpret_cast<float *>(take(items * sizes[i] * sizeof(float)));
    if (ws) *ws = Ws{plan[0], plan[1], a[0], a[1], a[2], a[3], a[4]};
    return off;
}

template <int D, typename TI, typename TB, typename TG>
hipError_t launch_t(const PrefillBackwardArgs &a) {
    constexpr int PO = sizeof(TG) == 2 ? 1 : 3;
    Ws ws;
    carve<D>(a.N, (long long)a.B * a.T, a.H, static_cast<char *>(a.ws), &ws);
    if (a.cu_seqlens) {
        hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(256), 0, a.stream, a.cu_seqlens, a.N, a.T, ws.cut, ws.chunk_off);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const SeqView sv{a.cu_seqlens ? ws.cut : nullptr, ws.chunk_off, a.N, a.T, C};
    const long long chunks = a.cu_seqlens ? max_chunks(a.N, a.T, C) : (long long)a.N * ((a.T + C - 1) / C);
    const Common p{sv, ws, a.g, a.H, (int)chunks, a.g_head, a.qk_norm, a.norm_eps, a.zero_rows};
    const unsigned items = static_cast<unsigned>(chunks * a.H);
    const TI *q = static_cast<const TI *>(a.q), *k = static_cast<const TI *>(a.k), *v = static_cast<const TI *>(a.v);
    const TB *beta = static_cast<const TB *>(a.beta);
    const TG *dout = static_cast<const TG *>(a.dout);
    const auto prep = prep_kernel<D, TI, TB>;
    // sums over a row's channels need the whole row in one workgroup
    const bool whole = D == 64 || a.qk_norm || a.g_head;
    const auto finish = whole ? finish_kernel<D, D, TI, TB, TG> : finish_kernel<D, 64, TI, TB, TG>;
    const int ch = whole ? D : 64, finish_lds = whole ? sizeof(FinishLds<D, PO>) : sizeof(FinishLds<64, PO>);
    // set on every call (idempotent; no process-wide flag to race on)
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(prep),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, sizeof(PrepLds<D>));
    if (e != hipSuccess) return e;
    e = hipFuncSetAttribute(reinterpret_cast<const void *>(finish), hipFuncAttributeMaxDynamicSharedMemorySize,
                            finish_lds);
    if (e != hipSuccess) return e;
    if (items > 0) {
        hipLaunchKernelGGL(prep, dim3(items), dim3(4 * D), sizeof(PrepLds<D>), a.stream, p, q, k, beta);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const unsigned groups = (static_cast<unsigned>(a.N * a.H) + 7) / 8;
    // 32 value channels per workgroup load each operand half as often, but on half
    // the workgroups. Whole calls at 32 / 16 channels, D = 128: one workgroup a CU (one
    // sequence of 8192 tokens, 32 heads) 1190 / 1282 us, two (2 x 4096) 1160 / 1272 us,
    // half a one (8192 tokens, 16 heads) 814 / 714 us. The longest of packed sequences
    // decides when a call ends: 64 chains of 1 to 2048 tokens (two a CU) 300 / 252 us, 96
    // (three) 651 / 697 us, 384 1815 / 1986 us.
    int dev = 0, cus = 0;
    if ((e = hipGetDevice(&dev)) != hipSuccess) return e;
    if ((e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev)) != hipSuccess) return e;
    const long long wide = 2ll * a.N * a.H * (D / 32);
    const int tv = wide >= (a.cu_seqlens && a.N > 1 ? 3ll : 1ll) * cus ? 32 : 16;
    const auto scan = tv == 32 ? scan_kernel<D, 32, TI, TB, TG> : scan_kernel<D, 16, TI, TB, TG>;
    hipLaunchKernelGGL(scan, dim3(2 * groups * 8 * (D / tv)), dim3(256), 0, a.stream, p, v, beta, dout, a.S0,
                       a.dS_out, a.dS0);
    e = hipGetLastError();
    if (e != hipSuccess || items == 0) return e;
    hipLaunchKernelGGL(finish, dim3((items + 7) / 8 * 8 * (D / ch)), dim3(4 * ch), finish_lds, a.stream, p, q, k, beta, dout,
                       static_cast<TI *>(a.dq), static_cast<TI *>(a.dk), static_cast<TI *>(a.dv), a.dg,
                       static_cast<TB *>(a.dbeta));
    return hipGetLastError();
}

template <int D>
hipError_t launch_d(const PrefillBackwardArgs &a) {
    if (a.io == Dt::F32) return launch_t<D, float, float, float>(a);
    if (a.beta_dt == Dt::F32)
        return a.dout_dt == Dt::F32 ? launch_t<D, bf16_t, float, float>(a) : launch_t<D, bf16_t, float, bf16_t>(a);
    return a.dout_dt == Dt::F32 ? launch_t<D, bf16_t, bf16_t, float>(a) : launch_t<D, bf16_t, bf16_t, bf16_t>(a);
}

}  // namespace

size_t prefill_backward_workspace(int N, long long T_total, int H, int Dk) {
    return Dk == 64 ? carve<64>(N, T_total, H, nullptr, nullptr) : carve<128>(N, T_total, H, nullptr, nullptr);
}

bool prefill_backward_fits(int N, long long T_total, int H, int Dk) {
    // a launch has fewer than 2^32 threads
    const unsigned long long items = (unsigned long long)max_chunks(N, T_total, C) * H;
    const unsigned long long scans = 2 * ((unsigned long long)N * H + 7) * (Dk / 16);
    // and one chunk of a tensor at most 2^31 bytes (offsets inside it have 32 bits)
    return (items + 8) * 512 < (1ull << 32) && scans * 256 < (1ull << 32) && (unsigned long long)H * Dk * C * 4 < (1ull << 31);
}

hipError_t launch_prefill_backward(const PrefillBackwardArgs &a) { return a.Dk == 64 ? launch_d<64>(a) : launch_d<128>(a); }

}  // namespace kda
