// lin_chunk.hip -- linear attention with a decay per head, chunked: the forward pass over
// whole sequences and the gradient.
//
//     S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = S_t q_t
//
// With a = the cumulative sum of g inside a chunk and S the state before it:
//     o_t = e^{a_t} S q_t + sum_{s <= t} e^{a_t - a_s} (q_t . k_s) v_s
//     S  <- e^{a_C} S + sum_s e^{a_C - a_s} v_s k_s^T
// The gradients of q, k and v are this form again, over other tensors and, for k and v,
// backwards in time: dq = F(dout, v, k), dk = F(v, dout, q) and dv = F(k, q, dout), F(x, y, z)
// being the outputs for queries x, keys y and values z. So one kernel serves all four.
//
// Split: the tokens of a sequence are cut into segments. Without states at the segments'
// borders a chain is one workgroup's serial walk; with them every (segment, head) is a
// workgroup of its own. state_kernel sums each segment's own contribution, border_kernel
// carries the states across segments, output_kernel walks a segment's chunks from its border
// state. Costs a second read of two of the tensors and 8 D^2 bytes a segment and pass.
//
// Arithmetic: bf16 matrix instructions with fp32 accumulators. An operand that is no bf16
// value (decayed, a state, fp32 input) is cut into bf16 parts whose sum it is to 2^-17 (two)
// or 2^-25 (three); of parts i and j the products i + j < the number of parts are taken.
// States take three always; outputs in bf16 two, outputs in fp32 and those that a decay's
// gradient is summed from three. (bf16 outputs, whose own rounding is 2^-9, are 1.66e-3 from 64 bits either way; with two
// parts some roundings fall the other way, 1.0e-4 of the norm, with three 1.7e-5, at 127 us instead of 116 for the 8k
// forward and 386 instead of 375 for its gradient.) The exponents of decays are differences of cumulative sums
// that are taken in 64 bits and held as whole and fractional part in base 2, so that no
// difference loses bits and no factor exceeds the decay that it stands for.
//
// A wavefront owns 16 value channels: its part of the state, transposed, stays in accumulator
// layout (16 x 16 tiles: column = value channel, rows = key channels), whose registers are, up
// to the order of the summed index, the A operand of the product with q^T; the scores q k^T are
// formed transposed for the same reason, a lane's four values being a lane's four values of the next
// product's operand. Only scores go through LDS, because the wavefronts share them. Eight wavefronts of
// 16 channels rather than four of 32 leave four to a SIMD, which the chunk's barriers and LDS reads need.
//
// 8192 tokens x 32 heads x 128, bf16, calls one behind the other: forward 115-119 us, gradient 375-381. Kernel by kernel under
// the profiler (average, least), whose times add up to more than a call's: forward states 37, 34 (4.5 TB/s), borders 11, 11,
// outputs 76, 75, bound by instruction issue and barriers (vector instructions 55% of their cycles, 47% without the
// matrix ones; matrix units 31%, LDS 44%; no less time with q and k from cache); gradient states 79, 72, borders 26, 24, dq
// and dk 243, 216, dv 84, 73, decays 12, 11.
#include "kda_device.h"
#include "kda_launch.h"

namespace kda {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kMinLog = -104.f;       // e^-104 rounds to zero: a smaller decay is no other

constexpr int kMaxSegment = 1024;

struct Segments {
    const int32_t *cu;      // packed offsets, or nullptr: N sequences of T tokens
    int N, T, T_total, L;   // L tokens a segment, 2^shift
    int shift;
};
struct Gate {
    const float *g;         // [tokens][H], fixed: [H]; nullptr: none
    bool fixed;
};
// One sum over segments: keys y, values z (a shared tensor has a head per group of heads).
struct StateJob {
    const void *y, *z;
    float *out;             // [ids][H][value channels][key channels]
    bool y_shared, z_shared, tail, skip_last;
};
struct StateJobs { StateJob job[2]; };
struct BorderArgs {
    const float *S0, *dS_out;
    float *states, *grads, *dS0, *dots, *starts;
    const float *whole;     // each segment's decay
    bool all;               // the gradients' states too
};
struct OutputJob {
    const void *x, *y, *z, *with;
    void *out;
    float *dot, *past;      // [H][T_total], and a chunk's part from the state [ids][H][chunks of a segment]
    const float *S;         // the state before each segment (border) or sequence, or nullptr
    float *S_out;           // the state behind each sequence, or nullptr
    bool x_shared, y_shared, z_shared, out_shared, border, key_rows, back, zero_rows;
};
struct OutputJobs { OutputJob job[3]; };

// ---- sequences and segments -------------------------------------------------
// Segment ids need no table: sequence n starts at id begin_n / L + n, which leaves room for
// ceil(length / L) ids (one for an empty sequence) and grows with n, so an id's sequence is
// found by a search, a wavefront's lanes at a time. Ids between two sequences' are holes.
struct Segment {
    int n, begin, end;      // the sequence and its tokens
    int b, blocks;          // this segment's index in it, and how many it has
};

// where sequence n begins; offsets outside the packed rows are cut to them
__device__ __forceinline__ int offset(const Segments &s, int n) {
    return s.cu ? min(max(s.cu[n], 0), s.T_total) : n * s.T;
}
// Where sequence i, one a lane, begins and ends. An offset below an earlier one would make sequences share ids; in a call
// of up to 64 sequences (i: the lane, or the last one) it is cut to it, so that every one has segments of its own and its
// state is written. With more there is no such look at all of them, and offsets that fall give undefined results (in bounds).
__device__ __forceinline__ void lane_bounds(const Segments &s, int i, int &begin, int &end) {
    begin = offset(s, i);
    const int next = offset(s, i + 1);
    if (s.cu && s.N <= 64 && __any(next < begin)) {
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) begin = max(begin, __shfl_up(begin, o, 64));
    }
    end = max(next, begin);
}
// The same for one sequence, n the same in every lane of a whole wavefront.
__device__ __forceinline__ void sequence_bounds(const Segments &s, int n, int &begin, int &end) {
    const bool all = s.cu && s.N <= 64;                     // uniform
    lane_bounds(s, all ? min((int)(threadIdx.x & 63), s.N - 1) : n, begin, end);
    begin = __builtin_amdgcn_readlane(begin, all ? n : 0);
    end = __builtin_amdgcn_readlane(end, all ? n : 0);
}
__device__ __forceinline__ int block_count(const Segments &s, int len) { return max(1, (len + s.L - 1) >> s.shift); }
__device__ __forceinline__ int first_id(const Segments &s, int n, int begin) { return (begin >> s.shift) + n; }

// false: a hole. The same in every lane.
__device__ __forceinline__ bool find_segment(const Segments &s, int id, Segment &x) {
    const int lane = threadIdx.x & 63;
    int lo = 0, span = s.N;                         // the sequence is one of span from lo on
    while (span > 64) {
        const int each = (span + 63) / 64, i = lo + lane * each;
        const bool before = lane * each < span && first_id(s, i, offset(s, i)) <= id;
        const int c = max(__popcll(__ballot(before)) - 1, 0);
        lo += c * each;
        span = min(each, span - c * each);
    }
    const int i = min(lo + lane, s.N - 1);
    int begin, end;
    lane_bounds(s, i, begin, end);
    const bool before = lane < span && first_id(s, i, begin) <= id;
    const int c = max(__popcll(__ballot(before)) - 1, 0);
    x.n = __builtin_amdgcn_readfirstlane(lo + c);
    x.begin = __builtin_amdgcn_readlane(begin, c);
    x.end = __builtin_amdgcn_readlane(end, c);
    x.blocks = block_count(s, x.end - x.begin);
    x.b = id - first_id(s, x.n, x.begin);
    return x.b >= 0 && x.b < x.blocks;
}

// ---- cutting ----------------------------------------------------------------
// Pairs at a time: one conversion instruction rounds two values into a word, whose halves are the rounded values.
__device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ f32x8 widen(bf16x8 x) {
    const u32x4 w = __builtin_bit_cast(u32x4, x);
    return f32x8{low(w[0]), high(w[0]), low(w[1]), high(w[1]), low(w[2]), high(w[2]), low(w[3]), high(w[3])};
}
__device__ __forceinline__ f32x4 widen(bf16x4 x) {
    const u32x2 w = __builtin_bit_cast(u32x2, x);
    return f32x4{low(w[0]), high(w[0]), low(w[1]), high(w[1])};
}
__device__ __forceinline__ bf16x4 narrow(f32x4 x) { return __builtin_bit_cast(bf16x4, u32x2{pack(x[0], x[1]), pack(x[2], x[3])}); }

template <int P> __device__ __forceinline__ void cut(f32x8 x, bf16x8 (&p)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = pack(x[2 * e], x[2 * e + 1]);
            x[2 * e] -= low(w[e]);
            x[2 * e + 1] -= high(w[e]);
        }
        p[i] = __builtin_bit_cast(bf16x8, w);
    }
}

// Rows in parts, as col_frag leaves them, times their weights W[0 .. 3] and W[16 .. 19], cut in three.
template <int NI> __device__ __forceinline__ void weigh(const bf16x8 (&x)[NI], const float *W, bf16x8 (&p)[3]) {
    f32x8 v = widen(x[NI - 1]);
#pragma unroll
    for (int i = NI - 2; i >= 0; --i) v += widen(x[i]);
    const f32x4 a = *reinterpret_cast<const f32x4 *>(W), b = *reinterpret_cast<const f32x4 *>(W + 16);
    v *= __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    cut<3>(v, p);
}

// acc += x y, x in PX parts and y in PY, products of parts whose indices add up to less than the larger count
template <int PX, int PY>
__device__ __forceinline__ f32x4 product(const bf16x8 (&x)[PX], const bf16x8 (&y)[PY], f32x4 acc) {
    constexpr int P = PX > PY ? PX : PY;
#pragma unroll
    for (int i = PX - 1; i >= 0; --i)
#pragma unroll
        for (int j = PY - 1; j >= 0; --j)
            if (i + j < P) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], y[j], acc, 0, 0, 0);
    return acc;
}

// The value again, as one the compiler knows nothing of: addresses derived from it are computed where
// they are used. Held over the chunk loop, as loop invariants, they cost more registers than there are.
__device__ __forceinline__ int afresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// ---- tiles in LDS -----------------------------------------------------------
// Rows of D bf16 values in blocks of four, a row's blocks permuted by an exclusive or with swz(row), which
// keeps pairs of blocks together, so that 32 lanes touch every bank once, whether they read two neighbouring blocks of 16 rows or (the transposing
// read) four blocks of eight rows.
template <int D> __device__ __forceinline__ int swz(int row) {
    return D == 128 ? ((row & 3) << 3) | (row & 4) | ((row >> 2) & 2) : ((row & 2) << 2) | (row & 4) | ((row >> 2) & 2);
}
template <int D> __device__ __forceinline__ int at(int row, int block) { return row * D + ((block ^ swz<D>(row)) << 2); }

// A sum over 32 channels (k-step m) runs in the order that a state's accumulator tiles dictate: lane group g
// (lane / 16) holds rows 4g .. 4g + 3 of two tiles. Keys lie in LDS so that those rows are channels 32m + 8g .. + 7:
// their block b at place(b). Queries then are read 16 bytes at a time, as they come.
__device__ __forceinline__ int place(int b) { return (b & ~7) | ((b & 1) << 2) | ((b >> 1) & 3); }
// The first of the four channels that lane group g holds in a state's tile d.
__device__ __forceinline__ int channel(int d, int g) { return 32 * (d >> 1) + 4 * (d & 1) + 8 * g; }
template <int D> __device__ __forceinline__ bf16x8 query_frag(const bf16_t *tile, int row, int m, int g) {
    return *reinterpret_cast<const bf16x8 *>(tile + at<D>(row, 8 * m + 2 * g));
}
template <int D> __device__ __forceinline__ bf16x8 key_frag(const bf16_t *tile, int row, int m, int g) {
    const bf16x4 x = *reinterpret_cast<const bf16x4 *>(tile + at<D>(row, 8 * m + g));
    const bf16x4 y = *reinterpret_cast<const bf16x4 *>(tile + at<D>(row, 8 * m + 4 + g));
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}
// The transpose: channel 16c + lane % 16 of tokens 32m + 4g .. + 3 and 32m + 16 + 4g .. + 3. Sixteen lanes read a
// 4 x 16 tile, lane j the four values of row j / 4 from column 4 (j % 4) on, and receive its column j.
__device__ __forceinline__ bf16x4 read_tr(const bf16_t *p) {
    const i16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4 *)p);
    return __builtin_bit_cast(bf16x4, r);
}
template <int D> __device__ __forceinline__ bf16x8 col_frag(const bf16_t *tile, int c, int m, int lane) {
    const int row = 32 * m + 4 * (lane >> 4) + ((lane >> 2) & 3), block = 4 * c + (lane & 3);
    const bf16x4 x = read_tr(tile + at<D>(row, block)), y = read_tr(tile + at<D>(row + 16, block));
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}

constexpr int kOnce = 2;        // a buffer access's hint that the line is not worth keeping

// One head of a token-major tensor over a segment's tokens: a load past them reads zeros, a store is dropped.
template <typename T> struct Strip {
    __amdgpu_buffer_rsrc_t r;
    int stride;                                             // bytes from a token to the next
    __device__ __forceinline__ Strip(const T *p, int start, int len, int heads, int h, int D)
        : r(buf_rsrc(p + ((size_t)start * heads + h) * D, len > 0 ? ((len - 1) * heads + 1) * D * (int)sizeof(T) : 0)),
          stride(heads * D * (int)sizeof(T)) {}
    // four values of the token `token` places behind the segment's first
    __device__ __forceinline__ f32x4 load4(int token, int c) const {
        const int off = token * stride + c * (int)sizeof(T);
        if constexpr (sizeof(T) == 2)
            return widen(__builtin_bit_cast(bf16x4, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0)));
        else
            return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
    }
    __device__ __forceinline__ void store4(int token, int c, f32x4 x) const {
        const int off = token * stride + c * (int)sizeof(T);
        if constexpr (sizeof(T) == 2)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, narrow(x)), r, off, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, off, 0, 0);
    }
};

// A chunk's rows of one tensor on their way from memory to LDS: C rows of D values by NT threads.
template <typename T, int D, int C, int NT, int NI> struct Rows {
    static constexpr int PER = 16 / sizeof(T);              // values of a 16-byte load
    static constexpr int N = C * D / PER / NT;              // loads of a thread
    static constexpr int PASS = NT * PER / D;               // rows between them
    static_assert(C * D % (PER * NT) == 0, "chunk rows per thread");
    u32x4 x[N];

    // the rows of tokens token0, token0 + step, ..., counted from the segment's first
    template <int AUX = 0> __device__ __forceinline__ void load(const Strip<T> &s, int token0, int step, int t) {
        const int off = (token0 + step * (t / (D / PER))) * s.stride + t % (D / PER) * 16;
#pragma unroll
        for (int n = 0; n < N; ++n)
            x[n] = __builtin_amdgcn_raw_buffer_load_b128(s.r, off + n * (step * PASS * s.stride), 0, AUX);
    }
    // KEYS: blocks at their places
    template <bool KEYS = false> __device__ __forceinline__ void store(bf16_t *tile, int t) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int u = t + n * NT, row = u / (D / PER), e = u % (D / PER);
            if constexpr (NI == 1) {
                if constexpr (KEYS) {
                    *reinterpret_cast<u32x2 *>(tile + at<D>(row, place(2 * e))) = u32x2{x[n][0], x[n][1]};
                    *reinterpret_cast<u32x2 *>(tile + at<D>(row, place(2 * e + 1))) = u32x2{x[n][2], x[n][3]};
                } else {
                    *reinterpret_cast<u32x4 *>(tile + at<D>(row, 2 * e)) = x[n];
                }
            } else {
                f32x4 y = __builtin_bit_cast(f32x4, x[n]);
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const bf16x4 p = narrow(y);
                    *reinterpret_cast<bf16x4 *>(tile + i * C * D + at<D>(row, KEYS ? place(e) : e)) = p;
                    y -= widen(p);
                }
            }
        }
    }
};

// ---- sums over lanes ---------------------------------------------------------
// over the four groups of 16 lanes, by exchanging rows and halves
__device__ __forceinline__ float group_sum(float x) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
// over the 16 lanes of a group
template <int BY> __device__ __forceinline__ float turned(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + BY, 0xf, 0xf, false));
}
__device__ __forceinline__ float lane_sum(float x) {
    x += turned<8>(x);
    x += turned<4>(x);
    x += turned<2>(x);
    return x + turned<1>(x);
}

// ---- decays -----------------------------------------------------------------
__device__ __forceinline__ double wave_prefix(double x, int lane) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double y = __shfl_up(x, o, 64);
        if (lane >= o) x += y;
    }
    return x;
}

__device__ __forceinline__ float gate_at(const Gate &g, long long token, int h, int H) {
    if (!g.g) return 0.f;
    const float x = g.fixed ? g.g[h] : g.g[token * H + h];
    return x < kMinLog ? kMinLog : x;
}

// Cumulative log2-decays of a segment's rows lo .. hi - 1: whole part in A[i].x, fraction in A[i].y (rows
// before lo: none; rows behind hi - 1, to the end of their chunk of C: as row hi - 1). Row i is the
// segment's token first + i * step. Backwards (step -1) the decay of row i is that of the token before it
// in walking order, and row lo has none. The gates are read by the constructor, ahead of the rows that
// would keep them waiting.
template <int NT, int C> struct SegmentDecays {
    static constexpr int PER = kMaxSegment / NT;            // rows of a thread, at most
    float g[PER];
    int rows, per;
    __device__ __forceinline__ SegmentDecays(const Gate &gate, int h, int H, int start, int first, int step, int lo, int hi,
                                             int t) {
        rows = (hi + C - 1) / C * C;
        per = (rows + NT - 1) / NT;
#pragma unroll
        for (int n = 0; n < PER; ++n) {
            const int i = t * per + n;
            const bool none = n >= per || i < lo || i >= hi || (step < 0 && i == lo);
            g[n] = none ? 0.f : gate_at(gate, start + (first + (step > 0 ? i : 1 - i)), h, H);
        }
    }
    // returns the sum
    __device__ __forceinline__ double write(float2 *A, double *waves, int t) const {
        constexpr int NW = NT / 64;
        const double log2e = 1.4426950408889634;
        double sum = 0.;
#pragma unroll
        for (int n = 0; n < PER; ++n) sum += (double)g[n] * log2e;
        const double incl = wave_prefix(sum, t & 63);
        if ((t & 63) == 63) waves[t >> 6] = incl;
        __syncthreads();
        double run = incl - sum, total = 0.;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < (t >> 6)) run += waves[w];
            total += waves[w];
        }
#pragma unroll
        for (int n = 0; n < PER; ++n) {
            const int i = t * per + n;
            run += (double)g[n] * log2e;
            const double whole = floor(run);
            if (n < per && i < rows) A[i] = float2{(float)whole, (float)(run - whole)};
        }
        __syncthreads();
        return total;
    }
};
__device__ __forceinline__ float decay(float2 to, float2 from) {
    return __builtin_amdgcn_exp2f((to.x - from.x) + (to.y - from.y));
}

// ---- a segment's own contribution to the state -------------------------------
// S^T = sum_i w_i y_i z_i^T over the segment, y [DA] keys and z [DC] values; w_i is the decay
// from row i to the segment's end (`tail`), or from its start through row i.
template <typename T, int DA, int DC, int NI, int C>
__global__ __launch_bounds__(DC * 4, 4) void state_kernel(Segments segs, Gate gate, StateJobs jobs, float *whole, int H,
                                                          int group) {
    constexpr int NT = DC * 4, ND = DA / 16;
    __shared__ bf16_t Y[NI * C * DA], Z[NI * C * DC];
    __shared__ float2 A[kMaxSegment];
    __shared__ float W[C];
    __shared__ double waves[NT / 64];
    const int id = blockIdx.x / H, h = blockIdx.x % H, t = threadIdx.x, lane = t & 63, w = t >> 6, g = lane >> 4;
    Segment x;
    if (!find_segment(segs, id, x)) return;
    const StateJob &job = jobs.job[blockIdx.y];
    if (job.skip_last && x.b == x.blocks - 1) return;
    const int start = x.begin + x.b * segs.L, len = min(segs.L, x.end - start), hs = h / group, HS = H / group;
    const Strip<T> y(static_cast<const T *>(job.y), start, len, job.y_shared ? HS : H, job.y_shared ? hs : h, DA);
    const Strip<T> z(static_cast<const T *>(job.z), start, len, job.z_shared ? HS : H, job.z_shared ? hs : h, DC);
    const SegmentDecays<NT, C> decays(gate, h, H, start, 0, 1, 0, len, t);
    Rows<T, DA, C, NT, NI> ry;
    Rows<T, DC, C, NT, NI> rz;
    ry.load(y, 0, 1, t);
    rz.load(z, 0, 1, t);
    const double total = decays.write(A, waves, t);
    if (t == 0 && blockIdx.y == 0) whole[(size_t)id * H + h] = (float)exp2(total);
    const double tw = floor(total);
    const float2 end = float2{(float)tw, (float)(total - tw)};

    f32x4 S[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) S[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < len; c0 += C) {
        __syncthreads();
        ry.store(Y, t);
        rz.store(Z, t);
        if (t < C) W[t] = job.tail ? decay(end, A[c0 + t]) : decay(A[c0 + t], float2{0.f, 0.f});
        __syncthreads();
        if (c0 + C < len) {
            ry.load(y, c0 + C, 1, t);
            rz.load(z, c0 + C, 1, t);
        }
        const int lane2 = afresh(lane);
#pragma unroll
        for (int m = 0; m < C / 32; ++m) {
            bf16x8 zv[NI], zp[3];
#pragma unroll
            for (int i = 0; i < NI; ++i) zv[i] = col_frag<DC>(Z + i * C * DC, w, m, lane2);
            weigh(zv, W + 32 * m + 4 * g, zp);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                bf16x8 yp[NI];
#pragma unroll
                for (int i = 0; i < NI; ++i) yp[i] = col_frag<DA>(Y + i * C * DA, d, m, lane2);
                S[d] = product<NI, 3>(yp, zp, S[d]);
            }
        }
    }
    float *out = job.out + ((size_t)id * H + h) * DA * DC + (size_t)(16 * w + (lane & 15)) * DA + 4 * g;
#pragma unroll
    for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4 *>(out + 16 * d) = S[d];
}

// ---- states at the segments' borders ------------------------------------------
// Forward: each segment's own sum is replaced by the state before it. Backward (dS): the same
// from the last segment on, for the gradient of the state behind a segment; with both, their
// inner products at every border, which the decays' gradients end on.
__global__ __launch_bounds__(256) void border_kernel(Segments segs, BorderArgs a, int H, int DD) {
    __shared__ float sums[4];
    const int n = blockIdx.x / H, h = blockIdx.x % H, t = threadIdx.x;
    const size_t e = ((size_t)blockIdx.y * 256 + t) * 4;
    int begin, end;
    sequence_bounds(segs, n, begin, end);
    const int blocks = block_count(segs, end - begin), id0 = first_id(segs, n, begin);
    const size_t own = ((size_t)n * H + h) * DD + e, step = (size_t)H * DD;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    auto load = [&](const float *p) { return *reinterpret_cast<const f32x4 *>(p); };
    f32x4 cur = a.S0 ? load(a.S0 + own) : zero;
    float *p = a.states + ((size_t)id0 * H + h) * DD + e;
    const float *g = a.whole + (size_t)id0 * H + h;
    const int sums_wanted = a.all ? blocks : blocks - 1;     // the last segment's own sum: only its state's gradient needs it
#pragma unroll 4
    for (int b = 0; b < sums_wanted; ++b) {
        const f32x4 add = load(p + b * step);
        *reinterpret_cast<f32x4 *>(p + b * step) = cur;
        cur = cur * g[(size_t)b * H] + add;
    }
    if (!a.all) {
        *reinterpret_cast<f32x4 *>(p + (blocks - 1) * step) = cur;
        return;
    }
    f32x4 after = cur;                                       // the state behind segment b
    cur = a.dS_out ? load(a.dS_out + own) : zero;
    float *d = a.grads + ((size_t)id0 * H + h) * DD + e;
    float *dots = a.dots + (((size_t)id0 * H + h) * gridDim.y + blockIdx.y);
    auto inner = [&](float *to) {
        const float x = warp_sum(cur.x * after.x + cur.y * after.y + cur.z * after.z + cur.w * after.w);
        if ((t & 63) == 0) sums[t >> 6] = x;
        __syncthreads();
        if (t == 0) *to = (sums[0] + sums[1]) + (sums[2] + sums[3]);
        __syncthreads();
    };
    for (int b = blocks - 1; b >= 0; --b) {
        const f32x4 add = load(d + b * step), before = load(p + b * step);
        *reinterpret_cast<f32x4 *>(d + b * step) = cur;
        inner(dots + (size_t)b * H * gridDim.y);
        after = before;
        cur = cur * g[(size_t)b * H] + add;
    }
    inner(a.starts + ((size_t)n * H + h) * gridDim.y + blockIdx.y);
    if (a.dS0) *reinterpret_cast<f32x4 *>(a.dS0 + own) = cur;
}

// ---- the outputs of a segment ---------------------------------------------------
template <typename TO> __device__ __forceinline__ void store4(TO *p, f32x4 x);
template <> __device__ __forceinline__ void store4<float>(float *p, f32x4 x) { *reinterpret_cast<f32x4 *>(p) = x; }
template <> __device__ __forceinline__ void store4<bf16_t>(bf16_t *p, f32x4 x) {
    *reinterpret_cast<bf16x4 *>(p) = narrow(x);
}

// F(x, y, z): queries x and keys y of DA channels, values z of DC. T: the tensors' type, in NI
// bf16 parts; TO the outputs'; NX parts of states and scores; chunks of C tokens; DOT: the
// sum over channels of each output row (its own token's share left out) times a row of `with`.
template <typename T, typename TO, int DA, int DC, int NI, int NX, int C, bool DOT>
__global__ __launch_bounds__(DC * 4, 4) void output_kernel(Segments segs, Gate gate, OutputJobs jobs, int H, int group) {
    constexpr int NT = DC * 4, NW = DC / 16, NC = C / 16, ND = DA / 16, TILES = NC * (NC + 1) / 2;
    constexpr bool ROWS = sizeof(TO) == 2 && DC == 128 && DC <= DA && !DOT;
    // ROWS: outputs leave through the queries' tile, whole rows at a time (8k forward 125 -> 115 us). Rows of 64 values are
    // half as long and gain 1% or nothing (8k x 32 x 64: 62 -> 61 us, 128 x 64 86 either way); with DOT six registers spill at
    // 128 x 128 (8k gradient 378 -> 400 us)
    __shared__ bf16_t X[NI * C * DA], Y[NI * C * DA], Z[NI * C * DC];
    __shared__ bf16x4 P[NC * NC / 4 + NC / 2][NX][64][2];  // scores(i, m): 16 query tokens, 32 key tokens, the two halves of the latter
    auto scores = [](int i, int m) { return (i / 2) * (i / 2 + 1) + (i & 1) * (i / 2 + 1) + m; };
    __shared__ float2 A[kMaxSegment];
    __shared__ float R[C], W[C];                           // decays from the chunk's start through a row, and from a row to its end
    __shared__ double waves[NW];
    __shared__ float own[DOT ? C : 1], dots[DOT ? NW : 1][DOT ? C : 1], past[DOT ? NW : 1];
    const int id = blockIdx.x / H, h = blockIdx.x % H, t = threadIdx.x, lane = t & 63, w = t >> 6, g = lane >> 4,
              col = lane & 15;
    Segment s;
    if (!find_segment(segs, id, s)) return;
    const OutputJob &job = jobs.job[blockIdx.y];
    const bool dot = DOT && (sizeof(T) == 2 || job.with);   // uniform; in fp32 a job may do without
    const int hs = h / group, HS = H / group;
    if (job.zero_rows) {
        // rows of no sequence lie before the first one and behind the last one
        TO *out = static_cast<TO *>(job.out) + (job.out_shared ? hs : h) * DC;
        const size_t os = (size_t)(job.out_shared ? HS : H) * DC;
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        if (s.n == 0 && s.b == 0)
            for (size_t u = t; u < (size_t)s.begin * (DC / 4); u += NT) store4(out + u / (DC / 4) * os + u % (DC / 4) * 4, zero);
        if (s.n == segs.N - 1 && s.b == s.blocks - 1)
            for (size_t u = t; u < (size_t)(segs.T_total - s.end) * (DC / 4); u += NT)
                store4(out + (s.end + u / (DC / 4)) * os + u % (DC / 4) * 4, zero);
    }
    // rows lo .. hi - 1; backwards the empty rows come first, so that chunks have the same borders both ways
    const int start = s.begin + s.b * segs.L, len = min(segs.L, s.end - start), step = job.back ? -1 : 1;
    const int hi = job.back ? (len + C - 1) / C * C : len, lo = hi - len, first = job.back ? hi - 1 : 0;
    const Strip<T> x(static_cast<const T *>(job.x), start, len, job.x_shared ? HS : H, job.x_shared ? hs : h, DA);
    const Strip<T> y(static_cast<const T *>(job.y), start, len, job.y_shared ? HS : H, job.y_shared ? hs : h, DA);
    const Strip<T> z(static_cast<const T *>(job.z), start, len, job.z_shared ? HS : H, job.z_shared ? hs : h, DC);
    const Strip<TO> out(static_cast<const TO *>(job.out), start, len, job.out_shared ? HS : H, job.out_shared ? hs : h, DC);
    const Strip<T> with(static_cast<const T *>(dot ? job.with : job.z), start, dot ? len : 0, HS, hs, DC);
    const SegmentDecays<NT, C> decays(gate, h, H, start, first, step, lo, hi, t);
    // the state before the segment, transposed: column = value channel, rows = key channels
    f32x4 S[ND];
    const float *Sp = job.S + ((size_t)(job.border ? id : s.n) * H + h) * DA * DC;
    if (!job.S) {
#pragma unroll
        for (int d = 0; d < ND; ++d) S[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    } else if (job.key_rows) {                             // as it lies: a row per key channel
        const float *p = Sp + 8 * g * DC + 16 * w + col;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[d][e] = p[(channel(d, 0) + e) * DC];
    } else {
        const float *p = Sp + (16 * w + col) * DA + 8 * g;
#pragma unroll
        for (int d = 0; d < ND; ++d) S[d] = *reinterpret_cast<const f32x4 *>(p + channel(d, 0));
    }
    Rows<T, DA, C, NT, NI> rx, ry;
    Rows<T, DC, C, NT, NI> rz;
    rx.template load<kOnce>(x, first, step, t);
    ry.load(y, first, step, t);
    rz.load(z, first, step, t);
    decays.write(A, waves, t);
    const bool last = job.back ? s.b == 0 : s.b == s.blocks - 1;
    const bool keep = last && job.S_out;

    for (int c0 = 0; c0 < hi; c0 += C) {
        __syncthreads();
        rx.store(X, t);
        ry.template store<true>(Y, t);
        rz.store(Z, t);
        if (t < C) {
            R[t] = decay(A[c0 + t], c0 ? A[c0 - 1] : float2{0.f, 0.f});
            W[t] = decay(A[c0 + C - 1], A[c0 + t]);
        }
        __syncthreads();

        // scores, transposed: rows = key tokens, column = query token
        for (int tile = w; tile < TILES; tile += NW) {
            const int ti = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3, ts = tile - ti * (ti + 1) / 2;
            const int lane2 = afresh(lane), c2 = lane2 & 15, g2 = lane2 >> 4;
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < DA / 32; ++m) {
                bf16x8 ky[NI], qx[NI];
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    ky[i] = key_frag<DA>(Y + i * C * DA, 16 * ts + c2, m, g2);
                    qx[i] = query_frag<DA>(X + i * C * DA, 16 * ti + c2, m, g2);
                }
                acc = product<NI, NI>(ky, qx, acc);
            }
            const int i = 16 * ti + col, sr = 16 * ts + 4 * g;
            const float2 ai = A[c0 + i];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float dec = decay(ai, A[c0 + sr + r]);
                if (dot && sr + r == i) own[i] = acc[r];
                acc[r] = sr + r < i + !dot ? acc[r] * dec : 0.f;
            }
#pragma unroll
            for (int j = 0; j < NX; ++j) {
                const bf16x4 p = narrow(acc);
                P[scores(ti, ts / 2)][j][lane][ts & 1] = p;
                if (ts == ti && !(ts & 1)) P[scores(ti, ts / 2)][j][lane][1] = bf16x4{};     // later keys than any query's
                acc -= widen(p);
            }
        }
        // e^{a_i} S x_i
        f32x4 O[NC];
        const int lane2 = afresh(lane), c2 = lane2 & 15, g2 = lane2 >> 4;
#pragma unroll
        for (int i = 0; i < NC; ++i) O[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < DA / 32; ++m) {
            bf16x8 sp[NX];
            cut<NX>(__builtin_shufflevector(S[2 * m], S[2 * m + 1], 0, 1, 2, 3, 4, 5, 6, 7), sp);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                bf16x8 qx[NI];
#pragma unroll
                for (int j = 0; j < NI; ++j) qx[j] = query_frag<DA>(X + j * C * DA, 16 * i + c2, m, g2);
                O[i] = product<NX, NI>(sp, qx, O[i]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) O[i] *= R[16 * i + col];
        if (dot) {
            // what the chunk's rows have from the state, against `with`
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const f32x4 y4 = with.load4(first + step * (c0 + 16 * i + col), 16 * w + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum += O[i][e] * y4[e];
            }
            sum = group_sum(lane_sum(sum));
            if (lane == 0) past[w] = sum;
        }
        const float over = R[C - 1];
        __syncthreads();
        // the next chunk's rows come while the values are summed: scores times them, and their share of the state
        const bool more = c0 + C < hi;
        if (more) {
            rx.template load<kOnce>(x, first + step * (c0 + C), step, t);
            ry.load(y, first + step * (c0 + C), step, t);
            rz.load(z, first + step * (c0 + C), step, t);
        }
        const int lane3 = afresh(lane);
#pragma unroll
        for (int m = 0; m < C / 32; ++m) {
            bf16x8 zv[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) zv[i] = col_frag<DC>(Z + i * C * DC, w, m, lane3);
#pragma unroll
            for (int i = 2 * m; i < NC; ++i) {
                bf16x8 p[NX];
#pragma unroll
                for (int j = 0; j < NX; ++j) p[j] = *reinterpret_cast<const bf16x8 *>(P[scores(i, m)][j][lane]);
                O[i] = product<NI, NX>(zv, p, O[i]);
            }
        }
        // out: a lane has four channels of token i; rows of no token fall behind the segment's end
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int token = first + step * (c0 + 16 * i + col), c = 16 * w + 4 * g;
            if (dot) {
                const f32x4 y4 = with.load4(token, c);
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) sum += O[i][e] * y4[e];
                sum = group_sum(sum);
                if (g == 0) dots[w][16 * i + col] = sum;
                f32x4 z4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int p = NI - 1; p >= 0; --p)
                    z4 += widen(*reinterpret_cast<const bf16x4 *>(Z + p * C * DC + at<DC>(16 * i + col, 4 * w + g)));
                O[i] += z4 * own[16 * i + col];
            }
            if constexpr (ROWS) *reinterpret_cast<bf16x4 *>(X + at<DC>(16 * i + col, 4 * w + g)) = narrow(O[i]);
            else out.store4(token, c, O[i]);
        }
        if constexpr (ROWS) {
            __syncthreads();
#pragma unroll
            for (int u = t; u < C * DC / 8; u += NT) {
                const int row = u / (DC / 8), e = u % (DC / 8);
                __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const u32x4 *>(X + at<DC>(row, 2 * e)), out.r,
                                                       (first + step * (c0 + row)) * out.stride + e * 16, 0, kOnce);
            }
        }
        if (more || keep) {
            __builtin_amdgcn_s_setprio(1);
            const int lane4 = afresh(lane);
#pragma unroll
            for (int d = 0; d < ND; ++d) S[d] *= over;
#pragma unroll
            for (int m = 0; m < C / 32; ++m) {
                bf16x8 zv[NI], zp[3];
#pragma unroll
                for (int i = 0; i < NI; ++i) zv[i] = col_frag<DC>(Z + i * C * DC, w, m, lane4);
                weigh(zv, W + 32 * m + 4 * g, zp);
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    bf16x8 ky[NI];
#pragma unroll
                    for (int i = 0; i < NI; ++i) ky[i] = col_frag<DA>(Y + i * C * DA, d, m, lane4);
                    S[d] = product<NI, 3>(ky, zp, S[d]);
                }
            }
            __builtin_amdgcn_s_setprio(0);
        }
        if (dot) {
            __syncthreads();
            if (t < C && c0 + t >= lo && c0 + t < hi) {
                float d = 0.f;
#pragma unroll
                for (int i = 0; i < NW; ++i) d += dots[i][t];
                job.dot[(size_t)h * segs.T_total + (size_t)(start + first + step * (c0 + t))] = d;
            }
            if (t == 0) {
                float d = 0.f;
#pragma unroll
                for (int i = 0; i < NW; ++i) d += past[i];
                const int chunk = job.back ? hi / C - 1 - c0 / C : c0 / C;
                job.past[((size_t)id * H + h) * (segs.L / C) + chunk] = d;
            }
        }
    }
    if (keep) {
        // backwards, the decay of the segment's first token is still to be applied
        const float rest = job.back && len > 0 ? expf(gate_at(gate, start, h, H)) : 1.f;
        float *so = job.S_out + ((size_t)s.n * H + h) * DA * DC + (size_t)(16 * w + col) * DA + 8 * g;
#pragma unroll
        for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4 *>(so + channel(d, 0)) = S[d] * rest;
    }
}

// ---- the decays' gradients --------------------------------------------------------
// What passes the decay of token t: with G(p) = <gradient of the state behind token p, that state>,
//     dg_t = G(t - 1) = G(p) + sum_{t <= i <= p} (q_i . dq_i - k_i . dk_i)
// (a token's own share left out of both). The terms of a long sum cancel, and their rounding would
// not, so it never runs further than a chunk: G at the chunks' borders follows from G at the segment's
// end by what the chunks' tokens have from the state (read, q . dq) and from its gradient (past,
// k . dk) alone, likewise from the segment's start, and inside a chunk from both of its borders. Either sum is off by
// some 2^-24 of what went into it, G and all terms, which strong decays make e^g times as much from a token to the
// next (in opposite directions), so the two are weighted by the squares of those magnitudes, each end's sum by the
// other's: 64 tokens of g = -8 and -16 between two states 2.5e-4 and 2.6 (weights by distance) -> 6e-7 relative.
// C tokens a chunk, a wavefront each; a workgroup a (segment, head); sums in 64 bits and a fixed order. `starts`: G before each
// sequence's first token, nullptr: zero, or (only_end) not known.
struct Carried { double x, size; };         // a sum, and the magnitudes that went into it
__device__ __forceinline__ Carried joined(Carried a, Carried b) {
    const double aa = a.size * a.size, bb = b.size * b.size;
    const double w = aa + bb > 0. ? aa / (aa + bb) : 0.5;
    return Carried{(1. - w) * a.x + w * b.x, fmin(a.size, b.size)};
}
__global__ __launch_bounds__(256) void decay_grad_kernel(Segments segs, Gate gate, const float *__restrict__ rows,
                                                         const float *__restrict__ cols, const float *__restrict__ read,
                                                         const float *__restrict__ past, const float *__restrict__ dots,
                                                         const float *__restrict__ starts, bool only_end, int parts, int C,
                                                         float *__restrict__ dg, double *__restrict__ sums, int H,
                                                         int zero_rows) {
    __shared__ double chunk_sums[kMaxSegment / 32];
    const int id = blockIdx.x / H, h = blockIdx.x % H, t = threadIdx.x, lane = t & 63, w = t >> 6;
    Segment s;
    if (!find_segment(segs, id, s)) {
        if (gate.fixed && t == 0) sums[(size_t)id * H + h] = 0.;
        return;
    }
    if (zero_rows && !gate.fixed) {
        if (s.n == 0 && s.b == 0)
            for (int i = t; i < s.begin; i += 256) dg[(size_t)i * H + h] = 0.f;
        if (s.n == segs.N - 1 && s.b == s.blocks - 1)
            for (int i = s.end + t; i < segs.T_total; i += 256) dg[(size_t)i * H + h] = 0.f;
    }
    const int start = s.begin + s.b * segs.L, len = min(segs.L, s.end - start);
    const size_t at = (size_t)h * segs.T_total + start, cell = (size_t)id * H + h;
    const int chunks = (len + C - 1) / C;
    const float *rd = read + cell * (segs.L / C), *pt = past + cell * (segs.L / C);
    auto total = [&](const float *p) {
        Carried x{0., 0.};
        for (int i = 0; i < parts; ++i) x = Carried{x.x + p[i], x.size + fabs((double)p[i])};
        return x;
    };
    // from c onwards by chunk i's tokens, and back
    auto term = [&](int i) { return Carried{(double)rd[i] - (double)pt[i], fabs((double)rd[i]) + fabs((double)pt[i])}; };
    auto plus = [](Carried a, Carried b) { return Carried{a.x + b.x, a.size + b.size}; };
    auto minus = [](Carried a, Carried b) { return Carried{a.x - b.x, a.size + b.size}; };
    const Carried last = total(dots + cell * parts);
    const Carried first = s.b > 0 ? total(dots + (cell - H) * parts)
                          : starts ? total(starts + ((size_t)s.n * H + h) * parts) : Carried{0., 0.};
    for (int c = w; c < chunks; c += 4) {                    // C <= 64 tokens, one a lane
        Carried to_c{0., 0.}, behind{0., 0.};                // what G loses up to this chunk, and behind it
        for (int i = 0; i < c; ++i) to_c = plus(to_c, term(i));
        for (int i = chunks - 1; i > c; --i) behind = plus(behind, term(i));
        const Carried own = term(c), from_end = plus(last, behind);
        const Carried begin = only_end ? plus(plus(from_end, own), to_c) : first, from_start = minus(begin, to_c);
        const Carried before = joined(from_start, plus(from_end, own)), after = joined(minus(from_start, own), from_end);
        const int i = c * C + lane, n = min(C, len - c * C);
        const double rw = lane < n ? rows[at + i] : 0., cl = lane < n ? cols[at + i] : 0.;
        const Carried x{rw - cl, fabs(rw) + fabs(cl)};
        const Carried upto{wave_prefix(x.x, lane), wave_prefix(x.size, lane)};
        const Carried rest{__shfl(upto.x, 63, 64) - upto.x, __shfl(upto.size, 63, 64) - upto.size};
        double d = joined(Carried{before.x - (upto.x - x.x), before.size + (upto.size - x.size)},
                          Carried{after.x + rest.x + x.x, after.size + rest.size + x.size}).x;
        // at -104 the decay is zero, and its gradient too
        if (lane >= n || gate.g[gate.fixed ? h : (size_t)(start + i) * H + h] <= kMinLog) d = 0.;
        if (gate.fixed) {
            d = wave_prefix(d, lane);
            if (lane == 63) chunk_sums[c] = d;
        } else if (lane < n) {
            dg[(size_t)(start + i) * H + h] = (float)d;
        }
    }
    if (gate.fixed) {
        __syncthreads();
        if (t == 0) {
            double sum = 0.;
            for (int c = 0; c < chunks; ++c) sum += chunk_sums[c];
            sums[cell] = sum;
        }
    }
}

// A fixed decay's gradient: the sum over all segments, in a fixed order.
__global__ __launch_bounds__(64) void fixed_grad_kernel(const double *__restrict__ sums, float *__restrict__ dg, int ids, int H) {
    const int h = blockIdx.x, lane = threadIdx.x;
    double x = 0.;
    for (int i = lane; i < ids; i += 64) x += sums[(size_t)i * H + h];
    x = wave_prefix(x, lane);
    if (lane == 63) dg[h] = (float)x;
}

// The gradients of shared query and key heads: the sums over their groups' heads.
template <typename TO>
__global__ __launch_bounds__(256) void share_kernel(Segments segs, const float *part0, const float *part1, TO *out0, TO *out1,
                                                    int H, int group, int D, int zero_bits) {
    const float *part = blockIdx.y ? part1 : part0;
    TO *out = blockIdx.y ? out1 : out0;
    const bool zero_rows = (zero_bits >> blockIdx.y) & 1;
    const size_t u = (size_t)blockIdx.x * 256 + threadIdx.x;
    const int HS = H / group, q = D / 4;
    const size_t token = u / ((size_t)HS * q);
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    bool live = true;
    if (segs.cu) {
        int b0, b1, e0, e1;
        sequence_bounds(segs, 0, b0, e0);
        sequence_bounds(segs, segs.N - 1, b1, e1);
        live = token >= (size_t)b0 && token < (size_t)e1;
    }
    if (token >= (size_t)segs.T_total || (!live && !zero_rows)) return;
    const int hs = (int)(u / q % HS), c = (int)(u % q) * 4;
    if (live)
        for (int i = 0; i < group; ++i) sum += *reinterpret_cast<const f32x4 *>(part + (token * H + hs * group + i) * D + c);
    store4(out + (token * HS + hs) * D + c, sum);
}

// ---- host -----------------------------------------------------------------------
// Tokens a segment, a power of two: the least that leaves one round of workgroups at two a CU, which is what the LDS of
// the bf16 kernels at 128 x 128 allows; more segments would be traffic (8 D^2 bytes each and pass) for nothing. In us, with
// half as many tokens a segment, these, twice as many:
//     forward, bf16: 8192 x 32 heads 137, 115, 130; 4832 packed x 16 (128 x 64) 53, 51, 61; 8192 x 32 at 64 x 64 (three workgroups
//     a CU) 68, 62, 78; 128 x 64 100, 86, 108; 64 x 128 96, 85, 95; 5000 x 8 45 with 64 tokens, 58 with 128
//     forward, fp32: 4096 x 16 at 128 x 128 (one workgroup a CU, so two rounds) 114, 87, 75; at 64 x 64 51, 41, 44
//     gradient, whose launches hold two or three jobs: bf16 8192 x 32 431, 378, 378; 64 x 64 218, 219, 225; fp32 4096 x 16 309, 242, 219
// So fp32 at 128 x 128 would take 10 to 14% less with segments twice as long; the rule is that of the others.
//
// Short sequences of a dense batch (`longest`: no sequence has more tokens) are one segment each, and their states need no
// passes of their own: 16 x 200 tokens x 8 heads 38 -> 25 us, 128 x 8 22 -> 15. `few`, 256 tokens, or 128 where
// T_total * H is below 16384: one of 256 x 8 has too few workgroups that way (gradient 34 -> 54 us). The lengths of packed
// sequences are not known on the host, so T_total stands for the longest: 64 x 256 x 32 heads take 157 us dense and 199
// packed. The gradient needs the passes where dS_out is given. A longest below T_total never makes segments shorter
// than T_total alone would, which the workspace is sized by.
int segment_length(long long longest, long long T_total, int H) {
    const long long L = T_total * H / 512;
    int p = 64;
    while (p < kMaxSegment && p < L) p *= 2;
    const long long few = T_total * H >= 64 * 256 ? 256 : 128;
    const long long whole = T_total <= few ? T_total : longest <= few ? longest : 0;
    while (p < whole) p *= 2;
    return p;
}
long long id_count(long long T_total, int N, int L) { return T_total / L + N; }
size_t round_up(size_t x) { return (x + 255) & ~(size_t)255; }

// The workspace of a call, piece after piece.
struct Carver {
    char *p;
    size_t used = 0;
    template <typename T> T *take(size_t n) {
        T *r = reinterpret_cast<T *>(p + used);
        used += round_up(n * sizeof(T));
        return r;
    }
};
struct ForwardSpace { float *states, *whole; };
struct BackwardSpace {
    float *states, *grads, *whole, *dots, *starts, *rows, *cols, *read, *past, *dq, *dk;
    double *sums;
};
ForwardSpace carve_forward(Carver &c, int N, long long longest, long long T_total, int H, int Dk, int Dv, int L) {
    ForwardSpace s{};
    if (longest <= L) return s;                             // every sequence is one segment
    const size_t cells = (size_t)id_count(T_total, N, L) * H;
    s.states = c.take<float>(cells * Dk * Dv);
    s.whole = c.take<float>(cells);
    return s;
}
BackwardSpace carve_backward(Carver &c, int N, long long T_total, int H, int group, int Dk, int Dv, int L) {
    BackwardSpace s{};
    const size_t cells = (size_t)id_count(T_total, N, L) * H;
    s.states = c.take<float>(cells * Dk * Dv);
    s.grads = c.take<float>(cells * Dk * Dv);
    s.whole = c.take<float>(cells);
    s.dots = c.take<float>(cells * (Dk * Dv / 1024));
    s.starts = c.take<float>((size_t)N * H * (Dk * Dv / 1024));
    s.sums = c.take<double>(cells);
    s.rows = c.take<float>((size_t)T_total * H);
    s.cols = c.take<float>((size_t)T_total * H);
    s.read = c.take<float>(cells * (L / 32));              // chunks of 32 tokens at least
    s.past = c.take<float>(cells * (L / 32));
    if (group > 1) {
        s.dq = c.take<float>((size_t)T_total * H * Dk);
        s.dk = c.take<float>((size_t)T_total * H * Dk);
    }
    return s;
}

template <typename T> struct Parts { static constexpr int N = 1, C = 64; };
template <> struct Parts<float> { static constexpr int N = 3, C = 32; };

template <typename T, int DA, int DC>
hipError_t run_states(const Segments &segs, const Gate &gate, const StateJobs &jobs, int n, float *whole, int H, int group,
                      hipStream_t stream) {
    const unsigned ids = (unsigned)id_count(segs.T_total, segs.N, segs.L);
    hipLaunchKernelGGL((state_kernel<T, DA, DC, Parts<T>::N, Parts<T>::C>), dim3(ids * H, n), dim3(DC * 4), 0, stream, segs,
                       gate, jobs, whole, H, group);
    return hipGetLastError();
}
hipError_t run_borders(const Segments &segs, const BorderArgs &a, int H, int DD, hipStream_t stream) {
    hipLaunchKernelGGL(border_kernel, dim3((unsigned)(segs.N * H), DD / 1024), dim3(256), 0, stream, segs, a, H, DD);
    return hipGetLastError();
}
template <typename T, typename TO, int DA, int DC, int NX, bool DOT>
hipError_t run_outputs(const Segments &segs, const Gate &gate, const OutputJobs &jobs, int n, int H, int group,
                       hipStream_t stream) {
    const unsigned ids = (unsigned)id_count(segs.T_total, segs.N, segs.L);
    hipLaunchKernelGGL((output_kernel<T, TO, DA, DC, Parts<T>::N, NX, Parts<T>::C, DOT>), dim3(ids * H, n), dim3(DC * 4),
                       0, stream, segs, gate, jobs, H, group);
    return hipGetLastError();
}

template <typename T, int DK, int DV> hipError_t prefill(const LinPrefillArgs &a) {
    const long long T_total = (long long)a.B * a.T;
    const long long longest = a.cu_seqlens ? T_total : a.T;
    const int L = segment_length(longest, T_total, a.H), group = a.H / a.Hk;
    const Segments segs{a.cu_seqlens, a.N, a.T, (int)T_total, L, __builtin_ctz((unsigned)L)};
    const Gate gate{a.g, a.fixed};
    Carver c{static_cast<char *>(a.ws)};
    const ForwardSpace ws = carve_forward(c, a.N, longest, T_total, a.H, DK, DV, L);
    OutputJobs out{};
    OutputJob &o = out.job[0];
    o.x = a.q; o.y = a.k; o.z = a.v; o.out = a.out; o.S = a.S0; o.S_out = a.S_out;
    o.x_shared = o.y_shared = true;
    o.zero_rows = a.zero_rows;
    if (ws.states) {
        StateJobs st{};
        st.job[0] = StateJob{a.k, a.v, ws.states, true, false, true, true};
        hipError_t e = run_states<T, DK, DV>(segs, gate, st, 1, ws.whole, a.H, group, a.stream);
        if (e != hipSuccess) return e;
        BorderArgs b{};
        b.S0 = a.S0; b.states = ws.states; b.whole = ws.whole;
        e = run_borders(segs, b, a.H, DK * DV, a.stream);
        if (e != hipSuccess) return e;
        o.S = ws.states;
        o.border = true;
    }
    if constexpr (sizeof(T) == 2)
        if (a.out_dt == Dt::BF16) return run_outputs<T, bf16_t, DK, DV, 2, false>(segs, gate, out, 1, a.H, group, a.stream);
    return run_outputs<T, float, DK, DV, 3, false>(segs, gate, out, 1, a.H, group, a.stream);
}

template <typename T, int DK, int DV> hipError_t backward(const LinBackwardArgs &a) {
    const long long T_total = (long long)a.B * a.T;
    const long long longest = a.cu_seqlens ? T_total : a.T;
    const int L = segment_length(longest, T_total, a.H), group = a.H / a.Hk, ids = (int)id_count(T_total, a.N, L);
    // sequences of one segment, whose last state has no gradient: states and gradients start from what the caller gives
    const bool borders = longest > L || a.dS_out;
    const Segments segs{a.cu_seqlens, a.N, a.T, (int)T_total, L, __builtin_ctz((unsigned)L)};
    const Gate gate{a.g, a.fixed};
    Carver c{static_cast<char *>(a.ws)};
    const BackwardSpace ws = carve_backward(c, a.N, T_total, a.H, group, DK, DV, L);
    hipError_t e = hipSuccess;
    if (borders) {
        StateJobs st{};
        st.job[0] = StateJob{a.k, a.v, ws.states, true, false, true, false};
        st.job[1] = StateJob{a.q, a.dout, ws.grads, true, false, false, false};
        e = run_states<T, DK, DV>(segs, gate, st, 2, ws.whole, a.H, group, a.stream);
        if (e != hipSuccess) return e;
        BorderArgs b{};
        b.S0 = a.S0; b.dS_out = a.dS_out; b.states = ws.states; b.grads = ws.grads; b.dS0 = a.dS0; b.dots = ws.dots; b.starts = ws.starts;
        b.whole = ws.whole; b.all = true;
        e = run_borders(segs, b, a.H, DK * DV, a.stream);
        if (e != hipSuccess) return e;
    }

    // dq = F(dout, v, k) from the states, dk = F(v, dout, q) and dv = F(k, q, dout) from their gradients
    OutputJobs qk{}, vj{};
    OutputJob &q = qk.job[0], &k = qk.job[1], &v = vj.job[0];
    q.x = a.dout; q.y = a.v; q.z = a.k; q.with = a.q; q.dot = ws.rows; q.past = ws.read; q.S = borders ? ws.states : a.S0;
    k.x = a.v; k.y = a.dout; k.z = a.q; k.with = a.k; k.dot = ws.cols; k.past = ws.past; k.S = borders ? ws.grads : nullptr;
    v.x = a.k; v.y = a.q; v.z = a.dout; v.S = borders ? ws.grads : nullptr; v.out = a.dv;
    v.S_out = borders ? nullptr : a.dS0;
    q.z_shared = k.z_shared = v.x_shared = v.y_shared = true;
    q.border = k.border = v.border = borders;
    q.key_rows = k.key_rows = k.back = v.back = true;
    v.zero_rows = a.zero_rows & 4;
    if (group == 1) {
        q.out = a.dq; k.out = a.dk;
        q.out_shared = k.out_shared = true;
        q.zero_rows = a.zero_rows & 1;
        k.zero_rows = a.zero_rows & 2;
    } else {
        q.out = ws.dq; k.out = ws.dk;
    }
    // fp32, square states: all three in one launch (their precision is the same), which small batches feel
    const bool together = sizeof(T) == 4 && DK == DV && a.g;
    if (together) qk.job[2] = v;
    if (group == 1 && sizeof(T) == 2) {
        if constexpr (sizeof(T) == 2)
            e = a.g ? run_outputs<T, bf16_t, DV, DK, 3, true>(segs, gate, qk, 2, a.H, group, a.stream)
                    : run_outputs<T, bf16_t, DV, DK, 2, false>(segs, gate, qk, 2, a.H, group, a.stream);
    } else {
        e = a.g ? run_outputs<T, float, DV, DK, 3, true>(segs, gate, qk, together ? 3 : 2, a.H, group, a.stream)
                : run_outputs<T, float, DV, DK, 3, false>(segs, gate, qk, 2, a.H, group, a.stream);
    }
    if (e != hipSuccess) return e;
    if constexpr (sizeof(T) == 2) e = run_outputs<T, bf16_t, DK, DV, 2, false>(segs, gate, vj, 1, a.H, group, a.stream);
    else if (!together) e = run_outputs<T, float, DK, DV, 3, false>(segs, gate, vj, 1, a.H, group, a.stream);
    if (e != hipSuccess) return e;
    if (group > 1) {
        const unsigned blocks = (unsigned)(((size_t)T_total * a.Hk * (DK / 4) + 255) / 256);
        hipLaunchKernelGGL((share_kernel<T>), dim3(blocks, 2), dim3(256), 0, a.stream, segs, ws.dq, ws.dk, static_cast<T *>(a.dq),
                           static_cast<T *>(a.dk), a.H, group, DK, a.zero_rows & 3);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.g) {
        hipLaunchKernelGGL(decay_grad_kernel, dim3((unsigned)(ids * a.H)), dim3(256), 0, a.stream, segs, gate, ws.rows, ws.cols,
                           ws.read, ws.past, ws.dots, borders ? ws.starts : nullptr, !borders && a.S0, borders ? DK * DV / 1024 : 0, Parts<T>::C, a.dg, ws.sums, a.H, a.zero_rows & 8);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (a.fixed) {
            hipLaunchKernelGGL(fixed_grad_kernel, dim3((unsigned)a.H), dim3(64), 0, a.stream, ws.sums, a.dg, ids, a.H);
            e = hipGetLastError();
        }
    }
    return e;
}

// No tokens at all: the states pass through.
__global__ __launch_bounds__(256) void pass_kernel(const float *from, float *to, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) to[i] = from ? from[i] : 0.f;
}
hipError_t pass(const float *from, float *to, size_t n, hipStream_t stream) {
    if (!to || from == to) return hipSuccess;
    hipLaunchKernelGGL(pass_kernel, dim3((unsigned)(n / 4096 + 1 < 4096 ? n / 4096 + 1 : 4096)), dim3(256), 0, stream, from, to, n);
    return hipGetLastError();
}

template <typename T, typename A, typename F> hipError_t by_width(const A &a, F) {
    if (a.Dk == 64) return a.Dv == 64 ? F::template run<T, 64, 64>(a) : F::template run<T, 64, 128>(a);
    return a.Dv == 64 ? F::template run<T, 128, 64>(a) : F::template run<T, 128, 128>(a);
}
struct Prefill { template <typename T, int DK, int DV> static hipError_t run(const LinPrefillArgs &a) { return prefill<T, DK, DV>(a); } };
struct Backward { template <typename T, int DK, int DV> static hipError_t run(const LinBackwardArgs &a) { return backward<T, DK, DV>(a); } };

}  // namespace

size_t lin_prefill_workspace(int N, long long T_total, int H, int Dk, int Dv) {
    Carver c{nullptr};
    carve_forward(c, N, T_total, T_total, H, Dk, Dv, segment_length(T_total, T_total, H));
    return c.used;
}
size_t lin_backward_workspace(int N, long long T_total, int H, int Hk, int Dk, int Dv) {
    if (T_total == 0) return 0;
    Carver c{nullptr};
    carve_backward(c, N, T_total, H, H / Hk, Dk, Dv, segment_length(T_total, T_total, H));
    return c.used;
}
bool lin_chunk_fits(int N, long long T_total, int H) {
    // workgroups of a launch times their threads stay below 2^32, a segment's tokens below 2^31 bytes
    return H <= 4096 && id_count(T_total, N, segment_length(T_total, T_total, H)) * H < (1ll << 23) && T_total * H < (1ll << 27);
}
hipError_t launch_lin_prefill(const LinPrefillArgs &a) {
    if ((long long)a.B * a.T == 0) return pass(a.S0, a.S_out, (size_t)a.N * a.H * a.Dk * a.Dv, a.stream);
    return a.io == Dt::F32 ? by_width<float>(a, Prefill{}) : by_width<bf16_t>(a, Prefill{});
}
hipError_t launch_lin_backward(const LinBackwardArgs &a) {
    if ((long long)a.B * a.T == 0) {
        const hipError_t e = pass(a.dS_out, a.dS0, (size_t)a.N * a.H * a.Dk * a.Dv, a.stream);
        return e != hipSuccess || !a.dg || !a.fixed ? e : pass(nullptr, a.dg, (size_t)a.H, a.stream);
    }
    return a.io == Dt::F32 ? by_width<float>(a, Backward{}) : by_width<bf16_t>(a, Backward{});
}

}  // namespace kda
