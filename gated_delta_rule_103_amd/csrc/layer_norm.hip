// layer_norm.hip -- layer norm and RMS norm of rows, and their gradients.
//
// Forward, per row x of W values:
//     mean = sum x / W (0 for RMS),  rstd = 1 / sqrt(sum (x - mean)^2 / W + eps)
//     y = (x - mean) rstd w + b
// Backward, with n = (x - mean) rstd and h = dy w:
//     dx = rstd (h - n mean(h n) - mean(h))        (no mean(h) term for RMS)
//     dw = sum over rows of dy n,  db = sum over rows of dy
//
// Both directions are bound by memory: x (and dy) is read once and held in
// registers while the row's sums are formed, so nothing is read twice. A row
// is spread over NW wavefronts, each thread holding K groups of eight
// channels: consecutive ones, loaded with 16-byte instructions, where every
// row starts on a 16-byte boundary (W a multiple of 8), else eight channels
// 64 * NW apart, so that a wavefront's scalar loads stay adjacent. The
// variance is the mean square of the centred values in registers (a second
// pass that costs no memory), not a difference of two sums.
//
// dw and db reduce over the rows: a thread keeps the same channels for every
// row that its workgroup takes and sums them in registers; each workgroup
// writes one partial row to the workspace, and a second kernel adds these in
// a fixed order, so results repeat bit for bit. No atomics.
//
// 8192 rows x 4096 channels, bf16, averages of 60 launches under the profiler: forward 134 MB
// in 28 us (4.8 TB/s), backward 201 MB in 34 us (5.9 TB/s, a part of it from the last-level
// cache) and 5 us for the sums. Loading the next row ahead and one barrier
// a row instead of four took the backward kernel from 60 to 36 us.
#include "kda_device.h"
#include "kda_launch.h"
#include "kda_vec8.h"

#include <type_traits>

namespace kda {
namespace {

// One group of eight channels: consecutive from `c`, or `step` apart.
template <bool VEC, typename T>
__device__ __forceinline__ f32x8 load8(const T *row, int c, int step, int W) {
    if constexpr (VEC) {
        return c < W ? vec8<T>::load(row + c) : f32x8{};
    } else {
        f32x8 x;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = c + i * step < W ? io<T>::load(row, c + i * step) : 0.f;
        return x;
    }
}
template <bool VEC, bool PUT = false, typename T>
__device__ __forceinline__ void store8(T *row, int c, int step, int W, f32x8 x) {
    if constexpr (VEC) {
        if (c < W) {
            if constexpr (PUT) vec8<T>::put(row + c, x);
            else vec8<T>::store(row + c, x);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i * step < W) io<T>::store(row, c + i * step, x[i]);
    }
}

// How a row lies over the threads of a workgroup: NW wavefronts per row, K
// groups per thread, 4 / NW rows side by side for NW < 4.
template <int NW, int K>
struct Shape {
    static constexpr int THREADS = NW < 4 ? 256 : 64 * NW;   // per workgroup
    static constexpr int ROWS = THREADS / (64 * NW);         // rows side by side
    static constexpr int SPAN = 64 * NW;                     // threads per row
    static constexpr int MAX_W = SPAN * 8 * K;
};

// first channel of group k of thread t, and the distance of its channels
template <bool VEC, int SPAN>
__device__ __forceinline__ int first_channel(int t, int k) {
    return VEC ? (k * SPAN + t) * 8 : k * SPAN * 8 + t;
}

// sum over the NW wavefronts of a row; `part` holds one float per wavefront
template <int NW>
__device__ __forceinline__ float row_sum(float x, float *part, int wave_in_row) {
    x = warp_sum(x);
    if constexpr (NW > 1) {
        __syncthreads();                       // the previous sum has been read
        if ((threadIdx.x & 63) == 0) part[wave_in_row] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) x += part[i];
    }
    return x;
}

// One group of eight channels as it lies in memory, so that a row can be loaded
// ahead in half the registers. Rows start on 16-byte boundaries, which is all that an
// fp32 group may be loaded by.
template <bool VEC, typename T> struct Group {
    std::conditional_t<VEC && sizeof(T) == 2, u32x4, f32x8> u;
    __device__ void load(const T *row, int c, int step, int W) {
        if constexpr (VEC && sizeof(T) == 2) u = c < W ? *reinterpret_cast<const u32x4 *>(row + c) : u32x4{};
        else u = load8<VEC>(row, c, step, W);
    }
    __device__ f32x8 value() const {
        if constexpr (!VEC || sizeof(T) == 4) {
            return u;
        } else {
            f32x8 x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(u[i] << 16);
                x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
            return x;
        }
    }
};

// A workgroup takes every gridDim.x-th row (group of ROWS rows) and loads the next
// while it reduces one.
template <int NW, int K, bool VEC, typename TI, typename TO>
__global__ __launch_bounds__((Shape<NW, K>::THREADS)) void norm_kernel(const TI *x, const float *__restrict__ w,
                                                                      const float *__restrict__ b, TO *y,
                                                                      float *__restrict__ mean_out,
                                                                      float *__restrict__ rstd_out, int rows, int W,
                                                                      float eps, bool rms) {
    using S = Shape<NW, K>;
    __shared__ float part[NW];
    const int t = threadIdx.x % S::SPAN, wave = t / 64;
    constexpr int STEP = VEC ? 1 : S::SPAN;
    const float inv = 1.f / W;
    const long long stride = (long long)gridDim.x * S::ROWS;
    long long r = (long long)blockIdx.x * S::ROWS + threadIdx.x / S::SPAN;
    Group<VEC, TI> ahead[K];
    auto fetch = [&](long long row) {
        if (row >= rows) return;
#pragma unroll
        for (int k = 0; k < K; ++k) ahead[k].load(x + (size_t)row * W, first_channel<VEC, S::SPAN>(t, k), STEP, W);
    };
    fetch(r);
    // NW > 1: one row per pass, so every thread makes the same number of passes
    for (; r < rows; r += stride) {
        f32x8 v[K];
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = ahead[k].value();
        fetch(r + stride);
        float mean = 0.f;
        if (!rms) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += v[k][i];
            mean = row_sum<NW>(s, part, wave) * inv;
        }
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = first_channel<VEC, S::SPAN>(t, k);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = c + i * STEP < W ? v[k][i] - mean : 0.f;
                v[k][i] = d;
                ss += d * d;
            }
        }
        const float rstd = 1.f / sqrtf(row_sum<NW>(ss, part, wave) * inv + eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = first_channel<VEC, S::SPAN>(t, k);
            f32x8 o = v[k] * rstd;
            if (w) o *= load8<VEC>(w, c, STEP, W);
            if (b) o += load8<VEC>(b, c, STEP, W);
            store8<VEC>(y + (size_t)r * W, c, STEP, W, o);
        }
        if (t == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
    }
}

// dw_part, db_part: [gridDim.x][W], null when that gradient is not wanted. The next
// row is loaded while the current one is reduced; both of a row's sums cross the
// wavefronts together, through slots that alternate, so a row takes one barrier.
template <int NW, int K, bool VEC, typename TI, typename TG>
__global__ __launch_bounds__((Shape<NW, K>::THREADS)) void norm_backward_kernel(
    const TI *__restrict__ x, const TG *__restrict__ dy, const float *__restrict__ mean_in,
    const float *__restrict__ rstd_in, const float *__restrict__ w, TI *__restrict__ dx, float *__restrict__ dw_part,
    float *__restrict__ db_part, int rows, int W) {
    using S = Shape<NW, K>;
    __shared__ float part[2][2][NW];
    __shared__ __align__(32) float fold[S::ROWS > 1 ? (S::ROWS - 1) * S::MAX_W : 1];
    const int t = threadIdx.x % S::SPAN, wave = t / 64, rg = threadIdx.x / S::SPAN;
    constexpr int STEP = VEC ? 1 : S::SPAN;
    f32x8 dw[K] = {}, db[K] = {}, wv[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        wv[k] = w ? load8<VEC>(w, first_channel<VEC, S::SPAN>(t, k), STEP, W) : f32x8{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    const float inv = 1.f / W;
    const long long stride = (long long)gridDim.x * S::ROWS;
    Group<VEC, TI> xn[K];
    Group<VEC, TG> dn[K];
    float mean_n = 0.f, rstd_n = 0.f;
    auto fetch = [&](long long r) {
        if (r >= rows) return;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = first_channel<VEC, S::SPAN>(t, k);
            xn[k].load(x + (size_t)r * W, c, STEP, W);
            dn[k].load(dy + (size_t)r * W, c, STEP, W);
        }
        mean_n = mean_in ? mean_in[r] : 0.f;
        rstd_n = rstd_in[r];
    };
    // NW > 1: one row per pass, so every thread makes the same number of passes
    long long r = (long long)blockIdx.x * S::ROWS + rg;
    fetch(r);
    for (int turn = 0; r < rows; r += stride, turn ^= 1) {
        const float mean = mean_n, rstd = rstd_n;
        f32x8 n[K], h[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            n[k] = xn[k].value();
            h[k] = dn[k].value();
        }
        fetch(r + stride);
        float shn = 0.f, sh = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            n[k] = (n[k] - mean) * rstd;       // past the row's end: h is 0 there
            dw[k] += h[k] * n[k];
            db[k] += h[k];
            h[k] *= wv[k];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                shn += h[k][i] * n[k][i];
                sh += h[k][i];
            }
        }
        shn = warp_sum(shn);
        if (mean_in) sh = warp_sum(sh);        // uniform
        if constexpr (NW > 1) {
            if ((threadIdx.x & 63) == 0) {
                part[turn][0][wave] = shn;
                part[turn][1][wave] = sh;
            }
            __syncthreads();
            shn = sh = 0.f;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                shn += part[turn][0][i];
                sh += part[turn][1][i];
            }
        }
        shn *= inv;
        sh = mean_in ? sh * inv : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            store8<VEC, true>(dx + (size_t)r * W, first_channel<VEC, S::SPAN>(t, k), STEP, W,
                        (h[k] - n[k] * shn - sh) * rstd);
    }
    auto put = [&](f32x8 (&a)[K], float *out) {
        if constexpr (S::ROWS > 1) {           // the rows side by side, added in a fixed order
            __syncthreads();
            if (rg > 0)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    *reinterpret_cast<f32x8 *>(&fold[(rg - 1) * S::MAX_W + (k * S::SPAN + t) * 8]) = a[k];
            __syncthreads();
            if (rg > 0) return;
            for (int g = 0; g < S::ROWS - 1; ++g)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    a[k] += *reinterpret_cast<f32x8 *>(&fold[g * S::MAX_W + (k * S::SPAN + t) * 8]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            store8<VEC>(out + (size_t)blockIdx.x * W, first_channel<VEC, S::SPAN>(t, k), STEP, W, a[k]);
    };
    if (dw_part) put(dw, dw_part);
    if (db_part) put(db, db_part);
}

// out[c] = sum over g of part[g][c]: 16 threads per channel group of 64, each
// summing every 16th partial row, then a fixed-order sum over the sixteen.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float *__restrict__ a, float *__restrict__ da,
                                                          const float *__restrict__ b, float *__restrict__ db, int G,
                                                          int W) {
    __shared__ float s[16][64];
    const float *p = blockIdx.y ? b : a;
    float *out = blockIdx.y ? db : da;
    if (!out) return;
    const int c = blockIdx.x * 64 + (threadIdx.x & 63), j = threadIdx.x >> 6;
    float x = 0.f;
    if (c < W) {
#pragma unroll 8
        for (int g = j; g < G; g += 16) x += p[(size_t)g * W + c];
    }
    s[j][threadIdx.x & 63] = x;
    __syncthreads();
    if (j == 0 && c < W) {
        for (int i = 1; i < 16; ++i) x += s[i][threadIdx.x];
        out[c] = x;
    }
}

// Rows of the partial sums, one for each workgroup: as many as keep the card busy, never
// more than there are rows for, and one for a few rows, whose sums then are the gradients
// themselves.
int partial_rows(long long rows, int rows_per_wg) {
    if (rows > 0 && rows <= 4 * rows_per_wg) return 1;
    const long long wgs = (rows + rows_per_wg - 1) / rows_per_wg;
    return static_cast<int>(wgs < 512 ? wgs : 512);
}

// Calls f with the smallest Shape that holds a row of W channels.
template <typename F>
hipError_t with_shape(int W, F f) {
    if (W <= 512) return f.template operator()<1, 1>();
    if (W <= 1024) return f.template operator()<1, 2>();
    if (W <= 2048) return f.template operator()<4, 1>();
    if (W <= 4096) return f.template operator()<4, 2>();
    if (W <= 8192) return f.template operator()<8, 2>();
    return f.template operator()<16, 2>();
}

bool aligned16(const void *a, const void *b, const void *c, const void *d) {
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c) |
             reinterpret_cast<uintptr_t>(d)) & 15u) == 0;
}

constexpr int FORWARD_GRID = 2048;

template <typename TI, typename TO, bool VEC>
struct Forward {
    const LayerNormArgs &a;
    template <int NW, int K>
    hipError_t operator()() const {
        using S = Shape<NW, K>;
        const long long groups = (a.rows + (long long)S::ROWS - 1) / S::ROWS;
        const unsigned grid = static_cast<unsigned>(groups < FORWARD_GRID ? groups : FORWARD_GRID);
        hipLaunchKernelGGL((norm_kernel<NW, K, VEC, TI, TO>), dim3(grid), dim3(S::THREADS), 0, a.stream,
                           static_cast<const TI *>(a.x), a.weight, a.bias, static_cast<TO *>(a.out), a.mean, a.rstd,
                           a.rows, a.W, a.eps, a.rms);
        return hipGetLastError();
    }
};

template <typename TI, typename TG, bool VEC>
struct Backward {
    const LayerNormBackwardArgs &a;
    template <int NW, int K>
    hipError_t operator()() const {
        using S = Shape<NW, K>;
        const int G = partial_rows(a.rows, S::ROWS);
        float *dwp = !a.dweight ? nullptr : G == 1 ? a.dweight : a.ws;
        float *dbp = !a.dbias ? nullptr : G == 1 ? a.dbias : a.ws + (a.dweight ? (size_t)G * a.W : 0);
        if (G > 0) {
            hipLaunchKernelGGL((norm_backward_kernel<NW, K, VEC, TI, TG>), dim3(G), dim3(S::THREADS), 0, a.stream,
                               static_cast<const TI *>(a.x), static_cast<const TG *>(a.dy), a.rms ? nullptr : a.mean,
                               a.rstd, a.weight, static_cast<TI *>(a.dx), dwp, dbp, a.rows, a.W);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        if (G == 1 || (!a.dweight && !a.dbias)) return hipSuccess;
        hipLaunchKernelGGL(column_sum_kernel, dim3((a.W + 63) / 64, 2), dim3(1024), 0, a.stream, dwp, a.dweight, dbp,
                           a.dbias, G, a.W);
        return hipGetLastError();
    }
};

}  // namespace

size_t layer_norm_backward_workspace(int rows, int W) {
    // partial rows of each gradient: no shape has more than the one with a row per workgroup
    const int G = partial_rows(rows, 1);
    return G == 1 ? 0 : 2 * sizeof(float) * (size_t)G * W;
}

hipError_t launch_layer_norm(const LayerNormArgs &a) {
    if (a.rows == 0) return hipSuccess;
    const bool vec = a.W % 8 == 0 && aligned16(a.x, a.out, a.weight, a.bias);
    auto run = [&](auto in, auto out) {
        using TI = decltype(in);
        using TO = decltype(out);
        return vec ? with_shape(a.W, Forward<TI, TO, true>{a}) : with_shape(a.W, Forward<TI, TO, false>{a});
    };
    if (a.x_dt == Dt::F32) return a.out_dt == Dt::F32 ? run(float{}, float{}) : run(float{}, bf16_t{});
    return a.out_dt == Dt::F32 ? run(bf16_t{}, float{}) : run(bf16_t{}, bf16_t{});
}

hipError_t launch_layer_norm_backward(const LayerNormBackwardArgs &a) {
    const bool vec = a.W % 8 == 0 && aligned16(a.x, a.dy, a.dx, a.weight) && aligned16(a.dweight, a.dbias, nullptr, nullptr);
    auto run = [&](auto in, auto grad) {
        using TI = decltype(in);
        using TG = decltype(grad);
        return vec ? with_shape(a.W, Backward<TI, TG, true>{a}) : with_shape(a.W, Backward<TI, TG, false>{a});
    };
    if (a.x_dt == Dt::F32) return a.dy_dt == Dt::F32 ? run(float{}, float{}) : run(float{}, bf16_t{});
    return a.dy_dt == Dt::F32 ? run(bf16_t{}, float{}) : run(bf16_t{}, bf16_t{});
}

}  // namespace kda
