// output_gate_backward.hip -- the gradient of the per-head output norm and
// gate, out_j = n_j w_j sigmoid(z_j) with n_j = o_j r, r = 1 / sqrt(mean_j o_j^2 + eps).
//
// Per (row, head), over the Dv channels, with s = sigmoid(z) and x = dout s w:
//     do = r (x - n mean_j(x n))
//     dz = dout n w s (1 - s)
//     dw = sum over rows and heads of dout s n
//
// o, z and dout are read once and do and dz written once, so the kernel is
// bound by memory. As in the forward kernel a head row is spread over Dv / 8
// lanes of eight consecutive channels; both of its sums are reduced inside
// those lanes. A lane keeps the same channels for every row it takes, so dw is
// summed in its registers, then over the workgroup's lanes in a fixed order;
// each workgroup writes one partial row, which a second kernel adds in a fixed
// order: no atomics, results repeat bit for bit. 8192 rows x 32 heads x 128 channels,
// bf16: 336 MB in 71 us (64-81 over 60 launches under the profiler, 4.8 TB/s), and 6 us for
// the weight's sum (65 us when one
// workgroup added the partial rows).
#include "kda_device.h"
#include "kda_launch.h"
#include "kda_vec8.h"

namespace kda {
namespace {

constexpr int THREADS = 256;
constexpr int MAX_PARTS = 2048;          // workgroups of a launch, and rows of its partial sums

template <int LR>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int m = 1; m < LR; m <<= 1) x += __shfl_xor(x, m, 64);
    return x;
}

template <int DV, typename TO, typename TZ, typename TG>
__global__ __launch_bounds__(THREADS) void output_gate_backward_kernel(
    const TO *__restrict__ o, const TZ *__restrict__ z, const TG *__restrict__ dout, const float *__restrict__ w,
    TO *__restrict__ do_, TZ *__restrict__ dz, float *__restrict__ dw_part, long long rowheads, float eps) {
    constexpr int LR = DV / 8, RPB = THREADS / LR;
    __shared__ float fold[THREADS / 64][DV];
    const int t = threadIdx.x, part = t % LR;
    f32x8 wv = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, dw = {};
    if (w) wv = vec8<float>::load(w + 8 * part);
    for (long long rh = (long long)blockIdx.x * RPB + t / LR; rh < rowheads; rh += (long long)gridDim.x * RPB) {
        // the LR lanes of a row leave the loop together
        const size_t off = (size_t)rh * DV + 8 * part;
        const f32x8 x = vec8<TO>::load(o + off), g = vec8<TZ>::load(z + off), d = vec8<TG>::load(dout + off);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
        const float r = 1.f / sqrtf(lanes_sum<LR>(ss) * (1.f / DV) + eps);
        const f32x8 n = x * r;
        f32x8 s, c;                      // sigmoid(z) and 1 - sigmoid(z), neither by cancellation
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = __expf(-fabsf(g[i])), q = 1.f / (1.f + e);
            s[i] = g[i] >= 0.f ? q : e * q;
            c[i] = g[i] >= 0.f ? e * q : q;
        }
        const f32x8 ds = d * s, y = ds * wv;
        dw += ds * n;
        float yn = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) yn += y[i] * n[i];
        yn = lanes_sum<LR>(yn) * (1.f / DV);
        vec8<TO>::store(do_ + off, (y - n * yn) * r);
        vec8<TZ>::store(dz + off, y * n * c);
    }
    if (!dw_part) return;
    // the rows of a wavefront, then the wavefronts
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int m = LR; m < 64; m <<= 1) dw[i] += __shfl_xor(dw[i], m, 64);
    }
    if ((t & 63) < LR)
#pragma unroll
        for (int i = 0; i < 8; ++i) fold[t / 64][8 * part + i] = dw[i];
    __syncthreads();
    if (t < DV) {
        float x = 0.f;
        for (int i = 0; i < THREADS / 64; ++i) x += fold[i][t];
        dw_part[(size_t)blockIdx.x * DV + t] = x;
    }
}

// dw[c] = sum over the G partial rows: a workgroup takes 16 channels in 64 strands,
// each adding every 64th row, then adds the strands in a fixed order.
constexpr int DW_CH = 16, DW_STRANDS = 64;
__global__ __launch_bounds__(DW_CH *DW_STRANDS) void dweight_kernel(const float *__restrict__ part,
                                                                   float *__restrict__ dw, int G, int Dv) {
    __shared__ float s[DW_STRANDS][DW_CH + 1];
    const int ch = threadIdx.x % DW_CH, j = threadIdx.x / DW_CH, c = blockIdx.x * DW_CH + ch;
    float x = 0.f;
#pragma unroll 8
    for (int g = j; g < G; g += DW_STRANDS) x += part[(size_t)g * Dv + c];
    s[j][ch] = x;
    __syncthreads();
    if (j == 0) {
        for (int i = 1; i < DW_STRANDS; ++i) x += s[i][ch];
        dw[c] = x;
    }
}

// Workgroups of a launch. A few rows are one workgroup's, whose sum is dw itself: a
// second launch would cost more than the four turns of its loop.
int parts(long long rowheads, int Dv) {
    const int rpb = THREADS / (Dv / 8);
    if (rowheads > 0 && rowheads <= 4 * rpb) return 1;
    const long long g = (rowheads + rpb - 1) / rpb;
    return static_cast<int>(g < MAX_PARTS ? g : MAX_PARTS);
}

template <int DV, typename TO, typename TZ, typename TG>
hipError_t launch_t(const OutputGateBackwardArgs &a) {
    const long long rowheads = (long long)a.rows * a.H;
    const int G = parts(rowheads, DV);
    if (G > 0) {
        hipLaunchKernelGGL((output_gate_backward_kernel<DV, TO, TZ, TG>), dim3(G), dim3(THREADS), 0, a.stream,
                           static_cast<const TO *>(a.o), static_cast<const TZ *>(a.gate),
                           static_cast<const TG *>(a.dout), a.weight, static_cast<TO *>(a.do_),
                           static_cast<TZ *>(a.dgate), G == 1 ? a.dweight : a.dweight ? a.ws : nullptr, rowheads,
                           a.eps);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.dweight || G == 1) return hipSuccess;
    hipLaunchKernelGGL(dweight_kernel, dim3(DV / DW_CH), dim3(DW_CH * DW_STRANDS), 0, a.stream, a.ws, a.dweight, G, DV);
    return hipGetLastError();
}

template <int DV, typename TO, typename TZ>
hipError_t launch_g(const OutputGateBackwardArgs &a) {
    return a.dout_dt == Dt::F32 ? launch_t<DV, TO, TZ, float>(a) : launch_t<DV, TO, TZ, bf16_t>(a);
}

template <int DV, typename TO>
hipError_t launch_z(const OutputGateBackwardArgs &a) {
    return a.gate_dt == Dt::F32 ? launch_g<DV, TO, float>(a) : launch_g<DV, TO, bf16_t>(a);
}

template <int DV>
hipError_t launch_o(const OutputGateBackwardArgs &a) {
    return a.o_dt == Dt::F32 ? launch_z<DV, float>(a) : launch_z<DV, bf16_t>(a);
}

}  // namespace

size_t output_gate_backward_workspace(long long rowheads, int Dv) {
    const int G = parts(rowheads, Dv);
    return G == 1 ? 0 : sizeof(float) * (size_t)G * Dv;
}

hipError_t launch_output_gate_backward(const OutputGateBackwardArgs &a) {
    return a.Dv == 64 ? launch_o<64>(a) : launch_o<128>(a);
}

}  // namespace kda
