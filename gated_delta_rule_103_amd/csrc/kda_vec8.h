// kda_vec8.h -- eight consecutive channels per lane: 16-byte loads and stores
// of bf16, two of fp32, as the row kernels use them.
#pragma once
#include "kda_device.h"

namespace kda {

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T> struct vec8;
template <> struct vec8<float> {
    __device__ static f32x8 load(const float *p) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
        return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
    __device__ static void store(float *p, f32x8 x) {
        *reinterpret_cast<f32x4 *>(p) = f32x4{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<f32x4 *>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
    }
    __device__ static void put(float *p, f32x8 x) { store(p, x); }
};
template <> struct vec8<bf16_t> {
    __device__ static f32x8 load(const bf16_t *p) {
        const u32x4 u = *reinterpret_cast<const u32x4 *>(p);
        f32x8 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
        return x;
    }
    __device__ static void store(bf16_t *p, f32x8 x) {
        u32x4 u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = static_cast<uint32_t>(f32_to_bf16(x[2 * i])) | (static_cast<uint32_t>(f32_to_bf16(x[2 * i + 1])) << 16);
        *reinterpret_cast<u32x4 *>(p) = u;
    }
    // the same rounding by the conversion instruction: fewer instructions than store's, which
    // pays where a kernel has many besides (norm gradient of 8192 x 4096 42.8 -> 41.0 us; the
    // norm itself 28.6 -> 29.0 and the gate's gradient 70.3 -> 71.0, which keep store)
    __device__ static void put(bf16_t *p, f32x8 x) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        u32x4 u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x[2 * i], x[2 * i + 1]}), bf16x2));
        *reinterpret_cast<u32x4 *>(p) = u;
    }
};

}  // namespace kda
