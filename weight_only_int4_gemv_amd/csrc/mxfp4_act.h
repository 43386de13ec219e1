// mxfp4_act.h — the activations of a product's epilogue and their slopes, in fp32.
// Private to libmxfp4.
#pragma once

#include "mxfp4_device.h"
#include "mxfp4_launch.h"

namespace mxfp4 {

enum Act { kNone = 0, kRelu = 1, kSilu = 2, kGelu = 3, kGeluTanh = 4, kSwiglu = 5 };

// z cut to [-c, c]; a NaN stays.
__device__ __forceinline__ float clamp_to(float z, float c) { return z > c ? c : z < -c ? -c : z; }

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

constexpr float kGeluTwoC = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;
constexpr float kRootHalf = 0.70710678118654752f;
constexpr float kRootTwoPi = 0.39894228040143268f;  // 1 / sqrt(2 pi)

// GELU as z Phi(z) = z erfc(-z / sqrt 2) / 2 (1 + erf loses the left tail), its tanh form as
// z / (1 + exp(-2u)), u = sqrt(2 / pi) (z + 0.044715 z^3), which is z (1 + tanh u) / 2.
__device__ __forceinline__ float act_value(int act, float z) {
    switch (act) {
        case kRelu: return z < 0.0f ? 0.0f : z;
        case kSilu: return silu(z);
        case kGelu: return 0.5f * z * erfcf(-kRootHalf * z);
        case kGeluTanh: return z / (1.0f + __expf(-kGeluTwoC * (z + kGeluCube * z * z * z)));
        default: return z;
    }
}

// d act / dz.  Beyond |z| of 40 (silu 150) the slopes are 0 and 1 in fp32: z is cut there, so
// that no product of an overflow and a zero arises.
__device__ __forceinline__ float silu_slope(float z) {
    z = clamp_to(z, 150.0f);
    const float s = sigmoid(z);
    return s * (1.0f + z * (1.0f - s));
}
__device__ __forceinline__ float act_slope(int act, float z) {
    switch (act) {
        case kRelu: return z <= 0.0f ? 0.0f : 1.0f;
        case kSilu: return silu_slope(z);
        case kGelu:
            z = clamp_to(z, 40.0f);
            return 0.5f * erfcf(-kRootHalf * z) + kRootTwoPi * z * __expf(-0.5f * z * z);
        case kGeluTanh: {
            z = clamp_to(z, 40.0f);
            const float s = sigmoid(kGeluTwoC * (z + kGeluCube * z * z * z));
            return s + z * s * (1.0f - s) * kGeluTwoC * (1.0f + 3.0f * kGeluCube * z * z);
        }
        default: return 1.0f;
    }
}

template <int N>
struct Int {
    static constexpr int value = N;
};

template <typename T, int VEC>
__device__ __forceinline__ void load_columns(const uint16_t* p, float (&v)[VEC]) {
    uint16_t b[VEC];
    __builtin_memcpy(b, __builtin_assume_aligned(p, 2 * VEC), 2 * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = T::load(b[j]);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_columns(uint16_t* p, const float (&v)[VEC]) {
    uint16_t b[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) b[j] = T::store(v[j]);
    __builtin_memcpy(__builtin_assume_aligned(p, 2 * VEC), b, 2 * VEC);
}

// Whether every row of the epilogue's tensors starts on 16 bytes.
__host__ __device__ inline bool finish_wide(const LinearArgs& a) {
    const int F = a.act == kSwiglu ? a.N / 2 : a.N;
    const uintptr_t at = (uintptr_t)a.Y | (uintptr_t)a.Y32 | (uintptr_t)a.bias |
                         (uintptr_t)a.residual | (uintptr_t)a.Z;
    return F % 8 == 0 && at % 16 == 0 && (a.residual == nullptr || a.r_stride % 8 == 0);
}

// The epilogue of VEC columns of Y from `col` on: h is their product (with SwiGLU the gates',
// up the up rows').  Sums are fp32; Z and Y are rounded once each, Y from the unrounded sums.
// Rows of no expert (their product is 0) take no bias.
template <typename T, int VEC>
__device__ __forceinline__ void finish_columns(const LinearArgs& a, int expert, int64_t row,
                                               int col, const float (&h)[VEC],
                                               const float (&up)[VEC]) {
    const bool swiglu = a.act == kSwiglu;
    const int F = swiglu ? a.N / 2 : a.N;
    float z[VEC], u[VEC], v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) z[j] = h[j], u[j] = up[j];
    if (a.bias != nullptr && expert >= 0) {
        const uint16_t* b = a.bias + (int64_t)expert * a.N + col;
        load_columns<T, VEC>(b, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) z[j] += v[j];
        if (swiglu) {
            load_columns<T, VEC>(b + F, v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[j] += v[j];
        }
    }
    if (a.Z != nullptr) {
        store_columns<T, VEC>(a.Z + row * a.N + col, z);
        if (swiglu) store_columns<T, VEC>(a.Z + row * a.N + F + col, u);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) z[j] = swiglu ? silu(z[j]) * u[j] : act_value(a.act, z[j]);
    if (a.residual != nullptr) {
        load_columns<T, VEC>(a.residual + row * a.r_stride + col, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) z[j] += v[j];
    }
    if (a.Y32 != nullptr) {
        constexpr int kAlign = 4 * VEC < 16 ? 4 * VEC : 16;
        __builtin_memcpy(__builtin_assume_aligned(a.Y32 + row * F + col, kAlign), z, 4 * VEC);
    } else {
        store_columns<T, VEC>(a.Y + row * F + col, z);
    }
}

}  // namespace mxfp4
