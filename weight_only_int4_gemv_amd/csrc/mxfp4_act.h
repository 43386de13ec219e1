// mxfp4_act.h — the activations of a product's epilogue and their slopes, in fp32.
// Private to libmxfp4.
#pragma once

#include "mxfp4_device.h"
#include "mxfp4_launch.h"

namespace mxfp4 {

enum Act { kNone = 0, kRelu = 1, kSilu = 2, kGelu = 3, kGeluTanh = 4, kSwiglu = 5 };

// z cut to [-c, c]; a NaN stays.
__device__ __forceinline__ float clamp_to(float z, float c) { return z > c ? c : z < -c ? -c : z; }

// 1 / (1 + exp(-z)); the reciprocal is good to an ulp.
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}

constexpr float kGeluTwoC = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;
constexpr float kRootHalf = 0.70710678118654752f;
constexpr float kRootTwoPi = 0.39894228040143268f;  // 1 / sqrt(2 pi)

// The activation of N values (of SwiGLU the gates').  GELU as z Phi(z) = z erfc(-z / sqrt 2) / 2
// (1 + erf loses the left tail), its tanh form as z sigmoid(2u), u = sqrt(2 / pi) (z + 0.044715
// z^3), which is z (1 + tanh u) / 2.  The choice is the same for all lanes and made once.
template <int N>
__device__ __forceinline__ void act_values(int act, float (&z)[N]) {
    switch (act) {
        case kRelu:
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] = z[j] < 0.0f ? 0.0f : z[j];
            break;
        case kSilu:
        case kSwiglu:
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] *= sigmoid(z[j]);
            break;
        case kGelu:
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] = 0.5f * z[j] * erfcf(-kRootHalf * z[j]);
            break;
        case kGeluTanh:
#pragma unroll
            for (int j = 0; j < N; ++j)
                z[j] *= sigmoid(z[j] * fmaf(kGeluTwoC * kGeluCube, z[j] * z[j], kGeluTwoC));
            break;
    }
}

// d act / dz.  Beyond |z| of 40 (silu 150) the slopes are 0 and 1 in fp32: z is cut there, so
// that no product of an overflow and a zero arises.
__device__ __forceinline__ float silu_slope(float z, float s) { return s * (1.0f + z * (1.0f - s)); }
template <int N>
__device__ __forceinline__ void act_slopes(int act, float (&z)[N]) {
    switch (act) {
        case kNone:
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] = 1.0f;
            break;
        case kRelu:
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] = z[j] <= 0.0f ? 0.0f : 1.0f;
            break;
        case kSilu:
#pragma unroll
            for (int j = 0; j < N; ++j) {
                z[j] = clamp_to(z[j], 150.0f);
                z[j] = silu_slope(z[j], sigmoid(z[j]));
            }
            break;
        case kGelu:
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float v = clamp_to(z[j], 40.0f);
                z[j] = 0.5f * erfcf(-kRootHalf * v) + kRootTwoPi * v * __expf(-0.5f * v * v);
            }
            break;
        case kGeluTanh:
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float v = clamp_to(z[j], 40.0f);
                const float s = sigmoid(v * fmaf(kGeluTwoC * kGeluCube, v * v, kGeluTwoC));
                z[j] = s + v * s * (1.0f - s) * fmaf(3.0f * kGeluTwoC * kGeluCube, v * v, kGeluTwoC);
            }
            break;
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

// The bias of VEC columns of Y from `col` on (with SwiGLU the gates', and of the up rows); rows of
// no expert take none.
template <int VEC>
struct Bias {
    float z[VEC], up[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Bias<VEC> load_bias(const LinearArgs& a, int expert, int col) {
    Bias<VEC> b;
#pragma unroll
    for (int j = 0; j < VEC; ++j) b.z[j] = b.up[j] = 0.0f;
    if (a.bias != nullptr && expert >= 0) {
        const uint16_t* p = a.bias + (int64_t)expert * a.N + col;
        load_columns<T, VEC>(p, b.z);
        if (a.act == kSwiglu) load_columns<T, VEC>(p + a.N / 2, b.up);
    }
    return b;
}

// The epilogue of VEC columns of Y from `col` on: h is their product (with SwiGLU the gates',
// up the up rows').  Sums are fp32; Z and Y are rounded once each, Y from the unrounded sums.
template <typename T, int VEC>
__device__ __forceinline__ void finish_columns(const LinearArgs& a, const Bias<VEC>& bias, int64_t row,
                                               int col, const float (&h)[VEC],
                                               const float (&up)[VEC]) {
    const bool swiglu = a.act == kSwiglu;
    const int F = swiglu ? a.N / 2 : a.N;
    float z[VEC], u[VEC], v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) z[j] = h[j] + bias.z[j], u[j] = up[j] + bias.up[j];
    if (a.Z != nullptr) {
        store_columns<T, VEC>(a.Z + row * a.N + col, z);
        if (swiglu) store_columns<T, VEC>(a.Z + row * a.N + F + col, u);
    }
    act_values(a.act, z);
    if (swiglu) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) z[j] *= u[j];
    }
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
