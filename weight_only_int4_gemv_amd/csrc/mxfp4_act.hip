// mxfp4_act.hip — the epilogue of products whose K was split, and the gradient through an
// activation with the bias's gradient.
#include "mxfp4_act.h"

namespace mxfp4 {
namespace {

// ------------------------------------------------------------------ epilogue
//
// Partial sums [slices][R][N] added in slice order, then bias, activation and residual;
// VEC columns of Y a thread.
template <typename T, int VEC>
__global__ __launch_bounds__(256) void finish_kernel(LinearArgs a) {
    const bool swiglu = a.act == kSwiglu;
    const int F = swiglu ? a.N / 2 : a.N, chunks = F / VEC;
    const int64_t n = (int64_t)a.R * a.N, total = (int64_t)a.R * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / chunks;
        const int col = (int)(i - row * chunks) * VEC;
        float h[VEC] = {}, up[VEC] = {};
        for (int s = 0; s < a.slices; ++s) {
            const float* p = a.part + s * n + row * a.N + col;
            constexpr int kAlign = 4 * VEC < 16 ? 4 * VEC : 16;
            float v[VEC];
            __builtin_memcpy(v, __builtin_assume_aligned(p, kAlign), 4 * VEC);
#pragma unroll
            for (int j = 0; j < VEC; ++j) h[j] += v[j];
            if (swiglu) {
                __builtin_memcpy(v, __builtin_assume_aligned(p + F, kAlign), 4 * VEC);
#pragma unroll
                for (int j = 0; j < VEC; ++j) up[j] += v[j];
            }
        }
        finish_columns<T, VEC>(a, load_bias<T, VEC>(a, 0, col), row, col, h, up);
    }
}

// --------------------------------------------------------- activation's gradient
//
// dZ = dY act'(Z), with SwiGLU dgate = dY up silu'(gate), dup = dY silu(gate); dbias is the sum
// of dZ's rows before their rounding, in fp32: each block adds its kRows rows, a second launch
// the blocks' sums in order, so that the result does not depend on scheduling.  Bound by HBM: 4095
// rows of 28672 columns with SwiGLU and bias (588 MB) take 114 us and 4.7 for the second launch,
// 5.1 TB/s.  One row in hand instead of four and loads that stay in the caches: 135 us together.
constexpr int kRows = 64;               // rows of a block
constexpr int kThreads = 256;
constexpr int kRowLanes = 4;            // rows a block has in hand
constexpr int kColLanes = kThreads / kRowLanes;

template <typename T, int VEC, bool SWIGLU, bool BIAS>
__global__ __launch_bounds__(kThreads) void act_grad_kernel(ActGradArgs a) {
    constexpr int H = SWIGLU ? 2 : 1;
    const int F = SWIGLU ? a.N / 2 : a.N;
    const int slot = blockIdx.z * gridDim.y + blockIdx.y;
    Tile t;
    if (a.offsets != nullptr) {
        t = find_tile(a.offsets, a.E, a.R, kRows, slot);
    } else {
        t.expert = 0;
        t.row0 = slot * kRows;
        t.rows = min(kRows, a.R - t.row0);
    }
    if (t.rows <= 0) return;
    const int lane = threadIdx.x % kColLanes, first = threadIdx.x / kColLanes;
    const int col = (blockIdx.x * kColLanes + lane) * VEC;
    float sum[H][VEC] = {};
    if (col < F) {
        constexpr int kHand = VEC == 8 ? 4 : 1;             // rows a lane has in hand
        for (int r0 = first; r0 < t.rows; r0 += kHand * kRowLanes) {
            Piece<uint16_t, VEC> dy[kHand], z[kHand], up[kHand];
#pragma unroll
            for (int h = 0; h < kHand; ++h) {
                const int64_t row = t.row0 + r0 + h * kRowLanes;
                if (r0 + h * kRowLanes >= t.rows) continue;
                dy[h].load_once(a.dY + row * a.y_stride + col);
                z[h].load_once(a.Z + row * a.z_stride + col);
                if constexpr (SWIGLU) up[h].load_once(a.Z + row * a.z_stride + F + col);
            }
#pragma unroll
            for (int h = 0; h < kHand; ++h) {
                const int64_t row = t.row0 + r0 + h * kRowLanes;
                if (r0 + h * kRowLanes >= t.rows) continue;
                Piece<uint16_t, VEC> out[H];
                float dz[H][VEC], g[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) g[j] = T::load(z[h].get(j));
                if constexpr (SWIGLU) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float d = T::load(dy[h].get(j)), u = T::load(up[h].get(j));
                        const float s = sigmoid(g[j]), c = clamp_to(g[j], 150.0f);
                        dz[0][j] = d * u * silu_slope(c, s);
                        dz[1][j] = d * (g[j] * s);
                    }
                } else {
                    act_slopes(a.act, g);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) dz[0][j] = T::load(dy[h].get(j)) * g[j];
                }
#pragma unroll
                for (int i = 0; i < H; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        out[i].set(j, T::store(dz[i][j]));
                        sum[i][j] += dz[i][j];
                    }
#pragma unroll
                for (int i = 0; i < H; ++i) out[i].store_once(a.dZ + row * a.N + i * F + col);
            }
        }
    }
    if constexpr (BIAS) {
        __shared__ float part[kRowLanes][H][kColLanes * VEC];
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int j = 0; j < VEC; ++j) part[first][h][lane * VEC + j] = sum[h][j];
        __syncthreads();
        float* out = a.part != nullptr ? a.part + (int64_t)slot * a.N : a.dbias;
        for (int i = threadIdx.x; i < H * kColLanes * VEC; i += kThreads) {
            const int h = i / (kColLanes * VEC), c = i % (kColLanes * VEC);
            const int n = blockIdx.x * kColLanes * VEC + c;
            if (n >= F) continue;
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < kRowLanes; ++k) s += part[k][h][c];
            out[h * F + n] = s;
        }
    }
}

// dbias[e] = the sums of the expert's blocks, in order.  A thread adds an expert's partial rows one
// after the other: 65536 rows of 4096 columns without an activation take 293 us, 30 more than without
// a bias; over 64 experts 268.
__global__ __launch_bounds__(kThreads) void bias_sum_kernel(ActGradArgs a) {
    const int e = blockIdx.y, n = blockIdx.x * kThreads + threadIdx.x;
    int first = 0, count = (a.R + kRows - 1) / kRows;
    if (a.offsets != nullptr) {
        // The slots of group e + 1.
        int before = 0, from = 0;
        for (int base = 0; base <= a.E + 1; base += kWave) {
            const Groups w = scan_groups(a.offsets, a.E, a.R, kRows, base, from);
            if (e + 1 < base + kWave) {
                const int src = e + 1 - base;
                first = before + __builtin_amdgcn_readlane(w.first, src);
                count = (__builtin_amdgcn_readlane(w.hi, src) -
                         __builtin_amdgcn_readlane(w.lo, src) + kRows - 1) / kRows;
                break;
            }
            before += w.count;
            from = w.end;
        }
    }
    if (n >= a.N) return;
    float s = 0.0f;
    const float* p = a.part + (int64_t)first * a.N + n;
#pragma unroll 8
    for (int i = 0; i < count; ++i) s += p[(int64_t)i * a.N];
    a.dbias[(int64_t)e * a.N + n] = s;
}

template <typename T, int VEC>
void act_grad(const ActGradArgs& a, hipStream_t stream) {
    const bool swiglu = a.act == kSwiglu;
    const int F = swiglu ? a.N / 2 : a.N;
    const int64_t slots = a.offsets ? tile_slots(a.R, a.E, kRows) : (a.R + kRows - 1) / kRows;
    const dim3 grid = slot_grid((F + kColLanes * VEC - 1) / (kColLanes * VEC), slots);
    if (swiglu && a.dbias) act_grad_kernel<T, VEC, true, true><<<grid, kThreads, 0, stream>>>(a);
    else if (swiglu) act_grad_kernel<T, VEC, true, false><<<grid, kThreads, 0, stream>>>(a);
    else if (a.dbias) act_grad_kernel<T, VEC, false, true><<<grid, kThreads, 0, stream>>>(a);
    else act_grad_kernel<T, VEC, false, false><<<grid, kThreads, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_finish(const LinearArgs& a, DType dt, hipStream_t stream) {
    const bool wide = finish_wide(a);
    const int F = a.act == kSwiglu ? a.N / 2 : a.N;
    const int64_t threads = (int64_t)a.R * (wide ? F / 8 : F), blocks = (threads + 255) / 256;
    const unsigned grid = (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20);
    if (dt == kF16 && wide) finish_kernel<F16, 8><<<grid, 256, 0, stream>>>(a);
    else if (dt == kF16) finish_kernel<F16, 1><<<grid, 256, 0, stream>>>(a);
    else if (wide) finish_kernel<BF16, 8><<<grid, 256, 0, stream>>>(a);
    else finish_kernel<BF16, 1><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

size_t activation_grad_workspace(int64_t R, int64_t N, int64_t E, bool grouped) {
    const int64_t slots = grouped ? tile_slots(R, E, kRows) : (R + kRows - 1) / kRows;
    return grouped || slots > 1 ? (size_t)slots * N * sizeof(float) : 0;
}

hipError_t launch_activation_grad(ActGradArgs a, DType dt, hipStream_t stream) {
    const int F = a.act == kSwiglu ? a.N / 2 : a.N;
    const uintptr_t at = (uintptr_t)a.dY | (uintptr_t)a.Z | (uintptr_t)a.dZ;
    const bool rows16 = F % 8 == 0 && at % 16 == 0 && a.y_stride % 8 == 0 && a.z_stride % 8 == 0;
    // One block of rows writes dbias itself.
    if (a.dbias == nullptr || activation_grad_workspace(a.R, a.N, a.E, a.offsets != nullptr) == 0)
        a.part = nullptr;
    if (a.R > 0) {
        // Eight columns a lane are 16 bytes, but as many slopes one after the other: few elements
        // are spread (6 x 4096 with GELU and bias 5.9 us of eight, 2.9 of one).
        const bool wide = rows16 && (int64_t)a.R * F >= 1 << 18;
        if (dt == kF16 && wide) act_grad<F16, 8>(a, stream);
        else if (dt == kF16) act_grad<F16, 1>(a, stream);
        else if (wide) act_grad<BF16, 8>(a, stream);
        else act_grad<BF16, 1>(a, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // No row: the sums are 0.
    if (a.dbias != nullptr && (a.part != nullptr || a.R == 0)) {
        const dim3 grid((unsigned)((a.N + kThreads - 1) / kThreads), (unsigned)a.E);
        bias_sum_kernel<<<grid, kThreads, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace mxfp4
