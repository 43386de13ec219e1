// moe_grad.hip — the balance loss with per-expert counts, the router's gradient and the
// gradient of the weighted sum over a token's expert rows.
#include <type_traits>

#include "mxfp4_device.h"
#include "mxfp4_launch.h"

namespace mxfp4 {
namespace {

struct F32 {
    typedef float type;
    static __device__ __forceinline__ float load(float f) { return f; }
    static __device__ __forceinline__ float store(float f) { return f; }
};
template <DType DT>
struct Of;
template <>
struct Of<kF16> { typedef F16 tag; };
template <>
struct Of<kBF16> { typedef BF16 tag; };
template <>
struct Of<kF32> { typedef F32 tag; };

template <DType DT>
__device__ __forceinline__ float load(const void* p, int64_t i) {
    typedef typename Of<DT>::tag T;
    return T::load(((const typename T::type*)p)[i]);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
    return v;
}
// The largest value; a NaN counts above every number.
__device__ __forceinline__ float wave_peak(float v) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const float o = __shfl_xor(v, d);
        v = o > v || o != o ? o : v;
    }
    return v;
}

// exp(l - max) of a token's logits, lane l holding experts l, l + 64, ..., and their sum.  A row
// without a usable expert (all -infinity) has sum 0.
template <DType DT, int PER_LANE>
struct Softmax {
    float p[PER_LANE], peak, sum;
    __device__ __forceinline__ void read(const void* logits, int64_t row, int E) {
        const int lane = threadIdx.x & (kWave - 1);
        peak = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
            const int e = lane + kWave * i;
            p[i] = e < E ? load<DT>(logits, row + e) : -INFINITY;
            peak = p[i] > peak || p[i] != p[i] ? p[i] : peak;
        }
        peak = wave_peak(peak);
        float s = 0.0f;
        const float from = peak == -INFINITY ? 0.0f : peak;
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
            p[i] = p[i] == -INFINITY ? 0.0f : expf(p[i] - from);
            s += p[i];
        }
        sum = wave_sum(s);
    }
};

// ------------------------------------------------------------------- balance
//
// loss = E sum_e (c_e / C) (S_e / T'): c_e the choices of expert e, C their sum, S_e the sum of
// the tokens' softmax at e, T' the tokens that may use an expert.  A wave adds a token at a time
// to its lanes' sums; blocks leave theirs to a second launch, which adds them in order.
constexpr int kBalanceWaves = 4;
constexpr int kBalanceThreads = kBalanceWaves * kWave;
constexpr int kMaxBalanceBlocks = 512;

struct BalancePart {            // of a block: sums fp32 [E], counts int32 [E + 1]
    float* sums;
    int* counts;
};
__host__ __device__ inline BalancePart balance_part(void* part, int64_t block, int E) {
    char* at = (char*)part + block * (2 * (int64_t)E + 1) * 4;
    return {(float*)at, (int*)(at + 4 * (int64_t)E)};
}

template <DType DT, int PER_LANE>
__global__ __launch_bounds__(kBalanceThreads) void balance_kernel(const void* logits, int T, int E,
                                                                  int64_t stride, const int* ids,
                                                                  int k, void* part) {
    __shared__ int hist[kWave * PER_LANE];
    __shared__ float sums[kBalanceWaves][kWave * PER_LANE];
    __shared__ int used[kBalanceWaves];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    for (int e = threadIdx.x; e < kWave * PER_LANE; e += kBalanceThreads) hist[e] = 0;
    __syncthreads();
    float sum[PER_LANE] = {};
    int tokens = 0;
    for (int t = blockIdx.x * kBalanceWaves + wave; t < T; t += gridDim.x * kBalanceWaves) {
        Softmax<DT, PER_LANE> s;
        s.read(logits, t * stride, E);
        const int id = lane < k ? ids[(int64_t)t * k + lane] : -1;
        if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
        if (s.sum == 0.0f) continue;
        ++tokens;
        const float inv = 1.0f / s.sum;
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) sum[i] += s.p[i] * inv;
    }
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) sums[wave][lane + kWave * i] = sum[i];
    if (lane == 0) used[wave] = tokens;
    __syncthreads();
    const BalancePart out = balance_part(part, blockIdx.x, E);
    for (int e = threadIdx.x; e < E; e += kBalanceThreads) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kBalanceWaves; ++w) s += sums[w][e];
        out.sums[e] = s;
        out.counts[e] = hist[e];
    }
    if (threadIdx.x == 0) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < kBalanceWaves; ++w) n += used[w];
        out.counts[E] = n;
    }
}

// One block: the blocks' sums in order, then the loss over the experts in order.
__global__ __launch_bounds__(1024) void balance_sum_kernel(void* part, int blocks, int E,
                                                           float* loss, int* counts) {
    __shared__ float product[1024];
    __shared__ int chosen[1024];
    __shared__ int tokens;
    const int e = threadIdx.x;
    float s = 0.0f;
    int c = 0;
    if (e < E) {
        for (int b = 0; b < blocks; ++b) {
            const BalancePart p = balance_part(part, b, E);
            s += p.sums[e];
            c += p.counts[e];
        }
        counts[e] = c;
    }
    if (e == 0) {
        int n = 0;
        for (int b = 0; b < blocks; ++b) n += balance_part(part, b, E).counts[E];
        tokens = n;
        counts[E] = n;
    }
    product[e] = (float)c * s;
    chosen[e] = c;
    __syncthreads();
    for (int d = 512; d > 0; d >>= 1) {
        if (e < d) {
            product[e] += product[e + d];
            chosen[e] += chosen[e + d];
        }
        __syncthreads();
    }
    if (e == 0) {
        const float scale = (float)E / (fmaxf((float)chosen[0], 1.0f) * fmaxf((float)tokens, 1.0f));
        *loss = product[0] * scale;
    }
}

// ------------------------------------------------------------- router's gradient
//
// A wave per token.  With P the softmax over the usable experts, the loss gives
//     dloss E / (C T') P_e (c_e - sum_i c_i P_i)
// and the routing weights, renormalized over the chosen j (w their softmax),
//     w_j (dw_j - sum_i w_i dw_i) at expert id_j,
// or not renormalized
//     P_e (sum of dw_j over the j with id_j = e, less sum_i P_(id_i) dw_i).
template <DType DT, int PER_LANE>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs a) {
    typedef typename Of<DT>::tag T;
    const int lane = threadIdx.x & (kWave - 1);
    const int t = blockIdx.x * 4 + threadIdx.x / kWave;
    if (t >= a.T) return;
    const int E = a.E;
    Softmax<DT, PER_LANE> s;
    s.read(a.logits, t * a.stride, E);
    const float inv = s.sum == 0.0f ? 0.0f : 1.0f / s.sum;
    float grad[PER_LANE];
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
        s.p[i] *= inv;
        grad[i] = 0.0f;
    }
    if (a.counts != nullptr) {
        float c[PER_LANE], all = 0.0f, mean = 0.0f;
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
            const int e = lane + kWave * i;
            c[i] = e < E ? (float)a.counts[e] : 0.0f;
            all += c[i];
            mean += c[i] * s.p[i];
        }
        all = wave_sum(all);
        mean = wave_sum(mean);
        const float tokens = fmaxf((float)a.counts[E], 1.0f);
        const float scale = *a.dloss * ((float)E / (fmaxf(all, 1.0f) * tokens));
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) grad[i] = scale * s.p[i] * (c[i] - mean);
    }
    if (a.dweights != nullptr) {
        // Lane j < k: choice j.
        int id = -1;
        float l = -INFINITY, dw = 0.0f;
        if (lane < a.k) {
            id = a.ids[(int64_t)t * a.k + lane];
            if (id < 0 || id >= E) id = -1;
            else l = load<DT>(a.logits, t * a.stride + id);
            if (id >= 0) dw = a.dweights[(int64_t)t * a.k + lane];
        }
        if (l == -INFINITY) id = -1, dw = 0.0f;         // an expert that cannot be used
        float w = 0.0f;
        if (a.renormalize) {
            const float peak = wave_peak(l);
            if (id >= 0) w = expf(l - peak);
            const float sum = wave_sum(w);
            if (id >= 0) w /= sum;
        } else if (id >= 0) {
            w = expf(l - s.peak) * inv;
        }
        const float mean = wave_sum(w * dw);
        const float mine = a.renormalize ? w * (dw - mean) : w * dw;
        if (!a.renormalize) {
#pragma unroll
            for (int i = 0; i < PER_LANE; ++i) grad[i] -= s.p[i] * mean;
        }
        for (int j = 0; j < a.k; ++j) {
            const int e = __builtin_amdgcn_readlane(id, j);
            const float v = __builtin_bit_cast(
                float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, mine), j));
#pragma unroll
            for (int i = 0; i < PER_LANE; ++i)
                if (e == lane + kWave * i) grad[i] += v;
        }
    }
    typename T::type* out = (typename T::type*)a.dlogits + (int64_t)t * E;
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
        const int e = lane + kWave * i;
        if (e < E) out[e] = T::store(grad[i]);
    }
}

// ----------------------------------------------------- the weighted sum's gradient
//
// dY[r] = weights[t, j] dout[t] and dweights[t, j] = <dout[t], Y[r]> for the row r =
// positions[t, j].  A wave per choice: it reads both rows once (the token's other choices find
// dout in the caches) and writes dY's row if tokens[r] names the token and no earlier choice of
// it the row; a row that no choice of its token names gets zeros from wave r.  So every row of
// dY is written once whatever the tensors hold.
template <typename T, typename ROW, int VEC>
__global__ __launch_bounds__(256) void combine_grad_kernel(const uint16_t* dout, const void* Y_,
                                                           int R, int N, const int* tokens,
                                                           const int* positions,
                                                           const float* weights, int T_, int k,
                                                           uint16_t* dY, float* dweights) {
    const auto* Y = (const typename ROW::type*)Y_;
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t choices = (int64_t)T_ * k;
    const int64_t waves = (int64_t)gridDim.x * 4;
    for (int64_t c = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
         c < choices || c < R; c += waves) {
        if (c < choices) {
            const int t = (int)(c / k), j = (int)(c - (int64_t)t * k);
            const int r = positions[c];
            float dot = 0.0f;
            if (r >= 0 && r < R) {
                // The choices of the token that name the row: the first one writes it.
                const bool same = lane < k && positions[(int64_t)t * k + lane] == r;
                const uint64_t named = __ballot(same);
                const bool write = tokens[r] == t && __builtin_ctzll(named) == j;
                const float w = wave_sum(same ? weights[(int64_t)t * k + lane] : 0.0f);
                for (int n = lane * VEC; n < N; n += kWave * VEC) {
                    uint16_t d[VEC], o[VEC];
                    typename ROW::type y[VEC];
                    constexpr int kAlign = sizeof(y) < 16 ? sizeof(y) : 16;
                    __builtin_memcpy(d, __builtin_assume_aligned(dout + (int64_t)t * N + n, 2 * VEC),
                                     sizeof(d));
                    __builtin_memcpy(y, __builtin_assume_aligned(Y + (int64_t)r * N + n, kAlign),
                                     sizeof(y));
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        dot = fmaf(T::load(d[i]), ROW::load(y[i]), dot);
                        o[i] = T::store(w * T::load(d[i]));
                    }
                    if (write)
                        __builtin_memcpy(__builtin_assume_aligned(dY + (int64_t)r * N + n, 2 * VEC),
                                         o, sizeof(o));
                }
                dot = wave_sum(dot);
            }
            if (lane == 0) dweights[c] = dot;
        }
        if (c < R) {
            const int t = tokens[c];
            const bool named = t >= 0 && t < T_ &&
                               __any(lane < k && positions[(int64_t)t * k + lane] == (int)c);
            if (!named) {
                const uint16_t o[VEC] = {};
                for (int n = lane * VEC; n < N; n += kWave * VEC)
                    __builtin_memcpy(__builtin_assume_aligned(dY + c * N + n, 2 * VEC), o, sizeof(o));
            }
        }
    }
}

template <typename T, typename ROW>
void combine_grad(const uint16_t* dout, const void* Y, int R, int N, const int* tokens,
                  const int* positions, const float* weights, int T_, int k, uint16_t* dY,
                  float* dweights, hipStream_t stream) {
    const bool wide = N % 8 == 0 && ((uintptr_t)dout | (uintptr_t)Y | (uintptr_t)dY) % 16 == 0;
    const int64_t most = (int64_t)T_ * k > R ? (int64_t)T_ * k : R, blocks = (most + 3) / 4;
    const unsigned grid = (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20);
    if (wide)
        combine_grad_kernel<T, ROW, 8><<<grid, 256, 0, stream>>>(dout, Y, R, N, tokens, positions,
                                                                 weights, T_, k, dY, dweights);
    else
        combine_grad_kernel<T, ROW, 1><<<grid, 256, 0, stream>>>(dout, Y, R, N, tokens, positions,
                                                                 weights, T_, k, dY, dweights);
}

// Experts a lane holds.
template <class F>
void by_experts(int E, F f) {
    if (E <= 64) f(std::integral_constant<int, 1>());
    else if (E <= 128) f(std::integral_constant<int, 2>());
    else if (E <= 256) f(std::integral_constant<int, 4>());
    else f(std::integral_constant<int, 16>());
}
template <class F>
void by_dtype(DType dt, F f) {
    if (dt == kF16) f(std::integral_constant<DType, kF16>());
    else if (dt == kBF16) f(std::integral_constant<DType, kBF16>());
    else f(std::integral_constant<DType, kF32>());
}

int balance_blocks(int64_t T) {
    const int64_t blocks = (T + kBalanceWaves - 1) / kBalanceWaves;
    return (int)(blocks < kMaxBalanceBlocks ? blocks : kMaxBalanceBlocks);
}

}  // namespace

size_t balance_workspace(int64_t T, int64_t E) {
    return (size_t)balance_blocks(T) * (2 * E + 1) * 4;
}

hipError_t launch_balance(const void* logits, DType dt, int T, int E, int64_t stride,
                          const int* ids, int k, float* loss, int* counts, void* part,
                          hipStream_t stream) {
    const int blocks = balance_blocks(T);
    if (blocks > 0) {
        by_dtype(dt, [&](auto d) {
            by_experts(E, [&](auto n) {
                balance_kernel<decltype(d)::value, decltype(n)::value>
                    <<<blocks, kBalanceThreads, 0, stream>>>(logits, T, E, stride, ids, k, part);
            });
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    balance_sum_kernel<<<1, 1024, 0, stream>>>(part, blocks, E, loss, counts);
    return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradArgs& a, DType dt, hipStream_t stream) {
    const unsigned grid = (unsigned)((a.T + 3) / 4);
    by_dtype(dt, [&](auto d) {
        by_experts(a.E, [&](auto n) {
            route_grad_kernel<decltype(d)::value, decltype(n)::value><<<grid, 256, 0, stream>>>(a);
        });
    });
    return hipGetLastError();
}

hipError_t launch_combine_grad(const uint16_t* dout, const void* Y, bool rows32, DType dt, int R,
                               int N, const int* tokens, const int* positions,
                               const float* weights, int T, int k, uint16_t* dY, float* dweights,
                               hipStream_t stream) {
    if (dt == kF16 && rows32)
        combine_grad<F16, F32>(dout, Y, R, N, tokens, positions, weights, T, k, dY, dweights, stream);
    else if (dt == kF16)
        combine_grad<F16, F16>(dout, Y, R, N, tokens, positions, weights, T, k, dY, dweights, stream);
    else if (rows32)
        combine_grad<BF16, F32>(dout, Y, R, N, tokens, positions, weights, T, k, dY, dweights, stream);
    else
        combine_grad<BF16, BF16>(dout, Y, R, N, tokens, positions, weights, T, k, dY, dweights,
                                 stream);
    return hipGetLastError();
}

}  // namespace mxfp4
