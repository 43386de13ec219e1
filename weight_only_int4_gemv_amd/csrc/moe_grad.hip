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

// ------------------------------------------------------------ softmax of logits
//
// A token takes LANES lanes of a wave, each with PER neighbouring experts: up to 64 experts eight
// lanes, so that a wave works on eight tokens, reads 16 bytes a lane and sums over a row of lanes
// with DPP steps.  (65521 tokens of 128 experts: a wave per token with shuffles through LDS takes
// 36 us for the loss's sums and 35 for the gradient.)

// The value of lane i ^ 1, i ^ 2, then of the other half of 8, of 16, of 32 and of 64 lanes whose
// own values are alike.
template <int D>
__device__ __forceinline__ float other(float v) {
    const int b = __builtin_bit_cast(int, v);
    if constexpr (D == 1) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, b, 0xB1, 0xF, 0xF, true));
    else if constexpr (D == 2) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, b, 0x4E, 0xF, 0xF, true));
    else if constexpr (D == 4) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, b, 0x141, 0xF, 0xF, true));
    else if constexpr (D == 8) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, b, 0x140, 0xF, 0xF, true));
    else return __shfl_xor(v, D);
}
template <int LANES, int D = 1>
__device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (D == LANES) return v;
    else return lanes_sum<LANES, 2 * D>(v + other<D>(v));
}
__device__ __forceinline__ float wave_sum(float v) { return lanes_sum<kWave>(v); }
// NaN aside, which enters by its own exponential.
template <int LANES, int D = 1>
__device__ __forceinline__ float lanes_peak(float v) {
    if constexpr (D == LANES) return v;
    else return lanes_peak<LANES, 2 * D>(fmaxf(v, other<D>(v)));
}

// exp(t) for t <= 0 to about an ulp: the product with log2 e in two parts, the low one as a factor
// 1 + low ln 2.  Below -200 it is 0; a NaN stays.
__device__ __forceinline__ float exp_down(float t) {
    t = t < -200.0f ? -200.0f : t;
    const float h = t * 1.44269502f;
    const float l = fmaf(t, 1.44269502f, -h) + t * 1.92596299e-8f;
    const float e = __builtin_amdgcn_exp2f(h);
    return fmaf(e, l * 0.693147181f, e);
}

// PER elements from p on, `left` of which are there: others are `fill`.
template <typename T, int PER>
__device__ __forceinline__ void load_some(const typename T::type* p, int left, bool wide, float fill,
                                          float (&v)[PER]) {
    if (wide && left >= PER) {
        typename T::type b[PER];
        __builtin_memcpy(b, __builtin_assume_aligned(p, 16), sizeof(b));
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = T::load(b[i]);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = i < left ? T::load(p[i]) : fill;
    }
}

// exp(l - peak) of a token's logits and their sum.  A row without a usable expert (all -infinity)
// has sum 0; one with a NaN or +infinity has sum NaN.
template <int LANES, int PER>
struct Softmax {
    float p[PER], peak, sum;
    __device__ __forceinline__ void make() {                // from the logits in p
        peak = p[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) peak = fmaxf(peak, p[i]);
        peak = lanes_peak<LANES>(peak);
        const float from = peak == -INFINITY ? 0.0f : peak;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            p[i] = exp_down(p[i] - from);
            s += p[i];
        }
        sum = lanes_sum<LANES>(s);
    }
};
template <DType DT, int PER>
__device__ __forceinline__ void load_logits(const void* logits, int64_t row, int e0, int E, bool wide,
                                            float (&p)[PER]) {
    typedef typename Of<DT>::tag T;
    load_some<T, PER>((const typename T::type*)logits + row + e0, E - e0, wide, -INFINITY, p);
}

// Whether rows of PER-element pieces start on 16 bytes.
inline bool wide_rows(const void* p, int64_t stride, DType dt) {
    return (uintptr_t)p % 16 == 0 && stride * (dt == kF32 ? 4 : 2) % 16 == 0;
}

// ------------------------------------------------------------------- balance
//
// loss = E sum_e (c_e / C) (S_e / T'): c_e the choices of expert e, C their sum, S_e the sum of
// the tokens' softmax at e, T' the tokens that may use an expert.  Lanes add their tokens' shares;
// blocks leave sums [block][E] and counts [block][E + 1] to a second launch, which adds them in
// order: the result does not depend on scheduling.  65521 tokens of 128 bf16 logits (16.8 MB and
// 2 MB of choices): 12 us of latency (two waves a SIMD, which wait 65 % of their time; vector units
// 24 % busy) and 6 us for the second launch, one block's latency; adding the blocks with atomics
// would save the launch and the fixed order.
constexpr int kBalanceThreads = 512;
constexpr int kMaxBalanceBlocks = 256;

struct BalancePart {
    float* sums;
    int* counts;
};
__host__ __device__ inline BalancePart balance_part(void* part, int64_t blocks, int64_t block, int E) {
    return {(float*)part + block * E, (int*)part + blocks * E + block * (E + 1)};
}

// The loss of a block's sums: thread e has expert e's choices c and sum s (0 from E on).
template <int THREADS>
__device__ __forceinline__ void write_loss(float s, int c, int tokens, int E, float* loss) {
    __shared__ float product[THREADS / kWave];
    __shared__ int chosen[THREADS / kWave];
    float p = wave_sum((float)c * s);
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) c += __shfl_xor(c, d);
    if (threadIdx.x % kWave == 0) product[threadIdx.x / kWave] = p, chosen[threadIdx.x / kWave] = c;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < THREADS / kWave; ++w) p += product[w], c += chosen[w];
    *loss = p * ((float)E / (fmaxf((float)c, 1.0f) * fmaxf((float)tokens, 1.0f)));
}

// loss: written by this kernel where one block has all tokens (E <= kBalanceThreads), else NULL.
template <DType DT, int LANES, int PER>
__global__ __launch_bounds__(kBalanceThreads) void balance_kernel(const void* logits, int T, int E,
                                                                  int64_t stride, bool wide,
                                                                  const int* ids, int k, void* part,
                                                                  float* loss, int* counts) {
    constexpr int kGroups = kBalanceThreads / LANES, kExperts = LANES * PER;
    // Sums of a wave's tokens meet in registers first: one row a wave.
    constexpr int kRows = kBalanceThreads / kWave;
    __shared__ int hist[kExperts];
    __shared__ float sums[kRows][kExperts];
    __shared__ int used;
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES, e0 = lane * PER;
    for (int e = threadIdx.x; e < kExperts; e += kBalanceThreads) hist[e] = 0;
    if (threadIdx.x == 0) used = 0;
    __syncthreads();
    float sum[PER] = {}, next[PER];
    int tokens = 0;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    int64_t t = (int64_t)blockIdx.x * kGroups + group;
    if (t < T) load_logits<DT>(logits, t * stride, e0, E, wide, next);
    for (; t < T; t += step) {
        Softmax<LANES, PER> s;
#pragma unroll
        for (int i = 0; i < PER; ++i) s.p[i] = next[i];
        if (t + step < T) load_logits<DT>(logits, (t + step) * stride, e0, E, wide, next);
        for (int j = lane; j < k; j += LANES) {
            const int id = ids[t * k + j];
            if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
        }
        s.make();
        if (s.sum == 0.0f) continue;
        ++tokens;
        const float inv = __builtin_amdgcn_rcpf(s.sum);
#pragma unroll
        for (int i = 0; i < PER; ++i) sum[i] += s.p[i] * inv;
    }
    if (lane == 0) atomicAdd(&used, tokens);
    // The groups of a wave, then the waves in order.
#pragma unroll
    for (int d = LANES; d < kWave; d <<= 1)
#pragma unroll
        for (int i = 0; i < PER; ++i) sum[i] += __shfl_xor(sum[i], d);
    if (threadIdx.x % kWave < LANES) {
#pragma unroll
        for (int i = 0; i < PER; ++i) sums[threadIdx.x / kWave][e0 + i] = sum[i];
    }
    __syncthreads();
    const BalancePart out = balance_part(part, gridDim.x, blockIdx.x, E);
    float s = 0.0f;
    int c = 0;
    for (int e = threadIdx.x; e < E; e += kBalanceThreads) {
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kRows; ++w) s += sums[w][e];
        c = hist[e];
        if (loss != nullptr) counts[e] = c;
        else out.sums[e] = s, out.counts[e] = c;
    }
    if (threadIdx.x == 0) *(loss != nullptr ? counts + E : out.counts + E) = used;
    if (loss != nullptr) write_loss<kBalanceThreads>(s, c, used, E, loss);
}

// One block: every expert's sums over the blocks, rows of them to each of 1024 / experts threads,
// then the loss.
__global__ __launch_bounds__(1024) void balance_sum_kernel(void* part, int blocks, int E, int log2_experts,
                                                           float* loss, int* counts) {
    __shared__ float sums[1024];
    __shared__ int chosen[1024];
    __shared__ int tokens[16];
    const int tid = threadIdx.x, experts = 1 << log2_experts;
    const int e = tid & (experts - 1), row = tid >> log2_experts, rows = 1024 >> log2_experts;
    float s = 0.0f;
    int c = 0, n = 0;
    const BalancePart p = balance_part(part, blocks, 0, E);
    if (e < E) {
#pragma unroll 8
        for (int b = row; b < blocks; b += rows) {
            s += p.sums[(int64_t)b * E + e];
            c += p.counts[(int64_t)b * (E + 1) + e];
        }
    }
    static_assert(kMaxBalanceBlocks <= 1024, "a thread a block");
    if (tid < blocks) n = p.counts[(int64_t)tid * (E + 1) + E];
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) n += __shfl_xor(n, d);
    if (tid % kWave == 0) tokens[tid / kWave] = n;
    sums[tid] = s;
    chosen[tid] = c;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) n += tokens[w];
    for (int r = 1; r < min(rows, blocks); ++r) {
        s += sums[(r * experts + tid) & 1023];              // of threads of row 0, the others' are not used
        c += chosen[(r * experts + tid) & 1023];
    }
    const bool mine = row == 0 && e < E;
    if (mine) counts[e] = c;
    if (tid == 0) counts[E] = n;
    write_loss<1024>(mine ? s : 0.0f, mine ? c : 0, n, E, loss);
}

// ------------------------------------------------------------- router's gradient
//
// Four waves a SIMD walk over the tokens, the next logits on their way (65521 tokens of 128 experts
// 14 us; as many waves as tokens need 23).  They wait 66 % of their time, vector units are 35 % busy.  With P the softmax over the usable experts, the loss gives
//     dloss E / (C T') P_e (c_e - sum_i c_i P_i)
// and the routing weights, renormalized over the chosen j (w their softmax),
//     w_j (dw_j - sum_i w_i dw_i) at expert id_j,
// or not renormalized
//     P_e (sum of dw_j over the j with id_j = e, less sum_i P_(id_i) dw_i).
template <DType DT, int LANES, int PER>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs a, bool wide, bool wide_out) {
    typedef typename Of<DT>::tag T;
    constexpr int kSlots = LANES >= 32 ? 1 : 32 / LANES;    // choices of a lane
    __shared__ __align__(16) float turn[256 / LANES][LANES * PER];
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES, e0 = lane * PER, E = a.E;
    const int64_t step = (int64_t)gridDim.x * (256 / LANES);
    int64_t t = (int64_t)blockIdx.x * (256 / LANES) + group;
    if (t >= a.T) return;                                   // all of a token's lanes
    const bool routed = a.dweights != nullptr;
    // The loss's factors, the same for all tokens.
    float c[PER], scale = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = 0.0f;
    if (a.counts != nullptr) {
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            c[i] = e0 + i < E ? (float)a.counts[e0 + i] : 0.0f;
            all += c[i];
        }
        all = lanes_sum<LANES>(all);
        scale = *a.dloss * ((float)E / (fmaxf(all, 1.0f) * fmaxf((float)a.counts[E], 1.0f)));
    }
    Softmax<LANES, PER> s;
    load_logits<DT>(a.logits, t * a.stride, e0, E, wide, s.p);
    for (;;) {
        // Lane j % LANES holds choice j in slot j / LANES.
        int id[kSlots];
        float l[kSlots], dw[kSlots];
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            const int j = lane + LANES * i;
            id[i] = -1, l[i] = -INFINITY, dw[i] = 0.0f;
            if (routed && j < a.k) {
                id[i] = a.ids[t * a.k + j];
                dw[i] = a.dweights[t * a.k + j];
            }
            if (id[i] < 0 || id[i] >= E) id[i] = -1;
            else l[i] = T::load(((const typename T::type*)a.logits)[t * a.stride + id[i]]);
            if (l[i] == -INFINITY) id[i] = -1;                  // an expert that cannot be used
        }
        float next[PER];
        if (t + step < a.T) load_logits<DT>(a.logits, (t + step) * a.stride, e0, E, wide, next);
        s.make();
        const float inv = s.sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(s.sum);
        float grad[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            s.p[i] *= inv;
            grad[i] = 0.0f;
        }
        if (a.counts != nullptr) {
            float mean = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) mean += c[i] * s.p[i];
            mean = lanes_sum<LANES>(mean);
#pragma unroll
            for (int i = 0; i < PER; ++i) grad[i] = scale * s.p[i] * (c[i] - mean);
        }
        if (routed) {
            float peak = s.peak, sum = 0.0f, mean = 0.0f, w[kSlots];
            if (a.renormalize) {
                peak = l[0];
#pragma unroll
                for (int i = 1; i < kSlots; ++i) peak = fmaxf(peak, l[i]);
                peak = lanes_peak<LANES>(peak);
            }
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                w[i] = id[i] >= 0 ? exp_down(l[i] - peak) : 0.0f;
                sum += w[i];
            }
            const float per = a.renormalize ? __builtin_amdgcn_rcpf(lanes_sum<LANES>(sum)) : inv;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                w[i] = id[i] >= 0 ? w[i] * per : 0.0f;
                mean += id[i] >= 0 ? w[i] * dw[i] : 0.0f;
            }
            mean = lanes_sum<LANES>(mean);
            if (!a.renormalize) {
#pragma unroll
                for (int i = 0; i < PER; ++i) grad[i] -= s.p[i] * mean;
            }
            // To the experts' lanes through LDS (the wave's own part of it).  Where a token names an
            // expert twice, a choice does not find its own number again: then one by one.
            float* mark = turn[group];
            auto settle = [] {
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            };
            bool twice = false;
#pragma unroll
            for (int i = 0; i < kSlots; ++i)
                if (id[i] >= 0) mark[id[i]] = (float)(lane + LANES * i);
            settle();
#pragma unroll
            for (int i = 0; i < kSlots; ++i)
                if (id[i] >= 0) twice = twice || mark[id[i]] != (float)(lane + LANES * i);
            settle();
            float add[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) turn[group][e0 + i] = 0.0f;
            settle();
            const bool one_by_one = __any(twice);
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                const float mine = a.renormalize ? w[i] * (dw[i] - mean) : w[i] * dw[i];
                if (!one_by_one) {
                    if (id[i] >= 0) turn[group][id[i]] = mine;
                } else {
                    for (int j = 0; j < LANES; ++j) {
                        if (lane == j && id[i] >= 0) turn[group][id[i]] += mine;
                        settle();
                    }
                }
            }
            settle();
#pragma unroll
            for (int i = 0; i < PER; ++i) add[i] = turn[group][e0 + i];
#pragma unroll
            for (int i = 0; i < PER; ++i) grad[i] += add[i];
        }
        typename T::type* out = (typename T::type*)a.dlogits + t * E + e0;
        typename T::type o[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) o[i] = T::store(grad[i]);
        if (wide_out && e0 + PER <= E) {
            __builtin_memcpy(__builtin_assume_aligned(out, 16), o, sizeof(o));
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (e0 + i < E) out[i] = o[i];
        }
        t += step;
        if (t >= a.T) return;
#pragma unroll
        for (int i = 0; i < PER; ++i) s.p[i] = next[i];
    }
}

// ----------------------------------------------------- the weighted sum's gradient
//
// dY[r] = weights[t, j] dout[t] and dweights[t, j] = <dout[t], Y[r]> for the row r =
// positions[t, j].  A wave per choice: it reads both rows once (the token's other choices find
// dout in the caches) and writes dY's row if tokens[r] names the token and no earlier choice of
// it the row; a row that no choice of its token names gets zeros from wave r.  So every row of
// dY is written once whatever the tensors hold.  Bound by HBM: 6000 tokens, one in
// sixteen of them padding, the others with eight rows of 4096 (787 MB), take 151 us, 5.2 TB/s; with one
// piece of the rows in hand 173.
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
                constexpr int kHand = VEC == 8 ? 4 : 1;     // pieces of the rows in hand
                for (int n0 = lane * VEC; n0 < N; n0 += kHand * kWave * VEC) {
                    Piece<uint16_t, VEC> d[kHand], o;
                    Piece<typename ROW::type, VEC> y[kHand];
#pragma unroll
                    for (int h = 0; h < kHand; ++h) {
                        const int n = n0 + h * kWave * VEC;
                        if (n >= N) continue;
                        d[h].load(dout + (int64_t)t * N + n);
                        y[h].load_once(Y + (int64_t)r * N + n);
                    }
#pragma unroll
                    for (int h = 0; h < kHand; ++h) {
                        const int n = n0 + h * kWave * VEC;
                        if (n >= N) continue;
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            const float e = T::load(d[h].get(i));
                            dot = fmaf(e, ROW::load(y[h].get(i)), dot);
                            o.set(i, T::store(w * e));
                        }
                        if (write) o.store_once(dY + (int64_t)r * N + n);
                    }
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
                Piece<uint16_t, VEC> o;
#pragma unroll
                for (int i = 0; i < VEC; ++i) o.set(i, 0);
                for (int n = lane * VEC; n < N; n += kWave * VEC) o.store_once(dY + c * N + n);
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

// Lanes of a token and experts of a lane.
template <int LANES, int PER>
struct Lanes {
    static constexpr int lanes = LANES, per = PER;
};
template <class F>
void by_experts(int E, F f) {
    if (E <= 64) f(Lanes<8, 8>());
    else if (E <= 128) f(Lanes<16, 8>());
    else if (E <= 256) f(Lanes<32, 8>());
    else if (E <= 512) f(Lanes<64, 8>());
    else f(Lanes<64, 16>());
}
template <class F>
void by_dtype(DType dt, F f) {
    if (dt == kF16) f(std::integral_constant<DType, kF16>());
    else if (dt == kBF16) f(std::integral_constant<DType, kBF16>());
    else f(std::integral_constant<DType, kF32>());
}

// Blocks of at least two tokens a group of lanes.
int balance_blocks(int64_t T, int E) {
    int lanes = 8;
    by_experts(E, [&](auto n) { lanes = decltype(n)::lanes; });
    const int64_t each = 2 * (kBalanceThreads / lanes), blocks = (T + each - 1) / each;
    return (int)(blocks < kMaxBalanceBlocks ? blocks : kMaxBalanceBlocks);
}

}  // namespace

size_t balance_workspace(int64_t T, int64_t E) {
    const int blocks = balance_blocks(T, (int)E);
    return blocks == 1 && E <= kBalanceThreads ? 0 : (size_t)blocks * (2 * E + 1) * 4;
}

hipError_t launch_balance(const void* logits, DType dt, int T, int E, int64_t stride,
                          const int* ids, int k, float* loss, int* counts, void* part,
                          hipStream_t stream) {
    const int blocks = balance_blocks(T, E);
    const bool wide = wide_rows(logits, stride, dt), one = blocks == 1 && E <= kBalanceThreads;
    if (blocks > 0) {
        by_dtype(dt, [&](auto d) {
            by_experts(E, [&](auto n) {
                typedef decltype(n) L;
                balance_kernel<decltype(d)::value, L::lanes, L::per>
                    <<<blocks, kBalanceThreads, 0, stream>>>(logits, T, E, stride, wide, ids, k, part,
                                                             one ? loss : nullptr, counts);
            });
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (one) return hipSuccess;
    int log2_experts = 0;
    while (1 << log2_experts < E) ++log2_experts;
    balance_sum_kernel<<<1, 1024, 0, stream>>>(part, blocks, E, log2_experts, loss, counts);
    return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradArgs& a, DType dt, hipStream_t stream) {
    const bool wide = wide_rows(a.logits, a.stride, dt), wide_out = wide_rows(a.dlogits, a.E, dt);
    by_dtype(dt, [&](auto d) {
        by_experts(a.E, [&](auto n) {
            typedef decltype(n) L;
            constexpr int kTokens = 256 / L::lanes;
            const int blocks = (a.T + kTokens - 1) / kTokens, most = 4 * 256;   // several tokens a lane
            route_grad_kernel<decltype(d)::value, L::lanes, L::per>
                <<<blocks < most ? blocks : most, 256, 0, stream>>>(a, wide, wide_out);
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
