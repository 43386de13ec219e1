// moe_route.hip — routing of tokens to experts, the expert-ordered plan and the
// weighted sum that takes the experts' rows back to their tokens.
#include "mxfp4_device.h"
#include "mxfp4_launch.h"

namespace mxfp4 {
namespace {

// ------------------------------------------------------------------ routing
//
// One wave per token; lane l holds the logits l, l + 64, ...  A choice is the
// largest key over the wave: the logit mapped to an unsigned number in its
// order (a NaN above everything, -infinity lowest), then the lower expert.

template <DType DT>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
    if constexpr (DT == kF32) return ((const float*)p)[i];
    else if constexpr (DT == kBF16) return BF16::load(((const uint16_t*)p)[i]);
    else return F16::load(((const uint16_t*)p)[i]);
}

// Rising with f; -infinity 0x007FFFFF, every NaN 0xFFFFFFFF; never 0.
__device__ __forceinline__ uint32_t order_key(float f) {
    if (f != f) return 0xFFFFFFFFu;
    const uint32_t b = __builtin_bit_cast(uint32_t, f == 0.0f ? 0.0f : f);    // -0 equals 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
constexpr uint32_t kMinusInf = 0x007FFFFFu;

__device__ __forceinline__ float key_value(uint32_t k) {
    if (k == 0xFFFFFFFFu) return __builtin_bit_cast(float, 0x7FC00000u);
    return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

template <DType DT, int PER_LANE>
__global__ __launch_bounds__(256) void route_kernel(const void* logits, int T, int E,
                                                    int64_t stride, int k, bool renormalize,
                                                    int* ids, float* weights) {
    const int lane = threadIdx.x & (kWave - 1);
    const int t = blockIdx.x * 4 + threadIdx.x / kWave;
    if (t >= T) return;
    uint32_t key[PER_LANE];
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
        const int e = lane + kWave * i;
        key[i] = e < E ? order_key(logit<DT>(logits, (int64_t)t * stride + e)) : 0;
    }
    float peak = 0.0f, all = 0.0f, mine = 0.0f;
    float chosen = 0.0f;             // lane j: exp(l_j - peak) of choice j
    int id = -1;
    for (int j = 0; j < k; ++j) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
            const uint64_t c = (uint64_t)key[i] << 32 | (uint32_t)~(lane + kWave * i);
            best = key[i] > kMinusInf && c > best ? c : best;
        }
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const uint64_t o = __shfl_xor((unsigned long long)best, d);
            best = o > best ? o : best;
        }
        const int e = best ? (int)~(uint32_t)best : -1;
        const float v = key_value((uint32_t)(best >> 32));
        if (j == 0) {
            peak = v;
            if (!renormalize && best) {
#pragma unroll
                for (int i = 0; i < PER_LANE; ++i)
                    if (key[i] > kMinusInf) all += expf(key_value(key[i]) - peak);
            }
        }
        const float p = best ? expf(v - peak) : 0.0f;
        mine += p;
        if (lane == j) { chosen = p; id = e; }
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i)
            if (e == lane + kWave * i) key[i] = 0;
    }
    if (!renormalize) {
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) all += __shfl_xor(all, d);
    }
    if (lane < k) {
        ids[(int64_t)t * k + lane] = id;
        weights[(int64_t)t * k + lane] = id < 0 ? 0.0f : chosen / (renormalize ? mine : all);
    }
}

template <DType DT>
void route(const void* logits, int T, int E, int64_t stride, int k, bool renorm, int* ids,
           float* weights, hipStream_t stream) {
    const unsigned grid = (unsigned)((T + 3) / 4);
    if (E <= 64)
        route_kernel<DT, 1><<<grid, 256, 0, stream>>>(logits, T, E, stride, k, renorm, ids, weights);
    else if (E <= 128)
        route_kernel<DT, 2><<<grid, 256, 0, stream>>>(logits, T, E, stride, k, renorm, ids, weights);
    else if (E <= 256)
        route_kernel<DT, 4><<<grid, 256, 0, stream>>>(logits, T, E, stride, k, renorm, ids, weights);
    else
        route_kernel<DT, 16><<<grid, 256, 0, stream>>>(logits, T, E, stride, k, renorm, ids, weights);
}

// --------------------------------------------------------------------- plan
//
// A stable counting sort with E + 1 buckets (the last takes the ids that name
// no expert).  Blocks own kPerBlock consecutive choices, waves kPerWave of
// them.  With more than one block a first launch counts every block's buckets;
// then each block forms its own bucket starts from all counts, and each wave
// ranks its choices 64 at a time, in order.  Integer sums only: the result
// does not depend on scheduling.

constexpr int kPlanThreads = 512;
constexpr int kPlanWaves = kPlanThreads / kWave;
constexpr int kPerWave = 512;
constexpr int kPerBlock = kPerWave * kPlanWaves;
constexpr int kMaxBuckets = 1025;

__device__ __forceinline__ int bucket(const int* ids, int i, int R, int E) {
    if (i >= R) return -1;
    const int e = ids[i];
    return e >= 0 && e < E ? e : E;
}

__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(const int* ids, int R, int E,
                                                                  int* counts) {
    __shared__ int hist[kMaxBuckets];
    for (int e = threadIdx.x; e <= E; e += kPlanThreads) hist[e] = 0;
    __syncthreads();
    const int base = blockIdx.x * kPerBlock;
    for (int i = threadIdx.x; i < kPerBlock; i += kPlanThreads) {
        const int b = bucket(ids, base + i, R, E);
        if (b >= 0) atomicAdd(&hist[b], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kPlanThreads)
        counts[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const int* ids, int R, int k, int E,
                                                            const int* counts, int blocks,
                                                            int* offsets, int* tokens,
                                                            int* positions) {
    __shared__ int next[kPlanWaves][kMaxBuckets];     // counts, then next free row
    __shared__ int total[kMaxBuckets];
    __shared__ int wave_sum[kPlanWaves];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int buckets = E + 1;
    for (int i = tid; i < kPlanWaves * buckets; i += kPlanThreads) next[i / buckets][i % buckets] = 0;
    __syncthreads();
    const int base = blockIdx.x * kPerBlock + wave * kPerWave;
    for (int i = lane; i < kPerWave; i += kWave) {
        const int b = bucket(ids, base + i, R, E);
        if (b >= 0) atomicAdd(&next[wave][b], 1);
    }
    __syncthreads();
    // Bucket sizes over all blocks, and what earlier blocks and waves hold.
    for (int e = tid; e < buckets; e += kPlanThreads) {
        int before = 0, sum = 0;
        for (int b = 0; b < blocks && counts != nullptr; ++b) {
            const int c = counts[(int64_t)b * buckets + e];
            sum += c;
            if (b < (int)blockIdx.x) before += c;
        }
#pragma unroll
        for (int v = 0; v < kPlanWaves; ++v) {
            const int c = next[v][e];
            next[v][e] = before;
            before += c;
        }
        total[e] = counts != nullptr ? sum : before;
    }
    __syncthreads();
    // Exclusive scan of the bucket sizes, kPlanThreads at a time.
    int carry = 0;
    for (int e0 = 0; e0 < buckets; e0 += kPlanThreads) {
        const int e = e0 + tid;
        const int c = e < buckets ? total[e] : 0;
        int sum = c;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int up = __shfl_up(sum, d);
            if (lane >= d) sum += up;
        }
        if (lane == kWave - 1) wave_sum[wave] = sum;
        __syncthreads();
        int start = carry + sum - c;
        for (int v = 0; v < kPlanWaves; ++v) {
            if (v < wave) start += wave_sum[v];
            carry += wave_sum[v];
        }
        if (e < buckets) {
            if (blockIdx.x == 0) offsets[e] = start;
#pragma unroll
            for (int v = 0; v < kPlanWaves; ++v) next[v][e] += start;
        }
        __syncthreads();
    }
    // Rank in order: lanes of one bucket take consecutive rows.
    for (int i0 = 0; i0 < kPerWave; i0 += kWave) {
        const int i = base + i0 + lane;
        if (base + i0 >= R) break;
        const int b = bucket(ids, i, R, E);
        uint64_t same = __ballot(b >= 0);
        for (int bit = 0; bit < 11; ++bit) {
            const uint64_t set = __ballot((b >> bit) & 1);
            same &= (b >> bit) & 1 ? set : ~set;
        }
        if (b >= 0) {
            const int rank = __popcll(same & ((1ull << lane) - 1));
            const int row = next[wave][b] + rank;
            const bool used = b < E;
            tokens[row] = used ? i / k : -1;
            positions[i] = used ? row : -1;
            if (rank == __popcll(same) - 1) next[wave][b] = row + 1;
        }
        // The wave's next reads of `next` come after this write.
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// ------------------------------------------------------------------ combine

template <typename T, int VEC>
__global__ __launch_bounds__(256) void combine_kernel(const uint16_t* Y, int R, int N,
                                                      const int* positions, const float* weights,
                                                      int T_, int k, uint16_t* out) {
    const int n = (blockIdx.x * 256 + threadIdx.x) * VEC;
    if (n >= N) return;
    for (int t = blockIdx.y; t < T_; t += gridDim.y) {
        float acc[VEC] = {};
        for (int j = 0; j < k; ++j) {
            const int r = positions[(int64_t)t * k + j];
            if (r < 0 || r >= R) continue;
            const float w = weights[(int64_t)t * k + j];
            uint16_t v[VEC];
            __builtin_memcpy(v, __builtin_assume_aligned(Y + (int64_t)r * N + n, 2 * VEC), 2 * VEC);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] = fmaf(w, T::load(v[i]), acc[i]);
        }
        uint16_t o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = T::store(acc[i]);
        __builtin_memcpy(__builtin_assume_aligned(out + (int64_t)t * N + n, 2 * VEC), o, 2 * VEC);
    }
}

template <typename T>
void combine(const uint16_t* Y, int R, int N, const int* positions, const float* weights, int T_,
             int k, uint16_t* out, hipStream_t stream) {
    // Eight columns a thread where every row starts on 16 bytes.
    const bool wide = N % 8 == 0 && ((uintptr_t)Y | (uintptr_t)out) % 16 == 0;
    const int vec = wide ? 8 : 1;
    const dim3 grid((unsigned)((N / vec + 255) / 256), (unsigned)(T_ < 65535 ? T_ : 65535));
    if (wide)
        combine_kernel<T, 8><<<grid, 256, 0, stream>>>(Y, R, N, positions, weights, T_, k, out);
    else
        combine_kernel<T, 1><<<grid, 256, 0, stream>>>(Y, R, N, positions, weights, T_, k, out);
}

}  // namespace

hipError_t launch_route(const void* logits, DType dt, int T, int E, int64_t stride, int k,
                        bool renormalize, int* ids, float* weights, hipStream_t stream) {
    if (dt == kF16) route<kF16>(logits, T, E, stride, k, renormalize, ids, weights, stream);
    else if (dt == kBF16) route<kBF16>(logits, T, E, stride, k, renormalize, ids, weights, stream);
    else route<kF32>(logits, T, E, stride, k, renormalize, ids, weights, stream);
    return hipGetLastError();
}

int64_t plan_blocks(int64_t R) { return (R + kPerBlock - 1) / kPerBlock; }

hipError_t launch_plan(const int* ids, int R, int k, int E, int* offsets, int* tokens,
                       int* positions, int* counts, hipStream_t stream) {
    const int blocks = (int)plan_blocks(R);
    if (blocks > 1) {
        plan_count_kernel<<<blocks, kPlanThreads, 0, stream>>>(ids, R, E, counts);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // R == 0: one block writes the offsets.
    plan_kernel<<<blocks > 0 ? blocks : 1, kPlanThreads, 0, stream>>>(
        ids, R, k, E, blocks > 1 ? counts : nullptr, blocks, offsets, tokens, positions);
    return hipGetLastError();
}

hipError_t launch_combine(const uint16_t* Y, DType dt, int R, int N, const int* positions,
                          const float* weights, int T, int k, uint16_t* out, hipStream_t stream) {
    if (dt == kF16) combine<F16>(Y, R, N, positions, weights, T, k, out, stream);
    else combine<BF16>(Y, R, N, positions, weights, T, k, out, stream);
    return hipGetLastError();
}

}  // namespace mxfp4
