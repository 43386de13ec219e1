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
// The maximum is taken between lanes' registers (DPP) and the expert found by
// comparing with it, without a trip through LDS.  Three tokens: 2.4 us, the latency
// of a launch.  Many tokens are bound by instruction issue: 8191 tokens, 8 of 128
// experts, 8.2 us (with 64-bit shuffles 13.5) are eight waves on every SIMD of 428
// vector instructions each, 14 of the launch's 20 thousand cycles; 2^20 tokens 510 us.

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

// The largest v of the wave: over 2, 4, 8 and 16 lanes of a row, then across rows.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true));    // row_shr:1
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true));    // row_shr:2
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true));    // row_shr:4
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true));    // row_shr:8
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, true));    // row_bcast:15
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, true));    // row_bcast:31
    return __builtin_amdgcn_readlane(v, kWave - 1);
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
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) best = max(best, key[i]);
        best = wave_max(best);
        int e = -1;
        if (best > kMinusInf) {
#pragma unroll
            for (int i = PER_LANE - 1; i >= 0; --i) {
                const uint64_t at = __ballot(key[i] == best);
                e = at ? kWave * i + __builtin_ctzll(at) : e;
            }
        }
        const float v = key_value(best);
        if (j == 0) {
            peak = v;
            if (!renormalize && e >= 0) {
#pragma unroll
                for (int i = 0; i < PER_LANE; ++i)
                    if (key[i] > kMinusInf) all += expf(key_value(key[i]) - peak);
            }
        }
        const float p = e >= 0 ? expf(v - peak) : 0.0f;
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
// Latency bounds it: 18 choices of 64 experts 3.4 us, 65528 of 128 in 5 + 10 us on
// 16 blocks.  Every block reads all counts, so the time grows with the square of the
// blocks in the end: 2^20 choices 27 us, 2^23 217 us, 2^24 (of 64 experts) 690 us.

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
    int mine[kPerBlock / kPlanThreads];
#pragma unroll
    for (int n = 0; n < kPerBlock / kPlanThreads; ++n)
        mine[n] = bucket(ids, base + n * kPlanThreads + threadIdx.x, R, E);
#pragma unroll
    for (int n = 0; n < kPerBlock / kPlanThreads; ++n)
        if (mine[n] >= 0) atomicAdd(&hist[mine[n]], 1);
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
    int mine[kPerWave / kWave];          // the lane's buckets, loaded together
#pragma unroll
    for (int n = 0; n < kPerWave / kWave; ++n) mine[n] = bucket(ids, base + n * kWave + lane, R, E);
#pragma unroll
    for (int n = 0; n < kPerWave / kWave; ++n)
        if (mine[n] >= 0) atomicAdd(&next[wave][mine[n]], 1);
    __syncthreads();
    // Bucket sizes over all blocks, and what earlier blocks and waves hold.
    for (int e = tid; e < buckets; e += kPlanThreads) {
        int before = 0, sum = 0;
#pragma unroll 8
        for (int b = 0; b < (counts != nullptr ? blocks : 0); ++b) {
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
    const int bits = 32 - __builtin_clz(E);
#pragma unroll
    for (int n = 0; n < kPerWave / kWave; ++n) {
        const int i = base + n * kWave + lane, b = mine[n];
        uint64_t same = __ballot(b >= 0);
        if (same == 0) break;
        for (int bit = 0; bit < bits; ++bit) {
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
//
// Memory bound: every chosen row is read once, eight columns a thread (300 tokens,
// 8 rows of 4096 each, 22 MB: 6.5-7 us).  Rows come in the result's type or, at
// twice the traffic, in fp32: then out is rounded once, where roundings of the rows
// make its error 1.4 times as large (bf16 2.35e-3 of the norm against 1.66e-3).

struct F32 {
    typedef float type;
    static __device__ __forceinline__ float load(float f) { return f; }
};

template <typename T, typename ROW, int VEC>
__global__ __launch_bounds__(256) void combine_kernel(const typename ROW::type* Y, int R, int N,
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
            typename ROW::type v[VEC];
            constexpr int kAlign = sizeof(v) < 16 ? sizeof(v) : 16;
            __builtin_memcpy(v, __builtin_assume_aligned(Y + (int64_t)r * N + n, kAlign), sizeof(v));
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] = fmaf(w, ROW::load(v[i]), acc[i]);
        }
        uint16_t o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = T::store(acc[i]);
        __builtin_memcpy(__builtin_assume_aligned(out + (int64_t)t * N + n, 2 * VEC), o, 2 * VEC);
    }
}

template <typename T, typename ROW>
void combine(const void* Y_, int R, int N, const int* positions, const float* weights, int T_,
             int k, uint16_t* out, hipStream_t stream) {
    const auto* Y = (const typename ROW::type*)Y_;
    // Eight columns a thread where every row starts on 16 bytes.
    const bool wide = N % 8 == 0 && ((uintptr_t)Y | (uintptr_t)out) % 16 == 0;
    const int vec = wide ? 8 : 1;
    const dim3 grid((unsigned)((N / vec + 255) / 256), (unsigned)(T_ < 65535 ? T_ : 65535));
    if (wide)
        combine_kernel<T, ROW, 8><<<grid, 256, 0, stream>>>(Y, R, N, positions, weights, T_, k, out);
    else
        combine_kernel<T, ROW, 1><<<grid, 256, 0, stream>>>(Y, R, N, positions, weights, T_, k, out);
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

hipError_t launch_combine(const void* Y, bool rows32, DType dt, int R, int N, const int* positions,
                          const float* weights, int T, int k, uint16_t* out, hipStream_t stream) {
    if (dt == kF16 && rows32) combine<F16, F32>(Y, R, N, positions, weights, T, k, out, stream);
    else if (dt == kF16) combine<F16, F16>(Y, R, N, positions, weights, T, k, out, stream);
    else if (rows32) combine<BF16, F32>(Y, R, N, positions, weights, T, k, out, stream);
    else combine<BF16, BF16>(Y, R, N, positions, weights, T, k, out, stream);
    return hipGetLastError();
}

}  // namespace mxfp4
