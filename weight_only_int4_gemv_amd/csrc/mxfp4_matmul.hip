// mxfp4_matmul.hip — product of two MXFP4 matrices on the block-scaled matrix
// instructions.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 with both operands fp4: lane l holds row
// l % 32 and the block (32 columns, 16 bytes) l / 32 of each operand, and one
// scale byte per operand and block; products and scales are exact, sums fp32.
#include "mxfp4_device.h"
#include "mxfp4_launch.h"

namespace mxfp4 {
namespace {

struct MatmulArgs {
    const uint8_t *ac, *as, *bc, *bs;
    void* Y;
    int M, N, K;
};

__device__ __forceinline__ float16_t mfma_fp4(uint4_t a, uint4_t b, float16_t c, int sa, int sb) {
    const int8_t_ av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const int8_t_ bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, 0, sa, 0, sb);
}

template <DType DT>
__device__ __forceinline__ void store(void* Y, int64_t i, float v) {
    if constexpr (DT == kF32) ((float*)Y)[i] = v;
    else if constexpr (DT == kBF16) ((uint16_t*)Y)[i] = BF16::store(v);
    else ((uint16_t*)Y)[i] = F16::store(v);
}

// Block of 64 x 64 outputs, four waves of 32 x 32, operands from L2.
template <DType DT>
__global__ __launch_bounds__(256) void matmul_kernel(MatmulArgs a) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int m0 = (blockIdx.z * gridDim.y + blockIdx.y) * 64 + (wave & 1) * 32;
    const int n0 = blockIdx.x * 64 + (wave >> 1) * 32;
    if (m0 >= a.M || n0 >= a.N) return;
    const int KB = a.K / kBlock;
    const int64_t m = min(m0 + (lane & 31), a.M - 1), n = min(n0 + (lane & 31), a.N - 1);
    const uint8_t *ac = a.ac + m * (a.K / 2), *bc = a.bc + n * (a.K / 2);
    const uint8_t *as = a.as + m * KB, *bs = a.bs + n * KB;
    float16_t acc = {};
    for (int kb = lane >> 5; kb < KB + (lane >> 5); kb += 2) {
        uint4_t x = {}, w = {};
        int sx = 127, sw = 127;
        if (kb < KB) {
            x = *(const uint4_t*)(ac + (int64_t)kb * 16);
            w = *(const uint4_t*)(bc + (int64_t)kb * 16);
            sx = as[kb];
            sw = bs[kb];
        }
        acc = mfma_fp4(x, w, acc, sx, sw);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = m0 + (i & 3) + 8 * (i >> 2) + 4 * (lane >> 5);
        const int c = n0 + (lane & 31);
        if (r < a.M && c < a.N) store<DT>(a.Y, (int64_t)r * a.N + c, acc[i]);
    }
}

}  // namespace

hipError_t launch_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                         const uint8_t* b_codes, const uint8_t* b_scales, int64_t N, int64_t K,
                         void* Y, DType dt, hipStream_t stream) {
    const MatmulArgs a{a_codes, a_scales, b_codes, b_scales, Y, (int)M, (int)N, (int)K};
    const dim3 grid = slot_grid((int)((N + 63) / 64), (M + 63) / 64);
    if (dt == kF16)
        matmul_kernel<kF16><<<grid, 256, 0, stream>>>(a);
    else if (dt == kBF16)
        matmul_kernel<kBF16><<<grid, 256, 0, stream>>>(a);
    else
        matmul_kernel<kF32><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace mxfp4
