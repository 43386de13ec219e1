// mxfp4_gemv.hip — products with an epilogue for one row (decode): each weight row read
// once, along the row.
//
// A wave takes four weight rows (with SwiGLU two gate rows and their up rows), a lane whole blocks
// of 32 columns: 16 bytes of codes and a scale byte, 1 KB and 64 bytes of a row at a time.  A
// block's sum is formed in fp32 of its codes times 2^-8 (no sum of 32 overflows) and then
// multiplied by its scale and 2^8, so that no scale and no x needs a special path.  X stands in
// LDS as fp32.  Waves that share rows split K in chunks of 64 blocks.
//
// What bounds it is reading the weights: one row of 4096 x 14336 takes 10.4 us (3.0 TB/s from HBM,
// 12 weights in turn), of 14336 x 4096 10.5, of 28672 x 8192 29.5 (4.2 TB/s); the 16-row tiles of the
// matrix cores, 64 bytes from each of 16 rows at a time, 16.5, 12.4 and 39.8.  Below 2^24 weights
// (4096 x 4096 5.9 against 6.2 us, 1000 x 2048 4.5 against 3.7) the X in LDS costs more than it gains.
// The weight-only INT4 row kernel reads as many bytes of 4096 x 14336 in 7.9 us.
#include "mxfp4_act.h"

namespace mxfp4 {
namespace {

constexpr int kWaves = 8;
constexpr int kRowsOfWave = 4;
// Bytes of X in LDS: two blocks a CU hold twice as many, and no longer K was measured.  One row of
// 3584 x 18944 takes 20.6 us on the 16-row tiles, of 8192 x 28672 45.7.
constexpr int kMaxX = 60000;

template <typename T>
__global__ __launch_bounds__(kWaves* kWave, 4) void gemv_kernel(LinearArgs a, int split) {
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const bool swiglu = a.act == kSwiglu;
    const int F = swiglu ? a.N / 2 : a.N, per = swiglu ? kRowsOfWave / 2 : kRowsOfWave;
    const int groups = kWaves / split;                      // row groups of the block
    const int group = wave / split, slice = wave % split;
    const int col0 = (blockIdx.x * groups + group) * per;   // first column of Y
    const int KB = a.K / kBlock, chunks = (KB + kWave - 1) / kWave;

    // Row i of the wave; rows past the end read the last and are not stored.
    const uint8_t *codes[kRowsOfWave], *scales[kRowsOfWave];
#pragma unroll
    for (int i = 0; i < kRowsOfWave; ++i) {
        const int64_t n = min(col0 + i % per, F - 1) + (i >= per ? F : 0);
        codes[i] = a.codes + n * (a.K / 2);
        scales[i] = a.scales + n * KB;
    }
    uint4_t w[kRowsOfWave];
    uint32_t sb[kRowsOfWave];
    auto load = [&](int c) {
        const int kb = c * kWave + lane;
#pragma unroll
        for (int i = 0; i < kRowsOfWave; ++i) {
            w[i] = (uint4_t){0, 0, 0, 0};
            sb[i] = 127;
            if (kb < KB) {
                w[i] = __builtin_nontemporal_load((const uint4_t*)codes[i] + kb);
                sb[i] = scales[i][kb];
            }
        }
    };
    if (slice < chunks) load(slice);
    // X as [row][block][32], 16-byte piece j of block b at j ^ (b / 2 % 8): 16 lanes that read a
    // piece of neighbouring blocks meet different banks.
    for (int p = threadIdx.x; p < KB * 4; p += kWaves * kWave) {
        const int b = p / 4;
        float v[8];
        load_columns<T, 8>(a.X + p * 8, v);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            ((float4_t*)lds)[b * 8 + ((p % 4 * 2 + h) ^ (b >> 1 & 7))] =
                (float4_t){v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    }
    __syncthreads();

    float acc[kRowsOfWave] = {};
    for (int c = slice; c < chunks; c += split) {
        uint4_t v[kRowsOfWave];
        float s[kRowsOfWave], sum[kRowsOfWave] = {};
#pragma unroll
        for (int i = 0; i < kRowsOfWave; ++i) v[i] = w[i], s[i] = scale_value(sb[i]);
        if (c + split < chunks) load(c + split);
        const int b = min(c * kWave + lane, KB - 1);        // past K the codes are 0
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float4_t x[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) x[h] = ((const float4_t*)lds)[b * 8 + ((2 * j + h) ^ (b >> 1 & 7))];
#pragma unroll
            for (int i = 0; i < kRowsOfWave; ++i) {
                const float2_t e[4] = {
                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[i][j], 0.00390625f, 0),
                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[i][j], 0.00390625f, 1),
                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[i][j], 0.00390625f, 2),
                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[i][j], 0.00390625f, 3)};
#pragma unroll
                for (int q = 0; q < 8; ++q) sum[i] = fmaf(e[q / 2][q % 2], x[q / 4][q % 4], sum[i]);
            }
        }
        // A lane past K meets the last block's X: an infinity there must not.
        if (c * kWave + lane < KB) {
#pragma unroll
            for (int i = 0; i < kRowsOfWave; ++i) acc[i] = fmaf(sum[i] * s[i], 256.0f, acc[i]);
        }
    }

    // Over the lanes, then the slices in order.
    __shared__ float part[kWaves][kRowsOfWave];
#pragma unroll
    for (int i = 0; i < kRowsOfWave; ++i) {
        float v = acc[i];
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
        if (lane == 0) part[wave][i] = v;
    }
    __syncthreads();
    if ((int)threadIdx.x >= groups * per) return;
    const int r = threadIdx.x % per, at = threadIdx.x / per;
    const int col = (blockIdx.x * groups + at) * per + r;
    if (col >= F) return;
    float h[1] = {0.0f}, up[1] = {0.0f};
    for (int v = 0; v < split; ++v) {
        h[0] += part[at * split + v][r];
        if (swiglu) up[0] += part[at * split + v][r + per];
    }
    finish_columns<T, 1>(a, load_bias<T, 1>(a, 0, col), 0, col, h, up);
}

template <typename T>
void launch(const LinearArgs& a, hipStream_t stream) {
    const int F = a.act == kSwiglu ? a.N / 2 : a.N, per = a.act == kSwiglu ? 2 : 4;
    const int64_t waves = (F + per - 1) / per, chunks = (a.K / kBlock + kWave - 1) / kWave;
    // Waves on the same rows, up to a block of eight a CU: 4096 x 14336 13.0 / 10.4 / 11.0 / 14.5 us
    // with 1 / 2 / 4 / 8 of them, 14336 x 4096 10.5 / 13.2 / 17.9 / 26.4.
    int split = 1;
    while (split < kWaves && 2 * split <= chunks && 2 * split * waves <= 256 * kWaves) split *= 2;
    const int groups = kWaves / split;
    const unsigned grid = (unsigned)((waves + groups - 1) / groups);
    const size_t bytes = (size_t)a.K * sizeof(float);
    gemv_kernel<T><<<grid, kWaves * kWave, bytes, stream>>>(a, split);
}

}  // namespace

bool gemv_fits(int64_t R, int64_t N, int64_t K) {
    return R == 1 && K * 4 <= kMaxX && N * K >= 1 << 24;
}

hipError_t launch_gemv(const LinearArgs& a, DType dt, hipStream_t stream) {
    if (dt == kF16) launch<F16>(a, stream);
    else launch<BF16>(a, stream);
    return hipGetLastError();
}

}  // namespace mxfp4
