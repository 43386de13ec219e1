// mxfp4_stream.hip — weight-only MXFP4 product for few rows per weight matrix
// (decode, small batches, experts with a few rows each).
//
// What bounds it is reading the weights once: 17/32 byte per weight.  A block
// owns 32 weight rows (two tiles of 16; with SwiGLU 16 gate rows and their 16
// up rows) and 16 MT rows of X; its eight waves split K in chunks of 128
// columns, each wave multiplies on the matrix cores, and the partial tiles are
// added through LDS in wave order.
//
// Matrix-core layout (16x16x32): A = weights, lane l holds row l % 16; B = X,
// lane l holds column (row of X) l % 16; lane group g = l / 16 supplies eight
// k values of each.  The sum over k may run in any order as long as A and B
// agree, so group g takes the whole block g of the chunk: one 16-byte load of
// codes, one scale byte, and MFMA i multiplies its columns 8i .. 8i+7.
#include "mxfp4_device.h"
#include "mxfp4_launch.h"

namespace mxfp4 {
namespace {

constexpr int kWaves = 8;
constexpr int kChunk = 128;      // columns a wave takes at a time
constexpr int kTile = 16;

template <typename T, int MT>
__global__ __launch_bounds__(kWaves* kWave) void stream_kernel(LinearArgs a) {
    constexpr bool kIsF16 = __is_same(T, F16);
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int slot = blockIdx.z * gridDim.y + blockIdx.y, nb = blockIdx.x;

    Tile t;
    if (a.offsets != nullptr) {
        t = find_tile(a.offsets, a.E, a.R, kTile * MT, slot);
    } else {
        t.expert = 0;
        t.row0 = slot * kTile * MT;
        t.rows = min(kTile * MT, a.R - t.row0);
    }
    if (t.rows <= 0) return;

    // Weight rows of the two tiles; rows past the end read the last row and
    // are not stored.
    const int F = a.swiglu ? a.N / 2 : a.N;                 // columns of Y
    const int col0 = nb * (a.swiglu ? kTile : 2 * kTile);   // first of this block
    const int KB = a.K / kBlock;
    float4_t acc[2][MT] = {};

    if (t.expert >= 0) {
        const uint8_t* codes = a.codes + (int64_t)t.expert * a.N * (a.K / 2);
        const uint8_t* scales = a.scales + (int64_t)t.expert * a.N * KB;
        const uint8_t *wc[2], *ws[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t n = a.swiglu ? (int64_t)j * F + min(col0 + (lane & 15), F - 1)
                                       : min(col0 + kTile * j + (lane & 15), F - 1);
            wc[j] = codes + n * (a.K / 2);
            ws[j] = scales + n * KB;
        }
        const uint16_t* xr[MT];
        bool live[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int i = kTile * m + (lane & 15);
            int src = -1;
            if (i < t.rows) src = a.tokens ? a.tokens[t.row0 + i] : t.row0 + i;
            live[m] = src >= 0 && src < a.x_rows;
            xr[m] = a.X + (live[m] ? src : 0) * a.x_stride;
        }
        for (int c = wave * kChunk; c < a.K; c += kWaves * kChunk) {
            const int kb = c / kBlock + (lane >> 4);
            const bool in = kb < KB;
            uint4_t w[2] = {};
            uint32_t sb[2] = {127, 127};
            uint4_t x[MT][4] = {};
            if (in) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    w[j] = *(const uint4_t*)(wc[j] + (int64_t)kb * 16);
                    sb[j] = ws[j][kb];
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (in && live[m]) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[m][i] = *(const uint4_t*)(xr[m] + (int64_t)kb * kBlock + 8 * i);
                }
            }
            float s[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) s[j] = scale_value(sb[j]);
            if (kIsF16 && __any(!(f16_scale_ok(sb[0]) && f16_scale_ok(sb[1])))) {
                // Weights outside fp16's range: exact in bf16, X as two bf16.
#pragma unroll
                for (int m = 0; m < MT; ++m) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        bf168_t hi, lo;
                        split_bf16(__builtin_bit_cast(half8_t, x[m][i]), hi, lo);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const bf168_t wv = values8(w[j][i], s[j], BF16());
                            acc[j][m] = BF16::mfma16(wv, hi, acc[j][m]);
                            acc[j][m] = BF16::mfma16(wv, lo, acc[j][m]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const typename T::vec8 wv = values8(w[j][i], s[j], T());
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            acc[j][m] = T::mfma16(
                                wv, __builtin_bit_cast(typename T::vec8, x[m][i]), acc[j][m]);
                    }
                }
            }
        }
    }

    // Partial tiles through LDS: [wave][m tile][j][row of X][weight row].
    __shared__ float part[kWaves][MT][2][kTile][kTile];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *(float4_t*)&part[wave][m][j][lane & 15][(lane >> 4) * 4] = acc[j][m];
    __syncthreads();
    const int per_row = a.swiglu ? kTile : 2 * kTile;
    for (int i = threadIdx.x; i < t.rows * per_row; i += kWaves * kWave) {
        const int r = i / per_row, n = i % per_row;
        if (col0 + n >= F) continue;
        float h[2] = {0.0f, 0.0f};
        const int j0 = a.swiglu ? 0 : n / kTile;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            h[0] += part[v][r / kTile][j0][r % kTile][n % kTile];
            if (a.swiglu) h[1] += part[v][r / kTile][1][r % kTile][n % kTile];
        }
        const float y = a.swiglu ? silu(h[0]) * h[1] : h[0];
        a.Y[(int64_t)(t.row0 + r) * F + col0 + n] = T::store(y);
    }
}

template <typename T, int MT>
hipError_t launch(const LinearArgs& a, hipStream_t stream) {
    const int F = a.swiglu ? a.N / 2 : a.N;
    const int per = a.swiglu ? kTile : 2 * kTile;
    const int nblocks = (F + per - 1) / per;
    const int64_t slots = a.offsets ? tile_slots(a.R, a.E, kTile * MT)
                                    : (a.R + kTile * MT - 1) / (kTile * MT);
    stream_kernel<T, MT><<<slot_grid(nblocks, slots), kWaves * kWave, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_stream(const LinearArgs& a, DType dt, hipStream_t stream) {
    const int64_t rows = a.offsets ? a.R / a.E : a.R;      // per expert, on average
    if (dt == kF16) {
        if (rows <= 16) return launch<F16, 1>(a, stream);
        if (rows <= 32) return launch<F16, 2>(a, stream);
        return launch<F16, 4>(a, stream);
    }
    if (rows <= 16) return launch<BF16, 1>(a, stream);
    if (rows <= 32) return launch<BF16, 2>(a, stream);
    return launch<BF16, 4>(a, stream);
}

}  // namespace mxfp4
