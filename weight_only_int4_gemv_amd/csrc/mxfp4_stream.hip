// mxfp4_stream.hip — weight-only MXFP4 product for up to 16 rows per weight
// matrix (decode, experts with a few rows each).
//
// What bounds it is reading the weights once: 17/32 byte per weight.  A block
// owns 16 J weight rows (J tiles; with SwiGLU J / 2 tiles of gate rows, then
// their up rows) and 16 rows of X; its eight waves split K in chunks of 128
// columns, each wave multiplies on the matrix cores, and the partial tiles are
// added through LDS in wave order.
//
// Matrix-core layout (16x16x32): A = weights, lane l holds row l % 16; B = X,
// lane l holds column (row of X) l % 16; lane group g = l / 16 supplies eight
// k values of each.  The sum over k may run in any order as long as A and B
// agree, so group g takes the whole block g of the chunk: one 16-byte load of
// codes, one scale byte, and MFMA i multiplies its columns 8i .. 8i+7.
//
// A wave loads a chunk and multiplies it; other waves of the CU cover its wait
// (holding a second chunk ahead costs as many waves as it gains: 1 x 4096 x
// 14336 12.3 us against 12.7, 8 x 28672 x 8192 42.3 against 41.1).
#include "mxfp4_device.h"
#include "mxfp4_launch.h"

namespace mxfp4 {
namespace {

constexpr int kWaves = 8;
constexpr int kChunkBlocks = 4;  // blocks of a row a wave takes at a time
constexpr int kTile = 16;

template <typename T, int J>
__global__ __launch_bounds__(kWaves* kWave) void stream_kernel(LinearArgs a) {
    constexpr bool kIsF16 = __is_same(T, F16);
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int slot = blockIdx.z * gridDim.y + blockIdx.y, nb = blockIdx.x;

    Tile t;
    if (a.offsets != nullptr) {
        t = find_tile(a.offsets, a.E, a.R, kTile, slot);
    } else {
        t.expert = 0;
        t.row0 = slot * kTile;
        t.rows = min(kTile, a.R - t.row0);
    }
    if (t.rows <= 0) return;

    // Weight rows of the tiles; rows past the end read the last row and are not
    // stored.
    const int F = a.swiglu ? a.N / 2 : a.N;                 // columns of Y
    const int per = a.swiglu ? J * kTile / 2 : J * kTile;   // of this block
    const int col0 = nb * per;
    const int KB = a.K / kBlock;
    float4_t acc[J] = {};

    if (t.expert >= 0) {
        const int64_t expert_row = (int64_t)t.expert * a.N;
        // Weight row r of tile j, and the row of X (-1: none), r = lane % 16.
        auto weight_row = [&](int j, int r) {
            // SwiGLU: the gate tiles, then their up tiles.
            const bool up = a.swiglu && j >= J / 2;
            const int col = min(col0 + kTile * (up ? j - J / 2 : j) + r, F - 1);
            return expert_row + col + (up ? F : 0);
        };
        auto x_row = [&](int r) {
            if (r >= t.rows) return -1;
            const int src = a.tokens ? a.tokens[t.row0 + r] : t.row0 + r;
            return src >= 0 && src < a.x_rows ? src : -1;
        };
        const uint8_t *wc[J], *ws[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t n = weight_row(j, lane & 15);
            wc[j] = a.codes + n * (a.K / 2);
            ws[j] = a.scales + n * KB;
        }
        const int src = x_row(lane & 15);
        const bool live = src >= 0;
        const uint16_t* xr = a.X + (live ? src : 0) * a.x_stride;

        uint4_t w[J], x[4];
        uint32_t sb[J];
        auto load = [&](int c) {
            const int kb = c * kChunkBlocks + (lane >> 4);
            const bool in = kb < KB;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                w[j] = (uint4_t){0, 0, 0, 0};
                sb[j] = 127;
                if (in) {
                    w[j] = *(const uint4_t*)(wc[j] + (int64_t)kb * 16);
                    sb[j] = ws[j][kb];
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = (uint4_t){0, 0, 0, 0};
                if (in && live) x[i] = *(const uint4_t*)(xr + (int64_t)kb * kBlock + 8 * i);
            }
        };
        auto multiply = [&]() {
            float s[J];
            bool ok = true;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                s[j] = scale_value(sb[j]);
                ok = ok && f16_scale_ok(sb[j]);
            }
            if (kIsF16 && __any(!ok)) {
                // Weights outside fp16's range: exact in bf16, X as two bf16.
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    bf168_t hi, lo;
                    split_bf16(__builtin_bit_cast(half8_t, x[i]), hi, lo);
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const bf168_t wv = values8(w[j][i], s[j], BF16());
                        acc[j] = BF16::mfma16(wv, hi, acc[j]);
                        acc[j] = BF16::mfma16(wv, lo, acc[j]);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        acc[j] = T::mfma16(values8(w[j][i], s[j], T()),
                                           __builtin_bit_cast(typename T::vec8, x[i]), acc[j]);
            }
        };
        const int chunks = (KB + kChunkBlocks - 1) / kChunkBlocks;
        uint64_t far = 0;               // lanes that met a scale bf16 does not hold
        load(wave);
        for (int c = wave; c < chunks; c += kWaves) {
#pragma unroll
            for (int j = 0; j < J; ++j) far |= __ballot(sb[j] >= kFarScale);
            multiply();
            if (c + kWaves < chunks) load(c + kWaves);
        }
        if (far != 0) {
            // Weights that bf16 does not hold: the chunks again, in quarters (a test and
            // branch in the loop costs every call 6 %: 1 x 14336 x 4096 11.15 us so, 11.8
            // with one).  The rows are found anew, for no register to stay taken above.
            int l = lane;
            asm volatile("" : "+v"(l));
            const int x_src = x_row(l & 15);
#pragma unroll
            for (int j = 0; j < J; ++j) acc[j] = (float4_t){0, 0, 0, 0};
#pragma unroll 1
            for (int i = 4 * wave; i < 4 * chunks; i += i % 4 == 3 ? 4 * kWaves - 3 : 1) {
                const int kb = i / 4 * kChunkBlocks + (l >> 4);
                const bool in = kb < KB;
                uint4_t xv = {0, 0, 0, 0};
                if (in && x_src >= 0)
                    xv = *(const uint4_t*)(a.X + x_src * a.x_stride + (int64_t)kb * kBlock + i % 4 * 8);
                bf168_t hi = __builtin_bit_cast(bf168_t, xv), lo;
                if constexpr (kIsF16) split_bf16(__builtin_bit_cast(half8_t, xv), hi, lo);
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int64_t n = weight_row(j, l & 15);
                    uint32_t word = 0, byte = 127;
                    if (in) {
                        word = *(const uint32_t*)(a.codes + n * (a.K / 2) + kb * 16 + i % 4 * 4);
                        byte = a.scales[n * KB + kb];
                    }
                    const bf168_t q = quarter8(word, byte);
                    acc[j] = BF16::mfma16(q, hi, acc[j]);
                    if constexpr (kIsF16) acc[j] = BF16::mfma16(q, lo, acc[j]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j) acc[j] *= 4.0f;
        }
    }

    // Partial tiles through LDS: [wave][j][row of X][weight row].
    __shared__ float part[kWaves][J][kTile][kTile];
#pragma unroll
    for (int j = 0; j < J; ++j)
        *(float4_t*)&part[wave][j][lane & 15][(lane >> 4) * 4] = acc[j];
    __syncthreads();
    for (int i = threadIdx.x; i < t.rows * per; i += kWaves * kWave) {
        const int r = i / per, n = i % per;
        if (col0 + n >= F) continue;
        float h[2] = {0.0f, 0.0f};
        const int j0 = n / kTile;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            h[0] += part[v][j0][r][n % kTile];
            if (J > 1 && a.swiglu) h[1] += part[v][j0 + J / 2][r][n % kTile];
        }
        const float y = a.swiglu ? silu(h[0]) * h[1] : h[0];
        const int64_t at = (int64_t)(t.row0 + r) * F + col0 + n;
        if (a.part != nullptr) a.part[at] = y;
        else a.Y[at] = T::store(y);
    }
}

template <int J>
hipError_t launch(const LinearArgs& a, DType dt, hipStream_t stream) {
    const int F = a.swiglu ? a.N / 2 : a.N, per = a.swiglu ? J * kTile / 2 : J * kTile;
    const int64_t slots = a.offsets ? tile_slots(a.R, a.E, kTile) : (a.R + kTile - 1) / kTile;
    const dim3 grid = slot_grid((F + per - 1) / per, slots);
    if (dt == kF16) stream_kernel<F16, J><<<grid, kWaves * kWave, 0, stream>>>(a);
    else stream_kernel<BF16, J><<<grid, kWaves * kWave, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_stream(const LinearArgs& a, DType dt, hipStream_t stream) {
    // Four tiles a block read X a quarter as often; one (with SwiGLU two) gives
    // more blocks, and is faster where four leave CUs without one (us, one / two /
    // four tiles): 8 x 28672 x 8192 59.9 / 48.6 / 41.1, 8 x 14336 x 4096 18.9 /
    // 14.7 / 13.5, 8 x 4096 x 14336 17.3 / 23.0 / 38.3, 1 x 4096 x 4096 5.4 / 7.4
    // / 11.8; four tokens, 8 of 64 experts, 4096 x 1792 39.5 / 37.0 / 31.0.
    const int64_t slots = a.offsets ? tile_slots(a.R, a.E, kTile) : (a.R + kTile - 1) / kTile;
    if (a.N / (4 * kTile) * slots >= 192) return launch<4>(a, dt, stream);
    return a.swiglu ? launch<2>(a, dt, stream) : launch<1>(a, dt, stream);
}

}  // namespace mxfp4
