// mxfp4_grad.hip — the gradient through the weight-only product, dX = dY W: 16-bit rows times
// untransposed MXFP4 weights, summed over the weight rows.
//
// Codes lie along K, the matrix instructions sum along N.  A lane loads one word or more of the
// same columns from eight weight rows, converts them (scales are those of a row and block) and
// pairs neighbouring rows with one byte permutation per pair; the lane then holds, for each of
// its columns, the eight weight rows that are its operand of a 16x16x32 instruction.  A wave's
// instructions j = 0, 1, ... take column j of every lane, so that a lane ends with neighbouring
// columns of dX: 16 lanes of 16 columns are 256 columns, and the results need no turning.
#include "mxfp4_device.h"
#include "mxfp4_launch.h"

namespace mxfp4 {
namespace {

constexpr int kTile = 16;               // rows of a matrix instruction
constexpr int kStepRows = 32;           // weight rows of one
constexpr int kWaves = 8;
constexpr int kCols = 256;              // columns of a block
constexpr int kLaneCols = kCols / kTile;
constexpr int kWords = kLaneCols / 8;

// Columns 2b and 2b + 1 of weight rows 2i and 2i + 1 as pairs along the rows.
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// Eight columns of eight weight rows (one word each) as operands: out[j] holds column j.
template <typename T, class CONVERT>
__device__ __forceinline__ void turn8(const uint32_t (&w)[8], CONVERT convert, uint4_t (&out)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4_t a = __builtin_bit_cast(uint4_t, convert(w[2 * i], 2 * i));
        const uint4_t b = __builtin_bit_cast(uint4_t, convert(w[2 * i + 1], 2 * i + 1));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            out[2 * c][i] = low_halves(a[c], b[c]);
            out[2 * c + 1][i] = high_halves(a[c], b[c]);
        }
    }
}

// The lane's eight weight rows n0 .. n0 + 7 of one row of dY; rows past N count 0.
__device__ __forceinline__ uint4_t load_dy(const uint16_t* row, int n0, int N, bool wide) {
    uint4_t v = {0, 0, 0, 0};
    if (row == nullptr || n0 >= N) return v;
    if (wide && n0 + 8 <= N) return *(const uint4_t*)(row + n0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (n0 + i < N) v[i / 2] |= (uint32_t)row[n0 + i] << (16 * (i & 1));
    return v;
}

template <typename T>
__global__ __launch_bounds__(kWaves* kWave) void stream_grad_kernel(GradArgs a) {
    constexpr bool kIsF16 = __is_same(T, F16);
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int r = lane & 15, g = lane >> 4;
    const int slot = blockIdx.z * gridDim.y + blockIdx.y;
    const int kblocks = (a.K + kCols - 1) / kCols;
    const int slice = blockIdx.x / kblocks, k0 = (blockIdx.x - slice * kblocks) * kCols;
    Tile t;
    if (a.offsets != nullptr) {
        t = find_tile(a.offsets, a.E, a.R, kTile, slot);
    } else {
        t.expert = 0;
        t.row0 = slot * kTile;
        t.rows = min(kTile, a.R - t.row0);
    }
    if (t.rows <= 0) return;

    float4_t acc[kWords][8] = {};
    const int KB = a.K / kBlock, row_bytes = a.K / 2;
    const int col = k0 + r * kLaneCols;
    const bool live = col < a.K;                        // all of a lane's columns or none
    const int total = (a.N + kStepRows - 1) / kStepRows;
    const int first = slice * a.steps, last = min(first + a.steps, total);
    if (t.expert >= 0) {
        const uint8_t* codes = a.codes + (int64_t)t.expert * a.N * row_bytes + (live ? col / 2 : 0);
        const uint8_t* scales = a.scales + (int64_t)t.expert * a.N * KB + (live ? col / kBlock : 0);
        const uint16_t* dy = r < t.rows ? a.dY + (t.row0 + r) * a.y_stride : nullptr;
        const bool wide = (uintptr_t)a.dY % 16 == 0 && (a.y_stride % 8 == 0 || a.R == 1);
        uint32_t w[kWords][8], sb[8];
        uint4_t x;
        auto load = [&](int s) {
            const int n0 = s * kStepRows + 8 * g;
            x = load_dy(dy, n0, a.N, wide);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // Rows past N: the last row's codes with scale 1 meet zeros.
                const int n = min(n0 + i, a.N - 1);
                const uint8_t* p = codes + (int64_t)n * row_bytes;
                static_assert(kWords == 2, "one load a row");
                const uint2_t v = *(const uint2_t*)p;
                w[0][i] = v[0], w[1][i] = v[1];
                sb[i] = n0 + i < a.N ? scales[(int64_t)n * KB] : 127;
            }
        };
        // The sums of one step: hi and lo are dY's halves where it is split.
        auto multiply = [&](auto type, auto convert, uint4_t hi, uint4_t lo, bool two) {
            typedef decltype(type) M;
            typedef typename M::vec8 vec8;
#pragma unroll
            for (int q = 0; q < kWords; ++q) {
                uint4_t f[8];
                turn8<M>(w[q], convert, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc[q][j] = M::mfma16(__builtin_bit_cast(vec8, f[j]),
                                          __builtin_bit_cast(vec8, hi), acc[q][j]);
                    if (two)
                        acc[q][j] = M::mfma16(__builtin_bit_cast(vec8, f[j]),
                                              __builtin_bit_cast(vec8, lo), acc[q][j]);
                }
            }
        };
        auto split = [&](uint4_t& hi, uint4_t& lo) {
            bf168_t h, l;
            split_bf16(__builtin_bit_cast(half8_t, x), h, l);
            hi = __builtin_bit_cast(uint4_t, h), lo = __builtin_bit_cast(uint4_t, l);
        };
        bool far = false;
        for (int s = first + wave; s < last; s += kWaves) {
            load(s);
            float sc[8];
            bool ok = true;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sc[i] = scale_value(sb[i]);
                ok = ok && f16_scale_ok(sb[i]);
                far = far || sb[i] >= kFarScale;
            }
            if (kIsF16 && __any(!ok)) {
                // Weights outside fp16's range: exact in bf16, dY as two bf16.
                uint4_t hi, lo;
                split(hi, lo);
                multiply(BF16(), [&](uint32_t v, int i) { return values8(v, sc[i], BF16()); }, hi,
                         lo, true);
            } else {
                multiply(T(), [&](uint32_t v, int i) { return values8(v, sc[i], T()); }, x, x,
                         false);
            }
        }
        if (__any(far)) {
            // Weights that bf16 does not hold: the steps again, in quarters.
#pragma unroll
            for (int q = 0; q < kWords; ++q)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[q][j] = (float4_t){0, 0, 0, 0};
#pragma unroll 1
            for (int s = first + wave; s < last; s += kWaves) {
                load(s);
                uint4_t hi = x, lo = x;
                if constexpr (kIsF16) split(hi, lo);
                multiply(BF16(), [&](uint32_t v, int i) { return quarter8(v, sb[i]); }, hi, lo,
                         kIsF16);
            }
#pragma unroll
            for (int q = 0; q < kWords; ++q)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[q][j] *= 4.0f;
        }
    }

    // The waves' sums through LDS, in wave order within each half.  Lane l holds row l % 16 of
    // dX; register i of acc[q][j] the column 16 (4 g + i) + 8 q + j.
    constexpr int kHalf = kWaves / 2, kPitch = kCols + 4;
    __shared__ __align__(16) float part[kHalf][kTile][kPitch];
    auto each = [&](auto f) {
        float* row = part[wave % kHalf][r];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < kWords; ++q)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    f(*(float4_t*)&row[kLaneCols * (4 * g + i) + 8 * q + 4 * h], i, q, 4 * h);
    };
    auto put = [&](float4_t& at, int i, int q, int j) {
        at = (float4_t){acc[q][j][i], acc[q][j + 1][i], acc[q][j + 2][i], acc[q][j + 3][i]};
    };
    if (wave >= kHalf) each(put);
    __syncthreads();
    if (wave < kHalf) {
        each([&](float4_t& at, int i, int q, int j) {
            const float4_t v = at;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[q][j + e][i] += v[e];
        });
        each(put);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < t.rows * (kCols / 8); i += kWaves * kWave) {
        const int m = i / (kCols / 8), c = i % (kCols / 8) * 8;
        if (k0 + c >= a.K) continue;
        float s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[j] = part[0][m][c + j];
#pragma unroll
            for (int v = 1; v < kHalf; ++v) s[j] += part[v][m][c + j];
        }
        const int64_t at = (int64_t)(t.row0 + m) * a.K + k0 + c;
        if (a.part != nullptr) {
            float* out = a.part + (int64_t)slice * a.R * a.K + at;
            __builtin_memcpy(__builtin_assume_aligned(out, 16), s, 32);
        } else {
            uint16_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = T::store(s[j]);
            __builtin_memcpy(__builtin_assume_aligned(a.dX + at, 16), o, 16);
        }
    }
}

// N slices (dense): as many as give every CU two blocks, of at least four steps a wave.
struct Choice {
    int slices, steps;
};
Choice choose(int64_t R, int64_t N, int64_t K, bool grouped, bool split) {
    const int64_t total = (N + kStepRows - 1) / kStepRows;
    Choice c{1, (int)(total > 0 ? total : 1)};
    if (grouped || !split) return c;
    const int64_t blocks = (R + kTile - 1) / kTile * ((K + kCols - 1) / kCols);
    int64_t s = 512 / blocks;
    if (s > total / (4 * kWaves)) s = total / (4 * kWaves);
    if (s > 1) {
        c.steps = (int)((total + s - 1) / s);
        c.slices = (int)((total + c.steps - 1) / c.steps);
    }
    return c;
}

}  // namespace

size_t grad_workspace(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || K <= 0) return 0;
    const Choice c = choose(M, N, K, false, true);
    return c.slices > 1 ? (size_t)c.slices * M * K * sizeof(float) : 0;
}

hipError_t launch_grad(GradArgs a, DType dt, float* part, hipStream_t stream) {
    const Choice c = choose(a.R, a.N, a.K, a.offsets != nullptr, part != nullptr);
    a.slices = c.slices, a.steps = c.steps;
    a.part = c.slices > 1 ? part : a.dX32;
    const int64_t slots = a.offsets ? tile_slots(a.R, a.E, kTile) : (a.R + kTile - 1) / kTile;
    const dim3 grid = slot_grid((a.K + kCols - 1) / kCols * a.slices, slots);
    if (dt == kF16) stream_grad_kernel<F16><<<grid, kWaves * kWave, 0, stream>>>(a);
    else stream_grad_kernel<BF16><<<grid, kWaves * kWave, 0, stream>>>(a);
    if (c.slices > 1) launch_add_slices(part, c.slices, (int64_t)a.R * a.K, a.dX, dt, stream);
    return hipGetLastError();
}

}  // namespace mxfp4
