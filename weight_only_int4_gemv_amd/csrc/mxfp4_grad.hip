// mxfp4_grad.hip — the gradient through the weight-only product, dX = dY W: 16-bit rows times
// untransposed MXFP4 weights, summed over the weight rows.
//
// Codes lie along K, the matrix instructions sum along N.  A lane loads one word or more of the
// same columns from eight weight rows, converts them (scales are those of a row and block) and
// pairs neighbouring rows with one byte permutation per pair; the lane then holds, for each of
// its columns, the eight weight rows that are its operand of a 16x16x32 instruction.  A wave's
// instructions j = 0, 1, ... take column j of every lane, so that a lane ends with neighbouring
// columns of dX: 16 lanes of 16 columns are 256 columns, and the results need no turning.
#include "mxfp4_launch.h"
#include "mxfp4_tile.h"

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

template <int N>
struct Int {
    static constexpr int value = N;
};

// f(Int<FROM>()) ... f(Int<TO - 1>()).
template <int FROM, int TO, class F>
__device__ __forceinline__ void units(F f) {
    if constexpr (FROM < TO) {
        f(Int<FROM>());
        units<FROM + 1, TO>(f);
    }
}

template <class F, int N>
__device__ __forceinline__ void each_of(F f, Int<N>) {
    units<0, N>(f);
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

// ------------------------------------------------------------------- tiled
//
// Many rows.  A block of four waves owns 16 MT rows of dY and 256 columns of dX, each wave all
// rows and 64 columns, so that a weight is converted once per block: a vector instruction per
// weight pair is what bounds the product (two of them fit beside a 16x16x32 matrix instruction,
// a third costs a quarter of the rate).  N is walked in steps of 64 weight rows, whose dY tile
// and codes go from global memory straight to LDS, kStages steps deep.  The scales' bytes go there
// a step earlier and become fp32 in LDS a step before their use.  (Loaded to registers they cost
// the copies their depth: the wait for them is a wait for every copy on its way.)
//
// In LDS, 16-byte chunk c of row m of dY stands at c ^ x_swizzle(m): 16 lanes that read one chunk
// of 16 rows meet all banks once.  Of each 32 weight rows, row 8 g + i has place 4 i + g (lane
// groups g = 0 .. 3 read one i together) and chunk c of it stands at c ^ w_swizzle(g).
//
// 3001 rows, 14336 x 4096, fp16: 352 us in a long row of calls, 302 to 331 in a short one, 1.0 to 1.15
// PFLOP/s (512 tiles of 96 rows, two a CU, fill one round); 8192 tokens' rows of 64 experts of 3584 x
// 4096: 856 us, 1.05 PFLOP/s.  Blocks of 2 x 2 waves, which convert each weight twice, took 475 us for
// the first, 256 x 256 with a wave a SIMD 619 (bf16).  32 rows each of 64 experts: 197 us, and 231
// without s_setprio around the products, 225 to 244 with the scales' conversion put off by a step or
// the copies spread between the products.
constexpr int kStep = 64;
constexpr int kXRow = kStep * 2;                            // bytes of a row of the dY tile
constexpr int kTiledWaves = 4, kTiledThreads = kTiledWaves * kWave;
constexpr int kWaveCols = 64;
constexpr int kTiledCols = kWaveCols * kTiledWaves;
constexpr int kWRow = kTiledCols / 2;                       // bytes of a weight row
constexpr int kSubBytes = kStepRows * kWRow;                // 32 weight rows
constexpr int kXRows = 8 * kTiledWaves;                     // rows of one copy of every wave
constexpr int kWCopies = 2;                                 // of a wave and step
constexpr int kBlocks = kTiledCols / kBlock;                // scales of a weight row
constexpr int kScales = kBlocks * kStep;                    // of a step: a byte each, then fp32

// What weight rows past N and rows past the tile are multiplied with.
__device__ const uint4_t kZeros = {0, 0, 0, 0};

template <int MT_, int STAGES, int PER_CU>
struct Tiling {
    static constexpr int MT = MT_, kStages = STAGES, kPerCu = PER_CU, BM = 16 * MT;
    static constexpr int kXBytes = BM * kXRow, kStage = kXBytes + 2 * kSubBytes;
    static constexpr int kXCopies = BM / kXRows;            // of a wave and step
    static constexpr int kBytes = kStages * kStage + 2 * kScales * 4, kFlags = kBytes + kStages * kScales;
    static constexpr int kLds = kFlags + 16;
    static_assert(BM % kXRows == 0, "whole copies");
    static_assert(kLds * PER_CU <= 160 * 1024, "blocks fit a CU");
};

__device__ __forceinline__ int x_swizzle(int m) { return (m >> 1) & 7; }
__device__ __forceinline__ int w_swizzle(int g) { return g & 2; }
// Place of the scale of weight row n (of 64) in block b: two blocks and four lane groups that are
// read together meet different banks.
__device__ __forceinline__ int scale_at(int b, int n) { return b * kStep + (n ^ ((b & 1) << 2)); }

// Byte C of a weight row's word, columns 2C and 2C + 1, as a pair of 16-bit values.
template <int C>
__device__ __forceinline__ uint32_t pair(uint32_t w, float s, F16) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, C));
}
template <int C>
__device__ __forceinline__ uint32_t pair(uint32_t w, float s, BF16) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, C));
}

template <typename T, class C, bool WIDE>
__global__ __launch_bounds__(kTiledThreads, C::kPerCu) void tiled_grad_kernel(GradArgs a) {
    constexpr bool kIsF16 = __is_same(T, F16);
    constexpr int MT = C::MT, kStages = C::kStages;
    constexpr int kAsync = (WIDE ? C::kXCopies : 0) + kWCopies;     // in flight, of a wave and step
    typedef typename T::vec8 vec8;
    __shared__ __align__(1024) char lds[C::kLds];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int nt = (a.K + kTiledCols - 1) / kTiledCols;

    // Tile of this block.  Grouped: column blocks innermost; the XCDs share the tiles in use.
    // Dense: bands of kBand row tiles, row tiles innermost.
    constexpr int kBand = 8;
    int64_t blocks = gridDim.x;
    if (a.offsets != nullptr) {
        blocks = (int64_t)count_tiles(a.offsets, a.E, a.R, C::BM) * nt - a.first;
        if (blockIdx.x >= blocks) return;
        blocks = min(blocks, (int64_t)gridDim.x);
    }
    const int64_t id = a.first + xcd_order(blockIdx.x, (int)blocks);
    Tile t;
    int nb, slice = 0;
    if (a.offsets != nullptr) {
        const int64_t slot = id / nt;
        nb = (int)(id - slot * nt);
        t = find_tile(a.offsets, a.E, a.R, C::BM, (int)slot);
        t.expert = __builtin_amdgcn_readfirstlane(t.expert);
        t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
        t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    } else {
        const int mt = (a.R + C::BM - 1) / C::BM;
        const int64_t tiles = (int64_t)mt * nt, run = (int64_t)kBand * nt;
        slice = (int)(id / tiles);
        const int64_t tile = id - slice * tiles;
        const int band = (int)(tile / run), in_band = (int)(tile - band * run);
        const int high = min(kBand, mt - band * kBand);
        t.expert = 0;
        t.row0 = (band * kBand + in_band % high) * C::BM;
        t.rows = min(C::BM, a.R - t.row0);
        nb = in_band / high;
    }
    if (t.rows <= 0) return;
    const int k0 = nb * kTiledCols;
    const int KB = a.K / kBlock, row_bytes = a.K / 2;
    const int total = (a.N + kStep - 1) / kStep, step0 = slice * a.steps;
    const int steps = t.expert < 0 ? 0 : min(a.steps, total - step0);
    const int64_t expert_row = (int64_t)max(t.expert, 0) * a.N;
    const uint32_t base = lds_address(lds);

    // Copies: a base that moves with the steps and a lane's offset that does not.
    // dY: wave w, copy c: the 8 rows from (c * kTiledWaves + w) * 8 on.
    const int x_row = wave * 8 + lane / 8, x_chunk = (lane & 7) ^ x_swizzle(x_row);
    const uint16_t* x_base = a.dY + t.row0 * a.y_stride + (int64_t)step0 * kStep;
    const uint32_t x_off = (uint32_t)(x_row * (uint32_t)a.y_stride + x_chunk * 8) * 2;
    const int64_t x_next = kXRows * a.y_stride;             // from copy to copy
    // Codes: copy j of wave w takes the eight places from 8 ((2 w + j) % 4) on of half w / 2 of
    // the step.  Columns past K are not stored: they read the block's first.
    const int w_g = lane / 8 & 3, w_chunk = (lane & 7) ^ w_swizzle(w_g);
    const int w_row = (wave >> 1) * kStepRows + 4 * (wave & 1) + 8 * w_g + lane / 32;   // j: + 2 j
    const uint8_t* w_base = a.codes + (expert_row + (int64_t)step0 * kStep) * row_bytes + k0 / 2;
    const uint32_t w_off = (uint32_t)w_row * row_bytes + (k0 / 2 + w_chunk * 16 < row_bytes ? w_chunk * 16 : 0);
    // Scales: wave w takes those of half w % 2 of the step's rows, four blocks a lane, where they
    // stand on words (two waves bring the same: a copy for part of a wave costs a branch).
    const bool words = KB % 4 == 0 && (uintptr_t)a.scales % 4 == 0;
    const int kb0 = k0 / kBlock, s_row0 = (wave & 1) * kStepRows;
    const uint32_t s_off = (uint32_t)(s_row0 + lane / 2) * KB + (kb0 + (lane & 1) * 4 < KB ? (lane & 1) * 4 : 0);
    const uint8_t* s_base = a.scales + (expert_row + (int64_t)step0 * kStep) * KB + kb0;
    uint32_t s_to = 0;
    auto copy_scales = [&](int s) {                         // one step after the other
        if (!words || s >= steps) return;
        const int n0 = (step0 + s) * kStep;
        uint32_t off = s_off;                               // rows past N: the last row's
        if (n0 + kStep > a.N) off -= (uint32_t)max(n0 + s_row0 + lane / 2 - (a.N - 1), 0) * KB;
        copy4(s_base, off, __builtin_amdgcn_readfirstlane(base + C::kBytes + s_to + s_row0 * kBlocks));
        s_base += kStep * KB;
        s_to = s_to + kScales == kStages * kScales ? 0 : s_to + kScales;
    };
    uint32_t to = 0;                                        // LDS offset of the copied stage
    auto copy = [&](int s) {
        const int n0 = (step0 + s) * kStep;
        const uint32_t x_to = base + to + wave * 8 * kXRow;
        const uint32_t w_to = base + to + C::kXBytes + wave * 2 * 8 * kWRow;
        if (WIDE && n0 + kStep <= a.N) {
            if (t.rows == C::BM) {
#pragma unroll
                for (int c = 0; c < C::kXCopies; ++c)
                    copy16(x_base + c * x_next, x_off, x_to + c * kXRows * kXRow);
            } else {
                // Rows past the tile: its last row, for dX rows that are not stored.
                int l = lane;                               // for no register to stay taken
                asm volatile("" : "+v"(l));
#pragma unroll
                for (int c = 0; c < C::kXCopies; ++c) {
                    const int row = min(wave * 8 + l / 8, t.rows - 1 - c * kXRows);
                    const uint32_t off = (uint32_t)(max(row, 0) * (uint32_t)a.y_stride + x_chunk * 8) * 2;
                    copy16(x_base + (c * kXRows < t.rows ? c * x_next : 0), off, x_to + c * kXRows * kXRow);
                }
            }
#pragma unroll
            for (int j = 0; j < kWCopies; ++j)
                copy16(w_base + 2 * j * row_bytes, w_off, w_to + j * 8 * kWRow);
        } else {
            int l = lane;                                   // for no register to stay taken
            asm volatile("" : "+v"(l));
            const int x_row = wave * 8 + l / 8, x_chunk = (l & 7) ^ x_swizzle(x_row);
            const int w_row = (wave >> 1) * kStepRows + 4 * (wave & 1) + 8 * (l / 8 & 3) + l / 32;
            auto copy_x = [&](int c) {
                const int n = n0 + x_chunk * 8;
                const bool live = x_row + c * kXRows < t.rows;
                const uint16_t* p = x_base + c * x_next + x_row * a.y_stride + x_chunk * 8;
                if constexpr (WIDE) {
                    copy16(live && n < a.N ? (const void*)p : &kZeros, x_to + c * kXRows * kXRow);
                } else {
                    uint4_t v = {0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (live && n + i < a.N) v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
                    *(uint4_t*)(lds + to + (c * kXRows + wave * 8) * kXRow + l * 16) = v;
                }
            };
            if constexpr (WIDE) {
#pragma unroll
                for (int c = 0; c < C::kXCopies; ++c) copy_x(c);
            } else {
#pragma unroll 1
                for (int c = 0; c < C::kXCopies; ++c) copy_x(c);
            }
#pragma unroll
            for (int j = 0; j < kWCopies; ++j) {            // rows past N: the last row's codes
                const int row = min(2 * j, a.N - 1 - n0 - w_row);
                copy16(w_base + w_off + (int64_t)row * row_bytes, w_to + j * 8 * kWRow);
            }
        }
        x_base += kStep;
        w_base += (int64_t)kStep * row_bytes;
        to = to + C::kStage == kStages * C::kStage ? 0 : to + C::kStage;
    };

    // Scales as fp32: two blocks of a weight row a thread.
    bool far = false;
    float* scales = (float*)(lds + kStages * C::kStage);
    volatile int* wide_at = (volatile int*)(lds + C::kFlags);   // of even and odd steps: the last
                                                                // one outside fp16's range
    auto convert_scales = [&](int s) {
        if (s >= steps) return;
        const int s_row = threadIdx.x / 4, s_block = threadIdx.x % 4 * 2;
        const int n = (step0 + s) * kStep + s_row;
        uint32_t v;
        if (words) {
            v = *(const uint16_t*)(lds + C::kBytes + s % kStages * kScales + threadIdx.x * 2);
        } else {                                            // past K: not stored
            const uint8_t* row = a.scales + (expert_row + min(n, a.N - 1)) * KB;
            const int kb = kb0 + s_block;
            v = row[min(kb, KB - 1)] | (uint32_t)row[min(kb + 1, KB - 1)] << 8;
        }
        if (n >= a.N) v = 0x7F7F;                           // past N: 1
        bool out = false;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint32_t byte = v >> 8 * b & 255;
            out = out || !f16_scale_ok(byte);
            far = far || byte >= kFarScale;
            scales[(s & 1) * kScales + scale_at(s_block + b, s_row)] = scale_value(byte);
        }
        if (kIsF16 && out) wide_at[s & 1] = s;
    };

    // Operands: of weights the words (four columns) and scales of the lane's eight rows, then a
    // pair of columns at a time; of dY a fragment per row tile.
    uint32_t w[8];
    float sc[8];
    vec8 x[MT];
    uint4_t f[2][2];
    float4_t acc[MT][4] = {};
    const int x_at = r * kXRow + (g ^ x_swizzle(r)) * 16;   // half 1's is 64 bytes on or back
    const int w_at = C::kXBytes + g * kWRow + ((wave * 2) ^ w_swizzle(g)) * 16 + r * 2;
    const int s_at = scale_at(wave * 2 + r / 8, 8 * g);
    auto load_w = [&](uint32_t stage, int s, int sub) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = *(const uint16_t*)(lds + stage + w_at + sub * kSubBytes + i * 4 * kWRow);
        const float* from = scales + (s & 1) * kScales + sub * kStepRows;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4_t v = *(const float4_t*)(from + (s_at ^ h * 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[4 * h + i] = v[i];
        }
    };
    auto load_x = [&](uint32_t stage, int sub, int m) {
        return *(const vec8*)(lds + stage + (x_at ^ sub * 64) + m * 16 * kXRow);
    };
    // Weight rows 2i and 2i + 1 of the columns 2c and 2c + 1.
    auto convert = [&](auto pair_of, auto rows, auto type) {
        constexpr int c = decltype(pair_of)::value, i = decltype(rows)::value;
        const uint32_t p = pair<c>(w[2 * i], sc[2 * i], type);
        const uint32_t q = pair<c>(w[2 * i + 1], sc[2 * i + 1], type);
        f[c][0][i] = low_halves(p, q);
        f[c][1][i] = high_halves(p, q);
    };

    if (steps > 0) {
        if (threadIdx.x < 2) wide_at[threadIdx.x] = -1;
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kStages; ++s) {
            if (s < steps) copy(s);
            copy_scales(s);
        }
        wait_copies<0>();
        convert_scales(0);
        convert_scales(1);
        __syncthreads();
        copy_scales(kStages);                               // where those of step 0 stood
        // To step s + 1, when a wave has all of step s in registers: its tile is free for the copy
        // kStages on, its scales for those of step s + 2.
        auto next_step = [&](int s) {
            if (s + kStages > steps) wait_copies<0>();
            else if (s + kStages + 1 <= steps && words) wait_copies<(kStages - 2) * (kAsync + 1)>();
            else wait_copies<(kStages - 2) * kAsync>();
        };
        uint32_t stage = 0;
        load_w(0, 0, 0);
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = load_x(0, 0, m);
        each_of([&](auto i) { convert(Int<0>(), i, T()); }, Int<4>());
        // The products of a pair of columns over the row tiles, while the next pair is converted:
        // pair 1 of these weight rows, or pair 0 of the next ones, which are half `sub` of step s
        // at `stage` and are read meanwhile, dY's fragments as their last use passes.
        auto products = [&](auto pair_of, uint32_t stage, int s, int sub) {
            constexpr int c = decltype(pair_of)::value;
            if constexpr (c == 1) load_w(stage, s, sub);
            each_of([&](auto mm) {
                constexpr int m = decltype(mm)::value;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    acc[m][2 * c + h] =
                        T::mfma16(__builtin_bit_cast(vec8, f[c][h]), x[m], acc[m][2 * c + h]);
                if constexpr (c == 1) x[m] = load_x(stage, sub, m);
                // The four units of the next pair, behind the reads of their weights.
                constexpr int F = MT / 2, kLeft = MT - F;
                if constexpr (m >= F)
                    units<(m - F) * 4 / kLeft, (m - F + 1) * 4 / kLeft>(
                        [&](auto i) { convert(Int<1 - c>(), i, T()); });
                __builtin_amdgcn_sched_barrier(0);
            }, Int<MT>());
        };
        int s = 0, wide = kIsF16 ? wide_at[0] : -1;
        for (; s < steps; ++s) {
            if (kIsF16 && __builtin_amdgcn_readfirstlane(wide) == s) break;
            products(Int<0>(), 0, 0, 0);
            products(Int<1>(), stage, s, 1);
            products(Int<0>(), 0, 0, 0);
            __builtin_amdgcn_s_setprio(0);
            if (s + 1 < steps) next_step(s);
            stage = stage + C::kStage == kStages * C::kStage ? 0 : stage + C::kStage;
            if (s + kStages < steps) copy(s + kStages);
            copy_scales(s + 1 + kStages);                   // where those of step s + 1 stood
            convert_scales(s + 2);
            if (kIsF16) wide = wide_at[(s + 1) & 1];
            __builtin_amdgcn_s_setprio(1);
            products(Int<1>(), stage, s + 1, 0);            // past the last step: not used
        }
        // From the first step with weights outside fp16's range on: weights are exact in bf16,
        // dY is the sum of two bf16 values.
        for (; kIsF16 && s < steps; ++s) {
#pragma unroll 1
            for (int sub = 0; sub < 2; ++sub) {
                load_w(stage, s, sub);
                each_of([&](auto i) {
                    convert(Int<0>(), i, BF16());
                    convert(Int<1>(), i, BF16());
                }, Int<4>());
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    bf168_t hi, lo;
                    split_bf16(__builtin_bit_cast(half8_t, load_x(stage, sub, m)), hi, lo);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bf168_t v = __builtin_bit_cast(bf168_t, f[j / 2][j % 2]);
                        acc[m][j] = BF16::mfma16(v, hi, acc[m][j]);
                        acc[m][j] = BF16::mfma16(v, lo, acc[m][j]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (s + 1 < steps) next_step(s);
            stage = stage + C::kStage == kStages * C::kStage ? 0 : stage + C::kStage;
            if (s + kStages < steps) copy(s + kStages);
            copy_scales(s + 1 + kStages);
            convert_scales(s + 2);
        }
        wait_copies<0>();
        if (__syncthreads_or(far)) {
            // Weights that bf16 does not hold: the block's sums again, in quarters, straight from
            // global memory.
            int l = lane;
            asm volatile("" : "+v"(l));
            const int r = l & 15, g = l >> 4;
            const int col = min(k0 + wave * kWaveCols + 4 * r, a.K - 4);
            const int last = min((step0 + steps) * kStep, a.N);
            each_of([&](auto tile) {                        // a row tile at a time: registers
                constexpr int m = decltype(tile)::value;
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][j] = (float4_t){0, 0, 0, 0};
                const uint16_t* from = a.dY + (t.row0 + min(m * 16 + r, t.rows - 1)) * a.y_stride;
#pragma unroll 1
                for (int n0 = step0 * kStep; n0 < last; n0 += kStepRows) {
                    uint32_t word[8], sb[8];
                    uint4_t v = {0, 0, 0, 0}, q[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int n = n0 + 8 * g + i, at = min(n, a.N - 1);
                        const int64_t row = expert_row + at;
                        word[i] = *(const uint16_t*)(a.codes + row * row_bytes + col / 2);
                        sb[i] = a.scales[row * KB + col / kBlock];
                        const uint32_t e = from[at];
                        if (n >= a.N) sb[i] = 127;
                        v[i / 2] |= (n < a.N ? e : 0) << (16 * (i & 1));
                    }
                    turn8<BF16>(word, [&](uint32_t u, int i) { return quarter8(u, sb[i]); }, q);
                    bf168_t hi = __builtin_bit_cast(bf168_t, v), lo;
                    if constexpr (kIsF16) split_bf16(__builtin_bit_cast(half8_t, v), hi, lo);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bf168_t u = __builtin_bit_cast(bf168_t, q[j]);
                        acc[m][j] = BF16::mfma16(u, hi, acc[m][j]);
                        if constexpr (kIsF16) acc[m][j] = BF16::mfma16(u, lo, acc[m][j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][j] *= 4.0f;
            }, Int<MT>());
        }
    }

    // Results: lane l holds row l % 16 of dX and, in register i of acc[m][j], the column
    // 4 (4 g + i) + j: 16 neighbouring columns.
    int l = lane;
    asm volatile("" : "+v"(l));
    const int col = k0 + wave * kWaveCols + 16 * (l >> 4);
    if (col >= a.K) return;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row = m * 16 + (l & 15);
        if (row >= t.rows) continue;
        const int64_t at = (int64_t)(t.row0 + row) * a.K + col;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = acc[m][j % 4][2 * h + j / 4];
            if (a.part != nullptr) {
                float* out = a.part + (int64_t)slice * a.R * a.K + at + 8 * h;
                __builtin_memcpy(__builtin_assume_aligned(out, 16), v, 32);
            } else {
                uint16_t o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = T::store(v[j]);
                __builtin_memcpy(__builtin_assume_aligned(a.dX + at + 8 * h, 16), o, 16);
            }
        }
    }
}

typedef Tiling<8, 3, 2> Large;      // 128 x 256
typedef Tiling<6, 3, 2> Mid;        // 96 x 256
typedef Tiling<4, 3, 2> Medium;     // 64 x 256
typedef Tiling<2, 3, 3> Low;        // 32 x 256

template <class C>
void launch(GradArgs a, DType dt, hipStream_t stream) {
    // The offset of a copy's rows has 32 bits.  Where a row's last chunk is part-filled or rows do
    // not start on 16 bytes, dY is read by element in every step: 3001 rows of 14336 x 4096 319 us,
    // of 14335 x 4096 978, with rows 14335 apart 1353; of 50257 x 2048 2712, of 50256 624.
    const bool wide = (uintptr_t)a.dY % 16 == 0 && a.N % 8 == 0 &&
                      (a.R == 1 || (a.y_stride % 8 == 0 && a.y_stride <= 1 << 25));
    const int64_t nt = (a.K + kTiledCols - 1) / kTiledCols;
    const int64_t slots = a.offsets ? tile_slots(a.R, a.E, C::BM) : (a.R + C::BM - 1) / C::BM;
    const int64_t blocks = slots * nt * a.slices;
    for (a.first = 0; a.first < blocks; a.first += kMaxGrid) {
        const unsigned grid = (unsigned)(blocks - a.first < kMaxGrid ? blocks - a.first : kMaxGrid);
        if (dt == kF16 && wide)
            tiled_grad_kernel<F16, C, true><<<grid, kTiledThreads, 0, stream>>>(a);
        else if (dt == kF16)
            tiled_grad_kernel<F16, C, false><<<grid, kTiledThreads, 0, stream>>>(a);
        else if (wide)
            tiled_grad_kernel<BF16, C, true><<<grid, kTiledThreads, 0, stream>>>(a);
        else
            tiled_grad_kernel<BF16, C, false><<<grid, kTiledThreads, 0, stream>>>(a);
    }
}

// Kernel and N slices.
//   Experts, by rows per expert on average (all rows / experts), as measured for 64 experts of
//   3584 x 4096; other counts and sizes follow the same borders (us):
//     rows     stream   Low   Medium   Mid   Large
//     2           117   135      202   224     248
//     16          168   143      214   227     252
//     32          260   197      207   230     256
//     64          443   274      277   243     266
//     96                372      312   313     283
//     320              1014      788   681     670
//   Dense: up to 16 rows the streaming kernel; else the tiling and the slices that the times below
//   say are fastest.
enum Kernel { kStream, kLow, kMedium, kMid, kLarge };
struct Choice {
    Kernel kernel;
    int slices, steps;
};
// A step of 64 weight rows takes `one` us with a block on a CU and `two` with two of them (measured on
// M x 4096, 8192 weight rows); a launch begins and ends with the time of about three steps.
struct Cost {
    Kernel kernel;
    int rows;
    double one, two;
};
constexpr Cost kCosts[] = {{kLarge, Large::BM, 1.20, 1.54}, {kMid, Mid::BM, 1.07, 1.33},
                           {kMedium, Medium::BM, 0.93, 1.08}, {kLow, Low::BM, 0.83, 0.87}};

Choice choose(int64_t R, int64_t E, int64_t N, int64_t K, bool grouped, bool split) {
    const int64_t steps = N > 0 ? (N + kStep - 1) / kStep : 1;
    Choice best{kStream, 1, (int)steps};
    if (grouped ? R < 12 * E : R <= kTile) {
        const int64_t total = N > 0 ? (N + kStepRows - 1) / kStepRows : 1;
        best.steps = (int)total;
        // Slices: as many as give every CU two blocks, of at least four steps a wave.
        int64_t s = split ? 512 / ((K + kCols - 1) / kCols) : 1;
        if (s > total / (4 * kWaves)) s = total / (4 * kWaves);
        if (!grouped && s > 1) {
            best.steps = (int)((total + s - 1) / s);
            best.slices = (int)((total + best.steps - 1) / best.steps);
        }
        return best;
    }
    if (grouped) {
        best.kernel = R < 28 * E ? kLow : R < 52 * E ? kMedium : R < 80 * E ? kMid : kLarge;
        return best;
    }
    double least = 0;
    for (const Cost& c : kCosts) {
        const int64_t tiles = (R + c.rows - 1) / c.rows * ((K + kTiledCols - 1) / kTiledCols);
        for (int64_t s = 1; s <= (split ? 16 : 1) && (s == 1 || steps / s >= 4); ++s) {
            const int64_t run = (steps + s - 1) / s, slices = (steps + run - 1) / run;
            const int64_t blocks = tiles * slices, left = blocks % 512;
            double us = (run + 3) * (double(blocks / 512) * c.two + (left > 256 ? c.two : left > 0 ? c.one : 0));
            // The slices' sums are written, read and added at about 4 TB/s by a second launch.
            if (slices > 1) us += 3 + double(slices) * R * K * 8 / 4e6;
            if (best.kernel == kStream || us < least) {
                least = us;
                best = {c.kernel, (int)slices, (int)run};
            }
        }
    }
    return best;
}

}  // namespace

size_t grad_workspace(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || K <= 0) return 0;
    const Choice c = choose(M, 1, N, K, false, true);
    return c.slices > 1 ? (size_t)c.slices * M * K * sizeof(float) : 0;
}

hipError_t launch_grad(GradArgs a, DType dt, float* part, hipStream_t stream) {
    const Choice c = choose(a.R, a.E, a.N, a.K, a.offsets != nullptr, part != nullptr);
    a.slices = c.slices, a.steps = c.steps;
    a.part = c.slices > 1 ? part : a.dX32;
    if (c.kernel == kLarge) {
        launch<Large>(a, dt, stream);
    } else if (c.kernel == kMid) {
        launch<Mid>(a, dt, stream);
    } else if (c.kernel == kMedium) {
        launch<Medium>(a, dt, stream);
    } else if (c.kernel == kLow) {
        launch<Low>(a, dt, stream);
    } else {
        const int64_t slots = a.offsets ? tile_slots(a.R, a.E, kTile) : (a.R + kTile - 1) / kTile;
        const dim3 grid = slot_grid((a.K + kCols - 1) / kCols * a.slices, slots);
        if (dt == kF16) stream_grad_kernel<F16><<<grid, kWaves * kWave, 0, stream>>>(a);
        else stream_grad_kernel<BF16><<<grid, kWaves * kWave, 0, stream>>>(a);
    }
    if (c.slices > 1) launch_add_slices(part, c.slices, (int64_t)a.R * a.K, a.dX, dt, stream);
    return hipGetLastError();
}

}  // namespace mxfp4
