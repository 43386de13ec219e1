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
// Many rows.  A block of WM x WK waves owns 16 MT WM rows of dY and 128 WK columns of dX; N is
// walked in steps of 64 weight rows, whose dY tile and codes go from global memory straight to
// LDS, STAGES steps deep.  Scales come through registers, as fp32: they follow the rows.
//
// In LDS, 16-byte chunk c of row m of dY stands at c ^ x_swizzle(m), so that 16 lanes that read
// one chunk of 16 rows meet all banks once; of each 32 weight rows those that lane groups 0 to 3
// read together (8 g + i for one i) stand side by side, 64 bytes of a wave's 128 columns each.
constexpr int kStep = 64;
constexpr int kXRow = kStep * 2;                            // bytes of a row of the dY tile
constexpr int kWaveCols = 128;
constexpr int kSubBytes = kStepRows * kWaveCols / 2;        // 32 weight rows of a wave's columns
constexpr int kChunk = 4;                                   // steps whose scales are loaded together

// What weight rows past N are multiplied with.
__device__ const uint4_t kZeros = {0, 0, 0, 0};

template <int WM_, int WK_, int MT_, int STAGES, int PER_CU>
struct Tiling {
    static constexpr int kPerCu = PER_CU;
    static constexpr int WM = WM_, WK = WK_, MT = MT_, kStages = STAGES;
    static constexpr int BM = 16 * MT * WM, BK = kWaveCols * WK;
    static constexpr int kWaves = WM * WK, kThreads = kWaves * kWave;
    static constexpr int kXBytes = BM * kXRow, kStage = kXBytes + 2 * WK * kSubBytes;
    static constexpr int kXRows = 8 * kWaves;               // rows of one copy of every wave
    static constexpr int kXCopies = BM / kXRows, kWCopies = 4 / WM;
    static constexpr int kBlocks = 4 * WK;                  // scales of a weight row
    static constexpr int kHeld = 4 / WM;                    // of them a thread's
    static constexpr int kScales = kBlocks * kStep * 4;
    static constexpr int kFlags = STAGES * kStage + 2 * kScales;
    static constexpr int kLds = kFlags + 16;
    static_assert(BM % kXRows == 0 && kXRows % 16 == 0, "a lane's copies share their swizzle");
    static_assert(kLds * PER_CU <= 160 * 1024, "blocks fit a CU");
};

__device__ __forceinline__ int x_swizzle(int m) { return (m >> 1) & 7; }
// Place of the scale of weight row n (of 64) in the row of block b: the four blocks and four
// lane groups of a wave's read meet different banks.
__device__ __forceinline__ int scale_at(int b, int n) {
    return b * kStep + (n ^ ((b & 1) << 2) ^ ((b & 2) << 4));
}

// Byte C of a weight row's word, columns 2C and 2C + 1, as a pair of 16-bit values.
template <int C>
__device__ __forceinline__ uint32_t pair(uint32_t w, float s, F16) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, C));
}
template <int C>
__device__ __forceinline__ uint32_t pair(uint32_t w, float s, BF16) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, C));
}
template <int C, typename T>
__device__ __forceinline__ void columns(const uint32_t (&w)[8], const float (&s)[8], T t,
                                        uint4_t& even, uint4_t& odd) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = pair<C>(w[2 * i], s[2 * i], t), b = pair<C>(w[2 * i + 1], s[2 * i + 1], t);
        even[i] = low_halves(a, b);
        odd[i] = high_halves(a, b);
    }
}

template <typename T, class C, bool WIDE>
__global__ __launch_bounds__(C::kThreads, C::kPerCu * C::kWaves / 4) void tiled_grad_kernel(GradArgs a) {
    constexpr bool kIsF16 = __is_same(T, F16);
    constexpr int MT = C::MT;
    constexpr int kAsync = (WIDE ? C::kXCopies : 0) + C::kWCopies;  // copies in flight, a wave and step
    typedef typename T::vec8 vec8;
    __shared__ __align__(1024) char lds[C::kLds];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / C::WK, wk = wave % C::WK;
    const int r = lane & 15, g = lane >> 4;
    const int nt = (a.K + C::BK - 1) / C::BK;

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
    const int k0 = nb * C::BK;
    const int KB = a.K / kBlock, row_bytes = a.K / 2;
    const int total = (a.N + kStep - 1) / kStep, step0 = slice * a.steps;
    const int steps = t.expert < 0 ? 0 : min(a.steps, total - step0);
    const int64_t expert_row = (int64_t)max(t.expert, 0) * a.N;
    const uint32_t base = lds_address(lds);

    // Copies of dY: wave w, copy c: the 8 rows from (c * kWaves + w) * 8 on.
    const int x_row = wave * 8 + lane / 8, x_chunk = (lane & 7) ^ x_swizzle(x_row);
    const uint16_t* xp = a.dY + (int64_t)(t.row0 + x_row) * a.y_stride + step0 * kStep + x_chunk * 8;
    // Of codes: 16 places of 64 bytes, place p of 32 rows being row 8 (p % 4) + p / 4; copy j of a
    // wave lies 4 (j % 2) + 32 (j / 2) rows behind its first.  Columns past K are not stored: they
    // read the row's first.
    const int q0 = wave * C::kWCopies;
    const int w_col = (k0 + q0 / 4 * kWaveCols) / 2 + (lane & 3) * 16;
    const int w_row = (q0 >> 1 & 1) * kStepRows + 8 * (lane / 4 & 3) + lane / 16;
    const uint8_t* wp = a.codes + (expert_row + step0 * kStep + w_row) * row_bytes +
                        (w_col < row_bytes ? w_col : 0);
    auto copy = [&](int s) {
        const uint32_t to = __builtin_amdgcn_readfirstlane(s % C::kStages * C::kStage);
        const int n0 = (step0 + s) * kStep;
        const bool tail = n0 + kStep > a.N;
        auto copy_x = [&](int c) {
            const uint32_t at = to + (c * C::kXRows + wave * 8) * kXRow;
            const int n = n0 + x_chunk * 8;
            const bool live = x_row + c * C::kXRows < t.rows;       // others are not stored
            const uint16_t* p = xp + c * C::kXRows * a.y_stride;
            if constexpr (WIDE) {
                copy16(live && !(tail && n >= a.N) ? (const void*)p : &kZeros, base + at);
            } else {
                uint4_t v = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (live && n + i < a.N) v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
                *(uint4_t*)(lds + at + lane * 16) = v;
            }
        };
        if constexpr (WIDE) {
#pragma unroll
            for (int c = 0; c < C::kXCopies; ++c) copy_x(c);
        } else {
#pragma unroll 1
            for (int c = 0; c < C::kXCopies; ++c) copy_x(c);
        }
        xp += kStep;
#pragma unroll
        for (int j = 0; j < C::kWCopies; ++j) {
            int row = 4 * (j & 1) + kStepRows * (j >> 1);
            // Rows past N: the last row's codes.
            if (tail) row = min(row, a.N - 1 - n0 - w_row);
            copy16(wp + (int64_t)row * row_bytes,
                   base + to + C::kXBytes + (q0 + j) * (kSubBytes / 2));
        }
        wp += (int64_t)kStep * row_bytes;
    };

    // Scales: a thread holds those of kHeld blocks of one weight row of each of kChunk steps.
    constexpr int kPerRow = C::kBlocks / C::kHeld;          // threads of a weight row
    const int s_row = threadIdx.x / kPerRow, s_block = threadIdx.x % kPerRow * C::kHeld;
    const int kb0 = k0 / kBlock + s_block;
    uint32_t held[kChunk];
    auto load_scales = [&](int s) {                         // of steps s .. s + kChunk - 1
#pragma unroll
        for (int c = 0; c < kChunk; ++c) {
            const int n = (step0 + s + c) * kStep + s_row;
            held[c] = 0x7F7F7F7Fu;                          // past N and K: 1
            if (n >= a.N) continue;
            const uint8_t* p = a.scales + (expert_row + n) * KB + kb0;
            if (kb0 + C::kHeld <= KB) {
                __builtin_memcpy(&held[c], p, C::kHeld);    // any byte
            } else {
#pragma unroll
                for (int b = 0; b < C::kHeld; ++b)
                    if (kb0 + b < KB) held[c] = (held[c] & ~(255u << 8 * b)) | (uint32_t)p[b] << 8 * b;
            }
        }
    };
    bool far = false;
    float* scales = (float*)(lds + C::kStages * C::kStage);
    volatile int* wide_at = (volatile int*)(lds + C::kFlags);   // of even and odd steps: the last
                                                                // one outside fp16's range
    auto store_scales = [&](int s) {
        bool out = false;
#pragma unroll
        for (int b = 0; b < C::kHeld; ++b) {
            const uint32_t byte = held[0] >> 8 * b & 255;
            out = out || !f16_scale_ok(byte);
            far = far || byte >= kFarScale;
            scales[(s & 1) * (C::kScales / 4) + scale_at(s_block + b, s_row)] = scale_value(byte);
        }
        if (kIsF16 && out) wide_at[s & 1] = s;
#pragma unroll
        for (int c = 0; c + 1 < kChunk; ++c) held[c] = held[c + 1];
        if (s % kChunk == kChunk - 1) load_scales(s + 1);
    };

    // Operands of 32 weight rows.
    struct Sub {
        uint32_t w[8];
        float s[8];
        vec8 x[MT];
    };
    const int x_at = (wm * MT * 16 + r) * kXRow, swizzle = x_swizzle(r);
    const int w_at = C::kXBytes + wk * 2 * kSubBytes + g * 64 + r * 4;
    const int block = wk * 4 + r / 4;
    auto load_w = [&](Sub& d, int s, int sub) {
        const char* stage = lds + s % C::kStages * C::kStage;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            d.w[i] = *(const uint32_t*)(stage + w_at + sub * kSubBytes + i * 256);
        const float* sc = scales + (s & 1) * (C::kScales / 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4_t v = *(const float4_t*)&sc[scale_at(block, sub * kStepRows + 8 * g + 4 * h)];
#pragma unroll
            for (int i = 0; i < 4; ++i) d.s[4 * h + i] = v[i];
        }
    };
    auto load_x = [&](int s, int sub, int m) {
        const char* stage = lds + s % C::kStages * C::kStage;
        return *(const vec8*)(stage + x_at + m * 16 * kXRow + ((4 * sub + g) ^ swizzle) * 16);
    };
    auto load = [&](Sub& d, int s, int sub) {
        load_w(d, s, sub);
#pragma unroll
        for (int m = 0; m < MT; ++m) d.x[m] = load_x(s, sub, m);
    };
    float4_t acc[MT][8] = {};
    // The products of d's pair C of columns (even and odd in f), while the next pair, next.w's byte
    // (C + 1) % 4, is converted.
    uint4_t f[2][2];
    auto convert = [&](auto c, const Sub& d) {
        constexpr int CC = decltype(c)::value;
        columns<CC>(d.w, d.s, T(), f[CC & 1][0], f[CC & 1][1]);
    };
    auto multiply = [&](auto c, const Sub& d, const Sub& next) {
        constexpr int CC = decltype(c)::value;
        convert(Int<(CC + 1) % 4>(), next);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[m][2 * CC + h] = T::mfma16(__builtin_bit_cast(vec8, f[CC & 1][h]), d.x[m],
                                               acc[m][2 * CC + h]);
        __builtin_amdgcn_sched_barrier(0);
    };

    if (steps > 0) {
        if (threadIdx.x < 2) wide_at[threadIdx.x] = -1;
        __syncthreads();
        load_scales(0);
        store_scales(0);
#pragma unroll
        for (int s = 0; s < C::kStages; ++s)
            if (s < steps) copy(s);
        wait_copies<0>();
        // To step s + 1, when a wave has all of step s in registers.
        auto advance = [&](int s) {
            if (s + 1 >= steps) return;
            store_scales(s + 1);
            if (s + C::kStages <= steps) wait_copies<(C::kStages - 2) * kAsync>();
            else wait_copies<0>();
            if (s + C::kStages < steps) copy(s + C::kStages);
        };
        Sub d[2];
        load(d[0], 0, 0);
        convert(Int<0>(), d[0]);
        int s = 0;
        for (; s < steps; ++s) {
            if (kIsF16 && __builtin_amdgcn_readfirstlane(wide_at[s & 1]) == s) break;
            load(d[1], s, 1);
            multiply(Int<0>(), d[0], d[0]);
            multiply(Int<1>(), d[0], d[0]);
            multiply(Int<2>(), d[0], d[0]);
            multiply(Int<3>(), d[0], d[1]);
            advance(s);
            load(d[0], s + 1, 0);                   // past the last step: not used
            multiply(Int<0>(), d[1], d[1]);
            multiply(Int<1>(), d[1], d[1]);
            multiply(Int<2>(), d[1], d[1]);
            multiply(Int<3>(), d[1], d[0]);
        }
        // From the first step with weights outside fp16's range on: weights are exact in bf16,
        // dY is the sum of two bf16 values.
        for (; kIsF16 && s < steps; ++s) {
#pragma unroll 1
            for (int sub = 0; sub < 2; ++sub) {
                load_w(d[0], s, sub);
                auto pairs = [&](auto c) {
                    constexpr int CC = decltype(c)::value;
                    uint4_t w[2];
                    columns<CC>(d[0].w, d[0].s, BF16(), w[0], w[1]);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        bf168_t hi, lo;
                        split_bf16(__builtin_bit_cast(half8_t, load_x(s, sub, m)), hi, lo);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float4_t& to = acc[m][2 * CC + h];
                            to = BF16::mfma16(__builtin_bit_cast(bf168_t, w[h]), hi, to);
                            to = BF16::mfma16(__builtin_bit_cast(bf168_t, w[h]), lo, to);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                };
                pairs(Int<0>()), pairs(Int<1>()), pairs(Int<2>()), pairs(Int<3>());
            }
            advance(s);
        }
        wait_copies<0>();
        if (__syncthreads_or(far)) {
            // Weights that bf16 does not hold: the block's sums again, in quarters, straight from
            // global memory.
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[m][j] = (float4_t){0, 0, 0, 0};
            const int col = min(k0 + wk * kWaveCols + 8 * r, a.K - 8);
            const int last = min((step0 + steps) * kStep, a.N);
            auto row_tile = [&](auto tile) {                // a row tile at a time: registers
                constexpr int m = decltype(tile)::value;
                const int row = min((wm * MT + m) * 16 + r, t.rows - 1);
                const uint16_t* from = a.dY + (t.row0 + row) * a.y_stride;
#pragma unroll 1
                for (int n0 = step0 * kStep; n0 < last; n0 += kStepRows) {
                    uint32_t w[8], sb[8];
                    uint4_t x = {0, 0, 0, 0}, q[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int n = n0 + 8 * g + i, at = min(n, a.N - 1);
                        const int64_t weight = expert_row + at;
                        w[i] = *(const uint32_t*)(a.codes + weight * row_bytes + col / 2);
                        sb[i] = a.scales[weight * KB + col / kBlock];
                        const uint32_t v = from[at];
                        if (n >= a.N) sb[i] = 127;
                        x[i / 2] |= (n < a.N ? v : 0) << (16 * (i & 1));
                    }
                    turn8<BF16>(w, [&](uint32_t v, int i) { return quarter8(v, sb[i]); }, q);
                    bf168_t hi = __builtin_bit_cast(bf168_t, x), lo;
                    if constexpr (kIsF16) split_bf16(__builtin_bit_cast(half8_t, x), hi, lo);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const bf168_t v = __builtin_bit_cast(bf168_t, q[j]);
                        acc[m][j] = BF16::mfma16(v, hi, acc[m][j]);
                        if constexpr (kIsF16) acc[m][j] = BF16::mfma16(v, lo, acc[m][j]);
                    }
                }
            };
            static_assert(MT == 1 || MT == 2 || MT == 4, "every row tile once");
            row_tile(Int<0>());
            if constexpr (MT > 1) row_tile(Int<1>());
            if constexpr (MT > 2) row_tile(Int<2>()), row_tile(Int<MT - 1>());
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[m][j] *= 4.0f;
        }
    }

    // Results: lane l holds row l % 16 of dX and, in register i of acc[m][j], the column
    // 8 (4 g + i) + j: 32 neighbouring columns.
    const int col = k0 + wk * kWaveCols + 32 * g;
    if (col >= a.K) return;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row = (wm * MT + m) * 16 + r;
        if (row >= t.rows) continue;
        const int64_t at = (int64_t)(t.row0 + row) * a.K + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = acc[m][j][i];
            if (a.part != nullptr) {
                float* out = a.part + (int64_t)slice * a.R * a.K + at + 8 * i;
                __builtin_memcpy(__builtin_assume_aligned(out, 16), v, 32);
            } else {
                uint16_t o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = T::store(v[j]);
                __builtin_memcpy(__builtin_assume_aligned(a.dX + at + 8 * i, 16), o, 16);
            }
        }
    }
}

typedef Tiling<2, 2, 4, 3, 2> Large;        // 128 x 256

template <class C>
void launch(GradArgs a, DType dt, hipStream_t stream) {
    const bool wide = (uintptr_t)a.dY % 16 == 0 && a.N % 8 == 0 && (a.y_stride % 8 == 0 || a.R == 1);
    const int64_t nt = (a.K + C::BK - 1) / C::BK;
    const int64_t slots = a.offsets ? tile_slots(a.R, a.E, C::BM) : (a.R + C::BM - 1) / C::BM;
    const int64_t blocks = slots * nt * a.slices;
    for (a.first = 0; a.first < blocks; a.first += kMaxGrid) {
        const unsigned grid = (unsigned)(blocks - a.first < kMaxGrid ? blocks - a.first : kMaxGrid);
        if (dt == kF16 && wide)
            tiled_grad_kernel<F16, C, true><<<grid, C::kThreads, 0, stream>>>(a);
        else if (dt == kF16)
            tiled_grad_kernel<F16, C, false><<<grid, C::kThreads, 0, stream>>>(a);
        else if (wide)
            tiled_grad_kernel<BF16, C, true><<<grid, C::kThreads, 0, stream>>>(a);
        else
            tiled_grad_kernel<BF16, C, false><<<grid, C::kThreads, 0, stream>>>(a);
    }
}

// Kernel and N slices.
enum Kernel { kStream, kLarge };
struct Choice {
    Kernel kernel;
    int slices, steps;
};
Choice choose(int64_t R, int64_t E, int64_t N, int64_t K, bool grouped, bool split) {
    Choice c{R > 32 * E ? kLarge : kStream, 1, 0};
    const int rows = c.kernel == kStream ? kStepRows : kStep;
    const int64_t total = N > 0 ? (N + rows - 1) / rows : 1;
    c.steps = (int)total;
    if (grouped || !split) return c;
    // As many as give every CU two blocks, of at least four steps a wave (tiled: eight).
    const int64_t blocks = c.kernel == kStream ? (R + kTile - 1) / kTile * ((K + kCols - 1) / kCols)
                                               : (R + Large::BM - 1) / Large::BM *
                                                     ((K + Large::BK - 1) / Large::BK);
    const int64_t least = c.kernel == kStream ? 4 * kWaves : 8;
    int64_t s = 512 / blocks;
    if (s > total / least) s = total / least;
    if (s > 1) {
        c.steps = (int)((total + s - 1) / s);
        c.slices = (int)((total + c.steps - 1) / c.steps);
    }
    return c;
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
