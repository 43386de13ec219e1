// mxfp4_tiled.hip — weight-only MXFP4 product for many rows (prefill, larger
// batches, experts with tens of rows and more): 16-bit X times MXFP4 weights,
// dequantized in registers, on the 32x32x16 matrix instructions.
//
// A block owns BM rows of X and BN weight rows; each of its waves all BM rows
// and WN weight rows, so that a weight is converted once per block.  K is
// walked in steps of 64 columns: X and code tiles go from global memory
// straight to LDS, kStages tiles deep, scales a chunk
// of blocks of each row at a time through registers.  The sum over k may run in any order as long as both
// operands agree: half h of a wave takes block h of the step (16 bytes of
// codes and one scale a lane), MFMA i its columns 8i .. 8i+7.
//
// What bounds it: the matrix cores and their feeding from LDS where tiles are
// full (2000 x 14336 x 4096 224 us in a row of calls, 1.05 PFLOP/s; matrix cores
// 49 % busy over the 241 us of a counted launch; 4096 x 16384 x 14336 1.21
// PFLOP/s); with few rows the latency of a step (0.45 us of LDS reads, barrier and
// 256 matrix-core cycles), which nothing hides where there is one block a CU.  A
// tile's rows are multiplied whether they are there or not.  Blocks of 256 weight rows read
// X from the caches least often; two or three of them a CU hide each other's
// barriers (one of 256 x 256: 8192 tokens over 64 experts 1091 us against 1000).
//
// With SwiGLU a block's weight rows are 32 gate rows, their 32 up rows, the
// next 32 gate rows ..., so that a wave holds both factors of its outputs.
#include "mxfp4_launch.h"
#include "mxfp4_tile.h"

namespace mxfp4 {
namespace {

constexpr int kStepCols = 64;
constexpr int kXRow = kStepCols * 2;        // bytes of a row of the X tile
constexpr int kGroup = 32;                  // weight rows copied together
constexpr int kGroupBytes = kGroup * kStepCols / 2;

// What rows of zeros are read from (no token, columns past K).
__device__ const uint4_t kZeros = {0, 0, 0, 0};

template <int BM_, int WN_, int WAVES, int STAGES, int SCALE_BLOCKS, int PER_CU>
struct Tiling {
    static constexpr int kPerCu = PER_CU;                   // blocks on a CU
    static constexpr int BM = BM_, WN = WN_, BN = WN * WAVES;
    static constexpr int MT = BM / 32, NT = WN / 32;
    static constexpr int kWaves = WAVES, kThreads = WAVES * kWave, kStages = STAGES;
    static constexpr int kXBytes = BM * kXRow, kStage = kXBytes + BN / kGroup * kGroupBytes;
    static constexpr int kScaleBlocks = SCALE_BLOCKS;       // scales of a row staged together
    static constexpr int kScaleSteps = kScaleBlocks * kBlock / kStepCols;
    static constexpr int kScales = BN * kScaleBlocks;
    static constexpr int kXRows = 8 * WAVES;                // rows of one X copy of every wave
    static constexpr int kXCopies = BM / kXRows;
    static constexpr int kWCopies = BN / kGroup / WAVES;
    static constexpr int kCopies = kXCopies + kWCopies;     // per wave and step
    static constexpr int kPitch = WN + 4;
    static constexpr int kTurn = 32 * kPitch * 4;           // a wave's 32 rows in fp32
    static constexpr int kLoop = STAGES * kStage + 2 * kScales;
    static constexpr int kLds = kLoop > kTurn * WAVES ? kLoop : kTurn * WAVES;
    static_assert(BM % kXRows == 0 && kXRows % 16 == 0, "a lane's copies share their swizzle");
    static_assert(kLds * PER_CU <= 160 * 1024, "blocks fit a CU");
    static_assert(BN <= kThreads, "a row's scales a thread");
    static_assert(BN % (kGroup * WAVES) == 0, "whole groups a wave");
};

// 16-byte chunk c of row r of the X tile stands at c ^ x_swizzle(r), block b of
// weight row r of a group at b ^ w_swizzle(r): 16 lanes that read the same chunk
// of 16 rows meet all 64 banks once.
__device__ __forceinline__ int x_swizzle(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int w_swizzle(int r) { return (r >> 3) & 1; }

template <typename T, class C>
__global__ __launch_bounds__(C::kThreads, C::kPerCu * C::kWaves / 4) void tiled_kernel(LinearArgs a) {
    constexpr bool kIsF16 = __is_same(T, F16);
    constexpr int MT = C::MT, NT = C::NT;
    typedef typename T::vec8 vec8;
    __shared__ __align__(1024) char lds[C::kLds];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int F = a.swiglu ? a.N / 2 : a.N;                 // columns of Y
    const int per = a.swiglu ? C::BN / 2 : C::BN;           // of one block

    // Tile of this block.  Grouped: column blocks innermost, so that blocks of one
    // row tile run together; the XCDs share the tiles in use, not the slots (300
    // tokens over 64 experts use 83 of 103 slots: 125 us by slots, 101 by tiles).  Dense: bands of kBand row tiles, row tiles innermost.
    constexpr int kBand = 8;
    int64_t blocks = gridDim.x;
    if (a.offsets != nullptr) {
        blocks = (int64_t)count_tiles(a.offsets, a.E, a.R, C::BM) * a.nt - a.first;
        if (blockIdx.x >= blocks) return;
        blocks = min(blocks, (int64_t)gridDim.x);
    }
    const int64_t id = a.first + xcd_order(blockIdx.x, (int)blocks);
    Tile t;
    int nb, slice = 0;
    if (a.offsets != nullptr) {
        const int64_t slot = id / a.nt;
        nb = (int)(id - slot * a.nt);
        t = find_tile(a.offsets, a.E, a.R, C::BM, (int)slot);
        t.expert = __builtin_amdgcn_readfirstlane(t.expert);
        t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
        t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    } else {
        const int64_t tiles = (int64_t)a.mt * a.nt, run = (int64_t)kBand * a.nt;
        slice = (int)(id / tiles);
        const int64_t tile = id - slice * tiles;
        const int band = (int)(tile / run), in_band = (int)(tile - band * run);
        const int high = min(kBand, a.mt - band * kBand);
        t.expert = 0;
        t.row0 = (band * kBand + in_band % high) * C::BM;
        t.rows = min(C::BM, a.R - t.row0);
        nb = in_band / high;
    }
    if (t.rows <= 0) return;
    const int col0 = nb * per;
    const int KB = a.K / kBlock, row_bytes = a.K / 2;
    const int step0 = slice * a.steps;
    const int steps = t.expert < 0 ? 0 : min(a.steps, (KB + 1) / 2 - step0);
    // K % 64 == 32: the last step's second block lies past K.
    const int odd_step = (KB & 1) ? KB / 2 - step0 : -1;
    const uint32_t base = lds_address(lds);

    // First weight row (of the expert) of group g, and how many of its 32 exist.
    auto group_row = [&](int g) {
        return a.swiglu ? (g & 1) * F + col0 + (g >> 1) * kGroup : col0 + g * kGroup;
    };
    auto group_rows = [&](int g) {
        return min(kGroup, F - (a.swiglu ? col0 + (g >> 1) * kGroup : col0 + g * kGroup));
    };
    const int64_t expert_row = (int64_t)max(t.expert, 0) * a.N;

    // Copies.  X: wave w, copy c: the 8 rows from (c * kWaves + w) * 8 on.
    const int x_row = wave * 8 + lane / 8, x_chunk = (lane & 7) ^ x_swizzle(x_row);
    const char* xp[C::kXCopies];
    uint32_t live = 0;
#pragma unroll
    for (int c = 0; c < C::kXCopies; ++c) {
        const int r = t.row0 + min(x_row + c * C::kXRows, t.rows - 1);   // not stored past rows
        const int src = a.tokens ? a.tokens[r] : r;
        const bool ok = src >= 0 && src < a.x_rows;
        xp[c] = ok ? (const char*)(a.X + src * a.x_stride + step0 * kStepCols + x_chunk * 8)
                   : (const char*)&kZeros;
        live |= (ok ? kXRow : 0u) << c;
    }
    uint4_t wrsrc[C::kWCopies];
#pragma unroll
    for (int j = 0; j < C::kWCopies; ++j) {
        const int g = j * C::kWaves + wave, rows = group_rows(g);
        wrsrc[j] = make_rsrc(a.codes + (expert_row + (rows > 0 ? group_row(g) : 0)) * row_bytes,
                             (uint32_t)max(rows, 0) * row_bytes);
#pragma unroll
        for (int i = 0; i < 4; ++i) wrsrc[j][i] = __builtin_amdgcn_readfirstlane(wrsrc[j][i]);
    }
    uint32_t w_off = (uint32_t)(lane / 2) * row_bytes + step0 * (kStepCols / 2) +
                     ((lane & 1) ^ w_swizzle(lane / 2)) * 16;
    auto copy = [&](int s) {
        const uint32_t to = base + s % C::kStages * C::kStage;
#pragma unroll
        for (int c = 0; c < C::kXCopies; ++c) {
            const char* p = s == odd_step && x_chunk >= 4 ? (const char*)&kZeros : xp[c];
            copy16(p, to + (c * C::kXRows + wave * 8) * kXRow);
            xp[c] += (live >> c) & kXRow;
        }
        // Blocks past K are the next row's first codes (or 0): they meet zeros.
#pragma unroll
        for (int j = 0; j < C::kWCopies; ++j)
            copy16(wrsrc[j], w_off, to + C::kXBytes + (j * C::kWaves + wave) * kGroupBytes);
        w_off += kStepCols / 2;
    };

    // Scales: thread t holds kHeld blocks of row t in registers (half a cache line,
    // so that lines are fetched once and the loop rarely waits for a load) and
    // passes on kScaleBlocks at a time: LDS holds word w (blocks 4w ..) of row r
    // at [w][r].  Blocks past K count as 1.
    constexpr int kScaleBlocks = C::kScaleBlocks, kScaleSteps = C::kScaleSteps;
    constexpr int kHeld = 64, kChunks = kHeld / kScaleBlocks;
    const int s_row = min((int)threadIdx.x, C::BN - 1), s_rows = group_rows(s_row / kGroup);
    const uint8_t* srow = a.scales + (expert_row + (s_rows > 0 ? group_row(s_row / kGroup) +
                                      min(s_row % kGroup, s_rows - 1) : 0)) * KB + step0 * 2;
    const int blocks_left = KB - step0 * 2;                 // from the slice's first on
    uint32_t held[kHeld / 4];
    auto load_scales = [&](int c) {                         // chunks c .. c + kChunks - 1
        const int kb = c * kScaleBlocks;
#pragma unroll
        for (int j = 0; j < kHeld / 8; ++j) {
            uint2_t v = {0, 0};
            if (kb + (j * 8 / kScaleBlocks + 1) * kScaleBlocks <= blocks_left)
                __builtin_memcpy(&v, srow + kb + 8 * j, 8);     // any byte
            held[2 * j] = v[0];
            held[2 * j + 1] = v[1];
        }
    };
    auto store_scale_chunk = [&](int c) {
        const int kb = c * kScaleBlocks;
        char* at = lds + C::kStages * C::kStage + (c & 1) * C::kScales;
        if (C::BN < C::kThreads && threadIdx.x >= C::BN) return;
        if (kb + kScaleBlocks <= blocks_left) {
#pragma unroll
            for (int w = 0; w < kScaleBlocks / 4; ++w) ((uint32_t*)at)[w * C::BN + s_row] = held[w];
#pragma unroll
            for (int w = 0; w < (kHeld - kScaleBlocks) / 4; ++w) held[w] = held[w + kScaleBlocks / 4];
        } else {
#pragma unroll 1
            for (int b = 0; b < kScaleBlocks; ++b)
                at[(b / 4 * C::BN + s_row) * 4 + b % 4] = kb + b < blocks_left ? srow[kb + b] : 127;
        }
    };
    // At the start of step s: the next kChunks, once the last chunk held is in LDS.
    auto more_scales = [&](int s) {
        const int c = s / kScaleSteps + 1;
        if (s % kScaleSteps == 0 && c % kChunks == 0 && c * kScaleSteps < steps) load_scales(c);
    };

    // Fragments of the wave.
    const int half = lane >> 5, r31 = lane & 31;
    const int x_at = r31 * kXRow;
    int x_off[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x_off[i] = x_at + ((4 * half + i) ^ x_swizzle(r31)) * 16;
    const int w_at = C::kXBytes + wave * NT * kGroupBytes + r31 * 16 * 2 + (half ^ w_swizzle(r31)) * 16;
    auto load_x = [&](vec8 (&x)[MT], const char* stage, int i) {
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = *(const vec8*)(stage + x_off[i] + m * 32 * kXRow);
    };
    uint32_t far = 0;                   // the largest scale byte the lane has met
    auto load_w = [&](uint4_t (&w)[NT], float (&sc)[NT], bool& wide, int s) {
        const char* stage = lds + s % C::kStages * C::kStage;
        const int in = s % kScaleSteps;
        const uint32_t* word = (const uint32_t*)(lds + C::kStages * C::kStage +
                                                 (s / kScaleSteps & 1) * C::kScales);
        bool out = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            w[n] = *(const uint4_t*)(stage + w_at + n * kGroupBytes);
            const uint32_t b = word[in / 2 * C::BN + wave * C::WN + 32 * n + r31] >>
                               (16 * (in & 1) + 8 * half) & 255;
            out |= !f16_scale_ok(b);
            far = max(far, b);
            sc[n] = scale_value(b);
        }
        wide = kIsF16 && __any(out);
    };
    float16_t acc[MT][NT] = {};
    auto multiply = [&](const vec8 (&x)[MT], const vec8 (&w)[NT]) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[m][n] = T::mfma32(w[n], x[m], acc[m][n]);
    };

    if (steps > 0) {
        load_scales(0);
#pragma unroll
        for (int s = 0; s < C::kStages; ++s)
            if (s < steps) copy(s);
        store_scale_chunk(0);
        wait_copies<0>();

        vec8 x[2][MT], wv[2][NT];
        uint4_t codes[NT];
        float sc[NT];
        bool wide;
        // To step s + 1: every wave has read the last of step s, so its tile is
        // free for the copy kStages on.
        auto advance = [&](int s) {
            if (s + 1 >= steps) return;
            if ((s + 1) % kScaleSteps == 0) store_scale_chunk((s + 1) / kScaleSteps);
            if (s + C::kStages <= steps) wait_copies<(C::kStages - 2) * C::kCopies>();
            else wait_copies<0>();
            if (s + C::kStages < steps) copy(s + C::kStages);
            load_w(codes, sc, wide, s + 1);
        };
        load_w(codes, sc, wide, 0);
        load_x(x[0], lds, 0);
#pragma unroll
        for (int n = 0; n < NT; ++n) wv[0][n] = values8(codes[n][0], sc[n], T());
        int s = 0;
        // A step's first fragments are read while the matrix cores work on the
        // last ones of the step before.
        for (; s < steps; ++s) {
            if (kIsF16 && wide) break;
            const char* stage = lds + s % C::kStages * C::kStage;
            more_scales(s);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                load_x(x[(i + 1) & 1], stage, i + 1);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    wv[(i + 1) & 1][n] = values8(codes[n][i + 1], sc[n], T());
                multiply(x[i & 1], wv[i & 1]);
                __builtin_amdgcn_sched_barrier(0);
            }
            advance(s);
            load_x(x[0], lds + (s + 1) % C::kStages * C::kStage, 0);
            multiply(x[1], wv[1]);
#pragma unroll
            for (int n = 0; n < NT; ++n) wv[0][n] = values8(codes[n][0], sc[n], T());
        }
        // From the first step with weights outside fp16's range on: weights are
        // exact in bf16, X is the sum of two bf16 values.
        for (; kIsF16 && s < steps; ++s) {
            const char* stage = lds + s % C::kStages * C::kStage;
            more_scales(s);
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                bf168_t w[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    w[n] = values8(*(const uint32_t*)(stage + w_at + n * kGroupBytes + 4 * i),
                                   sc[n], BF16());
                const int off = x_at + ((4 * half + i) ^ x_swizzle(r31)) * 16;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    bf168_t hi, lo;
                    split_bf16(*(const half8_t*)(stage + off + m * 32 * kXRow), hi, lo);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        acc[m][n] = BF16::mfma32(w[n], hi, acc[m][n]);
                        acc[m][n] = BF16::mfma32(w[n], lo, acc[m][n]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            advance(s);
        }
        wait_copies<0>();
        if (__builtin_expect(__any(far >= kFarScale), 0)) {
            // Weights that bf16 does not hold: the wave's rows again, in quarters,
            // straight from global memory.  A way out of the loops above instead costs
            // every bf16 call 1 to 4 %, this 0 to 2 % (50 x 4096 x 14336 22.5 / 23.3 / 23.0
            // us without, with a way out, and so).
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[m][n] = (float16_t){};
#pragma unroll 1
            for (int i = 0; i < 4 * steps; ++i) {
                const int kb = (step0 + i / 4) * 2 + half;
                const bool in = kb < KB;
                bf168_t w[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int g = wave * NT + n, rows = group_rows(g);
                    const int64_t row = expert_row + (rows > 0 ? group_row(g) + min(r31, rows - 1) : 0);
                    w[n] = quarter8(in ? *(const uint32_t*)(a.codes + row * row_bytes + kb * 16 + i % 4 * 4) : 0,
                                    in ? a.scales[row * KB + kb] : 127);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int r = t.row0 + min(r31 + 32 * m, t.rows - 1);
                    const int src = a.tokens ? a.tokens[r] : r;
                    uint4_t xv = {0, 0, 0, 0};
                    if (in && src >= 0 && src < a.x_rows)
                        xv = *(const uint4_t*)(a.X + src * a.x_stride + kb * kBlock + i % 4 * 8);
                    bf168_t hi = __builtin_bit_cast(bf168_t, xv), lo;
                    if constexpr (kIsF16) split_bf16(__builtin_bit_cast(half8_t, xv), hi, lo);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        acc[m][n] = BF16::mfma32(w[n], hi, acc[m][n]);
                        if constexpr (kIsF16) acc[m][n] = BF16::mfma32(w[n], lo, acc[m][n]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[m][n] *= 4.0f;
        }
    }

    // Results: lane l holds row l % 32 of X and the weight rows 8 g + 4 half + i
    // in registers 4 g + i.  Each wave turns 32 rows at a time in its own LDS, so
    // that stores run along the rows of Y.
    float* turn = (float*)(lds + wave * C::kTurn);
    const int wcols = a.swiglu ? C::WN / 2 : C::WN;
    const int wcol0 = col0 + wave * wcols, cols = min(wcols, F - wcol0);
    const bool wide_out = F % 8 == 0 && (uintptr_t)a.Y % 16 == 0;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (NT > 1 && a.swiglu && (n & 1)) continue;
            const int at = r31 * C::kPitch + (a.swiglu ? n / 2 : n) * 32 + 4 * half;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float4_t v;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = acc[m][n][4 * g + i];
                    if (NT > 1 && a.swiglu) v[i] = silu(v[i]) * acc[m][n | 1][4 * g + i];
                }
                *(float4_t*)&turn[at + 8 * g] = v;
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int rows = min(32, t.rows - 32 * m);
        const int64_t out0 = (int64_t)(t.row0 + 32 * m) * F + wcol0;
        if (a.part != nullptr) {
            float* p = a.part + (int64_t)slice * a.R * F + out0;
            if (F % 4 == 0 && (uintptr_t)a.part % 16 == 0) {
                for (int i = lane; i < 32 * C::WN / 4; i += kWave) {
                    const int r = i / (C::WN / 4), c = i % (C::WN / 4) * 4;
                    if (r < rows && c < cols)
                        *(float4_t*)(p + (int64_t)r * F + c) = *(const float4_t*)&turn[r * C::kPitch + c];
                }
            } else {
                for (int i = lane; i < 32 * C::WN; i += kWave) {
                    const int r = i / C::WN, c = i % C::WN;
                    if (r < rows && c < cols) p[(int64_t)r * F + c] = turn[r * C::kPitch + c];
                }
            }
        } else if (wide_out) {
            const int shift = a.swiglu ? 1 : 0;             // 8 columns a lane
            for (int i = lane; i < 32 * C::WN / 8 >> shift; i += kWave) {
                const int r = i / (C::WN / 8 >> shift), c = i % (C::WN / 8 >> shift) * 8;
                uint16_t v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = T::store(turn[r * C::kPitch + c + j]);
                if (r < rows && c < cols)
                    __builtin_memcpy(__builtin_assume_aligned(a.Y + out0 + (int64_t)r * F + c, 16), v, 16);
            }
        } else {
            for (int i = lane; i < 32 * wcols; i += kWave) {
                const int r = i / wcols, c = i % wcols;
                if (r < rows && c < cols)
                    a.Y[out0 + (int64_t)r * F + c] = T::store(turn[r * C::kPitch + c]);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

typedef Tiling<128, 64, 4, 3, 16, 2> Large;         // 128 x 256
typedef Tiling<64, 64, 4, 3, 8, 3> Medium;          // 64 x 256
typedef Tiling<32, 64, 4, 4, 8, 3> Low;             // 32 x 256
typedef Tiling<64, 32, 4, 4, 16, 3> Narrow;         // 64 x 128

template <class C>
void launch(LinearArgs a, DType dt, hipStream_t stream) {
    const int F = a.swiglu ? a.N / 2 : a.N, per = a.swiglu ? C::BN / 2 : C::BN;
    a.nt = (F + per - 1) / per;
    a.mt = (a.R + C::BM - 1) / C::BM;
    const int64_t slots = a.offsets ? tile_slots(a.R, a.E, C::BM) : a.mt;
    const int64_t blocks = slots * a.nt * a.slices;
    for (a.first = 0; a.first < blocks; a.first += kMaxGrid) {
        const unsigned grid = (unsigned)(blocks - a.first < kMaxGrid ? blocks - a.first : kMaxGrid);
        if (dt == kF16)
            tiled_kernel<F16, C><<<grid, C::kThreads, 0, stream>>>(a);
        else
            tiled_kernel<BF16, C><<<grid, C::kThreads, 0, stream>>>(a);
    }
}

// Kernel and K split.
//   Experts, by rows per expert on average (all rows / experts), as measured for 64
//   experts and one layer; other counts and sizes follow the same borders (us,
//   gate-up 3584 x 4096 / down 4096 x 1792):
//     rows       stream       Low     Medium     Large
//     0.5       54 / 32   57 / 33    72 / 41
//     2        117 / 63  101 / 48   111 / 56
//     16                 144 / 70   167 / 85
//     37                195 / 102   183 / 96
//     150                501 / 282  356 / 219  375 / 237
//     512              1504 / 844  1072 / 646  995 / 622
//   Dense: the largest tiles that give every CU a block; Narrow (32 rows: Low)
//   where none does.
//   K slices (dense): where the tiles are fewer than the blocks that fit on 256
//   CUs, as many as fill two a CU, of at least eight steps: 50 x 4096 x 14336
//   105 us unsplit, 24 in 8 or 16 slices; 17 rows 30 and 20 us.
enum Kernel { kStream, kLow, kNarrow, kMedium, kLarge };
struct Choice {
    Kernel kernel;
    int slices, steps;
};
Choice choose(int64_t R, int64_t E, int64_t N, int64_t K, bool grouped, bool split) {
    const int64_t total = (K / kBlock + 1) / 2;
    Choice c{kStream, 1, (int)total};
    if (grouped) {
        if (R >= E) c.kernel = R < 28 * E ? kLow : R < 192 * E ? kMedium : kLarge;
        return c;
    }
    if (R <= 16) return c;
    auto tiles = [&](int bm, int bn) { return (R + bm - 1) / bm * ((N + bn - 1) / bn); };
    int64_t n = tiles(128, 256);
    c.kernel = kLarge;
    if (n < 256) n = tiles(64, 256), c.kernel = kMedium;
    if (n < 256) n = tiles(64, 128), c.kernel = kNarrow;
    if (R <= 32) n = tiles(32, 256), c.kernel = kLow;
    if (split) {
        int64_t s = 512 / n, most = R <= 32 ? 16 : 8;
        if (s > most) s = most;
        if (s > total / 8) s = total / 8;
        if (s > 1) {
            c.steps = (int)((total + s - 1) / s);
            c.slices = (int)((total + c.steps - 1) / c.steps);
        }
    }
    return c;
}

}  // namespace

size_t linear_workspace(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0) return 0;
    const Choice c = choose(M, 1, N, K, false, true);
    return c.slices > 1 ? (size_t)c.slices * M * N * sizeof(float) : 0;
}

hipError_t launch_linear(LinearArgs a, DType dt, float* part, hipStream_t stream) {
    const Choice c = choose(a.R, a.E, a.N, a.K, a.offsets != nullptr, part != nullptr);
    a.slices = c.slices, a.steps = c.steps;
    a.part = c.slices > 1 ? part : a.Y32;
    switch (c.kernel) {
        case kStream: return launch_stream(a, dt, stream);
        case kLow: launch<Low>(a, dt, stream); break;
        case kNarrow: launch<Narrow>(a, dt, stream); break;
        case kMedium: launch<Medium>(a, dt, stream); break;
        case kLarge: launch<Large>(a, dt, stream); break;
    }
    if (c.slices > 1) launch_add_slices(a.part, a.slices, (int64_t)a.R * a.N, a.Y, dt, stream);
    return hipGetLastError();
}

}  // namespace mxfp4
