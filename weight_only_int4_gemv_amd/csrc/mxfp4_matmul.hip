// mxfp4_matmul.hip — product of two MXFP4 matrices on the block-scaled matrix
// instructions.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 with both operands fp4: lane l holds row
// l % 32 and one block (32 columns, 16 bytes) of each operand, lanes 32 up a
// second block, and one scale byte per operand and block; products and scales
// are exact, sums fp32.  The sum over k may run in any order as long as both
// operands agree: of the kStep blocks of a step, half h of the wave takes
// blocks h * kStep / 2 + i for MFMA i, so that the scale bytes a lane needs are
// neighbours (one word, its byte chosen by the instruction).
//
// What bounds it: copies to LDS and matrix instructions, 443 us each alone of the
// 546 that 4096 x 28672 x 8192 takes in a row of calls (3.5 PFLOP/s; 575-590 us
// and matrix cores 39 % busy in traced launches): they run largely in turn, since
// every wave waits for a whole stage at one barrier.  With few rows the latency of
// a step (1.4 us): one block a CU with one tile copy on its way.
//
// A block of BM x BN outputs walks K in steps of kStep blocks.  Code tiles go
// from global memory straight to LDS, kStages tiles deep; scales, 16 blocks of
// a row at a time, through registers.  16-byte chunks of a row are stored in
// an order that depends on the row, so that 16 lanes reading one chunk of 16
// rows meet different banks.
#include "mxfp4_launch.h"
#include "mxfp4_tile.h"

namespace mxfp4 {
namespace {

struct MatmulArgs {
    const uint8_t *ac, *as, *bc, *bs;
    void* Y;
    float* part;            // fp32 partial sums [slices][M][N], or NULL
    int M, N, K;
    int mt, nt;             // tiles
    int slices, steps;      // K slices, steps per slice
    int64_t first;          // first block of this launch
};

// Scale bytes S of both scale words apply.
template <int S>
__device__ __forceinline__ float16_t mfma_fp4(uint4_t a, uint4_t b, float16_t c, int sa, int sb) {
    const int8_t_ av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const int8_t_ bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, S, sa, S, sb);
}

template <DType DT>
struct Out;
template <>
struct Out<kF32> {
    typedef float type;
    static __device__ __forceinline__ float make(float v) { return v; }
};
template <>
struct Out<kBF16> {
    typedef uint16_t type;
    static __device__ __forceinline__ uint16_t make(float v) { return BF16::store(v); }
};
template <>
struct Out<kF16> {
    typedef uint16_t type;
    static __device__ __forceinline__ uint16_t make(float v) { return F16::store(v); }
};

constexpr int kScaleBlocks = 16;        // blocks of a row whose scales are staged together

template <int BM_, int BN_, int WM_, int WN_, int STAGES>
struct Tiling {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int kStep = 8, kStages = STAGES;
    static constexpr int kWavesN = BN / WN, kWaves = BM / WM * kWavesN, kThreads = kWaves * kWave;
    static constexpr int kRows = BM + BN;                   // A rows, then B rows
    static constexpr int kRowBytes = kStep * 16;
    static constexpr int kStage = kRows * kRowBytes;
    static constexpr int kScales = kRows * kScaleBlocks;
    static constexpr int kRowsPerCopy = 1024 / kRowBytes;   // rows of one wave's copy
    static constexpr int kCopyRows = kRowsPerCopy * kWaves; // of one copy of every wave
    static constexpr int kCopies = kRows / kCopyRows;
    static constexpr int kScaleSteps = kScaleBlocks / kStep;
    static constexpr int kScaleRows = (kRows + kThreads - 1) / kThreads;
    static constexpr int kLds = STAGES * kStage + 2 * kScales;
    static constexpr int kWaveLds = kLds / kWaves / 16 * 16;      // a wave's share in the epilogue
    static_assert(BM % kCopyRows == 0 && BN % kCopyRows == 0, "a copy stays in one operand");
    static_assert(kCopyRows % 16 == 0, "copies of a lane share its place in the swizzle");
    // Where 16-byte chunk c of a row stands: c ^ swizzle(row).
    static __device__ __forceinline__ int swizzle(int row) {
        return (row >> 1) & (kStep - 1);
    }
};

// Codes of one MFMA of every 32-row tile of the wave.
template <class T>
struct Fragments {
    uint4_t a[T::WM / 32], b[T::WN / 32];
    __device__ __forceinline__ void load(const char* a_row, const char* b_row, int at) {
#pragma unroll
        for (int m = 0; m < T::WM / 32; ++m)
            a[m] = *(const uint4_t*)(a_row + m * 32 * T::kRowBytes + at);
#pragma unroll
        for (int n = 0; n < T::WN / 32; ++n)
            b[n] = *(const uint4_t*)(b_row + n * 32 * T::kRowBytes + at);
    }
};

// MFMAs I .. of one step; `f` holds those of I.  The next ones are read ahead
// of the matrix instructions, and no further ahead (registers).
template <class T, int I>
struct Step {
    static __device__ __forceinline__ void run(const Fragments<T>& f, const char* a_row,
                                               const char* b_row, int swz, int half,
                                               const uint32_t (&sa)[T::WM / 32],
                                               const uint32_t (&sb)[T::WN / 32],
                                               float16_t (&acc)[T::WM / 32][T::WN / 32]) {
        Fragments<T> next;
        if constexpr (I + 1 < T::kStep / 2)
            next.load(a_row, b_row, ((half * (T::kStep / 2) + I + 1) ^ swz) * 16);
#pragma unroll
        for (int m = 0; m < T::WM / 32; ++m)
#pragma unroll
            for (int n = 0; n < T::WN / 32; ++n)
                acc[m][n] = mfma_fp4<I>(f.b[n], f.a[m], acc[m][n], sb[n], sa[m]);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (I + 1 < T::kStep / 2)
            Step<T, I + 1>::run(next, a_row, b_row, swz, half, sa, sb, acc);
    }
};

template <DType DT, class T>
__global__ __launch_bounds__(T::kThreads) void matmul_kernel(MatmulArgs a) {
    __shared__ __align__(1024) char lds[T::kLds];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t tiles = (int64_t)a.mt * a.nt;
    // Column tiles of a run of kBand row tiles, row tiles innermost.
    constexpr int kBand = 8;
    const int64_t id = a.first + xcd_order(blockIdx.x, gridDim.x);
    const int slice = (int)(id / tiles);
    const int64_t tile = id - slice * tiles, run = (int64_t)kBand * a.nt;
    const int band = (int)(tile / run), in_band = (int)(tile - band * run);
    const int high = min(kBand, a.mt - band * kBand);
    const int64_t m0 = (int64_t)(band * kBand + in_band % high) * T::BM;
    const int64_t n0 = (int64_t)(in_band / high) * T::BN;
    const int row_bytes = a.K / 2, KB = a.K / kBlock;
    const int step0 = slice * a.steps;
    const int steps = min(a.steps, (KB + T::kStep - 1) / T::kStep - step0);
    const int mrows = (int)min((int64_t)T::BM, a.M - m0), nrows = (int)min((int64_t)T::BN, a.N - n0);

    const uint4_t arsrc = make_rsrc(a.ac + m0 * row_bytes, (uint32_t)mrows * row_bytes);
    const uint4_t brsrc = make_rsrc(a.bc + n0 * row_bytes, (uint32_t)nrows * row_bytes);
    const uint32_t base = lds_address(lds);

    // Copy c of this wave takes the rows from (c * kWaves + wave) * kRowsPerCopy
    // on.  Rows past the matrix read 0; blocks past K read the next row's first
    // (or 0 past the end) and are taken out of the last step below.
    const int row0 = wave * T::kRowsPerCopy + lane / T::kStep;
    uint32_t voff = (uint32_t)row0 * row_bytes + step0 * T::kRowBytes +
                    ((lane & (T::kStep - 1)) ^ T::swizzle(row0)) * 16;
    auto copy = [&](int s) {
        const uint32_t to = base + s % T::kStages * T::kStage + wave * 1024;
#pragma unroll
        for (int c = 0; c < T::kCopies; ++c) {
            const int row = c * T::kCopyRows;
            const uint32_t from = (uint32_t)(row < T::BM ? row : row - T::BM) * row_bytes;
            copy16(row < T::BM ? arsrc : brsrc, voff + from, to + row * T::kRowBytes);
        }
        voff += T::kRowBytes;
    };

    // Scales: thread t takes rows t, t + kThreads, ...; LDS holds word w (blocks
    // 4w ..) of row r at [w][r].  Blocks past K count as 1.
    const uint8_t* srow[T::kScaleRows];
    uint4_t sreg[T::kScaleRows];
#pragma unroll
    for (int i = 0; i < T::kScaleRows; ++i) {
        const int r = min((int)threadIdx.x + i * T::kThreads, T::kRows - 1);
        srow[i] = r < T::BM ? a.as + (m0 + min(r, mrows - 1)) * KB
                            : a.bs + (n0 + min(r - T::BM, nrows - 1)) * KB;
    }
    auto load_scale_chunk = [&](int c) {
        const int kb = step0 * T::kStep + c * kScaleBlocks;
#pragma unroll
        for (int i = 0; i < T::kScaleRows; ++i)
            if (kb + kScaleBlocks <= KB) __builtin_memcpy(&sreg[i], srow[i] + kb, 16);   // any byte
    };
    auto store_scale_chunk = [&](int c) {
        const int kb = step0 * T::kStep + c * kScaleBlocks;
        char* at = lds + T::kStages * T::kStage + (c & 1) * T::kScales;
#pragma unroll
        for (int i = 0; i < T::kScaleRows; ++i) {
            const int r = threadIdx.x + i * T::kThreads;
            if (T::kRows % T::kThreads != 0 && r >= T::kRows) break;
            if (kb + kScaleBlocks <= KB) {
#pragma unroll
                for (int w = 0; w < 4; ++w) ((uint32_t*)at)[w * T::kRows + r] = sreg[i][w];
            } else {
#pragma unroll 1
                for (int b = 0; b < kScaleBlocks; ++b)
                    at[(b / 4 * T::kRows + r) * 4 + b % 4] = kb + b < KB ? srow[i][kb + b] : 127;
            }
        }
    };

    load_scale_chunk(0);
#pragma unroll
    for (int s = 0; s < T::kStages - 1; ++s)
        if (s < steps) copy(s);
    store_scale_chunk(0);

    const int wm = wave / T::kWavesN * T::WM, wn = wave % T::kWavesN * T::WN;
    const int half = lane >> 5, r31 = lane & 31;
    const int swz = T::swizzle(r31);
    float16_t acc[T::WM / 32][T::WN / 32] = {};
    for (int s = 0; s < steps; ++s) {
        const int sc = s / T::kScaleSteps, in_sc = s % T::kScaleSteps;
        // Copies of later steps stay in flight.
        if (s + T::kStages - 2 < steps) wait_copies<(T::kStages - 2) * T::kCopies>();
        else wait_copies<0>();
        if (s + T::kStages - 1 < steps) copy(s + T::kStages - 1);
        if (in_sc == 0 && s + T::kScaleSteps < steps) load_scale_chunk(sc + 1);
        const int left = KB - (step0 + s) * T::kStep;
        if (left < T::kStep) {                  // blocks past K: zero codes in A (scales are 1)
            for (int i = threadIdx.x; i < T::BM * T::kStep; i += T::kThreads) {
                const int r = i / T::kStep, chunk = i % T::kStep;
                if (chunk >= left)
                    *(uint4_t*)(lds + s % T::kStages * T::kStage + r * T::kRowBytes +
                                (chunk ^ T::swizzle(r)) * 16) = (uint4_t){0, 0, 0, 0};
            }
            wait_copies<0>();
        }

        const char* stage = lds + s % T::kStages * T::kStage;
        const uint32_t* scales = (const uint32_t*)(lds + T::kStages * T::kStage + (sc & 1) * T::kScales);
        uint32_t sa[T::WM / 32], sb[T::WN / 32];
        const int word = in_sc * 2 + half;
#pragma unroll
        for (int m = 0; m < T::WM / 32; ++m) sa[m] = scales[word * T::kRows + wm + 32 * m + r31];
#pragma unroll
        for (int n = 0; n < T::WN / 32; ++n)
            sb[n] = scales[word * T::kRows + T::BM + wn + 32 * n + r31];
        const char* ar = stage + (wm + r31) * T::kRowBytes;
        const char* br = stage + (T::BM + wn + r31) * T::kRowBytes;
        Fragments<T> f;
        f.load(ar, br, ((half * (T::kStep / 2)) ^ swz) * 16);
        Step<T, 0>::run(f, ar, br, swz, half, sa, sb, acc);
        if (in_sc == T::kScaleSteps - 1 && s + 1 < steps) store_scale_chunk(sc + 1);
    }
    wait_copies<0>();

    // Results: lane l holds row l % 32 of X and the weight rows 8 g + 4 half + i
    // in registers 4 g + i.  Each wave turns 32 rows at a time in its own LDS, so
    // that stores run along the rows of Y.
    const bool partial = a.part != nullptr;
    constexpr int kPitch = T::WN + 4;
    float* turn = (float*)(lds + wave * T::kWaveLds);
    static_assert(32 * kPitch * 4 <= T::kWaveLds, "a wave's 32 rows in fp32");
    typedef typename Out<DT>::type out_t;
    const int cols = (int)min((int64_t)T::WN, a.N - n0 - wn);
    constexpr int kVec = 16 / sizeof(out_t);
    const bool wide = a.N % kVec == 0 && (uintptr_t)a.Y % 16 == 0;
#pragma unroll
    for (int m = 0; m < T::WM / 32; ++m) {
#pragma unroll
        for (int n = 0; n < T::WN / 32; ++n)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *(float4_t*)&turn[r31 * kPitch + n * 32 + 8 * g + 4 * half] =
                    (float4_t){acc[m][n][4 * g], acc[m][n][4 * g + 1], acc[m][n][4 * g + 2],
                               acc[m][n][4 * g + 3]};
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int rows = min(32, mrows - wm - 32 * m);
        const int64_t out0 = (m0 + wm + 32 * m) * a.N + n0 + wn;
        if (partial) {
            float* p = a.part + (int64_t)slice * a.M * a.N + out0;
            if (a.N % 4 == 0) {
                for (int i = lane; i < 32 * T::WN / 4; i += kWave) {
                    const int r = i / (T::WN / 4), c = i % (T::WN / 4) * 4;
                    if (r < rows && c < cols)
                        *(float4_t*)(p + (int64_t)r * a.N + c) = *(const float4_t*)&turn[r * kPitch + c];
                }
            } else {
                for (int i = lane; i < 32 * T::WN; i += kWave) {
                    const int r = i / T::WN, c = i % T::WN;
                    if (r < rows && c < cols) p[(int64_t)r * a.N + c] = turn[r * kPitch + c];
                }
            }
        } else if (wide) {
            out_t* y = (out_t*)a.Y + out0;
#pragma unroll 2
            for (int i = lane; i < 32 * T::WN / kVec; i += kWave) {
                const int r = i / (T::WN / kVec), c = i % (T::WN / kVec) * kVec;
                out_t v[kVec];
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[j] = Out<DT>::make(turn[r * kPitch + c + j]);
                if (r < rows && c < cols) __builtin_memcpy(__builtin_assume_aligned(y + (int64_t)r * a.N + c, 16), v, 16);
            }
        } else {
            out_t* y = (out_t*)a.Y + out0;
            for (int i = lane; i < 32 * T::WN; i += kWave) {
                const int r = i / T::WN, c = i % T::WN;
                if (r < rows && c < cols) y[(int64_t)r * a.N + c] = Out<DT>::make(turn[r * kPitch + c]);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// Adds the K slices' partial sums in slice order; VEC outputs a thread.
template <DType DT, int VEC>
__global__ __launch_bounds__(256) void add_slices_kernel(const float* part, int slices, int64_t n,
                                                         typename Out<DT>::type* Y) {
    typedef typename Out<DT>::type out_t;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC; i < n;
         i += (int64_t)gridDim.x * 256 * VEC) {
        float sum[VEC] = {};
        for (int s = 0; s < slices; ++s) {
            float v[VEC];
            __builtin_memcpy(v, __builtin_assume_aligned(part + s * n + i, 4 * VEC), 4 * VEC);
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                sum[j] += v[j];
        }
        out_t o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = Out<DT>::make(sum[j]);
        __builtin_memcpy(__builtin_assume_aligned(Y + i, sizeof(out_t) * VEC), o, sizeof(o));
    }
}

template <DType DT>
void add_slices(const float* part, int slices, int64_t n, void* Y, hipStream_t stream) {
    typedef typename Out<DT>::type out_t;
    const bool wide = n % 4 == 0 && (uintptr_t)Y % (4 * sizeof(out_t)) == 0;
    const int64_t threads = wide ? n / 4 : n, blocks = (threads + 255) / 256;
    const unsigned grid = (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20);
    if (wide) add_slices_kernel<DT, 4><<<grid, 256, 0, stream>>>(part, slices, n, (out_t*)Y);
    else add_slices_kernel<DT, 1><<<grid, 256, 0, stream>>>(part, slices, n, (out_t*)Y);
}

typedef Tiling<256, 256, 128, 64, 2> Large;     // one block a CU
typedef Tiling<128, 128, 64, 64, 2> Medium;     // two
typedef Tiling<64, 64, 32, 32, 4> Small;        // two

// Tiling and K split, by how the output tiles fill 256 CUs.
//   Large against Medium: a round of 256 large tiles takes 5/3 of the time of a
//   round of 512 medium ones, for twice the work (K = 8192: 79 and 47 us); 4096
//   x 28672 552 against 658 us, 1000 x 8192 63 against 47 us.
//   Small: up to 64 rows of A (or B), where it wastes fewer rows and gives more
//   blocks: 16 x 14336 x 4096 9.4 us.
//   K slices: where the tiles are fewer than the 512 blocks that fit, as many
//   as fill them, of at least four steps (1024 columns): 200 x 4096 x 14336
//   52.1 us unsplit, 18.5 in 4 slices, 17.2 in 8 with twice the partial sums to
//   add (at most 4 for Medium); 1 x 4096 x 14336 35.1 and 9.7 us.
struct Choice {
    int tiling;         // 0 large, 1 medium, 2 small
    int slices, steps;
};
int64_t tile_count(int64_t M, int64_t N, int t) { return ((M + t - 1) / t) * ((N + t - 1) / t); }
Choice choose(int64_t M, int64_t N, int64_t K, bool split) {
    const int64_t kb = K / kBlock, total = (kb + 7) / 8;
    Choice c{1, 1, (int)total};
    if (M <= 64 || N <= 64) c.tiling = 2;
    else if ((tile_count(M, N, 256) + 255) / 256 * 5 <= (tile_count(M, N, 128) + 511) / 512 * 3)
        c.tiling = 0;
    if (c.tiling != 0 && split) {
        const int64_t tiles = tile_count(M, N, c.tiling == 1 ? 128 : 64);
        int64_t s = 512 / tiles, most = c.tiling == 1 ? 4 : 16;
        if (s > most) s = most;
        if (s > total / 4) s = total / 4;
        if (s > 1) {
            c.steps = (int)((total + s - 1) / s);
            c.slices = (int)((total + c.steps - 1) / c.steps);
        }
    }
    return c;
}

template <class T>
void launch(MatmulArgs a, DType dt, hipStream_t stream) {
    a.mt = (a.M + T::BM - 1) / T::BM;
    a.nt = (a.N + T::BN - 1) / T::BN;
    const int64_t blocks = (int64_t)a.mt * a.nt * a.slices;
    for (a.first = 0; a.first < blocks; a.first += kMaxGrid) {
        const unsigned grid = (unsigned)(blocks - a.first < kMaxGrid ? blocks - a.first : kMaxGrid);
        if (dt == kF16)
            matmul_kernel<kF16, T><<<grid, T::kThreads, 0, stream>>>(a);
        else if (dt == kBF16)
            matmul_kernel<kBF16, T><<<grid, T::kThreads, 0, stream>>>(a);
        else
            matmul_kernel<kF32, T><<<grid, T::kThreads, 0, stream>>>(a);
    }
}

}  // namespace

void launch_add_slices(const float* part, int slices, int64_t n, void* Y, DType dt,
                       hipStream_t stream) {
    if (dt == kF16) add_slices<kF16>(part, slices, n, Y, stream);
    else if (dt == kBF16) add_slices<kBF16>(part, slices, n, Y, stream);
    else add_slices<kF32>(part, slices, n, Y, stream);
}

size_t matmul_workspace(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0) return 0;
    const Choice c = choose(M, N, K, true);
    return c.slices > 1 ? (size_t)c.slices * M * N * sizeof(float) : 0;
}

hipError_t launch_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                         const uint8_t* b_codes, const uint8_t* b_scales, int64_t N, int64_t K,
                         void* Y, DType dt, float* part, hipStream_t stream) {
    const Choice c = choose(M, N, K, part != nullptr);
    MatmulArgs a{};
    a.ac = a_codes, a.as = a_scales, a.bc = b_codes, a.bs = b_scales, a.Y = Y;
    a.part = c.slices > 1 ? part : nullptr;
    a.M = (int)M, a.N = (int)N, a.K = (int)K;
    a.slices = c.slices, a.steps = c.steps;
    if (c.tiling == 0) launch<Large>(a, dt, stream);
    else if (c.tiling == 1) launch<Medium>(a, dt, stream);
    else launch<Small>(a, dt, stream);
    if (a.part) launch_add_slices(a.part, a.slices, (int64_t)a.M * a.N, Y, dt, stream);
    return hipGetLastError();
}

}  // namespace mxfp4
