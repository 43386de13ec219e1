// mxfp4_device.h — device-side helpers shared by the MXFP4 and expert kernels
// (gfx950 / CDNA4, wave64).  Private to libmxfp4.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxfp4 {

constexpr int kBlock = 32;       // columns per scale
constexpr int kWave = 64;

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf162_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf168_t __attribute__((ext_vector_type(8)));
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef float float16_t __attribute__((ext_vector_type(16)));
typedef int int8_t_ __attribute__((ext_vector_type(8)));
typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));

// 16-bit storage types by tag; arithmetic is always in fp32.
struct F16 {
    typedef uint16_t type;
    typedef half8_t vec8;
    static __device__ __forceinline__ float load(uint16_t b) {
        return (float)__builtin_bit_cast(_Float16, b);
    }
    static __device__ __forceinline__ uint16_t store(float f) {      // RNE
        return __builtin_bit_cast(uint16_t, (_Float16)f);
    }
    static __device__ __forceinline__ float4_t mfma16(vec8 a, vec8 b, float4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float16_t mfma32(vec8 a, vec8 b, float16_t c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};
struct BF16 {
    typedef uint16_t type;
    typedef bf168_t vec8;
    static __device__ __forceinline__ float load(uint16_t b) {
        return __builtin_bit_cast(float, (uint32_t)b << 16);
    }
    static __device__ __forceinline__ uint16_t store(float f) {      // RNE
        return __builtin_bit_cast(uint16_t, (__bf16)f);
    }
    static __device__ __forceinline__ float4_t mfma16(vec8 a, vec8 b, float4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float16_t mfma32(vec8 a, vec8 b, float16_t c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

// 2^(byte - 127), NaN for 255: the byte is the fp32 exponent field, with two
// exceptions (0 is the subnormal 2^-127, 255 needs a mantissa bit).
__device__ __forceinline__ float scale_value(uint32_t byte) {
    const uint32_t bits = byte << 23;
    return __builtin_bit_cast(float, byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : bits);
}

// Eight codes (one word, column i in bits 4i..4i+3) times the scale, as eight
// 16-bit values.  bf16 is exact for scale bytes up to 252 (values have two
// mantissa bits, down to the subnormal 2^-128 and up to 6 * 2^125; bytes 253 and
// 254 give values of 2^128 and more, which pass fp32 too: quarter8 below); fp16
// is exact for scale bytes kF16ScaleMin to kF16ScaleMax (0.5 * 2^-23 = 2^-24 up
// to 6 * 2^13 = 49152).
__device__ __forceinline__ bf168_t values8(uint32_t w, float s, BF16) {
    bf168_t v;
    const bf162_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    const bf162_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    const bf162_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    const bf162_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    v = (bf168_t){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    return v;
}
__device__ __forceinline__ half8_t values8(uint32_t w, float s, F16) {
    const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0);
    const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1);
    const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2);
    const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3);
    return (half8_t){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
constexpr uint32_t kF16ScaleMin = 104, kF16ScaleMax = 140;
__device__ __forceinline__ bool f16_scale_ok(uint32_t byte) {
    return byte - kF16ScaleMin <= kF16ScaleMax - kF16ScaleMin;
}

// A quarter of the values, exact in bf16 for every scale (2^-130 to 1.5 * 2^127):
// a wave that met a scale byte of kFarScale or more sums its products again as
// quarters and takes the sums times four.  Powers of two: only sums below 2^-124
// can lose a bit (2^-148).
constexpr uint32_t kFarScale = 253;
__device__ __forceinline__ bf168_t quarter8(uint32_t w, uint32_t byte) {
    bf168_t v = values8(w, scale_value(byte == 255 ? 255 : byte < 2 ? 0 : byte - 2), BF16());
    if (byte < 2) {                     // 2^-127 is the least scale
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (__bf16)((float)v[i] * (byte == 0 ? 0.25f : 0.5f));
    }
    return v;
}

// fp16 values as the exact sum of two bf16 values (11 significant bits = 8 +
// 3), for weights outside fp16's range: hi is x cut to 8 bits, lo the rest.
// An infinity has lo = 0, a NaN stays in both.
__device__ __forceinline__ void split_bf16(half8_t x, bf168_t& hi, bf168_t& lo) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = (float)x[i];
        const uint32_t bits = __builtin_bit_cast(uint32_t, f);
        const float h = __builtin_bit_cast(float, bits & 0xFFFF0000u);
        const float l = f != f ? f : (bits & 0x7F800000u) == 0x7F800000u ? 0.0f : f - h;
        hi[i] = (__bf16)h;
        lo[i] = (__bf16)l;
    }
}

// Largest value over the lanes l ^ 1 and l ^ 2 (groups of four lanes).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    const uint32_t a = __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);   // [1,0,3,2]
    v = max(v, a);
    const uint32_t b = __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);   // [2,3,0,1]
    return max(v, b);
}

// ---- Row groups of the expert product.
// The rows are cut into E + 2 groups: those before offsets[0], each expert's
// offsets[e] .. offsets[e+1], and those from offsets[E] on.  Every group is
// cut into tiles of `bm` rows, numbered by group, then row.  A grid of
// tile_slots(R, E, bm) slots covers every assignment of R rows, since
// sum ceil(r_g / bm) <= R / bm + the number of groups with a row.
__host__ __device__ inline int64_t tile_slots(int64_t R, int64_t E, int bm) {
    return R / bm + (E + 2 < R ? E + 2 : R);
}

struct Tile {
    int expert;      // -1: rows of no expert
    int row0;        // first row of the tile
    int rows;        // rows in it (1 .. bm); 0: no tile in this slot
};

// Tiles of 64 groups, lane l holding group base + l.  An offset counts as at
// least 0 and the ones before it, at most R: whatever the offsets hold, the
// groups are disjoint and cover the rows.
struct Groups {
    int lo, hi;      // rows of this lane's group
    int first;       // tiles of the earlier lanes' groups
    int count;       // tiles of all 64
    int end;         // where the last of them ends
};
__device__ __forceinline__ Groups scan_groups(const int* offsets, int E, int R, int bm, int base,
                                              int from) {
    const int lane = threadIdx.x & (kWave - 1), g = base + lane;
    Groups w;
    w.hi = g <= E ? min(max(offsets[g], from), R) : R;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int up = __shfl_up(w.hi, d);
        if (lane >= d) w.hi = max(w.hi, up);
    }
    w.lo = __shfl_up(w.hi, 1);
    if (lane == 0) w.lo = from;
    w.end = __builtin_amdgcn_readlane(w.hi, kWave - 1);
    const int tiles = (w.hi - w.lo + bm - 1) / bm;
    int sum = tiles;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int up = __shfl_up(sum, d);
        if (lane >= d) sum += up;
    }
    w.first = sum - tiles;
    w.count = __builtin_amdgcn_readlane(sum, kWave - 1);
    return w;
}

// Tiles in use, found by every wave for itself.
__device__ __forceinline__ int count_tiles(const int* offsets, int E, int R, int bm) {
    int n = 0, from = 0;
    for (int base = 0; base <= E + 1; base += kWave) {
        const Groups w = scan_groups(offsets, E, R, bm, base, from);
        n += w.count;
        from = w.end;
    }
    return n;
}

// Tile of a slot.
__device__ __forceinline__ Tile find_tile(const int* offsets, int E, int R, int bm, int slot) {
    int before = 0, from = 0;
    for (int base = 0; base <= E + 1; base += kWave) {
        const Groups w = scan_groups(offsets, E, R, bm, base, from);
        const int first = before + w.first;
        const int tiles = (w.hi - w.lo + bm - 1) / bm;
        const uint64_t hit = __ballot(slot >= first && slot < first + tiles);
        if (hit != 0) {
            const int src = __builtin_ctzll(hit);
            Tile t;
            t.expert = base + src - 1 < E ? base + src - 1 : -1;
            const int r0 = __builtin_amdgcn_readlane(w.lo, src);
            const int r1 = __builtin_amdgcn_readlane(w.hi, src);
            t.row0 = r0 + (slot - __builtin_amdgcn_readlane(first, src)) * bm;
            t.rows = min(bm, r1 - t.row0);
            return t;
        }
        before += w.count;
        from = w.end;
    }
    return Tile{-1, 0, 0};
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

}  // namespace mxfp4
