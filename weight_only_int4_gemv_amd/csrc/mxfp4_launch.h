// mxfp4_launch.h — host-side launchers of the MXFP4 and expert kernels
// (private).  Shapes, alignment and sizes are validated by the C ABI
// (mxfp4_api.hip) before any of these is called; no output is empty.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxfp4 {

enum DType { kF16 = 0, kBF16 = 1, kF32 = 2 };

hipError_t launch_quantize(const void* X, DType dt, int64_t rows, int64_t K, int64_t stride,
                           uint8_t* codes, uint8_t* scales, hipStream_t stream);
hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t n, void* Y,
                             DType dt, hipStream_t stream);

// The weight-only product.  Dense: offsets NULL, E = 1, x_rows = R = M.
struct LinearArgs {
    const uint16_t* X;
    const int* tokens;          // NULL: row r of X
    const uint8_t* codes;
    const uint8_t* scales;
    const int* offsets;         // NULL: all R rows belong to expert 0
    uint16_t* Y;                // rounded to X's type, or NULL:
    float* Y32;                 // the rows in fp32 (not with swiglu)
    int64_t x_stride;
    int x_rows, R, E;
    int N;                      // weight rows per expert
    int K;
    int swiglu;                 // Y has N / 2 columns
    // Set by launch_linear.
    float* part;                // fp32 partial sums [slices][R][N], or Y32, or NULL
    int slices, steps;          // K slices, steps of a slice
    int mt, nt;                 // row tiles (dense), column blocks
    int64_t first;              // first block of this launch
};
// Grid of `slots` row tiles by nblocks column blocks: slot = z * gridDim.y + y
// (slots past the last tile do nothing).
inline dim3 slot_grid(int nblocks, int64_t slots) {
    const int64_t y = slots < 32768 ? slots : 32768;
    return dim3((unsigned)nblocks, (unsigned)y, (unsigned)((slots + y - 1) / y));
}
constexpr int64_t kMaxGrid = (int64_t)1 << 22;      // blocks of a launch (threads stay below 2^32)

// The weight-only product by the kernel that suits its sizes.  part:
// linear_workspace bytes for the partial sums of K slices, or NULL for no split.
size_t linear_workspace(int64_t M, int64_t N, int64_t K);
hipError_t launch_linear(LinearArgs a, DType dt, float* part, hipStream_t stream);
// Few rows per weight matrix: weights straight into matrix-core registers.
hipError_t launch_stream(const LinearArgs& a, DType dt, hipStream_t stream);

// Y = the K slices' partial sums [slices][n], added in slice order.
void launch_add_slices(const float* part, int slices, int64_t n, void* Y, DType dt,
                       hipStream_t stream);

// Product of two MXFP4 matrices.  part: matmul_workspace bytes for the partial
// sums of K slices, or NULL for no split.
size_t matmul_workspace(int64_t M, int64_t N, int64_t K);
hipError_t launch_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                         const uint8_t* b_codes, const uint8_t* b_scales, int64_t N, int64_t K,
                         void* Y, DType dt, float* part, hipStream_t stream);

hipError_t launch_route(const void* logits, DType dt, int T, int E, int64_t stride, int k,
                        bool renormalize, int* ids, float* weights, hipStream_t stream);
int64_t plan_blocks(int64_t R);          // blocks of choices; one needs no workspace
hipError_t launch_plan(const int* ids, int R, int k, int E, int* offsets, int* tokens,
                       int* positions, int* counts, hipStream_t stream);
// Y: fp32 (rows32) or dt.
hipError_t launch_combine(const void* Y, bool rows32, DType dt, int R, int N, const int* positions,
                          const float* weights, int T, int k, uint16_t* out, hipStream_t stream);

}  // namespace mxfp4
