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
    // The epilogue (kernels with one only): Y = act(product + bias) + residual.
    bool epilogue;
    int act;                    // mxfp4_act.h's; kSwiglu with swiglu
    const uint16_t* bias;       // [E, N] or NULL
    const uint16_t* residual;   // [R, columns of Y], rows r_stride apart, or NULL
    int64_t r_stride;
    uint16_t* Z;                // product + bias [R, N], or NULL
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
// The same with the epilogue; dense with its own size of part.
size_t linear_act_workspace(int64_t M, int64_t N, int64_t K);
hipError_t launch_linear_act(LinearArgs a, DType dt, float* part, hipStream_t stream);
// Few rows per weight matrix: weights straight into matrix-core registers.
hipError_t launch_stream(const LinearArgs& a, DType dt, hipStream_t stream);

// One row with the epilogue, where X fits LDS and the weights are many.
bool gemv_fits(int64_t R, int64_t N, int64_t K);
hipError_t launch_gemv(const LinearArgs& a, DType dt, hipStream_t stream);
// The epilogue of the K slices' partial sums [slices][R][N], added in slice order.
hipError_t launch_finish(const LinearArgs& a, DType dt, hipStream_t stream);

// dZ [R, N] = dY act'(Z) and dbias [E, N] (NULL: not wanted), the sum of its rows by
// expert.  part: activation_grad_workspace bytes, NULL where that is 0.
struct ActGradArgs {
    const uint16_t *dY, *Z;
    int64_t y_stride, z_stride;
    uint16_t* dZ;
    float* dbias;
    const int* offsets;         // NULL: all R rows belong to expert 0
    int R, N, E, act;
    float* part;
};
size_t activation_grad_workspace(int64_t R, int64_t N, int64_t E, bool grouped);
hipError_t launch_activation_grad(ActGradArgs a, DType dt, hipStream_t stream);

// The product with the untransposed weights: dX[r, k] = sum_n dY[r, n] W[n, k].
struct GradArgs {
    const uint16_t* dY;
    const uint8_t* codes;
    const uint8_t* scales;
    const int* offsets;         // NULL: all R rows belong to expert 0
    uint16_t* dX;               // rounded to dY's type, or NULL:
    float* dX32;
    int64_t y_stride;
    int R, E, N, K;
    // Set by launch_grad.
    float* part;                // fp32 partial sums [slices][R][K], or dX32, or NULL
    int slices, steps;          // N slices, steps of a slice
    int64_t first;              // first block of this launch
};
size_t grad_workspace(int64_t M, int64_t N, int64_t K);
hipError_t launch_grad(GradArgs a, DType dt, float* part, hipStream_t stream);

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
// Gradient of the weighted sum.  Y: fp32 (rows32) or dt.
hipError_t launch_combine_grad(const uint16_t* dout, const void* Y, bool rows32, DType dt, int R,
                               int N, const int* tokens, const int* positions,
                               const float* weights, int T, int k, uint16_t* dY, float* dweights,
                               hipStream_t stream);

// Balance loss: part holds balance_workspace bytes.
size_t balance_workspace(int64_t T, int64_t E);
hipError_t launch_balance(const void* logits, DType dt, int T, int E, int64_t stride,
                          const int* ids, int k, float* loss, int* counts, void* part,
                          hipStream_t stream);
// Gradient of the routing weights (dweights, or NULL) and of the loss (counts, or NULL).
struct RouteGradArgs {
    const void* logits;
    const int* ids;
    const float* dweights;
    const int* counts;
    const float* dloss;
    void* dlogits;
    int64_t stride;
    int T, E, k;
    bool renormalize;
};
hipError_t launch_route_grad(const RouteGradArgs& a, DType dt, hipStream_t stream);

}  // namespace mxfp4
