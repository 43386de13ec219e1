// mxfp4_api.hip — the C ABI of include/mxfp4.h: host-side validation, device
// checks and dispatch to the kernels.
#include <hip/hip_runtime.h>

#include <mutex>
#include <string.h>

#include "mxfp4.h"
#include "mxfp4_act.h"
#include "mxfp4_launch.h"

namespace {

constexpr int64_t kMaxSize = (int64_t)1 << 24;

bool aligned(const void* p, uintptr_t a) { return (uintptr_t)p % a == 0; }

// A tensor's bytes, for the overlap rules.
struct Span {
    const void* p;
    uint64_t bytes;
};
bool overlap(Span a, Span b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + b.bytes && y < x + a.bytes;
}
template <int NO, int NI>
bool outputs_overlap(const Span (&out)[NO], const Span (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return true;
        for (const Span& s : in)
            if (overlap(out[i], s)) return true;
    }
    return false;
}

// Whether each device is gfx950, probed on first use.
constexpr int kMaxDevices = 64;
struct DeviceInfo {
    bool probed = false, ok = false;
};
DeviceInfo g_devices[kMaxDevices];
std::mutex g_mutex;

int check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return W4A16_ERR_DEVICE;
    std::lock_guard<std::mutex> lock(g_mutex);
    DeviceInfo& d = g_devices[dev];
    if (!d.probed) {
        hipDeviceProp_t prop;
        d.probed = true;
        d.ok = hipGetDeviceProperties(&prop, dev) == hipSuccess &&
               strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    }
    return d.ok ? W4A16_OK : W4A16_ERR_DEVICE;
}

int status_of(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_LAUNCH; }

bool bad_size(int64_t n) { return n < 0 || n > kMaxSize; }
bool bad_dtype(int dt, bool with_fp32) {
    return dt != MXFP4_FP16 && dt != MXFP4_BF16 && !(with_fp32 && dt == MXFP4_FP32);
}
// Takes MXFP4_FP32_ROWS out of a dtype; whether it was there.
bool take_fp32_rows(int& dt) {
    if (dt < MXFP4_FP32_ROWS) return false;
    dt -= MXFP4_FP32_ROWS;
    return true;
}
int elem_bytes(int dt) { return dt == MXFP4_FP32 ? 4 : 2; }
int check_k(int64_t K) {
    if (bad_size(K)) return W4A16_ERR_INVALID_ARG;
    return K % MXFP4_BLOCK ? W4A16_ERR_SHAPE : W4A16_OK;
}
// Bytes from the first to past the last element of rows x K, rows apart by stride.
uint64_t span_bytes(int64_t rows, int64_t K, int64_t stride, int bytes) {
    return rows > 0 && K > 0 ? ((uint64_t)(rows - 1) * stride + K) * bytes : 0;
}
uint64_t code_bytes(int64_t rows, int64_t K) { return (uint64_t)rows * (K / 2); }
uint64_t scale_bytes(int64_t rows, int64_t K) { return (uint64_t)rows * (K / MXFP4_BLOCK); }
// Strides stay far inside 64-bit offsets.
bool bad_stride(int64_t stride, int64_t K) { return stride < K || stride > ((int64_t)1 << 32); }

hipStream_t stream_of(void* s) { return (hipStream_t)s; }
mxfp4::DType dtype_of(int dt) { return (mxfp4::DType)dt; }

// workspace rules: NULL with 0 bytes, or aligned memory of at least `need`.
int check_workspace(const void* ws, size_t bytes, size_t need, uintptr_t align) {
    if (!ws) return bytes == 0 ? W4A16_OK : W4A16_ERR_INVALID_ARG;
    if (!aligned(ws, align)) return W4A16_ERR_MISALIGNED;
    return bytes < need ? W4A16_ERR_INVALID_ARG : W4A16_OK;
}

bool bad_activation(int act) { return act < MXFP4_ACT_NONE || act > MXFP4_ACT_SWIGLU; }
static_assert(MXFP4_ACT_RELU == (int)mxfp4::kRelu && MXFP4_ACT_SILU == (int)mxfp4::kSilu &&
                  MXFP4_ACT_GELU == (int)mxfp4::kGelu &&
                  MXFP4_ACT_GELU_TANH == (int)mxfp4::kGeluTanh &&
                  MXFP4_ACT_SWIGLU == (int)mxfp4::kSwiglu,
              "the activations' numbers");

}  // namespace

extern "C" {

int mxfp4_quantize(const void* X, int dtype, int64_t rows, int64_t K, int64_t x_stride,
                   uint8_t* codes, uint8_t* scales, void* stream) {
    if (bad_dtype(dtype, true) || bad_size(rows)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_k(K)) return st;
    if (bad_stride(x_stride, K)) return W4A16_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return W4A16_OK;
    if (!X || !codes || !scales) return W4A16_ERR_INVALID_ARG;
    const int eb = elem_bytes(dtype);
    if (!aligned(X, 16) || !aligned(codes, 16) || (rows > 1 && x_stride * eb % 16))
        return W4A16_ERR_MISALIGNED;
    const Span out[] = {{codes, code_bytes(rows, K)}, {scales, scale_bytes(rows, K)}};
    const Span in[] = {{X, span_bytes(rows, K, x_stride, eb)}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    return status_of(mxfp4::launch_quantize(X, dtype_of(dtype), rows, K, x_stride, codes, scales,
                                            stream_of(stream)));
}

int mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                     void* Y, int dtype, void* stream) {
    if (bad_dtype(dtype, true) || bad_size(rows)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_k(K)) return st;
    if (rows == 0 || K == 0) return W4A16_OK;
    if (!Y || !codes || !scales) return W4A16_ERR_INVALID_ARG;
    if (!aligned(Y, 16) || !aligned(codes, 16)) return W4A16_ERR_MISALIGNED;
    const Span out[] = {{Y, (uint64_t)rows * K * elem_bytes(dtype)}};
    const Span in[] = {{codes, code_bytes(rows, K)}, {scales, scale_bytes(rows, K)}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    return status_of(mxfp4::launch_dequantize(codes, scales, rows * K, Y, dtype_of(dtype),
                                              stream_of(stream)));
}

size_t mxfp4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (bad_size(M) || bad_size(N) || check_k(K)) return 0;
    return mxfp4::linear_workspace(M, N, K);
}

int mxfp4_linear(const void* X, int dtype, int64_t M, int64_t x_stride, const uint8_t* codes,
                 const uint8_t* scales, int64_t N, int64_t K, void* Y, void* workspace,
                 size_t workspace_bytes, void* stream) {
    if (bad_dtype(dtype, false) || bad_size(M) || bad_size(N)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_k(K)) return st;
    if (bad_stride(x_stride, K)) return W4A16_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return W4A16_OK;
    if (!Y || (K > 0 && (!X || !codes || !scales))) return W4A16_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(Y, 2) || (M > 1 && x_stride % 8))
        return W4A16_ERR_MISALIGNED;
    const size_t need = mxfp4_linear_workspace_bytes(M, N, K);
    if (const int st = check_workspace(workspace, workspace_bytes, need, 16)) return st;
    const Span out[] = {{Y, (uint64_t)M * N * 2}, {workspace, need}};
    const Span in[] = {{X, span_bytes(M, K, x_stride, 2)},
                       {codes, code_bytes(N, K)},
                       {scales, scale_bytes(N, K)}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    mxfp4::LinearArgs a{};
    a.X = (const uint16_t*)X;
    a.codes = codes;
    a.scales = scales;
    a.Y = (uint16_t*)Y;
    a.x_stride = x_stride;
    a.x_rows = a.R = (int)M;
    a.E = 1;
    a.N = (int)N;
    a.K = (int)K;
    return status_of(mxfp4::launch_linear(a, dtype_of(dtype), (float*)workspace,
                                          stream_of(stream)));
}

size_t mxfp4_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (bad_size(M) || bad_size(N) || check_k(K)) return 0;
    return mxfp4::matmul_workspace(M, N, K);
}

int mxfp4_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                 const uint8_t* b_codes, const uint8_t* b_scales, int64_t N, int64_t K,
                 void* Y, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (bad_dtype(dtype, true) || bad_size(M) || bad_size(N)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_k(K)) return st;
    if (M == 0 || N == 0) return W4A16_OK;
    if (!Y || (K > 0 && (!a_codes || !a_scales || !b_codes || !b_scales)))
        return W4A16_ERR_INVALID_ARG;
    const int eb = elem_bytes(dtype);
    if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(Y, eb))
        return W4A16_ERR_MISALIGNED;
    const size_t need = mxfp4_matmul_workspace_bytes(M, N, K);
    if (const int st = check_workspace(workspace, workspace_bytes, need, 16)) return st;
    const Span out[] = {{Y, (uint64_t)M * N * eb}, {workspace, need}};
    const Span in[] = {{a_codes, code_bytes(M, K)}, {a_scales, scale_bytes(M, K)},
                       {b_codes, code_bytes(N, K)}, {b_scales, scale_bytes(N, K)}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    return status_of(mxfp4::launch_matmul(a_codes, a_scales, M, b_codes, b_scales, N, K, Y,
                                          dtype_of(dtype), (float*)workspace, stream_of(stream)));
}

int moe_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t stride, int64_t k,
              int renormalize, int32_t* ids, float* weights, void* stream) {
    if (bad_dtype(dtype, true) || bad_size(T)) return W4A16_ERR_INVALID_ARG;
    if (E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > E || k > MOE_MAX_CHOICES ||
        bad_stride(stride, E))
        return W4A16_ERR_INVALID_ARG;
    if (T == 0) return W4A16_OK;
    if (!logits || !ids || !weights) return W4A16_ERR_INVALID_ARG;
    if (!aligned(logits, elem_bytes(dtype)) || !aligned(ids, 4) || !aligned(weights, 4))
        return W4A16_ERR_MISALIGNED;
    const Span out[] = {{ids, (uint64_t)T * k * 4}, {weights, (uint64_t)T * k * 4}};
    const Span in[] = {{logits, span_bytes(T, E, stride, elem_bytes(dtype))}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    return status_of(mxfp4::launch_route(logits, dtype_of(dtype), (int)T, (int)E, stride, (int)k,
                                         renormalize != 0, ids, weights, stream_of(stream)));
}

size_t moe_plan_workspace_bytes(int64_t T, int64_t k, int64_t E) {
    if (bad_size(T) || k < 1 || k > MOE_MAX_CHOICES || E < 1 || E > MOE_MAX_EXPERTS ||
        bad_size(T * k))
        return 0;
    const int64_t blocks = mxfp4::plan_blocks(T * k);
    return blocks > 1 ? (size_t)blocks * (E + 1) * 4 : 0;
}

int moe_plan(const int32_t* ids, int64_t T, int64_t k, int64_t E, int32_t* offsets,
             int32_t* tokens, int32_t* positions, void* workspace, size_t workspace_bytes,
             void* stream) {
    if (bad_size(T) || k < 1 || k > MOE_MAX_CHOICES || E < 1 || E > MOE_MAX_EXPERTS ||
        bad_size(T * k))
        return W4A16_ERR_INVALID_ARG;
    const size_t need = moe_plan_workspace_bytes(T, k, E);
    if (!offsets || (T > 0 && (!ids || !tokens || !positions)) || (need > 0 && !workspace))
        return W4A16_ERR_INVALID_ARG;
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(tokens, 4) || !aligned(positions, 4))
        return W4A16_ERR_MISALIGNED;
    if (const int st = check_workspace(workspace, workspace_bytes, need, 4)) return st;
    const uint64_t rb = (uint64_t)T * k * 4;
    const Span out[] = {{offsets, (uint64_t)(E + 1) * 4}, {tokens, rb}, {positions, rb},
                        {workspace, need}};
    const Span in[] = {{ids, rb}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    return status_of(mxfp4::launch_plan(ids, (int)(T * k), (int)k, (int)E, offsets, tokens,
                                        positions, (int*)workspace, stream_of(stream)));
}

int mxfp4_grouped_linear(const void* X, int dtype, int64_t x_rows, int64_t x_stride,
                         const int32_t* tokens, int64_t R, const uint8_t* codes,
                         const uint8_t* scales, const int32_t* offsets, int64_t E, int64_t N,
                         int64_t K, int swiglu, void* Y, void* stream) {
    const bool rows32 = take_fp32_rows(dtype);
    const int yb = rows32 ? 4 : 2;
    if (bad_dtype(dtype, false) || bad_size(x_rows) || bad_size(R) || bad_size(N) || E < 1 ||
        E > MOE_MAX_EXPERTS)
        return W4A16_ERR_INVALID_ARG;
    if (const int st = check_k(K)) return st;
    if (swiglu && N % 2) return W4A16_ERR_SHAPE;
    if (swiglu && rows32) return W4A16_ERR_INVALID_ARG;
    if (bad_stride(x_stride, K) || (!tokens && x_rows < R)) return W4A16_ERR_INVALID_ARG;
    if (R == 0 || N == 0) return W4A16_OK;
    if (!Y || !offsets || (K > 0 && ((x_rows > 0 && !X) || !codes || !scales)))
        return W4A16_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(Y, yb) || !aligned(tokens, 4) ||
        !aligned(offsets, 4) || (x_rows > 1 && x_stride % 8))
        return W4A16_ERR_MISALIGNED;
    const Span out[] = {{Y, (uint64_t)R * (swiglu ? N / 2 : N) * yb}};
    const Span in[] = {{X, span_bytes(x_rows, K, x_stride, 2)},
                       {tokens, (uint64_t)R * 4},
                       {codes, code_bytes(E * N, K)},
                       {scales, scale_bytes(E * N, K)},
                       {offsets, (uint64_t)(E + 1) * 4}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    mxfp4::LinearArgs a{};
    a.X = (const uint16_t*)X;
    a.tokens = tokens;
    a.codes = codes;
    a.scales = scales;
    a.offsets = offsets;
    a.Y = rows32 ? nullptr : (uint16_t*)Y;
    a.Y32 = rows32 ? (float*)Y : nullptr;
    a.x_stride = x_stride;
    a.x_rows = (int)x_rows;
    a.R = (int)R;
    a.E = (int)E;
    a.N = (int)N;
    a.K = (int)K;
    a.swiglu = swiglu != 0;
    return status_of(mxfp4::launch_linear(a, dtype_of(dtype), nullptr, stream_of(stream)));
}

int moe_combine(const void* Y, int dtype, int64_t R, int64_t N, const int32_t* positions,
                const float* weights, int64_t T, int64_t k, void* out_, void* stream) {
    const bool rows32 = take_fp32_rows(dtype);
    const int yb = rows32 ? 4 : 2;
    if (bad_dtype(dtype, false) || bad_size(R) || bad_size(N) || bad_size(T) || k < 1 ||
        k > MOE_MAX_CHOICES)
        return W4A16_ERR_INVALID_ARG;
    if (T == 0 || N == 0) return W4A16_OK;
    if (!out_ || !positions || !weights || (R > 0 && !Y)) return W4A16_ERR_INVALID_ARG;
    if (!aligned(Y, yb) || !aligned(out_, 2) || !aligned(positions, 4) || !aligned(weights, 4))
        return W4A16_ERR_MISALIGNED;
    const Span out[] = {{out_, (uint64_t)T * N * 2}};
    const Span in[] = {{Y, (uint64_t)R * N * yb}, {positions, (uint64_t)T * k * 4},
                       {weights, (uint64_t)T * k * 4}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    return status_of(mxfp4::launch_combine(Y, rows32, dtype_of(dtype), (int)R, (int)N, positions,
                                           weights, (int)T, (int)k, (uint16_t*)out_,
                                           stream_of(stream)));
}

size_t mxfp4_linear_act_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (bad_size(M) || bad_size(N) || check_k(K)) return 0;
    return mxfp4::linear_act_workspace(M, N, K);
}

int mxfp4_linear_act(const void* X, int dtype, int64_t M, int64_t x_stride, const uint8_t* codes,
                     const uint8_t* scales, int64_t N, int64_t K, const void* bias,
                     int activation, const void* residual, int64_t r_stride, void* Y, void* Z,
                     void* workspace, size_t workspace_bytes, void* stream) {
    if (bad_dtype(dtype, false) || bad_size(M) || bad_size(N) || bad_activation(activation))
        return W4A16_ERR_INVALID_ARG;
    if (const int st = check_k(K)) return st;
    const bool swiglu = activation == MXFP4_ACT_SWIGLU;
    if (swiglu && N % 2) return W4A16_ERR_SHAPE;
    const int64_t F = swiglu ? N / 2 : N;
    if (bad_stride(x_stride, K) || (residual && bad_stride(r_stride, F)))
        return W4A16_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return W4A16_OK;
    if (!Y || (K > 0 && (!X || !codes || !scales))) return W4A16_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(Y, 2) || !aligned(Z, 2) ||
        !aligned(bias, 2) || !aligned(residual, 2) || (M > 1 && x_stride % 8))
        return W4A16_ERR_MISALIGNED;
    const size_t need = mxfp4_linear_act_workspace_bytes(M, N, K);
    if (const int st = check_workspace(workspace, workspace_bytes, need, 16)) return st;
    const Span out[] = {{Y, (uint64_t)M * F * 2}, {Z, (uint64_t)M * N * 2}, {workspace, need}};
    const Span in[] = {{X, span_bytes(M, K, x_stride, 2)},
                       {codes, code_bytes(N, K)},
                       {scales, scale_bytes(N, K)},
                       {bias, (uint64_t)N * 2},
                       {residual, span_bytes(M, F, r_stride, 2)}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    mxfp4::LinearArgs a{};
    a.X = (const uint16_t*)X;
    a.codes = codes;
    a.scales = scales;
    a.Y = (uint16_t*)Y;
    a.x_stride = x_stride;
    a.x_rows = a.R = (int)M;
    a.E = 1;
    a.N = (int)N;
    a.K = (int)K;
    a.act = activation;
    a.bias = (const uint16_t*)bias;
    a.residual = (const uint16_t*)residual;
    a.r_stride = r_stride;
    a.Z = (uint16_t*)Z;
    return status_of(mxfp4::launch_linear_act(a, dtype_of(dtype), (float*)workspace,
                                              stream_of(stream)));
}

int mxfp4_grouped_linear_act(const void* X, int dtype, int64_t x_rows, int64_t x_stride,
                             const int32_t* tokens, int64_t R, const uint8_t* codes,
                             const uint8_t* scales, const int32_t* offsets, int64_t E, int64_t N,
                             int64_t K, const void* bias, int activation, void* Y, void* Z,
                             void* stream) {
    const bool rows32 = take_fp32_rows(dtype);
    const int yb = rows32 ? 4 : 2;
    if (bad_dtype(dtype, false) || bad_size(x_rows) || bad_size(R) || bad_size(N) || E < 1 ||
        E > MOE_MAX_EXPERTS || bad_activation(activation))
        return W4A16_ERR_INVALID_ARG;
    if (const int st = check_k(K)) return st;
    const bool swiglu = activation == MXFP4_ACT_SWIGLU;
    if (swiglu && N % 2) return W4A16_ERR_SHAPE;
    if (bad_stride(x_stride, K) || (!tokens && x_rows < R)) return W4A16_ERR_INVALID_ARG;
    if (R == 0 || N == 0) return W4A16_OK;
    if (!Y || !offsets || (K > 0 && ((x_rows > 0 && !X) || !codes || !scales)))
        return W4A16_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(Y, yb) || !aligned(tokens, 4) ||
        !aligned(offsets, 4) || !aligned(bias, 2) || !aligned(Z, 2) || (x_rows > 1 && x_stride % 8))
        return W4A16_ERR_MISALIGNED;
    const int64_t F = swiglu ? N / 2 : N;
    const Span out[] = {{Y, (uint64_t)R * F * yb}, {Z, (uint64_t)R * N * 2}};
    const Span in[] = {{X, span_bytes(x_rows, K, x_stride, 2)},
                       {tokens, (uint64_t)R * 4},
                       {codes, code_bytes(E * N, K)},
                       {scales, scale_bytes(E * N, K)},
                       {offsets, (uint64_t)(E + 1) * 4},
                       {bias, (uint64_t)E * N * 2}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    mxfp4::LinearArgs a{};
    a.X = (const uint16_t*)X;
    a.tokens = tokens;
    a.codes = codes;
    a.scales = scales;
    a.offsets = offsets;
    a.Y = rows32 ? nullptr : (uint16_t*)Y;
    a.Y32 = rows32 ? (float*)Y : nullptr;
    a.x_stride = x_stride;
    a.x_rows = (int)x_rows;
    a.R = (int)R;
    a.E = (int)E;
    a.N = (int)N;
    a.K = (int)K;
    a.act = activation;
    a.bias = (const uint16_t*)bias;
    a.Z = (uint16_t*)Z;
    return status_of(mxfp4::launch_linear_act(a, dtype_of(dtype), nullptr, stream_of(stream)));
}

size_t mxfp4_activation_grad_workspace_bytes(int64_t R, int64_t N, int64_t E) {
    if (bad_size(R) || bad_size(N) || E < 0 || E > MOE_MAX_EXPERTS || R == 0 || N == 0) return 0;
    return mxfp4::activation_grad_workspace(R, N, E > 0 ? E : 1, E > 0);
}

int mxfp4_activation_grad(const void* dY, int dtype, int64_t R, int64_t y_stride, const void* Z,
                          int64_t z_stride, int64_t N, int activation, const int32_t* offsets,
                          int64_t E, void* dZ, float* dbias, void* workspace,
                          size_t workspace_bytes, void* stream) {
    if (bad_dtype(dtype, false) || bad_size(R) || bad_size(N) || bad_activation(activation))
        return W4A16_ERR_INVALID_ARG;
    if (offsets ? E < 1 || E > MOE_MAX_EXPERTS : E != 0) return W4A16_ERR_INVALID_ARG;
    const bool swiglu = activation == MXFP4_ACT_SWIGLU;
    if (swiglu && N % 2) return W4A16_ERR_SHAPE;
    const int64_t F = swiglu ? N / 2 : N;
    if (bad_stride(y_stride, F) || bad_stride(z_stride, N)) return W4A16_ERR_INVALID_ARG;
    if (N == 0 || (R == 0 && !dbias)) return W4A16_OK;
    const size_t need = dbias ? mxfp4_activation_grad_workspace_bytes(R, N, E) : 0;
    if ((R > 0 && (!dY || !Z || !dZ)) || (need > 0 && !workspace)) return W4A16_ERR_INVALID_ARG;
    if (!aligned(dY, 2) || !aligned(Z, 2) || !aligned(dZ, 2) || !aligned(dbias, 4) ||
        !aligned(offsets, 4))
        return W4A16_ERR_MISALIGNED;
    if (const int st = check_workspace(workspace, workspace_bytes, need, 4)) return st;
    const Span out[] = {{dZ, (uint64_t)R * N * 2},
                        {dbias, (uint64_t)(E > 0 ? E : 1) * N * 4},
                        {workspace, need}};
    const Span in[] = {{dY, span_bytes(R, F, y_stride, 2)},
                       {Z, span_bytes(R, N, z_stride, 2)},
                       {offsets, (uint64_t)(E + 1) * 4}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    mxfp4::ActGradArgs a{};
    a.dY = (const uint16_t*)dY;
    a.Z = (const uint16_t*)Z;
    a.y_stride = y_stride;
    a.z_stride = z_stride;
    a.dZ = (uint16_t*)dZ;
    a.dbias = dbias;
    a.offsets = offsets;
    a.R = (int)R;
    a.N = (int)N;
    a.E = E > 0 ? (int)E : 1;
    a.act = activation;
    a.part = (float*)workspace;
    return status_of(mxfp4::launch_activation_grad(a, dtype_of(dtype), stream_of(stream)));
}

size_t mxfp4_linear_grad_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (bad_size(M) || bad_size(N) || check_k(K)) return 0;
    return mxfp4::grad_workspace(M, N, K);
}

int mxfp4_linear_grad(const void* dY, int dtype, int64_t M, int64_t y_stride,
                      const uint8_t* codes, const uint8_t* scales, int64_t N, int64_t K, void* dX,
                      void* workspace, size_t workspace_bytes, void* stream) {
    if (bad_dtype(dtype, false) || bad_size(M) || bad_size(N)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_k(K)) return st;
    if (bad_stride(y_stride, N)) return W4A16_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return W4A16_OK;
    if (!dX || (N > 0 && (!dY || !codes || !scales))) return W4A16_ERR_INVALID_ARG;
    if (!aligned(dY, 2) || !aligned(codes, 16) || !aligned(dX, 16)) return W4A16_ERR_MISALIGNED;
    const size_t need = mxfp4_linear_grad_workspace_bytes(M, N, K);
    if (const int st = check_workspace(workspace, workspace_bytes, need, 16)) return st;
    const Span out[] = {{dX, (uint64_t)M * K * 2}, {workspace, need}};
    const Span in[] = {{dY, span_bytes(M, N, y_stride, 2)},
                       {codes, code_bytes(N, K)},
                       {scales, scale_bytes(N, K)}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    mxfp4::GradArgs a{};
    a.dY = (const uint16_t*)dY;
    a.codes = codes;
    a.scales = scales;
    a.dX = (uint16_t*)dX;
    a.y_stride = y_stride;
    a.R = (int)M;
    a.E = 1;
    a.N = (int)N;
    a.K = (int)K;
    return status_of(mxfp4::launch_grad(a, dtype_of(dtype), (float*)workspace, stream_of(stream)));
}

int mxfp4_grouped_linear_grad(const void* dY, int dtype, int64_t R, int64_t y_stride,
                              const uint8_t* codes, const uint8_t* scales, const int32_t* offsets,
                              int64_t E, int64_t N, int64_t K, void* dX, void* stream) {
    const bool rows32 = take_fp32_rows(dtype);
    if (bad_dtype(dtype, false) || bad_size(R) || bad_size(N) || E < 1 || E > MOE_MAX_EXPERTS)
        return W4A16_ERR_INVALID_ARG;
    if (const int st = check_k(K)) return st;
    if (bad_stride(y_stride, N)) return W4A16_ERR_INVALID_ARG;
    if (R == 0 || K == 0) return W4A16_OK;
    if (!dX || !offsets || (N > 0 && (!dY || !codes || !scales))) return W4A16_ERR_INVALID_ARG;
    if (!aligned(dY, 2) || !aligned(codes, 16) || !aligned(dX, 16) || !aligned(offsets, 4))
        return W4A16_ERR_MISALIGNED;
    const Span out[] = {{dX, (uint64_t)R * K * (rows32 ? 4 : 2)}};
    const Span in[] = {{dY, span_bytes(R, N, y_stride, 2)},
                       {codes, code_bytes(E * N, K)},
                       {scales, scale_bytes(E * N, K)},
                       {offsets, (uint64_t)(E + 1) * 4}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    mxfp4::GradArgs a{};
    a.dY = (const uint16_t*)dY;
    a.codes = codes;
    a.scales = scales;
    a.offsets = offsets;
    a.dX = rows32 ? nullptr : (uint16_t*)dX;
    a.dX32 = rows32 ? (float*)dX : nullptr;
    a.y_stride = y_stride;
    a.R = (int)R;
    a.E = (int)E;
    a.N = (int)N;
    a.K = (int)K;
    return status_of(mxfp4::launch_grad(a, dtype_of(dtype), nullptr, stream_of(stream)));
}

size_t moe_balance_workspace_bytes(int64_t T, int64_t E, int64_t k) {
    if (bad_size(T) || E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > MOE_MAX_CHOICES) return 0;
    return mxfp4::balance_workspace(T, E);
}

int moe_balance(const void* logits, int dtype, int64_t T, int64_t E, int64_t stride,
                const int32_t* ids, int64_t k, float* loss, int32_t* counts, void* workspace,
                size_t workspace_bytes, void* stream) {
    if (bad_dtype(dtype, true) || bad_size(T)) return W4A16_ERR_INVALID_ARG;
    if (E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > MOE_MAX_CHOICES || bad_stride(stride, E))
        return W4A16_ERR_INVALID_ARG;
    const size_t need = moe_balance_workspace_bytes(T, E, k);
    if (!loss || !counts || (T > 0 && (!logits || !ids)) || (need > 0 && !workspace))
        return W4A16_ERR_INVALID_ARG;
    if (!aligned(logits, elem_bytes(dtype)) || !aligned(ids, 4) || !aligned(loss, 4) ||
        !aligned(counts, 4))
        return W4A16_ERR_MISALIGNED;
    if (const int st = check_workspace(workspace, workspace_bytes, need, 4)) return st;
    const Span out[] = {{loss, 4}, {counts, (uint64_t)(E + 1) * 4}, {workspace, need}};
    const Span in[] = {{logits, span_bytes(T, E, stride, elem_bytes(dtype))},
                       {ids, (uint64_t)T * k * 4}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    return status_of(mxfp4::launch_balance(logits, dtype_of(dtype), (int)T, (int)E, stride, ids,
                                           (int)k, loss, counts, workspace, stream_of(stream)));
}

int moe_route_grad(const void* logits, int dtype, int64_t T, int64_t E, int64_t stride,
                   const int32_t* ids, int64_t k, const float* dweights, int renormalize,
                   const int32_t* counts, const float* dloss, void* dlogits, void* stream) {
    if (bad_dtype(dtype, true) || bad_size(T)) return W4A16_ERR_INVALID_ARG;
    if (E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > MOE_MAX_CHOICES || bad_stride(stride, E))
        return W4A16_ERR_INVALID_ARG;
    if (T == 0) return W4A16_OK;
    if (!logits || !dlogits || (!dweights && !counts) || (dweights && !ids) || (counts && !dloss))
        return W4A16_ERR_INVALID_ARG;
    const int eb = elem_bytes(dtype);
    if (!aligned(logits, eb) || !aligned(dlogits, eb) || !aligned(ids, 4) ||
        !aligned(dweights, 4) || !aligned(counts, 4) || !aligned(dloss, 4))
        return W4A16_ERR_MISALIGNED;
    const Span out[] = {{dlogits, (uint64_t)T * E * eb}};
    const Span in[] = {{logits, span_bytes(T, E, stride, eb)},
                       {ids, (uint64_t)T * k * 4},
                       {dweights, (uint64_t)T * k * 4},
                       {counts, (uint64_t)(E + 1) * 4},
                       {dloss, 4}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    const mxfp4::RouteGradArgs a{logits,  ids,    dweights, counts, dloss, dlogits,
                                 stride,  (int)T, (int)E,   (int)k, renormalize != 0};
    return status_of(mxfp4::launch_route_grad(a, dtype_of(dtype), stream_of(stream)));
}

int moe_combine_grad(const void* dout, int dtype, int64_t T, int64_t N, const void* Y, int64_t R,
                     const int32_t* tokens, const int32_t* positions, const float* weights,
                     int64_t k, void* dY, float* dweights, void* stream) {
    const bool rows32 = take_fp32_rows(dtype);
    const int yb = rows32 ? 4 : 2;
    if (bad_dtype(dtype, false) || bad_size(R) || bad_size(N) || bad_size(T) || k < 1 ||
        k > MOE_MAX_CHOICES)
        return W4A16_ERR_INVALID_ARG;
    if (T == 0 && (R == 0 || N == 0)) return W4A16_OK;
    if ((T > 0 && (!positions || !weights || !dweights)) || (T > 0 && N > 0 && !dout) ||
        (R > 0 && !tokens) || (R > 0 && N > 0 && (!Y || !dY)))
        return W4A16_ERR_INVALID_ARG;
    if (!aligned(dout, 2) || !aligned(Y, yb) || !aligned(dY, 2) || !aligned(tokens, 4) ||
        !aligned(positions, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
        return W4A16_ERR_MISALIGNED;
    const uint64_t choices = (uint64_t)T * k * 4;
    const Span out[] = {{dY, (uint64_t)R * N * 2}, {dweights, choices}};
    const Span in[] = {{dout, (uint64_t)T * N * 2}, {Y, (uint64_t)R * N * yb},
                       {tokens, (uint64_t)R * 4},   {positions, choices},
                       {weights, choices}};
    if (outputs_overlap(out, in)) return W4A16_ERR_INVALID_ARG;
    if (const int st = check_device()) return st;
    return status_of(mxfp4::launch_combine_grad((const uint16_t*)dout, Y, rows32, dtype_of(dtype),
                                                (int)R, (int)N, tokens, positions, weights,
                                                (int)T, (int)k, (uint16_t*)dY, dweights,
                                                stream_of(stream)));
}

const char* mxfp4_status_string(int status) {
    switch (status) {
        case W4A16_OK: return "ok";
        case W4A16_ERR_INVALID_ARG: return "invalid argument";
        case W4A16_ERR_SHAPE: return "bad shape";
        case W4A16_ERR_MISALIGNED: return "misaligned pointer or stride";
        case W4A16_ERR_DEVICE: return "no gfx950 device";
        case W4A16_ERR_LAUNCH: return "launch failed";
        default: return "unknown status";
    }
}

}  // extern "C"
