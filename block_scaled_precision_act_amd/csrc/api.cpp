// api.cpp - the C ABI of libmxgemm (see include/mxgemm.h): argument checks on
// the host, then one launcher per call.  Nothing here allocates, synchronizes
// or keeps per-call state; the only state is a per-device "is this a gfx950"
// cache filled on first use.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "../../include/mxgemm.h"
#include "launch.hpp"

#define MX_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr int kAbiVersion = 1;
constexpr int kMaxDevices = 64;
int g_device_ok[kMaxDevices];  // 0 unknown, 1 gfx950, 2 other

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mx_status check_device() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return MX_ERROR_DEVICE;
    if (dev < kMaxDevices && g_device_ok[dev] != 0) return g_device_ok[dev] == 1 ? MX_SUCCESS : MX_ERROR_DEVICE;
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MX_ERROR_DEVICE;
    const bool ok = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < kMaxDevices) g_device_ok[dev] = ok ? 1 : 2;
    return ok ? MX_SUCCESS : MX_ERROR_DEVICE;
}

mx_status launched(hipError_t e) { return e == hipSuccess ? MX_SUCCESS : MX_ERROR_LAUNCH; }

// rows >= 0, 0 < K <= 2^31-1, K % kmod == 0, rows * K fits comfortably in int64
mx_status check_rows(int64_t rows, int64_t K, int64_t kmod) {
    if (rows < 0) return MX_ERROR_INVALID_VALUE;
    if (K <= 0 || K > INT32_MAX || K % kmod != 0) return MX_ERROR_UNSUPPORTED_SHAPE;
    if (rows > (INT64_C(1) << 40) / K) return MX_ERROR_UNSUPPORTED_SHAPE;
    return MX_SUCCESS;
}

mx_status check_gemm(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0) return MX_ERROR_INVALID_VALUE;
    if (K <= 0 || K % 128 != 0 || K > INT32_MAX) return MX_ERROR_UNSUPPORTED_SHAPE;
    if (M > INT32_MAX || N > INT32_MAX) return MX_ERROR_UNSUPPORTED_SHAPE;
    // 256 x 256 output tiles must fit one 1-D grid
    if (((M + 255) / 256) * ((N + 255) / 256) > INT32_MAX) return MX_ERROR_UNSUPPORTED_SHAPE;
    if (M > (INT64_C(1) << 40) / K || N > (INT64_C(1) << 40) / K) return MX_ERROR_UNSUPPORTED_SHAPE;
    return MX_SUCCESS;
}

}  // namespace

MX_API int mx_abi_version(void) { return kAbiVersion; }

MX_API const char* mx_status_string(mx_status status) {
    switch (status) {
        case MX_SUCCESS: return "MX_SUCCESS";
        case MX_ERROR_INVALID_VALUE: return "MX_ERROR_INVALID_VALUE: null pointer or negative size";
        case MX_ERROR_UNSUPPORTED_SHAPE: return "MX_ERROR_UNSUPPORTED_SHAPE: K (or a size) outside the supported rules";
        case MX_ERROR_MISALIGNED: return "MX_ERROR_MISALIGNED: a pointer misses its required alignment";
        case MX_ERROR_WORKSPACE: return "MX_ERROR_WORKSPACE: workspace smaller than the size query";
        case MX_ERROR_LAUNCH: return "MX_ERROR_LAUNCH: kernel launch failed";
        case MX_ERROR_DEVICE: return "MX_ERROR_DEVICE: current device is not a gfx950 GPU";
    }
    return "MX_ERROR_UNKNOWN";
}

static mx_status quant_mx(bool f32, const void* x, int64_t rows, int64_t K, void* q, void* s, void* stream) {
    mx_status st = check_rows(rows, K, 32);
    if (st != MX_SUCCESS) return st;
    if (rows == 0) return MX_SUCCESS;
    if (!x || !q || !s) return MX_ERROR_INVALID_VALUE;
    if (!aligned(x, 16) || !aligned(q, 16)) return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    return launched(f32 ? mx::launch_quant_mx_f32(x, rows, K, q, s, hs) : mx::launch_quant_mx_bf16(x, rows, K, q, s, hs));
}

MX_API mx_status mx_quant_act_bf16(const void* x_bf16, int64_t M, int64_t K, void* q, void* s, void* stream) {
    return quant_mx(false, x_bf16, M, K, q, s, stream);
}

MX_API mx_status mx_quant_weight_f32(const float* w, int64_t N, int64_t K, void* q, void* s, void* stream) {
    return quant_mx(true, w, N, K, q, s, stream);
}

MX_API size_t mx_gemm_a4w4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (check_gemm(M, N, K) != MX_SUCCESS || M == 0 || N == 0) return 0;
    return mx::gemm_a4w4_workspace_bytes(M, N, K);
}

MX_API mx_status mx_gemm_a4w4_bf16(const void* qa, const void* sa, const void* qw, const void* sw, void* y_bf16,
                                   int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    mx_status st = check_gemm(M, N, K);
    if (st != MX_SUCCESS) return st;
    if (M == 0 || N == 0) return MX_SUCCESS;
    if (!qa || !sa || !qw || !sw || !y_bf16) return MX_ERROR_INVALID_VALUE;
    const size_t need = mx_gemm_a4w4_workspace_bytes(M, N, K);
    if (workspace_bytes < need || (need && !workspace)) return MX_ERROR_WORKSPACE;
    if (!aligned(qa, 16) || !aligned(qw, 16) || !aligned(sa, 4) || !aligned(sw, 4) || !aligned(y_bf16, 2) ||
        (need && !aligned(workspace, 16)))
        return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_gemm_a4w4(qa, sa, qw, sw, y_bf16, M, N, K, workspace, reinterpret_cast<hipStream_t>(stream)));
}

MX_API mx_status mx_gemm_a4w4_bf16_noalloc(const void* qa, const void* sa, const void* qw, const void* sw,
                                           void* y_bf16, int64_t M, int64_t N, int64_t K, void* stream) {
    mx_status st = check_gemm(M, N, K);
    if (st != MX_SUCCESS) return st;
    if (M == 0 || N == 0) return MX_SUCCESS;
    if (!qa || !sa || !qw || !sw || !y_bf16) return MX_ERROR_INVALID_VALUE;
    if (mx_gemm_a4w4_workspace_bytes(M, N, K) > mx::kGemmScratchBytes) return MX_ERROR_WORKSPACE;
    if (!aligned(qa, 16) || !aligned(qw, 16) || !aligned(sa, 4) || !aligned(sw, 4) || !aligned(y_bf16, 2))
        return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_gemm_a4w4_noalloc(qa, sa, qw, sw, y_bf16, M, N, K, reinterpret_cast<hipStream_t>(stream)));
}

MX_API size_t mx_linear_a4w4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (check_gemm(M, N, K) != MX_SUCCESS || M == 0 || N == 0) return 0;
    return mx::linear_a4w4_workspace_bytes(M, N, K);
}

MX_API mx_status mx_linear_a4w4_bf16(const void* x_bf16, const void* qw, const void* sw, void* y_bf16, int64_t M,
                                     int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
    mx_status st = check_gemm(M, N, K);
    if (st != MX_SUCCESS) return st;
    if (M == 0 || N == 0) return MX_SUCCESS;
    if (!x_bf16 || !qw || !sw || !y_bf16) return MX_ERROR_INVALID_VALUE;
    const size_t need = mx_linear_a4w4_workspace_bytes(M, N, K);
    if (workspace_bytes < need || (need && !workspace)) return MX_ERROR_WORKSPACE;
    if (!aligned(x_bf16, 16) || !aligned(qw, 16) || !aligned(sw, 4) || !aligned(y_bf16, 2) ||
        (need && !aligned(workspace, 256)))
        return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_linear_a4w4(x_bf16, qw, sw, y_bf16, M, N, K, workspace,
                                           reinterpret_cast<hipStream_t>(stream)));
}

MX_API mx_status mx_gemm_a4w4_grouped_bf16(const void* qa, const void* sa, const void* qw, const void* sw,
                                           void* y_bf16, const int32_t* offsets, int64_t G, int64_t max_rows,
                                           int64_t N, int64_t K, void* stream) {
    if (G < 0 || N < 0 || max_rows < 0) return MX_ERROR_INVALID_VALUE;
    if (max_rows > INT32_MAX || G > 65535 || N > INT32_MAX || K <= 0 || K % 512 != 0 || K > 16384)
        return MX_ERROR_UNSUPPORTED_SHAPE;
    if (N > (INT64_C(1) << 40) / K / (G > 0 ? G : 1)) return MX_ERROR_UNSUPPORTED_SHAPE;
    if (G == 0 || N == 0 || max_rows == 0) return MX_SUCCESS;
    if (!qa || !sa || !qw || !sw || !y_bf16 || !offsets) return MX_ERROR_INVALID_VALUE;
    if (!aligned(qa, 16) || !aligned(qw, 16) || !aligned(sa, 16) || !aligned(sw, 16) || !aligned(y_bf16, 2) ||
        !aligned(offsets, 4))
        return MX_ERROR_MISALIGNED;
    mx_status st;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_a4w4_grouped(qa, sa, qw, sw, y_bf16, offsets, G, max_rows, N, K,
                                            reinterpret_cast<hipStream_t>(stream)));
}

static mx_status quant_ptpc(bool f32, const void* x, int64_t rows, int64_t K, void* q, float* s, void* stream) {
    mx_status st = check_rows(rows, K, 8);
    if (st != MX_SUCCESS) return st;
    if (rows == 0) return MX_SUCCESS;
    if (!x || !q || !s) return MX_ERROR_INVALID_VALUE;
    if (!aligned(x, 16) || !aligned(q, 8) || !aligned(s, 4)) return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    return launched(f32 ? mx::launch_quant_ptpc_f32(x, rows, K, q, s, hs)
                        : mx::launch_quant_ptpc_bf16(x, rows, K, q, s, hs));
}

MX_API mx_status ptpc_quant_act_fp8(const void* x_bf16, int64_t M, int64_t K, void* q, float* s, void* stream) {
    return quant_ptpc(false, x_bf16, M, K, q, s, stream);
}

MX_API mx_status ptpc_quant_weight_f32(const float* w, int64_t N, int64_t K, void* q, float* s, void* stream) {
    return quant_ptpc(true, w, N, K, q, s, stream);
}

MX_API size_t gemm_a8w8_ptpc_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (check_gemm(M, N, K) != MX_SUCCESS || M == 0 || N == 0) return 0;
    return mx::gemm_a8w8_workspace_bytes(M, N, K);
}

MX_API mx_status gemm_a8w8_ptpc_bf16(const void* qa, const float* sa, const void* qw, const float* sw, void* y_bf16,
                                     int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    mx_status st = check_gemm(M, N, K);
    if (st != MX_SUCCESS) return st;
    if (M == 0 || N == 0) return MX_SUCCESS;
    if (!qa || !sa || !qw || !sw || !y_bf16) return MX_ERROR_INVALID_VALUE;
    const size_t need = gemm_a8w8_ptpc_workspace_bytes(M, N, K);
    if (workspace_bytes < need || (need && !workspace)) return MX_ERROR_WORKSPACE;
    if (!aligned(qa, 16) || !aligned(qw, 16) || !aligned(sa, 4) || !aligned(sw, 4) || !aligned(y_bf16, 2) ||
        (need && !aligned(workspace, 16)))
        return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_gemm_a8w8(qa, sa, qw, sw, y_bf16, M, N, K, workspace,
                                         reinterpret_cast<hipStream_t>(stream)));
}

MX_API mx_status b128_quant_act_fp8(const void* x_bf16, int64_t M, int64_t K, void* q, float* s, void* stream) {
    mx_status st = check_rows(M, K, 128);
    if (st != MX_SUCCESS) return st;
    if (M == 0) return MX_SUCCESS;
    if (!x_bf16 || !q || !s) return MX_ERROR_INVALID_VALUE;
    if (!aligned(x_bf16, 16) || !aligned(q, 8) || !aligned(s, 4)) return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_quant_b128_act(x_bf16, M, K, q, s, reinterpret_cast<hipStream_t>(stream)));
}

MX_API mx_status b128_quant_weight_f32(const float* w, int64_t N, int64_t K, void* q, float* s, void* stream) {
    mx_status st = check_rows(N, K, 128);
    if (st != MX_SUCCESS) return st;
    if ((N + 127) / 128 > INT32_MAX / (K / 128)) return MX_ERROR_UNSUPPORTED_SHAPE;  // one workgroup per block
    if (N == 0) return MX_SUCCESS;
    if (!w || !q || !s) return MX_ERROR_INVALID_VALUE;
    if (!aligned(w, 16) || !aligned(q, 4) || !aligned(s, 4)) return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_quant_b128_weight(w, N, K, q, s, reinterpret_cast<hipStream_t>(stream)));
}

// K <= 2^22: a tile's rows are reached by 32-bit offsets; tiles of at least 32 x 64 must fit one 1-D grid
static mx_status check_gemm_b128(int64_t M, int64_t N, int64_t K) {
    const mx_status st = check_gemm(M, N, K);
    if (st != MX_SUCCESS) return st;
    if (K > (INT64_C(1) << 22)) return MX_ERROR_UNSUPPORTED_SHAPE;
    if ((M + 31) / 32 > INT32_MAX / ((N + 63) / 64 > 0 ? (N + 63) / 64 : 1)) return MX_ERROR_UNSUPPORTED_SHAPE;
    return MX_SUCCESS;
}

MX_API mx_status gemm_a8w8_b128_bf16(const void* qa, const float* sa, const void* qw, const float* sw, void* y_bf16,
                                     int64_t M, int64_t N, int64_t K, void* stream) {
    mx_status st = check_gemm_b128(M, N, K);
    if (st != MX_SUCCESS) return st;
    if (M == 0 || N == 0) return MX_SUCCESS;
    if (!qa || !sa || !qw || !sw || !y_bf16) return MX_ERROR_INVALID_VALUE;
    if (!aligned(qa, 16) || !aligned(qw, 16) || !aligned(sa, 4) || !aligned(sw, 4) || !aligned(y_bf16, 2))
        return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_gemm_b128(qa, sa, qw, sw, y_bf16, M, N, K, reinterpret_cast<hipStream_t>(stream)));
}

MX_API size_t linear_a8w8_b128_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (check_gemm_b128(M, N, K) != MX_SUCCESS || M == 0 || N == 0) return 0;
    return mx::linear_b128_workspace_bytes(M, N, K);
}

MX_API mx_status linear_a8w8_b128_bf16(const void* x_bf16, const void* qw, const float* sw, void* y_bf16, int64_t M,
                                       int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
    mx_status st = check_gemm_b128(M, N, K);
    if (st != MX_SUCCESS) return st;
    if (M == 0 || N == 0) return MX_SUCCESS;
    if (!x_bf16 || !qw || !sw || !y_bf16) return MX_ERROR_INVALID_VALUE;
    const size_t need = mx::linear_b128_workspace_bytes(M, N, K);
    if (workspace_bytes < need || (need && !workspace)) return MX_ERROR_WORKSPACE;
    if (!aligned(x_bf16, 16) || !aligned(qw, 16) || !aligned(sw, 4) || !aligned(y_bf16, 2) || (need && !aligned(workspace, 16)))
        return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_linear_b128(x_bf16, qw, sw, y_bf16, M, N, K, workspace, reinterpret_cast<hipStream_t>(stream)));
}

MX_API mx_status gemm_a8w8_b128_grouped_bf16(const void* qa, const float* sa, int64_t a_rows, const void* qw,
                                             const float* sw, void* y_bf16, const int32_t* offsets, const int32_t* rows,
                                             int64_t G, int64_t T, int64_t N, int64_t K, void* stream) {
    mx_status st = check_gemm_b128(T, N, K);
    if (st != MX_SUCCESS) return st;
    if (G < 0 || a_rows < 0) return MX_ERROR_INVALID_VALUE;
    if (G > 65535 || a_rows > (INT64_C(1) << 40) / K || N > (INT64_C(1) << 40) / K / (G > 0 ? G : 1))
        return MX_ERROR_UNSUPPORTED_SHAPE;
    // tiles of at least 32 x 64, one partial row tile per group, must fit one 1-D grid
    if ((T / 32 + (G < T ? G : T)) > INT32_MAX / ((N + 63) / 64 > 0 ? (N + 63) / 64 : 1)) return MX_ERROR_UNSUPPORTED_SHAPE;
    // named rows are reached by 32-bit offsets
    if (rows && a_rows > (INT64_C(1) << 32) / K - 1) return MX_ERROR_UNSUPPORTED_SHAPE;
    if (G == 0 || T == 0 || N == 0) return MX_SUCCESS;
    if (!qa || !sa || !qw || !sw || !y_bf16 || !offsets) return MX_ERROR_INVALID_VALUE;
    if (a_rows == 0 || (!rows && a_rows < T)) return MX_ERROR_INVALID_VALUE;
    if (!aligned(qa, 16) || !aligned(qw, 16) || !aligned(sa, 4) || !aligned(sw, 4) || !aligned(y_bf16, 2) ||
        !aligned(offsets, 4) || !aligned(rows, 4))
        return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_gemm_b128_grouped(qa, sa, a_rows, qw, sw, y_bf16, offsets, rows, G, T, N, K,
                                                 reinterpret_cast<hipStream_t>(stream)));
}

// T >= 0 rows of 1 .. 1024 experts
static mx_status check_router(int64_t T, int64_t E) {
    if (T < 0) return MX_ERROR_INVALID_VALUE;
    if (E < 1 || E > 1024 || T > INT32_MAX) return MX_ERROR_UNSUPPORTED_SHAPE;
    return MX_SUCCESS;
}

static mx_status check_route(int64_t T, int64_t top, int64_t E) {
    const mx_status st = check_router(T, E);
    if (st != MX_SUCCESS) return st;
    if (top < 0) return MX_ERROR_INVALID_VALUE;
    // choices are numbered in 32 bits, and so are the counts of their chunks, with room to spare
    if (top > 0 && T > (INT64_C(1) << 24) / top) return MX_ERROR_UNSUPPORTED_SHAPE;
    return MX_SUCCESS;
}

MX_API size_t moe_route_workspace_bytes(int64_t T, int64_t top, int64_t E) {
    return check_route(T, top, E) == MX_SUCCESS ? mx::moe_route_workspace_bytes(T * top, E) : 0;
}

MX_API mx_status moe_route(const void* ids, int id_bytes, int64_t T, int64_t top, int64_t E, int32_t* counts,
                           int32_t* offsets, int32_t* rows, int32_t* slots, void* workspace, size_t workspace_bytes,
                           void* stream) {
    mx_status st = check_route(T, top, E);
    if (st != MX_SUCCESS) return st;
    if (id_bytes != 4 && id_bytes != 8) return MX_ERROR_INVALID_VALUE;
    const bool any = T * top > 0;
    if (!counts || !offsets || (any && (!ids || !rows || !slots))) return MX_ERROR_INVALID_VALUE;
    const size_t need = mx::moe_route_workspace_bytes(T * top, E);
    if (workspace_bytes < need || (need && !workspace)) return MX_ERROR_WORKSPACE;
    if (!aligned(ids, id_bytes) || !aligned(counts, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4) ||
        (need && !aligned(workspace, 16)))
        return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_moe_route(ids, id_bytes == 8, T, top, E, counts, offsets, rows, slots, workspace,
                                         reinterpret_cast<hipStream_t>(stream)));
}

MX_API size_t moe_balance_loss_workspace_bytes(int64_t T, int64_t E) {
    return check_router(T, E) == MX_SUCCESS ? mx::moe_balance_workspace_bytes(T, E) : 0;
}

MX_API mx_status moe_balance_loss(const void* logits, mx_dtype dtype, int64_t T, int64_t E, const int32_t* counts,
                                  const uint8_t* mask, float coef, float* loss, float* weights, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    mx_status st = check_router(T, E);
    if (st != MX_SUCCESS) return st;
    if (dtype != MX_F32 && dtype != MX_BF16) return MX_ERROR_INVALID_VALUE;
    if (!counts || !loss || !weights || (T > 0 && !logits)) return MX_ERROR_INVALID_VALUE;
    const size_t need = mx::moe_balance_workspace_bytes(T, E);
    if (workspace_bytes < need || (need && !workspace)) return MX_ERROR_WORKSPACE;
    if (!aligned(logits, dtype == MX_F32 ? 4 : 2) || !aligned(counts, 4) || !aligned(loss, 4) || !aligned(weights, 4) ||
        (need && !aligned(workspace, 16)))
        return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_moe_balance(logits, dtype == MX_BF16, T, E, counts, mask, coef, loss, weights, workspace,
                                           reinterpret_cast<hipStream_t>(stream)));
}

MX_API mx_status moe_balance_loss_grad(const void* logits, mx_dtype dtype, int64_t T, int64_t E, const float* weights,
                                       const uint8_t* mask, const float* grad_loss, void* dlogits, void* stream) {
    mx_status st = check_router(T, E);
    if (st != MX_SUCCESS) return st;
    if (dtype != MX_F32 && dtype != MX_BF16) return MX_ERROR_INVALID_VALUE;
    if (T == 0) return MX_SUCCESS;
    if (!logits || !weights || !grad_loss || !dlogits) return MX_ERROR_INVALID_VALUE;
    const uintptr_t size = dtype == MX_F32 ? 4 : 2;
    if (!aligned(logits, size) || !aligned(dlogits, size) || !aligned(weights, 4) || !aligned(grad_loss, 4))
        return MX_ERROR_MISALIGNED;
    if ((st = check_device()) != MX_SUCCESS) return st;
    return launched(mx::launch_moe_balance_grad(logits, dtype == MX_BF16, T, E, weights, mask, grad_loss, dlogits,
                                                reinterpret_cast<hipStream_t>(stream)));
}
