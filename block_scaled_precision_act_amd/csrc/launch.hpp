// launch.hpp - internal launchers behind the C ABI (argument checks live in api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

// MXFP4 quantizer: rows x K values (K % 32 == 0) -> codes [rows, K/2], scales [rows, K/32].
hipError_t launch_quant_mx_bf16(const void* x, int64_t rows, int64_t K, void* q, void* s, hipStream_t st);
hipError_t launch_quant_mx_f32(const void* x, int64_t rows, int64_t K, void* q, void* s, hipStream_t st);

// PTPC FP8 quantizer: rows x K values (K % 8 == 0) -> E4M3 codes [rows, K], FP32 scales [rows].
hipError_t launch_quant_ptpc_bf16(const void* x, int64_t rows, int64_t K, void* q, float* s, hipStream_t st);
hipError_t launch_quant_ptpc_f32(const void* x, int64_t rows, int64_t K, void* q, float* s, hipStream_t st);

// GEMMs (K % 128 == 0, M, N > 0).
hipError_t launch_gemm_a4w4(const void* qa, const void* sa, const void* qw, const void* sw, void* y,
                            int64_t M, int64_t N, int64_t K, void* workspace, hipStream_t st);
size_t gemm_a4w4_workspace_bytes(int64_t M, int64_t N, int64_t K);
// The same GEMM with its workspace in a static per-device array of kGemmScratchBytes (no allocation):
// the largest workspace of any split-K plan (256 workgroups); the caller rejects shapes that need more.
constexpr size_t kGemmScratchBytes = (size_t)8 << 20;
hipError_t launch_gemm_a4w4_noalloc(const void* qa, const void* sa, const void* qw, const void* sw, void* y,
                                    int64_t M, int64_t N, int64_t K, hipStream_t st);
// A4W4 layer: BF16 X -> MXFP4 -> BF16 Y, in one launch for M <= 8 (quantization inside the split-K
// GEMM's workgroups), else the quantizer and the GEMM.
hipError_t launch_linear_a4w4(const void* x, const void* qw, const void* sw, void* y, int64_t M, int64_t N, int64_t K,
                              void* workspace, hipStream_t st);
size_t linear_a4w4_workspace_bytes(int64_t M, int64_t N, int64_t K);
// Grouped A4W4 GEMM over MoE experts (decode-sized groups, see mx_gemm_a4w4_grouped_bf16).
hipError_t launch_a4w4_grouped(const void* qa, const void* sa, const void* qw, const void* sw, void* y,
                               const int32_t* offsets, int64_t G, int64_t max_rows, int64_t N, int64_t K,
                               hipStream_t st);
hipError_t launch_gemm_a8w8(const void* qa, const float* sa, const void* qw, const float* sw, void* y,
                            int64_t M, int64_t N, int64_t K, void* workspace, hipStream_t st);
size_t gemm_a8w8_workspace_bytes(int64_t M, int64_t N, int64_t K);

// Block-128 FP8 (one FP32 scale per 128 values; K % 128 == 0): quantizers and GEMMs.
hipError_t launch_quant_b128_act(const void* x, int64_t M, int64_t K, void* q, float* s, hipStream_t st);
hipError_t launch_quant_b128_weight(const float* w, int64_t N, int64_t K, void* q, float* s, hipStream_t st);
hipError_t launch_gemm_b128(const void* qa, const float* sa, const void* qw, const float* sw, void* y, int64_t M, int64_t N,
                            int64_t K, hipStream_t st);
hipError_t launch_linear_b128(const void* x, const void* qw, const float* sw, void* y, int64_t M, int64_t N, int64_t K,
                              void* workspace, hipStream_t st);
size_t linear_b128_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_b128_grouped(const void* qa, const float* sa, int64_t arows, const void* qw, const float* sw,
                                    void* y, const int32_t* offsets, const int32_t* rows, int64_t G, int64_t M, int64_t N,
                                    int64_t K, hipStream_t st);

// Expert routing: packing of the experts' rows, and the balance loss with its gradient.
size_t moe_route_workspace_bytes(int64_t n, int64_t E);
hipError_t launch_moe_route(const void* ids, bool wide, int64_t T, int64_t top, int64_t E, int32_t* counts, int32_t* offsets,
                            int32_t* rows, int32_t* slots, void* workspace, hipStream_t st);
size_t moe_balance_workspace_bytes(int64_t T, int64_t E);
hipError_t launch_moe_balance(const void* logits, bool half, int64_t T, int64_t E, const int32_t* counts, const uint8_t* mask,
                              float coef, float* loss, float* w, void* workspace, hipStream_t st);
hipError_t launch_moe_balance_grad(const void* logits, bool half, int64_t T, int64_t E, const float* w, const uint8_t* mask,
                                   const float* grad_loss, void* dlogits, hipStream_t st);

// Compute units of the current device (cached per device); 0 if the query fails.
int device_cus();

}  // namespace mx
