// quant_b128.hip - FP8 E4M3 quantization with one FP32 scale per block of 128 values.
//
// Activations [M, K]: a block is 128 consecutive K-values of one row, scales [M, K/128].
// Weights [N, K]: a block is 128 rows x 128 K-values (the last row block may be short), scales
// [ceil(N/128), K/128].
//
// Per block: a = max|x| (an integer max over the magnitude bit patterns), s = fl32(a / 448), s = 1
// where that is 0, code = E4M3fn(fl32(x / s)), round to nearest even, saturating at 448.  Both
// divisions are IEEE binary32 divisions; for BF16 blocks the per-element one is div_corrected, which
// gives the same codes.  A block that holds a NaN or an infinity gets s = NaN and every code 0x7F.
// Quotients pass 448 only where s is subnormal and so rounded coarsely; they are clamped before the
// conversion, whose behaviour past the largest finite code is not relied on.
#include "fp8_device.hpp"
#include "launch.hpp"

namespace mx {
namespace {

constexpr int kThreads = 256;

// BF16 activations: 16 lanes own one block, 8 values (one 16-byte load, one 8-byte store) each, so a
// wave reads 1 KB and writes 512 bytes, both contiguous; the maximum over the 16 lanes is four DPP
// swaps.  Blocks are consecutive in memory whatever the row length, so the grid runs over blocks.
__global__ __launch_bounds__(kThreads) void quant_b128_act_kernel(const uint4* __restrict__ x, uint2* __restrict__ q,
                                                                  float* __restrict__ s, int64_t units) {
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += stride) {
        float sc;
        q[u] = quant_block_bf16x8(x[u], sc);  // units and the stride are multiples of 16: the lanes of a block run together
        if ((threadIdx.x & 15) == 0) s[u >> 4] = sc;
    }
}

// FP32 weights: one workgroup per 128 x 128 block; 32 lanes cover a row's 128 values (16-byte loads),
// eight rows at a time, so the block's 64 KB are read once into 64 registers per thread.
__global__ __launch_bounds__(kThreads) void quant_b128_weight_kernel(const float* __restrict__ w,
                                                                     uint8_t* __restrict__ q, float* __restrict__ s,
                                                                     int64_t N, int64_t K, int nkb) {
    __shared__ uint32_t red[kThreads / 64];
    const int64_t nb = blockIdx.x / nkb, kb = blockIdx.x % nkb;
    const int row = threadIdx.x >> 5, col = threadIdx.x & 31;
    uint4 v[16];
    uint32_t mag = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t n = nb * 128 + 8 * i + row;
        v[i] = make_uint4(0, 0, 0, 0);
        if (n < N) v[i] = *reinterpret_cast<const uint4*>(w + n * K + kb * 128 + 4 * col);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        mag = max(max(mag, max(v[i].x & 0x7fffffffu, v[i].y & 0x7fffffffu)),
                  max(v[i].z & 0x7fffffffu, v[i].w & 0x7fffffffu));
    mag = wave_max(mag);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mag;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) mag = max(mag, red[i]);
    const float sc = block_scale(mag);
    if (threadIdx.x == 0) s[blockIdx.x] = sc;
    const bool bad = mag >= 0x7f800000u;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t n = nb * 128 + 8 * i + row;
        if (n >= N) continue;
        const uint32_t c = bad ? 0x7f7f7f7fu
                               : e4m3fn_x4(clamped_quotient(__uint_as_float(v[i].x), sc),
                                           clamped_quotient(__uint_as_float(v[i].y), sc),
                                           clamped_quotient(__uint_as_float(v[i].z), sc),
                                           clamped_quotient(__uint_as_float(v[i].w), sc));
        *reinterpret_cast<uint32_t*>(q + n * K + kb * 128 + 4 * col) = c;
    }
}

}  // namespace

hipError_t launch_quant_b128_act(const void* x, int64_t M, int64_t K, void* q, float* s, hipStream_t st) {
    const int64_t units = M * (K / 8);
    const int64_t blocks = (units + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(quant_b128_act_kernel, dim3((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20))), dim3(kThreads),
                       0, st, reinterpret_cast<const uint4*>(x), reinterpret_cast<uint2*>(q), s, units);
    return hipGetLastError();
}

hipError_t launch_quant_b128_weight(const float* w, int64_t N, int64_t K, void* q, float* s, hipStream_t st) {
    const int64_t nkb = K / 128, blocks = ((N + 127) / 128) * nkb;
    hipLaunchKernelGGL(quant_b128_weight_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st, w,
                       reinterpret_cast<uint8_t*>(q), s, N, K, (int)nkb);
    return hipGetLastError();
}

}  // namespace mx
