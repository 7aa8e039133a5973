// gemm_b128.hip - A8W8 GEMM with one FP32 scale per block of 128: dense, and grouped over MoE experts.
//
//   Y[m, n] = sum_b sa[m, b] sw[n / 128, b] P_b[m, n],   P_b[m, n] = sum_{k in block b} qa[m, k] qw[n, k]
//
// with E4M3 codes and b the 128-value blocks of K.  P_b is one FP8 MFMA of depth 128 started from zero;
// the scaled sum over blocks runs in FP32 on the vector ALU: acc = fma(P_b, sa sw, acc).
//
// Precision.  The FP8 MFMA adds the 128 products of a block in groups of eight, and cuts each product at 2^-13
// of the power of two of its group's largest one (measured on this GPU, toward zero); the groups are added
// with FP32's width.  So a block's sum is off by less than 7 * 2^-13 of the sum of its products' magnitudes whatever the
// codes, and by 2^-15.5 at most over a million outputs of quantized normal values, 2^-19 in the mean: far
// below the rounding of the BF16 output except for strongly cancelling sums.  The per-row-scale GEMM of this
// library widens its codes to FP16 instead, which is exact up to FP32 but runs at half the matrix rate; with a
// scale per block, blocks have to leave the MFMA for their FP32 sum anyway, and the FP8 rate is kept.
//
// Operand layout: lane l holds row l % 16 of a fragment and, of the block's eight 16-byte chunks, chunks
// l / 16 and l / 16 + 4.  Both operands use the same order, and the order of K inside a block does not
// matter, so a wave's two loads of a fragment each take 64 contiguous bytes per row.  Weights are the
// first operand: a lane's four results are four consecutive n of one m, which share one activation scale.
#include "launch.hpp"
#include "mx_device.hpp"

namespace mx {

namespace {

constexpr int kFmtE4M3 = 0;   // scaled-MFMA operand format
constexpr int kOne = 0x7f;    // E8M0 1.0

__device__ __forceinline__ v8i operand(uint4 lo, uint4 hi) {
    v8i r = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    return r;
}
// 16 x 16 products of one block, from zero
__device__ __forceinline__ v4f block_mfma(v8i w, v8i x) {
    const v4f z = {0.f, 0.f, 0.f, 0.f};
    return mfma16<kFmtE4M3, 0>(w, x, z, kOne, kOne);
}

struct Args {
    const uint8_t* qa;      // [rows of A, K]
    const float* sa;        // [rows of A, K / 128]
    const uint8_t* qw;      // [groups, N, K]
    const float* sw;        // [groups, ceil(N / 128), K / 128]
    uint16_t* y;            // [M, N]
    const int32_t* offsets; // grouped: [G + 1], else null
    const int32_t* rows;    // grouped: A row of every Y row, or null (the same row)
    int64_t arows;          // rows of A
    int64_t M, N, K;
    int G;
};

// Rows r0 .. r1 - 1 of Y belong to group e.  Offsets that are out of order or past M give fewer rows, never
// rows outside Y.
__device__ __forceinline__ void group_rows(const Args& a, int e, int64_t& r0, int64_t& r1) {
    r0 = min((int64_t)max(a.offsets[e], 0), a.M);
    r1 = min((int64_t)max(a.offsets[e + 1], 0), a.M);
}
// A row that feeds row r of Y, -1 if there is none (its outputs are 0)
__device__ __forceinline__ int64_t a_row(const Args& a, int64_t r) {
    if (a.rows == nullptr) return r;
    const int64_t t = a.rows[r];
    return t >= 0 && t < a.arows ? t : -1;
}
__device__ __forceinline__ void store4(uint16_t* y, int64_t N, int64_t n, v4f v, bool vec) {
    uint16_t* dst = y + n;
    if (vec && n + 3 < N) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < N) dst[i] = (uint16_t)bf16_rne(v[i]);
    }
}

// Few rows: one workgroup per 16 FN columns (and group), its W waves take contiguous parts of K and meet
// in LDS, summed in wave order.  Operands go from memory to registers; rows in chunks of 16 FM.
template <int FM, int FN, int W>
__global__ __launch_bounds__(64 * W) void gemm_b128_rows(Args a) {
    __shared__ v4f red[W][FN][FM][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
    const int nkb = (int)(a.K / 128), per = (nkb + W - 1) / W;
    const int kb0 = min(wave * per, nkb), kb1 = min(kb0 + per, nkb);
    const int64_t n0 = (int64_t)blockIdx.x * 16 * FN;
    const int e = blockIdx.y;
    int64_t r0 = 0, r1 = a.M;
    if (a.offsets) group_rows(a, e, r0, r1);
    const uint8_t* wp[FN];
    const float* swp[FN];
#pragma unroll
    for (int f = 0; f < FN; ++f) {
        const int64_t n = min(n0 + 16 * f + l16, a.N - 1);
        wp[f] = a.qw + (e * a.N + n) * a.K + 16 * g;
        swp[f] = a.sw + (e * ((a.N + 127) / 128) + min(n0 + 16 * f, a.N - 1) / 128) * nkb;
    }
    for (int64_t m0 = r0; m0 < r1; m0 += 16 * FM) {
        const uint8_t* ap[FM];
        const float* sap[FM];
        bool live[FM];
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int64_t r = a_row(a, min(m0 + 16 * j + l16, r1 - 1));
            live[j] = r >= 0;
            ap[j] = a.qa + max(r, (int64_t)0) * a.K + 16 * g;
            sap[j] = a.sa + max(r, (int64_t)0) * nkb;
        }
        v4f acc[FN][FM] = {};
        for (int kb = kb0; kb < kb1; ++kb) {
            v8i x[FM];
            float sx[FM];
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                x[j] = operand(ldg16(ap[j] + (int64_t)kb * 128), ldg16(ap[j] + (int64_t)kb * 128 + 64));
                sx[j] = sap[j][kb];
            }
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                const v8i w = operand(ldg16(wp[f] + (int64_t)kb * 128), ldg16(wp[f] + (int64_t)kb * 128 + 64));
                const float sc = swp[f][kb];
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    const v4f p = block_mfma(w, x[j]);
                    const float s = sx[j] * sc;
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[f][j][i] = __builtin_fmaf(p[i], s, acc[f][j][i]);
                }
            }
        }
#pragma unroll
        for (int f = 0; f < FN; ++f)
#pragma unroll
            for (int j = 0; j < FM; ++j) red[wave][f][j][lane] = acc[f][j];
        __syncthreads();
        for (int t = threadIdx.x; t < FN * FM * 64; t += 64 * W) {
            const int f = t / (FM * 64), j = t / 64 % FM, l = t % 64;
            v4f s = red[0][f][j][l];
#pragma unroll
            for (int w = 1; w < W; ++w) s += red[w][f][j][l];
            const int64_t m = m0 + 16 * j + (l & 15);
            if (m < r1) {
                const bool ok = a_row(a, m) >= 0;
                const v4f zero = {0.f, 0.f, 0.f, 0.f};
                store4(a.y + m * a.N, a.N, n0 + 16 * f + 4 * (l >> 4), ok ? s : zero, a.N % 4 == 0 && ((uintptr_t)a.y & 7) == 0);
            }
        }
        __syncthreads();
    }
}

// Many rows: a 16 FM WM x 16 FN WN output tile per workgroup of WM x WN waves; K in steps of one block,
// double-buffered in LDS by direct copies.  Rows of 128 bytes hold eight 16-byte chunks, chunk c of row r at
// place c ^ (r / 2 % 8), so the 16 lanes of a fragment read 16 different places.
template <int FM, int FN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void gemm_b128_tile(Args a, int tiles_m, int tiles_n) {
    constexpr int TM = 16 * FM * WM, TN = 16 * FN * WN, W = WM * WN;
    constexpr int CA = TM / 8 / W, CW = TN / 8 / W;  // copies of eight rows per wave
    static_assert(TM % (8 * W) == 0 && TN % (8 * W) == 0, "whole copies");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2][(TM + TN) * 128];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4, wm = wave / WN, wn = wave % WN;
    const int nkb = (int)(a.K / 128);
    int tm = blockIdx.x / tiles_n, tn = blockIdx.x % tiles_n, e = 0;
    int64_t m0 = (int64_t)tm * TM, r1 = a.M;
    if (a.offsets) {  // the tm-th row tile over all groups
        int left = tm;
        bool found = false;
        for (int i = 0; i < a.G; ++i) {
            int64_t b, t;
            group_rows(a, i, b, t);
            const int n = t > b ? (int)((t - b + TM - 1) / TM) : 0;
            if (left < n) {
                e = i;
                m0 = b + (int64_t)left * TM;
                r1 = t;
                found = true;
                break;
            }
            left -= n;
        }
        if (!found) return;
    }
    const int64_t n0 = (int64_t)tn * TN;
    const int prow = lane >> 3, pchunk = lane & 7;
    const uint8_t* src[CA + CW];
#pragma unroll
    for (int i = 0; i < CA + CW; ++i) {
        const int row = 8 * (i < CA ? CA * wave + i : CW * wave + i - CA) + prow;
        const int chunk = pchunk ^ (row >> 1 & 7);
        if (i < CA) {
            const int64_t r = a_row(a, min(m0 + row, r1 - 1));
            src[i] = a.qa + max(r, (int64_t)0) * a.K + 16 * chunk;
        } else {
            src[i] = a.qw + (e * a.N + min(n0 + row, a.N - 1)) * a.K + 16 * chunk;
        }
    }
    auto issue = [&](int kb) {
#pragma unroll
        for (int i = 0; i < CA + CW; ++i) {
            uint8_t* dst = lds[kb & 1] + (i < CA ? (CA * wave + i) * 1024 : TM * 128 + (CW * wave + i - CA) * 1024);
            g2lds16(src[i] + (int64_t)kb * 128, dst);
        }
    };
    const float* sap[FM];
    bool live[FM];
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int64_t r = a_row(a, min(m0 + 16 * (FM * wm + j) + l16, r1 - 1));
        live[j] = r >= 0;
        sap[j] = a.sa + max(r, (int64_t)0) * nkb;
    }
    const float* swp[FN];
#pragma unroll
    for (int f = 0; f < FN; ++f)
        swp[f] = a.sw + (e * ((a.N + 127) / 128) + min(n0 + 16 * (FN * wn + f), a.N - 1) / 128) * nkb;
    const int key = l16 >> 1, c0 = 16 * (g ^ key), c1 = 16 * ((g + 4) ^ key);
    v4f acc[FN][FM] = {};
    issue(0);
    for (int kb = 0; kb < nkb; ++kb) {
        float sx[FM], sc[FN];
#pragma unroll
        for (int j = 0; j < FM; ++j) sx[j] = sap[j][kb];
#pragma unroll
        for (int f = 0; f < FN; ++f) sc[f] = swp[f][kb];
        wait_vmcnt<0>();
        __syncthreads();  // every wave's copies of kb have landed, and every wave has read kb - 1
        if (kb + 1 < nkb) issue(kb + 1);
        const uint8_t* la = lds[kb & 1] + (16 * FM * wm + l16) * 128;
        const uint8_t* lw = lds[kb & 1] + TM * 128 + (16 * FN * wn + l16) * 128;
        v8i x[FM];
#pragma unroll
        for (int j = 0; j < FM; ++j)
            x[j] = operand(*reinterpret_cast<const uint4*>(la + j * 2048 + c0), *reinterpret_cast<const uint4*>(la + j * 2048 + c1));
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            const v8i w = operand(*reinterpret_cast<const uint4*>(lw + f * 2048 + c0), *reinterpret_cast<const uint4*>(lw + f * 2048 + c1));
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                const v4f p = block_mfma(w, x[j]);
                const float s = sx[j] * sc[f];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[f][j][i] = __builtin_fmaf(p[i], s, acc[f][j][i]);
            }
        }
    }
    const bool vec = a.N % 4 == 0 && ((uintptr_t)a.y & 7) == 0;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int64_t m = m0 + 16 * (FM * wm + j) + l16;
        if (m >= r1) continue;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            const v4f zero = {0.f, 0.f, 0.f, 0.f};
            store4(a.y + m * a.N, a.N, n0 + 16 * (FN * wn + f) + 4 * g, live[j] ? acc[f][j] : zero, vec);
        }
    }
}

template <int FM, int FN, int W>
hipError_t launch_rows(const Args& a, hipStream_t st) {
    const int64_t tiles = (a.N + 16 * FN - 1) / (16 * FN);
    hipLaunchKernelGGL((gemm_b128_rows<FM, FN, W>), dim3((unsigned)tiles, a.offsets ? a.G : 1), dim3(64 * W), 0, st, a);
    return hipGetLastError();
}

template <int FM, int FN, int WM, int WN>
hipError_t launch_tile(const Args& a, hipStream_t st) {
    constexpr int TM = 16 * FM * WM, TN = 16 * FN * WN;
    // grouped: every group may end with a partial tile, and there are at most M non-empty groups
    const int64_t tm = a.M / TM + (a.offsets ? (a.G < a.M ? a.G : a.M) : a.M % TM != 0), tn = (a.N + TN - 1) / TN;
    if (tm * tn > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((gemm_b128_tile<FM, FN, WM, WN>), dim3((unsigned)(tm * tn)), dim3(64 * WM * WN), 0, st, a, (int)tm, (int)tn);
    return hipGetLastError();
}

hipError_t dispatch(const Args& a, int64_t rows, hipStream_t st) {
    if (rows <= 16) return launch_rows<1, 1, 8>(a, st);
    if (rows <= 32) return launch_rows<2, 1, 8>(a, st);
    if (rows <= 64) return launch_rows<4, 1, 8>(a, st);
    if (rows <= 512) return launch_tile<4, 4, 2, 2>(a, st);
    return launch_tile<4, 8, 4, 2>(a, st);
}

}  // namespace

hipError_t launch_gemm_b128(const void* qa, const float* sa, const void* qw, const float* sw, void* y, int64_t M, int64_t N,
                            int64_t K, hipStream_t st) {
    const Args a = {reinterpret_cast<const uint8_t*>(qa), sa, reinterpret_cast<const uint8_t*>(qw), sw,
                    reinterpret_cast<uint16_t*>(y), nullptr, nullptr, M, M, N, K, 1};
    return dispatch(a, M, st);
}

hipError_t launch_gemm_b128_grouped(const void* qa, const float* sa, int64_t arows, const void* qw, const float* sw,
                                    void* y, const int32_t* offsets, const int32_t* rows, int64_t G, int64_t M, int64_t N,
                                    int64_t K, hipStream_t st) {
    const Args a = {reinterpret_cast<const uint8_t*>(qa), sa, reinterpret_cast<const uint8_t*>(qw), sw,
                    reinterpret_cast<uint16_t*>(y), offsets, rows, arows, M, N, K, (int)G};
    return dispatch(a, (M + G - 1) / G, st);
}

}  // namespace mx
