// gemm_b128.hip - entries of the A8W8 GEMM with one FP32 scale per block of 128 (kernels: gemm_b128.hpp).
//
// Which kernel.  A dense product of at most kRows rows streams the weight to registers (rows_kernel).  Anything else
// takes the tile whose rounds over the CUs are estimated cheapest: time = rounds x the time of one round of that tile,
// rounds = ceil(tiles / CUs).  One round of each tile, measured at K = 8192 and N = 7168 (us, launch taken off):
//   32 x 64 14.5, 64 x 64 17.5, 64 x 128 29, 128 x 128 40, 256 x 128 70, 256 x 256 115
// so a small product fills the CUs with small tiles and a large one is read least by large tiles.  Grouped products
// count their row tiles from the mean group.
#include "gemm_b128.hpp"
#include "launch.hpp"

namespace mx {
namespace {

using b128::Args;

constexpr int64_t kRows = 8;

hipError_t launch_rows(const Args& a, hipStream_t st) {
    hipLaunchKernelGGL((b128::rows_kernel<1, 1, 8, 3>), dim3((unsigned)((a.N + 15) / 16)), dim3(512), 0, st, a);
    return hipGetLastError();
}

template <int FM, int FN, int WM, int WN, int KG, int S>
hipError_t launch_tile(const Args& a, hipStream_t st) {
    constexpr int TM = 16 * FM * WM, TN = 16 * FN * WN;
    // grouped: every group may end with a partial tile, and there are at most M non-empty groups
    const int64_t tm = a.M / TM + (a.offsets ? (a.G < a.M ? a.G : a.M) : a.M % TM != 0), tn = (a.N + TN - 1) / TN;
    if (tm * tn > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((b128::tile_kernel<FM, FN, WM, WN, KG, S>), dim3((unsigned)(tm * tn)), dim3(64 * WM * WN * KG), 0, st, a,
                       (int)tm, (int)tn);
    return hipGetLastError();
}

struct Tile {
    int m, n;
    double round;  // us, see above
    hipError_t (*launch)(const Args&, hipStream_t);
};
const Tile kTiles[] = {
    {32, 64, 14.5, launch_tile<2, 2, 1, 2, 2, 4>},   {64, 64, 17.5, launch_tile<2, 4, 2, 1, 2, 4>},
    {64, 128, 29.0, launch_tile<2, 4, 2, 2, 2, 2>},  {128, 128, 40.0, launch_tile<2, 4, 4, 2, 1, 3>},
    {256, 128, 70.0, launch_tile<4, 4, 4, 2, 1, 2>}, {256, 256, 115.0, launch_tile<4, 8, 4, 2, 1, 2>},
};

hipError_t launch(const Args& a, hipStream_t st) {
    if (!a.offsets && a.M <= kRows) return launch_rows(a, st);
    const double cus = device_cus() > 0 ? device_cus() : 256;
    const double groups = a.offsets ? (double)(a.G < a.M ? a.G : a.M) : 1.0;
    const Tile* best = nullptr;
    double least = 0;
    for (const Tile& t : kTiles) {
        const double tn = (double)((a.N + t.n - 1) / t.n), mean = (double)a.M / groups;
        const double tm = a.offsets ? groups * (mean > 0.5 * t.m ? mean / t.m + 0.5 : 1.0) : (double)((a.M + t.m - 1) / t.m);
        const double rounds = a.offsets ? (tm * tn > cus ? tm * tn / cus : 1.0) : (double)(int64_t)((tm * tn + cus - 1) / cus);
        const double time = rounds * t.round;
        if (!best || time < least) {
            best = &t;
            least = time;
        }
    }
    return best->launch(a, st);
}

}  // namespace

hipError_t launch_gemm_b128(const void* qa, const float* sa, const void* qw, const float* sw, void* y, int64_t M, int64_t N,
                            int64_t K, hipStream_t st) {
    return launch({reinterpret_cast<const uint8_t*>(qa), sa, reinterpret_cast<const uint8_t*>(qw), sw,
                   reinterpret_cast<uint16_t*>(y), nullptr, nullptr, M, M, N, K, 1}, st);
}

// codes [M, K], then scales [M, K / 128]
size_t linear_b128_workspace_bytes(int64_t M, int64_t, int64_t K) { return (size_t)M * K + (size_t)M * (K / 128) * 4; }

hipError_t launch_linear_b128(const void* x, const void* qw, const float* sw, void* y, int64_t M, int64_t N, int64_t K,
                              void* workspace, hipStream_t st) {
    uint8_t* q = reinterpret_cast<uint8_t*>(workspace);
    float* s = reinterpret_cast<float*>(q + M * K);
    const hipError_t err = launch_quant_b128_act(x, M, K, q, s, st);
    return err != hipSuccess ? err : launch_gemm_b128(q, s, qw, sw, y, M, N, K, st);
}

hipError_t launch_gemm_b128_grouped(const void* qa, const float* sa, int64_t arows, const void* qw, const float* sw,
                                    void* y, const int32_t* offsets, const int32_t* rows, int64_t G, int64_t M, int64_t N,
                                    int64_t K, hipStream_t st) {
    return launch({reinterpret_cast<const uint8_t*>(qa), sa, reinterpret_cast<const uint8_t*>(qw), sw,
                   reinterpret_cast<uint16_t*>(y), offsets, rows, arows, M, N, K, (int)G}, st);
}

}  // namespace mx
