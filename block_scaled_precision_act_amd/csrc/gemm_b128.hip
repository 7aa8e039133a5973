// gemm_b128.hip - entries of the A8W8 GEMM with one FP32 scale per block of 128 (kernels: gemm_b128.hpp).
//
// Dense products take the tile whose rounds over the CUs are estimated cheapest: rounds = ceil(tiles / CUs), times the time
// of one round of that tile (kTiles; measured at K = 8192 and N = 7168, us, launch taken off, weights in the last-level
// cache), so a small product fills the CUs with small tiles and a large one is read least by large tiles.  Over 67 shapes (M 3 to
// 8192, N 256 to 7168, K 512 to 8192) with weights in no cache the choice takes 1% more than the best of twelve tiles, 32% at worst.
//
// Few rows against weights in no cache take longer than the weights' stream (N = 7168, K = 8192, M = 16 / 32 / 64 / 128: 14.0 / 17.3
// / 19.5 / 24.9 us against 12.3 / 12.6 / 14.6 / 18.7 from the last-level cache): a CU's loads return in order, so its copies
// of activations, from L2, queue behind those of weights.  Fetching weight lines ahead, by the copying waves or by a
// wave of its own, takes places in the same queue and cost 2 to 4 us; tiles of 64 x 32 were as fast as 32 x 64.
//
// Grouped products take theirs by the same rule from the mean group (kGroupTiles; rounds at K = 7168 with weights from HBM),
// but not below the time that the weights take from memory at 5.4 TB/s; equal ones go to the larger tile.  Groups differ
// in size, so a group is counted as rows / height + 0.4 row tiles, one at least.  Over 90 measured combinations of 8 to 64
// groups, N 512 to 2048, K 2048 to 7168 and mean groups of 1 to 1024 rows (sizes off by 35%) the choice takes 1% more
// than the best tile, 19% at worst.  Some of them, 32 experts of [2048, 7168] and 8 of [2048, 7168], us:
//   mean rows        4    16    32    64   128   256   512  1024  |    4    16    64   256   512  1024
//   16 x 64         92   109   177   306   449   724                26    36    81
//   32 x 128        86    88   122   176   245   376   722          33    32    54    95
//   64 x 128        86    89    92   141   184   287   513   950    35    32    36    85   142   202
//   128 x 128       90    93    94   137   149   227   418   714    41    38    45    80   117   155
//   256 x 256       92    92    96   110   126   220   331   555    72    72    88   103   108   110
#include "gemm_b128.hpp"
#include "launch.hpp"

namespace mx {
namespace {

using b128::Args;

// The layer in one launch, for rows that the GEMM quantizes itself (see quant_rows_kernel).
constexpr int64_t kQuantRows = 2, kQuantLds = 32 * 1024;
constexpr int kQuantWaves = 16;
hipError_t launch_quant_rows(const Args& a, hipStream_t st) {
    hipLaunchKernelGGL((b128::quant_rows_kernel<kQuantWaves, 2>), dim3((unsigned)((a.N + 15) / 16)), dim3(64 * kQuantWaves),
                       (unsigned)b128::quant_lds_bytes(a.M, a.K, kQuantWaves), st, a);
    return hipGetLastError();
}
bool one_launch(int64_t M, int64_t K) { return M <= kQuantRows && b128::quant_lds_bytes(M, K, kQuantWaves) <= kQuantLds; }

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
template <int FN, int WM, int WN, int S>
hipError_t launch_heights(const Args& a, hipStream_t st) {
    constexpr int TM = 64 * WM, TN = 16 * FN * WN;
    const int64_t tm = a.M / TM + (a.G < a.M ? a.G : a.M), tn = (a.N + TN - 1) / TN;
    if (tm * tn > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((b128::tile_kernel_heights<FN, WM, WN, S>), dim3((unsigned)(tm * tn)), dim3(64 * WM * WN), 0, st, a, (int)tm,
                       (int)tn);
    return hipGetLastError();
}

struct Tile {
    int m, n;
    double round;  // us, see above
    hipError_t (*launch)(const Args&, hipStream_t);
};
const Tile kTiles[] = {
    {16, 32, 10.2, launch_tile<1, 2, 1, 1, 4, 4>},   {16, 64, 10.8, launch_tile<1, 4, 1, 1, 4, 3>},
    {32, 64, 12.5, launch_tile<2, 4, 1, 1, 4, 3>},   {64, 64, 15.8, launch_tile<2, 4, 2, 1, 2, 4>},
    {64, 128, 27.0, launch_tile<2, 4, 2, 2, 1, 4>},  {128, 128, 35.0, launch_tile<2, 4, 4, 2, 1, 3>},
    {256, 128, 64.8, launch_tile<4, 4, 4, 2, 1, 2>}, {256, 256, 109.0, launch_tile<4, 8, 4, 2, 1, 2>},
};
const Tile kGroupTiles[] = {
    {16, 64, 12.0, launch_tile<1, 4, 1, 1, 4, 3>},   {32, 128, 24.0, launch_tile<2, 4, 1, 2, 2, 3>},
    {64, 128, 34.0, launch_tile<2, 4, 2, 2, 1, 4>},  {128, 128, 46.0, launch_tile<2, 4, 4, 2, 1, 3>},
    {256, 256, 100.0, launch_heights<8, 4, 2, 2>},
};
constexpr double kWeightBytesPerUs = 5.4e6;

int cus() { return device_cus() > 0 ? device_cus() : 256; }

hipError_t launch(const Args& a, hipStream_t st) {
    const Tile* best = nullptr;
    double least = 0;
    for (const Tile& t : kTiles) {
        const int64_t tiles = ((a.M + t.m - 1) / t.m) * ((a.N + t.n - 1) / t.n);
        const double time = (double)((tiles + cus() - 1) / cus()) * t.round;
        if (!best || time < least) {
            best = &t;
            least = time;
        }
    }
    return best->launch(a, st);
}

hipError_t launch_grouped(const Args& a, hipStream_t st) {
    const double groups = (double)(a.G < a.M ? a.G : a.M), rows = (double)a.M / groups;
    const double stream = groups * (double)a.N * (double)a.K / kWeightBytesPerUs;
    const Tile* best = nullptr;
    double least = 0;
    for (const Tile& t : kGroupTiles) {
        const double high = rows / t.m + 0.4;
        const double tiles = groups * (high > 1 ? high : 1) * (double)((a.N + t.n - 1) / t.n);
        const double work = __builtin_ceil(tiles / cus()) * t.round * ((double)a.K / 7168), time = work > stream ? work : stream;
        if (!best || time <= least) {
            best = &t;
            least = time;
        }
    }
    return best->launch(a, st);
}

}  // namespace

hipError_t launch_gemm_b128(const void* qa, const float* sa, const void* qw, const float* sw, void* y, int64_t M, int64_t N,
                            int64_t K, hipStream_t st) {
    return launch({nullptr, reinterpret_cast<const uint8_t*>(qa), sa, reinterpret_cast<const uint8_t*>(qw), sw,
                   reinterpret_cast<uint16_t*>(y), nullptr, nullptr, M, M, N, K, 1}, st);
}

// codes [M, K], then scales [M, K / 128]
size_t linear_b128_workspace_bytes(int64_t M, int64_t, int64_t K) {
    return one_launch(M, K) ? 0 : (size_t)M * K + (size_t)M * (K / 128) * 4;
}

hipError_t launch_linear_b128(const void* x, const void* qw, const float* sw, void* y, int64_t M, int64_t N, int64_t K,
                              void* workspace, hipStream_t st) {
    if (one_launch(M, K))
        return launch_quant_rows({reinterpret_cast<const uint16_t*>(x), nullptr, nullptr, reinterpret_cast<const uint8_t*>(qw),
                                  sw, reinterpret_cast<uint16_t*>(y), nullptr, nullptr, M, M, N, K, 1}, st);
    uint8_t* q = reinterpret_cast<uint8_t*>(workspace);
    float* s = reinterpret_cast<float*>(q + M * K);
    const hipError_t err = launch_quant_b128_act(x, M, K, q, s, st);
    return err != hipSuccess ? err : launch_gemm_b128(q, s, qw, sw, y, M, N, K, st);
}

hipError_t launch_gemm_b128_grouped(const void* qa, const float* sa, int64_t arows, const void* qw, const float* sw,
                                    void* y, const int32_t* offsets, const int32_t* rows, int64_t G, int64_t M, int64_t N,
                                    int64_t K, hipStream_t st) {
    return launch_grouped({nullptr, reinterpret_cast<const uint8_t*>(qa), sa, reinterpret_cast<const uint8_t*>(qw), sw,
                           reinterpret_cast<uint16_t*>(y), offsets, rows, arows, M, N, K, (int)G}, st);
}

}  // namespace mx
