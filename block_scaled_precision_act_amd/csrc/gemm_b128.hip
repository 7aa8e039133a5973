// gemm_b128.hip - entries of the A8W8 GEMM with one FP32 scale per block of 128 (kernels: gemm_b128.hpp).
//
// Dense products take the tile whose rounds over the CUs are estimated cheapest: rounds = ceil(tiles / CUs), times the time
// of one round of that tile (kTiles; measured at K = 8192 and N = 7168, us, launch taken off), so a small product fills the
// CUs with small tiles and a large one is read least by large tiles.
//
// Grouped products stream the experts' weights, so a tile should hold a whole group and be wide: by the mean group's
// rows, with steps down while the tiles would leave half of the CUs idle.  Measured with 32 experts of [2048, 7168], us:
//   mean rows    2     4     8    16    32    64   128   256   512
//   16 x 64     87    91
//   32 x 128    79    85    87    98
//   64 x 128    78    84    87    89   102   118
//   128 x 128   86    90    90    93    97   116   142          405
//   256 x 256                                129   130   219   332
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
// for groups of up to `rows` rows in the mean; the first one only where wider tiles would be too few
struct GroupTile {
    double rows;
    int m, n;
    hipError_t (*launch)(const Args&, hipStream_t);
};
const GroupTile kGroupTiles[] = {
    {0, 16, 64, launch_tile<1, 4, 1, 1, 4, 3>},    {10, 32, 128, launch_tile<2, 4, 1, 2, 2, 3>},
    {24, 64, 128, launch_tile<2, 4, 2, 2, 1, 4>},  {90, 128, 128, launch_tile<2, 4, 4, 2, 1, 3>},
    {1e30, 256, 256, launch_tile<4, 8, 4, 2, 1, 2>},
};

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
    const GroupTile* t = kGroupTiles;
    while (rows > t->rows) ++t;
    auto tiles = [&](const GroupTile& g) {
        return groups * (double)(int64_t)((rows + g.m - 1) / g.m) * (double)((a.N + g.n - 1) / g.n);
    };
    while (t != kGroupTiles && 2 * tiles(*t) <= cus()) --t;
    return t->launch(a, st);
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
