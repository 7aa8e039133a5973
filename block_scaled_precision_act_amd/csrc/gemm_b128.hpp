// gemm_b128.hpp - kernels of the A8W8 GEMM with one FP32 scale per block of 128, dense and grouped over experts.
//
//   Y[m, n] = sum_b sa[m, b] sw[n / 128, b] P_b[m, n],   P_b[m, n] = sum_{k in block b} qa[m, k] qw[n, k]
//
// with E4M3 codes and b the 128-value blocks of K.  P_b is one FP8 MFMA of depth 128 started from zero;
// the scaled sum over blocks runs in FP32 on the vector ALU: acc = fma(P_b, sa sw, acc).
//
// Precision.  The FP8 MFMA adds the 128 products of a block in groups of eight, and cuts each product at 2^-13
// of the power of two of its group's largest one (measured on this GPU, toward zero); the groups are added
// with FP32's width.  So a block's sum is off by less than 7 * 2^-13 of the sum of its products' magnitudes whatever the
// codes; quantized normal values measured 2^-15.5 at most over a million outputs (2^-19 root mean square), and 2^-12
// beside a column of 448s.  That is far below the rounding of the BF16 output except for strongly cancelling sums.
// The per-row-scale GEMM of this library widens its codes to FP16 instead, which is exact up to FP32 but runs at half
// the matrix rate; with a scale per block, blocks have to leave the MFMA for their FP32 sum anyway, and the FP8 rate
// is kept.
//
// Operand layout: lane l holds row l % 16 of a fragment and, of the block's eight 16-byte chunks, chunks
// l / 16 and l / 16 + 4.  Both operands use the same order, and the order of K inside a block does not
// matter, so a wave's two loads of a fragment each take 64 contiguous bytes per row.  Weights are the
// first operand: a lane's four results are four consecutive n of one m, which share one activation scale.
#pragma once

#include "fp8_device.hpp"

namespace mx {
namespace b128 {

constexpr int kFmtE4M3 = 0;  // scaled-MFMA operand format; scale operands 0 select the MFMA without scales

__device__ __forceinline__ v8i operand(uint4 lo, uint4 hi) {
    v8i r = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    return r;
}
__device__ __forceinline__ v8i operand(v4u lo, v4u hi) {
    v8i r = {(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    return r;
}
// 16 x 16 products of one block, from zero
__device__ __forceinline__ v4f block_mfma(v8i w, v8i x) {
    const v4f z = {0.f, 0.f, 0.f, 0.f};
    return mfma16<kFmtE4M3, 0>(w, x, z, 0, 0);
}

// 16 or 4 bytes per lane from a buffer straight into LDS: lane i of the wave writes lds_base + 16 i or 4 i.
__device__ __forceinline__ void buffer2lds16(__amdgpu_buffer_rsrc_t r, void* lds_base, uint32_t lane_offset, int offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds_base, 16, lane_offset, offset, 0, 0);
}
__device__ __forceinline__ void buffer2lds4(__amdgpu_buffer_rsrc_t r, void* lds_base, uint32_t lane_offset, int offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds_base, 4, lane_offset, offset, 0, 0);
}

struct Args {
    const uint16_t* x;      // BF16 [M, K] instead of qa and sa, for the kernel that quantizes
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
// The A row that feeds row r of Y, -1 if there is none (its outputs are 0)
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

// ---------------------------------------------------------------------------- a row or two, quantized on the way
// The layer for M <= 16 rows of BF16, in one launch: one workgroup per 16 columns; its W waves take contiguous parts of K
// and meet in LDS, summed in wave order.  Every wave quantizes its part of the rows into LDS, bit for bit as the
// quantizer kernel, while its first weights are on the way; weights go from memory to registers through a ring of
// D stages of one block.  Every workgroup quantizes all rows, so this pays for very few of them only (measured at N =
// 7168, K = 8192, quantizer launch included: M = 1 / 2 12.3 / 12.9 us against 14.2 / 14.3, M = 4 15.0 against 14.4).
struct Stage {
    uint4 w[2];
    float sw;
};

// codes of one row and wave, padded by a chunk so that rows start in different banks
__host__ __device__ constexpr int quant_row_bytes(int blocks) { return blocks * 128 + 16; }
// bytes of dynamic LDS: codes and scales of M rows
__host__ inline int64_t quant_lds_bytes(int64_t M, int64_t K, int W) {
    const int64_t per = (K / 128 + W - 1) / W;
    return W * M * (per * 128 + 16 + per * 4);
}

template <int W, int D>
__global__ __launch_bounds__(64 * W) void quant_rows_kernel(Args a) {
    __shared__ v4f red[W][64];
    extern __shared__ __attribute__((aligned(16))) uint8_t codes[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4, M = (int)a.M;
    const int nkb = (int)(a.K / 128), per = (nkb + W - 1) / W;
    const int kb0 = min(wave * per, nkb), nk = min(per, nkb - kb0);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const uint8_t* wp = a.qw + min(n0 + l16, a.N - 1) * a.K + 16 * g + (int64_t)kb0 * 128;
    const float* swp = a.sw + n0 / 128 * nkb + kb0;
    const int pitch = quant_row_bytes(per), r = min(l16, M - 1);
    uint8_t* own = codes + wave * M * pitch;
    float* scales = reinterpret_cast<float*>(codes + W * M * pitch) + wave * M * per;

    v4f acc = {};
    Stage st[D];
    auto load = [&](Stage& s, int i) __attribute__((always_inline)) {
        s.w[0] = ldg16(wp + i * 128);
        s.w[1] = ldg16(wp + i * 128 + 64);
        s.sw = swp[i];
    };
    auto compute = [&](const Stage& s, int i) __attribute__((always_inline)) {
        const uint8_t* x = own + r * pitch + i * 128 + 16 * g;
        const v4f p = block_mfma(operand(s.w[0], s.w[1]), operand(ldg16(x), ldg16(x + 64)));
        const float sc = scales[r * per + i] * s.sw;
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = __builtin_fmaf(p[k], sc, acc[k]);
    };
    if (nk > 0) {
        static_for<D - 1>([&](auto d) { load(st[decltype(d)::value], min((int)decltype(d)::value, nk - 1)); });
        __builtin_amdgcn_sched_barrier(0);
        // 16 lanes per block of 128, four blocks of this wave's part at a time; only this wave reads them back
        for (int b0 = 0; b0 < M * nk; b0 += 4) {
            const int b = b0 + (lane >> 4);
            if (b < M * nk) {
                const int m = b / nk, i = b % nk;
                const uint4 x = *reinterpret_cast<const uint4*>(a.x + m * a.K + (int64_t)(kb0 + i) * 128 + 8 * l16);
                float s;
                *reinterpret_cast<uint2*>(own + m * pitch + i * 128 + 8 * l16) = quant_block_bf16x8(x, s);
                if (l16 == 0) scales[m * per + i] = s;
            }
        }
        for (int i = 0; i < nk; i += D)
            static_for<D>([&](auto dc) {
                constexpr int d = decltype(dc)::value;
                if (i + d < nk) {
                    if (i + d + D - 1 < nk) load(st[(d + D - 1) % D], i + d + D - 1);
                    compute(st[d], i + d);
                }
            });
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
        v4f s = red[0][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) s += red[w][lane];
        if (l16 < M) store4(a.y + l16 * a.N, a.N, n0 + 4 * g, s, a.N % 4 == 0 && ((uintptr_t)a.y & 7) == 0);
    }
}

// ---------------------------------------------------------------------------- many rows
// A TM x TN = 16 FM WM x 16 FN WN output tile per workgroup.  KG groups of WM x WN waves take every KG-th block of
// K (group q blocks q, q + KG, ...) and are summed in group order at the end; a step is one block per group.  Operands
// pass through a ring of S slots in LDS, filled by direct copies.
//
// Slot, per group: TM + TN rows of 128 bytes, chunk c of row r at place c ^ (r / 2 % 8), so that the 16 lanes of a
// fragment's read touch 16 different bank groups.  Scales come in batches of eight (or sixteen) blocks, three of
// them in LDS: a copy takes 32 bytes from each of eight rows (64 from four), and the copies of batch B travel with
// the codes of the steps of batch B - 1, one per wave and step.  The blocks of a row are permuted by the row's part of 16,
// so that the 16 rows of a fragment lie in different banks.  (Copying each step's scales, one 4-byte piece of a cache line per
// row, took as many line requests as the codes.)
//
// Step u of a wave, its first weight fragment, its row fragments and its scales already in registers:
//   1. all but the last two or three weight fragments times all row fragments, reading weight fragments ahead;
//   2. every operand of the step is now in registers: wait for the copies of u + 1, one barrier;
//   3. the last weight fragments, row fragment by row fragment, reading the next step's scales, first weight fragment
//      and row fragments as registers fall free.
// With three fragments behind the barrier where registers allow, LDS reads spread evenly over the MFMAs.
// So MFMAs run across the barrier.  The slot that the barrier frees is refilled with the copies of u + S, spread over the
// MFMAs of 3 and of the next step's 1: issued in one burst they hold up the waves behind the address unit.  The FMAs that scale a product follow two
// MFMAs behind it.
//
// LDS reads are inline assembly (the compiler would drain the copies before each one).  The compiler takes their
// results for ready at once, so nothing may touch a result register before the wait that covers it: every wait ties its
// results, and what is carried into the next step is waited for and tied before the step ends, ahead of any
// register copy the loop may need.  test_isa_hazards_b128.py checks that in the assembly.
struct TileAt {
    int e;            // group
    int64_t m0, r1;   // first row, end of the group's rows
    int64_t n0;
    int tm, tn;       // row and column tile
    int height;       // rows
    bool live;
};

// Row tiles of groups g0 .. g0 + 63, one group per lane: the lane's own, their height, and the running sum of tiles.  A
// group takes as few tiles of up to TM rows as it can, all of one height, the least multiple of STEP that does.
template <int TM, int STEP>
__device__ __forceinline__ int group_tiles(const Args& a, int g0, int64_t& r0, int64_t& r1, int& own, int& height) {
    const int lane = threadIdx.x & 63;
    r0 = r1 = 0;
    if (g0 + lane < a.G) group_rows(a, g0 + lane, r0, r1);
    own = r1 > r0 ? (int)((r1 - r0 + TM - 1) / TM) : 0;
    height = TM;
    if constexpr (STEP < TM) height = own > 0 ? (int)(((r1 - r0 + own - 1) / own + STEP - 1) / STEP * STEP) : TM;
    int sum = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(sum, d);
        if (lane >= d) sum += o;
    }
    return sum;
}

// Workgroup b's tile.  Consecutive workgroups go to the 8 XCDs in turn; each XCD takes a contiguous run of tiles,
// and walks it in bands of four row tiles, so tiles that run together share operand panels in its L2.  Grouped: the row
// tiles of all groups one after another; the grid has room for more than there are, and only those that there are are
// dealt out (dealing out the whole grid left an XCD idle).
template <int TM, int TN, int STEP>
__device__ __forceinline__ TileAt tile_of(const Args& a, int b, int tiles_m, int tiles_n) {
    int64_t r0, r1;
    int own, height;
    if (a.offsets) {
        int rows = 0;
        for (int g0 = 0; g0 < a.G; g0 += 64)
            rows += __builtin_amdgcn_readlane(group_tiles<TM, STEP>(a, g0, r0, r1, own, height), 63);
        tiles_m = min(tiles_m, rows);
    }
    const int T = tiles_m * tiles_n, T8 = T & ~7;
    const int L = b < T8 ? (b & 7) * (T8 >> 3) + (b >> 3) : b;
    TileAt t = {0, 0, a.M, 0, 0, 0, TM, b < T};
    if (!t.live) return t;
    const int band = L / (4 * tiles_n), high = min(tiles_m - 4 * band, 4), rem = L - band * 4 * tiles_n;
    t.tm = 4 * band + rem % high;
    t.tn = rem / high;
    t.m0 = (int64_t)t.tm * TM;
    t.n0 = (int64_t)t.tn * TN;
    if (a.offsets == nullptr) return t;
    t.live = false;
    int left = t.tm;
    for (int g0 = 0; g0 < a.G; g0 += 64) {
        const int sum = group_tiles<TM, STEP>(a, g0, r0, r1, own, height);
        const uint64_t past = __ballot(sum > left);
        if (past) {
            const int i = __builtin_ctzll(past);
            t.e = g0 + i;
            t.height = __builtin_amdgcn_readlane(height, i);
            t.m0 = __builtin_amdgcn_readlane((int)r0, i) + (int64_t)(left - __builtin_amdgcn_readlane(sum - own, i)) * t.height;
            t.r1 = __builtin_amdgcn_readlane((int)r1, i);
            t.live = true;
            break;
        }
        left -= __builtin_amdgcn_readlane(sum, 63);
    }
    return t;
}

// one tile's bytes of LDS: the ring, three batches of scales, their table, a place for lines fetched ahead
constexpr int tile_lds(int FM, int FN, int WM, int WN, int KG, int S) {
    return S * KG * 16 * (FM * WM + FN * WN) * 128 + 3 * (16 * FM * WM + 8) * (KG == 4 ? 16 : 8) * 4 + (16 * FM * WM + 8) * 4 + 256;
}

template <int FM, int FN, int WM, int WN, int KG, int S>
__device__ __forceinline__ void tile(const Args& a, const TileAt& t, uint8_t* lds) {
    constexpr int TM = 16 * FM * WM, TN = 16 * FN * WN, W = WM * WN * KG;
    constexpr int CA = (KG * TM / 8 + W - 1) / W, CW = (KG * TN / 8 + W - 1) / W;  // copies of eight rows per wave
    constexpr bool kAhead = S == 2 && TM * TN >= 256 * 128;                        // lines fetched ahead into L2
    constexpr int C = CA + CW + 1 + kAhead;                                        // and one of scales
    constexpr int kPart = (TM + TN) * 128, kSlot = KG * kPart, kBatches = S * kSlot;
    // a batch of scales: BB blocks of TM rows and of up to eight weight blocks, in parts of 64 scales
    constexpr int BB = KG == 4 ? 16 : 8, kBatch = (TM + 8) * BB * 4, kPer = 64 / BB, kParts = (TM + 8) / kPer;
    constexpr int kTable = kBatches + 3 * kBatch, kSink = kTable + (TM + 8) * 4, kLds = kSink + 256;
    constexpr int SB = BB / KG;  // steps per batch of scales
    // MFMAs of a step, and those ahead of its barrier; the copies issued behind the barrier that frees their slot (the
    // others follow in the next step, ahead of its barrier), and the MFMAs that those others are spread over
    constexpr int kLast = FN >= 6 ? 3 : 2, kAhd = FN - kLast, kPre = kAhd == 0 ? FN : 1;  // fragments behind, ahead of the barrier; read early
    constexpr int kMf = FN * FM, kFirst = kAhd * FM, kRest = kMf - kFirst;
    constexpr int kWish = kFirst == 0 ? C : kFirst >= 2 * C ? (kRest + 1) / 2 : kRest, kEarly = kWish < C ? kWish : C;
    constexpr int kLate = C - kEarly, kSpan = 2 * kLate < kFirst ? 2 * kLate : kFirst;
    constexpr bool kOneBlock = 128 % (16 * FN) == 0;    // a wave's columns lie in one weight block
    constexpr int kFree = FM > 2 && FN < 8 ? 2 : FM > 1 ? 1 : 0;  // row fragments read into registers of their own
    static_assert(kParts <= SB * W && S <= SB, "a batch's copies in its steps, and its place free in time");
    static_assert(kLds == tile_lds(FM, FN, WM, WN, KG, S) && kLds <= 160 * 1024 && (S - 1) * C < 64 && FN >= 2 && FN <= 8, "LDS, counters, weight scales");
    static_assert((KG - 1) * FM * FN * 1024 * WM * WN <= kBatches, "sums of the groups");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4, kg = wave / (WM * WN), wm = wave / WN % WM, wn = wave % WN;
    const int nkb = __builtin_amdgcn_readfirstlane((int)(a.K / 128)), steps = (nkb + KG - 1) / KG;
    const int64_t nblocks = (a.N + 127) / 128, nb0 = t.n0 / 128;

    // Copies are buffer loads: a 32-bit offset per lane, the block of K in the scalar offset.  Rows are counted from the
    // tile's first one, or from A's where a table names them.
    const int64_t arow0 = a.rows ? 0 : t.m0;
    constexpr int kRawWord3 = 0x00020000;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)(a.qa + arow0 * a.K), (short)0, -1, kRawWord3);
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc((void*)(a.qw + (t.e * a.N + t.n0) * a.K), (short)0, -1, kRawWord3);
    const __amdgpu_buffer_rsrc_t rsa = __builtin_amdgcn_make_buffer_rsrc((void*)(a.sa + arow0 * nkb), (short)0, -1, kRawWord3);
    const __amdgpu_buffer_rsrc_t rsw =
        __builtin_amdgcn_make_buffer_rsrc((void*)(a.sw + (t.e * nblocks + nb0) * nkb), (short)0, -1, kRawWord3);
    auto tile_row = [&](int i) { return (uint32_t)(max(a_row(a, min(t.m0 + i, t.r1 - 1)), (int64_t)0) - arow0); };

    // offsets of the rows of the scale copies: the tile's A rows, then weight blocks
    uint32_t* table = reinterpret_cast<uint32_t*>(lds + kTable);
    for (int i = threadIdx.x; i < TM + 8; i += 64 * W)
        table[i] = (i < TM ? tile_row(i) : (uint32_t)min((int64_t)i - TM, nblocks - 1 - nb0)) * (uint32_t)nkb * 4;

    // code copy i: eight rows of one group's block, a 16-byte chunk per lane.  Every wave issues C copies a step, so that
    // one count serves them all; where they do not divide, some repeat the last.
    uint32_t src[CA + CW];
    int dst[CA + CW], grp[CA + CW];
#pragma unroll
    for (int i = 0; i < CA + CW; ++i) {
        const int rows8 = i < CA ? TM / 8 : TN / 8;
        const int q = min(wave + (i < CA ? i : i - CA) * W, KG * rows8 - 1);
        grp[i] = q / rows8;
        const int row = q % rows8 * 8 + (lane >> 3);
        dst[i] = grp[i] * kPart + (i < CA ? 0 : TM * 128) + q % rows8 * 1024;
        const uint32_t r = i < CA ? tile_row(row) : (uint32_t)min((int64_t)row, a.N - 1 - t.n0);
        src[i] = r * (uint32_t)a.K + 16 * ((lane & 7) ^ (row >> 1 & 7));
    }
    // the scale copy that this wave issues in step c of a batch
    auto part_of = [&](int c) __attribute__((always_inline)) { return min((c & (SB - 1)) * W + wave, kParts - 1); };
    struct ScaleCopy {
        uint32_t at;  // the lane's offset
        int dst;
        bool weights;
    };
    auto scale_copy = [&](int b, int q, uint32_t row) __attribute__((always_inline)) {  // part q of batch b; row: from the table
        return ScaleCopy{row + 4 * min(BB * b + ((lane & (BB - 1)) ^ (q & (16 / kPer - 1))), nkb - 1),
                         kBatches + b % 3 * kBatch + q * 256, q >= TM / kPer};
    };
    auto issue_scale = [&](const ScaleCopy& c) __attribute__((always_inline)) { buffer2lds4(c.weights ? rsw : rsa, lds + c.dst, c.at, 0); };
    // Lines fetched ahead into L2: the 32 tiles that an XCD runs at a time are four row tiles by eight column tiles, so each
    // fetches an eighth of its A rows and a quarter of its weight rows, one 4-byte piece of every line, two steps before
    // the copies need them.  Without it every step waits for the first reader's miss.
    constexpr int kDistance = 2, kLines = (TM / 8 + TN / 4 + W - 1) / W;
    const int line = wave * kLines + min(lane, kLines - 1);
    const bool ahead_w = wave * kLines >= TM / 8;
    const uint32_t ahead = (ahead_w ? (uint32_t)min((int64_t)(t.tm & 3) * (TN / 4) + min(line - TM / 8, TN / 4 - 1), a.N - 1 - t.n0)
                                    : tile_row((t.tn & 7) * (TM / 8) + min(line, TM / 8 - 1))) * (uint32_t)a.K;
    const uint8_t* ahead_base = ahead_w ? a.qw + (t.e * a.N + t.n0) * a.K : a.qa + arow0 * a.K;
    const __amdgpu_buffer_rsrc_t rahead = __builtin_amdgcn_make_buffer_rsrc((void*)ahead_base, (short)0, -1, kRawWord3);
    int ahead_at = min(kDistance * KG, nkb - 1) * 128;
    // copy i of the C that go with step u, into its slot (blocks past the end: the last one again)
    auto issue = [&](int u, int slot, int i, const ScaleCopy& sc) __attribute__((always_inline)) {
        if (i == 0) issue_scale(sc);
        else if (i == CA + CW + 1) {
            buffer2lds4(rahead, lds + kSink, ahead, ahead_at);
            ahead_at = min(ahead_at + KG * 128, (nkb - 1) * 128);
        } else buffer2lds16(i <= CA ? ra : rw, lds + slot * kSlot + dst[i - 1], src[i - 1], min(u * KG + grp[i - 1], nkb - 1) * 128);
    };

    // LDS addresses: a per-lane base plus the slot and an immediate
    const uint32_t base = lds_addr(lds);
    const int key = l16 >> 1;
    const uint32_t c0 = 16 * (g ^ key), c1 = 16 * ((g + 4) ^ key);
    const uint32_t xrow = base + kg * kPart + (16 * FM * wm + l16) * 128, wrow = base + kg * kPart + TM * 128 + (16 * FN * wn + l16) * 128;
    const uint32_t x0 = xrow + c0, x1 = xrow + c1, w0 = wrow + c0, w1 = wrow + c1;
    const uint32_t xs = base + kBatches + 4 * BB * (16 * FM * wm + l16);
    // weight scales: fragment f is in block (n / 128) of its first column; the wave's fragments touch two at most
    const int nw = (int)(t.n0 - nb0 * 128) + 16 * FN * wn;  // from the first block's start
    const uint32_t ws = base + kBatches + 4 * BB * (TM + nw / 128);
    const int cut = 8 - nw % 128 / 16;  // fragments f < cut are in the first of the two
    const uint32_t trow = base + kTable + 4 * (lane / BB);

    v4f acc[FN][FM] = {};
    v4u wl[FN], wh[FN], xl[FM], xh[FM];
    uint32_t sx[FM], sw[2], row[1];

    __syncthreads();  // the table
    for (int q = wave; q < kParts; q += W) issue_scale(scale_copy(0, q, table[kPer * q + lane / BB]));
    uint32_t first[S];
#pragma unroll
    for (int s = 0; s < S; ++s) first[s] = table[kPer * part_of(s) + lane / BB];
    wait_vmcnt<0>();
    static_for<S>([&](auto s) {
        static_for<C>([&](auto i) {
            if (s < S - 1 || i < kEarly) issue(s, s, i, scale_copy(1, part_of(s), first[s]));
        });
    });
    // offsets of step u's scales (this group's block) in the batches: the weights', and this lane's rows'
    auto scales_at = [&](int u, int part) __attribute__((always_inline)) {
        const int b = u * KG + kg;
        return (uint32_t)(b / BB % 3 * kBatch + 4 * ((b & (BB - 1)) ^ part));
    };
    wait_vmcnt<(S - 2) * C + kEarly>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    static_for<2>([&](auto i) { sw[i] = lds_read4(scales_at(0, 0) + ws + 4 * BB * i); });
    static_for<kPre>([&](auto i) {
        wl[i] = lds_read16_at<i * 2048>(w0);
        wh[i] = lds_read16_at<i * 2048>(w1);
    });
    static_for<FM>([&](auto j) {
        sx[j] = lds_read4(scales_at(0, l16 / kPer) + xs + 64 * BB * j);
        xl[j] = lds_read16_at<j * 2048>(x0);
        xh[j] = lds_read16_at<j * 2048>(x1);
    });
    row[0] = lds_read4(trow + 4 * kPer * part_of(S));
    // ends a step: what is carried into the next one has arrived
    auto arrive = [&]() __attribute__((always_inline)) {
        lds_wait<0>();
#pragma unroll
        for (int i = 0; i < kPre; ++i) asm volatile("" : "+v"(wl[i]), "+v"(wh[i]));
        lds_tie(sx);
        lds_tie(sw);
        lds_tie(xl);
        lds_tie(xh);
        lds_tie(row);
        __builtin_amdgcn_sched_barrier(0);
    };
    arrive();

    // step u in slot s
    auto step = [&](int u, auto sc) __attribute__((always_inline)) {
        constexpr int s = decltype(sc)::value;
        constexpr uint32_t at = s * kSlot, next = (s + 1) % S * kSlot;
        // a group's block past the end repeats the last one, times 0
        const bool inside = KG == 1 || u * KG + kg < nkb;
        float fx[FM];
#pragma unroll
        for (int j = 0; j < FM; ++j) fx[j] = inside ? __uint_as_float(sx[j]) : 0.f;
        const float fw0 = inside ? __uint_as_float(__builtin_amdgcn_readfirstlane(sw[0])) : 0.f,
                    fw1 = inside ? __uint_as_float(__builtin_amdgcn_readfirstlane(sw[1])) : 0.f;
        if constexpr (kOneBlock) {
#pragma unroll
            for (int j = 0; j < FM; ++j) fx[j] *= fw0;
        }
        ScaleCopy copy = {};
        uint32_t sat = 0, xat = 0, tat = 0;  // addresses of the next step's scales and table entry
        auto place = [&](int part) __attribute__((always_inline)) {
            if (part == 0) copy = scale_copy((u + S) / SB + 1, part_of(u + S), row[0]);
            if (part == 1) sat = scales_at(u + 1, 0) + ws, xat = scales_at(u + 1, l16 / kPer) + xs;
            if (part == 2) tat = trow + 4 * kPer * part_of(u + 1 + S);
        };
        if constexpr (kFirst == 0) place(0), place(1), place(2);
        v4f p[3];
        v4u nwl[kPre], nwh[kPre], nxl[kFree + 1], nxh[kFree + 1];
        uint32_t nrow[1];
        auto scale = [&](auto ic, int f, int j) __attribute__((always_inline)) {
            const v4f v = p[decltype(ic)::value % 3];
            const float m = kOneBlock ? fx[j] : fx[j] * (f < cut ? fw0 : fw1);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[f][j][i] = __builtin_fmaf(v[i], m, acc[f][j][i]);
        };
        // MFMA i's fragments: weight-major, then the last weight fragments row by row
        auto fof = [](int i) constexpr { return i < kFirst ? i / FM : kAhd + (i - kFirst) % kLast; };
        auto jof = [](int i) constexpr { return i < kFirst ? i % FM : (i - kFirst) / kLast; };
        // the last weight fragment whose reads are issued by the start of fragment f: two ahead, or evenly
        auto upto = [](int f) constexpr {
            const int even = kAhd == 0 ? 0 : ((f + 1) * (FN - 1) + kAhd - 1) / (kAhd == 0 ? 1 : kAhd), two = f + 2;
            return f < 0 ? kPre - 1 : (even > two ? even : two) < FN - 1 ? (even > two ? even : two) : FN - 1;
        };
        static_for<kMf>([&](auto ic) {
            constexpr int i = decltype(ic)::value, f = fof(i), j = jof(i);
            if constexpr (i < kFirst && j == 0) {
                if constexpr (f >= kPre) {
                    lds_wait<2 * (upto(f - 1) - f)>();
                    asm volatile("" : "+v"(wl[f]), "+v"(wh[f]));
                }
                static_for<upto(f) - upto(f - 1)>([&](auto q) {
                    constexpr int r = upto(f - 1) + 1 + q;
                    wl[r] = lds_read16_at<r * 2048>(w0 + at);
                    wh[r] = lds_read16_at<r * 2048>(w1 + at);
                });
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (i == kFirst) {
                if constexpr (kAhd > 0) {
                    lds_wait<0>();
#pragma unroll
                    for (int q = kAhd; q < FN; ++q) asm volatile("" : "+v"(wl[q]), "+v"(wh[q]));
                }
                wait_vmcnt<(S - 2) * C + kAhead>();  // the line fetch is the last of a step's copies
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (kFirst == 0) static_for<C>([&](auto q) { issue(u + S, s, q, copy); });
            }
            p[i % 3] = block_mfma(operand(wl[f], wh[f]), operand(xl[j], xh[j]));
            __builtin_amdgcn_sched_barrier(0);  // the product two back is scaled behind this MFMA, not ahead of it
            if constexpr (i >= 2) scale(std::integral_constant<int, i - 2>{}, fof(i - 2), jof(i - 2));
            // ahead of the barrier: what the reads and copies behind it need
            if constexpr (kFirst > 0) static_for<3>([&](auto q) { if (i == q * kFirst / 3) place(q); });
            // behind it: the next step's first weight fragments, last row fragments, scales and table entry, spread evenly
            if constexpr (i >= kFirst) {
                constexpr int kReads = kPre + kFree + 2 + FM + 1, k = i - kFirst;
                static_for<(k + 1) * kReads / kRest - k * kReads / kRest>([&](auto z) {
                    constexpr int q = k * kReads / kRest + z, x = q - kPre, c = x - kFree, r = c - 2;
                    if constexpr (q < kPre) {
                        nwl[q] = lds_read16_at<q * 2048>(w0 + next);
                        nwh[q] = lds_read16_at<q * 2048>(w1 + next);
                    } else if constexpr (x < kFree) {
                        nxl[x] = lds_read16_at<(FM - kFree + x) * 2048>(x0 + next);
                        nxh[x] = lds_read16_at<(FM - kFree + x) * 2048>(x1 + next);
                    } else if constexpr (c < 2) {
                        sw[c] = lds_read4(sat + 4 * BB * c);
                    } else if constexpr (r < FM) {
                        sx[r] = lds_read4(xat + 64 * BB * r);
                    } else {
                        nrow[0] = lds_read4(tat);
                    }
                });
            }
            // copies: the slot of the step before, then this step's
            if constexpr (i < kSpan)
                static_for<(i + 1) * kLate / kSpan - i * kLate / kSpan>(
                    [&](auto q) { issue(u - 1 + S, (s + S - 1) % S, kEarly + i * kLate / kSpan + q, copy); });
            if constexpr (i >= kFirst && kFirst > 0) {
                constexpr int k = i - kFirst;
                static_for<(k + 1) * kEarly / kRest - k * kEarly / kRest>(
                    [&](auto q) { issue(u + S, s, k * kEarly / kRest + q, copy); });
            }
            // row fragment j is free one MFMA after its last use
            if constexpr (i > kFirst && (i - kFirst) % kLast == 0 && (i - kFirst) / kLast - 1 < FM - kFree) {
                constexpr int q = (i - kFirst) / kLast - 1;
                xl[q] = lds_read16_at<q * 2048>(x0 + next);
                xh[q] = lds_read16_at<q * 2048>(x1 + next);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        scale(std::integral_constant<int, kMf - 2>{}, fof(kMf - 2), jof(kMf - 2));
        if constexpr (kFree == 0) {
            xl[FM - 1] = lds_read16_at<(FM - 1) * 2048>(x0 + next);
            xh[FM - 1] = lds_read16_at<(FM - 1) * 2048>(x1 + next);
        }
        scale(std::integral_constant<int, kMf - 1>{}, fof(kMf - 1), jof(kMf - 1));
        __builtin_amdgcn_sched_barrier(0);
        lds_wait<0>();
        lds_tie(nrow);
        row[0] = nrow[0];
#pragma unroll
        for (int q = 0; q < kPre; ++q) {
            asm volatile("" : "+v"(nwl[q]), "+v"(nwh[q]));
            wl[q] = nwl[q], wh[q] = nwh[q];
        }
#pragma unroll
        for (int q = 0; q < kFree; ++q) {
            asm volatile("" : "+v"(nxl[q]), "+v"(nxh[q]));
            xl[FM - kFree + q] = nxl[q], xh[FM - kFree + q] = nxh[q];
        }
        arrive();
    };
    for (int u = 0; u < steps; u += S)
        static_for<S>([&](auto s) {
            if (u + s < steps) step(u + s, s);
        });
    wait_vmcnt<0>();  // the copies past the end still write to LDS

    if constexpr (KG > 1) {  // the groups' sums through LDS, in group order
        __syncthreads();
        v4f* red = reinterpret_cast<v4f*>(lds) + (wm * WN + wn) * FN * FM * 64 + lane;
        constexpr int kGroup = WM * WN * FN * FM * 64;
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < FN * FM; ++i) red[(kg - 1) * kGroup + i * 64] = acc[i / FM][i % FM];
        }
        __syncthreads();
        if (kg > 0) return;
#pragma unroll
        for (int q = 0; q < KG - 1; ++q)
#pragma unroll
            for (int i = 0; i < FN * FM; ++i) acc[i / FM][i % FM] += red[q * kGroup + i * 64];
    }
    const bool vec = a.N % 4 == 0 && ((uintptr_t)a.y & 7) == 0;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int64_t m = t.m0 + 16 * (FM * wm + j) + l16;
        if (m >= t.r1) continue;
        const bool ok = a_row(a, m) >= 0;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            const v4f zero = {0.f, 0.f, 0.f, 0.f};
            store4(a.y + m * a.N, a.N, t.n0 + 16 * (FN * wn + f) + 4 * g, ok ? acc[f][j] : zero, vec);
        }
    }
}

template <int FM, int FN, int WM, int WN, int KG, int S>
__global__ __launch_bounds__(64 * WM * WN * KG, WM * WN * KG >= 8 ? 2 : 1) void tile_kernel(Args a, int tiles_m, int tiles_n) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[tile_lds(FM, FN, WM, WN, KG, S)];
    constexpr int TM = 16 * FM * WM;
    const TileAt t = tile_of<TM, 16 * FN * WN, TM>(a, blockIdx.x, tiles_m, tiles_n);
    if (t.live) tile<FM, FN, WM, WN, KG, S>(a, t, lds);
}

// Groups of many rows: tiles of four heights, 16 WM to 64 WM.  A group's tiles being of one height keep step with each other,
// so that its weights come from memory once.  Measured with 32 groups of N = 2048, K = 7168, against tiles of 256 rows only:
// 384 rows each 198 instead of 243 us, 128 each 111 instead of 131, sizes about 512 (35% off) 328 instead of 337, 512
// each no change.  (Tiles of 256 with the idle waves of a group's last one skipped lose step: 384 each 247.)
template <int FN, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN, 2) void tile_kernel_heights(Args a, int tiles_m, int tiles_n) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[tile_lds(4, FN, WM, WN, 1, S)];
    constexpr int STEP = 16 * WM;
    const TileAt t = tile_of<4 * STEP, 16 * FN * WN, STEP>(a, blockIdx.x, tiles_m, tiles_n);
    if (!t.live) return;
    if (t.height == 4 * STEP) tile<4, FN, WM, WN, 1, S>(a, t, lds);
    else if (t.height == 3 * STEP) tile<3, FN, WM, WN, 1, S>(a, t, lds);
    else if (t.height == 2 * STEP) tile<2, FN, WM, WN, 1, S>(a, t, lds);
    else tile<1, FN, WM, WN, 1, S>(a, t, lds);
}

}  // namespace b128
}  // namespace mx
