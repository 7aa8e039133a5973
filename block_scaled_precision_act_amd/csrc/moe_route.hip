// moe_route.hip - what a router's choices become before the experts' grouped products, and the balance loss.
//
// Packing.  ids [T, top] names the expert of choice (t, j); an id outside 0 .. E - 1 is no choice.  The
// packed rows are the choices sorted by (expert, t, j), a stable counting sort: counts[e], offsets[e + 1] =
// offsets[e] + counts[e], rows[p] = t of packed row p (-1 behind the last), slots[t, j] = p (-1 for no choice).
// Every step is integer arithmetic whose result does not depend on the order of the atomic additions.
//   A workgroup places a chunk of the choices and needs every expert's count, in all and in the chunks before its own.
// Up to kAllMax choices each workgroup counts all ids itself, in LDS: one launch, no workspace.  Above, one kernel
// counts every chunk and a second one sums the counts of the chunks (chunks * E integers, read by every workgroup)
// before it places.  All of them together read those in quadratic time, so from kScanMin integers on a third kernel turns them
// into running sums in between (2^22 choices over 256 experts 55 us instead of 296, 2^24 190 us instead of 4.1 ms).
//   LDS atomics bound the first form (about 35 cycles for 64 random ids), a chain of memory and LDS latencies the second: 512
// choices over 32 experts 4.9 us, 8192 over 160 9.2 us, 24594 over 160 10.5 us (17 us in one launch), 131072 over 256 10.4 us.
//
// Balance loss.  p = softmax(logits[t]) over the experts, f_e = counts_e / sum(counts), n the tokens whose
// mask is not 0: loss = coef * E * sum_e f_e * mean_t p_te = sum_t sum_e w_e p_te with w_e = coef E f_e / n, so
// a row's share needs only its own logits, and the gradient is d loss / d logit_te = p_te (w_e - sum_j w_j p_tj).
// 64, 32, 16 or 8 lanes hold a row in registers: one read of the logits each way.  Few tokens are bound by launches and the
// chain of loads and reductions (T = 64, E = 32 in 3.7 us, gradient 2.3), many by memory: T = 16384, E = 256 FP32 masked, loss 10.5 us
// (its second launch, which joins the workgroups' sums, 2.9 of it), gradient 8.9 (3.8 TB/s).
#include "launch.hpp"
#include "mx_device.hpp"

namespace mx {
namespace {

constexpr int kMaxE = 1024;
constexpr int kThreads = 512, kChunk = 2048;  // choices per workgroup
constexpr int kAllMax = 8192;
constexpr int64_t kScanMin = 32768;

// Choices are numbered in 32 bits: T * top <= 2^24.
__device__ __forceinline__ int id_at(const void* ids, bool wide, int i, int E) {
    if (wide) {
        const int64_t v = reinterpret_cast<const int64_t*>(ids)[i];
        return v >= 0 && v < E ? (int)v : -1;
    }
    const int v = reinterpret_cast<const int32_t*>(ids)[i];
    return v >= 0 && v < E ? v : -1;
}

// lanes of the wave that hold the same id as this one (0 for id < 0)
__device__ __forceinline__ uint64_t same_id(int id, int bits) {
    uint64_t m = __ballot(id >= 0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t v = __ballot(id >> b & 1);
        m &= id >> b & 1 ? v : ~v;
    }
    return id >= 0 ? m : 0;
}

// exclusive prefix sum of v over the workgroup's threads; total is the sum
template <int THREADS>
__device__ __forceinline__ int block_scan(int v, int* tmp, int& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(s, d);
        if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 63) tmp[wave] = s;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        if (w < wave) before += tmp[w];
        total += tmp[w];
    }
    return before + s - v;
}

// hist[c, e]: the choices of expert e in chunk c
__global__ __launch_bounds__(kThreads) void moe_route_count(const void* ids, bool wide, int n, int E, int* __restrict__ hist) {
    __shared__ int h[kMaxE];
    for (int e = threadIdx.x; e < E; e += kThreads) h[e] = 0;
    __syncthreads();
    const int c0 = blockIdx.x * kChunk, c1 = min(c0 + kChunk, n);
    for (int i = c0 + threadIdx.x; i < c1; i += kThreads) {
        const int id = id_at(ids, wide, i, E);
        if (id >= 0) atomicAdd(h + id, 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) hist[(int64_t)blockIdx.x * E + e] = h[e];
}

// hist[c, e] becomes the choices of expert e in the chunks before c, totals[e] those of all.  16 experts per workgroup, 32
// threads for each, which take contiguous parts of the chunks.
constexpr int kScanExperts = 16;
__global__ __launch_bounds__(kThreads) void moe_route_scan(int* __restrict__ hist, int chunks, int E, int* __restrict__ totals) {
    constexpr int PARTS = kThreads / kScanExperts;
    __shared__ int sums[PARTS][kScanExperts];
    const int k = threadIdx.x % kScanExperts, part = threadIdx.x / kScanExperts, e = blockIdx.x * kScanExperts + k;
    const int per = (chunks + PARTS - 1) / PARTS, c0 = min(part * per, chunks), c1 = min(c0 + per, chunks);
    int sum = 0;
    if (e < E) {
#pragma unroll 8
        for (int c = c0; c < c1; ++c) sum += hist[(int64_t)c * E + e];
    }
    sums[part][k] = sum;
    __syncthreads();
    if (e >= E) return;
    int before = 0;
    for (int q = 0; q < part; ++q) before += sums[q][k];
    if (part == PARTS - 1) totals[e] = before + sum;
    constexpr int B = 8;  // reads ahead of the writes
    for (int c = c0; c < c1; c += B) {
        int v[B];
#pragma unroll
        for (int i = 0; i < B; ++i) v[i] = c + i < c1 ? hist[(int64_t)(c + i) * E + e] : 0;
#pragma unroll
        for (int i = 0; i < B; ++i) {
            if (c + i < c1) hist[(int64_t)(c + i) * E + e] = before;
            before += v[i];
        }
    }
}

// Places chunk blockIdx.x.  hist: the chunks' counts (running sums if there are totals), or null: this workgroup counts all ids.  Wave w takes the w-th
// part of the chunk in rounds of 64, its ids in registers from the start: what the kernel waits for is memory.
__global__ __launch_bounds__(kThreads) void moe_route_place(const void* ids, bool wide, int n, int top, int E,
                                                            const int* __restrict__ hist, const int* __restrict__ totals,
                                                            int32_t* counts, int32_t* offsets,
                                                            int32_t* rows, int32_t* slots) {
    constexpr int W = kThreads / 64, PER = kMaxE / kThreads, R = kChunk / kThreads;
    __shared__ int h[W * kMaxE], all[kMaxE], before[kMaxE];
    __shared__ int tmp[W];
    const int chunk = blockIdx.x, chunks = gridDim.x, lane = threadIdx.x & 63;
    const int bits = 32 - __builtin_clz(E > 1 ? E - 1 : 1);
    const int c0 = chunk * kChunk, c1 = min(c0 + kChunk, n), i0 = c0 + (threadIdx.x >> 6) * (R * 64) + lane;
    int id[R];
#pragma unroll
    for (int k = 0; k < R; ++k) id[k] = i0 + 64 * k < c1 ? id_at(ids, wide, i0 + 64 * k, E) : -1;
    int* mine = h + (threadIdx.x >> 6) * E;  // the wave's counts, later the running places
    for (int i = threadIdx.x; i < W * E; i += kThreads) h[i] = 0;
    for (int e = threadIdx.x; e < E; e += kThreads) all[e] = before[e] = 0;
    __syncthreads();
    if (totals) {
        for (int e = threadIdx.x; e < E; e += kThreads) {
            all[e] = totals[e];
            before[e] = hist[(int64_t)chunk * E + e];
        }
    } else if (hist) {
        // thread t takes expert t % span of chunks t / span, t / span + parts, ...
        const int sbits = bits < 9 ? bits : 9, span = 1 << sbits, parts = kThreads >> sbits;
        static_assert(kThreads == 512, "span");
        for (int e = threadIdx.x & (span - 1); e < E; e += span) {
            int sum = 0, low = 0;
#pragma unroll 16
            for (int b = threadIdx.x >> sbits; b < chunks; b += parts) {
                const int v = hist[(int64_t)b * E + e];
                sum += v;
                low += b < chunk ? v : 0;
            }
            atomicAdd(all + e, sum);
            atomicAdd(before + e, low);
        }
    } else if (chunks > 1) {
        constexpr int B = kAllMax / kThreads;
        int other[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int i = threadIdx.x + k * kThreads;
            other[k] = i < n ? id_at(ids, wide, i, E) : -1;
        }
#pragma unroll
        for (int k = 0; k < B; ++k)
            if (other[k] >= 0) {
                atomicAdd(all + other[k], 1);
                if ((int)threadIdx.x + k * kThreads < c0) atomicAdd(before + other[k], 1);
            }
    }
#pragma unroll
    for (int k = 0; k < R; ++k)
        if (id[k] >= 0) atomicAdd(mine + id[k], 1);
    __syncthreads();
    // thread t: expert t, or experts 2 t and 2 t + 1
    const int per = E > kThreads ? PER : 1;
    static_assert(PER <= 2, "experts per thread");
    int mine_all[PER] = {}, waves[PER][W] = {}, sum = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int e = per * threadIdx.x + k;
        if (k >= per || e >= E) continue;
#pragma unroll
        for (int w = 0; w < W; ++w) waves[k][w] = h[w * E + e];
        mine_all[k] = all[e];
        if (chunks == 1) {
#pragma unroll
            for (int w = 0; w < W; ++w) mine_all[k] += waves[k][w];
        }
        sum += mine_all[k];
    }
    int total;
    int start = block_scan<kThreads>(sum, tmp, total);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int e = per * threadIdx.x + k;
        if (k >= per || e >= E) continue;
        if (chunk == 0) {
            counts[e] = mine_all[k];
            offsets[e] = start;
        }
        int p = start + before[e];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            h[w * E + e] = p;
            p += waves[k][w];
        }
        start += mine_all[k];
    }
    if (chunk == 0 && threadIdx.x == 0) offsets[E] = total;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int i = i0 + 64 * k;
        if (i - lane >= c1) break;  // the wave's
        const uint64_t m = same_id(id[k], bits);
        const int ahead = __popcll(m & ((1ull << lane) - 1));
        int base = 0;
        if (id[k] >= 0 && ahead == 0) base = atomicAdd(mine + id[k], __popcll(m));  // one lane per id; its wave's own counter
        base = __shfl(base, m ? __ffsll((unsigned long long)m) - 1 : lane);
        if (i < c1) {
            const int p = id[k] >= 0 ? base + ahead : -1;
            slots[i] = p;
            if (p >= 0) rows[p] = (uint32_t)i / (uint32_t)top;
        }
    }
    for (int p = max(total, c0) + threadIdx.x; p < c1; p += kThreads) rows[p] = -1;
}

// ---------------------------------------------------------------- balance loss
constexpr int kLossThreads = 512, kLossBlocks = 1024;  // as many as fit at once
constexpr int kRows = 2;                                // of a group of lanes at a time

// Sums and maxima over the L lanes that hold a row (L = 8, 16, 32 or 64; every lane of them active), without LDS: lane
// swaps within 16 lanes by DPP, then rows of 16 and halves of the wave exchanged.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int L, typename F>
__device__ __forceinline__ float row_reduce(float v, F&& f) {
    v = f(v, dpp<0xB1>(v));   // quad_perm [1,0,3,2]
    v = f(v, dpp<0x4E>(v));   // quad_perm [2,3,0,1]
    v = f(v, dpp<0x141>(v));  // row_half_mirror
    if constexpr (L >= 16) v = f(v, dpp<0x140>(v));  // row_mirror
    if constexpr (L >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    if constexpr (L >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}
template <int L>
__device__ __forceinline__ float row_sum(float v) {
    return row_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float row_max(float v) {
    return row_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}

// A row as loaded: lane j of L holds experts j V .. j V + V - 1.  VEC: E is a multiple of V and rows start at multiples of their
// loads (row_vec).  Every lane loads, those past E from a place inside the row, so that nothing branches between the loads of
// two rows; values are taken out when they are needed.
template <int L, int V, bool HALF, bool VEC>
struct Row {
    static constexpr int kBytes = V * (HALF ? 2 : 4), kLoad = kBytes < 16 ? kBytes : 16;  // of the lane; of a load
    uint32_t w[VEC ? (kBytes + 3) / 4 : V];
    __device__ __forceinline__ void load(const void* logits, int64_t t, int E) {
        const int e0 = (threadIdx.x & (L - 1)) * V;
        const uint16_t* h = reinterpret_cast<const uint16_t*>(logits) + t * E;
        const uint32_t* f = reinterpret_cast<const uint32_t*>(logits) + t * E;
        if constexpr (VEC && kLoad > 2) {
            const int at = min(e0, E - V);
            const uint8_t* src = HALF ? reinterpret_cast<const uint8_t*>(h + at) : reinterpret_cast<const uint8_t*>(f + at);
#pragma unroll
            for (int c = 0; c < kBytes / kLoad; ++c)
                __builtin_memcpy(w + c * kLoad / 4, __builtin_assume_aligned(src + c * kLoad, kLoad), kLoad);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = HALF ? h[min(e0 + i, E - 1)] : f[min(e0 + i, E - 1)];
        }
    }
    // -infinity past E, and everywhere in a row that is not live
    __device__ __forceinline__ void take(bool live, int E, float (&p)[V]) const {
        const int e0 = (threadIdx.x & (L - 1)) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            uint32_t v;
            if constexpr (!HALF) v = w[i];
            else if constexpr (VEC && V > 1) v = i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16;
            else v = w[i] << 16;
            p[i] = live && (VEC ? e0 : e0 + i) < E ? __uint_as_float(v) : -__builtin_inff();
        }
    }
};
template <int V, bool HALF>
bool row_vec(const void* p, int64_t E) {
    constexpr int B = V * (HALF ? 2 : 4);
    return E % V == 0 && (uintptr_t)p % (B < 16 ? B : 16) == 0;
}

// e^d for d <= 0: the product with log2(e) in two parts, so off by little more than v_exp's last place; 0 below e^-87, where
// a probability is far below the last place of any sum that it enters
__device__ __forceinline__ float exp_neg(float d) {
    constexpr float kLog2e = 1.44269504f, kLow = 1.92596299e-8f, kLn2 = 0.693147181f;
    const float t = d * kLog2e, low = __builtin_fmaf(d, kLow, __builtin_fmaf(d, kLog2e, -t));
    const float v = __builtin_amdgcn_exp2f(t);
    return d < -87.f ? 0.f : __builtin_fmaf(v, low * kLn2, v);  // NaN stays NaN
}
// Logits to probabilities.  A row with no logit above -infinity has none (all 0); a NaN or +infinity makes the row NaN.
template <int L, int V>
__device__ __forceinline__ void row_softmax(float (&p)[V]) {
    float top = p[0], sum = 0.f;
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, p[i]);
    top = row_max<L>(top);
    const float base = top == -__builtin_inff() ? 0.f : top;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        p[i] = exp_neg(p[i] - base);
        sum += p[i];
    }
    sum = row_sum<L>(sum);
    const float r = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] *= r;
}

__device__ __forceinline__ uint32_t wave_sum(uint32_t v) {
    return __float_as_uint(row_reduce<64>(__uint_as_float(v), [](float a, float b) {
        return __uint_as_float(__float_as_uint(a) + __float_as_uint(b));  // lane swaps move bits, whatever they are
    }));
}

// The loss and the experts' weights from the threads' shares of sum_t sum_e counts_e p_te and of the unmasked tokens.  All
// sums in FP64 and in a fixed order: lanes, then waves.
__device__ __forceinline__ void balance_finish(double sum, double live, const int32_t* __restrict__ counts, int E, float coef,
                                               float* loss, float* __restrict__ w) {
    __shared__ double tmp[3][kLossThreads / 64];
    double v[3] = {sum, live, 0.0};
    for (int e = threadIdx.x; e < E; e += kLossThreads) v[2] += counts[e];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) v[i] += __shfl_xor(v[i], d);
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i) tmp[i][threadIdx.x >> 6] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        v[i] = tmp[i][0];
#pragma unroll
        for (int k = 1; k < kLossThreads / 64; ++k) v[i] += tmp[i][k];
    }
    const double unit = v[2] > 0 && v[1] > 0 ? (double)coef * E / (v[2] * v[1]) : 0.0;
    for (int e = threadIdx.x; e < E; e += kLossThreads) w[e] = (float)(unit * counts[e]);
    if (threadIdx.x == 0) *loss = (float)(unit * v[0]);
}

// Calls f(t, live, p) for the rows t of this lane's group of L, two at a time (their loads and reductions run beside each other);
// p are the lane's probabilities.  A row that is not live, masked or past T - 1, has none.  T > 0.
template <int L, int V, bool HALF, bool VEC, typename F>
__device__ __forceinline__ void for_rows(const void* __restrict__ logits, int64_t T, int E, const uint8_t* __restrict__ mask, F&& f) {
    const int64_t step = gridDim.x * (int64_t)(kLossThreads / L);  // rows per round
    const uint8_t* bytes = mask ? mask : reinterpret_cast<const uint8_t*>(logits);  // without a mask, any bytes do
    for (int64_t t = blockIdx.x * (int64_t)(kLossThreads / L) + threadIdx.x / L; t < T; t += kRows * step) {
        Row<L, V, HALF, VEC> row[kRows];
        uint8_t m[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t u = min(t + k * step, T - 1);
            row[k].load(logits, u, E);
            m[k] = bytes[u];
        }
        float p[kRows][V];
        bool live[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            live[k] = t + k * step < T && (!mask || m[k] != 0);
            row[k].take(live[k], E, p[k]);
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) row_softmax<L, V>(p[k]);
#pragma unroll
        for (int k = 0; k < kRows; ++k) f(t + k * step, live[k], p[k]);
    }
}

// Every workgroup sums its rows' shares and counts its unmasked rows, into part[2 b] and part[2 b + 1] for
// moe_balance_finish; one workgroup alone finishes by itself.
template <int L, int V, bool HALF>
__global__ __launch_bounds__(kLossThreads) void moe_balance_kernel(const void* __restrict__ logits, int64_t T, int E, bool vec,
                                                                   const int32_t* __restrict__ counts,
                                                                   const uint8_t* __restrict__ mask, float coef, float* loss,
                                                                   float* __restrict__ w, double* __restrict__ part) {
    __shared__ double tmp[2][kLossThreads / 64];
    const int e0 = (threadIdx.x & (L - 1)) * V;
    int held[V];
    float count[V];
#pragma unroll
    for (int i = 0; i < V; ++i) held[i] = counts[min(e0 + i, E - 1)];
#pragma unroll
    for (int i = 0; i < V; ++i) count[i] = e0 + i < E ? (float)held[i] : 0.f;
    double sum = 0;
    uint32_t live = 0;  // rows; the row's first lane counts
    auto row = [&](int64_t, bool counted, const float (&p)[V]) __attribute__((always_inline)) {
        float s = 0.f;
        live += counted && e0 == 0;
#pragma unroll
        for (int i = 0; i < V; ++i) s = __builtin_fmaf(p[i], count[i], s);
        sum += s;
    };
    if (T > 0) {
        if (V == 1 || !vec) for_rows<L, V, HALF, false>(logits, T, E, mask, row);
        else for_rows<L, V, HALF, true>(logits, T, E, mask, row);
    }
    if (gridDim.x == 1) {
        balance_finish(sum, live, counts, E, coef, loss, w);
        return;
    }
    live = wave_sum(live);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    if ((threadIdx.x & 63) == 0) {
        tmp[0][threadIdx.x >> 6] = sum;
        tmp[1][threadIdx.x >> 6] = live;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double s = 0;
#pragma unroll
        for (int k = 0; k < kLossThreads / 64; ++k) s += tmp[threadIdx.x][k];
        part[2 * blockIdx.x + threadIdx.x] = s;
    }
}

__global__ __launch_bounds__(kLossThreads) void moe_balance_finish(const double* __restrict__ part, int n, int E,
                                                                   const int32_t* __restrict__ counts, float coef, float* loss,
                                                                   float* __restrict__ w) {
    double sum = 0, live = 0;
    for (int b = threadIdx.x; b < n; b += kLossThreads) {
        sum += part[2 * b];
        live += part[2 * b + 1];
    }
    balance_finish(sum, live, counts, E, coef, loss, w);
}

template <int L, int V, bool HALF>
__global__ __launch_bounds__(kLossThreads) void moe_balance_grad_kernel(const void* __restrict__ logits, int64_t T, int E, bool vec,
                                                                        const float* __restrict__ w,
                                                                        const uint8_t* __restrict__ mask,
                                                                        const float* __restrict__ grad, void* __restrict__ d) {
    const int e0 = (threadIdx.x & (L - 1)) * V;
    const float g = *grad;
    float we[V];
#pragma unroll
    for (int i = 0; i < V; ++i) we[i] = w[min(e0 + i, E - 1)];
#pragma unroll
    for (int i = 0; i < V; ++i) we[i] = e0 + i < E ? we[i] : 0.f;
    auto row = [&](int64_t t, bool live, float (&p)[V], auto wide) __attribute__((always_inline)) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s = __builtin_fmaf(p[i], we[i], s);
        s = row_sum<L>(s);
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = live ? g * p[i] * (we[i] - s) : 0.f;
        uint16_t* h = reinterpret_cast<uint16_t*>(d) + t * E + e0;
        float* f = reinterpret_cast<float*>(d) + t * E + e0;
        if constexpr (decltype(wide)::value) {
            constexpr int B = V * (HALF ? 2 : 4), C = B < 16 ? B : 16;
            uint32_t o[(B + 3) / 4];
#pragma unroll
            for (int i = 0; i < B / 4; ++i) {
                if constexpr (HALF) o[i] = bf16x2_rne(p[2 * i], p[2 * i + 1]);
                else o[i] = __float_as_uint(p[i]);
            }
            if (t < T && e0 < E) {
                uint8_t* dst = HALF ? reinterpret_cast<uint8_t*>(h) : reinterpret_cast<uint8_t*>(f);
#pragma unroll
                for (int c = 0; c < B / C; ++c) __builtin_memcpy(__builtin_assume_aligned(dst + c * C, C), o + c * C / 4, C);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (t >= T || e0 + i >= E) continue;
                if constexpr (HALF) h[i] = (uint16_t)bf16_rne(p[i]);
                else f[i] = p[i];
            }
        }
    };
    if constexpr (V > 1) {
        if (vec) {
            for_rows<L, V, HALF, true>(logits, T, E, mask, [&](int64_t t, bool live, float (&p)[V]) __attribute__((always_inline)) {
                row(t, live, p, std::true_type{});
            });
            return;
        }
    }
    for_rows<L, V, HALF, false>(logits, T, E, mask, [&](int64_t t, bool live, float (&p)[V]) __attribute__((always_inline)) {
        row(t, live, p, std::false_type{});
    });
}

// calls f(L, V) for the lanes and values per lane of a row of E logits
template <typename F>
hipError_t by_width(int64_t E, F&& f) {
    using std::integral_constant;
    if (E <= 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    if (E <= 16) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    if (E <= 32) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
    if (E <= 64) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (E <= 128) return f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (E <= 256) return f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    if (E <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
    return f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}
int64_t lanes_of(int64_t E) { return E <= 8 ? 8 : E <= 16 ? 16 : E <= 32 ? 32 : 64; }
// One workgroup, and so one launch, for as many rounds as cost less than a second launch (2 us; a round after the first 0.6 us
// for one value per lane, 0.9 for four, 2.5 for sixteen: E = 256, T = 32 4.6 us; T = 64 5.8 with a second launch, 6.4 without).
int64_t loss_blocks(int64_t T, int64_t E) {
    const int64_t b = (T * lanes_of(E) + kRows * kLossThreads - 1) / (kRows * kLossThreads);
    const int64_t values = (E + 63) / 64;
    return b <= 1 + 24 / (6 + values) ? 1 : b < kLossBlocks ? b : kLossBlocks;
}

}  // namespace

// the chunks' counts, then the totals
size_t moe_route_workspace_bytes(int64_t n, int64_t E) {
    return n <= kAllMax ? 0 : (size_t)((n + kChunk - 1) / kChunk + 1) * E * sizeof(int);
}

hipError_t launch_moe_route(const void* ids, bool wide, int64_t T, int64_t top, int64_t E, int32_t* counts, int32_t* offsets,
                            int32_t* rows, int32_t* slots, void* workspace, hipStream_t st) {
    const int64_t n = T * top, chunks = n > 0 ? (n + kChunk - 1) / kChunk : 1;
    const dim3 grid((unsigned)chunks);
    int* hist = n <= kAllMax ? nullptr : reinterpret_cast<int*>(workspace);
    int* totals = hist && chunks * E >= kScanMin ? hist + chunks * E : nullptr;
    if (hist) {
        hipLaunchKernelGGL(moe_route_count, grid, dim3(kThreads), 0, st, ids, wide, (int)n, (int)E, hist);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    if (totals) {
        hipLaunchKernelGGL(moe_route_scan, dim3((unsigned)((E + kScanExperts - 1) / kScanExperts)), dim3(kThreads), 0, st, hist,
                           (int)chunks, (int)E, totals);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(moe_route_place, grid, dim3(kThreads), 0, st, ids, wide, (int)n, (int)top, (int)E, hist, totals, counts,
                       offsets, rows, slots);
    return hipGetLastError();
}

size_t moe_balance_workspace_bytes(int64_t T, int64_t E) {
    const int64_t b = loss_blocks(T, E);
    return b > 1 ? (size_t)b * 2 * sizeof(double) : 0;
}

hipError_t launch_moe_balance(const void* logits, bool half, int64_t T, int64_t E, const int32_t* counts, const uint8_t* mask,
                              float coef, float* loss, float* w, void* workspace, hipStream_t st) {
    const int64_t blocks = T > 0 ? loss_blocks(T, E) : 1;
    double* part = reinterpret_cast<double*>(workspace);
    hipError_t err = by_width(E, [&](auto l, auto v) {
        constexpr int L = decltype(l)::value, V = decltype(v)::value;
        const dim3 grid((unsigned)blocks), block(kLossThreads);
        if (half)
            hipLaunchKernelGGL((moe_balance_kernel<L, V, true>), grid, block, 0, st, logits, T, (int)E,
                               row_vec<V, true>(logits, E), counts, mask, coef, loss, w, part);
        else
            hipLaunchKernelGGL((moe_balance_kernel<L, V, false>), grid, block, 0, st, logits, T, (int)E,
                               row_vec<V, false>(logits, E), counts, mask, coef, loss, w, part);
        return hipGetLastError();
    });
    if (err != hipSuccess || blocks == 1) return err;
    hipLaunchKernelGGL(moe_balance_finish, dim3(1), dim3(kLossThreads), 0, st, part, (int)blocks, (int)E, counts, coef, loss, w);
    return hipGetLastError();
}

hipError_t launch_moe_balance_grad(const void* logits, bool half, int64_t T, int64_t E, const float* w, const uint8_t* mask,
                                   const float* grad_loss, void* dlogits, hipStream_t st) {
    const int64_t blocks = (T * lanes_of(E) + kRows * kLossThreads - 1) / (kRows * kLossThreads);
    return by_width(E, [&](auto l, auto v) {
        constexpr int L = decltype(l)::value, V = decltype(v)::value;
        const dim3 grid((unsigned)(blocks < kLossBlocks ? blocks : kLossBlocks)), block(kLossThreads);
        if (half)
            hipLaunchKernelGGL((moe_balance_grad_kernel<L, V, true>), grid, block, 0, st, logits, T, (int)E,
                               row_vec<V, true>(logits, E) && row_vec<V, true>(dlogits, E), w, mask, grad_loss, dlogits);
        else
            hipLaunchKernelGGL((moe_balance_grad_kernel<L, V, false>), grid, block, 0, st, logits, T, (int)E,
                               row_vec<V, false>(logits, E) && row_vec<V, false>(dlogits, E), w, mask, grad_loss, dlogits);
        return hipGetLastError();
    });
}

}  // namespace mx
