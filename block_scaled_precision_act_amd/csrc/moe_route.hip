// moe_route.hip - what a router's choices become before the experts' grouped products, and the balance loss.
//
// Packing.  ids [T, top] names the expert of choice (t, j); an id outside 0 .. E - 1 is no choice.  The
// packed rows are the choices sorted by (expert, t, j), a stable counting sort: counts[e], offsets[e + 1] =
// offsets[e] + counts[e], rows[p] = t of packed row p (-1 behind the last), slots[t, j] = p (-1 for no choice).
// Every step is integer arithmetic whose result does not depend on the order of the atomic additions.
//   A workgroup places a chunk of the choices and needs every expert's count, in all and in the chunks before its own.
// Up to kAllMax choices each workgroup counts all ids itself, in LDS: one launch, no workspace.  Above, one kernel
// counts every chunk and a second one sums the counts of the chunks (chunks * E integers, read by every workgroup)
// before it places.  LDS atomics bound the first form (about 35 cycles for 64 random ids), a chain of memory and LDS
// latencies the second: 512 choices over 32 experts 4.9 us, 8192 over 160 9.2 us, 24594 over 160 10.5 us (17 us in one
// launch), 131072 over 256 10.4 us.
//
// Balance loss.  p = softmax(logits[t]) over the experts, f_e = counts_e / sum(counts), n the tokens whose
// mask is not 0: loss = coef * E * sum_e f_e * mean_t p_te = sum_t sum_e w_e p_te with w_e = coef E f_e / n, so
// a row's share needs only its own logits, and the gradient is d loss / d logit_te = p_te (w_e - sum_j w_j p_tj).
// 64, 32, 16 or 8 lanes hold a row in registers (one read of the logits each way; the kernels are bound by
// that read, and by launches for few tokens).
#include "launch.hpp"
#include "mx_device.hpp"

namespace mx {
namespace {

constexpr int kMaxE = 1024;
constexpr int kThreads = 512, kChunk = 2048;  // choices per workgroup
constexpr int kAllMax = 8192;

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

// Places chunk blockIdx.x.  hist: the chunks' counts, or null: this workgroup counts all ids.  Wave w takes the w-th
// part of the chunk in rounds of 64, its ids in registers from the start: what the kernel waits for is memory.
__global__ __launch_bounds__(kThreads) void moe_route_place(const void* ids, bool wide, int n, int top, int E,
                                                            const int* __restrict__ hist, int32_t* counts, int32_t* offsets,
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
    if (hist) {
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
constexpr int kLossThreads = 512, kLossBlocks = 512;

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

// Row t's logits: lane j of L holds experts j, j + L, ...; -infinity past E, and everywhere if there is no such row.
template <int L, int V, bool HALF>
__device__ __forceinline__ void row_load(const void* logits, bool live, int64_t t, int E, float (&p)[V]) {
    const int j = threadIdx.x & (L - 1);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = j + i * L;
        p[i] = -__builtin_inff();
        if (live && e < E) {
            if constexpr (HALF) p[i] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(logits)[t * E + e] << 16);
            else p[i] = reinterpret_cast<const float*>(logits)[t * E + e];
        }
    }
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
        p[i] = expf(p[i] - base);
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
// Sums over the workgroup, in a fixed order: of each wave by shuffles or lane swaps, then of the waves.
__device__ __forceinline__ double block_sum(double v, double* tmp) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = tmp[0];
#pragma unroll
    for (int w = 1; w < kLossThreads / 64; ++w) s += tmp[w];
    return s;
}

// Every workgroup sums its rows' shares of the loss; part[b] (or the loss itself, when there is one workgroup).
template <int L, int V, bool HALF>
__global__ __launch_bounds__(kLossThreads) void moe_balance_kernel(const void* __restrict__ logits, int64_t T, int E,
                                                                   const int32_t* __restrict__ counts,
                                                                   const uint8_t* __restrict__ mask, float coef, float* loss,
                                                                   float* __restrict__ w, double* __restrict__ part) {
    __shared__ uint32_t tmp[kLossThreads / 64][3];
    __shared__ double dtmp[kLossThreads / 64];
    const int j = threadIdx.x & (L - 1);
    const int64_t per = kLossThreads / L, step = gridDim.x * per;  // rows per round of a workgroup, and of all
    int64_t t = blockIdx.x * per + threadIdx.x / L;
    auto is_live = [&](int64_t r) { return r < T && (!mask || mask[r] != 0); };
    float next[V];
    row_load<L, V, HALF>(logits, is_live(t), t, E, next);  // on its way while the counts are summed
    // choices in all (their halves of 16 bits apart: 1024 counts of 31 bits need 41) and unmasked tokens
    uint32_t low = 0, high = 0, unmasked = 0;
    for (int e = threadIdx.x; e < E; e += kLossThreads) {
        low += (uint32_t)counts[e] & 0xffffu;
        high += (uint32_t)counts[e] >> 16;
    }
    if (mask) {
        // 16 bytes at a time from the first aligned one; every workgroup counts them all
        const int64_t head = min((int64_t)(-(uintptr_t)mask & 15), T), vecs = (T - head) / 16;
        const uint4* v = reinterpret_cast<const uint4*>(mask + head);
        auto bytes = [](uint32_t w) { return __popc((((w & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w) & 0x80808080u); };  // not 0
        for (int64_t i = threadIdx.x; i < vecs; i += kLossThreads) {
            const uint4 m = v[i];
            unmasked += bytes(m.x) + bytes(m.y) + bytes(m.z) + bytes(m.w);
        }
        for (int64_t r = threadIdx.x; r < head; r += kLossThreads) unmasked += mask[r] != 0;
        for (int64_t r = head + 16 * vecs + threadIdx.x; r < T; r += kLossThreads) unmasked += mask[r] != 0;
    }
    low = wave_sum(low), high = wave_sum(high), unmasked = wave_sum(unmasked);
    if ((threadIdx.x & 63) == 0) {
        uint32_t* w = tmp[threadIdx.x >> 6];
        w[0] = low, w[1] = high, w[2] = unmasked;
    }
    __syncthreads();
    int64_t chosen = 0, live = 0;
#pragma unroll
    for (int w = 0; w < kLossThreads / 64; ++w) {
        chosen += tmp[w][0] + ((int64_t)tmp[w][1] << 16);
        live += tmp[w][2];
    }
    if (!mask) live = T;
    const double unit = chosen > 0 && live > 0 ? (double)coef * E / ((double)chosen * (double)live) : 0.0;
    float we[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = j + i * L;
        we[i] = e < E ? (float)(unit * counts[e]) : 0.f;
        if (blockIdx.x == 0 && (int)threadIdx.x < L && e < E) w[e] = we[i];
    }
    double sum = 0;
    for (; t < T; t += step) {
        float p[V], s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = next[i];
        row_load<L, V, HALF>(logits, is_live(t + step), t + step, E, next);  // while this row is reduced
        row_softmax<L, V>(p);  // a masked row has no logits: no probabilities
#pragma unroll
        for (int i = 0; i < V; ++i) s = __builtin_fmaf(p[i], we[i], s);
        sum += s;
    }
    sum = block_sum(sum, dtmp);
    if (threadIdx.x == 0) {
        if (gridDim.x == 1) *loss = (float)sum;
        else part[blockIdx.x] = sum;
    }
}

__global__ __launch_bounds__(kLossThreads) void moe_balance_finish(const double* __restrict__ part, int n, float* loss) {
    __shared__ double tmp[kLossThreads / 64];
    double s = (int)threadIdx.x < n ? part[threadIdx.x] : 0.0;
    s = block_sum(s, tmp);
    if (threadIdx.x == 0) *loss = (float)s;
}

template <int L, int V, bool HALF>
__global__ __launch_bounds__(kLossThreads) void moe_balance_grad_kernel(const void* __restrict__ logits, int64_t T, int E,
                                                                        const float* __restrict__ w,
                                                                        const uint8_t* __restrict__ mask,
                                                                        const float* __restrict__ grad, void* __restrict__ d) {
    const int j = threadIdx.x & (L - 1);
    const float g = *grad;
    float we[V];
#pragma unroll
    for (int i = 0; i < V; ++i) we[i] = j + i * L < E ? w[j + i * L] : 0.f;
    const int64_t per = kLossThreads / L, step = gridDim.x * per;
    int64_t t = blockIdx.x * per + threadIdx.x / L;
    auto is_live = [&](int64_t r) { return r < T && (!mask || mask[r] != 0); };
    float next[V];
    bool next_live = is_live(t);
    row_load<L, V, HALF>(logits, next_live, t, E, next);
    for (; t < T; t += step) {
        float p[V], s = 0.f;
        const bool live = next_live;
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = next[i];
        next_live = is_live(t + step);
        row_load<L, V, HALF>(logits, next_live, t + step, E, next);  // while this row is reduced
        row_softmax<L, V>(p);
#pragma unroll
        for (int i = 0; i < V; ++i) s = __builtin_fmaf(p[i], we[i], s);
        s = row_sum<L>(s);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = j + i * L;
            if (e >= E) continue;
            const float v = live ? g * p[i] * (we[i] - s) : 0.f;
            if constexpr (HALF) reinterpret_cast<uint16_t*>(d)[t * E + e] = (uint16_t)bf16_rne(v);
            else reinterpret_cast<float*>(d)[t * E + e] = v;
        }
    }
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
// One workgroup, and so one launch, up to eight rounds of it; a second launch costs about as much.
int64_t loss_blocks(int64_t T, int64_t E) {
    const int64_t b = (T * lanes_of(E) + kLossThreads - 1) / kLossThreads;
    return b <= 8 ? 1 : b < kLossBlocks ? b : kLossBlocks;
}

}  // namespace

size_t moe_route_workspace_bytes(int64_t n, int64_t E) {
    return n <= kAllMax ? 0 : (size_t)((n + kChunk - 1) / kChunk) * E * sizeof(int);
}

hipError_t launch_moe_route(const void* ids, bool wide, int64_t T, int64_t top, int64_t E, int32_t* counts, int32_t* offsets,
                            int32_t* rows, int32_t* slots, void* workspace, hipStream_t st) {
    const int64_t n = T * top;
    const dim3 grid((unsigned)(n > 0 ? (n + kChunk - 1) / kChunk : 1));
    int* hist = n <= kAllMax ? nullptr : reinterpret_cast<int*>(workspace);
    if (hist) {
        hipLaunchKernelGGL(moe_route_count, grid, dim3(kThreads), 0, st, ids, wide, (int)n, (int)E, hist);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(moe_route_place, grid, dim3(kThreads), 0, st, ids, wide, (int)n, (int)top, (int)E, hist, counts, offsets, rows,
                       slots);
    return hipGetLastError();
}

size_t moe_balance_workspace_bytes(int64_t T, int64_t E) {
    const int64_t b = loss_blocks(T, E);
    return b > 1 ? (size_t)b * sizeof(double) : 0;
}

hipError_t launch_moe_balance(const void* logits, bool half, int64_t T, int64_t E, const int32_t* counts, const uint8_t* mask,
                              float coef, float* loss, float* w, void* workspace, hipStream_t st) {
    const int64_t blocks = T > 0 ? loss_blocks(T, E) : 1;
    double* part = reinterpret_cast<double*>(workspace);
    hipError_t err = by_width(E, [&](auto l, auto v) {
        constexpr int L = decltype(l)::value, V = decltype(v)::value;
        const dim3 grid((unsigned)blocks), block(kLossThreads);
        if (half)
            hipLaunchKernelGGL((moe_balance_kernel<L, V, true>), grid, block, 0, st, logits, T, (int)E, counts, mask, coef, loss, w, part);
        else
            hipLaunchKernelGGL((moe_balance_kernel<L, V, false>), grid, block, 0, st, logits, T, (int)E, counts, mask, coef, loss, w, part);
        return hipGetLastError();
    });
    if (err != hipSuccess || blocks == 1) return err;
    hipLaunchKernelGGL(moe_balance_finish, dim3(1), dim3(kLossThreads), 0, st, part, (int)blocks, loss);
    return hipGetLastError();
}

hipError_t launch_moe_balance_grad(const void* logits, bool half, int64_t T, int64_t E, const float* w, const uint8_t* mask,
                                   const float* grad_loss, void* dlogits, hipStream_t st) {
    const int64_t blocks = (T * lanes_of(E) + kLossThreads - 1) / kLossThreads;
    return by_width(E, [&](auto l, auto v) {
        constexpr int L = decltype(l)::value, V = decltype(v)::value;
        const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096)), block(kLossThreads);
        if (half)
            hipLaunchKernelGGL((moe_balance_grad_kernel<L, V, true>), grid, block, 0, st, logits, T, (int)E, w, mask, grad_loss, dlogits);
        else
            hipLaunchKernelGGL((moe_balance_grad_kernel<L, V, false>), grid, block, 0, st, logits, T, (int)E, w, mask, grad_loss, dlogits);
        return hipGetLastError();
    });
}

}  // namespace mx
