// moe_route.hip - what a router's choices become before the experts' grouped products, and the balance loss.
//
// Packing.  ids [T, top] names the expert of choice (t, j); an id outside 0 .. E - 1 is no choice.  The
// packed rows are the choices sorted by (expert, t, j), a stable counting sort: counts[e], offsets[e + 1] =
// offsets[e] + counts[e], rows[p] = t of packed row p (-1 behind the last), slots[t, j] = p (-1 for no choice).
// Every step is integer arithmetic whose result does not depend on the order of the atomic additions.
//   Up to kOneMax choices one workgroup does it all in LDS, in one launch.  Above, one kernel counts the
// experts of every chunk of choices and a second one, a workgroup per chunk, sums the counts of the chunks
// before its own and places its chunk.  Every workgroup reads all counts (chunks * E integers, from L2), all its
// threads sharing them out by expert and chunk: with a few threads walking the chunks one after another, 131072
// choices over 256 experts took 51 us.
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
constexpr int kOneThreads = 1024, kOneMax = 8192;
constexpr int kThreads = 512, kChunk = 2048;  // choices per workgroup of the two-kernel form

__device__ __forceinline__ int id_at(const void* ids, bool wide, int64_t i, int E) {
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

// Counts the ids of choices c0 .. c1 - 1 into hist[W][E] (LDS, per wave: wave w takes the w-th part of
// whole rounds of 64), and afterwards places them: place(i, p) with p the running position of i's
// expert and wave, starting from what hist holds then.
template <int W>
struct Chunk {
    const void* ids;
    bool wide;
    int E, bits;
    int64_t a, b;  // this wave's choices
    __device__ __forceinline__ Chunk(const void* ids_, bool wide_, int E_, int64_t c0, int64_t c1) : ids(ids_), wide(wide_), E(E_) {
        bits = 32 - __builtin_clz(E > 1 ? E - 1 : 1);
        const int wave = threadIdx.x >> 6;
        const int64_t per = ((c1 - c0 + W - 1) / W + 63) / 64 * 64;
        a = min(c0 + wave * per, c1);
        b = min(a + per, c1);
    }
    __device__ __forceinline__ void count(int* hist) const {
        int* h = hist + (threadIdx.x >> 6) * E;
        for (int64_t i = a + (threadIdx.x & 63); i < b; i += 64) {
            const int id = id_at(ids, wide, i, E);
            if (id >= 0) atomicAdd(h + id, 1);
        }
    }
    template <typename F>
    __device__ __forceinline__ void place(int* hist, F&& put) const {
        int* h = hist + (threadIdx.x >> 6) * E;
        const int lane = threadIdx.x & 63;
        for (int64_t i0 = a; i0 < b; i0 += 64) {
            const int64_t i = i0 + lane;
            const int id = i < b ? id_at(ids, wide, i, E) : -1;
            const uint64_t m = same_id(id, bits);
            const int before = __popcll(m & ((1ull << lane) - 1));
            int base = 0;
            if (id >= 0 && before == 0) base = atomicAdd(h + id, __popcll(m));  // one lane per id; its wave's own counter
            base = __shfl(base, m ? __ffsll((unsigned long long)m) - 1 : lane);
            if (i < b) put(i, id >= 0 ? base + before : -1);
        }
    }
};

__global__ __launch_bounds__(kOneThreads) void moe_route_one(const void* ids, bool wide, int64_t n, int top, int E,
                                                             int32_t* counts, int32_t* offsets, int32_t* rows, int32_t* slots) {
    constexpr int W = kOneThreads / 64;
    __shared__ int hist[W * kMaxE];
    __shared__ int tmp[W];
    for (int i = threadIdx.x; i < W * E; i += kOneThreads) hist[i] = 0;
    __syncthreads();
    const Chunk<W> c(ids, wide, E, 0, n);
    c.count(hist);
    __syncthreads();
    int mine = 0;  // thread e: expert e
    if ((int)threadIdx.x < E)
        for (int w = 0; w < W; ++w) mine += hist[w * E + threadIdx.x];
    int total;
    const int start = block_scan<kOneThreads>(mine, tmp, total);
    if ((int)threadIdx.x < E) {
        counts[threadIdx.x] = mine;
        offsets[threadIdx.x] = start;
        int p = start;
        for (int w = 0; w < W; ++w) {
            const int h = hist[w * E + threadIdx.x];
            hist[w * E + threadIdx.x] = p;
            p += h;
        }
    }
    if (threadIdx.x == 0) offsets[E] = total;
    __syncthreads();
    c.place(hist, [&](int64_t i, int p) {
        slots[i] = p;
        if (p >= 0) rows[p] = (int)(i / top);
    });
    for (int64_t p = total + threadIdx.x; p < n; p += kOneThreads) rows[p] = -1;
}

// hist[c, e]: the choices of expert e in chunk c
__global__ __launch_bounds__(kThreads) void moe_route_count(const void* ids, bool wide, int64_t n, int E, int* __restrict__ hist) {
    __shared__ int h[kMaxE];
    for (int e = threadIdx.x; e < E; e += kThreads) h[e] = 0;
    __syncthreads();
    const int64_t c0 = (int64_t)blockIdx.x * kChunk, c1 = min(c0 + kChunk, n);
    for (int64_t i = c0 + threadIdx.x; i < c1; i += kThreads) {
        const int id = id_at(ids, wide, i, E);
        if (id >= 0) atomicAdd(h + id, 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) hist[(int64_t)blockIdx.x * E + e] = h[e];
}

__global__ __launch_bounds__(kThreads) void moe_route_place(const void* ids, bool wide, int64_t n, int top, int E,
                                                            const int* __restrict__ hist, int32_t* counts, int32_t* offsets,
                                                            int32_t* rows, int32_t* slots) {
    constexpr int W = kThreads / 64, PER = kMaxE / kThreads;
    __shared__ int h[W * kMaxE], all[kMaxE], before[kMaxE];
    __shared__ int tmp[W];
    const int chunk = blockIdx.x, chunks = gridDim.x;
    for (int i = threadIdx.x; i < W * E; i += kThreads) h[i] = 0;
    for (int e = threadIdx.x; e < E; e += kThreads) all[e] = before[e] = 0;
    __syncthreads();
    const int64_t c0 = (int64_t)chunk * kChunk, c1 = min(c0 + kChunk, n);
    const Chunk<W> c(ids, wide, E, c0, c1);
    c.count(h);
    // the counts of all chunks: thread t takes expert t % span of chunks t / span, t / span + parts, ...
    const int bits = c.bits < 9 ? c.bits : 9, span = 1 << bits, parts = kThreads >> bits;  // kThreads = 512
    for (int e = threadIdx.x & (span - 1); e < E; e += span) {
        int sum = 0, low = 0;
#pragma unroll 8
        for (int b = threadIdx.x >> bits; b < chunks; b += parts) {
            const int v = hist[(int64_t)b * E + e];
            sum += v;
            low += b < chunk ? v : 0;
        }
        atomicAdd(all + e, sum);
        atomicAdd(before + e, low);
    }
    __syncthreads();
    // thread t: experts PER t .. PER t + PER - 1
    int sum = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) sum += PER * (int)threadIdx.x + k < E ? all[PER * threadIdx.x + k] : 0;
    int total;
    int start = block_scan<kThreads>(sum, tmp, total);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int e = PER * threadIdx.x + k;
        if (e >= E) continue;
        if (chunk == 0) {
            counts[e] = all[e];
            offsets[e] = start;
        }
        int p = start + before[e];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int v = h[w * E + e];
            h[w * E + e] = p;
            p += v;
        }
        start += all[e];
    }
    if (chunk == 0 && threadIdx.x == 0) offsets[E] = total;
    __syncthreads();
    c.place(h, [&](int64_t i, int p) {
        slots[i] = p;
        if (p >= 0) rows[p] = (int)(i / top);
    });
    for (int64_t p = max((int64_t)total, c0) + threadIdx.x; p < c1; p += kThreads) rows[p] = -1;
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

// Row t's softmax: lane j of L holds experts j, j + L, ...  A row with no logit above -infinity has no
// probabilities (all 0); a NaN or +infinity makes the row NaN.
template <int L, int V, bool HALF>
__device__ __forceinline__ void row_softmax(const void* logits, int64_t t, int E, float (&p)[V]) {
    const int j = threadIdx.x & (L - 1);
    float top = -__builtin_inff(), sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = j + i * L;
        p[i] = -__builtin_inff();
        if (e < E) {
            if constexpr (HALF) p[i] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(logits)[t * E + e] << 16);
            else p[i] = reinterpret_cast<const float*>(logits)[t * E + e];
        }
        top = fmaxf(top, p[i]);
    }
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

// Workgroup sum in a fixed order
template <typename T, int THREADS>
__device__ __forceinline__ T block_sum(T v, T* tmp) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    T s = tmp[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) s += tmp[w];
    return s;
}

// Every workgroup sums its rows' shares of the loss; part[b] (or the loss itself, when there is one workgroup).
template <int L, int V, bool HALF>
__global__ __launch_bounds__(kLossThreads) void moe_balance_kernel(const void* __restrict__ logits, int64_t T, int E,
                                                                   const int32_t* __restrict__ counts,
                                                                   const uint8_t* __restrict__ mask, float coef, float* loss,
                                                                   float* __restrict__ w, double* __restrict__ part) {
    __shared__ int64_t tmp[kLossThreads / 64];
    __shared__ double dtmp[kLossThreads / 64];
    const int j = threadIdx.x & (L - 1);
    int64_t chosen = 0, live = 0;
    for (int e = threadIdx.x; e < E; e += kLossThreads) chosen += counts[e];
    chosen = block_sum<int64_t, kLossThreads>(chosen, tmp);
    if (mask) {
        // 16 bytes at a time from the first aligned one; every workgroup counts them all
        const int64_t head = min((int64_t)(-(uintptr_t)mask & 15), T), vecs = (T - head) / 16;
        const uint4* v = reinterpret_cast<const uint4*>(mask + head);
        for (int64_t i = threadIdx.x; i < vecs; i += kLossThreads) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int b = 0; b < 32; b += 8) live += (w[k] >> b & 0xff) != 0;
        }
        for (int64_t t = threadIdx.x; t < head; t += kLossThreads) live += mask[t] != 0;
        for (int64_t t = head + 16 * vecs + threadIdx.x; t < T; t += kLossThreads) live += mask[t] != 0;
        live = block_sum<int64_t, kLossThreads>(live, tmp);
    } else {
        live = T;
    }
    const double unit = chosen > 0 && live > 0 ? (double)coef * E / ((double)chosen * (double)live) : 0.0;
    float we[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = j + i * L;
        we[i] = e < E ? (float)(unit * counts[e]) : 0.f;
        if (blockIdx.x == 0 && (int)threadIdx.x < L && e < E) w[e] = we[i];
    }
    double sum = 0;
    const int per = kLossThreads / L;  // rows per workgroup and round
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < T; t0 += (int64_t)gridDim.x * per) {
        const int64_t t = t0 + threadIdx.x / L;
        if (t >= T || (mask && mask[t] == 0)) continue;
        float p[V], s = 0.f;
        row_softmax<L, V, HALF>(logits, t, E, p);
#pragma unroll
        for (int i = 0; i < V; ++i) s = __builtin_fmaf(p[i], we[i], s);
        sum += s;
    }
    sum = block_sum<double, kLossThreads>(sum, dtmp);
    if (threadIdx.x == 0) {
        if (gridDim.x == 1) *loss = (float)sum;
        else part[blockIdx.x] = sum;
    }
}

__global__ __launch_bounds__(kLossThreads) void moe_balance_finish(const double* __restrict__ part, int n, float* loss) {
    __shared__ double tmp[kLossThreads / 64];
    double s = (int)threadIdx.x < n ? part[threadIdx.x] : 0.0;
    s = block_sum<double, kLossThreads>(s, tmp);
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
    const int per = kLossThreads / L;
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < T; t0 += (int64_t)gridDim.x * per) {
        const int64_t t = t0 + threadIdx.x / L;
        if (t >= T) continue;
        float p[V], s = 0.f;
        const bool live = !mask || mask[t] != 0;
        if (live) {
            row_softmax<L, V, HALF>(logits, t, E, p);
#pragma unroll
            for (int i = 0; i < V; ++i) s = __builtin_fmaf(p[i], we[i], s);
            s = row_sum<L>(s);
        }
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
    return n <= kOneMax ? 0 : (size_t)((n + kChunk - 1) / kChunk) * E * sizeof(int);
}

hipError_t launch_moe_route(const void* ids, bool wide, int64_t T, int64_t top, int64_t E, int32_t* counts, int32_t* offsets,
                            int32_t* rows, int32_t* slots, void* workspace, hipStream_t st) {
    const int64_t n = T * top;
    if (n <= kOneMax) {
        hipLaunchKernelGGL(moe_route_one, dim3(1), dim3(kOneThreads), 0, st, ids, wide, n, (int)top, (int)E, counts, offsets,
                           rows, slots);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)((n + kChunk - 1) / kChunk));
    int* hist = reinterpret_cast<int*>(workspace);
    hipLaunchKernelGGL(moe_route_count, grid, dim3(kThreads), 0, st, ids, wide, n, (int)E, hist);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(moe_route_place, grid, dim3(kThreads), 0, st, ids, wide, n, (int)top, (int)E, hist, counts, offsets, rows,
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
