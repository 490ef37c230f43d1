// Rows sorted by expert and back (mpnn_route_*).  The pairs p = i k + s of row i and its slot s are ordered by
// expert with a stable counting sort; pairs whose expert is outside 0 .. E-1 keep a place after the last segment
// (treated as expert E), so `source` and `position` are inverse permutations of all n k pairs and every index that
// a kernel reads from them is one it can check against n k.
#include <type_traits>

#include "impl.h"
#include "rows.h"

namespace mpnn {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanItems = 16;                             // pairs per lane
constexpr int kPlanChunk = kPlanThreads * kPlanItems;      // pairs per block, contiguous
constexpr int kMaxBins = 1024 + 1;                         // experts and the dropped pairs

__device__ __forceinline__ int bin_of(int e, int n_experts) { return (unsigned)e < (unsigned)n_experts ? e : n_experts; }

// counts[bin][block]: pairs of each bin in the block's chunk (integer adds: the order does not matter)
__global__ void k_route_count(const int32_t *__restrict__ expert, int64_t pairs, int n_experts, int32_t *__restrict__ counts) {
    __shared__ int32_t h[kMaxBins];
    for (int b = threadIdx.x; b <= n_experts; b += kPlanThreads) h[b] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kPlanChunk;
    for (int j = 0; j < kPlanItems; ++j) {
        const int64_t p = base + j * kPlanThreads + threadIdx.x;
        if (p < pairs) atomicAdd(&h[bin_of(expert[p], n_experts)], 1);
    }
    __syncthreads();
    for (int b = threadIdx.x; b <= n_experts; b += kPlanThreads) counts[(int64_t)b * gridDim.x + blockIdx.x] = h[b];
}

// Inclusive prefix sum over the block's threads (kPlanThreads of them).
__device__ __forceinline__ int block_scan(int v, int32_t *sh) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int a = __shfl_up(v, d);
        if (lane >= d) v += a;
    }
    if (lane == 63) sh[wave] = v;
    __syncthreads();
    for (int w = 0; w < wave; ++w) v += sh[w];
    __syncthreads();
    return v;
}

// One block per bin: the counts of the bin become their exclusive prefix over the blocks; total[bin] the sum.
__global__ void k_route_scan(int32_t *__restrict__ counts, int blocks, int32_t *__restrict__ total) {
    __shared__ int32_t sh[kPlanWaves];
    __shared__ int32_t carry;
    int32_t *c = counts + (int64_t)blockIdx.x * blocks;
    if (threadIdx.x == 0) carry = 0;
    __syncthreads();
    for (int base = 0; base < blocks; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        const int v = i < blocks ? c[i] : 0;
        const int s = block_scan(v, sh) + carry;
        __syncthreads();
        if (i < blocks) c[i] = s - v;
        if (threadIdx.x == kPlanThreads - 1) carry = s;
        __syncthreads();
    }
    if (threadIdx.x == 0) total[blockIdx.x] = carry;
}

// Each wave takes a contiguous quarter of the block's chunk, 64 pairs at a time.  A pair's place is its bin's
// start, the bin's pairs in earlier blocks and in the block's earlier waves, and its rank among the wave's own pairs
// of the bin: those before this iteration, and the lower lanes of equal bin (one ballot per bit of the bin).
// Without earlier blocks (counts = nullptr, one block) the bins' totals come from the wave counts themselves.
__global__ void k_route_place(const int32_t *__restrict__ expert, int64_t pairs, int n_experts, const int32_t *__restrict__ counts,
                              const int32_t *__restrict__ total, int32_t *__restrict__ offsets, int32_t *__restrict__ source,
                              int32_t *__restrict__ position) {
    __shared__ int32_t h[kPlanWaves][kMaxBins];
    __shared__ int32_t sh[kPlanWaves];
    __shared__ int32_t carry;
    const int bins = n_experts + 1;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int b = threadIdx.x; b < bins; b += kPlanThreads)
        for (int w = 0; w < kPlanWaves; ++w) h[w][b] = 0;
    if (threadIdx.x == 0) carry = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kPlanChunk + wave * (64 * kPlanItems);
    int bin[kPlanItems];
#pragma unroll
    for (int j = 0; j < kPlanItems; ++j) {
        const int64_t p = base + j * 64 + lane;
        bin[j] = p < pairs ? bin_of(expert[p], n_experts) : -1;
        if (bin[j] >= 0) atomicAdd(&h[wave][bin[j]], 1);
    }
    __syncthreads();
    for (int b0 = 0; b0 < bins; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int mine = 0, all = 0;
        if (b < bins) {
            if (total) {
                all = total[b];
                mine = counts[(int64_t)b * gridDim.x + blockIdx.x];
            } else {
                for (int w = 0; w < kPlanWaves; ++w) all += h[w][b];
            }
        }
        const int start = block_scan(all, sh) - all + carry;
        __syncthreads();
        if (threadIdx.x == kPlanThreads - 1) carry = start + all;
        if (b < bins) {
            if (blockIdx.x == 0) offsets[b] = start;
            int run = start + mine;
            for (int w = 0; w < kPlanWaves; ++w) {
                const int c = h[w][b];
                h[w][b] = run;
                run += c;
            }
        }
        __syncthreads();
    }
    const int bits = 32 - __clz(n_experts);   // bins 0 .. n_experts
#pragma unroll
    for (int j = 0; j < kPlanItems; ++j) {
        const int64_t p = base + j * 64 + lane;
        uint64_t same = __ballot(bin[j] >= 0);
        for (int t = 0; t < bits; ++t) {
            const uint64_t set = __ballot((bin[j] >> t) & 1);
            same &= (bin[j] >> t) & 1 ? set : ~set;
        }
        if (bin[j] >= 0) {
            const int q = h[wave][bin[j]] + __popcll(same & ((1ull << lane) - 1));
            source[q] = (int32_t)p;
            position[p] = q;
            // the highest lane of the bin moves its start past this iteration's pairs
            if ((same >> lane) == 1) h[wave][bin[j]] = q + 1;
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Where a chunk of a row starts: the last chunk of a row is moved back to end with the row (its first values are
// then written twice, equally), so that every access is a whole chunk.  Rows shorter than a chunk go value by value.
template <class T> __device__ __forceinline__ int chunk_start(int c, int width) { return min(c * Chunk<T>::W, width - Chunk<T>::W); }

// sorted[position[i, s]] = x[i]; a pair without an expert gets a row of zeros.  Row-major over x, so that each row is
// read once for its k copies.
template <class T, bool SHORT>
__global__ __launch_bounds__(256) void k_route_scatter(Items it, int k, int width, const T *__restrict__ x, int64_t ldx,
                                                       const int32_t *__restrict__ position, const int32_t *__restrict__ used,
                                                       T *__restrict__ sorted) {
    const int64_t pairs = it.n * k;
    const int live = *used;
    int64_t row[kUnroll];
    int at[kUnroll];
    bool in[kUnroll];
    using V = typename std::conditional<SHORT, T, Chunk<T>>::type;
    V v[kUnroll], zero;
    __builtin_memset(&zero, 0, sizeof zero);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        in[u] = item_at(it, u, row[u], at[u]);
        if (!SHORT) at[u] = chunk_start<T>(at[u], width);
        if (in[u]) __builtin_memcpy(&v[u], x + row[u] * ldx + at[u], sizeof(V));
    }
    for (int s = 0; s < k; ++s)
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (!in[u]) continue;
            const int q = position[row[u] * k + s];
            if ((unsigned)q < (uint64_t)pairs) {
                const V w = q < live ? v[u] : zero;
                __builtin_memcpy(sorted + (int64_t)q * width + at[u], &w, sizeof(V));
            }
        }
}

// out[i] = sum over s of weight[i, s] sorted[position[i, s]], in the order of the slots, in fp32
template <class T, bool SHORT>
__global__ __launch_bounds__(256) void k_route_combine(Items it, int k, int width, const T *__restrict__ sorted,
                                                       const int32_t *__restrict__ position, const int32_t *__restrict__ used,
                                                       const float *__restrict__ weight, T *__restrict__ out) {
    constexpr int W = SHORT ? 1 : Chunk<T>::W, S = 4;     // S slots of a row are loaded together
    const int live = *used;
#pragma unroll 1
    for (int u = 0; u < kUnroll; ++u) {
        int64_t row;
        int at;
        if (!item_at(it, u, row, at)) continue;
        if (!SHORT) at = chunk_start<T>(at, width);
        float sum[W] = {};
        for (int s0 = 0; s0 < k; s0 += S) {
            struct { T v[W]; } y[S];
            bool on[S];
            float w[S];
#pragma unroll
            for (int j = 0; j < S; ++j) {
                const int64_t p = row * k + min(s0 + j, k - 1);
                const int q = position[p];
                on[j] = s0 + j < k && (unsigned)q < (unsigned)live;
                w[j] = weight ? weight[p] : 1.0f;
                // a place without an expert reads another row, whose values are not used
                __builtin_memcpy(&y[j], sorted + (int64_t)(on[j] ? q : 0) * width + at, sizeof y[j]);
            }
#pragma unroll
            for (int j = 0; j < S; ++j)
#pragma unroll
                for (int e = 0; e < W; ++e) sum[e] = on[j] ? fmaf(w[j], to_f32(y[j].v[e]), sum[e]) : sum[e];
        }
        struct { T v[W]; } o;
#pragma unroll
        for (int e = 0; e < W; ++e) o.v[e] = from_f32<T>(sum[e]);
        __builtin_memcpy(out + row * width + at, &o, sizeof o);
    }
}

// dsorted[q] = weight dout[i] and dweight = <dout[i], sorted[q]> for q = position[i, s]; zeros without an expert.
// G lanes take a row and kBackSlots of its slots, so that a chunk of dout is read once for them.
constexpr int kBackSlots = 4;
template <class T, int G>
__global__ __launch_bounds__(256) void k_route_combine_back(int64_t n, int k, int batches, int width, const T *__restrict__ dout, int64_t ld,
                                                            const T *__restrict__ sorted, const int32_t *__restrict__ position,
                                                            const int32_t *__restrict__ used, const float *__restrict__ weight,
                                                            T *__restrict__ dsorted, float *__restrict__ dweight) {
    constexpr int W = Chunk<T>::W, S = kBackSlots;
    const int64_t pairs = n * k;
    const int64_t job = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
    const int64_t i = batches == 1 ? job : job / batches;
    if (i >= n) return;                                   // a whole group of lanes
    const int s0 = batches == 1 ? 0 : (int)(job - i * batches) * S;
    const int lane = threadIdx.x % G, live = *used;
    int q[S];
    bool in[S], on[S];
    float w[S], dot[S] = {};
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const int64_t p = i * k + min(s0 + j, k - 1);
        q[j] = position[p];
        in[j] = s0 + j < k && (unsigned)q[j] < (uint64_t)pairs;
        on[j] = in[j] && q[j] < live;
        w[j] = weight ? weight[p] : 1.0f;
    }
    for (int c = lane * W; c < width; c += G * W) {
        const int left = width - c;
        const Chunk<T> d = load_chunk(dout + i * ld + c, left);
        Chunk<T> y[S];
        if (dweight) {
#pragma unroll
            for (int j = 0; j < S; ++j) y[j] = load_chunk(sorted + (int64_t)(on[j] ? q[j] : 0) * width + c, left);
        }
#pragma unroll
        for (int j = 0; j < S; ++j) {
            Chunk<T> o;
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float v = to_f32(d.v[e]);
                if (dweight) dot[j] = fmaf(v, to_f32(y[j].v[e]), dot[j]);
                o.v[e] = from_f32<T>(on[j] ? w[j] * v : 0.0f);
            }
            if (in[j]) store_chunk(dsorted + (int64_t)q[j] * width + c, o, left);
        }
    }
    if (dweight) {
#pragma unroll
        for (int j = 0; j < S; ++j) {
            const float t = lanes_sum<G>(dot[j]);
            if (lane == 0 && s0 + j < k) dweight[i * k + s0 + j] = on[j] ? t : 0.0f;
        }
    }
}

}  // namespace

Status route_plan(Context &cx, int64_t n, int k, int n_experts, const int32_t *expert, int32_t *offsets, int32_t *source,
                  int32_t *position) {
    const int64_t pairs = n * k;
    const int64_t blocks = (pairs + kPlanChunk - 1) / kPlanChunk;
    if (blocks <= 1) {
        k_route_place<<<1, kPlanThreads, 0, cx.stream>>>(expert, pairs, n_experts, nullptr, nullptr, offsets, source, position);
        MPNN_HIP(hipGetLastError());
        return Status::ok();
    }
    MPNN_TRY(cx.grow(cx.rows_ws, sizeof(int32_t) * (size_t)(n_experts + 1) * (size_t)(blocks + 1)));
    int32_t *counts = cx.rows_ws.as<int32_t>();
    int32_t *total = counts + (int64_t)(n_experts + 1) * blocks;
    k_route_count<<<(unsigned)blocks, kPlanThreads, 0, cx.stream>>>(expert, pairs, n_experts, counts);
    MPNN_HIP(hipGetLastError());
    k_route_scan<<<n_experts + 1, kPlanThreads, 0, cx.stream>>>(counts, (int)blocks, total);
    MPNN_HIP(hipGetLastError());
    k_route_place<<<(unsigned)blocks, kPlanThreads, 0, cx.stream>>>(expert, pairs, n_experts, counts, total, offsets, source, position);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

template <class T>
static Status scatter_t(Context &cx, int64_t n, int k, int width, const void *x, int64_t ldx, const int32_t *position,
                        const int32_t *used, void *sorted) {
    constexpr int W = Chunk<T>::W;
    const Items it = items_of(n, width < W ? width : (width + W - 1) / W);
    auto *kernel = width < W ? k_route_scatter<T, true> : k_route_scatter<T, false>;
    kernel<<<grid_of(it), 256, 0, cx.stream>>>(it, k, width, (const T *)x, ldx, position, used, (T *)sorted);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

Status route_scatter(Context &cx, int dtype, int64_t n, int k, int width, const void *x, int64_t ldx, const int32_t *position,
                     const int32_t *used, void *sorted) {
    if (n == 0) return Status::ok();
    return dtype == MPNN_BF16 ? scatter_t<bf16>(cx, n, k, width, x, ldx, position, used, sorted)
                              : scatter_t<float>(cx, n, k, width, x, ldx, position, used, sorted);
}

template <class T>
static Status combine_t(Context &cx, int64_t n, int k, int width, const void *sorted, const int32_t *position, const int32_t *used,
                        const float *weight, void *out) {
    constexpr int W = Chunk<T>::W;
    const Items it = items_of(n, width < W ? width : (width + W - 1) / W);
    auto *kernel = width < W ? k_route_combine<T, true> : k_route_combine<T, false>;
    kernel<<<grid_of(it), 256, 0, cx.stream>>>(it, k, width, (const T *)sorted, position, used, weight, (T *)out);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

Status route_combine(Context &cx, int dtype, int64_t n, int k, int width, const void *sorted, const int32_t *position,
                     const int32_t *used, const float *weight, void *out) {
    if (n == 0) return Status::ok();
    return dtype == MPNN_BF16 ? combine_t<bf16>(cx, n, k, width, sorted, position, used, weight, out)
                              : combine_t<float>(cx, n, k, width, sorted, position, used, weight, out);
}

template <class T>
static Status combine_back_t(Context &cx, int64_t n, int k, int width, const void *dout, int64_t ld, const void *sorted,
                             const int32_t *position, const int32_t *used, const float *weight, void *dsorted, float *dweight) {
    const int chunks = (width + Chunk<T>::W - 1) / Chunk<T>::W, batches = (k + kBackSlots - 1) / kBackSlots;
    auto run = [&](auto *kernel, int lanes) -> Status {
        kernel<<<grid_for(n * batches, 256 / lanes), 256, 0, cx.stream>>>(n, k, batches, width, (const T *)dout, ld, (const T *)sorted,
                                                                          position, used, weight, (T *)dsorted, dweight);
        MPNN_HIP(hipGetLastError());
        return Status::ok();
    };
    if (chunks <= 8) return run(k_route_combine_back<T, 8>, 8);
    if (chunks <= 16) return run(k_route_combine_back<T, 16>, 16);
    if (chunks <= 32) return run(k_route_combine_back<T, 32>, 32);
    return run(k_route_combine_back<T, 64>, 64);
}

Status route_combine_backward(Context &cx, int dtype, int64_t n, int k, int width, const void *dout, int64_t ld, const void *sorted,
                              const int32_t *position, const int32_t *used, const float *weight, void *dsorted, float *dweight) {
    if (n == 0) return Status::ok();
    return dtype == MPNN_BF16
               ? combine_back_t<bf16>(cx, n, k, width, dout, ld, sorted, position, used, weight, dsorted, dweight)
               : combine_back_t<float>(cx, n, k, width, dout, ld, sorted, position, used, weight, dsorted, dweight);
}

}  // namespace mpnn
