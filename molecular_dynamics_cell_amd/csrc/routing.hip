// Rows sorted by expert and back (mpnn_route_*).  The pairs p = i k + s of row i and its slot s are ordered by
// expert with a stable counting sort; pairs whose expert is outside 0 .. E-1 keep a place after the last segment
// (treated as expert E), so `source` and `position` are inverse permutations of all n k pairs and every index that
// a kernel reads from them is one it can check against n k.
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

// sorted[position[i, s]] = x[i]; a pair without an expert gets a row of zeros
template <class T>
__global__ void k_route_scatter(int64_t n, int k, int width, const T *__restrict__ x, int64_t ldx, const int32_t *__restrict__ position,
                                const int32_t *__restrict__ used, T *__restrict__ sorted) {
    const int64_t pairs = n * k;
    const int64_t p = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (p >= pairs) return;
    const int q = position[p];
    if ((unsigned)q >= (uint64_t)pairs) return;
    const bool live = q < *used;
    const T *from = x + (p / k) * ldx;
    T *to = sorted + (int64_t)q * width;
    for (int c = threadIdx.x & 63; c < width; c += 64) to[c] = live ? from[c] : from_f32<T>(0.0f);
}

// out[i] = sum over s of weight[i, s] sorted[position[i, s]], in the order of the slots, in fp32
template <class T>
__global__ void k_route_combine(int64_t n, int k, int width, const T *__restrict__ sorted, const int32_t *__restrict__ position,
                                const int32_t *__restrict__ used, const float *__restrict__ weight, T *__restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (i >= n) return;
    const int live = *used;
    for (int c = threadIdx.x & 63; c < width; c += 64) {
        float sum = 0.0f;
        for (int s = 0; s < k; ++s) {
            const int q = position[i * k + s];
            if ((unsigned)q < (unsigned)live) {
                const float v = to_f32(sorted[(int64_t)q * width + c]);
                sum = weight ? fmaf(weight[i * k + s], v, sum) : sum + v;
            }
        }
        out[i * width + c] = from_f32<T>(sum);
    }
}

// dsorted[q] = weight dout[i] and dweight = <dout[i], sorted[q]> for q = position[i, s]; zeros without an expert
template <class T>
__global__ void k_route_combine_back(int64_t n, int k, int width, const T *__restrict__ dout, int64_t ld, const T *__restrict__ sorted,
                                     const int32_t *__restrict__ position, const int32_t *__restrict__ used,
                                     const float *__restrict__ weight, T *__restrict__ dsorted, float *__restrict__ dweight) {
    const int64_t pairs = n * k;
    const int64_t p = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (p >= pairs) return;
    const int q = position[p];
    const bool in = (unsigned)q < (uint64_t)pairs, live = in && q < *used;
    const float w = live && weight ? weight[p] : 1.0f;
    const T *from = dout + (p / k) * ld;
    float dot = 0.0f;
    for (int c = threadIdx.x & 63; c < width && in; c += 64) {
        const int64_t at = (int64_t)q * width + c;
        const float d = live ? to_f32(from[c]) : 0.0f;
        if (live && dweight) dot = fmaf(d, to_f32(sorted[at]), dot);   // without dweight there may be no sorted rows
        dsorted[at] = from_f32<T>(live ? w * d : 0.0f);
    }
    dot = wave_sum(dot);
    if (dweight && (threadIdx.x & 63) == 0) dweight[p] = live ? dot : 0.0f;
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
    k_route_scatter<T><<<grid_for(n * k, 4), 256, 0, cx.stream>>>(n, k, width, (const T *)x, ldx, position, used, (T *)sorted);
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
    k_route_combine<T><<<grid_for(n, 4), 256, 0, cx.stream>>>(n, k, width, (const T *)sorted, position, used, weight, (T *)out);
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
    k_route_combine_back<T><<<grid_for(n * k, 4), 256, 0, cx.stream>>>(n, k, width, (const T *)dout, ld, (const T *)sorted, position,
                                                                       used, weight, (T *)dsorted, dweight);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

Status route_combine_backward(Context &cx, int dtype, int64_t n, int k, int width, const void *dout, int64_t ld, const void *sorted,
                              const int32_t *position, const int32_t *used, const float *weight, void *dsorted, float *dweight) {
    if (n == 0) return Status::ok();
    return dtype == MPNN_BF16
               ? combine_back_t<bf16>(cx, n, k, width, dout, ld, sorted, position, used, weight, dsorted, dweight)
               : combine_back_t<float>(cx, n, k, width, dout, ld, sorted, position, used, weight, dsorted, dweight);
}

}  // namespace mpnn
