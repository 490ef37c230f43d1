// Rows sorted by expert and back (mpnn_route_*), and the order of embedding rows (mpnn_embed_plan).  The pairs p = i k + s of row
// i and its slot s are ordered by
// expert with a stable counting sort; pairs whose expert is outside 0 .. E-1 keep a place after the last segment
// (treated as expert E), so `source` and `position` are inverse permutations of all n k pairs and every index that
// a kernel reads from them is one it can check against n k.
//
// All of it is bound by HBM, the plan by its launches.  Rows sent to their places: 128,000 x 312 fp32 to one place 65 us
// (320 MB, 4.9 TB/s), 16,384 x 2,048 bf16 to eight 130 us (604 MB, 4.6 TB/s); added up again 57 us (5.6 TB/s) and 122 us
// (5.0 TB/s; 156 us right after the rows were sent out, whose lines are still on their way to memory); the gradient with the
// weights' dot products, 65,536 x 1,024 bf16 from four: 224 us (1.21 GB, 5.4 TB/s).  The plan of 128,000 pairs: 11 us in two
// launches, one launch up to 1,024 pairs (4 us).
#include <algorithm>
#include <type_traits>

#include "impl.h"
#include "rows.h"

namespace mpnn {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kMaxBins = 1024 + 1;                         // experts and the dropped pairs
constexpr int kDigit = 10;                                 // bits of an index that one sort takes

__device__ __forceinline__ int bin_of(int e, int n_experts) { return (unsigned)e < (unsigned)n_experts ? e : n_experts; }

// What a counting sort orders by: the experts of the pairs, or a digit of an embedding's indexes, of which `order` has those that
// an earlier digit has put in order.
struct ByExpert {
    const int32_t *expert;
    __device__ __forceinline__ int key(int64_t p) const { return expert[p]; }
    __device__ __forceinline__ void placed(int64_t p, int q, int32_t *source, int32_t *position) const {
        source[q] = (int32_t)p;
        position[p] = q;
    }
};
struct ByDigit {
    const int32_t *index, *order;
    int entries, shift;
    int32_t *sorted;                       // the indexes in order (entries where one names none), or null
    __device__ __forceinline__ int64_t row(int64_t p) const { return order ? order[p] : p; }
    __device__ __forceinline__ int key(int64_t p) const {
        const int v = index[row(p)];
        return (unsigned)v < (unsigned)entries ? v >> shift & ((1 << kDigit) - 1) : -1;
    }
    __device__ __forceinline__ void placed(int64_t p, int q, int32_t *source, int32_t *) const {
        const int64_t i = row(p);
        source[q] = (int32_t)i;
        if (sorted) sorted[q] = (unsigned)index[i] < (unsigned)entries ? index[i] : entries;
    }
};

// counts[block][bin]: pairs of each bin among the block's 256 ITEMS ones (integer adds: the order does not matter)
template <int ITEMS, class By>
__global__ __launch_bounds__(kPlanThreads) void k_route_count(const By by, int64_t pairs, int n_experts,
                                                              int32_t *__restrict__ counts) {
    __shared__ int32_t h[kMaxBins];
    const int bins = n_experts + 1;
    const int64_t base = (int64_t)blockIdx.x * (kPlanThreads * ITEMS);
    int e[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) e[j] = by.key(min(base + j * kPlanThreads + threadIdx.x, pairs - 1));
    for (int b = threadIdx.x; b < bins; b += kPlanThreads) h[b] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j)
        if (base + j * kPlanThreads + threadIdx.x < pairs) atomicAdd(&h[bin_of(e[j], n_experts)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kPlanThreads) counts[(int64_t)blockIdx.x * bins + b] = h[b];
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

// Many blocks: the counts of 16 bins become their exclusive prefixes over the blocks, and total[bin] their sums.  64
// threads a bin take a stretch of the blocks each.
__global__ __launch_bounds__(1024) void k_route_scan(int32_t *__restrict__ counts, int blocks, int bins, int32_t *__restrict__ total) {
    __shared__ int32_t sh[64][17];
    const int lb = threadIdx.x & 15, slice = threadIdx.x >> 4, b = blockIdx.x * 16 + lb;
    const int each = (blocks + 63) / 64, from = min(slice * each, blocks), to = min(from + each, blocks);
    int s = 0;
    if (b < bins)
#pragma unroll 8
        for (int i = from; i < to; ++i) s += counts[(int64_t)i * bins + b];
    sh[slice][lb] = s;
    __syncthreads();
    int run = 0, all = 0;
    for (int i = 0; i < 64; ++i) {
        run += i < slice ? sh[i][lb] : 0;
        all += sh[i][lb];
    }
    if (b >= bins) return;
    if (slice == 0) total[b] = all;
#pragma unroll 8
    for (int i = from; i < to; ++i) {
        const int c = counts[(int64_t)i * bins + b];
        counts[(int64_t)i * bins + b] = run;
        run += c;
    }
}

// Each wave takes a contiguous quarter of the block's pairs, 64 at a time.  A pair's place is its bin's start, the bin's
// pairs in earlier blocks and in the block's earlier waves, and its rank among the wave's own pairs of the bin: those
// before this iteration, and the lower lanes of equal bin (one ballot per bit of the bin).
// The bins' totals and what earlier blocks hold of them: of one block from its own counts, of up to kSumCounts
// counts from all blocks' counts, which every block adds up for itself (a launch less), else from k_route_scan (`total`).
constexpr int kSumCounts = 16384;
template <int ITEMS, class By>
__global__ __launch_bounds__(kPlanThreads) void k_route_place(const By by, int64_t pairs, int n_experts,
                                                              const int32_t *__restrict__ counts, const int32_t *__restrict__ total,
                                                              int32_t *__restrict__ offsets, int32_t *__restrict__ source,
                                                              int32_t *__restrict__ position) {
    __shared__ int32_t h[kPlanWaves][kMaxBins];
    __shared__ int32_t before[kMaxBins], sums[kMaxBins];
    __shared__ int32_t part[2][kPlanThreads];
    __shared__ int32_t sh[kPlanWaves];
    __shared__ int32_t carry;
    const int bins = n_experts + 1, blocks = gridDim.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t base = (int64_t)blockIdx.x * (kPlanThreads * ITEMS) + wave * (64 * ITEMS);
    int bin[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const int64_t p = base + j * 64 + lane;
        bin[j] = pairs > 0 ? by.key(min(p, pairs - 1)) : 0;
    }
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) bin[j] = base + j * 64 + lane < pairs ? bin_of(bin[j], n_experts) : -1;
    for (int b = threadIdx.x; b < bins; b += kPlanThreads)
        for (int w = 0; w < kPlanWaves; ++w) h[w][b] = 0;
    if (threadIdx.x == 0) carry = 0;
    if (counts && !total) {
        // lanes of a column of bins, slices of the blocks
        const int columns = bins > 32 ? 64 : bins > 16 ? 32 : bins > 8 ? 16 : 8, slices = kPlanThreads / columns;
        const int column = threadIdx.x % columns, slice = threadIdx.x / columns;
        for (int b0 = 0; b0 < bins; b0 += columns) {
            const int b = b0 + column;
            int all = 0, early = 0;
            if (b < bins)
#pragma unroll 8
                for (int i = slice; i < blocks; i += slices) {
                    const int c = counts[(int64_t)i * bins + b];
                    all += c;
                    early += i < (int)blockIdx.x ? c : 0;
                }
            __syncthreads();
            part[0][threadIdx.x] = all;
            part[1][threadIdx.x] = early;
            __syncthreads();
            if (slice == 0 && b < bins) {
                for (int i = 1; i < slices; ++i) {
                    all += part[0][i * columns + column];
                    early += part[1][i * columns + column];
                }
                sums[b] = all;
                before[b] = early;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j)
        if (bin[j] >= 0) atomicAdd(&h[wave][bin[j]], 1);
    __syncthreads();
    for (int b0 = 0; b0 < bins; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int mine = 0, all = 0;
        if (b < bins) {
            if (total) {
                all = total[b];
                mine = counts[(int64_t)blockIdx.x * bins + b];
            } else if (counts) {
                all = sums[b];
                mine = before[b];
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
    for (int j = 0; j < ITEMS; ++j) {
        if (base + j * 64 >= pairs) break;    // all of the wave's
        const int64_t p = base + j * 64 + lane;
        uint64_t same = __ballot(bin[j] >= 0);
        for (int t = 0; t < bits; ++t) {
            const uint64_t set = __ballot((bin[j] >> t) & 1);
            same &= (bin[j] >> t) & 1 ? set : ~set;
        }
        if (bin[j] >= 0) {
            const int q = h[wave][bin[j]] + __popcll(same & ((1ull << lane) - 1));
            by.placed(p, q, source, position);
            // the highest lane of the bin moves its start past this iteration's pairs
            if ((same >> lane) == 1) h[wave][bin[j]] = q + 1;
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// A chunk of a row: the last one of a row is moved back to end with the row (its first values are then written twice,
// equally), so that every access is a whole chunk.  Rows shorter than a chunk go value by value (SHORT).
template <class T, bool SHORT>
struct Piece : Chunk<T, SHORT ? 1 : 16 / sizeof(T)> {
    __device__ __forceinline__ static int start(int c, int width) { return SHORT ? c : min(c * Piece::W, width - Piece::W); }
};
template <class T> int chunks_of(int width) { return width < Chunk<T>::W ? width : (width + Chunk<T>::W - 1) / Chunk<T>::W; }

// Places below this one have an expert.  The count is the caller's memory, and may be that of a longer plan: no place past
// the sorted rows is one, whatever it says.
__device__ __forceinline__ int live_places(const int32_t *used, int64_t pairs) { return (int)min(max((int64_t)*used, (int64_t)0), pairs); }

// out[i] = sum over s of weight[i, s] sorted[position[i, s]], in the order of the slots, in fp32.  S slots of kUnroll / S
// items are loaded together, a thread's only ones (with four items a thread at any S 165 us at 16,384 x 2,048 bf16 from
// eight right after they were sent out, 156 us with one).
template <class T, bool SHORT, int S>
__global__ __launch_bounds__(256) void k_route_combine(Items it, int64_t pairs, int k, int width, const T *__restrict__ sorted,
                                                       const int32_t *__restrict__ position, const int32_t *__restrict__ used,
                                                       const float *__restrict__ weight, T *__restrict__ out) {
    using P = Piece<T, SHORT>;
    constexpr int W = P::W, U = kUnroll / S;
    const int64_t block = xcd_block();
    const int live = live_places(used, pairs), units = it.items / 256;
    int64_t row[U];
    int at[U];
    float sum[U][W] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        item_at(it, block, min(u, units - 1), row[u], at[u]);
        at[u] = P::start(at[u], width);
    }
    for (int s0 = 0; s0 < k; s0 += S) {
        P y[U][S];
        bool on[U][S];
        float w[U][S];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < S; ++j) {
                const int64_t p = row[u] * k + min(s0 + j, k - 1);
                const int q = position[p];
                on[u][j] = s0 + j < k && (unsigned)q < (unsigned)live;
                w[u][j] = weight ? weight[p] : 1.0f;
                // a place without an expert reads another row, whose values are not used
                y[u][j].load(sorted + (int64_t)(on[u][j] ? q : 0) * width + at[u]);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < S; ++j)
#pragma unroll
                for (int e = 0; e < W; ++e)
                    sum[u][e] = on[u][j] ? fmaf(w[u][j], to_f32(y[u][j].v[e]), sum[u][e]) : sum[u][e];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        P o;
#pragma unroll
        for (int e = 0; e < W; ++e) o.v[e] = from_f32<T>(sum[u][e]);
        o.store(out + row[u] * width + at[u]);
    }
}

// dsorted[q] = weight dout[i] and dweight = <dout[i], sorted[q]> for q = position[i, s]; zeros without an expert.  Without
// weight and dweight: the rows dout sent to their places.
// G lanes take a row and S of its slots, so that a chunk of dout is read once for them; lanes past the row's last chunk
// repeat it without counting it in the sums.  (Rows sent to their places by flat items, four chunks of any rows a thread,
// took 107 us at 128,000 x 312 fp32 to one place and 181 us at 16,384 x 2,048 bf16 to eight; by groups of lanes 67 and
// 139 us.)
template <class T, bool SHORT, int G, int S>
__global__ __launch_bounds__(256) void k_route_combine_back(int64_t n, int64_t pairs, int k, int batches, int width, const T *__restrict__ dout, int64_t ld,
                                                            const T *__restrict__ sorted, const int32_t *__restrict__ position,
                                                            const int32_t *__restrict__ used, const float *__restrict__ weight,
                                                            T *__restrict__ dsorted, float *__restrict__ dweight) {
    using P = Piece<T, SHORT>;
    constexpr int W = P::W;
    const int64_t job = xcd_block() * (256 / G) + threadIdx.x / G;
    const int64_t i = batches == 1 ? job : job / batches;
    if (i >= n) return;                                   // a whole group of lanes
    const int s0 = batches == 1 ? 0 : (int)(job - i * batches) * S;
    const int lane = threadIdx.x % G, live = live_places(used, pairs), chunks = (width + W - 1) / W;
    int q[S];
    bool in[S], on[S], all_in = true;
    float w[S], dot[S] = {};
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const int64_t p = i * k + min(s0 + j, k - 1);     // slots past the last repeat it
        q[j] = position[p];
        in[j] = (unsigned)q[j] < (uint64_t)pairs;
        all_in = all_in && in[j];
        on[j] = (unsigned)q[j] < (unsigned)live;
        w[j] = weight ? weight[p] : 1.0f;
    }
    auto step = [&](int c0, auto checked) {
        const int c = c0 + lane, at = P::start(min(c, chunks - 1), width);
        const int skip = c < chunks ? c * W - at : W;      // values of this chunk that another one counts
        P d, y[S];
        d.load(dout + i * ld + at);
        if (dweight) {
#pragma unroll
            for (int j = 0; j < S; ++j) y[j].load(sorted + (int64_t)(on[j] ? q[j] : 0) * width + at);
        }
#pragma unroll
        for (int j = 0; j < S; ++j) {
            P o;
#pragma unroll
            for (int e = 0; e < W; ++e) o.v[e] = from_f32<T>(on[j] ? w[j] * to_f32(d.v[e]) : 0.0f);
            if (!checked() || in[j]) o.store(dsorted + (int64_t)q[j] * width + at);
        }
        if (dweight) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float v = e < skip ? 0.0f : to_f32(d.v[e]);
#pragma unroll
                for (int j = 0; j < S; ++j) dot[j] = e < skip ? dot[j] : fmaf(v, to_f32(y[j].v[e]), dot[j]);
            }
        }
    };
    if (__all(all_in)) {
        for (int c = 0; c < chunks; c += G) step(c, std::false_type{});
    } else {
        for (int c = 0; c < chunks; c += G) step(c, std::true_type{});
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

template <int ITEMS> static int64_t plan_blocks(int64_t pairs) {
    constexpr int kChunk = kPlanThreads * ITEMS;
    return std::max<int64_t>(1, (pairs + kChunk - 1) / kChunk);
}

template <int ITEMS, class By>
static Status plan(Context &cx, int64_t pairs, int n_experts, const By &by, int32_t *offsets, int32_t *source, int32_t *position, void *ws) {
    const int64_t blocks = plan_blocks<ITEMS>(pairs);
    const int bins = n_experts + 1;
    int32_t *counts = nullptr, *total = nullptr;
    if (blocks > 1) {
        counts = static_cast<int32_t *>(ws);
        k_route_count<ITEMS><<<(unsigned)blocks, kPlanThreads, 0, cx.stream>>>(by, pairs, n_experts, counts);
        MPNN_HIP(hipGetLastError());
        if (blocks * bins > kSumCounts) {
            total = counts + blocks * bins;
            k_route_scan<<<(bins + 15) / 16, 1024, 0, cx.stream>>>(counts, (int)blocks, bins, total);
            MPNN_HIP(hipGetLastError());
        }
    }
    k_route_place<ITEMS><<<(unsigned)blocks, kPlanThreads, 0, cx.stream>>>(by, pairs, n_experts, counts, total, offsets, source, position);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

// 1,024 pairs a block, so that the pairs of some 100,000 atoms already fill the GPU's CUs; 4,096 where there are enough
// of them, for fewer counts.
static bool many_pairs(int64_t pairs) { return pairs > (1 << 20); }

static size_t plan_scratch(int64_t pairs, int n_experts) {
    const int64_t blocks = many_pairs(pairs) ? plan_blocks<16>(pairs) : plan_blocks<4>(pairs);
    return blocks > 1 ? sizeof(int32_t) * (size_t)(n_experts + 1) * (size_t)(blocks + 1) : 0;
}

template <class By>
static Status plan_by(Context &cx, int64_t pairs, int n_experts, const By &by, int32_t *offsets, int32_t *source, int32_t *position, void *ws) {
    return many_pairs(pairs) ? plan<16>(cx, pairs, n_experts, by, offsets, source, position, ws)
                             : plan<4>(cx, pairs, n_experts, by, offsets, source, position, ws);
}

Status route_plan(Context &cx, int64_t n, int k, int n_experts, const int32_t *expert, int32_t *offsets, int32_t *source,
                  int32_t *position) {
    void *ws = nullptr;
    MPNN_TRY(cx.rows_scratch(plan_scratch(n * k, n_experts), &ws));
    return plan_by(cx, n * k, n_experts, ByExpert{expert}, offsets, source, position, ws);
}

// offsets[v]: the first place whose index is at least v
static __global__ __launch_bounds__(256) void k_embed_offsets(int64_t n, int entries, const int32_t *__restrict__ sorted, int32_t *__restrict__ offsets) {
    const int v = blockIdx.x * 256 + threadIdx.x;
    if (v > entries) return;
    int64_t low = 0, high = n;
    while (low < high) {
        const int64_t mid = (low + high) / 2;
        if (sorted[mid] < v) low = mid + 1;
        else high = mid;
    }
    offsets[v] = (int32_t)low;
}

// An embedding's order: one counting sort of up to 1,024 entries, else by the low ten bits of the index and then by the high
// ones, rows of no entry last both times (65,536 indexes of 32,000: 34 us, seven launches that wait for each other).
Status embed_plan(Context &cx, int64_t n, int entries, const int32_t *index, int32_t *offsets, int32_t *source) {
    void *ws = nullptr;
    if (entries <= 1 << kDigit) {
        MPNN_TRY(cx.rows_scratch(plan_scratch(n, entries), &ws));
        return plan_by(cx, n, entries, ByDigit{index, nullptr, entries, 0, nullptr}, offsets, source, nullptr, ws);
    }
    const int high = ((entries - 1) >> kDigit) + 1;
    const size_t counts = std::max(plan_scratch(n, 1 << kDigit), plan_scratch(n, high));
    MPNN_TRY(cx.rows_scratch(counts + sizeof(int32_t) * (2 * (size_t)n + (1 << kDigit) + 1), &ws));
    int32_t *const low = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + counts), *const sorted = low + n, *const ends = sorted + n;
    MPNN_TRY(plan_by(cx, n, 1 << kDigit, ByDigit{index, nullptr, entries, 0, nullptr}, ends, low, nullptr, ws));
    MPNN_TRY(plan_by(cx, n, high, ByDigit{index, low, entries, kDigit, sorted}, ends, source, nullptr, ws));
    k_embed_offsets<<<grid_for((int64_t)entries + 1), 256, 0, cx.stream>>>(n, entries, sorted, offsets);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

// Slots that a kernel takes together, as a constant.
template <class F> Status by_slots(int k, F run) {
    if (k == 1) return run(std::integral_constant<int, 1>{});
    if (k == 2) return run(std::integral_constant<int, 2>{});
    return run(std::integral_constant<int, 4>{});
}

template <class T>
static Status combine_t(Context &cx, int64_t n, int k, int width, const void *sorted, const int32_t *position, const int32_t *used,
                        const float *weight, void *out) {
    return by_slots(k, [&](auto slots) -> Status {
        const int per = chunks_of<T>(width);
        auto *kernel = width < Chunk<T>::W ? k_route_combine<T, true, slots()> : k_route_combine<T, false, slots()>;
        return by_launches(n, kLaunchBlocks * items_of(n, per, kUnroll / slots()).rows, [&](int64_t from, int64_t rows) -> Status {
            const Items it = items_of(rows, per, kUnroll / slots());
            kernel<<<grid_of(it), 256, 0, cx.stream>>>(it, n * k, k, width, (const T *)sorted, position + from * k, used,
                                                       weight ? weight + from * k : nullptr, (T *)out + from * width);
            MPNN_HIP(hipGetLastError());
            return Status::ok();
        });
    });
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
    return by_slots(k, [&](auto slots) -> Status {
        constexpr int S = slots();
        const int chunks = chunks_of<T>(width), batches = (k + S - 1) / S;
        auto run = [&](auto *kernel, int lanes) -> Status {
            return by_launches(n, kLaunchBlocks * (256 / lanes) / batches, [&](int64_t from, int64_t rows) -> Status {
                kernel<<<grid_xcd(rows * batches, 256 / lanes), 256, 0, cx.stream>>>(
                    rows, n * k, k, batches, width, (const T *)dout + from * ld, ld, (const T *)sorted, position + from * k, used,
                    weight ? weight + from * k : nullptr, (T *)dsorted, dweight ? dweight + from * k : nullptr);
                MPNN_HIP(hipGetLastError());
                return Status::ok();
            });
        };
        if (width < Chunk<T>::W) return run(k_route_combine_back<T, true, 8, S>, 8);
        if (chunks <= 8) return run(k_route_combine_back<T, false, 8, S>, 8);
        if (chunks <= 16) return run(k_route_combine_back<T, false, 16, S>, 16);
        if (chunks <= 32) return run(k_route_combine_back<T, false, 32, S>, 32);
        return run(k_route_combine_back<T, false, 64, S>, 64);
    });
}

Status route_combine_backward(Context &cx, int dtype, int64_t n, int k, int width, const void *dout, int64_t ld, const void *sorted,
                              const int32_t *position, const int32_t *used, const float *weight, void *dsorted, float *dweight) {
    if (n == 0) return Status::ok();
    return dtype == MPNN_BF16
               ? combine_back_t<bf16>(cx, n, k, width, dout, ld, sorted, position, used, weight, dsorted, dweight)
               : combine_back_t<float>(cx, n, k, width, dout, ld, sorted, position, used, weight, dsorted, dweight);
}

Status route_scatter(Context &cx, int dtype, int64_t n, int k, int width, const void *x, int64_t ldx, const int32_t *position,
                     const int32_t *used, void *sorted) {
    return route_combine_backward(cx, dtype, n, k, width, x, ldx, nullptr, position, used, nullptr, sorted, nullptr);
}

}  // namespace mpnn
