// Rows of a table by index (mpnn_embed), the stable order of the indexes (mpnn_embed_plan) and the table's gradient by
// that order (mpnn_embed_backward):
//   out[i] = scale table[index[i]],  dtable[v] = scale * sum of dout[i] over the rows i of index v.
// An entry's rows are added in their order, in fp32, by one block where there are at most `window` of them.  Longer
// ones are split at the multiples of `window` places, whose sums are added afterwards: a window has the end of at most one
// long entry and the start of at most one other, so two partial sums a window are enough whatever the entries' lengths.
#include <algorithm>

#include "impl.h"
#include "rows.h"

namespace mpnn {

namespace {

template <class T>
__global__ __launch_bounds__(256) void k_embed(Items it, int width, int entries, const int32_t *__restrict__ index, const T *__restrict__ table,
                                               float scale, T *__restrict__ out) {
    constexpr int W = Chunk<T>::W;
    const int64_t block = xcd_block();
    if (block * it.rows >= it.n) return;
    Chunk<T> v[kUnroll];
    int64_t row[kUnroll];
    int c[kUnroll], at[kUnroll];
    const int many = it.items / 256;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= many) break;
        item_at(it, block, u, row[u], c[u]);
        at[u] = index[row[u]];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= many) break;
        v[u].load(table + (int64_t)min(max(at[u], 0), entries - 1) * width + c[u] * W, width - c[u] * W);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= many) break;
        const bool there = (unsigned)at[u] < (unsigned)entries;
#pragma unroll
        for (int j = 0; j < W; ++j) v[u].v[j] = from_f32<T>(there ? scale * to_f32(v[u].v[j]) : 0.0f);
        v[u].store(out + row[u] * width + c[u] * W, width - c[u] * W);
    }
}

// The segment that has place q: the last entry whose offset is at most q (0 where there is none), by one wave.
__device__ __forceinline__ int entry_of(const int32_t *offsets, int entries, int64_t q) {
    const int lane = threadIdx.x & 63;
    int low = 0, count = entries;               // the answer is in low .. low + count - 1
    while (count > 1) {
        const int step = (count + 63) / 64, e = min(lane * step, count - 1);
        const uint64_t below = __ballot(offsets[low + e] <= q);
        const int l = max(63 - __clzll((long long)below), 0);      // offsets ascend
        const int at = min(l * step, count - 1);
        low += at;
        count = min(step, count - at);
    }
    return __builtin_amdgcn_readfirstlane(low);
}

constexpr int kAhead = 8;       // rows in flight

// Sums of the rows `from` .. `to` of the order, one chunk of columns a thread, every `slices`-th row; then over the slices.
template <class T>
__device__ __forceinline__ void add_rows(const T *dout, int64_t ld, const int32_t *source, int64_t n, int64_t from, int64_t to, int c, int width,
                                         int slice, int slices, float (&s)[Chunk<T>::W]) {
    constexpr int W = Chunk<T>::W;
    for (int64_t q = from + slice; q < to; q += kAhead * slices) {
        Chunk<T> v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t p = q + u * slices;
            const int64_t i = min((int64_t)(uint32_t)source[min(p, to - 1)], n - 1);
            v[u].load(dout + i * ld + c * W, width - c * W);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int j = 0; j < W; ++j) s[j] += q + u * slices < to ? to_f32(v[u].v[j]) : 0.0f;
    }
}
__device__ __forceinline__ void add_parts(const float *part, int width, int64_t window, int64_t from, int64_t to, int c, int W, int slice, int slices,
                                          float *s) {
    for (int64_t w = from / window + slice; w <= (to - 1) / window; w += slices) {
        const float *p = part + (2 * w + (from > w * window ? 1 : 0)) * width;
        for (int j = 0; j < W; ++j) s[j] += c * W + j < width ? p[c * W + j] : 0.0f;
    }
}
// The slices' sums of a chunk, in their order, by the first slice.
template <int W> __device__ __forceinline__ void join(float (*sums)[W], int chunks, int slice, int slices, int lc, float (&s)[W]) {
    __syncthreads();
    if (slice < slices)
#pragma unroll
        for (int j = 0; j < W; ++j) sums[slice * chunks + lc][j] = s[j];
    __syncthreads();
    if (slice != 0) return;
    for (int k = 1; k < slices; ++k)
#pragma unroll
        for (int j = 0; j < W; ++j) s[j] += sums[k * chunks + lc][j];
}

// A window's rows of entries that are longer than it.  blockIdx.y: a stripe of `chunks` chunks.
template <class T>
__global__ __launch_bounds__(256) void k_embed_windows(int64_t n, int width, int entries, int64_t window, int chunks, const int32_t *__restrict__ offsets,
                                                       const int32_t *__restrict__ source, const T *__restrict__ dout, int64_t ld,
                                                       float *__restrict__ part) {
    constexpr int W = Chunk<T>::W;
    __shared__ float sums[256][W];
    const int64_t used = min(max((int64_t)offsets[entries], (int64_t)0), n), from = (int64_t)blockIdx.x * window, to = min(from + window, used);
    if (from >= to) return;
    const int slices = 256 / chunks, slice = threadIdx.x / chunks, lc = threadIdx.x % chunks, c = blockIdx.y * chunks + lc;
    const int first = entry_of(offsets, entries, from), last = entry_of(offsets, entries, to - 1);
    for (int side = 0; side < 2; ++side) {
        const int e = side ? last : first;
        const int64_t start = max((int64_t)offsets[e], (int64_t)0), end = min((int64_t)offsets[e + 1], used);
        if ((side && (last == first || start <= from)) || end - start <= window) continue;
        float s[W] = {};
        const bool in = slice < slices && c * W < width;
        if (in) add_rows(dout, ld, source, n, max(start, from), min(end, to), c, width, slice, slices, s);
        join<W>(sums, chunks, slice, slices, lc, s);
        if (in && slice == 0)
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (c * W + j < width) part[(2 * (int64_t)blockIdx.x + side) * width + c * W + j] = s[j];
    }
}

template <class T>
__global__ __launch_bounds__(256) void k_embed_entries(int64_t n, int width, int entries, int64_t window, int chunks, int64_t first,
                                                       const int32_t *__restrict__ offsets, const int32_t *__restrict__ source,
                                                       const T *__restrict__ dout, int64_t ld, const float *__restrict__ part, float scale,
                                                       float *__restrict__ dtable) {
    constexpr int W = Chunk<T>::W;
    __shared__ float sums[256][W];
    const int64_t e = first + blockIdx.x;
    const int slices = 256 / chunks, slice = threadIdx.x / chunks, lc = threadIdx.x % chunks, c = blockIdx.y * chunks + lc;
    const int64_t used = min(max((int64_t)offsets[entries], (int64_t)0), n);
    const int64_t start = max((int64_t)offsets[e], (int64_t)0), end = min((int64_t)offsets[e + 1], used);
    const bool in = slice < slices && c * W < width;
    float s[W] = {};
    if (in && end > start) {
        if (end - start > window) add_parts(part, width, window, start, end, c, W, slice, slices, s);
        else add_rows(dout, ld, source, n, start, end, c, width, slice, slices, s);
    }
    join<W>(sums, chunks, slice, slices, lc, s);
    if (in && slice == 0)
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (c * W + j < width) dtable[e * width + c * W + j] = scale * s[j];
}

// The order of more entries than one counting sort takes: by the low ten bits of the index, then by the high ones.
constexpr int kDigit = 10;
__global__ __launch_bounds__(256) void k_embed_digit(int64_t n, int entries, int shift, const int32_t *__restrict__ index, const int32_t *__restrict__ order,
                                                     int32_t *__restrict__ digit) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int v = index[order ? order[i] : i];
    digit[i] = (unsigned)v < (unsigned)entries ? v >> shift & ((1 << kDigit) - 1) : -1;
}
__global__ __launch_bounds__(256) void k_embed_compose(int64_t n, int entries, const int32_t *__restrict__ index, const int32_t *__restrict__ low,
                                                       const int32_t *__restrict__ high, int32_t *__restrict__ source, int32_t *__restrict__ key) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int32_t p = low[high[i]], v = index[p];
    source[i] = p;
    key[i] = (unsigned)v < (unsigned)entries ? v : entries;
}
// offsets[v]: the first place whose key is at least v
__global__ __launch_bounds__(256) void k_embed_offsets(int64_t n, int entries, const int32_t *__restrict__ key, int32_t *__restrict__ offsets) {
    const int v = blockIdx.x * 256 + threadIdx.x;
    if (v > entries) return;
    int64_t low = 0, high = n;
    while (low < high) {
        const int64_t mid = (low + high) / 2;
        if (key[mid] < v) low = mid + 1;
        else high = mid;
    }
    offsets[v] = (int32_t)low;
}

template <class T>
Status embed_t(Context &cx, int64_t n, int width, int entries, const int32_t *index, const T *table, float scale, T *out) {
    const int per = (width + Chunk<T>::W - 1) / Chunk<T>::W;
    return by_launches(n, kLaunchBlocks * items_of(n, per).rows, [&](int64_t from, int64_t rows) -> Status {
        const Items it = items_of(rows, per);
        k_embed<T><<<grid_of(it), 256, 0, cx.stream>>>(it, width, entries, index + from, table, scale, out + from * width);
        MPNN_HIP(hipGetLastError());
        return Status::ok();
    });
}

template <class T>
Status embed_backward_t(Context &cx, int64_t n, int width, int entries, const T *dout, int64_t ld, const int32_t *offsets, const int32_t *source,
                        float scale, float *dtable) {
    const int per = (width + Chunk<T>::W - 1) / Chunk<T>::W;
    const int64_t window = std::max<int64_t>(64, (n + 1023) / 1024), windows = n > window ? (n + window - 1) / window : 0;
    int chunks = std::min(per, 256);
    void *ws = nullptr;
    MPNN_TRY(cx.rows_scratch(sizeof(float) * (size_t)(2 * windows * width), &ws));
    float *const part = static_cast<float *>(ws);
    if (windows) {
        k_embed_windows<T><<<dim3((unsigned)windows, (per + chunks - 1) / chunks), 256, 0, cx.stream>>>(n, width, entries, window, chunks, offsets, source,
                                                                                                    dout, ld, part);
        MPNN_HIP(hipGetLastError());
    }
    const unsigned stripes = (per + chunks - 1) / chunks;
    return by_launches(entries, kLaunchBlocks / stripes, [&](int64_t from, int64_t count) -> Status {
        k_embed_entries<T><<<dim3((unsigned)count, stripes), 256, 0, cx.stream>>>(n, width, entries, window, chunks, from, offsets, source, dout, ld, part,
                                                                                 scale, dtable);
        MPNN_HIP(hipGetLastError());
        return Status::ok();
    });
}

}  // namespace

Status embed(Context &cx, int dtype, int64_t n, int width, int entries, const int32_t *index, const void *table, float scale, void *out) {
    if (n == 0) return Status::ok();
    return dtype == MPNN_BF16 ? embed_t(cx, n, width, entries, index, (const bf16 *)table, scale, (bf16 *)out)
                              : embed_t(cx, n, width, entries, index, (const float *)table, scale, (float *)out);
}

Status embed_plan(Context &cx, int64_t n, int entries, const int32_t *index, int32_t *offsets, int32_t *source) {
    if (entries <= 1 << kDigit) {
        void *ws = nullptr;
        MPNN_TRY(cx.rows_scratch(route_plan_scratch(n, entries), &ws));
        return route_plan_at(cx, n, entries, index, offsets, source, nullptr, ws);
    }
    const int high = ((entries - 1) >> kDigit) + 1;
    const size_t counts = std::max(route_plan_scratch(n, 1 << kDigit), route_plan_scratch(n, high)), each = (size_t)std::max<int64_t>(n, 1);
    void *ws = nullptr;
    MPNN_TRY(cx.rows_scratch(counts + sizeof(int32_t) * (3 * each + (1 << kDigit) + 1), &ws));
    int32_t *const digit = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + counts), *const one = digit + each, *const two = one + each,
            *const ends = two + each;
    const unsigned grid = grid_for(n);
    k_embed_digit<<<grid, 256, 0, cx.stream>>>(n, entries, 0, index, nullptr, digit);
    MPNN_HIP(hipGetLastError());
    MPNN_TRY(route_plan_at(cx, n, 1 << kDigit, digit, ends, one, nullptr, ws));
    k_embed_digit<<<grid, 256, 0, cx.stream>>>(n, entries, kDigit, index, one, digit);
    MPNN_HIP(hipGetLastError());
    MPNN_TRY(route_plan_at(cx, n, high, digit, ends, two, nullptr, ws));
    k_embed_compose<<<grid, 256, 0, cx.stream>>>(n, entries, index, one, two, source, digit);
    MPNN_HIP(hipGetLastError());
    k_embed_offsets<<<grid_for((int64_t)entries + 1), 256, 0, cx.stream>>>(n, entries, digit, offsets);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

Status embed_backward(Context &cx, int dtype, int64_t n, int width, int entries, const void *dout, int64_t ld, const int32_t *offsets,
                      const int32_t *source, float scale, float *dtable) {
    return dtype == MPNN_BF16 ? embed_backward_t(cx, n, width, entries, (const bf16 *)dout, ld, offsets, source, scale, dtable)
                              : embed_backward_t(cx, n, width, entries, (const float *)dout, ld, offsets, source, scale, dtable);
}

}  // namespace mpnn
