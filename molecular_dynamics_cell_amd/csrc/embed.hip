// Rows of a table by index (mpnn_embed) and the table's gradient by the indexes' order (mpnn_embed_backward):
//   out[i] = scale table[index[i]],  dtable[v] = scale * sum of dout[i] over the rows i of index v.
// An entry's rows are added in their order, in fp32, by a few lanes where there are at most `window` of them.  Longer
// ones are split at the multiples of `window` places, whose sums are added afterwards: a window has the end of at most one
// long entry and the start of at most one other, so two partial sums a window are enough whatever the entries' lengths.
// Bound by HBM: 400,002 rows of 128 fp32 40 us (5.2 TB/s, all but the table is written); gradients of 128,000 x 312 fp32 of five
// entries 44 us (windows 30, 5.4 TB/s; their sums 8), of 65,536 x 1,024 bf16 of 32,000, a few frequent, without the order 96 us
// (windows 18, their sums 17, the other entries 49: 131 MB of fp32 gradients are written).
#include <algorithm>
#include <type_traits>

#include "impl.h"
#include "rows.h"

namespace mpnn {

namespace {

// A chunk of a row: the last one is moved back to end with the row (its first columns are then done twice, equally), so that
// no load has a condition beside it.  Rows shorter than a chunk go value by value (SHORT).
template <class T, bool SHORT> struct Part : Chunk<T, SHORT ? 1 : 16 / sizeof(T)> {
    __device__ __forceinline__ static int start(int c, int width) { return SHORT ? c : min(c * Part::W, width - Part::W); }
};
template <class T> int parts_of(int width) { return width < Chunk<T>::W ? width : (width + Chunk<T>::W - 1) / Chunk<T>::W; }

template <class T, bool SHORT>
__global__ __launch_bounds__(256) void k_embed(Items it, int width, int entries, const int32_t *__restrict__ index, const T *__restrict__ table,
                                               float scale, T *__restrict__ out) {
    using P = Part<T, SHORT>;
    const int64_t block = xcd_block();
    if (block * it.rows >= it.n) return;
    P v[kUnroll];
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
        v[u].load(table + (int64_t)min(max(at[u], 0), entries - 1) * width + P::start(c[u], width));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= many) break;
        const bool there = (unsigned)at[u] < (unsigned)entries;
#pragma unroll
        for (int j = 0; j < P::W; ++j) v[u].v[j] = from_f32<T>(there ? scale * to_f32(v[u].v[j]) : 0.0f);
        v[u].store(out + row[u] * width + P::start(c[u], width));
    }
}

// The segments that have places p <= q: of each the last entry whose offset is at most the place (0 where there is none), by
// one wave, both searches at once.
__device__ __forceinline__ void entries_of(const int32_t *offsets, int entries, int64_t p, int64_t q, int &first, int &last) {
    const int lane = threadIdx.x & 63;
    int low[2] = {0, 0}, count[2] = {entries, entries};     // the answers are in low .. low + count - 1
    const int64_t place[2] = {p, q};
    while (max(count[0], count[1]) > 1) {
        int at[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) at[k] = offsets[low[k] + min(lane * ((count[k] + 63) / 64), count[k] - 1)];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int step = (count[k] + 63) / 64;
            const uint64_t below = __ballot(at[k] <= place[k]);
            const int l = max(63 - __clzll((long long)below), 0), e = min(l * step, count[k] - 1);      // offsets ascend
            low[k] += e;
            count[k] = min(step, count[k] - e);
        }
    }
    first = __builtin_amdgcn_readfirstlane(low[0]);
    last = __builtin_amdgcn_readfirstlane(low[1]);
}

// s += the rows at places from, from + by .. below `to`, one chunk of columns, AHEAD rows in flight.  (Places are below 2^31 and
// those that are looked ahead to below 2^32: 32 bits without a sign hold them.  Where they are the same for a whole wave, so are a
// row's address and the loads of its place.)
template <class T, bool SHORT, int AHEAD>
__device__ __forceinline__ void add_rows(const T *dout, int64_t ld, const int32_t *source, uint32_t n, uint32_t from, uint32_t to, uint32_t by, int column,
                                         float (&s)[Part<T, SHORT>::W]) {
    using P = Part<T, SHORT>;
    for (uint32_t q = from; q < to; q += AHEAD * by) {
        P v[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const uint32_t i = min((uint32_t)source[min(q + u * by, to - 1)], n - 1);
            v[u].load(dout + (int64_t)i * ld + column);
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (q + u * by < to)
#pragma unroll
                for (int j = 0; j < P::W; ++j) s[j] += to_f32(v[u].v[j]);
    }
}

template <int W> __device__ __forceinline__ void store_sums(float *p, const float (&s)[W], float scale) {
    constexpr int V = W < 4 ? W : 4;
#pragma unroll
    for (int j = 0; j < W; j += V) {
        Chunk<float, V> o;
#pragma unroll
        for (int k = 0; k < V; ++k) o.v[k] = scale * s[j + k];
        o.store(p + j);
    }
}

// A window's rows of entries that are longer than it: blockIdx.x a window, blockIdx.y a stripe of `chunks` chunks, of which each
// thread has one and every slices-th row.  The sum of the entry that begins inside the window is its second one, that of an
// entry that has its first place the first one.  owner: the long entry that begins in the window, at its first place or inside, or -1.
template <class T, bool SHORT>
__global__ __launch_bounds__(256) void k_embed_windows(int64_t n, int width, int entries, int64_t window, int chunks, const int32_t *__restrict__ offsets,
                                                       const int32_t *__restrict__ source, const T *__restrict__ dout, int64_t ld,
                                                       float *__restrict__ part, int32_t *__restrict__ owner) {
    using P = Part<T, SHORT>;
    constexpr int W = P::W;
    __shared__ float sums[256][W];
    const int64_t used = min(max((int64_t)offsets[entries], (int64_t)0), n), from = (int64_t)blockIdx.x * window, to = min(from + window, used);
    int begins = -1;
    const int slices = 256 / chunks, slice = threadIdx.x / chunks, lc = threadIdx.x % chunks, c = blockIdx.y * chunks + lc;
    int entry[2] = {0, 0};
    if (from < to) entries_of(offsets, entries, from, to - 1, entry[0], entry[1]);
    for (int k = 0; k < 2 && from < to; ++k) {
        const int e = entry[k];
        const int64_t start = max((int64_t)offsets[e], (int64_t)0), end = min((int64_t)offsets[e + 1], used);
        // (the first entry stands for places before its own too)
        if ((k && entry[0] == e) || end - start <= window || start >= to) continue;
        if (start >= from) begins = e;
        float s[W] = {};
        const bool in = slice < slices && c * W < width;
        if (in) add_rows<T, SHORT, 8>(dout, ld, source, (uint32_t)n, (uint32_t)max(start, from) + slice, (uint32_t)min(end, to), slices, P::start(c, width), s);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < W; ++j) sums[threadIdx.x][j] = s[j];
        __syncthreads();
        if (!in || slice != 0) continue;
        for (int i = 1; i < slices; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) s[j] += sums[i * chunks + lc][j];
        store_sums<W>(part + (2 * (int64_t)blockIdx.x + (start > from ? 1 : 0)) * width + P::start(c, width), s, 1.0f);
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) owner[blockIdx.x] = begins;
}

// The windows' sums of each long entry, in their order: 16 columns by 64 slices of the windows a block, which takes every
// gridDim-th (entry, columns) of the windows' list.
template <bool SHORT>
__global__ __launch_bounds__(256) void k_embed_join(int64_t n, int width, int entries, int64_t window, int windows, const int32_t *__restrict__ offsets,
                                                    const float *__restrict__ part, const int32_t *__restrict__ owner, float scale,
                                                    float *__restrict__ dtable) {
    using P = Part<float, SHORT>;
    constexpr int W = P::W, CHUNKS = 4, SLICES = 64, EACH = 4;
    __shared__ P sums[SLICES][CHUNKS];
    __shared__ int list[256 * EACH], counts[4];
    const int64_t used = min(max((int64_t)offsets[entries], (int64_t)0), n);
    const int stripes = (width + CHUNKS * W - 1) / (CHUNKS * W), slice = threadIdx.x / CHUNKS, lc = threadIdx.x % CHUNKS;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t seen = 0;                                // items of the windows before
    for (int base = 0; base < windows; base += 256 * EACH) {
        int mine[EACH], held = 0;
#pragma unroll
        for (int u = 0; u < EACH; ++u) {
            const int w = base + threadIdx.x * EACH + u;
            mine[u] = w < windows ? owner[w] : -1;
            held += mine[u] >= 0;
        }
        int before = held;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(before, d);
            if (lane >= d) before += v;
        }
        __syncthreads();
        if (lane == 63) counts[wave] = before;
        __syncthreads();
        before -= held;
        for (int k = 0; k < wave; ++k) before += counts[k];
        const int found = counts[0] + counts[1] + counts[2] + counts[3];
#pragma unroll
        for (int u = 0; u < EACH; ++u)
            if (mine[u] >= 0) list[before++] = mine[u];
        __syncthreads();
        const int64_t items = (int64_t)found * stripes;
        for (int64_t i = ((int64_t)blockIdx.x - seen % gridDim.x + gridDim.x) % gridDim.x; i < items; i += gridDim.x) {
            const int e = list[i / stripes], c = (int)(i % stripes) * CHUNKS + lc;
            const int64_t start = max((int64_t)offsets[e], (int64_t)0), end = min((int64_t)offsets[e + 1], used);
            P s;
#pragma unroll
            for (int j = 0; j < W; ++j) s.v[j] = 0.0f;
            const int64_t last = (end - 1) / window;
            const int column = P::start(c, width);
            if (c * W < width)
#pragma unroll 4
                for (int64_t w = start / window + slice; w <= last; w += SLICES) {
                    P v;
                    v.load(part + (2 * w + (start > w * window ? 1 : 0)) * width + column);
#pragma unroll
                    for (int j = 0; j < W; ++j) s.v[j] += v.v[j];
                }
            sums[slice][lc] = s;
            __syncthreads();
            if (threadIdx.x < CHUNKS && c * W < width) {
                for (int k = 1; k < SLICES; ++k) {
                    const P v = sums[k][lc];
#pragma unroll
                    for (int j = 0; j < W; ++j) s.v[j] += v.v[j];
                }
                store_sums<W>(dtable + (int64_t)e * width + column, s.v, scale);
            }
            __syncthreads();
        }
        seen += items;
        __syncthreads();
    }
}

// Entries of at most `window` rows (zeros for none): LANES lanes an entry, a chunk of columns each; blockIdx.y: which chunks.
template <class T, bool SHORT, int LANES>
__global__ __launch_bounds__(256) void k_embed_entries(int64_t n, int width, int entries, int64_t window, const int32_t *__restrict__ offsets,
                                                       const int32_t *__restrict__ source, const T *__restrict__ dout, int64_t ld, float scale,
                                                       float *__restrict__ dtable) {
    using P = Part<T, SHORT>;
    constexpr int W = P::W;
    int64_t e = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    if (LANES == 64) e = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);       // known to be the wave's
    if (e >= entries) return;
    const int used = (int)min(max((int64_t)offsets[entries], (int64_t)0), n);
    const int start = max(offsets[e], 0), end = min(offsets[e + 1], used);
    if (end - (int64_t)start > window) return;
    const int c = blockIdx.y * LANES + threadIdx.x % LANES;
    if (c * W >= width) return;
    float s[W] = {};
    const int many = end - start, column = P::start(c, width);
    if (many > 6) add_rows<T, SHORT, 16>(dout, ld, source, (uint32_t)n, start, end, 1, column, s);
    else if (many > 2) add_rows<T, SHORT, 6>(dout, ld, source, (uint32_t)n, start, end, 1, column, s);
    else if (many > 0) add_rows<T, SHORT, 2>(dout, ld, source, (uint32_t)n, start, end, 1, column, s);
    store_sums<W>(dtable + e * width + column, s, scale);
}

template <class T, bool SHORT>
Status embed_t(Context &cx, int64_t n, int width, int entries, const int32_t *index, const T *table, float scale, T *out) {
    const int per = parts_of<T>(width);
    return by_launches(n, kLaunchBlocks * items_of(n, per).rows, [&](int64_t from, int64_t rows) -> Status {
        const Items it = items_of(rows, per);
        k_embed<T, SHORT><<<grid_of(it), 256, 0, cx.stream>>>(it, width, entries, index + from, table, scale, out + from * width);
        MPNN_HIP(hipGetLastError());
        return Status::ok();
    });
}

template <class T, bool SHORT>
Status embed_backward_t(Context &cx, int64_t n, int width, int entries, const T *dout, int64_t ld, const int32_t *offsets, const int32_t *source,
                        float scale, float *dtable) {
    const int per = parts_of<T>(width);
    // 64 rows: what a few lanes add up in a row's time or two; more where the windows would be many to look through
    const int64_t window = std::max<int64_t>(64, (n + 16383) / 16384), windows = n > window ? (n + window - 1) / window : 0;
    if (windows) {
        void *ws = nullptr;
        const size_t sums = sizeof(float) * (size_t)(2 * windows * width);
        MPNN_TRY(cx.rows_scratch(sums + sizeof(int32_t) * (size_t)windows, &ws));
        float *const part = static_cast<float *>(ws);
        int32_t *const owner = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + sums);
        // stripes of up to 32 chunks: eight slices and more of a window's rows in flight
        const int stripes = (per + 31) / 32, chunks = (per + stripes - 1) / stripes;
        k_embed_windows<T, SHORT><<<dim3((unsigned)windows, stripes), 256, 0, cx.stream>>>(n, width, entries, window, chunks, offsets, source, dout, ld,
                                                                                       part, owner);
        MPNN_HIP(hipGetLastError());
        auto *join = width < 4 ? k_embed_join<true> : k_embed_join<false>;
        join<<<2048, 256, 0, cx.stream>>>(n, width, entries, window, (int)windows, offsets, part, owner, scale, dtable);
        MPNN_HIP(hipGetLastError());
    }
    const auto run = [&](auto lanes) -> Status {
        constexpr int L = lanes();
        k_embed_entries<T, SHORT, L><<<dim3((unsigned)((entries + 256 / L - 1) / (256 / L)), (per + L - 1) / L), 256, 0, cx.stream>>>(
            n, width, entries, window, offsets, source, dout, ld, scale, dtable);
        MPNN_HIP(hipGetLastError());
        return Status::ok();
    };
    if (per <= 4) return run(std::integral_constant<int, 4>{});
    if (per <= 16) return run(std::integral_constant<int, 16>{});
    return run(std::integral_constant<int, 64>{});
}

template <class T> bool is_short(int width) { return width < Chunk<T>::W; }

}  // namespace

Status embed(Context &cx, int dtype, int64_t n, int width, int entries, const int32_t *index, const void *table, float scale, void *out) {
    if (n == 0) return Status::ok();
    const auto run = [&](auto one) -> Status {
        using T = decltype(one);
        return is_short<T>(width) ? embed_t<T, true>(cx, n, width, entries, index, (const T *)table, scale, (T *)out)
                                  : embed_t<T, false>(cx, n, width, entries, index, (const T *)table, scale, (T *)out);
    };
    return dtype == MPNN_BF16 ? run(bf16{}) : run(float{});
}

Status embed_backward(Context &cx, int dtype, int64_t n, int width, int entries, const void *dout, int64_t ld, const int32_t *offsets,
                      const int32_t *source, float scale, float *dtable) {
    const auto run = [&](auto one) -> Status {
        using T = decltype(one);
        return is_short<T>(width) ? embed_backward_t<T, true>(cx, n, width, entries, (const T *)dout, ld, offsets, source, scale, dtable)
                                  : embed_backward_t<T, false>(cx, n, width, entries, (const T *)dout, ld, offsets, source, scale, dtable);
    };
    return dtype == MPNN_BF16 ? run(bf16{}) : run(float{});
}

}  // namespace mpnn
