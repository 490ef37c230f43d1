// Device helpers of the row operators (routing.hip, residual.hip, checkpoint.hip, weight_grad.hip).
#pragma once

#include <algorithm>

#include "impl.h"

namespace mpnn {

using bf16 = __bf16;

// Values are read to and computed in fp32 and rounded once, to nearest even, when stored.
template <class T> __device__ __forceinline__ float to_f32(T v) { return (float)v; }
template <class T> __device__ __forceinline__ T from_f32(float v) { return (T)v; }

// W values of a row, 16 bytes of it unless said otherwise.  Rows may start on any value's boundary (odd widths, column
// blocks of wider rows): the access is declared with the value's alignment, and gfx950's global loads and stores take it
// in one instruction all the same.
template <class T, int WIDE = 16 / sizeof(T)>
struct Chunk {
    static constexpr int W = WIDE;
    T v[W];
    __device__ __forceinline__ void load(const T *p) { __builtin_memcpy(this, p, sizeof *this); }
    __device__ __forceinline__ void store(T *p) const { __builtin_memcpy(p, this, sizeof *this); }
    // the first `in` values (all of them from W on), zeros after them
    __device__ __forceinline__ void load(const T *p, int in) {
        if (in >= W) return load(p);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = j < in ? p[j] : from_f32<T>(0.0f);
    }
    __device__ __forceinline__ void store(T *p, int in) const {
        if (in >= W) return store(p);
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (j < in) p[j] = v[j];
    }
};

// Sum over G = 4 .. 64 neighbouring lanes, the same bits in each of them: exchanges inside 16 lanes by data-parallel
// primitives (neighbours, pairs, mirrored halves), across them by the lane swaps.
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int G> __device__ __forceinline__ float lanes_sum(float v) {
    v += dpp<0xb1>(v);                       // quad_perm 1 0 3 2
    v += dpp<0x4e>(v);                       // quad_perm 2 3 0 1
    if (G >= 8) v += dpp<0x141>(v);          // row_half_mirror
    if (G >= 16) v += dpp<0x140>(v);         // row_mirror
    if (G >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if (G >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    return v;
}

__device__ __forceinline__ float wave_sum(float v) { return lanes_sum<64>(v); }

// Items of a row operator without sums along the rows: `per` chunks a row.  A block takes `rows` whole rows, or, of
// rows longer than its `items`, one stretch (blockIdx.y); a thread takes every 256th item, `unroll` of them (one in
// small calls, which are spread over more blocks), whose loads are in flight together.  Consecutive stretches of rows
// go to one XCD, so that lines shared by neighbouring rows are completed in its L2.
constexpr int kUnroll = 4;
struct Items {
    int64_t n;
    int per, rows, items;
    float inv;      // 1 / per
};
inline Items items_of(int64_t n, int per, int unroll = kUnroll) {
    const int items = n * per > 256 * 2048 ? 256 * unroll : 256;
    const int rows = per < items ? items / per : 1;
    return Items{n, per, rows, items, 1.0f / (float)per};
}
// A launch counts its threads in 32 bits, and one of more leaves rows out without an error: rows past `most`, those of
// the most blocks of 256 threads that a launch holds, go into further launches.
constexpr int64_t kLaunchBlocks = (int64_t(1) << 24) - kXcds;
template <class F> Status by_launches(int64_t n, int64_t most, F run) {
    for (int64_t from = 0; from < n; from += most) MPNN_TRY(run(from, std::min(n - from, most)));
    return Status::ok();
}
inline dim3 grid_of(const Items &it) { return dim3(grid_xcd(it.n, it.rows), (unsigned)((it.per + it.items - 1) / it.items)); }

// This thread's u-th item: its row and chunk.  Threads past the block's last item, and blocks past the last row, repeat
// a last one (of the same place in a group of L chunks), so that no load or store has a condition: what they write is
// what its owner writes.
template <int L = 1> __device__ __forceinline__ void item_at(const Items &it, int64_t block, int u, int64_t &row, int &c) {
    int l = u * 256 + threadIdx.x;
    if (it.rows == 1) {
        row = min(block, it.n - 1);
        c = blockIdx.y * it.items + (l < it.items ? l : it.items - L + l % L);
        if (c >= it.per) c = it.per - L + l % L;
        return;
    }
    const int last = it.rows * it.per;
    if (l >= last) l = last - L + l % L;
    int q = (int)((float)l * it.inv);      // off by one at most
    q -= q * it.per > l;
    q += (q + 1) * it.per <= l;
    row = min(block * it.rows + q, it.n - 1);
    c = l - q * it.per;
}

}  // namespace mpnn
