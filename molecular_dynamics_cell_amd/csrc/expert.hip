// Rows sorted by expert times their experts' weights (mpnn_expert_product), the gradient towards the rows
// (mpnn_expert_input_grad) and the product with weights held in 4 bits (mpnn_micro_product):
//   y[q] = act(W_e x[q] + b_e),  dx[q] = W_e^T dy[q]  for the rows q of expert e.
#include <algorithm>
#include <type_traits>

#include "impl.h"
#include "rows.h"
#include "tiles.h"

namespace mpnn {

namespace {

struct Args {
    int64_t n, first;               // rows; the launch's first block
    int reduced, columns;           // length of the products' sums; columns of the result
    int n_experts, tiles_c;
    const int32_t *offsets;
    const int32_t *source;          // row q of x is source[q] / slots of n_x (null: q)
    int64_t n_x;
    int slots;
    const float *bias;
    int act;
    void *y;
    int y_bf16;
};

__device__ __forceinline__ float silu(float z) { return z / (1.0f + expf(-z)); }

template <class T> __device__ __forceinline__ void store_four(T *p, const float (&v)[4], int in) {
    Chunk<T, 4> o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o.v[j] = from_f32<T>(v[j]);
    o.store(p, in);
}

// Tiles of 32 MT WM columns by 32 NT WN rows.  ACROSS: the weights' rows are the reduced axis (dx).
template <class X, class W, bool ACROSS, int MT, int NT, int WM, int WN>
__global__ __launch_bounds__(256, 2) void k_product(const Args a, const RowsOf<X> x, const RowsOf<W> w) {
    constexpr int TP = kTerms<W>, TQ = kTerms<X>, WORDS = TP * TQ > 3 ? 4 : 8;
    constexpr int BC = 32 * MT * WM, BR = 32 * NT * WN;
    using P = std::conditional_t<ACROSS, Across<TP, BC, WORDS>, Along<TP, BC, WORDS>>;
    using Q = Along<TQ, BR, WORDS>;
    __shared__ uint4 lds[P::kWords + Q::kWords];
    uint4 *const lp = lds, *const lq = lds + P::kWords;

    const int64_t number = a.first + xcd_block();
    const Tile tile = find_tile(a.offsets, a.n_experts, a.n, BR, number / a.tiles_c);
    if (tile.from >= tile.to) return;
    const int c0 = (int)(number % a.tiles_c) * BC;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave / WN, wn = wave % WN;

    const auto place = [&](int64_t q) -> int64_t {
        if (!a.source) return q;
        return min((int64_t)((uint32_t)max(a.source[q], 0) / (uint32_t)a.slots), a.n_x - 1);
    };
    floatx16 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = (floatx16)(0.0f);
    float largest = 0.0f;
    if (tile.expert >= 0) {
        constexpr int XQ = BR * WORDS / 256, XP = BC * WORDS / 256;
        typename RowsOf<X>::Row xr[XQ];
        typename RowsOf<W>::Row wr[ACROSS ? 1 : XP];
        const int word = tid % WORDS, row = tid / WORDS;
        constexpr int STEP = 256 / WORDS;
#pragma unroll
        for (int i = 0; i < XQ; ++i) xr[i] = x.row(place(min(tile.from + row + i * STEP, tile.to - 1)));
        const int64_t w0 = (int64_t)tile.expert * (ACROSS ? a.reduced : a.columns);
        if constexpr (!ACROSS)
#pragma unroll
            for (int i = 0; i < XP; ++i) wr[i] = w.row(w0 + min(c0 + row + i * STEP, a.columns - 1));
        constexpr int WIDE = BC / 8, AT_ONCE = 256 / WIDE;      // words of a weight row, weight rows at once

        Word<X> xv[XQ];
        Word<W> wv[XP];
        auto fetch = [&](int k0) {
#pragma unroll
            for (int i = 0; i < XQ; ++i) RowsOf<X>::load(xv[i], xr[i], k0 + word * 8, a.reduced);
#pragma unroll
            for (int i = 0; i < XP; ++i) {
                if constexpr (ACROSS) {
                    const int k = k0 + tid / WIDE + i * AT_ONCE;
                    if (k < a.reduced) RowsOf<W>::load(wv[i], w.row(w0 + k), c0 + tid % WIDE * 8, a.columns);
                    else wv[i].clear();
                } else {
                    RowsOf<W>::load(wv[i], wr[i], k0 + word * 8, a.reduced);
                }
            }
        };
        fetch(0);
        for (int k0 = 0; k0 < a.reduced; k0 += 8 * WORDS) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < XQ; ++i) {
                uint4 t[TQ];
                xv[i].terms(t, largest);
                Q::store(lq, row + i * STEP, word, t);
            }
#pragma unroll
            for (int i = 0; i < XP; ++i) {
                uint4 t[TP];
                wv[i].terms(t, largest);
                if constexpr (ACROSS) P::store(lp, tid / WIDE + i * AT_ONCE, tid % WIDE, t);
                else P::store(lp, row + i * STEP, word, t);
            }
            __syncthreads();
            if (k0 + 8 * WORDS < a.reduced) fetch(k0 + 8 * WORDS);
            multiply<P, Q, TP, TQ, MT, NT, WORDS>(lp, lq, wm * MT * 32, wn * NT * 32, lane, acc);
        }
    }
    const bool huge = TP + TQ > 2 && __syncthreads_or(largest >= kHuge);

    // a lane has four neighbouring columns of a row in four registers
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t q = tile.from + (wn * NT + j) * 32 + (lane & 31);
        if (q >= tile.to) continue;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = c0 + (wm * MT + i) * 32 + 8 * g + 4 * (lane >> 5), in = a.columns - c;
                if (in <= 0) continue;
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = acc[i][j][4 * g + r];
                if (tile.expert >= 0) {
                    if (huge)
                        for (int r = 0; r < 4; ++r)
                            if (v[r] != v[r] && r < in) {
                                const int64_t w0 = (int64_t)tile.expert * (ACROSS ? a.reduced : a.columns), from = place(q);
                                float s = 0.0f;
                                for (int k = 0; k < a.reduced; ++k) s = fmaf(x.at(from, k), ACROSS ? w.at(w0 + k, c + r) : w.at(w0 + c + r, k), s);
                                v[r] = s;
                            }
                    if (a.bias)
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] += r < in ? a.bias[(int64_t)tile.expert * a.columns + c + r] : 0.0f;
                    if (a.act == MPNN_ACT_SILU)
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = silu(v[r]);
                }
                if (a.y_bf16) store_four(static_cast<bf16 *>(a.y) + q * a.columns + c, v, in);
                else store_four(static_cast<float *>(a.y) + q * a.columns + c, v, in);
            }
    }
}

template <class X, class W, bool ACROSS>
Status product_t(Context &cx, Args a, const RowsOf<X> &x, const RowsOf<W> &w) {
    constexpr int BC = 128, BR = 128;
    a.tiles_c = (a.columns + BC - 1) / BC;
    const int64_t blocks = row_tiles(a.n, a.n_experts, BR) * a.tiles_c;
    return by_launches(blocks, kLaunchBlocks, [&](int64_t from, int64_t count) -> Status {
        a.first = from;
        k_product<X, W, ACROSS, 2, 2, 2, 2><<<grid_xcd(count, 1), 256, 0, cx.stream>>>(a, x, w);
        MPNN_HIP(hipGetLastError());
        return Status::ok();
    });
}

}  // namespace

Status expert_product(Context &cx, int dtype, int64_t n, int width, int n_out, int n_experts, const int32_t *offsets, const void *x,
                      int64_t ldx, const int32_t *source, int64_t n_x, const void *weight, const float *bias, int act, void *y) {
    if (n == 0) return Status::ok();
    const Args a{n, 0, width, n_out, n_experts, 0, offsets, source, source ? n_x : n, source ? (int)(n / n_x) : 1, bias, act, y, dtype == MPNN_BF16};
    if (dtype == MPNN_BF16) return product_t<bf16, bf16, false>(cx, a, {(const bf16 *)x, ldx}, {(const bf16 *)weight, width});
    return product_t<float, float, false>(cx, a, {(const float *)x, ldx}, {(const float *)weight, width});
}

Status expert_input_grad(Context &cx, int dtype, int64_t n, int width, int n_out, int n_experts, const int32_t *offsets, const void *dy,
                         int64_t ld, const void *weight, void *dx) {
    if (n == 0) return Status::ok();
    const Args a{n, 0, n_out, width, n_experts, 0, offsets, nullptr, n, 1, nullptr, MPNN_ACT_NONE, dx, dtype == MPNN_BF16};
    if (dtype == MPNN_BF16) return product_t<bf16, bf16, true>(cx, a, {(const bf16 *)dy, ld}, {(const bf16 *)weight, width});
    return product_t<float, float, true>(cx, a, {(const float *)dy, ld}, {(const float *)weight, width});
}

Status micro_product(Context &cx, int x_dtype, int y_dtype, int64_t n, int width, int n_out, int n_experts, const int32_t *offsets,
                     const void *x, int64_t ldx, const uint8_t *x_scales, const int32_t *source, int64_t n_x, const uint8_t *codes,
                     const uint8_t *scales, const float *bias, int act, void *y) {
    if (n == 0) return Status::ok();
    const int64_t groups = (width + kMicroGroup - 1) / kMicroGroup;
    const Args a{n, 0, width, n_out, n_experts, 0, offsets, source, source ? n_x : n, source ? (int)(n / n_x) : 1, bias, act, y, y_dtype == MPNN_BF16};
    const RowsOf<Micro> w{codes, scales, groups};
    if (x_dtype == MPNN_MICRO) return product_t<Micro, Micro, false>(cx, a, {(const uint8_t *)x, x_scales, groups}, w);
    if (x_dtype == MPNN_BF16) return product_t<bf16, Micro, false>(cx, a, {(const bf16 *)x, ldx}, w);
    return product_t<float, Micro, false>(cx, a, {(const float *)x, ldx}, w);
}

}  // namespace mpnn
