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

constexpr int kCus = 256;

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

// z / (1 + exp(-z)) = z r for z >= 0, z a r below, a = exp(-|z|) <= 1, r = 1 / (1 + a): exp by the hardware's power of two with
// the rounding of its argument put back, the reciprocal of 1 .. 2 with one Newton step.  Beyond |z| = 128 a is zero.
__device__ __forceinline__ float silu(float z) {
    constexpr float kLog2e = 1.44269504f, kRest = 1.92596299e-8f, kLn2 = 0.693147181f;      // log2 e in two parts
    const float m = fminf(fabsf(z), 128.0f), t = -m * kLog2e, rest = fmaf(-m, kLog2e, -t) - m * kRest;
    const float e = __builtin_amdgcn_exp2f(t), a = fmaf(e, rest * kLn2, e);
    const float b = 1.0f + a, r0 = __builtin_amdgcn_rcpf(b), r = fmaf(r0, fmaf(-b, r0, 1.0f), r0);
    return z >= 0.0f ? z * r : z * a * r;
}

template <class T> __device__ __forceinline__ void store_four(T *p, const float (&v)[4], int in) {
    Chunk<T, 4> o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o.v[j] = from_f32<T>(v[j]);
    o.store(p, in);
}

// Bias, activation and the store of four neighbouring results (`in` of them are the row's) of row q; expert < 0: none.
__device__ __forceinline__ void finish(const Args &a, int expert, int64_t q, int c, int in, float (&v)[4]) {
    if (expert >= 0) {
        if (a.bias)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] += r < in ? a.bias[(int64_t)expert * a.columns + c + r] : 0.0f;
        if (a.act == MPNN_ACT_SILU)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = silu(v[r]);
    }
    if (a.y_bf16) store_four(static_cast<bf16 *>(a.y) + q * a.columns + c, v, in);
    else store_four(static_cast<float *>(a.y) + q * a.columns + c, v, in);
}

// 128 x 128 results at a time, four waves of 64 x 64, any types, strides and alignments: words go through registers, where
// fp32 is cut into terms and 4-bit codes become bf16.  A block stays for many tiles: the next one's first words are on
// their way while this one's results are stored.  ACROSS: the weights' rows are the reduced axis (dx).
// Two blocks a CU take turns at cutting and multiplying: fp32 128,000 rows 312 -> 128 x 5 with SiLU 78-92 us (47 at a large bf16
// product's rate), dx 95-117 us.  No unit bounds it: of a CU's cycles the matrix cores are busy 39 %, vector issue 49 %, LDS 22 %; of
// its waves' 39 % go by waiting for an issue slot and 24 % for memory or a barrier, so the turns do not fill each other's gaps.
// 32,768 rows 1024 -> 1024 x 8 fp32 355 us, 1.16 PFLOP/s of bf16 products; bf16 312 -> 128 30 us and dx 38 us.
constexpr int kTile = 128;
template <class X, class W, bool ACROSS>
__global__ __launch_bounds__(256, 2) void k_product(const Args a, const RowsOf<X> x, const RowsOf<W> w) {
    constexpr int TP = kTerms<W>, TQ = kTerms<X>, WORDS = TP * TQ > 1 ? 4 : 8, STAGE = 8 * WORDS, MT = 2, NT = 2;
    using P = std::conditional_t<ACROSS, Across<TP, kTile, WORDS>, Along<TP, kTile, WORDS>>;
    using Q = Along<TQ, kTile, WORDS>;
    __shared__ uint4 lds[P::kWords + Q::kWords];
    __shared__ uint4 results[4][kStoreBytes / 16];
    __shared__ Segments table;
    uint4 *const lp = lds, *const lq = lds + P::kWords;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave >> 1, wn = wave & 1;
    if (wave == 0) table.fill(a.offsets, a.n_experts, a.n, kTile);
    __syncthreads();
    const int64_t tiles = table.tiles(a.n_experts) * a.tiles_c;
    const auto place = [&](int64_t q) -> int64_t {
        if (!a.source) return q;
        return min((int64_t)((uint32_t)max(a.source[q], 0) / (uint32_t)a.slots), a.n_x - 1);
    };

    // The tile whose words are being loaded.
    constexpr int EACH = kTile * WORDS / 256, STEP = 256 / WORDS, WIDE = kTile / 8, AT_ONCE = 256 / WIDE;   // (of weight rows across: words, rows at once)
    const int word = tid % WORDS, row = tid / WORDS;
    Tile tile;
    int c0 = 0, at_column = 0;
    bool columns_whole = true, over = false;
    int64_t w0 = 0;
    typename RowsOf<X>::Row xr[EACH];
    typename RowsOf<W>::Row wr[ACROSS ? 1 : EACH];
    Word<X> xv[EACH];
    Word<W> wv[EACH];
    // A stage of whole words has no conditions beside its loads; nor has another one where eight rows follow the tile's rows and
    // the expert's weights (`over`), so that words may be loaded past a row's end (128,000 rows 311 -> 127 x 5 in bf16 42 us; with
    // 312 -> 128 30 us). bf16 across does without: its words would leave the registers (195 us in place of 52).
    constexpr bool kOver = !ACROSS || sizeof(X) == 4;
    const auto fetch = [&](int k0) {
        const int k = k0 + word * 8;
        const bool whole = columns_whole && k0 + STAGE <= a.reduced;
        if (whole) {
#pragma unroll
            for (int i = 0; i < EACH; ++i) RowsOf<X>::load(xv[i], xr[i], k);
        } else if (kOver && over) {
#pragma unroll
            for (int i = 0; i < EACH; ++i) RowsOf<X>::load_over(xv[i], xr[i], k, a.reduced);
        } else {
#pragma unroll
            for (int i = 0; i < EACH; ++i) RowsOf<X>::load(xv[i], xr[i], k, a.reduced);
        }
        const auto across = [&](int i) { return k0 + tid / WIDE + i * AT_ONCE; };
        if (whole) {
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                if constexpr (ACROSS) RowsOf<W>::load(wv[i], w.row(w0 + across(i)), at_column);
                else RowsOf<W>::load(wv[i], wr[i], k);
            }
        } else if (kOver && over) {
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                if constexpr (ACROSS) RowsOf<W>::load_over(wv[i], w.row(w0 + min(across(i), a.reduced - 1)), at_column, a.columns, across(i) < a.reduced);
                else RowsOf<W>::load_over(wv[i], wr[i], k, a.reduced);
            }
        } else {
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                if constexpr (ACROSS) RowsOf<W>::load(wv[i], w.row(w0 + min(across(i), a.reduced - 1)), at_column, across(i) < a.reduced ? a.columns : 0);
                else RowsOf<W>::load(wv[i], wr[i], k, a.reduced);
            }
        }
    };
    const auto begin = [&](int64_t number) {
        tile = table.find(a.offsets, a.n_experts, a.n, kTile, (int)(number / a.tiles_c));
        c0 = (int)(number % a.tiles_c) * kTile;
        // Across in bf16 the last tile ends with the row (its first columns are then the one's before too, the same bits), so that
        // no word of weights is cut: 361 rows 2639 -> 2910 59 us in place of 158, 128,000 rows 127 -> 311 x 5 52 in place of 66
        // (fp32, whose words go past their row's end, gains nothing).
        if (!kOver) c0 = min(c0, max(a.columns - kTile, 0));
        if (tile.expert < 0) return;
        w0 = (int64_t)tile.expert * (ACROSS ? a.reduced : a.columns);
        over = w0 + (ACROSS ? a.reduced : a.columns) + 8 <= (int64_t)a.n_experts * (ACROSS ? a.reduced : a.columns);
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int64_t at = place(min(tile.from + row + i * STEP, tile.to - 1));
            xr[i] = x.row(at);
            over = over && at + 8 < a.n_x;
        }
        over = __all(over);
        if constexpr (ACROSS) {
            columns_whole = c0 + kTile <= a.columns || a.columns % 8 == 0;
            at_column = c0 + tid % WIDE * 8;
            if (columns_whole) at_column = min(at_column, a.columns - 8);
        } else {
#pragma unroll
            for (int i = 0; i < EACH; ++i) wr[i] = w.row(w0 + min(c0 + row + i * STEP, a.columns - 1));
        }
        fetch(0);
    };

    int64_t number = tile_in_round(0, blockIdx.x, tiles);
    if (number < 0) return;
    begin(number);
    for (int64_t round = 1;; ++round) {
        floatx16 acc[MT][NT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = (floatx16)(0.0f);
        float largest = 0.0f;
        for (int k0 = 0; k0 < a.reduced && tile.expert >= 0; k0 += STAGE) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                uint4 t[TQ];
                xv[i].terms(t, largest);
                Q::store(lq, row + i * STEP, word, t);
            }
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                uint4 t[TP];
                wv[i].terms(t, largest);
                if constexpr (ACROSS) P::store(lp, tid / WIDE + i * AT_ONCE, tid % WIDE, t);
                else P::store(lp, row + i * STEP, word, t);
            }
            __syncthreads();
            if (k0 + STAGE < a.reduced) fetch(k0 + STAGE);
            multiply<P, Q, TP, TQ, MT, NT, WORDS>(lp, lq, wm * MT * 32, wn * NT * 32, lane, acc);
        }
        const bool large = TP + TQ > 2 && __syncthreads_or(largest >= kLarge);

        // the next tile, before this one's results
        const Tile done = tile;
        const int done_c0 = c0;
        number = tile_in_round(round, blockIdx.x, tiles);
        const bool again = number >= 0;
        if (again) begin(number);

        const bool act = a.act == MPNN_ACT_SILU, biased = a.bias && done.expert >= 0;      // silu(0) = 0: rows of no expert may take it too
        const auto out = [&](auto *y) {
            const auto bias = [&](int c) {
                Chunk<float, 4> b = {{0.0f, 0.0f, 0.0f, 0.0f}};
                if (biased) b.load(a.bias + (int64_t)done.expert * a.columns + c, a.columns - c);
                return b;
            };
            store_lines(reinterpret_cast<char *>(results[wave]), acc, lane, y, a.columns, done.from + wn * NT * 32, done.to, done_c0 + wm * MT * 32,
                        a.columns, bias, [&](float v) { return act ? silu(v) : v; });
            if (!large) return;
            // (sums that are all finite are right: 128,000 rows of values near 1e15 take no longer than of 1, and 141 us in place of 83
            // where results are looked through for it)
            float zero = 0.0f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) zero = fmaf(acc[i][j][r], 0.0f, zero);
            if (!__syncthreads_or(zero != 0.0f)) return;
            // results that are not finite, once more without terms
            __syncthreads();
            for (int e = tid; e < kTile * kTile; e += 256) {
                const int64_t q = done.from + e / kTile;
                const int c = done_c0 + e % kTile;
                if (q >= done.to || c >= a.columns) continue;
                if (isfinite(to_f32(y[q * a.columns + c]))) continue;
                const int64_t weights = (int64_t)done.expert * (ACROSS ? a.reduced : a.columns), from = place(q);
                float s = 0.0f;
                for (int k = 0; k < a.reduced && s == s; ++k) s = fmaf(x.at(from, k), ACROSS ? w.at(weights + k, c) : w.at(weights + c, k), s);
                if (biased) s += a.bias[(int64_t)done.expert * a.columns + c];
                y[q * a.columns + c] = from_f32<std::remove_pointer_t<decltype(y)>>(act ? silu(s) : s);
            }
        };
        if (a.y_bf16) out(static_cast<bf16 *>(a.y));
        else out(static_cast<float *>(a.y));
        if (!again) break;
    }
}

// ---- wide tiles ----
// The product of two 16-byte words that a lane of 32 rows has: 16 steps of bf16, or a group of 32 columns in 4 bits with its
// scales (byte S of each lane's word of scales).
typedef int intx8 __attribute__((ext_vector_type(8)));
template <class T> struct WideOp;
template <> struct WideOp<bf16> {
    static constexpr int kPerWord = 8;
    template <int S> __device__ __forceinline__ static floatx16 multiply(uint4 p, uint4 q, floatx16 c, uint32_t, uint32_t) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), c, 0, 0, 0);
    }
    __device__ __forceinline__ static const char *bytes(const RowsOf<bf16>::Row &r) { return reinterpret_cast<const char *>(r.p); }
};
template <> struct WideOp<Micro> {
    static constexpr int kPerWord = 32;
    template <int S> __device__ __forceinline__ static floatx16 multiply(uint4 p, uint4 q, floatx16 c, uint32_t ps, uint32_t qs) {
        const intx8 a = {(int)p.x, (int)p.y, (int)p.z, (int)p.w, 0, 0, 0, 0}, b = {(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, S, ps, S, qs);
    }
    __device__ __forceinline__ static const char *bytes(const RowsOf<Micro>::Row &r) { return reinterpret_cast<const char *>(r.codes); }
};

// 256 x 256 results at a time, eight waves of 128 columns x 64 rows.  Stages are 64 bytes of every row; they go to LDS without
// passing through registers, two stages ahead.  A block stays for many tiles: the next one's first stages are on their way
// while this one's results are stored.  (One block a CU: without that a tile of 2,048 columns takes 29 us of products and
// 23 us to find its rows, wait for the first of them and store its results.)
// 65,536 rows 2048 -> 1024 x 64 bf16 260-318 us with equal shares (up to 1.06 PFLOP/s) and 321-372 with a router's, whose tiles are not
// all full; 16,384 rows 2048 -> 4096 x 8 in 4 bits 149 us (1.84 PFLOP/s), of which SiLU at the ends of tiles is 24-32 and uneven shares
// 15-24; dx of 32,768 rows 1024 -> 1024 x 8 68-78 us.  No unit bounds it: of a CU's cycles the matrix cores are busy 45 % (in 4 bits
// 26 %), vector issue 28 % (50 %), LDS 21 % (18 %), and 39 % (33 %) of the waves' go by waiting for loads and barriers; the clock is
// 2.0 GHz meanwhile.  (The bf16 products alone, of random data from registers, run at 1.75 PFLOP/s, of zeros at 2.47.)
constexpr int kWide = 256, kWideWords = 4, kBuffers = 3, kWideThreads = 512;
using WideTile = Along<1, kWide, kWideWords>;

// ACROSS (bf16): the weights' rows are the reduced axis; a stage is 32 of them, 512 bytes each.
template <class T, bool ACROSS>
__global__ __launch_bounds__(kWideThreads, 2) void k_product_wide(const Args a, const RowsOf<T> x, const RowsOf<T> w) {
    using Op = WideOp<T>;
    constexpr bool MICRO = std::is_same<T, Micro>::value;
    constexpr int STAGE = kWideWords * Op::kPerWord;                   // columns of a stage
    constexpr int SIDE = WideTile::kWords, BOTH = SIDE + (ACROSS ? Pairs::kWords : SIDE);     // words of a stage: rows, then weights
    constexpr int MT = 4, NT = 2;
    __shared__ uint4 lds[kBuffers * BOTH];
    __shared__ uint32_t scales[MICRO ? kBuffers : 1][2][MICRO ? kWide : 1];
    __shared__ uint4 results[kWideThreads / 64][kStoreBytes / 16];
    __shared__ Segments table;
    typedef const __attribute__((address_space(1))) void *Global;
    typedef __attribute__((address_space(3))) void *Local;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave & 1, wn = wave >> 1;

    [[maybe_unused]] const Pairs pairs(lane);
    if (wave == 0) table.fill(a.offsets, a.n_experts, a.n, kWide);
    __syncthreads();
    const int64_t tiles = table.tiles(a.n_experts) * a.tiles_c;

    const auto place = [&](int64_t q) -> int64_t {
        if (!a.source) return q;
        return min((int64_t)((uint32_t)max(a.source[q], 0) / (uint32_t)a.slots), a.n_x - 1);
    };
    const int words = (a.reduced + Op::kPerWord - 1) / Op::kPerWord;
    const int full = MICRO ? words / kWideWords : a.reduced / STAGE, stages = (words + kWideWords - 1) / kWideWords;

    // The tile that is being brought, multiplied and stored.
    int expert = 0, c0 = 0;
    int64_t from = 0, to = 0;
    const char *px[2], *pw[2];
    const uint8_t *ps_row = nullptr;
    uint32_t next_scales = 0;
    int at = 0;                                    // buffer of the tile's first stage
    const auto w_row = [&](int r) { return w.row(ACROSS ? (int64_t)expert * a.reduced + r : (int64_t)expert * a.columns + min(c0 + r, a.columns - 1)); };
    const auto x_row = [&](int r) { return x.row(place(min(from + r, to - 1))); };
    const auto buffer_of = [&](int s) { return s % kBuffers; };
    // A wave brings 32 rows of each side, 16 at once; lane l the word that stands at place l of those rows in LDS.
    const auto bring = [&](int buffer, int i) {
        const int of = wave * 2 + i;
        __builtin_amdgcn_global_load_lds((Global)px[i], (Local)&lds[buffer * BOTH + of * 64], 16, 0, 0);
        __builtin_amdgcn_global_load_lds((Global)pw[i], (Local)&lds[buffer * BOTH + SIDE + of * (ACROSS ? Pairs::kPair : 64)], 16, 0, 0);
        px[i] += 64;
        pw[i] += ACROSS ? a.columns * (int64_t)64 : 64;       // bytes of 32 rows of weights
    };
    // Scales: a thread brings the four of a stage of one row, by way of a register (rows of scales start on any byte).  Past
    // a row's last group they are those of 1, since its codes are zeros there.
    const auto fetch_scales = [&](int stage) {
        stage = min(stage, stages - 1);
        const int left = words - stage * kWideWords;
        const uint8_t *p = ps_row + stage * kWideWords;
        uint32_t v = 0;
        if (left >= kWideWords) __builtin_memcpy(&v, p, 4);
        else
#pragma unroll
            for (int k = 0; k < 4; ++k) v |= (k < left ? (uint32_t)p[k] : 127u) << 8 * k;
        next_scales = v;
    };
    const auto store_scales = [&](int buffer) { scales[buffer][threadIdx.x >> 8][threadIdx.x & 255] = next_scales; };
    const auto begin = [&](int64_t number) {
        const Tile tile = table.find(a.offsets, a.n_experts, a.n, kWide, (int)(number / a.tiles_c));
        expert = tile.expert;
        from = tile.from;
        to = tile.to;
        c0 = (int)(number % a.tiles_c) * kWide;
        if (expert < 0) return;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = wave * 32 + i * 16 + lane / 4, word = (lane & 3) ^ (r >> 2 & 3);
            px[i] = Op::bytes(x_row(r)) + word * 16;
            if constexpr (ACROSS) {
                // words past the last column bring the last one again
                const int k = (wave * 2 + i) * 2 + Pairs::step_of(lane), at_column = c0 + 8 * Pairs::word_of(lane);
                pw[i] = Op::bytes(w_row(min(k, a.reduced - 1))) + 2 * min(at_column, a.columns - 8);
            } else {
                pw[i] = Op::bytes(w_row(r)) + word * 16;
            }
        }
        if constexpr (MICRO) {
            ps_row = wave < 4 ? x_row(threadIdx.x).scales : w_row(threadIdx.x - 256).scales;
            fetch_scales(0);
            store_scales(at);
            fetch_scales(1);
        }
        for (int s = 0; s < min(full, kBuffers - 1); ++s) {
            bring(buffer_of(at + s), 0);
            bring(buffer_of(at + s), 1);
        }
    };

    int64_t number = tile_in_round(0, blockIdx.x, tiles);
    if (number < 0) return;
    begin(number);
    for (int64_t round = 1;; ++round) {
        floatx16 acc[MT][NT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = (floatx16)(0.0f);
        // Waves whose rows are past the tile's last one bring their share and rest: each SIMD has a wave of the tile's first
        // half and one of the second, so a tile of up to 128 rows takes half the time.
        const bool idle = wn * 32 * NT >= to - from;
        const auto stage = [&](int s, auto more) {
            const int buffer = buffer_of(at + s);
            const uint4 *lq = lds + buffer * BOTH, *lp = lq + SIDE;
            uint4 p[2][MT], q[2][NT];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if constexpr (ACROSS) p[t][i] = __builtin_bit_cast(uint4, pairs.read(lp + wm * 16, i, t));
                    else p[t][i] = lp[WideTile::slot((wm * MT + i) * 32 + (lane & 31), 2 * t + (lane >> 5))];
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) q[t][j] = lq[WideTile::slot((wn * NT + j) * 32 + (lane & 31), 2 * t + (lane >> 5))];
            }
            uint32_t ps[MT] = {}, qs[NT] = {};
            if constexpr (MICRO) {
                // of a row's four scales a lane has the words of its half: 0 and 2, or 1 and 3
                const int shift = 8 * (lane >> 5);
#pragma unroll
                for (int i = 0; i < MT; ++i) ps[i] = scales[buffer][1][(wm * MT + i) * 32 + (lane & 31)] >> shift;
#pragma unroll
                for (int j = 0; j < NT; ++j) qs[j] = scales[buffer][0][(wn * NT + j) * 32 + (lane & 31)] >> shift;
                store_scales(buffer_of(at + s + 1));
                fetch_scales(s + 2);
            }
            const auto step = [&](auto t) {
                if constexpr (more()) bring(buffer_of(at + s + kBuffers - 1), t());
                if (idle) return;
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[i][j] = Op::template multiply<2 * t()>(p[t()][i], q[t()][j], acc[i][j], ps[i], qs[j]);
                __builtin_amdgcn_sched_barrier(0);
            };
            step(std::integral_constant<int, 0>{});
            step(std::integral_constant<int, 1>{});
        };
        if (expert >= 0) {
            int s = 0;
            // a stage is there when only the loads of the next one are out, and its buffer's last reads are over when all
            // waves have come to the stage after them
            for (; s + kBuffers - 1 < full; ++s) {
                asm volatile("s_waitcnt vmcnt(4) lgkmcnt(0)\n\ts_barrier" ::: "memory");
                stage(s, std::true_type{});
            }
            for (; s < full; ++s) {
                if (s + 1 < full) asm volatile("s_waitcnt vmcnt(4) lgkmcnt(0)\n\ts_barrier" ::: "memory");
                else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
                stage(s, std::false_type{});
            }
            if (s < stages) {
                // the last columns, short of a stage: by way of registers, zeros after them
                const int word = threadIdx.x % 4, left = a.reduced - full * STAGE - word * Op::kPerWord;
                const int64_t bytes = (int64_t)full * kWideWords * 16 + word * 16;
                const auto last = [&](const char *p, uint4 *side, int r) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if constexpr (MICRO) {
                        if (left > 0) __builtin_memcpy(&v, p, 16);     // a group's codes past the last column are zeros
                    } else if (left > 0) {
                        Word<T> t;
                        if (left >= 8) t.load(reinterpret_cast<const T *>(p));
                        else t.load(reinterpret_cast<const T *>(p), left);
                        v = make_uint4(t.v[0], t.v[1], t.v[2], t.v[3]);
                    }
                    side[WideTile::slot(r, word)] = v;
                };
#pragma unroll 1
                for (int r = threadIdx.x / 4; r < kWide; r += kWideThreads / 4) {
                    last(Op::bytes(x_row(r)) + bytes, lds + buffer_of(at + s) * BOTH, r);
                    if constexpr (!ACROSS) last(Op::bytes(w_row(r)) + bytes, lds + buffer_of(at + s) * BOTH + SIDE, r);
                }
                if constexpr (ACROSS)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = threadIdx.x / 32 + i * 16, k = full * STAGE + r, column = min(c0 + 8 * (int)(threadIdx.x % 32), a.columns - 8);
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (k < a.reduced) __builtin_memcpy(&v, Op::bytes(w_row(k)) + 2 * column, 16);
                        lds[buffer_of(at + s) * BOTH + SIDE + Pairs::slot(r, threadIdx.x % 32)] = v;
                    }
                __syncthreads();
                stage(s, std::false_type{});
                ++s;
            }
            at = buffer_of(at + s);
        }

        // the next tile, before this one's results
        const int this_expert = expert, this_c0 = c0;
        const int64_t this_from = from, this_to = to;
        number = tile_in_round(round, blockIdx.x, tiles);
        const bool again = number >= 0;
        if (again) begin(number);

        const auto out = [&](auto *y) {
            const bool act = a.act == MPNN_ACT_SILU, biased = a.bias && this_expert >= 0;      // silu(0) = 0: rows of no expert may take it too
            const auto bias = [&](int c) {
                Chunk<float, 4> b = {{0.0f, 0.0f, 0.0f, 0.0f}};
                if (biased) b.load(a.bias + (int64_t)this_expert * a.columns + c, a.columns - c);
                return b;
            };
            store_lines(reinterpret_cast<char *>(results[wave]), acc, lane, y, a.columns, this_from + wn * NT * 32, this_to,
                        this_c0 + wm * MT * 32, a.columns, bias, [&](float v) { return act ? silu(v) : v; });
        };
        if (a.y_bf16) out(static_cast<bf16 *>(a.y));
        else out(static_cast<float *>(a.y));
        if (!again) break;
    }
}

// ---- few rows ----
// 16 columns by 16 NT rows a wave, operands straight from memory to registers: what bounds a call of few rows is reading the
// weights, so each lane reads 64 neighbouring bytes of a weight row at once (32 of 4-bit codes) and the reduced axis is split
// among the waves of a block, whose sums are added in their order.  A lane's word holds the same steps of the reduced axis for
// rows and weights; which lane holds which does not matter to the sum.  8 rows of eight experts 2048 -> 1024 bf16 9.1 us, 4 rows
// 4096 -> 4096 by 4-bit weights 8.0 us, 216 rows of four 64 -> 128 fp32 10.4 us (a tile's rows found, loads, products and the waves'
// sums one after another); the host needs 10-11 us for such a call.
typedef float floatx4 __attribute__((ext_vector_type(4)));

// PER steps of a row as loaded, and the products of a lane's word of weights with its word of rows.
template <class X, class W> struct FewOp;
template <> struct FewOp<bf16, bf16> {
    static constexpr int kPer = 8, kWords = 4;
    struct Raw {
        Word<bf16> v;
        template <class R> __device__ __forceinline__ void load(const R &r, int k) { RowsOf<bf16>::load(v, r, k); }
        template <class R> __device__ __forceinline__ void load(const R &r, int k, int width) { RowsOf<bf16>::load(v, r, k, width); }
        __device__ __forceinline__ bf16x8 operand() const { return __builtin_bit_cast(bf16x8, make_uint4(v.v[0], v.v[1], v.v[2], v.v[3])); }
    };
    using RawX = Raw;
    using RawW = Raw;
    __device__ __forceinline__ static floatx4 multiply(const RawW &w, const RawX &x, floatx4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.operand(), x.operand(), c, 0, 0, 0);
    }
};
template <> struct FewOp<float, float> {       // fp32 matrix cores: few rows leave them time enough
    static constexpr int kPer = 8, kWords = 4;
    struct Raw {
        Word<float> v;
        template <class R> __device__ __forceinline__ void load(const R &r, int k) { RowsOf<float>::load(v, r, k); }
        template <class R> __device__ __forceinline__ void load(const R &r, int k, int width) { RowsOf<float>::load(v, r, k, width); }
    };
    using RawX = Raw;
    using RawW = Raw;
    __device__ __forceinline__ static floatx4 multiply(const RawW &w, const RawX &x, floatx4 c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(w.v.v[j], x.v.v[j], c, 0, 0, 0);
        return c;
    }
};
struct FewMicro {                               // a whole group
    uint4 v;
    uint32_t scale;
    __device__ __forceinline__ void load(const RowsOf<Micro>::Row &r, int k, int width) {
        v = make_uint4(0, 0, 0, 0);
        scale = 127;
        if (k < width) load(r, k);
    }
    __device__ __forceinline__ void load(const RowsOf<Micro>::Row &r, int k) {
        __builtin_memcpy(&v, r.codes + k / 2, 16);
        scale = r.scales[k / kMicroGroup];
    }
};
template <class T> struct FewRows {             // 32 columns of rows that are not held
    Word<T> v[4];
    template <class R> __device__ __forceinline__ void load(const R &r, int k, int width) {
#pragma unroll
        for (int u = 0; u < 4; ++u) RowsOf<T>::load(v[u], r, k + 8 * u, width);
    }
    template <class R> __device__ __forceinline__ void load(const R &r, int k) {
#pragma unroll
        for (int u = 0; u < 4; ++u) RowsOf<T>::load(v[u], r, k + 8 * u);
    }
};
template <> struct FewOp<Micro, Micro> {
    static constexpr int kPer = 32, kWords = 2;
    using RawX = FewMicro;
    using RawW = FewMicro;
    __device__ __forceinline__ static floatx4 multiply(const RawW &w, const RawX &x, floatx4 c) {
        const intx8 a = {(int)w.v.x, (int)w.v.y, (int)w.v.z, (int)w.v.w, 0, 0, 0, 0}, b = {(int)x.v.x, (int)x.v.y, (int)x.v.z, (int)x.v.w, 0, 0, 0, 0};
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, 0, w.scale, 0, x.scale);
    }
};
template <> struct FewOp<bf16, Micro> {
    static constexpr int kPer = 32, kWords = 2;
    using RawX = FewRows<bf16>;
    using RawW = FewMicro;
    __device__ __forceinline__ static floatx4 multiply(const RawW &w, const RawX &x, floatx4 c) {
        const uint32_t codes[4] = {w.v.x, w.v.y, w.v.z, w.v.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            Word<Micro> m;
            m.v = codes[u];
            m.scale = (uint8_t)w.scale;
            uint4 t[1];
            float unused = 0.0f;
            m.terms(t, unused);
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, t[0]), __builtin_bit_cast(bf16x8, make_uint4(x.v[u].v[0], x.v[u].v[1], x.v[u].v[2], x.v[u].v[3])), c, 0, 0, 0);
        }
        return c;
    }
};
template <> struct FewOp<float, Micro> {
    static constexpr int kPer = 32, kWords = 1;
    using RawX = FewRows<float>;
    using RawW = FewMicro;
    __device__ __forceinline__ static floatx4 multiply(const RawW &w, const RawX &x, floatx4 c) {
        const uint32_t codes[4] = {w.v.x, w.v.y, w.v.z, w.v.w};
        const float step = micro_step(w.scale);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const auto two = [&](auto k) {
                const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[u], step, k());
                c = __builtin_amdgcn_mfma_f32_16x16x4f32(p[0], x.v[u].v[2 * k()], c, 0, 0, 0);
                c = __builtin_amdgcn_mfma_f32_16x16x4f32(p[1], x.v[u].v[2 * k() + 1], c, 0, 0, 0);
            };
            two(std::integral_constant<int, 0>{});
            two(std::integral_constant<int, 1>{});
            two(std::integral_constant<int, 2>{});
            two(std::integral_constant<int, 3>{});
        }
        return c;
    }
};

// Of the block's eight waves `split` share a tile's reduced axis, so it has 8 / split tiles of 16 columns.
constexpr int kFewThreads = 512, kFewWaves = kFewThreads / 64;
template <class X, class W, int NT>
__global__ __launch_bounds__(kFewThreads) void k_product_few(const Args a, int split, const RowsOf<X> x, const RowsOf<W> w) {
    using Op = FewOp<X, W>;
    constexpr int STRIDE = 4 * Op::kWords * Op::kPer;                  // of the reduced axis, a wave at once
    __shared__ floatx4 sums[kFewWaves][NT][64];
    const int64_t number = a.first + blockIdx.x;       // (the last row tiles may be none: all XCDs have their share of the others)
    const Tile tile = find_tile(a.offsets, a.n_experts, a.n, 16 * NT, number / a.tiles_c);
    if (tile.from >= tile.to) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = wave % split;
    const int c0 = ((int)(number % a.tiles_c) * (kFewWaves / split) + wave / split) * 16;
    floatx4 acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = (floatx4)(0.0f);
    if (tile.expert >= 0 && c0 < a.columns) {
        const auto place = [&](int64_t q) -> int64_t {
            if (!a.source) return q;
            return min((int64_t)((uint32_t)max(a.source[q], 0) / (uint32_t)a.slots), a.n_x - 1);
        };
        typename RowsOf<X>::Row xr[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) xr[j] = x.row(place(min(tile.from + 16 * j + (lane & 15), tile.to - 1)));
        const typename RowsOf<W>::Row wr = w.row((int64_t)tile.expert * a.columns + min(c0 + (lane & 15), a.columns - 1));
        const int turns = (a.reduced + STRIDE - 1) / STRIDE, each = (turns + split - 1) / split;
        const int first = part * each, last = min(first + each, turns);
        typename Op::RawW wv[2][Op::kWords];
        typename Op::RawX xv[2][NT][Op::kWords];
        const auto fetch = [&](int turn, int b) {
            const int k = turn * STRIDE + (lane >> 4) * (Op::kWords * Op::kPer);
            if ((turn + 1) * STRIDE <= a.reduced) {      // whole words, no conditions beside the loads
#pragma unroll
                for (int u = 0; u < Op::kWords; ++u) wv[b][u].load(wr, k + u * Op::kPer);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int u = 0; u < Op::kWords; ++u) xv[b][j][u].load(xr[j], k + u * Op::kPer);
                return;
            }
#pragma unroll
            for (int u = 0; u < Op::kWords; ++u) wv[b][u].load(wr, k + u * Op::kPer, a.reduced);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int u = 0; u < Op::kWords; ++u) xv[b][j][u].load(xr[j], k + u * Op::kPer, a.reduced);
        };
        const auto use = [&](int b) {
#pragma unroll
            for (int u = 0; u < Op::kWords; ++u)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[j] = Op::multiply(wv[b][u], xv[b][j][u], acc[j]);
        };
        if (first < last) fetch(first, 0);
        for (int t = first; t < last; t += 2) {
            if (t + 1 < last) fetch(t + 1, 1);
            use(0);
            if (t + 1 < last) {
                if (t + 2 < last) fetch(t + 2, 0);
                use(1);
            }
        }
    }
    if (split > 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j) sums[wave][j][lane] = acc[j];
        __syncthreads();
        if (part != 0) return;
        for (int p = 1; p < split; ++p)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j] += sums[wave + p][j][lane];
    }
    // a lane has four neighbouring columns of a row
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t q = tile.from + 16 * j + (lane & 15);
        const int c = c0 + 4 * (lane >> 4);
        float v[4] = {acc[j][0], acc[j][1], acc[j][2], acc[j][3]};
        if (q < tile.to && c < a.columns) finish(a, tile.expert, q, c, a.columns - c, v);
    }
}

// The same across (dx): a lane has four neighbouring columns of a weight row and four steps of a gradient row, which are fp32
// operands whatever their type; a wave has 64 columns, a lane's results are sixteen neighbouring ones.  64 rows of eight experts
// 2048 -> 1024: 67 MB of fp32 weights in 16 us, bf16 in 14.
template <class T> struct FewAcross {
    T v[4];
    __device__ __forceinline__ void load(const T *p) { __builtin_memcpy(v, p, 4 * sizeof(T)); }
    // `in` of them are the row's: one value at least lies at or before p
    __device__ __forceinline__ void load(const T *p, int in) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = p[min(j, in - 1)];
    }
    __device__ __forceinline__ void keep(int in) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = j < in ? v[j] : from_f32<T>(0.0f);
    }
};
template <class T, int NT>
__global__ __launch_bounds__(kFewThreads) void k_input_grad_few(const Args a, int split, const RowsOf<T> dy, const RowsOf<T> w) {
    constexpr int STRIDE = 16;
    __shared__ floatx4 sums[kFewWaves][4 * NT][64];
    const int64_t number = a.first + blockIdx.x;
    const Tile tile = find_tile(a.offsets, a.n_experts, a.n, 16 * NT, number / a.tiles_c);
    if (tile.from >= tile.to) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = wave % split;
    const int c0 = ((int)(number % a.tiles_c) * (kFewWaves / split) + wave / split) * 64;
    floatx4 acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = (floatx4)(0.0f);
    if (tile.expert >= 0 && c0 < a.columns) {
        const T *yr[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) yr[j] = dy.row(min(tile.from + 16 * j + (lane & 15), tile.to - 1)).p + 4 * (lane >> 4);
        const int c = c0 + 4 * (lane & 15), in = a.columns - c;
        const bool whole = c0 + 64 <= a.columns;
        const T *const wr = w.row((int64_t)tile.expert * a.reduced).p + (in > 0 ? c : 0);       // columns past the last are not stored
        const int turns = (a.reduced + STRIDE - 1) / STRIDE, each = (turns + split - 1) / split;
        const int first = part * each, last = min(first + each, turns);
        FewAcross<T> wv[2][4], yv[2][NT];
        const auto fetch = [&](int turn, int b) {
            const int k = turn * STRIDE, mine = k + 4 * (lane >> 4);
            if (whole && k + STRIDE <= a.reduced) {
#pragma unroll
                for (int u = 0; u < 4; ++u) wv[b][u].load(wr + (int64_t)(mine + u) * w.ld);
#pragma unroll
                for (int j = 0; j < NT; ++j) yv[b][j].load(yr[j] + k);
                return;
            }
            const int steps = a.reduced - mine;          // steps past the last are zeros on both sides
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                wv[b][u].load(wr + (int64_t)min(mine + u, a.reduced - 1) * w.ld, in > 0 ? in : 1);
                wv[b][u].keep(u < steps ? 4 : 0);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                yv[b][j].load(yr[j] + k, steps);
                yv[b][j].keep(steps);
            }
        };
        const auto use = [&](int b) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(to_f32(wv[b][u].v[i]), to_f32(yv[b][j].v[u]), acc[j][i], 0, 0, 0);
        };
        if (first < last) fetch(first, 0);
        for (int t = first; t < last; t += 2) {
            if (t + 1 < last) fetch(t + 1, 1);
            use(0);
            if (t + 1 < last) {
                if (t + 2 < last) fetch(t + 2, 0);
                use(1);
            }
        }
    }
    if (split > 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[wave][4 * j + i][lane] = acc[j][i];
        __syncthreads();
        if (part != 0) return;
        for (int p = 1; p < split; ++p)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] += sums[wave + p][4 * j + i][lane];
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t q = tile.from + 16 * j + (lane & 15);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int c = c0 + 16 * (lane >> 4) + 4 * r;
            float v[4] = {acc[j][0][r], acc[j][1][r], acc[j][2][r], acc[j][3][r]};
            if (q < tile.to && c < a.columns) finish(a, tile.expert, q, c, a.columns - c, v);
        }
    }
}

// Every block of a tiling, in launches of as many as one holds.
template <class F> Status by_tiles(Args &a, int columns, int rows, F run) {
    a.tiles_c = (a.columns + columns - 1) / columns;
    return by_launches(row_tiles(a.n, a.n_experts, rows) * a.tiles_c, kLaunchBlocks, [&](int64_t from, int64_t count) -> Status {
        a.first = from;
        run(grid_xcd(count, 1));
        MPNN_HIP(hipGetLastError());
        return Status::ok();
    });
}

// Blocks that stay for many tiles: as many as run at once, or as there are tiles.
inline unsigned resident(int64_t tiles, int64_t most) { return grid_xcd(std::min(tiles, most), 1); }

// Rows that start on 16 bytes, as the loads to LDS need them.
inline bool whole_words(const void *p, int64_t row_bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row_bytes % 16 == 0; }
inline bool wide_fits(const RowsOf<bf16> &x, const RowsOf<bf16> &w) { return whole_words(x.p, 2 * x.ld) && whole_words(w.p, 2 * w.ld); }
inline bool wide_fits(const RowsOf<Micro> &x, const RowsOf<Micro> &w) { return whole_words(x.codes, 16) && whole_words(w.codes, 16); }

template <class X, class W, bool ACROSS>
Status product_t(Context &cx, Args a, const RowsOf<X> &x, const RowsOf<W> &w) {
    // Few results: straight from memory.  Its time goes with the rows that every 16 columns read again, a tile's with the length
    // of its sums, so the sides meet at a number of results: 512 rows of eight experts 2048 -> 1024 bf16 30 us and 40 in tiles,
    // 640 rows 46 and 41; fp32 73 and 118, 800 rows 126 and 118; 200 rows 4096 -> 4096 fp32 199 and 227, 400 rows 370 and 233.
    if constexpr (!ACROSS) {
        constexpr bool both32 = std::is_same<X, float>::value && std::is_same<W, float>::value;
        if (a.n * a.columns <= (both32 ? 768 << 10 : 512 << 10)) {
            int split = 1;
            while (split < kFewWaves && split * 4 * FewOp<X, W>::kWords * FewOp<X, W>::kPer < a.reduced) split *= 2;
            const auto few = [&](auto nt) {
                return by_tiles(a, 16 * (kFewWaves / split), 16 * nt(), [&](unsigned grid) { k_product_few<X, W, nt()><<<grid, kFewThreads, 0, cx.stream>>>(a, split, x, w); });
            };
            const int64_t rows = (a.n + std::min<int64_t>(a.n, a.n_experts) - 1) / std::min<int64_t>(a.n, a.n_experts);    // of an expert
            if (rows <= 16) return few(std::integral_constant<int, 1>{});
            // four row groups of operands fit the registers where both sides have the same 16-bit or smaller type
            if constexpr (std::is_same<X, W>::value && !std::is_same<X, float>::value)
                if (rows > 32) return few(std::integral_constant<int, 4>{});
            return few(std::integral_constant<int, 2>{});
        }
    }
    // Few results across likewise, in groups of 64 columns: eight experts' 2048 -> 1024 take 64 rows of dx fp32 16 us (tiles 70),
    // 1,024 rows 66 (71); bf16 64 rows 14 (25), 256 rows 20 (25), 512 rows 31 (25); 400 rows 4096 -> 4096 fp32 215 (256);
    // 1,000 rows 256 -> 4096 fp32 47 (254), bf16 57 (104); 40,000 rows 15 -> 500 of twenty fp32 72 (63).
    if constexpr (ACROSS) {
        if (a.n * ((a.columns + 63) / 64 * 64) <= (std::is_same<X, float>::value ? 1536 << 10 : 512 << 10)) {
            int split = 1;
            while (split < kFewWaves && split * 32 < a.reduced) split *= 2;
            const auto few = [&](auto nt) {
                return by_tiles(a, 64 * (kFewWaves / split), 16 * nt(), [&](unsigned grid) { k_input_grad_few<X, nt()><<<grid, kFewThreads, 0, cx.stream>>>(a, split, x, w); });
            };
            const int64_t rows = (a.n + std::min<int64_t>(a.n, a.n_experts) - 1) / std::min<int64_t>(a.n, a.n_experts);    // of an expert
            return rows <= 16 ? few(std::integral_constant<int, 1>{}) : few(std::integral_constant<int, 2>{});
        }
    }
    if constexpr (std::is_same<X, W>::value && !std::is_same<X, float>::value) {
        if (a.columns > kTile && wide_fits(x, w)) {
            a.tiles_c = (a.columns + kWide - 1) / kWide;
            k_product_wide<X, ACROSS><<<resident(row_tiles(a.n, a.n_experts, kWide) * a.tiles_c, kCus), kWideThreads, 0, cx.stream>>>(a, x, w);
            MPNN_HIP(hipGetLastError());
            return Status::ok();
        }
    }
    a.tiles_c = (a.columns + kTile - 1) / kTile;
    k_product<X, W, ACROSS><<<resident(row_tiles(a.n, a.n_experts, kTile) * a.tiles_c, 2 * kCus), 256, 0, cx.stream>>>(a, x, w);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
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
