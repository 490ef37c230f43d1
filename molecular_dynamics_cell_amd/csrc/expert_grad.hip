// Weight gradients of the experts' products (mpnn_expert_weight_grad):
//   dW_e[o][c] = sum over the rows q of expert e of dy[q][o] x[q][c],  db_e[o] = sum of dy[q][o].
// Rows are cut into pieces as for the gradient from checkpoints; both operands have the rows as their slow axis and are
// turned by the transposing reads of LDS.
// 128,000 rows 312 -> 128 x 5 fp32: 96-103 us, and 7 to add the pieces; six products and the cutting of both operands into terms
// share the issue slots (35 us are the products at a large bf16 product's rate).
#include <algorithm>
#include <type_traits>

#include "impl.h"
#include "pieces.h"
#include "rows.h"
#include "tiles.h"

namespace mpnn {

namespace {

struct Args {
    int64_t n, rows;                // rows; of a piece
    int out, width, n_experts, tiles_c, tiles;
    const int32_t *offsets, *source;
    int64_t n_x;
    int slots;
    int64_t part_slots;
    float *part, *dweight, *dbias;
};

template <class T, int MT, int NT, int WM, int WN>
__global__ __launch_bounds__(256, 2) void k_expert_weight_grad(const Args a, const RowsOf<T> dy, const RowsOf<T> x) {
    constexpr int TERMS = kTerms<T>, WORDS = TERMS > 1 ? 4 : 8, STEPS = 8 * WORDS;
    constexpr int BC = 32 * MT * WM, BO = 32 * NT * WN;
    using P = Across<TERMS, BC, WORDS>;
    using Q = Across<TERMS, BO, WORDS>;
    __shared__ uint4 lds[P::kWords + Q::kWords];
    __shared__ float sums[256][8];
    uint4 *const lp = lds, *const lq = lds + P::kWords;

    const uint32_t number = (uint32_t)xcd_block();
    const int tile = (int)(number % (uint32_t)a.tiles);
    const Piece pc = find_piece(a.offsets, a.n_experts, a.n, a.rows, (int)(number / (uint32_t)a.tiles), -1);
    if (pc.expert < 0) return;
    int64_t from, to;
    pieces_of(a.offsets, pc.expert, a.n, a.rows, from, to);
    from += pc.piece * a.rows;
    to = min(to, from + a.rows);
    const int o0 = tile / a.tiles_c * BO, c0 = tile % a.tiles_c * BC;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave / WN, wn = wave % WN;

    constexpr int WP = BC / 8, WQ = BO / 8, XP = STEPS * WP / 256, XQ = STEPS * WQ / 256;     // words a row; words a thread
    static_assert(STEPS * WP % 256 == 0 && STEPS * WQ % 256 == 0, "whole words a thread");
    Word<T> pv[XP], qv[XQ];
    int32_t at[XP];
    const auto places = [&](int64_t q0) {
#pragma unroll
        for (int i = 0; i < XP; ++i) {
            const int64_t q = min(q0 + tid / WP + i * (256 / WP), a.n - 1);
            at[i] = a.source ? (int32_t)min((int64_t)((uint32_t)max(a.source[q], 0) / (uint32_t)a.slots), a.n_x - 1) : (int32_t)q;
        }
    };
    // A stage of whole words has no conditions beside its loads; nor has another one where eight rows follow those that a wave
    // loads, so that words may be loaded past a row's end.
    const bool columns_whole = (c0 + BC <= a.width || a.width % 8 == 0) && (o0 + BO <= a.out || a.out % 8 == 0);
    const int pc0 = c0 + tid % WP * 8, qc0 = o0 + tid % WQ * 8, pc1 = min(pc0, a.width - 8), qc1 = min(qc0, a.out - 8);
    const auto fetch = [&](int64_t q0) {
        bool over = q0 + STEPS <= to && q0 + STEPS + 8 <= a.n;
#pragma unroll
        for (int i = 0; i < XP; ++i) over = over && at[i] < a.n_x - 8;
        if (columns_whole && q0 + STEPS <= to) {
#pragma unroll
            for (int i = 0; i < XP; ++i) RowsOf<T>::load(pv[i], x.row(at[i]), pc1);
#pragma unroll
            for (int i = 0; i < XQ; ++i) RowsOf<T>::load(qv[i], dy.row(q0 + tid / WQ + i * (256 / WQ)), qc1);
        } else if (__all(over)) {
#pragma unroll
            for (int i = 0; i < XP; ++i) RowsOf<T>::load_over(pv[i], x.row(at[i]), pc0, a.width);
#pragma unroll
            for (int i = 0; i < XQ; ++i) RowsOf<T>::load_over(qv[i], dy.row(q0 + tid / WQ + i * (256 / WQ)), qc0, a.out);
        } else {
#pragma unroll
            for (int i = 0; i < XP; ++i) {
                if (q0 + tid / WP + i * (256 / WP) < to) RowsOf<T>::load(pv[i], x.row(at[i]), pc0, a.width);
                else pv[i].clear();
            }
#pragma unroll
            for (int i = 0; i < XQ; ++i) {
                const int64_t q = q0 + tid / WQ + i * (256 / WQ);
                if (q < to) RowsOf<T>::load(qv[i], dy.row(q), qc0, a.out);
                else qv[i].clear();
            }
        }
    };
    floatx16 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = (floatx16)(0.0f);
    float bias[8] = {}, largest = 0.0f;
    if (from < to) {
        places(from);
        fetch(from);
    }
    for (int64_t q0 = from; q0 < to; q0 += STEPS) {
        places(q0 + STEPS);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < XP; ++i) {
            uint4 t[TERMS];
            pv[i].terms(t, largest);
            P::store(lp, tid / WP + i * (256 / WP), tid % WP, t);
        }
#pragma unroll
        for (int i = 0; i < XQ; ++i) {
            uint4 t[TERMS];
            qv[i].terms(t, largest);
            Q::store(lq, tid / WQ + i * (256 / WQ), tid % WQ, t);
            if (c0 == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) bias[j] += qv[i].at(j);
        }
        __syncthreads();
        if (q0 + STEPS < to) fetch(q0 + STEPS);
        multiply<P, Q, TERMS, TERMS, MT, NT, WORDS>(lp, lq, wm * MT * 32, wn * NT * 32, lane, acc);
    }
    const bool large = TERMS > 1 && __syncthreads_or(largest >= kLarge);       // then results that are not finite, once more without terms

    const int64_t matrix = (int64_t)a.out * a.width;
    const bool whole = pc.pieces == 1;
    if (!whole && pc.slot + pc.piece >= a.part_slots) return;     // offsets that do not ascend name more pieces than there are
    float *to_w = whole ? a.dweight + pc.expert * matrix : a.part + (int64_t)(pc.slot + pc.piece) * slot_size(matrix + a.out);
    float *to_b = whole ? (a.dbias ? a.dbias + (int64_t)pc.expert * a.out : nullptr) : to_w + matrix;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int o = o0 + (wn * NT + j) * 32 + (lane & 31);
        if (o >= a.out) continue;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = c0 + (wm * MT + i) * 32 + 8 * g + 4 * (lane >> 5), in = a.width - c;
                if (in <= 0) continue;
                Chunk<float, 4> v;
#pragma unroll
                for (int r = 0; r < 4; ++r) v.v[r] = acc[i][j][4 * g + r];
                if (large)
                    for (int r = 0; r < 4; ++r)
                        if (!isfinite(v.v[r]) && r < in) {
                            float s = 0.0f;
                            for (int64_t q = from; q < to && s == s; ++q) {
                                const int64_t at = a.source ? min((int64_t)((uint32_t)max(a.source[q], 0) / (uint32_t)a.slots), a.n_x - 1) : q;
                                s = fmaf(dy.at(q, o), x.at(at, c + r), s);
                            }
                            v.v[r] = s;
                        }
                v.store(to_w + (int64_t)o * a.width + c, in);
            }
    }
    if (c0 == 0 && to_b) {
        // the threads of a word's columns, in their order
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[tid][j] = bias[j];
        __syncthreads();
        if (tid < BO && o0 + tid < a.out) {
            float s = 0.0f;
            for (int k = tid / 8; k < 256; k += WQ) s += sums[k][tid % 8];
            to_b[o0 + tid] = s;
        }
    }
}

// Wide tiles, bf16: 256 columns of x by 256 of dy, eight waves of 128 x 64, stages of 32 rows that go to LDS without passing
// through registers, two stages ahead; a bias is the product of dy with ones.  A block stays for many tiles: the next one's
// first stages are on their way while this one's results are stored.
// Whole pieces are dealt to the blocks first, then what is left of each expert, in turn from the first block to the last and
// back, so that a block with one tile more has a short one.
// 32,768 rows 1024 -> 1024 x 8: 93-135 us by the experts' shares (46 at a large product's rate), and 21 to add the pieces.
constexpr int kWide = 256, kWideThreads = 512, kBuffers = 3, kWideStage = 32, kCus = 256, kMostExperts = 1024;

__global__ __launch_bounds__(kWideThreads, 2) void k_expert_weight_grad_wide(const Args a, const RowsOf<bf16> dy, const RowsOf<bf16> x) {
    constexpr int MT = 4, NT = 2, SIDE = Pairs::kWords, BOTH = 2 * SIDE;
    __shared__ uint4 lds[kBuffers * BOTH];                             // dy, then x
    __shared__ uint4 results[kWideThreads / 64][kStoreBytes / 16];
    __shared__ int before[kMostExperts + 1], slot[kMostExperts];       // whole pieces before each expert's; its partial sums
    typedef const __attribute__((address_space(1))) void *Global;
    typedef __attribute__((address_space(3))) void *Local;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave & 1, wn = wave >> 1;
    const Pairs pairs(lane);
    if (wave == 0) {
        int wholes = 0, slots = 0;
        for (int base = 0; base < a.n_experts; base += 64) {
            const int e = base + lane;
            int64_t from = 0, to = 0;
            const int p = e < a.n_experts ? pieces_of(a.offsets, e, a.n, a.rows, from, to) : 0, c = (int)((to - from) / a.rows), m = p > 1 ? p : 0;
            int s = c, t = m;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int u = __shfl_up(s, d), v = __shfl_up(t, d);
                if (lane >= d) {
                    s += u;
                    t += v;
                }
            }
            if (e < a.n_experts) {
                before[e] = wholes + s - c;
                slot[e] = slots + t - m;
            }
            wholes += __builtin_amdgcn_readlane(s, 63);
            slots += __builtin_amdgcn_readlane(t, 63);
        }
        if (lane == 0) before[a.n_experts] = wholes;
    }
    __syncthreads();
    const int64_t wholes = (int64_t)before[a.n_experts] * a.tiles, all = wholes + (int64_t)a.n_experts * a.tiles;
    const int64_t matrix = (int64_t)a.out * a.width;

    // The tile that is being brought, multiplied and stored.
    float *to_w = nullptr, *to_b = nullptr;        // (null: nothing is stored)
    int o0 = 0, c0 = 0, full = 0, stages = 0, at = 0;
    int64_t from = 0, to = 0, next[2];             // next: the row of x that is brought next (by source)
    const bf16 *px[2], *pd[2];
    const auto place = [&](int64_t q) -> int64_t { return min((int64_t)((uint32_t)max(a.source[q], 0) / (uint32_t)a.slots), a.n_x - 1); };
    // Lane l of a wave's i-th load of a stage brings one word of step (2 wave + i) 2 + l / 32; words past the last column bring
    // the last one again.
    const int step0 = wave * 4 + Pairs::step_of(lane);
    const auto look_up = [&](int s, int i) { next[i] = place(min(from + (int64_t)s * kWideStage + step0 + i * 2, to - 1)); };
    const auto bring = [&](int s, int i) {
        const int words = (at + s) % kBuffers * BOTH + (wave * 2 + i) * Pairs::kPair;
        const bf16 *p = px[i];
        if (a.source) {
            p += next[i] * x.ld;
            look_up(s + 1, i);
        } else {
            px[i] += kWideStage * x.ld;
        }
        __builtin_amdgcn_global_load_lds((Global)pd[i], (Local)&lds[words], 16, 0, 0);
        __builtin_amdgcn_global_load_lds((Global)p, (Local)&lds[words + SIDE], 16, 0, 0);
        pd[i] += kWideStage * dy.ld;
    };
    const auto begin = [&](int64_t number) {
        const int64_t piece = number / a.tiles;
        const int tile = (int)(number % a.tiles);
        int e, k;                                  // expert, and the piece of its pieces
        if (number < wholes) {
            int low = 0, high = a.n_experts - 1;   // the last expert with at most `piece` pieces before its own
            while (low < high) {
                const int mid = (low + high + 1) / 2;
                if (before[mid] <= piece) low = mid;
                else high = mid - 1;
            }
            e = low;
            k = (int)piece - before[low];
        } else {
            e = (int)(piece - before[a.n_experts]);
            k = before[e + 1] - before[e];
        }
        e = __builtin_amdgcn_readfirstlane(e);
        k = __builtin_amdgcn_readfirstlane(k);
        const int pieces = pieces_of(a.offsets, e, a.n, a.rows, from, to);
        from += k * a.rows;
        to = min(to, from + a.rows);
        const int place_of = slot[e] + k;
        const bool none = k >= pieces || (pieces > 1 && place_of >= a.part_slots);    // (offsets that do not ascend: more pieces than there are)
        if (none) to = from;
        to_w = none ? nullptr : pieces == 1 ? a.dweight + e * matrix : a.part + place_of * slot_size(matrix + a.out);
        to_b = none ? nullptr : pieces == 1 ? (a.dbias ? a.dbias + (int64_t)e * a.out : nullptr) : to_w + matrix;
        o0 = tile / a.tiles_c * kWide;
        c0 = tile % a.tiles_c * kWide;
        full = (int)((to - from) / kWideStage);
        stages = (int)((to - from + kWideStage - 1) / kWideStage);
        if (stages == 0) return;
        const int xc = min(c0 + 8 * Pairs::word_of(lane), a.width - 8), oc = min(o0 + 8 * Pairs::word_of(lane), a.out - 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t q = min(from + step0 + i * 2, to - 1);
            pd[i] = dy.p + q * dy.ld + oc;
            px[i] = x.p + (a.source ? 0 : q * x.ld) + xc;
            if (a.source) look_up(0, i);
        }
        for (int s = 0; s < min(full, kBuffers - 1); ++s) {
            bring(s, 0);
            bring(s, 1);
        }
    };

    int64_t number = tile_in_round(0, blockIdx.x, all);
    if (number < 0) return;
    begin(number);
    for (int64_t round = 1;; ++round) {
        floatx16 acc[MT][NT], sum[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            sum[j] = (floatx16)(0.0f);
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i][j] = (floatx16)(0.0f);
        }
        const bool biased = c0 == 0 && wm == 0 && to_b;
        const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
        const auto stage = [&](int s, auto more) {
            const uint4 *lq = lds + (at + s) % kBuffers * BOTH + wn * 8, *lp = lds + (at + s) % kBuffers * BOTH + SIDE + wm * 16;
            bf16x8 p[2][MT], q[2][NT];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int i = 0; i < MT; ++i) p[t][i] = pairs.read(lp, i, t);
#pragma unroll
                for (int j = 0; j < NT; ++j) q[t][j] = pairs.read(lq, j, t);
            }
            const auto step = [&](int t) {
                if constexpr (more()) bring(s + kBuffers - 1, t);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(p[t][i], q[t][j], acc[i][j], 0, 0, 0);
                if (biased)
#pragma unroll
                    for (int j = 0; j < NT; ++j) sum[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, ones), q[t][j], sum[j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            };
            step(0);
            step(1);
        };
        // a stage is there when only the loads of the next one are out, and its buffer's last reads are over when all waves have
        // come to the stage after them
        int s = 0;
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
            // the last rows, short of a stage: by way of registers, zeros after them
            const int word = threadIdx.x % 32, oc = min(o0 + 8 * word, a.out - 8), xc = min(c0 + 8 * word, a.width - 8);
            uint4 *const to_lds = lds + (at + s) % kBuffers * BOTH;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int step = threadIdx.x / 32 + i * 16;
                const int64_t q = from + (int64_t)full * kWideStage + step;
                uint4 d = make_uint4(0, 0, 0, 0), v = d;
                if (q < to) {
                    __builtin_memcpy(&d, dy.p + q * dy.ld + oc, 16);
                    __builtin_memcpy(&v, x.p + (a.source ? place(q) : q) * x.ld + xc, 16);
                }
                to_lds[Pairs::slot(step, word)] = d;
                to_lds[SIDE + Pairs::slot(step, word)] = v;
            }
            __syncthreads();
            stage(s, std::false_type{});
            ++s;
        }
        at = (at + s) % kBuffers;

        // the next tile, before this one's results
        float *const this_w = to_w, *const this_b = to_b;
        const int this_o0 = o0, this_c0 = c0;
        number = tile_in_round(round, round % 2 ? gridDim.x - 1 - blockIdx.x : blockIdx.x, all);
        const bool again = number >= 0;            // a block without a tile in this round has none in a later one
        if (again) begin(number);
        if (this_w) {
            if (biased && lane < 32)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (const int o = this_o0 + (wn * NT + j) * 32 + lane; o < a.out) this_b[o] = sum[j][0];
            // by L2: the pieces' sums are read again
            store_lines_to<false>(reinterpret_cast<char *>(results[wave]), acc, lane, this_w, a.width, this_o0 + wn * NT * 32, a.out, this_c0 + wm * MT * 32,
                        a.width, [](int) { return Chunk<float, 4>{{0.0f, 0.0f, 0.0f, 0.0f}}; }, [](float v) { return v; });
        }
        if (!again) break;
    }
}

template <class T>
Status weight_grad_t(Context &cx, Args a, const RowsOf<T> &dy, const RowsOf<T> &x) {
    const auto whole = [](const void *p, int64_t ld, int width) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 && width % 8 == 0; };
    const bool wide = std::is_same<T, bf16>::value && a.out > 128 && a.width > 128 && a.n / a.n_experts >= 128 && whole(dy.p, dy.ld, a.out) &&
                      whole(x.p, x.ld, a.width);
    const int tile = wide ? kWide : 128;
    a.tiles_c = (a.width + tile - 1) / tile;
    a.tiles = a.tiles_c * ((a.out + tile - 1) / tile);
    const int64_t want = wide ? std::max<int64_t>(1, 256 / a.tiles) : std::max<int64_t>(1, 512 / a.tiles - a.n_experts);
    // The least rows of a piece: few, as a piece's time is that of its stages one after another where there are too few pieces for
    // the GPU (30,000 rows 64 -> 64 x 4 fp32 43 us with 512, 30 with 256, 23 with 128, bf16 21, 17, 17; 3,000 rows fp32 42 and 19);
    // more where a stage is longer (20,000 rows 256 -> 256 x 8 bf16 27 us with 256, 30 with 128) and where tiles are wide (4,000 rows
    // 1024 -> 1024 x 8 32 us with 512, 53 with 256); and up to 512 rows are not cut, which spares a launch (454 rows 11 and 15 us).
    const int64_t least = wide || a.n <= 512 ? 512 : std::is_same<T, float>::value ? 128 : 256;
    a.rows = std::max<int64_t>(least, ((a.n + want - 1) / want + 63) / 64 * 64);
    const int64_t pieces = a.n / a.rows + a.n_experts;
    const int64_t matrix = (int64_t)a.out * a.width;
    a.part_slots = a.n > a.rows ? 2 * (a.n / a.rows) : 0;
    void *ws = nullptr;
    MPNN_TRY(cx.rows_scratch(sizeof(float) * (size_t)(a.part_slots * slot_size(matrix + a.out)), &ws));
    a.part = static_cast<float *>(ws);
    if constexpr (std::is_same<T, bf16>::value)
        if (wide) k_expert_weight_grad_wide<<<(unsigned)std::min<int64_t>(grid_xcd(std::min<int64_t>(pieces * a.tiles, kCus), 1), kCus), kWideThreads, 0, cx.stream>>>(a, dy, x);
    if (!wide) k_expert_weight_grad<T, 2, 2, 2, 2><<<grid_xcd(pieces * a.tiles, 1), 256, 0, cx.stream>>>(a, dy, x);
    MPNN_HIP(hipGetLastError());
    return a.part_slots ? join_pieces(cx, a.n_experts, a.n, a.rows, a.part_slots, matrix, a.out, a.offsets, a.part, a.dweight, a.dbias) : Status::ok();
}

}  // namespace

Status expert_weight_grad(Context &cx, int dtype, int64_t n, int width, int n_out, int n_experts, const int32_t *offsets, const void *dy,
                          int64_t ld_dy, const void *x, int64_t ldx, const int32_t *source, int64_t n_x, float *dweight, float *dbias) {
    if (n == 0) source = nullptr;       // no places to look up, and n_x may be zero
    const Args a{n, 0, n_out, width, n_experts, 0, 0, offsets, source, source ? n_x : n, source ? (int)(n / n_x) : 1, 0, nullptr, dweight, dbias};
    if (dtype == MPNN_BF16) return weight_grad_t<bf16>(cx, a, {(const bf16 *)dy, ld_dy}, {(const bf16 *)x, ldx});
    return weight_grad_t<float>(cx, a, {(const float *)dy, ld_dy}, {(const float *)x, ldx});
}

}  // namespace mpnn
