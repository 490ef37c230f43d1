// Rows of experts cut into pieces, for sums over the rows that are split among blocks (weight_grad.hip, expert_grad.hip).
#pragma once

#include "impl.h"

namespace mpnn {

// Pieces of each expert: at least one (an expert without rows writes its zeros).
__device__ __forceinline__ int pieces_of(const int32_t *offsets, int e, int64_t n, int64_t rows, int64_t &from, int64_t &to) {
    from = min(max((int64_t)offsets[e], (int64_t)0), n);
    to = min(max((int64_t)offsets[e + 1], from), n);
    return (int)max((int64_t)1, (to - from + rows - 1) / rows);
}

struct Piece {
    int expert, piece, pieces;   // piece of its expert's pieces; expert < 0: past the last
    int slot;                    // partial sums of the expert's first piece (pieces > 1)
};

// Floats of a piece's partial sums, dW then db, in whole 16 bytes.
__host__ __device__ __forceinline__ int64_t slot_size(int64_t values) { return (values + 3) / 4 * 4; }

// The piece with the given number, by one wave: a prefix sum over the experts, 64 at a time.  want_expert >= 0 looks
// that expert up instead.
__device__ __forceinline__ Piece find_piece(const int32_t *offsets, int n_experts, int64_t n, int64_t rows, int number, int want_expert) {
    const int lane = threadIdx.x & 63;
    int before = 0, slots = 0;
    for (int base = 0; base < n_experts; base += 64) {
        const int e = base + lane;
        int64_t from, to;
        const int c = e < n_experts ? pieces_of(offsets, e, n, rows, from, to) : 0;
        const int m = c > 1 ? c : 0;
        int s = c, t = m;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int a = __shfl_up(s, d), b = __shfl_up(t, d);
            if (lane >= d) {
                s += a;
                t += b;
            }
        }
        const uint64_t hit = __ballot(want_expert >= 0 ? e == want_expert : e < n_experts && number < before + s);
        if (hit) {
            // the same in all lanes, and known to be: what follows from it is computed once a wave
            const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
            const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
            const int pc = of(c);
            return Piece{base + l, number - (before + of(s) - pc), pc, slots + of(t) - of(m)};
        }
        before += __builtin_amdgcn_readlane(s, 63);
        slots += __builtin_amdgcn_readlane(t, 63);
    }
    return Piece{-1, 0, 0, 0};
}

// With an expert a piece (and at most 64 experts, one a lane): the expert whose tiles are the number-th to start.  The
// longest experts start first, `row` of them on all CUs, and the next ones in turn from the shortest and the longest, so that
// a CU that holds two blocks holds a long and a short one (16,384 rows 1024 -> 1024 x 8, shares from 4 to 20 %: bf16 85 -> 79 us,
// fp32 163 -> 156 us).
__device__ __forceinline__ int expert_in_turn(const int32_t *offsets, int n_experts, int64_t n, int row, int number) {
    const int lane = threadIdx.x & 63, e = min(lane, n_experts - 1);
    const int from = (int)min(max((int64_t)offsets[e], (int64_t)0), n), to = (int)min(max((int64_t)offsets[e + 1], (int64_t)from), n);
    const int length = to - from;
    int rank = 0;
    for (int f = 0; f < n_experts; ++f) {
        const int other = __builtin_amdgcn_readlane(length, f);
        rank += other > length || (other == length && f < lane);
    }
    const int in = number % row, want = (number / row & 1) && number - in + row <= n_experts ? number - in + row - 1 - in : number;
    return __ffsll((unsigned long long)__ballot(lane < n_experts && rank == want)) - 1;
}

// The pieces of each expert that has several, added in a fixed order (weight_grad.hip): dW of `matrix` values and db of `out`.
Status join_pieces(Context &cx, int n_experts, int64_t n, int64_t rows, int64_t slots, int64_t matrix, int out, const int32_t *offsets,
                   const float *part, float *dweight, float *dbias);

}  // namespace mpnn
