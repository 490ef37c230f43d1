// Tiles of matrix products on the bf16 matrix cores (expert.hip, expert_grad.hip): words of eight values are loaded to
// registers, turned into matrix-core operands and held in LDS.
//
// Operands.  A bf16 value is one as it stands, and so is a 4-bit value times its power-of-two step.  An fp32 value is cut
// into three bf16 terms by rounding, each to nearest: the second is at most 2^-9 of the value, the third 2^-18, and the three add
// up to it exactly.  Of the nine products of two such values the six largest are taken; what is left out is below
// 2 * 2^-9 * 2^-18 = 2^-26 of the product, less than fp32's own rounding of it.  Terms overflow where their values do not: a
// value of 0x1.ffp127 and more rounds to an infinity, whose other terms are not numbers, products of first terms may be 2^-8 larger
// than those of the values, and the remainders' products may overflow with the other sign.  Kernels keep the largest magnitude
// they have met and compute the results that are not finite again from the values, one by one, where it is large enough for any
// of it: below 2^48 products are below 2^96, and 2^31 of them below 2^127.
// The matrix cores take terms below 2^-126 as zero, so that at most as much is lost of a value (its third term is that small
// from 2^-109 down).
//
// Layouts in LDS (a word is 16 bytes: eight bf16 values).  For rows along the reduced axis [row][word], for a reduced
// axis across the rows [step along it][word of eight columns], which the transposing reads turn.  Words are permuted inside
// a row by exclusive-or, so that neither the stores nor the reads of a wave meet in a bank.
#pragma once

#include <type_traits>

#include "impl.h"
#include "rows.h"

namespace mpnn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef short shortx4 __attribute__((ext_vector_type(4)));

struct Micro {};                             // values in 4 bits: 16 bytes of codes and a scale byte for 32 columns
constexpr int kMicroGroup = 32;

constexpr float kLarge = 0x1p48f;            // sums of products of smaller values do not overflow

template <class T> constexpr int kTerms = std::is_same<T, float>::value ? 3 : 1;

__device__ __forceinline__ float micro_step(uint32_t byte) { return __uint_as_float(byte == 255 ? 0x7fc00000u : byte << 23); }

// Eight neighbouring values of a row as they are loaded.
template <class T> struct Word;
template <> struct Word<float> {
    float v[8];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    }
    __device__ __forceinline__ void load(const float *p) { __builtin_memcpy(v, p, 32); }
    __device__ __forceinline__ void load(const float *p, int in) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < in ? p[j] : 0.0f;
    }
    __device__ __forceinline__ void keep(int in) {       // the first `in` values, zeros after them
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < in ? v[j] : 0.0f;
    }
    __device__ __forceinline__ float at(int j) const { return v[j]; }
    __device__ __forceinline__ void terms(uint4 (&w)[3], float &largest) const {
        float a[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[j] = v[j];
            largest = fmaxf(largest, fabsf(a[j]));
        }
#pragma unroll
        for (int t = 0; t < 3; ++t) {
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(floatx2{a[2 * j], a[2 * j + 1]}, bf16x2));
                if (t < 2) {
                    a[2 * j] -= __uint_as_float(h[j] << 16);
                    a[2 * j + 1] -= __uint_as_float(h[j] & 0xffff0000u);
                }
            }
            w[t] = make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
};
typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));
template <> struct Word<bf16> {
    uintx4 v;
    __device__ __forceinline__ void clear() { v = (uintx4)(0u); }
    __device__ __forceinline__ void load(const bf16 *p) { __builtin_memcpy(&v, p, 16); }
    __device__ __forceinline__ void load(const bf16 *p, int in) {
        const uint16_t *u = reinterpret_cast<const uint16_t *>(p);
        uint32_t s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = j < in ? (uint32_t)u[j] : 0u;
        v = (uintx4){s[0] | s[1] << 16, s[2] | s[3] << 16, s[4] | s[5] << 16, s[6] | s[7] << 16};
    }
    __device__ __forceinline__ void keep(int in) {
        const auto mask = [&](int j) { return (2 * j < in ? 0xffffu : 0u) | (2 * j + 1 < in ? 0xffff0000u : 0u); };
        v &= (uintx4){mask(0), mask(1), mask(2), mask(3)};
    }
    __device__ __forceinline__ float at(int j) const { return __uint_as_float(j & 1 ? v[j >> 1] & 0xffff0000u : v[j >> 1] << 16); }
    __device__ __forceinline__ void terms(uint4 (&w)[1], float &) const { w[0] = make_uint4(v[0], v[1], v[2], v[3]); }
};
template <> struct Word<Micro> {
    uint32_t v;         // eight codes, the first in the low bits
    uint8_t scale;
    __device__ __forceinline__ void clear() {
        v = 0;
        scale = 127;
    }
    __device__ __forceinline__ void terms(uint4 (&w)[1], float &largest) const {
        const float s = micro_step(scale);
        largest = fmaxf(largest, 8.0f * s);
        const auto two = [&](auto k) { return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, k())); };
        w[0] = make_uint4(two(std::integral_constant<int, 0>{}), two(std::integral_constant<int, 1>{}),
                          two(std::integral_constant<int, 2>{}), two(std::integral_constant<int, 3>{}));
    }
};

// Rows of values, `ld` apart; of 4-bit codes, `groups` groups a row.
template <class T> struct RowsOf {
    const T *p;
    int64_t ld;
    struct Row {
        const T *p;
    };
    __device__ __forceinline__ Row row(int64_t i) const { return {p + i * ld}; }
    // a word that is all the row's
    __device__ __forceinline__ static void load(Word<T> &w, const Row &r, int c) { w.load(r.p + c); }
    // the word at column c of a row that has `width` of them (zeros past the end), without a condition beside the load: eight
    // further rows come after this one, so that what is read past its end is of theirs (zeros alone where not `any`)
    __device__ __forceinline__ static void load_over(Word<T> &w, const Row &r, int c, int width, bool any = true) {
        w.load(r.p + min(c, width - 1));
        w.keep(any ? width - c : 0);
    }
    // the same for any row
    __device__ __forceinline__ static void load(Word<T> &w, const Row &r, int c, int width) {
        const int in = width - c;
        if (in >= 8) w.load(r.p + c);
        else w.load(r.p + c, in);
    }
    __device__ __forceinline__ float at(int64_t i, int c) const { return to_f32(p[i * ld + c]); }
};
template <> struct RowsOf<Micro> {
    const uint8_t *codes, *scales;
    int64_t groups;
    struct Row {
        const uint8_t *codes, *scales;
    };
    __device__ __forceinline__ Row row(int64_t i) const { return {codes + i * groups * (kMicroGroup / 2), scales + i * groups}; }
    __device__ __forceinline__ static void load(Word<Micro> &w, const Row &r, int c, int width) {
        if (c >= width) return w.clear();
        load(w, r, c);
    }
    __device__ __forceinline__ static void load_over(Word<Micro> &w, const Row &r, int c, int width) { load(w, r, c, width); }
    __device__ __forceinline__ static void load(Word<Micro> &w, const Row &r, int c) {
        __builtin_memcpy(&w.v, r.codes + c / 2, 4);
        w.scale = r.scales[c / kMicroGroup];
    }
    __device__ __forceinline__ float at(int64_t i, int c) const {
        const Row r = row(i);
        const uint32_t code = r.codes[c / 2] >> 4 * (c & 1) & 15, m = code & 7;
        const float v = m < 2 ? 0.5f * m : __uint_as_float(((m >> 1) + 126) << 23 | (m & 1) << 22);
        return (code & 8 ? -v : v) * micro_step(r.scales[c / kMicroGroup]);
    }
};

// A tile in LDS of `ROWS` rows with WORDS words of the reduced axis each (4 or 8).
template <int TERMS, int ROWS, int WORDS> struct Along {
    static constexpr int kWords = TERMS * ROWS * WORDS;
    // a row's words are permuted by the bits of the row that its 16 neighbours in a read do not share a bank by
    __device__ __forceinline__ static int slot(int row, int word) {
        return row * WORDS + (WORDS == 8 ? word ^ (row >> 1 & 7) : word ^ (row >> 2 & 3));
    }
    __device__ __forceinline__ static void store(uint4 *lds, int row, int word, const uint4 (&w)[TERMS]) {
#pragma unroll
        for (int t = 0; t < TERMS; ++t) lds[t * ROWS * WORDS + slot(row, word)] = w[t];
    }
    // the operand of 32 rows from `first` at step s (16 values of the reduced axis)
    __device__ __forceinline__ static bf16x8 read(const uint4 *lds, int t, int first, int s, int lane) {
        return __builtin_bit_cast(bf16x8, lds[t * ROWS * WORDS + slot(first + (lane & 31), 2 * s + (lane >> 5))]);
    }
};

// The same with the reduced axis across the rows: 8 WORDS of its steps, COLUMNS columns each.
template <int TERMS, int COLUMNS, int WORDS> struct Across {
    static constexpr int kWords = TERMS * COLUMNS * WORDS;
    static constexpr int kWide = COLUMNS / 8;      // words of a step
    // pairs of words (32 bytes, what the lanes of a transposing read take together) are permuted by the step
    __device__ __forceinline__ static int slot(int step, int word) { return step * kWide + (word ^ (step & (kWide / 2 - 1) & 7) * 2); }
    __device__ __forceinline__ static void store(uint4 *lds, int step, int word, const uint4 (&w)[TERMS]) {
#pragma unroll
        for (int t = 0; t < TERMS; ++t) lds[t * COLUMNS * WORDS + slot(step, word)] = w[t];
    }
    // Lane i of 16 names four columns of step i / 4 and gets column i of four steps.
    __device__ __forceinline__ static bf16x8 read(const uint4 *lds, int t, int first, int s, int lane) {
        const int i = lane & 15, step = 16 * s + 8 * (lane >> 5) + i / 4, word = (first + (lane & 16)) / 8 + (i >> 1 & 1);
        typedef __attribute__((address_space(3))) shortx4 *Ptr;
        const auto four = [&](int k) {
            const char *p = reinterpret_cast<const char *>(lds + t * COLUMNS * WORDS + slot(k, word)) + (i & 1) * 8;
            return __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(p));
        };
        const shortx4 a = four(step), b = four(step + 4);
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// Tiles of 256 columns whose steps come to LDS two at a time without passing through registers (64 lanes, a word each, end up
// one after another): the odd step of a pair has its groups of four words swapped, and pairs are 128 bytes further apart than
// their length, so that four steps of a transposing read lie in different banks, at addresses that differ by constants.
struct Pairs {
    static constexpr int kPair = 2 * 32 + 8;                            // words
    static constexpr int kWords = 16 * kPair;                           // of a stage of 32 steps
    __device__ __forceinline__ static int slot(int step, int word) { return (step >> 1) * kPair + (step & 1) * 32 + (word ^ (step & 1) * 4); }
    // of the pair's words the one that a lane brings: its step of the two, and its word
    __device__ __forceinline__ static int step_of(int lane) { return lane >> 5; }
    __device__ __forceinline__ static int word_of(int lane) { return (lane & 31) ^ (lane >> 5) * 4; }
    int even, odd;          // byte offsets of the lane's reads of the first and the second 32 columns
    __device__ __forceinline__ explicit Pairs(int lane) {
        const int i = lane & 15, step = 8 * (lane >> 5) + i / 4, word = (lane & 16) / 8 + (i >> 1 & 1), low = (i & 1) * 8;
        even = slot(step, word) * 16 + low;
        odd = slot(step, word + 4) * 16 + low;
    }
    // the operand of 32 columns from 32 i on at step s (16 steps along the reduced axis)
    __device__ __forceinline__ bf16x8 read(const uint4 *lds, int i, int s) const {
        typedef __attribute__((address_space(3))) shortx4 *Ptr;
        const char *p = reinterpret_cast<const char *>(lds) + (i & 1 ? odd : even) + (i >> 1) * 128 + s * (8 * kPair * 16);
        const shortx4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)p), b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(p + 2 * kPair * 16));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// acc[i][j] += P_i^T Q_j over the WORDS / 2 steps of a stage, P columns of the result and Q its rows: smallest terms first.
template <class P, class Q, int TP, int TQ, int MT, int NT, int WORDS>
__device__ __forceinline__ void multiply(const uint4 *p, const uint4 *q, int pfirst, int qfirst, int lane, floatx16 (&acc)[MT][NT]) {
#pragma unroll
    for (int s = 0; s < WORDS / 2; ++s) {
        bf16x8 a[TP][MT], b[TQ][NT];
#pragma unroll
        for (int t = 0; t < TP; ++t)
#pragma unroll
            for (int i = 0; i < MT; ++i) a[t][i] = P::read(p, t, pfirst + 32 * i, s, lane);
#pragma unroll
        for (int t = 0; t < TQ; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j) b[t][j] = Q::read(q, t, qfirst + 32 * j, s, lane);
#pragma unroll
        for (int sum = 2; sum >= 0; --sum)
#pragma unroll
            for (int u = 0; u < TP; ++u) {
                const int v = sum - u;
                if (v < 0 || v >= TQ) continue;
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[u][i], b[v][j], acc[i][j], 0, 0, 0);
            }
    }
}

// 16 bytes that are not read again soon.
template <class T> __device__ __forceinline__ void store_past(T *p, const Chunk<T> &v) {
    typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
    __builtin_nontemporal_store(__builtin_bit_cast(Words, v), reinterpret_cast<Words *>(p));
}

// A wave's results (32 MT columns from col0, 32 NT rows from row0) by way of LDS, 32 rows of 128 bytes at once, so that lines are
// stored whole, and past L2 where rows are whole lines (279,184 rows 32 -> 512 bf16 55 us, by L2 72).  Others' parts of lines have
// to meet in L2 (32 -> 463 bf16 130 us, past it 217; 128,000 rows 128 -> 312 bf16 38 and 53; fp32 98 and 113).
// mine: the wave's kStoreBytes of LDS; bias(c): what is added to four columns from c on; act(v) then is the result.
constexpr int kStorePitch = 128 + 16, kStoreBytes = 32 * kStorePitch;
template <bool PAST, class Y, int MT, int NT, class B, class F>
__device__ __forceinline__ void store_lines_to(char *mine, const floatx16 (&acc)[MT][NT], int lane, Y *y, int64_t ld, int64_t row0, int64_t rows,
                                               int col0, int columns, B bias, F act) {
    constexpr int V = 16 / sizeof(Y), GROUPS = 8 * V / 32;       // columns a lane; groups of 32 columns a line
#pragma unroll
    for (int i = 0; i < MT; i += GROUPS) {
        const int c = col0 + i * 32 + lane % 8 * V, in = columns - c;
        Chunk<float, 4> b[GROUPS][4];
#pragma unroll
        for (int u = 0; u < GROUPS; ++u)
#pragma unroll
            for (int g = 0; g < 4; ++g) b[u][g] = bias(col0 + (i + u) * 32 + 8 * g + 4 * (lane >> 5));
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int u = 0; u < GROUPS; ++u)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    Chunk<Y, 4> o;
#pragma unroll
                    for (int r = 0; r < 4; ++r) o.v[r] = from_f32<Y>(act(acc[i + u][j][4 * g + r] + b[u][g].v[r]));
                    __builtin_memcpy(__builtin_assume_aligned(mine + (lane & 31) * kStorePitch + (u * 32 + 8 * g + 4 * (lane >> 5)) * sizeof(Y), 4 * sizeof(Y)), &o,
                                     sizeof o);
                }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int r = 0; r < 32; r += 8) {
                const int64_t row = row0 + j * 32 + r + lane / 8;
                Chunk<Y> o;
                __builtin_memcpy(&o, __builtin_assume_aligned(mine + (r + lane / 8) * kStorePitch + lane % 8 * 16, 16), 16);
                if (row < rows && in >= V) {
                    if constexpr (PAST) store_past(y + row * ld + c, o);
                    else o.store(y + row * ld + c);
                } else if (row < rows && in > 0) {
                    o.store(y + row * ld + c, in);
                }
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}
template <class Y, int MT, int NT, class B, class F>
__device__ __forceinline__ void store_lines(char *mine, const floatx16 (&acc)[MT][NT], int lane, Y *y, int64_t ld, int64_t row0, int64_t rows,
                                            int col0, int columns, B bias, F act) {
    if (ld % (128 / (int)sizeof(Y)) == 0) store_lines_to<true>(mine, acc, lane, y, ld, row0, rows, col0, columns, bias, act);
    else store_lines_to<false>(mine, acc, lane, y, ld, row0, rows, col0, columns, bias, act);
}

// Row tiles of the experts' segments, and of the rows that no expert has (before the first segment and after the last;
// expert < 0), which get zeros.
struct Tile {
    int expert;
    int64_t from, to;       // its rows; from >= to: past the last tile
};
__device__ __forceinline__ int64_t clamped(int32_t v, int64_t low, int64_t n) { return min(max((int64_t)v, low), n); }
// Rows of segment e: an expert's, and then those after the last one's and before the first one's.
__device__ __forceinline__ void segment_of(const int32_t *offsets, int n_experts, int64_t n, int e, int64_t &from, int64_t &to) {
    from = to = 0;
    if (e < n_experts) {
        from = clamped(offsets[e], 0, n);
        to = clamped(offsets[e + 1], from, n);
    } else if (e == n_experts) {
        from = clamped(offsets[n_experts], 0, n);
        to = n;
    } else if (e == n_experts + 1) {
        to = clamped(offsets[0], 0, n);
    }
}
__device__ __forceinline__ Tile find_tile(const int32_t *offsets, int n_experts, int64_t n, int rows, int64_t number) {
    const int lane = threadIdx.x & 63;
    int64_t before = 0;
    for (int base = 0; base < n_experts + 2; base += 64) {
        const int e = base + lane;
        int64_t from, to;
        segment_of(offsets, n_experts, n, e, from, to);
        const int c = (int)((to - from + rows - 1) / rows);
        int s = c;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int a = __shfl_up(s, d);
            if (lane >= d) s += a;
        }
        const uint64_t hit = __ballot(number < before + s);
        if (hit) {
            const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
            const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
            const int64_t first = (int64_t)of((int)from) + (number - (before + of(s) - of(c))) * rows;     // n is below 2^31
            const int64_t last = of((int)to);
            return Tile{base + l < n_experts ? base + l : -1, first, min(last, first + rows)};
        }
        before += __builtin_amdgcn_readlane(s, 63);
    }
    return Tile{-1, 0, 0};
}
// The same for blocks that take many tiles: of each segment its first tile and row, in LDS.
constexpr int kSegments = 1024 + 2;
struct Segments {
    int first[kSegments + 1], start[kSegments];
    // by the first wave; the others see it after a barrier
    __device__ __forceinline__ void fill(const int32_t *offsets, int n_experts, int64_t n, int rows) {
        const int lane = threadIdx.x & 63, segments = n_experts + 2;
        int before = 0;
        for (int base = 0; base < segments; base += 64) {
            int64_t from, to;
            segment_of(offsets, n_experts, n, base + lane, from, to);
            const int c = (int)((to - from + rows - 1) / rows);
            int s = c;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int t = __shfl_up(s, d);
                if (lane >= d) s += t;
            }
            if (base + lane < segments) {
                first[base + lane] = before + s - c;
                start[base + lane] = (int)from;
            }
            before += __builtin_amdgcn_readlane(s, 63);
        }
        if (lane == 0) first[segments] = before;
    }
    __device__ __forceinline__ int64_t tiles(int n_experts) const { return first[n_experts + 2]; }
    __device__ __forceinline__ Tile find(const int32_t *offsets, int n_experts, int64_t n, int rows, int tile) const {
        int low = 0, high = n_experts + 1;         // the last segment whose first tile is at most this one
        while (low < high) {
            const int mid = (low + high + 1) / 2;
            if (first[mid] <= tile) low = mid;
            else high = mid - 1;
        }
        low = __builtin_amdgcn_readfirstlane(low);
        const int64_t from = __builtin_amdgcn_readfirstlane(start[low] + (tile - first[low]) * rows);
        int64_t f, e;
        segment_of(offsets, n_experts, n, low, f, e);
        return Tile{low < n_experts ? low : -1, from, min(e, from + rows)};
    }
};
// The tile that block `block` of a grid of whole eighths takes in a round, or -1: neighbouring tiles on one XCD, and those of a
// round that is not full on all XCDs alike.
__device__ __forceinline__ int64_t tile_in_round(int64_t round, int block, int64_t tiles) {
    const int64_t base = round * gridDim.x;
    const int left = (int)min(tiles - base, (int64_t)gridDim.x), per = (left + kXcds - 1) / kXcds, i = block / kXcds, at = block % kXcds * per + i;
    return left > 0 && i < per && at < left ? base + at : -1;
}
// At most so many row tiles: one short one for each expert that has rows, and for the two outer segments.
inline int64_t row_tiles(int64_t n, int n_experts, int rows) { return n / rows + std::min<int64_t>(n, n_experts) + 2; }

}  // namespace mpnn
