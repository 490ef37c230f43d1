// Weight gradients of one linear layer per expert from its saved input (mpnn_checkpoint_weight_grad):
//   dW_e[o][c] = sum over the rows q of expert e of dy[q][o] x[q][c],  db_e[o] = sum of dy[q][o],
// with x the values that the checkpoint holds: a product whose long axis is the rows.
//
// The rows of an expert are cut into pieces of at most `rows`; a block takes one piece and one BM x 128 tile of dW.  How
// long a piece is follows from the experts being alike: where they and their tiles fill the GPU already none is cut, and
// one that holds most of the rows takes its few blocks' time (65,536 rows 256 -> 512 x 64 bf16: 43 us with equal shares,
// 1,164 us with 95 % in one).  An expert of one piece is written at once, the pieces of the others are added afterwards in their order, so results
// do not depend on the launch.
//
// Operands on the bf16 matrix cores: x is exact in bf16 (7 bits and a power of two).  A bf16 dy is one as it stands;
// an fp32 dy is cut into three bf16 terms of 8 bits each, top, middle and last, which add up to it exactly, so that
// every product is exact and the sums are fp32 as with fp32 products.
//
// 128,000 rows 312 -> 128 x 5 fp32: 51 us and 7 us for the pieces' sums (10 GFLOP, three products each: 0.6 PFLOP/s on the
// matrix cores in the first; the operands are 107 MB, 22 us); bf16 38 us together; 16,384 rows 1024 -> 1024 x 8 bf16: 65 .. 75 us
// by the run (0.46 .. 0.53 PFLOP/s).  A stage of 64 rows costs a wave, with two waves a SIMD: 600 .. 700 cycles to cut and
// store dy in bf16 (1,900 in fp32), 600 for x, 800 for the products (512 are the instructions; fp32 2,100 and 1,536) and 1,000 to get its 17 loads
// issued.  Without the loads the time is the same: it is the issue of vector, LDS and matrix instructions by few waves.
// What is read of memory is 5 TB/s at most, mostly from the L2s.
#include <algorithm>
#include <type_traits>

#include "impl.h"
#include "pieces.h"
#include "rows.h"

namespace mpnn {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));

constexpr int kBK = 64;          // rows per stage: 8 chunks of 8, one matrix-core operand word each
constexpr int kChunks = kBK / 8;

__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Four neighbouring columns of dy in one row.
struct Quad32 {
    float v[4];
    __device__ __forceinline__ float at(int j) const { return v[j]; }
};
struct Quad16 {
    uint32_t v[2];
    __device__ __forceinline__ float at(int j) const { return __uint_as_float(j & 1 ? v[j >> 1] & 0xffff0000u : v[j >> 1] << 16); }
};
template <class T> struct QuadOf;
template <> struct QuadOf<float> { using type = Quad32; };
template <> struct QuadOf<bf16> { using type = Quad16; };

// `last`: the last of the four columns that is there; those past it repeat it (their results are not written).
__device__ __forceinline__ void load_quad(Quad32 &q, const float *p) { __builtin_memcpy(&q, p, sizeof q); }
__device__ __forceinline__ void load_quad(Quad32 &q, const float *p, int last) {
#pragma unroll
    for (int j = 0; j < 4; ++j) q.v[j] = p[min(j, last)];
}
__device__ __forceinline__ void load_quad(Quad16 &q, const bf16 *p) { __builtin_memcpy(&q, p, sizeof q); }
__device__ __forceinline__ void load_quad(Quad16 &q, const bf16 *p, int last) {
    const uint16_t *u = reinterpret_cast<const uint16_t *>(p);
    q.v[0] = (uint32_t)u[0] | (uint32_t)u[min(1, last)] << 16;
    q.v[1] = (uint32_t)u[min(2, last)] | (uint32_t)u[min(3, last)] << 16;
}
__device__ __forceinline__ void clear_quad(Quad32 &q) { q.v[0] = q.v[1] = q.v[2] = q.v[3] = 0.0f; }
__device__ __forceinline__ void clear_quad(Quad16 &q) { q.v[0] = q.v[1] = 0u; }

// Column j of eight rows as the operand words of each term.
__device__ __forceinline__ void column(const Quad16 (&q)[8], int j, uint4 (&w)[1]) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        p[i] = j & 1 ? high_halves(q[2 * i].v[j >> 1], q[2 * i + 1].v[j >> 1]) : low_halves(q[2 * i].v[j >> 1], q[2 * i + 1].v[j >> 1]);
    w[0] = make_uint4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ bool infinite(const Quad16 (&)[8]) { return false; }
__device__ __forceinline__ bool infinite(const Quad32 (&q)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        m = fmaxf(fmaxf(m, fabsf(q[r].v[0])), fabsf(q[r].v[1]));
        m = fmaxf(fmaxf(m, fabsf(q[r].v[2])), fabsf(q[r].v[3]));
    }
    return m == __uint_as_float(0x7f800000u);
}
__device__ __forceinline__ void column(const Quad32 (&q)[8], int j, uint4 (&w)[3]) {
    uint32_t t[3][8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const float v = q[r].v[j];
        const uint32_t top = __float_as_uint(v) & 0xffff0000u;
        const float left = v - __uint_as_float(top);                   // exact: 16 significant bits
        const uint32_t middle = __float_as_uint(left) & 0xffff0000u;
        t[0][r] = top;
        t[1][r] = middle;
        t[2][r] = __float_as_uint(left - __uint_as_float(middle));   // 8 bits: its low half is zero
    }
#pragma unroll
    for (int s = 0; s < 3; ++s)
        w[s] = make_uint4(high_halves(t[s][0], t[s][1]), high_halves(t[s][2], t[s][3]), high_halves(t[s][4], t[s][5]),
                          high_halves(t[s][6], t[s][7]));
}

// Layout.  Both operands have the rows as their slow axis, while a matrix-core operand word holds eight of them for
// one column: a thread loads 4 neighbouring columns of 8 rows, turns them in registers and writes four 16-byte words.
// LDS holds [chunk][position][8 rows].  Column m of a tile of B columns sits at position (m % 4) (B / 4) + m / 4, so
// that neighbouring threads write neighbouring words (no bank conflict), and the operand reads are neighbouring words
// too; the permutation only reorders the tile's results (of 128 columns of x a lane ends up with NT neighbouring ones,
// which it stores together).
// WM x WN waves own 32 MT x 32 NT positions each.
// VEC: quads are loaded whole, at any alignment; the last one of a row is moved back to end with it, and the window of the
// last stage to end with the array (what it holds of other rows is cleared when it is staged).  Otherwise (fewer than kBK
// rows or 4 columns, or a moved quad of two groups) values are loaded one by one, rows and columns past the last repeat it.
template <class T, int MT, int NT, int WM, int WN, bool VEC>
__global__ __launch_bounds__(256, 2) void k_weight_grad(int out, int width, int groups, int n_experts, int64_t n, int64_t rows, int tiles_n,
                                                        int tiles, const int32_t *__restrict__ offsets, const T *__restrict__ dy, int64_t ld,
                                                        const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t slots, float *__restrict__ part, float *__restrict__ dweight,
                                                        float *__restrict__ dbias) {
    constexpr int TERMS = sizeof(T) == 4 ? 3 : 1;
    constexpr int BM = 32 * MT * WM, BN = 32 * NT * WN;
    constexpr int QA = BM / 4, QX = BN / 4, GX = BN / 32;               // quads and groups of columns
    constexpr int XT = (QX * kChunks + 255) / 256, ST = (GX * kBK + 255) / 256;   // x quads and scales per thread
    constexpr bool kAllA = QA * kChunks == 256, kAllX = QX * kChunks % 256 == 0;   // every thread has a quad to stage
    static_assert(BN == 128 && WM * WN == 4 && QA * kChunks <= 256, "four waves, one quad of dy a thread");
    using Quad = typename QuadOf<T>::type;
    __shared__ uint4 A[TERMS][kChunks][BM];
    __shared__ uint4 B[kChunks][BN];
    __shared__ __attribute__((aligned(16))) float steps[2][GX][kBK];
    __shared__ float sums[kChunks][BM];

    // Blocks are dealt to the XCDs in turn: where experts are cut into pieces, give the tiles of one piece (the same rows)
    // to one XCD; with an expert a piece deal each expert's tiles to all of them, since experts differ in length
    // (16,384 rows 1024 -> 1024 x 8 with shares from 4 to 20 %: bf16 111 -> 92 us, fp32 254 -> 177 us).
    const uint32_t number = n > rows ? (uint32_t)xcd_block() : blockIdx.x;
    const int tile = (int)(number % (uint32_t)tiles);
    int turn = (int)(number / (uint32_t)tiles);
    if (n <= rows && n_experts <= 64 && turn < n_experts) turn = expert_in_turn(offsets, n_experts, n, max(1, 256 / tiles), turn);
    const Piece pc = find_piece(offsets, n_experts, n, rows, turn, -1);
    if (pc.expert < 0) return;
    int64_t from, to;
    pieces_of(offsets, pc.expert, n, rows, from, to);
    from += pc.piece * rows;
    to = min(to, from + rows);
    const int o0 = tile / tiles_n * BM, c0 = tile % tiles_n * BN;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int am = tid % QA, ak = tid / QA;                   // dy: column quad, chunk (threads with ak < 8)
    // quads past the last (VEC) or columns past the last repeat it
    const int ac = min(o0 + 4 * am, out - (VEC ? 4 : 1));
    [[maybe_unused]] const int alast = out - 1 - ac;
    const uint32_t abase = ((uint32_t)ak * 8 * (uint32_t)ld + ac) * sizeof(T);      // bytes; ld is at most 2^24
    int xm[XT], xk[XT];
    uint32_t xbase[XT];
    bool x_in[XT];
#pragma unroll
    for (int i = 0; i < XT; ++i) {
        const int t = tid + i * 256;
        xm[i] = t % QX;
        xk[i] = t / QX;
        x_in[i] = kAllX || xk[i] < kChunks;
        if (!x_in[i]) xk[i] = kChunks - 1;                    // loads what another thread does, stores nothing
        xbase[i] = (uint32_t)xk[i] * 8 * (uint32_t)width + min(c0 + 4 * xm[i], width - (VEC ? 4 : 1));
    }

    Quad a[8];
    uint32_t x[XT][8];
    uint8_t scale[ST];
    uint32_t sbase[ST];
#pragma unroll
    for (int i = 0; i < ST; ++i) {
        const int t = min(tid + i * 256, GX * kBK - 1);
        sbase[i] = (uint32_t)(t / GX) * (uint32_t)groups + min(c0 / 32 + t % GX, groups - 1);
    }
    const auto window = [&](int64_t q0) { return VEC ? min(q0, n - kBK) : min(q0, to - 1); };
    // The loads of a stage: its rows from a uniform row address and this thread's distance from it.
    auto fetch = [&](int64_t q0) {
        q0 = window(q0);
        const T *ap = dy + q0 * ld;
        const int8_t *xp = codes + q0 * width;
        if constexpr (VEC) {
            // Each load is a scalar row address and a 32-bit distance, which the empty asm keeps apart: otherwise the additions
            // become one of 64 bits a load and thread (16,384 rows 1024 -> 1024 x 8 bf16 79 -> 74 us).
            uint32_t adist = abase, xdist[XT];
#pragma unroll
            for (int i = 0; i < XT; ++i) xdist[i] = xbase[i];
            if (kAllA || ak < kChunks) {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    asm volatile("" : "+v"(adist));
                    load_quad(a[r], reinterpret_cast<const T *>(reinterpret_cast<const char *>(ap + r * ld) + adist));
                }
            }
#pragma unroll
            for (int i = 0; i < XT; ++i)
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    asm volatile("" : "+v"(xdist[i]));
                    __builtin_memcpy(&x[i][r], xp + r * (int64_t)width + xdist[i], 4);
                }
        } else {
            const int last = (int)min(to - 1 - q0, (int64_t)(kBK - 1));
            if (kAllA || ak < kChunks) {
#pragma unroll
                for (int r = 0; r < 8; ++r) load_quad(a[r], ap + (uint32_t)min(ak * 8 + r, last) * (uint32_t)ld + ac, alast);
            }
#pragma unroll
            for (int i = 0; i < XT; ++i) {
                const int xc = min(c0 + 4 * xm[i], width - 1), xlast = width - 1 - xc;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const uint8_t *u = reinterpret_cast<const uint8_t *>(xp) + (uint32_t)min(xk[i] * 8 + r, last) * (uint32_t)width + xc;
                    x[i][r] = (uint32_t)u[0] | (uint32_t)u[min(1, xlast)] << 8 | (uint32_t)u[min(2, xlast)] << 16 | (uint32_t)u[min(3, xlast)] << 24;
                }
            }
        }
    };
    // The scales go through LDS a stage ahead: [group][row], as steps, 0 for rows that are not this stage's.
    auto fetch_scales = [&](int64_t q0) {
        const int64_t w = window(q0);
        const uint8_t *sp = scales + w * groups;
#pragma unroll
        for (int i = 0; i < ST; ++i) scale[i] = VEC ? sp[sbase[i]] : sp[min((int64_t)sbase[i], (to - w) * groups - 1)];
    };
    auto store_scales = [&](int64_t q0, int buffer) {
#pragma unroll
        for (int i = 0; i < ST; ++i) {
            const int t = min(tid + i * 256, GX * kBK - 1), r = t / GX;
            float step = __uint_as_float(scale[i] == 255 ? 0x7fc00000u : (uint32_t)scale[i] << 23);
            if (q0 + kBK > to) {
                const int64_t q = window(q0) + r;
                if (q < q0 || q >= to) step = 0.0f;
            }
            steps[buffer][t % GX][r] = step;
        }
    };

    floatx16 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = (floatx16)(0.0f);
    float bias[4] = {};
    const int wm = wave / WN, wn = wave % WN;
    if (from < to) {
        fetch_scales(from);
        fetch(from);
        store_scales(from, 0);
        fetch_scales(from + kBK);
    }
    int buffer = 0;
    for (int64_t q0 = from; q0 < to; q0 += kBK) {
        __syncthreads();
        if (q0 + kBK > to) {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int64_t q = window(q0) + ak * 8 + r;
                if (q < q0 || q >= to) clear_quad(a[r]);
            }
        }
        if (kAllA || ak < kChunks) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint4 w[TERMS];
                column(a, j, w);
#pragma unroll
                for (int t = 0; t < TERMS; ++t) A[t][ak][j * QA + am] = w[t];
            }
            if (TERMS > 1 && __any(infinite(a))) {
                // the terms of an infinity after the first are nothing, not the difference of two infinities
                for (int e = 0; e < 32; ++e) {
                    float v = 0.0f;
#pragma unroll
                    for (int f = 0; f < 32; ++f) v = e == f ? a[f >> 2].at(f & 3) : v;
                    if (fabsf(v) == __uint_as_float(0x7f800000u))
#pragma unroll
                        for (int t = 1; t < TERMS; ++t) reinterpret_cast<uint16_t *>(&A[t][ak][(e & 3) * QA + am])[e >> 2] = 0;
                }
            }
            if (c0 == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int r = 0; r < 8; ++r) bias[j] += a[r].at(j);
            }
        }
#pragma unroll
        for (int i = 0; i < XT; ++i) {
            const float4 lo = *reinterpret_cast<const float4 *>(&steps[buffer][xm[i] / 8][xk[i] * 8]);
            const float4 hi = *reinterpret_cast<const float4 *>(&steps[buffer][xm[i] / 8][xk[i] * 8 + 4]);
            const float step[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = __float_as_uint((float)(int8_t)(x[i][r] >> 8 * j) * step[r]);   // exact
                if (x_in[i])
                    B[xk[i]][j * QX + xm[i]] = make_uint4(high_halves(v[0], v[1]), high_halves(v[2], v[3]), high_halves(v[4], v[5]),
                                                          high_halves(v[6], v[7]));
            }
        }
        store_scales(q0 + kBK, buffer ^ 1);
        buffer ^= 1;
        __syncthreads();
        if (q0 + kBK < to) {
            fetch(q0 + kBK);
            fetch_scales(q0 + 2 * kBK);
        }
        bf16x8 af[2][TERMS][MT], bf[2][NT];
        auto operands = [&](int s) {
            const int c = 2 * s + (lane >> 5);
#pragma unroll
            for (int j = 0; j < NT; ++j) bf[s & 1][j] = __builtin_bit_cast(bf16x8, B[c][(wn * NT + j) * 32 + (lane & 31)]);
#pragma unroll
            for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
                for (int i = 0; i < MT; ++i) af[s & 1][t][i] = __builtin_bit_cast(bf16x8, A[t][c][(wm * MT + i) * 32 + (lane & 31)]);
        };
        // operands are read a step ahead, and a wave that multiplies goes before one that stages (128,000 rows 312 -> 128 x 5
        // fp32 66 -> 63 us; 16,384 rows 1024 -> 1024 x 8 fp32 153 -> 147 us, bf16 74 and 75 us)
        operands(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < kChunks / 2; ++s) {
            if (s + 1 < kChunks / 2) operands(s + 1);
#pragma unroll
            for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[s & 1][t][i], bf[s & 1][j], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
    }

    const int64_t matrix = (int64_t)out * width;
    const bool whole = pc.pieces == 1;
    if (!whole && pc.slot + pc.piece >= slots) return;   // offsets that do not ascend name more pieces than there are
    float *to_w = whole ? dweight + pc.expert * matrix : part + (int64_t)(pc.slot + pc.piece) * slot_size(matrix + out);
    float *to_b = whole ? (dbias ? dbias + (int64_t)pc.expert * out : nullptr) : to_w + matrix;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int pm = (wm * MT + i) * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
            const int oq = o0 + 4 * (pm % QA), o = (VEC ? min(oq, out - 4) : oq) + pm / QA;
            if (oq >= out || o >= out) continue;
            const int cl = c0 + 4 * (lane & 31) + wn * NT;          // this lane's NT columns
            float *row = to_w + (int64_t)o * width;
            if (!VEC || cl + NT > width || (cl + NT > width - 4 && width % 4)) {
                // at the row's end: the last quad was moved back to end with it
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int cq = (cl + j) / 4 * 4, c = (VEC ? min(cq, width - 4) : cq) + (cl + j) % 4;
                    if (cq < width && c < width) row[c] = acc[i][j][r];
                }
            } else {
                float v[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) v[j] = acc[i][j][r];
                __builtin_memcpy(row + cl, v, sizeof v);
            }
        }
    if (c0 == 0 && to_b) {
        if (kAllA || ak < kChunks)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (o0 + 4 * am < out && ac + j >= o0) sums[ak][ac - o0 + j] = bias[j];   // a moved quad begins in the tile before
        __syncthreads();
        if (tid < BM && o0 + tid < out) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < kChunks; ++k) s += sums[k][tid];
            to_b[o0 + tid] = s;
        }
    }
}

// The pieces of each expert that has several, added in a fixed order: a thread takes four values of every fourth piece,
// then the four sums of a value are added.
__global__ __launch_bounds__(256) void k_weight_grad_sum(int n_experts, int64_t n, int64_t rows, int64_t slots, int64_t matrix, int out,
                                                         const int32_t *__restrict__ offsets, const float *__restrict__ part,
                                                         float *__restrict__ dweight, float *__restrict__ dbias) {
    __shared__ float4 sums[4][64];
    const int e = blockIdx.y, lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const Piece pc = find_piece(offsets, n_experts, n, rows, 0, e);
    if (pc.pieces <= 1 || pc.slot + (int64_t)pc.pieces > slots) return;
    const int64_t stride = slot_size(matrix + out);
    for (int64_t from = (int64_t)blockIdx.x * 256; from < stride; from += (int64_t)gridDim.x * 256) {
        const int64_t v = from + lane * 4;
        const float *p = part + (int64_t)pc.slot * stride + min(v, stride - 4);
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int i = slice; i < pc.pieces; i += 4) {
            const float4 t = *reinterpret_cast<const float4 *>(p + i * stride);
            s.x += t.x; s.y += t.y; s.z += t.z; s.w += t.w;
        }
        __syncthreads();
        sums[slice][lane] = s;
        __syncthreads();
        if (slice != 0) continue;
#pragma unroll
        for (int k = 1; k < 4; ++k) {
            const float4 t = sums[k][lane];
            s.x += t.x; s.y += t.y; s.z += t.z; s.w += t.w;
        }
        const float o[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (v + j < matrix) dweight[e * matrix + v + j] = o[j];
            else if (v + j < matrix + out && dbias) dbias[(int64_t)e * out + (v + j - matrix)] = o[j];
        }
    }
}

template <class T, int MT, int NT, int WM, int WN>
Status launch(Context &cx, int64_t n, int out, int width, int n_experts, const int32_t *offsets, const T *dy, int64_t ld,
              const int8_t *codes, const uint8_t *scales, float *dweight, float *dbias) {
    constexpr int BM = 32 * MT * WM, BN = 32 * NT * WN;
    const int tiles_n = (width + BN - 1) / BN, tiles = tiles_n * ((out + BM - 1) / BM);
    // The blocks that run at once, two a CU of the widest tile, three of the narrower ones; an expert's last piece may be
    // short, so a few pieces less than fill them.  (128,000 rows 312 -> 128 x 5 fp32 with one, two and three blocks a CU:
    // 86, 65 and 79 us; 2,000,000 rows 108 -> 64 bf16: 179, 119 and 109 us.)
    constexpr int kResident = BM > 64 ? 512 : 768;
    const int64_t want = std::max<int64_t>(1, kResident / tiles - n_experts);
    const int64_t rows = std::max<int64_t>(512, ((n + want - 1) / want + kBK - 1) / kBK * kBK);
    const int64_t pieces = n / rows + n_experts;              // at most; an expert of several pieces has more than `rows` rows
    const int64_t matrix = (int64_t)out * width, slots = n > rows ? 2 * (n / rows) : 0;   // an expert of p > 1 pieces fills p / 2 whole ones
    void *ws = nullptr;
    MPNN_TRY(cx.rows_scratch(sizeof(float) * (size_t)(slots * slot_size(matrix + out)), &ws));
    float *const part = static_cast<float *>(ws);
    const bool vec = n >= kBK && out >= 4 && width >= 4 && (width % 32 == 0 || width % 32 > 3);
    auto *kernel = vec ? k_weight_grad<T, MT, NT, WM, WN, true> : k_weight_grad<T, MT, NT, WM, WN, false>;
    kernel<<<grid_xcd(pieces * tiles, 1), 256, 0, cx.stream>>>(out, width, (width + 31) / 32, n_experts, n, rows, tiles_n, tiles, offsets,
                                                               dy, ld, codes, scales, slots, part, dweight, dbias);
    MPNN_HIP(hipGetLastError());
    return slots ? join_pieces(cx, n_experts, n, rows, slots, matrix, out, offsets, part, dweight, dbias) : Status::ok();
}

template <class T>
Status weight_grad_t(Context &cx, int64_t n, int out, int width, int n_experts, const int32_t *offsets, const void *dy, int64_t ld,
                     const int8_t *codes, const uint8_t *scales, float *dweight, float *dbias) {
    // tiles of 32, 64 or 128 x 128: of the wider ones tried, 64 x 192, 64 x 320 and 64 x 128 were slower at 128,000 rows
    // 312 -> 128 (81, 78, 86 us, 70 us with 128 x 128; bf16 52, 49, 49 and 44 us)
    constexpr std::integral_constant<int, 1> one{};
    constexpr std::integral_constant<int, 2> two{};
    constexpr std::integral_constant<int, 4> four{};
    auto tile = [&](auto mt, auto nt, auto wm, auto wn) -> Status {
        return launch<T, mt(), nt(), wm(), wn()>(cx, n, out, width, n_experts, offsets, (const T *)dy, ld, codes, scales, dweight, dbias);
    };
    if (out <= 32) return tile(one, one, one, four);
    if (out <= 64) return tile(one, two, two, two);
    return tile(two, two, two, two);
}

}  // namespace

Status join_pieces(Context &cx, int n_experts, int64_t n, int64_t rows, int64_t slots, int64_t matrix, int out, const int32_t *offsets,
                   const float *part, float *dweight, float *dbias) {
    // about 8,192 blocks: most experts have one piece, and a block of theirs ends at once (64 experts of 2048 x 1024: 390 us
    // with a block for every 256 values)
    const unsigned most = (unsigned)std::max(1, 8192 / n_experts);
    k_weight_grad_sum<<<dim3(std::min(grid_for(slot_size(matrix + out) / 4, 64), most), n_experts), 256, 0, cx.stream>>>(
        n_experts, n, rows, slots, matrix, out, offsets, part, dweight, dbias);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

Status weight_grad(Context &cx, int dtype, int64_t n, int out, int width, int n_experts, const int32_t *offsets, const void *dy,
                   int64_t ld, const int8_t *codes, const uint8_t *scales, float *dweight, float *dbias) {
    return dtype == MPNN_BF16 ? weight_grad_t<bf16>(cx, n, out, width, n_experts, offsets, dy, ld, codes, scales, dweight, dbias)
                              : weight_grad_t<float>(cx, n, out, width, n_experts, offsets, dy, ld, codes, scales, dweight, dbias);
}

}  // namespace mpnn
