// Norms before and after a block, fused with the block's gate and residual scale (mpnn_norm_residual*).
//   r = x + scale * sigma(gate) * N_post(block),  h = N_pre(r),
//   N(v) = (v - mean) / sqrt(mean((v - mean)^2) + eps) * weight + bias   (rms: without the mean)
// h comes from the unrounded r.  The reverse pass takes the statistics again from the rows it reads anyway, so the
// forward pass stores none.
//
// One pass over the rows: G lanes hold a row in registers, CH 16-byte chunks each (G = 8 .. 64 inside a wave, or
// waves of one block for wide rows), so that means and mean squares are taken from registers (the mean first, then
// the squares about it) and every array is read and written once.  Groups walk over the rows with their columns'
// weights in registers, and in the reverse pass with their columns' sums; the sums of all groups are added at the end
// in a fixed order.
//
// Bound by HBM: forward of 400,002 x 128 fp32 187 us (1.02 GB, 5.5 TB/s), reverse of 128,000 x 312 fp32 with a gate a row
// 184 us (959 MB, 5.2 TB/s), of 8,192 x 4,096 bf16 125 us (537 MB, 4.3 TB/s: 115 us and 8 us for 33 MB of blocks' sums,
// which rows this wide cost).  One row alone takes 3 us.
#include <algorithm>
#include <type_traits>

#include "impl.h"
#include "rows.h"

namespace mpnn {

namespace {

struct NormArgs {
    int64_t n;
    int width, layer;
    int gate_width;        // 0: no gate
    float eps, inv_width;
    const float *post_weight, *post_bias, *scale, *pre_weight, *pre_bias;
};

// 1 / (1 + 2^(-g log2 e)).  The exponent's rounding is off by |g| 2^-24 relative, which s (1 - s) |g| < 0.23 keeps
// below half an ulp of 1 in the result; infinities and NaN come out as the formula has them.
__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * g)); }

// sigma(g) and sigma(-g) = 1 - sigma(g) for the gate's derivative, with full accuracy at both ends: the difference loses a
// large gate's (1 % at 12, all of it from 17.4 on), so there it is 2^(-g log2 e) sigma(g).  Off by |g| 2^-24 relative from the
// exponent's rounding and a few units from the rest.  (From 2^(-|g| log2 e) for both signs: 24,000 x 2,600 bf16 gradient 228 us,
// 222 us this way, which takes fewer registers.)
__device__ __forceinline__ void sigmoids(float g, float &s, float &rest) {
    const float a = __builtin_amdgcn_exp2f(-1.44269504f * g);
    s = __builtin_amdgcn_rcpf(1.0f + a);
    rest = g >= 0.0f ? a * s : 1.0f - s;
}

// What a launch is compiled for.  kAny: some of the optional arrays may be missing.  The others: every array there, and
// the gate of that kind, in fewer registers, so with more waves (gradient of 8,192 x 4,096 bf16: 242 us with the
// conditions, 140 us without).
enum Mode { kAny = -1, kNoGate = 0, kRowGate = 1, kElementGate = 2 };

// A row's place in the block's registers: W values a chunk, CH chunks a lane, G lanes.  The chunk that would pass the
// row's end is moved back to end with it, and lanes past the last chunk repeat it, so that every access is a whole chunk
// of the row; the values that another lane has too (the first `skip` of a lane's last chunk: every chunk before it lies
// inside the row) count in no sum, and what is stored of them is what their owner stores.  EXACT: there are none.
template <class T, int W, int G, int CH, bool EXACT>
struct Lanes {
    static constexpr int E = CH * W;                       // values of a row per lane
    static constexpr int kThreads = G > 64 ? G : 256, kGroups = kThreads / G;   // several waves a row: one row a block
    static constexpr int kWaves = G / 64;                  // waves of a row (0: part of one)
    int lane, group;
    int width;
    int column[CH];
    int skip;
    __device__ __forceinline__ Lanes(int w) : lane(threadIdx.x % G), group(threadIdx.x / G), width(w) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int at = (c * G + lane) * W;
            column[c] = EXACT ? at : min(at, width - W);
            skip = at - column[c];
        }
    }
    // A row as it is in memory.
    struct Raw {
        Chunk<T, W> c[CH];
    };
    __device__ __forceinline__ void fetch(Raw &t, const T *row) const {
#pragma unroll
        for (int c = 0; c < CH; ++c) t.c[c].load(row + column[c]);
    }
    __device__ __forceinline__ void values(float (&v)[E], const Raw &t) const {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < W; ++j) v[c * W + j] = to_f32(t.c[c].v[j]);
    }
    __device__ __forceinline__ void store(T *row, const float (&v)[E]) const {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            Chunk<T, W> t;
#pragma unroll
            for (int j = 0; j < W; ++j) t.v[j] = from_f32<T>(v[c * W + j]);
            t.store(row + column[c]);
        }
    }
    // a vector's values of this lane's columns
    __device__ __forceinline__ void vector(float (&v)[E], const float *p, float otherwise) const {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = otherwise;
        if (!p) return;
#pragma unroll
        for (int c = 0; c < CH; ++c) __builtin_memcpy(&v[c * W], p + column[c], W * sizeof(float));
    }
    // one value's share of a sum: the value or nothing, not a product with 0, which of an infinity is NaN
    __device__ __forceinline__ float share(float v, int e) const { return EXACT || e < E - W || e - (E - W) >= skip ? v : 0.0f; }
    // The reverse pass keeps its vectors in LDS (zeros past the width), whose registers its sums need.  The offset is
    // zero, but not to the compiler, which would move the reads out of the row loop, into registers.
    static constexpr int kSlots = G * E;
    __device__ __forceinline__ void keep(float *sh, const float *p, float otherwise, const float *factor) const {
        for (int c = threadIdx.x; c < width; c += kThreads) sh[c] = (p ? p[c] : otherwise) * (factor ? factor[c] : 1.0f);
    }
    __device__ __forceinline__ void kept(float (&v)[E], const float *sh) const {
        int z = 0;
        asm volatile("" : "+v"(z));
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if constexpr (EXACT && W % 4 == 0) {
#pragma unroll
                for (int j = 0; j < W; j += 4) {
                    const float4 t = *reinterpret_cast<const float4 *>(sh + column[c] + j + z);
                    v[c * W + j] = t.x; v[c * W + j + 1] = t.y; v[c * W + j + 2] = t.z; v[c * W + j + 3] = t.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) v[c * W + j] = sh[column[c] + j + z];
            }
        }
    }
    // sums over the row's lanes, the same bits in each
    template <int N, int M> __device__ __forceinline__ void sums(float (&s)[N], float (&sh)[2][M], int &turn) const {
        if constexpr (kWaves <= 1) {
#pragma unroll
            for (int q = 0; q < N; ++q) s[q] = lanes_sum<G>(s[q]);
        } else {
            static_assert(M >= N * kWaves, "room for the waves' sums");
            // the waves' sums through LDS; two buffers in turn, so that one barrier a sum is enough
            float *b = sh[turn];
            turn ^= 1;
#pragma unroll
            for (int q = 0; q < N; ++q) {
                s[q] = lanes_sum<64>(s[q]);
                if ((threadIdx.x & 63) == 0) b[q * kWaves + (lane >> 6)] = s[q];
            }
            __syncthreads();
#pragma unroll
            for (int q = 0; q < N; ++q) {
                s[q] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) s[q] += b[q * kWaves + w];
            }
        }
    }
    // v becomes its normed values; returns one over the root
    template <int M> __device__ __forceinline__ float normalise(float (&v)[E], bool layer, float eps, float inv_width, float (&sh)[2][M],
                                                                int &turn) const {
        if (layer) {
            float m[1] = {0.0f};
#pragma unroll
            for (int e = 0; e < E; ++e) m[0] += share(v[e], e);
            sums(m, sh, turn);
            m[0] *= inv_width;
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] -= m[0];
        }
        float q[1] = {0.0f};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float mine = share(v[e], e);
            q[0] = fmaf(mine, mine, q[0]);
        }
        sums(q, sh, turn);
        const float inv = rsqrtf(q[0] * inv_width + eps);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= inv;
        return inv;
    }
};

// In a group of several waves all waves of the block take the same row, so barriers inside the row loop are uniform.
// r may be x, so neither is __restrict__: where a row does not fill its lanes, another wave stores columns that this one
// loads too, and the loads have to stay before the barriers of the block's norm, which that store comes after.  (Rows without
// a block are stored as they were loaded.)
template <class T, int W, int G, int CH, int MODE, bool EXACT>
__global__ __launch_bounds__((Lanes<T, W, G, CH, false>::kThreads)) void k_norm_residual(NormArgs a, const T *x, int64_t ldx,
                                                                             const T *__restrict__ block, int64_t ldb,
                                                                             const T *__restrict__ gate, int64_t ldg, T *r,
                                                                             T *__restrict__ h) {
    constexpr bool FULL = MODE != kAny;
    using L = Lanes<T, W, G, CH, EXACT>;
    constexpr int E = L::E;
    __shared__ float sh[2][L::kWaves > 1 ? L::kWaves : 1];
    int turn = 0;
    const L at(a.width);
    const int gate_kind = FULL ? (int)MODE : a.gate_width > 1 ? (int)kElementGate : a.gate_width;   // widths of 1 count as one gate a row
    const bool has_block = FULL || block, has_r = FULL || r, has_h = FULL || h;
    float pw[E], pb[E], qw[E], qb[E];
    if (has_block) {
        float sc[E];
        at.vector(pw, a.post_weight, 1.0f);
        at.vector(pb, a.post_bias, 0.0f);
        at.vector(sc, a.scale, 1.0f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            pw[e] *= sc[e];
            pb[e] *= sc[e];
        }
    }
    if (has_h) {
        at.vector(qw, a.pre_weight, 1.0f);
        at.vector(qb, a.pre_bias, 0.0f);
    }
    auto normalise = [&](float (&v)[E]) { at.normalise(v, a.layer, a.eps, a.inv_width, sh, turn); };
    // the next row's loads are under way while a row is worked on
    typename L::Raw rx, rb, rg;
    T row_gate{};
    auto fetch = [&](int64_t i) {
        at.fetch(rx, x + i * ldx);
        if (has_block) {
            at.fetch(rb, block + i * ldb);
            if (gate_kind == kElementGate) at.fetch(rg, gate + i * ldg);
            else if (gate_kind == kRowGate) row_gate = gate[i * ldg];
        }
    };
    const int64_t stride = (int64_t)gridDim.x * L::kGroups;
    int64_t i = (int64_t)blockIdx.x * L::kGroups + at.group;
    if (i < a.n) fetch(i);
    for (; i < a.n; i += stride) {
        float v[E], b[E], g[E];
        at.values(v, rx);
        if (has_block) {
            at.values(b, rb);
            if (gate_kind == kElementGate) at.values(g, rg);
            else g[0] = to_f32(row_gate);
        }
        if (i + stride < a.n) fetch(i + stride);
        if (has_block) {
            normalise(b);
            if (gate_kind == kElementGate) {
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = fmaf(sigmoid(g[e]), fmaf(b[e], pw[e], pb[e]), v[e]);
            } else {
                const float s = gate_kind == kRowGate ? sigmoid(g[0]) : 1.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = fmaf(s, fmaf(b[e], pw[e], pb[e]), v[e]);
            }
        }
        if (has_r) at.store(r + i * a.width, v);
        if (has_h) {
            normalise(v);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = fmaf(v[e], qw[e], qb[e]);
            at.store(h + i * a.width, v);
        }
    }
}

// Gradients of the rows.  total = dr + N_pre'(dh), dx = total, and with u = N_post(block):
//   dgate = total scale u sigma'(gate), du = total scale sigma(gate), dblock = N_post'(du),
//   N'(d) = inv (a - mean(a) - hat mean(a hat)), a = d weight   (rms: without mean(a))
// and of the vectors, summed over the group's rows:
//   post weight: du hat_b, post bias: du, scale: total sigma(gate) u, pre weight: dh hat_r, pre bias: dh
// The first three are combinations of two sums, of total sigma hat_b (P) and of total sigma (Q), by the column's own
// values: scale P, scale Q and weight P + bias Q.
template <class T, int W, int G, int CH, int MODE, bool EXACT>
__global__ __launch_bounds__((Lanes<T, W, G, CH, false>::kThreads)) void k_norm_residual_back(NormArgs a, const T *dr, const T *__restrict__ dh,
                                                                                  const T *__restrict__ r, int64_t ldr,
                                                                                  const T *__restrict__ block, int64_t ldb,
                                                                                  const T *__restrict__ gate, int64_t ldg, T *dx,
                                                                                  T *__restrict__ dblock, T *__restrict__ dgate,
                                                                                  float *__restrict__ part) {
    constexpr bool FULL = MODE != kAny;
    using L = Lanes<T, W, G, CH, EXACT>;
    constexpr int E = L::E;
    constexpr int kShared = L::kWaves > 1 ? 3 * L::kWaves : 1;
    __shared__ float sh1[2][L::kWaves > 1 ? L::kWaves : 1], sh2[2][L::kWaves > 1 ? 2 * L::kWaves : 1], sh3[2][kShared];
    __shared__ float columns[L::kGroups > 1 ? L::kGroups * G * E : 1];
    // Rows of several waves that do not fill their slots take more registers, and run in fewer waves: there the block's and
    // the gate's loads go out with the first ones, if they are short (bf16: 24,000 x 2,600 257 -> 225 us, x 1,400 121 -> 124 us,
    // 8,192 x 5,000 194 us either way; where rows fill their slots 214 -> 220 us at 32,768 x 2,048, so not there).
    constexpr bool kEarly = sizeof(T) == 2 && !EXACT && L::kWaves > 1;
    int turn1 = 0, turn2 = 0, turn3 = 0;
    const L at(a.width);
    const int gate_kind = FULL ? (int)MODE : a.gate_width > 1 ? (int)kElementGate : a.gate_width;   // widths of 1 count as one gate a row
    const bool has_dr = FULL || dr, has_dh = FULL || dh, has_block = FULL || block;
    __shared__ __attribute__((aligned(16))) float vectors[3][L::kSlots];
    at.keep(vectors[0], a.post_weight, 1.0f, a.scale);
    at.keep(vectors[1], a.post_bias, 0.0f, a.scale);
    at.keep(vectors[2], a.pre_weight, 1.0f, nullptr);
    __syncthreads();
    // sums over the group's rows: total sigma hat_b, total sigma, dh hat_r, dh
    float s0[E] = {}, s1[E] = {}, s3[E] = {}, s4[E] = {};
    auto normalise = [&](float (&v)[E]) { return at.normalise(v, a.layer, a.eps, a.inv_width, sh1, turn1); };
    typename L::Raw rdr, rdh, rr, rb, rg;
    T row_gate{};
    auto fetch_pre = [&](int64_t i) {
        if (has_dr) at.fetch(rdr, dr + i * a.width);
        if (has_dh) {
            at.fetch(rr, r + i * ldr);
            at.fetch(rdh, dh + i * a.width);
        }
    };
    auto fetch_post = [&](int64_t i) {
        if (!has_block) return;
        at.fetch(rb, block + i * ldb);
        if (gate_kind == kElementGate) at.fetch(rg, gate + i * ldg);
        else if (gate_kind == kRowGate) row_gate = gate[i * ldg];
    };
    const int64_t stride = (int64_t)gridDim.x * L::kGroups;
    int64_t i = (int64_t)blockIdx.x * L::kGroups + at.group;
    for (; i < a.n; i += stride) {
        fetch_pre(i);
        if (kEarly) fetch_post(i);
        float t[E];
        if (has_dr) at.values(t, rdr);
        else
#pragma unroll
            for (int e = 0; e < E; ++e) t[e] = 0.0f;
        if (has_dh) {
            float hat[E], d[E];
            at.values(hat, rr);
            at.values(d, rdh);
            const float inv = normalise(hat);
            float qw[E];
            at.kept(qw, vectors[2]);
            float m[2] = {0.0f, 0.0f};
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s3[e] = fmaf(d[e], hat[e], s3[e]);
                s4[e] += d[e];
                d[e] *= qw[e];
                const float mine = at.share(d[e], e);
                m[0] += mine;
                m[1] = fmaf(mine, hat[e], m[1]);
            }
            at.sums(m, sh2, turn2);
            const float m1 = a.layer ? m[0] * a.inv_width : 0.0f, m2 = m[1] * a.inv_width;
#pragma unroll
            for (int e = 0; e < E; ++e) t[e] = fmaf(inv, d[e] - m1 - hat[e] * m2, t[e]);
        }
        if (FULL || dx) at.store(dx + i * a.width, t);
        if (has_block) {
            if (!kEarly) fetch_post(i);
            float b[E], g[E];
            at.values(b, rb);
            if (gate_kind == kElementGate) at.values(g, rg);
            else g[0] = to_f32(row_gate);
            const float inv = normalise(b);
            float pw[E], pb[E];   // times the scale
            at.kept(pw, vectors[0]);
            at.kept(pb, vectors[1]);
            float m[3] = {0.0f, 0.0f, 0.0f};
            float s = 1.0f, rest = 0.0f;
            if (gate_kind == kRowGate) sigmoids(g[0], s, rest);
            float du[E], dg[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (gate_kind == kElementGate) sigmoids(g[e], s, rest);
                const float ts = t[e] * s;
                s0[e] = fmaf(ts, b[e], s0[e]);
                s1[e] += ts;
                dg[e] = ts * fmaf(b[e], pw[e], pb[e]) * rest;
                du[e] = ts * pw[e];
                const float mine = at.share(du[e], e);
                m[0] += mine;
                m[1] = fmaf(mine, b[e], m[1]);
                m[2] += at.share(dg[e], e);
            }
            if (gate_kind == kElementGate) at.store(dgate + i * a.width, dg);
            at.sums(m, sh3, turn3);
            if (gate_kind == kRowGate && at.lane == 0) dgate[i] = from_f32<T>(m[2]);
            const float m1 = a.layer ? m[0] * a.inv_width : 0.0f, m2 = m[1] * a.inv_width;
#pragma unroll
            for (int e = 0; e < E; ++e) du[e] = inv * (du[e] - m1 - b[e] * m2);
            at.store(dblock + i * a.width, du);
        }
    }
    if (!part) return;
    // the block's sums of each column, its groups in order: part[block][4][width]
    auto write = [&](int q, const float (&s)[E]) {
        float *to = part + ((int64_t)blockIdx.x * 4 + q) * a.width;
        // columns that several lanes have hold the same sum in each
        if constexpr (L::kGroups == 1) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < W; ++j) to[at.column[c] + j] = s[c * W + j];
        } else {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < W; ++j) columns[at.group * L::kSlots + at.column[c] + j] = s[c * W + j];
            __syncthreads();
            for (int c = threadIdx.x; c < a.width; c += L::kThreads) {
                float v = 0.0f;
#pragma unroll
                for (int g = 0; g < L::kGroups; ++g) v += columns[g * L::kSlots + c];
                to[c] = v;
            }
            __syncthreads();
        }
    };
    write(0, s0);
    write(1, s1);
    write(2, s3);
    write(3, s4);
}

// The blocks' sums of 32 columns (blockIdx.y 0: P and Q, 1: the pre norm's two): 32 threads a column take every 32nd
// block, then their sums in order (8,192 x 4,096 bf16, 512 blocks' 33 MB: the gradient 126 us, with 16 columns 129 us).
constexpr int kColumns = 32, kSlices = 1024 / kColumns;
struct Vectors {
    float *v[5];
};
__global__ __launch_bounds__(1024) void k_norm_columns(NormArgs a, int parts, const float *__restrict__ part, Vectors out) {
    __shared__ float sh[2][kSlices][kColumns + 1];
    const int c = blockIdx.x * kColumns + threadIdx.x % kColumns, slice = threadIdx.x / kColumns;
    float s[2] = {};
    if (c < a.width)
#pragma unroll 8
        for (int b = slice; b < parts; b += kSlices) {
            const float *p = part + ((int64_t)b * 4 + blockIdx.y * 2) * a.width + c;
            s[0] += p[0];
            s[1] += p[a.width];
        }
    sh[0][slice][threadIdx.x % kColumns] = s[0];
    sh[1][slice][threadIdx.x % kColumns] = s[1];
    __syncthreads();
    if (slice != 0 || c >= a.width) return;
    float p = 0.0f, q = 0.0f;
#pragma unroll
    for (int b = 0; b < kSlices; ++b) {
        p += sh[0][b][threadIdx.x];
        q += sh[1][b][threadIdx.x];
    }
    if (blockIdx.y == 0) {
        const float sc = a.scale ? a.scale[c] : 1.0f, w = a.post_weight ? a.post_weight[c] : 1.0f, b = a.post_bias ? a.post_bias[c] : 0.0f;
        if (out.v[0]) out.v[0][c] = sc * p;
        if (out.v[1]) out.v[1][c] = sc * q;
        if (out.v[2]) out.v[2][c] = fmaf(w, p, b * q);
    } else {
        if (out.v[3]) out.v[3][c] = p;
        if (out.v[4]) out.v[4][c] = q;
    }
}

NormArgs args_of(const mpnn_norm &p, int64_t n, bool gate) {
    return NormArgs{n, p.width, p.kind == MPNN_NORM_LAYER, gate ? p.gate_width : 0, (float)p.eps, 1.0f / (float)p.width,
                    p.post_weight, p.post_bias, p.scale, p.pre_weight, p.pre_bias};
}

// Values a chunk, lanes and chunks of a lane: the fewest slots that hold the row, in steps of a half (312 values: 32
// lanes of 3 chunks of 4 have 384 slots, 64 lanes of 2 would have 512), up to 12 values a lane, which leaves room for the
// reverse pass's four sums a column in registers; 16 where another wave a row would cost more than it brings.  Rows
// shorter than a chunk go value by value.  Three waves a row (8 values of 192 lanes, for 1,536) are not used: four such
// blocks fill a CU's registers only if their waves fall evenly on its SIMDs (24,000 x 1,400 bf16 133 us or 177 us, 137 us
// with 128 lanes of 12).  BACK: of the widest rows, whose vectors leave LDS for one block a CU, the
// reverse pass takes more waves (bf16 8,192 x 8,192 512 lanes of 16 and 1024 of 8: 289 and 231 us, forward 137 and 150 us;
// 8,192 x 6,144 512 of 12 and 768 of 8: 233 and 186 us, forward 100 and 116 us; fp32 8,192 x 8,192 512
// of 16 and 1024 of 8: reverse 449 and 418 us, forward 251 and 249 us).
template <bool BACK, class F>
Status by_width(int dtype, int width, F run) {
#define MPNN_ROW(type, limit, wide, lanes, chunks)                                                                      \
    if (width <= limit && width > wide * lanes * (chunks - 1))                                                          \
        return run(type{}, std::integral_constant<int, wide>{}, std::integral_constant<int, lanes>{}, std::integral_constant<int, chunks>{});
    if (dtype == MPNN_BF16) {
        MPNN_ROW(bf16, 7, 1, 8, 1)
        MPNN_ROW(bf16, 64, 8, 8, 1)
        MPNN_ROW(bf16, 96, 4, 8, 3)
        MPNN_ROW(bf16, 128, 8, 16, 1)
        MPNN_ROW(bf16, 192, 4, 16, 3)
        MPNN_ROW(bf16, 256, 8, 32, 1)
        MPNN_ROW(bf16, 384, 4, 32, 3)
        MPNN_ROW(bf16, 512, 8, 64, 1)
        MPNN_ROW(bf16, 768, 4, 64, 3)
        MPNN_ROW(bf16, 1024, 8, 64, 2)
        MPNN_ROW(bf16, 1536, 4, 128, 3)
        MPNN_ROW(bf16, 2048, 8, 256, 1)
        MPNN_ROW(bf16, 256 * 12, 4, 256, 3)
        MPNN_ROW(bf16, 4096, 8, 512, 1)
        if constexpr (BACK) {
            MPNN_ROW(bf16, 6144, 8, 768, 1)
            MPNN_ROW(bf16, 8192, 8, 1024, 1)
        } else {
            MPNN_ROW(bf16, 6144, 4, 512, 3)
            MPNN_ROW(bf16, 8192, 8, 512, 2)
        }
    } else {
        MPNN_ROW(float, 3, 1, 8, 1)
        MPNN_ROW(float, 32, 4, 8, 1)
        MPNN_ROW(float, 64, 4, 8, 2)
        MPNN_ROW(float, 96, 4, 8, 3)
        MPNN_ROW(float, 128, 4, 16, 2)
        MPNN_ROW(float, 192, 4, 16, 3)
        MPNN_ROW(float, 256, 4, 32, 2)
        MPNN_ROW(float, 384, 4, 32, 3)
        MPNN_ROW(float, 512, 4, 64, 2)
        MPNN_ROW(float, 768, 4, 64, 3)
        MPNN_ROW(float, 1024, 4, 128, 2)
        MPNN_ROW(float, 1536, 4, 128, 3)
        MPNN_ROW(float, 2048, 4, 256, 2)
        MPNN_ROW(float, 256 * 12, 4, 256, 3)
        MPNN_ROW(float, 4096, 4, 512, 2)
        MPNN_ROW(float, 6144, 4, 512, 3)
        MPNN_ROW(float, 8192, 4, 1024, 2)
    }
#undef MPNN_ROW
    return Status::err(MPNN_E_INVALID_ARG, "bad width");
}

// Blocks for n rows: enough that the rows which a CU's blocks ask for at a time come to `bytes`, no more than run at once.
// More of them bring no bandwidth, and each writes partial sums (gradient of 128,000 x 312 fp32 with one and two blocks of
// four rows a CU: 237 and 255 us, bf16 185 and 138 us; forward of 400,002 x 128 fp32 with 32 KB a CU, with all that fit and
// with eight blocks a CU: 186, 201 and 198 us; of 8,192 x 8,192 bf16 with one block and eight: 122 and 137 us).
constexpr int kForwardBytes = 32 * 1024, kBackBytes = 52 * 1024;
template <auto *Kernel, class L, class T>
int64_t blocks_for(int64_t n, int arrays, int bytes) {
    static const int resident = [] {
        int per = 0;
        return hipOccupancyMaxActiveBlocksPerMultiprocessor(&per, Kernel, L::kThreads, 0) == hipSuccess && per > 0 ? per : 1;
    }();
    const int span = L::kThreads * L::E * (int)sizeof(T) * arrays;
    return std::min<int64_t>((n + L::kGroups - 1) / L::kGroups, 256 * (int64_t)std::min(resident, (bytes + span - 1) / span));
}

// The kernel for a call: run gets the mode, and whether the rows fill their slots, as constants.
template <class F>
Status by_mode(bool full, bool exact, int gate_width, F run) {
    const auto with = [&](auto mode) -> Status { return exact ? run(mode, std::true_type{}) : run(mode, std::false_type{}); };
    if (!full) return run(std::integral_constant<int, kAny>{}, std::false_type{});
    if (gate_width == 0) return with(std::integral_constant<int, kNoGate>{});
    if (gate_width == 1) return with(std::integral_constant<int, kRowGate>{});
    return with(std::integral_constant<int, kElementGate>{});
}

}  // namespace

Status norm_residual(Context &cx, const mpnn_norm &p, int64_t n, const void *x, int64_t ldx, const void *block, int64_t ldb,
                     const void *gate, int64_t ldg, void *r, void *h) {
    if (n == 0) return Status::ok();
    const NormArgs a = args_of(p, n, gate);
    return by_width<false>(p.dtype, p.width, [&](auto type, auto wide, auto lanes, auto chunks) -> Status {
        using T = decltype(type);
        using L = Lanes<T, wide(), lanes(), chunks(), false>;
        return by_mode(block && r && h, p.width == L::kSlots, a.gate_width, [&](auto mode, auto exact) -> Status {
            constexpr auto *kernel = k_norm_residual<T, wide(), lanes(), chunks(), mode(), exact()>;
            const int64_t blocks = blocks_for<kernel, L, T>(n, mode() == kElementGate ? 3 : 2, kForwardBytes);
            kernel<<<(unsigned)blocks, L::kThreads, 0, cx.stream>>>(a, (const T *)x, ldx, (const T *)block, ldb, (const T *)gate, ldg,
                                                                    (T *)r, (T *)h);
            MPNN_HIP(hipGetLastError());
            return Status::ok();
        });
    });
}

Status norm_residual_backward(Context &cx, const mpnn_norm &p, int64_t n, const void *dr, const void *dh, const void *r, int64_t ldr,
                              const void *block, int64_t ldb, const void *gate, int64_t ldg, void *dx, void *dblock, void *dgate,
                              float *const dvec[5]) {
    const NormArgs a = args_of(p, n, gate);
    return by_width<true>(p.dtype, p.width, [&](auto type, auto wide, auto lanes, auto chunks) -> Status {
        using T = decltype(type);
        using L = Lanes<T, wide(), lanes(), chunks(), false>;
        const bool columns = dvec[0] || dvec[1] || dvec[2] || dvec[3] || dvec[4];
        int64_t blocks = 0;
        float *part = nullptr;
        MPNN_TRY(by_mode(dr && dh && block && dx, p.width == L::kSlots, a.gate_width, [&](auto mode, auto exact) -> Status {
            constexpr auto *kernel = k_norm_residual_back<T, wide(), lanes(), chunks(), mode(), exact()>;
            blocks = blocks_for<kernel, L, T>(n, mode() == kElementGate ? 5 : 4, kBackBytes);
            void *ws = nullptr;
            if (columns) MPNN_TRY(cx.rows_scratch(sizeof(float) * (size_t)(blocks * 4 * p.width), &ws));
            part = static_cast<float *>(ws);
            if (n == 0) return Status::ok();
            kernel<<<(unsigned)blocks, L::kThreads, 0, cx.stream>>>(a, (const T *)dr, (const T *)dh, (const T *)r, ldr, (const T *)block, ldb,
                                                                   (const T *)gate, ldg, (T *)dx, (T *)dblock, (T *)dgate, part);
            MPNN_HIP(hipGetLastError());
            return Status::ok();
        }));
        if (columns) {
            k_norm_columns<<<dim3((p.width + kColumns - 1) / kColumns, 2), 1024, 0, cx.stream>>>(a, (int)blocks, part,
                                                                                 Vectors{{dvec[0], dvec[1], dvec[2], dvec[3], dvec[4]}});
            MPNN_HIP(hipGetLastError());
        }
        return Status::ok();
    });
}

}  // namespace mpnn
