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

// What a launch is compiled for.  kAny: any width up to the lanes' slots, any of the optional arrays missing.  The
// others: rows that fill the slots exactly, every array there, and the gate of that kind.  Their row loop has no
// condition around a load or a store, so a wait for a load is a wait for that load alone; with conditions it waits for
// all that is under way, the stores of the row before among it (gradient of 8,192 x 4,096 bf16: 242 us, 140 us without).
enum Mode { kAny = -1, kNoGate = 0, kRowGate = 1, kElementGate = 2 };

// A row's place in the block's registers.
template <class T, int G, int CH, bool EXACT>
struct Lanes {
    static constexpr int W = Chunk<T>::W, E = CH * W;      // values of a row per lane
    static constexpr int kThreads = G > 64 ? G : 256, kGroups = kThreads / G;   // several waves a row: one row a block
    static constexpr int kWaves = G / 64;                  // waves of a row (0: part of one)
    int lane, group;
    int width;
    bool whole;            // a row is whole chunks: each is all inside it or all outside (EXACT: inside)
    __device__ __forceinline__ Lanes(int w) : lane(threadIdx.x % G), group(threadIdx.x / G), width(w), whole(w % W == 0) {}
    __device__ __forceinline__ int column(int c) const { return (c * G + lane) * W; }
    // A row as it is in memory; zeros past its end.
    struct Raw {
        Chunk<T> c[CH];
    };
    __device__ __forceinline__ void fetch(Raw &t, const T *row) const {
        if (EXACT) {
#pragma unroll
            for (int c = 0; c < CH; ++c) t.c[c] = load_chunk(row + column(c));
            return;
        }
        __builtin_memset(&t, 0, sizeof t);
        if (whole) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (column(c) < width) t.c[c] = load_chunk(row + column(c));
        } else {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int left = width - column(c);
                if (left > 0) t.c[c] = load_chunk(row + column(c), left);
            }
        }
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
            Chunk<T> t;
#pragma unroll
            for (int j = 0; j < W; ++j) t.v[j] = from_f32<T>(v[c * W + j]);
            const int left = width - column(c);
            if (EXACT) {
                store_chunk(row + column(c), t);
            } else if (whole) {
                if (left > 0) store_chunk(row + column(c), t);
            } else {
                if (left > 0) store_chunk(row + column(c), t, left);
            }
        }
    }
    // a vector's values of this lane's columns; zeros past the width
    __device__ __forceinline__ void vector(float (&v)[E], const float *p, float otherwise) const {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = p ? 0.0f : column(e / W) + e % W < width ? otherwise : 0.0f;
        if (!p) return;
        if (whole) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (column(c) < width) __builtin_memcpy(&v[c * W], p + column(c), W * sizeof(float));
        } else {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (column(c) + j < width) v[c * W + j] = p[column(c) + j];
        }
    }
    // The reverse pass keeps its vectors in LDS (zeros past the width), whose registers its sums need.  The offset is
    // zero, but not to the compiler, which would move the reads out of the row loop, into registers.
    static constexpr int kSlots = G * E;
    __device__ __forceinline__ void keep(float *sh, const float *p, float otherwise) const {
        for (int c = threadIdx.x; c < kSlots; c += kThreads) sh[c] = c < width ? (p ? p[c] : otherwise) : 0.0f;
    }
    __device__ __forceinline__ void kept(float (&v)[E], const float *sh) const {
        int z = 0;
        asm volatile("" : "+v"(z));
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < W; j += 4) {
                const float4 t = *reinterpret_cast<const float4 *>(sh + column(c) + j + z);
                v[c * W + j] = t.x; v[c * W + j + 1] = t.y; v[c * W + j + 2] = t.z; v[c * W + j + 3] = t.w;
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
    // v becomes its distance from m (0 past the width)
    __device__ __forceinline__ void centre(float (&v)[E], float m) const {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const float mc = EXACT || column(c) < width ? m : 0.0f;      // a chunk outside holds zeros
#pragma unroll
            for (int j = 0; j < W; ++j) v[c * W + j] -= mc;
        }
        if (!EXACT && !whole) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (column(c) + j >= width) v[c * W + j] = 0.0f;
        }
    }
};

template <int E> __device__ __forceinline__ float sum_of(const float (&v)[E]) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += v[e];
    return s;
}
template <int E> __device__ __forceinline__ float dot_of(const float (&v)[E], const float (&w)[E]) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(v[e], w[e], s);
    return s;
}

// In a group of several waves all waves of the block take the same row, so barriers inside the row loop are uniform.
template <class T, int G, int CH, int MODE>
__global__ __launch_bounds__((Lanes<T, G, CH, false>::kThreads)) void k_norm_residual(NormArgs a, const T *__restrict__ x, int64_t ldx,
                                                                             const T *__restrict__ block, int64_t ldb,
                                                                             const T *__restrict__ gate, int64_t ldg, T *r,
                                                                             T *__restrict__ h) {
    constexpr bool EXACT = MODE != kAny;
    using L = Lanes<T, G, CH, EXACT>;
    constexpr int E = L::E;
    __shared__ float sh[2][L::kWaves > 1 ? L::kWaves : 1];
    int turn = 0;
    const L at(a.width);
    const int gate_kind = EXACT ? (int)MODE : a.gate_width > 1 ? (int)kElementGate : a.gate_width;   // widths of 1 count as one gate a row
    const bool has_block = EXACT || block, has_r = EXACT || r, has_h = EXACT || h;
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
    auto normalise = [&](float (&v)[E]) {
        if (a.layer) {
            float m[1] = {sum_of(v)};
            at.sums(m, sh, turn);
            at.centre(v, m[0] * a.inv_width);
        }
        float q[1] = {dot_of(v, v)};
        at.sums(q, sh, turn);
        const float inv = rsqrtf(q[0] * a.inv_width + a.eps);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= inv;
    };
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
template <class T, int G, int CH, int MODE>
__global__ __launch_bounds__((Lanes<T, G, CH, false>::kThreads)) void k_norm_residual_back(NormArgs a, const T *dr, const T *__restrict__ dh,
                                                                                  const T *__restrict__ r, int64_t ldr,
                                                                                  const T *__restrict__ block, int64_t ldb,
                                                                                  const T *__restrict__ gate, int64_t ldg, T *dx,
                                                                                  T *__restrict__ dblock, T *__restrict__ dgate,
                                                                                  float *__restrict__ part) {
    constexpr bool EXACT = MODE != kAny;
    using L = Lanes<T, G, CH, EXACT>;
    constexpr int E = L::E;
    constexpr int kShared = L::kWaves > 1 ? 3 * L::kWaves : 1;
    __shared__ float sh1[2][L::kWaves > 1 ? L::kWaves : 1], sh2[2][L::kWaves > 1 ? 2 * L::kWaves : 1], sh3[2][kShared];
    __shared__ float columns[L::kGroups > 1 ? L::kGroups * G * E : 1];
    int turn1 = 0, turn2 = 0, turn3 = 0;
    const L at(a.width);
    const int gate_kind = EXACT ? (int)MODE : a.gate_width > 1 ? (int)kElementGate : a.gate_width;   // widths of 1 count as one gate a row
    const bool has_dr = EXACT || dr, has_dh = EXACT || dh, has_block = EXACT || block;
    __shared__ __attribute__((aligned(16))) float vectors[4][L::kSlots];
    at.keep(vectors[0], a.post_weight, 1.0f);
    at.keep(vectors[1], a.post_bias, 0.0f);
    at.keep(vectors[2], a.scale, 1.0f);
    at.keep(vectors[3], a.pre_weight, 1.0f);
    __syncthreads();
    // sums over the group's rows: total sigma hat_b, total sigma, dh hat_r, dh
    float s0[E] = {}, s1[E] = {}, s3[E] = {}, s4[E] = {};
    // v becomes its normed values; returns one over the root
    auto normalise = [&](float (&v)[E]) {
        if (a.layer) {
            float m[1] = {sum_of(v)};
            at.sums(m, sh1, turn1);
            at.centre(v, m[0] * a.inv_width);
        }
        float q[1] = {dot_of(v, v)};
        at.sums(q, sh1, turn1);
        const float inv = rsqrtf(q[0] * a.inv_width + a.eps);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= inv;
        return inv;
    };
    // the next row's loads are under way while a row is worked on
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
    constexpr bool kAhead = !EXACT;      // without conditions the block's other waves hide the loads, in fewer registers
    const int64_t stride = (int64_t)gridDim.x * L::kGroups;
    int64_t i = (int64_t)blockIdx.x * L::kGroups + at.group;
    if (kAhead && i < a.n) {
        fetch_pre(i);
        fetch_post(i);
    }
    for (; i < a.n; i += stride) {
        const int64_t next = i + stride;
        if (!kAhead) fetch_pre(i);
        float t[E];
        if (has_dr) at.values(t, rdr);
        else
#pragma unroll
            for (int e = 0; e < E; ++e) t[e] = 0.0f;
        if (has_dh) {
            float hat[E], d[E];
            at.values(hat, rr);
            at.values(d, rdh);
            if (kAhead && next < a.n) fetch_pre(next);
            const float inv = normalise(hat);
            float qw[E];
            at.kept(qw, vectors[3]);
            float m[2] = {0.0f, 0.0f};
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s3[e] = fmaf(d[e], hat[e], s3[e]);
                s4[e] += d[e];
                d[e] *= qw[e];
                m[0] += d[e];
                m[1] = fmaf(d[e], hat[e], m[1]);
            }
            at.sums(m, sh2, turn2);
            const float m1 = a.layer ? m[0] * a.inv_width : 0.0f, m2 = m[1] * a.inv_width;
#pragma unroll
            for (int e = 0; e < E; ++e) t[e] = fmaf(inv, d[e] - m1 - hat[e] * m2, t[e]);
        }
        if (!has_dh && kAhead && next < a.n) fetch_pre(next);
        if (EXACT || dx) at.store(dx + i * a.width, t);
        if (has_block) {
            if (!kAhead) fetch_post(i);
            float b[E], g[E];
            at.values(b, rb);
            if (gate_kind == kElementGate) at.values(g, rg);
            else g[0] = to_f32(row_gate);
            if (kAhead && next < a.n) fetch_post(next);
            const float inv = normalise(b);
            float pw[E], pb[E], sc[E];
            at.kept(pw, vectors[0]);
            at.kept(pb, vectors[1]);
            at.kept(sc, vectors[2]);
            float m[3] = {0.0f, 0.0f, 0.0f};
            if (gate_kind == kRowGate) g[0] = sigmoid(g[0]);
            float du[E], dg[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float s = gate_kind == kElementGate ? sigmoid(g[e]) : gate_kind == kRowGate ? g[0] : 1.0f;
                const float ts = t[e] * s;
                s0[e] = fmaf(ts, b[e], s0[e]);
                s1[e] += ts;
                du[e] = ts * sc[e];
                dg[e] = du[e] * fmaf(b[e], pw[e], pb[e]) * (1.0f - s);
                du[e] *= pw[e];
                m[0] += du[e];
                m[1] = fmaf(du[e], b[e], m[1]);
                m[2] += dg[e];
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
        if constexpr (L::kGroups == 1) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < L::W; ++j)
                    if (at.column(c) + j < a.width) to[at.column(c) + j] = s[c * L::W + j];
        } else {
            constexpr int kRow = G * E;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < L::W; ++j) columns[at.group * kRow + at.column(c) + j] = s[c * L::W + j];
            __syncthreads();
            for (int c = threadIdx.x; c < a.width; c += L::kThreads) {
                float v = 0.0f;
#pragma unroll
                for (int g = 0; g < L::kGroups; ++g) v += columns[g * kRow + c];
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

// The blocks' sums of 16 columns (blockIdx.y 0: P and Q, 1: the pre norm's two): 64 threads a column take every 64th
// block, then their sums in order.
struct Vectors {
    float *v[5];
};
__global__ __launch_bounds__(1024) void k_norm_columns(NormArgs a, int parts, const float *__restrict__ part, Vectors out) {
    __shared__ float sh[2][64][17];
    const int c = blockIdx.x * 16 + (threadIdx.x & 15), slice = threadIdx.x >> 4;
    float s[2] = {};
    if (c < a.width)
#pragma unroll 8
        for (int b = slice; b < parts; b += 64) {
            const float *p = part + ((int64_t)b * 4 + blockIdx.y * 2) * a.width + c;
            s[0] += p[0];
            s[1] += p[a.width];
        }
    sh[0][slice][threadIdx.x & 15] = s[0];
    sh[1][slice][threadIdx.x & 15] = s[1];
    __syncthreads();
    if (slice != 0 || c >= a.width) return;
    float p = 0.0f, q = 0.0f;
#pragma unroll
    for (int b = 0; b < 64; ++b) {
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

// Lanes of a row and chunks of a lane: the fewest slots that hold the row's chunks (312 fp32 values are 78 chunks: 32
// lanes of 3 waste 18 of 96 slots, 64 lanes of 2 would waste 50 of 128), up to 12 values a lane, which leaves room for
// the reverse pass's five sums a column in registers; 16 values for the widest rows, whose 1,024 lanes would leave only
// 128 registers each.
template <class F>
Status by_width(int dtype, int width, F run) {
#define MPNN_ROW(type, limit, lanes, chunks) \
    if (width <= limit) return run(type{}, std::integral_constant<int, lanes>{}, std::integral_constant<int, chunks>{});
    if (dtype == MPNN_BF16) {
        MPNN_ROW(bf16, 64, 8, 1)
        MPNN_ROW(bf16, 128, 16, 1)
        MPNN_ROW(bf16, 256, 32, 1)
        MPNN_ROW(bf16, 512, 64, 1)
        MPNN_ROW(bf16, 1024, 128, 1)
        MPNN_ROW(bf16, 2048, 256, 1)
        MPNN_ROW(bf16, 4096, 512, 1)
        MPNN_ROW(bf16, 8192, 512, 2)
    } else {
        MPNN_ROW(float, 32, 8, 1)
        MPNN_ROW(float, 64, 8, 2)
        MPNN_ROW(float, 96, 8, 3)
        MPNN_ROW(float, 128, 16, 2)
        MPNN_ROW(float, 192, 16, 3)
        MPNN_ROW(float, 256, 32, 2)
        MPNN_ROW(float, 384, 32, 3)
        MPNN_ROW(float, 512, 64, 2)
        MPNN_ROW(float, 768, 64, 3)
        MPNN_ROW(float, 1024, 128, 2)
        MPNN_ROW(float, 2048, 256, 2)
        MPNN_ROW(float, 4096, 512, 2)
        MPNN_ROW(float, 8192, 512, 4)
    }
#undef MPNN_ROW
    return Status::err(MPNN_E_INVALID_ARG, "bad width");
}

constexpr int64_t kForwardBlocks = 2048, kBackBlocks = 1024;

// The kernel for a call: run gets the mode as a constant.
template <class F>
Status by_mode(bool exact, int gate_width, F run) {
    if (!exact) return run(std::integral_constant<int, kAny>{});
    if (gate_width == 0) return run(std::integral_constant<int, kNoGate>{});
    if (gate_width == 1) return run(std::integral_constant<int, kRowGate>{});
    return run(std::integral_constant<int, kElementGate>{});
}

}  // namespace

Status norm_residual(Context &cx, const mpnn_norm &p, int64_t n, const void *x, int64_t ldx, const void *block, int64_t ldb,
                     const void *gate, int64_t ldg, void *r, void *h) {
    if (n == 0) return Status::ok();
    const NormArgs a = args_of(p, n, gate);
    return by_width(p.dtype, p.width, [&](auto type, auto lanes, auto chunks) -> Status {
        using T = decltype(type);
        using L = Lanes<T, lanes(), chunks(), false>;
        const int64_t blocks = std::min<int64_t>((n + L::kGroups - 1) / L::kGroups, kForwardBlocks);
        return by_mode(p.width == L::kSlots && block && r && h, a.gate_width, [&](auto mode) -> Status {
            k_norm_residual<T, lanes(), chunks(), mode()><<<(unsigned)blocks, L::kThreads, 0, cx.stream>>>(
                a, (const T *)x, ldx, (const T *)block, ldb, (const T *)gate, ldg, (T *)r, (T *)h);
            MPNN_HIP(hipGetLastError());
            return Status::ok();
        });
    });
}

Status norm_residual_backward(Context &cx, const mpnn_norm &p, int64_t n, const void *dr, const void *dh, const void *r, int64_t ldr,
                              const void *block, int64_t ldb, const void *gate, int64_t ldg, void *dx, void *dblock, void *dgate,
                              float *const dvec[5]) {
    const NormArgs a = args_of(p, n, gate);
    return by_width(p.dtype, p.width, [&](auto type, auto lanes, auto chunks) -> Status {
        using T = decltype(type);
        using L = Lanes<T, lanes(), chunks(), false>;
        const int64_t blocks = std::min<int64_t>((n + L::kGroups - 1) / L::kGroups, kBackBlocks * 256 / L::kThreads);
        const bool columns = dvec[0] || dvec[1] || dvec[2] || dvec[3] || dvec[4];
        if (columns) MPNN_TRY(cx.grow(cx.rows_ws, sizeof(float) * (size_t)(blocks * 4 * p.width)));
        float *part = columns ? cx.rows_ws.as<float>() : nullptr;
        if (n > 0)
            MPNN_TRY(by_mode(p.width == L::kSlots && dr && dh && block && dx, a.gate_width, [&](auto mode) -> Status {
                k_norm_residual_back<T, lanes(), chunks(), mode()><<<(unsigned)blocks, L::kThreads, 0, cx.stream>>>(
                    a, (const T *)dr, (const T *)dh, (const T *)r, ldr, (const T *)block, ldb, (const T *)gate, ldg, (T *)dx,
                    (T *)dblock, (T *)dgate, part);
                MPNN_HIP(hipGetLastError());
                return Status::ok();
            }));
        if (columns) {
            k_norm_columns<<<dim3((p.width + 15) / 16, 2), 1024, 0, cx.stream>>>(a, (int)blocks, part,
                                                                                 Vectors{{dvec[0], dvec[1], dvec[2], dvec[3], dvec[4]}});
            MPNN_HIP(hipGetLastError());
        }
        return Status::ok();
    });
}

}  // namespace mpnn
