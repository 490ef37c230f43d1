// Norms before and after a block, fused with the block's gate and residual scale (mpnn_norm_residual*).
//   r = x + scale * sigma(gate) * N_post(block),  h = N_pre(r),
//   N(v) = (v - mean) / sqrt(mean((v - mean)^2) + eps) * weight + bias   (rms: without the mean)
// h comes from the unrounded r.  The reverse pass takes the statistics again from the rows it reads anyway, so the
// forward pass stores none.
#include "impl.h"
#include "rows.h"

namespace mpnn {

namespace {

struct NormArgs {
    int64_t n;
    int width, layer;
    int gate_width;
    float eps;
    const float *post_weight, *post_bias, *scale, *pre_weight, *pre_bias;
};

__device__ __forceinline__ float at_or(const float *p, int c, float otherwise) { return p ? p[c] : otherwise; }
__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

// mean (0 for rms) and 1 / sqrt(mean square + eps) of a row, by one wave
template <class F>
__device__ __forceinline__ void row_stats(const NormArgs &a, int lane, F value, float &mean, float &inv) {
    mean = 0.0f;
    if (a.layer) {
        float s = 0.0f;
        for (int c = lane; c < a.width; c += 64) s += value(c);
        mean = wave_sum(s) / a.width;
    }
    float q = 0.0f;
    for (int c = lane; c < a.width; c += 64) {
        const float v = value(c) - mean;
        q = fmaf(v, v, q);
    }
    inv = rsqrtf(wave_sum(q) / a.width + a.eps);
}

template <class T>
__global__ void k_norm_residual(NormArgs a, const T *__restrict__ x, int64_t ldx, const T *__restrict__ block, int64_t ldb,
                                const T *__restrict__ gate, int64_t ldg, T *r, T *__restrict__ h) {
    const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (i >= a.n) return;
    const int lane = threadIdx.x & 63;
    float bm = 0.0f, bi = 0.0f;
    if (block) row_stats(a, lane, [&](int c) { return to_f32(block[i * ldb + c]); }, bm, bi);
    auto sum = [&](int c) {
        float v = to_f32(x[i * ldx + c]);
        if (block) {
            const float u = (to_f32(block[i * ldb + c]) - bm) * bi * at_or(a.post_weight, c, 1.0f) + at_or(a.post_bias, c, 0.0f);
            const float g = gate ? sigmoid(to_f32(gate[i * ldg + (a.gate_width == 1 ? 0 : c)])) : 1.0f;
            v += at_or(a.scale, c, 1.0f) * g * u;
        }
        return v;
    };
    float rm, ri;
    if (h) {
        row_stats(a, lane, sum, rm, ri);
        for (int c = lane; c < a.width; c += 64)
            h[i * a.width + c] = from_f32<T>((sum(c) - rm) * ri * at_or(a.pre_weight, c, 1.0f) + at_or(a.pre_bias, c, 0.0f));
    }
    if (r)
        for (int c = lane; c < a.width; c += 64) r[i * a.width + c] = from_f32<T>(sum(c));
}

// Gradients of the rows.  total = dr + N_pre'(dh), dx = total, and with u = N_post(block):
//   dgate = total scale u sigma'(gate), du = total scale sigma(gate), dblock = N_post'(du),
//   N'(d) = inv (a - mean(a) - hat mean(a hat)), a = d weight   (rms: without mean(a))
// The row's statistics and sums go to stats[i][kStats] for the columns' pass.
constexpr int kStats = 6;   // block mean, block inverse, r mean, r inverse, mean(a_pre), mean(a_pre hat)

template <class T>
__global__ void k_norm_residual_back(NormArgs a, const T *__restrict__ dr, const T *__restrict__ dh, const T *__restrict__ r,
                                     int64_t ldr, const T *__restrict__ block, int64_t ldb, const T *__restrict__ gate, int64_t ldg,
                                     T *dx, T *__restrict__ dblock, T *__restrict__ dgate, float *__restrict__ stats) {
    const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (i >= a.n) return;
    const int lane = threadIdx.x & 63;
    float bm = 0, bi = 0, rm = 0, ri = 0, m1 = 0, m2 = 0;
    if (dh) {
        row_stats(a, lane, [&](int c) { return to_f32(r[i * ldr + c]); }, rm, ri);
        for (int c = lane; c < a.width; c += 64) {
            const float w = to_f32(dh[i * a.width + c]) * at_or(a.pre_weight, c, 1.0f);
            m1 += w;
            m2 = fmaf(w, (to_f32(r[i * ldr + c]) - rm) * ri, m2);
        }
        m1 = a.layer ? wave_sum(m1) / a.width : 0.0f;
        m2 = wave_sum(m2) / a.width;
    }
    auto total = [&](int c) {
        float v = dr ? to_f32(dr[i * a.width + c]) : 0.0f;
        if (dh) {
            const float hat = (to_f32(r[i * ldr + c]) - rm) * ri;
            v += ri * (to_f32(dh[i * a.width + c]) * at_or(a.pre_weight, c, 1.0f) - m1 - hat * m2);
        }
        return v;
    };
    if (block) {
        row_stats(a, lane, [&](int c) { return to_f32(block[i * ldb + c]); }, bm, bi);
        float n1 = 0, n2 = 0, gs = 0;
        auto sig = [&](int c) { return gate ? sigmoid(to_f32(gate[i * ldg + (a.gate_width == 1 ? 0 : c)])) : 1.0f; };
        for (int c = lane; c < a.width; c += 64) {
            const float t = total(c) * at_or(a.scale, c, 1.0f), hat = (to_f32(block[i * ldb + c]) - bm) * bi;
            const float g = sig(c), d = t * g * at_or(a.post_weight, c, 1.0f);
            n1 += d;
            n2 = fmaf(d, hat, n2);
            const float dg = t * (hat * at_or(a.post_weight, c, 1.0f) + at_or(a.post_bias, c, 0.0f)) * g * (1.0f - g);
            if (gate && a.gate_width != 1) dgate[i * a.width + c] = from_f32<T>(dg);
            gs += dg;
        }
        n1 = a.layer ? wave_sum(n1) / a.width : 0.0f;
        n2 = wave_sum(n2) / a.width;
        gs = wave_sum(gs);
        if (gate && a.gate_width == 1 && lane == 0) dgate[i] = from_f32<T>(gs);
        for (int c = lane; c < a.width; c += 64) {
            const float hat = (to_f32(block[i * ldb + c]) - bm) * bi;
            const float d = total(c) * at_or(a.scale, c, 1.0f) * sig(c) * at_or(a.post_weight, c, 1.0f);
            dblock[i * a.width + c] = from_f32<T>(bi * (d - n1 - hat * n2));
        }
    }
    if (stats && lane == 0) {
        const float v[kStats] = {bm, bi, rm, ri, m1, m2};
        for (int q = 0; q < kStats; ++q) stats[i * kStats + q] = v[q];
    }
    if (dx)
        for (int c = lane; c < a.width; c += 64) dx[i * a.width + c] = from_f32<T>(total(c));
}

// Sums over the rows, for the five vectors: one thread per column and block of rows, then one per column.
template <class T>
__global__ void k_norm_columns(NormArgs a, const T *__restrict__ dr, const T *__restrict__ dh, const T *__restrict__ r, int64_t ldr,
                               const T *__restrict__ block, int64_t ldb, const T *__restrict__ gate, int64_t ldg,
                               const float *__restrict__ stats, int64_t rows, float *__restrict__ part) {
    const int c = blockIdx.y * 64 + threadIdx.x;
    if (c >= a.width) return;
    const int64_t end = min(a.n, (int64_t)(blockIdx.x + 1) * rows);
    float s[5] = {};
    for (int64_t i = (int64_t)blockIdx.x * rows; i < end; ++i) {
        const float *st = stats + i * kStats;
        float total = dr ? to_f32(dr[i * a.width + c]) : 0.0f;
        if (dh) {
            const float hat = (to_f32(r[i * ldr + c]) - st[2]) * st[3], d = to_f32(dh[i * a.width + c]);
            total += st[3] * (d * at_or(a.pre_weight, c, 1.0f) - st[4] - hat * st[5]);
            s[3] = fmaf(d, hat, s[3]);
            s[4] += d;
        }
        if (block) {
            const float hat = (to_f32(block[i * ldb + c]) - st[0]) * st[1];
            const float g = gate ? sigmoid(to_f32(gate[i * ldg + (a.gate_width == 1 ? 0 : c)])) : 1.0f;
            const float du = total * at_or(a.scale, c, 1.0f) * g;
            s[0] = fmaf(du, hat, s[0]);
            s[1] += du;
            s[2] = fmaf(total * g, hat * at_or(a.post_weight, c, 1.0f) + at_or(a.post_bias, c, 0.0f), s[2]);
        }
    }
    for (int q = 0; q < 5; ++q) part[((int64_t)blockIdx.x * 5 + q) * a.width + c] = s[q];
}

__global__ void k_norm_columns_sum(int width, int parts, const float *__restrict__ part, float *o0, float *o1, float *o2, float *o3,
                                   float *o4) {
    const int c = blockIdx.x * 64 + threadIdx.x, q = blockIdx.y;
    float *o = q == 0 ? o0 : q == 1 ? o1 : q == 2 ? o2 : q == 3 ? o3 : o4;
    if (c >= width || !o) return;
    float s = 0.0f;
    for (int b = 0; b < parts; ++b) s += part[((int64_t)b * 5 + q) * width + c];
    o[c] = s;
}

NormArgs args_of(const mpnn_norm &p, int64_t n, bool gate) {
    return NormArgs{n, p.width, p.kind == MPNN_NORM_LAYER, gate ? p.gate_width : 0, (float)p.eps,
                    p.post_weight, p.post_bias, p.scale, p.pre_weight, p.pre_bias};
}

template <class T>
Status forward_t(Context &cx, const mpnn_norm &p, int64_t n, const void *x, int64_t ldx, const void *block, int64_t ldb,
                 const void *gate, int64_t ldg, void *r, void *h) {
    k_norm_residual<T><<<grid_for(n, 4), 256, 0, cx.stream>>>(args_of(p, n, gate), (const T *)x, ldx, (const T *)block, ldb,
                                                              (const T *)gate, ldg, (T *)r, (T *)h);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

template <class T>
Status backward_t(Context &cx, const mpnn_norm &p, int64_t n, const void *dr, const void *dh, const void *r, int64_t ldr,
                  const void *block, int64_t ldb, const void *gate, int64_t ldg, void *dx, void *dblock, void *dgate,
                  float *const dvec[5]) {
    const NormArgs a = args_of(p, n, gate);
    const bool columns = dvec[0] || dvec[1] || dvec[2] || dvec[3] || dvec[4];
    const int64_t rows = std::max<int64_t>(16, (n + 1023) / 1024);
    const int64_t parts = (n + rows - 1) / rows;
    float *stats = nullptr, *part = nullptr;
    if (columns) {
        MPNN_TRY(cx.grow(cx.rows_ws, sizeof(float) * (size_t)(n * kStats + parts * 5 * p.width)));
        stats = cx.rows_ws.as<float>();
        part = stats + n * kStats;
    }
    if (n > 0) {
        k_norm_residual_back<T><<<grid_for(n, 4), 256, 0, cx.stream>>>(a, (const T *)dr, (const T *)dh, (const T *)r, ldr,
                                                                       (const T *)block, ldb, (const T *)gate, ldg, (T *)dx,
                                                                       (T *)dblock, (T *)dgate, stats);
        MPNN_HIP(hipGetLastError());
    }
    if (columns) {
        if (parts > 0) {
            k_norm_columns<T><<<dim3((unsigned)parts, (p.width + 63) / 64), 64, 0, cx.stream>>>(
                a, (const T *)dr, (const T *)dh, (const T *)r, ldr, (const T *)block, ldb, (const T *)gate, ldg, stats, rows, part);
            MPNN_HIP(hipGetLastError());
        }
        k_norm_columns_sum<<<dim3((p.width + 63) / 64, 5), 64, 0, cx.stream>>>(p.width, (int)parts, part, dvec[0], dvec[1], dvec[2],
                                                                              dvec[3], dvec[4]);
        MPNN_HIP(hipGetLastError());
    }
    return Status::ok();
}

}  // namespace

Status norm_residual(Context &cx, const mpnn_norm &p, int64_t n, const void *x, int64_t ldx, const void *block, int64_t ldb,
                     const void *gate, int64_t ldg, void *r, void *h) {
    if (n == 0) return Status::ok();
    return p.dtype == MPNN_BF16 ? forward_t<bf16>(cx, p, n, x, ldx, block, ldb, gate, ldg, r, h)
                                : forward_t<float>(cx, p, n, x, ldx, block, ldb, gate, ldg, r, h);
}

Status norm_residual_backward(Context &cx, const mpnn_norm &p, int64_t n, const void *dr, const void *dh, const void *r, int64_t ldr,
                              const void *block, int64_t ldb, const void *gate, int64_t ldg, void *dx, void *dblock, void *dgate,
                              float *const dvec[5]) {
    return p.dtype == MPNN_BF16 ? backward_t<bf16>(cx, p, n, dr, dh, r, ldr, block, ldb, gate, ldg, dx, dblock, dgate, dvec)
                                : backward_t<float>(cx, p, n, dr, dh, r, ldr, block, ldb, gate, ldg, dx, dblock, dgate, dvec);
}

}  // namespace mpnn
