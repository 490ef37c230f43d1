// Activation checkpoints in 8 bits (mpnn_checkpoint_*).  A group of 32 channels of a row shares one power-of-two
// step 2^e, the smallest that keeps the group's largest value within 127 steps:
//   largest = m 2^E, 1 <= m < 2:  e = E - 6 + (m > 127/64), clamped to -100 .. 121;  code = rint(v 2^-e) in +-127
// The scale byte holds e + 127; 255 marks a group with a value that is not finite and reads back as NaN.  With a
// power of two every code 2^e is exact in bf16 (and in fp32), so a checkpoint is a matrix-core operand as it stands
// and reading one back rounds nothing.
//
// Bound by HBM: a lane takes 16 bytes of the rows, and a group's largest value comes from its 4 or 8 neighbouring lanes
// without LDS.  400,002 x 128: fp32 saved in 42 us (258 MB, 6.1 TB/s), with SiLU and both checkpoints 102 us (515 MB,
// 5.0 TB/s), its gradient 88 us (5.2 TB/s), read back 38 us; bf16 29, 69, 52 and 24 us in a loop of one of them, 73, 55 and
// 30 us for the last three one after another.
#include "impl.h"
#include "rows.h"

namespace mpnn {

namespace {

constexpr int kGroup = 32;
constexpr int kStepMin = -100, kStepMax = 121;

__device__ __forceinline__ int scale_byte(float largest) {
    const uint32_t u = __float_as_uint(largest);
    if (u >= 0x7f800000u) return 255;
    // exponent E + 127 in the top bits; m > 127/64 by its 23 fraction bits (127/64 - 1 = 63/64)
    const int e = (int)(u >> 23) - 127 - 6 + ((u & 0x7fffffu) > (63u << 17) ? 1 : 0);
    return min(max(e, kStepMin), kStepMax) + 127;
}
__device__ __forceinline__ float step_of(int byte) { return byte == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)byte << 23); }
// Lanes of a group: each holds one 16-byte chunk.
template <class T> constexpr int kGroupLanes = kGroup / Chunk<T>::W;

// Largest magnitude of a group from its lanes' values.  Magnitudes order as integers, a NaN above infinity.
template <class T> __device__ __forceinline__ float group_max(const float (&v)[Chunk<T>::W]) {
    uint32_t u = 0;
#pragma unroll
    for (int j = 0; j < Chunk<T>::W; ++j) u = max(u, __float_as_uint(v[j]) & 0x7fffffffu);
    float f = __uint_as_float(u);
    auto step = [&](float o) { f = __uint_as_float(max(__float_as_uint(f), __float_as_uint(o))); };
    step(dpp<0xb1>(f));
    step(dpp<0x4e>(f));
    if (kGroupLanes<T> == 8) step(dpp<0x141>(f));
    return f;
}

// sigma(z) and 1 - sigma(z) from a = exp(-|z|) <= 1, without a reciprocal of a large number (1 / (1 + exp(-z)) would pass
// through one that the hardware's reciprocal flushes to zero): r = 1 / (1 + a) and a r. The reciprocal of 1 .. 2 gets one
// Newton step, r + r (1 - (1 + a) r): its own error of an ulp moves more codes across a rounding edge than exp's does.
__device__ __forceinline__ void sigmoids(float z, float &s, float &rest) {
    const float a = expf(-fabsf(z)), r0 = __builtin_amdgcn_rcpf(1.0f + a);
    const float r = fmaf(r0, fmaf(-(1.0f + a), r0, 1.0f), r0), ar = a * r;
    s = z >= 0.0f ? r : ar;
    rest = z >= 0.0f ? ar : r;
}

// The codes of one chunk and, by the group's first lane, the scale.
template <class T>
__device__ __forceinline__ void save_chunk(const float (&v)[Chunk<T>::W], int in, int8_t *codes, uint8_t *scale, bool first) {
    constexpr int W = Chunk<T>::W;
    const int b = scale_byte(group_max<T>(v));
    const float to = b == 255 ? 0.0f : __uint_as_float((uint32_t)(254 - b) << 23);   // 2^-e
    int8_t q[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
        // the clamp's order sends NaN (0 times an infinity, or a NaN) to -127; such a group's codes are not used, but defined
        const float r = fminf(fmaxf(rintf(v[j] * to), -127.0f), 127.0f);
        q[j] = b == 255 ? 0 : (int8_t)(int)r;
    }
    if (in >= W) {
        __builtin_memcpy(codes, q, W);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (j < in) codes[j] = q[j];
    }
    if (first) *scale = (uint8_t)b;
}

// A lane per chunk of a whole number of groups (chunks past the row's end hold zeros), kUnroll chunks in flight.
// MOVED: the last group holds at least a chunk.  A chunk that would pass the row's end, or begins after it, is moved back
// to end with the row: it stays in its group, so the group's largest value and the codes are the same, and what two lanes
// store they store alike.  No load or store has a condition then (128,000 x 312 fp32 with SiLU 83 us, 107 with them; x 311 bf16
// read back 20 us, 41 with them).
template <class T, bool SILU, bool MOVED>
__global__ __launch_bounds__(256) void k_checkpoint_save(Items it, int groups, int width, const T *__restrict__ z, int64_t ld,
                                                         T *__restrict__ y, int8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                         int8_t *__restrict__ ycodes, uint8_t *__restrict__ yscales) {
    constexpr int W = Chunk<T>::W, L = kGroupLanes<T>;
    const int64_t block = xcd_block();
    const int units = it.items / 256;
    int64_t row[kUnroll];
    int c[kUnroll];
    Chunk<T> v[kUnroll];
    const auto column = [&](int u) { return MOVED ? min(c[u] * W, width - W) : c[u] * W; };
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= units) break;
        item_at<L>(it, block, u, row[u], c[u]);
        const int left = MOVED ? W : width - c[u] * W;
        if (MOVED || left > 0) v[u].load(z + row[u] * ld + column(u), left);
        else __builtin_memset(&v[u], 0, sizeof v[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= units) break;
        const int left = MOVED ? W : width - c[u] * W;
        const int64_t at = row[u] * width + column(u), g = row[u] * groups + c[u] / L;
        float f[W];
#pragma unroll
        for (int j = 0; j < W; ++j) f[j] = to_f32(v[u].v[j]);
        save_chunk<T>(f, left, codes + at, scales + g, c[u] % L == 0);
        if (SILU) {
            Chunk<T> o;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float s, rest;
                sigmoids(f[j], s, rest);
                f[j] *= s;
                o.v[j] = from_f32<T>(f[j]);
            }
            if (MOVED || left > 0) o.store(y + at, left);
            if (ycodes) save_chunk<T>(f, left, ycodes + at, yscales + g, c[u] % L == 0);
        }
    }
}

// One chunk of a checkpoint as it is in memory.
template <int W>
struct Held {
    int8_t code[W];
    uint8_t scale;
    __device__ __forceinline__ void load(const int8_t *codes, const uint8_t *scales, int left) {
        if (left >= W) {
            __builtin_memcpy(code, codes, W);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) code[j] = j < left ? codes[j] : (int8_t)0;
        }
        scale = *scales;
    }
};

// out = the held values, or with dy the gradient dz = dy s (1 + z (1 - s)), s = sigma(z), at the held z
template <class T, bool BACK, bool MOVED>
__global__ __launch_bounds__(256) void k_checkpoint_use(Items it, int groups, int width, const T *__restrict__ dy, int64_t ld,
                                                        const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                                        T *__restrict__ out) {
    constexpr int W = Chunk<T>::W, L = kGroupLanes<T>;
    const int64_t block = xcd_block();
    const int units = it.items / 256;
    int64_t row[kUnroll];
    int c[kUnroll];
    Chunk<T> d[kUnroll];
    Held<W> z[kUnroll];
    const auto column = [&](int u) { return MOVED ? min(c[u] * W, width - W) : c[u] * W; };
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= units) break;
        item_at(it, block, u, row[u], c[u]);
        const int left = MOVED ? W : width - c[u] * W;
        if (BACK) d[u].load(dy + row[u] * ld + column(u), left);
        z[u].load(codes + row[u] * width + column(u), scales + row[u] * groups + c[u] / L, left);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= units) break;
        Chunk<T> o;
        const float step = step_of(z[u].scale);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float v = (float)z[u].code[j] * step;
            if (BACK) {
                float s, rest;
                sigmoids(v, s, rest);
                v = to_f32(d[u].v[j]) * s * fmaf(v, rest, 1.0f);
            }
            o.v[j] = from_f32<T>(v);
        }
        o.store(out + row[u] * width + column(u), MOVED ? W : width - c[u] * W);
    }
}

}  // namespace

// A row's last chunk may be moved back inside its group.
template <class T> static bool can_move(int width) { return width % kGroup == 0 || width % kGroup >= Chunk<T>::W; }

template <class T>
static Status save_t(Context &cx, bool silu, int64_t n, int width, const void *z, int64_t ld, void *y, int8_t *codes, uint8_t *scales,
                     int8_t *ycodes, uint8_t *yscales) {
    const int groups = (width + kGroup - 1) / kGroup;
    const bool moved = can_move<T>(width);
    auto *kernel = silu ? (moved ? k_checkpoint_save<T, true, true> : k_checkpoint_save<T, true, false>)
                        : (moved ? k_checkpoint_save<T, false, true> : k_checkpoint_save<T, false, false>);
    return by_launches(n, kLaunchBlocks * items_of(n, groups * kGroupLanes<T>).rows, [&](int64_t from, int64_t rows) -> Status {
        const Items it = items_of(rows, groups * kGroupLanes<T>);
        kernel<<<grid_of(it), 256, 0, cx.stream>>>(it, groups, width, (const T *)z + from * ld, ld, y ? (T *)y + from * width : nullptr,
                                                   codes + from * width, scales + from * groups,
                                                   ycodes ? ycodes + from * width : nullptr, yscales ? yscales + from * groups : nullptr);
        MPNN_HIP(hipGetLastError());
        return Status::ok();
    });
}

Status checkpoint_save(Context &cx, int dtype, bool silu, int64_t n, int width, const void *z, int64_t ld, void *y, int8_t *codes,
                       uint8_t *scales, int8_t *ycodes, uint8_t *yscales) {
    if (n == 0) return Status::ok();
    return dtype == MPNN_BF16 ? save_t<bf16>(cx, silu, n, width, z, ld, y, codes, scales, ycodes, yscales)
                              : save_t<float>(cx, silu, n, width, z, ld, y, codes, scales, ycodes, yscales);
}

template <class T, bool BACK>
static Status use_t(Context &cx, int64_t n, int width, const void *dy, int64_t ld, const int8_t *codes, const uint8_t *scales,
                    void *out) {
    const int groups = (width + kGroup - 1) / kGroup, chunks = (width + Chunk<T>::W - 1) / Chunk<T>::W;
    auto *kernel = can_move<T>(width) ? k_checkpoint_use<T, BACK, true> : k_checkpoint_use<T, BACK, false>;
    return by_launches(n, kLaunchBlocks * items_of(n, chunks).rows, [&](int64_t from, int64_t rows) -> Status {
        const Items it = items_of(rows, chunks);
        kernel<<<grid_of(it), 256, 0, cx.stream>>>(it, groups, width, dy ? (const T *)dy + from * ld : nullptr, ld, codes + from * width,
                                                   scales + from * groups, (T *)out + from * width);
        MPNN_HIP(hipGetLastError());
        return Status::ok();
    });
}

Status checkpoint_load(Context &cx, int dtype, int64_t n, int width, const int8_t *codes, const uint8_t *scales, void *out) {
    if (n == 0) return Status::ok();
    return dtype == MPNN_BF16 ? use_t<bf16, false>(cx, n, width, nullptr, 0, codes, scales, out)
                              : use_t<float, false>(cx, n, width, nullptr, 0, codes, scales, out);
}

Status checkpoint_silu_backward(Context &cx, int dtype, int64_t n, int width, const void *dy, int64_t ld, const int8_t *codes,
                                const uint8_t *scales, void *dz) {
    if (n == 0) return Status::ok();
    return dtype == MPNN_BF16 ? use_t<bf16, true>(cx, n, width, dy, ld, codes, scales, dz)
                              : use_t<float, true>(cx, n, width, dy, ld, codes, scales, dz);
}

}  // namespace mpnn
