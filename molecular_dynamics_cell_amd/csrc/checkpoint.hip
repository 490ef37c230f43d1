// Activation checkpoints in 8 bits (mpnn_checkpoint_*).  A group of 32 channels of a row shares one power-of-two
// step 2^e, the smallest that keeps the group's largest value within 127 steps:
//   largest = m 2^E, 1 <= m < 2:  e = E - 6 + (m > 127/64), clamped to -100 .. 121;  code = rint(v 2^-e) in +-127
// The scale byte holds e + 127; 255 marks a group with a value that is not finite and reads back as NaN.  With a
// power of two every code 2^e is exact in bf16 (and in fp32), so a checkpoint is a matrix-core operand as it stands
// and reading one back rounds nothing.
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
__device__ __forceinline__ int code_of(float v, int byte) {
    if (byte == 255) return 0;
    const float q = rintf(v * __uint_as_float((uint32_t)(254 - byte) << 23));   // 2^-e
    return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

// largest magnitude of a group; a NaN counts as the largest
__device__ __forceinline__ float group_max(float v) {
    uint32_t u = __float_as_uint(v) & 0x7fffffffu;   // magnitudes order as integers, NaN above infinity
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) u = max(u, (uint32_t)__shfl_xor((int)u, d));
    return __uint_as_float(u);
}

// One lane per channel, 32 lanes per group.
template <class T, bool SILU>
__global__ void k_checkpoint_save(int64_t items, int groups, int width, const T *__restrict__ z, int64_t ld, T *__restrict__ y,
                                  int8_t *__restrict__ codes, uint8_t *__restrict__ scales, int8_t *__restrict__ ycodes,
                                  uint8_t *__restrict__ yscales) {
    const int64_t g = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (g >= items) return;
    const int64_t i = g / groups;
    const int c = (int)(g - i * groups) * kGroup + (threadIdx.x & 31);
    const bool in = c < width;
    const float v = in ? to_f32(z[i * ld + c]) : 0.0f;
    int b = scale_byte(group_max(v));
    if (in) codes[i * width + c] = (int8_t)code_of(v, b);
    if ((threadIdx.x & 31) == 0) scales[g] = (uint8_t)b;
    if (SILU) {
        const float o = v / (1.0f + expf(-v));
        if (in) y[i * width + c] = from_f32<T>(o);
        if (ycodes) {
            b = scale_byte(group_max(o));
            if (in) ycodes[i * width + c] = (int8_t)code_of(o, b);
            if ((threadIdx.x & 31) == 0) yscales[g] = (uint8_t)b;
        }
    }
}

template <class T>
__global__ void k_checkpoint_load(int64_t n, int groups, int width, const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                  T *__restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (i >= n) return;
    for (int c = threadIdx.x & 63; c < width; c += 64)
        out[i * width + c] = from_f32<T>((float)codes[i * width + c] * step_of(scales[i * groups + c / kGroup]));
}

// dz = dy s (1 + z (1 - s)), s = sigma(z), for the z that the checkpoint holds
template <class T>
__global__ void k_checkpoint_silu_back(int64_t n, int groups, int width, const T *__restrict__ dy, int64_t ld,
                                       const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales, T *__restrict__ dz) {
    const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (i >= n) return;
    for (int c = threadIdx.x & 63; c < width; c += 64) {
        const float z = (float)codes[i * width + c] * step_of(scales[i * groups + c / kGroup]);
        const float s = 1.0f / (1.0f + expf(-z));
        dz[i * width + c] = from_f32<T>(to_f32(dy[i * ld + c]) * s * fmaf(z, 1.0f - s, 1.0f));
    }
}

}  // namespace

template <class T>
static Status save_t(Context &cx, bool silu, int64_t n, int width, const void *z, int64_t ld, void *y, int8_t *codes, uint8_t *scales,
                     int8_t *ycodes, uint8_t *yscales) {
    const int groups = (width + kGroup - 1) / kGroup;
    const int64_t items = n * groups;
    if (silu)
        k_checkpoint_save<T, true><<<grid_for(items, 8), 256, 0, cx.stream>>>(items, groups, width, (const T *)z, ld, (T *)y, codes,
                                                                              scales, ycodes, yscales);
    else
        k_checkpoint_save<T, false><<<grid_for(items, 8), 256, 0, cx.stream>>>(items, groups, width, (const T *)z, ld, nullptr, codes,
                                                                               scales, nullptr, nullptr);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

Status checkpoint_save(Context &cx, int dtype, bool silu, int64_t n, int width, const void *z, int64_t ld, void *y, int8_t *codes,
                       uint8_t *scales, int8_t *ycodes, uint8_t *yscales) {
    if (n == 0) return Status::ok();
    return dtype == MPNN_BF16 ? save_t<bf16>(cx, silu, n, width, z, ld, y, codes, scales, ycodes, yscales)
                              : save_t<float>(cx, silu, n, width, z, ld, y, codes, scales, ycodes, yscales);
}

Status checkpoint_load(Context &cx, int dtype, int64_t n, int width, const int8_t *codes, const uint8_t *scales, void *out) {
    if (n == 0) return Status::ok();
    const int groups = (width + kGroup - 1) / kGroup;
    if (dtype == MPNN_BF16)
        k_checkpoint_load<bf16><<<grid_for(n, 4), 256, 0, cx.stream>>>(n, groups, width, codes, scales, (bf16 *)out);
    else
        k_checkpoint_load<float><<<grid_for(n, 4), 256, 0, cx.stream>>>(n, groups, width, codes, scales, (float *)out);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

Status checkpoint_silu_backward(Context &cx, int dtype, int64_t n, int width, const void *dy, int64_t ld, const int8_t *codes,
                                const uint8_t *scales, void *dz) {
    if (n == 0) return Status::ok();
    const int groups = (width + kGroup - 1) / kGroup;
    if (dtype == MPNN_BF16)
        k_checkpoint_silu_back<bf16><<<grid_for(n, 4), 256, 0, cx.stream>>>(n, groups, width, (const bf16 *)dy, ld, codes, scales,
                                                                            (bf16 *)dz);
    else
        k_checkpoint_silu_back<float><<<grid_for(n, 4), 256, 0, cx.stream>>>(n, groups, width, (const float *)dy, ld, codes, scales,
                                                                             (float *)dz);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

}  // namespace mpnn
