// Rows in microscaled 4-bit floating point (mpnn_micro_save, mpnn_micro_load).  32 columns of a row share one
// power-of-two step 2^e:
//   largest = m 2^E, 1 <= m < 2:  e = E - 2, at least -100;  code = sign, nearest of 0 0.5 1 1.5 2 3 4 6 steps (6 at most)
// The scale byte holds e + 127; 255 marks a group with a value that is not finite and reads back as NaN.  A code times its
// step has two significant bits: exact in bf16 and fp32, so reading rounds nothing and a held row is a matrix-core operand.
// Rows are whole groups (the codes past the last column are zeros), so every group starts on 16 bytes.
//
// Bound by HBM: a lane takes eight columns, a group's largest comes from its three neighbours without LDS, and the hardware's
// conversions round (to nearest, ties to the even code) and keep in range.  8,192 x 4,096 bf16: held in 18 us (4.7 TB/s), read
// back in 14 (6.2 TB/s).
#include "impl.h"
#include "rows.h"
#include "tiles.h"

namespace mpnn {

namespace {

constexpr int kLeast = 127 - 100;

// WHOLE: rows of whole chunks of eight columns, whose loads and stores then have no condition beside them.
template <class T, bool WHOLE>
__global__ __launch_bounds__(256) void k_micro_save(Items it, int width, const T *__restrict__ x, int64_t ld, uint8_t *__restrict__ codes,
                                                    uint8_t *__restrict__ scales) {
    constexpr int W = 8;
    const int64_t block = xcd_block();
    if (block * it.rows >= it.n) return;
    Chunk<T, W> v[kUnroll];
    int64_t row[kUnroll];
    int c[kUnroll];
    const int many = it.items / 256;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= many) break;
        item_at<4>(it, block, u, row[u], c[u]);
        if (WHOLE) v[u].load(x + row[u] * ld + min(c[u] * W, width - W));
        else v[u].load(x + row[u] * ld + c[u] * W, width - c[u] * W);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= many) break;
        uint32_t m = 0;
        float f[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            f[j] = !WHOLE || c[u] * W < width ? to_f32(v[u].v[j]) : 0.0f;
            m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);      // magnitudes order as integers, a NaN above infinity
        }
        m = max(m, __float_as_uint(dpp<0xb1>(__uint_as_float(m))));
        m = max(m, __float_as_uint(dpp<0x4e>(__uint_as_float(m))));
        const bool fine = m < 0x7f800000u;
        const int byte = max((int)(m >> 23) - 2, kLeast);
        const float step = __uint_as_float((uint32_t)byte << 23);
        uint32_t o = 0;
        o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f[0], f[1], step, 0);
        o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f[2], f[3], step, 1);
        o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f[4], f[5], step, 2);
        o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f[6], f[7], step, 3);
        o = fine ? o : 0u;
        __builtin_memcpy(codes + (row[u] * it.per + c[u]) * 4, &o, 4);
        if (c[u] % 4 == 0) scales[row[u] * (it.per / 4) + c[u] / 4] = fine ? (uint8_t)byte : 255;
    }
}

template <class T, bool WHOLE>
__global__ __launch_bounds__(256) void k_micro_load(Items it, int width, const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                                    T *__restrict__ out) {
    const int64_t block = xcd_block();
    if (block * it.rows >= it.n) return;
    const int64_t groups = (width + kMicroGroup - 1) / kMicroGroup;
    uint32_t v[kUnroll];
    uint8_t s[kUnroll];
    int64_t row[kUnroll];
    int c[kUnroll];
    const int many = it.items / 256;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= many) break;
        item_at(it, block, u, row[u], c[u]);
        __builtin_memcpy(&v[u], codes + row[u] * groups * (kMicroGroup / 2) + c[u] * 4, 4);
        s[u] = scales[row[u] * groups + c[u] / 4];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (u >= many) break;
        const float step = micro_step(s[u]);
        Chunk<T, 8> o;
        const auto two = [&](auto k) {
            const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[u], step, k());
            o.v[2 * k()] = from_f32<T>(p[0]);
            o.v[2 * k() + 1] = from_f32<T>(p[1]);
        };
        two(std::integral_constant<int, 0>{});
        two(std::integral_constant<int, 1>{});
        two(std::integral_constant<int, 2>{});
        two(std::integral_constant<int, 3>{});
        if (WHOLE) o.store(out + row[u] * width + c[u] * 8);
        else o.store(out + row[u] * width + c[u] * 8, width - c[u] * 8);
    }
}

template <class T> Status save_t(Context &cx, int64_t n, int width, const T *x, int64_t ld, uint8_t *codes, uint8_t *scales) {
    const int groups = (width + kMicroGroup - 1) / kMicroGroup;
    return by_launches(n, kLaunchBlocks * items_of(n, groups * 4).rows, [&](int64_t from, int64_t rows) -> Status {
        const Items it = items_of(rows, groups * 4);
        auto *kernel = width % 8 ? k_micro_save<T, false> : k_micro_save<T, true>;
        kernel<<<grid_of(it), 256, 0, cx.stream>>>(it, width, x + from * ld, ld, codes + from * groups * (kMicroGroup / 2),
                                                           scales + from * groups);
        MPNN_HIP(hipGetLastError());
        return Status::ok();
    });
}

template <class T> Status load_t(Context &cx, int64_t n, int width, const uint8_t *codes, const uint8_t *scales, T *out) {
    const int groups = (width + kMicroGroup - 1) / kMicroGroup, per = (width + 7) / 8;
    return by_launches(n, kLaunchBlocks * items_of(n, per).rows, [&](int64_t from, int64_t rows) -> Status {
        const Items it = items_of(rows, per);
        auto *kernel = width % 8 ? k_micro_load<T, false> : k_micro_load<T, true>;
        kernel<<<grid_of(it), 256, 0, cx.stream>>>(it, width, codes + from * groups * (kMicroGroup / 2), scales + from * groups,
                                                           out + from * width);
        MPNN_HIP(hipGetLastError());
        return Status::ok();
    });
}

}  // namespace

Status micro_save(Context &cx, int dtype, int64_t n, int width, const void *x, int64_t ld, uint8_t *codes, uint8_t *scales) {
    if (n == 0) return Status::ok();
    return dtype == MPNN_BF16 ? save_t(cx, n, width, (const bf16 *)x, ld, codes, scales) : save_t(cx, n, width, (const float *)x, ld, codes, scales);
}

Status micro_load(Context &cx, int dtype, int64_t n, int width, const uint8_t *codes, const uint8_t *scales, void *out) {
    if (n == 0) return Status::ok();
    return dtype == MPNN_BF16 ? load_t(cx, n, width, codes, scales, (bf16 *)out) : load_t(cx, n, width, codes, scales, (float *)out);
}

}  // namespace mpnn
