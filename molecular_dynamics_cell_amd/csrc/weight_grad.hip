// Weight gradients of one linear layer per expert from its saved input (mpnn_checkpoint_weight_grad):
//   dW_e[o][c] = sum over the rows q of expert e of dy[q][o] x[q][c],  db_e[o] = sum of dy[q][o],
// with x the values that the checkpoint holds.  The rows of an expert are cut into pieces of at most `rows`; each
// piece's product is a block's own partial sum, and the pieces of an expert are added in order, so results do not
// depend on the launch.
#include "impl.h"
#include "rows.h"

namespace mpnn {

namespace {

constexpr int kTile = 32;

// One block per (expert piece, 32 x 32 tile of dW): rows are read through LDS, 32 at a time.
template <class T>
__global__ void k_weight_grad(int out, int width, int groups, int n_experts, int64_t n, int64_t rows, int pieces,
                              const int32_t *__restrict__ offsets, const T *__restrict__ dy, int64_t ld,
                              const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales, float *__restrict__ part) {
    __shared__ float a[kTile][kTile + 1], b[kTile][kTile + 1];
    const int e = blockIdx.z / pieces, piece = blockIdx.z % pieces;
    const int64_t lo = min(max((int64_t)offsets[e], (int64_t)0), n), hi = min(max((int64_t)offsets[e + 1], lo), n);
    const int64_t from = lo + piece * rows, to = min(hi, from + rows);
    const int o0 = blockIdx.y * kTile, c0 = blockIdx.x * kTile;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    float s[4] = {}, sb[4] = {};
    for (int64_t q0 = from; q0 < to; q0 += kTile) {
        for (int j = ty; j < kTile; j += 8) {
            const int64_t q = q0 + j;
            a[j][tx] = q < to && o0 + tx < out ? to_f32(dy[q * ld + o0 + tx]) : 0.0f;
            float v = 0.0f;
            if (q < to && c0 + tx < width) {
                const int byte = scales[q * groups + (c0 + tx) / 32];
                v = (float)codes[q * width + c0 + tx] * (byte == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)byte << 23));
            }
            b[j][tx] = v;
        }
        __syncthreads();
        for (int j = 0; j < kTile; ++j)
            for (int u = 0; u < 4; ++u) {
                s[u] = fmaf(a[j][ty + 8 * u], b[j][tx], s[u]);
                sb[u] += a[j][ty + 8 * u];
            }
        __syncthreads();
    }
    float *to_p = part + (int64_t)blockIdx.z * out * (width + 1);
    for (int u = 0; u < 4; ++u) {
        const int o = o0 + ty + 8 * u;
        if (o >= out) continue;
        if (c0 + tx < width) to_p[(int64_t)o * width + c0 + tx] = s[u];
        if (c0 == 0 && tx == 0) to_p[(int64_t)out * width + o] = sb[u];
    }
}

__global__ void k_weight_grad_sum(int64_t values, int64_t matrix, int pieces, const float *__restrict__ part, float *__restrict__ dweight,
                                  float *__restrict__ dbias) {
    const int64_t v = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (v >= values) return;
    const int64_t e = blockIdx.y;
    float s = 0.0f;
    for (int p = 0; p < pieces; ++p) s += part[(e * pieces + p) * values + v];
    if (v < matrix) dweight[e * matrix + v] = s;
    else if (dbias) dbias[e * (values - matrix) + (v - matrix)] = s;
}

}  // namespace

template <class T>
static Status weight_grad_t(Context &cx, int64_t n, int out, int width, int n_experts, const int32_t *offsets, const void *dy,
                            int64_t ld, const int8_t *codes, const uint8_t *scales, float *dweight, float *dbias) {
    const int64_t tiles = (int64_t)((width + kTile - 1) / kTile) * ((out + kTile - 1) / kTile) * n_experts;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>((n + 255) / 256, 2048 / tiles));
    const int64_t rows = std::max<int64_t>(1, (n + want - 1) / want);
    const int pieces = (int)want;
    const int64_t values = (int64_t)out * (width + 1);
    MPNN_TRY(cx.grow(cx.rows_ws, sizeof(float) * (size_t)(values * pieces * n_experts)));
    k_weight_grad<T><<<dim3((width + kTile - 1) / kTile, (out + kTile - 1) / kTile, (unsigned)(pieces * n_experts)), 256, 0, cx.stream>>>(
        out, width, (width + 31) / 32, n_experts, n, rows, pieces, offsets, (const T *)dy, ld, codes, scales, cx.rows_ws.as<float>());
    MPNN_HIP(hipGetLastError());
    k_weight_grad_sum<<<dim3(grid_for(values), n_experts), kBlock, 0, cx.stream>>>(values, (int64_t)out * width, pieces,
                                                                                   cx.rows_ws.as<float>(), dweight, dbias);
    MPNN_HIP(hipGetLastError());
    return Status::ok();
}

Status weight_grad(Context &cx, int dtype, int64_t n, int out, int width, int n_experts, const int32_t *offsets, const void *dy,
                   int64_t ld, const int8_t *codes, const uint8_t *scales, float *dweight, float *dbias) {
    return dtype == MPNN_BF16 ? weight_grad_t<bf16>(cx, n, out, width, n_experts, offsets, dy, ld, codes, scales, dweight, dbias)
                              : weight_grad_t<float>(cx, n, out, width, n_experts, offsets, dy, ld, codes, scales, dweight, dbias);
}

}  // namespace mpnn
