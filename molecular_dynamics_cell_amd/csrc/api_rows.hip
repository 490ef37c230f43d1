// C ABI entry points of the row operators (include/mpnn.h): argument checks before any launch.
#include <cmath>

#include "impl.h"

using mpnn::Status;

namespace {

constexpr int32_t kMaxWidth = 1 << 20;      // columns of a routed or saved row
constexpr int32_t kMaxNorm = 8192;          // columns of a normed row
constexpr int32_t kMaxSlots = 64, kMaxExperts = 1024;

Status bad(const char *what) { return Status::err(MPNN_E_INVALID_ARG, what); }

// Runs the body and records its error on the context; nothing is thrown across the C boundary.
template <class F>
mpnn_status guarded(mpnn_ctx *ctx, F body) {
    if (!ctx) return MPNN_E_INVALID_ARG;
    try {
        const Status s = body(ctx->cx);
        ctx->cx.last_error = s.msg;
        return s.code;
    } catch (...) {
        return MPNN_E_OOM;
    }
}

Status check_rows(int32_t dtype, int64_t n, int32_t width, int32_t most) {
    if (dtype != MPNN_F32 && dtype != MPNN_BF16) return bad("dtype must be MPNN_F32 or MPNN_BF16");
    if (n < 0 || n > INT32_MAX) return bad("bad row count");
    if (width < 1 || width > most) return bad("bad width");
    return Status::ok();
}

Status check_pairs(int64_t n, int32_t k, int32_t n_experts) {
    if (n < 0) return bad("bad row count");
    if (k < 1 || k > kMaxSlots) return bad("slots per row must be in 1..64");
    if (n_experts < 1 || n_experts > kMaxExperts) return bad("n_experts must be in 1..1024");
    if (n > INT32_MAX / k) return Status::err(MPNN_E_CAPACITY, "more than 2^31-1 (row, slot) pairs");
    return Status::ok();
}

Status check_ld(int64_t ld, int32_t width, const char *what) { return ld < width ? bad(what) : Status::ok(); }

}  // namespace

extern "C" {

mpnn_status mpnn_route_plan(mpnn_ctx *ctx, int64_t n, int32_t k, int32_t n_experts, const int32_t *expert, int32_t *offsets,
                            int32_t *source, int32_t *position) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_pairs(n, k, n_experts));
        if (!offsets || (n > 0 && (!expert || !source || !position))) return bad("null array");
        return mpnn::route_plan(cx, n, k, n_experts, expert, offsets, source, position);
    });
}

mpnn_status mpnn_route_scatter(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t k, int32_t width, const void *x, int64_t ldx,
                               const int32_t *position, const int32_t *offsets, int32_t n_experts, void *sorted) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_rows(dtype, n, width, kMaxWidth));
        MPNN_TRY(check_pairs(n, k, n_experts));
        MPNN_TRY(check_ld(ldx, width, "ldx smaller than the width"));
        if (n > 0 && (!x || !position || !offsets || !sorted)) return bad("null array");
        return mpnn::route_scatter(cx, dtype, n, k, width, x, ldx, position, offsets + n_experts, sorted);
    });
}

mpnn_status mpnn_route_combine(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t k, int32_t width, const void *sorted,
                               const int32_t *position, const int32_t *offsets, int32_t n_experts, const float *weight, void *out) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_rows(dtype, n, width, kMaxWidth));
        MPNN_TRY(check_pairs(n, k, n_experts));
        if (n > 0 && (!sorted || !position || !offsets || !out)) return bad("null array");
        return mpnn::route_combine(cx, dtype, n, k, width, sorted, position, offsets + n_experts, weight, out);
    });
}

mpnn_status mpnn_route_combine_backward(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t k, int32_t width, const void *dout,
                                        int64_t ld_dout, const void *sorted, const int32_t *position, const int32_t *offsets,
                                        int32_t n_experts, const float *weight, void *dsorted, float *dweight) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_rows(dtype, n, width, kMaxWidth));
        MPNN_TRY(check_pairs(n, k, n_experts));
        MPNN_TRY(check_ld(ld_dout, width, "ld_dout smaller than the width"));
        if (n > 0 && (!dout || !position || !offsets || !dsorted)) return bad("null array");
        if (n > 0 && dweight && !sorted) return bad("dweight needs the sorted rows");
        return mpnn::route_combine_backward(cx, dtype, n, k, width, dout, ld_dout, sorted, position, offsets + n_experts, weight,
                                            dsorted, dweight);
    });
}

static Status check_norm(const mpnn_norm *p, int64_t n, bool block, bool gate) {
    if (!p) return bad("null norm description");
    MPNN_TRY(check_rows(p->dtype, n, p->width, kMaxNorm));
    if (p->kind != MPNN_NORM_RMS && p->kind != MPNN_NORM_LAYER) return bad("kind must be MPNN_NORM_RMS or MPNN_NORM_LAYER");
    if (!(p->eps > 0) || !std::isfinite(p->eps) || !((float)p->eps > 0.0f)) return bad("eps must be positive");
    if (gate && !block) return bad("a gate without a block");
    if (gate && p->gate_width != 1 && p->gate_width != p->width) return bad("gate_width must be 1 or the width");
    return Status::ok();
}

mpnn_status mpnn_norm_residual(mpnn_ctx *ctx, const mpnn_norm *p, int64_t n, const void *x, int64_t ldx, const void *block,
                               int64_t ld_block, const void *gate, int64_t ld_gate, void *r, void *h) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_norm(p, n, block, gate));
        MPNN_TRY(check_ld(ldx, p->width, "ldx smaller than the width"));
        if (block) MPNN_TRY(check_ld(ld_block, p->width, "ld_block smaller than the width"));
        if (gate) MPNN_TRY(check_ld(ld_gate, p->gate_width, "ld_gate smaller than gate_width"));
        if (n > 0 && !x) return bad("null array");
        if (n > 0 && !r && !h) return bad("no output");
        return mpnn::norm_residual(cx, *p, n, x, ldx, block, ld_block, gate, ld_gate, r, h);
    });
}

mpnn_status mpnn_norm_residual_backward(mpnn_ctx *ctx, const mpnn_norm *p, int64_t n, const void *dr, const void *dh, const void *r,
                                        int64_t ldr, const void *block, int64_t ld_block, const void *gate, int64_t ld_gate,
                                        void *dx, void *dblock, void *dgate, float *dpost_weight, float *dpost_bias, float *dscale,
                                        float *dpre_weight, float *dpre_bias) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_norm(p, n, block, gate));
        if (dh) MPNN_TRY(check_ld(ldr, p->width, "ldr smaller than the width"));
        if (block) MPNN_TRY(check_ld(ld_block, p->width, "ld_block smaller than the width"));
        if (gate) MPNN_TRY(check_ld(ld_gate, p->gate_width, "ld_gate smaller than gate_width"));
        if (n > 0 && !dr && !dh) return bad("no incoming gradient");
        if (n > 0 && dh && !r) return bad("dh needs r");
        if (n > 0 && block && !dblock) return bad("null dblock");
        if (n > 0 && gate && !dgate) return bad("null dgate");
        float *const d[5] = {dpost_weight, dpost_bias, dscale, dpre_weight, dpre_bias};
        return mpnn::norm_residual_backward(cx, *p, n, dr, dh, r, ldr, block, ld_block, gate, ld_gate, dx, dblock, dgate, d);
    });
}

mpnn_status mpnn_checkpoint_save(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t width, const void *x, int64_t ldx, int8_t *codes,
                                 uint8_t *scales) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_rows(dtype, n, width, kMaxWidth));
        MPNN_TRY(check_ld(ldx, width, "ldx smaller than the width"));
        if (n > 0 && (!x || !codes || !scales)) return bad("null array");
        return mpnn::checkpoint_save(cx, dtype, false, n, width, x, ldx, nullptr, codes, scales, nullptr, nullptr);
    });
}

mpnn_status mpnn_checkpoint_load(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t width, const int8_t *codes, const uint8_t *scales,
                                 void *out) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_rows(dtype, n, width, kMaxWidth));
        if (n > 0 && (!codes || !scales || !out)) return bad("null array");
        return mpnn::checkpoint_load(cx, dtype, n, width, codes, scales, out);
    });
}

mpnn_status mpnn_checkpoint_silu(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t width, const void *z, int64_t ldz, void *y,
                                 int8_t *z_codes, uint8_t *z_scales, int8_t *y_codes, uint8_t *y_scales) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_rows(dtype, n, width, kMaxWidth));
        MPNN_TRY(check_ld(ldz, width, "ldz smaller than the width"));
        if (n > 0 && (!z || !y || !z_codes || !z_scales)) return bad("null array");
        if ((y_codes == nullptr) != (y_scales == nullptr)) return bad("y_codes and y_scales go together");
        return mpnn::checkpoint_save(cx, dtype, true, n, width, z, ldz, y, z_codes, z_scales, y_codes, y_scales);
    });
}

mpnn_status mpnn_checkpoint_silu_backward(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t width, const void *dy, int64_t ld_dy,
                                          const int8_t *codes, const uint8_t *scales, void *dz) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_rows(dtype, n, width, kMaxWidth));
        MPNN_TRY(check_ld(ld_dy, width, "ld_dy smaller than the width"));
        if (n > 0 && (!dy || !codes || !scales || !dz)) return bad("null array");
        return mpnn::checkpoint_silu_backward(cx, dtype, n, width, dy, ld_dy, codes, scales, dz);
    });
}

mpnn_status mpnn_checkpoint_weight_grad(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t n_out, int32_t width, int32_t n_experts,
                                        const int32_t *offsets, const void *dy, int64_t ld_dy, const int8_t *codes,
                                        const uint8_t *scales, float *dweight, float *dbias) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_rows(dtype, n, width, 1 << 16));
        if (n_out < 1 || n_out > 1 << 16) return bad("bad output width");
        if (n_experts < 1 || n_experts > kMaxExperts) return bad("n_experts must be in 1..1024");
        MPNN_TRY(check_ld(ld_dy, n_out, "ld_dy smaller than the output width"));
        if (ld_dy > 1 << 24) return bad("ld_dy larger than 2^24");
        if (!offsets || !dweight || (n > 0 && (!dy || !codes || !scales))) return bad("null array");
        return mpnn::weight_grad(cx, dtype, n, n_out, width, n_experts, offsets, dy, ld_dy, codes, scales, dweight, dbias);
    });
}

static Status check_product(int32_t dtype, int64_t n, int32_t width, int32_t n_out, int32_t n_experts, const int32_t *offsets) {
    MPNN_TRY(check_rows(dtype, n, width, 1 << 16));
    if (n_out < 1 || n_out > 1 << 16) return bad("bad output width");
    if (n_experts < 1 || n_experts > kMaxExperts) return bad("n_experts must be in 1..1024");
    if (!offsets) return bad("null array");
    return Status::ok();
}

static Status check_source(int64_t n, const int32_t *source, int64_t n_x) {
    if (!source || n == 0) return Status::ok();
    if (n_x < 1 || n % n_x || n / n_x > kMaxSlots) return bad("with a source n must be n_x times 1..64 slots");
    return Status::ok();
}

static Status check_act(int32_t act) { return act == MPNN_ACT_NONE || act == MPNN_ACT_SILU ? Status::ok() : bad("bad activation"); }

mpnn_status mpnn_expert_product(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t width, int32_t n_out, int32_t n_experts,
                                const int32_t *offsets, const void *x, int64_t ldx, const int32_t *source, int64_t n_x,
                                const void *weight, const float *bias, int32_t act, void *y) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_product(dtype, n, width, n_out, n_experts, offsets));
        MPNN_TRY(check_ld(ldx, width, "ldx smaller than the width"));
        MPNN_TRY(check_source(n, source, n_x));
        MPNN_TRY(check_act(act));
        if (n > 0 && (!x || !weight || !y)) return bad("null array");
        return mpnn::expert_product(cx, dtype, n, width, n_out, n_experts, offsets, x, ldx, source, n_x, weight, bias, act, y);
    });
}

mpnn_status mpnn_expert_input_grad(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t width, int32_t n_out, int32_t n_experts,
                                   const int32_t *offsets, const void *dy, int64_t ld_dy, const void *weight, void *dx) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_product(dtype, n, width, n_out, n_experts, offsets));
        MPNN_TRY(check_ld(ld_dy, n_out, "ld_dy smaller than the output width"));
        if (n > 0 && (!dy || !weight || !dx)) return bad("null array");
        return mpnn::expert_input_grad(cx, dtype, n, width, n_out, n_experts, offsets, dy, ld_dy, weight, dx);
    });
}

mpnn_status mpnn_expert_weight_grad(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t width, int32_t n_out, int32_t n_experts,
                                    const int32_t *offsets, const void *dy, int64_t ld_dy, const void *x, int64_t ldx,
                                    const int32_t *source, int64_t n_x, float *dweight, float *dbias) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_product(dtype, n, width, n_out, n_experts, offsets));
        MPNN_TRY(check_ld(ld_dy, n_out, "ld_dy smaller than the output width"));
        MPNN_TRY(check_ld(ldx, width, "ldx smaller than the width"));
        MPNN_TRY(check_source(n, source, n_x));
        if (!dweight || (n > 0 && (!dy || !x))) return bad("null array");
        return mpnn::expert_weight_grad(cx, dtype, n, width, n_out, n_experts, offsets, dy, ld_dy, x, ldx, source, n_x, dweight, dbias);
    });
}

mpnn_status mpnn_micro_save(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t width, const void *x, int64_t ldx, uint8_t *codes,
                            uint8_t *scales) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_rows(dtype, n, width, kMaxWidth));
        MPNN_TRY(check_ld(ldx, width, "ldx smaller than the width"));
        if (n > 0 && (!x || !codes || !scales)) return bad("null array");
        return mpnn::micro_save(cx, dtype, n, width, x, ldx, codes, scales);
    });
}

mpnn_status mpnn_micro_load(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t width, const uint8_t *codes, const uint8_t *scales,
                            void *out) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_rows(dtype, n, width, kMaxWidth));
        if (n > 0 && (!codes || !scales || !out)) return bad("null array");
        return mpnn::micro_load(cx, dtype, n, width, codes, scales, out);
    });
}

mpnn_status mpnn_micro_product(mpnn_ctx *ctx, int32_t x_dtype, int32_t y_dtype, int64_t n, int32_t width, int32_t n_out,
                               int32_t n_experts, const int32_t *offsets, const void *x, int64_t ldx, const uint8_t *x_scales,
                               const int32_t *source, int64_t n_x, const uint8_t *codes, const uint8_t *scales, const float *bias,
                               int32_t act, void *y) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_product(x_dtype == MPNN_MICRO ? MPNN_F32 : x_dtype, n, width, n_out, n_experts, offsets));
        if (y_dtype != MPNN_F32 && y_dtype != MPNN_BF16) return bad("y_dtype must be MPNN_F32 or MPNN_BF16");
        if (x_dtype != MPNN_MICRO) MPNN_TRY(check_ld(ldx, width, "ldx smaller than the width"));
        MPNN_TRY(check_source(n, source, n_x));
        MPNN_TRY(check_act(act));
        if (n > 0 && (!x || !codes || !scales || !y || (x_dtype == MPNN_MICRO && !x_scales))) return bad("null array");
        return mpnn::micro_product(cx, x_dtype, y_dtype, n, width, n_out, n_experts, offsets, x, ldx, x_scales, source, n_x, codes, scales, bias, act, y);
    });
}

static Status check_entries(int64_t n, int32_t n_entries, double scale) {
    if (n < 0 || n > INT32_MAX) return bad("bad row count");
    if (n_entries < 1 || n_entries > 1 << 20) return bad("n_entries must be in 1..2^20");
    if (!std::isfinite(scale) || !std::isfinite((float)scale)) return bad("scale must be finite");
    return Status::ok();
}

mpnn_status mpnn_embed(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t width, int32_t n_entries, const int32_t *index,
                       const void *table, double scale, void *out) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_rows(dtype, n, width, kMaxWidth));
        MPNN_TRY(check_entries(n, n_entries, scale));
        if (n > 0 && (!index || !table || !out)) return bad("null array");
        return mpnn::embed(cx, dtype, n, width, n_entries, index, table, (float)scale, out);
    });
}

mpnn_status mpnn_embed_plan(mpnn_ctx *ctx, int64_t n, int32_t n_entries, const int32_t *index, int32_t *offsets, int32_t *source) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_entries(n, n_entries, 1.0));
        if (!offsets || (n > 0 && (!index || !source))) return bad("null array");
        return mpnn::embed_plan(cx, n, n_entries, index, offsets, source);
    });
}

mpnn_status mpnn_embed_backward(mpnn_ctx *ctx, int32_t dtype, int64_t n, int32_t width, int32_t n_entries, const void *dout,
                                int64_t ld_dout, const int32_t *offsets, const int32_t *source, double scale, float *dtable) {
    return guarded(ctx, [&](mpnn::Context &cx) -> Status {
        MPNN_TRY(check_rows(dtype, n, width, kMaxWidth));
        MPNN_TRY(check_entries(n, n_entries, scale));
        MPNN_TRY(check_ld(ld_dout, width, "ld_dout smaller than the width"));
        if (!offsets || !dtable || (n > 0 && (!dout || !source))) return bad("null array");
        return mpnn::embed_backward(cx, dtype, n, width, n_entries, dout, ld_dout, offsets, source, (float)scale, dtable);
    });
}

}  // extern "C"
