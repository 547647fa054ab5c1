// C ABI of the rows sorted by expert and of the products with block scales
// (declared in include/spconv.h): argument checks.
#include "rows_args.cuh"

using namespace spconv;

namespace {

bool bad_pairs(int64_t tokens, int32_t k, int32_t n_experts) {
    return tokens < 0 || k < 1 || k > kMaxExperts || n_experts < 1 || n_experts > kMaxExperts || tokens * k >= (int64_t(1) << 30);
}
bool bad_dtype(int32_t dtype) { return dtype != SPCONV_BF16 && dtype != SPCONV_FP32; }
Rows ints(const int32_t* p, int64_t n) { return {p, 1, n, n, 4}; }
bool overlaps_any(const Rows& out, const Rows* ins, int count) {
    for (int i = 0; i < count; ++i)
        if (out.overlaps(ins[i])) return true;
    return false;
}

// The arguments that both products have; out and what it may not lie on.
int check_blocks(const BlockOp& op, int32_t c_in, int32_t c_out) {
    if (bad_sizes(op.n, c_in, c_out) || bad_act(op.act) || op.experts < 1 || op.experts > kMaxExperts ||
        (!op.offsets && op.experts != 1) || !aligned(op.offsets, 4))
        return SPCONV_ERR_INVALID_ARG;
    return c_in % 16 ? SPCONV_ERR_UNSUPPORTED : SPCONV_OK;
}
int run_blocks(const BlockOp& op, cudaStream_t s) {
    const int64_t wn = int64_t(op.experts) * op.h * op.k, kb = ceil_div(op.k, 128), hb = ceil_div(op.h, 128);
    const bool dual = op.w[1] != nullptr, eight = op.out_scale != nullptr;
    const Rows x{op.x, op.n, op.k, op.ldx, 1}, out{op.out, op.n, op.h, op.ld_out, eight ? size_t(1) : size_t(2)},
        scale = vec(op.out_scale, op.n * hb), res{op.extra, op.n, op.h, op.ld_extra, 2};
    const Rows ins[8] = {x, vec(op.x_scale, kb * op.n), {op.w[0], 1, wn, wn, 1}, {op.w[1], 1, wn, wn, 1},
                         vec(op.w_scale[0], op.experts * hb * kb), vec(op.w_scale[1], op.experts * hb * kb),
                         ints(op.offsets, op.experts + 1), vec(op.bias, int64_t(op.experts) * op.h)};
    if (!x.ok() || !out.ok() || !op.w[0] || !aligned(op.w[0], 16) || !aligned(op.w[1], 16) || (op.extra && !res.ok()))
        return SPCONV_ERR_INVALID_ARG;
    if (!op.x_scale || !op.w_scale[0] || (dual && !op.w_scale[1])) return SPCONV_ERR_INVALID_ARG;
    for (const float* v : {op.x_scale, op.w_scale[0], op.w_scale[1], op.bias, static_cast<const float*>(op.out_scale)})
        if (bad_vec(v)) return SPCONV_ERR_INVALID_ARG;
    if (overlaps_any(out, ins, 8) || overlaps_any(scale, ins, 8) || scale.overlaps(out) || (out.overlaps(res) && !out.same(res)))
        return SPCONV_ERR_ALIAS;
    return blocks_run(op, s);
}

}  // namespace

extern "C" {

int spconv_expert_plan(const void* experts_dev, int32_t index_bytes, int64_t tokens, int32_t k, int32_t n_experts,
                       int32_t* offsets_dev, int32_t* pairs_dev, int32_t* slots_dev, void* stream) {
    reset_launch_count();
    if (bad_pairs(tokens, k, n_experts) || (index_bytes != 4 && index_bytes != 8) || !offsets_dev || !aligned(offsets_dev, 4))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t pairs = tokens * k;
    if (pairs > 0) {
        if (!experts_dev || !aligned(experts_dev, index_bytes) || !pairs_dev || !aligned(pairs_dev, 4) || !slots_dev ||
            !aligned(slots_dev, 4))
            return SPCONV_ERR_INVALID_ARG;
        const Rows in{experts_dev, 1, pairs, pairs, static_cast<size_t>(index_bytes)};
        const Rows outs[3] = {ints(offsets_dev, n_experts + 1), ints(pairs_dev, pairs), ints(slots_dev, pairs)};
        for (int i = 0; i < 3; ++i)
            if (outs[i].overlaps(in) || overlaps_any(outs[i], outs, i)) return SPCONV_ERR_ALIAS;
    }
    return expert_plan(experts_dev, index_bytes, pairs, n_experts, offsets_dev, pairs_dev, slots_dev, static_cast<cudaStream_t>(stream));
}

int spconv_expert_gather(const void* x_dev, int64_t ld_x, const int32_t* slots_dev, const int32_t* offsets_dev, int64_t tokens,
                         int32_t k, int32_t n_experts, int32_t c, int32_t dtype, void* out_dev, int32_t out_dtype,
                         float* scale_dev, void* stream) {
    reset_launch_count();
    if (bad_pairs(tokens, k, n_experts) || bad_sizes(tokens, c, 1) || bad_dtype(dtype) ||
        (out_dtype != dtype && out_dtype != SPCONV_E4M3))
        return SPCONV_ERR_INVALID_ARG;
    if (tokens == 0) return SPCONV_OK;
    if ((scale_dev != nullptr) != (out_dtype == SPCONV_E4M3) || bad_vec(scale_dev)) return SPCONV_ERR_INVALID_ARG;
    const int64_t pairs = tokens * k;
    const Rows ins[3] = {{x_dev, tokens, c, ld_x, size_of(dtype)}, ints(slots_dev, pairs), ints(offsets_dev, n_experts + 1)};
    const Rows out{out_dev, pairs, c, c, size_of(out_dtype)}, scale = vec(scale_dev, pairs * ceil_div(c, 128));
    if (!ins[0].ok() || !ins[1].ok() || !ins[2].ok() || !out.ok()) return SPCONV_ERR_INVALID_ARG;
    if (overlaps_any(out, ins, 3) || overlaps_any(scale, ins, 3) || out.overlaps(scale)) return SPCONV_ERR_ALIAS;
    return expert_gather({x_dev, ld_x, slots_dev, offsets_dev, n_experts, tokens, k, c, dtype, out_dev, scale_dev, false},
                         static_cast<cudaStream_t>(stream));
}

int spconv_expert_combine(const void* y_dev, int64_t ld_y, const int32_t* slots_dev, const float* weights_dev,
                          const void* residual_dev, int64_t ld_residual, int64_t tokens, int32_t k, int32_t c, int32_t dtype,
                          void* out_dev, void* stream) {
    reset_launch_count();
    if (bad_pairs(tokens, k, 1) || bad_sizes(tokens, c, 1) || bad_dtype(dtype) || bad_vec(weights_dev)) return SPCONV_ERR_INVALID_ARG;
    if (tokens == 0) return SPCONV_OK;
    const int64_t pairs = tokens * k;
    const size_t es = size_of(dtype);
    const Rows ins[3] = {{y_dev, pairs, c, ld_y, es}, ints(slots_dev, pairs), vec(weights_dev, pairs)};
    const Rows res{residual_dev, tokens, c, ld_residual, es}, out{out_dev, tokens, c, c, es};
    if (!ins[0].ok() || !ins[1].ok() || !out.ok() || (residual_dev && !res.ok())) return SPCONV_ERR_INVALID_ARG;
    if (overlaps_any(out, ins, 3) || (out.overlaps(res) && !out.same(res))) return SPCONV_ERR_ALIAS;
    return expert_combine({y_dev, ld_y, slots_dev, weights_dev, residual_dev, ld_residual, tokens, k, c, dtype, out_dev},
                          static_cast<cudaStream_t>(stream));
}

int spconv_expert_combine_backward(const void* dout_dev, int64_t ld_dout, const void* y_dev, int64_t ld_y,
                                   const int32_t* slots_dev, const int32_t* offsets_dev, const float* weights_dev, int64_t tokens,
                                   int32_t k, int32_t n_experts, int32_t c, int32_t dtype, void* dy_dev, float* dweights_dev,
                                   void* stream) {
    reset_launch_count();
    if (bad_pairs(tokens, k, n_experts) || bad_sizes(tokens, c, 1) || bad_dtype(dtype)) return SPCONV_ERR_INVALID_ARG;
    if (tokens == 0) return SPCONV_OK;
    const int64_t pairs = tokens * k;
    const size_t es = size_of(dtype);
    const Rows ins[5] = {{dout_dev, tokens, c, ld_dout, es}, {y_dev, pairs, c, ld_y, es}, ints(slots_dev, pairs),
                         ints(offsets_dev, n_experts + 1), vec(weights_dev, pairs)};
    const Rows dy{dy_dev, pairs, c, c, es}, dw = vec(dweights_dev, pairs);
    for (const Rows& r : ins)
        if (!r.ok()) return SPCONV_ERR_INVALID_ARG;
    if (!dy.ok() || !dw.ok()) return SPCONV_ERR_INVALID_ARG;
    if (overlaps_any(dy, ins, 5) || overlaps_any(dw, ins, 5) || dy.overlaps(dw)) return SPCONV_ERR_ALIAS;
    return expert_combine_backward({dout_dev, ld_dout, y_dev, ld_y, slots_dev, offsets_dev, n_experts, weights_dev, tokens, k, c,
                                    dtype, dy_dev, dweights_dev},
                                   static_cast<cudaStream_t>(stream));
}

int spconv_quantize_blocks(const void* x_dev, int64_t ld_x, int64_t n, int32_t c, int32_t dtype, void* q_dev, float* scale_dev,
                           void* stream) {
    reset_launch_count();
    if (bad_sizes(n, c, 1) || bad_dtype(dtype)) return SPCONV_ERR_INVALID_ARG;
    if (n == 0) return SPCONV_OK;
    const Rows x{x_dev, n, c, ld_x, size_of(dtype)}, q{q_dev, n, c, c, 1}, scale = vec(scale_dev, n * ceil_div(c, 128));
    if (!x.ok() || !q.ok() || !scale.ok()) return SPCONV_ERR_INVALID_ARG;
    if (q.overlaps(x) || scale.overlaps(x) || q.overlaps(scale)) return SPCONV_ERR_ALIAS;
    return expert_gather({x_dev, ld_x, nullptr, nullptr, 0, n, 1, c, dtype, q_dev, scale_dev, false},
                         static_cast<cudaStream_t>(stream));
}

int spconv_quantize_weight_blocks(const void* w_dev, int32_t count, int32_t c_in, int32_t c_out, void* q_dev, float* scale_dev,
                                  void* stream) {
    reset_launch_count();
    if (bad_sizes(0, c_in, c_out) || count < 1 || count > kMaxExperts) return SPCONV_ERR_INVALID_ARG;
    const int64_t wn = int64_t(count) * c_in * c_out;
    const Rows w{w_dev, 1, wn, wn, 2}, q{q_dev, 1, wn, wn, 1}, scale = vec(scale_dev, count * ceil_div(c_in, 128) * ceil_div(c_out, 128));
    if (!w.ok() || !q.ok() || !scale.ok()) return SPCONV_ERR_INVALID_ARG;
    if (q.overlaps(w) || scale.overlaps(w) || q.overlaps(scale)) return SPCONV_ERR_ALIAS;
    return quantize_weight_blocks(w_dev, count, c_in, c_out, q_dev, scale_dev, static_cast<cudaStream_t>(stream));
}

int spconv_linear_blocks(const void* x_dev, int64_t ld_x, const float* x_scale_dev, const void* w_dev, const float* w_scale_dev,
                         const int32_t* offsets_dev, int32_t n_experts, int64_t n, int32_t c_in, int32_t c_out,
                         const float* bias_dev, int32_t activation, const void* residual_dev, int64_t ld_residual, void* out_dev,
                         int64_t ld_out, float* out_scale_dev, void* stream) {
    reset_launch_count();
    const BlockOp op{x_dev, ld_x, x_scale_dev, {w_dev, nullptr}, {w_scale_dev, nullptr}, offsets_dev, n_experts, n, c_in, c_out,
                     bias_dev, activation, residual_dev, ld_residual, out_dev, ld_out, out_scale_dev};
    SPCONV_CHECK(check_blocks(op, c_in, c_out));
    if (residual_dev && out_scale_dev) return SPCONV_ERR_UNSUPPORTED;
    if (n == 0) return SPCONV_OK;
    return run_blocks(op, static_cast<cudaStream_t>(stream));
}

int spconv_gated_ffn_blocks(const void* x_dev, int64_t ld_x, const float* x_scale_dev, const void* w_gate_dev,
                            const float* gate_scale_dev, const void* w_up_dev, const float* up_scale_dev,
                            const int32_t* offsets_dev, int32_t n_experts, int64_t n, int32_t c_in, int32_t c_hidden,
                            int32_t activation, void* out_dev, int64_t ld_out, float* out_scale_dev, void* stream) {
    reset_launch_count();
    const BlockOp op{x_dev, ld_x, x_scale_dev, {w_gate_dev, w_up_dev}, {gate_scale_dev, up_scale_dev}, offsets_dev, n_experts, n,
                     c_in, c_hidden, nullptr, activation, nullptr, 0, out_dev, ld_out, out_scale_dev};
    SPCONV_CHECK(check_blocks(op, c_in, c_hidden));
    if (n == 0) return SPCONV_OK;
    if (!w_up_dev) return SPCONV_ERR_INVALID_ARG;
    return run_blocks(op, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
