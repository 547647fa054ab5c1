// C ABI of the row-wise operators (declared in include/spconv.h): argument
// checks, and the products that each operator is made of.
#include "rows.cuh"

using namespace spconv;

namespace {

constexpr int32_t kMaxChannels = 65536;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A row matrix as the caller gave it: n rows of c elements, ld elements apart.
struct Rows {
    const void* p;
    int64_t n, c, ld;
    size_t es;
    bool ok() const { return p && aligned(p, es) && ld >= c && ld < (int64_t(1) << 38); }
    size_t bytes() const { return n == 0 ? 0 : (static_cast<size_t>(n - 1) * ld + c) * es; }
    bool overlaps(const Rows& o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        if (!p || !o.p || a >= b + o.bytes() || b >= a + bytes()) return false;
        // column ranges of one wider matrix: the rows interleave without touching
        const uintptr_t pitch = static_cast<uintptr_t>(ld) * es;
        if (n > 1 && o.n > 1 && pitch == static_cast<uintptr_t>(o.ld) * o.es) {
            const uintptr_t d = b >= a ? (b - a) % pitch : (pitch - (a - b) % pitch) % pitch;   // o's row after this one's
            return d < static_cast<uintptr_t>(c) * es || d + static_cast<uintptr_t>(o.c) * o.es > pitch;
        }
        return true;
    }
    // the same rows at the same places: an in-place update
    bool same(const Rows& o) const { return p == o.p && (ld == o.ld || n <= 1); }
};

// fp32 values in a row (absent: null, which overlaps nothing)
Rows vec(const float* p, int64_t c) { return {p, 1, c, c, 4}; }

size_t size_of(int32_t dtype) { return dtype == SPCONV_FP32 ? 4 : dtype == SPCONV_E4M3 ? 1 : 2; }

bool bad_sizes(int64_t n, int32_t c_in, int32_t c_out) {
    return n < 0 || n >= (int64_t(1) << 30) || c_in < 1 || c_out < 1 || c_in > kMaxChannels || c_out > kMaxChannels;
}
bool bad_act(int32_t a) { return a < SPCONV_ACT_NONE || a > SPCONV_ACT_GELU_TANH; }
bool bad_vec(const float* v) { return !aligned(v, 4); }

// e4m3 operands need their scales, bf16 ones have none.
int check_scales(int32_t dtype, const float* a, const float* b) {
    if (dtype != SPCONV_BF16 && dtype != SPCONV_E4M3)
        return dtype == SPCONV_FP32 ? SPCONV_ERR_UNSUPPORTED : SPCONV_ERR_INVALID_ARG;
    const bool eight = dtype == SPCONV_E4M3;
    if ((a != nullptr) != eight || (b != nullptr) != eight || bad_vec(a) || bad_vec(b)) return SPCONV_ERR_INVALID_ARG;
    return SPCONV_OK;
}

// x [n][c_in] times a weight: bf16 [c_in][c_out], e4m3 [c_out][c_in], its rows
// ld_w apart.
DenseOp product(const Rows& x, const void* w, int64_t ld_w, int32_t c_out, int32_t dtype) {
    DenseOp op;
    op.m = x.n;
    op.n = c_out;
    op.k = x.c;
    op.dtype = dtype;
    op.a.p[0] = x.p;
    op.a.ld = x.ld;
    op.a.k_major = true;
    op.b.p[0] = w;
    op.b.k_major = dtype == SPCONV_E4M3;
    op.b.ld = ld_w;
    return op;
}

// dz [n][c_out] times the transposed bf16 weight [c_in][c_out].
DenseOp product_t(const Rows& dz, const void* w, int64_t ld_w, int32_t c_in) {
    DenseOp op;
    op.m = dz.n;
    op.n = c_in;
    op.k = dz.c;
    op.a.p[0] = dz.p;
    op.a.ld = dz.ld;
    op.b.p[0] = w;
    op.b.ld = ld_w;
    return op;
}

// x^T dz, [c_in][c_out], over the rows.
DenseOp outer(const Rows& x, const Rows& dz) {
    DenseOp op;
    op.m = x.c;
    op.n = dz.c;
    op.k = x.n;
    op.a.p[0] = x.p;
    op.a.ld = x.ld;
    op.a.k_major = false;
    op.b.p[0] = dz.p;
    op.b.ld = dz.ld;
    op.b.k_major = false;
    op.ld_out = dz.c;
    return op;
}

int zero(void* p, size_t bytes, cudaStream_t s) { return p ? cuda_status(cudaMemsetAsync(p, 0, bytes, s)) : SPCONV_OK; }

}  // namespace

extern "C" {

int spconv_rms_norm(const void* x_dev, int64_t ld_x, const void* residual_dev, int64_t ld_residual, const float* weight_dev,
                    int64_t n, int32_t c, int32_t dtype, float eps, void* sum_dev, void* out_dev, int32_t out_dtype,
                    float* scale_dev, void* stream) {
    reset_launch_count();
    if (bad_sizes(n, c, 1) || !(eps >= 0.0f)) return SPCONV_ERR_INVALID_ARG;
    if (dtype != SPCONV_BF16 && dtype != SPCONV_FP32) return SPCONV_ERR_INVALID_ARG;
    if (out_dtype != dtype && out_dtype != SPCONV_E4M3) return SPCONV_ERR_INVALID_ARG;
    if (n == 0) return SPCONV_OK;
    if ((scale_dev != nullptr) != (out_dtype == SPCONV_E4M3) || bad_vec(scale_dev)) return SPCONV_ERR_INVALID_ARG;
    const size_t es = size_of(dtype);
    const Rows x{x_dev, n, c, ld_x, es}, res{residual_dev, n, c, ld_residual, es}, sum{sum_dev, n, c, c, es},
        out{out_dev, n, c, c, size_of(out_dtype)}, scale = vec(scale_dev, n), w = vec(weight_dev, c);
    if (!x.ok() || !out.ok() || !weight_dev || bad_vec(weight_dev)) return SPCONV_ERR_INVALID_ARG;
    if ((residual_dev && !res.ok()) || (sum_dev && !sum.ok())) return SPCONV_ERR_INVALID_ARG;
    if (out.overlaps(x) || out.overlaps(res) || out.overlaps(sum) || scale.overlaps(out) || scale.overlaps(x) ||
        scale.overlaps(res) || scale.overlaps(sum) || w.overlaps(out) || w.overlaps(sum) || w.overlaps(scale))
        return SPCONV_ERR_ALIAS;
    if ((sum.overlaps(x) && !sum.same(x)) || (sum.overlaps(res) && !sum.same(res))) return SPCONV_ERR_ALIAS;
    return norm_forward({x_dev, ld_x, residual_dev, ld_residual, weight_dev, n, c, dtype, eps, sum_dev, out_dev, out_dtype,
                         scale_dev},
                        static_cast<cudaStream_t>(stream));
}

int spconv_rms_norm_backward(const void* dy_dev, int64_t ld_dy, const void* x_dev, int64_t ld_x, const float* weight_dev,
                             const void* dres_dev, int64_t ld_dres, int64_t n, int32_t c, int32_t dtype, float eps,
                             void* dx_dev, float* dweight_dev, void* stream) {
    reset_launch_count();
    if (bad_sizes(n, c, 1) || !(eps >= 0.0f)) return SPCONV_ERR_INVALID_ARG;
    if (dtype != SPCONV_BF16 && dtype != SPCONV_FP32) return SPCONV_ERR_INVALID_ARG;
    if (!dweight_dev || bad_vec(dweight_dev)) return SPCONV_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n == 0) return zero(dweight_dev, static_cast<size_t>(c) * 4, s);
    const size_t es = size_of(dtype);
    const Rows dy{dy_dev, n, c, ld_dy, es}, x{x_dev, n, c, ld_x, es}, dres{dres_dev, n, c, ld_dres, es},
        dx{dx_dev, n, c, c, es}, dw = vec(dweight_dev, c), w = vec(weight_dev, c);
    if (!dy.ok() || !x.ok() || !dx.ok() || !weight_dev || bad_vec(weight_dev) || (dres_dev && !dres.ok()))
        return SPCONV_ERR_INVALID_ARG;
    if (dx.overlaps(x) || dx.overlaps(dy) || (dx.overlaps(dres) && !dx.same(dres)) || dw.overlaps(dx) || dw.overlaps(x) ||
        dw.overlaps(dy) || dw.overlaps(dres) || w.overlaps(dx) || w.overlaps(dw))
        return SPCONV_ERR_ALIAS;
    return norm_backward({dy_dev, ld_dy, x_dev, ld_x, weight_dev, dres_dev, ld_dres, n, c, dtype, eps, dx_dev, dweight_dev}, s);
}

int spconv_linear(const void* x_dev, int64_t ld_x, const float* x_scale_dev, const void* w_dev, const float* w_scale_dev,
                  int64_t n, int32_t c_in, int32_t c_out, int32_t dtype, const float* bias_dev, int32_t activation,
                  const void* residual_dev, int64_t ld_residual, void* out_dev, int64_t ld_out, void* stream) {
    reset_launch_count();
    if (bad_sizes(n, c_in, c_out) || bad_act(activation) || bad_vec(bias_dev)) return SPCONV_ERR_INVALID_ARG;
    if (n == 0) return SPCONV_OK;
    SPCONV_CHECK(check_scales(dtype, x_scale_dev, w_scale_dev));
    const size_t es = size_of(dtype);
    const Rows x{x_dev, n, c_in, ld_x, es}, w{w_dev, 1, int64_t(c_in) * c_out, int64_t(c_in) * c_out, es},
        res{residual_dev, n, c_out, ld_residual, 2}, out{out_dev, n, c_out, ld_out, 2};
    if (!x.ok() || !w.ok() || !out.ok() || (residual_dev && !res.ok())) return SPCONV_ERR_INVALID_ARG;
    if (out.overlaps(x) || out.overlaps(w) || (out.overlaps(res) && !out.same(res)) || out.overlaps(vec(bias_dev, c_out)) ||
        out.overlaps(vec(x_scale_dev, n)) || out.overlaps(vec(w_scale_dev, c_out)))
        return SPCONV_ERR_ALIAS;
    DenseOp op = product(x, w_dev, dtype == SPCONV_E4M3 ? c_in : c_out, c_out, dtype);
    op.row_scale = x_scale_dev;
    op.col_scale[0] = w_scale_dev;
    op.bias = bias_dev;
    op.act = activation;
    op.extra = residual_dev;
    op.ld_extra = ld_residual;
    op.out[0] = out_dev;
    op.ld_out = ld_out;
    return dense_run(op, static_cast<cudaStream_t>(stream));
}

int spconv_linear_backward(const void* dy_dev, int64_t ld_dy, const void* x_dev, int64_t ld_x, const void* w_dev, int64_t n,
                           int32_t c_in, int32_t c_out, int32_t dtype, const float* bias_dev, int32_t activation,
                           void* dx_dev, void* dw_dev, float* dbias_dev, void* stream) {
    reset_launch_count();
    if (bad_sizes(n, c_in, c_out) || bad_act(activation) || bad_vec(bias_dev) || bad_vec(dbias_dev))
        return SPCONV_ERR_INVALID_ARG;
    if (dtype != SPCONV_BF16) return dtype == SPCONV_FP32 || dtype == SPCONV_E4M3 ? SPCONV_ERR_UNSUPPORTED : SPCONV_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t wn = int64_t(c_in) * c_out;
    if (n == 0) {
        SPCONV_CHECK(zero(dw_dev, wn * 2, s));
        return zero(dbias_dev, static_cast<size_t>(c_out) * 4, s);
    }
    Rows dy{dy_dev, n, c_out, ld_dy, 2}, x{x_dev, n, c_in, ld_x, 2};
    const Rows w{w_dev, 1, wn, wn, 2};
    const Rows outs[3] = {{dx_dev, n, c_in, c_in, 2}, {dw_dev, 1, wn, wn, 2}, vec(dbias_dev, c_out)};
    if (!dy.ok() || !x.ok() || !w.ok()) return SPCONV_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) {
        if (!outs[i].p) continue;
        if (!outs[i].ok()) return SPCONV_ERR_INVALID_ARG;
        if (outs[i].overlaps(dy) || outs[i].overlaps(x) || outs[i].overlaps(w) || outs[i].overlaps(vec(bias_dev, c_out)))
            return SPCONV_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (outs[i].overlaps(outs[j])) return SPCONV_ERR_ALIAS;
    }
    if (!dx_dev && !dw_dev && !dbias_dev) return SPCONV_OK;
    const bool act = activation != SPCONV_ACT_NONE;
    // what two products read is brought into alignment once
    AlignedRows rows;
    int64_t ld_w = c_out;
    if (act || dw_dev) rows.add(&x.p, 1, &x.ld, n, c_in, 2);
    if (act || dx_dev) rows.add(&w_dev, 1, &ld_w, c_in, c_out, 2);
    if (act || dw_dev || dx_dev) rows.add(&dy.p, 1, &dy.ld, n, c_out, 2);
    SPCONV_CHECK(rows.run(s));
    const int64_t ld_dz = static_cast<int64_t>(round_up(c_out, 8));   // whole 16-byte rows
    ColumnSums cols;
    cols.n = c_out;
    cols.out = dbias_dev;
    if (dbias_dev) cols.rows = act ? col_part_rows(n) : column_part_rows(n, c_out);
    // dz, then the partial column sums.  dz is an operand of two products on the
    // bf16 tensor pipe, so it is rounded once like any other: dx and dw are off by
    // 2.3e-3 of their size, by their own rounding alone 1.7e-3.  Kept in 32 bits it
    // would need products at half the rate (tf32) or twice as many (two halves).
    const size_t dz_bytes = act ? round_up(static_cast<size_t>(n) * ld_dz * 2, 256) : 0;
    Scratch buf(dz_bytes + static_cast<size_t>(cols.rows) * c_out * 4, s);
    if (buf.failed()) return SPCONV_ERR_OOM;
    float* col_part = buf.as<float>(dz_bytes);
    cols.part = col_part;
    Rows dz = dy;
    if (act) {
        DenseOp op = product(x, w_dev, ld_w, c_out, SPCONV_BF16);
        op.epi = kEpiActGrad;
        op.act = activation;
        op.bias = bias_dev;
        op.extra = dy.p;
        op.ld_extra = dy.ld;
        op.out[0] = buf.as<void>();
        op.ld_out = ld_dz;
        op.out_padded = true;
        op.col_part = dbias_dev ? col_part : nullptr;
        SPCONV_CHECK(dense_run(op, s));
        dz = Rows{buf.as<void>(), n, c_out, ld_dz, 2};
    } else if (dbias_dev) {
        SPCONV_CHECK(column_parts(dy.p, dy.ld, n, c_out, col_part, s));
    }
    DenseOp ops[2];
    int count = 0;
    if (dw_dev) {
        ops[count] = outer(x, dz);
        ops[count++].out[0] = dw_dev;
    }
    if (dx_dev) {
        ops[count] = product_t(dz, w_dev, ld_w, c_in);
        ops[count].ld_out = c_in;
        ops[count++].out[0] = dx_dev;
    }
    return dense_run_plain(ops, count, cols, s);
}

int spconv_gated_ffn(const void* x_dev, int64_t ld_x, const float* x_scale_dev, const void* w_gate_dev,
                     const float* gate_scale_dev, const void* w_up_dev, const float* up_scale_dev, int64_t n, int32_t c_in,
                     int32_t c_hidden, int32_t dtype, int32_t activation, void* out_dev, int64_t ld_out, void* stream) {
    reset_launch_count();
    if (bad_sizes(n, c_in, c_hidden) || bad_act(activation)) return SPCONV_ERR_INVALID_ARG;
    if (n == 0) return SPCONV_OK;
    SPCONV_CHECK(check_scales(dtype, x_scale_dev, gate_scale_dev));
    SPCONV_CHECK(check_scales(dtype, x_scale_dev, up_scale_dev));
    const size_t es = size_of(dtype);
    const int64_t wn = int64_t(c_in) * c_hidden;
    const Rows x{x_dev, n, c_in, ld_x, es}, wg{w_gate_dev, 1, wn, wn, es}, wu{w_up_dev, 1, wn, wn, es},
        out{out_dev, n, c_hidden, ld_out, 2};
    if (!x.ok() || !wg.ok() || !wu.ok() || !out.ok()) return SPCONV_ERR_INVALID_ARG;
    if (out.overlaps(x) || out.overlaps(wg) || out.overlaps(wu) || out.overlaps(vec(x_scale_dev, n)) ||
        out.overlaps(vec(gate_scale_dev, c_hidden)) || out.overlaps(vec(up_scale_dev, c_hidden)))
        return SPCONV_ERR_ALIAS;
    DenseOp op = product(x, w_gate_dev, dtype == SPCONV_E4M3 ? c_in : c_hidden, c_hidden, dtype);
    op.epi = kEpiGated;
    op.b.p[1] = w_up_dev;
    op.row_scale = x_scale_dev;
    op.col_scale[0] = gate_scale_dev;
    op.col_scale[1] = up_scale_dev;
    op.act = activation;
    op.out[0] = out_dev;
    op.ld_out = ld_out;
    return dense_run(op, static_cast<cudaStream_t>(stream));
}

int spconv_gated_ffn_backward(const void* dh_dev, int64_t ld_dh, const void* x_dev, int64_t ld_x, const void* w_gate_dev,
                              const void* w_up_dev, int64_t n, int32_t c_in, int32_t c_hidden, int32_t dtype,
                              int32_t activation, void* dx_dev, void* dw_gate_dev, void* dw_up_dev, void* stream) {
    reset_launch_count();
    if (bad_sizes(n, c_in, c_hidden) || bad_act(activation)) return SPCONV_ERR_INVALID_ARG;
    if (dtype != SPCONV_BF16) return dtype == SPCONV_FP32 || dtype == SPCONV_E4M3 ? SPCONV_ERR_UNSUPPORTED : SPCONV_ERR_INVALID_ARG;
    if ((dw_gate_dev != nullptr) != (dw_up_dev != nullptr)) return SPCONV_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t wn = int64_t(c_in) * c_hidden;
    if (n == 0) {
        SPCONV_CHECK(zero(dw_gate_dev, wn * 2, s));
        return zero(dw_up_dev, wn * 2, s);
    }
    Rows dh{dh_dev, n, c_hidden, ld_dh, 2}, x{x_dev, n, c_in, ld_x, 2};
    const Rows ins[4] = {dh, x, {w_gate_dev, 1, wn, wn, 2}, {w_up_dev, 1, wn, wn, 2}};
    const Rows outs[3] = {{dx_dev, n, c_in, c_in, 2}, {dw_gate_dev, 1, wn, wn, 2}, {dw_up_dev, 1, wn, wn, 2}};
    for (const Rows& r : ins)
        if (!r.ok()) return SPCONV_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) {
        if (!outs[i].p) continue;
        if (!outs[i].ok()) return SPCONV_ERR_INVALID_ARG;
        for (const Rows& r : ins)
            if (outs[i].overlaps(r)) return SPCONV_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (outs[i].overlaps(outs[j])) return SPCONV_ERR_ALIAS;
    }
    if (!dx_dev && !dw_gate_dev) return SPCONV_OK;
    // what two products read is brought into alignment once, and dh with it
    AlignedRows rows;
    const void* w[2] = {w_gate_dev, w_up_dev};
    int64_t ld_w = c_hidden;
    rows.add(&x.p, 1, &x.ld, n, c_in, 2);
    rows.add(w, 2, &ld_w, c_in, c_hidden, 2);
    rows.add(&dh.p, 1, &dh.ld, n, c_hidden, 2);
    SPCONV_CHECK(rows.run(s));
    // gate and up are formed again in the product's epilogue, which writes their
    // gradients, rounded as operands of the products that follow (as dz above)
    const int64_t ld_d = static_cast<int64_t>(round_up(c_hidden, 8));
    const size_t one = static_cast<size_t>(n) * ld_d * 2;
    Scratch d_buf(2 * one, s);
    if (d_buf.failed()) return SPCONV_ERR_OOM;
    const Rows dg{d_buf.as<void>(), n, c_hidden, ld_d, 2}, du{d_buf.as<void>(one), n, c_hidden, ld_d, 2};
    DenseOp op = product(x, w[0], ld_w, c_hidden, SPCONV_BF16);
    op.epi = kEpiGatedGrad;
    op.b.p[1] = w[1];
    op.act = activation;
    op.extra = dh.p;
    op.ld_extra = dh.ld;
    op.out[0] = d_buf.as<void>();
    op.out[1] = d_buf.as<void>(one);
    op.ld_out = ld_d;
    op.out_padded = true;
    SPCONV_CHECK(dense_run(op, s));
    DenseOp ops[2];
    int count = 0;
    if (dw_gate_dev) {
        DenseOp& o = ops[count++];
        o = outer(x, dg);
        o.n_sources = 2;
        o.b.p[1] = du.p;
        o.out[0] = dw_gate_dev;
        o.out[1] = dw_up_dev;
    }
    if (dx_dev) {
        DenseOp& o = ops[count++];
        o = product_t(dg, w[0], ld_w, c_in);
        o.k_sources = 2;
        o.a.p[1] = du.p;
        o.b.p[1] = w[1];
        o.out[0] = dx_dev;
        o.ld_out = c_in;
    }
    return dense_run_plain(ops, count, {}, s);
}

int spconv_rows_status(void* stream) {
    int32_t* word = nullptr;
    SPCONV_CHECK(rows_status_word(&word));
    int32_t st = 0;
    SPCONV_CHECK_CUDA(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
    SPCONV_CHECK_CUDA(cudaMemcpy(&st, word, sizeof(st), cudaMemcpyDeviceToHost));
    if (st == 0) return SPCONV_OK;
    const int32_t zero_word = 0;
    SPCONV_CHECK_CUDA(cudaMemcpy(word, &zero_word, sizeof(zero_word), cudaMemcpyHostToDevice));
    return status_from_flags(st);
}

int spconv_selftest_rows_wait(int64_t limit_ns, void* stream) {
    reset_launch_count();
    if (limit_ns < 1000000 || limit_ns > 100000000) return SPCONV_ERR_INVALID_ARG;
    return rows_wait_probe(static_cast<uint64_t>(limit_ns), static_cast<cudaStream_t>(stream));
}

int spconv_quantize_weight(const void* w_dev, int32_t c_in, int32_t c_out, void* q_dev, float* scale_dev, void* stream) {
    reset_launch_count();
    if (bad_sizes(0, c_in, c_out) || !w_dev || !aligned(w_dev, 2) || !q_dev || !scale_dev || bad_vec(scale_dev))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t wn = int64_t(c_in) * c_out;
    const Rows w{w_dev, 1, wn, wn, 2}, q{q_dev, 1, wn, wn, 1}, sc{scale_dev, 1, c_out, c_out, 4};
    if (q.overlaps(w) || sc.overlaps(w) || sc.overlaps(q)) return SPCONV_ERR_ALIAS;
    return quantize_weight(w_dev, c_in, c_out, q_dev, scale_dev, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
