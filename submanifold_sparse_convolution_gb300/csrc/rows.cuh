// Shared by the row-wise operators (RMS norm, linear, gated feed-forward):
// activations, vector loads and stores, stream-ordered scratch, and the
// description of one matrix product with its epilogue.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "common.cuh"

namespace spconv {

// ---- activations -----------------------------------------------------------
// Evaluated on the fp32 sum in every epilogue, so they are made of few
// instructions: 2^x and 1/x of the special-function unit (relative error about
// 2^-22, far below the bf16 rounding of whatever is stored) and FMAs.  2^x of a
// large argument is infinity and 1/infinity is 0, which are the limits wanted.
//
// The functions take one value (V = float) or two (V = F2): the tensor-core
// epilogues issue the packed multiplies and adds, one instruction for both
// values with the same roundings.
struct F2 {
    uint64_t v;
    F2() = default;
    __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit F2(float a) : F2(a, a) {}
    // f of each value
    template <typename F>
    __device__ __forceinline__ F2 each(F&& f) const {
        float a, b;
        get(a, b);
        return F2(f(a), f(b));
    }
    __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma_v(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float fma_v(float a, float b, float c) { return fmaf(a, b, c); }

template <typename F>
__device__ __forceinline__ float each(float x, F&& f) { return f(x); }
template <typename F>
__device__ __forceinline__ F2 each(F2 x, F&& f) { return x.each(f); }
template <typename F>
__device__ __forceinline__ float each(float x, float y, F&& f) { return f(x, y); }
template <typename F>
__device__ __forceinline__ F2 each(F2 x, F2 y, F&& f) {
    float a, b, c, d;
    x.get(a, b);
    y.get(c, d);
    return F2(f(a, c), f(b, d));
}

template <typename V>
__device__ __forceinline__ V exp2_approx(V x) {
    return each(x, [](float t) {
        float y;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t));
        return y;
    });
}
template <typename V>
__device__ __forceinline__ V rcp_approx(V x) {
    return each(x, [](float t) {
        float y;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t));
        return y;
    });
}
template <typename V>
__device__ __forceinline__ V sigmoid_f(V z) { return rcp_approx(V(1.0f) + exp2_approx(V(-1.44269504f) * z)); }

// tanh form of GELU: 0.5 (1 + tanh(v / 2)) is the logistic function of
// v = z (A + A B z^2)
constexpr float kGeluA = 1.5957691216057308f;   // sqrt(8 / pi)
constexpr float kGeluB = 0.044715f;

// The normal distribution function Phi(z) = erfc(-z / sqrt 2) / 2 and e =
// exp(-z^2 / 2), with erfc of x = |z| / sqrt 2 from Abramowitz and Stegun,
// Handbook of Mathematical Functions, 7.1.26: (a1 t + .. + a5 t^5) exp(-x^2),
// t = 1 / (1 + p x), absolute error at most 1.5e-7.
template <typename V>
__device__ __forceinline__ V normal_cdf(V z, V* e) {
    const V t = rcp_approx(each(z, [](float x) { return fmaf(0.3275911f * 0.70710678f, fabsf(x), 1.0f); }));
    V q = fma_v(t, V(0.5f * 1.061405429f), V(0.5f * -1.453152027f));
    q = fma_v(t, q, V(0.5f * 1.421413741f));
    q = fma_v(t, q, V(0.5f * -0.284496736f));
    q = fma_v(t, q, V(0.5f * 0.254829592f));
    *e = exp2_approx(V(-0.72134752f) * z * z);   // log2(e) / 2
    q = q * t * *e;
    return each(z, q, [](float x, float y) { return x < 0.0f ? y : 1.0f - y; });
}

template <int ACT, typename V>
__device__ __forceinline__ V act_f(V z) {
    if (ACT == SPCONV_ACT_RELU) return each(z, [](float x) { return x < 0.0f ? 0.0f : x; });   // keeps NaN
    if (ACT == SPCONV_ACT_SILU) return z * sigmoid_f(z);
    if (ACT == SPCONV_ACT_GELU) {
        V e;
        return z * normal_cdf(z, &e);
    }
    if (ACT == SPCONV_ACT_GELU_TANH) return z * sigmoid_f(z * fma_v(V(kGeluA * kGeluB) * z, z, V(kGeluA)));
    return z;
}

// *a = act(z), returns act'(z)
template <int ACT, typename V>
__device__ __forceinline__ V act_grad_f(V z, V* a) {
    if (ACT == SPCONV_ACT_RELU) {
        *a = act_f<ACT>(z);
        return each(z, [](float x) { return x > 0.0f ? 1.0f : 0.0f; });
    }
    if (ACT == SPCONV_ACT_SILU) {
        const V s = sigmoid_f(z);
        *a = z * s;
        return fma_v(*a, fma_v(s, V(-1.0f), V(1.0f)), s);
    }
    if (ACT == SPCONV_ACT_GELU) {
        V e;
        const V phi = normal_cdf(z, &e);
        *a = z * phi;
        return fma_v(V(0.39894228f) * z, e, phi);
    }
    if (ACT == SPCONV_ACT_GELU_TANH) {
        const V s = sigmoid_f(z * fma_v(V(kGeluA * kGeluB) * z, z, V(kGeluA)));
        *a = z * s;
        return fma_v(fma_v(*a * V(-1.0f), s, *a), fma_v(V(3.0f * kGeluA * kGeluB) * z, z, V(kGeluA)), s);
    }
    *a = z;
    return V(1.0f);
}

// Calls f with the activation as a compile-time constant.
template <typename F>
__device__ __forceinline__ void with_act(int32_t act, F&& f) {
    switch (act) {
        case SPCONV_ACT_RELU: f(std::integral_constant<int, SPCONV_ACT_RELU>()); break;
        case SPCONV_ACT_SILU: f(std::integral_constant<int, SPCONV_ACT_SILU>()); break;
        case SPCONV_ACT_GELU: f(std::integral_constant<int, SPCONV_ACT_GELU>()); break;
        case SPCONV_ACT_GELU_TANH: f(std::integral_constant<int, SPCONV_ACT_GELU_TANH>()); break;
        default: f(std::integral_constant<int, SPCONV_ACT_NONE>()); break;
    }
}

// ---- scratch ---------------------------------------------------------------
// Device memory for the length of one call: allocated and freed in stream
// order from the library's pool, so it follows the call's stream by itself.
class Scratch {
public:
    Scratch() = default;
    Scratch(size_t bytes, cudaStream_t s) { alloc(bytes, s); }
    ~Scratch() {
        if (ptr_) cudaFreeAsync(ptr_, stream_);
    }
    Scratch(const Scratch&) = delete;
    Scratch& operator=(const Scratch&) = delete;
    // (once per object)
    bool alloc(size_t bytes, cudaStream_t s) {
        stream_ = s;
        if (bytes && pool_alloc(&ptr_, bytes, s) != cudaSuccess) {
            cudaGetLastError();
            ptr_ = nullptr;
            failed_ = true;
        }
        return !failed_;
    }
    bool failed() const { return failed_; }
    template <typename T>
    T* as(size_t byte_offset = 0) const {
        return reinterpret_cast<T*>(static_cast<uint8_t*>(ptr_) + byte_offset);
    }

private:
    void* ptr_ = nullptr;
    cudaStream_t stream_ = nullptr;
    bool failed_ = false;
};

// Launches a kernel with programmatic dependent launch: it calls pdl_wait()
// before its first access to what an earlier kernel wrote or reads.
template <typename... K, typename... A>
int launch_pdl(void (*kernel)(K...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchAttribute at[1] = {pdl_attr()};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    count_launch();
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, args...));
}

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int launch_status() { return cuda_status(cudaGetLastError()); }

// ---- RMS norm (norm.cu) ----------------------------------------------------
struct NormArgs {
    const void* x;          // [n] rows of c, ldx elements apart
    int64_t ldx;
    const void* residual;   // or null
    int64_t ldr;
    const float* weight;    // [c]
    int64_t n;
    int32_t c;
    int32_t dtype;          // of x, residual, sum
    float eps;
    void* sum;              // [n][c] x + residual, or null
    void* out;              // [n][c]
    int32_t out_dtype;      // dtype, or SPCONV_E4M3
    float* scale;           // [n], with SPCONV_E4M3
};
int norm_forward(const NormArgs& a, cudaStream_t s);

struct NormGradArgs {
    const void* dy;
    int64_t ldy;
    const void* x;
    int64_t ldx;
    const float* weight;
    const void* dres;       // or null
    int64_t ldr;
    int64_t n;
    int32_t c;
    int32_t dtype;
    float eps;
    void* dx;               // [n][c]
    float* dweight;         // [c]
};
int norm_backward(const NormGradArgs& a, cudaStream_t s);

// ---- products with an epilogue (dense.cu, dense_tc.cu) ----------------------------------
// Element (i, k) of an operand is p[i ld + k] (k_major) or p[k ld + i].
struct Operand {
    const void* p[2] = {nullptr, nullptr};
    int64_t ld = 0;
    bool k_major = true;
};

enum : int32_t {
    kEpiLinear = 0,      // out0 = act(acc * row_scale * col_scale + bias) + extra
    kEpiGated = 1,       // out0 = act(acc0 ..) * (acc1 ..), acc1 from b.p[1]
    kEpiActGrad = 2,     // out0 = extra * act'(acc + bias); col_part: sums of the unrounded values
    kEpiGatedGrad = 3,   // out0 = extra * acc1 * act'(acc0), out1 = extra * act(acc0)
};

// out[m][n] = epilogue(sum_k A(m, k) B(n, k)), fp32 sums, bf16 out.
struct DenseOp {
    int32_t epi = kEpiLinear;
    int64_t m = 0, n = 0, k = 0;
    int32_t dtype = SPCONV_BF16;     // of A and B: SPCONV_BF16 or SPCONV_E4M3
    Operand a, b;
    int32_t k_sources = 1;           // 2: acc = A0 B0 + A1 B1
    int32_t n_sources = 1;           // 2: out[1] = A B1 beside out[0] = A B0 (kEpiLinear, no epilogue terms)
    int32_t act = SPCONV_ACT_NONE;
    const float* row_scale = nullptr;            // [m]
    const float* col_scale[2] = {nullptr, nullptr};   // [n] of b.p[0], b.p[1]
    const float* bias = nullptr;                 // [n]
    const void* extra = nullptr;                 // bf16 [m] rows, ld_extra apart
    int64_t ld_extra = 0;
    void* out[2] = {nullptr, nullptr};           // bf16 [m] rows, ld_out apart
    int64_t ld_out = 0;
    bool out_padded = false;                     // columns n .. up to whole 16 bytes are the library's to write
    float* col_part = nullptr;                   // fp32 [col_part_rows(m)][n] (kEpiActGrad), or null

    // no epilogue: bf16 operands, the sums rounded and stored
    bool plain() const {
        return epi == kEpiLinear && act == SPCONV_ACT_NONE && !extra && !bias && !col_scale[0];
    }
};

// Rows of a matrix of partial column sums: one per 32 rows of a 256-row tile.
inline int64_t col_part_rows(int64_t m) { return 8 * ceil_div(m, 256); }

// out[j] = sum_i part[i][j] over fp32 rows of n.
struct ColumnSums {
    const float* part = nullptr;
    int64_t rows = 0, n = 0;
    float* out = nullptr;
};
int dense_run(const DenseOp& op, cudaStream_t s);

// Matrices brought into the alignment that the tensor maps need (tma_ok): those
// whose rows (odd channel counts, strides or addresses) do not have it are copied
// to workspace rows that do, all in one launch.  A product does so with what it
// reads; what two products of a gradient read is brought over before both (35309
// x 459 x 228 with SiLU: 93.6 us, by each product 105.4).
constexpr int kMaxCopies = 5;
struct RowCopy {
    const void* src;
    void* dst;
    int64_t pitch_src, pitch_dst, rows;   // bytes, bytes, rows
    int32_t cols, row_warps, blocks, e;   // elements of a row, warps for them, their blocks, bytes of an element
};
struct RowCopies {
    RowCopy copy[kMaxCopies];
};
class AlignedRows {
public:
    // `count` matrices of one shape and row stride (kMaxCopies of all calls)
    void add(const void** p, int count, int64_t* ld, int64_t rows, int64_t cols, size_t es);
    // after the last add: allocates and copies, and sets their addresses
    int run(cudaStream_t s);

private:
    RowCopies args_ = {};
    const void** out_[kMaxCopies];
    size_t off_[kMaxCopies], bytes_ = 0;
    int64_t blocks_ = 0;
    int count_ = 0;
    Scratch buf_;
};
// Up to two plain products in one launch, and column sums, if any, with them.
int dense_run_plain(const DenseOp* ops, int count, const ColumnSums& cols, cudaStream_t s);
// On the tensor cores (dense_tc.cu); operands and extra satisfy tma_ok.
int dense_tc_run(const DenseOp& op, int32_t* status, cudaStream_t s);
// (one product may have an epilogue: dense_tc_cuts
// says whether cutting its K is worth the workspace; plain ones always go here)
bool dense_tc_cuts(const DenseOp& op);
int dense_tc_plain(const DenseOp* ops, int count, const ColumnSums& cols, int32_t* status, cudaStream_t s);
// the same for few rows (dense_few.cu): dense_few_takes says which
bool dense_few_takes(const DenseOp& op);
int dense_few_run(const DenseOp& op, int32_t* status, cudaStream_t s);
// The device status word of the row-wise operators on the current device.
int rows_status_word(int32_t** word);
// Runs their wait against a barrier that nothing arrives on (spconv_selftest_rows_wait).
int rows_wait_probe(uint64_t limit_ns, cudaStream_t s);

// What a tensor map takes: 16-byte aligned rows.
inline bool tma_ok(const void* p, int64_t ld, size_t es) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * static_cast<int64_t>(es)) % 16 == 0;
}

// Partial column sums of bf16 rows: fills part (column_part_rows(m, n) fp32 rows of n).
int64_t column_part_rows(int64_t m, int64_t n);
int column_parts(const void* v, int64_t ld, int64_t m, int64_t n, float* part, cudaStream_t s);
// What is left after partial results: for up to two products the sums of their
// slices of K (fp32 [splits][outputs][m][ld_part], outputs one or two), the
// epilogue and the rounding; and column sums.  One launch.
struct SliceSums {
    const float* part = nullptr;
    int64_t ld_part = 0;
    int32_t splits = 0;
    int64_t m = 0, n = 0;
    int32_t outputs = 0;
    __nv_bfloat16* out[2] = {nullptr, nullptr};
    int64_t ld = 0;
    bool vec_out = false;   // (set by finish_sums: the rows take 8-byte stores)
    // kEpiLinear's or kEpiGated's terms (DenseOp); kEpiGated makes one output of two
    int32_t epi = kEpiLinear, act = SPCONV_ACT_NONE;
    const float* row_scale = nullptr;
    const float* col_scale[2] = {nullptr, nullptr};
    const float* bias = nullptr;
    const __nv_bfloat16* extra = nullptr;
    int64_t ld_extra = 0;
    float* col_part = nullptr;   // (finish_grad; DenseOp's)
};
// The same for one product with kEpiActGrad or kEpiGatedGrad.
int finish_grad(const SliceSums& a, cudaStream_t s);
int finish_sums(const SliceSums* slices, int count, const ColumnSums& cols, cudaStream_t s);
// bf16 w [c_in][c_out] -> e4m3 q [c_out][c_in] with scale [c_out]
int quantize_weight(const void* w, int32_t c_in, int32_t c_out, void* q, float* scale, cudaStream_t s);

}  // namespace spconv
