// Root-mean-square norm of rows, with the residual's addition, an optional
// 8-bit output, and its backward pass.
//
//   h = x + residual;  r = 1 / sqrt(mean_c h^2 + eps);  y = h r w
//   8 bits: scale = max_c |y| / 448,  q = e4m3(y / scale)
//
// Everything between the loads and the stores is fp32, with one rounding per
// output.  The kernels are bound by HBM: a row is read once into registers,
// reduced, and written; the next row's loads are in flight meanwhile.
#include "rows.cuh"

namespace spconv {
namespace {

constexpr int kBlock = 256;          // threads of a block that holds several rows
constexpr int kLongThreads = 512;    // threads of a block that walks a row too long to hold
constexpr float kE4m3Max = 448.0f;

// W consecutive elements as they lie in memory (W = 8 is one or two 16-byte loads).
template <typename T, int W>
struct Pack {
    T v[W];
};
template <>
struct alignas(16) Pack<__nv_bfloat16, 8> {
    __nv_bfloat16 v[8];
};
template <>
struct alignas(16) Pack<float, 8> {
    float v[8];
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

template <int W>
__device__ __forceinline__ void store_e4m3(uint8_t* dst, const float* v) {
    if (W == 8) {
        uint32_t q[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * j], v[4 * j + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * j + 2], v[4 * j + 3]), __NV_SATFINITE, __NV_E4M3);
            q[j] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) dst[j] = __nv_cvt_float_to_fp8(v[j], __NV_SATFINITE, __NV_E4M3);
    }
}

// What a row's threads add up: sum of squares and, forward with 8 bits, the
// largest |h w| as its bits (non-negative floats order as integers, with NaN
// above infinity, so NaN is kept); backward, the sum of g h.
struct SumMax {
    float s;
    uint32_t m;
};
__device__ __forceinline__ SumMax join(SumMax a, SumMax b) { return {a.s + b.s, a.m > b.m ? a.m : b.m}; }
__device__ __forceinline__ SumMax shfl_xor(SumMax v, int o) {
    return {__shfl_xor_sync(0xFFFFFFFFu, v.s, o), __shfl_xor_sync(0xFFFFFFFFu, v.m, o)};
}
struct Sum2 {
    float s, t;
};
__device__ __forceinline__ Sum2 join(Sum2 a, Sum2 b) { return {a.s + b.s, a.t + b.t}; }
__device__ __forceinline__ Sum2 shfl_xor(Sum2 v, int o) {
    return {__shfl_xor_sync(0xFFFFFFFFu, v.s, o), __shfl_xor_sync(0xFFFFFFFFu, v.t, o)};
}

// Over TPR <= 32 neighbouring lanes, the result in all of them.
template <int TPR, typename V>
__device__ __forceinline__ V lanes_reduce(V v) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) v = join(v, shfl_xor(v, o));
    return v;
}

// Over the block, the result in all threads.  `sh` holds two sets of 32 slots
// that successive calls take in turn (`turn`), so one barrier per call is
// enough: a set is written again only after the barrier of the call between.
template <typename V>
__device__ __forceinline__ V block_reduce(V v, V* sh, int turn) {
    v = lanes_reduce<32>(v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    V* slot = sh + 32 * (turn & 1);
    if (lane == 0) slot[warp] = v;
    __syncthreads();
    V r{};
    if (lane < warps) r = slot[lane];
    return lanes_reduce<32>(r);
}

// The scale of a row whose largest |y| is amax, and the factors with
// q = (y * pre) * inv.  448 / amax overflows for amax below 2^-119, so tiny
// rows are first brought up by 2^100.  A row of zeros has scale 0, q 0.
__device__ __forceinline__ float row_scale_of(float amax, float* pre, float* inv) {
    *pre = amax < 0x1p-100f ? 0x1p100f : 1.0f;
    *inv = amax == 0.0f ? 0.0f : kE4m3Max / (amax * *pre);
    return amax / kE4m3Max;
}

// ---- forward ------------------------------------------------------------------
// The VPT vectors of W elements of one row that one of its TPR threads handles:
// elements (v TPR + t) W ..
template <typename T, int W, int VPT>
struct RowPart {
    Pack<T, W> x[VPT], r[VPT];

    __device__ __forceinline__ void load(const NormArgs& a, int64_t row, int t, int tpr) {
        const T* x0 = static_cast<const T*>(a.x) + row * a.ldx;
        const T* r0 = static_cast<const T*>(a.residual) + row * a.ldr;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * tpr + t) * W;
            if (e < a.c) {
                x[v] = *reinterpret_cast<const Pack<T, W>*>(x0 + e);
                if (a.residual) r[v] = *reinterpret_cast<const Pack<T, W>*>(r0 + e);
            }
        }
    }
};

// h = x + residual, this thread's share of the row's statistics.
template <typename T, int W, int VPT, bool EIGHT>
__device__ __forceinline__ SumMax row_stats(const NormArgs& a, const RowPart<T, W, VPT>& p, const Pack<float, W> (&w)[VPT],
                                            float (&h)[VPT * W], int t, int tpr) {
    SumMax st{0.0f, 0u};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if ((v * tpr + t) * W >= a.c) continue;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float f = to_f(p.x[v].v[j]);
            if (a.residual) f += to_f(p.r[v].v[j]);
            h[v * W + j] = f;
            st.s = fmaf(f, f, st.s);
            if (EIGHT) {
                const uint32_t b = __float_as_uint(fabsf(f * w[v].v[j]));
                st.m = b > st.m ? b : st.m;
            }
        }
    }
    return st;
}

// Writes the row.  y = (h w) r: r is one positive factor, so max |y| is
// (max |h w|) r, rounding included, and the two reductions are one.
template <typename T, int W, int VPT, bool EIGHT>
__device__ __forceinline__ void row_write(const NormArgs& a, int64_t row, SumMax st, const Pack<float, W> (&w)[VPT],
                                          const float (&h)[VPT * W], int t, int tpr) {
    using P = Pack<T, W>;
    const float r = rsqrtf(st.s / static_cast<float>(a.c) + a.eps);
    float pre = 1.0f, inv = 1.0f;
    if (EIGHT) {
        const float scale = row_scale_of(__uint_as_float(st.m) * r, &pre, &inv);
        if (t == 0) a.scale[row] = scale;
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * tpr + t) * W;
        if (e >= a.c) continue;
        P o;
        if (a.sum) {
#pragma unroll
            for (int j = 0; j < W; ++j) from_f(h[v * W + j], o.v[j]);
            *reinterpret_cast<P*>(static_cast<T*>(a.sum) + row * a.c + e) = o;
        }
        float y[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            y[j] = h[v * W + j] * w[v].v[j] * r;
            if (EIGHT) y[j] = y[j] * pre * inv;
        }
        if (EIGHT) {
            store_e4m3<W>(static_cast<uint8_t*>(a.out) + row * a.c + e, y);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) from_f(y[j], o.v[j]);
            *reinterpret_cast<P*>(static_cast<T*>(a.out) + row * a.c + e) = o;
        }
    }
}

template <int W, int VPT>
__device__ __forceinline__ void load_weight(const float* weight, int32_t c, Pack<float, W> (&w)[VPT], int t, int tpr) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * tpr + t) * W;
        if (e < c) w[v] = *reinterpret_cast<const Pack<float, W>*>(weight + e);
    }
}

// Short rows: TPR lanes per row, many rows per block; enough
// independent warps that the loads of some cover the arithmetic of others.
template <typename T, int W, int TPR, int VPT, bool EIGHT>
__global__ void __launch_bounds__(kBlock) k_rms_norm(const NormArgs a) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kBlock / TPR) + threadIdx.x / TPR;
    const int t = threadIdx.x % TPR;
    const bool live = row < a.n;   // (lanes of absent rows still take part in the shuffles)
    RowPart<T, W, VPT> p;
    Pack<float, W> w[VPT];
    float h[VPT * W];
    SumMax st{0.0f, 0u};
    load_weight<W, VPT>(a.weight, a.c, w, t, TPR);
    pdl_wait();
    pdl_trigger();
    if (live) {
        p.load(a, row, t, TPR);
        st = row_stats<T, W, VPT, EIGHT>(a, p, w, h, t, TPR);
    }
    st = lanes_reduce<TPR>(st);
    if (live) row_write<T, W, VPT, EIGHT>(a, row, st, w, h, t, TPR);
}

// Up to 8192 elements: one block per row, persistent, the next row's loads in
// flight while this one is reduced and written; the weight stays in registers.
template <typename T, int W, int VPT, bool EIGHT>
__global__ void __launch_bounds__(512) k_rms_norm_block(const NormArgs a) {
    __shared__ SumMax sh[64];
    const int t = threadIdx.x, tpr = blockDim.x;
    RowPart<T, W, VPT> p, next;
    Pack<float, W> w[VPT];
    float h[VPT * W];
    load_weight<W, VPT>(a.weight, a.c, w, t, tpr);
    pdl_wait();
    pdl_trigger();
    int64_t row = blockIdx.x;
    p.load(a, row, t, tpr);   // (the grid has at most n blocks)
    for (int turn = 0; row < a.n; ++turn) {
        const int64_t after = row + gridDim.x;
        if (after < a.n) next.load(a, after, t, tpr);
        const SumMax st = block_reduce(row_stats<T, W, VPT, EIGHT>(a, p, w, h, t, tpr), sh, turn);
        row_write<T, W, VPT, EIGHT>(a, row, st, w, h, t, tpr);
        p = next;
        row = after;
    }
}

// Longer rows: one block per row, the row read once per pass (the second
// mostly from L2).  Every element is read by the thread that writes it, after
// the first pass, so sum may be the residual.
template <typename T, int W, bool EIGHT>
__global__ void __launch_bounds__(kLongThreads) k_rms_norm_long(const NormArgs a) {
    __shared__ SumMax sh[64];
    pdl_wait();
    pdl_trigger();
    int turn = 0;
    const int step = kLongThreads;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, ++turn) {
        SumMax st{0.0f, 0u};
        RowPart<T, W, 1> p;
        Pack<float, W> w[1];
        float h[W];
#pragma unroll 4
        for (int t = threadIdx.x; t * W < a.c; t += step) {
            p.load(a, row, t, 0);
            load_weight<W, 1>(a.weight, a.c, w, t, 0);
            st = join(st, row_stats<T, W, 1, EIGHT>(a, p, w, h, t, 0));
        }
        st = block_reduce(st, sh, turn);
#pragma unroll 2
        for (int t = threadIdx.x; t * W < a.c; t += step) {
            p.load(a, row, t, 0);
            load_weight<W, 1>(a.weight, a.c, w, t, 0);
            row_stats<T, W, 1, false>(a, p, w, h, t, 0);
            row_write<T, W, 1, EIGHT>(a, row, st, w, h, t, 0);
        }
    }
}

// ---- backward -----------------------------------------------------------------
// With g = dy w and r as above:
//   dx = r g - h r^3 mean_c(g h) + dres,   dw_c = sum_rows dy h r
// Each row's threads walk the rows first, first + step, ...; the weight and the
// running dw of their columns stay in registers, a block's rows are added in a
// fixed order and the block writes one row of partial sums (sum_partials adds
// those): no atomics, the same bits every run.
template <typename T, int W, int VPT>
struct GradPart {
    Pack<T, W> x[VPT], d[VPT], r[VPT];

    __device__ __forceinline__ void load(const NormGradArgs& a, int64_t row, int t, int tpr) {
        const T* x0 = static_cast<const T*>(a.x) + row * a.ldx;
        const T* d0 = static_cast<const T*>(a.dy) + row * a.ldy;
        const T* r0 = static_cast<const T*>(a.dres) + row * a.ldr;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * tpr + t) * W;
            if (e < a.c) {
                x[v] = *reinterpret_cast<const Pack<T, W>*>(x0 + e);
                d[v] = *reinterpret_cast<const Pack<T, W>*>(d0 + e);
                if (a.dres) r[v] = *reinterpret_cast<const Pack<T, W>*>(r0 + e);
            }
        }
    }
};

template <typename T, int W, int VPT>
__device__ __forceinline__ Sum2 grad_stats(const NormGradArgs& a, const GradPart<T, W, VPT>& p, const Pack<float, W> (&w)[VPT],
                                           int t, int tpr) {
    Sum2 st{0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if ((v * tpr + t) * W >= a.c) continue;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float h = to_f(p.x[v].v[j]);
            st.s = fmaf(h, h, st.s);
            st.t = fmaf(to_f(p.d[v].v[j]) * w[v].v[j], h, st.t);
        }
    }
    return st;
}

// r = 1 / rms and k = r^3 mean(g h) of a row
__device__ __forceinline__ Sum2 grad_factors(Sum2 st, int32_t c, float eps) {
    const float inv_c = 1.0f / static_cast<float>(c);
    const float r = rsqrtf(st.s * inv_c + eps);
    return {r, r * r * r * st.t * inv_c};
}

template <typename T, int W, int VPT>
__device__ __forceinline__ void grad_write(const NormGradArgs& a, int64_t row, Sum2 f, const GradPart<T, W, VPT>& p,
                                           const Pack<float, W> (&w)[VPT], float (&dw)[VPT * W], int t, int tpr) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * tpr + t) * W;
        if (e >= a.c) continue;
        Pack<T, W> o;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float h = to_f(p.x[v].v[j]), d = to_f(p.d[v].v[j]);
            float dx = fmaf(d * w[v].v[j], f.s, -h * f.t);
            if (a.dres) dx += to_f(p.r[v].v[j]);
            from_f(dx, o.v[j]);
            dw[v * W + j] = fmaf(d, h * f.s, dw[v * W + j]);
        }
        *reinterpret_cast<Pack<T, W>*>(static_cast<T*>(a.dx) + row * a.c + e) = o;
    }
}

// Short rows: TPR lanes per row.
template <typename T, int W, int TPR, int VPT>
__global__ void __launch_bounds__(kBlock) k_rms_norm_grad(const NormGradArgs a, float* part) {
    constexpr int kRows = kBlock / TPR, kCols = TPR * VPT * W;
    extern __shared__ float sh_dw[];   // [kRows][kCols]
    const int grp = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    Pack<float, W> w[VPT];
    float dw[VPT * W] = {};
    GradPart<T, W, VPT> p, next;
    load_weight<W, VPT>(a.weight, a.c, w, t, TPR);
    pdl_wait();
    pdl_trigger();
    int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
    if (base + grp < a.n) p.load(a, base + grp, t, TPR);
    // (every lane of the block runs the same number of rounds: shuffles inside)
    for (; base < a.n; base += step) {
        const int64_t row = base + grp;
        if (row + step < a.n) next.load(a, row + step, t, TPR);
        Sum2 st{0.0f, 0.0f};
        if (row < a.n) st = grad_stats<T, W, VPT>(a, p, w, t, TPR);
        st = lanes_reduce<TPR>(st);
        if (row < a.n) grad_write<T, W, VPT>(a, row, grad_factors(st, a.c, a.eps), p, w, dw, t, TPR);
        p = next;
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int j = 0; j < W; ++j) sh_dw[grp * kCols + (v * TPR + t) * W + j] = dw[v * W + j];
    __syncthreads();
    for (int e = threadIdx.x; e < a.c; e += kBlock) {
        float s = 0.0f;
#pragma unroll
        for (int g = 0; g < kRows; ++g) s += sh_dw[g * kCols + e];
        part[static_cast<int64_t>(blockIdx.x) * a.c + e] = s;
    }
}

// Up to 8192 elements: one block per row.
template <typename T, int W, int VPT>
__global__ void __launch_bounds__(512) k_rms_norm_grad_block(const NormGradArgs a, float* part) {
    __shared__ Sum2 sh[64];
    const int t = threadIdx.x, tpr = blockDim.x;
    Pack<float, W> w[VPT];
    float dw[VPT * W] = {};
    GradPart<T, W, VPT> p, next;
    load_weight<W, VPT>(a.weight, a.c, w, t, tpr);
    pdl_wait();
    pdl_trigger();
    int64_t row = blockIdx.x;
    p.load(a, row, t, tpr);
    for (int turn = 0; row < a.n; ++turn) {
        const int64_t after = row + gridDim.x;
        if (after < a.n) next.load(a, after, t, tpr);
        const Sum2 st = block_reduce(grad_stats<T, W, VPT>(a, p, w, t, tpr), sh, turn);
        grad_write<T, W, VPT>(a, row, grad_factors(st, a.c, a.eps), p, w, dw, t, tpr);
        p = next;
        row = after;
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int e = (v * tpr + t) * W + j;
            if (e < a.c) part[static_cast<int64_t>(blockIdx.x) * a.c + e] = dw[v * W + j];
        }
}

// Longer rows in two passes: the factors of each row, then dx and the partial
// dw of a block of columns over a run of rows.
template <typename T, int W>
__global__ void __launch_bounds__(kLongThreads) k_rms_norm_grad_factors(const NormGradArgs a, Sum2* factors) {
    __shared__ Sum2 sh[64];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, ++turn) {
        Sum2 st{0.0f, 0.0f};
        NormGradArgs b = a;
        b.dres = nullptr;
        GradPart<T, W, 1> p;
        Pack<float, W> w[1];
#pragma unroll 4
        for (int t = threadIdx.x; t * W < a.c; t += kLongThreads) {
            p.load(b, row, t, 0);
            load_weight<W, 1>(a.weight, a.c, w, t, 0);
            st = join(st, grad_stats<T, W, 1>(b, p, w, t, 0));
        }
        st = block_reduce(st, sh, turn);
        if (threadIdx.x == 0) factors[row] = grad_factors(st, a.c, a.eps);
    }
}

template <typename T, int W>
__global__ void __launch_bounds__(kBlock) k_rms_norm_grad_columns(const NormGradArgs a, const Sum2* factors, int64_t rows,
                                                                  float* part) {
    const int t = blockIdx.x * kBlock + threadIdx.x;
    if (t * W >= a.c) return;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows, r1 = r0 + rows < a.n ? r0 + rows : a.n;
    Pack<float, W> w[1];
    float dw[W] = {};
    load_weight<W, 1>(a.weight, a.c, w, t, 0);
#pragma unroll 2
    for (int64_t row = r0; row < r1; ++row) {
        GradPart<T, W, 1> p;
        p.load(a, row, t, 0);
        grad_write<T, W, 1>(a, row, factors[row], p, w, dw, t, 0);
    }
#pragma unroll
    for (int j = 0; j < W; ++j) part[static_cast<int64_t>(blockIdx.y) * a.c + t * W + j] = dw[j];
}

bool vec_ok(const void* p, int64_t ld, size_t elem) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * static_cast<int64_t>(elem)) % 16 == 0;
}

// Launches with programmatic dependent launch: each kernel waits (pdl_wait)
// before its first read of what an earlier one wrote.
template <typename... K, typename... A>
int launch(void (*kernel)(K...), int64_t blocks, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchAttribute at[1] = {pdl_attr()};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    count_launch();
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, args...));
}

constexpr int64_t kSms = 152;

// Threads of a block that holds a row of c elements, `per` of them each.
int block_threads(int32_t c, int per) { return static_cast<int>(round_up(static_cast<size_t>(ceil_div(c, per)), 32)); }

// Rows of up to 512 elements (1024 with WIDE): calls f(TPR, VPT) (as
// constants) with the smallest layout that holds c elements, VPT counting
// vectors of 8.
template <bool WIDE, typename F>
int with_lanes(int32_t c, F&& f) {
#define SPCONV_NORM_LAYOUT(TPR, VPT) \
    if (c <= TPR * VPT * 8) return f(std::integral_constant<int, TPR>(), std::integral_constant<int, VPT>());
    SPCONV_NORM_LAYOUT(2, 1)
    SPCONV_NORM_LAYOUT(4, 1)
    SPCONV_NORM_LAYOUT(8, 1)
    SPCONV_NORM_LAYOUT(16, 1)
    SPCONV_NORM_LAYOUT(32, 1)
    if constexpr (WIDE) {
        SPCONV_NORM_LAYOUT(32, 2)
        return f(std::integral_constant<int, 32>(), std::integral_constant<int, 4>());
    }
#undef SPCONV_NORM_LAYOUT
    return f(std::integral_constant<int, 32>(), std::integral_constant<int, 2>());
}

// How long a row a thread's registers allow to hold: vectors of 8 take fewer
// than single elements, the forward pass fewer than the backward one (which
// also keeps dy, dres and the running dw), bf16 fewer than fp32.
template <typename T, int W, bool EIGHT>
int forward_t(const NormArgs& a, cudaStream_t s) {
    constexpr int S = 8 / W;   // W = 1 holds the same elements in eight times the loads
    constexpr bool kVec = W == 8;
    if (a.c <= (kVec ? 1024 : 512))
        return with_lanes<kVec>(a.c, [&](auto tpr, auto vpt) {
            return launch(k_rms_norm<T, W, tpr, vpt * S, EIGHT>, ceil_div(a.n, kBlock / tpr), kBlock, 0, s, a);
        });
    auto persistent = [&](auto kernel, int per) {
        const int threads = block_threads(a.c, per);
        const int64_t most = kSms * (1024 / threads);
        return launch(kernel, a.n < most ? a.n : most, threads, 0, s, a);
    };
    if (a.c <= 4096) return persistent(k_rms_norm_block<T, W, S, EIGHT>, 8);
    if constexpr (kVec) {
        if (a.c <= 8192) return persistent(k_rms_norm_block<T, W, 2, EIGHT>, 16);
    }
    const int64_t most = kSms * 4;
    return launch(k_rms_norm_long<T, W, EIGHT>, a.n < most ? a.n : most, kLongThreads, 0, s, a);
}

template <typename T, int W>
int backward_t(const NormGradArgs& a, cudaStream_t s) {
    constexpr int S = 8 / W;
    constexpr bool kVec = W == 8;
    // blocks: partial sums of dw, one row each
    auto with_part = [&](int64_t blocks, auto&& run) -> int {
        Scratch part(static_cast<size_t>(blocks) * a.c * 4, s);
        if (part.failed()) return SPCONV_ERR_OOM;
        SPCONV_CHECK(run(part.as<float>()));
        return sum_partials(part.as<float>(), blocks, a.c, a.dweight, s);
    };
    if (a.c <= 512)
        return with_lanes<false>(a.c, [&](auto tpr, auto vpt) {
            const int64_t want = ceil_div(a.n, kBlock / tpr), most = kSms * 4;
            const int64_t blocks = want < most ? want : most;
            return with_part(blocks, [&](float* part) {
                return launch(k_rms_norm_grad<T, W, tpr, vpt * S>, blocks, kBlock, size_t(kBlock) * vpt * 8 * 4, s, a, part);
            });
        });
    auto persistent = [&](auto kernel, int per) {
        const int threads = block_threads(a.c, per);
        const int64_t most = kSms * (1024 / threads);
        const int64_t blocks = a.n < most ? a.n : most;
        return with_part(blocks, [&](float* part) { return launch(kernel, blocks, threads, 0, s, a, part); });
    };
    constexpr int kPer = kVec ? 8 : 4;
    if (a.c <= 512 * kPer) return persistent(k_rms_norm_grad_block<T, W, kPer / W>, kPer);
    if constexpr (kVec && sizeof(T) == 2) {
        if (a.c <= 8192) return persistent(k_rms_norm_grad_block<T, W, 2>, 16);
    }
    Scratch factors(static_cast<size_t>(a.n) * sizeof(Sum2), s);
    if (factors.failed()) return SPCONV_ERR_OOM;
    const int64_t most = kSms * 4;
    count_launch();
    k_rms_norm_grad_factors<T, W><<<static_cast<unsigned>(a.n < most ? a.n : most), kLongThreads, 0, s>>>(a, factors.as<Sum2>());
    SPCONV_CHECK(launch_status());
    const int64_t bx = ceil_div(a.c, kBlock * W);
    int64_t chunks = ceil_div(kSms * 8, bx);
    if (chunks > ceil_div(a.n, 16)) chunks = ceil_div(a.n, 16);
    const int64_t rows = ceil_div(a.n, chunks);
    return with_part(chunks, [&](float* part) {
        count_launch();
        k_rms_norm_grad_columns<T, W><<<dim3(static_cast<unsigned>(bx), static_cast<unsigned>(chunks)), kBlock, 0, s>>>(
            a, factors.as<Sum2>(), rows, part);
        return launch_status();
    });
}

}  // namespace

int norm_forward(const NormArgs& a, cudaStream_t s) {
    const size_t es = a.dtype == SPCONV_FP32 ? 4 : 2;
    const bool vec = a.c % 8 == 0 && vec_ok(a.x, a.ldx, es) && vec_ok(a.residual, a.ldr, es) &&
                     vec_ok(a.weight, 0, 4) && vec_ok(a.sum, 0, es) && vec_ok(a.out, 0, es);
    const bool eight = a.out_dtype == SPCONV_E4M3;
    if (a.dtype == SPCONV_FP32)
        return vec ? (eight ? forward_t<float, 8, true>(a, s) : forward_t<float, 8, false>(a, s))
                   : (eight ? forward_t<float, 1, true>(a, s) : forward_t<float, 1, false>(a, s));
    return vec ? (eight ? forward_t<__nv_bfloat16, 8, true>(a, s) : forward_t<__nv_bfloat16, 8, false>(a, s))
               : (eight ? forward_t<__nv_bfloat16, 1, true>(a, s) : forward_t<__nv_bfloat16, 1, false>(a, s));
}

int norm_backward(const NormGradArgs& a, cudaStream_t s) {
    const size_t es = a.dtype == SPCONV_FP32 ? 4 : 2;
    const bool vec = a.c % 8 == 0 && vec_ok(a.dy, a.ldy, es) && vec_ok(a.x, a.ldx, es) && vec_ok(a.dres, a.ldr, es) &&
                     vec_ok(a.weight, 0, 4) && vec_ok(a.dx, 0, es);
    if (a.dtype == SPCONV_FP32) return vec ? backward_t<float, 8>(a, s) : backward_t<float, 1>(a, s);
    return vec ? backward_t<__nv_bfloat16, 8>(a, s) : backward_t<__nv_bfloat16, 1>(a, s);
}

}  // namespace spconv
