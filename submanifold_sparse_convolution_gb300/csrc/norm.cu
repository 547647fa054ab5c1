// Root-mean-square norm of rows, with the residual's addition, an optional
// 8-bit output, and its backward pass.
//
//   h = x + residual;  r = 1 / sqrt(mean_c h^2 + eps);  y = h r w
//   8 bits: scale = max_c |y| / 448,  q = e4m3(y / scale)
//
// Everything between the loads and the stores is fp32, with one rounding per
// output.  The kernels are bound by HBM: a row is read once into registers
// (TPR threads per row, VPT vectors of W elements each), reduced, and written.
// Rows of more than 16384 elements (backward: 8192) are read again for the
// second pass.
#include "rows.cuh"

namespace spconv {
namespace {

constexpr int kBlock = 256;          // threads of a block that holds several rows
constexpr int kWideThreads = 512;    // threads of a block that walks a row too long to hold
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

struct AddF {
    __device__ float operator()(float a, float b) const { return a + b; }
};
// of |y| as its bits: the order of non-negative floats, with NaN above infinity, so NaN is kept
struct MaxU {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};

// Reduction over the TPR threads of a row, the result in all of them.  With
// TPR > 32 the block is one row and `sh` (32 words) is free before the call.
template <int TPR, typename V, typename Op>
__device__ __forceinline__ V row_reduce(V v, Op op, V* sh) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (TPR > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) sh[warp] = v;
        __syncthreads();
        v = sh[lane & (TPR / 32 - 1)];   // TPR / 32 is a power of two: every slot read is written
#pragma unroll
        for (int o = TPR / 64; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
        __syncthreads();
    }
    return v;
}

// The scale of a row whose largest |y| has the bits `amax`, and the factors
// with q = (y * pre) * inv.  448 / amax overflows for amax below 2^-119, so
// tiny rows are first brought up by 2^100.  A row of zeros has scale 0, q 0.
__device__ __forceinline__ float row_scale_of(uint32_t amax_bits, float* pre, float* inv) {
    const float amax = __uint_as_float(amax_bits);
    *pre = amax < 0x1p-100f ? 0x1p100f : 1.0f;
    *inv = amax == 0.0f ? 0.0f : kE4m3Max / (amax * *pre);
    return amax / kE4m3Max;
}

template <typename T, int W, int TPR, int VPT, bool EIGHT>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock) k_rms_norm(const NormArgs a) {
    constexpr int kThreads = TPR > 32 ? TPR : kBlock;
    __shared__ float sh_f[32];
    __shared__ uint32_t sh_u[32];
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
    const int t = threadIdx.x % TPR;
    const bool live = row < a.n;   // (threads of absent rows still take part in the shuffles)
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* res = static_cast<const T*>(a.residual) + row * a.ldr;
    using P = Pack<T, W>;
    P px[VPT], pr[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * TPR + t) * W;
        if (live && e < a.c) {
            px[v] = *reinterpret_cast<const P*>(x + e);
            if (a.residual) pr[v] = *reinterpret_cast<const P*>(res + e);
        }
    }
    float h[VPT * W];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const bool in = live && (v * TPR + t) * W < a.c;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float f = 0.0f;
            if (in) {
                f = to_f(px[v].v[j]);
                if (a.residual) f += to_f(pr[v].v[j]);
            }
            h[v * W + j] = f;
            ss = fmaf(f, f, ss);
        }
    }
    ss = row_reduce<TPR>(ss, AddF(), sh_f);
    const float r = rsqrtf(ss / static_cast<float>(a.c) + a.eps);
    uint32_t amax = 0;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * TPR + t) * W;
        if (!(live && e < a.c)) continue;
        if (a.sum) {
            P o;
#pragma unroll
            for (int j = 0; j < W; ++j) from_f(h[v * W + j], o.v[j]);
            *reinterpret_cast<P*>(static_cast<T*>(a.sum) + row * a.c + e) = o;
        }
        Pack<float, W> w = *reinterpret_cast<const Pack<float, W>*>(a.weight + e);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            h[v * W + j] *= r * w.v[j];
            if (EIGHT) amax = MaxU()(amax, __float_as_uint(fabsf(h[v * W + j])));
        }
        if (!EIGHT) {
            P o;
#pragma unroll
            for (int j = 0; j < W; ++j) from_f(h[v * W + j], o.v[j]);
            *reinterpret_cast<P*>(static_cast<T*>(a.out) + row * a.c + e) = o;
        }
    }
    if (EIGHT) {
        amax = row_reduce<TPR>(amax, MaxU(), sh_u);
        float pre, inv;
        const float scale = row_scale_of(amax, &pre, &inv);
        if (live && t == 0) a.scale[row] = scale;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * TPR + t) * W;
            if (!(live && e < a.c)) continue;
#pragma unroll
            for (int j = 0; j < W; ++j) h[v * W + j] = h[v * W + j] * pre * inv;
            store_e4m3<W>(static_cast<uint8_t*>(a.out) + row * a.c + e, h + v * W);
        }
    }
}

// Rows too long to hold: one block per row, the row read once
// per pass (the later passes mostly from L2).  Every element is read by the
// thread that writes it, after all other passes, so sum may be the residual.
template <typename T, int W, bool EIGHT>
__global__ void __launch_bounds__(kWideThreads) k_rms_norm_wide(const NormArgs a) {
    __shared__ float sh_f[32];
    __shared__ uint32_t sh_u[32];
    using P = Pack<T, W>;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* res = static_cast<const T*>(a.residual) + row * a.ldr;
        auto load = [&](int e, float* h) {
            const P p = *reinterpret_cast<const P*>(x + e);
#pragma unroll
            for (int j = 0; j < W; ++j) h[j] = to_f(p.v[j]);
            if (a.residual) {
                const P q = *reinterpret_cast<const P*>(res + e);
#pragma unroll
                for (int j = 0; j < W; ++j) h[j] += to_f(q.v[j]);
            }
        };
        float ss = 0.0f, h[W];
        for (int e = threadIdx.x * W; e < a.c; e += kWideThreads * W) {
            load(e, h);
#pragma unroll
            for (int j = 0; j < W; ++j) ss = fmaf(h[j], h[j], ss);
        }
        ss = row_reduce<kWideThreads>(ss, AddF(), sh_f);
        const float r = rsqrtf(ss / static_cast<float>(a.c) + a.eps);
        float pre = 1.0f, inv = 1.0f;
        if (EIGHT) {
            uint32_t amax = 0;
            for (int e = threadIdx.x * W; e < a.c; e += kWideThreads * W) {
                load(e, h);
#pragma unroll
                for (int j = 0; j < W; ++j) amax = MaxU()(amax, __float_as_uint(fabsf(h[j] * (r * a.weight[e + j]))));
            }
            amax = row_reduce<kWideThreads>(amax, MaxU(), sh_u);
            const float scale = row_scale_of(amax, &pre, &inv);
            if (threadIdx.x == 0) a.scale[row] = scale;
        }
        for (int e = threadIdx.x * W; e < a.c; e += kWideThreads * W) {
            load(e, h);
            if (a.sum) {
                P o;
#pragma unroll
                for (int j = 0; j < W; ++j) from_f(h[j], o.v[j]);
                *reinterpret_cast<P*>(static_cast<T*>(a.sum) + row * a.c + e) = o;
            }
#pragma unroll
            for (int j = 0; j < W; ++j) h[j] *= r * a.weight[e + j];
            if (EIGHT) {
#pragma unroll
                for (int j = 0; j < W; ++j) h[j] = h[j] * pre * inv;
                store_e4m3<W>(static_cast<uint8_t*>(a.out) + row * a.c + e, h);
            } else {
                P o;
#pragma unroll
                for (int j = 0; j < W; ++j) from_f(h[j], o.v[j]);
                *reinterpret_cast<P*>(static_cast<T*>(a.out) + row * a.c + e) = o;
            }
        }
    }
}

// Backward.  With g = dy w and r as above:
//   dx = r g - h r^3 mean_c(g h) + dres,   dw_c = sum_rows dy h r
// Each group of TPR threads walks the rows first, first + step, ...; the
// weight and the running dw of its columns stay in registers, the block's
// groups are added in a fixed order and the block writes one row of partial
// sums (sum_partials adds those): no atomics, the same bits every run.
template <typename T, int W, int TPR, int VPT>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock) k_rms_norm_grad(const NormGradArgs a, float* part) {
    constexpr int kThreads = TPR > 32 ? TPR : kBlock;
    constexpr int kGroups = kThreads / TPR;
    __shared__ float sh_f[32];
    extern __shared__ float sh_dw[];   // [kGroups][TPR VPT W], kGroups > 1
    const int grp = threadIdx.x / TPR, t = threadIdx.x % TPR;
    using P = Pack<T, W>;
    Pack<float, W> w[VPT];
    float dw[VPT * W];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * TPR + t) * W;
        if (e < a.c) w[v] = *reinterpret_cast<const Pack<float, W>*>(a.weight + e);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[v * W + j] = 0.0f;
    }
    // every group of the block runs the same number of rounds (shuffles and barriers inside)
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kGroups; base < a.n;
         base += static_cast<int64_t>(gridDim.x) * kGroups) {
        const int64_t row = base + grp;
        const bool live = row < a.n;
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* dy = static_cast<const T*>(a.dy) + row * a.ldy;
        const T* dres = static_cast<const T*>(a.dres) + row * a.ldr;
        P px[VPT], pd[VPT], pr[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * TPR + t) * W;
            if (live && e < a.c) {
                px[v] = *reinterpret_cast<const P*>(x + e);
                pd[v] = *reinterpret_cast<const P*>(dy + e);
                if (a.dres) pr[v] = *reinterpret_cast<const P*>(dres + e);
            }
        }
        float ss = 0.0f, gh = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (!(live && (v * TPR + t) * W < a.c)) continue;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float h = to_f(px[v].v[j]);
                ss = fmaf(h, h, ss);
                gh = fmaf(to_f(pd[v].v[j]) * w[v].v[j], h, gh);
            }
        }
        ss = row_reduce<TPR>(ss, AddF(), sh_f);
        gh = row_reduce<TPR>(gh, AddF(), sh_f);
        const float inv_c = 1.0f / static_cast<float>(a.c);
        const float r = rsqrtf(ss * inv_c + a.eps);
        const float k = r * r * r * gh * inv_c;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * TPR + t) * W;
            if (!(live && e < a.c)) continue;
            P o;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float h = to_f(px[v].v[j]), d = to_f(pd[v].v[j]);
                float dx = fmaf(d * w[v].v[j], r, -h * k);
                if (a.dres) dx += to_f(pr[v].v[j]);
                from_f(dx, o.v[j]);
                dw[v * W + j] = fmaf(d, h * r, dw[v * W + j]);
            }
            *reinterpret_cast<P*>(static_cast<T*>(a.dx) + row * a.c + e) = o;
        }
    }
    float* dst = part + static_cast<int64_t>(blockIdx.x) * a.c;
    if (kGroups == 1) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int e = (v * TPR + t) * W + j;
                if (e < a.c) dst[e] = dw[v * W + j];
            }
    } else {
        constexpr int kCols = TPR * VPT * W;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int j = 0; j < W; ++j) sh_dw[grp * kCols + (v * TPR + t) * W + j] = dw[v * W + j];
        __syncthreads();
        for (int e = threadIdx.x; e < a.c; e += kThreads) {
            float s = 0.0f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) s += sh_dw[g * kCols + e];
            dst[e] = s;
        }
    }
}

// Rows too long to hold: each block keeps its running dw in its
// own row of `part` (zeroed), each element touched by one thread only.
template <typename T, int W>
__global__ void __launch_bounds__(kWideThreads) k_rms_norm_grad_wide(const NormGradArgs a, float* part) {
    __shared__ float sh_f[32];
    using P = Pack<T, W>;
    float* dw = part + static_cast<int64_t>(blockIdx.x) * a.c;
    const float inv_c = 1.0f / static_cast<float>(a.c);
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* dy = static_cast<const T*>(a.dy) + row * a.ldy;
        const T* dres = static_cast<const T*>(a.dres) + row * a.ldr;
        float ss = 0.0f, gh = 0.0f;
        for (int e = threadIdx.x * W; e < a.c; e += kWideThreads * W) {
            const P p = *reinterpret_cast<const P*>(x + e), d = *reinterpret_cast<const P*>(dy + e);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float h = to_f(p.v[j]);
                ss = fmaf(h, h, ss);
                gh = fmaf(to_f(d.v[j]) * a.weight[e + j], h, gh);
            }
        }
        ss = row_reduce<kWideThreads>(ss, AddF(), sh_f);
        gh = row_reduce<kWideThreads>(gh, AddF(), sh_f);
        const float r = rsqrtf(ss * inv_c + a.eps);
        const float k = r * r * r * gh * inv_c;
        for (int e = threadIdx.x * W; e < a.c; e += kWideThreads * W) {
            const P p = *reinterpret_cast<const P*>(x + e), d = *reinterpret_cast<const P*>(dy + e);
            P q, o;
            if (a.dres) q = *reinterpret_cast<const P*>(dres + e);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float h = to_f(p.v[j]), dj = to_f(d.v[j]);
                float dx = fmaf(dj * a.weight[e + j], r, -h * k);
                if (a.dres) dx += to_f(q.v[j]);
                from_f(dx, o.v[j]);
                dw[e + j] = fmaf(dj, h * r, dw[e + j]);
            }
            *reinterpret_cast<P*>(static_cast<T*>(a.dx) + row * a.c + e) = o;
        }
    }
}

bool vec_ok(const void* p, int64_t ld, size_t elem) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * static_cast<int64_t>(elem)) % 16 == 0;
}

// Calls f(W, TPR, VPT) (as constants) with the smallest row layout that holds
// c elements, W per load.  The backward pass holds a row's x, dy and weight and
// the running dw: 512 threads x 4 vectors would spill.
template <int W, bool BACKWARD, typename F>
bool with_layout(int32_t c, F&& f) {
    constexpr int S = 8 / W;   // W = 1 holds the same elements in eight times the loads
#define SPCONV_NORM_LAYOUT(TPR, VPT)                                                                           \
    if (c <= TPR * VPT * 8) {                                                                                  \
        f(std::integral_constant<int, W>(), std::integral_constant<int, TPR>(), std::integral_constant<int, VPT * S>()); \
        return true;                                                                                           \
    }
    SPCONV_NORM_LAYOUT(8, 1)
    SPCONV_NORM_LAYOUT(16, 1)
    SPCONV_NORM_LAYOUT(32, 1)
    SPCONV_NORM_LAYOUT(32, 2)
    SPCONV_NORM_LAYOUT(128, 1)
    SPCONV_NORM_LAYOUT(128, 2)
    SPCONV_NORM_LAYOUT(256, 2)
    SPCONV_NORM_LAYOUT(512, 2)
    if constexpr (!BACKWARD) {
        SPCONV_NORM_LAYOUT(512, 4)
    }
#undef SPCONV_NORM_LAYOUT
    return false;
}

template <typename T, int W, bool EIGHT>
int forward_t(const NormArgs& a, cudaStream_t s) {
    count_launch();
    const bool held = with_layout<W, false>(a.c, [&](auto w, auto tpr, auto vpt) {
        constexpr int kThreads = tpr > 32 ? tpr : kBlock;
        const int64_t blocks = ceil_div(a.n, kThreads / tpr);
        k_rms_norm<T, w, tpr, vpt, EIGHT><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
    });
    if (!held) k_rms_norm_wide<T, W, EIGHT><<<static_cast<unsigned>(a.n < 1216 ? a.n : 1216), kWideThreads, 0, s>>>(a);
    return launch_status();
}

template <typename T, int W>
int backward_t(const NormGradArgs& a, cudaStream_t s) {
    int rc = SPCONV_OK;
    const bool held = with_layout<W, true>(a.c, [&](auto w, auto tpr, auto vpt) {
        constexpr int kThreads = tpr > 32 ? tpr : kBlock;
        constexpr int kGroups = kThreads / tpr;
        constexpr int kSmem = kGroups > 1 ? kThreads * vpt * w * 4 : 0;
        const int64_t want = ceil_div(a.n, kGroups);
        const int64_t most = 152 * (1024 / kThreads);
        const int64_t blocks = want < most ? want : most;
        Scratch part(static_cast<size_t>(blocks) * a.c * 4, s);
        if (part.failed()) {
            rc = SPCONV_ERR_OOM;
            return;
        }
        count_launch();
        k_rms_norm_grad<T, w, tpr, vpt><<<static_cast<unsigned>(blocks), kThreads, kSmem, s>>>(a, part.as<float>());
        rc = launch_status();
        if (rc == SPCONV_OK) rc = sum_partials(part.as<float>(), blocks, a.c, a.dweight, s);
    });
    if (held) return rc;
    const int64_t blocks = a.n < 304 ? a.n : 304;
    const size_t bytes = static_cast<size_t>(blocks) * a.c * 4;
    Scratch part(bytes, s);
    if (part.failed()) return SPCONV_ERR_OOM;
    SPCONV_CHECK_CUDA(cudaMemsetAsync(part.as<float>(), 0, bytes, s));
    count_launch();
    k_rms_norm_grad_wide<T, W><<<static_cast<unsigned>(blocks), kWideThreads, 0, s>>>(a, part.as<float>());
    SPCONV_CHECK(launch_status());
    return sum_partials(part.as<float>(), blocks, a.c, a.dweight, s);
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
