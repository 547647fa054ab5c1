// Root-mean-square norm of rows, with the residual's addition, an optional
// 8-bit output, and its backward pass.
//
//   h = x + residual;  r = 1 / sqrt(mean_c h^2 + eps);  y = h r w
//   8 bits: scale = max_c |y| / 448,  q = e4m3(y / scale)
//
// Everything between the loads and the stores is fp32, with one rounding per
// output.  The kernels are bound by HBM: a row is read once into registers,
// reduced, and written; the next row's loads are in flight meanwhile.
#include "ptx_sm100.cuh"
#include "rows.cuh"

namespace spconv {
namespace {

constexpr int kBlock = 256;          // threads of a block that holds several rows
constexpr int kLongThreads = 512;    // threads of a block that walks a row too long to hold
constexpr float kE4m3Max = 448.0f;

// W consecutive elements as they lie in memory (W = 8 is one or two 16-byte loads).
template <typename T, int W>
struct alignas(sizeof(T) * W < 16 ? sizeof(T) * W : 16) Pack {
    T v[W];
};

// To fp32 and back (one rounding); pairs of bf16 take one instruction each.
template <int W>
__device__ __forceinline__ void unpack(const Pack<float, W>& p, float (&f)[W]) {
#pragma unroll
    for (int j = 0; j < W; ++j) f[j] = p.v[j];
}
template <int W>
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, W>& p, float (&f)[W]) {
    if constexpr (W == 8) {
        const uint4 q = reinterpret_cast<const uint4&>(p);
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(u[j] << 16);
            f[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) f[j] = __bfloat162float(p.v[j]);
    }
}
template <int W>
__device__ __forceinline__ void pack(const float (&f)[W], Pack<float, W>& p) {
#pragma unroll
    for (int j = 0; j < W; ++j) p.v[j] = f[j];
}
template <int W>
__device__ __forceinline__ void pack(const float (&f)[W], Pack<__nv_bfloat16, W>& p) {
    if constexpr (W == 8) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
            u[j] = reinterpret_cast<const uint32_t&>(v);
        }
        reinterpret_cast<uint4&>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) p.v[j] = __float2bfloat16_rn(f[j]);
    }
}

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
    } else if (W == 2) {
        *reinterpret_cast<uint16_t*>(dst) = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1 % W]), __NV_SATFINITE, __NV_E4M3);
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
                                            float (&h)[VPT][W], int t, int tpr) {
    SumMax st{0.0f, 0u};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if ((v * tpr + t) * W >= a.c) continue;
        unpack<W>(p.x[v], h[v]);
        if (a.residual) {
            float r[W];
            unpack<W>(p.r[v], r);
#pragma unroll
            for (int j = 0; j < W; ++j) h[v][j] += r[j];
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            st.s = fmaf(h[v][j], h[v][j], st.s);
            if (EIGHT) {
                const uint32_t b = __float_as_uint(fabsf(h[v][j] * w[v].v[j]));
                st.m = b > st.m ? b : st.m;
            }
        }
    }
    return st;
}

// Writes the row.  y = (h w) r, and r is one positive factor: max |y| is
// (max |h w|) r, so the two reductions are one, and y / scale is
// (h w) 448 / max |h w| without r.  That factor overflows where the maximum is
// below 2^-119: such rows are first brought up by 2^100.  A row of zeros has
// scale 0 and q 0.
template <typename T, int W, int VPT, bool EIGHT>
__device__ __forceinline__ void row_write(const NormArgs& a, int64_t row, SumMax st, const Pack<float, W> (&w)[VPT],
                                          const float (&h)[VPT][W], int t, int tpr) {
    using P = Pack<T, W>;
    const float r = rsqrtf(st.s / static_cast<float>(a.c) + a.eps);
    float factor = r, pre = 1.0f;
    if (EIGHT) {
        const float amax = __uint_as_float(st.m);
        if (t == 0) a.scale[row] = amax * r / kE4m3Max;
        pre = amax < 0x1p-100f ? 0x1p100f : 1.0f;
        factor = amax == 0.0f ? 0.0f : kE4m3Max / (amax * pre);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * tpr + t) * W;
        if (e >= a.c) continue;
        P o;
        if (a.sum) {
            pack<W>(h[v], o);
            *reinterpret_cast<P*>(static_cast<T*>(a.sum) + row * a.c + e) = o;
        }
        float y[W];
#pragma unroll
        for (int j = 0; j < W; ++j) y[j] = h[v][j] * w[v].v[j];
        if (EIGHT && pre != 1.0f) {
#pragma unroll
            for (int j = 0; j < W; ++j) y[j] *= pre;
        }
#pragma unroll
        for (int j = 0; j < W; ++j) y[j] *= factor;
        if (EIGHT) {
            store_e4m3<W>(static_cast<uint8_t*>(a.out) + row * a.c + e, y);
        } else {
            pack<W>(y, o);
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

// Rows of up to 1024 elements (512 where no 16-byte load takes them): TPR lanes per
// row, many rows per block; enough independent warps that the loads of some cover the
// arithmetic of others.  With a residual, bf16: 600000 x 128 89 us, 6.9 TB/s; 75000 x
// 1024 89 us, where the ring below takes 102.
template <typename T, int W, int TPR, int VPT, bool EIGHT>
__global__ void __launch_bounds__(kBlock) k_rms_norm(const NormArgs a) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kBlock / TPR) + threadIdx.x / TPR;
    const int t = threadIdx.x % TPR;
    const bool live = row < a.n;   // (lanes of absent rows still take part in the shuffles)
    RowPart<T, W, VPT> p;
    Pack<float, W> w[VPT];
    float h[VPT][W];
    SumMax st{0.0f, 0u};
    pdl_wait();   // (also before the weight: the kernel before this one may write it)
    pdl_trigger();
    load_weight<W, VPT>(a.weight, a.c, w, t, TPR);
    if (live) {
        p.load(a, row, t, TPR);
        st = row_stats<T, W, VPT, EIGHT>(a, p, w, h, t, TPR);
    }
    st = lanes_reduce<TPR>(st);
    if (live) row_write<T, W, VPT, EIGHT>(a, row, st, w, h, t, TPR);
}

// Rows of 513 to 4096 elements that no vector load takes: one block per row,
// persistent, the next row's loads in flight while this one is reduced and
// written; the weight stays in registers.  75000 x 1001 bf16 133 us, 4.5 TB/s: the
// loads of two bytes bound it (in two passes as below 306; 25000 x 3001 167, 189).
template <typename T, int W, int VPT, bool EIGHT>
__global__ void __launch_bounds__(512) k_rms_norm_block(const NormArgs a) {
    __shared__ SumMax sh[64];
    const int t = threadIdx.x, tpr = blockDim.x;
    RowPart<T, W, VPT> p, next;
    Pack<float, W> w[VPT];
    float h[VPT][W];
    pdl_wait();
    pdl_trigger();
    load_weight<W, VPT>(a.weight, a.c, w, t, tpr);
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
// mostly from L2; 3000 x 24000 bf16 113 us, 5.1 TB/s).  Every element is read by the thread that writes it, after
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
        float h[1][W];
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
//   dx = r (g - (h r) m) + dres,  m = r mean_c(g h),   dw_c = sum_rows dy h r
// h r has unit size and m the size of g whatever the size of the row; the cube
// of r, which the same formula has when multiplied out, leaves the range of fp32
// for rows below 1e-13 (eps = 0) and above 1e13.
// Each row's threads walk the rows first, first + step, ...; the weight and the
// running dw of their columns stay in registers, a block's rows are added in a
// fixed order and the block writes one row of partial sums (finish_sums adds
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
        float h[W], d[W];
        unpack<W>(p.x[v], h);
        unpack<W>(p.d[v], d);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            st.s = fmaf(h[j], h[j], st.s);
            st.t = fmaf(d[j] * w[v].v[j], h[j], st.t);
        }
    }
    return st;
}

// r = 1 / rms and m = r mean(g h) of a row
__device__ __forceinline__ Sum2 grad_factors(Sum2 st, int32_t c, float eps) {
    const float inv_c = 1.0f / static_cast<float>(c);
    const float r = rsqrtf(st.s * inv_c + eps);
    return {r, r * st.t * inv_c};
}

template <typename T, int W, int VPT>
__device__ __forceinline__ void grad_write(const NormGradArgs& a, int64_t row, Sum2 f, const GradPart<T, W, VPT>& p,
                                           const Pack<float, W> (&w)[VPT], float (&dw)[VPT][W], int t, int tpr) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * tpr + t) * W;
        if (e >= a.c) continue;
        float h[W], d[W], dx[W];
        unpack<W>(p.x[v], h);
        unpack<W>(p.d[v], d);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float unit = h[j] * f.s;
            dx[j] = f.s * fmaf(-unit, f.t, d[j] * w[v].v[j]);
            dw[v][j] = fmaf(d[j], unit, dw[v][j]);
        }
        if (a.dres) {
            float r[W];
            unpack<W>(p.r[v], r);
#pragma unroll
            for (int j = 0; j < W; ++j) dx[j] += r[j];
        }
        Pack<T, W> o;
        pack<W>(dx, o);
        *reinterpret_cast<Pack<T, W>*>(static_cast<T*>(a.dx) + row * a.c + e) = o;
    }
}

// Rows of 513 elements and more that no 16-byte load takes: one block per row, while
// the weight and the running dw fit the registers (with single elements up to 3584,
// fp32 4096: 25000 x 3001 bf16 199 us, the two passes below 479; with pairs up to
// 4096: of 6002 elements the passes take 170 us for 9000 rows, this 198).  75000 x
// 1001 takes 234 us, 2.6 TB/s: loads of two bytes keep too few on their way.
template <typename T, int W, int VPT>
__global__ void __launch_bounds__(512) k_rms_norm_grad_block(const NormGradArgs a, float* part) {
    __shared__ Sum2 sh[64];
    const int t = threadIdx.x, tpr = blockDim.x;
    Pack<float, W> w[VPT];
    float dw[VPT][W] = {};
    GradPart<T, W, VPT> p, next;
    pdl_wait();
    load_weight<W, VPT>(a.weight, a.c, w, t, tpr);
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
            if (e < a.c) part[static_cast<int64_t>(blockIdx.x) * a.c + e] = dw[v][j];
        }
}

// Longer rows in two passes: the factors of each row, then dx and the partial
// dw of a block of columns over a run of rows.  The second pass finds part of the
// rows in L2: 4600 x 16384 bf16 158 us, 3.8 TB/s of the bytes that one pass has.
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
    float dw[1][W] = {};
    load_weight<W, 1>(a.weight, a.c, w, t, 0);
#pragma unroll 2
    for (int64_t row = r0; row < r1; ++row) {
        GradPart<T, W, 1> p;
        p.load(a, row, t, 0);
        grad_write<T, W, 1>(a, row, factors[row], p, w, dw, t, 0);
    }
#pragma unroll
    for (int j = 0; j < W; ++j) part[static_cast<int64_t>(blockIdx.y) * a.c + t * W + j] = dw[0][j];
}

// ---- rows through shared memory -------------------------------------------------
// A load in flight costs a thread its destination registers: threads x 16 bytes
// x inputs is what an SM keeps on its way, and HBM wants some 60 KB per SM at
// its loaded latency.  Here bulk asynchronous copies bring stages of rows (one
// copy per input where the rows are dense) into a ring and the threads compute
// from it, so the bytes in flight are the ring's size.
constexpr int kMaxStages = 8;

struct Ring {
    int32_t stages, rows;       // of the ring; of a stage
    uint32_t bytes;             // of one input in a stage (a multiple of 16)
    int32_t* status;
};

// Consumers and producer of a ring of IN inputs.
template <typename T, int IN>
struct RingState {
    uint8_t* base;
    uint64_t *full, *empty;
    volatile int* abort_flag;

    // all threads; ends with a barrier
    __device__ __forceinline__ void init(uint8_t* smem, const Ring& g, int consumer_warps) {
        base = smem;
        full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(g.stages) * IN * g.bytes);
        empty = full + kMaxStages;
        abort_flag = reinterpret_cast<volatile int*>(empty + kMaxStages);
        if (threadIdx.x == 0) {
            for (int s = 0; s < g.stages; ++s) {
                ptx::mbar_init(&full[s], 1);
                ptx::mbar_init(&empty[s], consumer_warps);
            }
            *abort_flag = 0;
            ptx::fence_mbar_init();
        }
        __syncthreads();
    }
    __device__ __forceinline__ const T* rows(const Ring& g, int s, int in) const {
        return reinterpret_cast<const T*>(base + (static_cast<size_t>(s) * IN + in) * g.bytes);
    }
    __device__ __forceinline__ void fail(const Ring& g) {
        atomicOr(g.status, kStatusTimeout);
        *abort_flag = 1;
    }
    // Starts fill number k, tile `tile`, by `lanes` lanes of one warp (1: the calling thread).
    __device__ __forceinline__ void fill(const Ring& g, int64_t k, int64_t tile, int64_t n, int32_t c, const T* const (&src)[IN],
                                         const int64_t (&ld)[IN], int lane, int lanes) const {
        const int s = static_cast<int>(k % g.stages);
        const uint32_t row_bytes = static_cast<uint32_t>(c) * sizeof(T);
        const int64_t r0 = tile * g.rows;
        const int32_t rows_here = static_cast<int32_t>(n - r0 < g.rows ? n - r0 : g.rows);
        int inputs = 0;
#pragma unroll
        for (int i = 0; i < IN; ++i) inputs += src[i] != nullptr;
        // bulk copies move 16 bytes at a time: what dense rows of another size
        // leave over at the matrix's end is stored before the stage is published
        const uint32_t all = rows_here * row_bytes, over = all & 15;
        if (over) {
            const int32_t first = static_cast<int32_t>((all - over) / sizeof(T)), count = static_cast<int32_t>(all / sizeof(T));
#pragma unroll
            for (int i = 0; i < IN; ++i)
                for (int e = first + lane; src[i] && e < count; e += lanes)
                    const_cast<T*>(rows(g, s, i))[e] = src[i][r0 * ld[i] + e];
            if (lanes > 1) __syncwarp();
        }
        if (lane == 0) ptx::mbar_arrive_expect_tx(&full[s], inputs * (all - over));
        if (lanes > 1) __syncwarp();
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            if (!src[i]) continue;
            const uint32_t dst = ptx::smem_u32(rows(g, s, i));
            if (ld[i] == c) {
                if (lane == 0 && all > over) ptx::bulk_copy_g2s(dst, src[i] + r0 * ld[i], all - over, &full[s]);
            } else {
                for (int r = lane; r < rows_here; r += lanes)
                    ptx::bulk_copy_g2s(dst + r * row_bytes, src[i] + (r0 + r) * ld[i], row_bytes, &full[s]);
            }
        }
    }
    // After an abort: the copies of the fills before number k land before the block exits.
    __device__ __forceinline__ void drain(const Ring& g, int64_t k) const {
        for (int64_t j = k > g.stages ? k - g.stages : 0; j < k; ++j)
            ptx::mbar_wait(&full[j % g.stages], static_cast<uint32_t>(j / g.stages) & 1, nullptr);
    }
};

// Keeps the shared-memory loads of one vector behind the work on the one
// before: all of a row's loaded at once would cost the registers that hold dw.
__device__ __forceinline__ void apart() { asm volatile("" ::: "memory"); }

// Rows of 513 elements and more: a row per block and stage, so a block needs
// 1/32 of the row's elements as threads and many blocks share an SM (the
// barriers of one fall into the work of others).  There is no copying warp:
// when the block meets to reduce row k, every thread is done with row k - 1,
// and thread 0 refills that row's stage.  Rows of 1025 to 16384 elements (fp32
// 8192), as many as two stages of an SM's shared memory hold: to e4m3, 37000 x 2048
// 85 us, 6.2 TB/s (the two passes above 198), 16381 x 8192 154 us; 4600 x 16384 to
// bf16 104 us (110).
template <typename T, bool EIGHT>
__global__ void __launch_bounds__(512, 1) k_rms_norm_ring(const NormArgs a, const Ring g) {
    constexpr int VPT = 4;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ SumMax sh[64];
    RingState<T, 2> ring;
    ring.init(smem, g, 1);
    const int t = threadIdx.x, threads = blockDim.x;
    Pack<float, 8> w[VPT];
    const T* const src[2] = {static_cast<const T*>(a.x), static_cast<const T*>(a.residual)};
    const int64_t ld[2] = {a.ldx, a.ldr};
    pdl_wait();
    pdl_trigger();
    int64_t filled = 0;   // (thread 0)
    if (t == 0)
        for (int64_t row = blockIdx.x; row < a.n && filled < g.stages; row += gridDim.x, ++filled)
            ring.fill(g, filled, row, a.n, a.c, src, ld, 0, 1);
    load_weight<8, VPT>(a.weight, a.c, w, t, threads);
    int k = 0;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, ++k) {
        const int s = k % g.stages;
        // (a thread that gave up still meets the others at the barrier)
        if (!ptx::mbar_wait(&ring.full[s], static_cast<uint32_t>(k / g.stages) & 1, ring.abort_flag)) ring.fail(g);
        NormArgs b = a;   // the stage's row in place of the global one
        b.x = ring.rows(g, s, 0);
        b.residual = a.residual ? ring.rows(g, s, 1) : nullptr;
        RowPart<T, 8, 1> p;
        Pack<float, 8> wv[1];
        float h[1][8];
        SumMax st{0.0f, 0u};
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            p.load(b, 0, v * threads + t, 0);
            wv[0] = w[v];
            st = join(st, row_stats<T, 8, 1, EIGHT>(a, p, wv, h, v * threads + t, 0));
        }
        st = block_reduce(st, sh, k);
        if (*ring.abort_flag) break;
        const int64_t next = row + (g.stages - 1) * static_cast<int64_t>(gridDim.x);
        if (t == 0 && k > 0 && next < a.n) ring.fill(g, filled++, next, a.n, a.c, src, ld, 0, 1);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            apart();
            p.load(b, 0, v * threads + t, 0);
            wv[0] = w[v];
            row_stats<T, 8, 1, false>(a, p, wv, h, v * threads + t, 0);
            row_write<T, 8, 1, EIGHT>(a, row, st, wv, h, v * threads + t, 0);
        }
    }
    if (t == 0 && *ring.abort_flag) ring.drain(g, filled);   // (set before the last barrier, if at all)
}

// The backward pass of such rows, up to 8192 elements (fp32 4096).  The row's
// vectors are taken from shared memory again for the second pass, and the weight's
// from L1 or L2: the registers hold the running dw.  Bound by issue and the row's
// barriers rather than HBM: 9000 x 8192 bf16 117 us, 5.1 TB/s (in two passes 160),
// 37000 x 2048 118 (231).
template <typename T, int VPT>
__global__ void __launch_bounds__(512, 1) k_rms_norm_grad_ring(const NormGradArgs a, const Ring g, float* part) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Sum2 sh[64];
    RingState<T, 3> ring;
    ring.init(smem, g, 1);
    const int t = threadIdx.x, threads = blockDim.x;
    float dw[VPT][1][8] = {};
    const T* const src[3] = {static_cast<const T*>(a.x), static_cast<const T*>(a.dy), static_cast<const T*>(a.dres)};
    const int64_t ld[3] = {a.ldx, a.ldy, a.ldr};
    pdl_wait();
    int64_t filled = 0;
    if (t == 0)
        for (int64_t row = blockIdx.x; row < a.n && filled < g.stages; row += gridDim.x, ++filled)
            ring.fill(g, filled, row, a.n, a.c, src, ld, 0, 1);
    int k = 0;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, ++k) {
        const int s = k % g.stages;
        if (!ptx::mbar_wait(&ring.full[s], static_cast<uint32_t>(k / g.stages) & 1, ring.abort_flag)) ring.fail(g);
        NormGradArgs b = a;
        b.x = ring.rows(g, s, 0);
        b.dy = ring.rows(g, s, 1);
        b.dres = nullptr;
        GradPart<T, 8, 1> p;
        Pack<float, 8> wv[1];
        Sum2 st{0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            apart();
            p.load(b, 0, v * threads + t, 0);
            load_weight<8, 1>(a.weight, a.c, wv, v * threads + t, 0);
            st = join(st, grad_stats<T, 8, 1>(a, p, wv, v * threads + t, 0));
        }
        st = block_reduce(st, sh, k);
        if (*ring.abort_flag) break;
        const int64_t next = row + (g.stages - 1) * static_cast<int64_t>(gridDim.x);
        if (t == 0 && k > 0 && next < a.n) ring.fill(g, filled++, next, a.n, a.c, src, ld, 0, 1);
        const Sum2 f = grad_factors(st, a.c, a.eps);
        b.dres = a.dres ? ring.rows(g, s, 2) : nullptr;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            apart();
            p.load(b, 0, v * threads + t, 0);
            load_weight<8, 1>(a.weight, a.c, wv, v * threads + t, 0);
            grad_write<T, 8, 1>(a, row, f, p, wv, dw[v], v * threads + t, 0);
        }
    }
    if (t == 0 && *ring.abort_flag) ring.drain(g, filled);   // (set before the last barrier, if at all)
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = (v * threads + t) * 8 + j;
            if (e < a.c) part[static_cast<int64_t>(blockIdx.x) * a.c + e] = dw[v][0][j];
        }
}

// Shorter rows, backward (up to 1024 elements; fp32, and where no 16-byte load takes
// them, 512): a row per TPR lanes, one warp of the block copies stages of many rows;
// no barrier of the block.  75000 x 1000 bf16 92 us, 6.5 TB/s (the ring above 129);
// 300000 x 255 133 (a block per row 241).  A stage starts a multiple of eight rows in, which is 16
// bytes aligned for any number of elements where the rows are dense (W < 8).
template <typename T, int W, int TPR, int VPT>
__global__ void __launch_bounds__(kBlock + 32, VPT * W > 16 || (VPT * W > 8 && (sizeof(T) == 4 || W < 8)) ? 1 : 2)
    k_rms_norm_grad_lanes(const NormGradArgs a, const Ring g, float* part) {
    constexpr int kGroups = kBlock / TPR, kCols = TPR * VPT * W;
    extern __shared__ __align__(128) uint8_t smem[];
    RingState<T, 3> ring;
    ring.init(smem, g, kBlock / 32);
    const bool consumer = threadIdx.x < kBlock;
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    Pack<float, W> w[VPT];
    float dw[VPT][1][W] = {};
    const int64_t tiles = (a.n + g.rows - 1) / g.rows;
    pdl_wait();
    if (consumer) load_weight<W, VPT>(a.weight, a.c, w, t, TPR);
    int64_t k = 0;
    if (!consumer) {
        const T* const src[3] = {static_cast<const T*>(a.x), static_cast<const T*>(a.dy), static_cast<const T*>(a.dres)};
        const int64_t ld[3] = {a.ldx, a.ldy, a.ldr};
        const int lane = threadIdx.x & 31;
        for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++k) {
            if (k >= g.stages &&
                !__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&ring.empty[k % g.stages], static_cast<uint32_t>(k / g.stages - 1) & 1,
                                                        ring.abort_flag))) {
                if (lane == 0) ring.fail(g);
                break;
            }
            ring.fill(g, k, tile, a.n, a.c, src, ld, lane, 32);
        }
    } else {
        for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++k) {
            const int s = static_cast<int>(k % g.stages);
            if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&ring.full[s], static_cast<uint32_t>(k / g.stages) & 1, ring.abort_flag))) {
                if ((threadIdx.x & 31) == 0) ring.fail(g);
                break;
            }
            NormGradArgs b = a;   // the stage's rows in place of global ones
            b.x = ring.rows(g, s, 0);
            b.dy = ring.rows(g, s, 1);
            b.dres = a.dres ? ring.rows(g, s, 2) : nullptr;
            b.ldx = b.ldy = b.ldr = a.c;
            for (int r = grp; r < g.rows; r += kGroups) {
                const int64_t row = tile * g.rows + r;
                const bool live = row < a.n;
                GradPart<T, W, 1> p;
                Pack<float, W> wv[1];
                Sum2 st{0.0f, 0.0f};
                if (live) {
#pragma unroll
                    for (int v = 0; v < VPT; ++v) {
                        p.load(b, r, v * TPR + t, 0);
                        wv[0] = w[v];
                        st = join(st, grad_stats<T, W, 1>(a, p, wv, v * TPR + t, 0));
                    }
                }
                st = lanes_reduce<TPR>(st);
                if (live) {
                    const Sum2 f = grad_factors(st, a.c, a.eps);
#pragma unroll
                    for (int v = 0; v < VPT; ++v) {
                        apart();
                        p.load(b, r, v * TPR + t, 0);
                        wv[0] = w[v];
                        grad_write<T, W, 1>(a, row, f, p, wv, dw[v], v * TPR + t, 0);
                    }
                }
            }
            __syncwarp();
            if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&ring.empty[s]);
        }
    }
    // the block's rows are added through the ring's memory, free by now
    float* sh_dw = reinterpret_cast<float*>(smem);   // [kGroups][kCols]
    __syncthreads();
    if (!consumer && *ring.abort_flag) ring.drain(g, k);
    if (consumer) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int j = 0; j < W; ++j) sh_dw[grp * kCols + (v * TPR + t) * W + j] = dw[v][0][j];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.c; e += blockDim.x) {
        float sum = 0.0f;
        for (int q = 0; q < kGroups; ++q) sum += sh_dw[q * kCols + e];
        part[static_cast<int64_t>(blockIdx.x) * a.c + e] = sum;
    }
}

bool vec_ok(const void* p, int64_t ld, size_t elem) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * static_cast<int64_t>(elem)) % 16 == 0;
}

// bf16 rows that two-element loads may take
bool pair_ok(const void* p, int64_t ld, uintptr_t align = 4) {
    return (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0 && ld % 2 == 0;
}

template <typename... K, typename... A>
int launch(void (*kernel)(K...), int64_t blocks, int threads, size_t smem, cudaStream_t s, A... args) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), threads, smem, s, args...);
}

constexpr int64_t kSms = 152;

// The ring of a kernel with `in` inputs and `rows` rows a stage.  *per_sm
// blocks share an SM's shared memory: the most asked for, or fewer where that
// leaves less than two stages.
int make_ring(Ring* g, size_t* smem, int32_t c, size_t es, int in, int64_t rows, int* per_sm) {
    g->rows = static_cast<int32_t>(rows);
    g->bytes = static_cast<uint32_t>(round_up(static_cast<size_t>(rows) * c * es, 128));
    for (;; --*per_sm) {
        if (*per_sm < 1) return SPCONV_ERR_UNSUPPORTED;
        g->stages = static_cast<int32_t>((static_cast<size_t>(220 * 1024) / *per_sm - 2048) / (in * g->bytes));
        if (g->stages >= 2) break;
    }
    if (g->stages > kMaxStages) g->stages = kMaxStages;
    *smem = static_cast<size_t>(g->stages) * in * g->bytes + 2 * kMaxStages * 8 + 16;
    return rows_status_word(&g->status);
}

template <auto KERNEL, typename... A>
int launch_ring(int64_t blocks, int threads, size_t smem, cudaStream_t s, A... args) {
    static bool set[kMaxDevices] = {};
    int dev = 0;
    SPCONV_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return SPCONV_ERR_UNSUPPORTED;
    if (!set[dev]) {
        SPCONV_CHECK_CUDA(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024));
        set[dev] = true;
    }
    return launch(KERNEL, blocks, threads, smem, s, args...);
}

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

template <typename T, int W, bool EIGHT>
int forward_t(const NormArgs& a, cudaStream_t s) {
    constexpr int S = 8 / W;   // fewer elements per load: as many times the loads
    constexpr bool kVec = W == 8;
    if constexpr (kVec) {
        if (a.c > 1024 && a.c <= (sizeof(T) == 2 ? 16384 : 8192)) {
            Ring g;
            size_t smem;
            const int threads = block_threads(a.c, 32);
            int per_sm = 512 / threads;
            SPCONV_CHECK(make_ring(&g, &smem, a.c, sizeof(T), 2, 1, &per_sm));
            const int64_t most = kSms * per_sm;
            return launch_ring<k_rms_norm_ring<T, EIGHT>>(a.n < most ? a.n : most, threads, smem, s, a, g);
        }
    }
    if (a.c <= (kVec ? 1024 : 512))
        return with_lanes<kVec>(a.c, [&](auto tpr, auto vpt) {
            return launch(k_rms_norm<T, W, tpr, vpt * S, EIGHT>, ceil_div(a.n, kBlock / tpr), kBlock, 0, s, a);
        });
    if constexpr (W == 1) {
        if (a.c <= 4096) {
            const int threads = block_threads(a.c, 8);
            const int64_t most = kSms * (1024 / threads);
            return launch(k_rms_norm_block<T, W, S, EIGHT>, a.n < most ? a.n : most, threads, 0, s, a);
        }
    }
    const int64_t most = kSms * 4;
    return launch(k_rms_norm_long<T, W, EIGHT>, a.n < most ? a.n : most, kLongThreads, 0, s, a);
}

template <typename T, int W>
int backward_t(const NormGradArgs& a, cudaStream_t s) {
    constexpr bool kVec = W == 8;
    // blocks: partial sums of dw, one row each
    auto with_part = [&](int64_t blocks, auto&& run) -> int {
        Scratch part(static_cast<size_t>(blocks) * a.c * 4, s);
        if (part.failed()) return SPCONV_ERR_OOM;
        SPCONV_CHECK(run(part.as<float>()));
        return finish_sums(nullptr, 0, {part.as<float>(), blocks, a.c, a.dweight}, s);
    };
    Ring g;
    size_t smem;
    auto dense = [&](const void* p, int64_t ld) { return !p || (vec_ok(p, 0, 2) && ld == a.c); };
    constexpr bool kWide = kVec && sizeof(T) == 2;   // (others would spill)
    if (a.c <= (kWide ? 1024 : 512) && (kVec || (dense(a.x, a.ldx) && dense(a.dy, a.ldy) && dense(a.dres, a.ldr))))
        return with_lanes<kWide>(a.c, [&](auto tpr, auto vpt) {
            // stages of 8 KB per input at least, so that barriers are few
            const int64_t unit = kBlock / tpr, row = static_cast<int64_t>(a.c) * sizeof(T);
            int per_sm = vpt > 2 || (vpt > 1 && !kWide) ? 1 : 2;
            SPCONV_CHECK(make_ring(&g, &smem, a.c, sizeof(T), 3, unit * ceil_div(8192, unit * row), &per_sm));
            const int64_t tiles = ceil_div(a.n, g.rows), most = kSms * per_sm, blocks = tiles < most ? tiles : most;
            return with_part(blocks, [&](float* part) {
                return launch_ring<k_rms_norm_grad_lanes<T, W, tpr, vpt * (8 / W)>>(blocks, kBlock + 32, smem, s, a, g, part);
            });
        });
    if constexpr (kVec) {
        if (a.c <= (sizeof(T) == 2 ? 8192 : 4096)) {
            constexpr int kVpt = sizeof(T) == 2 ? 4 : 2;
            const int threads = block_threads(a.c, 8 * kVpt);
            int per_sm = 512 / threads;
            SPCONV_CHECK(make_ring(&g, &smem, a.c, sizeof(T), 3, 1, &per_sm));
            const int64_t most = kSms * per_sm, blocks = a.n < most ? a.n : most;
            return with_part(blocks, [&](float* part) {
                return launch_ring<k_rms_norm_grad_ring<T, kVpt>>(blocks, threads, smem, s, a, g, part);
            });
        }
    }
    if constexpr (!kVec) {
        auto block = [&](auto vpt) {
            const int threads = block_threads(a.c, vpt * W);
            const int64_t most = kSms * (1024 / threads), blocks = a.n < most ? a.n : most;
            return with_part(blocks, [&](float* part) {
                return launch(k_rms_norm_grad_block<T, W, vpt>, blocks, threads, 0, s, a, part);
            });
        };
        if (a.c <= 512 * 4 * W) return block(std::integral_constant<int, 4>());
        if constexpr (W == 1) {
            constexpr int kMost = sizeof(T) == 2 ? 7 : 8;   // (bf16 rows would spill)
            if (a.c <= 512 * kMost) return block(std::integral_constant<int, kMost>());
        }
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
    // (between, a block per row with single loads is faster: 75000 x 1002 133 us, by pairs 268)
    const bool pairs = (a.c <= 512 || a.c > 4096) && a.c % 2 == 0 && pair_ok(a.x, a.ldx) && pair_ok(a.residual, a.ldr) && pair_ok(a.weight, 0, 8) &&
                       pair_ok(a.sum, 0) && pair_ok(a.out, 0, eight ? 2 : 4);
    if (a.dtype == SPCONV_FP32)
        return vec ? (eight ? forward_t<float, 8, true>(a, s) : forward_t<float, 8, false>(a, s))
                   : (eight ? forward_t<float, 1, true>(a, s) : forward_t<float, 1, false>(a, s));
    if (vec) return eight ? forward_t<__nv_bfloat16, 8, true>(a, s) : forward_t<__nv_bfloat16, 8, false>(a, s);
    if (pairs) return eight ? forward_t<__nv_bfloat16, 2, true>(a, s) : forward_t<__nv_bfloat16, 2, false>(a, s);
    return eight ? forward_t<__nv_bfloat16, 1, true>(a, s) : forward_t<__nv_bfloat16, 1, false>(a, s);
}

int norm_backward(const NormGradArgs& a, cudaStream_t s) {
    const size_t es = a.dtype == SPCONV_FP32 ? 4 : 2;
    const bool vec = a.c % 8 == 0 && vec_ok(a.dy, a.ldy, es) && vec_ok(a.x, a.ldx, es) && vec_ok(a.dres, a.ldr, es) &&
                     vec_ok(a.weight, 0, 4) && vec_ok(a.dx, 0, es);
    if (a.dtype == SPCONV_FP32) return vec ? backward_t<float, 8>(a, s) : backward_t<float, 1>(a, s);
    // (from 2049 on a thread's pairs take the registers of the other blocks of its SM: 25000 x 3002
    // 263 us, by single elements 199; 37000 x 2046 197, 225)
    const bool pairs = (a.c <= 2048 || a.c > 3584) && a.c % 2 == 0 && pair_ok(a.dy, a.ldy) && pair_ok(a.x, a.ldx) && pair_ok(a.dres, a.ldr) &&
                       pair_ok(a.weight, 0, 8) && pair_ok(a.dx, 0);
    return vec     ? backward_t<__nv_bfloat16, 8>(a, s)
           : pairs ? backward_t<__nv_bfloat16, 2>(a, s)
                   : backward_t<__nv_bfloat16, 1>(a, s);
}

}  // namespace spconv
