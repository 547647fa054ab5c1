// Products with an epilogue, the column sums of the bias gradients, and the
// 8-bit weight layout.
#include "rows.cuh"

#include <type_traits>

namespace spconv {
namespace {

// ---- the product: 64 x 64 tiles in fp32 ---------------------------------------
constexpr int kT = 64, kTK = 16;

__device__ __forceinline__ float elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float elem(const __nv_fp8_e4m3* p) { return static_cast<float>(*p); }

template <typename T, int EPI>
__global__ void __launch_bounds__(256) k_dense_simt(const DenseOp op, int32_t n_tiles, float* part) {
    __shared__ float sa[kTK][kT + 4], sb[2][kTK][kT + 4];
    __shared__ float sh_cols[16][kT];
    constexpr int kAcc = (EPI == kEpiGated || EPI == kEpiGatedGrad) ? 2 : 1;
    const int src = static_cast<int>(blockIdx.y);   // n source
    const int64_t m0 = static_cast<int64_t>(blockIdx.x / n_tiles) * kT, n0 = static_cast<int64_t>(blockIdx.x % n_tiles) * kT;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[kAcc][4][4] = {};
    for (int ks = 0; ks < op.k_sources; ++ks) {
        const T* A = static_cast<const T*>(op.a.p[ks]);
        for (int64_t k0 = 0; k0 < op.k; k0 += kTK) {
            for (int i = threadIdx.x; i < kT * kTK; i += 256) {
                const int r = op.a.k_major ? i / kTK : i % kT, k = op.a.k_major ? i % kTK : i / kT;
                const int64_t gm = m0 + r, gk = k0 + k;
                sa[k][r] = gm < op.m && gk < op.k ? elem(A + (op.a.k_major ? gm * op.a.ld + gk : gk * op.a.ld + gm)) : 0.0f;
            }
#pragma unroll
            for (int q = 0; q < kAcc; ++q) {
                const T* B = static_cast<const T*>(op.b.p[kAcc == 2 ? q : (op.k_sources == 2 ? ks : src)]);
                for (int i = threadIdx.x; i < kT * kTK; i += 256) {
                    const int r = op.b.k_major ? i / kTK : i % kT, k = op.b.k_major ? i % kTK : i / kT;
                    const int64_t gn = n0 + r, gk = k0 + k;
                    sb[q][k][r] =
                        gn < op.n && gk < op.k ? elem(B + (op.b.k_major ? gn * op.b.ld + gk : gk * op.b.ld + gn)) : 0.0f;
                }
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kTK; ++k)
#pragma unroll
                for (int q = 0; q < kAcc; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[q][i][j] = fmaf(sa[k][ty + 16 * i], sb[q][k][tx + 16 * j], acc[q][i][j]);
            __syncthreads();
        }
    }
    const __nv_bfloat16* extra = static_cast<const __nv_bfloat16*>(op.extra);
    __nv_bfloat16* out0 = static_cast<__nv_bfloat16*>(op.out[EPI == kEpiLinear ? src : 0]);
    __nv_bfloat16* out1 = static_cast<__nv_bfloat16*>(op.out[1]);
    float cols[4] = {};
    with_act(op.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (m >= op.m || n >= op.n) continue;
                float z = acc[0][i][j];
                const float rs = op.row_scale ? op.row_scale[m] : 1.0f;
                if (op.col_scale[0]) z *= rs * op.col_scale[0][n];
                const int64_t o = m * op.ld_out + n;
                const float ex = extra ? __bfloat162float(extra[m * op.ld_extra + n]) : 0.0f;
                if (EPI == kEpiLinear) {
                    if (op.bias) z += op.bias[n];
                    out0[o] = __float2bfloat16_rn(act_f<act>(z) + ex);
                } else if (EPI == kEpiActGrad) {
                    if (op.bias) z += op.bias[n];
                    float a;
                    const float dz = ex * act_grad_f<act>(z, &a);
                    cols[j] += dz;
                    out0[o] = __float2bfloat16_rn(dz);
                } else {
                    float u = acc[kAcc - 1][i][j];
                    if (op.col_scale[1]) u *= rs * op.col_scale[1][n];
                    if (EPI == kEpiGated) {
                        out0[o] = __float2bfloat16_rn(act_f<act>(z) * u);
                    } else {
                        float a;
                        const float slope = act_grad_f<act>(z, &a);
                        out0[o] = __float2bfloat16_rn(ex * u * slope);
                        out1[o] = __float2bfloat16_rn(ex * a);
                    }
                }
            }
    });
    if (EPI == kEpiActGrad && part) {
#pragma unroll
        for (int j = 0; j < 4; ++j) sh_cols[ty][tx + 16 * j] = cols[j];
        __syncthreads();
        if (threadIdx.x < kT && n0 + threadIdx.x < op.n) {
            float t = 0.0f;
            for (int y = 0; y < 16; ++y) t += sh_cols[y][threadIdx.x];
            part[(blockIdx.x / n_tiles) * op.n + n0 + threadIdx.x] = t;
        }
    }
}

template <typename T>
int run_simt(const DenseOp& op, cudaStream_t s) {
    const int64_t tm = ceil_div(op.m, kT), tn = ceil_div(op.n, kT);
    if (tm * tn > 0x7FFFFFFF) return SPCONV_ERR_UNSUPPORTED;
    Scratch part(op.col_sums ? static_cast<size_t>(tm) * op.n * 4 : 0, s);
    if (part.failed()) return SPCONV_ERR_OOM;
    const dim3 grid(static_cast<unsigned>(tm * tn), static_cast<unsigned>(op.n_sources));
    const int32_t nt = static_cast<int32_t>(tn);
    count_launch();
    switch (op.epi) {
        case kEpiGated: k_dense_simt<T, kEpiGated><<<grid, 256, 0, s>>>(op, nt, nullptr); break;
        case kEpiActGrad: k_dense_simt<T, kEpiActGrad><<<grid, 256, 0, s>>>(op, nt, part.as<float>()); break;
        case kEpiGatedGrad: k_dense_simt<T, kEpiGatedGrad><<<grid, 256, 0, s>>>(op, nt, nullptr); break;
        default: k_dense_simt<T, kEpiLinear><<<grid, 256, 0, s>>>(op, nt, nullptr);
    }
    SPCONV_CHECK(launch_status());
    return op.col_sums ? sum_partials(part.as<float>(), tm, op.n, op.col_sums, s) : SPCONV_OK;
}

// ---- column sums ----------------------------------------------------------------
// 32 columns per block, 32 threads down each column, added through shared memory
// in a fixed order.
__global__ void __launch_bounds__(1024) k_sum_partials(const float* part, int64_t p, int64_t n, float* out) {
    __shared__ float sh[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + x;
    float s = 0.0f;
    if (col < n) {
#pragma unroll 8
        for (int64_t i = y; i < p; i += 32) s += part[i * n + col];
    }
    sh[y][x] = s;
    __syncthreads();
    float v = sh[x][y];   // thread (x, y) now holds part x of column y
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + y;
    if (x == 0 && c < n) out[c] = v;
}

// One row of partial sums per block of `rows` rows: 64 columns, 8 per thread
// (W = 8: one 16-byte load) or one (W = 1).
template <int W>
__global__ void __launch_bounds__(256) k_column_sums(const __nv_bfloat16* v, int64_t ld, int64_t m, int64_t n, int64_t rows,
                                                     float* part) {
    constexpr int kX = 64 / W, kY = 256 / kX;
    __shared__ float sh[kY][64 + 1];
    const int x = threadIdx.x % kX, y = threadIdx.x / kX;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + x * W;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows, r1 = r0 + rows < m ? r0 + rows : m;
    float s[W] = {};
    if (col < n) {
#pragma unroll 4
        for (int64_t r = r0 + y; r < r1; r += kY) {
            const __nv_bfloat16* p = v + r * ld + col;
            if (W == 8) {
                const uint4 q = *reinterpret_cast<const uint4*>(p);
                const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[(2 * j) % W] += __uint_as_float(u[j] << 16);
                    s[(2 * j + 1) % W] += __uint_as_float(u[j] & 0xFFFF0000u);
                }
            } else {
                s[0] += __bfloat162float(*p);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < W; ++j) sh[y][x * W + j] = s[j];
    __syncthreads();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    if (threadIdx.x < 64 && c < n) {
        float t = 0.0f;
        for (int i = 0; i < kY; ++i) t += sh[i][threadIdx.x];
        part[static_cast<int64_t>(blockIdx.y) * n + c] = t;
    }
}

// ---- 8-bit weights --------------------------------------------------------------
// |w| per output channel as its bits (non-negative floats order as integers, NaN on
// top); a maximum does not depend on the order of the atomics.
__global__ void __launch_bounds__(256) k_weight_amax(const __nv_bfloat16* w, int32_t c_in, int32_t c_out, uint32_t* amax) {
    const int32_t o = blockIdx.x * 64 + threadIdx.x % 64;
    uint32_t m = 0;
    if (o < c_out)
        for (int64_t c = blockIdx.y * 4 + threadIdx.x / 64; c < c_in; c += gridDim.y * 4) {
            const uint32_t b = __float_as_uint(fabsf(__bfloat162float(w[c * c_out + o])));
            m = b > m ? b : m;
        }
    if (m) atomicMax(amax + o, m);
}

// 64 x 64 tiles, transposed through shared memory.
__global__ void __launch_bounds__(256) k_quantize_weight(const __nv_bfloat16* w, int32_t c_in, int32_t c_out,
                                                         const uint32_t* amax, uint8_t* q, float* scale) {
    __shared__ float sh[64][65];
    const int32_t c0 = blockIdx.x * 64, o0 = blockIdx.y * 64;
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
        const int32_t c = c0 + i / 64, o = o0 + i % 64;
        sh[i / 64][i % 64] = c < c_in && o < c_out ? __bfloat162float(w[static_cast<int64_t>(c) * c_out + o]) : 0.0f;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
        const int32_t o = o0 + i / 64, c = c0 + i % 64;
        if (o >= c_out || c >= c_in) continue;
        const float m = __uint_as_float(amax[o]);
        // (448 / m overflows below 2^-119: bring such channels up first)
        const float pre = m < 0x1p-100f ? 0x1p100f : 1.0f;
        const float inv = m == 0.0f ? 0.0f : 448.0f / (m * pre);
        q[static_cast<int64_t>(o) * c_in + c] = __nv_cvt_float_to_fp8(sh[i % 64][i / 64] * pre * inv, __NV_SATFINITE, __NV_E4M3);
        if (c == 0) scale[o] = m / 448.0f;
    }
}

}  // namespace

int dense_run(const DenseOp& op, cudaStream_t s) {
    if (op.m == 0 || op.n == 0) return SPCONV_OK;
    return op.dtype == SPCONV_E4M3 ? run_simt<__nv_fp8_e4m3>(op, s) : run_simt<__nv_bfloat16>(op, s);
}

int sum_partials(const float* part, int64_t p, int64_t n, float* out, cudaStream_t s) {
    count_launch();
    k_sum_partials<<<static_cast<unsigned>(ceil_div(n, 32)), 1024, 0, s>>>(part, p, n, out);
    return launch_status();
}

int column_sums(const void* v, int64_t ld, int64_t m, int64_t n, float* out, cudaStream_t s) {
    const int64_t bx = ceil_div(n, 64);
    // about eight blocks per SM, each of 64 rows at least
    int64_t chunks = ceil_div(8 * 152, bx);
    if (chunks > ceil_div(m, 64)) chunks = ceil_div(m, 64);
    if (chunks < 1) chunks = 1;
    const int64_t rows = ceil_div(m, chunks);
    Scratch part(static_cast<size_t>(chunks) * n * 4, s);
    if (part.failed()) return SPCONV_ERR_OOM;
    const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>(chunks));
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(v);
    count_launch();
    if (n % 8 == 0 && ld % 8 == 0 && (reinterpret_cast<uintptr_t>(v) & 15) == 0)
        k_column_sums<8><<<grid, 256, 0, s>>>(p, ld, m, n, rows, part.as<float>());
    else
        k_column_sums<1><<<grid, 256, 0, s>>>(p, ld, m, n, rows, part.as<float>());
    SPCONV_CHECK(launch_status());
    return sum_partials(part.as<float>(), chunks, n, out, s);
}

int quantize_weight(const void* w, int32_t c_in, int32_t c_out, void* q, float* scale, cudaStream_t s) {
    Scratch amax(static_cast<size_t>(c_out) * 4, s);
    if (amax.failed()) return SPCONV_ERR_OOM;
    SPCONV_CHECK_CUDA(cudaMemsetAsync(amax.as<uint32_t>(), 0, static_cast<size_t>(c_out) * 4, s));
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(w);
    const unsigned bo = static_cast<unsigned>(ceil_div(c_out, 64)), bc = static_cast<unsigned>(ceil_div(c_in, 64));
    count_launch(2);
    k_weight_amax<<<dim3(bo, bc < 64 ? bc : 64), 256, 0, s>>>(p, c_in, c_out, amax.as<uint32_t>());
    k_quantize_weight<<<dim3(bc, bo), 256, 0, s>>>(p, c_in, c_out, amax.as<uint32_t>(), static_cast<uint8_t*>(q), scale);
    return launch_status();
}

}  // namespace spconv
