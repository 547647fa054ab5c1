// Around the tensor-core products: rows brought into the alignment that the
// tensor maps need, the column sums of the bias gradients, and the 8-bit weight
// layout.
#include "rows.cuh"

namespace spconv {
namespace {

__device__ int32_t g_rows_status;   // kStatus* bits of the row-wise operators' bounded waits

// ---- copies between aligned and unaligned rows ------------------------------------
// Eight elements per thread; the side whose rows are 16-byte aligned moves as one
// vector.
template <typename T>
__global__ void __launch_bounds__(256) k_copy_rows(const T* src, int64_t ld_src, T* dst, int64_t ld_dst, int64_t rows,
                                                   int64_t cols, int64_t row_groups, bool vec_src, bool vec_dst) {
    pdl_wait();
    pdl_trigger();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t r = i / row_groups, c = (i - r * row_groups) * 8;
    if (r >= rows) return;
    struct alignas(8 * sizeof(T)) V {
        T v[8];
    } t;
    const T* s = src + r * ld_src + c;
    T* d = dst + r * ld_dst + c;
    const bool whole = c + 8 <= cols;
    if (vec_src && whole) {
        t = *reinterpret_cast<const V*>(s);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) t.v[j] = c + j < cols ? s[j] : T(0);
    }
    if (vec_dst && whole) {
        *reinterpret_cast<V*>(d) = t;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < cols) d[j] = t.v[j];
    }
}

// ---- column sums ----------------------------------------------------------------
// 32 columns per block, 32 threads down each column, added through shared memory
// in a fixed order.
__global__ void __launch_bounds__(1024) k_sum_partials(const float* part, int64_t p, int64_t n, float* out) {
    __shared__ float sh[32][33];
    pdl_wait();
    pdl_trigger();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + x;
    float s = 0.0f;
    if (col < n) {
#pragma unroll 16
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
    pdl_wait();
    pdl_trigger();
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

int copy_rows(const void* src, int64_t ld_src, void* dst, int64_t ld_dst, int64_t rows, int64_t cols, size_t es, cudaStream_t s) {
    const int64_t groups = ceil_div(cols, 8), blocks = ceil_div(rows * groups, 256);
    if (blocks > 0x7FFFFFFF) return SPCONV_ERR_UNSUPPORTED;
    auto vec = [&](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % (8 * es) == 0 && ld % 8 == 0; };
    const bool vs = vec(src, ld_src), vd = vec(dst, ld_dst);
    const dim3 grid(static_cast<unsigned>(blocks));
    if (es == 1)
        return launch_pdl(k_copy_rows<uint8_t>, grid, 256, 0, s, static_cast<const uint8_t*>(src), ld_src,
                          static_cast<uint8_t*>(dst), ld_dst, rows, cols, groups, vs, vd);
    return launch_pdl(k_copy_rows<uint16_t>, grid, 256, 0, s, static_cast<const uint16_t*>(src), ld_src,
                      static_cast<uint16_t*>(dst), ld_dst, rows, cols, groups, vs, vd);
}

}  // namespace

int rows_status_word(int32_t** word) {
    static int32_t* words[kMaxDevices] = {};
    int dev = 0;
    SPCONV_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return SPCONV_ERR_UNSUPPORTED;
    if (!words[dev]) {
        void* p = nullptr;
        SPCONV_CHECK_CUDA(cudaGetSymbolAddress(&p, g_rows_status));
        words[dev] = static_cast<int32_t*>(p);
    }
    *word = words[dev];
    return SPCONV_OK;
}

int dense_run(const DenseOp& op, cudaStream_t s) {
    if (op.m == 0 || op.n == 0) return SPCONV_OK;
    int32_t* status = nullptr;
    SPCONV_CHECK(rows_status_word(&status));
    // The tensor maps need 16-byte aligned rows.  Matrices without them (odd
    // channel counts, strides or addresses) are copied to rows that have them,
    // and such an output is copied back: one extra pass over that matrix.
    const size_t es = op.dtype == SPCONV_E4M3 ? 1 : 2;
    const bool dual = op.epi == kEpiGated || op.epi == kEpiGatedGrad;
    const int na = op.k_sources, nb = dual || op.k_sources == 2 || op.n_sources == 2 ? 2 : 1;
    const int nc = op.epi == kEpiGatedGrad || op.n_sources == 2 ? 2 : 1;
    struct Matrix {   // up to two matrices of one shape
        int64_t rows, cols;
        size_t es;
        bool move;
        size_t off[2];
        int64_t ld() const { return static_cast<int64_t>(round_up(static_cast<size_t>(cols), 16 / es)); }
    };
    size_t bytes = 0;
    auto plan = [&](const void* const* ptr, int count, int64_t ld, int64_t rows, int64_t cols, size_t e) {
        Matrix t{rows, cols, e, false, {0, 0}};
        for (int i = 0; i < count; ++i) t.move = t.move || !tma_ok(ptr[i], ld, e);
        for (int i = 0; t.move && i < count; ++i) {
            t.off[i] = bytes;
            bytes += round_up(static_cast<size_t>(rows) * t.ld() * e, 256);
        }
        return t;
    };
    const Matrix ma = op.a.k_major ? plan(op.a.p, na, op.a.ld, op.m, op.k, es) : plan(op.a.p, na, op.a.ld, op.k, op.m, es);
    const Matrix mb = op.b.k_major ? plan(op.b.p, nb, op.b.ld, op.n, op.k, es) : plan(op.b.p, nb, op.b.ld, op.k, op.n, es);
    const Matrix mx = plan(&op.extra, op.extra ? 1 : 0, op.ld_extra, op.m, op.n, 2);
    const Matrix mc = plan(op.out, nc, op.ld_out, op.m, op.n, 2);
    auto run = [&](const DenseOp& o) { return dense_few_takes(o) ? dense_few_run(o, status, s) : dense_tc_run(o, status, s); };
    if (bytes == 0) return run(op);
    Scratch buf(bytes, s);
    if (buf.failed()) return SPCONV_ERR_OOM;
    DenseOp o = op;
    auto bring = [&](const Matrix& t, const void** ptr, int count, int64_t* ld) -> int {
        if (!t.move) return SPCONV_OK;
        for (int i = 0; i < count; ++i) {
            SPCONV_CHECK(copy_rows(ptr[i], *ld, buf.as<void>(t.off[i]), t.ld(), t.rows, t.cols, t.es, s));
            ptr[i] = buf.as<void>(t.off[i]);
        }
        *ld = t.ld();
        return SPCONV_OK;
    };
    SPCONV_CHECK(bring(ma, o.a.p, na, &o.a.ld));
    SPCONV_CHECK(bring(mb, o.b.p, nb, &o.b.ld));
    SPCONV_CHECK(bring(mx, &o.extra, 1, &o.ld_extra));
    if (mc.move) {
        for (int i = 0; i < nc; ++i) o.out[i] = buf.as<void>(mc.off[i]);
        o.ld_out = mc.ld();
    }
    SPCONV_CHECK(run(o));
    for (int i = 0; mc.move && i < nc; ++i)
        SPCONV_CHECK(copy_rows(o.out[i], o.ld_out, op.out[i], op.ld_out, op.m, op.n, 2, s));
    return SPCONV_OK;
}

int sum_partials(const float* part, int64_t p, int64_t n, float* out, cudaStream_t s) {
    return launch_pdl(k_sum_partials, dim3(static_cast<unsigned>(ceil_div(n, 32))), 1024, 0, s, part, p, n, out);
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
    const bool vec = n % 8 == 0 && ld % 8 == 0 && (reinterpret_cast<uintptr_t>(v) & 15) == 0;
    SPCONV_CHECK(launch_pdl(vec ? k_column_sums<8> : k_column_sums<1>, grid, 256, 0, s, p, ld, m, n, rows, part.as<float>()));
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
