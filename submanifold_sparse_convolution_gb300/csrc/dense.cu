// Around the tensor-core products: rows brought into the alignment that the
// tensor maps need, the column sums of the bias gradients, and the 8-bit weight
// layout.
#include "ptx_sm100.cuh"
#include "rows.cuh"

namespace spconv {
namespace {

__device__ int32_t g_rows_status;   // kStatus* bits of the row-wise operators' bounded waits

// A warp's wait as the operators make it, on a barrier without copies or
// arrivals: it gives up after limit_ns and records that.
__global__ void __launch_bounds__(32) k_rows_wait_probe(int32_t* status, uint64_t limit_ns) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        ptx::mbar_init(&bar, 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&bar, 0, nullptr, limit_ns)) && threadIdx.x == 0) atomicOr(status, kStatusTimeout);
}

// ---- copies to aligned rows ---------------------------------------------------------
// A warp per 256 elements E of a row, neighbouring lanes on neighbouring
// elements: rows of any alignment move in whole 32-byte sectors.  Bound by HBM
// and the loads in flight: 120000 x 459 bf16 41.7 us, 5.3 TB/s.  All matrices of a
// call in one launch (gated, 1 x 930 x 62: 9.3 us, a launch each 11.1).
template <typename E>
__device__ __forceinline__ void copy_rows(const RowCopy& c, int32_t block) {
    const int64_t w = (static_cast<int64_t>(block) * 256 + threadIdx.x) >> 5;
    const int64_t r = w / c.row_warps;
    if (r >= c.rows) return;
    const int32_t c0 = static_cast<int32_t>(w - r * c.row_warps) * 256 + (threadIdx.x & 31);
    const E* src = reinterpret_cast<const E*>(static_cast<const uint8_t*>(c.src) + r * c.pitch_src);
    E* dst = reinterpret_cast<E*>(static_cast<uint8_t*>(c.dst) + r * c.pitch_dst);
    E v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (c0 + 32 * k < c.cols) v[k] = src[c0 + 32 * k];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (c0 + 32 * k < c.cols) dst[c0 + 32 * k] = v[k];
}

__global__ void __launch_bounds__(256) k_copy_rows(const RowCopies a) {
    pdl_wait();
    pdl_trigger();
    int32_t b = static_cast<int32_t>(blockIdx.x);
#pragma unroll
    for (int i = 0; i < kMaxCopies; ++i) {
        const RowCopy& c = a.copy[i];
        if (b < c.blocks) {
            if (c.e == 4) copy_rows<uint32_t>(c, b);
            else if (c.e == 2) copy_rows<uint16_t>(c, b);
            else copy_rows<uint8_t>(c, b);
            return;
        }
        b -= c.blocks;
    }
}

// ---- column sums ----------------------------------------------------------------
// The sums that are left after partial results, by block: slices of the first
// product, of the second, then columns.  A chain of latencies: the 19 slices of a
// 512 x 512 weight gradient with 512 column sums 8.7 us cold, about 4 after the
// products (the slices are in L2), most of it the launch.
struct FinishArgs {
    SliceSums slices[2];
    ColumnSums cols;
    int32_t blocks[2];   // of each product's slices
};

constexpr int kFinishCols = 8;   // columns of a block, 32 threads down each

// W (4 or 1) neighbouring sums of the slices, eight loads in flight, added in order.
template <int W>
__device__ __forceinline__ void add_slices(const float* q, int32_t splits, int64_t slice, float (&s)[W]) {
    struct alignas(4 * W) V {
        float v[W];
    };
#pragma unroll
    for (int j = 0; j < W; ++j) s[j] = 0.0f;
    for (int32_t k = 0; k < splits; k += 8) {
        V v[8];
#pragma unroll
        for (int32_t t = 0; t < 8; ++t)
            if (k + t < splits) v[t] = *reinterpret_cast<const V*>(q + (k + t) * slice);
#pragma unroll
        for (int32_t t = 0; t < 8; ++t)
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (k + t < splits) s[j] += v[t].v[j];
    }
}

// W elements of one row of one output (W = 4 where n % 4 == 0).
template <int W>
__device__ __forceinline__ void sum_slices(const SliceSums& a, int32_t block) {
    const int64_t mn = a.m * a.n, one = a.m * a.ld_part, slice = one * a.outputs;
    const bool gated = a.epi == kEpiGated;
    const int64_t i = (static_cast<int64_t>(block) * 256 + threadIdx.x) * W;
    if (i >= (gated ? mn : mn * a.outputs)) return;
    const int src = !gated && i >= mn;
    const int64_t r = i - (src ? mn : 0);
    const int64_t row = mn < 0x7FFFFFFF ? static_cast<uint32_t>(r) / static_cast<uint32_t>(a.n) : r / a.n, col = r - row * a.n;
    float z[W], u[W];
    const float* q = a.part + src * one + row * a.ld_part + col;
    add_slices<W>(q, a.splits, slice, z);
    if (gated) add_slices<W>(q + one, a.splits, slice, u);
    if (a.row_scale) {
        const float rs = a.row_scale[row];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            z[j] *= rs * a.col_scale[0][col + j];
            if (gated) u[j] *= rs * a.col_scale[1][col + j];
        }
    }
    if (a.bias) {
#pragma unroll
        for (int j = 0; j < W; ++j) z[j] += a.bias[col + j];
    }
    with_act(a.act, [&](auto act) {
#pragma unroll
        for (int j = 0; j < W; ++j) z[j] = act_f<act>(z[j]);
    });
    struct alignas(2 * W) V {
        __nv_bfloat16 v[W];
    } o;
    if (gated) {
#pragma unroll
        for (int j = 0; j < W; ++j) z[j] *= u[j];
    } else if (a.extra) {
        const V x = *reinterpret_cast<const V*>(a.extra + row * a.ld_extra + col);   // (tma_ok)
#pragma unroll
        for (int j = 0; j < W; ++j) z[j] += __bfloat162float(x.v[j]);
    }
#pragma unroll
    for (int j = 0; j < W; ++j) o.v[j] = __float2bfloat16_rn(z[j]);
    __nv_bfloat16* out = a.out[src] + row * a.ld + col;
    if (a.vec_out) {
        *reinterpret_cast<V*>(out) = o;
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) out[j] = o.v[j];
    }
}

// The gradients' epilogues after slices of K: 32 rows of 32 W columns a block, eight
// rows at a time, and one row of the column sums.  467 x 7832 x 912 with SiLU: the
// whole backward pass 40.9 us, with K in one piece 61.3; 2000 x 512 x 512 is not cut.
template <int W>
__global__ void __launch_bounds__(256) k_finish_grad(const SliceSums a) {
    struct alignas(2 * W) V {
        __nv_bfloat16 v[W];
    };
    __shared__ float sh[8][32 * W];
    pdl_wait();
    pdl_trigger();
    const bool gated = a.epi == kEpiGatedGrad;
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 * W + x * W, one = a.m * a.ld_part, slice = one * a.outputs;
    float s[W] = {};
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * 32 + y; col < a.n && row < a.m && row < (blockIdx.y + 1) * int64_t(32); row += 8) {
        float z[W], u[W] = {};
        const float* q = a.part + row * a.ld_part + col;
        add_slices<W>(q, a.splits, slice, z);
        if (gated) add_slices<W>(q + one, a.splits, slice, u);
        const V d = *reinterpret_cast<const V*>(a.extra + row * a.ld_extra + col);   // (tma_ok)
        V o0, o1;
        with_act(a.act, [&](auto act) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (a.bias) z[j] += a.bias[col + j];
                float v;
                const float dy = __bfloat162float(d.v[j]), slope = act_grad_f<act>(z[j], &v);
                const float dz = gated ? dy * u[j] * slope : dy * slope;
                s[j] += dz;
                o0.v[j] = __float2bfloat16_rn(dz);
                o1.v[j] = __float2bfloat16_rn(dy * v);
            }
        });
        *reinterpret_cast<V*>(a.out[0] + row * a.ld + col) = o0;
        if (gated) *reinterpret_cast<V*>(a.out[1] + row * a.ld + col) = o1;
    }
    if (!a.col_part) return;
#pragma unroll
    for (int j = 0; j < W; ++j) sh[y][x * W + j] = s[j];
    __syncthreads();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 * W + threadIdx.x;
    if (threadIdx.x < 32 * W && c < a.n) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += sh[i][threadIdx.x];
        a.col_part[blockIdx.y * a.n + c] = t;
    }
}

__global__ void __launch_bounds__(256) k_finish(const FinishArgs a) {
    __shared__ float sh[32][kFinishCols + 1];
    pdl_wait();
    pdl_trigger();
    int32_t b = static_cast<int32_t>(blockIdx.x);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        if (b < a.blocks[g]) {
            if (a.slices[g].n % 4 == 0) sum_slices<4>(a.slices[g], b);
            else sum_slices<1>(a.slices[g], b);
            return;
        }
        b -= a.blocks[g];
    }
    const int x = threadIdx.x % kFinishCols, y = threadIdx.x / kFinishCols;
    const int64_t col = static_cast<int64_t>(b) * kFinishCols + x;
    float s = 0.0f;
    if (col < a.cols.n) {
        // eight loads in flight, added in order
        for (int64_t i = y; i < a.cols.rows; i += 8 * 32) {
            float v[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) v[t] = i + 32 * t < a.cols.rows ? a.cols.part[(i + 32 * t) * a.cols.n + col] : 0.0f;
#pragma unroll
            for (int t = 0; t < 8; ++t) s += v[t];
        }
    }
    sh[y][x] = s;
    __syncthreads();
    // a warp per column adds its 32 parts
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float v = sh[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int64_t c = static_cast<int64_t>(b) * kFinishCols + warp;
    if (lane == 0 && c < a.cols.n) a.cols.out[c] = v;
}

// One row of partial sums per block of `rows` rows: 64 columns, 8 per thread
// (W = 8: one 16-byte load) or one (W = 1).  240000 x 512 46.3 us, 5.3 TB/s.
template <int W>
__global__ void __launch_bounds__(256) k_column_parts(const __nv_bfloat16* v, int64_t ld, int64_t m, int64_t n, int64_t rows,
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
// Once per weight, so kept simple: two passes, 4096 x 8192 72 us together.
// |w| per output channel as its bits (non-negative floats order as integers, NaN on
// top); a maximum does not depend on the order of the atomics.
__global__ void __launch_bounds__(256) k_weight_amax(const __nv_bfloat16* w, int32_t c_in, int32_t c_out, uint32_t* amax) {
    const int32_t o = blockIdx.x * 64 + threadIdx.x % 64;
    uint32_t m = 0;
    if (o < c_out)
#pragma unroll 8
        for (int64_t c = blockIdx.y * 4 + threadIdx.x / 64; c < c_in; c += gridDim.y * 4) {
            const uint32_t b = __float_as_uint(fabsf(__bfloat162float(w[c * c_out + o])));
            m = b > m ? b : m;
        }
    if (m) atomicMax(amax + o, m);
}

// 64 x 64 tiles, transposed through shared memory; four values a store where the
// rows of q are whole words.
__global__ void __launch_bounds__(256) k_quantize_weight(const __nv_bfloat16* w, int32_t c_in, int32_t c_out,
                                                         const uint32_t* amax, uint8_t* q, float* scale, bool words) {
    __shared__ float sh[64][65];
    __shared__ float first[64], then[64];   // factors of a channel
    const int32_t c0 = blockIdx.x * 64, o0 = blockIdx.y * 64;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int i = k * 256 + threadIdx.x;
        const int32_t c = c0 + i / 64, o = o0 + i % 64;
        sh[i / 64][i % 64] = c < c_in && o < c_out ? __bfloat162float(w[static_cast<int64_t>(c) * c_out + o]) : 0.0f;
    }
    const int32_t ch = o0 + static_cast<int32_t>(threadIdx.x);
    if (threadIdx.x < 64 && ch < c_out) {
        const float m = __uint_as_float(amax[ch]);
        // (448 / m overflows below 2^-119: bring such channels up first)
        const float pre = m < 0x1p-100f ? 0x1p100f : 1.0f;
        first[threadIdx.x] = pre;
        then[threadIdx.x] = m == 0.0f ? 0.0f : 448.0f / (m * pre);
        if (c0 == 0) scale[ch] = m / 448.0f;
    }
    __syncthreads();
    const int c4 = threadIdx.x % 16 * 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int j = k * 16 + threadIdx.x / 16;
        const int32_t o = o0 + j, c = c0 + c4;
        if (o >= c_out || c >= c_in) continue;
        uint32_t v = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            v |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(sh[c4 + t][j] * first[j] * then[j], __NV_SATFINITE, __NV_E4M3)) << (8 * t);
        uint8_t* out = q + static_cast<int64_t>(o) * c_in + c;
        if (words) {
            *reinterpret_cast<uint32_t*>(out) = v;
        } else {
            for (int t = 0; t < 4 && c + t < c_in; ++t) out[t] = static_cast<uint8_t>(v >> (8 * t));
        }
    }
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

int rows_wait_probe(uint64_t limit_ns, cudaStream_t s) {
    int32_t* status = nullptr;
    SPCONV_CHECK(rows_status_word(&status));
    count_launch();
    k_rows_wait_probe<<<1, 32, 0, s>>>(status, limit_ns);
    return launch_status();
}

void AlignedRows::add(const void** p, int count, int64_t* ld, int64_t rows, int64_t cols, size_t es) {
    bool move = false;
    for (int i = 0; i < count; ++i) move = move || !tma_ok(p[i], *ld, es);
    if (!move) return;
    const int64_t pitch = static_cast<int64_t>(round_up(static_cast<size_t>(cols), 16 / es));
    for (int i = 0; i < count; ++i) {
        // the largest elements that the rows allow
        const uintptr_t all = reinterpret_cast<uintptr_t>(p[i]) | static_cast<uintptr_t>(*ld * es) | static_cast<uintptr_t>(cols * es);
        RowCopy& c = args_.copy[count_];
        c.e = all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
        c.src = p[i];
        c.pitch_src = *ld * static_cast<int64_t>(es);
        c.pitch_dst = pitch * static_cast<int64_t>(es);
        c.rows = rows;
        c.cols = static_cast<int32_t>(cols * static_cast<int64_t>(es) / c.e);
        c.row_warps = static_cast<int32_t>(ceil_div(c.cols, 256));
        const int64_t b = ceil_div(rows * c.row_warps, 8);
        blocks_ += b;
        c.blocks = static_cast<int32_t>(b);
        off_[count_] = bytes_;
        bytes_ += round_up(static_cast<size_t>(rows) * c.pitch_dst, 256);
        out_[count_++] = &p[i];
    }
    *ld = pitch;
}

int AlignedRows::run(cudaStream_t s) {
    if (count_ == 0) return SPCONV_OK;
    if (blocks_ > 0x7FFFFFFF) return SPCONV_ERR_UNSUPPORTED;
    if (!buf_.alloc(bytes_, s)) return SPCONV_ERR_OOM;
    for (int i = 0; i < count_; ++i) *out_[i] = args_.copy[i].dst = buf_.as<void>(off_[i]);
    return launch_pdl(k_copy_rows, dim3(static_cast<unsigned>(blocks_)), 256, 0, s, args_);
}

namespace {

// Brings the operands of a product, and what its epilogue reads, into alignment.
int align(DenseOp* op, AlignedRows* rows, cudaStream_t s) {
    const size_t es = op->dtype == SPCONV_E4M3 ? 1 : 2;
    const bool dual = op->epi == kEpiGated || op->epi == kEpiGatedGrad;
    const int nb = dual || op->k_sources == 2 || op->n_sources == 2 ? 2 : 1;
    auto add = [&](Operand& t, int count, int64_t r) {
        rows->add(t.p, count, &t.ld, t.k_major ? r : op->k, t.k_major ? op->k : r, es);
    };
    add(op->a, op->k_sources, op->m);
    add(op->b, nb, op->n);
    if (op->extra) rows->add(&op->extra, 1, &op->ld_extra, op->m, op->n, 2);
    return rows->run(s);
}

}  // namespace

int dense_run(const DenseOp& op, cudaStream_t s) {
    if (op.m == 0 || op.n == 0) return SPCONV_OK;
    int32_t* status = nullptr;
    SPCONV_CHECK(rows_status_word(&status));
    AlignedRows rows;
    DenseOp o = op;
    SPCONV_CHECK(align(&o, &rows, s));
    if (dense_few_takes(o)) return dense_few_run(o, status, s);
    return dense_tc_cuts(o) ? dense_tc_plain(&o, 1, {}, status, s) : dense_tc_run(o, status, s);
}

int dense_run_plain(const DenseOp* ops, int count, const ColumnSums& cols, cudaStream_t s) {
    if (count == 0) return cols.out ? finish_sums(nullptr, 0, cols, s) : SPCONV_OK;
    int32_t* status = nullptr;
    SPCONV_CHECK(rows_status_word(&status));
    AlignedRows rows[2];
    DenseOp o[2];
    for (int i = 0; i < count; ++i) {
        o[i] = ops[i];
        SPCONV_CHECK(align(&o[i], &rows[i], s));
    }
    return dense_tc_plain(o, count, cols, status, s);
}

int finish_grad(const SliceSums& a, cudaStream_t s) {
    const bool quads = a.n % 4 == 0;   // (the outputs are aligned workspace)
    const int64_t rows = a.col_part ? col_part_rows(a.m) : ceil_div(a.m, 32);
    if (rows > 65535) return SPCONV_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(ceil_div(a.n, quads ? 128 : 32)), static_cast<unsigned>(rows));
    return launch_pdl(quads ? k_finish_grad<4> : k_finish_grad<1>, grid, 256, 0, s, a);
}

int finish_sums(const SliceSums* slices, int count, const ColumnSums& cols, cudaStream_t s) {
    FinishArgs a = {};
    int64_t blocks = 0;
    for (int i = 0; i < count; ++i) {
        a.slices[i] = slices[i];
        const SliceSums& t = slices[i];
        a.slices[i].vec_out = t.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(t.out[0]) | reinterpret_cast<uintptr_t>(t.out[1])) % 8 == 0;
        const int64_t elems = t.m * t.n * (t.epi == kEpiGated ? 1 : t.outputs);
        const int64_t b = t.splits ? ceil_div(elems, t.n % 4 == 0 ? 1024 : 256) : 0;
        if (b > 0x3FFFFFFF) return SPCONV_ERR_UNSUPPORTED;
        a.blocks[i] = static_cast<int32_t>(b);
        blocks += b;
    }
    if (cols.out) {
        a.cols = cols;
        blocks += ceil_div(cols.n, kFinishCols);
    }
    if (blocks == 0) return SPCONV_OK;
    return launch_pdl(k_finish, dim3(static_cast<unsigned>(blocks)), 256, 0, s, a);
}

namespace {
// about eight blocks per SM, each of 64 rows at least
int64_t column_chunk(int64_t m, int64_t n) {
    int64_t chunks = ceil_div(8 * 152, ceil_div(n, 64));
    if (chunks > ceil_div(m, 64)) chunks = ceil_div(m, 64);
    return ceil_div(m, chunks < 1 ? 1 : chunks);
}
}  // namespace

int64_t column_part_rows(int64_t m, int64_t n) { return ceil_div(m, column_chunk(m, n)); }

int column_parts(const void* v, int64_t ld, int64_t m, int64_t n, float* part, cudaStream_t s) {
    const int64_t rows = column_chunk(m, n);
    const dim3 grid(static_cast<unsigned>(ceil_div(n, 64)), static_cast<unsigned>(ceil_div(m, rows)));
    const bool vec = n % 8 == 0 && ld % 8 == 0 && (reinterpret_cast<uintptr_t>(v) & 15) == 0;
    return launch_pdl(vec ? k_column_parts<8> : k_column_parts<1>, grid, 256, 0, s, static_cast<const __nv_bfloat16*>(v), ld, m, n,
                      rows, part);
}

int quantize_weight(const void* w, int32_t c_in, int32_t c_out, void* q, float* scale, cudaStream_t s) {
    Scratch amax(static_cast<size_t>(c_out) * 4, s);
    if (amax.failed()) return SPCONV_ERR_OOM;
    SPCONV_CHECK_CUDA(cudaMemsetAsync(amax.as<uint32_t>(), 0, static_cast<size_t>(c_out) * 4, s));
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(w);
    const unsigned bo = static_cast<unsigned>(ceil_div(c_out, 64)), bc = static_cast<unsigned>(ceil_div(c_in, 64));
    count_launch(2);
    k_weight_amax<<<dim3(bo, bc < 64 ? bc : 64), 256, 0, s>>>(p, c_in, c_out, amax.as<uint32_t>());
    k_quantize_weight<<<dim3(bc, bo), 256, 0, s>>>(p, c_in, c_out, amax.as<uint32_t>(), static_cast<uint8_t*>(q), scale,
                                                  c_in % 4 == 0 && reinterpret_cast<uintptr_t>(q) % 4 == 0);
    return launch_status();
}

}  // namespace spconv
