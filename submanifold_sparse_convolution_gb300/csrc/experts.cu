// Rows sorted by expert and back, and rows and weights in e4m3 with a scale for
// each block of 128.
//
// A pair is a row's j-th choice, numbered token k + j.  Pairs are sorted stably
// by expert (a counting sort), so an expert's rows keep the tokens' order:
//
//   rows[slot(t, j)] = x[t]                       its gradient: dx[t] = sum_j drows[slot(t, j)]
//   out[t] = residual[t] + sum_j w[t, j] y[slot(t, j)]
//   dy[slot(t, j)] = w[t, j] dout[t];  dw[t, j] = dout[t] . y[slot(t, j)]
//
// All of them walk the tokens, so that a token's row is read once for all its
// choices and no sum needs an atomic.  They are bound by HBM: a thread holds one
// vector of a row, and the warps of an SM have enough of them in flight (bf16, four
// choices: 16381 tokens of 1024 channels, gather 24.5 us, 6.8 TB/s, combine 27.5;
// 8189 of 2048, the gradient of combine 47 us, 6.4 TB/s; 40000 rows of 2048 to e4m3
// blocks 85 us, 2.9 TB/s: there the arithmetic of a value is the bound).  The sort is
// two kernels of 3 and 6 us for 32756 pairs, most of it latency.
#include "row_vectors.cuh"

namespace spconv {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxChunks = 128;

// ---- the sort -----------------------------------------------------------------
struct SortArgs {
    const void* experts;   // [pairs] int32 or int64
    int64_t pairs;
    int32_t n_experts;
    int32_t tiles;         // of kSortThreads pairs, of a chunk
    int32_t* counts;       // [chunks][n_experts]
    int32_t* offsets;      // [n_experts + 1]
    int32_t* sorted;       // [pairs] the pair of each slot
    int32_t* slots;        // [pairs]
    int32_t* status;
};

// The expert of a pair; -1: none.
template <typename I>
__device__ __forceinline__ int32_t expert_of(const SortArgs& a, int64_t pair) {
    if (pair >= a.pairs) return -1;
    const I e = static_cast<const I*>(a.experts)[pair];
    return e >= 0 && e < a.n_experts ? static_cast<int32_t>(e) : -1;
}

// How often a chunk's pairs name each expert (whole numbers: the atomics' order
// does not matter).
template <typename I>
__global__ void __launch_bounds__(kSortThreads) k_expert_count(const SortArgs a) {
    __shared__ int32_t count[kSortThreads];
    count[threadIdx.x] = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    for (int32_t i = 0; i < a.tiles; ++i) {
        const int32_t e = expert_of<I>(a, (static_cast<int64_t>(blockIdx.x) * a.tiles + i) * kSortThreads + threadIdx.x);
        if (e >= 0) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    if (static_cast<int32_t>(threadIdx.x) < a.n_experts)
        a.counts[static_cast<int64_t>(blockIdx.x) * a.n_experts + threadIdx.x] = count[threadIdx.x];
}

// Exclusive sums of one value per thread over the block.
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t* sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) sh[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int32_t w = sh[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w += u;
        }
        sh[lane] = w;
    }
    __syncthreads();
    const int32_t before = warp ? sh[warp - 1] : 0;
    __syncthreads();
    return before + inc - v;
}

// Each pair's slot: the experts before its own, the chunks before this one, the
// tiles and warps before its own, the lanes before it.  With one chunk nothing
// was counted before: the block counts for itself.
template <typename I>
__global__ void __launch_bounds__(kSortThreads) k_expert_place(const SortArgs a) {
    extern __shared__ __align__(16) uint16_t in_warp[];   // [kSortWarps][n_experts] (cleared by 32 bits)
    __shared__ int32_t next[kSortThreads], part[2][kSortThreads], sh[32];
    const int32_t tid = static_cast<int32_t>(threadIdx.x), lane = tid & 31, warp = tid >> 5, ne = a.n_experts;
    const int32_t chunks = static_cast<int32_t>(gridDim.x), b = static_cast<int32_t>(blockIdx.x);
    pdl_wait();
    pdl_trigger();
    int32_t before = 0, all = 0;
    if (chunks > 1) {
        // several threads an expert, each every so many chunks
        const int32_t deep = kSortThreads / ne, e = tid % ne;
        if (tid < deep * ne) {
#pragma unroll 8
            for (int32_t c = tid / ne; c < chunks; c += deep) {
                const int32_t v = __ldcg(a.counts + static_cast<int64_t>(c) * ne + e);
                all += v;
                before += c < b ? v : 0;
            }
        }
        part[0][tid] = before;
        part[1][tid] = all;
        __syncthreads();
        before = all = 0;
        if (tid < ne)
            for (int32_t d = 0; d < deep; ++d) {
                before += part[0][d * ne + tid];
                all += part[1][d * ne + tid];
            }
    } else {
        part[0][tid] = 0;
        __syncthreads();
        for (int32_t i = 0; i < a.tiles; ++i) {
            const int32_t e = expert_of<I>(a, static_cast<int64_t>(i) * kSortThreads + tid);
            if (e >= 0) atomicAdd(&part[0][e], 1);
        }
        __syncthreads();
        if (tid < ne) all = part[0][tid];
    }
    const int32_t first = block_scan(all, sh);
    next[tid] = first + before;
    if (tid == kSortThreads - 1) part[1][0] = first + all;
    if (b == 0 && tid < ne) a.offsets[tid + 1] = first + all;
    if (b == 0 && tid == 0) a.offsets[0] = 0;
    __syncthreads();
    const int64_t live = part[1][0];
    for (int64_t i = live + static_cast<int64_t>(b) * kSortThreads + tid; i < a.pairs; i += static_cast<int64_t>(chunks) * kSortThreads)
        a.sorted[i] = -1;
    for (int32_t i = 0; i < a.tiles; ++i) {
        const int64_t pair = (static_cast<int64_t>(b) * a.tiles + i) * kSortThreads + tid;
        if (pair - tid >= a.pairs) break;
        for (int32_t j = tid; j < kSortWarps * ne / 2; j += kSortThreads) reinterpret_cast<uint32_t*>(in_warp)[j] = 0;
        __syncthreads();
        const int32_t e = expert_of<I>(a, pair);
        if (e < 0 && pair < a.pairs && static_cast<const I*>(a.experts)[pair] >= ne) atomicOr(a.status, kStatusRange);
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e), lower = same & ((1u << lane) - 1);
        if (e >= 0 && lower == 0) in_warp[warp * ne + e] = static_cast<uint16_t>(__popc(same));
        __syncthreads();
        if (tid < ne) {
            int32_t at = 0;
#pragma unroll 8
            for (int32_t w = 0; w < kSortWarps; ++w) {
                const int32_t v = in_warp[w * ne + tid];
                in_warp[w * ne + tid] = static_cast<uint16_t>(at);
                at += v;
            }
            part[0][tid] = at;
        }
        __syncthreads();
        if (pair < a.pairs) {
            const int32_t slot = e < 0 ? -1 : next[e] + in_warp[warp * ne + e] + __popc(lower);
            a.slots[pair] = slot;
            if (slot >= 0) a.sorted[slot] = static_cast<int32_t>(pair);
        }
        __syncthreads();
        if (tid < ne) next[tid] += part[0][tid];
        __syncthreads();
    }
}

// Which row and which of its vectors a flat index is: by a product where the index
// has 31 bits (a division of 64 bits takes longer than the rest).
struct RowVector {
    FastDiv by;
    int32_t vectors, small;
    RowVector(int64_t threads, int64_t vectors_)
        : by(static_cast<uint32_t>(vectors_)), vectors(static_cast<int32_t>(vectors_)), small(threads + 256 < 0x7FFFFFFF) {}
    __device__ __forceinline__ int64_t row(int64_t i) const { return small ? by(static_cast<int32_t>(i)) : i / vectors; }
};

// ---- rows to their slots ----------------------------------------------------------
// Rows at and behind offsets[n_experts] have no pair: the blocks' threads write
// zeros there.
template <typename V>
__device__ __forceinline__ void zero_tail(V* out, int64_t row_vectors, const int32_t* offsets, int32_t n_experts, int64_t rows) {
    int64_t live = __ldg(offsets + n_experts);
    live = live < 0 ? 0 : live;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const V zero = {};
    for (int64_t i = live * row_vectors + static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < rows * row_vectors; i += step)
        out[i] = zero;
}

__device__ __forceinline__ bool in_range(int64_t slot, int64_t rows) {
    return static_cast<uint64_t>(slot) < static_cast<uint64_t>(rows);   // (whatever a caller's plan holds)
}

template <typename T, int W>
__global__ void __launch_bounds__(256) k_expert_gather(const ExpertRows a, const RowVector at) {
    using P = Pack<T, W>;
    pdl_wait();
    pdl_trigger();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int32_t vectors = a.c / W;
    const int64_t rows = a.tokens * a.k;
    P* out = static_cast<P*>(a.out);
    if (i < a.tokens * vectors) {
        const int64_t t = at.row(i);
        const int32_t v = static_cast<int32_t>(i - t * vectors);
        const P x = *reinterpret_cast<const P*>(static_cast<const T*>(a.x) + t * a.ldx + v * W);
        for (int32_t j = 0; j < a.k; ++j) {
            const int32_t slot = __ldg(a.slots + t * a.k + j);
            if (in_range(slot, rows)) out[static_cast<int64_t>(slot) * vectors + v] = x;
        }
    }
    zero_tail(out, vectors, a.offsets, a.n_experts, rows);
}

// A block of 128 values is half a warp's: eight values a lane.  scale = max |x| /
// 448, q = e4m3(x / scale), both divisions rounded to nearest: bf16 values often
// lie halfway between two e4m3 ones, where the scale's last bit decides.  The product
// with the inverse, which is within 2.5 units in the last place of the quotient, is
// taken first, and the division only where that is within 4 of halfway between two
// e4m3 values (three mantissa bits: the other twenty are near 0x80000) or below 2^-6,
// where those lie elsewhere.  (us, and with a division for every value: 5000 x 1001,
// read one value at a time, 8.7 and 14.0; 32371 x 128 5.9 and 5.4, 40000 x 2048 84.8
// and 78.8: for whole vectors the test costs more than it saves.)
//
// Without slots a row keeps its place (spconv_quantize_blocks).
template <typename T, int W, int ROWS>
__global__ void __launch_bounds__(256) k_rows_to_blocks(const ExpertRows a, const RowVector at) {
    using P = Pack<T, W>;
    pdl_wait();
    pdl_trigger();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int32_t blocks = (a.c + 127) / 128;
    const int64_t t0 = at.row(i), rows = a.tokens * a.k, apart = (a.tokens + ROWS - 1) / ROWS;
    const int32_t v = static_cast<int32_t>(i - t0 * (blocks * 16)), e = v * 8;
    uint8_t* out = static_cast<uint8_t*>(a.out);
    // the vectors of ROWS rows are on their way together
    P x[ROWS][8 / W];
    bool live[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t t = t0 + r * apart;
        live[r] = t0 < apart && t < a.tokens && e < a.c;
#pragma unroll
        for (int j = 0; j < 8; j += W)
            if (live[r] && e + j < a.c) x[r][j / W] = *reinterpret_cast<const P*>(static_cast<const T*>(a.x) + t * a.ldx + e + j);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t t = t0 + r * apart;
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; j += W) {
            float g[W] = {};
            if (live[r] && e + j < a.c) unpack<W>(x[r][j / W], g);
#pragma unroll
            for (int u = 0; u < W; ++u) f[j + u] = g[u];
        }
        uint32_t most = 0;   // the bits of |x| order as whole numbers, NaN on top
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __float_as_uint(fabsf(f[j]));
            most = b > most ? b : most;
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            const uint32_t u = __shfl_xor_sync(0xFFFFFFFFu, most, o);
            most = u > most ? u : most;
        }
        const float scale = __fdiv_rn(__uint_as_float(most), 448.0f);
        if (!live[r]) continue;
        const bool tiny = scale < 0x1p-100f;   // (its inverse may be infinite)
        const float inverse = tiny ? 0.0f : __fdiv_rn(1.0f, scale);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q = f[j] * inverse;
            const uint32_t b = __float_as_uint(fabsf(q));
            const bool near = ((b & 0xFFFFFu) - 0x7FFFCu) <= 8u || (b != 0 && b < 0x3C800000u);
            if (tiny || near) f[j] = scale == 0.0f ? 0.0f : __fdiv_rn(f[j], scale);
            else f[j] = q;
        }
        const uint32_t q[2] = {pack_e4m3(f), pack_e4m3(f + 4)};
        float* to_scale = v % 16 == 0 ? a.scale + static_cast<int64_t>(v / 16) * rows : nullptr;
        const int32_t* slots = a.slots + t * a.k;
        for (int32_t j = 0; j < a.k; ++j) {
            const int64_t slot = a.slots ? __ldg(slots + j) : t;
            if (!in_range(slot, rows)) continue;
            uint8_t* to = out + slot * a.c + e;
            if (a.wide) {
                *reinterpret_cast<uint2*>(to) = make_uint2(q[0], q[1]);
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (e + u < a.c) to[u] = static_cast<uint8_t>(q[u / 4] >> (8 * (u % 4)));
            }
            if (to_scale) to_scale[slot] = scale;
        }
    }
    if (a.slots) {
        zero_tail(out, a.c, a.offsets, a.n_experts, rows);
        int64_t last = __ldg(a.offsets + a.n_experts);
        last = last < 0 ? 0 : last;
        const int64_t left = rows - last, step = static_cast<int64_t>(gridDim.x) * 256;
        for (int64_t z = i; z < left * blocks; z += step) a.scale[(z / left) * rows + last + z % left] = 0.0f;
    }
}

// ---- slots to their rows ----------------------------------------------------------
// Up to four choices' rows are in flight at once.
template <typename T, int W>
__global__ void __launch_bounds__(256) k_expert_combine(const ExpertSums a, const RowVector at) {
    using P = Pack<T, W>;
    pdl_wait();
    pdl_trigger();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int32_t vectors = a.c / W;
    if (i >= a.tokens * vectors) return;
    const int64_t t = at.row(i), rows = a.tokens * a.k;
    const int32_t v = static_cast<int32_t>(i - t * vectors);
    float sum[W] = {};
    if (a.residual) unpack<W>(*reinterpret_cast<const P*>(static_cast<const T*>(a.residual) + t * a.ldr + v * W), sum);
    constexpr int U = 4;
    for (int32_t j0 = 0; j0 < a.k; j0 += U) {
        P y[U];
        float w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int32_t slot = -1;
            w[u] = 0.0f;
            if (j0 + u < a.k) slot = __ldg(a.slots + t * a.k + j0 + u);
            if (in_range(slot, rows)) {
                y[u] = *reinterpret_cast<const P*>(static_cast<const T*>(a.y) + slot * a.ldy + v * W);
                w[u] = a.weights ? __ldg(a.weights + t * a.k + j0 + u) : 1.0f;
            } else {
                const float none[W] = {};
                pack<W>(none, y[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[W];
            unpack<W>(y[u], f);
#pragma unroll
            for (int q = 0; q < W; ++q) sum[q] = fmaf(w[u], f[q], sum[q]);
        }
    }
    P o;
    pack<W>(sum, o);
    *reinterpret_cast<P*>(static_cast<T*>(a.out) + t * a.c + v * W) = o;
}

// Gradients of the weighted sum: THREADS (32 or the block's 128) a token, four
// choices at a time.
template <typename T, int W, int THREADS>
__global__ void __launch_bounds__(128) k_expert_combine_grad(const ExpertGrad a) {
    using P = Pack<T, W>;
    __shared__ float sh[4][4];
    pdl_wait();
    pdl_trigger();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (128 / THREADS) + threadIdx.x / THREADS, rows = a.tokens * a.k;
    const int32_t vectors = a.c / W, first = threadIdx.x % THREADS;
    constexpr int U = 4;
    if (t < a.tokens) {   // (the same for all threads of a token)
        const T* dout = static_cast<const T*>(a.dout) + t * a.ldd;
        for (int32_t j0 = 0; j0 < a.k; j0 += U) {
            int32_t slot[U];
            float w[U], dot[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                slot[u] = j0 + u < a.k ? __ldg(a.slots + t * a.k + j0 + u) : -1;
                if (!in_range(slot[u], rows)) slot[u] = -1;
                w[u] = slot[u] >= 0 ? __ldg(a.weights + t * a.k + j0 + u) : 0.0f;
                dot[u] = 0.0f;
            }
            for (int32_t v = first; v < vectors; v += THREADS) {
                float d[W];
                unpack<W>(*reinterpret_cast<const P*>(dout + v * W), d);
                P y[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (slot[u] >= 0) y[u] = *reinterpret_cast<const P*>(static_cast<const T*>(a.y) + slot[u] * a.ldy + v * W);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (slot[u] < 0) continue;
                    float f[W];
                    unpack<W>(y[u], f);
#pragma unroll
                    for (int q = 0; q < W; ++q) {
                        dot[u] = fmaf(d[q], f[q], dot[u]);
                        f[q] = w[u] * d[q];
                    }
                    P o;
                    pack<W>(f, o);
                    *reinterpret_cast<P*>(static_cast<T*>(a.dy) + static_cast<int64_t>(slot[u]) * a.c + v * W) = o;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot[u] += __shfl_xor_sync(0xFFFFFFFFu, dot[u], o);
            if (THREADS > 32) {
                if ((threadIdx.x & 31) == 0)
#pragma unroll
                    for (int u = 0; u < U; ++u) sh[threadIdx.x >> 5][u] = dot[u];
                __syncthreads();
#pragma unroll
                for (int u = 0; u < U; ++u) dot[u] = (sh[0][u] + sh[1][u]) + (sh[2][u] + sh[3][u]);
                __syncthreads();
            }
            if (first == 0)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (j0 + u < a.k) a.dweights[t * a.k + j0 + u] = dot[u];
        }
    }
    zero_tail(static_cast<P*>(a.dy), vectors, a.offsets, a.n_experts, rows);
}

// ---- weights in blocks --------------------------------------------------------------
// A block of threads per 128 x 128 values: the largest, then the values turned
// through shared memory.  Once per weight.
__global__ void __launch_bounds__(256) k_weight_to_blocks(const __nv_bfloat16* w, int32_t c_in, int32_t c_out, uint8_t* q,
                                                          float* scale) {
    __shared__ __nv_bfloat16 sh[128][130];
    __shared__ uint32_t warps[8];
    const int32_t c0 = blockIdx.x * 128, o0 = blockIdx.y * 128;
    const int64_t m = blockIdx.z;
    w += m * c_in * c_out;
    q += m * c_in * c_out;
    uint32_t most = 0;
#pragma unroll 8
    for (int i = threadIdx.x; i < 128 * 128; i += 256) {
        const int32_t c = c0 + i / 128, o = o0 + i % 128;
        const __nv_bfloat16 v = c < c_in && o < c_out ? w[static_cast<int64_t>(c) * c_out + o] : __float2bfloat16_rn(0.0f);
        sh[i / 128][i % 128] = v;
        const uint32_t b = __float_as_uint(fabsf(__bfloat162float(v)));
        most = b > most ? b : most;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint32_t u = __shfl_xor_sync(0xFFFFFFFFu, most, o);
        most = u > most ? u : most;
    }
    if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = most;
    __syncthreads();
    for (int i = 0; i < 8; ++i) most = warps[i] > most ? warps[i] : most;
    const float s = __fdiv_rn(__uint_as_float(most), 448.0f);
    if (threadIdx.x == 0) scale[(m * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = s;
    const int32_t c4 = threadIdx.x % 32 * 4;
    for (int j = threadIdx.x / 32; j < 128; j += 8) {
        const int32_t o = o0 + j, c = c0 + c4;
        if (o >= c_out || c >= c_in) continue;
        uint32_t v = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float x = s == 0.0f ? 0.0f : __fdiv_rn(__bfloat162float(sh[c4 + t][j]), s);
            v |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3)) << (8 * t);
        }
        uint8_t* out = q + static_cast<int64_t>(o) * c_in + c;
        if (c_in % 4 == 0 && reinterpret_cast<uintptr_t>(q) % 4 == 0) {
            *reinterpret_cast<uint32_t*>(out) = v;
        } else {
            for (int t = 0; t < 4 && c + t < c_in; ++t) out[t] = static_cast<uint8_t>(v >> (8 * t));
        }
    }
}

// ---- host -----------------------------------------------------------------------
template <typename F>
int with_type(int32_t dtype, uintptr_t all, int64_t ld, int32_t c, F&& f) {
    if (dtype == SPCONV_FP32) return with_width<float>(all | static_cast<uintptr_t>(ld * 4), c, [&](auto w) { return f(0.0f, w); });
    return with_width<__nv_bfloat16>(all | static_cast<uintptr_t>(ld * 2), c, [&](auto w) { return f(__nv_bfloat16(), w); });
}

uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// A thread a vector of `rows` rows.
template <typename... K, typename A>
int launch_flat(void (*kernel)(K...), int64_t rows, int64_t vectors, cudaStream_t s, const A& a) {
    const int64_t blocks = ceil_div(rows * vectors, 256);
    if (blocks > 0x7FFFFFFF) return SPCONV_ERR_UNSUPPORTED;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), 256, 0, s, a, RowVector(rows * vectors, vectors));
}

template <typename I>
int sort_pairs(const SortArgs& args, cudaStream_t s) {
    SortArgs a = args;
    const int64_t all = ceil_div(a.pairs > 0 ? a.pairs : 1, kSortThreads);
    a.tiles = static_cast<int32_t>(ceil_div(all, kMaxChunks));
    const unsigned chunks = static_cast<unsigned>(ceil_div(all, a.tiles));
    Scratch counts(chunks > 1 ? static_cast<size_t>(chunks) * a.n_experts * 4 : 0, s);
    if (counts.failed()) return SPCONV_ERR_OOM;
    a.counts = counts.as<int32_t>();
    if (chunks > 1) SPCONV_CHECK(launch_pdl(k_expert_count<I>, dim3(chunks), kSortThreads, 0, s, a));
    static bool set[kMaxDevices] = {};
    int dev = 0;
    SPCONV_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return SPCONV_ERR_UNSUPPORTED;
    if (!set[dev]) {
        SPCONV_CHECK_CUDA(cudaFuncSetAttribute(k_expert_place<I>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSortWarps * kMaxExperts * 2));
        set[dev] = true;
    }
    return launch_pdl(k_expert_place<I>, dim3(chunks), kSortThreads, static_cast<size_t>(kSortWarps) * a.n_experts * 2, s, a);
}

}  // namespace

int expert_plan(const void* experts, int32_t index_bytes, int64_t pairs, int32_t n_experts, int32_t* offsets, int32_t* sorted,
                int32_t* slots, cudaStream_t s) {
    SortArgs a = {};
    a.experts = experts;
    a.pairs = pairs;
    a.n_experts = n_experts;
    a.offsets = offsets;
    a.sorted = sorted;
    a.slots = slots;
    SPCONV_CHECK(rows_status_word(&a.status));
    return index_bytes == 8 ? sort_pairs<int64_t>(a, s) : sort_pairs<int32_t>(a, s);
}

int expert_gather(const ExpertRows& args, cudaStream_t s) {
    ExpertRows a = args;
    if (a.scale) {
        a.wide = a.c % 8 == 0 && bits(a.out) % 8 == 0;
        // two rows a thread where one each would fill the GPU twice over (2048 channels, us:
        // 64 rows 2.7 and with one row 2.1, 4000 rows 10.3 and 10.5, 40000 rows 85 and 97)
        const int64_t threads = a.tokens * ceil_div(a.c, 128) * 16;
        const bool two = threads > 2 * 152 * 2048;
        return with_type(a.dtype, bits(a.x), a.ldx, a.c, [&](auto t, auto w) {
            using T = decltype(t);
            return two ? launch_flat(k_rows_to_blocks<T, w, 2>, ceil_div(a.tokens, 2), ceil_div(a.c, 128) * 16, s, a)
                       : launch_flat(k_rows_to_blocks<T, w, 1>, a.tokens, ceil_div(a.c, 128) * 16, s, a);
        });
    }
    return with_type(a.dtype, bits(a.x) | bits(a.out), a.ldx, a.c,
                     [&](auto t, auto w) { return launch_flat(k_expert_gather<decltype(t), w>, a.tokens, a.c / w, s, a); });
}

int expert_combine(const ExpertSums& a, cudaStream_t s) {
    return with_type(a.dtype, bits(a.y) | bits(a.residual) | bits(a.out), a.residual ? a.ldy | a.ldr : a.ldy, a.c,
                     [&](auto t, auto w) { return launch_flat(k_expert_combine<decltype(t), w>, a.tokens, a.c / w, s, a); });
}

int expert_combine_backward(const ExpertGrad& a, cudaStream_t s) {
    return with_type(a.dtype, bits(a.dout) | bits(a.y) | bits(a.dy), a.ldd | a.ldy, a.c, [&](auto t, auto w) {
        using T = decltype(t);
        // a token's vectors are a warp's, or a block's where that takes each several times
        // (8189 tokens, us: 512 channels 9.4 and 14.8, 1024 26.6 and 28.0, 2048 49.8 and 47.4)
        const bool wide = a.c / w > 128;
        const int64_t blocks = wide ? a.tokens : ceil_div(a.tokens, 4);
        const dim3 grid(static_cast<unsigned>(blocks));   // (tokens < 2^30)
        return wide ? launch_pdl(k_expert_combine_grad<T, w, 128>, grid, 128, 0, s, a)
                    : launch_pdl(k_expert_combine_grad<T, w, 32>, grid, 128, 0, s, a);
    });
}

int quantize_weight_blocks(const void* w, int64_t count, int32_t c_in, int32_t c_out, void* q, float* scale, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(ceil_div(c_in, 128)), static_cast<unsigned>(ceil_div(c_out, 128)), static_cast<unsigned>(count));
    count_launch();
    k_weight_to_blocks<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(w), c_in, c_out, static_cast<uint8_t*>(q), scale);
    return launch_status();
}

}  // namespace spconv
