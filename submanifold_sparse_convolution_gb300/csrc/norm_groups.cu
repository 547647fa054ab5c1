// Group norm of ragged scans with an activation, and its backward pass.
//
// Rows offsets[s] .. offsets[s + 1] - 1 are scan s; a group is D = c / groups
// neighbouring channels; M = rows of the scan x D values share statistics:
//
//   u = (x - mean) r,  r = 1 / sqrt(var + eps);  z = u w + b;  y = act(z)
//   dz = dy act'(z),  p = dz w:   dx = r (p - mean(p) - u mean(p u))
//   dw = sum_rows dz u;  db = sum_rows dz
//
// A scan's statistics need all of it, so each pass is two kernels: sums of
// pieces, then the rows again (from L2 where they fit it).  Block b of both
// holds the rows [b R, (b + 1) R): the offsets stay on the device, so the rows
// are cut without looking at them, and a block walks the pieces of the scans
// that it meets.  The piece of scan s in block b has the number b + s, which no
// other piece has (along the rows both only grow, one of them strictly), and a
// scan's pieces have consecutive ones.  The second kernel's blocks add up the
// pieces of their scans in that order: no atomics, the same bits every run.
//
// Bound by HBM, and for small inputs by the chain of latencies (two launches,
// the loads, the pieces).
#include "row_vectors.cuh"

namespace spconv {
namespace {

constexpr int kSms = 152;
constexpr int kMaxPieces = 160;          // blocks that a warp adds up: five pieces a lane
constexpr int kPerLane = kMaxPieces / 32;
constexpr int kStatThreads = 1024, kApplyThreads = 640, kBwdThreads = 512;   // (registers)

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The scans' borders, brought into order and range, whatever they hold.
struct Scans {
    const int32_t* offsets;   // [scans + 1] or null: one scan of all rows
    int32_t scans;
    int32_t n;

    __device__ __forceinline__ int32_t raw(int32_t i) const { return offsets ? offsets[i] : (i == 0 ? 0 : n); }
    __device__ __forceinline__ int32_t at(int32_t i) const {
        const int32_t v = raw(i);
        return v < 0 ? 0 : v > n ? n : v;
    }
    // Number of borders at or before `row`, by the whole block.
    __device__ __forceinline__ int32_t borders(int32_t row) const {
        if (!offsets) return 1;   // (0 <= row < n)
        int32_t count = 0;
        for (int32_t i0 = 0; i0 <= scans; i0 += blockDim.x) {
            const int32_t i = i0 + static_cast<int32_t>(threadIdx.x);
            count += __syncthreads_count(i <= scans && offsets[i] <= row);
        }
        return count;
    }
    // f(scan, first row, last row + 1) for each piece of [row0, row1): scans
    // outside [0, scans) are rows of no scan.  The same for all threads.
    template <typename F>
    __device__ __forceinline__ void pieces(int32_t row0, int32_t row1, F&& f) const {
        int32_t s = borders(row0) - 1, row = row0;
        while (row < row1) {
            int32_t end = s < scans ? at(s + 1) : n;
            if (end > row1) end = row1;
            if (end > row) {
                f(s, row, end);
                row = end;
            }
            ++s;
        }
    }
};

struct Shape {
    int32_t c, groups, width;      // width: channels of a group
    int32_t vectors, tx, ty;       // vectors of a row; threads across and down
    int32_t rows;                  // of a block (R)
    int32_t joined;                // channels of a group that a thread of k_group_stats joins: a power of two
    int64_t slots;                 // blocks + scans
};

// Where piece sums lie: [groups][slots], so that a warp reads a group's run.
__device__ __forceinline__ int64_t slot_of(const Shape& h, int32_t group, int32_t scan) {
    return group * h.slots + static_cast<int32_t>(blockIdx.x) + scan;
}

// This lane's share of a scan's pieces of one group, in order, and how many
// rows each has.
struct PieceSet {
    float2 v[kPerLane];
    float rows[kPerLane];
    __device__ __forceinline__ void load(const Shape& h, const float2* part, int32_t group, int32_t s, int32_t lo, int32_t hi) {
        const int32_t b0 = lo / h.rows, b1 = (hi - 1) / h.rows, lane = threadIdx.x & 31;
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
            const int32_t b = b0 + 32 * k + lane;
            v[k] = make_float2(0.0f, 0.0f);
            rows[k] = 0.0f;
            if (b <= b1) {
                v[k] = __ldcg(part + group * h.slots + b + s);
                const int32_t first = b * h.rows > lo ? b * h.rows : lo, last = (b + 1) * h.rows < hi ? (b + 1) * h.rows : hi;
                rows[k] = static_cast<float>(last - first);
            }
        }
    }
};

// ---- forward ------------------------------------------------------------------
struct NormPass {
    GroupNormArgs a;
    Shape h;
    Scans scans;
    float2* part;        // of each piece: mean, sum of squares about it
    int32_t* status;
};

// Statistics of the block's pieces.  A thread's sums are about its first value
// of the channel, so a mean far from zero costs no digits; it joins its channels
// of a group, and a warp the threads' about the group's mean, in two passes over
// shared memory.
template <typename T, int W>
__global__ void __launch_bounds__(kStatThreads, 1) k_group_stats(const __grid_constant__ NormPass p) {
    using P = Pack<T, W>;
    extern __shared__ float sh[];
    const Shape& h = p.h;
    const int32_t entries = h.c / h.joined;
    float* sh_mean = sh;                                            // [ty][entries]
    float* sh_m2 = sh + static_cast<size_t>(h.ty) * entries;
    const int tx = threadIdx.x % h.tx, ty = threadIdx.x / h.tx, lane = threadIdx.x & 31;
    const int32_t row0 = static_cast<int32_t>(blockIdx.x) * h.rows;
    const int32_t row1 = row0 + h.rows < p.scans.n ? row0 + h.rows : p.scans.n;
    pdl_wait();
    pdl_trigger();
    p.scans.pieces(row0, row1, [&](int32_t s, int32_t lo, int32_t hi) {
        if (s < 0 || s >= p.scans.scans) return;
        const int32_t each = (hi - lo) / h.ty, extra = (hi - lo) % h.ty;   // rows of a thread; threads with one more
        for (int32_t v = tx; v < h.vectors && ty < h.ty; v += h.tx) {
            const T* x = static_cast<const T*>(p.a.x) + v * W;
            float first[W], sum[W], sq[W];
            int32_t r = lo + ty;
            if (r < hi) {
                unpack<W>(*reinterpret_cast<const P*>(x + r * p.a.ldx), first);
#pragma unroll
                for (int j = 0; j < W; ++j) sum[j] = sq[j] = 0.0f;
                r += h.ty;
                auto add = [&](const P& q) {
                    float f[W];
                    unpack<W>(q, f);
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        const float d = f[j] - first[j];
                        sum[j] += d;
                        sq[j] = fmaf(d, d, sq[j]);
                    }
                };
                constexpr int U = 4;
                for (; r + (U - 1) * h.ty < hi; r += U * h.ty) {
                    P q[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) q[u] = *reinterpret_cast<const P*>(x + (r + u * h.ty) * p.a.ldx);
#pragma unroll
                    for (int u = 0; u < U; ++u) add(q[u]);
                }
                for (; r < hi; r += h.ty) add(*reinterpret_cast<const P*>(x + r * p.a.ldx));
                const float n = static_cast<float>(each + (ty < extra)), by_n = 1.0f / n;
                float mean[W], m2[W];
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const float m = sum[j] * by_n;   // of x - first
                    mean[j] = first[j] + m;
                    const float q = fmaf(-m, sum[j], sq[j]);
                    m2[j] = q < 0.0f ? 0.0f : q;     // (keeps NaN)
                }
                // neighbouring channels of a group, as many as lie in one vector
#pragma unroll
                for (int w = 1; w < W; w *= 2)
                    if (h.joined > w) {
#pragma unroll
                        for (int j = 0; j < W; j += 2 * w) {
                            const float d = mean[j + w] - mean[j];
                            mean[j] = fmaf(0.5f, d, mean[j]);
                            m2[j] += fmaf(0.5f * n * static_cast<float>(w) * d, d, m2[j + w]);
                        }
                    }
                const int32_t at = ty * entries + v * W / h.joined;
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (j % h.joined == 0) {
                        sh_mean[at + j / h.joined] = mean[j];
                        sh_m2[at + j / h.joined] = m2[j];
                    }
            }
        }
        __syncthreads();
        const int32_t deep = hi - lo < h.ty ? hi - lo : h.ty;   // thread rows that have any
        const float by_count = 1.0f / (static_cast<float>(hi - lo) * static_cast<float>(h.width));
        // lanes across a group's entries, and down the thread rows where those are few
        const int32_t wide = h.width / h.joined, down = wide < 32 ? 32 / wide : 1;
        const int32_t k0 = wide < 32 ? lane % wide : lane, t0 = wide < 32 ? lane / wide : 0;
        for (int32_t g = threadIdx.x >> 5; g < h.groups; g += blockDim.x >> 5) {
            const float base = sh_mean[g * wide];
            float sum = 0.0f, m2 = 0.0f;
            auto entries_of = [&](auto&& f) {
                if (t0 >= down) return;
                for (int32_t t = t0; t < deep; t += down) {
                    const float n = static_cast<float>((each + (t < extra)) * h.joined);
                    for (int32_t k = k0; k < wide; k += 32) f(t * entries + g * wide + k, n);
                }
            };
            entries_of([&](int32_t i, float n) { sum = fmaf(n, sh_mean[i] - base, sum); });
            const float mean = base + warp_sum(sum) * by_count;
            entries_of([&](int32_t i, float n) {
                const float d = sh_mean[i] - mean;
                m2 += fmaf(n * d, d, sh_m2[i]);
            });
            m2 = warp_sum(m2);
            if (lane == 0) p.part[slot_of(h, g, s)] = make_float2(mean, m2);
        }
        __syncthreads();
    });
}

// The rows again, last ones first: those are the ones that L2 still has where
// the input is larger.
template <typename T, int W>
__global__ void __launch_bounds__(kApplyThreads, 1) k_group_apply(const __grid_constant__ NormPass p) {
    using P = Pack<T, W>;
    extern __shared__ float sh[];
    const Shape& h = p.h;
    const GroupNormArgs& a = p.a;
    float* sh_mean = sh;              // [groups]
    float* sh_r = sh + h.groups;
    const int tx = threadIdx.x % h.tx, ty = threadIdx.x / h.tx, lane = threadIdx.x & 31;
    const int32_t row0 = static_cast<int32_t>(blockIdx.x) * h.rows;
    const int32_t row1 = row0 + h.rows < p.scans.n ? row0 + h.rows : p.scans.n;
    pdl_wait();
    pdl_trigger();
    // what the scans without a row have for statistics; borders out of order or range
    if (p.scans.offsets)
        for (int32_t s = blockIdx.x * blockDim.x + threadIdx.x; s < p.scans.scans; s += gridDim.x * blockDim.x) {
            const int32_t lo = p.scans.raw(s), hi = p.scans.raw(s + 1);
            if (lo > hi || lo < 0 || hi > p.scans.n) atomicOr(p.status, kStatusRange);
            if (a.stats && p.scans.at(s) >= p.scans.at(s + 1))
                for (int32_t g = 0; g < h.groups; ++g)
                    a.stats[static_cast<int64_t>(s) * h.groups + g] = make_float2(0.0f, rsqrtf(a.eps));
        }
    p.scans.pieces(row0, row1, [&](int32_t s, int32_t lo, int32_t hi) {
        T* out = static_cast<T*>(a.out);
        if (s < 0 || s >= p.scans.scans) {
            P zero;
            float f[W] = {};
            pack<W>(f, zero);
            for (int32_t v = tx; v < h.vectors && ty < h.ty; v += h.tx)
                for (int32_t r = lo + ty; r < hi; r += h.ty) *reinterpret_cast<P*>(out + static_cast<int64_t>(r) * h.c + v * W) = zero;
            return;
        }
        const int32_t s_lo = p.scans.at(s), s_hi = p.scans.at(s + 1);
        const float by_count = 1.0f / (static_cast<float>(s_hi - s_lo) * static_cast<float>(h.width));
        __syncthreads();   // (the last piece's statistics have been read)
        for (int32_t g = threadIdx.x >> 5; g < h.groups; g += blockDim.x >> 5) {
            PieceSet set;
            set.load(h, p.part, g, s, s_lo, s_hi);
            const float base = __shfl_sync(0xFFFFFFFFu, set.v[0].x, 0), width = static_cast<float>(h.width);
            float sum = 0.0f, m2 = 0.0f;
#pragma unroll
            for (int k = 0; k < kPerLane; ++k) sum = fmaf(set.rows[k] * width, set.rows[k] > 0.0f ? set.v[k].x - base : 0.0f, sum);
            const float mean = base + warp_sum(sum) * by_count;
#pragma unroll
            for (int k = 0; k < kPerLane; ++k) {
                const float d = set.rows[k] > 0.0f ? set.v[k].x - mean : 0.0f;
                m2 += fmaf(set.rows[k] * width * d, d, set.v[k].y);
            }
            const float r = rsqrtf(warp_sum(m2) * by_count + a.eps);
            if (lane == 0) {
                sh_mean[g] = mean;
                sh_r[g] = r;
                if (a.stats && lo == s_lo) a.stats[static_cast<int64_t>(s) * h.groups + g] = make_float2(mean, r);
            }
        }
        __syncthreads();
        with_act(a.act, [&](auto act) {
            for (int32_t v = tx; v < h.vectors && ty < h.ty; v += h.tx) {
                const T* x = static_cast<const T*>(a.x) + v * W;
                T* y = out + v * W;
                float mean[W], scale[W], bias[W];
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const int32_t ch = v * W + j, g = ch / h.width;
                    mean[j] = sh_mean[g];
                    scale[j] = sh_r[g] * __ldg(a.weight + ch);
                    bias[j] = a.bias ? __ldg(a.bias + ch) : 0.0f;
                }
                auto one = [&](const P& q, int32_t r) {
                    float f[W];
                    unpack<W>(q, f);
#pragma unroll
                    for (int j = 0; j < W; ++j) f[j] = act_f<act>(fmaf(f[j] - mean[j], scale[j], bias[j]));
                    P o;
                    pack<W>(f, o);
                    *reinterpret_cast<P*>(y + static_cast<int64_t>(r) * h.c) = o;
                };
                constexpr int U = 4;
                int32_t r = hi - 1 - ty;
                for (; r - (U - 1) * h.ty >= lo; r -= U * h.ty) {
                    P q[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) q[u] = *reinterpret_cast<const P*>(x + (r - u * h.ty) * a.ldx);
#pragma unroll
                    for (int u = 0; u < U; ++u) one(q[u], r - u * h.ty);
                }
                for (; r >= lo; r -= h.ty) one(*reinterpret_cast<const P*>(x + r * a.ldx), r);
            }
        });
    });
}

// Statistics where there is no row at all.
__global__ void __launch_bounds__(256) k_empty_stats(float2* stats, int64_t count, float eps) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (i < count) stats[i] = make_float2(0.0f, rsqrtf(eps));
}

// ---- backward -----------------------------------------------------------------
struct GradPass {
    GroupNormGradArgs a;
    Shape h;
    Scans scans;
    float2* part;        // of each piece: sums of p and of p u
    float* cols;         // [blocks][2][c]: sums of dz u, of dz
    int32_t blocks;      // of rows; the blocks after them add up cols
    int32_t* status;
};

// What a thread needs of its W channels in a scan.
template <int W>
struct Channels {
    float mean[W], r[W], w[W], b[W];
    __device__ __forceinline__ void load(const GradPass& p, int32_t s, int32_t v) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int32_t ch = v * W + j;
            const float2 st = __ldg(p.a.stats + static_cast<int64_t>(s) * p.h.groups + ch / p.h.width);
            mean[j] = st.x;
            r[j] = st.y;
            w[j] = __ldg(p.a.weight + ch);
            b[j] = p.a.bias ? __ldg(p.a.bias + ch) : 0.0f;
        }
    }
};

template <typename T, int W>
__global__ void __launch_bounds__(kBwdThreads, 1) k_group_grad_sums(const __grid_constant__ GradPass p) {
    using P = Pack<T, W>;
    extern __shared__ float sh[];
    const Shape& h = p.h;
    float* total = sh;                                              // [2][c]: of all pieces
    float* sh_u = sh + 2 * h.c;                                     // [ty][c]: sums of dz u
    float* sh_z = sh_u + static_cast<size_t>(h.ty) * h.c;           // sums of dz
    const int tx = threadIdx.x % h.tx, ty = threadIdx.x / h.tx, lane = threadIdx.x & 31;
    const int32_t row0 = static_cast<int32_t>(blockIdx.x) * h.rows;
    const int32_t row1 = row0 + h.rows < p.scans.n ? row0 + h.rows : p.scans.n;
    pdl_wait();
    pdl_trigger();
    for (int32_t i = threadIdx.x; i < 2 * h.c; i += blockDim.x) total[i] = 0.0f;
    p.scans.pieces(row0, row1, [&](int32_t s, int32_t lo, int32_t hi) {
        if (s < 0 || s >= p.scans.scans) return;
        with_act(p.a.act, [&](auto act) {
            for (int32_t v = tx; v < h.vectors && ty < h.ty; v += h.tx) {
                const T* x = static_cast<const T*>(p.a.x) + v * W;
                const T* dy = static_cast<const T*>(p.a.dy) + v * W;
                Channels<W> ch;
                ch.load(p, s, v);
                float su[W] = {}, sz[W] = {};
                auto add = [&](const P& qx, const P& qd) {
                    float f[W], d[W];
                    unpack<W>(qx, f);
                    unpack<W>(qd, d);
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        const float u = (f[j] - ch.mean[j]) * ch.r[j];
                        float unused;
                        const float dz = d[j] * act_grad_f<act>(fmaf(u, ch.w[j], ch.b[j]), &unused);
                        su[j] = fmaf(dz, u, su[j]);
                        sz[j] += dz;
                    }
                };
                constexpr int U = 2;
                int32_t r = lo + ty;
                for (; r + (U - 1) * h.ty < hi; r += U * h.ty) {
                    P qx[U], qd[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        qx[u] = *reinterpret_cast<const P*>(x + (r + u * h.ty) * p.a.ldx);
                        qd[u] = *reinterpret_cast<const P*>(dy + (r + u * h.ty) * p.a.ldy);
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) add(qx[u], qd[u]);
                }
                for (; r < hi; r += h.ty)
                    add(*reinterpret_cast<const P*>(x + r * p.a.ldx), *reinterpret_cast<const P*>(dy + r * p.a.ldy));
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    sh_u[ty * h.c + v * W + j] = su[j];
                    sh_z[ty * h.c + v * W + j] = sz[j];
                }
            }
        });
        __syncthreads();
        // down the thread rows: by several threads where a row has fewer channels than the block threads
        const int32_t deep = hi - lo < h.ty ? hi - lo : h.ty;
        const int32_t threads = static_cast<int32_t>(blockDim.x);
        int32_t rows = h.c < threads ? threads / h.c : 1;
        if (rows > deep) rows = deep;
        for (int32_t i = threadIdx.x; i < rows * h.c; i += threads) {
            const int32_t c = i % h.c;
            float u = 0.0f, z = 0.0f;
            for (int32_t t = i / h.c; t < deep; t += rows) {
                u += sh_u[t * h.c + c];
                z += sh_z[t * h.c + c];
            }
            sh_u[i] = u;   // (row i / c, which no other thread reads)
            sh_z[i] = z;
        }
        __syncthreads();
        for (int32_t c = threadIdx.x; c < h.c; c += threads) {
            float u = 0.0f, z = 0.0f;
            for (int32_t t = 0; t < rows; ++t) {
                u += sh_u[t * h.c + c];
                z += sh_z[t * h.c + c];
            }
            total[c] += u;
            total[h.c + c] += z;
            const float w = __ldg(p.a.weight + c);
            sh_u[c] = u * w;
            sh_z[c] = z * w;
        }
        __syncthreads();
        for (int32_t g = threadIdx.x >> 5; g < h.groups; g += blockDim.x >> 5) {
            float u = 0.0f, z = 0.0f;
            for (int32_t k = lane; k < h.width; k += 32) {
                u += sh_u[g * h.width + k];
                z += sh_z[g * h.width + k];
            }
            u = warp_sum(u);
            z = warp_sum(z);
            if (lane == 0) p.part[slot_of(h, g, s)] = make_float2(z, u);
        }
        __syncthreads();
    });
    __syncthreads();
    for (int32_t i = threadIdx.x; i < 2 * h.c; i += blockDim.x) p.cols[static_cast<int64_t>(blockIdx.x) * 2 * h.c + i] = total[i];
}

// Columns of the blocks' sums: 32 of them a block, 16 threads down each.
__device__ __forceinline__ void add_columns(const GradPass& p, float* sh) {
    const int32_t col = (static_cast<int32_t>(blockIdx.x) - p.blocks) * 32 + (threadIdx.x & 31), deep = threadIdx.x >> 5;
    float sum = 0.0f;
    if (col < 2 * p.h.c)
        for (int32_t b = deep; b < p.blocks; b += kBwdThreads / 32) sum += __ldcg(p.cols + static_cast<int64_t>(b) * 2 * p.h.c + col);
    sh[threadIdx.x] = sum;
    __syncthreads();
    if (deep != 0 || col >= 2 * p.h.c) return;
    for (int32_t t = 1; t < kBwdThreads / 32; ++t) sum += sh[t * 32 + threadIdx.x];
    if (col < p.h.c) p.a.dweight[col] = sum;
    else if (p.a.dbias) p.a.dbias[col - p.h.c] = sum;
}

template <typename T, int W>
__global__ void __launch_bounds__(kBwdThreads, 1) k_group_grad_apply(const __grid_constant__ GradPass p) {
    using P = Pack<T, W>;
    extern __shared__ float sh[];
    const Shape& h = p.h;
    const GroupNormGradArgs& a = p.a;
    float* sh_z = sh;                 // [groups]: means of p, of p u
    float* sh_u = sh + h.groups;
    pdl_wait();
    pdl_trigger();
    if (static_cast<int32_t>(blockIdx.x) >= p.blocks) {
        add_columns(p, sh);
        return;
    }
    const int tx = threadIdx.x % h.tx, ty = threadIdx.x / h.tx, lane = threadIdx.x & 31;
    const int32_t row0 = static_cast<int32_t>(blockIdx.x) * h.rows;
    const int32_t row1 = row0 + h.rows < p.scans.n ? row0 + h.rows : p.scans.n;
    if (p.scans.offsets)
        for (int32_t s = blockIdx.x * blockDim.x + threadIdx.x; s < p.scans.scans; s += p.blocks * blockDim.x) {
            const int32_t lo = p.scans.raw(s), hi = p.scans.raw(s + 1);
            if (lo > hi || lo < 0 || hi > p.scans.n) atomicOr(p.status, kStatusRange);
        }
    p.scans.pieces(row0, row1, [&](int32_t s, int32_t lo, int32_t hi) {
        T* out = static_cast<T*>(a.dx);
        if (s < 0 || s >= p.scans.scans) {
            P zero;
            float f[W] = {};
            pack<W>(f, zero);
            for (int32_t v = tx; v < h.vectors && ty < h.ty; v += h.tx)
                for (int32_t r = lo + ty; r < hi; r += h.ty) *reinterpret_cast<P*>(out + static_cast<int64_t>(r) * h.c + v * W) = zero;
            return;
        }
        const int32_t s_lo = p.scans.at(s), s_hi = p.scans.at(s + 1);
        const float by_count = 1.0f / (static_cast<float>(s_hi - s_lo) * static_cast<float>(h.width));
        __syncthreads();
        for (int32_t g = threadIdx.x >> 5; g < h.groups; g += blockDim.x >> 5) {
            PieceSet set;
            set.load(h, p.part, g, s, s_lo, s_hi);
            float z = 0.0f, u = 0.0f;
#pragma unroll
            for (int k = 0; k < kPerLane; ++k) {
                z += set.v[k].x;
                u += set.v[k].y;
            }
            z = warp_sum(z);
            u = warp_sum(u);
            if (lane == 0) {
                sh_z[g] = z * by_count;
                sh_u[g] = u * by_count;
            }
        }
        __syncthreads();
        with_act(a.act, [&](auto act) {
            for (int32_t v = tx; v < h.vectors && ty < h.ty; v += h.tx) {
                const T* x = static_cast<const T*>(a.x) + v * W;
                const T* dy = static_cast<const T*>(a.dy) + v * W;
                T* dx = out + v * W;
                Channels<W> ch;
                ch.load(p, s, v);
                float mz[W], mu[W];
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const int32_t g = (v * W + j) / h.width;
                    mz[j] = sh_z[g];
                    mu[j] = sh_u[g];
                }
                auto one = [&](const P& qx, const P& qd, int32_t r) {
                    float f[W], d[W];
                    unpack<W>(qx, f);
                    unpack<W>(qd, d);
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        const float u = (f[j] - ch.mean[j]) * ch.r[j];
                        float unused;
                        const float dz = d[j] * act_grad_f<act>(fmaf(u, ch.w[j], ch.b[j]), &unused);
                        f[j] = ch.r[j] * (fmaf(dz, ch.w[j], -mz[j]) - u * mu[j]);
                    }
                    P o;
                    pack<W>(f, o);
                    *reinterpret_cast<P*>(dx + static_cast<int64_t>(r) * h.c) = o;
                };
                constexpr int U = 2;
                int32_t r = hi - 1 - ty;
                for (; r - (U - 1) * h.ty >= lo; r -= U * h.ty) {
                    P qx[U], qd[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        qx[u] = *reinterpret_cast<const P*>(x + (r - u * h.ty) * a.ldx);
                        qd[u] = *reinterpret_cast<const P*>(dy + (r - u * h.ty) * a.ldy);
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) one(qx[u], qd[u], r - u * h.ty);
                }
                for (; r >= lo; r -= h.ty)
                    one(*reinterpret_cast<const P*>(x + r * a.ldx), *reinterpret_cast<const P*>(dy + r * a.ldy), r);
            }
        });
    });
}

// ---- host -----------------------------------------------------------------------
// A block of at most `most` threads over vectors of a row; how many it uses.
int set_threads(Shape* h, int most) {
    h->tx = h->vectors < most ? h->vectors : most;
    h->ty = most / h->tx;
    return static_cast<int>(round_up(static_cast<size_t>(h->tx) * h->ty, 32));
}

// Vectors of W elements, and the rows of a block: one block per SM, fewer where
// each would have less than one step of loads.
Shape make_shape(int64_t n, int32_t c, int32_t groups, int64_t scans, int w, int most, int* blocks, int* threads) {
    Shape h = {};
    h.c = c;
    h.groups = groups;
    h.width = c / groups;
    h.vectors = c / w;
    h.joined = 1;
    while (h.joined < w && h.width % (2 * h.joined) == 0) h.joined *= 2;
    *threads = set_threads(&h, most);
    int64_t b = ceil_div(n, static_cast<int64_t>(4) * h.ty);
    if (b > kSms) b = kSms;
    h.rows = static_cast<int32_t>(ceil_div(n, b));
    *blocks = static_cast<int>(ceil_div(n, h.rows));
    h.slots = *blocks + scans;
    return h;
}

template <auto KERNEL, typename A>
int launch_wide(int blocks, int threads, size_t smem, cudaStream_t s, const A& args) {
    static bool set[kMaxDevices] = {};
    int dev = 0;
    SPCONV_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return SPCONV_ERR_UNSUPPORTED;
    if (!set[dev]) {
        SPCONV_CHECK_CUDA(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024));
        set[dev] = true;
    }
    return launch_pdl(KERNEL, dim3(static_cast<unsigned>(blocks)), threads, smem, s, args);
}

template <typename T, int W>
int forward_w(const GroupNormArgs& a, cudaStream_t s) {
    NormPass p = {};
    p.a = a;
    int blocks = 0, threads = 0;
    p.h = make_shape(a.n, a.c, a.groups, a.scans, W, kStatThreads, &blocks, &threads);
    p.scans = Scans{a.offsets, static_cast<int32_t>(a.scans), static_cast<int32_t>(a.n)};
    SPCONV_CHECK(rows_status_word(&p.status));
    Scratch part(static_cast<size_t>(p.h.slots) * a.groups * sizeof(float2), s);
    if (part.failed()) return SPCONV_ERR_OOM;
    p.part = part.as<float2>();
    SPCONV_CHECK((launch_wide<k_group_stats<T, W>>(blocks, threads, static_cast<size_t>(2) * p.h.ty * (a.c / p.h.joined) * 4, s, p)));
    threads = set_threads(&p.h, kApplyThreads);
    return launch_wide<k_group_apply<T, W>>(blocks, threads, static_cast<size_t>(2) * a.groups * 4, s, p);
}

template <typename T, int W>
int backward_w(const GroupNormGradArgs& a, cudaStream_t s) {
    GradPass p = {};
    p.a = a;
    int threads = 0;
    p.h = make_shape(a.n, a.c, a.groups, a.scans, W, kBwdThreads, &p.blocks, &threads);
    p.scans = Scans{a.offsets, static_cast<int32_t>(a.scans), static_cast<int32_t>(a.n)};
    SPCONV_CHECK(rows_status_word(&p.status));
    const size_t part_bytes = round_up(static_cast<size_t>(p.h.slots) * a.groups * sizeof(float2), 256);
    Scratch buf(part_bytes + static_cast<size_t>(p.blocks) * 2 * a.c * 4, s);
    if (buf.failed()) return SPCONV_ERR_OOM;
    p.part = buf.as<float2>();
    p.cols = buf.as<float>(part_bytes);
    SPCONV_CHECK((launch_wide<k_group_grad_sums<T, W>>(p.blocks, threads, static_cast<size_t>(2) * (p.h.ty + 1) * a.c * 4, s, p)));
    size_t smem = static_cast<size_t>(2) * a.groups * 4;
    if (smem < kBwdThreads * 4) smem = kBwdThreads * 4;
    return launch_wide<k_group_grad_apply<T, W>>(p.blocks + static_cast<int>(ceil_div(2 * a.c, 32)), kBwdThreads, smem, s, p);
}

}  // namespace

int group_norm_forward(const GroupNormArgs& a, cudaStream_t s) {
    if (a.n == 0) {
        const int64_t count = a.scans * a.groups;
        return launch_pdl(k_empty_stats, dim3(static_cast<unsigned>(ceil_div(count, 256))), 256, 0, s, a.stats, count, a.eps);
    }
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out);
    if (a.dtype == SPCONV_FP32)
        return with_width<float>(all | static_cast<uintptr_t>(a.ldx * 4), a.c, [&](auto w) { return forward_w<float, w>(a, s); });
    return with_width<__nv_bfloat16>(all | static_cast<uintptr_t>(a.ldx * 2), a.c,
                                     [&](auto w) { return forward_w<__nv_bfloat16, w>(a, s); });
}

int group_norm_backward(const GroupNormGradArgs& a, cudaStream_t s) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.dx);
    if (a.dtype == SPCONV_FP32)
        return with_width<float>(all | static_cast<uintptr_t>((a.ldx | a.ldy) * 4), a.c,
                                 [&](auto w) { return backward_w<float, w>(a, s); });
    return with_width<__nv_bfloat16>(all | static_cast<uintptr_t>((a.ldx | a.ldy) * 2), a.c,
                                     [&](auto w) { return backward_w<__nv_bfloat16, w>(a, s); });
}

}  // namespace spconv
