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
// scan's pieces have consecutive ones.  They are added up in that order: no
// atomics, the same bits every run.
//
// One scan of up to kSmallBytes, and every backward pass, have one block per SM at most;
// the second kernel's blocks add up the pieces of their scans themselves, and they load
// their first rows while the first kernel ends.  A forward pass over several scans, or
// beyond kSmallBytes, has blocks of kBlockBytes, or smaller ones where those would be fewer
// than four an SM; a small kernel between the two adds the pieces up, and the second takes
// the blocks from the last to the first, whose rows L2 read last (160000 x 256, 82 MB: 44.7
// us, from the first on 46.4; beyond L2 at most 1 %: of 307 MB the second kernel reads 306
// from HBM again).
//
// Scans of at most kScanBytes on the average are taken whole by a cluster of up
// to eight CTAs, which keep the rows in registers and exchange their sums through
// distributed shared memory: one launch, the rows read once.
//
// What bounds it: small inputs the launches and the chain offsets - rows - sums -
// rows (3000 x 64 in bf16: 7 us, 32371 x 128: 14 us for 25 MB), large ones HBM, which
// has the rows twice and the result (1000000 x 256: 249 us, 6.2 TB/s of 1.54 GB;
// backward 420 us, 6.1 TB/s of 2.56 GB).
#include "ptx_sm100.cuh"
#include "row_vectors.cuh"

namespace spconv {
namespace {

constexpr int kSms = 152;
constexpr int kPerLane = 5;              // pieces that a lane adds up where a block does so for itself
static_assert(kSms <= 32 * kPerLane, "blocks of a small input");
constexpr int kThreads = 448;            // blocks of a small input (72 registers a thread, two on an SM); half of it for those of a large one
constexpr int kApplyThreads = 320;       // (96 registers a thread, and room on an SM beside a block of k_group_stats)
// (us, bf16, 256 channels, as a small input and otherwise: one scan of 10 MB 13.3 and 14.1, 41 MB 24.2
// and 24.4, 64 MB 36.2 and 34.9, 82 MB 48.7 and 45.9, seven scans of 10 MB together 19.1 and 16.5, of 64 MB
// 43 and 37.  A backward pass gains nothing from more blocks: 41 MB 44 and 51, 512 MB 420 and 446; only very
// many scans would, 2000 of 50 rows 106 and 85.)
constexpr int64_t kSmallBytes = 40 << 20;
// (154 MB: 81 us, with 64 kB 83; 512 MB: 249, 256, with 1 MB 275.  At least four blocks an SM
// all the same: 72 MB 40 us, with blocks of 1 MB alone 104)
constexpr int64_t kBlockBytes = 256 << 10;
constexpr int64_t kScanBytes = 512 << 10;
constexpr int kMaxCluster = 8;           // portable cluster size

// W values in fp32, two in a register pair where there are two: the packed
// instructions do both in one issue.
template <int W>
struct Values {
    using V = std::conditional_t<W == 1, float, F2>;
    static constexpr int n = W == 1 ? 1 : W / 2;
    V v[n];
    __device__ __forceinline__ void set(float x) {
#pragma unroll
        for (int j = 0; j < n; ++j) v[j] = V(x);
    }
    __device__ __forceinline__ void put(const float (&f)[W]) {
        if constexpr (W == 1) {
            v[0] = f[0];
        } else {
#pragma unroll
            for (int j = 0; j < n; ++j) v[j] = F2(f[2 * j], f[2 * j + 1]);
        }
    }
    __device__ __forceinline__ void get(float (&f)[W]) const {
        if constexpr (W == 1) {
            f[0] = v[0];
        } else {
#pragma unroll
            for (int j = 0; j < n; ++j) v[j].get(f[2 * j], f[2 * j + 1]);
        }
    }
    template <typename T>
    __device__ __forceinline__ void unpack(const Pack<T, W>& p) {
        float f[W];
        spconv::unpack<W>(p, f);
        put(f);
    }
    template <typename T>
    __device__ __forceinline__ void pack(Pack<T, W>& p) const {
        float f[W];
        get(f);
        spconv::pack<W>(f, p);
    }
};

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
    int32_t blocks;
    int32_t shift;                 // 2^shift channels of a group lie in a vector and are joined by a thread
    int32_t lanes;                 // of a warp that join one group's entries: a power of two
    FastDiv by_tx, by_ty, by_wide, by_blocks;   // wide: entries of a group in a row
    int64_t slots;                 // blocks + scans
};

// Where piece sums lie: [groups][slots], so that a warp reads a group's run.
__device__ __forceinline__ int64_t slot_of(const Shape& h, int32_t group, int32_t scan) {
    return group * h.slots + static_cast<int32_t>(blockIdx.x) + scan;
}

// U vectors, `step` rows apart from row r on, those before `end`.
template <typename P, typename T, int U>
__device__ __forceinline__ void load_rows(P (&q)[U], const T* at, int64_t ld, int32_t r, int32_t step, int32_t end) {
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (r + u * step < end) q[u] = *reinterpret_cast<const P*>(at + (r + u * step) * ld);
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

// A thread's vectors of N matrices on their way through its own slots of shared
// memory: D rows ahead, without registers for them.
template <typename P, int N, int D>
struct Stream {
    P* slots;        // this thread's: slot (s, a) at (s N + a) threads
    int32_t threads;
    __device__ __forceinline__ Stream(void* shared) : slots(static_cast<P*>(shared) + threadIdx.x), threads(blockDim.x) {}
    static __host__ __device__ constexpr size_t bytes(int threads) { return static_cast<size_t>(D) * N * threads * sizeof(P); }
    __device__ __forceinline__ void put(int32_t s, int a, const P* from) {
        P* to = slots + (s * N + a) * threads;
        if constexpr (sizeof(P) >= 4) ptx::cp_async_n<sizeof(P)>(ptx::smem_u32(to), from);
        else *to = *from;
    }
    // The first rows of `count`: from(a, i) is row i of matrix a.
    template <typename From>
    __device__ __forceinline__ void begin(int32_t count, From&& from) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
            if (i < count)
#pragma unroll
                for (int a = 0; a < N; ++a) put(i, a, from(a, i));
            ptx::cp_async_commit();
        }
    }
    // use(i, vectors) for each row in turn, after begin with at least as many.
    template <typename From, typename Use>
    __device__ __forceinline__ void run(int32_t count, From&& from, Use&& use) {
        int32_t s = 0;
#pragma unroll 2
        for (int32_t i = 0; i < count; ++i) {
            ptx::cp_async_wait_group<D - 1>();
            P q[N];
#pragma unroll
            for (int a = 0; a < N; ++a) q[a] = *(slots + (s * N + a) * threads);
            use(i, q);
            if (i + D < count)
#pragma unroll
                for (int a = 0; a < N; ++a) put(s, a, from(a, i + D));
            ptx::cp_async_commit();
            s = s + 1 == D ? 0 : s + 1;
        }
        ptx::cp_async_wait_all();   // (what was begun past `count`)
    }
};
constexpr int kDeep = 6;         // rows of one matrix ahead
constexpr int kDeepGrad = 4;     // of two

// Rows of no scan, by the block.
template <typename P>
__device__ __forceinline__ void zero_rows(const Shape& h, void* out, int32_t lo, int32_t hi) {
    const P zero = {};
    for (int64_t i = static_cast<int64_t>(lo) * h.vectors + threadIdx.x; i < static_cast<int64_t>(hi) * h.vectors; i += blockDim.x)
        static_cast<P*>(out)[i] = zero;
}

// The group of channel v W + j, given that of the channel before it.
template <int W>
__device__ __forceinline__ int32_t group_of(const Shape& h, int32_t v, int j, int32_t before) {
    if (j & ((1 << h.shift) - 1)) return before;
    return h.by_wide((v * W + j) >> h.shift);
}

// ---- forward ------------------------------------------------------------------
struct NormPass {
    GroupNormArgs a;
    Shape h;
    Scans scans;
    float2* part;        // of each piece: mean, sum of squares about it
    const float2* stats; // [scans][groups], or null: the second kernel adds up the pieces
    int32_t* status;
};

// A thread's sums of its channels, about its first value of each, so that a mean
// far from zero costs no digits.
template <int W>
struct Moments {
    Values<W> first, sum, sq;
    template <typename P>
    __device__ __forceinline__ void begin(const P& q) {
        float f[W];
        first.unpack(q);
        first.get(f);
#pragma unroll
        for (int j = 0; j < W; ++j) f[j] = -f[j];
        first.put(f);   // (negated: it is added)
        sum.set(0.0f);
        sq.set(0.0f);
    }
    template <typename P>
    __device__ __forceinline__ void add(const P& q) {
        Values<W> x;
        x.unpack(q);
#pragma unroll
        for (int j = 0; j < Values<W>::n; ++j) {
            const auto d = x.v[j] + first.v[j];
            sum.v[j] = sum.v[j] + d;
            sq.v[j] = fma_v(d, d, sq.v[j]);
        }
    }
    // n rows: joins the channels of a group that lie in the vector, and writes mean and
    // sum of squares about it of each, from entry `at` on
    __device__ __forceinline__ void write(float n, int shift, float* sh_mean, float* sh_m2, int32_t at) const {
        float mean[W], m2[W], s[W], q[W];
        const float by_n = 1.0f / n;
        first.get(mean);
        sum.get(s);
        sq.get(q);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float m = s[j] * by_n;   // of x - first
            mean[j] = m - mean[j];
            const float v = fmaf(-m, s[j], q[j]);
            m2[j] = v < 0.0f ? 0.0f : v;   // (keeps NaN)
        }
#pragma unroll
        for (int l = 0; (1 << l) < W; ++l)
            if (shift > l) {
#pragma unroll
                for (int j = 0; j < W; j += 2 << l) {
                    const float d = mean[j + (1 << l)] - mean[j];
                    mean[j] = fmaf(0.5f, d, mean[j]);
                    m2[j] += fmaf(0.5f * n * static_cast<float>(1 << l) * d, d, m2[j + (1 << l)]);
                }
            }
#pragma unroll
        for (int j = 0; j < W; ++j)
            if ((j & ((1 << shift) - 1)) == 0) {
                sh_mean[at + (j >> shift)] = mean[j];
                sh_m2[at + (j >> shift)] = m2[j];
            }
    }
};

// Rows of the block's threads: each of the first `extra` of `ty` has one more.
struct Deal {
    int32_t rows, each, extra, deep;
    __device__ __forceinline__ Deal(int32_t rows_, const Shape& h)
        : rows(rows_), each(h.by_ty(rows_)), extra(rows_ - each * h.ty), deep(rows_ < h.ty ? rows_ : h.ty) {}
    __device__ __forceinline__ int32_t of(int32_t t) const { return each + (t < extra); }
};

// What the threads wrote, joined about each group's mean in two passes over shared
// memory, by as many lanes a group as it has entries for: f(group, mean, sum of
// squares) by one of them.
template <typename F>
__device__ __forceinline__ void join_threads(const Shape& h, const Deal& deal, const float* sh_mean, const float* sh_m2, F&& f) {
    const int lane = threadIdx.x & 31;
    const int32_t entries = h.c >> h.shift, wide = h.width >> h.shift, count = deal.deep * wide, lanes = h.lanes;
    const float by_count = 1.0f / (static_cast<float>(deal.rows) * static_cast<float>(h.width)), joined = static_cast<float>(1 << h.shift);
    const int32_t log = 31 - __clz(lanes), per = 32 >> log, i0 = lane & (lanes - 1);
    auto sum_lanes = [&](float v) {
        for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        return v;
    };
    for (int32_t g0 = (threadIdx.x >> 5) * per; g0 < h.groups; g0 += (blockDim.x >> 5) * per) {
        const int32_t g = g0 + (lane >> log);
        const bool live = g < h.groups;
        const float base = live ? sh_mean[g * wide] : 0.0f;
        float sum = 0.0f, m2 = 0.0f;
        auto entries_of = [&](auto&& each) {
            if (live)
                for (int32_t i = i0; i < count; i += lanes) {
                    const int32_t t = h.by_wide(i);
                    each(t * entries + g * wide + (i - t * wide), static_cast<float>(deal.of(t)) * joined);
                }
        };
        entries_of([&](int32_t i, float n) { sum = fmaf(n, sh_mean[i] - base, sum); });
        const float mean = base + sum_lanes(sum) * by_count;
        entries_of([&](int32_t i, float n) {
            const float d = sh_mean[i] - mean;
            m2 += fmaf(n * d, d, sh_m2[i]);
        });
        m2 = sum_lanes(m2);
        if (live && i0 == 0) f(g, mean, m2);
    }
}

// act(norm) of one vector
template <int W>
struct Affine {
    Values<W> mean, scale, bias;   // (mean negated)
    __device__ __forceinline__ void load(const NormPass& p, const float2* stats, int32_t v) {
        float m[W], s[W], b[W];
        int32_t g = 0;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            g = group_of<W>(p.h, v, j, g);
            const float2 st = stats[g];
            m[j] = -st.x;
            s[j] = st.y * __ldg(p.a.weight + v * W + j);
            b[j] = p.a.bias ? __ldg(p.a.bias + v * W + j) : 0.0f;
        }
        mean.put(m);
        scale.put(s);
        bias.put(b);
    }
    template <int ACT, typename P>
    __device__ __forceinline__ P apply(const P& q) const {
        Values<W> x;
        x.unpack(q);
#pragma unroll
        for (int j = 0; j < Values<W>::n; ++j) x.v[j] = act_f<ACT>(fma_v(x.v[j] + mean.v[j], scale.v[j], bias.v[j]));
        P o;
        x.pack(o);
        return o;
    }
};

// Statistics of the block's pieces.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads, 2) k_group_stats(const __grid_constant__ NormPass p) {
    using P = Pack<T, W>;
    extern __shared__ __align__(16) uint8_t sh_raw[];
    Stream<P, 1, kDeep> stream(sh_raw);
    float* sh = reinterpret_cast<float*>(sh_raw + stream.bytes(blockDim.x));
    const Shape& h = p.h;
    const int32_t entries = h.c >> h.shift;
    float* sh_mean = sh;                                            // [ty][entries]
    float* sh_m2 = sh + static_cast<size_t>(h.ty) * entries;
    const int ty = h.by_tx(threadIdx.x), tx = threadIdx.x - ty * h.tx;
    const int32_t row0 = static_cast<int32_t>(blockIdx.x) * h.rows;
    const int32_t row1 = row0 + h.rows < p.scans.n ? row0 + h.rows : p.scans.n;
    const T* x0 = static_cast<const T*>(p.a.x);
    pdl_wait();
    pdl_trigger();
    // the first rows are on their way while the offsets are read
    auto rows_from = [&](int32_t first, int32_t v) {
        return [=, &p, &h](int, int32_t i) { return reinterpret_cast<const P*>(x0 + v * W + (first + ty + i * h.ty) * p.a.ldx); };
    };
    if (ty < h.ty) stream.begin(Deal(row1 - row0, h).of(ty), rows_from(row0, tx));
    p.scans.pieces(row0, row1, [&](int32_t s, int32_t lo, int32_t hi) {
        if (s < 0 || s >= p.scans.scans) return;
        const Deal deal(hi - lo, h);
        for (int32_t v = tx; v < h.vectors && ty < deal.deep; v += h.tx) {
            const auto from = rows_from(lo, v);
            if (lo != row0 || v != tx) {
                ptx::cp_async_wait_all();
                stream.begin(deal.of(ty), from);
            }
            Moments<W> m;
            stream.run(deal.of(ty), from, [&](int32_t i, const P (&q)[1]) {
                if (i == 0) m.begin(q[0]);
                m.add(q[0]);
            });
            m.write(static_cast<float>(deal.of(ty)), h.shift, sh_mean, sh_m2, ty * entries + ((v * W) >> h.shift));
        }
        __syncthreads();
        join_threads(h, deal, sh_mean, sh_m2, [&](int32_t g, float mean, float m2) {
            p.part[slot_of(h, g, s)] = make_float2(mean, m2);
        });
        __syncthreads();
    });
    ptx::cp_async_wait_all();
}

// The pieces of a scan's group: mean and 1 / sqrt(var + eps) for all of the warp.
__device__ __forceinline__ float2 join_pieces(const NormPass& p, int32_t g, int32_t s, int32_t lo, int32_t hi) {
    const float width = static_cast<float>(p.h.width), by_count = 1.0f / (static_cast<float>(hi - lo) * width);
    PieceSet set;
    set.load(p.h, p.part, g, s, lo, hi);
    const float base = __shfl_sync(0xFFFFFFFFu, set.v[0].x, 0);
    float sum = 0.0f, m2 = 0.0f;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) sum = fmaf(set.rows[k] * width, set.rows[k] > 0.0f ? set.v[k].x - base : 0.0f, sum);
    const float mean = base + warp_sum(sum) * by_count;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
        const float d = set.rows[k] > 0.0f ? set.v[k].x - mean : 0.0f;
        m2 += fmaf(set.rows[k] * width * d, d, set.v[k].y);
    }
    return make_float2(mean, rsqrtf(warp_sum(m2) * by_count + p.a.eps));
}

// The rows again.
template <typename T, int W>
__global__ void __launch_bounds__(kApplyThreads, 2) k_group_apply(const __grid_constant__ NormPass p) {
    using P = Pack<T, W>;
    extern __shared__ __align__(16) uint8_t sh_raw[];
    Stream<P, 1, kDeep> stream(sh_raw);
    float2* sh_stats = reinterpret_cast<float2*>(sh_raw + stream.bytes(blockDim.x));   // [groups]
    const Shape& h = p.h;
    const GroupNormArgs& a = p.a;
    const int ty = h.by_tx(threadIdx.x), tx = threadIdx.x - ty * h.tx, lane = threadIdx.x & 31;
    const int32_t block = p.stats ? h.blocks - 1 - static_cast<int32_t>(blockIdx.x) : static_cast<int32_t>(blockIdx.x);
    const int32_t row0 = block * h.rows;
    const int32_t row1 = row0 + h.rows < p.scans.n ? row0 + h.rows : p.scans.n;
    const T* x0 = static_cast<const T*>(a.x);
    T* out = static_cast<T*>(a.out);
    // The kernel before this one began once all before it had ended, so what the caller
    // gave may be read already; only the pieces' sums and what is written here wait.
    auto rows_from = [&](int32_t first, int32_t v) {
        return [=, &a, &h](int, int32_t i) { return reinterpret_cast<const P*>(x0 + v * W + (first + ty + i * h.ty) * a.ldx); };
    };
    if (ty < h.ty) stream.begin(Deal(row1 - row0, h).of(ty), rows_from(row0, tx));
    bool waited = false;
    auto wait = [&]() {
        if (!waited) {
            pdl_wait();
            pdl_trigger();
        }
        waited = true;
    };
    p.scans.pieces(row0, row1, [&](int32_t s, int32_t lo, int32_t hi) {
        if (s < 0 || s >= p.scans.scans) {
            wait();
            zero_rows<P>(h, out, lo, hi);
            return;
        }
        const int32_t s_lo = p.scans.at(s), s_hi = p.scans.at(s + 1);
        wait();
        __syncthreads();   // (the last piece's statistics have been read)
        if (p.stats) {
            for (int32_t g = threadIdx.x; g < h.groups; g += blockDim.x) sh_stats[g] = __ldcg(p.stats + static_cast<int64_t>(s) * h.groups + g);
        } else {
            for (int32_t g = threadIdx.x >> 5; g < h.groups; g += blockDim.x >> 5) {
                const float2 st = join_pieces(p, g, s, s_lo, s_hi);
                if (lane == 0) {
                    sh_stats[g] = st;
                    if (a.stats && lo == s_lo) a.stats[static_cast<int64_t>(s) * h.groups + g] = st;
                }
            }
        }
        __syncthreads();
        const Deal deal(hi - lo, h);
        with_act(a.act, [&](auto act) {
            for (int32_t v = tx; v < h.vectors && ty < deal.deep; v += h.tx) {
                const auto from = rows_from(lo, v);
                if (lo != row0 || v != tx) {
                    ptx::cp_async_wait_all();
                    stream.begin(deal.of(ty), from);
                }
                Affine<W> f;
                f.load(p, sh_stats, v);
                P* y = reinterpret_cast<P*>(out + static_cast<int64_t>(lo + ty) * h.c + v * W);
                const int64_t step = static_cast<int64_t>(h.ty) * h.vectors;
                stream.run(deal.of(ty), from, [&](int32_t, const P (&q)[1]) {
                    *y = f.template apply<act>(q[0]);
                    y += step;
                });
            }
        });
    });
    ptx::cp_async_wait_all();
    wait();
    if (p.scans.offsets) {
        // borders out of order or range; what the scans without a row have for statistics
        for (int32_t s = blockIdx.x * blockDim.x + threadIdx.x; s < p.scans.scans; s += gridDim.x * blockDim.x) {
            const int32_t lo = p.scans.raw(s), hi = p.scans.raw(s + 1);
            if (lo > hi || lo < 0 || hi > p.scans.n) atomicOr(p.status, kStatusRange);
            if (a.stats && !p.stats && p.scans.at(s) >= p.scans.at(s + 1))
                for (int32_t g = 0; g < h.groups; ++g)
                    a.stats[static_cast<int64_t>(s) * h.groups + g] = make_float2(0.0f, rsqrtf(a.eps));
        }
    }
}

// Between the two for large inputs: THREADS (32 or 256) a scan and group.
__device__ __forceinline__ float2 sum_of(float2 v, float2* sh, int threads) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (threads == 32) return v;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float2 r = sh[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        r.x += sh[i].x;
        r.y += sh[i].y;
    }
    return r;
}
template <int THREADS>
__global__ void __launch_bounds__(256) k_group_join(const __grid_constant__ NormPass p, float2* stats) {
    __shared__ float2 sh[8];
    const int64_t i = static_cast<int64_t>(blockIdx.x) * (256 / THREADS) + threadIdx.x / THREADS;
    pdl_wait();
    pdl_trigger();
    if (i >= static_cast<int64_t>(p.scans.scans) * p.h.groups) return;   // (all threads of a scan and group)
    const int32_t s = static_cast<int32_t>(i / p.h.groups), g = static_cast<int32_t>(i - static_cast<int64_t>(s) * p.h.groups);
    const int32_t lo = p.scans.at(s), hi = p.scans.at(s + 1), t = threadIdx.x % THREADS, rows = p.h.rows;
    if (lo >= hi) {
        if (t == 0) stats[i] = make_float2(0.0f, rsqrtf(p.a.eps));
        return;
    }
    const int32_t b0 = lo / rows, b1 = (hi - 1) / rows;
    const float2* part = p.part + g * p.h.slots + s;
    const float base = __ldcg(part + b0).x, width = static_cast<float>(p.h.width);
    const float by_count = 1.0f / (static_cast<float>(hi - lo) * width);
    auto values = [&](int32_t b) {   // of piece b: as many, over all channels of the group
        const int32_t first = b * rows > lo ? b * rows : lo, last = (b + 1) * rows < hi ? (b + 1) * rows : hi;
        return static_cast<float>(last - first) * width;
    };
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int32_t b = b0 + t; b <= b1; b += THREADS) sum.x = fmaf(values(b), __ldcg(part + b).x - base, sum.x);
    const float mean = base + sum_of(sum, sh, THREADS).x * by_count;
    sum = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int32_t b = b0 + t; b <= b1; b += THREADS) {
        const float2 v = __ldcg(part + b);
        const float d = v.x - mean;
        sum.y += fmaf(values(b) * d, d, v.y);
    }
    const float m2 = sum_of(sum, sh, THREADS).y;
    if (t == 0) stats[i] = make_float2(mean, rsqrtf(m2 * by_count + p.a.eps));
}

// A scan's rows by a cluster: the statistics of each CTA's share, joined through
// distributed shared memory, then the rows again from the registers that keep the
// first ones (a longer share is read again).
template <typename T, int W>
__global__ void __launch_bounds__(kThreads, 1) k_group_scan(const __grid_constant__ NormPass p) {
    using P = Pack<T, W>;
    constexpr int KEEP = W == 8 ? 6 : 8, U = 4;   // (registers)
    extern __shared__ __align__(16) float sh[];
    const Shape& h = p.h;
    const GroupNormArgs& a = p.a;
    const int32_t entries = h.c >> h.shift;
    float2* own = reinterpret_cast<float2*>(sh);                    // [groups] of this CTA's rows: mean, sum of squares
    float2* stats = own + h.groups;                                 // [groups]
    float* sh_mean = reinterpret_cast<float*>(stats + h.groups);    // [ty][entries]
    float* sh_m2 = sh_mean + static_cast<size_t>(h.ty) * entries;
    const int ty = h.by_tx(threadIdx.x), tx = threadIdx.x - ty * h.tx;
    const uint32_t rank = ptx::cluster_rank();
    const int32_t size = h.blocks, s = h.by_blocks(static_cast<int32_t>(blockIdx.x));
    const T* x0 = static_cast<const T*>(a.x);
    T* out = static_cast<T*>(a.out);
    pdl_wait();
    pdl_trigger();
    const int32_t lo = p.scans.at(s), hi = p.scans.at(s + 1);
    if (p.scans.offsets) {
        if (rank == 0 && threadIdx.x == 0) {
            const int32_t l = p.scans.raw(s), u = p.scans.raw(s + 1);
            if (l > u || l < 0 || u > p.scans.n) atomicOr(p.status, kStatusRange);
        }
        // rows of no scan, a share each
        const int32_t before = p.scans.at(0), after = p.scans.at(p.scans.scans), skip = after > before ? after - before : 0;
        if (const int32_t rest = p.scans.n - skip; rest > 0) {
            const int32_t blocks = static_cast<int32_t>(gridDim.x), share = (rest + blocks - 1) / blocks;
            const int32_t z0 = static_cast<int64_t>(blockIdx.x) * share < rest ? static_cast<int32_t>(blockIdx.x) * share : rest;
            const int32_t z1 = z0 + share < rest ? z0 + share : rest;
            if (z0 < before) zero_rows<P>(h, out, z0, z1 < before ? z1 : before);
            if (z1 > before) zero_rows<P>(h, out, (z0 > before ? z0 : before) + skip, z1 + skip);
        }
    }
    if (lo >= hi) {   // (the whole cluster)
        if (a.stats && rank == 0)
            for (int32_t g = threadIdx.x; g < h.groups; g += blockDim.x)
                a.stats[static_cast<int64_t>(s) * h.groups + g] = make_float2(0.0f, rsqrtf(a.eps));
        return;
    }
    const int32_t share = h.by_blocks(hi - lo + size - 1);
    const int32_t r0 = lo + static_cast<int32_t>(rank) * share < hi ? lo + static_cast<int32_t>(rank) * share : hi;
    const int32_t r1 = r0 + share < hi ? r0 + share : hi;
    const Deal deal(r1 - r0, h);
    P keep[KEEP];
    if (ty < deal.deep) load_rows(keep, x0 + tx * W, a.ldx, r0 + ty, h.ty, r1);
    for (int32_t v = tx; v < h.vectors && ty < deal.deep; v += h.tx) {
        const T* x = x0 + v * W;
        Moments<W> m;
        int32_t r = r0 + ty;
        if (v == tx) {
            m.begin(keep[0]);
#pragma unroll
            for (int u = 0; u < KEEP; ++u)
                if (r + u * h.ty < r1) m.add(keep[u]);
            r += KEEP * h.ty;
        } else {
            m.begin(*reinterpret_cast<const P*>(x + r * a.ldx));
        }
        for (; r < r1; r += U * h.ty) {
            P q[U];
            load_rows(q, x, a.ldx, r, h.ty, r1);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * h.ty < r1) m.add(q[u]);
        }
        m.write(static_cast<float>(deal.of(ty)), h.shift, sh_mean, sh_m2, ty * entries + ((v * W) >> h.shift));
    }
    __syncthreads();
    if (r0 < r1)
        join_threads(h, deal, sh_mean, sh_m2, [&](int32_t g, float mean, float m2) {
            own[g] = make_float2(mean, m2);
        });
    if (size > 1) ptx::cluster_sync();
    else __syncthreads();
    for (int32_t g = threadIdx.x; g < h.groups; g += blockDim.x) {
        const float width = static_cast<float>(h.width), by_count = 1.0f / (static_cast<float>(hi - lo) * width);
        float mean = own[g].x, m2 = own[g].y;
        if (size > 1) {
            float2 v[kMaxCluster];
            float n[kMaxCluster];
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) {
                const int32_t left = hi - lo - c * share;
                n[c] = c < size && left > 0 ? static_cast<float>(left < share ? left : share) * width : 0.0f;
                v[c] = n[c] > 0.0f ? ptx::ld_cluster_f32x2(ptx::map_to_rank(ptx::smem_u32(own + g), c)) : make_float2(0.0f, 0.0f);
            }
            float sum = 0.0f;
#pragma unroll
            for (int c = 1; c < kMaxCluster; ++c) sum = fmaf(n[c], n[c] > 0.0f ? v[c].x - v[0].x : 0.0f, sum);
            mean = v[0].x + sum * by_count;
            m2 = 0.0f;
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) {
                const float d = n[c] > 0.0f ? v[c].x - mean : 0.0f;
                m2 += fmaf(n[c] * d, d, v[c].y);
            }
        }
        const float2 st = make_float2(mean, rsqrtf(m2 * by_count + a.eps));
        stats[g] = st;
        if (a.stats && rank == 0) a.stats[static_cast<int64_t>(s) * h.groups + g] = st;
    }
    if (size > 1) ptx::cluster_arrive();   // (its sums are read until all have come here)
    __syncthreads();
    with_act(a.act, [&](auto act) {
        for (int32_t v = tx; v < h.vectors && ty < deal.deep; v += h.tx) {
            const T* x = x0 + v * W;
            Affine<W> f;
            f.load(p, stats, v);
            int32_t r = r0 + ty;
            auto write = [&](int32_t row, const P& q) { *reinterpret_cast<P*>(out + static_cast<int64_t>(row) * h.c + v * W) = f.template apply<act>(q); };
            if (v == tx) {
#pragma unroll
                for (int u = 0; u < KEEP; ++u)
                    if (r + u * h.ty < r1) write(r + u * h.ty, keep[u]);
                r += KEEP * h.ty;
            }
            for (; r < r1; r += U * h.ty) {
                P q[U];
                load_rows(q, x, a.ldx, r, h.ty, r1);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (r + u * h.ty < r1) write(r + u * h.ty, q[u]);
            }
        }
    });
    if (size > 1) ptx::cluster_wait();
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
    int32_t col_blocks;  // the second kernel's first blocks add up cols
    int32_t* status;
};

// What a thread needs of its W channels in a scan.
template <int W>
struct Channels {
    Values<W> mean, r, w, b;   // (mean negated)
    __device__ __forceinline__ void load(const GradPass& p, int32_t s, int32_t v) {
        float fm[W], fr[W], fw[W], fb[W];
        int32_t g = 0;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            g = group_of<W>(p.h, v, j, g);
            const float2 st = __ldg(p.a.stats + static_cast<int64_t>(s) * p.h.groups + g);
            fm[j] = -st.x;
            fr[j] = st.y;
            fw[j] = __ldg(p.a.weight + v * W + j);
            fb[j] = p.a.bias ? __ldg(p.a.bias + v * W + j) : 0.0f;
        }
        mean.put(fm);
        r.put(fr);
        w.put(fw);
        b.put(fb);
    }
    // u of the j-th values (pairs) of x; *dz their gradient
    template <int ACT, typename V>
    __device__ __forceinline__ V unit(int j, V x, V dy, V* dz) const {
        const V u = (x + mean.v[j]) * r.v[j];
        V unused;
        *dz = dy * act_grad_f<ACT>(fma_v(u, w.v[j], b.v[j]), &unused);
        return u;
    }
};

// Sums over a thread's rows of dz u and dz.
template <int W>
struct GradSums {
    Values<W> u, z;
    __device__ __forceinline__ void begin() {
        u.set(0.0f);
        z.set(0.0f);
    }
    template <int ACT, typename P>
    __device__ __forceinline__ void add(const Channels<W>& ch, const P& qx, const P& qd) {
        Values<W> x, d;
        x.unpack(qx);
        d.unpack(qd);
#pragma unroll
        for (int j = 0; j < Values<W>::n; ++j) {
            typename Values<W>::V dz;
            const auto un = ch.template unit<ACT>(j, x.v[j], d.v[j], &dz);
            u.v[j] = fma_v(dz, un, u.v[j]);
            z.v[j] = z.v[j] + dz;
        }
    }
    __device__ __forceinline__ void write(float* sh_u, float* sh_z) const {
        float f[W];
        u.get(f);
#pragma unroll
        for (int j = 0; j < W; ++j) sh_u[j] = f[j];
        z.get(f);
#pragma unroll
        for (int j = 0; j < W; ++j) sh_z[j] = f[j];
    }
};

// The threads' sums: added to the block's totals [2][c], then, times the weight,
// to each group's (group, sum of p, sum of p u) by a warp.  Ends at a barrier.
template <typename F>
__device__ __forceinline__ void join_grad_threads(const GradPass& p, int32_t deep, float* total, float* sh_u, float* sh_z, F&& f) {
    const Shape& h = p.h;
    const int lane = threadIdx.x & 31;
    __syncthreads();
    // down the thread rows: by several threads where a row has fewer channels than the block threads
    const int32_t threads = static_cast<int32_t>(blockDim.x);
    int32_t rows = h.c < threads ? threads / h.c : 1;
    if (rows > deep) rows = deep;
    for (int32_t i = threadIdx.x; i < rows * h.c; i += threads) {
        const int32_t r = i >= h.c ? i / h.c : 0, c = i - r * h.c;
        float u = 0.0f, z = 0.0f;
        for (int32_t t = r; t < deep; t += rows) {
            u += sh_u[t * h.c + c];
            z += sh_z[t * h.c + c];
        }
        sh_u[i] = u;   // (row r, which no other thread reads)
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
    // (as many lanes a group as it has channels, up to a warp)
    const int32_t lanes = h.width >= 32 ? 32 : h.width > 8 ? 16 : h.width > 4 ? 8 : h.width > 1 ? 4 : 1;
    const int32_t k0 = lane & (lanes - 1), per = 32 / lanes;
    for (int32_t g0 = (threadIdx.x >> 5) * per; g0 < h.groups; g0 += (threads >> 5) * per) {
        const int32_t g = g0 + lane / lanes;
        float u = 0.0f, z = 0.0f;
        if (g < h.groups)
            for (int32_t k = k0; k < h.width; k += lanes) {
                u += sh_u[g * h.width + k];
                z += sh_z[g * h.width + k];
            }
        for (int32_t o = lanes >> 1; o > 0; o >>= 1) {
            u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
            z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
        }
        if (g < h.groups && k0 == 0) f(g, z, u);
    }
    __syncthreads();
}

// dx of one vector
template <int W>
struct GradAffine {
    Channels<W> ch;
    Values<W> mz, mu;   // means of p and p u (negated)
    __device__ __forceinline__ void load(const GradPass& p, const float2* means, int32_t s, int32_t v) {
        ch.load(p, s, v);
        float a[W], b[W];
        int32_t g = 0;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            g = group_of<W>(p.h, v, j, g);
            const float2 m = means[g];
            a[j] = -m.x;
            b[j] = -m.y;
        }
        mz.put(a);
        mu.put(b);
    }
    template <int ACT, typename P>
    __device__ __forceinline__ P apply(const P& qx, const P& qd) const {
        Values<W> x, d;
        x.unpack(qx);
        d.unpack(qd);
#pragma unroll
        for (int j = 0; j < Values<W>::n; ++j) {
            typename Values<W>::V dz;
            const auto u = ch.template unit<ACT>(j, x.v[j], d.v[j], &dz);
            x.v[j] = ch.r.v[j] * fma_v(u, mu.v[j], fma_v(dz, ch.w.v[j], mz.v[j]));
        }
        P o;
        x.pack(o);
        return o;
    }
};

template <typename T, int W>
__global__ void __launch_bounds__(kThreads, 1) k_group_grad_sums(const __grid_constant__ GradPass p) {
    using P = Pack<T, W>;
    extern __shared__ __align__(16) uint8_t sh_raw[];
    Stream<P, 2, kDeepGrad> stream(sh_raw);
    float* sh = reinterpret_cast<float*>(sh_raw + stream.bytes(blockDim.x));
    const Shape& h = p.h;
    float* total = sh;                                              // [2][c]: of all pieces
    float* sh_u = sh + 2 * h.c;                                     // [ty][c]: sums of dz u
    float* sh_z = sh_u + static_cast<size_t>(h.ty) * h.c;           // sums of dz
    const int ty = h.by_tx(threadIdx.x), tx = threadIdx.x - ty * h.tx;
    const int32_t row0 = static_cast<int32_t>(blockIdx.x) * h.rows;
    const int32_t row1 = row0 + h.rows < p.scans.n ? row0 + h.rows : p.scans.n;
    const T* x0 = static_cast<const T*>(p.a.x);
    const T* dy0 = static_cast<const T*>(p.a.dy);
    pdl_wait();
    pdl_trigger();
    auto rows_from = [&](int32_t first, int32_t v) {
        return [=, &p, &h](int m, int32_t i) {
            const int32_t row = first + ty + i * h.ty;
            return reinterpret_cast<const P*>(m ? dy0 + v * W + row * p.a.ldy : x0 + v * W + row * p.a.ldx);
        };
    };
    if (ty < h.ty) stream.begin(Deal(row1 - row0, h).of(ty), rows_from(row0, tx));
    for (int32_t i = threadIdx.x; i < 2 * h.c; i += blockDim.x) total[i] = 0.0f;
    p.scans.pieces(row0, row1, [&](int32_t s, int32_t lo, int32_t hi) {
        if (s < 0 || s >= p.scans.scans) return;
        const Deal deal(hi - lo, h);
        with_act(p.a.act, [&](auto act) {
            for (int32_t v = tx; v < h.vectors && ty < deal.deep; v += h.tx) {
                const auto from = rows_from(lo, v);
                if (lo != row0 || v != tx) {
                    ptx::cp_async_wait_all();
                    stream.begin(deal.of(ty), from);
                }
                Channels<W> ch;
                ch.load(p, s, v);
                GradSums<W> sums;
                sums.begin();
                stream.run(deal.of(ty), from, [&](int32_t, const P (&q)[2]) { sums.template add<act>(ch, q[0], q[1]); });
                sums.write(sh_u + ty * h.c + v * W, sh_z + ty * h.c + v * W);
            }
        });
        join_grad_threads(p, deal.deep, total, sh_u, sh_z,
                          [&](int32_t g, float z, float u) { p.part[slot_of(h, g, s)] = make_float2(z, u); });
    });
    ptx::cp_async_wait_all();
    __syncthreads();
    for (int32_t i = threadIdx.x; i < 2 * h.c; i += blockDim.x) p.cols[static_cast<int64_t>(blockIdx.x) * 2 * h.c + i] = total[i];
}

// Columns of the blocks' sums: kColumns of them a block, the other threads down each.
constexpr int kColumns = 8;
__device__ __forceinline__ void add_columns(const GradPass& p, int32_t blocks, float* sh) {
    const int32_t col = static_cast<int32_t>(blockIdx.x) * kColumns + (threadIdx.x & (kColumns - 1));
    const int32_t down = static_cast<int32_t>(blockDim.x) / kColumns;
    float sum = 0.0f;
    if (col < 2 * p.h.c)
#pragma unroll 8
        for (int32_t b = threadIdx.x / kColumns; b < blocks; b += down) sum += __ldcg(p.cols + static_cast<int64_t>(b) * 2 * p.h.c + col);
#pragma unroll
    for (int32_t o = kColumns; o < 32; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if ((threadIdx.x & 31) < kColumns) sh[(threadIdx.x >> 5) * kColumns + (threadIdx.x & 31)] = sum;
    __syncthreads();
    if (threadIdx.x >= kColumns || col >= 2 * p.h.c) return;
    sum = sh[threadIdx.x];
    for (int32_t w = 1; w < static_cast<int32_t>(blockDim.x >> 5); ++w) sum += sh[w * kColumns + threadIdx.x];
    if (col < p.h.c) p.a.dweight[col] = sum;
    else if (p.a.dbias) p.a.dbias[col - p.h.c] = sum;
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads, 1) k_group_grad_apply(const __grid_constant__ GradPass p) {
    using P = Pack<T, W>;
    extern __shared__ __align__(16) uint8_t sh_raw[];
    Stream<P, 2, kDeepGrad> stream(sh_raw);
    float* sh = reinterpret_cast<float*>(sh_raw + stream.bytes(blockDim.x));
    const Shape& h = p.h;
    const GroupNormGradArgs& a = p.a;
    float2* sh_means = reinterpret_cast<float2*>(sh);   // [groups]: of p, of p u
    if (static_cast<int32_t>(blockIdx.x) < p.col_blocks) {
        pdl_wait();
        pdl_trigger();
        add_columns(p, h.blocks, sh);
        return;
    }
    const int ty = h.by_tx(threadIdx.x), tx = threadIdx.x - ty * h.tx, lane = threadIdx.x & 31;
    const int32_t index = static_cast<int32_t>(blockIdx.x) - p.col_blocks;
    const int32_t row0 = index * h.rows;
    const int32_t row1 = row0 + h.rows < p.scans.n ? row0 + h.rows : p.scans.n;
    const T* x0 = static_cast<const T*>(a.x);
    const T* dy0 = static_cast<const T*>(a.dy);
    T* out = static_cast<T*>(a.dx);
    // (as in the forward pass, what the caller gave may be read before the wait)
    auto rows_from = [&](int32_t first, int32_t v) {
        return [=, &p, &h](int m, int32_t i) {
            const int32_t row = first + ty + i * h.ty;
            return reinterpret_cast<const P*>(m ? dy0 + v * W + row * p.a.ldy : x0 + v * W + row * p.a.ldx);
        };
    };
    if (ty < h.ty) stream.begin(Deal(row1 - row0, h).of(ty), rows_from(row0, tx));
    bool waited = false;
    auto wait = [&]() {
        if (!waited) {
            pdl_wait();
            pdl_trigger();
        }
        waited = true;
    };
    p.scans.pieces(row0, row1, [&](int32_t s, int32_t lo, int32_t hi) {
        if (s < 0 || s >= p.scans.scans) {
            wait();
            zero_rows<P>(h, out, lo, hi);
            return;
        }
        const int32_t s_lo = p.scans.at(s), s_hi = p.scans.at(s + 1);
        const float by_count = 1.0f / (static_cast<float>(s_hi - s_lo) * static_cast<float>(h.width));
        wait();
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
            if (lane == 0) sh_means[g] = make_float2(z * by_count, u * by_count);
        }
        __syncthreads();
        const Deal deal(hi - lo, h);
        with_act(a.act, [&](auto act) {
            for (int32_t v = tx; v < h.vectors && ty < deal.deep; v += h.tx) {
                const auto from = rows_from(lo, v);
                if (lo != row0 || v != tx) {
                    ptx::cp_async_wait_all();
                    stream.begin(deal.of(ty), from);
                }
                GradAffine<W> f;
                f.load(p, sh_means, s, v);
                P* dx = reinterpret_cast<P*>(out + static_cast<int64_t>(lo + ty) * h.c + v * W);
                const int64_t step = static_cast<int64_t>(h.ty) * h.vectors;
                stream.run(deal.of(ty), from, [&](int32_t, const P (&q)[2]) {
                    *dx = f.template apply<act>(q[0], q[1]);
                    dx += step;
                });
            }
        });
    });
    ptx::cp_async_wait_all();
    wait();
    if (p.scans.offsets)
        for (int32_t s = index * blockDim.x + threadIdx.x; s < p.scans.scans; s += h.blocks * blockDim.x) {
            const int32_t lo = p.scans.raw(s), hi = p.scans.raw(s + 1);
            if (lo > hi || lo < 0 || hi > p.scans.n) atomicOr(p.status, kStatusRange);
        }
}

// ---- host -----------------------------------------------------------------------
// Vectors of W elements and the rows of a block; large: enough blocks to be taken
// in turn, their pieces added up between.
int set_threads(Shape* h, int most) {
    h->tx = h->vectors < most ? h->vectors : most;
    h->ty = most / h->tx;
    h->by_tx = FastDiv(static_cast<uint32_t>(h->tx));
    h->by_ty = FastDiv(static_cast<uint32_t>(h->ty));
    const int32_t wide = h->width >> h->shift;
    h->by_wide = FastDiv(static_cast<uint32_t>(wide));
    h->lanes = 1;
    while (h->lanes < 32 && h->lanes < h->ty * wide) h->lanes *= 2;
    return static_cast<int>(round_up(static_cast<size_t>(h->tx) * h->ty, 32));
}
Shape make_shape(int64_t n, int32_t c, int32_t groups, int64_t scans, int w, size_t es, bool large, int* threads) {
    Shape h = {};
    h.c = c;
    h.groups = groups;
    h.width = c / groups;
    h.vectors = c / w;
    while ((2 << h.shift) <= w && h.width % (2 << h.shift) == 0) ++h.shift;
    *threads = set_threads(&h, large ? kThreads / 2 : kThreads);
    int64_t blocks = ceil_div(n, static_cast<int64_t>(4) * h.ty);   // (one step of loads each, at least)
    int64_t limit = large ? ceil_div(n * c * static_cast<int64_t>(es), kBlockBytes) : kSms;
    if (large && limit < 4 * kSms) limit = 4 * kSms;
    if (blocks > limit) blocks = limit;
    h.rows = static_cast<int32_t>(ceil_div(n, blocks));
    h.blocks = static_cast<int32_t>(ceil_div(n, h.rows));
    h.slots = h.blocks + scans;
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

// The kernel between the two: a warp a scan and group, or a block where a scan
// has many pieces (one scan of 512 MB: 249 us with blocks and 279 with warps in
// all; 64 scans of as much 247 either way).
int launch_join(const NormPass& p, float2* to, cudaStream_t s) {
    const int64_t count = static_cast<int64_t>(p.scans.scans) * p.h.groups;
    const bool many = p.h.blocks / p.scans.scans > 64;
    const int64_t blocks = many ? count : ceil_div(count, 8);
    if (blocks > 0x7FFFFFFF) return SPCONV_ERR_UNSUPPORTED;
    return launch_pdl(many ? k_group_join<256> : k_group_join<32>, dim3(static_cast<unsigned>(blocks)), 256, 0, s, p, to);
}

template <auto KERNEL, typename A>
int launch_clusters(int64_t blocks, int cluster, int threads, size_t smem, cudaStream_t s, const A& args) {
    if (blocks > 0x7FFFFFFF) return SPCONV_ERR_UNSUPPORTED;
    static bool set[kMaxDevices] = {};
    int dev = 0;
    SPCONV_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return SPCONV_ERR_UNSUPPORTED;
    if (!set[dev]) {
        SPCONV_CHECK_CUDA(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024));
        set[dev] = true;
    }
    cudaLaunchAttribute at[2] = {pdl_attr(), {}};
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    count_launch();
    return cuda_status(cudaLaunchKernelEx(&cfg, KERNEL, args));
}

// CTAs of a cluster that takes a scan of average size whole, with at most `keep`
// bytes each while there are CTAs; 0: too large, or so many CTAs that they run in
// turns.  (us, bf16, 128 channels, clusters and pieces: 160 scans of 32 kB 9 and 23,
// of 128 kB 24 and 31, of 256 kB 45 and 39; 600 of 64 kB 36 and 54, of 128 kB 83 and
// 53; one of 512 kB 10.4 and 11.3, 40 of them 25 and 26.)
int scan_cluster(int64_t bytes, int64_t scans, int64_t keep) {
    const int64_t each = ceil_div(bytes, scans);
    if (each > kScanBytes) return 0;
    int size = 1;
    while (size < kMaxCluster && each > size * keep) size *= 2;
    return each <= 2 * keep || scans * size <= 5 * kSms ? size : 0;
}

template <typename T, int W>
int forward_w(const GroupNormArgs& a, cudaStream_t s) {
    NormPass p = {};
    p.a = a;
    int threads = 0;
    const int64_t bytes = a.n * a.c * static_cast<int64_t>(sizeof(T));
    const bool large = a.scans > 1 || bytes > kSmallBytes;
    if (const int size = scan_cluster(bytes, a.scans, 32 << 10)) {
        p.h = make_shape(a.n, a.c, a.groups, a.scans, W, sizeof(T), false, &threads);
        // (half as many where two CTAs then share an SM: 300000 rows in 160 scans 69 us, not 123;
        // one scan of 3000 x 64 8.0, not 7.2)
        threads = set_threads(&p.h, a.scans * size <= kSms ? kThreads : kThreads / 2);
        p.h.blocks = size;
        p.h.by_blocks = FastDiv(static_cast<uint32_t>(size));
        p.scans = Scans{a.offsets, static_cast<int32_t>(a.scans), static_cast<int32_t>(a.n)};
        SPCONV_CHECK(rows_status_word(&p.status));
        const size_t smem = static_cast<size_t>(4) * a.groups * 4 + static_cast<size_t>(2) * p.h.ty * (a.c >> p.h.shift) * 4;
        return launch_clusters<k_group_scan<T, W>>(a.scans * size, size, threads, smem, s, p);
    }
    p.h = make_shape(a.n, a.c, a.groups, a.scans, W, sizeof(T), large, &threads);
    p.scans = Scans{a.offsets, static_cast<int32_t>(a.scans), static_cast<int32_t>(a.n)};
    SPCONV_CHECK(rows_status_word(&p.status));
    const size_t part_bytes = round_up(static_cast<size_t>(p.h.slots) * a.groups * sizeof(float2), 256);
    const size_t stats_bytes = large && !a.stats ? static_cast<size_t>(a.scans) * a.groups * sizeof(float2) : 0;
    Scratch part(part_bytes + stats_bytes, s);
    if (part.failed()) return SPCONV_ERR_OOM;
    p.part = part.as<float2>();
    using Rows1 = Stream<Pack<T, W>, 1, kDeep>;
    SPCONV_CHECK((launch_wide<k_group_stats<T, W>>(p.h.blocks, threads, Rows1::bytes(threads) + static_cast<size_t>(2) * p.h.ty * (a.c >> p.h.shift) * 4, s, p)));
    if (large) {
        float2* stats = a.stats ? a.stats : part.as<float2>(part_bytes);
        SPCONV_CHECK(launch_join(p, stats, s));
        p.stats = stats;
    }
    threads = set_threads(&p.h, large ? kApplyThreads / 2 : kApplyThreads);
    return launch_wide<k_group_apply<T, W>>(p.h.blocks, threads, Rows1::bytes(threads) + static_cast<size_t>(2) * a.groups * 4, s, p);
}

template <typename T, int W>
int backward_w(const GroupNormGradArgs& a, cudaStream_t s) {
    GradPass p = {};
    p.a = a;
    int threads = 0;
    p.h = make_shape(a.n, a.c, a.groups, a.scans, W, sizeof(T), false, &threads);
    p.scans = Scans{a.offsets, static_cast<int32_t>(a.scans), static_cast<int32_t>(a.n)};
    SPCONV_CHECK(rows_status_word(&p.status));
    const size_t part_bytes = round_up(static_cast<size_t>(p.h.slots) * a.groups * sizeof(float2), 256);
    Scratch buf(part_bytes + static_cast<size_t>(p.h.blocks) * 2 * a.c * 4, s);
    if (buf.failed()) return SPCONV_ERR_OOM;
    p.part = buf.as<float2>();
    p.cols = buf.as<float>(part_bytes);
    using Rows2 = Stream<Pack<T, W>, 2, kDeepGrad>;
    SPCONV_CHECK((launch_wide<k_group_grad_sums<T, W>>(p.h.blocks, threads, Rows2::bytes(threads) + static_cast<size_t>(2) * (p.h.ty + 1) * a.c * 4, s, p)));
    p.col_blocks = static_cast<int32_t>(ceil_div(2 * a.c, kColumns));
    size_t smem = static_cast<size_t>(2) * a.groups * 4;
    if (smem < kThreads * 4) smem = kThreads * 4;
    return launch_wide<k_group_grad_apply<T, W>>(p.h.blocks + p.col_blocks, threads, Rows2::bytes(threads) + smem, s, p);
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
