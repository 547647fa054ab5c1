// Products of e4m3 operands with a scale for each block of 128, and of sorted
// rows with the weights of their experts.
//
//   z[i][o] = sum_b xs[b][i] ws[o / 128][b] sum_{k in block b} x[i][k] W[o][k]
//
// The tensor cores sum one block of 128 at a time into TMEM (fp32); the scales
// differ from block to block, so the block's sums are read back, scaled and added
// up in registers: one fp32 multiply-add a sum and block.
//
// A pair of CTAs works on a tile of 256 rows by 256 columns (gated: 128 of the
// gate's weight and the same 128 of the up weight), CTA rank r bringing 128 rows of
// x and 128 of W.  Two accumulators of 256 columns take turns: while the tensor
// pipe fills one with a block of K (4 MMAs, 512 clocks at the e4m3 rate), eight
// warps add the other to their registers (128 sums a thread; 256 clocks of TMEM
// loads and as many of packed multiply-adds over an SM).  (Halves of 128 columns,
// which would leave more time between a half's last MMA and its next, are slower:
// shared memory then has to feed the pipe 1.5 times as much; 162 us, not 123, for
// 8192 x 4096 x 4096 with one of the first forms.)
//
// What bounds it: in the main loop the chain of a block's commit, its adding up, the
// arrival and the issue of the next but one (790 clocks a block, not 512: 8192 x
// 4096 x 4096 106 us, 2.6 PFLOP/s; 8192^3 405 to 417 us, 327 without the adding up); between
// tiles the epilogue, which nothing hides because the sums fill the registers (plain
// 3000 clocks, GELU 9000: 123 us with it, with a bias too 128, SiLU 117, residual 129;
// gated 207, to e4m3 211).
// Much of that is waiting for instructions: it is run once a tile.
//
// Sorted rows: expert e's rows are offsets[e] .. offsets[e + 1] - 1, and its
// weight rows e H .. (e + 1) H - 1 of the stacked weights.  The offsets stay on
// the device: each CTA sums up the experts' row tiles and looks its tiles up.  A
// tile reads past its expert's rows and columns (whatever is there, or zeros
// behind the last) and stores only its own.
#include "ptx_sm100.cuh"
#include "row_vectors.cuh"
#include "tensor_map.cuh"

namespace spconv {
namespace {

constexpr int kPairs = 76;
constexpr int kGroupM = 16;              // row tiles that share the column tiles in L2
constexpr int kStageA = 128 * 128, kStage = 2 * kStageA;
constexpr int kStages = 5;
constexpr int kEpiWarps = 8;
constexpr int kFirstEpi = 4;             // warp 0 loads, warp 1 issues MMAs, warp 3 brings scales, warps 4 .. 11 add up
constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
constexpr int kStaging = 32 * 128;       // of an epilogue warp: twice 32 rows of 32 bf16, or 32 of 128 e4m3
constexpr int kScaleSlots = 4;           // blocks of K whose scales lie in shared memory: [2 blocks of columns][128 rows] each
constexpr int kBiasSlots = 4;            // tiles whose bias lies in shared memory: [256 columns] each
constexpr int kScaleBytes = kScaleSlots * 2 * 128 * 4 + kBiasSlots * 256 * 4 + kEpiWarps * 16;   // (and the epilogue warps' tiles)
// Registers a thread: 168 at the launch (three warps on each quarter of an SM), then
// 80 for the first four warps and 208 for the others (bf16 results of one product,
// which have a residual on its way: 56 and 224): where neither side spills.
template <bool DUAL, bool EIGHT>
struct Regs {
    static constexpr int first = DUAL || EIGHT ? 80 : 56, epi = DUAL || EIGHT ? 208 : 224;
    static_assert(128 * first + 32 * kEpiWarps * epi <= kThreads * 168, "register split");
};
constexpr int kTableSize = 256;
constexpr int kSmem = 1024 + kStages * kStage + kEpiWarps * kStaging + kScaleBytes + 256 + 4 * (kTableSize + 1);
static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
static_assert(ptx::tmem_fits(kSmem, 512), "TMEM of an SM");

// Experts' runs of rows, in order and range whatever the offsets hold.
struct Runs {
    const int32_t* offsets;   // [count + 1] or null: one run of all rows
    int32_t count;
    int32_t n;
    __device__ __forceinline__ void get(int32_t e, int32_t& lo, int32_t& hi) const {
        lo = 0;
        hi = n;
        if (!offsets) return;
        lo = __ldg(offsets + e);
        hi = __ldg(offsets + e + 1);
        lo = lo < 0 ? 0 : lo > n ? n : lo;
        hi = hi < lo ? lo : hi > n ? n : hi;
    }
    // Borders out of order or range; by any number of threads.
    __device__ __forceinline__ void check(int32_t first, int32_t step, int32_t* status) const {
        if (!offsets) return;
        for (int32_t e = first; e < count; e += step) {
            const int32_t lo = __ldg(offsets + e), hi = __ldg(offsets + e + 1);
            if (lo > hi || lo < 0 || hi > n) atomicOr(status, kStatusRange);
        }
    }
};

struct BlockArgs {
    CUtensorMap x, w[2], c, map_extra;   // c: of out, where map_out; map_extra: where vec_extra
    Runs runs;
    int32_t h;                // columns of an expert's weight
    int32_t kb;               // blocks of K
    int32_t hb;               // blocks of columns
    int32_t act;
    const float* x_scale;     // [kb][n]
    const float* w_scale[2];  // [experts][hb][kb]
    const float* bias;        // [experts][h] or null
    const __nv_bfloat16* extra;   // [n] rows of h, or null
    int64_t ld_extra;
    void* out;                // bf16 [n] rows of h; or e4m3 [n][h] with scale
    int64_t ld_out;
    float* scale;             // [hb][n]
    int32_t vec_out, vec_extra;   // rows take 16-byte stores, loads
    int32_t map_out;
    int32_t* status;
};

// Rows of no expert are zeros: before the first run, behind the last.
template <bool EIGHT>
__device__ __forceinline__ void zero_rest(const BlockArgs& p, int64_t first, int64_t step) {
    if (!p.runs.offsets) return;
    int32_t from = __ldg(p.runs.offsets), to = __ldg(p.runs.offsets + p.runs.count);
    from = from < 0 ? 0 : from > p.runs.n ? p.runs.n : from;
    to = to < from ? from : to > p.runs.n ? p.runs.n : to;
    const int64_t rows = from + (p.runs.n - to);
#pragma unroll 1
    for (int64_t i = first; i < rows * p.h; i += step) {
        const int64_t r = i / p.h, row = r < from ? r : to + (r - from);
        if (EIGHT) static_cast<uint8_t*>(p.out)[row * p.ld_out + i % p.h] = 0;
        else static_cast<__nv_bfloat16*>(p.out)[row * p.ld_out + i % p.h] = __float2bfloat16_rn(0.0f);
    }
    if (EIGHT)
#pragma unroll 1
        for (int64_t i = first; i < rows * p.hb; i += step) {
            const int64_t r = i / p.hb, row = r < from ? r : to + (r - from);
            p.scale[i % p.hb * p.runs.n + row] = 0.0f;
        }
}

// 1 / s rounded towards zero, from the nearest.
__device__ __forceinline__ float inverse_towards_zero(float s, float nearest) {
    return fmaf(-s, nearest, 1.0f) < 0.0f ? __uint_as_float(__float_as_uint(nearest) - 1) : nearest;
}

// The quotients of a block's values and its scale s (largest magnitude / 448), of which
// e4m3(v / s) is formed with both divisions rounded to nearest, as spconv_quantize_blocks
// has them.  1 / s is held in two parts, y rounded towards zero and y2 = (1 - s y) y, whose
// first factor is exact; neither is negative, so a zero keeps its sign.  v y + v y2, rounded
// once by the multiply-add, is v / s (1 + e) before that rounding, with e at most 1.5 2^-46
// (y2) + 2^-47 (v y2) = 2^-45.  What the e4m3 value turns on is on which side of T + 2^-24
// and of T - 2^-24 v / s lies, T the middle of two e4m3 values, t sixteenths in [1, 2)
// (powers of two aside; where T is one, T - 2^-25).  With s = B 2^-23 and v = A 2^-23, 24
// bits each, v differs from s (T +- 2^-24) by N 2^-47, N = A 2^24 - B (t 2^20 +- 1), so N =
// -+B modulo 2^20, and |N| > 16 is more than e can pass over (s T < 4).
//
// That fails for scales whose last 20 bits are near 0 (20 is kept), but not 0, and says nothing
// of those far from 1: those rows take AnyQuotient.  (Measured: 8192 x 4096 x 4096 gated
// 208 us, with one product by 448 / max, which gives other values near T, 208; 32 experts'
// rows, 2048 x 1408, 178 and 175.  A division a value where both a product with a little
// less and one with a little more than 1 / s do not agree: 214 and 183.)
struct Quotient {
    F2 y, y2;
    bool serves;
    __device__ __forceinline__ explicit Quotient(float s) {
        const uint32_t last = __float_as_uint(s) & 0xFFFFFu;
        serves = s == 0.0f || (s >= 0x1p-60f && s <= 0x1p60f && (last == 0 || ((last + 20) & 0xFFFFFu) > 40));
        const float inverse = s == 0.0f ? 0.0f : inverse_towards_zero(s, __fdiv_rn(1.0f, s));
        y = F2(inverse);
        y2 = F2(fmaf(-s, inverse, 1.0f) * inverse);
    }
    __device__ __forceinline__ F2 operator()(F2 v) const { return fma_v(v, y, v * y2); }
};

// For every scale: the step that makes a quotient q within a unit in the last place the
// rounded one, q + (v - s q) y, y = 1 / s rounded to nearest (P. Markstein, IBM Journal of
// Research and Development 34, 1990), with s and v times a power of two that keeps every
// factor in fp32's range.
struct AnyQuotient {
    F2 s, pre, y, y2, nearest;   // (pre and the inverses negated: with v - s q the other way about a zero keeps its sign here too)
    __device__ __forceinline__ explicit AnyQuotient(float scale) {
        const bool infinite = scale == __int_as_float(0x7F800000);   // (0 for what is finite, NaN for the infinities)
        const float by = scale < 0x1p-60f ? 0x1p100f : scale > 0x1p60f ? 0x1p-60f : 1.0f, d = scale * by;
        const float n = scale == 0.0f ? 0.0f : __fdiv_rn(1.0f, d), z = inverse_towards_zero(d, n);
        s = F2(infinite ? 0.0f : d);
        pre = F2(-by);
        y = F2(-z);
        y2 = F2(infinite ? -0.0f : -fmaf(-d, z, 1.0f) * z);
        nearest = F2(-n);
    }
    __device__ __forceinline__ F2 operator()(F2 v) const {
        v = v * pre;
        const F2 q = fma_v(v, y, v * y2);
        return fma_v(fma_v(q, s, v), nearest, q);
    }
};

// Four values; a block of zeros (scale 0) is +0.
template <typename Q>
__device__ __forceinline__ uint32_t to_e4m3(const Q& quotient, float scale, F2 ab, F2 cd) {
    float a, b, c, d;
    quotient(ab).get(a, b);
    quotient(cd).get(c, d);
    const uint32_t q = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
                       static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3)) << 16;
    return scale == 0.0f ? 0u : q;
}

// A tile: its expert, first row, the run's end and its column tile.
struct Tile {
    int32_t e, row, end, tn;
};

// Tiles of all experts, WIDTH columns wide (below 2^31 where the borders are in order).
template <int WIDTH>
__device__ __forceinline__ int64_t tiles_of(const BlockArgs& p, const int32_t* table) {
    const int32_t stride = (p.runs.count + kTableSize - 1) / kTableSize, slots = (p.runs.count + stride - 1) / stride;
    const int64_t all = static_cast<int64_t>(table[slots]) * ((p.h + WIDTH - 1) / WIDTH);
    return all < 0x7FFFFFFF ? all : 0x7FFFFFFF;
}

// Issues the MMAs of `blocks` blocks of K, the accumulators in turn.  What the tensor
// pipe waits for between a block and the next but one is this loop too, so its values
// are kept the same for the warp to the compiler's knowledge (the descriptors lie in
// uniform registers then) and the next stage is looked at before it is needed.
__device__ __forceinline__ bool issue_blocks(uint32_t blocks, uint32_t tmem, uint32_t smem_base, uint64_t* full, uint64_t* empty,
                                             uint64_t* acc_full, uint64_t* acc_empty, const volatile int* abort_flag) {
    const uint32_t idesc = ptx::idesc_dense(true, true, true, 256, 256), leader = ptx::elect_one();
    const uint64_t a0 = ptx::sdesc_k128(smem_base), b0 = ptx::sdesc_k128(smem_base + kStageA);
    uint32_t s = 0, filled = 0;   // stage, and the parity of its fill
    bool ready = false;
#pragma unroll 1
    for (uint32_t f = 0; f < blocks; ++f) {
        const uint32_t turn = f & 1;
        bool ok = ready || ptx::mbar_wait(&full[s], filled, abort_flag);
        if (f >= 2) ok = ok && ptx::mbar_wait(&acc_empty[turn], ((f >> 1) - 1) & 1, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, ok)) return false;
        ptx::tc_fence_after();
        const uint32_t off = s * (kStage >> 4);
        ptx::mma_pair_k128_e4m3_if(leader, tmem + turn * 256, a0 + off, b0 + off, idesc);
        ptx::mma_commit_pair_if(leader, &acc_full[turn]);
        ptx::mma_commit_pair_if(leader, &empty[s]);
        if (++s == kStages) {
            s = 0;
            filled ^= 1;
        }
        ready = ptx::mbar_test_wait(&full[s], filled);
    }
    return true;
}

// The k-th tile of this pair of CTAs, WIDTH columns wide; false past its last one.
template <int WIDTH>
__device__ __forceinline__ bool find_tile(const BlockArgs& p, const int32_t* table, int32_t k, Tile& t) {
    const int32_t stride = (p.runs.count + kTableSize - 1) / kTableSize, slots = (p.runs.count + stride - 1) / stride;
    const int32_t tiles_n = (p.h + WIDTH - 1) / WIDTH;
    const int64_t next = (blockIdx.x >> 1) + static_cast<int64_t>(k) * (gridDim.x >> 1);
    if (next >= tiles_of<WIDTH>(p, table)) return false;
    const int32_t u = static_cast<int32_t>(next);
    const int32_t mt = u / tiles_n;   // (only which expert: its tiles are in an order of their own)
    int32_t a = 0, b = slots;         // table[a] <= mt < table[b]
#pragma unroll 1
    while (b - a > 1) {
        const int32_t mid = (a + b) >> 1;
        if (table[mid] <= mt) a = mid;
        else b = mid;
    }
    int32_t first = table[a], lo = 0, hi = 0, tiles = 0;
    bool found = false;
#pragma unroll 1
    for (int32_t e = a * stride; e < p.runs.count && !found; ++e) {
        p.runs.get(e, lo, hi);
        tiles = (hi - lo + 255) / 256;
        t.e = e;
        found = mt < first + tiles;
        if (!found) first += tiles;
    }
    if (!found) return false;
    int32_t i = u - first * tiles_n;
    const int32_t group = i / (kGroupM * tiles_n) * kGroupM;
    i -= group * tiles_n;
    const int32_t height = tiles - group < kGroupM ? tiles - group : kGroupM;
    t.tn = i / height;
    t.row = lo + (group + i - t.tn * height) * 256;
    t.end = hi;
    return true;
}

template <bool DUAL, bool EIGHT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) k_blocks_tc(const __grid_constant__ BlockArgs p) {
    constexpr int S = kStages;
    constexpr int kOut = DUAL ? 64 : 128;   // output columns of a warp
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
    uint8_t* staging = smem + S * kStage;
    float* scales = reinterpret_cast<float*>(staging + kEpiWarps * kStaging);
    float* biases = scales + kScaleSlots * 256;
    int4* tiles = reinterpret_cast<int4*>(biases + kBiasSlots * 256);   // [kEpiWarps]
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpiWarps * kStaging + kScaleBytes);   // [S]  (CTA 0's are used)
    uint64_t* empty = full + S;             // [S]
    uint64_t* acc_full = empty + S;         // [2]
    uint64_t* acc_empty = acc_full + 2;     // [2]  (CTA 0's are used)
    uint64_t* exit_bar = acc_empty + 2;
    uint64_t* shared_max = exit_bar + 1;    // [4]  the two warps that share a block of a gated e4m3 output's columns
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(shared_max + 4);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int32_t* table = reinterpret_cast<int32_t*>(staging + kEpiWarps * kStaging + kScaleBytes + 256);   // row tiles before every `stride`-th expert

    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&acc_full[b], 2);    // the MMAs and the scales
            ptx::mbar_init(&acc_empty[b], 2 * kEpiWarps);
        }
        ptx::mbar_init(exit_bar, 1);
        for (int g = 0; g < 4; ++g) ptx::mbar_init(&shared_max[g], 2);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_map(&p.x);
        ptx::prefetch_map(&p.w[0]);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(tmem_slot, 512);
        ptx::tmem_relinquish_pair();
    }
    pdl_wait();
    const int32_t stride = (p.runs.count + kTableSize - 1) / kTableSize;
    if (warp == 2) {
        int32_t sum = 0;
        for (int32_t i0 = 0; i0 * stride < p.runs.count; i0 += 32) {
            const int32_t e0 = (i0 + lane) * stride;
            int32_t tiles = 0;
            for (int32_t e = e0; e < e0 + stride && e < p.runs.count; ++e) {
                int32_t lo, hi;
                p.runs.get(e, lo, hi);
                tiles += (hi - lo + 255) / 256;
            }
            int32_t inc = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += u;
            }
            // (at most 2^30, whatever the borders)
            if (e0 < p.runs.count) table[i0 + lane] = min(sum + inc - tiles, 1 << 30);
            sum = min(sum + __shfl_sync(0xFFFFFFFFu, inc, 31), 1 << 30);
        }
        if (lane == 0) table[(p.runs.count + stride - 1) / stride] = sum;
    }
    if (warp == 3 && blockIdx.x == 0) p.runs.check(lane, 32, p.status);
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    pdl_trigger();   // (once TMEM is allocated: the next kernel's blocks may want theirs on this SM)
    const uint32_t tmem = __reduce_max_sync(0xFFFFFFFFu, *tmem_slot);   // (uniform)
    const uint32_t smem_base = ptx::smem_u32(smem);
    constexpr int kTileN = DUAL ? 128 : 256;

    auto fail = [&]() {
        atomicOr(p.status, kStatusTimeout);
        *abort_flag = 1;
    };
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, ptx::mbar_wait(bar, parity, abort_flag));
    };
    auto tile_at = [&](int32_t k, Tile& t) { return find_tile<DUAL ? 128 : 256>(p, table, k, t); };
    uint32_t fills = 0;   // stages this thread has filled
    if (warp < kFirstEpi) ptx::regs_dec<Regs<DUAL, EIGHT>::first>();
    if (warp == 0) {
        if (lane == 0) {
            uint32_t& f = fills;
            bool ok = true;
            Tile t;
            for (int32_t q = 0; ok && tile_at(q, t); ++q) {
                const int32_t r0 = t.row + static_cast<int32_t>(rank) * 128;
                const int32_t o0 = t.e * p.h + (DUAL ? t.tn * 128 : t.tn * 256 + static_cast<int32_t>(rank) * 128);
                const CUtensorMap* w = &p.w[DUAL ? rank : 0];
                if (!DUAL && p.vec_extra)   // the residual to L2
                    for (int32_t o = t.tn * 256; o < p.h && o < t.tn * 256 + 256; o += 64) ptx::tma_prefetch_2d(&p.map_extra, o, r0);
#pragma unroll 1
                for (int32_t it = 0; it < p.kb; ++it, ++f) {
                    const uint32_t s = f % S;
                    if (f >= S && !ptx::mbar_wait(&empty[s], (f / S - 1) & 1, abort_flag)) {
                        fail();
                        ok = false;
                        break;
                    }
                    if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * kStage);   // of both CTAs
                    const uint32_t bar = ptx::map_to_rank(ptx::smem_u32(&full[s]), 0);
                    ptx::tma_load_2d_pair(smem_base + s * kStage, &p.x, it * 128, r0, bar);
                    ptx::tma_load_2d_pair(smem_base + s * kStage + kStageA, w, it * 128, o0, bar);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const int64_t all = tiles_of<kTileN>(p, table), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
            const uint32_t blocks = static_cast<uint32_t>(all > pair ? (all - pair + pairs - 1) / pairs : 0) * static_cast<uint32_t>(p.kb);
            const bool ok = issue_blocks(__reduce_max_sync(0xFFFFFFFFu, blocks), tmem, smem_base, full, empty, acc_full, acc_empty, abort_flag);
            if (!ok && lane == 0) fail();
            ptx::mma_commit_pair_if(ptx::elect_one(), exit_bar);   // (the lane that issued)
            const bool done = __all_sync(0xFFFFFFFFu, ptx::mbar_wait(exit_bar, 0, nullptr));
            if (!done && lane == 0) atomicOr(p.status, kStatusTimeout);
        }
    } else if (warp == 3) {
        // The products of the two scales, four rows a lane: read two to four blocks
        // before they are used, written once the accumulator's last turn is over
        // (which means that the turn before it, whose slot this is, has been added up).
        uint32_t f = 0;
        bool ok = true;
        Tile t;
        for (int32_t q = 0; ok && tile_at(q, t); ++q) {
            const int32_t row = t.row + static_cast<int32_t>(rank) * 128 + lane;
            const float* xs = p.x_scale + row;
            // (columns past the last block are not stored: any scale serves)
            const int32_t wi0 = (t.e * p.hb + (DUAL ? t.tn : t.tn * 2)) * p.kb;
            const int32_t wi1 = DUAL ? wi0 : (t.e * p.hb + min(t.tn * 2 + 1, p.hb - 1)) * p.kb;
            const float* ws1 = DUAL ? p.w_scale[1] : p.w_scale[0];
            constexpr int G = 2;
            float x[2][G][4], w0 = 0.0f, w1 = 0.0f;   // [group of blocks][block][quarter]
            auto load = [&](float (&v)[G][4], int32_t it0) {
#pragma unroll
                for (int j = 0; j < G; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        v[j][r] = it0 + j < p.kb && row + 32 * r < t.end ? __ldg(xs + static_cast<int64_t>(it0 + j) * p.runs.n + 32 * r) : 0.0f;
            };
            load(x[0], 0);
            if (!DUAL && p.bias) {   // (once the slot's tile before has been added up: as for the first block's scales)
                if (f >= 2 && !warp_wait(&acc_full[f & 1], ((f >> 1) - 1) & 1)) {
                    if (lane == 0) fail();
                    break;
                }
#pragma unroll
                for (int k = 0; k < 256; k += 32) {
                    const int32_t o = t.tn * 256 + k + lane;
                    biases[(q & (kBiasSlots - 1)) * 256 + k + lane] = o < p.h ? __ldg(p.bias + static_cast<int64_t>(t.e) * p.h + o) : 0.0f;
                }
            }
#pragma unroll 1
            for (int32_t it0 = 0; ok && it0 < p.kb; it0 += 2 * G) {
                if ((it0 & 31) == 0) {   // one block's in each lane
                    w0 = it0 + lane < p.kb ? __ldg(p.w_scale[0] + wi0 + it0 + lane) : 0.0f;
                    w1 = it0 + lane < p.kb ? __ldg(ws1 + wi1 + it0 + lane) : 0.0f;
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    load(x[g ^ 1], it0 + G * g + G);
#pragma unroll
                    for (int j = 0; j < G; ++j) {
                        const int32_t it = it0 + G * g + j;
                        if (!ok || it >= p.kb) continue;
                        const float a = __shfl_sync(0xFFFFFFFFu, w0, it & 31), b = __shfl_sync(0xFFFFFFFFu, w1, it & 31);
                        if (f >= 2 && !warp_wait(&acc_full[f & 1], ((f >> 1) - 1) & 1)) {
                            if (lane == 0) fail();
                            ok = false;
                            continue;
                        }
                        float* slot = scales + (f % kScaleSlots) * 256 + lane;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            slot[32 * r] = x[g][j][r] * a;
                            slot[128 + 32 * r] = x[g][j][r] * b;
                        }
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&acc_full[f & 1]);
                        ++f;
                    }
                }
            }
        }
    } else if (warp >= kFirstEpi) {
        ptx::regs_inc<Regs<DUAL, EIGHT>::epi>();
        const int e = warp - kFirstEpi;
        const int quarter = warp & 3, part = e >> 2;   // TMEM lanes; half of the columns
        uint8_t* stage0 = staging + e * kStaging;
        volatile int4* tile = reinterpret_cast<volatile int4*>(tiles) + e;
        const uint32_t acc_bar = ptx::map_to_rank(ptx::smem_u32(&acc_empty[0]), 0);
        // accumulator columns of each 32: 128 next to each other, or 64 of gate and 64 of up
        const uint32_t ta = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        auto column = [&](int c) { return DUAL ? (c < 2 ? part * 64 + c * 32 : 128 + part * 64 + (c - 2) * 32) : part * 128 + c * 32; };
        uint32_t f = 0;
        bool ok = true;
        Tile t;
        for (int32_t q = 0; ok && tile_at(q, t); ++q) {
            // (the tile waits in shared memory: the loop has no registers for it)
            __syncwarp();
            if (lane == 0) tile->x = t.e, tile->y = t.row, tile->z = t.end, tile->w = t.tn;
            __syncwarp();
            F2 acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = F2(0.0f);
            bool ready = false;
            if (!DUAL && p.bias) {   // the sums begin with it: it comes with the first block's scales
                ready = ptx::mbar_wait(&acc_full[f & 1], (f >> 1) & 1, abort_flag);
                __syncwarp();
                const volatile float4* bias = reinterpret_cast<const volatile float4*>(biases + (q & (kBiasSlots - 1)) * 256 + part * 128);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    acc[2 * j] = F2(bias[j].x, bias[j].y);
                    acc[2 * j + 1] = F2(bias[j].z, bias[j].w);
                }
            }
            // What can is done while TMEM's loads or the multiply-adds run: a warp has about 600
            // clocks a block for all of it, and only one other warp to share them with.
#pragma unroll 1
            for (int32_t it = 0; it < p.kb; ++it, ++f) {
                const uint32_t buf = f & 1;
                if (!ready && !ptx::mbar_wait(&acc_full[buf], (f >> 1) & 1, abort_flag)) {
                    if (lane == 0) fail();
                    ok = false;
                }
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                uint32_t z[2][32];
                ptx::tmem_ld_32x32b_x32(ta + buf * 256 + column(0), z[0]);
                ptx::tmem_ld_32x32b_x32(ta + buf * 256 + column(1), z[1]);
                const volatile float* scale = scales + (f % kScaleSlots) * 256 + quarter * 32 + lane;
                const F2 now0(scale[DUAL ? 0 : part * 128]), now1(DUAL ? scale[128] : 0.0f);
                auto add = [&](int c) {
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        acc[(c * 32 + j) / 2] = fma_v(F2(__uint_as_float(z[c & 1][j]), __uint_as_float(z[c & 1][j + 1])),
                                                      DUAL && c >= 2 ? now1 : now0, acc[(c * 32 + j) / 2]);
                };
                ptx::tmem_ld_wait_for(z[0]);
                ptx::tmem_ld_wait_for(z[1]);
                add(0);
                ptx::tmem_ld_32x32b_x32(ta + buf * 256 + column(2), z[0]);
                add(1);
                ptx::tmem_ld_32x32b_x32(ta + buf * 256 + column(3), z[1]);
                ptx::tmem_ld_wait_for(z[0]);
                ptx::tmem_ld_wait_for(z[1]);
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(acc_bar + buf * 8);
                ready = ptx::mbar_test_wait(&acc_full[buf ^ 1], ((f + 1) >> 1) & 1);
                add(2);
                add(3);
            }
            if (!ok) break;
            const int32_t end = tile->z;
            const int32_t m0 = tile->y + static_cast<int32_t>(ptx::cluster_rank()) * 128 + quarter * 32, row = m0 + lane;
            const int32_t n0 = tile->w * kTileN + part * kOut;   // first output column
            const int32_t rows = end - m0 < 32 ? end - m0 : 32, left = p.h - n0;   // (either may be negative)
            const bool live = row < end;
            // Whole groups of 32 rows leave by tensor-map copies, which nobody waits for; a run's
            // last ones, which a copy would not clip, and unaligned outputs by plain stores.
            const bool mapped = p.map_out && rows == 32;
            // Activations in place, some columns at a time: the empty statements keep the compiler from
            // working on more of them at once, which would take more registers than there are.  A gated
            // result's chunks are of one case of the switch, another's a switch each: the other way about
            // the main loop gets spills, or both take longer (8192 x 512 x 4096: gated to e4m3 without
            // activation 53 and 61 us; ReLU in 32 columns 39, in 16 44).  No loop over them: moving the
            // sums to where it finds them takes longer than the unrolled code's wait for instructions (a
            // plain product 39 us, not 31).
            auto activate = [&]() {
                constexpr int kChunk = DUAL ? 8 : 16;   // of columns
                auto apply = [&](int c, auto act) {
#pragma unroll
                    for (int j = c; j < c + kChunk; ++j) acc[j] = DUAL ? act_f<act>(acc[j]) * acc[(j + 32) % 64] : act_f<act>(acc[j]);
                };
                if constexpr (DUAL) {
                    with_act(p.act, [&](auto act) {
#pragma unroll
                        for (int c = 0; c < kOut / 2; c += kChunk) {
#pragma unroll
                            for (int j = c; j < c + kChunk; ++j) asm volatile("" : "+l"(acc[j].v));
                            apply(c, act);
#pragma unroll
                            for (int j = c; j < c + kChunk; ++j) asm volatile("" : "+l"(acc[j].v));
                        }
                    });
                } else {
#pragma unroll
                    for (int c = 0; c < kOut / 2; c += kChunk) {
                        int32_t a = p.act;
                        asm volatile("" : "+r"(a));
                        with_act(a, [&](auto act) { apply(c, act); });
                    }
                }
            };
            if (DUAL || p.act != SPCONV_ACT_NONE) activate();
            if (!EIGHT) {
                // two staging buffers in turn: rows of 64 bytes in 16-byte pieces whose places are
                // turned by the row (the copies' 64-byte swizzle)
                auto place = [](int r, int piece) { return r * 64 + ((piece ^ ((r >> 1) & 3)) << 4); };
                const int i0 = lane >> 2, c8 = lane & 3;   // of eight rows at a time: row; eight columns
                // the residual of the next 32 columns is on its way while these are stored
                uint4 ahead[4];
                auto whole = [&](int c, int i) { return p.vec_extra && i < rows && c * 32 + c8 * 8 + 8 <= left; };
                auto read_ahead = [&](int c) {
#pragma unroll
                    for (int r = 0; r < 32; r += 8)
                        if (whole(c, r + i0))
                            ahead[r / 8] = *reinterpret_cast<const uint4*>(p.extra + (m0 + r + i0) * p.ld_extra + n0 + c * 32 + c8 * 8);
                };
                if (!DUAL && p.extra) read_ahead(0);
                auto store = [&](int c, F2 (&v)[16]) {     // 32 columns
                    const int32_t cols = left - 32 * c;    // (may be negative)
                    uint8_t* stage = stage0 + (c & 1) * 2048;
                    if (lane == 0) ptx::bulk_wait_read_but<1>();   // (the other buffer's copy may still run)
                    __syncwarp();
                    if (!DUAL && p.extra) {
#pragma unroll
                        for (int r = 0; r < 32; r += 8) {
                            const int i = r + i0;
                            uint4 x4 = ahead[r / 8];
                            if (!whole(c, i) && i < rows && c8 * 8 < cols) {
                                const __nv_bfloat16* x = p.extra + (m0 + i) * p.ld_extra + n0 + c * 32 + c8 * 8;
                                uint32_t u[4] = {};
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    if (c8 * 8 + j < cols) u[j / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(x[j])) << (16 * (j & 1));
                                x4 = make_uint4(u[0], u[1], u[2], u[3]);
                            }
                            *reinterpret_cast<uint4*>(stage + place(i, c8)) = x4;
                        }
                        if (c < 3) read_ahead(c + 1);
                        __syncwarp();
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint4* at = reinterpret_cast<uint4*>(stage + place(lane, k));
                        if (!DUAL && p.extra) {
                            const uint4 x4 = *at;
                            const uint32_t u[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                v[k * 4 + j] = v[k * 4 + j] + F2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xFFFF0000u));
                        }
                        uint32_t u[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float a, b;
                            v[k * 4 + j].get(a, b);
                            const __nv_bfloat162 y = __floats2bfloat162_rn(a, b);
                            u[j] = reinterpret_cast<const uint32_t&>(y);
                        }
                        *at = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                    if (mapped) ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (mapped) {
                        if (lane == 0 && cols > 0) ptx::tma_store_2d(&p.c, n0 + c * 32, m0, ptx::smem_u32(stage));
                    } else {
                        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + n0 + c * 32 + c8 * 8;
#pragma unroll
                        for (int r = 0; r < 32; r += 8) {
                            const int i = r + i0;
                            if (i >= rows || c8 * 8 >= cols) continue;
                            const uint4 y4 = *reinterpret_cast<const uint4*>(stage + place(i, c8));
                            __nv_bfloat16* o = out + (m0 + i) * p.ld_out;
                            if (p.vec_out && c8 * 8 + 8 <= cols) {
                                *reinterpret_cast<uint4*>(o) = y4;
                            } else {
                                const uint32_t u[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    if (c8 * 8 + j < cols) o[j] = __ushort_as_bfloat16(static_cast<uint16_t>(u[j / 2] >> (16 * (j & 1))));
                            }
                        }
                        __syncwarp();
                    }
                    if (lane == 0) ptx::bulk_commit();
                };
#pragma unroll
                for (int c = 0; c < kOut / 32; ++c) store(c, reinterpret_cast<F2(&)[16]>(acc[c * 16]));
            } else {
                // the largest of the row's 128 columns: this warp's, or its half and another warp's
                uint32_t most = 0;
#pragma unroll
                for (int j = 0; j < kOut / 2; ++j) {
                    float a, b;
                    acc[j].get(a, b);
                    if (2 * j < left) most = max(most, __float_as_uint(fabsf(a)));
                    if (2 * j + 1 < left) most = max(most, __float_as_uint(fabsf(b)));
                }
                if (DUAL) {
                    // (behind the staged output, by the tiles' parity: a slot is written again two tiles
                    // later, when both have passed the barrier of the tile between)
                    uint64_t* bar = &shared_max[quarter];
                    const uint32_t slot = 2048 + (q & 1) * 128 + lane * 4;
                    *reinterpret_cast<volatile uint32_t*>(stage0 + slot) = most;
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar);
                    if (!warp_wait(bar, q & 1)) {
                        if (lane == 0) fail();
                        ok = false;
                        break;
                    }
                    most = max(most, *reinterpret_cast<volatile uint32_t*>(staging + (e ^ 4) * kStaging + slot));
                }
                const float scale = __fdiv_rn(__uint_as_float(most), 448.0f);
                if ((!DUAL || part == 0) && live && left > 0) p.scale[static_cast<int64_t>(n0 / 128) * p.runs.n + row] = scale;
                if (lane == 0) ptx::bulk_wait_read();
                __syncwarp();
                constexpr int kPieces = kOut / 16, kRows = 32 / kPieces;   // 16-byte pieces of a row
                auto place = [](int r, int piece) { return r * kOut + ((piece ^ (kPieces == 8 ? r & 7 : (r >> 1) & 3)) << 4); };
                auto stage_row = [&](const auto& quotient) {
#pragma unroll
                    for (int c = 0; c < kPieces; ++c) {
                        uint32_t u[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) u[j] = to_e4m3(quotient, scale, acc[c * 8 + j * 2], acc[c * 8 + j * 2 + 1]);
                        *reinterpret_cast<uint4*>(stage0 + place(lane, c)) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                };
                const Quotient quotient(scale);
                if (__all_sync(0xFFFFFFFFu, quotient.serves)) stage_row(quotient);
                else stage_row(AnyQuotient(scale));
                if (mapped) ptx::fence_proxy_async_smem();
                __syncwarp();
                if (mapped) {
                    if (lane == 0 && left > 0) ptx::tma_store_2d(&p.c, n0, m0, ptx::smem_u32(stage0));
                    if (lane == 0) ptx::bulk_commit();
                } else {
                    uint8_t* out = static_cast<uint8_t*>(p.out);
#pragma unroll 4
                    for (int r = 0; r < 32; r += kRows) {
                        const int i = r + lane / kPieces, c = lane % kPieces;
                        if (i >= rows || c * 16 >= left) continue;
                        const uint4 v = *reinterpret_cast<const uint4*>(stage0 + place(i, c));
                        uint8_t* o = out + (m0 + i) * p.ld_out + n0 + c * 16;
                        if (p.vec_out && c * 16 + 16 <= left) {
                            *reinterpret_cast<uint4*>(o) = v;
                        } else {
                            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (c * 16 + j < left) o[j] = static_cast<uint8_t>(u[j / 4] >> (8 * (j % 4)));
                        }
                    }
                }
            }
            __syncwarp();
        }
        if (lane == 0) ptx::bulk_wait();
        __syncwarp();
        zero_rest<EIGHT>(p, static_cast<int64_t>(blockIdx.x) * (32 * kEpiWarps) + threadIdx.x - 32 * kFirstEpi, static_cast<int64_t>(gridDim.x) * (32 * kEpiWarps));
    }
    // (as in dense_tc.cu: neither CTA leaves, or frees TMEM, while the other may still signal it)
    ptx::tc_fence_before();
    ptx::cluster_sync();
    const uint32_t side = ptx::cluster_rank();   // (read again: no register is kept for it)
    if (side == 0 && fills && *abort_flag)
        for (uint32_t q = fills > S ? fills - S : 0; q < fills; ++q) ptx::mbar_wait(&full[q % S], (q / S) & 1, nullptr);
    __syncwarp();
    if (warp == 1 && side == 1 && !ptx::mbar_wait(exit_bar, 0, nullptr)) atomicOr(p.status, kStatusTimeout);
    __syncwarp();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc_pair(*tmem_slot, 512);
}

// ---- few rows -------------------------------------------------------------------
// The weights are the traffic, so they are streamed once and the operands change
// places: 128 output channels (one block of the weight's scales) are the MMA's M,
// R rows of x its N.  A cluster of `splits` CTAs cuts K between them; each adds
// its blocks up in registers (a thread a channel), and the cluster's partial sums
// are added through distributed shared memory in the order of the ranks.
// Accumulators of one block of K take turns in a ring in TMEM.  The weights' stream
// bounds it: 64 rows of 28 experts, gated 2048 x 1408, 27 us at 6.0 TB/s; one row
// of 4096 x 4096 7 us, where the start and the cluster's sums are 4.  An expert with
// more than R rows streams its weight again for each R of them.
constexpr int kFewThreads = 192;       // warp 0 loads, warp 1 issues MMAs, warps 2-5 add up
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kTileW = 128 * 128;
constexpr int kMaxStages = 8;
constexpr int kMaxAcc = 4;
constexpr int kFewRing = 100 * 1024;   // of one of two CTAs on an SM
constexpr int kMaxSplits = 8;

struct FewBlockArgs {
    BlockArgs b;
    int32_t stages, stage_bytes;
};

template <bool DUAL, int R>
struct FewShape {
    static constexpr int kAcc = DUAL ? 2 : 1;
    static constexpr int kCols = kAcc * R;                        // TMEM columns of an accumulator
    static constexpr int kBufs = 256 / kCols < kMaxAcc ? 256 / kCols : kMaxAcc;
    static constexpr uint32_t kTmem = kBufs * kCols;
    static constexpr int kSmallRing = R == 16 && !DUAL ? kFewRing / 2 : kFewRing;   // (four CTAs on an SM)
    static_assert(kTmem >= 32 && (kTmem & (kTmem - 1)) == 0, "TMEM columns");
    static_assert(kAcc * R * 128 * 4 <= kSmallRing, "the sums take the ring's place");
    // two CTAs with the large ring, or one and those with the small one in what it leaves (of
    // the other kernels that take TMEM k_dense_few's small form has as much shared memory and a
    // quarter of the columns, and the others leave no room beside them)
    static_assert(ptx::tmem_fits(kFewRing + 1024, kTmem) && ptx::tmem_fits(kSmallRing + 1024, kTmem), "TMEM of an SM");
    static_assert(kSmallRing == kFewRing ||
                      256 + (ptx::kSmShared - ptx::cta_shared(kFewRing + 1024)) / ptx::cta_shared(kSmallRing + 1024) * kTmem <= ptx::kSmTmemColumns,
                  "TMEM of an SM");
};

template <bool DUAL, bool EIGHT, int R>
__global__ void __launch_bounds__(kFewThreads, 2) k_blocks_few(const __grid_constant__ FewBlockArgs a) {
    using Shape = FewShape<DUAL, R>;
    constexpr int kAcc = Shape::kAcc, kCols = Shape::kCols, kBufs = Shape::kBufs;
    constexpr uint32_t kTmem = Shape::kTmem;
    const BlockArgs& p = a.b;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[kBufs], acc_empty[kBufs];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    uint8_t* ring = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t splits = gridDim.y, rank = blockIdx.y;   // the cluster is one column of the grid
    const int32_t e = static_cast<int32_t>(blockIdx.z), tn = static_cast<int32_t>(blockIdx.x);
    pdl_wait();
    if (tn == 0 && rank == 0 && e == 0) p.runs.check(threadIdx.x, kFewThreads, p.status);
    if (rank == 0) {
        const int64_t block = static_cast<int64_t>(e) * gridDim.x + tn, step = static_cast<int64_t>(gridDim.z) * gridDim.x * kFewThreads;
        zero_rest<EIGHT>(p, block * kFewThreads + threadIdx.x, step);
    }
    int32_t lo, hi;
    p.runs.get(e, lo, hi);
    if (lo == hi) return;   // (the whole cluster)
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kBufs; ++s) {
            ptx::mbar_init(&acc_full[s], 1);
            ptx::mbar_init(&acc_empty[s], 4);
        }
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(&tmem_slot, kTmem);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    pdl_trigger();   // (once TMEM is allocated, as above)
    const uint32_t tmem = tmem_slot;
    const int32_t n0 = tn * 128;
    const int32_t it0 = static_cast<int32_t>(rank * static_cast<uint32_t>(p.kb) / splits);
    const int32_t it1 = static_cast<int32_t>((rank + 1) * static_cast<uint32_t>(p.kb) / splits);
    auto fail = [&]() {
        atomicOr(p.status, kStatusTimeout);
        *abort_flag = 1;
    };
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, ptx::mbar_wait(bar, parity, abort_flag));
    };
    const uint32_t base = ptx::smem_u32(ring);
    float* sums = reinterpret_cast<float*>(ring);   // [kAcc][R][128]
    uint32_t f = 0;                                 // blocks that this role has handled
    uint32_t fills = 0;                             // of the loading thread
    for (int32_t r0 = lo; r0 < hi; r0 += R) {
        const int32_t rows = hi - r0 < R ? hi - r0 : R;
        if (warp == 0) {
            if (lane == 0) {
                for (int32_t it = it0; it < it1; ++it, ++fills) {
                    const uint32_t s = fills % a.stages;
                    if (fills >= static_cast<uint32_t>(a.stages) && !ptx::mbar_wait(&empty[s], (fills / a.stages - 1) & 1, abort_flag)) {
                        fail();
                        break;
                    }
                    const uint32_t at = base + s * a.stage_bytes, bar = ptx::smem_u32(&full[s]);
                    ptx::mbar_arrive_expect_tx(&full[s], kAcc * kTileW + R * 128);
#pragma unroll
                    for (int w = 0; w < kAcc; ++w) ptx::tma_load_2d(at + w * kTileW, &p.w[w], it * 128, e * p.h + n0, bar);
                    ptx::tma_load_2d(at + kAcc * kTileW, &p.x, it * 128, r0, bar);
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            const uint32_t leader = lane == 0;
            const uint32_t idesc = ptx::idesc_dense(true, true, true, 128, R);
            for (int32_t it = it0; it < it1; ++it, ++f) {
                const uint32_t s = f % a.stages, buf = f % kBufs;
                if ((f >= kBufs && !warp_wait(&acc_empty[buf], (f / kBufs - 1) & 1)) || !warp_wait(&full[s], (f / a.stages) & 1)) {
                    if (lane == 0) fail();
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t at = base + s * a.stage_bytes;
#pragma unroll
                for (int w = 0; w < kAcc; ++w)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        ptx::mma_if<true>(leader, tmem + buf * kCols + w * R, ptx::sdesc_k128(at + w * kTileW) + 2 * j,
                                          ptx::sdesc_k128(at + kAcc * kTileW) + 2 * j, idesc, j > 0 ? 1u : 0u);
                ptx::mma_commit_if(leader, &empty[s]);
                ptx::mma_commit_if(leader, &acc_full[buf]);
            }
        } else {
            const int quarter = warp & 3;
            const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
            float acc[kAcc][R];
#pragma unroll
            for (int w = 0; w < kAcc; ++w)
#pragma unroll
                for (int j = 0; j < R; ++j) acc[w][j] = 0.0f;
            for (int32_t it = it0; it < it1; ++it, ++f) {
                const uint32_t buf = f % kBufs;
                // lane j has the scale of row j (and j + 32), passed round below
                const float* xs = p.x_scale + static_cast<int64_t>(it) * p.runs.n + r0;
                const float x0 = lane < rows ? __ldg(xs + lane) : 0.0f, x1 = R > 32 && lane + 32 < rows ? __ldg(xs + lane + 32) : 0.0f;
                float ws[kAcc];
#pragma unroll
                for (int w = 0; w < kAcc; ++w) ws[w] = __ldg(p.w_scale[w] + (static_cast<int64_t>(e) * p.hb + tn) * p.kb + it);
                if (!warp_wait(&acc_full[buf], (f / kBufs) & 1)) {
                    if (lane == 0) fail();
                    break;
                }
                ptx::tc_fence_after();
#pragma unroll
                for (int w = 0; w < kAcc; ++w)
#pragma unroll
                    for (int c = 0; c < R; c += 16) {
                        uint32_t z[16];
                        ptx::tmem_ld_32x32b_x16(tmem + lanes + buf * kCols + w * R + c, z);
                        ptx::tmem_ld_wait();
                        if (w == kAcc - 1 && c == R - 16) {
                            ptx::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(&acc_empty[buf]);
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float s = ws[w] * __shfl_sync(0xFFFFFFFFu, c + j < 32 ? x0 : x1, (c + j) & 31);
                            // (a row past the run's end is some other row: its sums are not used)
                            acc[w][c + j] = fmaf(__uint_as_float(z[j]), s, acc[w][c + j]);
                        }
                    }
            }
            // every block has been added up: the ring is free once all four warps are here
            ptx::named_barrier_sync(1, 128);
#pragma unroll
            for (int w = 0; w < kAcc; ++w)
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (j < rows) sums[(w * R + j) * 128 + quarter * 32 + lane] = acc[w][j];
        }
        ptx::cluster_sync();
        // this CTA's share: rows rank, rank + splits, ..; a warp a row, a lane four channels
        const int32_t left = p.h - n0 - 4 * lane;
        const uint32_t sums_addr = ptx::smem_u32(sums);
        for (int32_t i = static_cast<int32_t>(rank) + warp * static_cast<int32_t>(splits); i < rows; i += kFewWarps * static_cast<int32_t>(splits)) {
            const int64_t row = r0 + i;
            float z[kAcc][4] = {};
#pragma unroll
            for (int w = 0; w < kAcc; ++w) {
                const uint32_t at = sums_addr + static_cast<uint32_t>(((w * R + i) * 128 + 4 * lane) * 4);
                float4 part[kMaxSplits];
#pragma unroll
                for (uint32_t r = 0; r < kMaxSplits; ++r)
                    part[r] = r < splits ? ptx::ld_cluster_f32x4(ptx::map_to_rank(at, r)) : make_float4(0, 0, 0, 0);
#pragma unroll
                for (uint32_t r = 0; r < kMaxSplits; ++r) {
                    z[w][0] += part[r].x;
                    z[w][1] += part[r].y;
                    z[w][2] += part[r].z;
                    z[w][3] += part[r].w;
                }
            }
            if (!DUAL && p.bias)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < left) z[0][j] += __ldg(p.bias + static_cast<int64_t>(e) * p.h + n0 + 4 * lane + j);
            with_act(p.act, [&](auto act) {
#pragma unroll
                for (int j = 0; j < 4; ++j) z[0][j] = DUAL ? act_f<act>(z[0][j]) * z[kAcc - 1][j] : act_f<act>(z[0][j]);
            });
            if (!DUAL && p.extra)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < left) z[0][j] += __bfloat162float(p.extra[row * p.ld_extra + n0 + 4 * lane + j]);
            if (EIGHT) {
                uint32_t most = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < left) most = max(most, __float_as_uint(fabsf(z[0][j])));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
                const float scale = __fdiv_rn(__uint_as_float(most), 448.0f);
                if (lane == 0) p.scale[static_cast<int64_t>(tn) * p.runs.n + row] = scale;
                const uint32_t v = to_e4m3(AnyQuotient(scale), scale, F2(z[0][0], z[0][1]), F2(z[0][2], z[0][3]));
                uint8_t* out = static_cast<uint8_t*>(p.out) + row * p.ld_out + n0 + 4 * lane;
                if (p.vec_out && left >= 4) {
                    *reinterpret_cast<uint32_t*>(out) = v;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < left) out[j] = static_cast<uint8_t>(v >> (8 * j));
                }
            } else {
                alignas(8) __nv_bfloat16 y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = __float2bfloat16_rn(z[0][j]);
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * p.ld_out + n0 + 4 * lane;
                if (p.vec_out && left >= 4) {
                    *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(y);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < left) out[j] = y[j];
                }
            }
        }
        // no CTA's sums go away while another may still read them; loads come into the same bytes
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        ptx::cluster_sync();
        ptx::tc_fence_after();
    }
    if (warp == 0 && lane == 0 && *abort_flag)   // given up: loads still in flight land first
        for (uint32_t j = fills > static_cast<uint32_t>(a.stages) ? fills - a.stages : 0; j < fills; ++j)
            ptx::mbar_wait(&full[j % a.stages], (j / a.stages) & 1, nullptr);
    __syncthreads();
    if (warp == 1) ptx::tmem_dealloc(tmem, kTmem);
}

// ---- host -----------------------------------------------------------------------
template <auto KERNEL>
int allow_smem(int bytes) {
    static bool set[kMaxDevices] = {};
    int dev = 0;
    SPCONV_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return SPCONV_ERR_UNSUPPORTED;
    if (!set[dev]) {
        SPCONV_CHECK_CUDA(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
        set[dev] = true;
    }
    return SPCONV_OK;
}

int make_maps(const BlockOp& op, const void* x, int64_t ldx, int32_t rows, BlockArgs* p) {
    SPCONV_CHECK(make_tensor_map(&p->x, x, 1, op.k, op.n, ldx, rows));
    for (int i = 0; i < (op.w[1] ? 2 : 1); ++i)
        SPCONV_CHECK(make_tensor_map(&p->w[i], op.w[i], 1, op.k, static_cast<int64_t>(op.experts) * op.h, op.k, 128));
    return SPCONV_OK;
}

template <bool DUAL, bool EIGHT>
int run_tc(const BlockOp& op, const BlockArgs& p, cudaStream_t s) {
    const int64_t tiles = (op.n / 256 + op.experts) * ceil_div(op.h, DUAL ? 128 : 256);
    if (tiles >= 0x7FFFFFFF) return SPCONV_ERR_UNSUPPORTED;
    const unsigned pairs = static_cast<unsigned>(tiles < kPairs ? tiles : kPairs);
    SPCONV_CHECK((allow_smem<k_blocks_tc<DUAL, EIGHT>>(kSmem)));
    return launch_pdl(k_blocks_tc<DUAL, EIGHT>, dim3(2 * pairs), kThreads, kSmem, s, p);
}

template <bool DUAL, bool EIGHT, int R>
int run_few(const BlockOp& op, const BlockArgs& p, int64_t active, cudaStream_t s) {
    FewBlockArgs a = {};
    a.b = p;
    const int64_t tiles = ceil_div(op.h, 128);
    int32_t splits = 1;
    while (splits < kMaxSplits && tiles * active * splits * 2 <= 304 && p.kb >= 4 * splits) splits *= 2;
    a.stage_bytes = (DUAL ? 2 : 1) * kTileW + R * 128;
    // a smaller ring where all CTAs then run at once and do not otherwise (512 rows of 32
    // experts, 1408 x 2048: 16.7 us, not 23.3)
    const int64_t ctas = tiles * active * splits;
    const int32_t ring = ctas > 304 && ctas <= 608 ? FewShape<DUAL, R>::kSmallRing : kFewRing;
    a.stages = ring / a.stage_bytes < kMaxStages ? ring / a.stage_bytes : kMaxStages;
    SPCONV_CHECK((allow_smem<k_blocks_few<DUAL, EIGHT, R>>(kFewRing + 1024)));
    cudaLaunchAttribute at[2] = {pdl_attr(), {}};
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 1;
    at[1].val.clusterDim.y = static_cast<unsigned>(splits);
    at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(splits), static_cast<unsigned>(op.experts));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(ring) + 1024;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    count_launch();
    return cuda_status(cudaLaunchKernelEx(&cfg, k_blocks_few<DUAL, EIGHT, R>, static_cast<const FewBlockArgs&>(a)));
}

template <bool DUAL, bool EIGHT>
int run(const BlockOp& op, cudaStream_t s) {
    BlockArgs p = {};
    p.runs = Runs{op.offsets, op.experts, static_cast<int32_t>(op.n)};
    p.h = op.h;
    p.kb = static_cast<int32_t>(ceil_div(op.k, 128));
    p.hb = static_cast<int32_t>(ceil_div(op.h, 128));
    p.act = op.act;
    p.x_scale = op.x_scale;
    p.w_scale[0] = op.w_scale[0];
    p.w_scale[1] = op.w_scale[1];
    p.bias = op.bias;
    p.extra = static_cast<const __nv_bfloat16*>(op.extra);
    p.ld_extra = op.ld_extra;
    p.out = op.out;
    p.ld_out = op.ld_out;
    p.scale = op.out_scale;
    p.vec_extra = op.extra && tma_ok(op.extra, op.ld_extra, 2);
    p.vec_out = tma_ok(op.out, op.ld_out, EIGHT ? 1 : 2);
    SPCONV_CHECK(rows_status_word(&p.status));
    // x in the alignment that its tensor map needs
    AlignedRows rows;
    const void* x = op.x;
    int64_t ldx = op.ldx;
    rows.add(&x, 1, &ldx, op.n, op.k, 1);
    SPCONV_CHECK(rows.run(s));
    // Few rows a run (an expert has n / experts of them where all are chosen alike): the
    // weight's stream is the bound, which many CTAs share.  One weight of 4096 x 4096, us, and
    // as 256-row tiles: 32 rows 8.0 and 16.9, 64 rows 9.4 and 17.0; 32 experts of 1408 x 2048:
    // 16 rows each 16.7 and 23.3, 64 rows 31.9 and 33.0.  A gated product of more than 32 rows
    // has room for two stages, which is too few where its CTAs do not all run at once: 32
    // experts of 2048 x 1408 with 40 rows each 56 and 49, 8 experts with 48 rows 16.8 and 22.1.
    const int64_t active = op.experts < op.n ? op.experts : op.n;
    const int64_t each = ceil_div(op.n, active);
    if (each <= 32 || (each <= 64 && !(DUAL && active * p.hb > 304))) {
        const int32_t r = each <= 16 ? 16 : each <= 32 ? 32 : 64;
        SPCONV_CHECK(make_maps(op, x, ldx, r, &p));
        return r == 16 ? run_few<DUAL, EIGHT, 16>(op, p, active, s) : r == 32 ? run_few<DUAL, EIGHT, 32>(op, p, active, s)
                                                                             : run_few<DUAL, EIGHT, 64>(op, p, active, s);
    }
    SPCONV_CHECK(make_maps(op, x, ldx, 128, &p));
    p.map_out = p.vec_out && op.h % (EIGHT ? 16 : 8) == 0;
    if (p.map_out)
        SPCONV_CHECK(make_tensor_map(&p.c, op.out, EIGHT ? 1 : 2, op.h, op.n, op.ld_out, 32, EIGHT && !DUAL ? 128 : 64));
    if (p.vec_extra) SPCONV_CHECK(make_tensor_map(&p.map_extra, op.extra, 2, op.h, op.n, op.ld_extra, 128));
    return run_tc<DUAL, EIGHT>(op, p, s);
}

}  // namespace

int blocks_run(const BlockOp& op, cudaStream_t s) {
    if (op.w[1]) return op.out_scale ? run<true, true>(op, s) : run<true, false>(op, s);
    return op.out_scale ? run<false, true>(op, s) : run<false, false>(op, s);
}

}  // namespace spconv
