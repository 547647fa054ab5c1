// Products with an epilogue on the 5th-generation tensor cores.
//
//   out[m][n] = epilogue(sum_k A(m, k) B(n, k))
//
// A pair of CTAs works on one tile of 256 rows by 2 `hb` columns (hb = 64 or
// 128): tcgen05.mma with cta_group::2, each CTA bringing its 128 rows of A and
// hb rows of B, so an operand byte fetched from L2 feeds twice the products it
// would in one CTA.  For a gated product CTA 0 brings hb rows of the gate's
// weight and CTA 1 the same rows of the up weight: columns [0, hb) of the
// accumulator are gate, [hb, 2 hb) up, side by side in each thread's row.
//
// Either operand may be K-major or have its rows contiguous (forward weights
// [c_in][c_out], and x^T, dz^T of the weight gradients): the tensor maps and
// the shared-memory descriptors take both as they lie in memory.
//
// Warps of each CTA (persistent over the tiles):
//   warps 0, 18  tensor-map loads of one operand each into a ring of stages;
//              both CTAs' loads complete on CTA 0's barrier
//   warp 1     MMA issue (CTA 0), TMEM allocation
//   warps 2-17 epilogue, in two sets of eight: each set takes every other
//              tile, so that the chain of latencies of one tile's epilogue
//              (accumulator wait, TMEM loads, staging, store) runs beside that
//              of the next.  Two warps share 32 accumulator rows and take
//              blocks of columns in turn: 16 columns at a time from TMEM, fp32
//              epilogue, one rounding, staged in shared memory and stored by a
//              tensor-map copy, which also clips the ragged edges; the residual
//              or incoming gradient arrives in the same staging buffer by a
//              tensor-map load before the accumulator is ready
// The accumulator is double-buffered in TMEM (2 x 256 columns), so the
// epilogue of one tile runs beside the main loop of the next.
//
// What bounds it: with many steps of K the tensor pipe and the power cap (gated,
// 7777 x 4096 x 8192: 533 us alone, 94 % of the pipe's cycles, 587 in a long run;
// 8192 x 8192 x 8192 bf16 591, the library's 620); with e4m3 the loads, 50 bytes a
// clock and SM (8192 x 4096 x 4096 with bias and GELU 86 us, 75 %); with few
// steps the epilogue's instructions and latencies (gated, 32371 x 128 x 512:
// 14.4 us; of 240000 rows 74, where the activation keeps the special-function
// unit at 35 % of its rate) or the output's stores (53280 x 144 x 1624: 51.9 us;
// a fill of the output alone takes 43.6).
#include "ptx_sm100.cuh"
#include "tensor_map.cuh"

namespace spconv {
namespace {

constexpr int kRowsA = 128;                   // rows of A per CTA
constexpr int kStageA = kRowsA * 128;         // 128 bytes of K per stage
constexpr int kStageB = 128 * 128;            // hb <= 128 rows
constexpr int kStage = kStageA + kStageB;
constexpr int kEpiWarps = 16;
constexpr int kLoadA = 0, kLoadB = 2 + kEpiWarps;   // warps that load an operand each
constexpr int kThreads = 32 * (3 + kEpiWarps);
constexpr int kStaging = 32 * 128;            // of an epilogue warp: 32 rows of 64 bf16, or twice 32 of 32
constexpr int kTmemCols = 512;
constexpr int kGroupM = 16;                   // row tiles that share the column tiles in L2
constexpr int kPairs = 76;                    // CTA pairs of a full GPU

constexpr int32_t kEpiPlain = 4;              // the sums, rounded; or, of one slice of K, fp32 to a workspace

// x / d for 0 <= x < 2^31, without a division: x m / 2^(31 + s) with
// s = ceil(log2 d) and m = ceil(2^(31 + s) / d).
struct FastDiv {
    uint32_t d, m, s;
    FastDiv() = default;
    explicit FastDiv(uint32_t v) : d(v), s(0) {
        while ((1ull << s) < v) ++s;
        m = static_cast<uint32_t>(((1ull << (31 + s)) + v - 1) / v);
    }
    __device__ __forceinline__ int32_t operator()(int32_t x) const {
        return static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(x)) * m) >> (31 + s));
    }
};

// How an operand lies in memory: K contiguous; rows contiguous; rows contiguous
// and a multiple of 64, which one copy takes whole.
enum : int32_t { kLayoutK = 0, kLayoutRows = 1, kLayoutBlocks = 2 };

struct TcArgs {
    CUtensorMap a[2], b[2], c[2], x;
    FastDiv by_tiles, by_group, by_height, by_last_height, by_tiles_n;   // divisors of the unit numbers
    int64_t m, n;
    int32_t k_iters;       // stages of one source
    int32_t k_total;       // stages of all sources
    int32_t tiles_m, tiles_n, n_sources;
    int32_t splits, split_iters;   // slices of K, stages of a slice
    int32_t hb;
    int32_t a_layout, b_layout;    // kLayout*
    int32_t act;
    int32_t has_extra;
    const float* row_scale;
    const float* col_scale[2];
    const float* bias;
    float* part;           // kEpiActGrad: column sums of 32 rows each, [8 tiles_m][n], or null;
                           // kEpiPlain: with splits > 1, [splits][n_sources][m][n] by c[0]
    int32_t tiles, units;  // of the product; tiles splits
    // outputs that a tensor-map store does not take (it wants 16-byte aligned rows
    // and clips them at 16 bytes): stored a row at a time
    int32_t direct;        // 0: by c[]; 1: rows of whole 4-byte words; 2: others
    __nv_bfloat16* out[2];
    int64_t ld_out;
};

// A launch: one product, or two plain ones.  The units (tile, slice of K) of
// the first come before those of the second, and CTA pairs take them in turn.
// Where the first product's last turn is short, the pairs without a unit in it
// take `rounds` units of the second instead (about as long), and the others
// follow.
template <int EPI>
struct TcLaunch {
    static constexpr int kMax = EPI == kEpiPlain ? 2 : 1;
    TcArgs g[kMax];
    int32_t count;
    int32_t late, rounds;  // first pair without a unit in the short turn (0: none is short)
    int32_t trigger;       // whether the next kernel may be scheduled early
    int32_t* status;
};

constexpr int kStages = 5;
constexpr int kSmem = 1024 + kStages * kStage + kEpiWarps * kStaging + 512;
static_assert(kSmem <= 227 * 1024, "shared memory per CTA");

// Columns of an epilogue warp's block: one staging buffer of 128-byte rows, or
// two of 64-byte rows where there are two outputs.
__host__ __device__ constexpr int block_columns(int epi) { return epi == kEpiGatedGrad ? 32 : 64; }

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
}

// Eight fp32 values, as their bits, to bf16.
__device__ __forceinline__ uint4 pack8(const uint32_t* v) {
    auto two = [&](int j) { return bf16x2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])); };
    return make_uint4(two(0), two(2), two(4), two(6));
}

// Sums of the fp32 values v[j] (as bits) over the 32 lanes: lanes l and l + 16
// return that of column l < 16.
__device__ __forceinline__ float column_sum16(uint32_t (&v)[16], int lane) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const uint32_t send = up ? v[j] : v[j + o];
            const float keep = __uint_as_float(up ? v[j + o] : v[j]);
            v[j] = __float_as_uint(keep + __uint_as_float(__shfl_xor_sync(0xFFFFFFFFu, send, o)));
        }
    }
    const float s = __uint_as_float(v[0]);
    return s + __shfl_xor_sync(0xFFFFFFFFu, s, 16);
}

// A block's 64 values of a column vector, two in each lane, from where the
// epilogue passes them round: loaded where they are used, each 16 of them would
// wait on L1 (8192 x 4096 x 4096 e4m3 with bias and GELU 97.9 us, passed round 93.1).
struct Columns {
    float v[2];
    __device__ __forceinline__ void load(const float* p, int64_t n0, int64_t n, int lane) {
        v[0] = n0 + lane < n ? __ldg(p + n0 + lane) : 0.0f;
        v[1] = n0 + lane + 32 < n ? __ldg(p + n0 + lane + 32) : 0.0f;
    }
    __device__ __forceinline__ float at(int c) const { return __shfl_sync(0xFFFFFFFFu, c < 32 ? v[0] : v[1], c & 31); }
};

template <int EPI, bool E4M3>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) k_dense_tc(const __grid_constant__ TcLaunch<EPI> L) {
    constexpr int S = kStages;
    constexpr int kBC = block_columns(EPI);
    constexpr bool kDual = EPI == kEpiGated || EPI == kEpiGatedGrad;
    constexpr bool kExtra = EPI != kEpiGated && EPI != kEpiPlain;
    constexpr bool kDirect = EPI == kEpiLinear || EPI == kEpiGated || EPI == kEpiPlain;   // (the others' outputs are the library's)
    constexpr bool kScaled = E4M3 && EPI != kEpiPlain;
    constexpr bool kBias = EPI == kEpiLinear || EPI == kEpiActGrad;
    constexpr int kBK = E4M3 ? 128 : 64;      // K elements of a stage
    constexpr int CW = 16;                    // accumulator columns a thread takes at once
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
    uint8_t* staging = smem + S * kStage;
    uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kEpiWarps * kStaging);
    uint64_t* full = bars;              // [S]  (CTA 0's are used)
    uint64_t* empty = full + S;         // [S]
    uint64_t* acc_full = empty + S;     // [2]
    uint64_t* acc_empty = acc_full + 2; // [2]  (CTA 0's are used)
    uint64_t* exit_bar = acc_empty + 2;
    uint64_t* extra_full = exit_bar + 1;   // [kEpiWarps]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(extra_full + kEpiWarps);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(&full[s], 2);   // one arrival per operand
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&acc_full[b], 1);
            ptx::mbar_init(&acc_empty[b], kEpiWarps);   // a set of either CTA
        }
        ptx::mbar_init(exit_bar, 1);
        for (int w = 0; w < kEpiWarps; ++w) ptx::mbar_init(&extra_full[w], 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_map(&L.g[0].a[0]);
        ptx::prefetch_map(&L.g[0].b[0]);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(tmem_slot, kTmemCols);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    pdl_wait();
    // The next product's blocks may be scheduled as this one's leave the SMs.
    // The sums that follow partial results may not: their small blocks would
    // crowd on the SMs that are free first (a weight gradient and its sum of
    // slices, 15052 x 512 x 512: 22.7 us, against 19.7).
    if (L.trigger) pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    const uint32_t smem_base = ptx::smem_u32(smem);

    auto fail = [&]() {
        atomicOr(L.status, kStatusTimeout);
        *abort_flag = 1;
    };
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, ptx::mbar_wait(bar, parity, abort_flag));
    };
    const int32_t pair = static_cast<int32_t>(blockIdx.x >> 1), n_pairs = static_cast<int32_t>(gridDim.x >> 1);
    struct Unit {
        int32_t g, tm, tn, src, k0, k1, split;
    };
    // The k-th unit of this pair; false past its last one.
    const int32_t mine0 = (L.g[0].units - pair + n_pairs - 1) / n_pairs;   // its units of the first product
    auto unit_at = [&](int32_t k, Unit& t) -> bool {
        int32_t u;
        if (k < mine0) {
            t.g = 0;
            u = pair + k * n_pairs;
        } else {
            if (EPI != kEpiPlain || L.count == 1) return false;
            t.g = 1;
            k -= mine0;
            const int32_t idle = n_pairs - L.late, ahead = L.rounds * idle;   // (late = 0: rounds = 0)
            if (pair < L.late || L.rounds == 0) u = ahead + pair + k * n_pairs;
            else u = k < L.rounds ? pair - L.late + k * idle : ahead + pair + (k - L.rounds) * n_pairs;
            if (u >= L.g[TcLaunch<EPI>::kMax - 1].units) return false;
        }
        const TcArgs& p = L.g[EPI == kEpiPlain ? t.g : 0];
        const int32_t tiles_nn = p.tiles_n * p.n_sources;
        t.split = p.by_tiles(u);
        const int32_t i = u - t.split * p.tiles;
        const int32_t grp = p.by_group(i);
        const int32_t first = grp * kGroupM;
        const int32_t r = i - grp * kGroupM * tiles_nn;
        const bool last = p.tiles_m - first < kGroupM;
        const int32_t gm = last ? p.tiles_m - first : kGroupM;
        const int32_t nn = last ? p.by_last_height(r) : p.by_height(r);
        t.tm = first + r - nn * gm;
        t.src = p.by_tiles_n(nn);
        t.tn = nn - t.src * p.tiles_n;
        t.k0 = t.split * p.split_iters;
        t.k1 = t.k0 + p.split_iters < p.k_total ? t.k0 + p.split_iters : p.k_total;
        return true;
    };
    auto args_of = [&](const Unit& t) -> const TcArgs& { return L.g[EPI == kEpiPlain ? t.g : 0]; };

    uint32_t fills = 0;   // stages this thread has filled
    if (warp == kLoadA || warp == kLoadB) {
        // ---------------- loads of one operand
        if (lane == 0) {
            const bool is_a = warp == kLoadA;
            uint32_t& f = fills;
            bool ok = true;
            Unit t;
            for (int32_t q = 0; ok && unit_at(q, t); ++q) {
                const TcArgs& p = args_of(t);
                const int32_t rows = is_a ? kRowsA : p.hb;
                const int32_t layout = is_a ? p.a_layout : p.b_layout;
                const uint32_t bytes = 2u * static_cast<uint32_t>(rows) * 128u;   // of both CTAs
                const int32_t r0 = is_a    ? t.tm * 256 + static_cast<int32_t>(rank) * kRowsA
                                   : kDual ? t.tn * p.hb
                                           : t.tn * 2 * p.hb + static_cast<int32_t>(rank) * p.hb;
                const CUtensorMap* map0 = is_a ? &p.a[0] : &p.b[kDual ? rank : t.src];
                for (int32_t it = t.k0; it < t.k1; ++it, ++f) {
                    const uint32_t s = f % S;
                    if (f >= S && !ptx::mbar_wait(&empty[s], (f / S - 1) & 1, abort_flag)) {
                        fail();
                        ok = false;
                        break;
                    }
                    const bool second = it >= p.k_iters;   // the second source of a sum over two
                    const int32_t k = (second ? it - p.k_iters : it) * kBK;
                    const CUtensorMap* map = second ? map0 + 1 : map0;
                    if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], bytes);
                    const uint32_t bar = ptx::map_to_rank(ptx::smem_u32(&full[s]), 0);
                    const uint32_t dst = smem_base + s * kStage + (is_a ? 0 : kStageA);
                    if (layout == kLayoutK) {
                        ptx::tma_load_2d_pair(dst, map, k, r0, bar);
                    } else if (layout == kLayoutBlocks) {
                        ptx::tma_load_3d_pair(dst, map, 0, k, r0 >> 6, bar);
                    } else {
                        ptx::tma_load_2d_pair(dst, map, r0, k, bar);
                        if (rows > 64) ptx::tma_load_2d_pair(dst + 8192, map, r0 + 64, k, bar);
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issue (the warp runs the loop, lane 0 of CTA 0 issues)
        if (rank == 0) {
            const uint32_t leader = lane == 0;
            uint32_t f = 0;
            bool ok = true;
            Unit t;
            for (int32_t ai = 0; ok && unit_at(ai, t); ++ai) {
                const TcArgs& p = args_of(t);
                const bool a_k = p.a_layout == kLayoutK, b_k = p.b_layout == kLayoutK;
                const uint32_t idesc = ptx::idesc_dense(E4M3, a_k, b_k, 256, static_cast<uint32_t>(2 * p.hb));
                const uint64_t a0 = a_k ? ptx::sdesc_k128(smem_base) : ptx::sdesc_mn128(smem_base, 64);
                const uint64_t b0 = b_k ? ptx::sdesc_k128(smem_base + kStageA) : ptx::sdesc_mn128(smem_base + kStageA, 64);
                // one MMA contracts 32 bytes of a K-major row, or 16 rows of 128 bytes
                const uint64_t da = a_k ? 2 : 128, db = b_k ? 2 : 128;
                const int buf = ai & 1;
                const uint32_t v = static_cast<uint32_t>(ai >> 1);
                if (v > 0 && !warp_wait(&acc_empty[buf], (v - 1) & 1)) {
                    if (lane == 0) fail();
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(buf * 256);
                for (int32_t it = t.k0; it < t.k1; ++it, ++f) {
                    const uint32_t s = f % S;
                    if (!warp_wait(&full[s], (f / S) & 1)) {
                        if (lane == 0) fail();
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint64_t off = static_cast<uint64_t>((s * kStage) >> 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        ptx::mma_pair_if<E4M3>(leader, d, a0 + off + j * da, b0 + off + j * db, idesc,
                                               (it > t.k0 || j > 0) ? 1u : 0u);
                    ptx::mma_commit_pair_if(leader, &empty[s]);
                }
                if (ok) ptx::mma_commit_pair_if(leader, &acc_full[buf]);
            }
            // every MMA, and every arrival it sends to either CTA, is done once
            // exit_bar flips; TMEM is freed after that
            ptx::mma_commit_pair_if(leader, exit_bar);
            const bool done = __all_sync(0xFFFFFFFFu, ptx::mbar_wait(exit_bar, 0, nullptr));
            if (!done && lane == 0) atomicOr(L.status, kStatusTimeout);
        }
    } else {
        // ---------------- epilogue
        const int e = warp - 2;
        const int quarter = warp & 3;            // the TMEM lanes a warp may read
        const int half = (e >> 2) & 1, buf = e >> 3;   // which blocks of columns; the set, and its accumulator
        uint8_t* stage0 = staging + e * kStaging;
        const uint32_t st0 = ptx::smem_u32(stage0);
        const uint32_t row_off = static_cast<uint32_t>(lane) * (kBC * 2);
        const uint32_t sw = kBC == 64 ? lane & 7 : (lane >> 1) & 3;   // the copies' 128- or 64-byte swizzle
        uint64_t* xbar = &extra_full[e];
        uint32_t xphase = 0;
        const uint32_t acc_bar = ptx::map_to_rank(ptx::smem_u32(&acc_empty[0]), 0);
        bool ok = true;
        Unit t;
        for (int32_t ai = buf; ok && unit_at(ai, t); ai += 2) {
            const TcArgs& p = args_of(t);
            const int blocks = (kDual ? p.hb : 2 * p.hb) / kBC;
            const bool to_part = EPI == kEpiPlain && p.part;   // fp32 sums of a slice, not staged
            const int32_t m0 = t.tm * 256 + static_cast<int32_t>(rank) * kRowsA + quarter * 32;
            const int64_t row = m0 + lane;
            const int32_t col0 = t.tn * (kDual ? p.hb : 2 * p.hb);
            const bool rows_live = m0 < p.m;
            const bool row_live = row < p.m;
            const float rs = (kScaled && row_live) ? p.row_scale[row] : 1.0f;
            bool waited = false;
            auto wait_acc = [&]() {
                if (waited) return;
                waited = true;
                if (!warp_wait(&acc_full[buf], (static_cast<uint32_t>(ai) >> 1) & 1)) {
                    if (lane == 0) fail();
                    ok = false;
                }
                ptx::tc_fence_after();
            };
            for (int c = half; ok && c < blocks; c += 2) {
                const int32_t n0 = col0 + c * kBC;
                if (!(rows_live && n0 < p.n)) continue;
                if (!to_part) {
                    // the staging buffer is free once its last store has been read out
                    if (lane == 0) {
                        ptx::bulk_wait_read();
                        if (kExtra && p.has_extra) {
                            ptx::mbar_arrive_expect_tx(xbar, 32 * kBC * 2);
                            ptx::tma_load_2d(st0, &p.x, n0, m0, ptx::smem_u32(xbar));
                        }
                    }
                    __syncwarp();
                }
                Columns scale0, scale1, bias;
                if (kScaled) scale0.load(p.col_scale[0], n0, p.n, lane);
                if (kScaled && kDual) scale1.load(p.col_scale[1], n0, p.n, lane);
                if (kBias && p.bias) bias.load(p.bias, n0, p.n, lane);
                wait_acc();
                if (kExtra && p.has_extra) {
                    // (also after a failed wait: the copy must land before the CTA exits)
                    if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(xbar, xphase, nullptr))) {
                        if (lane == 0) fail();
                        ok = false;
                    }
                    xphase ^= 1;
                }
                const uint32_t ta = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                    static_cast<uint32_t>(buf * 256 + c * kBC);
                if (!ok) break;
                if (to_part) {
                    // 32 columns of fp32 fill the staging buffer
#pragma unroll 1
                    for (int q = 0; q < 2 && n0 + q * 32 < p.n; ++q) {
                        if (lane == 0) ptx::bulk_wait_read();
                        __syncwarp();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t z[CW];
                            ptx::tmem_ld_32x32b_x16(ta + q * 32 + h * CW, z);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < CW; j += 4)
                                *reinterpret_cast<uint4*>(stage0 + row_off + (((h * 4 + j / 4) ^ sw) << 4)) =
                                    make_uint4(z[j], z[j + 1], z[j + 2], z[j + 3]);
                        }
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            ptx::tma_store_3d(&p.c[0], n0 + q * 32, m0, t.split * p.n_sources + t.src, st0);
                            ptx::bulk_commit();
                        }
                    }
                    continue;
                }
#pragma unroll 2
                for (int h = 0; h < kBC / CW; ++h) {
                    uint32_t z[CW], w[CW];
                    ptx::tmem_ld_32x32b_x16(ta + h * CW, z);
                    if (kDual) ptx::tmem_ld_32x32b_x16(ta + p.hb + h * CW, w);
                    ptx::tmem_ld_wait();
                    const int32_t nc = n0 + h * CW;
                    const uint32_t piece = h * (CW / 8);   // first 16-byte piece of these columns in a row
                    // extra: this thread's CW columns, 16-byte pieces in the 128-byte swizzle
                    uint32_t x[CW / 2];
                    if (kExtra) {
#pragma unroll
                        for (int q = 0; q < CW / 8; ++q) {
                            uint4 v = make_uint4(0, 0, 0, 0);
                            if (p.has_extra) v = *reinterpret_cast<const uint4*>(stage0 + row_off + (((piece + q) ^ sw) << 4));
                            x[4 * q] = v.x;
                            x[4 * q + 1] = v.y;
                            x[4 * q + 2] = v.z;
                            x[4 * q + 3] = v.w;
                        }
                    }
                    // two columns at a time; the results take the places of what they are
                    // made of: y in z, the second output in w
                    auto pair_of = [](const uint32_t* v) { return F2(__uint_as_float(v[0]), __uint_as_float(v[1])); };
                    auto keep = [](uint32_t* v, F2 y) {
                        float lo, hi;
                        y.get(lo, hi);
                        v[0] = __float_as_uint(lo);
                        v[1] = __float_as_uint(hi);
                    };
                    auto columns = [&](const Columns& v, int j) { return F2(v.at(h * CW + j), v.at(h * CW + j + 1)); };
                    if (kScaled) {
#pragma unroll
                        for (int j = 0; j < CW; j += 2) {
                            keep(z + j, pair_of(z + j) * (F2(rs) * columns(scale0, j)));
                            if (kDual) keep(w + j, pair_of(w + j) * (F2(rs) * columns(scale1, j)));
                        }
                    }
                    if (kBias && p.bias) {
#pragma unroll
                        for (int j = 0; j < CW; j += 2) keep(z + j, pair_of(z + j) + columns(bias, j));
                    }
                    if (EPI != kEpiPlain) with_act(p.act, [&](auto act) {
#pragma unroll
                        for (int j = 0; j < CW; j += 2) {
                            const F2 zz = pair_of(z + j), ww = kDual ? pair_of(w + j) : F2(0.0f);
                            const F2 xx = kExtra ? F2(__uint_as_float(x[j / 2] << 16), __uint_as_float(x[j / 2] & 0xFFFF0000u)) : F2(0.0f);
                            F2 y;
                            if (EPI == kEpiLinear) {
                                y = act_f<act>(zz) + xx;
                            } else if (EPI == kEpiGated) {
                                y = act_f<act>(zz) * ww;
                            } else {
                                F2 a;
                                const F2 slope = act_grad_f<act>(zz, &a);
                                if (EPI == kEpiActGrad) {
                                    y = row_live ? xx * slope : F2(0.0f);
                                } else {
                                    y = xx * ww * slope;
                                    keep(w + j, xx * a);
                                }
                            }
                            keep(z + j, y);
                        }
                    });
#pragma unroll
                    for (int q = 0; q < CW / 8; ++q) {
                        const uint32_t at = row_off + (((piece + q) ^ sw) << 4);
                        *reinterpret_cast<uint4*>(stage0 + at) = pack8(z + 8 * q);
                        if (EPI == kEpiGatedGrad) *reinterpret_cast<uint4*>(stage0 + kStaging / 2 + at) = pack8(w + 8 * q);
                    }
                    if constexpr (EPI == kEpiActGrad) {
                        if (p.part) {
                            const float s = column_sum16(z, lane);
                            const int64_t pr = static_cast<int64_t>(t.tm) * 8 + rank * 4 + quarter;
                            if (lane < CW && nc + lane < p.n) p.part[pr * p.n + nc + lane] = s;
                        }
                    }
                }
                if (kDirect && p.direct) {
                    __syncwarp();
                    // lane l has columns 2 l and 2 l + 1 of a row: one 128-byte row a store
                    __nv_bfloat16* out = p.out[EPI == kEpiPlain ? t.src : 0] + m0 * p.ld_out + n0 + 2 * lane;
                    const int32_t left = static_cast<int32_t>(p.n - n0 - 2 * lane < 3 ? p.n - n0 - 2 * lane : 3);
                    const int32_t rows = static_cast<int32_t>(p.m - m0 < 32 ? p.m - m0 : 32);
                    auto lo = [](uint32_t v) { return __ushort_as_bfloat16(static_cast<uint16_t>(v & 0xFFFFu)); };
                    auto hi = [](uint32_t v) { return __ushort_as_bfloat16(static_cast<uint16_t>(v >> 16)); };
                    auto staged = [&](int32_t r) {
                        return *reinterpret_cast<const uint32_t*>(stage0 + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
                    };
                    if (p.direct == 1) {
#pragma unroll 4
                        for (int32_t r = 0; r < rows; ++r, out += p.ld_out) {
                            const uint32_t v = staged(r);
                            if (left > 1) *reinterpret_cast<uint32_t*>(out) = v;
                            else if (left == 1) out[0] = lo(v);
                        }
                    } else {
                        // a row that starts inside a 4-byte word takes columns 2 l + 1 and
                        // 2 l + 2 (dx of 35309 x 459 x 228: 31.8 us, by single columns 35.7)
#pragma unroll 4
                        for (int32_t r = 0; r < rows; ++r, out += p.ld_out) {
                            const uint32_t v = staged(r), next = __shfl_down_sync(0xFFFFFFFFu, v, 1);
                            if ((reinterpret_cast<uintptr_t>(out) & 2) == 0) {
                                if (left > 1) *reinterpret_cast<uint32_t*>(out) = v;
                                else if (left == 1) out[0] = lo(v);
                            } else {
                                if (lane == 0 && left > 0) out[0] = lo(v);
                                if (lane < 31 && left > 2) *reinterpret_cast<uint32_t*>(out + 1) = (v >> 16) | (next << 16);
                                else if (left > 1) out[1] = hi(v);
                            }
                        }
                    }
                    ptx::fence_proxy_async_smem();   // (the next residual's copy comes into the same bytes)
                    __syncwarp();
                    continue;
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ptx::tma_store_2d(&p.c[EPI == kEpiPlain ? t.src : 0], n0, m0, st0);
                    if (EPI == kEpiGatedGrad) ptx::tma_store_2d(&p.c[1], n0, m0, st0 + kStaging / 2);
                    ptx::bulk_commit();
                }
            }
            wait_acc();   // (a warp without a block of this tile still takes its turn)
            // rows past m of the column sums: whole 32-row groups without a row
            if (EPI == kEpiActGrad && p.part && !rows_live) {
                const int64_t pr = static_cast<int64_t>(t.tm) * 8 + rank * 4 + quarter;
                for (int c = half; c < blocks; c += 2)
                    for (int32_t n = col0 + c * kBC + lane; n < col0 + (c + 1) * kBC && n < p.n; n += 32)
                        p.part[pr * p.n + n] = 0.0f;
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) ptx::mbar_arrive_cluster(acc_bar + static_cast<uint32_t>(buf) * 8);
        }
        if (lane == 0) ptx::bulk_wait();
        __syncwarp();
    }
    // neither CTA leaves, or frees TMEM, while the other may still signal it:
    // once both have ended their roles, CTA 1 waits for the last arrival that
    // CTA 0's MMAs send it
    ptx::tc_fence_before();
    ptx::cluster_sync();
    if (rank == 0 && fills && *abort_flag)   // given up: loads of either CTA still in flight land first
        for (uint32_t q = fills > S ? fills - S : 0; q < fills; ++q) ptx::mbar_wait(&full[q % S], (q / S) & 1, nullptr);
    __syncwarp();
    if (warp == 1 && rank == 1 && !ptx::mbar_wait(exit_bar, 0, nullptr)) atomicOr(L.status, kStatusTimeout);
    __syncwarp();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc_pair(tmem, kTmemCols);
}

// ---- host -------------------------------------------------------------------
template <int EPI, bool E4M3>
int launch(const TcLaunch<EPI>& args, int64_t units, cudaStream_t s) {
    static bool set[kMaxDevices] = {};
    int dev = 0;
    SPCONV_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return SPCONV_ERR_UNSUPPORTED;
    if (!set[dev]) {
        SPCONV_CHECK_CUDA(cudaFuncSetAttribute(k_dense_tc<EPI, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSmem));
        set[dev] = true;
    }
    const unsigned pairs = static_cast<unsigned>(units < kPairs ? units : kPairs);
    return launch_pdl(k_dense_tc<EPI, E4M3>, dim3(2 * pairs), kThreads, kSmem, s, args);
}

}  // namespace

namespace {
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

}  // namespace

int make_tensor_map(CUtensorMap* map, const void* base, size_t es, int64_t inner, int64_t outer, int64_t ld, int32_t box_outer,
                    int32_t box_bytes) {
    const EncodeFn fn = encode_fn();
    if (!fn) return SPCONV_ERR_CUDA;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * es};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes / es), static_cast<cuuint32_t>(box_outer)};
    const cuuint32_t unit[2] = {1, 1};
    const CUresult r = fn(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                          const_cast<void*>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SPCONV_OK : SPCONV_ERR_CUDA;
}

int make_tensor_map_blocks(CUtensorMap* map, const void* base, int64_t inner, int64_t outer, int64_t ld, int32_t blocks) {
    const EncodeFn fn = encode_fn();
    if (!fn) return SPCONV_ERR_CUDA;
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(outer), static_cast<cuuint64_t>(inner / 64)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, 128};
    const cuuint32_t box[3] = {64, 64, static_cast<cuuint32_t>(blocks)};
    const cuuint32_t unit[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, unit,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SPCONV_OK : SPCONV_ERR_CUDA;
}

namespace {

// How a product is cut into units, and a model of its time in us.  A step of K
// of a 256-column tile takes 0.37 us and one of a 128-column tile 0.34 (both
// bound by the loads: 32 and 24 KB per SM and step; 1024 and 300 rows x 4096 x
// 4096).  Where there are few steps the epilogue bounds a tile: 1.6 and 1.1 us,
// or 2.6 and 1.7 with an activation per column or with a residual (32371 x 96 x
// 384 with SiLU in narrow tiles 12.6 us, in wide ones 14.2; x 128 x 512: 14.9 and
// 14.7), and that of the last tile runs alone.  A launch of sums takes 3 us and the fp32
// partial results move at 6 TB/s.
struct Cut {
    int32_t hb = 128, splits = 1, split_iters = 1;
    int64_t tiles = 0;
    double us = 0.0;
};

Cut best_cut(const DenseOp& op, bool dual, int outputs, bool may_split) {
    const int64_t k_total = ceil_div(op.k, op.dtype == SPCONV_E4M3 ? 128 : 64) * op.k_sources;
    const int64_t tiles_m = ceil_div(op.m, 256);
    const bool more = !may_split && (op.epi == kEpiActGrad || op.epi == kEpiGatedGrad ||
                                     (op.epi == kEpiLinear && (op.act != SPCONV_ACT_NONE || op.extra)));
    Cut best;
    best.us = 1e30;
    for (int32_t hb : {128, 64}) {
        const double step = hb == 128 ? 0.37 : 0.34, epi = hb == 128 ? (more ? 2.6 : 1.6) : (more ? 1.7 : 1.1);
        const int64_t tiles = tiles_m * ceil_div(op.n, dual ? hb : 2 * hb) * outputs;
        int64_t most = may_split && tiles < kPairs ? kPairs / tiles : 1;
        if (most > k_total / 8) most = k_total / 8;
        for (int64_t splits = 1; splits == 1 || splits <= most; ++splits) {
            const int64_t iters = ceil_div(k_total, splits), used = ceil_div(k_total, iters);
            if (used != splits) continue;   // the same cut as a smaller count
            const double unit = static_cast<double>(iters) * step > epi ? static_cast<double>(iters) * step : epi;
            double us = static_cast<double>(ceil_div(tiles * splits, kPairs)) * unit + epi;
            if (splits > 1) us += 3.0 + 8.0e-6 / 6.0 * static_cast<double>(op.m * op.n * outputs) * static_cast<double>(splits);
            if (us < best.us) {
                best.hb = hb;
                best.splits = static_cast<int32_t>(splits);
                best.split_iters = static_cast<int32_t>(iters);
                best.tiles = tiles;
                best.us = us;
            }
        }
    }
    return best;
}

// Rows of the fp32 partial results: whole 16 bytes.
int64_t part_ld(int64_t n) { return static_cast<int64_t>(round_up(static_cast<size_t>(n), 4)); }

// The slices [slices][m][part_ld(n)], stored in boxes of 32 columns x 32 rows,
// clipped at each slice's last row.
int make_part_map(CUtensorMap* map, float* base, int64_t n, int64_t m, int32_t slices) {
    const EncodeFn fn = encode_fn();
    if (!fn) return SPCONV_ERR_CUDA;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(m), static_cast<cuuint64_t>(slices)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(part_ld(n)) * 4, static_cast<cuuint64_t>(part_ld(n) * m) * 4};
    const cuuint32_t box[3] = {32, 32, 1}, unit[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, unit,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SPCONV_OK : SPCONV_ERR_CUDA;
}

// An epilogue's product with K cut: gate and up are two outputs of a plain one.
DenseOp as_plain(const DenseOp& op) {
    DenseOp o = op;
    if (op.epi == kEpiGated || op.epi == kEpiGatedGrad) o.n_sources = 2;
    o.epi = kEpiLinear;
    return o;
}

// Everything of a product but its workspace.
int set_args(const DenseOp& op, bool may_split, TcArgs* args) {
    const size_t es = op.dtype == SPCONV_E4M3 ? 1 : 2;
    const int32_t bk = static_cast<int32_t>(128 / es);
    const bool dual = op.epi == kEpiGated || op.epi == kEpiGatedGrad;
    TcArgs& p = *args;
    p = {};
    p.m = op.m;
    p.n = op.n;
    p.k_iters = static_cast<int32_t>(ceil_div(op.k, bk));
    p.k_total = p.k_iters * op.k_sources;
    p.n_sources = op.n_sources;
    auto layout = [](const Operand& t, int64_t rows) { return t.k_major ? kLayoutK : rows % 64 == 0 ? kLayoutBlocks : kLayoutRows; };
    p.a_layout = layout(op.a, op.m);
    p.b_layout = layout(op.b, op.n);
    p.act = op.act;
    p.has_extra = op.extra != nullptr;
    p.row_scale = op.row_scale;
    p.col_scale[0] = op.col_scale[0];
    p.col_scale[1] = op.col_scale[1];
    p.bias = op.bias;
    const Cut cut = best_cut(op, dual, op.n_sources, may_split);
    p.hb = cut.hb;
    p.tiles_m = static_cast<int32_t>(ceil_div(op.m, 256));
    p.tiles_n = static_cast<int32_t>(ceil_div(op.n, dual ? p.hb : 2 * p.hb));
    p.splits = cut.splits;
    p.split_iters = cut.split_iters;
    if (cut.tiles * p.splits > 0x3FFFFFFF) return SPCONV_ERR_UNSUPPORTED;
    p.tiles = static_cast<int32_t>(cut.tiles);
    p.units = p.tiles * p.splits;
    p.by_tiles = FastDiv(static_cast<uint32_t>(p.tiles));
    p.by_group = FastDiv(static_cast<uint32_t>(kGroupM * p.tiles_n * p.n_sources));
    p.by_height = FastDiv(kGroupM);
    p.by_last_height = FastDiv(p.tiles_m % kGroupM ? p.tiles_m % kGroupM : kGroupM);
    p.by_tiles_n = FastDiv(static_cast<uint32_t>(p.tiles_n));
    auto operand = [&](CUtensorMap* map, const Operand& t, int i, int32_t lay, int64_t rows, int32_t box) {
        return lay == kLayoutK      ? make_tensor_map(map, t.p[i], es, op.k, rows, t.ld, box)
               : lay == kLayoutRows ? make_tensor_map(map, t.p[i], es, rows, op.k, t.ld, 64)
                                    : make_tensor_map_blocks(map, t.p[i], rows, op.k, t.ld, box / 64);
    };
    for (int i = 0; i < op.k_sources; ++i) SPCONV_CHECK(operand(&p.a[i], op.a, i, p.a_layout, op.m, kRowsA));
    for (int i = 0; i < ((dual || op.k_sources == 2 || op.n_sources == 2) ? 2 : 1); ++i)
        SPCONV_CHECK(operand(&p.b[i], op.b, i, p.b_layout, op.n, p.hb));
    const int outs = op.epi == kEpiGatedGrad || op.n_sources == 2 ? 2 : 1;
    uintptr_t at = static_cast<uintptr_t>(op.ld_out) * 2;
    bool mapped = op.n % 8 == 0 || op.out_padded;
    for (int i = 0; i < outs; ++i) {
        mapped = mapped && tma_ok(op.out[i], op.ld_out, 2);
        at |= reinterpret_cast<uintptr_t>(op.out[i]);
        p.out[i] = static_cast<__nv_bfloat16*>(op.out[i]);
    }
    p.ld_out = op.ld_out;
    p.direct = mapped ? 0 : at % 4 == 0 ? 1 : 2;
    for (int i = 0; p.splits == 1 && mapped && i < outs; ++i)
        SPCONV_CHECK(make_tensor_map(&p.c[i], op.out[i], 2, op.n, op.m, op.ld_out, 32, 2 * block_columns(op.epi)));
    if (op.extra && p.splits == 1) SPCONV_CHECK(make_tensor_map(&p.x, op.extra, 2, op.n, op.m, op.ld_extra, 32, 2 * block_columns(op.epi)));
    return SPCONV_OK;
}

template <int EPI, bool E4M3>
int run_one(const DenseOp& op, int32_t* status, cudaStream_t s) {
    TcLaunch<EPI> l = {};
    SPCONV_CHECK(set_args(op, false, &l.g[0]));
    l.count = 1;
    l.g[0].part = op.col_part;
    l.trigger = op.col_part == nullptr;
    l.status = status;
    return launch<EPI, E4M3>(l, l.g[0].units, s);
}

}  // namespace

int dense_tc_run(const DenseOp& op, int32_t* status, cudaStream_t s) {
    const bool eight = op.dtype == SPCONV_E4M3;
    switch (op.epi) {
        case kEpiGated: return eight ? run_one<kEpiGated, true>(op, status, s) : run_one<kEpiGated, false>(op, status, s);
        case kEpiActGrad: return run_one<kEpiActGrad, false>(op, status, s);
        case kEpiGatedGrad: return run_one<kEpiGatedGrad, false>(op, status, s);
        default: return eight ? run_one<kEpiLinear, true>(op, status, s) : run_one<kEpiLinear, false>(op, status, s);
    }
}

bool dense_tc_cuts(const DenseOp& op) {
    if (op.plain()) return true;
    const DenseOp o = as_plain(op);
    const Cut cut = best_cut(o, false, o.n_sources, true);
    return cut.splits > 1 && cut.us < best_cut(op, op.epi == kEpiGated || op.epi == kEpiGatedGrad, 1, false).us;
}

int dense_tc_plain(const DenseOp* ops, int count, const ColumnSums& cols, int32_t* status, cudaStream_t s) {
    TcLaunch<kEpiPlain> l = {};
    l.count = count;
    l.status = status;
    // the product of the longer units first
    int order[2] = {0, 1};
    int64_t cost[2] = {0, 0};
    for (int i = 0; i < count; ++i) {
        SPCONV_CHECK(set_args(as_plain(ops[i]), true, &l.g[i]));
        cost[i] = static_cast<int64_t>(l.g[i].split_iters) * l.g[i].hb;
    }
    if (count == 2 && cost[1] > cost[0]) {
        const TcArgs t = l.g[0];
        l.g[0] = l.g[1];
        l.g[1] = t;
        order[0] = 1;
        order[1] = 0;
    }
    int64_t units = 0;
    size_t bytes = 0, off[2] = {0, 0};
    for (int i = 0; i < count; ++i) {
        units += l.g[i].units;
        off[i] = bytes;
        if (l.g[i].splits > 1)
            bytes += round_up(static_cast<size_t>(l.g[i].m) * part_ld(l.g[i].n) * l.g[i].n_sources * l.g[i].splits * 4, 256);
    }
    Scratch part(bytes, s);
    if (part.failed()) return SPCONV_ERR_OOM;
    SliceSums sums[2];
    for (int i = 0; i < count; ++i) {
        TcArgs& p = l.g[i];
        if (p.splits == 1) continue;
        const DenseOp& op = ops[order[i]];
        p.part = part.as<float>(off[i]);
        SPCONV_CHECK(make_part_map(&p.c[0], p.part, p.n, p.m, p.splits * p.n_sources));
        sums[i].ld_part = part_ld(p.n);
        sums[i].part = p.part;
        sums[i].splits = p.splits;
        sums[i].m = p.m;
        sums[i].n = p.n;
        sums[i].outputs = p.n_sources;
        sums[i].out[0] = static_cast<__nv_bfloat16*>(op.out[0]);
        sums[i].out[1] = static_cast<__nv_bfloat16*>(op.out[1]);
        sums[i].ld = op.ld_out;
        sums[i].epi = op.epi;
        sums[i].act = op.act;
        sums[i].row_scale = op.row_scale;
        sums[i].col_scale[0] = op.col_scale[0];
        sums[i].col_scale[1] = op.col_scale[1];
        sums[i].bias = op.bias;
        sums[i].extra = static_cast<const __nv_bfloat16*>(op.extra);
        sums[i].ld_extra = op.ld_extra;
        sums[i].col_part = op.col_part;
    }
    const bool sums_follow = bytes > 0 || cols.out;
    l.trigger = !sums_follow;
    if (count == 2 && units > kPairs) {
        l.late = l.g[0].units % kPairs;
        const int64_t c0 = cost[order[0]], c1 = cost[order[1]];
        if (l.late) l.rounds = static_cast<int32_t>((2 * c0 + c1) / (2 * c1));
    }
    SPCONV_CHECK(ops[0].dtype == SPCONV_E4M3 ? (launch<kEpiPlain, true>(l, units, s)) : (launch<kEpiPlain, false>(l, units, s)));
    if (ops[0].epi == kEpiActGrad || ops[0].epi == kEpiGatedGrad) return finish_grad(sums[0], s);   // (K is cut: dense_tc_cuts)
    return sums_follow ? finish_sums(sums, count, cols, s) : SPCONV_OK;
}

}  // namespace spconv
