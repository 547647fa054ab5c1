// Products with an epilogue for few rows (single tokens up to a small batch).
//
// The weight is the traffic: every byte of it is used for a handful of
// products, so the kernel streams it at the memory's rate and the tensor cores
// only have to keep up.  The roles of the operands are exchanged: 128 output
// channels are the MMA's M (the weight's columns as they lie in memory, or the
// e4m3 weight's rows) and the rows of x its N, padded to 16 instead of 256.
//
// 128 channels x all of K would leave most SMs without work, so a cluster of
// `splits` CTAs cuts K between them.  Each keeps its fp32 sums in shared
// memory and every CTA adds the partial sums of its share of the rows through
// distributed shared memory, in the order of the ranks, applies the epilogue
// and stores: one launch, no workspace, the same bits every run.  An SM keeps
// about 200 KB of loads in flight: two CTAs up to 128 rows (gated: 64), one up
// to twice that, where the sums need the room.  1 x 8192 x 16384 takes 47.5 us,
// 5.7 TB/s of weight; 1 x 4096 x 4096 7.1, of which about 3 are the launch, the
// first loads' latency and the sums.
#include "ptx_sm100.cuh"
#include "tensor_map.cuh"

namespace spconv {
namespace {

constexpr int kThreads = 192;          // warp 0 loads, warp 1 issues MMAs, warps 2-5 read the accumulator
constexpr int kChannels = 128;         // output channels per CTA (MMA M)
constexpr int kTileA = kChannels * 128;
constexpr int kMaxSplits = 8;          // portable cluster size
constexpr int kMaxStages = 8;
constexpr int kWarps = kThreads / 32;

// Four channels of `rows` (<= kBatch) rows summed over the cluster's ranks (S of
// them at most), in their order; at: their addresses in this CTA.
template <int S, int kBatch>
__device__ __forceinline__ void add_ranks(const uint32_t (&at)[kBatch], int rows, uint32_t splits, float (&z)[kBatch][4]) {
    constexpr int kAtOnce = S == 8 ? 1 : kBatch;   // (the loads in flight are registers)
#pragma unroll
    for (int b0 = 0; b0 < kBatch; b0 += kAtOnce) {
        float4 part[kAtOnce][S];
#pragma unroll
        for (int b = 0; b < kAtOnce; ++b)
#pragma unroll
            for (uint32_t r = 0; r < S; ++r)
                part[b][r] = b0 + b < rows && (S < kMaxSplits || r < splits)
                                 ? ptx::ld_cluster_f32x4(ptx::map_to_rank(at[b0 + b], r))
                                 : make_float4(0, 0, 0, 0);
#pragma unroll
        for (int b = 0; b < kAtOnce; ++b) {
            float4 t = part[b][0];
#pragma unroll
            for (int r = 1; r < S; ++r) {
                t.x += part[b][r].x;
                t.y += part[b][r].y;
                t.z += part[b][r].z;
                t.w += part[b][r].w;
            }
            z[b0 + b][0] = t.x;
            z[b0 + b][1] = t.y;
            z[b0 + b][2] = t.z;
            z[b0 + b][3] = t.w;
        }
    }
}

// BIG: one CTA per SM.
template <bool DUAL, bool BIG>
struct FewConfig {
    static constexpr int kRows = (BIG ? 256 : 128) / (DUAL ? 2 : 1);   // of an accumulator
    static constexpr int kCols = (DUAL ? 2 : 1) * kRows;              // TMEM columns (a power of two)
    static constexpr int kRing = (BIG ? 200 : 100) * 1024;            // stages, of one CTA
    static constexpr int kPerSm = BIG ? 1 : 2;
    static_assert(kCols * kChannels * 4 <= kRing, "the sums take the ring's place");
};

struct FewArgs {
    CUtensorMap w[2], x;
    int64_t n;             // channels
    int32_t rows, rows_pad;
    int32_t k_iters;
    int32_t stages, stage_bytes;
    int32_t w_kmajor;
    int32_t act;
    const float* row_scale;
    const float* col_scale[2];
    const float* bias;
    const __nv_bfloat16* extra;
    int64_t ld_extra;
    __nv_bfloat16* out;
    int64_t ld_out;
    int32_t vec_out;       // rows of out take 8-byte stores
    int32_t* status;
};

template <bool DUAL, bool E4M3, bool BIG>
__global__ void __launch_bounds__(kThreads, FewConfig<DUAL, BIG>::kPerSm) k_dense_few(const __grid_constant__ FewArgs p) {
    constexpr int kAcc = DUAL ? 2 : 1;
    constexpr int kBK = E4M3 ? 128 : 64;
    // Rows of a warp's step of the epilogue: more loads together (128 x 512 x 2048 7.4 us,
    // one row at a time 11.9), but more code to fetch (1 row, gated, 1024 x 2048 with two
    // 6.1 us, with one 5.7)
    constexpr int kBatch = DUAL ? 1 : 2;
    constexpr int kRows = FewConfig<DUAL, BIG>::kRows;
    constexpr uint32_t kCols = FewConfig<DUAL, BIG>::kCols;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    uint8_t* ring = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t splits = gridDim.y, rank = blockIdx.y;   // the cluster is one column of the grid
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        ptx::mbar_init(&done, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_map(&p.w[0]);
        ptx::prefetch_map(&p.x);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&tmem_slot, kCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    pdl_wait();
    pdl_trigger();
    const uint32_t tmem = tmem_slot;
    const int32_t n0 = static_cast<int32_t>(blockIdx.x) * kChannels;
    // (k_iters >= splits: no slice is empty)
    const int32_t it0 = static_cast<int32_t>(rank * static_cast<uint32_t>(p.k_iters) / splits);
    const int32_t it1 = static_cast<int32_t>((rank + 1) * static_cast<uint32_t>(p.k_iters) / splits);
    auto fail = [&]() {
        atomicOr(p.status, kStatusTimeout);
        *abort_flag = 1;
    };
    int32_t fills = 0;   // stages this thread has filled
    if (warp == 0) {
        if (lane == 0) {
            const uint32_t bytes = kAcc * kTileA + static_cast<uint32_t>(p.rows_pad) * 128u;
            int32_t& f = fills;
            for (int32_t it = it0; it < it1; ++it, ++f) {
                const int32_t s = f % p.stages;
                if (f >= p.stages && !ptx::mbar_wait(&empty[s], static_cast<uint32_t>(f / p.stages - 1) & 1, abort_flag)) {
                    fail();
                    break;
                }
                const uint32_t base = ptx::smem_u32(ring) + static_cast<uint32_t>(s * p.stage_bytes);
                const uint32_t bar = ptx::smem_u32(&full[s]);
                ptx::mbar_arrive_expect_tx(&full[s], bytes);
#pragma unroll
                for (int a = 0; a < kAcc; ++a) {
                    if (p.w_kmajor) {
                        ptx::tma_load_2d(base + a * kTileA, &p.w[a], it * kBK, n0, bar);
                    } else {
                        ptx::tma_load_2d(base + a * kTileA, &p.w[a], n0, it * kBK, bar);
                        ptx::tma_load_2d(base + a * kTileA + 8192, &p.w[a], n0 + 64, it * kBK, bar);
                    }
                }
                ptx::tma_load_2d(base + kAcc * kTileA, &p.x, it * kBK, 0, bar);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t leader = lane == 0;
        const uint32_t idesc = ptx::idesc_dense(E4M3, p.w_kmajor, true, kChannels, static_cast<uint32_t>(p.rows_pad));
        const uint32_t base = ptx::smem_u32(ring);
        const uint64_t a0 = p.w_kmajor ? ptx::sdesc_k128(base) : ptx::sdesc_mn128(base, 64);
        const uint64_t b0 = ptx::sdesc_k128(base + kAcc * kTileA);
        const uint64_t da = p.w_kmajor ? 2 : 128;
        int32_t f = 0;
        for (int32_t it = it0; it < it1; ++it, ++f) {
            const int32_t s = f % p.stages;
            if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&full[s], static_cast<uint32_t>(f / p.stages) & 1, abort_flag))) {
                if (lane == 0) fail();
                break;
            }
            ptx::tc_fence_after();
            const uint64_t off = static_cast<uint64_t>(s * p.stage_bytes) >> 4;
#pragma unroll
            for (int a = 0; a < kAcc; ++a)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    ptx::mma_if<E4M3>(leader, tmem + a * kRows, a0 + off + a * (kTileA >> 4) + j * da, b0 + off + 2 * j,
                                      idesc, (f > 0 || j > 0) ? 1u : 0u);
            ptx::mma_commit_if(leader, &empty[s]);
        }
        ptx::mma_commit_if(leader, &done);
    }
    // the terms of this lane's channels, while the last products run
    const int64_t n = n0 + 4 * lane;
    float bias[4] = {}, scale[kAcc][4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n + j >= p.n) continue;
        if (!DUAL && p.bias) bias[j] = p.bias[n + j];
        if (E4M3) {
#pragma unroll
            for (int a = 0; a < kAcc; ++a) scale[a][j] = p.col_scale[a][n + j];
        }
    }
    __syncthreads();
    if (*abort_flag)   // given up: loads still in flight land first
        for (int32_t j = fills > p.stages ? fills - p.stages : 0; j < fills; ++j)
            ptx::mbar_wait(&full[j % p.stages], static_cast<uint32_t>(j / p.stages) & 1, nullptr);
    // every MMA of this CTA has completed: its sums are whole, its ring is free
    const bool whole = ptx::mbar_wait(&done, 0, nullptr);
    if (!whole && threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    __syncthreads();
    ptx::tc_fence_after();
    float* sums = reinterpret_cast<float*>(ring);   // [kAcc][rows][kChannels]
    if (warp >= 2) {
        const int quarter = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
#pragma unroll
        for (int a = 0; a < kAcc; ++a)
            for (int32_t r0 = 0; r0 < p.rows; r0 += 16) {
                uint32_t v[16];
                ptx::tmem_ld_32x32b_x16(tmem + lanes + a * kRows + r0, v);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (r0 + j < p.rows) sums[(a * p.rows + r0 + j) * kChannels + quarter * 32 + lane] = __uint_as_float(v[j]);
            }
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    // this CTA's share: rows rank, rank + splits, ..; a warp takes kBatch of them at
    // once (their loads travel together), a lane four channels
    const int32_t mine = (p.rows - static_cast<int32_t>(rank) + static_cast<int32_t>(splits) - 1) / static_cast<int32_t>(splits);
    const uint32_t sums_addr = ptx::smem_u32(sums);
    for (int32_t i0 = warp; i0 < mine && n < p.n; i0 += kBatch * kWarps) {
        const int32_t left = (mine - i0 + kWarps - 1) / kWarps, rows = left < kBatch ? left : kBatch;
        int32_t row[kBatch];
        uint2 x[kBatch];
        float z[kAcc][kBatch][4];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            row[b] = static_cast<int32_t>(rank) + (i0 + b * kWarps) * static_cast<int32_t>(splits);
            x[b] = make_uint2(0, 0);
            if (!DUAL && p.extra && b < rows) {
                const __nv_bfloat16* e = p.extra + row[b] * p.ld_extra + n;   // (tma_ok: 8-byte loads, where the row has four)
                if (n + 4 <= p.n) {
                    x[b] = *reinterpret_cast<const uint2*>(e);
                } else {
                    uint32_t v[3] = {};
                    for (int j = 0; j < 3 && n + j < p.n; ++j) v[j] = __bfloat16_as_ushort(e[j]);
                    x[b] = make_uint2(v[0] | v[1] << 16, v[2]);
                }
            }
        }
#pragma unroll
        for (int a = 0; a < kAcc; ++a) {
            uint32_t at[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) at[b] = sums_addr + static_cast<uint32_t>(((a * p.rows + row[b]) * kChannels + 4 * lane) * 4);
            if (DUAL || splits == 8) add_ranks<8>(at, rows, splits, z[a]);
            else if (splits == 4) add_ranks<4>(at, rows, splits, z[a]);
            else if (splits == 2) add_ranks<2>(at, rows, splits, z[a]);
            else add_ranks<1>(at, rows, splits, z[a]);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (E4M3) {
                const float rs = b < rows ? p.row_scale[row[b]] : 0.0f;
#pragma unroll
                for (int a = 0; a < kAcc; ++a)
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[a][b][j] *= rs * scale[a][j];
            }
            if (!DUAL) {
#pragma unroll
                for (int j = 0; j < 4; ++j) z[0][b][j] += bias[j];
            }
        }
        with_act(p.act, [&](auto act) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (b >= rows) break;
                alignas(8) __nv_bfloat16 y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t h = j < 2 ? x[b].x : x[b].y;
                    const float v = __uint_as_float(j & 1 ? h & 0xFFFF0000u : h << 16);
                    y[j] = __float2bfloat16_rn(DUAL ? act_f<act>(z[0][b][j]) * z[kAcc - 1][b][j] : act_f<act>(z[0][b][j]) + v);
                }
                __nv_bfloat16* out = p.out + row[b] * p.ld_out + n;
                if (p.vec_out && n + 4 <= p.n) {
                    *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(y);
                } else {
                    for (int j = 0; j < 4 && n + j < p.n; ++j) out[j] = y[j];
                }
            }
        });
    }
    // no CTA's sums go away while another may still read them
    ptx::cluster_sync();
    if (warp == 1) ptx::tmem_dealloc(tmem, kCols);
}

template <bool DUAL, bool E4M3, bool BIG>
int launch(FewArgs& p, cudaStream_t s) {
    using Cfg = FewConfig<DUAL, BIG>;
    constexpr int kAcc = DUAL ? 2 : 1;
    // As many CTAs as the SMs hold, each with four steps of K at least.  Clusters of
    // eight lie within a GPC, so fewer fit: with one CTA per SM 12 of them run at once
    // and 16 do not (160 x 2048 x 2048: 16.6 us, with clusters of four 9.6), with two 36
    // and not 37 (1 x 4096 x 4736: 13.0 us, with clusters of four 9.4)
    const int32_t tiles = static_cast<int32_t>(ceil_div(p.n, kChannels));
    int32_t splits = 1;
    while (splits < kMaxSplits && tiles * splits * 2 <= (splits == 4 ? (BIG ? 96 : 288) : Cfg::kPerSm * 152) && p.k_iters >= 8 * splits) splits *= 2;
    p.stage_bytes = static_cast<int32_t>(round_up(kAcc * kTileA + p.rows_pad * 128, 1024));
    p.stages = Cfg::kRing / p.stage_bytes < kMaxStages ? Cfg::kRing / p.stage_bytes : kMaxStages;
    static bool set[kMaxDevices] = {};
    int dev = 0;
    SPCONV_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return SPCONV_ERR_UNSUPPORTED;
    if (!set[dev]) {
        SPCONV_CHECK_CUDA(cudaFuncSetAttribute(k_dense_few<DUAL, E4M3, BIG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Cfg::kRing + 1024));
        set[dev] = true;
    }
    cudaLaunchAttribute at[2] = {pdl_attr(), {}};
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 1;
    at[1].val.clusterDim.y = static_cast<unsigned>(splits);
    at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(splits));
    cfg.blockDim = dim3(kThreads);
    // (at most the ring's room: the sums fit it too)
    const size_t ring = static_cast<size_t>(p.stages) * p.stage_bytes, sums = static_cast<size_t>(kAcc) * p.rows * kChannels * 4;
    cfg.dynamicSmemBytes = (ring > sums ? ring : sums) + 1024;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    count_launch();
    return cuda_status(cudaLaunchKernelEx(&cfg, k_dense_few<DUAL, E4M3, BIG>, static_cast<const FewArgs&>(p)));
}

template <bool DUAL, bool E4M3>
int launch(FewArgs& p, cudaStream_t s) {
    return p.rows <= FewConfig<DUAL, false>::kRows ? launch<DUAL, E4M3, false>(p, s) : launch<DUAL, E4M3, true>(p, s);
}

}  // namespace

bool dense_few_takes(const DenseOp& op) {
    if (op.k_sources != 1 || op.n_sources != 1 || !op.a.k_major) return false;
    if (op.epi != kEpiGated && op.epi != kEpiLinear) return false;
    const bool dual = op.epi == kEpiGated;
    if (op.m <= (dual ? FewConfig<true, false>::kRows : FewConfig<false, false>::kRows)) return true;
    // Beyond, the pairs' tiles of 256 rows are no longer mostly empty and win where
    // there are enough of them (256 rows x 2048 x 8192, 64 tiles of channels: 15.4 us,
    // 20.3 here), where the weight's rows are short (200 x 512 x 2048: 7.3, 8.8) and where
    // each CTA here would stream too many (256 x 8192 x 1024: 13.7, 15.7).  Between: 256
    // x 4096 x 4096 16.3, 15.2 here; 160 x 2048 x 1024 10.7, 8.9 here
    const int64_t k_bytes = op.k * (op.dtype == SPCONV_E4M3 ? 1 : 2);
    return op.m <= (dual ? FewConfig<true, true>::kRows : FewConfig<false, true>::kRows) && ceil_div(op.n, kChannels) <= 38 &&
           k_bytes >= 2048 && k_bytes <= 8192;
}

int dense_few_run(const DenseOp& op, int32_t* status, cudaStream_t s) {
    const bool dual = op.epi == kEpiGated, eight = op.dtype == SPCONV_E4M3;
    const size_t es = eight ? 1 : 2;
    FewArgs p = {};
    p.n = op.n;
    p.rows = static_cast<int32_t>(op.m);
    p.rows_pad = static_cast<int32_t>(round_up(static_cast<size_t>(op.m), 16));
    p.k_iters = static_cast<int32_t>(ceil_div(op.k, static_cast<int64_t>(128 / es)));
    p.w_kmajor = op.b.k_major;
    p.act = op.act;
    p.row_scale = op.row_scale;
    p.col_scale[0] = op.col_scale[0];
    p.col_scale[1] = op.col_scale[1];
    p.bias = op.bias;
    p.extra = static_cast<const __nv_bfloat16*>(op.extra);
    p.ld_extra = op.ld_extra;
    p.out = static_cast<__nv_bfloat16*>(op.out[0]);
    p.ld_out = op.ld_out;
    p.vec_out = op.ld_out % 4 == 0 && reinterpret_cast<uintptr_t>(op.out[0]) % 8 == 0;
    p.status = status;
    for (int a = 0; a < (dual ? 2 : 1); ++a)
        SPCONV_CHECK(op.b.k_major ? make_tensor_map(&p.w[a], op.b.p[a], es, op.k, op.n, op.b.ld, kChannels)
                                  : make_tensor_map(&p.w[a], op.b.p[a], es, op.n, op.k, op.b.ld, 64));
    SPCONV_CHECK(make_tensor_map(&p.x, op.a.p[0], es, op.k, op.m, op.a.ld, p.rows_pad));
    if (dual) return eight ? launch<true, true>(p, s) : launch<true, false>(p, s);
    return eight ? launch<false, true>(p, s) : launch<false, false>(p, s);
}

}  // namespace spconv
