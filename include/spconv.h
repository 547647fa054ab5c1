/*
 * spconv.h -- C ABI of the GB300 (sm_103a) submanifold sparse convolution
 * (3x3x3 and 5x5x5 kernels, stride 1) and of the row-wise operators between
 * two convolutions (RMS norm, linear, gated feed-forward).
 *
 * The operation (FlyDSL PR #942, "Add submanifold sparse 3D convolution",
 * Summary: raw voxel coordinates in, output features out, the kernel map built
 * internally; "Sparse convolution in FP32", section "The starting point": for
 * every active voxel, the sum over its 27 neighbours of the neighbour's
 * features times the weights of that kernel offset; FlyDSL PR #942, "Test
 * plan": kernel sizes 3 and 5):
 *
 *     out[i][o] = sum_{k=0..V-1} sum_{c} f[nbr[i][k]][c] * W[k][c][o]
 *
 * over the rows i of the input, where nbr[i][k] is the row of the voxel at
 * coords[i] + d_k (same batch index), the term skipped when there is none.
 * Kernel size K (3 or 5), radius r = (K-1)/2, V = K^3 taps; tap order
 * k = K*K*(dx+r) + K*(dy+r) + (dz+r) for d = (dx,dy,dz) in {-r..r}^3, i.e.
 * k = 9*(dx+1) + 3*(dy+1) + (dz+1) for K = 3 (cross-correlation, as torch
 * conv3d with padding r).  Outputs live at the input sites, in the input row
 * order.
 *
 * Memory: every pointer argument named *_dev is a device pointer that the
 * caller owns; host pointers are marked host.  The library allocates map
 * handles and packed-weight handles (stream-ordered, on the stream passed to
 * the creating call) and frees them in the matching destroy call; the row-wise
 * operators below take scratch memory in stream order for the length of a call.
 * All of it comes from a pool of the library's own on each device, which keeps
 * what is freed for later calls (a gated gradient of n rows and c_hidden
 * channels leaves 4 n c_hidden bytes there); spconv_trim_pool gives it back.
 *
 * Streams: all work is enqueued on the caller's stream; nothing synchronises
 * the device except where a function says it does.
 *
 * Devices: every call works on the calling thread's current device: its device
 * pointers, its stream and the handles that it is given belong to that one.
 *
 * Errors: functions return SPCONV_OK (0) or a negative spconv_status_t.
 * Argument errors are detected on the host before any work is enqueued.
 * Data errors found on the device (duplicate or out-of-range coordinates) are
 * recorded in the map handle and reported by spconv_map_status(); the map's
 * contents are then unspecified, but every kernel stays within its buffers.
 * No kernel traps; bounded waits inside kernels report SPCONV_ERR_TIMEOUT.
 */
#ifndef SPCONV_H_
#define SPCONV_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SPCONV_OK = 0,
    SPCONV_ERR_INVALID_ARG = -1,   /* null pointer, bad size, bad enum, misaligned buffer */
    SPCONV_ERR_UNSUPPORTED = -2,   /* valid request outside what this build implements    */
    SPCONV_ERR_OOM = -3,           /* device allocation failed                             */
    SPCONV_ERR_CUDA = -4,          /* a CUDA runtime call failed                            */
    SPCONV_ERR_DUPLICATE_COORD = -5,
    SPCONV_ERR_COORD_RANGE = -6,   /* b, x, y or z outside [0, batch) x [0, shape)          */
    SPCONV_ERR_ALIAS = -7,         /* out overlaps feats                                     */
    SPCONV_ERR_TIMEOUT = -8,       /* a bounded wait inside a kernel ran out                 */
    SPCONV_ERR_INTERNAL = -9       /* a kernel's consistency guard fired (a library bug)     */
} spconv_status_t;

typedef enum {
    SPCONV_BF16 = 0,
    SPCONV_FP32 = 1,
    SPCONV_E4M3 = 2    /* 8-bit floats with separate scales: the row-wise operators only */
} spconv_dtype_t;

typedef enum {
    SPCONV_MAPPER_AUTO = 0,   /* dense grid iff padded cells <= dense_max_cells, else HASH when
                                 the WIDE pipeline or a grouped K = 3 build makes the map, else
                                 SORTED                                                           */
    SPCONV_MAPPER_DENSE = 1,  /* presence grid over the padded bounding box                       */
    SPCONV_MAPPER_SORTED = 2, /* sorted 64-bit keys + binary search, memory O(N)                   */
    SPCONV_MAPPER_HASH = 3    /* the same packed keys in an open-addressing hash table, one
                                 bucket read per pair of z neighbours; memory O(N).  The WIDE
                                 pipeline and grouped builds only (the FUSED and MULTI
                                 pipelines with one group: SPCONV_ERR_UNSUPPORTED)                 */
} spconv_mapper_t;

typedef enum {
    SPCONV_ORDER_CALIBRATED = 0, /* sort key bits by descending tap frequency (rarest tap = MSB) */
    SPCONV_ORDER_PLAIN = 1       /* sort key = the mask itself                                    */
} spconv_bit_order_t;

typedef enum {
    SPCONV_PIPELINE_AUTO = 0,  /* WIDE when it applies, else FUSED when it applies, else MULTI    */
    SPCONV_PIPELINE_FUSED = 1, /* whole build in one thread-block-cluster launch (n <= 2^20)     */
    SPCONV_PIPELINE_MULTI = 2, /* one kernel per step, three per 8-bit sort pass (any n)          */
    SPCONV_PIPELINE_WIDE = 3   /* one kernel per step on the whole GPU, look-back sort passes     */
                               /* (n <= 2^26; sorted mapper: coordinate keys of at most 40 bits) */
} spconv_pipeline_t;

/* Work decomposition of the bf16 tensor-core forward ("Compaction is the
 * largest single win", FlyDSL PR #942; "Offset-group partitioning", "Sparse
 * convolution in FP32").  Both give the same sums up to fp32 rounding order. */
typedef enum {
    SPCONV_GEMM_AUTO = 0,        /* TILE_UNION (measured faster on every tested workload)      */
    SPCONV_GEMM_TILE_UNION = 1,  /* output-stationary: 128 mask-sorted rows per tile, all taps of
                                    the tile's mask union accumulated on chip, one bf16 store;
                                    deterministic                                             */
    SPCONV_GEMM_TAP_MAJOR = 2    /* 128 pairs of one tap per tile (compacted pair lists, no
                                    zero rows), fp32 sums added in an [n][c_out] workspace,
                                    then rounded to bf16; summation order varies run to run   */
} spconv_gemm_t;

/* Options of spconv_build_map.  Pass NULL for the defaults.  None of them
 * changes any result beyond fp32 rounding order; they select how the same
 * map is built and used. */
typedef struct {
    int32_t mapper;          /* spconv_mapper_t, default AUTO                          */
    int32_t bit_order;       /* spconv_bit_order_t, default CALIBRATED                 */
    int64_t dense_max_cells; /* AUTO threshold on B*(X+2)*(Y+2)*(Z+2); default 1<<24   */
    int32_t pipeline;        /* spconv_pipeline_t, default AUTO                        */
    int32_t gemm;            /* spconv_gemm_t for the bf16 forward on this map, default AUTO */
    int32_t groups;          /* offset groups ("Sparse convolution in FP32", "Offset-group
                                partitioning"): the V taps split into G runs of V/G
                                consecutive taps (G = K: the taps of one dx each), every
                                group with its own masks, row order and tiles, the forward
                                one GEMM pass per group.  0: default (1 for K = 3, 5 for
                                K = 5); 1 (K = 3 only) or K.  G > 1 builds with the MULTI
                                pipeline and the TILE_UNION forward; other choices of
                                pipeline or gemm return SPCONV_ERR_UNSUPPORTED.           */
} spconv_options_t;

typedef struct spconv_map_s* spconv_map_t;
typedef struct spconv_wpack_s* spconv_wpack_t;

/*
 * Epilogue of a forward: what happens to each fp32 sum of output row i,
 * channel o before its one rounding to the output dtype.  The inference form
 * of a layer's batch norm (a per-channel scale and shift), its bias, a
 * residual branch and the ReLU between layers, fused into the store so that
 * they cost no extra pass over [n][c_out].  The pages' networks are stacks of
 * such layers (FlyDSL PR #942, "Open questions": a layer stack with
 * normalisation and residuals; "Sparse convolution in FP32", "Offset-group
 * partitioning": the convolution's last launch applies the ReLU to every row):
 *
 *   y = sum * scale[o] + bias[o] + residual[i][o];   out[i][o] = relu ? max(y, 0) : y
 *
 *   scale_dev     fp32 [c_out], device, 16-byte aligned; NULL means 1.
 *   bias_dev      fp32 [c_out], device, 16-byte aligned; NULL means 0.
 *   residual_dev  [n][c_out] in the forward's dtype, device, 16-byte aligned,
 *                 row-major in the original row order; NULL means 0.  It may
 *                 be out_dev itself (an in-place add) or feats_dev, but must
 *                 not partly overlap out_dev (SPCONV_ERR_ALIAS).
 *   relu          0: none, 1: max(y, 0).  Other values: SPCONV_ERR_INVALID_ARG.
 * The caller owns every buffer; the library only reads them, in stream order.
 */
typedef struct {
    const float* scale_dev;
    const float* bias_dev;
    const void* residual_dev;
    int32_t relu;
} spconv_epilogue_t;

/* Summary of a built map.  Filling it synchronises the map's stream. */
typedef struct {
    int64_t n;           /* active voxels (rows)                                  */
    int64_t pairs;       /* P = number of (row, tap) with a neighbour (>= n)      */
    int64_t n_tiles;     /* 128-row tiles of the mask-sorted order (per group)    */
    int64_t tile_taps;   /* sum over tiles (all groups) of the taps in the tile's mask union */
    int32_t mapper;      /* spconv_mapper_t actually used (DENSE, SORTED or HASH) */
    int32_t pipeline;    /* spconv_pipeline_t actually used (FUSED, MULTI, WIDE)  */
    int32_t key_bits;    /* live bits of the packed coordinate key                */
    int32_t shape[3];    /* spatial shape used                                    */
    int32_t batch_size;  /* batch size used                                       */
    int32_t gemm;        /* spconv_gemm_t the bf16 forward uses (TILE_UNION or TAP_MAJOR) */
    int32_t kernel_size; /* K                                                     */
    int32_t groups;      /* G offset groups                                       */
    int64_t n_in;        /* rows of the features a forward reads (n but for strided and inverse maps) */
    int32_t conv;        /* 0 submanifold, 1 strided, 2 inverse of a strided map  */
    int32_t out_shape[3];/* spatial shape of the map's rows (a strided map: the output grid) */
} spconv_map_info_t;

/*
 * Build the kernel map of a coordinate set (FlyDSL PR #942, "Two mappers, both
 * required"; "Sparse convolution in FP32", "Neighbour masks and sorted rows";
 * FlyDSL PR #942, "Compaction is the largest single win").
 *
 *   coords_dev     int32 [n][4] rows (b, x, y, z), device, row-major.  Must stay
 *                  valid until the stream has passed this call; the handle
 *                  keeps what it needs.
 *   n              number of rows, 0 <= n < 2^30.
 *   spatial_shape  host int32[3] {X, Y, Z}, each >= 1; NULL derives max+1 per
 *                  axis on the device (synchronises the stream).
 *   batch_size     frames, >= 1; 0 derives max(b)+1 (synchronises the stream).
 *   kernel_size    3 or 5 (others return SPCONV_ERR_UNSUPPORTED).
 *   opt            options, NULL for defaults.
 *   stream         CUDA stream (cudaStream_t) the work is enqueued on.
 *   out_map        receives the handle; free it with spconv_map_destroy.
 *
 * Device-side results (all in the handle): the kernel map nbr[n][V]; per
 * offset group its masks (bit j: the group's tap j present), perm (rows in
 * ascending sort-key order, ties by row) and 128-row tile work list; the
 * per-tap pair lists, each in the order of its tap's group.
 */
int spconv_build_map(const int32_t* coords_dev, int64_t n, const int32_t* spatial_shape,
                     int32_t batch_size, int32_t kernel_size, const spconv_options_t* opt,
                     void* stream, spconv_map_t* out_map);

/*
 * The map of a strided (downsampling) sparse convolution: kernel 3, stride 2,
 * padding 1 per axis ("Sparse convolution in FP32", "Calibrated bit order":
 * the strided kernels, which change the coordinate set).  Its rows are the
 * output sites: every o of the output grid, X' = (X - 1) / 2 + 1 per axis,
 * whose window {2o + d : d in {-1,0,1}^3} holds an input site of the same
 * batch, in ascending (b, x, y, z) order; tap k of row o is the input row at
 * 2o + d_k.  A forward on it computes out[o] = sum_k W[k]^T f(2o + d_k):
 * feats [n][c_in] on the input sites, out [n_out][c_out] (torch conv3d with
 * stride 2 and padding 1, read at the output sites).
 *
 *   coords_dev, n, spatial_shape, batch_size: as spconv_build_map (n < 2^27).
 *   kernel_size 3 and stride 2 only (else SPCONV_ERR_UNSUPPORTED).
 *   opt: mapper AUTO or HASH, pipeline AUTO or MULTI, gemm not TAP_MAJOR,
 *        groups 0 or 1 (else SPCONV_ERR_UNSUPPORTED).
 * Synchronises the stream once: the number of output sites sizes the map.
 * spconv_map_rows gives n (output sites) and n_in without a second
 * synchronisation; spconv_map_info also out_shape;
 * spconv_map_out_coords copies the output sites' coordinates.
 */
int spconv_build_map_strided(const int32_t* coords_dev, int64_t n, const int32_t* spatial_shape,
                             int32_t batch_size, int32_t kernel_size, int32_t stride, const spconv_options_t* opt,
                             void* stream, spconv_map_t* out_map);

/*
 * The map of the inverse (transposed) convolution of a strided map: rows are
 * the strided map's input sites (its n_in), tap k of row i is the output site
 * o with 2o + d_k at site i, or none.  A forward on it computes
 * out[i] = sum_k W[k]^T g(o_k(i)) with g [n_out][c_in] on the strided map's
 * output sites and out [n_in][c_out] (torch conv_transpose3d, stride 2,
 * padding 1, read at the input sites).  Enqueued on the strided map's stream,
 * which the strided map must outlive until then; no synchronisation.
 * opt: bit_order and gemm (not TAP_MAJOR) are used; NULL for defaults.
 */
int spconv_build_map_inverse(spconv_map_t strided, const spconv_options_t* opt, spconv_map_t* out_map);

/* Copy a strided map's output sites, int32 [n][4] (b, x, y, z), to caller
 * device memory, enqueued on stream.  SPCONV_ERR_INVALID_ARG for other maps. */
int spconv_map_out_coords(spconv_map_t map, int32_t* out_coords_dev, void* stream);

/*
 * out = subm_conv(feats, weights) over the map's sites (the definition at the
 * top of this file).
 *
 *   feats_dev    [n_in][c_in] row-major, dtype elements, 16-byte aligned
 *                (n_in = n but for strided and inverse maps, spconv_map_info).
 *   weights_dev  [V][c_in][c_out] row-major, dtype elements (V = K^3 of the map).
 *   out_dev      [n][c_out] row-major, dtype elements, 16-byte aligned; must
 *                not overlap feats (SPCONV_ERR_ALIAS).
 *   dtype        SPCONV_BF16: bf16 in/out, fp32 accumulation, one rounding to
 *                bf16 at the store (tensor cores when c_in % 8 == 0 and
 *                c_out % 16 == 0, else a SIMT kernel).  SPCONV_FP32: fp32
 *                in/out with fp32 FMA on the SIMT path (exact mode).
 * Packs the weights into a workspace owned by the map on every call; use
 * spconv_wpack_create + spconv_subm_forward_packed to pack once.
 */
int spconv_subm_forward(spconv_map_t map, const void* feats_dev, const void* weights_dev,
                        void* out_dev, int32_t c_in, int32_t c_out, int32_t dtype, void* stream);

/* spconv_subm_forward with an epilogue (spconv_epilogue_t above; NULL is the
 * plain forward).  Same arguments, layouts and errors otherwise. */
int spconv_subm_forward_ex(spconv_map_t map, const void* feats_dev, const void* weights_dev,
                           void* out_dev, int32_t c_in, int32_t c_out, int32_t dtype,
                           const spconv_epilogue_t* epi, void* stream);

/*
 * Pre-pack weights [27][c_in][c_out] of a 3x3x3 kernel for repeated forwards (FlyDSL PR #942,
 * "Weight layout is [kv, t, k_outer, u, k_inner]": a packed tile layout; here
 * the tensor-core shared-memory image).  The handle owns a copy; the source
 * may be freed once the stream has passed this call.
 */
int spconv_wpack_create(const void* weights_dev, int32_t c_in, int32_t c_out, int32_t dtype,
                        void* stream, spconv_wpack_t* out_wpack);
int spconv_subm_forward_packed(spconv_map_t map, const void* feats_dev, spconv_wpack_t wpack,
                               void* out_dev, void* stream);
/* spconv_subm_forward_packed with an epilogue (NULL: none). */
int spconv_subm_forward_packed_ex(spconv_map_t map, const void* feats_dev, spconv_wpack_t wpack,
                                  void* out_dev, const spconv_epilogue_t* epi, void* stream);
/* spconv_wpack_create for a kernel of size kernel_size (3 or 5): weights
 * [K^3][c_in][c_out].  A packed forward on a map of another kernel size returns
 * SPCONV_ERR_INVALID_ARG. */
int spconv_wpack_create_ex(const void* weights_dev, int32_t kernel_size, int32_t c_in, int32_t c_out,
                           int32_t dtype, void* stream, spconv_wpack_t* out_wpack);
void spconv_wpack_destroy(spconv_wpack_t wpack);

/*
 * A stack of n_layers submanifold convolutions over one kernel map in a single
 * launch ("Sparse convolution in FP32", "Offset-group partitioning": the
 * convolution's last step applies the ReLU to every output row; layers that
 * share one coordinate set share one map, FlyDSL PR #942, "API style").
 * Layer l computes out_l = epilogue_l(conv(in_l, W_l)) with in_0 = feats and
 * in_l = out_{l-1}; every layer visits the same mask-sorted tiles and gather
 * table.  A layer's gathers start only after every CTA has stored the layer
 * before it, so each layer's result equals that of a separate
 * spconv_subm_forward_packed_ex call, bit for bit.
 *
 *   map        a submanifold map with one offset group and the tile-union GEMM
 *              (else SPCONV_ERR_UNSUPPORTED when n_layers > 1).
 *   feats_dev  bf16 [n][c_in], 16-byte aligned.
 *   wpacks     n_layers bf16 tensor-core weight packs (spconv_wpack_create),
 *              all c_in -> c_out with c_in == c_out when n_layers > 1.
 *   outs_dev   n_layers bf16 [n][c_out] outputs, 16-byte aligned, caller-owned;
 *              outs_dev[l] must not overlap its own input (feats_dev for l = 0,
 *              else outs_dev[l - 1]): SPCONV_ERR_ALIAS.  outs_dev[l] may equal
 *              outs_dev[l - 2] (two buffers ping-pong).
 *   n_layers   1 .. 8.
 *   epis       n_layers epilogues (each as in spconv_subm_forward_ex), or NULL.
 *   stream     CUDA stream; with n_layers > 1 the launch is cooperative (one
 *              CTA per SM, all resident) and uses a small per-map counter array.
 * Device-side waits between layers are bounded: a stall sets
 * SPCONV_ERR_TIMEOUT in the map's status (spconv_map_status).
 */
int spconv_subm_forward_layers(spconv_map_t map, const void* feats_dev, const spconv_wpack_t* wpacks,
                               void* const* outs_dev, int32_t n_layers, const spconv_epilogue_t* epis,
                               void* stream);

/* Synchronise the map's stream and return the first device-detected error
 * (duplicate or out-of-range coordinates, kernel timeouts), else SPCONV_OK. */
int spconv_map_status(spconv_map_t map);

/* Fill *info (synchronises the map's stream). */
int spconv_map_info(spconv_map_t map, spconv_map_info_t* info);

/*
 * The map's row count (output sites) and the count of the sites its
 * neighbours index (n_in; = rows but for strided and inverse maps), both
 * known on the host once the build call has returned: no synchronisation
 * and no device access.  Either pointer may be NULL.  Returns
 * SPCONV_ERR_INVALID_ARG for a NULL map.
 */
int spconv_map_rows(spconv_map_t map, int64_t* n, int64_t* n_in);

/*
 * Copy the map's arrays into caller device buffers (any may be NULL):
 *   nbr_dev int32 [n][V]; mask_dev uint32 [G][n]; perm_dev int32 [G][n];
 *   tap_off_dev int32 [V + 1]; in_rows_dev, out_rows_dev int32 [pairs].
 * Enqueued on stream; no synchronisation.
 */
int spconv_map_export(spconv_map_t map, int32_t* nbr_dev, uint32_t* mask_dev, int32_t* perm_dev,
                      int32_t* tap_off_dev, int32_t* in_rows_dev, int32_t* out_rows_dev,
                      void* stream);

/* Free the handle (stream-ordered on the stream of the build). */
void spconv_map_destroy(spconv_map_t map);

/*
 * The kernel map nbr[n][27] of a coordinate set without allocating any device
 * memory.  The pages have no counterpart to this entry point; it exists for
 * callers that cannot allocate at the point where they run this code (a
 * plugin's enqueue step in an inference runtime that plans all device memory
 * up front, runtimes that forbid allocation after start-up).
 *
 *   coords_dev     int32 [n][4] rows (b, x, y, z), device, 16-byte aligned.
 *   n              0 <= n <= 65536; larger n returns SPCONV_ERR_INVALID_ARG
 *                  (the working buffers live in a fixed 1.6 MB device array).
 *   spatial_shape  host int32[3] {X, Y, Z} (required).
 *   batch_size     >= 1 (required).
 *   nbr_dev        int32 [n][27] output, caller-owned: the same values as the
 *                  nbr that spconv_map_export returns for this input.
 *   stream         CUDA stream; the call synchronises it before returning and
 *                  returns SPCONV_ERR_DUPLICATE_COORD / SPCONV_ERR_COORD_RANGE
 *                  for bad coordinates.
 *
 * No cudaMalloc, cudaFree or allocating library routine is called.  The
 * working buffers are one file-scope device array that every GPU loading this
 * library holds until the process exits; the first call on a device looks up
 * its address (make that first call before any stream capture).  All calls
 * share the array, so calls whose work overlaps on the GPU (different streams
 * or threads) race; serialise them.
 */
int spconv_kernel_map_static(const int32_t* coords_dev, int64_t n, const int32_t* spatial_shape,
                             int32_t batch_size, int32_t* nbr_dev, void* stream);

/*
 * Row-wise operators of a network over voxels: what stands between two
 * convolutions on the same sites.  They need no map: each works on n rows of
 * features, [n][c] as the convolution reads and writes them.  The pages' open
 * question of "a layer stack with normalisation and residuals" (FlyDSL PR #942,
 * "Open questions") for networks whose norm has row statistics and whose
 * layers have a feed-forward part.
 *
 *   Rows       every [n][c] argument has a row stride ld_* in elements (>= c);
 *              its rows are contiguous.  Outputs without a stride are dense.
 *              Any element-aligned address and stride is taken.
 *   Sizes      0 <= n < 2^30, 1 <= c <= 65536.  n = 0 writes only the
 *              gradients of the parameters (zeros).
 *   Rounding   sums, statistics and epilogues are fp32, with one rounding to
 *              the output type.
 *   Order      every sum has a fixed order: the same call gives the same bits.
 *   Scratch    taken from the library's pool in stream order for the length
 *              of the call.
 *   Capture    calls can be captured into a CUDA graph.  Which kernels a call
 *              takes depends on its sizes, types, strides, alignment and
 *              options, and each is loaded at its first launch on a device: make
 *              the call that is to be captured once before.
 *   Aliasing   an output must not overlap an input (biases, scales and weights
 *              included) or another output, unless said below
 *              (SPCONV_ERR_ALIAS).  Column ranges of one wider matrix do not
 *              overlap.
 *   NaN, inf   pass through the formulas as in IEEE arithmetic.
 */
typedef enum {
    SPCONV_ACT_NONE = 0,
    SPCONV_ACT_RELU = 1,       /* max(z, 0)                                            */
    SPCONV_ACT_SILU = 2,       /* z / (1 + exp(-z))                                    */
    SPCONV_ACT_GELU = 3,       /* z (1 + erf(z / sqrt 2)) / 2                          */
    SPCONV_ACT_GELU_TANH = 4   /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2    */
} spconv_act_t;

/*
 * Root-mean-square norm of rows with the residual's addition:
 *
 *   h = x + residual;  y = h / sqrt(mean_c h^2 + eps) * weight;  sum = h
 *
 *   x_dev, residual_dev  [n] rows of c, dtype (SPCONV_BF16 or SPCONV_FP32);
 *                        residual_dev NULL means 0.
 *   weight_dev           fp32 [c].
 *   sum_dev              [n][c] dtype, h rounded (the next residual), or NULL.
 *                        May be x_dev or residual_dev themselves when dense.
 *   out_dev              [n][c]: y in dtype, or with out_dtype SPCONV_E4M3 the
 *                        e4m3 values q of y / scale, scale_dev fp32 [n] being
 *                        max_c |y| / 448 of each row (0 for a row of zeros, with
 *                        q 0).  scale_dev NULL exactly when y is in dtype.
 */
int spconv_rms_norm(const void* x_dev, int64_t ld_x, const void* residual_dev, int64_t ld_residual, const float* weight_dev,
                    int64_t n, int32_t c, int32_t dtype, float eps, void* sum_dev, void* out_dev, int32_t out_dtype,
                    float* scale_dev, void* stream);

/*
 * Its backward pass.  x is the normalised sum h, r = 1 / sqrt(mean_c x^2 + eps):
 *
 *   dx = r (dy w - x r^2 mean_c(dy w x)) + dres;   dweight_c = sum_rows dy x r
 *
 *   dres_dev   gradient that reaches the sum by another way (the residual
 *              stream), or NULL; dx_dev may be dres_dev when dense.
 *   dx_dev     [n][c] dtype: the gradient of x and of the residual alike.
 *   dweight_dev fp32 [c], overwritten.
 */
int spconv_rms_norm_backward(const void* dy_dev, int64_t ld_dy, const void* x_dev, int64_t ld_x, const float* weight_dev,
                             const void* dres_dev, int64_t ld_dres, int64_t n, int32_t c, int32_t dtype, float eps,
                             void* dx_dev, float* dweight_dev, void* stream);

/*
 * out = act(z) + residual,  z = x W + bias.
 *
 *   dtype SPCONV_BF16   x bf16 [n] rows of c_in, W bf16 [c_in][c_out] (one tap
 *                       of a convolution's weights); the scales are NULL.
 *   dtype SPCONV_E4M3   x e4m3 with fp32 x_scale [n], W e4m3 [c_out][c_in] with
 *                       fp32 w_scale [c_out] (spconv_rms_norm and
 *                       spconv_quantize_weight make them): the product of row i
 *                       and channel o is multiplied by x_scale[i] w_scale[o].
 *   bias_dev            fp32 [c_out] or NULL.
 *   residual_dev        bf16 [n] rows of c_out or NULL; may be out_dev with the
 *                       same stride.
 *   out_dev             bf16 [n] rows of c_out.
 * SPCONV_FP32 returns SPCONV_ERR_UNSUPPORTED.
 */
int spconv_linear(const void* x_dev, int64_t ld_x, const float* x_scale_dev, const void* w_dev, const float* w_scale_dev,
                  int64_t n, int32_t c_in, int32_t c_out, int32_t dtype, const float* bias_dev, int32_t activation,
                  const void* residual_dev, int64_t ld_residual, void* out_dev, int64_t ld_out, void* stream);

/*
 * Gradients of the bf16 form (the residual's is dy itself).  z is formed again:
 *
 *   dz = dy act'(z);  dx = dz W^T;  dw = x^T dz;  dbias = sum_rows dz
 *
 * dz is rounded to bf16 as an operand of the two products (dbias sums it
 * unrounded).  dx_dev bf16 [n][c_in], dw_dev bf16 [c_in][c_out], dbias_dev
 * fp32 [c_out]; each may be NULL, which leaves its work out.
 */
int spconv_linear_backward(const void* dy_dev, int64_t ld_dy, const void* x_dev, int64_t ld_x, const void* w_dev, int64_t n,
                           int32_t c_in, int32_t c_out, int32_t dtype, const float* bias_dev, int32_t activation,
                           void* dx_dev, void* dw_dev, float* dbias_dev, void* stream);

/*
 * Gated feed-forward: out = act(x W_gate) * (x W_up), both products, the
 * activation and the product of the two in one kernel (for a few hundred rows
 * and a long c_in, where that is cut, in two).  Operands as
 * spconv_linear (gate_scale, up_scale fp32 [c_hidden] with e4m3);
 * out_dev bf16 [n] rows of c_hidden.
 */
int spconv_gated_ffn(const void* x_dev, int64_t ld_x, const float* x_scale_dev, const void* w_gate_dev,
                     const float* gate_scale_dev, const void* w_up_dev, const float* up_scale_dev, int64_t n, int32_t c_in,
                     int32_t c_hidden, int32_t dtype, int32_t activation, void* out_dev, int64_t ld_out, void* stream);

/*
 * Gradients of the bf16 form, from dh, the gradient of out.  g = x W_gate and
 * u = x W_up are formed again:
 *
 *   dg = dh u act'(g);  du = dh act(g)      (rounded to bf16 as operands)
 *   dx = dg W_gate^T + du W_up^T;  dw_gate = x^T dg;  dw_up = x^T du
 *
 * dx_dev may be NULL, or dw_gate_dev and dw_up_dev both.
 */
int spconv_gated_ffn_backward(const void* dh_dev, int64_t ld_dh, const void* x_dev, int64_t ld_x, const void* w_gate_dev,
                              const void* w_up_dev, int64_t n, int32_t c_in, int32_t c_hidden, int32_t dtype,
                              int32_t activation, void* dx_dev, void* dw_gate_dev, void* dw_up_dev, void* stream);

/*
 * A weight for the e4m3 forms, made once: w bf16 [c_in][c_out] to q e4m3
 * [c_out][c_in] with scale[o] = max_c |w[c][o]| / 448 (0, with q 0, for a
 * channel of zeros).
 */
int spconv_quantize_weight(const void* w_dev, int32_t c_in, int32_t c_out, void* q_dev, float* scale_dev, void* stream);

/*
 * Group norm of ragged scans with an activation.  Rows offsets[s] ..
 * offsets[s + 1] - 1 are scan s, a group is c / groups neighbouring channels,
 * and the rows of a scan share each group's statistics:
 *
 *   out = act((x - mean) / sqrt(var + eps) * weight + bias)
 *
 * with the variance of the whole population (divided by the count).
 *
 *   x_dev        [n] rows of c, dtype (SPCONV_BF16 or SPCONV_FP32).
 *   weight_dev   fp32 [c];  bias_dev fp32 [c] or NULL (0).
 *   offsets_dev  int32 [scans + 1], ascending, in [0, n]; or NULL: one scan of
 *                all rows (scans = 1).  A scan may be empty.  Rows of no scan
 *                (before the first border, behind the last) are written as
 *                zeros.  Borders out of order or range are an error that
 *                spconv_rows_status returns (SPCONV_ERR_COORD_RANGE); no memory
 *                outside the arguments is touched, and out is undefined.
 *   out_dev      [n][c] dtype.
 *   stats_dev    fp32 [scans][groups][2], mean and 1 / sqrt(var + eps), for the
 *                backward pass (8-byte aligned); or NULL.  An empty scan has
 *                mean 0 and variance 0.
 * groups divides c; scans <= 2^20.  c > 8192 returns SPCONV_ERR_UNSUPPORTED.
 */
int spconv_group_norm(const void* x_dev, int64_t ld_x, const float* weight_dev, const float* bias_dev,
                      const int32_t* offsets_dev, int64_t scans, int64_t n, int32_t c, int32_t groups, int32_t dtype,
                      int32_t activation, float eps, void* out_dev, float* stats_dev, void* stream);

/*
 * Its backward pass, from the statistics that the forward pass wrote: with
 * u = (x - mean) r, dz = dy act'(u weight + bias), p = dz weight, and means over
 * a scan's group,
 *
 *   dx = r (p - mean(p) - u mean(p u));  dweight = sum dz u;  dbias = sum dz
 *
 *   dx_dev       [n][c] dtype, zeros in rows of no scan.
 *   dweight_dev  fp32 [c]; dbias_dev fp32 [c] or NULL: over the rows of scans.
 */
int spconv_group_norm_backward(const void* dy_dev, int64_t ld_dy, const void* x_dev, int64_t ld_x, const float* weight_dev,
                               const float* bias_dev, const float* stats_dev, const int32_t* offsets_dev, int64_t scans,
                               int64_t n, int32_t c, int32_t groups, int32_t dtype, int32_t activation, void* dx_dev,
                               float* dweight_dev, float* dbias_dev, void* stream);

/*
 * Rows sorted by expert.  Row t chooses k experts: pair (t, j) has the number
 * t k + j.  The pairs are sorted by expert, those of one expert in their own
 * order; a pair's place among them is its slot.
 *
 *   experts_dev  int32 (index_bytes 4) or int64 (8) [tokens][k], each in
 *                [0, n_experts), or negative: no expert, and no slot.  One that
 *                is too large counts as none and is an error that
 *                spconv_rows_status returns (SPCONV_ERR_COORD_RANGE).  A row may
 *                name an expert twice.
 *   offsets_dev  int32 [n_experts + 1]: expert e's rows are the slots
 *                offsets[e] .. offsets[e + 1] - 1.
 *   pairs_dev    int32 [tokens k]: the pair of each slot, -1 behind the last.
 *   slots_dev    int32 [tokens][k]: the slot of each pair, -1 for no expert.
 * 1 <= k, n_experts <= 1024; tokens k < 2^30.  tokens = 0 writes the offsets.
 */
int spconv_expert_plan(const void* experts_dev, int32_t index_bytes, int64_t tokens, int32_t k, int32_t n_experts,
                       int32_t* offsets_dev, int32_t* pairs_dev, int32_t* slots_dev, void* stream);

/*
 * Each row to the slots of its pairs: out[slots[t][j]] = x[t], for slots and
 * offsets from spconv_expert_plan.  Rows of out at and behind
 * offsets[n_experts] are zeros.
 *
 *   x_dev      [tokens] rows of c, dtype (SPCONV_BF16 or SPCONV_FP32).
 *   out_dev    [tokens k][c] in dtype; or, with out_dtype SPCONV_E4M3, e4m3
 *              values q with scale_dev fp32 [ceil(c / 128)][tokens k], one for
 *              each 128 values of a row, as spconv_quantize_blocks makes them.
 *              scale_dev NULL exactly when out is in dtype.
 * The gradient of x is spconv_expert_combine of out's without weights.
 */
int spconv_expert_gather(const void* x_dev, int64_t ld_x, const int32_t* slots_dev, const int32_t* offsets_dev, int64_t tokens,
                         int32_t k, int32_t n_experts, int32_t c, int32_t dtype, void* out_dev, int32_t out_dtype,
                         float* scale_dev, void* stream);

/*
 * And back: out[t] = residual[t] + sum_j weights[t][j] y[slots[t][j]], in the
 * order of j, over the pairs that have a slot (whatever the weights of the
 * others are).
 *
 *   y_dev         [tokens k] rows of c, dtype.
 *   weights_dev   fp32 [tokens][k], or NULL (1).
 *   residual_dev  [tokens] rows of c, dtype, or NULL; may be out_dev when dense.
 *   out_dev       [tokens][c] dtype.
 */
int spconv_expert_combine(const void* y_dev, int64_t ld_y, const int32_t* slots_dev, const float* weights_dev,
                          const void* residual_dev, int64_t ld_residual, int64_t tokens, int32_t k, int32_t c, int32_t dtype,
                          void* out_dev, void* stream);

/*
 * Its gradients: dy[slots[t][j]] = weights[t][j] dout[t], zeros at and behind
 * offsets[n_experts], and dweights[t][j] = dout[t] . y[slots[t][j]], 0 for a
 * pair without a slot.  The residual's gradient is dout itself.
 *
 *   dy_dev        [tokens k][c] dtype;  dweights_dev fp32 [tokens][k].
 */
int spconv_expert_combine_backward(const void* dout_dev, int64_t ld_dout, const void* y_dev, int64_t ld_y,
                                   const int32_t* slots_dev, const int32_t* offsets_dev, const float* weights_dev, int64_t tokens,
                                   int32_t k, int32_t n_experts, int32_t c, int32_t dtype, void* dy_dev, float* dweights_dev,
                                   void* stream);

/*
 * Rows in e4m3 with a scale for each 128 values (the last of a row: what is
 * left): scale[b][i] = max |x| / 448 over block b of row i, q = e4m3(x / scale),
 * both divisions rounded to nearest; 0, with q 0, for a block of zeros.  A block
 * with an infinity or a NaN stands for NaN.
 *
 *   x_dev      [n] rows of c, dtype (SPCONV_BF16 or SPCONV_FP32).
 *   q_dev      e4m3 [n][c];  scale_dev fp32 [ceil(c / 128)][n].
 */
int spconv_quantize_blocks(const void* x_dev, int64_t ld_x, int64_t n, int32_t c, int32_t dtype, void* q_dev, float* scale_dev,
                           void* stream);

/*
 * Weights for the block-scaled products, made once: w bf16
 * [count][c_in][c_out] to q e4m3 [count][c_out][c_in] with a scale for each 128
 * x 128 values, scale_dev fp32 [count][ceil(c_out / 128)][ceil(c_in / 128)].
 * count <= 1024.
 */
int spconv_quantize_weight_blocks(const void* w_dev, int32_t count, int32_t c_in, int32_t c_out, void* q_dev, float* scale_dev,
                                  void* stream);

/*
 * spconv_linear for e4m3 operands with a scale for each block of 128, and for
 * sorted rows and the weights of their experts:
 *
 *   out = act(z + bias) + residual
 *   z[i][o] = sum_b x_scale[b][i] w_scale[o / 128][b] sum_{c in block b} x[i][c] W[o][c]
 *
 *   x_dev          e4m3 [n] rows of c_in, x_scale_dev fp32 [ceil(c_in / 128)][n]
 *                  (spconv_quantize_blocks, spconv_expert_gather).
 *   w_dev          e4m3 [n_experts][c_out][c_in], 16-byte aligned, w_scale_dev
 *                  fp32 [n_experts][ceil(c_out / 128)][ceil(c_in / 128)]
 *                  (spconv_quantize_weight_blocks).
 *   offsets_dev    int32 [n_experts + 1], ascending, in [0, n]: rows offsets[e]
 *                  .. offsets[e + 1] - 1 are expert e's, any number of them.
 *                  Rows of no expert are written as zeros.  Borders out of order
 *                  or range are an error that spconv_rows_status returns
 *                  (SPCONV_ERR_COORD_RANGE); out is undefined then.  NULL with
 *                  n_experts 1: one weight for all rows.
 *   bias_dev       fp32 [n_experts][c_out] or NULL.
 *   residual_dev   bf16 [n] rows of c_out or NULL; may be out_dev with the same
 *                  stride.
 *   out_dev        bf16 [n] rows of c_out; or, with out_scale_dev fp32
 *                  [ceil(c_out / 128)][n], e4m3 with a scale for each 128 values
 *                  of a row, as spconv_quantize_blocks forms them (from the fp32
 *                  values, and without a residual).
 * The sums are fp32 throughout.  c_in is a multiple of 16
 * (SPCONV_ERR_UNSUPPORTED otherwise: the rows of the dense weight are read by
 * tensor-map copies, which take strides of whole 16 bytes); n_experts <= 1024.
 */
int spconv_linear_blocks(const void* x_dev, int64_t ld_x, const float* x_scale_dev, const void* w_dev, const float* w_scale_dev,
                         const int32_t* offsets_dev, int32_t n_experts, int64_t n, int32_t c_in, int32_t c_out,
                         const float* bias_dev, int32_t activation, const void* residual_dev, int64_t ld_residual, void* out_dev,
                         int64_t ld_out, float* out_scale_dev, void* stream);

/*
 * spconv_gated_ffn of the same operands: out = act(z_gate) * z_up.
 */
int spconv_gated_ffn_blocks(const void* x_dev, int64_t ld_x, const float* x_scale_dev, const void* w_gate_dev,
                            const float* gate_scale_dev, const void* w_up_dev, const float* up_scale_dev,
                            const int32_t* offsets_dev, int32_t n_experts, int64_t n, int32_t c_in, int32_t c_hidden,
                            int32_t activation, void* out_dev, int64_t ld_out, float* out_scale_dev, void* stream);

/*
 * Synchronise the stream and return the first error that the row-wise
 * operators' kernels recorded on the current device since the last call of
 * this function (SPCONV_ERR_TIMEOUT: a bounded wait ran out and the results
 * of a call are incomplete), else SPCONV_OK.
 */
int spconv_rows_status(void* stream);

/*
 * Synchronise the current device and give the memory that the library's pool
 * holds there without using it back to the device, down to keep_bytes in all.
 * Maps and weight packs stay.
 */
int spconv_trim_pool(int64_t keep_bytes);

/* Number of kernel launches enqueued by the last call on this thread. */
int32_t spconv_last_launch_count(void);

/*
 * Diagnostics: runs one of the bounded device waits of the sort passes
 * against a state that nothing will ever publish, so that it must give up.
 * The pages have no counterpart; every device wait of the library ends after
 * a time limit (2 s in the product path) with SPCONV_ERR_TIMEOUT instead of
 * hanging the GPU, and this call shows that path working with a short limit.
 *
 *   which     0: the decoupled look-back of a sort pass, waiting for a
 *             predecessor partition whose state stays unpublished;
 *             1: the grid barrier of a two-CTA grid of which only one CTA
 *             runs;
 *             2: the flag wait of a pass that sums its predecessors'
 *             counts, on a flag that stays unset.
 *   limit_ns  the wait's limit, 1 ms .. 100 ms.
 *   stream    CUDA stream; the call allocates a few hundred bytes
 *             stream-ordered, synchronises the stream and frees them.
 *
 * Returns SPCONV_ERR_TIMEOUT when the wait ran out as designed (the GPU
 * context stays usable), SPCONV_ERR_INVALID_ARG for a bad argument, or
 * SPCONV_ERR_CUDA.
 */
int spconv_selftest_wait_timeout(int32_t which, int64_t limit_ns, void* stream);

/*
 * Diagnostics: the same for the row-wise operators.  Enqueues a kernel that
 * waits, as theirs do, on a barrier that nothing arrives on and gives up after
 * limit_ns (1 ms .. 100 ms).  spconv_rows_status then returns
 * SPCONV_ERR_TIMEOUT once.  Returns SPCONV_OK, SPCONV_ERR_INVALID_ARG for a
 * limit out of range, or SPCONV_ERR_CUDA.
 */
int spconv_selftest_rows_wait(int64_t limit_ns, void* stream);

const char* spconv_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* SPCONV_H_ */
