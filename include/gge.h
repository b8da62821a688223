/*
 * gge.h -- C ABI of libgge.so: fused persistent GEMM epilogues on one GB300
 * (sm_103a).
 *
 * The operation is the one the QuACK pages implement for Hopper
 * (quack-kernels 0.2.0: quack/dense_gemm_sm90.py ``GemmSm90``,
 * quack/gemm_act_sm90.py ``GemmActSm90`` / ``gemm_act_sm90``):
 *
 *   D[m,n,l]       = alpha * sum_k A[m,k,l] * B[n,k,l] + beta * C[m,n,l]
 *   PostAct[m,n,l] = act( same value, before rounding )
 *
 * with fp32 accumulation; each output is rounded once (round to nearest even)
 * to its own dtype.  Without C there is no beta term (the pages' epilogue
 * visit adds ``beta * C`` only when C is given).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller.  Nothing is
 *     allocated, freed or synchronised by the library (except
 *     gge_read_device_status and gge_read_static_scratch_status, which
 *     synchronise the given stream).
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default).
 *     Kernels are launched with programmatic stream serialization: a launch may
 *     begin its setup (shared memory, TMEM) while the previous kernel in the
 *     stream is finishing, but reads and writes no global memory before that
 *     kernel has completed, so stream order holds as for any launch.
 *   - Validation happens on the host before any launch; a rejected call
 *     launches nothing and returns GGE_ERR_INVALID_ARG / GGE_ERR_UNSUPPORTED /
 *     GGE_ERR_ALIGNMENT / GGE_ERR_WORKSPACE.  A failed launch returns
 *     GGE_ERR_CUDA.  Faults found on the device (a wait that ran out of time,
 *     a gather index or group offset out of range) are written to the
 *     workspace and read back with gge_read_device_status.
 *   - Strides are in ELEMENTS.  The contiguous dimension of every tensor must
 *     have stride 1, every other stride and every base pointer must be 16-byte
 *     aligned (the pages' rule: the contiguous dimension 16-byte aligned).
 *   - Sizes are int64 in the structs but every extent must be < 2^31.
 */
#ifndef GGE_H_
#define GGE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* gge_stream_t; /* same type as cudaStream_t */

typedef enum gge_status {
  GGE_OK = 0,
  GGE_ERR_INVALID_ARG = 1, /* NULL where a pointer is required, inconsistent shapes */
  GGE_ERR_UNSUPPORTED = 2, /* valid request outside what the kernels implement      */
  GGE_ERR_ALIGNMENT = 3,   /* base pointer or stride not 16-byte aligned             */
  GGE_ERR_WORKSPACE = 4,   /* workspace NULL or smaller than gge_workspace_size      */
  GGE_ERR_CUDA = 5,        /* a CUDA runtime / driver call failed                    */
  GGE_ERR_TIMEOUT = 6,     /* device: a pipeline wait ran past its time limit        */
  GGE_ERR_INDEX_RANGE = 7  /* device: gather index / group offset out of range       */
} gge_status;

typedef enum gge_dtype {
  GGE_BF16 = 0,
  GGE_F16 = 1,
  GGE_E4M3 = 2, /* float8_e4m3fn */
  GGE_E5M2 = 3, /* float8_e5m2   */
  GGE_F32 = 4
} gge_dtype;

/* Activations of the fused epilogue.  The pages list relu and
 * gelu_tanh_approx (quack/gemm_act_sm90.py ``act_fn_map``); SiLU is the
 * textbook x / (1 + exp(-x)). */
typedef enum gge_act {
  GGE_ACT_NONE = 0,
  GGE_ACT_RELU = 1,      /* x > 0 ? x : 0                                        */
  GGE_ACT_GELU_TANH = 2, /* 0.5 x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3)))      */
  GGE_ACT_SILU = 3,      /* x / (1 + exp(-x))                                    */
  GGE_ACT_RELU_SQ = 4    /* relu(x)^2 (act_fn_map's relu_sq)                     */
} gge_act;

/* A strided 3-D view [rows, cols, batch]. */
typedef struct gge_tensor {
  void* ptr;            /* device pointer to element [0,0,0]                    */
  int32_t dtype;        /* gge_dtype                                            */
  int32_t reserved;     /* must be 0                                            */
  int64_t rows, cols, batch;
  int64_t stride_row, stride_col, stride_batch; /* in elements                  */
} gge_tensor;

/* Optional tuning / debug knobs; pass NULL for the defaults. */
typedef struct gge_config {
  int32_t tile_n;         /* 0 = auto; else output columns per tile: 64 (TMA forms),
                             128 or 256 on one CTA, 256, 224, 192 or 160 on a
                             CTA pair (the narrower pair tiles need a K-major B) */
  int32_t num_ctas;       /* 0 = one persistent CTA per SM                         */
  int32_t raster_band;    /* 0 = auto; tiles per raster band (plain problems): auto
                             takes the width that keeps a wave's A and B rows
                             fewest, sqrt(units * tile_n / tile_m) m-tiles     */
  int32_t stages;         /* 0 = as many as shared memory holds                    */
  int32_t flags;          /* bit 0: count tile visits into tile_counts;
                             bit 1: test hook -- the MMA warp never signals a
                             finished accumulator, so the epilogue's bounded wait
                             runs out and the call reports GGE_ERR_TIMEOUT;
                             bit 2: dynamic tile scheduler -- after its first
                             tile each CTA (pair) claims the next one from a
                             counter in the workspace (needs a workspace);
                             bit 3: direct epilogue stores -- each lane stores its
                             own output row instead of staging 32 x 32 chunks in
                             shared memory (frees 16-32 KiB: one more pipeline
                             stage on a CTA pair; best when K is long);
                             bit 4: reserved (a call that sets it returns
                             GGE_ERR_UNSUPPORTED);
                             bit 5: never split the last wave.  By default a
                             plain problem whose last wave of tiles is at most
                             half full cuts those tiles into 2-8 K-slices that
                             otherwise idle CTAs compute.  Each slice leaves its
                             fp32 partial sums in the workspace; whichever unit
                             finishes a tile's slices last adds them, in slice
                             order, and runs the epilogue.  No CTA waits for
                             another, so the result does not depend on when the
                             CTAs run.  Not with the dynamic scheduler or the
                             gather and varlen forms; needs gge_workspace_size
                             bytes;
                             bit 6: reserved (a call that sets it returns
                             GGE_ERR_UNSUPPORTED);
                             bit 7: raster along N -- plain problems walk bands
                             of raster_band n-tiles, the n-tile varying fastest
                             (default: bands of m-tiles, the m-tile fastest);
                             bit 8: cluster launch control -- the grid has one
                             CTA (pair) per tile, and a running one takes over
                             the tiles of those not launched yet
                             (clusterlaunchcontrol.try_cancel) instead of a
                             fixed stride; no workspace needed; not with bit 2;
                             the last wave is not split;
                             bit 9: swap_ab -- compute D^T = B A^T: the kernel's
                             tiles run over the caller's N (rows) and M
                             (columns) and the epilogue stores C / D / PostAct
                             transposed into the caller's N-major [M, N]
                             layout (plain problems: gge_gemm, gge_gemm_act,
                             gge_gemm_dact).  For small M, so that M becomes the
                             tile width (64-wide one-CTA tiles exist for this);
                             bit 10: serpentine K -- work items of odd waves
                             (item index / resident units) walk K backwards, so
                             each wave starts on the k-slices the previous one
                             read last, still in L2 (plain and varlen-M forms
                             with TMA-loaded A; reproducible, the direction is
                             fixed by the plan).                               */
  int32_t cta_group;      /* 0 = auto; 1 = one CTA per 128-row tile; 2 = a CTA pair
                             per 256-row tile (tcgen05 cta_group::2; with gather-A
                             256-column tiles only; not with gather-K)           */
  int32_t* tile_counts;   /* device int32 per tile (debug coverage), or NULL       */
  uint64_t timeout_ns;    /* 0 = default (2 s) limit for each pipeline wait        */
  const int32_t* batch_idx_permute;
                          /* NULL, or device int32[L], a permutation of 0..L-1
                             (the pages' batch_idx_permute; plain problems with
                             L <= 1024 only, else GGE_ERR_UNSUPPORTED): the
                             scheduler visits batch batch_idx_permute[b] where it
                             would visit batch b, so it fixes the order in which
                             batches run, never the results.  Every CTA checks
                             it on the device before any work: an entry outside
                             [0, L) or a batch listed twice records
                             GGE_ERR_INDEX_RANGE (where 14, tile = the first bad
                             position, or the first batch not listed) and the
                             launch computes and writes nothing.               */
} gge_config;

/*
 * Arguments of one GEMM.
 *   A : [M, K, L]  rows = M, cols = K.  K-major (stride_col == 1) or, for
 *       16-bit operands loaded by TMA (every form but the gathers), M-major
 *       (stride_row == 1).  In gather-A, A is the SOURCE matrix
 *       [rows_src, K, 1], K-major; in gather-K, the M-major source [M, K_src, 1].
 *   B : [N, K, L]  rows = N, cols = K.  K-major (stride_col == 1) or, for
 *       16-bit operands, N-major (stride_row == 1).  8-bit operands must be
 *       K-major (as on the pages).
 *   C : optional [M, N, L] input, N-major.  NULL: no beta term.
 *   D : optional [M, N, L] output, N-major.
 *   PostAct : optional [M, N, L] output of act(...), N-major.  Required when
 *       act != GGE_ACT_NONE.
 *   Dtypes: A and B both 16-bit and equal (bf16 or f16), or both 8-bit
 *       (e4m3 / e5m2 in any combination).  C, D, PostAct: bf16, f16 or f32.
 *   N must be a multiple of 8.
 *   alpha_dev / beta_dev: optional device float scalars that override alpha /
 *       beta (read once per CTA).
 */
typedef struct gge_gemm_args {
  gge_tensor A;
  gge_tensor B;
  const gge_tensor* C;
  const gge_tensor* D;
  const gge_tensor* PostAct;
  float alpha;
  float beta;
  const float* alpha_dev;
  const float* beta_dev;
  int32_t act;               /* gge_act */
  int32_t reserved;
  const gge_config* config;  /* NULL = defaults */
} gge_gemm_args;

/* Bytes of device workspace that let a call run at full speed, for every
 * entry point except gge_gemm_varlen_k and gge_gemm_gather_k (see
 * gge_workspace_size_varlen_k): 256 bytes of status words and scheduler
 * counters, plus, for plain problems, room to split the last, partly filled
 * wave of tiles along K (16 KiB of tickets, then one 128 x 256 fp32 partial
 * block per SM: about 20 MiB on a 152-SM GPU; the split needs a 256-byte
 * aligned workspace).  Any workspace of at least 256 bytes works: with less
 * room the last wave runs unsplit.  Layout: bytes 0-255 status words, then
 * the tickets, then the partial blocks (or, for varlen-K, the tensor-map
 * slots), so one workspace serves every entry point in turn.  The workspace is caller-owned, at least 16-byte
 * aligned, must be zeroed once before first use, and is reusable across calls
 * on the same stream (not by calls running concurrently on other streams).
 * The arguments are not inspected (they may be NULL); the size depends on the
 * current device. */
size_t gge_workspace_size(const gge_gemm_args* args, int32_t num_groups);

/* Workspace bytes gge_gemm_varlen_k and gge_gemm_gather_k need on the current
 * device: the status words and the ticket region plus 4 KiB of tensor-map copies for each CTA a
 * launch can have (one per SM: about 0.6 MiB on a 152-SM GPU).  The arguments
 * are not inspected (they may be NULL); returns 0 if the device cannot be
 * queried.  (The slots start after the 16 KiB ticket region, which these
 * calls leave untouched.) */
size_t gge_workspace_size_varlen_k(const gge_gemm_args* args, int32_t num_groups);

/* D = alpha A B^T + beta C (PostAct must be NULL and act NONE).
 * Page: quack/dense_gemm_sm90.py, gemm_sm90 / GemmSm90.epi_visit_acc_subtile. */
gge_status gge_gemm(const gge_gemm_args* args, void* workspace, size_t workspace_bytes,
                    gge_stream_t stream);

/* D (optional) and PostAct = act(alpha A B^T + beta C), act applied to the
 * unrounded fp32 value.  Page: quack/gemm_act_sm90.py, gemm_act_sm90 /
 * GemmActSm90.epi_visit_acc_subtile. */
gge_status gge_gemm_act(const gge_gemm_args* args, void* workspace, size_t workspace_bytes,
                        gge_stream_t stream);

/* Backward activation epilogue: the accumulator S = A B^T is the incoming
 * gradient dout, C (required) holds the pre-activation x, and
 *   D = act'(x) * S      (required)        PostAct = act(x)   (optional)
 * with act in {relu, relu_sq, gelu_tanh, silu}; alpha and beta are not used.
 * Page: quack-kernels 0.2.0 diff, quack/gemm_dact_sm90.py, gemm_dact_sm90 /
 * GemmDActSm90.epi_visit_acc_subtile (act_bwd(x, dout) -> (dx, out)). */
gge_status gge_gemm_dact(const gge_gemm_args* args, void* workspace, size_t workspace_bytes,
                         gge_stream_t stream);

/* Varlen-M grouped GEMM: A is [total_M, K, 1], B is [N, K, G] (batch = G
 * groups), C / D / PostAct are [total_M, N, 1].  Group g owns rows
 * cu_seqlens_m[g] .. cu_seqlens_m[g+1]-1 and multiplies them by B[:,:,g];
 * rows outside every group are not written.  cu_seqlens_m: DEVICE int32
 * [G+1], non-decreasing, cu[0] >= 0, cu[G] <= total_M (an offset that breaks
 * this is held to [0, total_M] and to the largest before it, and reported as
 * GGE_ERR_INDEX_RANGE by gge_read_device_status).
 * 1 <= G <= 1024.  act as in gge_gemm_act.
 * Page: quack/dense_gemm_sm90.py, GemmSm90 with VarlenArguments(mCuSeqlensM). */
gge_status gge_gemm_varlen_m(const gge_gemm_args* args, const int32_t* cu_seqlens_m,
                             int32_t num_groups, void* workspace, size_t workspace_bytes,
                             gge_stream_t stream);

/* Varlen-K grouped GEMM (the weight-gradient shape of grouped experts):
 * A is [M, total_K, 1], B is [N, total_K, 1], C / D / PostAct are [M, N, G]
 * (batch = G groups).  Group g contracts the K columns
 * cu_seqlens_k[g] .. cu_seqlens_k[g+1]-1:
 *   D[:,:,g] = alpha * A[:, K_g] B[:, K_g]^T + beta * C[:,:,g]
 * and an empty group gives alpha * 0 + beta * C.  Columns outside every group
 * take part in no product.  cu_seqlens_k: DEVICE int32 [G+1], non-decreasing,
 * cu[0] >= 0, cu[G] <= total_K.  When A or B is K-major, every non-empty
 * group must start on a 16-byte boundary of the K-major rows (a multiple of 8
 * for 16-bit, 16 for 8-bit operands); with A M-major and B N-major any
 * offsets are allowed.  A group that breaks these rules contracts nothing and
 * is reported as GGE_ERR_INDEX_RANGE by gge_read_device_status.
 * 1 <= G <= 1024.  act as in gge_gemm_act.  The workspace (256-byte aligned,
 * zeroed once) must hold gge_workspace_size_varlen_k bytes: the kernel keeps
 * per-CTA copies of the A / B tensor maps there, rewritten with each group's
 * K extent.  Page: quack/dense_gemm_sm90.py, GemmSm90 with
 * VarlenArguments(mCuSeqlensK) (update_tensormap_shape per group; a group
 * with k_tile_cnt == 0 keeps a zero accumulator). */
gge_status gge_gemm_varlen_k(const gge_gemm_args* args, const int32_t* cu_seqlens_k,
                             int32_t num_groups, void* workspace, size_t workspace_bytes,
                             gge_stream_t stream);

/* Gather-K: the varlen-K GEMM above whose A is gathered along K.  args->A is
 * the SOURCE [M, K_src, 1], M-major (stride_row == 1; the usual storage of
 * X [K_src, M] row-major), 16-bit, M a multiple of 8; a_idx is DEVICE int32
 * [total_K] with total_K = columns of B.  Column k of the effective A is
 * column a_idx[k] of the source; B [N, total_K] is read at column k itself.
 * Group rules as in gge_gemm_varlen_k (with a K-major B, non-empty groups
 * start on multiples of 8); an index outside [0, K_src) reads zeros and is
 * reported as GGE_ERR_INDEX_RANGE.  One CTA per 128 x BN tile; the rows are
 * copied by four gather warps with 16-byte cp.async (a TMA row gather issues
 * too slowly for four rows of 128 bytes at a time).  The workspace (256-byte
 * aligned) must hold gge_workspace_size_varlen_k bytes.  Page: quack/dense_gemm_sm90.py,
 * GemmSm90 with gather_A and VarlenArguments(mCuSeqlensK)
 * (copy_utils.gather_k_get_copy_fn). */
gge_status gge_gemm_gather_k(const gge_gemm_args* args, const int32_t* a_idx,
                             const int32_t* cu_seqlens_k, int32_t num_groups, void* workspace,
                             size_t workspace_bytes, gge_stream_t stream);

/* Gather-A GEMM: row r of the effective A is row a_idx[r] of the source
 * matrix args->A ([rows_src, K, 1], K-major, 16-bit).  With cu_seqlens_m
 * (DEVICE int32 [G+1]) it is the varlen-M problem above, a_idx being
 * [total_M] with total_M = rows of D / PostAct; with cu_seqlens_m == NULL it
 * is a plain batched problem of M = rows of D per batch and a_idx [L][M].
 * An index outside [0, rows_src) reads zeros and is reported as
 * GGE_ERR_INDEX_RANGE.  Page: quack/dense_gemm_sm90.py,
 * GemmSm90.load_AB_gather_A (mAIdx). */
gge_status gge_gemm_gather_a(const gge_gemm_args* args, const int32_t* a_idx,
                             const int32_t* cu_seqlens_m, int32_t num_groups, void* workspace,
                             size_t workspace_bytes, gge_stream_t stream);

/* ---- low-precision linear layers ----------------------------------------
 * Microscaled operands (narrow codes, one scale per block of K), what makes
 * them (quantisation, and the RMS norm that ends in one), their product, and
 * the norm's backward.  The pages have no counterpart: these are additions of
 * this library.  The conventions above hold (asynchronous on `stream`,
 * validated before any launch, strides in elements unless a field says bytes).
 * Rows of an output may not overlap, nor may its batches: each lies behind the one
 * before, or row r of every batch before row r + 1 of any.  Inputs may overlap. */

/* Formats.  value = code * block scale (* the tensor scale, GGE_NVFP4).
 *   GGE_MXFP8  e4m3 codes, blocks of 32, scales 2^(byte - 127), byte 255 = NaN
 *   GGE_MXFP4  e2m1 codes, blocks of 32, scales as above
 *   GGE_NVFP4  e2m1 codes, blocks of 16, e4m3 scales, one fp32 scale a tensor   */
typedef enum gge_mx_format { GGE_MXFP8 = 0, GGE_MXFP4 = 1, GGE_NVFP4 = 2 } gge_mx_format;

/*
 * A microscaled matrix [rows, cols, batch] whose blocks run along cols (a
 * product's K).
 *   codes  row-major; two 4-bit codes a byte, the even column in the low half.
 *          A row takes gge_mx_row_bytes bytes (whole 32s of columns; the codes
 *          past `cols` are zero).  16-byte aligned, as are the byte strides.
 *   scales tiles of 512 bytes for 128 rows x 4 blocks, ceil(blocks / 4) tiles
 *          along K for each 128 rows: the scale of row r, block b is byte
 *          (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4 of tile [r / 128][b / 4].
 *          Bytes of blocks past the row's last one are zero; rows past the last
 *          one may hold anything.  gge_mx_scale_bytes in all, 128-byte aligned.
 */
typedef struct gge_mx_tensor {
  void* codes;
  void* scales;
  const float* tensor_scale; /* device scalar (GGE_NVFP4; NULL: 1), must be > 0   */
  int32_t format;            /* gge_mx_format                                     */
  int32_t reserved;          /* must be 0                                         */
  int64_t rows, cols, batch;
  int64_t stride_row;        /* BYTES between rows of codes                       */
  int64_t stride_batch;      /* BYTES between batches of codes                    */
  int64_t scale_stride_batch; /* BYTES between batches of scales (a multiple of a
                                128-row block's scales)                           */
} gge_mx_tensor;

/* Bytes of one row of codes, and of one batch's scales (0 for a bad format). */
size_t gge_mx_row_bytes(int32_t format, int64_t cols);
size_t gge_mx_scale_bytes(int32_t format, int64_t rows, int64_t cols);

/* q = x quantised.  x: [rows, cols, batch] in bf16, f16 or f32, with
 * stride_col == 1 or stride_row == 1 (the transpose of a row-major matrix, as
 * the weight-gradient products need it, of at most 65535 * 64 rows:
 * GGE_ERR_UNSUPPORTED beyond); rows may start on any element.
 *   GGE_MXFP8, GGE_MXFP4: a block's scale is the smallest power of two 2^e (e >=
 *     -127) with max|x| <= 2^e * (448 or 6); code = round(x / 2^e), exact but for
 *     the rounding (to nearest, ties to even).
 *   GGE_NVFP4, t the tensor scale: scale s = e4m3(min(max(max|x| / (6 t), 2^-9),
 *     448)), code = round(x * (1 / (s t))) in fp32 arithmetic, at most 6 in size.
 *     t = max over the tensor / (6 * 448) uses the scales' whole range.
 * A block that holds an infinity or a NaN becomes NaN throughout.
 * values (may be NULL): the numbers that the codes stand for, [rows, cols,
 * batch] row-major in bf16, f16 or f32 (rounded once). */
gge_status gge_mx_quantize(const gge_tensor* x, const gge_mx_tensor* q, const gge_tensor* values,
                           gge_stream_t stream);

/* y = the numbers that q's codes stand for, row-major in bf16, f16 or f32. */
gge_status gge_mx_dequantize(const gge_mx_tensor* q, const gge_tensor* y, gge_stream_t stream);

/*
 * D       = alpha * tA * tB * sum_k (a_k sa_k) (b_k sb_k) + beta * C
 * PostAct = act(same value, before rounding)
 *   A [M, K, L] and B [N, K, L] of one format (tA, tB: their tensor scales);
 *   C, D, PostAct, act, alpha, beta as in gge_gemm_act (D and PostAct each
 *   optional, not both NULL; PostAct required when act is not NONE).  N must be
 *   a multiple of 8, M, K and L may be anything.  K == 0 gives beta * C.
 *   config (may be NULL): tile_n 0 (automatic), 256 (a CTA pair, 256 x 256), 128
 *   (one CTA, 128 x 128) or 64 (one CTA, for few rows of A: the roles of A and B
 *   are exchanged); num_ctas, raster_band, stages, timeout_ns; of the flags
 *   those for direct stores, no split, raster along N and the test hook.
 * Few tiles are split along K over a cluster of 2, 4 or 8 CTAs, which add their
 * sums in a fixed order through shared memory.  The workspace holds the status
 * words (at least 256 bytes; NULL: device errors go unrecorded).
 */
typedef struct gge_gemm_mx_args {
  gge_mx_tensor A;
  gge_mx_tensor B;
  const gge_tensor* C;
  const gge_tensor* D;
  const gge_tensor* PostAct;
  float alpha;
  float beta;
  const float* alpha_dev;
  const float* beta_dev;
  int32_t act;
  int32_t reserved;
  const gge_config* config;
} gge_gemm_mx_args;
gge_status gge_gemm_mx(const gge_gemm_mx_args* args, void* workspace, size_t workspace_bytes,
                       gge_stream_t stream);

/* The backward activation epilogue on microscaled operands (as gge_gemm_dact):
 * with S = tA * tB * sum_k (a_k sa_k) (b_k sb_k) the incoming gradient and C
 * (required) the pre-activation x, D = act'(x) * S (required) and PostAct =
 * act(x) (optional); act is not NONE, alpha and beta are not used. */
gge_status gge_gemm_mx_dact(const gge_gemm_mx_args* args, void* workspace, size_t workspace_bytes,
                            gge_stream_t stream);

/*
 * RMS norm with the residual's addition:
 *   h = round(x + residual)  (h = x without one)
 *   inv = 1 / sqrt(mean over a row of h^2 + eps)       y = (h * inv) * weight
 *   x, residual, residual_out (h), y: [rows, cols, 1] of one type (bf16, f16 or
 *     f32), stride_col == 1, rows may start on any element; every output may be
 *     NULL, and residual_out may be x or residual itself.  residual_out is
 *     written only when there is a residual.
 *   weight: `cols` contiguous values of weight_dtype.  inv_rms: fp32 [rows].
 *   q, values: y quantised from fp32 as gge_mx_quantize does, and the numbers
 *     that its codes stand for (values needs q).
 */
typedef struct gge_rmsnorm_args {
  gge_tensor x;
  const gge_tensor* residual;
  const gge_tensor* residual_out;
  const gge_tensor* y;
  const gge_mx_tensor* q;
  const gge_tensor* values;
  const void* weight;
  int32_t weight_dtype; /* gge_dtype */
  float eps;
  float* inv_rms;
} gge_rmsnorm_args;
gge_status gge_rmsnorm(const gge_rmsnorm_args* args, gge_stream_t stream);

/*
 * Its backward, from the saved h and inv_rms:
 *   g = dy * weight      dx = inv * (g - h * inv^2 * mean(g * h)) + dh
 *   dweight = sum over rows of dy * (h * inv)     (fp32, in a fixed order)
 * dx is the gradient of x and of the residual alike.  dh (may be NULL): the
 * gradient that reaches residual_out directly.  dy, h, dh and dx: [rows, cols, 1]
 * of one type; dx may be dy, h or dh itself.  dweight may be NULL.  A quantised
 * output's dy passes through unchanged.  The workspace (256-byte aligned) must hold
 * gge_workspace_size_rmsnorm_bwd(cols) bytes when dweight is given.
 */
typedef struct gge_rmsnorm_bwd_args {
  gge_tensor dy;
  gge_tensor h;
  const gge_tensor* dh;
  gge_tensor dx;
  const void* weight;
  int32_t weight_dtype;
  int32_t reserved;
  const float* inv_rms;
  float* dweight;
} gge_rmsnorm_bwd_args;
size_t gge_workspace_size_rmsnorm_bwd(int64_t cols);
gge_status gge_rmsnorm_bwd(const gge_rmsnorm_bwd_args* args, void* workspace,
                           size_t workspace_bytes, gge_stream_t stream);

/* ---- 8 bits with a scale for each block of 128 ---------------------------
 * Operands in 8-bit floating point with one fp32 scale for each
 * block of 128 columns of a row, or of 128 rows x 128 columns; what makes them
 * (quantisation, transposition, the layer norm and the product's own epilogue),
 * their product, and the backward from activations that were kept in this form.
 * Additions of this library, under the conventions of the section above. */

/*
 * A matrix [rows, cols, batch] of 8-bit codes; blocks run along cols (a product's K).
 *   codes   row-major, dtype GGE_E4M3 or GGE_E5M2; base and byte strides 16-byte
 *           aligned.  Bytes between a row's end and the next row are not touched.
 *   scales  fp32; the scale of row r, column block b (b = col / 128) of batch l is
 *           scales[(r / block_rows) * scale_stride_row + b * scale_stride_col +
 *           l * scale_stride_batch].  block_rows is 1 or 128.  The kernels read
 *           scale_stride_row == 1 best (blocks of neighbouring rows together).
 * value = code * scale.
 */
typedef struct gge_b128_tensor {
  void* codes;
  float* scales;
  int32_t dtype;      /* GGE_E4M3 or GGE_E5M2 */
  int32_t block_rows; /* 1 or 128             */
  int64_t rows, cols, batch;
  int64_t stride_row, stride_batch; /* of codes */
  int64_t scale_stride_row, scale_stride_col, scale_stride_batch; /* in floats */
} gge_b128_tensor;

/* q = x quantised.  x: [rows, cols, batch] in bf16, f16 or f32, with stride_col == 1
 * or stride_row == 1 (a transposed view); rows may start on any element.  For each
 * block, in fp32 arithmetic with the top value t = 448 (e4m3) or 57344 (e5m2):
 *   scale = max(max|x| * (1 / t), 2^-126)     code = round(x * (1 / scale))
 * to nearest, ties to even, at most t in size.  A block that holds an infinity or a
 * NaN gets a NaN scale: all of it reads back as NaN.
 * values (may be NULL): the numbers that the codes stand for, [rows, cols, batch]
 * row-major in bf16, f16 or f32 (rounded once). */
gge_status gge_b128_quantize(const gge_tensor* x, const gge_b128_tensor* q, const gge_tensor* values,
                             gge_stream_t stream);

/* q = the transpose of x's numbers, quantised anew along its own rows: x [rows, cols,
 * batch] -> q [cols, rows, batch], as the weight gradient's product needs an
 * activation that was kept in 8 bits.  values as above. */
gge_status gge_b128_transpose(const gge_b128_tensor* x, const gge_b128_tensor* q,
                              const gge_tensor* values, gge_stream_t stream);

/* y = the numbers that q's codes stand for, row-major in bf16, f16 or f32. */
gge_status gge_b128_dequantize(const gge_b128_tensor* q, const gge_tensor* y, gge_stream_t stream);

/*
 * D       = alpha * S + beta * C      S[m, n] = sum over blocks b of K of
 * PostAct = act(same value, before rounding)      sA[m, b] sB[n, b] sum_{k in b} a[m, k] b[n, k]
 *   A [M, K, L] and B [N, K, L], each with codes of either type and blocks of 1 or
 *   128 rows.  The sum within a block runs on the tensor core in fp32; blocks are
 *   scaled and added in fp32, in the order of K.  A block's term is its sum times the
 *   product sA sB, which is rounded to fp32 first: a product below 2^-126 loses up to
 *   2^-150, so the term as much times its sum (which is 2^25 at most in e4m3, 2^39 in
 *   e5m2); one of 2^128 or more makes the term an infinity or a NaN.
 *   C, D and PostAct: [M, N, L] as a gge_tensor (16 bits or fp32, as in gge_gemm) or,
 *   in the field that ends in 8, as a gge_b128_tensor with block_rows 1; at most one of the
 *   two each.  An 8-bit output is quantised from the fp32 value as gge_b128_quantize does
 *   (D8: a pre-activation kept for the backward; PostAct8: the next product's operand).
 *   D and PostAct are optional, not both absent; PostAct is required when act is not NONE.
 *   N must be a multiple of 8; M, K and L may be anything.  K == 0 gives beta * C.
 *   cu_seqlens_m (may be NULL): grouped rows, as gge_gemm_varlen_m: DEVICE int32
 *   [num_groups + 1], A [total_M, K, 1], B [N, K, num_groups], C, D and PostAct
 *   [total_M, N, 1]; row r of group g, cu[g] <= r < cu[g + 1], is multiplied with B[g].
 *   Rows of no group are not written.  At most 1024 groups.  An offset outside [0, total_M]
 *   or below one before it is held to these bounds and reported as GGE_ERR_INDEX_RANGE.
 *   config (may be NULL): tile_n 0 (automatic), 256 (a CTA pair, 256 x 256), 128 or 64
 *   (one CTA, 128 rows; 64 not with 8-bit outputs); num_ctas, raster_band, stages, timeout_ns;
 *   of the flags those for no split, raster along N and the test hook.
 * Few tiles are split along K over a cluster of 2 or 4 CTAs, which add their sums in a
 * fixed order through shared memory (not grouped rows).  D may be C itself (a gradient
 * added to in place).  The workspace holds the status
 * words (at least 256 bytes; NULL: device errors go unrecorded).
 */
typedef struct gge_gemm_b128_args {
  gge_b128_tensor A;
  gge_b128_tensor B;
  const gge_tensor* C;
  const gge_tensor* D;
  const gge_tensor* PostAct;
  const gge_b128_tensor* C8;
  const gge_b128_tensor* D8;
  const gge_b128_tensor* PostAct8;
  const int32_t* cu_seqlens_m;
  int32_t num_groups;
  int32_t act;
  float alpha;
  float beta;
  const float* alpha_dev;
  const float* beta_dev;
  const gge_config* config;
} gge_gemm_b128_args;
gge_status gge_gemm_b128(const gge_gemm_b128_args* args, void* workspace, size_t workspace_bytes,
                         gge_stream_t stream);

/* The backward activation epilogue (as gge_gemm_dact): with S the incoming gradient and
 * C or C8 (one of them required) the pre-activation x, D = act'(x) * S (required, in either
 * form) and PostAct = act(x) (optional); act is not NONE, alpha and beta are not used.
 * Neither output may be C or C8, which is read again after D is written: INVALID_ARG.
 * Grouped rows as above. */
gge_status gge_gemm_b128_dact(const gge_gemm_b128_args* args, void* workspace,
                              size_t workspace_bytes, gge_stream_t stream);

/*
 * Layer norm with the residual's addition:
 *   h = round(x + residual)  (h = x without one)
 *   mean, var = of a row of h      rstd = 1 / sqrt(var + eps)
 *   y = (h - mean) * rstd * weight + bias
 *   x, residual, residual_out (h), y: [rows, cols, 1] of one type (bf16, f16 or f32),
 *     stride_col == 1, rows may start on any element; every output may be NULL, and
 *     residual_out may be x or residual itself.  residual_out is written only when there
 *     is a residual.
 *   weight, bias (each may be NULL: 1 and 0): `cols` contiguous values of param_dtype.
 *   mean, rstd: fp32 [rows].  A row that holds an infinity or a NaN has a NaN rstd and y, as may one
 *     whose squares leave fp32 (values above 2^63 in size).
 *   q, values: y quantised from fp32 as gge_b128_quantize does (block_rows 1), and the
 *     numbers that its codes stand for (values needs q).
 *   h8: h quantised (block_rows 1), as the backward may read it.
 */
typedef struct gge_layernorm_args {
  gge_tensor x;
  const gge_tensor* residual;
  const gge_tensor* residual_out;
  const gge_tensor* y;
  const gge_b128_tensor* q;
  const gge_tensor* values;
  const gge_b128_tensor* h8;
  const void* weight;
  const void* bias;
  int32_t param_dtype; /* gge_dtype */
  float eps;
  float* mean;
  float* rstd;
} gge_layernorm_args;
gge_status gge_layernorm(const gge_layernorm_args* args, gge_stream_t stream);

/*
 * Its backward, from the saved h (in 16 or 32 bits, or in 8 bits: exactly one of h and h8),
 * mean and rstd:
 *   n = (h - mean) * rstd      g = dy * weight
 *   dx = rstd * (g - mean(g) - n * mean(g * n)) + dh
 *   dweight = sum over rows of dy * n      dbias = sum over rows of dy   (fp32, in a fixed
 *   order)
 * dx is the gradient of x and of the residual alike.  dh (may be NULL): the gradient that
 * reaches residual_out directly.  dy, h, dh and dx: [rows, cols, 1] of one type; dx may be dy,
 * h or dh itself.  weight, dweight and dbias may be NULL.  A quantised output's dy passes
 * through unchanged.  The workspace (256-byte aligned) must hold
 * gge_workspace_size_layernorm_bwd(cols) bytes when dweight or dbias is given.
 */
typedef struct gge_layernorm_bwd_args {
  gge_tensor dy;
  const gge_tensor* h;
  const gge_b128_tensor* h8;
  const gge_tensor* dh;
  gge_tensor dx;
  const void* weight;
  int32_t weight_dtype;
  int32_t reserved;
  const float* mean;
  const float* rstd;
  float* dweight;
  float* dbias;
} gge_layernorm_bwd_args;
size_t gge_workspace_size_layernorm_bwd(int64_t cols);
gge_status gge_layernorm_bwd(const gge_layernorm_bwd_args* args, void* workspace,
                             size_t workspace_bytes, gge_stream_t stream);

/* gge_gemm_act without a caller workspace, for callers that cannot allocate
 * device memory where they run the GEMM (a host framework that owns all device
 * memory through its own arena or caching allocator, or a latency-critical path
 * that must not call the allocator).  The pages have no counterpart: it is an
 * addition of this library.
 *   - The scratch (the 256 bytes of status words) lives in a fixed 1024-byte
 *     __device__ area inside the library, held on every GPU that loads it until
 *     process exit.  It has no room for partial sums, so the last wave of tiles
 *     is never split along K on this path (see gge_workspace_size).
 *   - The first call on a device looks up that area's device address (on the
 *     current device); make that first call before any stream capture.  A
 *     failed lookup returns GGE_ERR_CUDA and is tried again by the next call.
 *   - Each call clears the area's scheduler counters (an async memset on
 *     `stream`), then launches the same kernel as gge_gemm_act.  Nothing is
 *     allocated.
 *   - Device errors (a wait past its limit, GGE_ERR_TIMEOUT) are recorded in
 *     the area and kept until gge_read_static_scratch_status reads them.
 *   - All calls on a device share the one area: calls that overlap on the GPU
 *     (different streams without ordering) race on it. */
gge_status gge_gemm_act_static_scratch(const gge_gemm_args* args, gge_stream_t stream);

/* gge_read_device_status for the library's own scratch area: synchronises
 * `stream`, returns the device status that gge_gemm_act_static_scratch calls
 * on the current device recorded since it was last read (GGE_OK or
 * GGE_ERR_TIMEOUT), and clears it.  `detail` (may be NULL) receives
 * [where, tile].  No counterpart on the pages. */
gge_status gge_read_static_scratch_status(gge_stream_t stream, int32_t* detail);

/* Synchronises `stream`, returns the device status recorded in `workspace`
 * since it was last cleared (GGE_OK, GGE_ERR_TIMEOUT or GGE_ERR_INDEX_RANGE)
 * and clears it.  `detail` (may be NULL) receives [where, tile]. */
gge_status gge_read_device_status(void* workspace, gge_stream_t stream, int32_t* detail);

const char* gge_status_string(gge_status status);

/* ---- host-side helpers (no GPU needed) -------------------------------- */

/* FastDivmod parameters as quack/fast_math.py FastDivmod.create builds them:
 * p = 31 + ceil(log2 d), multiplier = ceil(2^p / d), shift = p - 32. */
void gge_fastdivmod_params(int32_t divisor, uint32_t* multiplier, uint32_t* shift);

/* q = n / d by the FastDivmod formula (host build of the device code),
 * for 0 <= n < 2^31. */
int32_t gge_fastdivmod_div(int32_t divisor, int32_t n);

/* The plain persistent schedule: tile index t -> (batch, m-tile, n-tile) for a
 * grid of tiles_m x tiles_n tiles per batch and `batches` batches, with
 * `band` m-tiles per raster band (n-tiles when along_n != 0, config flag
 * bit 7).  Writes `count` triples into out[3*count] for t = 0 .. count-1.
 * Returns the number of tiles of the problem.  Page: quack/dense_gemm_sm90.py,
 * the tile scheduler's raster_order and max_swizzle_size. */
int32_t gge_schedule_map(int32_t tiles_m, int32_t tiles_n, int32_t batches, int32_t band,
                         int32_t along_n, int32_t count, int32_t* out);

/* The launch plan the library would use for `args` (tile and pipeline
 * shape).  form: GGE_FORM_DEFAULT (plain, or varlen-M when num_groups > 0),
 * GGE_FORM_GATHER_A, GGE_FORM_VARLEN_K or GGE_FORM_GATHER_K.  Returns GGE_OK or the validation
 * error of the call. */
enum { GGE_FORM_DEFAULT = 0, GGE_FORM_GATHER_A = 1, GGE_FORM_VARLEN_K = 2, GGE_FORM_GATHER_K = 3 };
typedef struct gge_plan_info {
  int32_t tile_m, tile_n, tile_k, stages;  /* tile_m: rows per (pair) tile */
  int32_t num_tiles;  /* plain and varlen-K problems; -1 for varlen-M (known on
                         the device only) */
  int32_t grid;
  int32_t threads;
  int32_t smem_bytes;
  int32_t raster_band;
  int32_t cta_group;  /* 1 or 2 CTAs per tile */
  int32_t raster_along_n; /* 1: bands of n-tiles (config flag bit 7) */
  int32_t tail_tiles; /* tiles of the last, partly filled wave that are split along K
                         (plain problems; 0: none).  Reported only when the unit
                         count is known here, i.e. config->num_ctas is set. */
  int32_t tail_splits; /* K-slices per split tile (1: none) */
} gge_plan_info;
gge_status gge_plan(const gge_gemm_args* args, int32_t num_groups, int32_t form,
                    gge_plan_info* out);

/* ---- autotuning ---------------------------------------------------------
 * Page: quack-kernels 0.2.0 diff, quack/gemm_config.py (GemmConfig and
 * get_all_configs: a space of tile shapes, cooperative / ping-pong
 * warpgroups, 1x2 / 2x1 clusters and swap_ab to search by timing).  Here the space is the launch shapes this library
 * has: one CTA per 128 x 128 or 128 x 256 tile, or a CTA pair per 256 x 256,
 * 224, 192 or 160 tile (not with the gather forms), times the raster of
 * plain problems (bands of m-tiles of the automatic width or 8, or bands of
 * n-tiles: flag bit 7), times staged or direct epilogue stores.  The pages' swap_ab is not in the space: it needs M-major
 * output stores, which the epilogue does not have. */

/* Which entry point a tuning call times. */
enum {
  GGE_OP_GEMM = 0,      /* gge_gemm (PostAct NULL) or gge_gemm_act          */
  GGE_OP_DACT = 1,      /* gge_gemm_dact                                      */
  GGE_OP_VARLEN_M = 2,  /* gge_gemm_varlen_m (cu = cu_seqlens_m)              */
  GGE_OP_GATHER_A = 3,  /* gge_gemm_gather_a (idx = a_idx, cu may be NULL)    */
  GGE_OP_VARLEN_K = 4,  /* gge_gemm_varlen_k (cu = cu_seqlens_k)              */
  GGE_OP_GATHER_K = 5   /* gge_gemm_gather_k (idx = a_idx, cu = cu_seqlens_k) */
};

/* Writes up to `max` candidate configurations for (args, op) into `out`
 * (host only, no GPU needed: shapes the planner rejects are left out) and
 * returns how many there are (which may exceed `max`).  Each candidate is
 * args->config (or the defaults) with tile_n, cta_group and raster_band set. */
int32_t gge_tune_candidates(const gge_gemm_args* args, int32_t op, int32_t num_groups,
                            gge_config* out, int32_t max);

/* Times every candidate of (args, op) on `stream` -- `reps` launches each
 * after one warm-up launch, CUDA events around them -- and writes the fastest
 * configuration to *best (and its mean time in ms to *best_ms, if not NULL).
 * Every launch computes the real outputs, so they hold the result on return.
 * Synchronises `stream`.  The result is also stored in an in-process cache
 * keyed by the problem's shapes, dtypes, strides pattern, activation and op,
 * which gge_tuned_config reads.  Errors of a launch are returned as they are;
 * a candidate rejected by the planner is skipped. */
gge_status gge_autotune(const gge_gemm_args* args, int32_t op, const int32_t* idx,
                        const int32_t* cu, int32_t num_groups, void* workspace,
                        size_t workspace_bytes, gge_stream_t stream, int32_t reps,
                        gge_config* best, float* best_ms);

/* The configuration gge_autotune found for a problem of the same key, or
 * GGE_ERR_INVALID_ARG if there is none (no GPU work).  The launch-shape
 * fields are the search's; tile_counts, timeout_ns and batch_idx_permute are
 * taken from args->config (NULL / 0 without one). */
gge_status gge_tuned_config(const gge_gemm_args* args, int32_t op, int32_t num_groups,
                            gge_config* out);

/* Library version string. */
const char* gge_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GGE_H_ */
