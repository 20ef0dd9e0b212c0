/*
 * fg.h -- C ABI of the GB300 (sm_103a) preshuffled-weight GEMM library.
 *
 *   Y[M,N] = dequant(A[M,K]) . dequant(B[N,K])^T,  fp32 accumulation, bf16 Y.
 *
 * Sources of the operation (titles of the pages that state the method):
 *  - aiter PR "FlyDSL split-K preshuffle decode GEMM for small-M shapes
 *    (FP8 + MX, gfx950/gfx942)", sections Summary and What's included: the
 *    two-pass split-K GEMM for small M (fp32 partials in a workspace, then a
 *    reduce that downcasts once at the final store), the direct-output
 *    epilogue for split_k = 1, the three scale modes (FP8 per-tensor, FP8
 *    128-block blockscale, MX: mxfp8 with one E8M0 per 128 K, mxfp4 with
 *    one E8M0 per 32 K; the OCP-standard 32-element mxfp8 block is offered
 *    beside the pages' 128-element one), the weight/scale preshuffle helpers and the
 *    shape-keyed dispatch; Copilot review: K must be a multiple of the scale
 *    block, and already-preshuffled weights must not be shuffled again.
 *  - FlyDSL PR "Enable the gmem->LDS async copy for f16/bf16 preshuffle
 *    GEMM", Summary and Performance: the large-M bf16 preshuffle GEMM
 *    (M=54560, N=K=8192), and the early, clear error off the supported arch.
 *  - FlyDSL PR "Migrate kernels to fx.copy / .llvm_ptr; expand
 *    kernel-code-cleanup skill", Validation and the later commit "Reject
 *    tiles whose A tile is only partially loaded": the fp8 large-M shape
 *    (M=N=4096, K=8192) and the rule that a shape the kernel cannot load
 *    whole is refused up front instead of computed wrongly.
 *
 * Conventions for every call:
 *  - Device pointers are caller-owned (allocate them with any allocator).
 *    The library never allocates, frees or synchronises device memory, and
 *    never writes outside the buffers it is given.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Launches are asynchronous; errors found on the host are
 *    returned before anything is launched.  A kernel that gives up on a
 *    bounded wait records FG_ERR_TIMEOUT in a device word that
 *    fg_get_error() returns.
 *  - Only compute capability 10.3 devices are accepted
 *    (FG_ERR_UNSUPPORTED_ARCH otherwise).
 *  - Layouts are row-major.  A: [M][K] bf16 | e4m3 bytes | packed e2m1
 *    ([M][K/2] bytes, low nibble = even k).  B likewise [N][K] (for
 *    MXFP4_FP8A, A is e4m3 [M][K] and B packed e2m1 [N][K/2]).
 *    Y: [M][N] bf16.  Workspace: [split_k][M][N] fp32.
 *  - Shapes: N % 128 == 0; K * element bits / 8 must be a multiple of 128
 *    bytes (K % 64 for bf16, K % 128 for fp8 and MXFP4_FP8A, K % 256 for
 *    mxfp4); the 128-K scale blocks of FP8_BLOCK128 / MXFP8 and the 32-K
 *    blocks of MXFP4 then divide K exactly.  M >= 0 (M == 0 is a no-op).
 */
#ifndef FG_H
#define FG_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FG_API __attribute__((visibility("default")))
#else
#define FG_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fg_status {
  FG_OK = 0,
  FG_ERR_INVALID_ARG = 1,      /* null pointer, bad enum, bad flag, bad split_k   */
  FG_ERR_SHAPE = 2,            /* N, K or M violate the shape rules above          */
  FG_ERR_ALIGN = 3,            /* a pointer is not 16-byte aligned (4 for scales)  */
  FG_ERR_LAYOUT = 4,           /* descriptor is not one fg_preshuffle_b made, or   */
                               /* its mode differs from the call's                 */
  FG_ERR_WORKSPACE = 5,        /* workspace missing or too small                   */
  FG_ERR_UNSUPPORTED_ARCH = 6, /* current device is not compute capability 10.3    */
  FG_ERR_CUDA = 7,             /* a CUDA runtime/driver call failed                */
  FG_ERR_TIMEOUT = 8           /* a kernel gave up on a bounded wait               */
} fg_status;

typedef enum fg_mode {
  FG_BF16 = 0,         /* bf16 A and B, no scales                                   */
  FG_FP8_TENSOR = 1,   /* e4m3 A and B; fp32 scalars a_s, b_s                       */
  FG_FP8_BLOCK128 = 2, /* e4m3; a_s fp32 [M][K/128]; b_s fp32 [N/128][K/128]        */
  FG_MXFP8 = 3,        /* e4m3; E8M0 a_sf [M][K/128], b_sf [N][K/128]               */
  FG_MXFP4 = 4,        /* packed e2m1; E8M0 a_sf [M][K/32], b_sf [N][K/32]          */
  FG_MXFP8_B32 = 5,    /* e4m3; E8M0 a_sf [M][K/32], b_sf [N][K/32] (OCP MX block)  */
  FG_MXFP4_FP8A = 6    /* A e4m3, E8M0 a_sf [M][K/32]; B packed e2m1, E8M0 b_sf     */
                       /* [N][K/32] ("MXFP4 fp8-A": fp8 activations, fp4 weights)   */
} fg_mode;

/* fg_gemm flags */
#define FG_FLAG_DEFER_REDUCE 0x1u /* split_k > 1: stop after writing the fp32 partials */
#define FG_FLAG_DEBUG_STALL 0x40000000u /* test hook: the MMA issuer waits on a barrier */
                                        /* nothing arrives at, so every bounded wait    */
                                        /* runs out and the call ends in FG_ERR_TIMEOUT */

/* element types of the operators' plain inputs and outputs */
typedef enum fg_type { FG_TYPE_F32 = 0, FG_TYPE_BF16 = 1 } fg_type;

/* what fg_quantize applies to its input first */
typedef enum fg_act {
  FG_ACT_NONE = 0,
  FG_ACT_SWIGLU = 1 /* rows of 2K values (g, u): silu(g) * u = g / (1 + exp(-g)) * u, */
                    /* in 32 bits: zero below g = -88.7, where exp(-g) overflows   */
} fg_act;

/* fg_moe_route flag: weights over the chosen experts only (they sum to 1) */
#define FG_FLAG_RENORMALIZE 0x1u

#define FG_BSHUF_MAGIC 0x31424746u /* "FGB1" */
#define FG_BSHUF_VERSION 1u

/*
 * Descriptor of a preshuffled weight, filled by fg_preshuffle_b.  It points
 * at caller-owned device buffers and carries a check word over its fields;
 * fg_gemm accepts only descriptors whose check word matches (a raw pointer,
 * a hand-made or edited descriptor, or one of another mode is rejected with
 * FG_ERR_LAYOUT).  Keep the buffers alive while the descriptor is used.
 *
 * Weight image layout: B viewed as N rows of Kb bytes (Kb = 2K bf16, K fp8,
 * K/2 fp4) cut into slabs of 128 rows x 128 bytes, slab (nb, kb) at index
 * nb*(Kb/128)+kb (16 KiB each); in a slab, 16-byte chunk c of row r sits at
 * byte r*128 + ((c ^ (r%8))*16) -- the image a 128-byte-swizzled K-major
 * tensor-core operand has in shared memory, so one pipeline stage of one
 * 128-row tile is one contiguous copy.  MXFP4_FP8A instead keeps the packed
 * fp4 bytes (Kb = K/2) in unswizzled blocks of 128 rows x 64 bytes (128 K),
 * block (nb, kb) at index nb*(K/128)+kb, row r at byte r*64; the image must
 * be 32-byte aligned.  The kernels load one block per tensor copy that puts
 * every 16 codes in the low half of a 16-byte shared-memory chunk (the
 * e2m1 operand form of the fp8/fp6/fp4 block-scaled MMA), so HBM moves
 * only the packed bytes.
 *
 * Scale image (sf): FP8_TENSOR: the fp32 b_s (16 bytes reserved);
 * FP8_BLOCK128: b_s fp32 [N/128][K/128] unchanged; MXFP8_B32 / MXFP4_FP8A
 * (one atom per 128 K) / MXFP4 (two atoms per 256 K): for each 128-row tile
 * and slab, atoms of 512 bytes, atom byte 16*(r%32) + 4*(r/32) + j = the
 * E8M0 of row r for the j-th 32-K block the atom covers; MXFP8 (one scale
 * per 128 K): one atom per four consecutive 128-K slabs of a 128-row tile,
 * byte j of row r = the E8M0 of slab 4g + j (zero past the last slab);
 * BF16: none.
 */
typedef struct fg_bshuf {
  uint32_t magic;
  uint32_t version;
  int32_t mode;
  int32_t tile_rows; /* 128 */
  int64_t N;
  int64_t K;
  void* data;        /* device: weight image, data_bytes long */
  void* sf;          /* device: scale image, sf_bytes long (NULL for BF16) */
  uint64_t data_bytes;
  uint64_t sf_bytes;
  uint64_t check;
} fg_bshuf;

/* Chosen kernel configuration for one GEMM shape (fg_gemm_plan). */
typedef struct fg_plan {
  int32_t path;        /* 0 = split-K decode kernel (weights on the MMA M side), 1 = large-M kernel */
  int32_t split_k;     /* K splits (1 = direct bf16 output, no workspace)                          */
  int32_t tile_m;      /* rows of A per CTA tile                                                   */
  int32_t tile_n;      /* rows of B per CTA tile                                                   */
  int32_t stage_slabs; /* 128-byte K slabs per pipeline stage                                      */
  int32_t stages;      /* pipeline depth                                                           */
  int32_t ctas;        /* CTAs launched by the main kernel                                         */
  int32_t from_table;  /* 1 if an exact dispatch-table row matched, 0 if the heuristic chose       */
  char name[96];       /* kernel/config name: arch, mode, shape identity                          */
} fg_plan;

/* Library version (major*10000 + minor*100 + patch). */
FG_API int fg_version(void);

/* Human-readable name of a status code. */
FG_API const char* fg_status_str(int status);

/* Message with the details of the last error returned on this host thread. */
FG_API const char* fg_last_error_message(void);

/*
 * Sizes of the buffers fg_preshuffle_b writes for a weight of the given mode
 * and shape: the weight image (N*Kb bytes) and the scale image (0 for BF16).
 * Errors: FG_ERR_INVALID_ARG (mode, null outputs), FG_ERR_SHAPE.
 */
FG_API fg_status fg_preshuffle_b_size(int mode, int64_t N, int64_t K, uint64_t* b_bytes, uint64_t* sf_bytes);

/*
 * One-time relayout of the weight B[N][K] (and of its scales) into the
 * images described above; fills *desc_out.  b_scales: FP8_TENSOR: device
 * fp32 scalar; FP8_BLOCK128: device fp32 [N/128][K/128]; MX: device uint8
 * E8M0 [N][K/128] (MXFP8) or [N][K/32] (MXFP4, MXFP8_B32, MXFP4_FP8A); BF16: must be NULL.  B and the images must
 * not overlap.  Errors: INVALID_ARG, SHAPE, ALIGN (16 bytes for B and the
 * images -- 32 for the MXFP4_FP8A weight image --, 4 for fp32 scales),
 * WORKSPACE (an image buffer smaller than
 * fg_preshuffle_b_size says), UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_preshuffle_b(int mode, const void* B, const void* b_scales, int64_t N, int64_t K, void* b_image,
                          uint64_t b_image_bytes, void* sf_image, uint64_t sf_image_bytes, fg_bshuf* desc_out,
                          void* stream);

/*
 * Inverse of fg_preshuffle_b: writes B[N][K] (and, if b_scales_out is not
 * NULL, the scales in the caller's layout) back from the images.  Used to
 * check that the relayout is a bijection.  Errors as fg_preshuffle_b, plus
 * FG_ERR_LAYOUT for a bad descriptor.
 */
FG_API fg_status fg_unshuffle_b(const fg_bshuf* desc, void* B_out, void* b_scales_out, void* stream);

/*
 * The configuration fg_gemm would use (split_k = 0 lets the dispatch table
 * choose; a positive split_k is taken as given).  Errors: INVALID_ARG, SHAPE.
 */
FG_API fg_status fg_gemm_plan(int mode, int64_t M, int64_t N, int64_t K, int split_k, fg_plan* out);

/*
 * Workspace bytes a call of fg_gemm without FG_FLAG_DEFER_REDUCE needs for
 * this shape and split: 0 when the split resolves to 1 or to at most 8 (the
 * splits of a tile then reduce inside one thread-block cluster, with no
 * global scratch), split_k*M*N*4 for larger splits, and the A scale image
 * for large-M MX shapes.  For large-M bf16 / fp8 shapes whose tiles leave a
 * partial last wave it is the optional stream-K workspace (fp32 partial
 * tiles of the CTAs that split a tile): with less, those shapes still run,
 * every tile whole.  A call with FG_FLAG_DEFER_REDUCE always needs
 * split_k*M*N*4 bytes.
 */
FG_API fg_status fg_gemm_workspace_size(int mode, int64_t M, int64_t N, int64_t K, int split_k, uint64_t* bytes);

/*
 * Y = dequant(A) . dequant(B)^T for the preshuffled weight `b`.
 *  A        device [M][K] codes (layout per mode, see top).
 *  a_scales FP8_TENSOR: device fp32 scalar; FP8_BLOCK128: fp32 [M][K/128];
 *           MXFP8: uint8 E8M0 [M][K/128]; MXFP4, MXFP8_B32, MXFP4_FP8A:
 *           uint8 E8M0 [M][K/32];
 *           BF16: ignored (pass NULL).
 *  mode     must equal b->mode (FG_ERR_LAYOUT otherwise).
 *  split_k  0 = dispatch chooses; 1..16 = number of K splits.  Split s takes
 *           the contiguous run of 128-byte K slabs [s*q + min(s,r), ...) of
 *           length q + (s < r), q = U/S, r = U%S, U = Kb/128 (for
 *           MXFP4_FP8A, U = K/128: the slabs of the fp8 A).
 *  Y        device bf16 [M][N].
 *  workspace / workspace_bytes: as fg_gemm_workspace_size says; may be
 *           NULL when that is 0.  With FG_FLAG_DEFER_REDUCE (or a split
 *           above 8) it holds fp32 [split_k][M][N], per split the partial
 *           sum: unscaled for FP8_TENSOR (the per-tensor scale is applied
 *           once, in the reduce), fully scaled for the other modes.  Splits
 *           of 2..8 without the flag sum their partials in split order
 *           inside one thread-block cluster, which gives the same bits as
 *           the workspace + fg_gemm_splitk_reduce pair.
 *  flags    FG_FLAG_DEFER_REDUCE: leave the partials in the workspace and do
 *           not write Y (call fg_gemm_splitk_reduce later).
 * Errors: INVALID_ARG, SHAPE, ALIGN, LAYOUT, WORKSPACE, UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_gemm(const void* A, const void* a_scales, int64_t M, const fg_bshuf* b, int mode, int split_k,
                  void* Y, void* workspace, uint64_t workspace_bytes, uint32_t flags, void* stream);

/*
 * Second pass of the split-K GEMM:
 *   Y[m][n] = bf16_rne( a_s * b_s * sum_{s=0}^{split_k-1} ws[s][m][n] )
 * summed in split order; a_s and b_s are device fp32 scalars (both NULL
 * means a factor of 1; exactly one NULL is an error).  Errors: INVALID_ARG,
 * SHAPE (N % 8 != 0, split_k outside 1..16), ALIGN, UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_gemm_splitk_reduce(const float* ws, int split_k, int64_t M, int64_t N, const float* a_s,
                                const float* b_s, void* Y, void* stream);

/*
 * fg_gemm without a caller workspace (no counterpart in the pages).  For
 * callers that cannot allocate device memory while they run -- a serving
 * loop whose buffers are all sized at start-up (cudaMalloc can synchronise
 * the device and stall every stream), or a plug-in whose host framework owns
 * all device memory and offers no allocator.  Whatever fg_gemm would keep in
 * a caller workspace goes to one 8 MiB array that the library keeps in every
 * device's memory until the process exits; this call allocates nothing.
 * The array holds, depending on the call:
 *  - the fp32 split-K partials of a split above 8 (splits 9..16):
 *    split_k * M * N * 4 bytes, refused with FG_ERR_WORKSPACE (before
 *    anything is launched) when above 8 MiB;
 *  - the A scale image of a large-M MX call (M > 32, MX modes):
 *    M/128 rounded up * K/128 * 512 bytes (twice that for MXFP4; a quarter,
 *    rounded up, for MXFP8), refused with FG_ERR_WORKSPACE when above 8 MiB;
 *  - the optional stream-K partials and flags of a large-M bf16 / fp8 call,
 *    when they fit (about 128 KiB per CTA for 128 x 256 tiles, 256 KiB for
 *    256 x 256 tiles; more than 8 MiB once the grid has more than 63 / 31
 *    CTAs).  When they do not fit the call is not refused: every tile then
 *    runs whole, as fg_gemm does with a smaller workspace.
 * Splits of 2..8 and split 1 need no scratch.
 *  - Arguments as fg_gemm, minus the workspace.  FG_FLAG_DEFER_REDUCE is
 *    refused (FG_ERR_INVALID_ARG): the partials would stay in the private
 *    scratch.
 *  - The first call on a device looks up the scratch's device address (once
 *    per device, with that device current); make that first call before any
 *    stream capture.
 *  - All calls share the one array and it keeps the last call's contents.
 *    Nothing in it has to start at zero (every split writes its whole
 *    partial before the reduce reads it, every large-M MX call rewrites its
 *    whole A scale image, a partial's flag matches only the launch that
 *    wrote it and is cleared once read), but two calls that overlap on the
 *    GPU (e.g. on two streams) race on it: serialise them.
 * Errors: as fg_gemm.
 */
FG_API fg_status fg_gemm_noalloc(const void* A, const void* a_scales, int64_t M, const fg_bshuf* b, int mode,
                                 int split_k, void* Y, uint32_t flags, void* stream);

/* ------------------------------------------------------------------------
 * Operators around the GEMM: activations into the A formats, and a
 * mixture-of-experts layer (routing, products grouped by expert, weighted
 * sum).  Conventions as above; no pointer may alias another unless said.
 * ------------------------------------------------------------------------ */

/*
 * Codes and scales of the A operand of `mode` from x [M][K] (or, with
 * FG_ACT_SWIGLU, from rows (g, u) of 2K values), rows ldx elements apart.
 *  mode    MXFP8, MXFP4, MXFP8_B32, MXFP4_FP8A (its activations: e4m3, 32-K
 *          blocks) or FP8_BLOCK128.
 *  codes   [M][K] e4m3, or [M][K/2] packed e2m1 for MXFP4; scales as a_scales
 *          of fg_gemm.
 * E8M0 c = 127 + ceil(log2(amax / elem_max)) clamped to 0..254 (127 for an
 * all-zero block), code = RNE(v * 2^(127-c)); FP8_BLOCK128: scale = amax / 448
 * (1 for an all-zero block; rounded to nearest, for amax < 2^-132 upwards, so
 * never 0), code = RNE(v / scale).  A block with a NaN or an infinity gets the
 * NaN scale (255; fp32 NaN) and zero codes.
 * A weight's [N][K] rows quantise the same way (FP8_BLOCK128's weights have
 * 128 x 128 blocks: fg_quantize_weight).
 * Errors: INVALID_ARG, SHAPE (K not a multiple of the block), ALIGN (x and its
 * rows 16 bytes, codes 16, fp32 scales 4), UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_quantize(int mode, int act, const void* x, int type, int64_t M, int64_t K, int64_t ldx,
                             void* codes, void* scales, void* stream);

/*
 * h = x + residual (x alone when residual is NULL),
 * y = h / sqrt(mean(h^2) + eps) * weight, all in 32 bits; residual_out = h and
 * y rounded once to the type (each only if not NULL), and y's codes and scales
 * as fg_quantize gives them (from the unrounded y).  x and residual: rows ldx
 * and ldr elements apart; weight [K]; outputs contiguous.  mode FG_BF16: no
 * codes and scales (both NULL), y required.  residual_out may be residual, and
 * residual_out or y may be x, where that has contiguous rows.
 * Errors as fg_quantize (K at most 32768; a multiple of 8 for FG_BF16).
 */
FG_API fg_status fg_rmsnorm_quantize(int mode, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                     const void* weight, float eps, int type, int64_t M, int64_t K,
                                     void* residual_out, void* y, void* codes, void* scales, void* stream);

/* Workspace of fg_moe_route: 0 for up to 64 tokens, else the blocks' counts. */
FG_API fg_status fg_moe_route_workspace_size(int64_t T, int E, uint64_t* bytes);

/*
 * Routing of T tokens to top_k of E experts (E <= 1024, top_k <= 32) by their
 * logits (rows ldl elements apart).  Per token the top_k largest logits, the
 * lowest expert first among equals; NaN counts as -infinity, and -infinity is
 * never picked.  weights [T][top_k] (fp32): softmax over all experts, or with
 * FG_FLAG_RENORMALIZE over the chosen ones (where the largest logit is
 * +infinity, the infinite ones share the weight).  experts [T][top_k].
 * The pairs (t, j) in stable order of their expert: offsets [E+1], expert e's
 * pairs are slots offsets[e] .. offsets[e+1]-1; rows[slot] = t, slots[t][j] =
 * the pair's slot.  Where a token has fewer than top_k logits to pick, its last
 * choices are expert -1, weight 0, slot -1, and the rows from offsets[E] on are
 * -1.  Errors: INVALID_ARG, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_moe_route(const void* logits, int type, int64_t T, int E, int64_t ldl, int top_k, uint32_t flags,
                              float* weights, int32_t* experts, int32_t* offsets, int32_t* rows, int32_t* slots,
                              void* workspace, uint64_t workspace_bytes, void* stream);

/*
 * Products grouped by expert: Y[i] = dequant(A[rows[i]]) . dequant(B_e)^T for
 * offsets[e] <= i < offsets[e+1], fp32 accumulation, bf16 Y [R][N].
 *  b        the experts' weights stacked to one [E * N][K] and preshuffled as
 *           one weight (fg_preshuffle_b; FP8_TENSOR: one b_s for all); N, the
 *           rows of one expert, a multiple of 128.
 *  A        [T][K] codes as in fg_gemm, a_scales likewise ([T] rows).
 *  rows     device int32 [R]: the row of A that row i multiplies, clamped into
 *           0..T-1; NULL: row i itself (T >= R).
 *  offsets  device int32 [E + 1], not decreasing (one that does counts as the
 *           largest before it), clamped into 0..R.  Rows of Y before offsets[0]
 *           and from offsets[E] on are not written.
 *  workspace  fg_grouped_gemm_workspace_size bytes (gather: rows given); any contents.  Calls that
 *           overlap on the GPU need a workspace each.  FP8_BLOCK128 runs with the bytes for
 *           gather = 0 too, which never fall with more rows; gathered calls of many rows an
 *           expert are slower then (and may differ in last bits, by the order of their sums).
 * All modes; E <= 1024; R, T <= 2^24.
 * Errors: INVALID_ARG, SHAPE, ALIGN, LAYOUT, WORKSPACE, UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_grouped_gemm_workspace_size(int mode, int64_t R, int E, int64_t N, int64_t K, int gather,
                                                uint64_t* bytes);
FG_API fg_status fg_grouped_gemm(const void* A, const void* a_scales, int64_t T, const int32_t* rows, int64_t R,
                                 const int32_t* offsets, int E, const fg_bshuf* b, int mode, void* Y, void* workspace,
                                 uint64_t workspace_bytes, uint32_t flags, void* stream);

/*
 * out[t] = residual[t] + sum_j weights[t][j] * Y[slots[t][j]] (bf16, 32-bit
 * sums in the order of j, rounded once; residual may be NULL).  Y [R][N]; a slot
 * outside 0..R-1 counts as no choice.  out may be residual.  top_k <= 32.
 * Errors: INVALID_ARG, SHAPE (N % 8), ALIGN, UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_moe_combine(const void* Y, int64_t R, const int32_t* slots, const float* weights,
                                const void* residual, int64_t T, int top_k, int64_t N, void* out, void* stream);

/* ------------------------------------------------------------------------
 * Training a mixture-of-experts layer in 8 bits: what its backward pass needs
 * beside the products above.  Input gradients are grouped products with the
 * transposed weight; weight gradients sum over rows, which their operands are
 * quantised along ("column operands"); activations are kept as 8-bit codes and
 * scales.  Codes and scales stand for code * scale, rounded to 32 bits.
 * ------------------------------------------------------------------------ */

/*
 * Codes and scales of E weights w [N][K] (rows ldw, weights `stride` elements
 * apart) in FP8_BLOCK128's 128 x 128 blocks, ready for fg_preshuffle_b: scale =
 * amax / 448 (as fg_quantize rounds it; 1 for an all-zero block), code = RNE(w /
 * scale); a block with a NaN or an infinity gets a NaN scale and zero codes.
 *  transpose  0: codes [E * N][K], scales [E * N/128][K/128]; else of the
 *             transposed weights: codes [E * K][N], scales [E * K/128][N/128].
 * Errors: INVALID_ARG (another mode: fg_quantize does its rows), SHAPE (N or K not
 * a multiple of 128), ALIGN (w and its rows 16 bytes), UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_quantize_weight(int mode, const void* w, int type, int E, int64_t N, int64_t K, int64_t ldw,
                                    int64_t stride, int transpose, void* codes, void* scales, void* stream);

/*
 * fg_quantize of silu(g) * u, x's rows being (g, u), and in the same pass the
 * checkpoint of the backward pass: codes and scales of the rows themselves
 * (saved [M][2K]).  mode: MXFP8, MXFP8_B32, MXFP4_FP8A (its activations) or
 * FP8_BLOCK128.  Errors as fg_quantize.
 */
FG_API fg_status fg_swiglu_checkpoint(int mode, const void* x, int type, int64_t M, int64_t K, int64_t ldx, void* codes,
                                      void* scales, void* saved, void* saved_scales, void* stream);

/*
 * Sizes of a column operand of C columns (a multiple of 128) for R rows of E
 * experts: `places` P = 128 * max(1, R / 128 + min(E, R)), at most 2^20.  Every
 * expert's rows begin a new slab of 128 places, the rest of its last slab and the
 * slabs behind the last expert hold zeros.  data and sf are the weight image and
 * the scale image of an MXFP8_B32 matrix [C][P] (see fg_bshuf): e4m3 codes and one
 * E8M0 for each column and 32 places; fg_unshuffle_b gives the plain matrix.
 */
FG_API fg_status fg_columns_size(int64_t C, int64_t R, int E, int64_t* places, uint64_t* data_bytes, uint64_t* sf_bytes);

/*
 * Column operand of x's rows: row rows[i] of x [T][C] (clamped into 0..T-1; rows
 * NULL: row i) is row i of the expert e with offsets[e] <= i < offsets[e+1]
 * (offsets as for fg_grouped_gemm; NULL with E = 1: one expert with all R rows).
 *  mode    FG_BF16: x holds values of `type`, rows ldx apart, scales NULL; else x
 *          holds e4m3 codes (ldx = C) with scales as fg_quantize gives them for
 *          MXFP8, MXFP8_B32, MXFP4_FP8A or FP8_BLOCK128.
 * Scales and codes as fg_quantize's 32-blocks, along the places.  Errors:
 * INVALID_ARG, SHAPE, ALIGN (x and its rows 16 bytes, data 128, sf 16), UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_quantize_columns(int mode, const void* x, const void* scales, int type, int64_t T, int64_t C,
                                     int64_t ldx, const int32_t* rows, int64_t R, const int32_t* offsets, int E,
                                     void* data, void* sf, fg_bshuf* desc_out, void* stream);

/*
 * Backward pass of y = silu(g) * u from the checkpoint's g and u, for the gradient
 * dy [R][K] of the experts' rows (type fp32 or bf16, rows ldd apart).  With s = 1 /
 * (1 + exp(-g)), 0 where that is under 2^-126, and w the row's routing weight (1
 * without weights), in 32 bits:
 *   dg = w dy u s (1 + g (1 - s)),  du = w dy g s,  act = g s u.
 * s comes from the fast power and reciprocal: it is within (8 + 1.3 |g|) 2^-24 of
 * itself where g is negative, within 8 * 2^-24 elsewhere; 32-bit dx and dweights
 * carry that error.
 *  codes, scales  of (dg, du) [R][2K] in `mode`, which is the checkpoint's too;
 *  dx             (dg, du) in dy's type (NULL: not wanted);
 *  dx_data .. dx_desc, act_data .. act_desc  column operands of (dg, du) (2K
 *                 columns) and of w * act (K columns) by the offsets (all NULL: none);
 *  weights, rows, slots, T, top_k  as fg_moe_route gives them (all NULL: no
 *                 weights); then dweights [T][top_k] = sum_i dy[slot][i] act[slot][i]
 *                 (0 where there is no choice), the gradient of the weights that
 *                 fg_moe_combine takes;
 *  offsets        [E + 1] (NULL with E = 1: all rows).  Rows of no expert are not
 *                 read; their codes and dx are zero, their scales 127 (fp32: 1).
 *  workspace      fg_swiglu_backward_workspace_size bytes (weighted: weights given).
 * Errors: INVALID_ARG, SHAPE (K not a multiple of the block, or of 128 with
 * columns; R / 128 + min(E, R) above 65535), ALIGN, WORKSPACE, UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_swiglu_backward_workspace_size(int64_t R, int64_t K, int weighted, uint64_t* bytes);
FG_API fg_status fg_swiglu_backward(int mode, const void* dy, int type, int64_t R, int64_t K, int64_t ldd, const void* saved,
                                    const void* saved_scales, const float* weights, const int32_t* rows,
                                    const int32_t* slots, int64_t T, int top_k, const int32_t* offsets, int E, void* codes,
                                    void* scales, void* dx, float* dweights, void* dx_data, void* dx_sf, fg_bshuf* dx_desc,
                                    void* act_data, void* act_sf, fg_bshuf* act_desc, void* workspace,
                                    uint64_t workspace_bytes, void* stream);

/*
 * Weight gradients grouped by expert: out[e][n][k] = the sum over the rows i of
 * expert e of a[i][n] * b[i][k], fp32 accumulation, for column operands a and b
 * (N and K columns) of the same offsets, R and E.  out [E][N][K] in fp32 or bf16;
 * accumulate: fp32 out is added to, by additions in memory, which may take values
 * and sums under 2^-126 for 0; after FG_ERR_TIMEOUT part of it has been added.  An
 * expert without rows has gradient 0.
 * Errors: INVALID_ARG, SHAPE (operands of another R or E), ALIGN, LAYOUT,
 * UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_grouped_wgrad(const fg_bshuf* a, const fg_bshuf* b, const int32_t* offsets, int64_t R, int E, int type,
                                  int accumulate, void* out, uint32_t flags, void* stream);

/* Workspace of fg_moe_balance_loss: 0 for few tokens, else the blocks' sums. */
FG_API fg_status fg_moe_balance_loss_workspace_size(int64_t T, int E, uint64_t* bytes);

/*
 * Balance loss of a routing: with p = softmax of a token's logits (0 where there is
 * nothing to pick; NaN counts as -infinity), T' the tokens that have something to
 * pick, counts[e] = offsets[e+1] - offsets[e] (0 where that is negative) and f_e
 * their share of all counts:
 *   probs[e] = sum_t p_te / T',  loss = coefficient * E * sum_e f_e probs[e],
 *   slopes[e] = coefficient * E * f_e / T', the loss's derivative by each p_te.
 * Errors: INVALID_ARG, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_moe_balance_loss(const void* logits, int type, int64_t T, int E, int64_t ldl, const int32_t* offsets,
                                     float coefficient, float* loss, int32_t* counts, float* probs, float* slopes,
                                     void* workspace, uint64_t workspace_bytes, void* stream);

/*
 * Gradient of the logits (out [T][E], their type) from the gradients dweights
 * [T][top_k] of the routing weights of `experts` (both as fg_moe_route orders them;
 * NULL: none; an expert outside 0..E-1, or whose logit is NaN or -infinity, is no
 * choice, whatever lies in its dweights) and the balance loss's slopes (NULL: none):
 *   out[t][e] = p_te (slopes[e] - sum_i p_ti slopes[i])
 *             + q_j (dweights[t][j] - sum_i q_i dweights[t][i])   where e = experts[t][j],
 * q being the softmax over the chosen experts with FG_FLAG_RENORMALIZE; without it
 * q_j = p_te, and the last sum is subtracted from every p_te's factor instead.
 * Errors: INVALID_ARG, SHAPE, ALIGN, UNSUPPORTED_ARCH, CUDA.
 */
FG_API fg_status fg_moe_route_backward(const void* logits, int type, int64_t T, int E, int64_t ldl, const int32_t* experts,
                                       const float* dweights, int top_k, const float* slopes, uint32_t flags, void* out,
                                       void* stream);

/*
 * Synchronises the current device and returns (and clears) the error word
 * the library's kernels write when a bounded wait runs out: FG_OK or
 * FG_ERR_TIMEOUT.  A failed synchronisation returns FG_ERR_CUDA.
 * After FG_ERR_TIMEOUT capture launches of fg_gemm anew before replaying them
 * (partials of its large-M form that were not taken stay marked as present).
 */
FG_API fg_status fg_get_error(void);

/*
 * Limit for every wait inside the kernels, in nanoseconds (default 4e9).
 * Values below 1e6 (1 ms) are raised to 1 ms: a wait that gives up must not
 * end while the cluster peers' shared-memory stores it waits for (a few
 * microseconds apart) may still be on their way.
 */
FG_API void fg_set_wait_timeout_ns(uint64_t ns);

/*
 * Test hook: make the architecture check see the given compute capability
 * instead of the device's (major < 0 restores the real one).  Lets host
 * tests reach FG_ERR_UNSUPPORTED_ARCH without a second kind of GPU.
 */
FG_API void fg_debug_override_cc(int major, int minor);

#ifdef __cplusplus
}
#endif

#endif /* FG_H */
