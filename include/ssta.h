/*
 * ssta.h — C ABI of the SSTA library (libssta.so) for NVIDIA B200 (sm_100a).
 *
 * Selective and Sliding Tile Attention (SSTA) is the block-sparse self-attention
 * over the 3D (latent frame x height x width) token grid of a video diffusion
 * transformer, described in "HunyuanVideo 1.5 Technical Report" (paper-graph-ui
 * summary), section "SSTA: Selective and Sliding Tile Attention", in four steps:
 *   Step 1  3D Block Partition                     -> ssta_tile_reorder
 *   Step 2  Selective Mask Generation (top-k)      -> ssta_build_block_mask
 *   Step 3  STA sliding tile window mask           -> ssta_build_block_mask
 *   Step 4  Combine masks + block-sparse attention -> ssta_build_block_mask (union,
 *                                                     compact lists) and
 *                                                     ssta_attention_fwd
 * plus ssta_tile_unorder, the inverse layout change of Step 1, ssta_attention_bwd, the
 * gradients of Step 4, and the operators around the attention in a transformer block
 * (norms, gated residuals, 8-bit activation checkpoints).
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Memory: every tensor argument is a DEVICE pointer to caller-owned, dense,
 *    row-major storage.  The library never allocates, frees or synchronises;
 *    each call only enqueues kernels on `stream` (a cudaStream_t passed as
 *    void*, NULL = the legacy default stream) and returns.
 *  - Alignment: tensor pointers must be 16-byte aligned, the workspace 256-byte
 *    aligned; otherwise SSTA_ERR_ALIGNMENT.
 *  - Errors: arguments are checked on the host before anything is launched.
 *    Launch failures return SSTA_ERR_LAUNCH.  Faults the kernels detect on the
 *    device (an out-of-range kept-tile id, a pipeline wait that exceeded its
 *    time limit, or - in the backward dK/dV kernel, whose shared-memory layout
 *    leaves under 1 KB to align its base - a dynamic shared-memory base the
 *    runtime did not place 1024-byte aligned, SSTA_ERR_ALIGNMENT) do not trap:
 *    the kernel records a code in the first 4 bytes of the workspace (an int32;
 *    0 = no error, else an ssta_status value) and returns; read it with
 *    ssta_read_device_status after the stream completes.
 *  - Calls are stateless and thread-safe; separate calls may run concurrently
 *    on different streams if their workspaces differ.
 *  - Dtypes: SSTA_BF16 (bfloat16 storage; tensor-core attention with fp32
 *    softmax and accumulation) or SSTA_F32 (fp32 storage and arithmetic).
 *
 * Layouts (B = batch, H = heads, D = head dim = 128)
 * --------------------------------------------------
 *  raster  [B, H, T, Y, X, D]     tokens of the valid latent grid.
 *  text    [B, H, L_text, D]      optional text tokens (L_text may be 0).
 *  packed  [B, H, Lq, D]          Lq = NT*N + L_text.  The grid is padded up to
 *          whole tiles (tT x tY x tX tokens, N = tT*tY*tX); video tile
 *          c = (cT*nY + cY)*nX + cX owns rows c*N .. c*N+N-1 with its tokens in
 *          raster order; pad rows are zero; text rows follow all video tiles.
 *  kv_idx  [B, H, NQ, max_kept] int32, NQ = NT + ceil(L_text/N) query tiles; row
 *          (b,h,i) lists the key tiles query tile i attends, ascending, padded
 *          with -1.  Key tiles NT.. are the text tiles.
 *  kv_cnt  [B, H, NQ] int32 number of valid entries of each kv_idx row.
 *  lse     [B, H, Lq] fp32, natural-log sum of exp of the scaled scores of a row.
 */
#ifndef SSTA_H
#define SSTA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SSTA_OK = 0,
  SSTA_ERR_INVALID_ARG = 1,    /* NULL pointer, negative or zero size, bad field */
  SSTA_ERR_UNSUPPORTED = 2,    /* well-formed but outside what the kernels implement */
  SSTA_ERR_ALIGNMENT = 3,      /* pointer not 16-byte (tensors) / 256-byte (workspace) aligned */
  SSTA_ERR_WORKSPACE = 4,      /* workspace NULL or smaller than ssta_plan's workspace_bytes */
  SSTA_ERR_LAUNCH = 5,         /* CUDA refused a launch (see cudaGetLastError) */
  SSTA_ERR_DEVICE_TIMEOUT = 6, /* device code: a pipeline wait exceeded its limit */
  SSTA_ERR_DEVICE_BOUNDS = 7   /* device code: a kept-tile id or count was out of range */
} ssta_status;

typedef enum { SSTA_BF16 = 0, SSTA_F32 = 1 } ssta_dtype;

/* Block score ranked by top-k (Step 2, "Selective Mask Generation"). */
typedef enum {
  SSTA_SCORE_SIMILARITY = 0, /* Score_s = Qbar . Kbar (raw dot product of the tile means) */
  SSTA_SCORE_IMPORTANCE = 1  /* lambda (cos(Qbar, Kbar) + 1) / 2 - (1 - lambda) * redundancy, where the
                                redundancy of key tile j is the mean over the other key tiles j' of
                                (cos(Kbar_j', Kbar_j) + 1) / 2 (0 when NT = 1); an all-zero mean has
                                cosine 0 with everything */
} ssta_score_mode;

/* How selection and window combine (Step 4). */
typedef enum {
  SSTA_COMBINE_UNION = 0,    /* selected OR in the window */
  SSTA_COMBINE_AND = 1       /* selected AND in the window (Algorithm 1 as printed) */
} ssta_combine;

/* Window at the grid edges (Step 3).  The window of tile c on an axis of n tiles
 * covers [c - w/2, c - w/2 + w) (integer w/2). */
typedef enum {
  SSTA_WINDOW_SHIFT = 0,     /* slid inward so it keeps min(w, n) tiles */
  SSTA_WINDOW_TRUNCATE = 1   /* cut at 0 and n */
} ssta_window;

/* Problem descriptor.  All fields are plain integers or floats; see the layouts
 * above.  A descriptor whose mode fields are all zero selects the similarity
 * score, the union and the shifted window. */
typedef struct {
  int B, H, D;      /* batch, heads, head dim (D must be 128) */
  int T, Y, X;      /* valid latent grid: frames, height, width (each >= 1) */
  int tT, tY, tX;   /* tile extent per axis in tokens (each >= 1) */
  int wT, wY, wX;   /* sliding window per axis, in tiles (each >= 1; odd = centred) */
  int topk;         /* key tiles selected per query tile (>= 0; clamped to NT) */
  int L_text;       /* appended text tokens (>= 0) */
  int dtype;        /* ssta_dtype */
  float scale;      /* softmax scale; 0 means 1/sqrt(D) */
  int score_mode;   /* ssta_score_mode */
  float lambda;     /* importance score: weight of the similarity term, in [0, 1] (the pages use 0.9);
                       ignored by the similarity score */
  int combine;      /* ssta_combine */
  int window_mode;  /* ssta_window */
} ssta_desc;

/* Sizes derived from a descriptor. */
typedef struct {
  int64_t packed_len;      /* Lq */
  int num_tiles;           /* NT video tiles */
  int num_text_tiles;      /* ceil(L_text / N) */
  int num_q_tiles;         /* NQ = NT + num_text_tiles */
  int tile_tokens;         /* N */
  int topk;                /* min(topk, NT) */
  int window_tiles;        /* prod over axes of min(w, n) */
  int max_kept;            /* row width of kv_idx */
  size_t workspace_bytes;  /* workspace for ssta_build_block_mask (>= 256) */
  size_t attn_workspace_bytes; /* workspace for ssta_attention_fwd (256) */
  size_t bwd_workspace_bytes;  /* workspace for ssta_attention_bwd */
} ssta_plan_info;

/*
 * ssta_plan — derive every size from `desc` (host only, no CUDA call).
 * Step 1, "3D Block Partition": NT = ceil(T/tT)*ceil(Y/tY)*ceil(X/tX).
 * max_kept = NT + num_text_tiles when L_text > 0 (text query tiles attend every
 * tile), else min(NT, topk + window_tiles).  window_tiles is the largest window
 * (with SSTA_WINDOW_TRUNCATE edge tiles keep fewer).  workspace_bytes depends on
 * score_mode (the importance score keeps per-tile norms and redundancies).
 * Returns SSTA_ERR_INVALID_ARG also for an unknown mode or lambda outside [0, 1].
 * Returns SSTA_ERR_INVALID_ARG for malformed descriptors, SSTA_ERR_UNSUPPORTED
 * when D != 128, N > 4096, NT > 2048, B*H > 65535 or Lq >= 2^31.
 */
ssta_status ssta_plan(const ssta_desc* desc, ssta_plan_info* info);

/*
 * ssta_tile_reorder — Step 1 ("3D Block Partition"): gather raster tokens into
 * the packed tile-major layout, zero the pad rows and append the text tokens.
 *   x_raster [B,H,T,Y,X,D] (read), x_text [B,H,L_text,D] (read; NULL iff
 *   L_text == 0), x_packed [B,H,Lq,D] (written in full).  Element type = dtype.
 * Exact copy.  The three buffers must not overlap.
 */
ssta_status ssta_tile_reorder(const ssta_desc* desc, const void* x_raster, const void* x_text,
                              void* x_packed, void* stream);

/*
 * ssta_build_block_mask — Steps 2-4 up to the mask: per (b, h, video tile) mean
 * of q and k over the tile's valid tokens; fp32 block scores (Step 2: Score_s =
 * Qbar Kbar^T, computed on the tensor cores with each fp32 mean split into three
 * bf16 parts and six products accumulated in fp32, or the importance score of
 * desc->score_mode, computed with fp32 FMA); per query tile the
 * top-k key tiles by score, ties to the lower tile index (Step 2,
 * Topk/Indexes2mask); combined (desc->combine: union, or AND) with the sliding
 * tile window (Step 3; desc->window_mode: slid inward at the grid edges so it
 * always spans min(w, n) tiles per axis, or truncated), and with every text tile;
 * text query tiles keep every tile (Step 4).  Writes the compact lists; a video
 * query tile can keep no tile at all (AND, no text), its count is then 0.
 *   q_packed, k_packed [B,H,Lq,D] (read; pad rows are ignored),
 *   kv_idx [B,H,NQ,max_kept] and kv_cnt [B,H,NQ] (written),
 *   tile_scores [B,H,NT,NT] fp32: the block scores top-k ranks (written when
 *   non-NULL, else kept in workspace),
 *   workspace >= info.workspace_bytes (contents overwritten).
 */
ssta_status ssta_build_block_mask(const ssta_desc* desc, const void* q_packed, const void* k_packed,
                                  int32_t* kv_idx, int32_t* kv_cnt, float* tile_scores,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * ssta_attention_fwd — Step 4 ("flex_block_attention"): for every packed query
 * row, softmax(q k^T * scale) v over the valid keys of the kept key tiles of
 * its query tile (full attention inside each kept tile; key tiles that are not
 * listed are never read).  Pad query rows are computed but carry no meaning.
 * A query tile with no valid kept key gets O = 0 and LSE = -inf.
 *   q/k/v_packed [B,H,Lq,D] (read), kv_idx/kv_cnt as written by
 *   ssta_build_block_mask (read; ids must be < NQ and ascending order is not
 *   required), o_packed [B,H,Lq,D] (written, dtype), lse [B,H,Lq] fp32
 *   (written), workspace >= info.attn_workspace_bytes (device status word).
 * bf16: tcgen05 tensor-core kernel; needs N % 128 == 0, else
 * SSTA_ERR_UNSUPPORTED (the paper's 4x8x8 tiles hold 256 tokens).
 * f32: SIMT kernel, any N.
 */
ssta_status ssta_attention_fwd(const ssta_desc* desc, const void* q_packed, const void* k_packed,
                               const void* v_packed, const int32_t* kv_idx, const int32_t* kv_cnt,
                               void* o_packed, float* lse, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * ssta_attention_bwd — gradients of ssta_attention_fwd (Step 4) for training: with
 * P = exp(q k^T * scale - LSE) over the valid keys of each query tile's kept tiles,
 * D = rowsum(dO * O) and dS = P * (dO v^T - D):
 *   dQ = scale * dS K,  dK = scale * dS^T Q,  dV = P^T dO.
 * Pad query rows take no part (dQ = 0 there); pad key rows get dK = dV = 0.
 *   q/k/v/o/do_packed [B,H,Lq,D] (read; o and lse as ssta_attention_fwd wrote them,
 *   do = dL/dO), kv_idx/kv_cnt as ssta_build_block_mask wrote them (ascending lists
 *   required), dq/dk/dv_packed [B,H,Lq,D] (written in full), all of `dtype`;
 *   workspace >= info.bwd_workspace_bytes (status word, per-row D, per-row -LSE and -D
 *   over whole tiles for the bf16 kernels, and for every key tile the list of query
 *   tiles keeping it).
 * bf16 (N % 128 == 0 required, as for ssta_attention_fwd): one tcgen05 tensor-core
 * kernel, whose blocks form dK and dV over the query tiles keeping each key tile, or dQ
 * over each query tile's kept list; P and dS enter their products rounded to bf16.
 * fp32: SIMT kernels with fp32 arithmetic.
 * Returns SSTA_ERR_UNSUPPORTED for bf16 with N % 128 != 0, SSTA_ERR_WORKSPACE for a
 * missing or short workspace, SSTA_ERR_ALIGNMENT for a workspace not 256-byte aligned
 * or a tensor not 16-byte aligned, SSTA_ERR_INVALID_ARG for a NULL tensor.
 */
ssta_status ssta_attention_bwd(const ssta_desc* desc, const void* q_packed, const void* k_packed,
                               const void* v_packed, const void* o_packed, const float* lse,
                               const void* do_packed, const int32_t* kv_idx, const int32_t* kv_cnt,
                               void* dq_packed, void* dk_packed, void* dv_packed, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * ssta_tile_unorder — inverse of ssta_tile_reorder: scatter packed rows back to
 * the raster layout, dropping pad rows, and split off the text rows.
 *   x_packed [B,H,Lq,D] (read), x_raster [B,H,T,Y,X,D] (written),
 *   x_text [B,H,L_text,D] (written; may be NULL to drop the text rows).
 */
ssta_status ssta_tile_unorder(const ssta_desc* desc, const void* x_packed, void* x_raster,
                              void* x_text, void* stream);

/*
 * ssta_build_block_mask_noalloc — the same computation and outputs as
 * ssta_build_block_mask, for callers that cannot allocate device memory at call
 * time (for instance a plugin that an inference engine hands only pre-planned
 * tensors, or a service that reserved all device memory for its own pool).  The
 * paper has no counterpart to this call; it exists for those callers only.
 *   Scratch: a device array of SSTA_STATIC_SCRATCH_BYTES built into the library,
 *   one per GPU that loads it, resident until the process exits.  It holds the
 *   workspace layout of ssta_build_block_mask: a 256-byte header, the pooled q and
 *   k means, in importance mode the inverse norms and the key sums, and the score
 *   matrix unless tile_scores is given.  Problems whose layout exceeds the array
 *   return SSTA_ERR_WORKSPACE.  The mask kernels report no device-side errors and
 *   the array's address is not exported, so this call keeps no device status word
 *   (there is nothing for ssta_read_device_status to read).
 *   The call allocates nothing.  All calls on a device share the array, so calls
 *   whose kernels overlap on the GPU race: serialise them.  The first call on a
 *   device looks up the array's device address (with that device current); make
 *   it before any stream capture.
 *   Arguments as for ssta_build_block_mask, without the workspace.
 */
#define SSTA_STATIC_SCRATCH_BYTES (32u << 20)
ssta_status ssta_build_block_mask_noalloc(const ssta_desc* desc, const void* q_packed, const void* k_packed,
                                          int32_t* kv_idx, int32_t* kv_cnt, float* tile_scores, void* stream);

/*
 * Around the attention: norms, gated residuals and 8-bit checkpoints
 * -------------------------------------------------------------------
 * What stands before and after the attention (or the MLP) of a diffusion
 * transformer block ("HunyuanVideo 1.5 Technical Report", the DiT the attention
 * runs in), and a way to keep what the backward reads in 8 bits.  These calls
 * work on rows of C channels: tokens of the residual stream, [rows, C] =
 * [B * L, H * D], or heads, [B * H * T * Y * X, D].  The conventions above hold
 * (device pointers, dense storage except the modulation's row stride, alignment,
 * no allocation, host-checked arguments); none of these calls reports device-side
 * errors, so they have no status word.
 *
 *   norm(x)   layer: (x - mean) * rstd, rstd = 1 / sqrt(mean((x - mean)^2) + eps)
 *             rms:   x * rstd,          rstd = 1 / sqrt(mean(x^2) + eps)
 *             statistics over the C channels of a row, in fp32.
 *   modulation  scale, shift, gate [G, C]: row i uses modulation row i / mod_rows,
 *             G = ceil(rows / mod_rows); mod_stride elements lie between two rows,
 *             so the chunks of one [G, 6 C] tensor serve as they are.
 *   weights   weight, post_weight [C].
 * Weights and modulation are of param_dtype; their gradients, and mean and rstd
 * [rows], are fp32.  A NULL weight counts as 1, a NULL scale or shift as 0, a
 * NULL gate as 1.
 */
typedef enum { SSTA_NORM_NONE = 0, SSTA_NORM_LAYER = 1, SSTA_NORM_RMS = 2 } ssta_norm;

typedef struct {
  int64_t rows;        /* >= 1 and < 2^31 */
  int64_t mod_rows;    /* rows sharing one modulation row; 0 = all rows */
  int64_t mod_stride;  /* elements between modulation rows; 0 = C; a multiple of 8, >= C */
  int C;               /* channels: a multiple of 8, 8 .. 8192 */
  int dtype;           /* ssta_dtype of the activations and their gradients */
  int param_dtype;     /* ssta_dtype of weights and modulation */
  int norm;            /* ssta_norm before the block (the output y or n) */
  int post_norm;       /* ssta_norm after the block (of y, before its gate) */
  float eps;           /* > 0, finite */
  float res_scale;     /* factor of the residual x, finite */
} ssta_norm_desc;

typedef struct {
  int64_t groups;               /* G */
  int exponents_per_row;        /* ceil(C / 128) */
  size_t bwd_workspace_bytes;   /* workspace for ssta_norm_bwd and ssta_residual_norm_bwd: 12 bytes per channel
                                   and run of rows, a few hundred runs, or one per group where there are more
                                   groups (mod_rows = 1: 12 bytes per element) */
} ssta_norm_plan_info;

/*
 * An activation kept in 8 bits.  128 consecutive channels of a row (fewer at its
 * end) share one exponent byte E: value = code * 2^(E - 127), with E the smallest
 * in [1, 254] that gives the group's largest magnitude a code.  Codes are rounded
 * to nearest, ties to even.  A group that holds an infinity, a NaN or a magnitude
 * whose nearest value would be 2^128 has E = 255 and all its values read as NaN.
 * Largest error of a value: half a step, 2^(E - 128) (int8), which is at most
 * max|group| / 127.5 unless E is held at 1 (max|group| below 63.75 * 2^-126); or
 * |x| * 2^-4, and 2^(E - 137) below 2^(E - 133), where the steps are equal (e4m3).
 * Every int8 value is exact in bf16, and so is every e4m3 value of a bf16 tensor; of an
 * fp32 tensor, e4m3 values with E = 1 or 2 go down to 2^-135, below bf16's smallest
 * number 2^-133, and reading them as bf16 rounds.
 */
typedef enum { SSTA_INT8 = 0, SSTA_E4M3 = 1 } ssta_code_format;
typedef struct {
  void* codes;         /* [rows, C] one byte each */
  uint8_t* exponents;  /* [rows, ceil(C / 128)] */
  int format;          /* ssta_code_format */
} ssta_checkpoint;

/*
 * ssta_norm_plan — derive sizes from `desc` (host only, no CUDA call).
 * SSTA_ERR_INVALID_ARG for malformed descriptors, SSTA_ERR_UNSUPPORTED when C is
 * no multiple of 8 or above 8192, mod_stride is no multiple of 8, or rows >= 2^31.
 */
ssta_status ssta_norm_plan(const ssta_norm_desc* desc, ssta_norm_plan_info* info);

/*
 * ssta_norm_fwd — the norm before a block, with its modulation:
 *   y = norm(x) * weight * (1 + scale) + shift.
 *   x [rows, C] (read), y [rows, C] (written; may be x), mean, rstd [rows]
 *   (written when non-NULL; mean must be NULL for the RMS norm), x_save (NULL, or
 *   a checkpoint of x to write in the same pass).
 * desc->norm must not be SSTA_NORM_NONE; post_norm and res_scale are not used (but have
 * to be valid, as in every call).
 */
ssta_status ssta_norm_fwd(const ssta_norm_desc* desc, const void* x, const void* weight, const void* scale,
                          const void* shift, void* y, float* mean, float* rstd, const ssta_checkpoint* x_save,
                          void* stream);

/*
 * ssta_norm_bwd — gradients of ssta_norm_fwd.  With xh = norm(x) from the saved
 * statistics and g = dy * weight * (1 + scale):
 *   dx = dres + rstd * (g - mean(g) - xh * mean(g * xh))   (rms: without mean(g))
 *   dshift = sum dy, dscale = sum dy * xh * weight   over the rows of each group
 *   dweight = sum dy * (1 + scale) * xh              over all rows
 *   dy [rows, C] (read), x [rows, C] or x_saved (exactly one non-NULL; read),
 *   mean (layer norm), rstd (read), dres [rows, C] (read when non-NULL: the
 *   gradient that reaches x past the block), dx [rows, C] (written; may be dy or
 *   dres), dweight [C], dscale, dshift [G, C] dense fp32 (written when non-NULL),
 *   workspace >= info.bwd_workspace_bytes (contents overwritten).
 * Sums run in a fixed order: equal inputs give equal bytes.
 */
ssta_status ssta_norm_bwd(const ssta_norm_desc* desc, const void* dy, const void* x, const ssta_checkpoint* x_saved,
                          const float* mean, const float* rstd, const void* weight, const void* scale,
                          const void* dres, void* dx, float* dweight, float* dscale, float* dshift, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * ssta_residual_norm_fwd — behind a block whose output is y: the residual with the
 * block's gate, and the norm before the next block, in one pass:
 *   h = post_norm(y) * post_weight   (post_norm none: h = y)
 *   r = res_scale * x + gate * h
 *   n = norm(r) * weight * (1 + scale) + shift   (norm none: n is not written)
 *   x, y [rows, C] (read), r [rows, C] (written; may be x), n [rows, C] (written;
 *   may be y; NULL iff norm is none), post_mean, post_rstd, mean, rstd [rows]
 *   (written when non-NULL; each must be NULL where its norm has none), y_save,
 *   r_save (NULL, or checkpoints of y and of the stored r to write in the same
 *   pass).  n and the statistics are those of r before it is rounded to dtype.
 */
ssta_status ssta_residual_norm_fwd(const ssta_norm_desc* desc, const void* x, const void* y, const void* post_weight,
                                   const void* gate, const void* weight, const void* scale, const void* shift,
                                   void* r, void* n, float* post_mean, float* post_rstd, float* mean, float* rstd,
                                   const ssta_checkpoint* y_save, const ssta_checkpoint* r_save, void* stream);

/*
 * ssta_residual_norm_bwd — gradients of ssta_residual_norm_fwd, from dr and dn, the
 * gradients of r and n (either may be NULL, not both; dn must be NULL when norm is
 * none).  With rh = norm(r), yh = post_norm(y) (none: y), g = dn * weight * (1 + scale):
 *   dR = dr + rstd * (g - mean(g) - rh * mean(g * rh)),  dx = res_scale * dR
 *   dh = dR * gate * post_weight,  dy = dh, or its gradient through post_norm
 *   dgate = sum dR * yh * post_weight, dshift, dscale as above   over each group
 *   dpost_weight = sum dR * gate * yh, dweight as above          over all rows
 *   r or r_saved (needed with dn), y or y_saved (needed for post_norm, dgate and
 *   dpost_weight): at most one of each pair, and where both r and y are given, both
 *   dense or both checkpoints of one format.  dx, dy [rows, C] (written; dx may be
 *   dr, dy may be dn), gradients of the vectors written when non-NULL
 *   (dpost_weight needs a post_norm; dweight, dscale, dshift need dn).
 */
ssta_status ssta_residual_norm_bwd(const ssta_norm_desc* desc, const void* dr, const void* dn, const void* r,
                                   const ssta_checkpoint* r_saved, const void* y, const ssta_checkpoint* y_saved,
                                   const float* post_mean, const float* post_rstd, const float* mean,
                                   const float* rstd, const void* post_weight, const void* gate, const void* weight,
                                   const void* scale, void* dx, void* dy, float* dpost_weight, float* dgate,
                                   float* dweight, float* dscale, float* dshift, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * ssta_checkpoint_save — write the checkpoint of x [rows, C] (dtype, read).
 * ssta_checkpoint_load — write the values of a checkpoint to x [rows, C] (dtype).
 * rows >= 1, C >= 8 and a multiple of 8, at most 2^36 groups (rows * ceil(C / 128)).
 */
ssta_status ssta_checkpoint_save(int64_t rows, int C, int dtype, const void* x, const ssta_checkpoint* out,
                                 void* stream);
ssta_status ssta_checkpoint_load(int64_t rows, int C, int dtype, const ssta_checkpoint* in, void* x, void* stream);

/*
 * ssta_attention_bwd_checkpoint — ssta_attention_bwd with q, k, v and O kept in 8
 * bits: checkpoints of the packed tensors ([B*H*Lq, 128], one format for all
 * four).  The formulas of ssta_attention_bwd at the checkpoints' values.  lse and O are
 * those of ssta_attention_fwd over these values of q, k and v: with the LSE of other q and
 * k (the tensors before they were rounded, say) the rows of P = exp(S - LSE) sum to
 * exp(LSE(values) - LSE), which is unbounded and grows with the logits.  workspace >= ssta_attention_bwd_checkpoint_workspace (which is
 * info.bwd_workspace_bytes and room for the values of q, k and v; status word
 * first).  Otherwise as ssta_attention_bwd.
 */
ssta_status ssta_attention_bwd_checkpoint_workspace(const ssta_desc* desc, size_t* bytes);
ssta_status ssta_attention_bwd_checkpoint(const ssta_desc* desc, const ssta_checkpoint* q, const ssta_checkpoint* k,
                                          const ssta_checkpoint* v, const ssta_checkpoint* o, const float* lse,
                                          const void* do_packed, const int32_t* kv_idx, const int32_t* kv_cnt,
                                          void* dq_packed, void* dk_packed, void* dv_packed, void* workspace,
                                          size_t workspace_bytes, void* stream);

/*
 * ssta_selftest_bounded_wait — runs the device-side bounded wait that guards every
 * pipeline wait of ssta_attention_fwd on a barrier phase that never completes
 * (complete == 0) or that completes at once (complete != 0).  The paper has no
 * counterpart; this exists to test failure handling without faulting a GPU.
 *   timeout_us in [1, 2,000,000]: the wait's limit; workspace >= 256 bytes.
 * Afterwards the workspace status word (ssta_read_device_status) holds
 * SSTA_ERR_DEVICE_TIMEOUT (never-completing phase, after about timeout_us) or 0.
 */
ssta_status ssta_selftest_bounded_wait(int32_t timeout_us, int32_t complete, void* workspace,
                                       size_t workspace_bytes, void* stream);

/*
 * ssta_read_device_status — copy the device status word (first int32 of a
 * workspace used by the calls above) to *code, synchronising `stream` first.
 * Diagnostic call: the only function of this library that synchronises.
 */
ssta_status ssta_read_device_status(const void* workspace, void* stream, int32_t* code);

/* Static, human-readable name of a status code. */
const char* ssta_status_string(ssta_status status);

#ifdef __cplusplus
}
#endif

#endif /* SSTA_H */
