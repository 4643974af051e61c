/*
 * mega_moe.h -- C ABI of the MegaMoE expert layer for AMD Instinct MI355X (gfx950).
 *
 * One call computes, on one GPU, the forward of a mixture-of-experts FFN layer:
 *
 *   1. dispatch   every (token t, top-k slot j) pair with expert id e in [0, E)
 *                 joins expert e's pool; rows of a pool keep row-major (t, j) order.
 *                 (Research report "MegaMoE on SM100/SM90", section 3.1, dispatch
 *                 role; design page "MegaMoE SM90 Implementation Design",
 *                 section 9.2, source metadata {rank, token, topk}.)
 *   2. L1 GEMM    acc = sum_kb sx[t,kb] * sw1[e,n,kb] * sum_{k in kb} x[t,k] w1[e,n,k]
 *                 over n in [0, 2I)  (design page section 5.3, scale application;
 *                 section 15.2, weight-scale layout).
 *   3. SwiGLU     v = clamp(silu(acc[:, :I]) * acc[:, I:]) * topk_w[t, j]
 *                 then per group of G channels: float scale amax/448 (G = 128) or
 *                 UE8M0 scale (G = 32) and an E4M3 cast  (design page section 10.1).
 *   4. L2 GEMM    o = the same block-scaled product of the re-quantised
 *                 intermediate with w2, cast to BF16 per (token, slot) row
 *                 (design page section 11.1).
 *   5. combine    y[t] = bf16( sum_j f32(slot row (t, j)) ), ascending j, float32
 *                 accumulation (design page section 11.2).
 *
 * Recipes:
 *   MEGA_MOE_RECIPE_FP8_B128   x, w1, w2 and the intermediate are OCP E4M3FN bytes;
 *                              float32 scales: x per (token, 128 channels), weights
 *                              per 128x128 block, intermediate per (row, 128 channels).
 *                              (The SM90 FP8 path of the design page, section 1.1.)
 *   MEGA_MOE_RECIPE_MXFP4W_B32 x and the intermediate are E4M3FN with a UE8M0 scale per
 *                              32 channels; w1, w2 are E2M1 nibbles (two per byte, low
 *                              nibble = even K index) with a UE8M0 scale per (row, 32 K).
 *                              (PR #411 "SM90 FP8 x MXFP4 MegaMoE"; UE8M0 = 2^(code-127).)
 *   MEGA_MOE_RECIPE_MXFP8_B32  as MXFP4W_B32, but w1, w2 are E4M3FN bytes (one per K index) with a
 *                              UE8M0 scale per (row, 32 K): FP8 activations and weights with the
 *                              SM100 scale format, packed UE8M0 per 32 K for activations, weights
 *                              and the intermediate (research report "MegaMoE on SM100/SM90",
 *                              section 8.4, scale-factor formats; design page section 2, the
 *                              scale-factor row of the SM100/SM90 comparison).
 *
 * Layouts (all row-major, contiguous, device memory):
 *   x        u8  [T, H]                     x_sf  f32 [T, H/128]  | u8 [T, H/32]  (per-32 recipes)
 *   topk_idx i32 [T, k]                     topk_w f32 [T, k]
 *   l1_w     u8  [E, 2I, H]  | [E, 2I, H/2] rows 0..I-1 gate, I..2I-1 up   (MXFP8: [E, 2I, H])
 *   l1_sf    f32 [E, 2I/128, H/128]         | u8 [E, 2I, H/32]            (MXFP8: as MXFP4)
 *   l2_w     u8  [E, H, I]   | [E, H, I/2]                                 (MXFP8: [E, H, I])
 *   l2_sf    f32 [E, H/128, I/128]          | u8 [E, H, I/32]             (MXFP8: as MXFP4)
 *   y        bf16 (u16 bits) [T, H]
 * Every pointer must be 16-byte aligned.  Ids < 0 in topk_idx mark masked slots; ids
 * >= E are dropped (contribute nothing) and counted in the num_invalid view.
 *
 * Ownership: the caller allocates every buffer, including the workspace.  The library
 * allocates, frees and synchronises nothing; all work is enqueued on `stream` and the
 * call returns at once.  Inputs are read only; y is fully overwritten.  The workspace
 * needs no initialisation (each call re-initialises what it uses) and stays readable
 * through mega_moe_workspace_views() until the next call that uses it.  Concurrent
 * calls need distinct workspaces.
 *
 * Errors: the functions validate their arguments synchronously and return 0 or one of
 * the negative MEGA_MOE_ERR_* codes.  Nothing is enqueued when validation fails; after
 * MEGA_MOE_ERR_HIP (a failed launch) part of the sequence may have been enqueued and y is
 * undefined.  T * k must stay below 2^30.
 */
#ifndef MEGA_MOE_H
#define MEGA_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MEGA_MOE_ABI_VERSION 1

typedef enum {
  MEGA_MOE_RECIPE_FP8_B128 = 0,
  MEGA_MOE_RECIPE_MXFP4W_B32 = 1,
  MEGA_MOE_RECIPE_MXFP8_B32 = 2
} mega_moe_recipe;

/* flags: bits 0-1 select the GEMM tile class (0 = library default, chosen per expert from
   its row count (currently the large-M class for every expert), 1 = small-M class only,
   2 = large-M class only); bit 2 is MEGA_MOE_FLAG_CLAMP_INPUTS, bit 3 MEGA_MOE_FLAG_PRECISE_SILU,
   bit 4 MEGA_MOE_FLAG_WEIGHT_SF_KMAJOR, bit 5 MEGA_MOE_FLAG_INTER_SF64, bit 6 MEGA_MOE_FLAG_FUSED,
   bit 7 MEGA_MOE_FLAG_WEIGHT_E2M1_PAIRED; other bits must be 0. */
#define MEGA_MOE_FLAG_TILE_AUTO  0u
#define MEGA_MOE_FLAG_TILE_SMALL 1u
#define MEGA_MOE_FLAG_TILE_LARGE 2u
#define MEGA_MOE_FLAG_TILE_MASK  3u
/* flags bit 2: with swiglu_clamp = c > 0, clamp the gate and up halves of the L1 result to
 * [-c, c] before SiLU and leave silu(g)*u unclamped (the activation clamp of the design page
 * "MegaMoE SM90 Implementation Design", section 10.1, step 3).  Without it, c clamps
 * silu(g)*u, the reading of the mid-size workload's "SwiGLU output clamped".  Ignored when
 * there is no clamp. */
#define MEGA_MOE_FLAG_CLAMP_INPUTS 4u
/* flags bit 3: SiLU with the device library's expf and an IEEE division (the pages' fast_math =
 * false, design page section 10.1 step 3); by default the hardware exp and reciprocal
 * instructions (fast_math = true), float32 to a few ulp. */
#define MEGA_MOE_FLAG_PRECISE_SILU 8u
/* flags bit 4 (per-32 recipes only; INVALID_ARG with MEGA_MOE_RECIPE_FP8_B128): l1_sf and l2_sf
 * are in the K-major layout that mega_moe_transform_weight_scales() writes, [E][K/128][rows]
 * 32-bit words, each the four UE8M0 codes of one row's 128-K block (K = H, rows = 2I for l1_sf;
 * K = I, rows = H for l2_sf).  Same sizes as the row-major layout; the results are identical. */
#define MEGA_MOE_FLAG_WEIGHT_SF_KMAJOR 16u
/* flags bit 7 (MEGA_MOE_RECIPE_MXFP4W_B32 only; INVALID_ARG with the other recipes): l1_w and
 * l2_w are in the row-pair layout that mega_moe_transform_weights() writes: for each pair of
 * weight rows (2q, 2q + 1) of an expert and each 128-K block kb, the 64 bytes of row 2q's block
 * followed by the 64 bytes of row 2q + 1's, so one K block of two rows is one 128-byte line
 * (offset (q * K/128 + kb) * 128 + (row % 2) * 64 within the expert).  Same sizes as the
 * row-major layout; the results are identical. */
#define MEGA_MOE_FLAG_WEIGHT_E2M1_PAIRED 128u
/* flags bit 5 (MEGA_MOE_RECIPE_FP8_B128 only; INVALID_ARG with the per-32 recipes): the SM90
 * design's per-64 intermediate scales.  The L1 epilogue re-quantises the SwiGLU output with one
 * float scale amax/448 per 64 channels instead of per 128, and the L2 GEMM sums each 128-K block
 * of w2 as two 64-K halves, each scaled by its own intermediate scale times the block's weight
 * scale (design page "MegaMoE SM90 Implementation Design", section 5.4, L2 per-64 dual-half
 * scale application; section 10.1 step 6, the per-64 scale layout).  The inter_sf view is then
 * [I/64, T*k] float32. */
#define MEGA_MOE_FLAG_INTER_SF64 32u
/* flags bit 6: the fused forward, the whole layer (dispatch, L1 GEMM + SwiGLU, L2 GEMM, combine)
 * in one persistent cooperative launch, one workgroup per compute unit (design page "MegaMoE SM90
 * Implementation Design", section 3.3, the fused kernel pipeline; section 14.3, cross-phase
 * synchronisation: the L2 GEMM of a pool tile starts as soon as every L1 slab of that tile is
 * stored, while other L1 work still runs).  Same results bit for bit as the split forward.  Every
 * expert runs in the large-M class: INVALID_ARG with MEGA_MOE_FLAG_TILE_SMALL or for a problem too
 * large for the large-M kernels' 32-bit offsets.  Fused forwards on one GPU must not overlap
 * (each needs every compute unit; cooperative launches are not run side by side).  The events of
 * mega_moe_forward_profiled are all recorded after the one launch except events[0]. */
#define MEGA_MOE_FLAG_FUSED 64u

enum {
  MEGA_MOE_OK = 0,
  MEGA_MOE_ERR_INVALID_ARG = -1,        /* a field out of range or not a multiple of 128 */
  MEGA_MOE_ERR_NULL_POINTER = -2,       /* a required pointer is NULL */
  MEGA_MOE_ERR_MISALIGNED = -3,         /* a pointer is not 16-byte aligned */
  MEGA_MOE_ERR_WORKSPACE_TOO_SMALL = -4,/* workspace_bytes < mega_moe_workspace_size() */
  MEGA_MOE_ERR_UNSUPPORTED_DEVICE = -5, /* the current device is not gfx950 */
  MEGA_MOE_ERR_HIP = -6,                /* a HIP runtime call or launch failed */
  MEGA_MOE_ERR_SCRATCH_TOO_SMALL = -7   /* mega_moe_forward_noalloc: the problem needs more workspace
                                           than the library's static scratch holds */
};

typedef struct {
  int64_t num_tokens;    /* T >= 0; T == 0 is a valid no-op */
  int32_t hidden;        /* H in (0, 16384], multiple of 128 */
  int32_t intermediate;  /* I in (0, 16384], multiple of 128 */
  int32_t num_experts;   /* E in [1, 8192]; an always-on shared expert is one more expert */
  int32_t topk;          /* k in [1, 64] columns of topk_idx / topk_w */
  int32_t recipe;        /* mega_moe_recipe */
  float swiglu_clamp;    /* 0 or +inf: no clamp; c > 0: silu(g)*u clamped to [-c, c]
                            before the top-k weight multiplies it (or, with
                            MEGA_MOE_FLAG_CLAMP_INPUTS, gate and up clamped before SiLU) */
  uint32_t flags;        /* MEGA_MOE_FLAG_* */
} mega_moe_problem;

/* Device pointers into a workspace after a forward call (for inspection and tests): the buffer
   views the pages' buffer query hands back for correctness checks of the dispatch state (research
   report "MegaMoE on SM100/SM90", section 6.4, the buffer-size query that lays out the workspace,
   pools and combine buffer and returns tensor views of them; development log of the SM90 port,
   first entry, the Phase 1 buffer query returning its views).  Every pointer lies inside the
   caller's workspace; nothing is allocated. */
typedef struct {
  const int32_t* expert_count;   /* [E]   rows per expert */
  const int32_t* expert_offset;  /* [E+1] exclusive prefix of expert_count */
  const int32_t* pool_src;       /* [T*k] pool row -> pair t*k+j (first offset[E] valid) */
  const int32_t* pair_pos;       /* [T*k] pair -> pool row, -1 when masked or invalid */
  const int32_t* num_invalid;    /* [1]   ids >= E seen in topk_idx */
  const uint8_t* inter_q;        /* [T*k, I] E4M3 intermediate per pool row */
  const void* inter_sf;          /* K-major: [I/128, T*k] f32 | [I/128, T*k, 4] u8 (the four
                                    per-32 codes of one 128 block); pool row r, block b at b*T*k+r;
                                    with MEGA_MOE_FLAG_INTER_SF64 [I/64, T*k] f32 */
  const uint16_t* slot;          /* [T*k, H] BF16 L2 output per pair (t*k+j order) */
} mega_moe_views;

/* Bytes of workspace a forward call of this problem needs: the separate sizing query of the
   pages' interface (research report "MegaMoE on SM100/SM90", section 6.4, key APIs: the buffer-size
   query; design page "MegaMoE SM90 Implementation Design", section 16.1, the SM90 entry's size
   query registered beside the forward).  The workspace holds the dispatch counts and offsets,
   the pool metadata, the GEMM tile lists, the pool-order activation scales, the E4M3 intermediate
   with its scales and the BF16 slot rows, each region 256-byte aligned.  A forward accepts any
   workspace of at least this many bytes (a >= check, not ==).
   Errors: NULL_POINTER (p or bytes_out), INVALID_ARG (a field out of range); *bytes_out is
   written only on success. */
int mega_moe_workspace_size(const mega_moe_problem* p, size_t* bytes_out);

/* The layer forward; see the top of this file for the arithmetic and the layouts.
   stream: a hipStream_t, NULL for the default stream. */
int mega_moe_forward(const mega_moe_problem* p,
                     const void* x, const void* x_sf,
                     const int32_t* topk_idx, const float* topk_w,
                     const void* l1_w, const void* l1_sf,
                     const void* l2_w, const void* l2_sf,
                     void* y, void* workspace, size_t workspace_bytes,
                     void* stream);

/* mega_moe_forward, additionally recording caller-created hipEvent_t handles on `stream` at
   the phase boundaries, for timing each kernel of the layer on the stream it runs on:
     events[0] before dispatch, [1] after dispatch (before L1), [2] after the L1 GEMM,
     [3] after the L2 GEMM, [4] after the combine.
   num_events in [0, MEGA_MOE_NUM_PHASE_EVENTS]; events beyond num_events are not recorded.
   The caller owns the events.  With T == 0 nothing is recorded. */
#define MEGA_MOE_NUM_PHASE_EVENTS 5
int mega_moe_forward_profiled(const mega_moe_problem* p,
                              const void* x, const void* x_sf,
                              const int32_t* topk_idx, const float* topk_w,
                              const void* l1_w, const void* l1_sf,
                              const void* l2_w, const void* l2_sf,
                              void* y, void* workspace, size_t workspace_bytes,
                              void* stream, void* const* events, int num_events);

/* mega_moe_forward for callers that cannot allocate device memory (code under HIP graph capture,
   tight serving loops, harnesses that forbid allocation): no workspace argument; the call uses
   the library's own static device scratch of MEGA_MOE_NOALLOC_SCRATCH_BYTES (32 MiB) per GPU,
   which each GPU the library runs on holds until the process ends.  Problems whose
   mega_moe_workspace_size exceeds it are rejected with MEGA_MOE_ERR_SCRATCH_TOO_SMALL before
   anything is enqueued (the decode shape T = 128, H = 7168, I = 2048, E = 256, k = 8 needs
   16.3 MiB; about 250 tokens fit at that shape).  The call allocates, frees and synchronises
   nothing.  Every call on one GPU shares that GPU's scratch: calls that overlap on one GPU (on
   different streams, or from several threads) race and must be ordered by the caller; the scratch
   keeps the last call's contents, and each call re-initialises everything it reads.  Same
   arguments, results and errors as mega_moe_forward otherwise (bit-identical y). */
#define MEGA_MOE_NOALLOC_SCRATCH_BYTES (32u << 20)
int mega_moe_forward_noalloc(const mega_moe_problem* p,
                             const void* x, const void* x_sf,
                             const int32_t* topk_idx, const float* topk_w,
                             const void* l1_w, const void* l1_sf,
                             const void* l2_w, const void* l2_sf,
                             void* y, void* stream);

/* mega_moe_forward that also adds each expert's received row count (its pool size: pairs
   routed to it, masked and invalid slots excluded) of this call to the caller's device array
   cumulative_expert_recv_stats[E] (int32), the per-expert receive statistics of the research
   report's and the design page's interface (`cumulative_local_expert_recv_stats`; design page
   section 10.2).  The array is never cleared by the library; NULL skips the update.  The add
   runs on `stream` after the dispatch counts are known; calls that share one array must be
   ordered on one stream (concurrent calls race on it). */
int mega_moe_forward_stats(const mega_moe_problem* p,
                           const void* x, const void* x_sf,
                           const int32_t* topk_idx, const float* topk_w,
                           const void* l1_w, const void* l1_sf,
                           const void* l2_w, const void* l2_sf,
                           void* y, void* workspace, size_t workspace_bytes,
                           int32_t* cumulative_expert_recv_stats, void* stream);

/* The per-32 recipes' weight-scale transform, run once when the weights are loaded (the pages'
   model-load weight transform re-lays the UE8M0 scale factors out for the kernels' loads: design
   page "MegaMoE SM90 Implementation Design", section 15; research report section 6.2).  Reads the
   row-major l1_sf [E, 2I, H/32] and l2_sf [E, H, I/32] codes and writes the same codes K-major
   into l1_sf_kmajor [E, H/128, 2I, 4] and l2_sf_kmajor [E, I/128, H, 4] (caller-allocated, same
   sizes, distinct from the inputs), for forward calls with MEGA_MOE_FLAG_WEIGHT_SF_KMAJOR, whose
   GEMMs then fetch one K block's scales of 64 consecutive rows as 256 contiguous bytes instead of
   64 scattered words.  Enqueued on `stream` (a hipStream_t, NULL for the default stream).
   Errors: INVALID_ARG for the FP8_B128 recipe, an invalid problem or overlapping buffers;
   NULL_POINTER; MISALIGNED (16 bytes); UNSUPPORTED_DEVICE; HIP. */
int mega_moe_transform_weight_scales(const mega_moe_problem* p, const void* l1_sf, const void* l2_sf,
                                     void* l1_sf_kmajor, void* l2_sf_kmajor, void* stream);

/* The MXFP4 recipe's weight transform, run once when the weights are loaded (the same model-load
   weight re-layout: design page "MegaMoE SM90 Implementation Design", section 15; research report
   section 6.2).  Reads the row-major E2M1 weights l1_w [E, 2I, H/2] and l2_w [E, H, I/2] bytes and
   writes them in the row-pair layout of MEGA_MOE_FLAG_WEIGHT_E2M1_PAIRED into l1_w_paired and
   l2_w_paired (caller-allocated, same sizes, distinct from the inputs): a 128-K block of an E2M1
   row is half a 128-byte line, and in this layout the GEMMs fetch whole lines (and can stream the
   weights of single-tile experts past the caches).  Enqueued on `stream` (NULL: default stream).
   Errors: INVALID_ARG for a recipe other than MXFP4W_B32, an invalid problem or overlapping
   buffers; NULL_POINTER; MISALIGNED (16 bytes); UNSUPPORTED_DEVICE; HIP. */
int mega_moe_transform_weights(const mega_moe_problem* p, const void* l1_w, const void* l2_w,
                               void* l1_w_paired, void* l2_w_paired, void* stream);

/* Fill *out with device pointers into `workspace` for problem p (the layout of
   mega_moe_workspace_size; see mega_moe_views).  The views stay valid while the workspace does and
   hold the last forward's results until the next call that uses the workspace.
   Errors: NULL_POINTER (p, workspace or out), INVALID_ARG (a field out of range). */
int mega_moe_workspace_views(const mega_moe_problem* p, const void* workspace,
                             mega_moe_views* out);

/* Diagnostic: n_tiles independent 16 x 16 block dot products over one 128-long K block, computed
   with the same matrix-core instruction, operand layout and scale encoding the grouped GEMMs use,
   so that the error of the hardware block sum against the exact sum of its products can be
   measured (it bounds how far an intermediate value, and so its E4M3 code, may lie from the
   exactly summed one; design page "MegaMoE SM90 Implementation Design", section 20.3, tolerance,
   and the development log entry of 2026-06-18 01:10 on accumulator error and E4M3 code flips).
     out[t][m][n] = sum_{k<128} A[t][m][k] * B[t][n][k] * 2^(sa[t][m][k/32]-127) * 2^(sb[t][n][k/32]-127)
   fmt 0: A, B E4M3FN bytes [n_tiles][16][128], unit scales (scale arrays ignored, may be NULL);
   fmt 1: A E2M1 nibbles [n_tiles][16][64] (low nibble = even k), B E4M3FN [n_tiles][16][128],
          UE8M0 scales sa, sb [n_tiles][16][4];
   fmt 2: A, B E4M3FN [n_tiles][16][128] with UE8M0 scales sa, sb [n_tiles][16][4].
   out: float32 [n_tiles][16][16].  Device pointers, 16-byte aligned (scales: any alignment).
   Enqueued on `stream` (a hipStream_t, NULL for the default stream).  Errors: INVALID_ARG (fmt or
   n_tiles), NULL_POINTER, MISALIGNED, UNSUPPORTED_DEVICE, HIP. */
int mega_moe_diag_mfma_block_sums(int fmt, const void* a, const void* b, const void* a_scale,
                                  const void* b_scale, float* out, int n_tiles, void* stream);

/* ------------------------------------------------------------------------------------------
 * The operators in front of the layer: what turns a model's hidden state into the inputs of
 * mega_moe_forward.  In the order of their use:
 *
 *   mega_moe_norm_quant    residual addition, RMS norm, 8-bit rows with the recipe's scales
 *                          (x and x_sf of the forward) and the BF16 rows the gate reads
 *   mega_moe_gate_logits   logits[t, e] = sum_h x[t, h] * w[e, h]
 *   mega_moe_gate_topk     scores, balance bias, expert groups, top-k, weights (topk_idx and
 *                          topk_w of the forward), always-on shared experts appended
 *
 * They need no workspace, allocate and synchronise nothing, keep nothing between calls and can be
 * captured into a HIP graph; each is one kernel launch on `stream` (a hipStream_t, NULL for the
 * default stream; the gate product: one for every 2^23 tokens), whose device has to be the current
 * one.  Pointers are device memory, 16-byte aligned unless stated.  Arguments are validated
 * synchronously, before the device is touched; num_tokens == 0 is a valid no-op.  An output overlaps
 * no input and no other output, from its first element to its last, except where stated
 * (INVALID_ARG).
 *
 * The same call gives the same results bit for bit.  A row's outputs depend on its own inputs alone.
 * Those of the norm and of the choice of experts do not depend on the row's place in the batch
 * either (num_tokens may change the last bits of topk_w); those of the gate product as stated there.
 * Errors: INVALID_ARG, NULL_POINTER, MISALIGNED, UNSUPPORTED_DEVICE, HIP. */
typedef enum {
  MEGA_MOE_DTYPE_BF16 = 0,
  MEGA_MOE_DTYPE_F32 = 1,
  MEGA_MOE_DTYPE_E4M3 = 2   /* mega_moe_sort_tokens only */
} mega_moe_dtype;
typedef enum { MEGA_MOE_SCORE_SOFTMAX = 0, MEGA_MOE_SCORE_SIGMOID = 1 } mega_moe_score;

typedef struct {
  int64_t num_tokens;      /* T in [0, 2^30) */
  int32_t hidden;          /* H in (0, 16384], multiple of 128 */
  int32_t recipe;          /* mega_moe_recipe: which scales q_sf holds */
  int32_t x_dtype;         /* mega_moe_dtype of x, residual and residual_out */
  int32_t weight_dtype;    /* mega_moe_dtype of weight */
  float eps;               /* finite, > 0 */
  uint32_t flags;          /* 0 */
  int64_t x_stride;        /* elements from one row of x to the next: 0 (= H), or >= H in whole
                              16-byte steps (a multiple of 8 for BF16, of 4 for F32), < 2^40 */
  int64_t residual_stride; /* the same for residual and residual_out */
} mega_moe_norm_problem;

/* Residual addition, RMS norm and quantisation of each row:
 *   h = x + residual              (float32; x alone where residual is NULL)
 *   residual_out = h              (rounded to x_dtype)
 *   v = h / sqrt(mean(h^2) + eps) * weight          (from the unrounded h; the mean in float64)
 *   normed = bf16(v)
 *   q, q_sf = v in 8 bits as the forward's x, x_sf of the recipe: per group of 128 columns
 *     q_sf = amax/448 (float32), q = E4M3(v / q_sf); or per group of 32 the UE8M0 code of the
 *     smallest power of two s with amax/s <= 448 (at least 2^-127; decided as if in float64), and
 *     q = E4M3(v / s).  A group whose scale is 0 (code 0 for one that is
 *     all zero) has codes 0.
 * A row with a value that is not finite (in h) has NaN normed, q and q_sf (E4M3 0x7F or 0xFF, UE8M0
 * code 255), a group with a v that is not finite has NaN q and q_sf; other rows and groups are
 * not affected.
 *   x            [T, H] x_dtype, rows x_stride apart
 *   residual     [T, H] x_dtype, rows residual_stride apart, or NULL
 *   weight       [H] weight_dtype
 *   residual_out [T, H] x_dtype, rows residual_stride apart, or NULL; may be the residual itself
 *                (in place), or x where both strides are the same
 *   normed       bf16 [T, H], or NULL
 *   q            u8 [T, H], q_sf f32 [T, H/128] | u8 [T, H/32] (per-32 recipes): both or neither
 * normed, or q and q_sf, must be given (INVALID_ARG otherwise). */
int mega_moe_norm_quant(const mega_moe_norm_problem* p, const void* x, const void* residual,
                        const void* weight, void* residual_out, void* normed, void* q, void* q_sf,
                        void* stream);

typedef struct {
  int64_t num_tokens;    /* T in [0, 2^30) */
  int32_t hidden;        /* H in (0, 16384], multiple of 128 */
  int32_t num_experts;   /* E in [1, 8192] */
  int32_t weight_dtype;  /* mega_moe_dtype of w */
  uint32_t flags;        /* 0 */
  int64_t x_stride;      /* elements from one row of x to the next: 0 (= H), or >= H and a multiple
                            of 8, at most 2^22 */
} mega_moe_gate_problem;

/* Gate product: logits[t, e] = sum_h x[t, h] * w[e, h], products exact, sums in float32.
 *   x bf16 [T, H], rows x_stride apart;  w [E, H] weight_dtype;  logits f32 [T, E]
 * Float32 weights are multiplied as they stand where there are few logits (num_tokens at most 64 and num_tokens *
 * num_experts at most 2048), otherwise as the sum of three BF16 terms, which hold every float32 of magnitude 2^-102
 * or more exactly; with them an infinity in x or w gives an infinity or NaN, and smaller weights lose their last bits.
 * The order of a logit's sum, and so its last bits, goes by num_tokens and by the row's place in the batch: a row among
 * other rows need not give the bits that it gives alone.  A value that is not finite affects only the logits of its row
 * of x or of its expert. */
int mega_moe_gate_logits(const mega_moe_gate_problem* p, const void* x, const void* w, float* logits,
                         void* stream);

/* flags of mega_moe_topk_problem: divide the chosen experts' scores by their sum + 1e-20. */
#define MEGA_MOE_FLAG_TOPK_RENORM 1u

typedef struct {
  int64_t num_tokens;     /* T >= 0, T * (topk + num_shared) below 2^30 */
  int32_t num_experts;    /* E routed experts, E >= 1, E + num_shared <= 8192 */
  int32_t topk;           /* k >= 1 experts a token, k + num_shared <= 64,
                             k <= topk_groups * E / num_groups */
  int32_t score;          /* mega_moe_score */
  int32_t logits_dtype;   /* mega_moe_dtype of logits */
  int32_t num_groups;     /* groups of E / num_groups consecutive experts, in [1, 64], divides E */
  int32_t topk_groups;    /* groups kept a token, in [1, num_groups] */
  int32_t group_top;      /* a group's value: 1: its best expert's, 2: the sum of its two best */
  int32_t num_shared;     /* S >= 0 always-on experts, ids E .. E + S - 1, in the last S columns */
  float scale;            /* finite; the routed experts' weights are multiplied by it */
  float shared_weight;    /* finite; the shared experts' weight */
  uint32_t flags;         /* MEGA_MOE_FLAG_TOPK_* */
  int64_t logits_stride;  /* elements from one row of logits to the next: 0 (= E), or >= E, < 2^40 */
} mega_moe_topk_problem;

/* Choice of experts.  For each row of logits l:
 *   s_e = softmax(l)_e or sigmoid(l_e);  c_e = s_e + bias_e, or s_e where bias is NULL
 *   a group's value is the largest c_e in it, or the sum of its two largest (of one where it has no
 *   second candidate); the topk_groups best groups are kept
 *   the k experts with the largest c_e in these groups, in descending order, go to topk_idx[t, 0..k)
 *   w_e = s_e (without the bias), divided by the sum over the chosen + 1e-20 with
 *   MEGA_MOE_FLAG_TOPK_RENORM, times scale, go to topk_w
 *   (in float64, rounded once to float32; up to 512 experts the softmax's sum is good to 2^-19 of itself, which
 *   counts without the renormalisation, or where the chosen hold so little of it that 1e-20 does)
 * Order is decided as if c were computed in float64, without a bias in the order of l itself; of
 * equal ones the lowest id (group) comes first.  A logit that is NaN or -inf counts in no softmax and its
 * expert is never chosen; nor is one whose bias is NaN or -inf.  Experts with a logit of +inf share
 * the whole softmax.  Where there are fewer than k experts to choose, the columns left have id -1
 * and weight 0.
 *   logits     [T, E] logits_dtype, rows logits_stride apart
 *   bias       f32 [E] or NULL
 *   topk_idx   i32 [T, k + S], topk_w f32 [T, k + S]
 *   num_valid  i32 [1] in device memory (4-byte aligned) or NULL: rows from *num_valid on (the padding
 *              of a captured batch) get ids -1 and weights 0, the shared columns too; their logits are
 *              not looked at */
int mega_moe_gate_topk(const mega_moe_topk_problem* p, const void* logits, const float* bias,
                       const int32_t* num_valid, int32_t* topk_idx, float* topk_w, void* stream);

/* ------------------------------------------------------------------------------------------
 * The layer in parts: what mega_moe_forward does in one call, as operators of its own, for what the
 * one call does not do: other activations or adapters between the two products, dense 8-bit layers,
 * and the gradients of what stands between the router and the experts (the experts' 8-bit weights
 * themselves are held fixed).  In the order of their use:
 *
 *   mega_moe_sort_tokens     each routed pair's row to its expert's place, with the plan
 *   mega_moe_block_product   y = x w^T in 8 bits with a scale for each block of 128, by expert or dense
 *   mega_moe_act_quant       activation, 8-bit rows with the recipe's scales: the next product's x
 *   mega_moe_unsort_tokens   weighted sum of each token's expert rows
 *
 * and backwards:
 *
 *   mega_moe_unsort_backward   gradients of the rows and of the weights
 *   mega_moe_act_backward      gradient of the activation
 *   mega_moe_block_product     gradient of x: the product of the 8-bit gradient (mega_moe_act_quant with
 *                              MEGA_MOE_ACT_NONE) with the transposed weights
 *   mega_moe_unsort_tokens     gradient of the sort: without weights
 *
 * As for the operators in front of the layer, they allocate and synchronise nothing, keep nothing
 * between calls, can be captured into a HIP graph, run on `stream`, whose device has to be the current
 * one, and validate their arguments synchronously, before the device is touched.  Pointers are device
 * memory, 16-byte aligned unless stated.  An output overlaps no input and no other output, from its
 * first element to its last, except where stated (INVALID_ARG).  The same call gives the same results
 * bit for bit.
 * Errors: INVALID_ARG, NULL_POINTER, MISALIGNED, WORKSPACE_TOO_SMALL, UNSUPPORTED_DEVICE, HIP. */
typedef struct {
  int64_t num_tokens;    /* T >= 0, T * topk below 2^30 */
  int32_t hidden;        /* H in (0, 16384], multiple of 128 */
  int32_t num_experts;   /* E in [1, 8192] */
  int32_t topk;          /* k in [1, 64] */
  int32_t dtype;         /* mega_moe_dtype of x and rows */
  int32_t recipe;        /* mega_moe_recipe: which scales go with rows in MEGA_MOE_DTYPE_E4M3 */
  uint32_t flags;        /* 0 */
  int64_t x_stride;      /* elements from one row of x to the next: 0 (= H), or >= H in whole 16-byte steps,
                            < 2^40 */
} mega_moe_sort_problem;

/* Bytes of workspace a mega_moe_sort_tokens call of this problem needs; 0 for small batches.
   Errors: NULL_POINTER, INVALID_ARG; *bytes_out is written only on success. */
int mega_moe_sort_workspace_size(const mega_moe_sort_problem* p, size_t* bytes_out);

/* Tokens sorted by expert.  The pairs t*k + j with an id in [0, E) take places in the order of their
 * ids, pairs of one expert in their own order; other ids have no place.  n of them have one:
 *   expert_offset[e] = pairs with an id below e   (expert_offset[E] = n)
 *   pool_src[r] = the pair at place r;  pair_pos[t*k + j] = its place, or -1
 *   rows[r] = x[pool_src[r] / k],  rows_sf[r] = x_sf[pool_src[r] / k]
 * the dispatch of mega_moe_forward (its views have the same names).  Places from n on are left as they
 * were in pool_src, rows and rows_sf.  With num_tokens == 0, expert_offset is zeroed and nothing else is
 * looked at.  Its gradient: mega_moe_unsort_tokens of the rows' gradients without weights.
 *   x         [T, H] dtype, rows x_stride apart, or NULL with rows NULL: the plan alone
 *   x_sf      f32 [T, H/128] | u8 [T, H/32] (per-32 recipes) with MEGA_MOE_DTYPE_E4M3, otherwise NULL
 *   topk_idx  i32 [T, k]
 *   rows      [T*k, H] dtype;  rows_sf [T*k, H/128] | [T*k, H/32] as x_sf
 *   pool_src  i32 [T*k];  pair_pos i32 [T, k];  expert_offset i32 [E + 1]
 *   workspace of mega_moe_sort_workspace_size() bytes (NULL where that is 0), used by no other call at the
 *             same time; it needs no initialisation */
int mega_moe_sort_tokens(const mega_moe_sort_problem* p, const void* x, const void* x_sf, const int32_t* topk_idx,
                         void* rows, void* rows_sf, int32_t* pool_src, int32_t* pair_pos, int32_t* expert_offset,
                         void* workspace, size_t workspace_bytes, void* stream);

typedef struct {
  int64_t num_tokens;    /* T >= 0, T * topk below 2^30 */
  int64_t num_rows;      /* rows of `rows` and d_rows: 0 (= T * topk), or up to 2^30 */
  int32_t hidden;        /* H in (0, 16384], multiple of 128 */
  int32_t topk;          /* k in [1, 64] */
  int32_t dtype;         /* BF16 or F32: rows and y (dy, d_rows) */
  uint32_t flags;        /* 0 */
  int64_t stride;        /* elements from one row of y (dy) to the next: 0 (= H), or >= H in whole 16-byte
                            steps, < 2^40 */
} mega_moe_unsort_problem;

/* Expert rows back in token order:
 *   y[t] = sum_j topk_w[t, j] * rows[pair_pos[t, j]]
 * in float32, ascending j, rounded once.  Pairs whose pair_pos is not in [0, num_rows) contribute
 * nothing (their weight and any row without a pair are not looked at); a token without pairs gives 0.
 *   rows [num_rows, H] dtype;  pair_pos i32 [T, k];  topk_w f32 [T, k], or NULL: 1
 *   y    [T, H] dtype, rows `stride` apart */
int mega_moe_unsort_tokens(const mega_moe_unsort_problem* p, const void* rows, const int32_t* pair_pos,
                           const float* topk_w, void* y, void* stream);

/* Gradients of mega_moe_unsort_tokens, for each pair with a place r = pair_pos[t, j]:
 *   d_rows[r] = topk_w[t, j] * dy[t]               (rounded once)
 *   d_w[t, j] = sum_h rows[r, h] * dy[t, h]        (sums of 8 columns in float32, joined in float64)
 * d_w of other pairs is 0; places without a pair are left as they were in d_rows.  No two pairs share a place
 * (as mega_moe_sort_tokens makes them): of two that do, either may be left in d_rows.
 *   dy   [T, H] dtype, rows `stride` apart;  rows as above, may be NULL where d_w is
 *   d_rows [num_rows, H] dtype or NULL, may be `rows` itself;  d_w f32 [T, k] or NULL; not both NULL */
int mega_moe_unsort_backward(const mega_moe_unsort_problem* p, const void* dy, const void* rows,
                             const int32_t* pair_pos, const float* topk_w, void* d_rows, float* d_w, void* stream);

typedef struct {
  int64_t num_rows;      /* M in [0, 2^30), M * N below 2^45 */
  int32_t n;             /* N in (0, 2^20], multiple of 8: rows of each group's weights */
  int32_t k;             /* K in (0, 16384], multiple of 128 */
  int32_t num_groups;    /* G in [1, 8192] */
  uint32_t flags;        /* 0 */
  int64_t x_stride;      /* elements from one row of x to the next: 0 (= K), or >= K and a multiple of 16,
                            at most 2^22 */
  int64_t y_stride;      /* the same for y: 0 (= N), or >= N and a multiple of 8, < 2^40 */
} mega_moe_product_problem;

/* Matrix product in 8 bits with a scale for each block of 128, of each group's rows with its weights:
 *   y[m, n] = bf16( sum_b x_sf[m, b] * w_sf[g, n / 128, b] * sum_{k in block b} x[m, k] * w[g, n, k] )
 * for group_offset[g] <= m < group_offset[g + 1]: the scales and weights of MEGA_MOE_RECIPE_FP8_B128.
 * Block sums are the matrix cores' (see mega_moe_diag_mfma_block_sums), scaled and added up in float32.
 * Rows outside the groups are left as they were in y and not looked at in x.  A row's values depend on its own
 * inputs and its group's weights alone, but the order of their sums, and so their last bits, goes by the problem's
 * sizes, by the row's place in its group and by the sizes of the groups before it.
 *   x  u8 (E4M3) [M, K], rows x_stride apart;  x_sf f32 [M, K/128]
 *   w  u8 (E4M3) [G, N, K];  w_sf f32 [G, ceil(N/128), K/128]
 *   group_offset  i32 [G + 1] in device memory (4-byte aligned), ascending (expert_offset of
 *                 mega_moe_sort_tokens), or NULL with one group: every row.  Values outside [0, M] are taken as the
 *                 nearest inside.  Where they descend no memory outside the buffers is touched, but a row of two
 *                 groups gets the values of either, and groups may be left out.
 *   y  bf16 [M, N], rows y_stride apart
 * The gradient of x is the same product with y's gradient in 8 bits and the weights transposed,
 * w^T [G, K, N] with w_sf transposed alike, where N is a multiple of 128. */
int mega_moe_block_product(const mega_moe_product_problem* p, const void* x, const float* x_sf, const void* w,
                           const float* w_sf, const int32_t* group_offset, void* y, void* stream);

typedef enum { MEGA_MOE_ACT_NONE = 0, MEGA_MOE_ACT_SWIGLU = 1 } mega_moe_act;

typedef struct {
  int64_t num_rows;      /* M in [0, 2^30) */
  int32_t width;         /* I in (0, 16384], multiple of 128: columns of the result */
  int32_t act;           /* mega_moe_act */
  int32_t recipe;        /* mega_moe_recipe: which scales q_sf holds */
  int32_t x_dtype;       /* BF16 or F32: x (d_out, d_x) */
  float swiglu_clamp;    /* as in mega_moe_problem: 0 or +inf: none; only with MEGA_MOE_ACT_SWIGLU */
  uint32_t flags;        /* 0 or MEGA_MOE_FLAG_CLAMP_INPUTS */
  int64_t x_stride;      /* elements from one row of x (d_x) to the next: 0 (= its columns), or more in whole
                            16-byte steps, < 2^40 */
} mega_moe_act_problem;

/* Activation and quantisation of each row:
 *   v = x                          (MEGA_MOE_ACT_NONE, x [M, I])
 *   v = clamp(silu(g) * u)         (MEGA_MOE_ACT_SWIGLU, x [M, 2I]: g the first I columns, u the others; with
 *                                   MEGA_MOE_FLAG_CLAMP_INPUTS the clamp is on g and u instead)
 *   q, q_sf = v in 8 bits with the recipe's scales, out = bf16(v)
 * in float32 (v within 9 half steps, 2^-24 of its value each, or within 2^-141), each output rounded once; scales and codes
 * as mega_moe_norm_quant makes them, a UE8M0 code decided as if in float64.  A group with a v that is not finite has NaN q
 * and q_sf; others are not affected.
 *   x          [M, I] | [M, 2I] x_dtype, rows x_stride apart
 *   num_valid  i32 [1] in device memory (4-byte aligned) or NULL: rows from *num_valid on are not looked at, and
 *              left as they were in the outputs (expert_offset + E of mega_moe_sort_tokens, say)
 *   q          u8 [M, I], q_sf f32 [M, I/128] | u8 [M, I/32] (per-32 recipes): both or neither
 *   out        bf16 [M, I] or NULL; out, or q and q_sf, must be given (INVALID_ARG otherwise) */
int mega_moe_act_quant(const mega_moe_act_problem* p, const void* x, const int32_t* num_valid, void* q, void* q_sf,
                       void* out, void* stream);

/* Gradient of the SwiGLU (INVALID_ARG with another activation; the recipe is not looked at, the rounding to
 * 8 bits passes gradients on as they are), with s = 1 / (1 + exp(-g)):
 *   d_g = d_out * u * s * (1 + g (1 - s)),  d_u = d_out * g * s
 * both 0 where silu(g) * u lies outside [-c, c] (decided as in float64), or with MEGA_MOE_FLAG_CLAMP_INPUTS each
 * where its own input does (g and u in the formulas are then the clamped ones); in float32 (d_u within 9 half steps, d_g
 * within 18 of |d_out u s| (1 + |g (1 - s)|), or both within 2^-141), rounded once.
 *   x [M, 2I] x_dtype, rows x_stride apart;  d_out [M, I] x_dtype;  num_valid as above
 *   d_x [M, 2I] x_dtype, rows x_stride apart; may be x itself */
int mega_moe_act_backward(const mega_moe_act_problem* p, const void* x, const void* d_out, const int32_t* num_valid,
                          void* d_x, void* stream);

/* Static text for a status code. */
const char* mega_moe_strerror(int status);

/* MEGA_MOE_ABI_VERSION of the loaded library. */
int mega_moe_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MEGA_MOE_H */
