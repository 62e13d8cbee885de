/*
 * mok.h — C ABI of a single-GPU, deterministic mixture-of-experts layer for GB300 (sm_103a).
 *
 * One call of the layer routes T tokens of width H to k of E experts, runs each expert
 * (a SwiGLU FFN of intermediate width I) on its tokens, and merges the k expert outputs
 * of each token with the router's gate weights.  The steps and their order follow the
 * pages on Mixture-of-Kittens (MoK):
 *   - "把 MoE 通信延迟从 103μs 压到 18μs：Cursor 开源 GPU 内核 MoK" (aientropygate.com),
 *     §02: router decision -> dispatch -> grouped GEMM -> combine; the schedule step
 *     counts each expert's tokens, places them and keeps an expert's tokens together;
 *     §03 ①: the dispatch is a pull (the expert side reads the rows it needs);
 *     §03 ③: MXFP8 activation quantisation sits on the dispatch / GEMM / SwiGLU path;
 *     §04: the measured layer ends in a weighted merge.
 *   - "Mixture-of-Kittens (MoK)" (sd114.wiki), pull-dispatch section: one schedule table
 *     serves all four transfers; benchmark section: BF16 and MXFP8, router-weight
 *     gradient computed inside the SwiGLU backward; introduction: fully deterministic.
 *   - "Cursor Open-Sources Mixture-of-Kittens (MoK) ..." (aitrending.vip),
 *     "Technical Details": the same, plus the ring token buffer.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers on the current device; the caller owns and
 *     allocates all memory (inputs, outputs, ctx, ws).  The library never allocates,
 *     frees or synchronises inside the compute calls; everything is enqueued on `stream`
 *     (a cudaStream_t passed as void*; NULL = legacy default stream).
 *   - Row-major layouts, bf16 = IEEE bfloat16 bit patterns (uint16), f32 = IEEE float.
 *   - Return values report host-side validation only (shapes, alignment, sizes) plus
 *     launch errors.  Errors found on the device (a bounded wait that ran out, an expert
 *     index out of range) go to a status word inside `ws`; read it with mok_read_status.
 *   - Outputs are overwritten, never accumulated.  Results are bitwise reproducible for
 *     the same inputs, descriptor and device: every reduction runs in a fixed order and
 *     no floating-point atomics are used.
 *   - One call at a time per `ws`: calls that may overlap on the GPU (different streams)
 *     need a `ws` each.  Besides the temporaries, `ws` holds the status word and the work
 *     counters from which the expert GEMMs and weight-gradient kernels take their tiles
 *     (cleared by each call); two overlapping calls on one `ws` would share them and skip
 *     tiles.
 *   - The descriptors carry neither their size nor a version, and grow at their ends: a caller is
 *     compiled with the header of the library that it loads, and zero-fills what it does not set
 *     (the last fields of mok_layer_desc are n_group, topk_group and group_score).
 *   - No C++ exception crosses this boundary.  No global mutable state besides per-device
 *     caches of the SM count and of how many CTA pairs of each pair kernel fit at once, the
 *     driver entry point used to encode TMA descriptors, the optional per-kernel trace
 *     (mok_trace_start / mok_trace_stop) and the fixed device scratch of
 *     mok_schedule_noalloc.  The caches are filled on first use with idempotent values.
 */
#ifndef MOK_H_
#define MOK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOK_OK = 0,
  MOK_ERR_INVALID_ARG = 1,          /* null pointer, bad shape, misaligned pointer */
  MOK_ERR_UNSUPPORTED = 2,          /* shape outside what the kernels tile (see mok_layer_desc) */
  MOK_ERR_WORKSPACE_TOO_SMALL = 3,  /* ws/ctx smaller than mok_workspace_size reports */
  MOK_ERR_CUDA = 4,                 /* a CUDA runtime/driver call or kernel launch failed */
  MOK_ERR_TIMEOUT = 5,              /* device: a bounded wait ran out (status word only) */
  MOK_ERR_INVALID_ROUTING = 6       /* device: an expert index outside [0, E) or repeated */
} mok_status;

typedef enum { MOK_ROUTER_SOFTMAX = 0, MOK_ROUTER_SIGMOID = 1 } mok_router_kind;
typedef enum { MOK_BF16 = 0, MOK_MXFP8 = 1 } mok_precision;
typedef enum { MOK_ELEM_F32 = 0, MOK_ELEM_BF16 = 1 } mok_elem_type;

/* Layer descriptor.
 *   T       tokens of this call, 1 <= T
 *   H       hidden width; multiple of 128 (MOK_ERR_UNSUPPORTED otherwise)
 *   I       expert intermediate width; multiple of 128 (MOK_ERR_UNSUPPORTED otherwise).
 *           128 is one CTA's share of a CTA pair's 256-row weight tile and the K step of
 *           the MXFP8 kernels; where H or I is an odd multiple of 128 the last pair tile
 *           reads zeros past the end and stores nothing there
 *   E       routed experts, 1 <= E <= 1024
 *   k       experts per token, 1 <= k <= min(E, 16)
 *   router  mok_router_kind: softmax over E logits, or elementwise sigmoid
 *   renorm  nonzero: the k selected gates are divided by their sum
 *   route_scale  factor on every gate (1.0 for the workloads here)
 *   precision    mok_precision of the expert GEMMs
 *   ring_bytes   0: the forward gathers all T*k rows at once.  > 0: ring forward — the
 *                gathered (dispatched) rows pass through a fixed ring of this many bytes in
 *                minibatches, gathered by comm_sms CTAs while the other SMs run GEMM1 on
 *                earlier minibatches, in one persistent launch that signals through device
 *                counters ("Mixture-of-Kittens (MoK)", sd114.wiki, ring-buffer section;
 *                aientropygate.com §03 ② and ③).  The ring must hold one minibatch.
 *   minibatch    ring forward: rows per minibatch, consecutive rows of the expert-sorted
 *                order (0 = mok_min_minibatch(0, I), two full SM waves of GEMM1 tiles)
 *   flags        MOK_FLAG_WGRAD_BF16: the expert weight gradients dw13 / dw2 of
 *                mok_moe_backward are bf16 instead of the default f32.
 *                Expert GEMM kernels.  Default: GEMM1, GEMM2 and dX_g on CTA pairs with
 *                the expert's rows as the MMA's N, padded to 16 rows (tcgen05
 *                cta_group::2, 256 weight rows per pair).  MOK_FLAG_GEMM_PAIR: GEMM1 and
 *                GEMM2 on CTA pairs with 256-row tiles of an expert's rows, dX_g on
 *                single CTAs with 128-row tiles.  MOK_FLAG_GEMM_SINGLE: all three on
 *                single CTAs with 128-row tiles.  The weight gradients run on CTA pairs
 *                (256 x 256 tiles) by default and on single CTAs (128 x 128) with either
 *                flag.  Results are bitwise the same in every case.  Setting both flags
 *                is an invalid argument.
 *                MOK_FLAG_W2_F16: mok_moe_forward reads w2 as IEEE fp16 [E][H][I] (the
 *                layer's bf16 W2 converted once with mok_convert_f16, exact for weights of
 *                magnitude 2^-14 and above), keeps a = silu(h) * u as one fp16 value (11
 *                significant bits) instead of a bf16 hi / lo pair, and runs GEMM2 on fp16
 *                operands, one MMA per K step instead of two.  Default GEMM kernels and no
 *                ring only (else MOK_ERR_UNSUPPORTED); mok_moe_backward ignores the flag and
 *                takes w2 in bf16 (the backward does not read a).
 *                MOK_FLAG_RING_PERSISTENT: the ring forward (ring_bytes > 0, default GEMM
 *                kernels, k <= 8) runs GEMM2 and the weighted merge in its persistent launch
 *                too: the CTA pairs take GEMM2 tiles of each minibatch whose GEMM1 tiles have
 *                stored their rows of a, and every CTA takes tokens of the merge once every
 *                GEMM2 tile has stored its rows of o ("把 MoE 通信延迟从 103μs 压到 18μs",
 *                aientropygate.com §03 ②: one SM group for dispatch and combine, the other
 *                for the expert FFN).  Results are bitwise those of the separate launches.
 *   comm_sms     ring forward: CTAs (one per SM) that gather rows (0 = 12); even when GEMM1
 *                runs on the narrow-segment CTA-pair kernel (the default), since those
 *                CTAs are launched in clusters of two
 *   n_group      0 or 1: the k experts are chosen among all E.  > 1: among those of the topk_group
 *                best of n_group equal groups of consecutive experts, as mok_route does it
 *                (group_score as there); a given selection is taken as it is
 *   topk_group, group_score  read where n_group > 1
 * T*k*max(H, 2I) must stay below 2^31 elements. */
#define MOK_FLAG_WGRAD_BF16 1
#define MOK_FLAG_GEMM_PAIR 2
#define MOK_FLAG_GEMM_SINGLE 4
#define MOK_FLAG_W2_F16 8
#define MOK_FLAG_RING_PERSISTENT 16
typedef struct {
  int32_t T, H, I, E, k;
  int32_t router;
  int32_t renorm;
  float route_scale;
  int32_t precision;
  int32_t minibatch;
  int64_t ring_bytes;
  int32_t flags;
  int32_t comm_sms;
  int32_t n_group, topk_group, group_score;
} mok_layer_desc;

/* Byte offsets (from the base pointer) of the tensors inside ctx and ws.  ctx holds what
 * the forward saves for the backward; ws holds temporaries.  An offset of -1 means the
 * tensor is absent for this descriptor.  Every offset is a multiple of 256. */
typedef struct {
  /* ctx */
  int64_t topk_idx;   /* i32 [T][k]   selected experts, best first (ties -> lower index) */
  int64_t gates;      /* f32 [T][k]   gate weights */
  int64_t scores;     /* f32 [T][E]   router scores (softmax probabilities or sigmoids) */
  int64_t counts;     /* i32 [E]      rows per expert */
  int64_t offsets;    /* i32 [E+1]    exclusive prefix sum of counts */
  int64_t row_of;     /* i32 [T*k]    sorted row of assignment a = t*k + j */
  int64_t src_of;     /* i32 [T*k]    assignment held by sorted row r */
  int64_t tile_off;   /* i32 [E+1]    prefix sum of ceil(counts/128) (GEMM m-tiles) */
  int64_t gate_row;   /* f32 [T*k]    gate of each sorted row */
  int64_t x_g;        /* bf16 [T*k][H]  dispatched (expert-sorted) token rows */
  int64_t hu;         /* f32 [T*k][2I]  gate and up projections h | u */
  int64_t ring_stamp; /* u64 [2]      ring forward only: a count of the ring forwards on this ctx */
  int64_t ctx_bytes;
  /* ws.  "hi/lo" pairs hold v as bf16 hi = bf16(v) plus bf16 lo = bf16(v - hi), so that a
   * GEMM operand produced inside the layer keeps about 16 significant bits. */
  int64_t status;     /* i32 [64]     device status word (code, site), then per-call work counters */
  int64_t logits;     /* f32 [T][E]   router logits */
  int64_t sched;      /* i32 [ceil(T*k/1024)][E]  schedule-table scratch: per-block counts, then starts */
  int64_t act;        /* bf16 [T*k][I]  SwiGLU output a = silu(h) * u, hi part */
  int64_t act_lo;     /* bf16 [T*k][I]  lo part */
  int64_t expert_out; /* f32 [T*k][H]   expert outputs o (unweighted) */
  int64_t dy_g;       /* bf16 [T*k][H]  dispatched upstream gradient (backward) */
  int64_t dhu;        /* bf16 [T*k][2I] gradient of h | u, hi part (backward) */
  int64_t dhu_lo;     /* bf16 [T*k][2I] lo part */
  int64_t gact;       /* bf16 [T*k][I]  gate * a, operand of dW2, hi part (backward) */
  int64_t gact_lo;    /* bf16 [T*k][I]  lo part */
  int64_t dx_g;       /* f32 [T*k][H]   per-row input gradient (backward) */
  int64_t dg_part;    /* f32 [T*k][I/128] partial gate gradients per GEMM column tile (bf16: ceil(I/256) used) */
  int64_t dlogits;    /* f32 [T][E]   router logit gradient (backward) */
  /* ring forward only (-1 otherwise) */
  int64_t ring;       /* bf16 [n_mb * minibatch][H]  the dispatched rows of every minibatch: the
                          token ring is the last slots * minibatch rows, minibatch mb in slot
                          (mb + n_mb * (slots - 1)) % slots, so that the minibatches the ring still
                          holds after the forward sit at their own rows; the backward replays the
                          rest in front of them */
  int64_t mb_tables;  /* i32 [n_mb][E+1] row offsets, [n_mb][E+1] tile offsets, [n_mb] tiles,
                          [n_mb+1] tile starts (exclusive prefix of the tiles) */
  int64_t mb_counters;/* i32 [2][n_mb]  rows gathered, tile epilogues finished, per minibatch; i32
                          the GEMM1 tile counter the CTA pairs take tiles from; then (16-byte
                          aligned) u64 [2] {ctx address, ctx ring_stamp} of the forward whose rows
                          the ring holds */
  /* MXFP8 backward only (-1 otherwise): operands quantised along their GEMM's reduction
   * dimension, as exact bf16 values */
  int64_t mx_dhu_r;   /* bf16 [T*k][2I] dh | du in 32-row blocks of each expert (dW13) */
  int64_t mx_xg_r;    /* bf16 [T*k][H]  dispatched x in 32-row blocks (dW13) */
  int64_t mx_do_r;    /* bf16 [T*k][H]  gate * dY rows in 32-row blocks (dW2) */
  int64_t mx_a_r;     /* bf16 [T*k][I]  a = silu(h) * u in 32-row blocks (dW2) */
  int64_t mx_blk_off; /* i32 [E+1]      32-row blocks before each expert (forward and backward) */
  /* MXFP8 forward only (-1 otherwise): E4M3 row operands of the FP8 GEMMs in a padded row space,
   * expert e owning rows [32 mx_blk_off[e], 32 mx_blk_off[e+1]) (its rows in schedule order, then
   * zero rows); RP = 32 (ceil(T*k / 32) + E) rows, G = RP / 32 + 4 row groups.  Scales: 512-byte
   * blocks of 128 rows x 4 blocks of 32 along the row, row 32 j + l and block b at byte
   * 16 l + 4 j + b; block (g, s) holds rows 32 g .. 32 g + 127 of 128-element stage s. */
  int64_t mx_xq;      /* E4M3 [RP][H]            dispatched rows quantised along H */
  int64_t mx_xsf;     /* E8M0 [G][H/128][512]    their scale blocks */
  int64_t mx_aq;      /* E4M3 [RP][I]            a = silu(h) * u quantised along I */
  int64_t mx_asf;     /* E8M0 [G][I/128][512]    its scale blocks */
  /* MXFP8 backward, same padded row space */
  int64_t mx_dyq;     /* E4M3 [RP][H]            dispatched dY rows quantised along H */
  int64_t mx_dysf;    /* E8M0 [G][H/128][512]    their scale blocks */
  int64_t mx_dhuq;    /* E4M3 [RP][2I]           dh | du quantised along 2I */
  int64_t mx_dhusf;   /* E8M0 [G][2I/128][512]   its scale blocks */
  int64_t ws_bytes;
} mok_layout;

/* Fills *layout (and so the ctx and ws sizes) for a descriptor.  Host only. */
mok_status mok_get_layout(const mok_layer_desc* desc, mok_layout* layout);

/* The two sizes alone: *ws_bytes and *ctx_bytes are layout.ws_bytes and layout.ctx_bytes of
 * mok_get_layout.  Host only; MOK_ERR_INVALID_ARG for a null output, otherwise the descriptor's
 * validation status (outputs untouched on error). */
mok_status mok_workspace_size(const mok_layer_desc* desc, size_t* ws_bytes, size_t* ctx_bytes);

/* Router + schedule table (the "unified schedule table" of the pull-dispatch section of
 * "Mixture-of-Kittens (MoK)", sd114.wiki; fields and reading as in the layout above).
 *   x [T][H] bf16, w_router [E][H] bf16, router_bias f32 [E] or NULL (added to the
 *   selection score only).  given_topk i32 [T][k] or NULL: when non-NULL the selection is
 *   taken from it (each row k distinct experts in [0, E); a violation is reported as
 *   MOK_ERR_INVALID_ROUTING in the status word) and the gates are the router scores at
 *   those experts; x and w_router may then be NULL only if gates are not needed (pass
 *   gates = NULL too).
 *   Outputs (i32 unless noted): topk_idx [T][k], gates f32 [T][k] (nullable), counts [E],
 *   offsets [E+1], row_of [T*k], src_of [T*k].  ws: at least layout.ws_bytes.
 * The table is exact integer work: rows of an expert are in ascending assignment order. */
mok_status mok_schedule(const mok_layer_desc* desc, const void* x, const void* w_router,
                        const float* router_bias, const int32_t* given_topk, int32_t* topk_idx,
                        float* gates, int32_t* counts, int32_t* offsets, int32_t* row_of,
                        int32_t* src_of, void* ws, size_t ws_bytes, void* stream);

/* mok_schedule without a workspace (the pages have no counterpart of this entry point).
 * For callers that cannot allocate device memory when they route tokens: code running under
 * an allocator that forbids new allocations (a step whose memory plan is fixed), a runtime
 * that only hands out its own pre-sized buffers, or a plain C caller without a CUDA
 * allocator.  Same arguments, outputs and results as mok_schedule, minus ws / ws_bytes; the
 * scratch (status word and router logits) is one array compiled into the library:
 * MOK_NOALLOC_MAX_LOGITS floats plus 256 bytes (about 4 MiB), held in the memory of every
 * GPU that loads the library until the process exits.
 *   - Rejects T * E > MOK_NOALLOC_MAX_LOGITS with MOK_ERR_WORKSPACE_TOO_SMALL when the router
 *     runs (x and w_router given); the given_topk-only path has no size limit beyond
 *     mok_layer_desc's.
 *   - device_status: NULL, or a DEVICE buffer of 2 int32 that receives (code, site) of the
 *     first device-side error of this call, as mok_read_status would report it.
 *   - The first call on a device looks up the array's device address (cudaGetSymbolAddress,
 *     with that device current); make that first call before any stream capture.
 *   - Every call on a device shares the array and it keeps the last call's contents (the
 *     status word is cleared at the start of each call).  Calls whose work overlaps on the
 *     GPU (other streams, other host threads) race on it: order them.
 *   - Allocates nothing: no cudaMalloc, cudaFree or allocating library routine. */
#define MOK_NOALLOC_MAX_LOGITS (1 << 20)
mok_status mok_schedule_noalloc(const mok_layer_desc* desc, const void* x, const void* w_router,
                                const float* router_bias, const int32_t* given_topk, int32_t* topk_idx,
                                float* gates, int32_t* counts, int32_t* offsets, int32_t* row_of,
                                int32_t* src_of, int32_t* device_status, void* stream);

/* Layer forward: y [T][H] bf16 = sum over the k selected experts of gate * SwiGLU-FFN(x).
 *   w13 [E][2I][H] bf16 (rows 0..I-1 gate projection, I..2I-1 up projection),
 *   w2 [E][H][I] bf16, router_bias and given_topk as in mok_schedule.
 *   ctx (layout.ctx_bytes) receives what the backward needs; ws (layout.ws_bytes) is
 *   scratch and also holds the status word.  Pointers to x, weights, y, ctx and ws must be
 *   16-byte aligned (TMA).  MXFP8 is not accepted here (MOK_ERR_UNSUPPORTED).
 *   With ring_bytes > 0 the dispatched rows live only in the ring (ctx x_g is not written) and y
 *   is bitwise the same as without the ring.  The ring-based backward (mok_moe_backward on the
 *   same ctx and ws) reuses the minibatches the ring still holds and gathers again only those it
 *   overwrote ("Mixture-of-Kittens (MoK)", sd114.wiki, ring-buffer section); given another ws it
 *   gathers them all, with the same results.  The ring launch is cooperative: all of its CTAs
 *   must be resident at once (one per SM). */
mok_status mok_moe_forward(const mok_layer_desc* desc, const void* x, const void* w_router,
                           const float* router_bias, const int32_t* given_topk, const void* w13,
                           const void* w2, void* y, void* ctx, size_t ctx_bytes, void* ws,
                           size_t ws_bytes, void* stream);

/* IEEE fp16 copy of a bf16 tensor: dst [n] fp16 = src [n] bf16 rounded to nearest even (exact
 * for magnitudes 2^-14 .. 65504; smaller values become fp16 subnormals, larger ones infinities).
 * For the fp16 W2 of MOK_FLAG_W2_F16 (no counterpart on the pages: a precision choice of this
 * library for the tensor-bound GEMM2).  Device pointers, 16-byte aligned; async on `stream`. */
mok_status mok_convert_f16(const void* src, void* dst, int64_t n, void* stream);

/* MXFP8 weights for mok_moe_forward_mxfp8.  MXFP8 is one of the two precisions of the pages'
 * kernel ("Mixture-of-Kittens (MoK)", sd114.wiki, benchmark section); the format is read as OCP
 * Microscaling v1.0: E4M3 elements, one E8M0 scale per 32 consecutive elements along the GEMM's
 * reduction dimension, X = clamp(floor(log2 amax) - 8, -127, 127), elements RNE(v / 2^X)
 * saturated at +-448, scale byte X + 127.
 *   w13 [E][2I][H] bf16 -> w13_q [E][2I][H] E4M3 bytes, w13_scale [E][I/64][H/128][512] bytes
 *   w2  [E][H][I]  bf16 -> w2_q  [E][H][I]  E4M3 bytes, w2_scale  [E][H/128][I/128][512]  bytes
 * Scales come in 512-byte blocks, one per 128-row tile and 128-element stage of the reduction
 * dimension, in the order the tensor cores read them from tensor memory: row 32 j + l (of the
 * tile) and 32-element block b (of the stage) at byte 16 l + 4 j + b.  The 128-row tiles of W13
 * pair the gate rows 64 t .. 64 t + 63 (tile rows 0..63) with the up rows I + 64 t .. I + 64 t + 63
 * (tile rows 64..127): the rows one CTA of the SwiGLU GEMM multiplies.  All device pointers,
 * 16-byte aligned. */
mok_status mok_quantize_weights(const mok_layer_desc* desc, const void* w13, const void* w2, void* w13_q,
                                void* w13_scale, void* w2_q, void* w2_scale, void* stream);

/* Backward-direction MXFP8 weights for mok_moe_backward_mxfp8: each GEMM of the backward
 * quantises its operands along its own reduction dimension, so the weights are quantised again,
 * along the other axis, and stored transposed so that the reduction dimension is contiguous:
 *   w2  [E][H][I]  -> w2t_q  [E][I][H]  E4M3, quantised along H (for dA' = dY_g W2[e]),
 *                     w2t_scale [E][I/128][H/128][512]
 *   w13 [E][2I][H] -> w13t_q [E][H][2I] E4M3, quantised along 2I (for dX_g = dHU W13[e]),
 *                     w13t_scale [E][H/128][2I/128][512]
 * Scale blocks as for mok_quantize_weights (row 32 j + l of a 128-row tile and 32-element block b
 * of a 128-element stage at byte 16 l + 4 j + b).  Same rule as mok_quantize_weights.  All device
 * pointers, 16-byte aligned. */
mok_status mok_quantize_weights_backward(const mok_layer_desc* desc, const void* w13, const void* w2, void* w13t_q,
                                         void* w13t_scale, void* w2t_q, void* w2t_scale, void* stream);

/* Layer backward with MXFP8 expert GEMMs (desc->precision must be MOK_MXFP8), after
 * mok_moe_forward_mxfp8 with the same ctx.  Every expert GEMM operand is quantised in 32-element
 * blocks along that GEMM's reduction dimension: dY_g (gathered, along H) and W2 along H for dA';
 * dh|du along 2I and W13 along 2I for dX_g; for the weight gradients both operands along the
 * expert's rows (gate * dY and a for dW2, dh|du and the dispatched x for dW13), in 32-row blocks
 * that start at the expert's first row.  dA' and dX_g run on the FP8 tensor path (block-scaled MMAs
 * on the E4M3 weights of mok_quantize_weights_backward); the weight gradients multiply the exact
 * values of their quantised operands on the bf16 tensor path.  The gate gradient is <dA', a> in the
 * SwiGLU backward epilogue, with dA' the quantised product; the router backward and the reverse
 * dispatch are the bf16 path's.  Outputs and ws as for mok_moe_backward (ws layout from an MXFP8
 * descriptor). */
mok_status mok_moe_backward_mxfp8(const mok_layer_desc* desc, const void* dy, const void* x, const void* w_router,
                                  const void* w13t_q, const void* w13t_scale, const void* w2t_q, const void* w2t_scale,
                                  const void* ctx, size_t ctx_bytes, void* dx, float* dw_router, void* dw13, void* dw2,
                                  float* dgates, void* ws, size_t ws_bytes, void* stream);

/* Layer forward with MXFP8 expert GEMMs (desc->precision must be MOK_MXFP8, no ring).  As
 * mok_moe_forward, with the expert weights given as mok_quantize_weights output.  The MXFP8
 * activation quantisation sits on the data path ("把 MoE 通信延迟从 103μs 压到 18μs：Cursor 开源
 * GPU 内核 MoK", aientropygate.com, §03 ③): the gather quantises each dispatched row in
 * 32-element blocks along H and the GEMM1 epilogue quantises a = silu(h) * u along I, both into
 * E4M3 bytes and scale blocks (layout.mx_xq / mx_xsf, mx_aq / mx_asf in ws).  The expert GEMMs
 * run on the FP8 tensor path (block-scaled MMAs that apply the E8M0 scales themselves) and
 * accumulate in fp32.  The router stays in bf16.  ctx as for mok_moe_forward except that ctx x_g
 * is not written (the MXFP8 backward takes the dispatched rows from x).  The MXFP8 backward is
 * mok_moe_backward_mxfp8; mok_moe_backward returns MOK_ERR_UNSUPPORTED for an MXFP8 descriptor. */
mok_status mok_moe_forward_mxfp8(const mok_layer_desc* desc, const void* x, const void* w_router,
                                 const float* router_bias, const int32_t* given_topk, const void* w13_q,
                                 const void* w13_scale, const void* w2_q, const void* w2_scale, void* y,
                                 void* ctx, size_t ctx_bytes, void* ws, size_t ws_bytes, void* stream);

/* Layer backward for upstream gradient dy [T][H] bf16, using the ctx written by the
 * matching mok_moe_forward (same desc, inputs and weights).  Outputs:
 *   dx [T][H] bf16, dw_router [E][H] f32, dw13 [E][2I][H] and dw2 [E][H][I] in f32 (bf16
 *   with MOK_FLAG_WGRAD_BF16), dgates [T][k] f32 (nullable): gradient w.r.t. each gate.
 *   An expert that received no rows gets an all-zero weight gradient.
 * The selection is held fixed; the router bias gets no gradient.  The gate gradient
 * <dA', a> of each row is formed in the SwiGLU-backward epilogue (the router-weight
 * gradient "fused into the SwiGLU backward" of the pages' benchmark section). */
mok_status mok_moe_backward(const mok_layer_desc* desc, const void* dy, const void* x,
                            const void* w_router, const void* w13, const void* w2,
                            const void* ctx, size_t ctx_bytes, void* dx, float* dw_router,
                            void* dw13, void* dw2, float* dgates, void* ws, size_t ws_bytes,
                            void* stream);

/* ------------------------------------------------------------------ group-limited routing
 * Expert selection from router logits in hand, with what load balancing needs of it (readings: the
 * pages name a router that picks a few experts per token and no rule; this is DeepSeek-V3's, whose
 * layout they target, with its softmax predecessor).
 *   T        tokens, >= 0
 *   E        experts, 1 .. 1024;  k  experts per token, 1 .. min(16, topk_group * E / n_group)
 *   router, renorm, route_scale  as in mok_layer_desc
 *   n_group  equal groups of consecutive experts, 1 .. 32, a divisor of E
 *   topk_group   groups a token's experts come from, 1 .. n_group
 *   group_score  mok_group_score: a group's value is its best rank value, or the sum of its two best
 *   logits_type  mok_elem_type of the logits (and of their gradient)
 *   logits_stride  elements between rows, >= E (0 = E)
 *   balance_coef, bias_rate  factors of the balance loss and of the bias step
 * With s the scores, an expert's rank value is s + bias (softmax without a bias: its logit, and
 * e^(logit - max) in a sum of two, the same order without the rounding of the softmax's sum).  An
 * expert whose logit or bias is -inf (masked) or NaN ranks behind all others and counts in no group's
 * value; every other bias is added as it is, the type's lowest and largest values and +inf too.
 * The topk_group best groups stay, then the k best experts in them; ties go to the lower index. */
typedef enum { MOK_GROUP_MAX = 0, MOK_GROUP_TOP2 = 1 } mok_group_score;
typedef struct {
  int64_t T, logits_stride;
  int32_t E, k;
  int32_t router, renorm;
  float route_scale;
  int32_t n_group, topk_group, group_score;
  int32_t logits_type;
  float balance_coef, bias_rate;
  int32_t reserved; /* 0 */
} mok_route_desc;

/* logits [T][E] (device; rows logits_stride apart), bias f32 [E] or NULL (added to the rank value
 * only).  Outputs, each NULL if not wanted unless noted:
 *   topk_idx   i32 [T][k] (required): best first
 *   gates      f32 [T][k]: route_scale * s, or route_scale * s / (sum of the k selected s) with renorm
 *              (0 where that sum is 0, e.g. with every expert masked)
 *   scores     f32 [T][E]
 *   counts     i32 [E]: tokens of each expert
 *   prob_sum   f32 [E]: sum over the tokens of s / (sum of the token's s)
 *   loss       f32 [1]: balance_coef * E / (k T^2) * sum_e counts[e] * prob_sum[e]
 *   dprob      f32 [E]: the loss's derivative by prob_sum (the counts are constants), for
 *              mok_route_backward
 *   bias_next  f32 [E]: bias + bias_rate * sign(T k / E - counts), may be bias itself
 * The five from counts on need ws: at least MOK_ROUTE_WS_BYTES, 256-byte aligned, zero-filled once
 * before its first use (each call leaves it ready for the next; calls that may overlap need one
 * each); otherwise ws may be NULL.  With them T stays below 2^31.  A logit that makes a token's
 * scores NaN makes prob_sum and loss NaN. */
#define MOK_ROUTE_WS_BYTES 98560
mok_status mok_route(const mok_route_desc* desc, const void* logits, const float* bias, int32_t* topk_idx,
                     float* gates, float* scores, int32_t* counts, float* prob_sum, float* loss, float* dprob,
                     float* bias_next, void* ws, size_t ws_bytes, void* stream);

/* dlogits [T][E] (the logits' type, rows dlogits_stride apart, 0 = E) for the gates' gradient
 * dgates f32 [T][k] at the experts topk_idx i32 [T][k] (distinct) and the gradient dprob f32 [E] of
 * prob_sum; either gradient may be NULL (topk_idx too without dgates), not both.  The selection is
 * held fixed, the bias gets no gradient.  An index outside [0, E) is left out and reported as
 * (MOK_ERR_INVALID_ROUTING, site) in device_status, a DEVICE buffer of 2 int32 that the caller has
 * cleared, or NULL.
 * With the layer: mok_moe_backward's router gradient is that of its gates alone.  The balance loss's
 * gradient of the logits (dgates NULL) is added to its outputs by the caller: dw_router += dlogits^T x and
 * dx += dlogits w_router (examples/train_step.py). */
mok_status mok_route_backward(const mok_route_desc* desc, const void* logits, const int32_t* topk_idx,
                              const float* dgates, const float* dprob, void* dlogits, int64_t dlogits_stride,
                              int32_t* device_status, void* stream);

/* ------------------------------------------------------------------ optimizer step
 * The step that consumes the layer's gradients (the pages end with the backward pass; the update
 * is plain AdamW, I. Loshchilov and F. Hutter, "Decoupled Weight Decay Regularization").  Tensors
 * are given as a host array that is read before the call returns; nothing of it is kept. */
typedef enum { MOK_STATE_F32 = 0, MOK_STATE_MX8 = 1 } mok_state_type;

typedef struct {
  const void* grad;   /* n contiguous elements */
  int64_t n;          /* >= 0 */
  int32_t grad_type;  /* mok_elem_type */
  int32_t reserved;   /* 0 */
} mok_grad_tensor;

/* out[0] = the 2-norm of all gradients together, out[1] = min(1, max_norm / (out[0] + 1e-6)), the
 * factor that clips them to max_norm (> 0, may be infinite), or NaN where the norm is not finite.
 * out is f32 [2] on the device.  ws: at least MOK_GRAD_NORM_WS_BYTES, 16-byte aligned, zero-filled
 * once before its first use (each call leaves it ready for the next; calls that may overlap need one
 * each).  The squares are formed and added in f32, the blocks' sums in f64, in a fixed order; a block
 * whose squares pass f32's range is taken again in a smaller unit, so that every norm below 3.4e38 is
 * found.
 * Squares have f32's lower end: below gradients of 1e-19 they lose bits, below 2.6e-23 they are 0. */
#define MOK_GRAD_NORM_WS_BYTES 16640
mok_status mok_grad_norm(const mok_grad_tensor* tensors, int32_t count, float max_norm, float* out, void* ws,
                         size_t ws_bytes, void* stream);

/* One tensor of an AdamW step, n contiguous elements:
 *   param    f32, or bf16; with bf16, master is its f32 copy (param becomes the rounded master) or
 *            NULL (param is then rounded at random, up or down, with the mean unchanged: a step is
 *            mostly smaller than half of a bf16 spacing, and rounded to nearest would be lost; an
 *            infinity or NaN stays one).
 *            master must be NULL for an f32 param
 *   grad     f32 or bf16
 *   state_type  MOK_STATE_F32: m and v are f32 [n], v_scale and m_scale NULL.
 *               MOK_STATE_MX8: m and v are E4M3 [n] holding m and sqrt(v) in blocks of 32 elements,
 *               m_scale and v_scale [ceil(n / 32)] E8M0 bytes b standing for 2^(b - 127): the OCP
 *               Microscaling layout the layer's MXFP8 operands have.  Elements are rounded at random,
 *               with the mean unchanged; a nonzero sqrt(v) never becomes zero.  v below 2^-126
 *               counts as 0.  An m or sqrt(v) that is not finite (an infinite gradient, or one whose
 *               square is beyond f32) is kept as a NaN; the other elements of its block and the
 *               block's scale are what they would be with a zero in its place.  Scale bytes are written
 *               from 1 to 254; a block under byte 0 reads as zeros, one under byte 255 (the format's
 *               NaN) as not finite.  All-zero states: zero elements with scale bytes 0 to 254.
 *   counter  multiple of 8: element i takes the rounding bits of number counter + i.  Tensors whose
 *            ranges [counter, counter + n) do not overlap are rounded independently
 * Pointers are aligned to their element; 16-byte aligned ones are accessed in 16 bytes. */
typedef struct {
  void* param;
  float* master;
  const void* grad;
  void* m;
  void* v;
  uint8_t* m_scale;
  uint8_t* v_scale;
  int64_t n;
  uint64_t counter;
  float lr, weight_decay;
  int32_t param_type, grad_type; /* mok_elem_type */
  int32_t state_type;            /* mok_state_type */
  int32_t reserved;              /* 0 */
} mok_adamw_tensor;

/* beta1, beta2 in [0, 1), eps >= 0; step >= 1 is this step's number; seed chooses the rounding bits
 * (with the step and the element's counter; the same three give the same bits). */
typedef struct {
  double beta1, beta2, eps;
  int64_t step;
  uint32_t seed;
  uint32_t reserved; /* 0 */
} mok_adamw_hyper;

/* AdamW on every tensor, in place:
 *   g' = c * grad, c = *grad_scale (f32 on the device, NULL = 1), e.g. out + 1 of mok_grad_norm
 *   m = beta1 m + (1 - beta1) g';  v = beta2 v + (1 - beta2) g'^2
 *   param -= lr * ((m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps) + weight_decay * param)
 * in f32.  Where c is NaN nothing is changed (the host does not see it: a caller that counts on has
 * skipped that number).  The step's number and rates are in the launch: a captured graph repeats them
 * and the rounding bits at each replay. */
mok_status mok_adamw_step(const mok_adamw_tensor* tensors, int32_t count, const mok_adamw_hyper* hyper,
                          const float* grad_scale, void* stream);

/* ------------------------------------------------------------------ experts outside the layer
 * For experts that are not the layer's (another FFN, weights in 8 bits with a scale for each 128 x 128, a shared
 * expert): the layer's table (mok_schedule) moves the rows, and the products run on E4M3 operands.  The pages have
 * no counterpart: their experts are SwiGLU FFNs in BF16 or MXFP8.  Rows, and assignments, stay below 2^31, widths below
 * 2^28, groups are at most 1024 (MOK_ERR_UNSUPPORTED).  No call has a workspace: calls may overlap.
 *
 * Rows by a table.
 *   T  tokens, R  rows of the sorted order (mok_schedule: T k; fewer or more where assignments are dropped or rows
 *   padded), both >= 0;  H  width >= 1;  k  assignments of a token, 1 .. 16
 *   token_stride, row_stride  elements between tokens and between rows, >= H (0 = H)
 *   type  mok_elem_type of tokens and rows
 * src_of i32 [R]: the assignment a = t k + j in row r; row_of i32 [T k]: the row of assignment a.  -1 is an empty row
 * and an assignment without a row (dropped); any other index out of range counts as -1 and is reported as
 * (MOK_ERR_INVALID_ROUTING, site) in device_status, a DEVICE buffer of 2 int32 that the caller has cleared, or NULL.
 * gates f32 [T][k], or NULL: all 1.  Outputs do not overlap inputs. */
typedef struct {
  int64_t T, R, H;
  int64_t token_stride, row_stride;
  int32_t k, type;
} mok_rows_desc;

/* x_g[r] = gates[a] x[a / k], a = src_of[r]: every row of x_g is written, empty ones with zeros.  Its gradient with
 * respect to x is mok_merge_rows of dx_g with the same gates. */
mok_status mok_gather_rows(const mok_rows_desc* desc, const void* x, const int32_t* src_of, const float* gates,
                           void* x_g, int32_t* device_status, void* stream);

/* y[t] = sum_j gates[t][j] o[row_of[t k + j]], j ascending, in f32, rounded once; zeros for a token without rows. */
mok_status mok_merge_rows(const mok_rows_desc* desc, const void* o, const int32_t* row_of, const float* gates, void* y,
                          int32_t* device_status, void* stream);

/* d_o[row_of[t k + j]] = gates[t][j] dy[t]; dgates[t][j] = <dy[t], o[row_of[t k + j]]> (f32, NULL if not wanted), 0 for
 * an assignment without a row.  Rows of d_o that no assignment names are left as they were; a row that two name
 * holds either's. */
mok_status mok_merge_rows_backward(const mok_rows_desc* desc, const void* dy, const void* o, const int32_t* row_of,
                                   const float* gates, void* d_o, float* dgates, int32_t* device_status, void* stream);

/* E4M3 with an f32 scale for each block of 128: scale = max(amax, 2^-110) / 448 over the block's finite elements,
 * element = the E4M3 value nearest to 448 x / amax, ties to even; an element that is not finite becomes a NaN.  Rows
 * of E4M3 elements start at multiples of 16 bytes.
 *   R  rows, C  width of the quantised rows;  x_stride, grad_stride  elements between rows (0 = packed)
 *   source   MOK_FP8_PLAIN: x [R][C]; with src_of, rows gates[a] x[a / k] of x [T][C] as in mok_gather_rows
 *            (gates may be NULL; an index out of range is reported in device_status)
 *            MOK_FP8_SWIGLU: x [R][2C] = h | u; quantised is silu(h) u
 *            MOK_FP8_SWIGLU_GRAD: x [R][C] = h | u, grad [R][C/2] = da; quantised is the gradient dh | du [R][C] of
 *            a = silu(h) u
 *   type     mok_elem_type of x and grad
 * Outputs, either pair NULL if not wanted:
 *   q [R][C], scale f32 [ceil(C/128)][R]: blocks along the row (q_stride bytes, a multiple of 16, 0 = C rounded up to
 *     one; scale_stride floats, 0 = R)
 *   qt [C][P], qt_scale f32 [P/128][C], P = 128 (R / 128 + E): blocks along the rows of each of E groups (offsets i32
 *     [E+1], as of mok_schedule), transposed: group e's rows follow each other from 128 times the 128-row blocks of
 *     the groups before it, with zeros behind its last up to a multiple of 128 (qt_stride bytes, 0 = P).  Blocks
 *     behind the last group's are left as they were.  With it, q and scale too are written for the rows of the
 *     groups only.
 * Without columns E and offsets are not read.  Offsets that do not ascend within [0, R] give results that are not
 * defined; nothing outside the tensors is read or written. */
typedef enum { MOK_FP8_PLAIN = 0, MOK_FP8_SWIGLU = 1, MOK_FP8_SWIGLU_GRAD = 2 } mok_fp8_source;
typedef struct {
  int64_t R, C, T;
  int64_t x_stride, grad_stride, q_stride, scale_stride, qt_stride;
  int32_t E, k;
  int32_t source, type;
} mok_fp8_quantize_desc;
mok_status mok_fp8_quantize(const mok_fp8_quantize_desc* desc, const void* x, const void* grad, const int32_t* src_of,
                            const float* gates, const int32_t* offsets, uint8_t* q, float* scale, uint8_t* qt,
                            float* qt_scale, int32_t* device_status, void* stream);

/* Weights w [E][N][K] (contiguous) with a scale for each 128 x 128, by the same rule.  Outputs, either pair NULL if not
 * wanted: q [E][N][K] and scale f32 [E][ceil(N/128)][ceil(K/128)] for x W^T, qt [E][K][N] and qt_scale f32
 * [E][ceil(K/128)][ceil(N/128)] for dy W (the same elements and scales, transposed).  Strides in bytes between
 * elements' rows, multiples of 16 (0 = the width rounded up to one). */
typedef struct {
  int64_t N, K;
  int64_t q_stride, qt_stride;
  int32_t E, type;
} mok_fp8_weights_desc;
mok_status mok_fp8_quantize_weights(const mok_fp8_weights_desc* desc, const void* w, uint8_t* q, float* scale,
                                    uint8_t* qt, float* qt_scale, void* stream);

/* out[r][n] = sum_b x_scale[b][r] w_scale[e][n/128][b] sum_{k in block b} x[r][k] w[e][n][k] for the rows r of group e,
 * offsets[e] <= r < offsets[e+1] (as for mok_fp8_quantize; NULL with E = 1: all R rows).  x [R][K] and x_scale as q and
 * scale of mok_fp8_quantize, w [E][N][K] and w_scale as of mok_fp8_quantize_weights: q and scale for x W^T, qt and
 * qt_scale for dy W.  The sums of a block are formed by the tensor cores, the blocks are added in f32, in a fixed
 * order.  The two scales' product may leave f32's range where the result does not (a block at the least scale, 2^-110 / 448, may
 * be off by 2^-125 then).  out f32 or bf16 (out_type, rounded once), out_stride elements between rows (0 = N); rows of no group are
 * left as they were.  device_status as for mok_gather_rows; it also takes a wait that ran out (MOK_ERR_TIMEOUT). */
typedef struct {
  int64_t R, N, K;
  int64_t x_stride, x_scale_stride, w_stride, out_stride;
  int32_t E, out_type;
} mok_fp8_matmul_desc;
mok_status mok_fp8_matmul(const mok_fp8_matmul_desc* desc, const uint8_t* x, const float* x_scale, const uint8_t* w,
                          const float* w_scale, const int32_t* offsets, void* out, int32_t* device_status,
                          void* stream);

/* out[e][n][h] = sum over group e's blocks b of dy_scale[b][n] x_scale[b][h] sum_{r in b} dy[n][r] x[h][r] (a block's sum
 * meets dy_scale first, and that product has to lie within f32: any dy below 2^112; x may be as large as its type): the gradient
 * of the weights, with dy [N][P], x [H][P] and their scales as qt and qt_scale of mok_fp8_quantize for the same R, E and
 * offsets.  Zeros for a group without rows.  out f32 or bf16 [E][N][H], contiguous.  device_status (or NULL) takes a wait that
 * ran out (MOK_ERR_TIMEOUT); part of out is unwritten then, as of mok_fp8_matmul's. */
typedef struct {
  int64_t R, N, H;
  int64_t dy_stride, x_stride;
  int32_t E, out_type;
} mok_fp8_weight_grad_desc;
mok_status mok_fp8_weight_grad(const mok_fp8_weight_grad_desc* desc, const uint8_t* dy, const float* dy_scale,
                               const uint8_t* x, const float* x_scale, const int32_t* offsets, void* out,
                               int32_t* device_status, void* stream);

/* Synchronises `stream`, copies the device status word out of ws into
 * device_status[0] (code, a mok_status value) and device_status[1] (site), then clears it.
 * Host-blocking; not for use inside captured graphs. */
mok_status mok_read_status(void* ws, size_t ws_bytes, void* stream, int32_t* device_status);

/* Test hook for the bounded waits (no counterpart on the pages): launches one kernel
 * whose single thread waits on an mbarrier that nothing will complete, with the given
 * limit in milliseconds; the wait gives up, records MOK_ERR_TIMEOUT in the status word
 * of ws and the kernel returns normally.  Used to show that a stuck wait ends cleanly. */
mok_status mok_test_bounded_wait(void* ws, size_t ws_bytes, int32_t limit_ms, void* stream);

/* Per-kernel timing (tracing; no counterpart on the pages).  mok_trace_start enables it
 * for the whole process: every kernel the library launches from then on is bracketed by
 * two CUDA events recorded on the stream it is launched on, up to max_launches launches.
 * mok_trace_stop synchronises those events, sums the elapsed time per kernel name into
 * out[0..cap) (names in launch order of first appearance), stores the number of entries in
 * *n_out, frees the events and disables tracing.  Host-side state only; not thread-safe;
 * do not start it while a stream capture is active. */
typedef struct {
  char name[32];
  int32_t launches;
  float total_ms;
} mok_trace_entry;

mok_status mok_trace_start(int32_t max_launches);
mok_status mok_trace_stop(mok_trace_entry* out, int32_t cap, int32_t* n_out);

/* Human-readable name of a status code. */
const char* mok_status_string(mok_status s);

/* Number of SMs of the current device and the minimum minibatch (rows) whose expert-
 * grouped GEMM1 fills two full SM waves of 128x256 output tiles: ceil(2*n_sm*128*256/(2I)).
 * The pages state the two-wave rule and its result, 2,368 tokens, for hidden 7168 and
 * intermediate 2048 ("Mixture-of-Kittens (MoK)", sd114.wiki, overlap-granularity section;
 * aientropygate.com, §03 ②) but no formula; this is the reading that reproduces it for
 * 148 SMs.  n_sm <= 0 means: query the current device. */
int32_t mok_min_minibatch(int32_t n_sm, int32_t I);

#ifdef __cplusplus
}
#endif

#endif /* MOK_H_ */
