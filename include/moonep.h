/*
 * moonep.h -- C ABI of the balanced expert-parallel MoE layer on one MI355X (gfx950).
 *
 * R virtual expert-parallel ranks live in one GPU's HBM.  The library plans,
 * from top-K router output, how many pairs each rank processes so that every
 * rank handles exactly S*K (token, expert) pairs, then moves rows and runs the
 * expert GEMMs under that plan.
 *
 * Sources (web pages about MoonEP; a section name follows each citation):
 *   [P1] "Valhalla static engineering review #004 -- MoonshotAI MoonEP"
 *        (wsisp.com), section 2 "Project background".
 *   [P2] "Moonshot open-sources MoonEP: an expert-parallel communication
 *        library for MoE training" (umios.umi6.com), sections "Core problem",
 *        "Core technique: dynamic redundant experts", "Memory contract and
 *        weight layout".
 *   [P3] "Moonshot AI Open-Sources MoonEP for Expert Parallelism"
 *        (interestana.com), paragraphs two (maxvio) and three (S*K invariant).
 *
 * Notation ([P2] "Memory contract and weight layout"): E routed experts, E/R
 * home experts per rank (expert e lives on rank e / (E/R)), B prefetch slots
 * per rank, S tokens per rank, K experts per token, H hidden size, Hp = H'
 * FFN width.  P = S*K rows per rank, N = R*P rows in total.  Rank r sees a
 * logical [E+B, H, Hp] weight tensor: row g < E is W_home[g], row E+j is its
 * slot W_slots[r, j].
 *
 * Conventions shared by every call
 *   - All array pointers are DEVICE memory owned by the caller, dense and
 *     row-major with the shapes given.  The library never allocates, frees,
 *     copies to the host or synchronises: each call only enqueues kernels on
 *     `stream` (a hipStream_t; NULL is the null stream), so a call sequence
 *     can be captured in a HIP graph.
 *   - Shapes are static: no output size depends on the routing.
 *   - Return value: MOONEP_OK, or a negative code.  MOONEP_EINVAL (bad
 *     dimension, null pointer, misaligned pointer) and MOONEP_EUNSUPPORTED
 *     are returned before anything is enqueued.  MOONEP_EHIP means a launch
 *     failed; the device state of the outputs is then unspecified.
 *     moonep_last_error() gives a human-readable reason for the calling thread.
 *   - Device-side contract violations are never trapped: top-K ids outside
 *     [0, E) and a repeated expert within one token are counted in
 *     stats[3] by moonep_plan; other results are then unspecified (but every
 *     kernel stays inside its buffers).
 *   - Row pointers whose rows are a multiple of 16 bytes must be 16-byte
 *     aligned (checked).
 */
#ifndef MOONEP_H
#define MOONEP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct moonep_dims {
  int32_t R; /* virtual ranks, >= 1 */
  int32_t E; /* routed experts, >= 1, E % R == 0 */
  int32_t B; /* prefetch slots per rank, >= 0 (training uses E/R, inference 3-4) */
  int32_t S; /* tokens per rank, >= 0 */
  int32_t K; /* experts per token, 1 <= K <= E; R*S*K < 2^31 */
} moonep_dims;

typedef enum moonep_dtype {
  MOONEP_F32 = 0, /* float32 activations and weights */
  MOONEP_BF16 = 1 /* bfloat16 activations and weights, float32 accumulation */
} moonep_dtype;

enum {
  MOONEP_OK = 0,
  MOONEP_EINVAL = -1,
  MOONEP_EHIP = -2,
  MOONEP_EUNSUPPORTED = -3
};

typedef void* moonep_stream; /* a hipStream_t */

/* Text of the last error raised on the calling thread ("" when none). */
const char* moonep_last_error(void);

/* Planners of moonep_plan_ex. */
typedef enum moonep_planner {
  MOONEP_PLAN_PREFIX = 0, /* home-first prefix: each rank keeps the first S*K pairs of its home experts */
  MOONEP_PLAN_MINCOPY = 1 /* fewest copies: an overloaded rank's excess leaves through its largest experts */
} moonep_planner;

/* Bytes of device workspace moonep_plan needs for these dims (256-byte aligned pointer). */
size_t moonep_plan_workspace_bytes(moonep_dims d);

/*
 * moonep_plan -- histogram, maxvio and the home-first prefix-sum plan.
 *   maxvio = max_e(T_e / Tbar) - 1, Tbar = N / E ([P2] "Core problem"; [P3]
 *   paragraph two), evaluated as (double)(E * max_e T_e) / (double)N - 1.0
 *   (0.0 when N == 0).  Every rank then receives exactly P = S*K pairs
 *   ([P1] section 2; [P2] "Core technique"; [P3] paragraph three): rank r keeps
 *   the first P pairs of its home experts' pairs taken in (expert, src rank,
 *   token, k) order; the rest, in ascending (expert, order), are cut
 *   contiguously into the deficits P - L_r of the underloaded ranks in rank
 *   order.  On a receiving rank the arriving experts, in ascending order, take
 *   slots j = 0..B-1 (group E+j); beyond B they are read from their home row
 *   (group e) ([P2] "Memory contract and weight layout").
 * In:  topk_idx [R,S,K] int32 expert ids, pair (r,s,k) is flat id (r*S+s)*K+k.
 * Out: expert_counts [E]        int32  T_e.
 *      maxvio        [1]        double.
 *      cu_seqlens    [R,E+B+1]  int32  rank r's group g occupies local rows
 *                                      [cu[r,g], cu[r,g+1]); cu[r,0]=0, cu[r,E+B]=P
 *                                      (less where ids outside [0,E) leave rows without a pair).
 *      slot_expert   [R,B]      int32  expert held by slot j of rank r, -1 unused
 *                                      (may be NULL when B == 0).
 *      dest_idx      [R,S,K]    int32  global row r'*P + local row of each pair;
 *                                      -1 for an id outside [0,E).
 *      src_of_row    [R*S*K]    int32  inverse of dest_idx (flat pair id per row, -1
 *                                      for a row without a pair), or NULL to skip.
 *      stats         [4]        int32  copies (expert, non-home rank) used,
 *                                      of them slotted, of them direct reads,
 *                                      invalid ids + repeated ids within a token.
 * workspace: moonep_plan_workspace_bytes(d) bytes of device memory, contents
 * ignored on entry.
 * Limits (MOONEP_EINVAL beyond them): E <= 4096, R <= 4096, and each planner
 * block keeps per-expert and per-rank tables in LDS, so the largest of
 * E + max(1024, K), 5E + 4R and 8E + 3R int32 values must fit in 158 KiB
 * (E = 4096 allows R <= 2048; E = 2048 any R that divides it).
 */
int moonep_plan(moonep_dims d, const int32_t* topk_idx, int32_t* expert_counts, double* maxvio,
                int32_t* cu_seqlens, int32_t* slot_expert, int32_t* dest_idx, int32_t* src_of_row,
                int32_t* stats, void* workspace, moonep_stream stream);

/*
 * moonep_plan_ex -- moonep_plan with a choice of planner (a moonep_planner value; anything else is
 * MOONEP_EINVAL).  The pages describe their planner as one that keeps the number of redundant experts
 * small ([P1] abstract; [P2] "Core technique: dynamic redundant experts") without printing its program.
 * MOONEP_PLAN_PREFIX is moonep_plan.  MOONEP_PLAN_MINCOPY changes only which pairs stay home: a rank
 * with L_r > P pairs sends its excess L_r - P out of its home experts taken largest first (equal counts:
 * lower id first), each overflowing what is still needed, so the excess leaves through the fewest
 * experts; every expert keeps the first keep_e pairs of its (src rank, token, k)-ordered list.  The
 * overflow list, the contiguous cut into deficits in rank order, slots, direct reads past B, cu_seqlens
 * and destinations then follow exactly as in moonep_plan.  Arguments, layouts, workspace (the same
 * moonep_plan_workspace_bytes) and limits are those of moonep_plan.
 */
int moonep_plan_ex(moonep_dims d, int32_t planner, const int32_t* topk_idx, int32_t* expert_counts,
                   double* maxvio, int32_t* cu_seqlens, int32_t* slot_expert, int32_t* dest_idx,
                   int32_t* src_of_row, int32_t* stats, void* workspace, moonep_stream stream);

/*
 * moonep_plan_static -- moonep_plan_ex for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  It takes no workspace: the
 * planner's scratch is a device array inside the library, moonep_plan_static_scratch_bytes() (8 MiB)
 * large, of which every GPU the library runs on holds its own copy until the process ends.  The call
 * allocates and frees nothing.  Arguments, outputs and limits are those of moonep_plan_ex; dims whose
 * moonep_plan_workspace_bytes exceed the scratch size are refused with MOONEP_EINVAL (use moonep_plan_ex
 * with a workspace then).  Every call on one GPU uses that GPU's one array: calls that overlap on a GPU
 * (concurrent streams, or threads) race and give unspecified plans; calls in stream order do not.  No
 * scratch contents carry over between calls (every planner kernel writes its part before reading it).
 * MOONEP_EHIP when the array's device address cannot be obtained on the current device.
 */
size_t moonep_plan_static_scratch_bytes(void);
int moonep_plan_static(moonep_dims d, int32_t planner, const int32_t* topk_idx, int32_t* expert_counts,
                       double* maxvio, int32_t* cu_seqlens, int32_t* slot_expert, int32_t* dest_idx,
                       int32_t* src_of_row, int32_t* stats, moonep_stream stream);

/*
 * moonep_dispatch -- fused permute ([P2] "Core technique": each token row is
 * written straight into its expert-grouped row of the fixed S*K buffer).
 *   Xp[dest_idx[r,s,k], :] = X[r,s,:] for every k; rows with dest -1 are skipped.
 * In:  X [R,S,H] dtype t;  dest_idx [R,S,K] int32 from moonep_plan.
 * Out: Xp [R*S*K, H] dtype t (bit-exact copies).
 */
int moonep_dispatch(moonep_dims d, int32_t H, moonep_dtype t, const void* X, const int32_t* dest_idx,
                    void* Xp, moonep_stream stream);

/*
 * moonep_prefetch -- copy each used slot's expert weights into the slot
 * ([P2] "Core technique" and "Memory contract": redundant experts are fetched
 * into rows [E, E+B) before expert compute).
 *   W_slots[r,j] = W_home[slot_expert[r,j]] when slot_expert[r,j] >= 0;
 *   unused slots are not written.
 * In:  W_home [E,H,Hp] dtype t;  slot_expert [R,B] int32.
 * Out: W_slots [R,B,H,Hp] dtype t (bit-exact copies).
 */
int moonep_prefetch(moonep_dims d, int32_t H, int32_t Hp, moonep_dtype t, const void* W_home,
                    const int32_t* slot_expert, void* W_slots, moonep_stream stream);

/* Bytes of device workspace moonep_group_gemm needs. */
size_t moonep_group_gemm_workspace_bytes(moonep_dims d);

/*
 * moonep_group_gemm -- the VM group GEMM over each rank's logical [E+B,H,Hp]
 * weight tensor, groups delimited by cu_seqlens ([P2] "Memory contract").
 *   For rank r, group g: Yp[rows] = Xp[rows] @ W_r[g], rows = r*P + [cu[r,g], cu[r,g+1]).
 *   bf16: float32 accumulation, result rounded to nearest-even bf16.
 *   f32:  float32 throughout.
 * In:  Xp [R*S*K,H], W_home [E,H,Hp], W_slots [R,B,H,Hp] (NULL when B == 0), dtype t;
 *      cu_seqlens [R,E+B+1] int32.
 * Out: Yp [R*S*K,Hp] dtype t.
 * workspace: moonep_group_gemm_workspace_bytes(d) bytes.
 */
int moonep_group_gemm(moonep_dims d, int32_t H, int32_t Hp, moonep_dtype t, const void* Xp,
                      const void* W_home, const void* W_slots, const int32_t* cu_seqlens, void* Yp,
                      void* workspace, moonep_stream stream);

/*
 * moonep_combine -- gate-weighted fused unpermute ([P2] "Core technique").
 *   out[r,s,:] = sum_{k=0..K-1} gates[r,s,k] * Yp[dest_idx[r,s,k], :]
 *   float32 accumulation in ascending k (fused multiply-add); dest -1 is skipped.
 * In:  Yp [R*S*K, D] dtype t;  dest_idx [R,S,K] int32;  gates [R,S,K] float32.
 * Out: out [R,S,D] float32.
 */
int moonep_combine(moonep_dims d, int32_t D, moonep_dtype t, const void* Yp, const int32_t* dest_idx,
                   const float* gates, float* out, moonep_stream stream);

/*
 * Backward of the data path.  The pages state that the backward pass runs through the same
 * buffers and that redundant experts' gradients go back to their home experts ([P2] "Core
 * technique"; [P3] third paragraph); read plainly, the data gradients are the chain rule of
 * dispatch -> group GEMM -> combine, each stage the transpose of its forward.
 */

/*
 * moonep_combine_backward -- gradients of moonep_combine given dout = d(loss)/d(out).
 *   For every pair (r,s,k) with q = dest_idx[r,s,k]:
 *     dYp[q] = gates[r,s,k] * dout[r,s]            (float32 product, then rounded to dtype t)
 *     dgates[r,s,k] = sum_n dout[r,s,n] * Yp[q,n]  (float32 accumulation)
 *   Every row of dYp is the destination of exactly one pair, so all of dYp is written.
 * In:  dout [R,S,D] float32;  Yp [R*S*K,D] dtype t;  dest_idx [R,S,K] int32;  gates [R,S,K] float32.
 * Out: dYp [R*S*K,D] dtype t;  dgates [R,S,K] float32.
 */
int moonep_combine_backward(moonep_dims d, int32_t D, moonep_dtype t, const float* dout, const void* Yp,
                            const int32_t* dest_idx, const float* gates, void* dYp, float* dgates,
                            moonep_stream stream);

/*
 * moonep_group_gemm_dgrad -- gradient of the VM group GEMM with respect to its input, through the
 * same groups and the same weight rows (home, slot, or a home row read directly):
 *   For rank r, group g: dXp[rows] = dYp[rows] @ W_r[g]^T, rows = r*P + [cu[r,g], cu[r,g+1]).
 *   bf16: float32 accumulation, result rounded to nearest-even bf16;  f32: float32 throughout.
 * In:  dYp [R*S*K,Hp], W_home [E,H,Hp], W_slots [R,B,H,Hp] (NULL when B == 0), dtype t;
 *      cu_seqlens [R,E+B+1] int32.
 * Out: dXp [R*S*K,H] dtype t.
 * workspace: moonep_group_gemm_workspace_bytes(d) bytes (the same workspace as the forward).
 */
int moonep_group_gemm_dgrad(moonep_dims d, int32_t H, int32_t Hp, moonep_dtype t, const void* dYp,
                            const void* W_home, const void* W_slots, const int32_t* cu_seqlens, void* dXp,
                            void* workspace, moonep_stream stream);

/*
 * moonep_dispatch_backward -- gradient of moonep_dispatch (the fused permute):
 *   dX[r,s] = sum over k ascending of dXp[dest_idx[r,s,k]], float32 additions.
 * In:  dXp [R*S*K,H] dtype t;  dest_idx [R,S,K] int32.
 * Out: dX [R,S,H] float32.
 */
int moonep_dispatch_backward(moonep_dims d, int32_t H, moonep_dtype t, const void* dXp, const int32_t* dest_idx,
                             float* dX, moonep_stream stream);

/*
 * Full gated expert FFN.  The pages ask for one [E+B, H, H'] tensor per expert projection ([P2]
 * "Memory contract and weight layout") without naming the FFN; read plainly it is the gated expert:
 * a gate|up projection [E+B, H, 2H'] (gate in output columns [0, H'), up in [H', 2H')), then
 * act = silu(gate) * up, then a down projection [E+B, H', H].  Both projections run through
 * moonep_group_gemm / moonep_group_gemm_dgrad / moonep_wgrad / moonep_reduce_grad with their own
 * (H, Hp) -- (H, 2H') and (H', H) -- and the same plan; these two calls are the activation.
 */

/*
 * moonep_swiglu -- A[q, c] = silu(Ygu[q, c]) * Ygu[q, Hp + c] for every dispatched row q < R*S*K and
 *   c < Hp, silu(g) = g * sigmoid(g); float32 arithmetic, rounded once to dtype t.
 * In:  Ygu [R*S*K, 2*Hp] dtype t.   Out: A [R*S*K, Hp] dtype t.
 */
int moonep_swiglu(moonep_dims d, int32_t Hp, moonep_dtype t, const void* Ygu, void* A, moonep_stream stream);

/*
 * moonep_swiglu_backward -- gradient of moonep_swiglu: with g = Ygu[q,c], u = Ygu[q,Hp+c],
 *   s = sigmoid(g), da = dA[q,c]:  dYgu[q,c] = da * u * s * (1 + g * (1 - s)),  dYgu[q,Hp+c] = da * g * s;
 *   float32 arithmetic, rounded once to dtype t.
 * In:  Ygu [R*S*K, 2*Hp], dA [R*S*K, Hp] dtype t.   Out: dYgu [R*S*K, 2*Hp] dtype t.
 */
int moonep_swiglu_backward(moonep_dims d, int32_t Hp, moonep_dtype t, const void* Ygu, const void* dA, void* dYgu,
                           moonep_stream stream);

/* Bytes of device workspace moonep_wgrad needs. */
size_t moonep_wgrad_workspace_bytes(moonep_dims d);

/*
 * moonep_wgrad -- weight-gradient group GEMM into the float32 gradient
 * buffers ([P2] "Memory contract": an fp32 [E+B,H,Hp] gradient per projection
 * whose rows [E,E+B) are separate reduce buffers).
 *   For every rank r and group g: dW_r[g] += Xp[rows]^T @ dY[rows].
 *   g < E adds into dW_home[g]; when several ranks hold rows of home row g
 *   (the home rank plus direct reads) their rows are summed in ascending rank
 *   order into one float32 accumulator and added once.  g = E+j adds into
 *   dW_slots[r,j].  Groups with no rows leave their gradient untouched.
 * In:  Xp [R*S*K,H], dY [R*S*K,Hp] dtype t;  cu_seqlens [R,E+B+1].
 * In/Out: dW_home [E,H,Hp] float32;  dW_slots [R,B,H,Hp] float32 (NULL when B == 0).
 * workspace: moonep_wgrad_workspace_bytes(d) bytes of device memory (256-byte aligned), contents
 * ignored on entry (it holds the size-ordered list of gradient jobs that have rows, the work
 * queue counters and a row of zeros, all of which the call itself writes before use).
 */
int moonep_wgrad(moonep_dims d, int32_t H, int32_t Hp, moonep_dtype t, const void* Xp, const void* dY,
                 const int32_t* cu_seqlens, float* dW_home, float* dW_slots, void* workspace,
                 moonep_stream stream);

/*
 * moonep_reduce_grad -- fold redundant-expert gradients back to their home
 * expert and clear them ([P2] "Core technique" and "Memory contract": the
 * R reduce buffers viewed as [R,B,H,Hp]; each slot's gradient is added into
 * the parameter gradient, then the consumed slot is zeroed).
 *   For each expert e and each element, in float32:
 *     acc = dW_home[e]; for r = 0..R-1: for the slot j of rank r holding e:
 *       acc += dW_slots[r,j]; dW_slots[r,j] = 0;   then dW_home[e] = acc.
 *   Unused slots (slot_expert -1) are neither read nor written.
 * In:  slot_expert [R,B] int32.
 * In/Out: dW_home [E,H,Hp] float32;  dW_slots [R,B,H,Hp] float32.
 */
int moonep_reduce_grad(moonep_dims d, int32_t H, int32_t Hp, const int32_t* slot_expert, float* dW_home,
                       float* dW_slots, moonep_stream stream);

/*
 * Activation checkpoints in 8 bits.  The pages describe a backward pass through the same buffers as the
 * forward ([P2] "Core technique") and say nothing about what is kept between the two; these calls keep
 * the two tensors that the gated expert FFN's backward needs, its input and the activation's input, in
 * 8 bits, and read them there, so that the row buffers of the forward pass are free for the next layer.
 *
 * 8-bit rows: a [rows, C] tensor is kept as codes [rows, C] int8 and exps [rows, moonep_save8_blocks(C)]
 * uint8, one byte per 32 columns of a row (the last one covers what is left).  For a block of columns
 *   b = max(1, biased float32 exponent of its largest magnitude),  step = 2^(b - 133),
 *   code = x / step rounded to the nearest even whole number, held within +-127;  value = code * step.
 * A value is off by at most step / 2 (by step where |x| is within step / 2 of 128 steps), and step is at
 * most 1/64 of the block's largest magnitude (2^-132 where that is below 2^-126).  x / step and code * step are exact, and every value is a
 * bfloat16 number.  A block with an infinity or a NaN has b = 255: all its values are NaN, its codes
 * unspecified.
 *
 * In these calls and in the layer norm, output arrays do not overlap inputs or each other; row pointers
 * need the alignment of their elements only (rows of whole 8-column chunks at 16-byte aligned pointers,
 * 8 for codes, move fastest).  Widths (C, H, Hp, D) are at most 2^30, the norm's 32768 (MOONEP_EINVAL).
 */

/* ceil(C / 32): exponent bytes of a row of C columns (0 for C < 1). */
int32_t moonep_save8_blocks(int32_t C);

/*
 * moonep_save8 -- rows into 8 bits;  moonep_load8 -- the values that 8-bit rows stand for.
 * In/Out: X [rows, C] dtype t;  codes [rows, C] int8;  exps [rows, moonep_save8_blocks(C)] uint8.
 * moonep_load8 writes bf16 and f32 values exactly.  rows >= 0.
 */
int moonep_save8(int64_t rows, int32_t C, moonep_dtype t, const void* X, int8_t* codes, uint8_t* exps,
                 moonep_stream stream);
int moonep_load8(int64_t rows, int32_t C, moonep_dtype t, const int8_t* codes, const uint8_t* exps, void* X,
                 moonep_stream stream);

/*
 * moonep_swiglu_save8 -- moonep_swiglu (the same A, bit for bit), and its input kept in 8 bits in the same pass.
 *   Each row's gate and up halves are coded as rows of their own: the codes are those of moonep_save8 of Ygu as
 *   [2*R*S*K, Hp].
 * In:  Ygu [R*S*K, 2*Hp] dtype t.
 * Out: A [R*S*K, Hp] dtype t;  codes [R*S*K, 2, Hp] int8;  exps [R*S*K, 2, moonep_save8_blocks(Hp)] uint8.
 */
int moonep_swiglu_save8(moonep_dims d, int32_t Hp, moonep_dtype t, const void* Ygu, void* A, int8_t* codes,
                        uint8_t* exps, moonep_stream stream);

/*
 * moonep_swiglu_backward8 -- gradient of moonep_swiglu from its 8-bit input, with the gates applied here
 *   instead of in combine's backward.  For every row q, with p = src_of_row[q] and w = gates[p]:
 *     h = silu(g) * u,  A[q] = w * h,  dgates[p] = sum_c dA[q,c] * h[c]  (float32),
 *     dYgu[q] = w * dA * (u * s * (1 + g * (1 - s)) | g * s),  s = sigmoid(g);
 *   float32 arithmetic, each result rounded once to dtype t.
 *   dA is the gradient of the ungated expert output carried through the down projection: dout laid out by
 *   moonep_combine_backward_ungated and multiplied by W_down^T (moonep_group_gemm_dgrad).  Then
 *   sum_c dA * h = <dout, Z> is the gate's gradient without Z, and moonep_wgrad of (A, the ungated rows) is
 *   the down projection's.  src_of_row, gates and dgates may all be NULL: w is then 1.  A row whose
 *   src_of_row is outside [0, R*S*K) counts as w = 0 and has no dgates; pairs without a row (ids outside
 *   [0, E)) keep theirs, so a caller that may have such pairs clears dgates first.
 * In:  codes [R*S*K, 2, Hp] int8, exps;  dA [R*S*K, Hp] dtype t;  src_of_row [R*S*K] int32 from moonep_plan;
 *      gates [R,S,K] float32.
 * Out: A [R*S*K, Hp], dYgu [R*S*K, 2*Hp] dtype t;  dgates [R,S,K] float32.
 */
int moonep_swiglu_backward8(moonep_dims d, int32_t Hp, moonep_dtype t, const int8_t* codes, const uint8_t* exps,
                            const void* dA, const int32_t* src_of_row, const float* gates, void* A, void* dYgu,
                            float* dgates, moonep_stream stream);

/*
 * moonep_dispatch8 -- moonep_dispatch from 8-bit token rows: Xp[dest_idx[r,s,k], :] = v[r,s,:] with
 *   v = value * gamma + beta (one float32 fused multiply-add per element), rounded once to dtype t; with
 *   gamma and beta NULL, v = value.  beta alone may be NULL.  Rows with dest -1 are skipped.
 * In:  codes [R,S,H] int8, exps [R,S,moonep_save8_blocks(H)] uint8;  gamma, beta [H] float32;
 *      dest_idx [R,S,K] int32.
 * Out: Xp [R*S*K, H] dtype t.
 */
int moonep_dispatch8(moonep_dims d, int32_t H, moonep_dtype t, const int8_t* codes, const uint8_t* exps,
                     const float* gamma, const float* beta, const int32_t* dest_idx, void* Xp, moonep_stream stream);

/*
 * moonep_combine_backward_ungated -- the output gradient's rows by expert, without gates:
 *   dYp[dest_idx[r,s,k], :] = dout[r,s,:], rounded to dtype t; rows with dest -1 are skipped.
 * In:  dout [R,S,D] float32;  dest_idx [R,S,K] int32.   Out: dYp [R*S*K, D] dtype t.
 */
int moonep_combine_backward_ungated(moonep_dims d, int32_t D, moonep_dtype t, const float* dout,
                                    const int32_t* dest_idx, void* dYp, moonep_stream stream);

/*
 * Layer norm of the token rows, in front of the expert layer.
 */

/*
 * moonep_layernorm -- with m and v the mean and variance (divided by H) of a row x, r = 1 / sqrt(v + eps) and
 *   z = (x - m) * r:  Y = z * gamma + beta;  float32 arithmetic, rounded once to dtype t.  Rows are not scaled first:
 *   where their sum passes float32's range Y is NaN, where the sum of (x - m)^2 does r is 0 and Y is beta.
 * In:  X [R,S,H] dtype t;  gamma [H] float32;  beta [H] float32 or NULL (0);  eps > 0.
 * Out: Y [R,S,H] dtype t;  mean [R,S] (m), rstd [R,S] (r) float32, each NULL to skip;
 *      codes [R,S,H] int8, exps [R,S,moonep_save8_blocks(H)] uint8: z in 8 bits, both NULL to skip.
 */
int moonep_layernorm(moonep_dims d, int32_t H, moonep_dtype t, const void* X, const float* gamma, const float* beta,
                     float eps, void* Y, float* mean, float* rstd, int8_t* codes, uint8_t* exps,
                     moonep_stream stream);

/*
 * moonep_layernorm_dispatch -- moonep_layernorm and moonep_dispatch of its rows in one pass: Xp[dest_idx[r,s,k], :] =
 *   Y[r,s,:] of moonep_layernorm (the same bits), Y itself is not stored; rows with dest -1 are skipped.
 * In:  as moonep_layernorm;  dest_idx [R,S,K] int32 from moonep_plan.
 * Out: Xp [R*S*K, H] dtype t;  mean, rstd, codes, exps as moonep_layernorm.
 */
int moonep_layernorm_dispatch(moonep_dims d, int32_t H, moonep_dtype t, const void* X, const float* gamma,
                              const float* beta, float eps, const int32_t* dest_idx, void* Xp, float* mean,
                              float* rstd, int8_t* codes, uint8_t* exps, moonep_stream stream);

/* Bytes of device workspace moonep_layernorm_backward and moonep_layernorm_backward8 need on the current device. */
size_t moonep_layernorm_backward_workspace_bytes(moonep_dims d, int32_t H);

/*
 * moonep_layernorm_backward -- gradients of moonep_layernorm, with gy = dY * gamma and means over a row:
 *   dX = r * (gy - mean(gy) - z * mean(gy * z));
 *   dgamma[c] += sum over rows of dY * z;  dbeta[c] += sum over rows of dY  (one addition to what is there).
 *   float32 sums in a fixed order.  moonep_layernorm_backward forms z from X, mean and rstd,
 *   moonep_layernorm_backward8 reads it from 8 bits.
 * In:  dY [R,S,H] float32 (as moonep_dispatch_backward writes it);  X [R,S,H] dtype t and mean [R,S] float32, or
 *      codes and exps;  rstd [R,S], gamma [H] float32.
 * Out: dX [R,S,H] float32.   In/Out: dgamma, dbeta [H] float32 (dbeta NULL to skip).
 * workspace: moonep_layernorm_backward_workspace_bytes(d, H) bytes of device memory (256-byte aligned), contents
 * ignored on entry; calls that can overlap (two streams, two replayed graphs) need one each.
 */
int moonep_layernorm_backward(moonep_dims d, int32_t H, moonep_dtype t, const float* dY, const void* X,
                              const float* mean, const float* rstd, const float* gamma, float* dX, float* dgamma,
                              float* dbeta, void* workspace, moonep_stream stream);
int moonep_layernorm_backward8(moonep_dims d, int32_t H, const float* dY, const int8_t* codes, const uint8_t* exps,
                               const float* rstd, const float* gamma, float* dX, float* dgamma, float* dbeta,
                               void* workspace, moonep_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* MOONEP_H */
