/*
 * q4moe — affine 4-bit mixture-of-experts feed-forward on AMD MI355X (gfx950).
 *
 * Weight format (lily README, introduction and "Requirements": MLX affine
 * 4-bit weights, group size 64).  A Q4 matrix of n rows and k columns is
 *   codes  uint32 [n][k/8]   eight 4-bit codes per word; column j of a row is
 *                             in word j/8 at bits [4*(j%8), 4*(j%8)+4)
 *   scales bf16   [n][k/64]  one scale per 64 consecutive columns of a row
 *   biases bf16   [n][k/64]  one bias per 64 consecutive columns of a row
 * and stands for w[r][j] = scale[r][j/64] * code[r][j] + bias[r][j/64].
 * All arrays are row-major and contiguous.  Stacked matrices (count > 1) are
 * laid out [count][n][...].  Activations are bfloat16 bit patterns.
 *
 * Conventions for every entry point:
 *  - Pointers named in the argument lists are DEVICE pointers owned by the
 *    caller, except the descriptor structs, which are host memory read during
 *    the call only.  The library allocates nothing and keeps no state between
 *    calls; scratch comes from the caller's workspace (size from
 *    q4moe_workspace_bytes, 256-byte aligned).
 *  - Work is enqueued on `stream` (a hipStream_t; NULL is the null stream) and
 *    the call returns without synchronising.  Inputs must stay unmodified and
 *    the workspace untouched until the stream reaches the end of the call.
 *  - Arguments are validated on the host before any HIP call.  Invalid shapes,
 *    null pointers or misaligned buffers return Q4MOE_EINVAL (or
 *    Q4MOE_EUNSUPPORTED for valid shapes outside what the kernels handle) and
 *    enqueue nothing.  A HIP launch error returns Q4MOE_EHIP.  There is no
 *    fallback path.  No C++ exception crosses this interface.
 *  - Alignment: codes, activations and outputs 16-byte aligned; scale and bias
 *    arrays 2-byte aligned; workspaces 256-byte aligned.
 */
#ifndef Q4MOE_H
#define Q4MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t q4moe_bf16;   /* raw bfloat16 bits */
typedef void* q4moe_stream;    /* hipStream_t */

enum {
  Q4MOE_OK = 0,
  Q4MOE_EINVAL = 1,        /* null pointer, bad shape, misaligned buffer */
  Q4MOE_EUNSUPPORTED = 2,  /* valid but outside the kernels' limits */
  Q4MOE_EWORKSPACE = 3,    /* workspace missing or smaller than required */
  Q4MOE_EHIP = 4           /* a HIP runtime or launch error */
};

/* Output forms.  Q4MOE_OUT_BF16_RESIDUAL is accepted by moe_ffn_decode only: it
 * writes bf16(x + y), the next layer's input on a residual stream. */
enum { Q4MOE_OUT_F32 = 0, Q4MOE_OUT_BF16 = 1, Q4MOE_OUT_BF16_RESIDUAL = 2 };

/* Operation ids for q4moe_workspace_bytes. */
enum {
  Q4MOE_OP_GEMV = 0,
  Q4MOE_OP_GEMM = 1,
  Q4MOE_OP_ROUTE = 2,
  Q4MOE_OP_PERMUTE = 3,
  Q4MOE_OP_FFN_DECODE = 4,
  Q4MOE_OP_FFN_PREFILL = 5,
  Q4MOE_OP_LMHEAD = 6,
  Q4MOE_OP_FFN_DECODE_BATCH = 7,
  Q4MOE_OP_ROUTE_RULE = 8
};

/* An affine matrix of 4-bit codes (the default), or of 8-bit codes (the
 * checkpoint's 8-bit exceptions: "lily-qwen3.8-flash-next" README, "The model";
 * "2026-09-02: Lily vs MLX 0.32.2", "Hardware and software"), or `count` stacked
 * matrices of the same shape.  8-bit codes: uint32 [count][n][k/4], code j of a
 * row in byte j%4 of word j/4 (least significant first), same groups and
 * w = scale*q + bias.  q4_gemv and lmhead_argmax take 8-bit matrices, the layer
 * calls an 8-bit router (router_q8) and an 8-bit shared expert, and
 * moe_route_topk_q8 and moe_route an 8-bit router; the other calls return Q4MOE_EUNSUPPORTED
 * for them.
 *
 * codes_gm (optional, 4-bit only): the same codes group-major, as written by
 * q4moe_pack_group_major: uint32 [count][k/64][n][8], the 32 code bytes of group
 * g of row r at word ((e*k/64 + g)*n + r)*8, so that a group's bytes of consecutive
 * rows are contiguous.  q4_gemm and moe_ffn_prefill read it for their grouped GEMMs
 * (the products, their order and the results are those of the `codes` form) when
 * every 4-bit matrix they multiply carries it; every other call reads `codes`.  It is
 * a layout of the prefill's own, next to the MLX layout that decode streams row by
 * row. */
typedef struct {
  const uint32_t* codes;
  const q4moe_bf16* scales;
  const q4moe_bf16* biases;
  int64_t count;  /* >= 1 */
  int64_t n;      /* rows per matrix */
  int64_t k;      /* columns, a multiple of 64 */
  int32_t bits;   /* code width: 4 (0 also means 4) or 8 */
  int32_t reserved;  /* 0 */
  const uint32_t* codes_gm;  /* null, or the group-major copy of codes (16-byte aligned) */
} q4moe_matrix;

/*
 * One MoE feed-forward layer.  Routed expert e has gate and up matrices of
 * `inter` rows by `hidden` columns and a down matrix of `hidden` rows by
 * `inter` columns (gate/up/down stacked with count = n_experts).  The shared
 * expert, when sh_gate.codes is non-null, has the same shapes with count 1
 * and is added with weight 1, or with weight sigmoid(sh_gate_w . x) when the
 * layer carries a shared-expert gate vector (Qwen-family MoE layers do).  The router is bf16 [n_experts][hidden], or, when
 * router_q8.codes is non-null, the 8-bit affine matrix router_q8 (count 1,
 * n_experts x hidden, bits 8: the benchmark checkpoint's affine Q8 router-gate
 * exceptions, "2026-09-02: Lily vs MLX 0.32.2", "Hardware and software"), and
 * `router` may be null.  moe_ffn_decode, moe_ffn_decode_batch and moe_ffn_prefill
 * all take an 8-bit router (the standalone routers: moe_route_topk_q8, moe_route).  The
 * shared expert's three matrices may be 8-bit together (the q4-xl conversion
 * keeps it at 8 bits: "lily-qwen3.8-flash-next" README, "The model"); the layer
 * calls take that form (a mix of 4- and 8-bit shared matrices is
 * Q4MOE_EUNSUPPORTED).  Routed experts are 4-bit.
 */
typedef struct {
  int32_t hidden;
  int32_t inter;
  int32_t n_experts;
  int32_t top_k;
  const q4moe_bf16* router;
  q4moe_matrix gate, up, down;
  q4moe_matrix sh_gate, sh_up, sh_down;
  q4moe_matrix router_q8;  /* codes null: the bf16 router is used */
  const q4moe_bf16* sh_gate_w;  /* null, or bf16 [hidden]: the shared expert is weighted by
                                   sigmoid(sh_gate_w . x) in every layer call */
} q4moe_layer;

/*
 * A matrix of symmetric 8-bit codes, or `count` stacked matrices of the same shape:
 * codes int8 [count][n][k] and one fp32 scale per row (output channel), scales
 * [count][n], for w[r][j] = scales[r] * codes[r][j].  i8_quantize writes this form.
 * k a multiple of 64; codes 16-byte aligned, scales 4-byte aligned.
 */
typedef struct {
  const int8_t* codes;
  const float* scales;
  int64_t count;  /* >= 1 */
  int64_t n;      /* rows per matrix */
  int64_t k;      /* columns, a multiple of 64 */
} q4moe_i8_matrix;

/*
 * The experts of a layer in 8-bit integers: gate and up (count n_experts, inter x
 * hidden), down (count n_experts, hidden x inter); the shared expert, when
 * sh_gate.codes is non-null, has the same shapes with count 1 and is added with
 * weight 1.  (A shared expert with a weight of its own per token, a sigmoid gate say,
 * goes in as one more of the stacked experts, chosen by every token in a further slot
 * with that weight.)
 */
typedef struct {
  int32_t hidden;
  int32_t inter;
  int32_t n_experts;
  int32_t reserved;  /* 0 */
  q4moe_i8_matrix gate, up, down;
  q4moe_i8_matrix sh_gate, sh_up, sh_down;
} q4moe_i8_experts;

/*
 * A matrix in microscaled 4-bit floating point (OCP MXFP4), or `count` stacked matrices of
 * the same shape.  Each 32 consecutive columns of a row share a scale, a power of two held
 * as its exponent (E8M0): scales uint8 [count][n][k/32], a byte b for 2^(b - 127), 255 for
 * NaN.  codes uint8 [count][n][k/2]: column 2j of a row in the low four bits of byte j,
 * column 2j + 1 in the high four; a code is e2m1, a sign (bit 3) and one of 0, 0.5, 1, 1.5,
 * 2, 3, 4, 6.  w[r][j] = 2^(scale - 127) * code.  mx4_quantize writes this form.
 * k a multiple of 64; codes 16-byte aligned, scales 2-byte aligned.
 */
typedef struct {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t count;  /* >= 1 */
  int64_t n;      /* rows per matrix */
  int64_t k;      /* columns, a multiple of 64 */
} q4moe_mx4_matrix;

/*
 * The experts of a layer in microscaled 4-bit floating point, shaped as q4moe_i8_experts.
 */
typedef struct {
  int32_t hidden;
  int32_t inter;
  int32_t n_experts;
  int32_t reserved;  /* 0 */
  q4moe_mx4_matrix gate, up, down;
  q4moe_mx4_matrix sh_gate, sh_up, sh_down;  /* codes null: no shared expert */
} q4moe_mx4_experts;

/* Scores of q4moe_routing. */
enum { Q4MOE_SCORE_SOFTMAX = 0, Q4MOE_SCORE_SIGMOID = 1 };

/*
 * A routing rule.  With logits l (fp32), scores s = softmax(l) over all experts or
 * s = sigmoid(l) each, and choices c = s + bias:
 *  - an expert is closed for a token when its logit or its bias is NaN or
 *    -infinity; a closed expert is never chosen;
 *  - with n_groups > 1 the experts form n_groups groups of n_experts / n_groups
 *    consecutive ones.  A group's value is the sum of the open ones among its
 *    group_terms largest choices (1 or 2); the top_groups groups of largest value
 *    stay and the experts of the others are not chosen;
 *  - the top_k largest choices among what stays are chosen, in descending order.
 *    Equal values, of experts or of groups, go to the lower index;
 *  - the weight of a chosen expert is its score s, without the bias; with
 *    renormalise divided by the sum of the chosen scores (all 0 where that sum is
 *    0); then times scale;
 *  - where fewer than top_k experts are open the last slots get id -1 and weight 0.
 * Scores, choices and sums are computed in 64 bits from the fp32 logits (without a
 * bias, and with groups valued by one term, choices are compared by their logits)
 * and each weight is rounded once to fp32.  In a softmax a closed logit counts as 0,
 * and +infinity takes the whole row (several share it).
 */
typedef struct {
  int32_t n_experts;    /* 1..1024 */
  int32_t hidden;       /* a multiple of 64; moe_route only */
  int32_t top_k;        /* 1..32, at most top_groups * (n_experts / n_groups) */
  int32_t score;        /* Q4MOE_SCORE_* */
  int32_t n_groups;     /* 1..64, divides n_experts */
  int32_t top_groups;   /* 1..n_groups */
  int32_t group_terms;  /* 1 or 2 */
  int32_t renormalise;  /* 0 or 1 */
  float scale;          /* finite */
  int32_t reserved;     /* 0 */
  const float* bias;    /* null, or fp32 [n_experts] */
  const q4moe_bf16* router;  /* moe_route: bf16 [n_experts][hidden], may be null with router_q8 */
  q4moe_matrix router_q8;    /* moe_route: codes null, or the 8-bit router used in its place */
} q4moe_routing;

/*
 * y = W x, one bf16 vector x[k] against every row of W (count*n rows), fp32
 * accumulation, y written as fp32 or bf16 [count*n].  The decode form of the
 * 4-bit weight stream (lily-qwen3.8-flash-next README, "How the speed was
 * achieved": decode reads every weight once and is bandwidth-bound).
 */
int q4_gemv(const q4moe_matrix* W, const q4moe_bf16* x, void* y, int out_dtype,
            q4moe_stream stream);

/*
 * Y[m][r] = sum_j X[m][j] W[r][j] for bf16 rows X[m][k], Y [m][count*n] fp32 or
 * bf16.  The prefill form, run on fp16 matrix cores (lily-qwen3.8-flash-next
 * README, "How the speed was achieved": prefill GEMMs on the tensor units):
 * each row of X is scaled by an exact power of two into fp16 (exact for bf16
 * values within 2^-23 of the row's largest), each scale*q is rounded once to
 * fp16 (at most 2^-12 relative), the bias term is exact up to fp32 summation,
 * and accumulation is fp32.  Scales must be below 64 in magnitude.  Needs
 * Q4MOE_OP_GEMM workspace (m).
 */
int q4_gemm(const q4moe_matrix* W, const q4moe_bf16* X, int64_t m, void* Y, int out_dtype,
            void* workspace, size_t workspace_bytes, q4moe_stream stream);

/*
 * Router of the mixture-of-experts layer (lily README, introduction: the
 * checkpoint is a 35B-A3B model, about 3B of its 35B parameters active per
 * token, which is a router picking a few experts per token; the pages give no
 * rule, and softmax -> top-k -> renormalise is the plain reading):
 * logits[t][e] = router[e] . X[t] (fp32 accumulation), softmax over
 * all n_experts, the top_k largest kept in descending order (equal logits:
 * lower expert id first), their probabilities renormalised to sum to 1.
 * Writes ids int32 [T][top_k] and weights fp32 [T][top_k].  1 <= top_k <= 32,
 * top_k <= n_experts <= 1024, hidden a multiple of 64.  Needs
 * Q4MOE_OP_ROUTE workspace (T).
 */
int moe_route_topk(const q4moe_bf16* router, int32_t n_experts, int32_t hidden,
                   const q4moe_bf16* X, int64_t T, int32_t top_k, int32_t* ids, float* weights,
                   void* workspace, size_t workspace_bytes, q4moe_stream stream);

/*
 * moe_route_topk with the benchmark checkpoint's affine-Q8 router gate
 * ("2026-09-02: Lily vs MLX 0.32.2", "Hardware and software": the Q4 checkpoint
 * keeps its router gates at 8 bits): router_q8 is an 8-bit matrix (bits 8,
 * count 1) of n = n_experts rows by k = hidden columns, its logits
 * logits[t][e] = sum_j (scale*q + bias)[e][j] X[t][j] in fp32, the rest as
 * moe_route_topk.  The same workspace (Q4MOE_OP_ROUTE with n_experts).
 */
int moe_route_topk_q8(const q4moe_matrix* router_q8, const q4moe_bf16* X, int64_t T, int32_t top_k,
                      int32_t* ids, float* weights, void* workspace, size_t workspace_bytes,
                      q4moe_stream stream);

/*
 * moe_route_topk with a routing rule (see q4moe_routing): logits of the rows
 * X bf16 [T][hidden] through rule->router or rule->router_q8 in fp32, then the rule.
 * Rows of one call are summed alike, but few rows (T up to 64) in another order than
 * more, and than moe_route_topk sums them: where choices lie within such a sum's
 * rounding of each other, another T or the other call may choose another expert.
 * Writes ids int32 [T][top_k] and weights fp32 [T][top_k], which overlap neither X nor
 * each other nor the workspace (Q4MOE_EINVAL); T up to 2^26.  Needs
 * Q4MOE_OP_ROUTE_RULE workspace (n_experts; T), its first 256 bytes zero-filled before
 * its first use and used by moe_route alone: few rows run as one launch whose last
 * workgroups select, by arrival counts in these bytes that each call leaves at zero
 * again.  Counts that were not zero give id -1 and weight NaN in every slot, until they
 * are zeroed.  Calls that share a workspace must not overlap.
 */
int moe_route(const q4moe_routing* rule, const q4moe_bf16* X, int64_t T, int32_t* ids, float* weights,
              void* workspace, size_t workspace_bytes, q4moe_stream stream);

/*
 * The rule alone, on logits fp32 [T][n_experts] that the caller has; rule->hidden,
 * router and router_q8 are not read.  ids and weights overlap neither the logits nor
 * each other (Q4MOE_EINVAL).  No workspace.
 */
int moe_route_logits(const q4moe_routing* rule, const float* logits, int64_t T, int32_t* ids, float* weights,
                     q4moe_stream stream);

/*
 * Stable counting sort of the T*top_k rows r = t*top_k + slot by expert id
 * (token-to-expert grouping for the prefill expert GEMM; lily-qwen3.8-flash-next
 * README, "How the speed was achieved").  Writes offsets int32 [n_experts+1]
 * (offsets[e]..offsets[e+1] is expert e's segment), sorted_rows int32 [T*top_k]
 * (rows of each segment in increasing r) and inv_rows int32 [T*top_k] with
 * inv_rows[sorted_rows[p]] = p.  ids must lie in [0, n_experts); an
 * out-of-range id is skipped by the kernels and leaves the outputs
 * inconsistent.  Needs Q4MOE_OP_PERMUTE workspace (T*top_k).
 */
int moe_permute(const int32_t* ids, int64_t T, int32_t top_k, int32_t n_experts,
                int32_t* offsets, int32_t* sorted_rows, int32_t* inv_rows,
                void* workspace, size_t workspace_bytes, q4moe_stream stream);

/*
 * One token through the MoE layer (batch-1 greedy decode step):
 *   y = sum_i w_i down_{e_i}(silu(gate_{e_i} x) * up_{e_i} x) + shared(x)
 * with (e_i, w_i) from the router as in moe_route_topk.  x bf16 [hidden]; y fp32
 * or bf16 [hidden], or with Q4MOE_OUT_BF16_RESIDUAL the bf16 rounding (nearest,
 * ties to even) of x + y computed in fp32, which is the next layer's input when
 * layers are chained through a residual stream (lily-qwen3.8-flash-next, "How
 * the speed was achieved": a decode step runs every layer on the GPU, so the
 * host is off the critical path); y must not overlap x (Q4MOE_EINVAL).  ids_out
 * int32 [top_k] and w_out fp32 [top_k] may be null.  Intermediates stay fp32.  Runs as one launch of one workgroup per compute
 * unit; values passed between workgroups carry a per-launch tag kept in the
 * workspace, so the Q4MOE_OP_FFN_DECODE workspace must be zero-filled before
 * its first use and must stay with one device; each call leaves it ready for
 * the next.  Calls that share a workspace must not overlap.  Every wait inside
 * the kernel is bounded (about a quarter second): if one ever gives up, the
 * result is wrong and the 32-bit word at byte offset 2048 of the workspace is
 * incremented (it stays 0 in correct use).
 */
int moe_ffn_decode(const q4moe_layer* layer, const q4moe_bf16* x, void* y, int out_dtype,
                   int32_t* ids_out, float* w_out, void* workspace, size_t workspace_bytes,
                   q4moe_stream stream);

/*
 * moe_ffn_decode for callers that cannot allocate: code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation.  Same arguments, result
 * and kernels, without a workspace: the call uses a fixed scratch array of 1 MiB
 * inside the library (one per device, held until the process ends; zero at load,
 * and every call leaves it ready for the next).  The call allocates nothing.
 * Layers whose Q4MOE_OP_FFN_DECODE workspace would exceed 1 MiB return
 * Q4MOE_EUNSUPPORTED (no layer that moe_ffn_decode takes needs that much).  All calls on one device share the array: calls that
 * overlap on one device (on different streams without ordering) race and give
 * wrong results.  Its abandoned-wait counter is internal (use moe_ffn_decode to
 * read one).
 */
int moe_ffn_decode_noalloc(const q4moe_layer* layer, const q4moe_bf16* x, void* y, int out_dtype,
                           int32_t* ids_out, float* w_out, q4moe_stream stream);

/*
 * B tokens, one per request, through the MoE layer in one decode step
 * (lily-qwen3.8-flash-next, "Running it": up to four requests by default
 * decode together), 1 <= B <= 8: row b of Y equals moe_ffn_decode on X[b] up
 * to rounding (intermediates stay fp32).  X bf16 [B][hidden]; Y fp32 or bf16
 * [B][hidden]; ids_out int32 [B][top_k] and w_out fp32 [B][top_k] may be null.
 * Each expert chosen by any of the tokens is read once for all of them.  Runs
 * as two launches: one of one workgroup per compute unit (router, every
 * token's top-k, the step's expert plan, gate/up with SwiGLU), whose
 * workgroups pass the router logits to each other as tagged words as
 * moe_ffn_decode does, then the down projection with the weighted sum.  B = 1
 * runs moe_ffn_decode's single launch when it applies (y not overlapping x,
 * and a workspace as large as Q4MOE_OP_FFN_DECODE needs: the
 * Q4MOE_OP_FFN_DECODE_BATCH size for one row includes it).  The
 * Q4MOE_OP_FFN_DECODE_BATCH workspace (B) must be zero-filled before its
 * first use and stay with one device; each call leaves it ready for the next,
 * and calls that share a workspace must not overlap.  Waits are bounded as in
 * moe_ffn_decode (the same counter at byte offset 2048).  Q4MOE_EUNSUPPORTED:
 * shapes whose staged vectors exceed 64 KB of LDS (B * hidden * 21 / 8 bytes
 * of inputs, or (top_k + 1) * inter * 37 / 8 bytes of SwiGLU outputs for one
 * token), or a device on which one front workgroup per compute unit cannot be
 * resident at once.
 */
int moe_ffn_decode_batch(const q4moe_layer* layer, const q4moe_bf16* X, int64_t B, void* Y,
                         int out_dtype, int32_t* ids_out, float* w_out, void* workspace,
                         size_t workspace_bytes, q4moe_stream stream);

/*
 * T tokens through the MoE layer (a prefill chunk, 2,048 tokens in the
 * "Measurement contract" of "2026-09-02: Lily vs MLX 0.32.2"): route, permute
 * by expert, grouped fp16-MFMA GEMMs (as q4_gemm) for gate/up with SwiGLU and
 * for down with the routing weight, then combine back in token order.  Row t
 * of Y equals moe_ffn_decode on X[t] up to rounding; the SwiGLU output is
 * computed in fp32 and rounded once to fp16 (after an exact power-of-two row
 * scaling; a value that lands below fp16's normal range there, under 2^-22 of
 * its row's largest, may round twice) before the down GEMM, and each expert's
 * weighted output is rounded
 * once to fp16 precision (11 significant bits, kept in range by a power of two
 * per four columns) before the combine adds them in fp32.  The GEMMs read the experts' group-major
 * codes when every 4-bit expert matrix of the layer (routed and shared) carries
 * them (q4moe_matrix.codes_gm; the results are the same bits either way).
 * Y fp32 or bf16 [T][hidden].  Needs Q4MOE_OP_FFN_PREFILL workspace (T).
 */
int moe_ffn_prefill(const q4moe_layer* layer, const q4moe_bf16* X, int64_t T, void* Y,
                    int out_dtype, void* workspace, size_t workspace_bytes, q4moe_stream stream);

/*
 * Symmetric 8-bit form of bf16 rows X[rows][k]: scales[r] is the fp32 nearest to
 * max|X[r]| / 127 and codes[r][j] the integer nearest to X[r][j] / scales[r] (ties to
 * even; -127..127).  A row of zeros gets scale 0 and codes 0; a row that holds an
 * infinity or a NaN gets scale NaN and codes 0, so products with it are NaN.  The
 * load-time step for weights (a row is an output channel), and what i8_gemm does to
 * its activations (a row is a token).  k a multiple of 64 up to 65536; X and codes
 * 16-byte aligned, codes and scales not overlapping X.
 */
int i8_quantize(const q4moe_bf16* X, int64_t rows, int64_t k, int8_t* codes, float* scales,
                q4moe_stream stream);

/*
 * Y[m][r] = (sum_j q[m][j] codes[r][j] * sx[m]) * scales[r] for bf16 rows X[m][k],
 * with q, sx the 8-bit form of X's rows (i8_quantize), taken inside the call.  The
 * product in 8-bit integers next to q4_gemm's fp16 one: the integer sum is exact
 * (int32) and is rounded where it becomes fp32, at each scale, and to Y's type.
 * Y fp32 or bf16 [m][count*n], not overlapping X; k up to 65536.  Needs a workspace
 * of i8_gemm_workspace_bytes, which overlaps neither.
 */
int i8_gemm(const q4moe_i8_matrix* W, const q4moe_bf16* X, int64_t m, void* Y, int out_dtype,
            void* workspace, size_t workspace_bytes, q4moe_stream stream);

/*
 * i8_gemm on rows that are in 8-bit form already: codes int8 [m][k] (16-byte aligned) and
 * scales fp32 [m], as i8_quantize and rms_norm write them; the results are i8_gemm's bits
 * on the rows that these came from.  For several products of the same rows, and after a
 * norm.  Y overlaps neither.  No workspace.
 */
int i8_gemm_rows(const q4moe_i8_matrix* W, const int8_t* codes, const float* scales, int64_t m, void* Y,
                 int out_dtype, q4moe_stream stream);

/* Workspace bytes of i8_gemm on m rows; 0 for invalid arguments. */
size_t i8_gemm_workspace_bytes(const q4moe_i8_matrix* W, int64_t m);

/*
 * Root-mean-square norm of bf16 rows X[rows][k], after the residual's addition:
 *   t = bf16(X + residual)  (or X, where residual and total are null)
 *   y = t / sqrt(sum_j t_j^2 / k + eps) * weight
 * total bf16 [rows][k] receives t, the residual stream that the next addition takes; it
 * may be X or residual itself.  The result goes to y as bf16 [rows][k] (rounded once from
 * fp32 that is within 2^-22 of it, or 2^-136 where that is more), or in i8_quantize's 8-bit
 * form to codes int8 [rows][k] and scales fp32 [rows], or to both: codes and scales are those
 * of the unrounded y (scales[r] the fp32 nearest to max|y| / 127, codes computed in fp64,
 * halves to the even one), so that a product takes them with one rounding less than a bf16 y
 * would bring.  y is null, or codes and scales are.  A row that holds an infinity or a NaN
 * (in t, or in weight) gives scale NaN and codes 0; its y is what the formula gives.  weight
 * bf16 [k]; k a multiple of 8 up to 65536; eps at least 1.2e-38 and finite.  Buffers overlap
 * no other (but total as said).
 */
int rms_norm(const q4moe_bf16* X, const q4moe_bf16* residual, const q4moe_bf16* weight, int64_t rows, int64_t k,
             double eps, q4moe_bf16* total, q4moe_bf16* y, int8_t* codes, float* scales, q4moe_stream stream);

/*
 * T tokens through the 8-bit experts that a router chose for them: with ids int32
 * [T][top_k] and weights fp32 [T][top_k] (moe_route's, moe_route_topk's or the
 * caller's),
 *   y[t] = sum_i weights[t][i] * down_e(act_e(x[t])), e = ids[t][i], + shared(x[t])
 *   act_e(x) = silu(gate_e x) * up_e x
 * Both products are i8_gemm's: x in 8-bit form per token, the fp32 activations in
 * 8-bit form per token and expert.  A slot whose id lies outside [0, n_experts) adds
 * nothing (a token all of whose slots do gets the shared expert alone, or zeros); an
 * id may stand in several slots of a token.  The slots' products are summed in fp32
 * in slot order, the shared expert last; a bf16 Y is that sum rounded once.  A
 * token's result is the same bits whatever other tokens the call has.
 * X bf16 [T][hidden], Y fp32 or bf16 [T][hidden], not overlapping X, ids or weights;
 * hidden and inter multiples of 64 up to 16384, n_experts up to 1024, top_k up to 32
 * (not bounded by n_experts).  Needs a workspace of moe_experts_i8_workspace_bytes that
 * overlaps none of them.
 */
int moe_experts_i8(const q4moe_i8_experts* experts, const q4moe_bf16* X, int64_t T, const int32_t* ids,
                   const float* weights, int32_t top_k, void* Y, int out_dtype, void* workspace,
                   size_t workspace_bytes, q4moe_stream stream);

/* Workspace bytes of moe_experts_i8 on T tokens of top_k slots; 0 for invalid arguments. */
size_t moe_experts_i8_workspace_bytes(const q4moe_i8_experts* experts, int64_t T, int32_t top_k);

/*
 * Microscaled 4-bit form (see q4moe_mx4_matrix) of bf16 rows X[rows][k].  A block's scale is
 * 2^(floor(log2(max|x|)) - 2), at least 2^-127, and its codes are x / scale rounded to the
 * nearest of e2m1's values (ties to the even code; beyond 6 to 6).  A block of zeros gets
 * scale byte 0; a block that holds an infinity or a NaN gets scale byte 255 and codes 0, so
 * products with it are NaN.  The load-time step for weights, and what mx4_gemm does to its
 * activations.  k a multiple of 64 up to 65536; X and codes 16-byte aligned, scales 2-byte
 * aligned; no buffer overlaps another.
 */
int mx4_quantize(const q4moe_bf16* X, int64_t rows, int64_t k, uint8_t* codes, uint8_t* scales, q4moe_stream stream);

/*
 * The values of a matrix (all count * n rows) as bf16 [count*n][k], exact: magnitudes of 2^128
 * and more, which mx4_quantize does not write, become infinite.  Y overlaps neither input.
 */
int mx4_dequantize(const q4moe_mx4_matrix* W, q4moe_bf16* Y, q4moe_stream stream);

/*
 * Y[m][r] = sum_j xq[m][j] w[r][j] for bf16 rows X[m][k], with xq the microscaled 4-bit form
 * of X's rows (mx4_quantize), taken inside the call.  The product in 4-bit floating point
 * next to i8_gemm's in integers, on the matrix cores that take the blocks' scales: each
 * product is exact, sums are fp32 (rows of one call alike, few rows in another order than
 * more).  Y fp32 or bf16 [m][count*n], not overlapping X; k up to 65536.  Needs a workspace
 * of mx4_gemm_workspace_bytes, which overlaps neither.
 */
int mx4_gemm(const q4moe_mx4_matrix* W, const q4moe_bf16* X, int64_t m, void* Y, int out_dtype, void* workspace,
             size_t workspace_bytes, q4moe_stream stream);

/* Workspace bytes of mx4_gemm on m rows; 0 for invalid arguments. */
size_t mx4_gemm_workspace_bytes(const q4moe_mx4_matrix* W, int64_t m);

/*
 * moe_experts_i8 with experts in microscaled 4-bit floating point: x in that form per token,
 * silu(gate x) * up x (fp32) per token and expert, both products mx4_gemm's.  Ids, weights,
 * empty and repeated slots, the order of the sum and the shared expert as there.  X bf16
 * [T][hidden], Y fp32 or bf16 [T][hidden], not overlapping X, ids or weights; hidden and
 * inter multiples of 64 up to 16384, n_experts up to 1024, top_k up to 32 (not bounded by
 * n_experts).  A token's result may differ in its sums' last bits, and in an activation next
 * to a border between two codes, with the number of tokens in the call.  Needs a workspace of
 * moe_experts_mx4_workspace_bytes that overlaps none of them.
 */
int moe_experts_mx4(const q4moe_mx4_experts* experts, const q4moe_bf16* X, int64_t T, const int32_t* ids,
                    const float* weights, int32_t top_k, void* Y, int out_dtype, void* workspace,
                    size_t workspace_bytes, q4moe_stream stream);

/* Workspace bytes of moe_experts_mx4 on T tokens of top_k slots; 0 for invalid arguments. */
size_t moe_experts_mx4_workspace_bytes(const q4moe_mx4_experts* experts, int64_t T, int32_t top_k);

/*
 * Greedy LM head: logits[b][r] = W[r] . X[b] in fp32 for b < B (1 <= B <= 8),
 * ids[b] = the lowest index of the largest logit (Lily decodes greedily: lily
 * README, introduction).  max_logit fp32 [B] may be null.  Needs
 * Q4MOE_OP_LMHEAD workspace (B), zero-filled before its first use: the call
 * keeps an arrival count of its workgroups and one running 64-bit maximum per
 * batch row there (the last workgroup to arrive reads them) and leaves both at
 * zero again, so calls that share a workspace must not overlap.
 */
int lmhead_argmax(const q4moe_matrix* W, const q4moe_bf16* X, int64_t B, int32_t* ids,
                  float* max_logit, void* workspace, size_t workspace_bytes, q4moe_stream stream);

/*
 * The next token of B rows of logits [B][V], drawn by given random numbers u fp32 [B] in
 * [0, 1): what lmhead_argmax's greedy choice is to one, on logits that a product wrote.
 * logits_dtype: Q4MOE_OUT_F32 or Q4MOE_OUT_BF16.  Each row has its own parameters (each
 * array [B], or null for none): temperature fp32, top_k int32, top_p fp32, min_p fp32.
 *  - temperature t: weights are w_i = exp((l_i - max l) / t).  Where t is not above 0 the
 *    row is greedy: its largest logit, the filters aside.
 *  - The filters keep a first part of the tokens in descending order of their logits
 *    (equal ones: the lower index first).  top_k in 1..V-1: that many tokens (others: all).
 *    top_p below 1: of these the fewest whose weights sum to at least top_p of theirs, one at
 *    least.  min_p above 0: of these the ones with w_i >= min_p (1 where it is larger), the
 *    weight of the likeliest being 1.
 *  - ids[b] is the first token in the order of the vocabulary with which the kept weights'
 *    running sum exceeds u times their total; probs[b] (may be null) its weight over the total.
 * A NaN logit is closed, as -infinity is: never kept.  A row without an open logit gets id -1
 * and probability 0; of a row with a logit of +infinity these share the weight.  A u outside
 * [0, 1) counts as the nearest in it, a NaN as 0.  NaN parameters are: a temperature greedy,
 * a top_p or min_p none.  Weights are taken in fp64 to multiples of 2^-45 of the largest and
 * added as integers, and top_p's and u's shares of their totals are exact, so a row gets the
 * same token in any batch and on any run.
 * V up to 262144, B up to 65536; logits aligned to their type; ids and probs overlap no
 * input, each other or the workspace (Q4MOE_EINVAL).  Needs a workspace of
 * sample_logits_workspace_bytes; calls that share one must not overlap.
 */
int sample_logits(const void* logits, int logits_dtype, int64_t B, int64_t V, const float* u,
                  const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p, int32_t* ids,
                  float* probs, void* workspace, size_t workspace_bytes, q4moe_stream stream);

/* Workspace bytes of sample_logits on B rows; 0 for invalid arguments. */
size_t sample_logits_workspace_bytes(int64_t B, int64_t V);

/*
 * Write the group-major copy of a 4-bit matrix's codes (see q4moe_matrix) to dst:
 * uint32 [count][k/64][n][8] (count*n*k/8 words, 16-byte aligned, device memory the
 * caller owns; it must not overlap W->codes).  A layout step for prefill, done once per
 * matrix (when weights are loaded), not per call.  W must be 4-bit (8-bit:
 * Q4MOE_EUNSUPPORTED); W->codes_gm is ignored.  Asynchronous on `stream`.
 */
int q4moe_pack_group_major(const q4moe_matrix* W, uint32_t* dst, q4moe_stream stream);

/*
 * Workspace bytes for an operation.  `layer` is read for the FFN and ROUTE
 * ops (ROUTE and ROUTE_RULE use layer->n_experts), `W` for GEMM and LMHEAD; `rows` is T, m
 * or B.  Returns 0 when no workspace is needed or the arguments are invalid.
 */
size_t q4moe_workspace_bytes(int op, const q4moe_layer* layer, const q4moe_matrix* W, int64_t rows);

/* Static text for a status code. */
const char* q4moe_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* Q4MOE_H */
