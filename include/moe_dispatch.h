/*
 * moe_dispatch.h -- C ABI of the MI355X (gfx950) MoE token dispatch / unpermute-combine library
 * (libmoe_dispatch.so).
 *
 * The operations follow these web pages (cited by title and section):
 *   [Combine]   "03 · Combine 与 forward / backward 对称性" (llm-infra-atlas, EP chapter)
 *   [Scratch]   "从零理解 MoE 算子：路由、专家并行与 Token 重排" (171host)
 *   [CANN]      CANN Dispatch&Combine optimisation notes (cann.csdn.net), "Dispatch&Combine优化"
 *   [Megatron]  "token dispatcher + fuse_a2a" (obnotes, Megatron/transformer-moe)
 *
 * Conventions for every call:
 *   - Pointers to tensors are DEVICE memory owned by the caller (the library never allocates
 *     and never frees). Tensors are row-major and contiguous. Indices and counts are int32,
 *     router weights and probabilities float32, hidden rows float32 or bf16 (moe_dtype).
 *   - Calls are asynchronous: they enqueue kernels on `stream` (a hipStream_t; NULL is the
 *     null stream) and return. Results are visible to later work on the same stream.
 *   - Argument errors are reported synchronously, before anything is launched:
 *     MOE_ERR_INVALID (null pointer where data is needed, negative size, K < 1, K > E,
 *     H < 1, group size not dividing E, ...) or MOE_ERR_UNSUPPORTED (E > 1024, K > 32, a
 *     hidden row longer than 2^31 - 1 bytes, more than 2^31 - 1 tokens, or a combination the
 *     call does not implement). MOE_ERR_HIP means a launch failed.
 *   - A size of zero tokens / rows is valid (an empty rank or an expert with no tokens must
 *     work, [Scratch] §26.1-26.2): a call with nothing to write launches nothing, and
 *     moe_build_index with T = 0 still writes its per-expert results (zero counts) and the
 *     marks of its rows (padding or unused).
 *   - Memory safety does not depend on the data: an expert id outside [0, E) routes nowhere
 *     (the pages write -1 for "no expert"), a row index outside the source range selects a
 *     zero row (permute) or no term (combine). Expert ids in one row of topk_idx must be
 *     distinct for the pages' routing map to be defined; if they repeat, slots of the same
 *     expert are ordered by slot.
 *   - The library holds no global state (apart from the scratch of moe_build_index_noalloc);
 *     calls on different streams may run concurrently as long as they do not write the same
 *     memory.
 */
#ifndef MOE_DISPATCH_H
#define MOE_DISPATCH_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID = 1,
    MOE_ERR_UNSUPPORTED = 2,
    MOE_ERR_HIP = 3
} moe_status;

/* Element types of hidden rows. MOE_FP8_E4M3 (1-byte OCP E4M3 codes, the FP8 dispatch) is
 * accepted by the permutes only, which copy bytes; the combines work in bf16 / float32 and
 * return MOE_ERR_UNSUPPORTED for it. */
typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_FP8_E4M3 = 2 } moe_dtype;

/* Upper limits of the kernels. */
#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_TOPK 32
#define MOE_MAX_FEW_TOKENS 256 /* tokens of moe_few_token_layer and moe_few_token_experts */

/* Markers in gather maps (sorted_indices, esrc): a padding row, written as zeros by the
 * permutes; and an unused row after the last expert segment (buffer slack when the buffer is
 * sized by an upper bound), which no call writes. */
#define MOE_ROW_PAD (-1)
#define MOE_ROW_UNUSED (-2)

/* Static, human-readable name of a status code. Never NULL. */
const char *moe_status_string(moe_status s);

/* Expert capacity, [Scratch] §18: ceil(tokens * top_k / num_experts * capacity_factor) with the
 * capacity factor given as the exact fraction cf_num / cf_den (1.25 = 5/4), computed in
 * integers on the host. 1024 tokens, top_k 2, 8 experts, 5/4 -> 320.
 * Returns -1 for tokens < 0, top_k < 1, num_experts < 1, cf_num < 0, cf_den < 1 or a result
 * that does not fit in int32. */
int64_t moe_expert_capacity(int64_t tokens, int32_t top_k, int32_t num_experts,
                            int32_t cf_num, int32_t cf_den);

/* Top-k routing, [Scratch] §3 and §27: for each token t the K experts with the largest logits,
 * then a softmax over those K logits only.
 *   logits   [T, E] float32, finite.
 *   topk_idx [T, K] int32 out: slot k is the k-th expert in the order (logit descending,
 *            expert id ascending); equal logits (+0 and -0 are equal) go to the lower id.
 *   topk_w   [T, K] float32 out: w_k = exp(s_k - s_0) / sum_j exp(s_j - s_0), evaluated in
 *            double (the router softmax is precision sensitive, [Scratch] §26.7) and rounded
 *            once to float32; the sum runs in slot order.
 * Requires 1 <= K <= E, E <= MOE_MAX_EXPERTS, K <= MOE_MAX_TOPK. */
moe_status moe_route_topk(const float *logits, int64_t T, int32_t E, int32_t K,
                          int32_t *topk_idx, float *topk_w, hipStream_t stream);

/* Group-limited routing, [Scratch] §21: the experts form G = E / group_size contiguous groups
 * (g = e / group_size; a group stands for a rank or node); the router first keeps the
 * topk_groups groups with the best scores, then picks the top K experts among the experts of
 * those groups only, and the weights are the softmax over the K selected logits exactly as in
 * moe_route_topk. A group's score is its largest logit (the pages define no score: with the
 * maximum, topk_groups = G is plain routing and the token's best expert is always kept); equal
 * scores go to the lower group id. A token's K experts then lie in at most topk_groups groups,
 * so the group dispatch sends each token at most topk_groups times.
 * Requires group_size dividing E, 1 <= topk_groups <= G, K <= topk_groups * group_size
 * (else MOE_ERR_INVALID) and G <= 256 (else MOE_ERR_UNSUPPORTED). */
moe_status moe_route_topk_grouped(const float *logits, int64_t T, int32_t E, int32_t K, int32_t group_size,
                                  int32_t topk_groups, int32_t *topk_idx, float *topk_w, hipStream_t stream);

/* The dispatch "handle" ([Combine] §3: computed once by dispatch, reused by combine).
 * All members are caller-owned device arrays, written by moe_build_index.
 * R = moe_index_rows(...): T*K in the standard and group modes, E*capacity in drop-and-pad
 * mode, T*K + E*(alignment-1) with expert alignment. */
typedef struct moe_index {
    int32_t *counts;         /* [E] rows routed to each expert, before capacity ([Megatron] §1.2
                                num_tokens_per_expert). Required. */
    int32_t *group_list;     /* [E] inclusive running sum of counts ([Scratch] §7:
                                [3,2,4] -> [3,5,9]); in the standard and group modes expert e
                                owns rows [group_list[e]-counts[e], group_list[e]). With expert
                                alignment A the running sum of the aligned lengths
                                ceil(counts/A)*A (expert e's segment ends at group_list[e], its
                                tokens come first, then padding rows). In drop-and-pad mode it
                                stays the running sum of the counts before capacity and
                                describes no row layout: there expert e owns rows
                                [e*capacity, e*capacity + kept_counts[e]), then padding up to
                                (e+1)*capacity. Required. */
    int32_t *kept_counts;    /* [E] min(counts, capacity) in drop-and-pad mode, counts
                                otherwise. May be NULL. */
    int32_t *sorted_indices; /* [R] source token of each expert-major row ([Megatron] §1.1,
                                masked_select over the transposed routing map): experts in
                                ascending order, tokens ascending inside an expert. Padding
                                rows hold MOE_ROW_PAD (-1), rows after the last segment
                                MOE_ROW_UNUSED (-2). Required. */
    int32_t *row_of;         /* [T, K] expert-major row of slot (t,k), -1 if the slot routes
                                nowhere or was dropped (the saved mapping that makes the permute
                                invertible, [Scratch] §26.5). Required. */
    float *permuted_probs;   /* [R] topk_w of the slot in each row ([Megatron] §1.1 step 4),
                                0 on padding/unused rows, 1 if topk_w is NULL. May be NULL. */
    /* group mode only (group_size > 0), else ignored; all required in group mode: */
    int32_t *slot_of;        /* [T, G] slot of (token t, group g) in the send-once list, -1 if
                                token t uses no expert of group g ([CANN] §1(1)). */
    int32_t *gsrc;           /* [T*min(K,G)] source token of each group slot, groups ascending
                                then tokens ascending; only the first n_slots entries are
                                written. */
    int32_t *esrc;           /* [R] group slot feeding each expert-major row; MOE_ROW_PAD on
                                padding rows, MOE_ROW_UNUSED after the last segment. */
    int32_t *group_counts;   /* [G] slots per group. */
    int32_t *n_slots;        /* [1] number of group slots M_g (the caller reads it back if it
                                needs the exact size; gsrc may be sized by the upper bound). */
    int32_t *slot_src;       /* [T, K] group mode, may be NULL (not written): the group slot
                                feeding routing slot (t,k), i.e. slot_of[t, group of its expert]
                                = esrc[row_of[t,k]]; -1 if the slot routes nowhere. The receive
                                side passes it to moe_permute_grouped as src_of, so that each
                                destination's source is known without a lookup. */
} moe_index;

/* Rows R of the expert-major arrays (sorted_indices, permuted_probs, esrc) and buffers for
 * these sizes: E*capacity with capacity > 0, else T*K + E*(alignment-1) (alignment <= 1: T*K),
 * the most that the segments rounded up to a multiple of the alignment can need. Returns -1 for
 * invalid sizes, capacity together with alignment > 1, or R above 2^31 - 1. */
int64_t moe_index_rows(int64_t T, int32_t K, int32_t E, int32_t capacity, int32_t alignment);

/* Bytes of device workspace that moe_build_index needs for these sizes: the tile counts of the
 * experts (and of the groups), at most 128 tiles. The caller allocates it, 16-byte aligned
 * (NULL when the size is 0); its contents need no initialisation and mean nothing after the
 * call. */
moe_status moe_build_index_workspace_size(int64_t T, int32_t K, int32_t E, int32_t group_size,
                                          size_t *bytes);

/* Builds the expert-major index from the routing result ([Megatron] §1.1; [Scratch] §6, §7,
 * §11-13, §16).
 *   topk_idx [T, K] int32 expert ids (-1 or any id outside [0, E) = no expert).
 *   topk_w   [T, K] float32 or NULL (then permuted_probs holds 1 on routed rows).
 *   capacity > 0 selects drop-and-pad ([Scratch] §18, §26.6): expert e owns rows
 *            [e*capacity, (e+1)*capacity); the p-th token of expert e (tokens in ascending
 *            order) is kept at row e*capacity + p iff p < capacity, later ones are dropped
 *            (row_of = -1) and the rest of the expert's rows are padding.
 *   group_size > 0 selects group mode ([CANN] §1(1)): experts e form G = E / group_size
 *            contiguous groups g = e / group_size, and slot_of/gsrc/esrc/group_counts/n_slots
 *            are written. capacity > 0 together with group_size > 0 is MOE_ERR_UNSUPPORTED.
 *   alignment > 1 selects expert alignment ([Combine] §6, dispatch(..., expert_alignment=128)):
 *            each expert segment is rounded up to a multiple of the alignment, its tokens first
 *            and MOE_ROW_PAD rows after them, so that every segment of the grouped GEMM input
 *            starts at a multiple of the alignment; group_list follows the aligned segments.
 *            Not with capacity (MOE_ERR_UNSUPPORTED); 0 or 1 means none.
 * Rows after the last segment are MOE_ROW_UNUSED. The build is deterministic: no position
 * depends on the timing of atomics. */
moe_status moe_build_index(const int32_t *topk_idx, const float *topk_w, int64_t T, int32_t K,
                           int32_t E, int32_t capacity, int32_t group_size, int32_t alignment,
                           const moe_index *out, void *workspace, size_t workspace_bytes,
                           hipStream_t stream);

/* moe_build_index without a workspace argument, for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * tile counts go to a scratch array inside the library instead -- 1 MiB of device memory per GPU,
 * enough for every input moe_build_index accepts (at most 128 tiles of 1024 expert and 1024 group
 * counts), held by each GPU the library runs on until the process ends. Nothing is allocated;
 * arguments, results and errors are those of moe_build_index (bit for bit the same arrays), plus:
 *   - the stream must belong to the current device (else MOE_ERR_INVALID): the scratch used is
 *     the current device's, whose address is looked up on the first call on that device
 *     (MOE_ERR_HIP if that fails);
 *   - a plan larger than the scratch returns MOE_ERR_UNSUPPORTED (no valid input makes one);
 *   - every call on one GPU shares that GPU's scratch: calls on the same stream are ordered, but
 *     calls that overlap on one GPU (different streams, or different host threads without
 *     ordering between their streams) race and may write wrong results. The scratch needs no
 *     clearing: each call writes the counts it reads. */
moe_status moe_build_index_noalloc(const int32_t *topk_idx, const float *topk_w, int64_t T, int32_t K,
                                   int32_t E, int32_t capacity, int32_t group_size, int32_t alignment,
                                   const moe_index *out, hipStream_t stream);

/* Routing and index build in one call ([Scratch] §3, §27: top-k and the softmax over the K
 * selected logits; §7: the per-expert counts behind group_list; [Megatron] §1.1: the index):
 * the same topk_idx, topk_w and moe_index arrays, bit for bit, as moe_route_topk (route_group_size
 * <= 0) or moe_route_topk_grouped(route_group_size, topk_groups) followed by moe_build_index(
 * topk_idx, topk_w, T, K, E, capacity, group_size, alignment, ...). Where moe_build_index would
 * count its tiles in a launch of its own, the workgroups that route a tile count its slots
 * instead, one launch fewer. Arguments are those of the two calls (route_group_size and
 * topk_groups as moe_route_topk_grouped's group_size and topk_groups; group_size is the index's);
 * the workspace (16-byte aligned; contents need no initialisation and mean nothing after the
 * call) must hold moe_route_topk_index_workspace_size bytes. Every argument error of either call
 * is returned before anything is launched. */
moe_status moe_route_topk_index_workspace_size(int64_t T, int32_t K, int32_t E, int32_t group_size, size_t *bytes);
moe_status moe_route_topk_index(const float *logits, int64_t T, int32_t E, int32_t K, int32_t route_group_size,
                                int32_t topk_groups, int32_t *topk_idx, float *topk_w, int32_t capacity,
                                int32_t group_size, int32_t alignment, const moe_index *out, void *workspace,
                                size_t workspace_bytes, hipStream_t stream);

/* Row gather ([Megatron] §1.1 step 5, permuted_input = tokens.index_select(0, sorted_indices);
 * [Scratch] §12, permuted_tokens = tokens[permute_indices]):
 *   dst[i, :] = src[src_row[i], :] copied bit for bit, for i in [0, N); a src_row outside
 *   [0, src_rows) (MOE_ROW_PAD of padding rows) writes a row of zeros, except MOE_ROW_UNUSED,
 *   which leaves row i untouched (this holds for every call that takes a gather map).
 *   src [src_rows, H] of dtype dt, src_row [N] int32, dst [N, H] of dtype dt.
 * Used for the standard dispatch (src_row = sorted_indices, N = R), drop-and-pad (which also
 * zero-fills the padding rows) and the two stages of the group dispatch (src_row = gsrc, then
 * esrc). moe_permute_scatter below computes the same rows reading each source row once. */
moe_status moe_permute(const void *src, int64_t src_rows, int64_t H, moe_dtype dt,
                       const int32_t *src_row, int64_t N, void *dst, hipStream_t stream);

/* The same row copy as moe_permute, taken source-major: each source row is read once and
 * written to every destination that names it, instead of being read again for each destination
 * (with top-k routing a token row feeds K expert rows, [Scratch] §4).
 *   dst_of  [src_rows, J] int32: dst[dst_of[t*J + j], :] = src[t, :] for every entry in [0, N);
 *           other entries (-1) are skipped. J <= MOE_MAX_EXPERTS (one column per expert group
 *           at most); the entries are read 64 at a time, so a wide map costs a little more.
 *   src_row [N] int32 or NULL: rows i with src_row[i] outside [0, src_rows) are written as zeros
 *           (the padding rows of drop-and-pad); NULL writes no zero rows.
 * When dst_of is the inverse of src_row -- row_of and sorted_indices of one moe_index are -- the
 * result is bit for bit that of moe_permute(src, src_rows, H, dt, src_row, N, dst). Every
 * destination row must be named at most once; rows named by neither map are left untouched. */
moe_status moe_permute_scatter(const void *src, int64_t src_rows, int64_t H, moe_dtype dt,
                               const int32_t *dst_of, int32_t J, const int32_t *src_row, int64_t N,
                               void *dst, hipStream_t stream);

/* The row gather of moe_permute, worked through in groups of destination rows: the result is
 * defined by the gather map alone,
 *   dst[r, :] = src[src_row[r], :]   (bit for bit) for every r listed in dst_of,
 *   dst[r, :] = 0                     for every r in [0, N) with src_row[r] outside [0, src_rows),
 * and dst_of only decides which rows are copied together: within one group (a row of dst_of),
 * a source row named by several destinations is read once. This is the receive side of the
 * send-once-per-rank dispatch ([CANN] §1(1)) put back in expert-major order ([Scratch] §11-12,
 * rank-major to expert-major): src = the group buffer, src_row = moe_index.esrc, dst_of =
 * moe_index.row_of (one group per token, J = K), where each group slot feeds every expert of
 * its group that the token chose.
 *   src     [src_rows, H] (dt); src_row [N] int32 (required); dst [N, H] (dt).
 *   dst_of  [M, J] int32 destination rows, J <= 64; entries outside [0, N) are ignored. A row
 *           may be listed more than once (each copy writes the same bytes); rows with a valid
 *           src_row that dst_of never lists are left untouched.
 *   src_of  [M, J] int32 or NULL: the source row of each listed destination, which must equal
 *           src_row[dst_of[m*J + j]] (moe_index.slot_src is that for the group receive); with it
 *           the sources load together with the destinations instead of after them. Its entries
 *           for unlisted columns (dst_of outside [0, N)) are ignored. The result is the same.
 * With dst_of = the inverse of src_row (every row listed), the result equals
 * moe_permute(src, src_rows, H, dt, src_row, N, dst) bit for bit. */
moe_status moe_permute_grouped(const void *src, int64_t src_rows, int64_t H, moe_dtype dt,
                               const int32_t *src_row, int64_t N, const int32_t *dst_of, int64_t M,
                               int32_t J, const int32_t *src_of, void *dst, hipStream_t stream);

/* FP8 dispatch ([Combine] §3: the dispatch sends FP8, the combine stays BF16; the DeepEP
 * dispatch call in [Megatron] passes x together with x_scales, num_scales scale groups per token
 * along the hidden dimension). Each token's row is cut into H / block blocks of `block`
 * consecutive elements; per block
 *   amax = max |x|,  scale = amax / 448 (float32 division; 1 when amax is 0),
 *   q[i] = E4M3 code of x[i] / scale (float32 division, nearest even, saturating at 448),
 * E4M3 being the OCP 8-bit format (bias 7, no infinities, 448 the largest finite value).
 * x must be finite (then |x / scale| exceeds 448 by at most the division's rounding and the
 * code is at most 448 in magnitude).
 *   moe_quantize_fp8: x [T, H] (x_dt float32 or bf16) -> q [T, H] bytes, scales [T, H/block]
 *     float32. block must divide H.
 *   moe_permute_scatter_fp8: the same codes and scales, computed once per source row and
 *     written source-major like moe_permute_scatter: dst[dst_of[t*J+j]] = q[t],
 *     dst_scales[...] = scales[t]; rows with src_row outside [0, src_rows) get zero codes and
 *     zero scales (padding), MOE_ROW_UNUSED rows are left untouched. Equal, bit for bit, to
 *     moe_quantize_fp8 followed by moe_permute_scatter of the codes (MOE_FP8_E4M3) and of the
 *     scales (float32, H / block columns). block must be a power of two in [8, 1024] dividing H
 *     (else MOE_ERR_UNSUPPORTED), J <= MOE_MAX_EXPERTS, src and dst 16-byte aligned.
 * The moved rows then hold half the bytes of bf16 rows; moe_permute / moe_permute_grouped move
 * FP8 rows (and float32 scale rows) as they move any rows. */
moe_status moe_quantize_fp8(const void *x, moe_dtype x_dt, int64_t T, int64_t H, int32_t block, uint8_t *q,
                            float *scales, hipStream_t stream);
moe_status moe_permute_scatter_fp8(const void *src, moe_dtype src_dt, int64_t src_rows, int64_t H, int32_t block,
                                   const int32_t *dst_of, int32_t J, const int32_t *src_row, int64_t N, uint8_t *dst,
                                   float *dst_scales, hipStream_t stream);

/* The receive side of the FP8 group dispatch: FP8 rows and their scale rows moved together, in one
 * launch ([Combine] §3 and the DeepEP dispatch call in [Megatron]: the codes travel with their
 * scales; [CANN] §1(1), [Scratch] §11-12: group slots back to expert-major rows). Bit for bit
 * moe_permute_grouped of the codes (MOE_FP8_E4M3 rows of H bytes) followed by moe_permute_grouped
 * of the scales (float32 rows of H / block values) with the same src_row, dst_of and src_of:
 * every listed row gets its source's codes and scales, every row whose src_row lies outside
 * [0, src_rows) (MOE_ROW_UNUSED excepted) gets zero codes and zero scales.
 *   src [src_rows, H] codes, src_scales [src_rows, H/block] float32, dst [N, H], dst_scales
 *   [N, H/block]; block >= 1 must divide H (else MOE_ERR_INVALID); the other arguments, limits
 *   and errors as in moe_permute_grouped. The group dispatch's receive:
 *   moe_permute_grouped_fp8(codes, scales, ..., moe_index.esrc, R, moe_index.row_of, T, K,
 *   moe_index.slot_src, ...) after moe_permute_scatter_fp8 over moe_index.slot_of. */
moe_status moe_permute_grouped_fp8(const uint8_t *src, const float *src_scales, int64_t src_rows, int64_t H,
                                   int32_t block, const int32_t *src_row, int64_t N, const int32_t *dst_of,
                                   int64_t M, int32_t J, const int32_t *src_of, uint8_t *dst, float *dst_scales,
                                   hipStream_t stream);

/* Unpermute + weighted top-k merge ([Combine] §1: out[t] = sum over the token's top-k experts
 * of probs[t,e] * expert_e(x[t]); [Scratch] §13, §16):
 *   out[t, :] = sum_{k = 0..K-1, row_of[t,k] in [0, y_rows)} w[t,k] * y[row_of[t,k], :]
 * with a float32 accumulator starting at +0 and one fused multiply-add per term in slot order
 * k = 0, 1, ..., K-1 (deterministic: no atomics, no reordering), then stored as float32 or
 * rounded to bf16 (nearest, ties to even).
 *   y      [y_rows, H] expert outputs in expert-major order (dtype y_dt).
 *   row_of [T, K] int32 (moe_index.row_of).
 *   w      [T, K] float32, or NULL for unit weights (the pure-add combine, [Combine] §3).
 *   bias   [T, H] of dtype out_dt, or NULL: the final bias of [Combine] §3, added in float32
 *          after the sum (one addition) before the output is rounded.
 *   out    [T, H] dtype out_dt.
 * K may be up to 1024 here: the group-mode final sum calls it with y = partials,
 * row_of = slot_of, w = NULL and K = G. */
moe_status moe_unpermute_combine(const void *y, moe_dtype y_dt, int64_t y_rows, int64_t H,
                                 const int32_t *row_of, const float *w, const void *bias, int64_t T,
                                 int32_t K, void *out, moe_dtype out_dt, hipStream_t stream);

/* Local pre-combine per group ([CANN] §1(2): the outputs of a token's experts on the same rank
 * are merged with their weights before leaving the rank; here a group of group_size experts
 * stands for a rank). For every (t, g) with s = slot_of[t*G + g] in [0, slots_cap):
 *   partials[s, :] = sum_{k: topk_idx[t,k] in group g, row_of[t,k] in [0, y_rows)}
 *                    w[t,k] * y[row_of[t,k], :]
 * float32, fused multiply-add in slot order, an empty sum being +0. With slot_of from
 * moe_build_index the partials are stored compactly ([n_slots, H], one row per (token,
 * group) that exists); a slot_of numbering every (t, g) gives the dense [T, G, H] layout.
 * Rows of partials not named by slot_of are left untouched.
 *   y [y_rows, H] (y_dt), row_of/topk_idx/w [T, K], slot_of [T, G], partials [slots_cap, H]
 *   of dtype partials_dt: MOE_F32 stores the float32 sums, MOE_BF16 rounds each once to bf16
 *   (nearest, ties to even) -- the BF16 exchange of [Combine] §3 (DeepEP's combine sends BF16),
 *   half the bytes; the final sum then reads bf16 partials. w may be NULL (unit weights). */
moe_status moe_group_precombine(const void *y, moe_dtype y_dt, int64_t y_rows, int64_t H,
                                const int32_t *row_of, const float *w, const int32_t *topk_idx,
                                int64_t T, int32_t K, int32_t E, int32_t group_size,
                                const int32_t *slot_of, int64_t slots_cap, void *partials,
                                moe_dtype partials_dt, hipStream_t stream);

/* Backward of moe_unpermute_combine ([Combine] §4: the combine is linear in the expert outputs,
 * so its backward is the transposed map -- a dispatch of the output gradient back to the expert
 * rows -- and the router gradient reaches only the selected slots):
 *   dy[row_of[t,k], :] = w[t,k] * dout[t, :]   (float32 product, stored as dy_dt)
 *   dw[t, k] = sum_h dout[t,h] * y[row_of[t,k], h]   (float32, summed in a fixed order: each
 *              thread's elements in order, a reduce-scatter butterfly over the wavefront, the
 *              wavefronts in order; 0 for a slot whose row is outside [0, y_rows))
 * and, when src_row is given, every row r of dy with src_row[r] outside [0, T) is written as
 * zeros (padding rows, which fed no output) -- except MOE_ROW_UNUSED rows. Each row of dy must be
 * named by at most one slot; other rows are left untouched.
 *   dout [T, H] (dout_dt); y [y_rows, H] (y_dt; may be NULL when dw is NULL); row_of, w [T, K]
 *   (w NULL: unit weights, dy = dout); src_row [y_rows] (moe_index.sorted_indices) or NULL;
 *   dy [y_rows, H] (dy_dt); dw [T, K] float32 or NULL (not computed).
 * The backward of the dispatch needs no call of its own ([Combine] §4.1): it is the unit-weight
 * combine of the expert-row gradient, moe_unpermute_combine(dxp, ..., row_of, NULL, NULL, ...); in
 * group mode moe_group_precombine with w = NULL followed by the final sum over groups. */
moe_status moe_unpermute_combine_backward(const void *dout, moe_dtype dout_dt, const void *y, moe_dtype y_dt,
                                          int64_t y_rows, int64_t H, const int32_t *row_of, const float *w,
                                          int64_t T, int32_t K, const int32_t *src_row, void *dy, moe_dtype dy_dt,
                                          float *dw, hipStream_t stream);

/* Backward of moe_route_topk's softmax over the K selected logits ([Scratch] §3, §27: the
 * softmax runs over the selected scores; [Combine] §6: only the selected experts carry router
 * gradient, the selection itself being piecewise constant). With w = topk_w, g = d_topk_w:
 *   d_logits[t, topk_idx[t,k]] += w[t,k] * (g[t,k] - sum_j w[t,j] g[t,j])
 * in double (the sum over j in slot order, the slots in order), rounded once to float32; every
 * other logit of the row gets 0. Slots with an id outside [0, E) give nothing.
 *   topk_idx, topk_w, d_topk_w [T, K]; d_logits [T, E] float32, every entry written. */
moe_status moe_route_topk_backward(const int32_t *topk_idx, const float *topk_w, const float *d_topk_w, int64_t T,
                                   int32_t E, int32_t K, float *d_logits, hipStream_t stream);

/* The router's balance loss, beside the routing weights' own gradient: with p[t,:] the softmax of token t's logits over
 * all E experts, n the number of tokens that count and f_e = counts[e] / (n K) each expert's share of the slots,
 *   loss = coef * E * sum_e f_e * (1/n) sum_t p[t,e]      (coef for a router that spreads its tokens evenly; 0 when n = 0)
 *   logits [T, E] float32 (-inf: p = 0; a row with nothing but -inf gives p = 0 throughout); topk_idx [T, K], ids outside
 *   [0, E) count nowhere; token_mask [T] bytes or NULL: tokens with 0 (padding) count nowhere, whatever their logits hold.
 *   loss [1] float32; counts [E] int32: slots of each expert; prob_sum [E] float32: sum_t p[t,e]; tokens [1] int32: n. With
 *   tokens on several ranks counts, prob_sum and tokens are what is summed over the ranks (the loss follows from them).
 * p is float32; its sums are double (eight tokens at a time, and a workgroup's, float32), the loss double, rounded once; no
 * result depends on timing. coef must be finite.
 * T * K <= 2^31 - 1 (else MOE_ERR_UNSUPPORTED). T = 0 writes zeros. The workspace (16-byte aligned, contents need no
 * initialisation and mean nothing after the call) must hold moe_balance_loss_workspace_size bytes; calls that may overlap
 * need one each. */
moe_status moe_balance_loss_workspace_size(int64_t T, int32_t E, size_t *bytes);
moe_status moe_balance_loss(const float *logits, const int32_t *topk_idx, const uint8_t *token_mask, int64_t T, int32_t E,
                            int32_t K, float coef, float *loss, int32_t *counts, float *prob_sum, int32_t *tokens,
                            void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Backward of moe_balance_loss, from its counts and tokens (or their sums over ranks: the gradient is then that of the loss
 * of all ranks' tokens):
 *   d_logits[t,e] = d_loss * coef * (E/n) * p[t,e] * (f_e - sum_j f_j p[t,j])  (+ d_logits_in[t,e])
 * and 0 (+ d_logits_in) for tokens that do not count, and where n <= 0; the counts, piecewise constant, have no gradient. In
 * float32.
 *   d_loss [1] float32 (NULL: 1); d_logits_in [T, E] or NULL: the gradient that reaches the logits by other ways
 *   (moe_route_topk_backward's); d_logits [T, E], which may be d_logits_in and overlaps no other
 *   input. */
moe_status moe_balance_loss_backward(const float *logits, const uint8_t *token_mask, const int32_t *counts,
                                     const int32_t *tokens, const float *d_loss, int64_t T, int32_t E, int32_t K,
                                     float coef, const float *d_logits_in, float *d_logits, hipStream_t stream);

/* Residual addition and RMS norm, the step before an MoE layer's router and dispatch:
 *   h[t,j] = x[t,j] + residual[t,j]   (residual NULL: h = x)
 *   s[t]   = 1 / sqrt(mean_j h[t,j]^2 + eps)
 *   out[t,j] = h[t,j] * s[t] * weight[j]
 * in float32 from the loads to the one rounding of each output: the norm is that of the unrounded
 * float32 sum, also where sum_out stores it as bf16.
 *   x [T, H] (x_dt), residual [T, H] (sum_dt) or NULL, weight [H] (weight_dt); each float32 or bf16;
 *   eps finite, >= 0 (with eps 0 a row of zeros gives NaN; a row whose sum of squares passes float32's
 *   range gives zeros);
 *   sum_out [T, H] (sum_dt) or NULL: h, the new residual; out [T, H] (out_dt); rstd [T] float32 or
 *   NULL: s, for the backward.
 * sum_out may be x or residual, and out may be x or residual, where the types are the same (each
 * element is read before it is written); otherwise outputs overlap nothing.
 * T <= 2^31 - 1 and H <= 2^26 (else MOE_ERR_UNSUPPORTED). */
moe_status moe_add_rmsnorm(const void *x, moe_dtype x_dt, const void *residual, moe_dtype sum_dt,
                           const void *weight, moe_dtype weight_dt, int64_t T, int64_t H, float eps,
                           void *sum_out, void *out, moe_dtype out_dt, float *rstd, hipStream_t stream);

/* moe_add_rmsnorm with its output as the rows of the FP8 dispatch: per block of `block` consecutive
 * elements the scale of moe_quantize_fp8, taken from the float32 values of out (not those of out's type), and
 * the codes of 448 h[t,j] weight[j] / max_k |h[t,k] weight[k]|, in which s has no part: with h in float32, that
 * in float64 up to one rounding to float32. They are moe_quantize_fp8's of the float32 values but for about one
 * in a million, whose value float32's roundings carry over a boundary between two codes there. Blocks whose
 * scale is under 2^-100 have moe_quantize_fp8's codes.
 *   q [T, H] E4M3 codes, scales [T, H/block] float32; out [T, H] (out_dt) or NULL: the rows themselves
 *   too (the router's input). block >= 1 must divide H (else MOE_ERR_INVALID). A block that holds a NaN
 *   or an infinity has unspecified codes. The other arguments as in moe_add_rmsnorm; q and scales overlap
 *   no input. */
moe_status moe_add_rmsnorm_fp8(const void *x, moe_dtype x_dt, const void *residual, moe_dtype sum_dt,
                               const void *weight, moe_dtype weight_dt, int64_t T, int64_t H, float eps,
                               int32_t block, void *sum_out, void *out, moe_dtype out_dt, uint8_t *q,
                               float *scales, float *rstd, hipStream_t stream);

/* Backward of moe_add_rmsnorm, given its h (sum_out, or x without a residual) and s (rstd): with
 * a = dout * weight and m[t] = s[t]^2 * mean_j a[t,j] h[t,j],
 *   dx[t,j]    = s[t] * (a[t,j] - h[t,j] * m[t]) + d_sum[t,j]   (the gradient of x and of residual alike)
 *   dweight[j] = sum_t dout[t,j] * h[t,j] * s[t]
 * in float32, summed in an order that depends on the sizes alone (no atomics).
 *   dout [T, H] (dout_dt), h [T, H] (h_dt), d_sum [T, H] (dx_dt) or NULL: the gradient that reaches
 *   sum_out by other ways; dx [T, H] (dx_dt), which may be d_sum and overlaps no other input;
 *   dweight [H] float32 or NULL (not computed). T = 0 writes zeros to dweight.
 * The workspace (16-byte aligned, contents need no initialisation; needed with dweight only) must hold
 * moe_add_rmsnorm_backward_workspace_size bytes. */
moe_status moe_add_rmsnorm_backward_workspace_size(int64_t T, int64_t H, size_t *bytes);
moe_status moe_add_rmsnorm_backward(const void *dout, moe_dtype dout_dt, const void *h, moe_dtype h_dt,
                                    const void *weight, moe_dtype weight_dt, const float *rstd,
                                    const void *d_sum, int64_t T, int64_t H, void *dx, moe_dtype dx_dt,
                                    float *dweight, void *workspace, size_t workspace_bytes,
                                    hipStream_t stream);

/* The whole MoE layer for a few tokens (a decode step), from hidden rows to combined rows: the router's
 * product, moe_route_topk, each chosen expert's gated products and the weighted merge, without the
 * dispatched and permuted rows in between ([Scratch] §3, §16 for the routing and the merge):
 *   logits[t,e] = sum_j x[t,j] router[e,j]   summed in double, rounded once to float32
 *   topk_idx, topk_w as moe_route_topk of them (route_group_size > 0: moe_route_topk_grouped, with its
 *              limits)
 *   h[t,k,:] = topk_w[t,k] * silu(G_e x[t]) * (U_e x[t]),   e = topk_idx[t,k], silu(g) = g / (1 + exp(-g))
 *   out[t,:] = sum_k D_e h[t,k,:] (+ bias[t,:])
 * where w_gate_up [E, 2I, H] holds G_e in rows [0, I) and U_e in rows [I, 2I) of expert e, and w_down
 * [E, H, I] holds D_e. Sums are float32 (no atomics: their order depends on the sizes, the routing and the
 * alignment of the arrays alone), h is kept to 16 significant bits or more, and out is rounded once.
 *   x [T, H] and router [E, H] of dtype dt (float32 or bf16); bias [T, H] of dtype out_dt or NULL, which
 *   may be out itself; out [T, H] (out_dt), which overlaps no other input; topk_idx [T, K], topk_w [T, K] out.
 *   weight_dt: dt, or MOE_FP8_E4M3 beside bf16 rows: codes with float32 scales, one per row and block of
 *   `block` consecutive elements of the row, as moe_quantize_fp8 of the weight rows gives them
 *   (gate_up_scales [E, 2I, H/block], down_scales [E, H, I/block]); block must divide H and I (else
 *   MOE_ERR_INVALID) and be a multiple of 128 (else MOE_ERR_UNSUPPORTED). Other types of weights:
 *   MOE_ERR_UNSUPPORTED; block and scales are ignored without FP8.
 *   K <= E (else MOE_ERR_INVALID); T <= MOE_MAX_FEW_TOKENS, H and I <= 2^20 (else MOE_ERR_UNSUPPORTED): for more
 *   tokens dispatch them.
 * Weights of experts that no token uses are not read. Rows are independent: what is not finite in one token's row
 * or in an expert's weights reaches only the tokens that use it. A row whose logits are NaN may route anywhere or
 * nowhere, and an infinite element of a bf16 w_down may give NaN where the formula gives an infinity.
 * The workspace (16-byte aligned, contents need no initialisation and mean nothing after the call) must
 * hold moe_few_token_workspace_size bytes; calls that may overlap need one each. */
moe_status moe_few_token_workspace_size(int64_t T, int64_t H, int64_t I, int32_t E, int32_t K, size_t *bytes);
moe_status moe_few_token_layer(const void *x, moe_dtype dt, const void *router, int64_t T, int64_t H, int64_t I,
                               int32_t E, int32_t K, int32_t route_group_size, int32_t topk_groups,
                               const void *w_gate_up, const void *w_down, moe_dtype weight_dt,
                               const float *gate_up_scales, const float *down_scales, int32_t block,
                               const void *bias, void *out, moe_dtype out_dt, int32_t *topk_idx, float *topk_w,
                               void *workspace, size_t workspace_bytes, hipStream_t stream);

/* The experts of moe_few_token_layer after a routing that the caller has: topk_idx [T, K] (an id outside
 * [0, E) routes nowhere, so a rank can name the experts it does not hold -1; an id may repeat within a row, each slot
 * counting), topk_w [T, K] or NULL (unit weights). A token without experts gets zeros (or its bias). E is the number of
 * experts whose weights are given, and may be less than K <= MOE_MAX_TOPK.
 * Arguments, limits and workspace otherwise as above; its size is moe_few_token_experts_workspace_size's, which is
 * moe_few_token_workspace_size's where K <= E. */
moe_status moe_few_token_experts_workspace_size(int64_t T, int64_t H, int64_t I, int32_t E, int32_t K, size_t *bytes);
moe_status moe_few_token_experts(const void *x, moe_dtype dt, int64_t T, int64_t H, int64_t I, int32_t E,
                                 int32_t K, const int32_t *topk_idx, const float *topk_w, const void *w_gate_up,
                                 const void *w_down, moe_dtype weight_dt, const float *gate_up_scales,
                                 const float *down_scales, int32_t block, const void *bias, void *out,
                                 moe_dtype out_dt, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Rows in microscaled 4-bit floating point (the OCP MX format MXFP4): each 32 consecutive elements of a row share a scale, a
 * power of two, and an element is one of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} times it:
 *   amax = max |x|, scale = 2^(floor(log2 amax) - 2), but at least 2^-127; 1 when amax is 0
 *   code = the nearest of those values to x / scale (a tie goes to the even code, what is above 6 to 6; the sign is kept)
 *   x [T, H] (x_dt float32 or bf16); H a multiple of 32 (else MOE_ERR_INVALID), at most 2^26;
 *   T * H / 8 <= 2^32 - 2^8 for float32, T * H / 32 for bf16 (else MOE_ERR_UNSUPPORTED).
 *   q [T, H/2] bytes: two codes each, the even element's in the low half. scales [T, H/32] bytes: the exponent + 127; 255
 *   (which stands for NaN) for a block that holds a NaN or an infinity, whose codes are 0.
 * Both are byte rows that the permutes move as MOE_FP8_E4M3 rows of H/2 and H/32 elements; they overlap neither x nor each other. */
moe_status moe_quantize_mxfp4(const void *x, moe_dtype x_dt, int64_t T, int64_t H, uint8_t *q, uint8_t *scales,
                              hipStream_t stream);

/* Each expert's product of its rows with its weights, between dispatch and combine ([Scratch] §11-13: the grouped product over
 * expert-major rows; [Combine] §6 for aligned segments), both operands as moe_quantize_mxfp4's rows:
 *   y[r, :] = W_e X[r]  for the rows r of expert e's segment; float32 sums, no atomics, an order that depends on the sizes alone
 *   out[r, n] = y[r, n], or with gated != 0: silu(y[r, n]) * y[r, N + n],  silu(g) = g / (1 + exp(-g)); rounded once
 *   w [E, N, H/2], w_scales [E, N, H/32]; gated: [E, 2N, ...], expert e's gate rows first, then its up rows.
 *   X[r] is row r of x, or row src_row[r] of it (a row of zeros where that is outside [0, x_rows)): with
 *   moe_index.sorted_indices the token rows need not be dispatched first. x [x_rows, H/2], x_scales [x_rows, H/32];
 *   src_row [R] or NULL (then x_rows >= R).
 *   Segments: group_list [E] is moe_index.group_list, expert e's rows ending before group_list[e] and beginning where the
 *   previous expert's end; with counts [E] (may be NULL) only the first counts[e] of them (moe_index.counts with expert
 *   alignment: the padding rows take no part). capacity > 0 is the drop-and-pad layout: the first counts[e]
 *   (moe_index.kept_counts) rows from e * capacity, group_list is not read, R >= E * capacity.
 *   out [R, N] (float32 or bf16), which overlaps no input. Rows in no segment are left untouched. Segments are cut to [0, R);
 *   ones that overlap give unspecified rows.
 * R and E choose the kernel, and R counts rows that take no part too: segments aligned to 8 and more, or of a capacity past 8, take
 * calls with few tokens off the kernel for few rows (one token twice the time, 64 tokens a fifth more).
 * Rows are independent: a NaN scale makes NaN of its own row or column alone. H a multiple of 32 (else MOE_ERR_INVALID);
 * H, N <= 2^20, x and w 16-byte aligned (else MOE_ERR_UNSUPPORTED, as for a launch that would pass 2^32 threads: R * N from 2^38
 * on, or up to 8 rows of each of more than 680 experts with some 2^20 columns). */
moe_status moe_grouped_product_mxfp4(const uint8_t *x, const uint8_t *x_scales, int64_t x_rows, const int32_t *src_row,
                                     int64_t R, int64_t H, const uint8_t *w, const uint8_t *w_scales, int32_t E, int64_t N,
                                     int32_t gated, const int32_t *group_list, const int32_t *counts, int32_t capacity,
                                     void *out, moe_dtype out_dt, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DISPATCH_H */
