/*
 * moe_ep.h -- C ABI of the MI355X (gfx950) MoE expert-parallel layout,
 * dispatch and combine library (libmoe_ep.so).
 *
 * The three calls are the data-parallel hot path of expert parallelism:
 *
 *   moe_layout    top-k routing -> per-expert / per-rank counts, padded segment
 *                 offsets, and the maps between (token, k) entries and rows of
 *                 the receive buffer.
 *   moe_dispatch  token rows -> rows of the expert-grouped, rank-partitioned
 *                 receive buffer, bit-copied bf16 or FP8 E4M3 with one fp32
 *                 scale per 128 channels.
 *   moe_combine   expert output rows -> token order, as the route-weighted sum
 *                 of each token's K rows (fp32 accumulation), plus an optional
 *                 shared-expert output.
 *
 * Before the layout, moe_router turns a router's logits into the top-k routing
 * and its weights, with the load-balance loss and the gradients
 * (moe_balance_loss, moe_router_backward).  Between dispatch and combine,
 * moe_dispatch_mx4 carries the rows in microscaled 4-bit floating point
 * (MXFP4), moe_quantize_mx4 / moe_dequantize_mx4 convert rows, and
 * moe_expert_gemm_mx4 multiplies every expert's rows with its weights.  The same
 * in 8-bit integers: moe_dispatch_i8, moe_quantize_i8 / moe_dequantize_i8,
 * moe_expert_gemm_i8.  In bf16, with what training needs: moe_expert_gemm,
 * moe_expert_gemm_backward_x / _w, moe_combine_backward.
 *
 * Around them: moe_layout_dispatch (layout + dispatch in one launch for
 * decode-sized batches), moe_layout_balanced (every rank receives the same
 * number of rows through redundant-expert slots), moe_zero_padding (optional
 * zero fill of padding rows), moe_stream_create_cu_limited /
 * moe_stream_create_cu_range / moe_stream_destroy (a stream confined to a set
 * of CUs), and the sizing helpers
 * moe_max_recv_rows, moe_layout_workspace_bytes,
 * moe_layout_balanced_workspace_bytes, plus moe_status_str.
 *
 * What the operations are (passages):
 *   - Experts of a layer are spread over the ranks of an EP group; E must
 *     divide by the group size R and each rank holds E/R local experts
 *     (delect.ru glossary "Expert parallelism (EP)", confirmed facts: the
 *     DeepSpeed v0.14.5 example, 8 experts on 4 ranks).  Rank r owns experts
 *     [r*E/R, (r+1)*E/R) (MoonEP article, section 3 and Fig. 3: rows [0,E) of
 *     the weight buffer hold every rank's local experts in order).
 *   - Activations travel to the experts and the results travel back and are
 *     merged (same glossary, the MOELayer.forward fact); the all-to-all pair
 *     is called dispatch and combine (DeepEP analysis, "DeepEP introduction").
 *   - Dispatch sends FP8, combine returns BF16 (DeepEP analysis, feature list
 *     and the set-up of both benchmark tables).
 *   - Each token is written straight into its final expert-grouped row on the
 *     receiving rank; static shapes avoid any per-layer host sync (MoonEP
 *     article, section 2, "zero copy" and static layout).  Per-expert padding
 *     to a static shape (search-results page, the dynamic-routing snippet:
 *     drop tokens or zero-pad; MoonEP basic usage, token_padding=128).
 *
 * The R ranks of one EP group are simulated on one GPU as rank-major
 * partitions of one receive buffer: partition r is exactly what GPU r would
 * receive.
 *
 * Conventions for every call:
 *   - All array arguments are DEVICE pointers, row-major and contiguous, owned
 *     by the caller; the library never allocates, frees or keeps them.
 *     Descriptor structs are HOST pointers read during the call only.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = the null stream) and
 *     runs asynchronously; no call copies device -> host or synchronises.
 *   - Argument errors are returned synchronously, before anything is
 *     enqueued.  Data errors (an expert id outside [0,E), a capacity
 *     overflow) are found on the device and written to layout->status[0].
 *   - The library holds no global state: calls are reentrant and thread safe.
 *     Calls on one stream run in order; calls on different streams that share
 *     output buffers race.
 *   - Limits: 0 <= S, 1 <= K <= 16, 1 <= E <= 1024, R divides E,
 *     S*K and every row count below 2^31; dispatch: S*ceil(H/512) (bf16) or
 *     S*ceil(H/1024) (FP8) below 2^31, S*ceil(H/2048) (MXFP4) below 2^26;
 *     combine: S*ceil(H/512) below 2^31.  Offsets inside every array are 64-bit.
 *     The router's, the conversions' and the products' stand at their calls.
 */
#ifndef MOE_EP_H
#define MOE_EP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_NULL = 1,      /* a required pointer is NULL */
    MOE_ERR_SHAPE = 2,     /* a size or mode is outside the limits above */
    MOE_ERR_ALIGN = 3,     /* a row buffer is not 16-byte aligned */
    MOE_ERR_WORKSPACE = 4, /* workspace missing or smaller than required */
    MOE_ERR_HIP = 5        /* the HIP runtime refused a launch */
} moe_status;

/* How each expert's segment of the receive buffer is sized. */
typedef enum {
    MOE_PAD_NONE = 0,      /* exactly the expert's entries */
    MOE_PAD_MULTIPLE = 1,  /* rounded up to a multiple of pad_rows (0 stays 0) */
    MOE_PAD_CAPACITY = 2   /* exactly pad_rows; entries beyond are not placed */
} moe_pad_mode;

/* Bits of layout->status[0]. */
enum {
    MOE_FLAG_BAD_EXPERT = 1, /* some topk_idx outside [0,E); that entry got pos = -1 */
    MOE_FLAG_CAPACITY = 2    /* some expert had more than pad_rows entries (CAPACITY);
                                the entries past the capacity got pos = -1 */
};

/* Shape of one batch (host struct). */
typedef struct {
    int32_t S;        /* tokens */
    int32_t K;        /* experts per token */
    int32_t E;        /* experts */
    int32_t R;        /* EP ranks; rank r owns experts [r*E/R, (r+1)*E/R) */
    int32_t pad_mode; /* moe_pad_mode */
    int32_t pad_rows; /* multiple or capacity; ignored for MOE_PAD_NONE */
} moe_layout_desc;

/* The layout of one batch: outputs of moe_layout, inputs of dispatch and
 * combine (host struct holding device pointers, all int32). */
typedef struct {
    int32_t *tokens_per_expert; /* [E]   rows placed in each expert's segment */
    int32_t *tokens_per_rank;   /* [R]   rows placed in each rank's partition */
    int32_t *expert_offset;     /* [E+1] first row of each expert's segment; [E] = rows used */
    int32_t *rank_offset;       /* [R+1] first row of each rank's partition */
    int32_t *pos;               /* [S*K] row of entry (t,k) at t*K+k, or -1 */
    int32_t *src;               /* [moe_max_recv_rows] entry t*K+k held by each row, -1 if none */
    int32_t *status;            /* [1]   MOE_FLAG_* of this batch (overwritten) */
} moe_layout_bufs;

/* Rows the receive buffer (and src) must hold for ANY routing of this shape:
 * S*K (NONE), S*K + E*(pad_rows-1) (MULTIPLE), E*pad_rows (CAPACITY).
 * Host only.  Returns -1 if the shape is invalid. */
int64_t moe_max_recv_rows(const moe_layout_desc *desc);

/* Device workspace bytes moe_layout needs for this shape: 0 when
 * S*K <= 32768 (those batches run as one launch with no scratch), else one
 * histogram of E counts per tile.  Host only.  Returns 0 for an invalid shape
 * too; moe_layout then reports MOE_ERR_SHAPE. */
size_t moe_layout_workspace_bytes(const moe_layout_desc *desc);

/* Layout of one batch from its top-k routing.
 *   topk_idx  [S,K] int32 device: expert of entry (t,k).
 *   out       every pointer required; src has moe_max_recv_rows entries.
 *   workspace device scratch of at least moe_layout_workspace_bytes (may be
 *             NULL when that is 0); 16-byte aligned; contents need no init.
 * Inside each expert's segment, rows follow ascending t*K+k (stable); ranks
 * and experts appear in ascending order (rank-major).  Padding rows are not
 * touched in the row buffers; their src is -1. */
moe_status moe_layout(const moe_layout_desc *desc, const int32_t *topk_idx,
                      const moe_layout_bufs *out, void *workspace, size_t workspace_bytes,
                      void *stream);

/* moe_layout without a workspace argument, for callers that cannot allocate
 * device memory (code under graph capture, tight serving loops, harnesses that
 * forbid allocation).  Same results as moe_layout.  The two-launch form
 * (S*K > 32768) keeps its per-tile histograms in a device array inside the
 * library, 4 MiB per GPU, held from the first call on a GPU until the process
 * ends: MOE_ERR_WORKSPACE when moe_layout_workspace_bytes exceeds 4 MiB (about
 * 4M entries at E = 1024, 16M at E = 256).  Every call on one GPU shares that
 * array, so calls that overlap in time on one GPU (other streams, other host
 * threads) race; calls on one stream are fine.  The array needs no clearing:
 * each call writes every histogram and flag it reads.  The current device must
 * be the stream's device.  No allocation, free or host sync. */
moe_status moe_layout_noalloc(const moe_layout_desc *desc, const int32_t *topk_idx,
                              const moe_layout_bufs *out, void *stream);

/* Dispatch: row pos[t,k] of the receive buffer gets token t's hidden row.
 *   hidden      [S,H] bf16 device, 16-byte aligned, H % 8 == 0.
 *   topk_idx    [S,K] int32; the expert ids already folded into `layout`
 *               (kept for the calling convention; may be NULL).
 *   topk_w      [S,K] fp32 or NULL; with recv_w, recv_w[pos[t,k]] = topk_w[t,k].
 *   fp8 == 0    recv [max_recv,H] bf16 gets the row bit for bit.
 *   fp8 != 0    H % 128 == 0; recv [max_recv,H] E4M3FN bytes and recv_scales
 *               [max_recv,H/128] fp32: per 128-channel block b of token t,
 *               scale = amax/448 (fp32 division, amax = max |x|) and
 *               code = E4M3FN(x/scale) (fp32 division, round to nearest even,
 *               saturating at +-448); an all-zero block has scale 0 and codes 0.
 *   recv_w      [max_recv] fp32 or NULL.
 * Rows that no entry maps to (padding, unused tail) are not written. */
moe_status moe_dispatch(const moe_layout_desc *desc, const moe_layout_bufs *layout,
                        const void *hidden, int32_t H, const int32_t *topk_idx,
                        const float *topk_w, int32_t fp8, void *recv, float *recv_scales,
                        float *recv_w, void *stream);

/* Layout + dispatch in one call: the same results as moe_layout followed by
 * moe_dispatch with these arguments (every output of both).  Batches with
 * S*K <= 4096 and S <= 512 (decode-sized) run as ONE kernel launch in which
 * each workgroup rebuilds the layout counts it needs in LDS; other batches run
 * the two calls' kernels back to back.  Arguments as in moe_layout and moe_dispatch; the
 * workspace rule is moe_layout's.  This is the low-latency variant for
 * inference decoding (DeepEP analysis, feature list: low-latency kernels for
 * decoding). */
moe_status moe_layout_dispatch(const moe_layout_desc *desc, const int32_t *topk_idx,
                               const moe_layout_bufs *out, void *workspace, size_t workspace_bytes,
                               const void *hidden, int32_t H, const float *topk_w, int32_t fp8,
                               void *recv, float *recv_scales, float *recv_w, void *stream);

/* Combine: out[t,c] = bf16_rne( (fma chain over k = 0..K-1 of
 *                                w[t,k] * expert_out[pos[t,k], c], from +0.0)
 *                               + shared_out[t,c] ).
 *   expert_out  [max_recv,H] bf16 device, 16-byte aligned, H % 8 == 0; only rows
 *               some pos[t,k] points to are read.
 *   w           [S,K] fp32 in token order, or NULL for weight 1.
 *   shared_out  [S,H] bf16 or NULL (then nothing is added).
 *   out         [S,H] bf16, 16-byte aligned.
 * Entries with pos = -1 are skipped: their expert_out row is not read. */
moe_status moe_combine(const moe_layout_desc *desc, const moe_layout_bufs *layout,
                       const void *expert_out, int32_t H, const float *w,
                       const void *shared_out, void *out, void *stream);

/* Zero padding (optional, after dispatch): clears every receive row that no
 * entry maps to -- src[r] = -1: padding inside the segments and the unused
 * tail -- so a consumer that runs over whole padded segments reads zeros
 * there (search-results page, the snippet on the limits of dynamic routing:
 * drop tokens or zero-pad).  Dispatch itself never writes those rows.
 *   layout      moe_layout's output for this batch (its src is read).
 *   H, fp8      as given to moe_dispatch.
 *   recv        [max_recv,H] bf16 or E4M3 bytes, 16-byte aligned.
 *   recv_scales [max_recv,H/128] fp32 (required when fp8, ignored otherwise);
 *               scale rows of cleared rows become 0.0f.
 * Rows that hold an entry are not written.  Cost: one write of every padding
 * row (at the decode shape 31,744 rows x 7 KB). */
moe_status moe_zero_padding(const moe_layout_desc *desc, const moe_layout_bufs *layout, int32_t H, int32_t fp8,
                            void *recv, float *recv_scales, void *stream);

/* Balanced layout: every rank receives the same number of rows (N/R, the
 * first N%R ranks one more; N = entries with a valid expert) however skewed
 * the routing, through redundant copies of experts held in per-rank slots --
 * the perfect-balance scheme of the MoonEP article (section 1: a few
 * redundant experts planned online; section 3, Fig. 3: each rank's local
 * experts followed by B prefetch slots).  The planning rule (the pages give
 * none): overloaded ranks in ascending order shed their surplus from their
 * largest experts first (ties: lower id); each piece goes to the lowest rank
 * still below its quota that has a free slot, as much as its room allows;
 * each (expert, destination) piece takes one slot; an expert's first entries
 * (t*K+k order) stay home, later ones fill its replicas in creation order.
 * If slots run out the rest stays home and status bit 4 is set.
 *   desc       pad_mode must be MOE_PAD_NONE; rows used <= S*K (src has S*K).
 *   slots_per_rank  B, 0..64, R*B <= 512.
 *   out        as moe_layout; expert_offset[e] = first row of e's home segment,
 *              expert_offset[E] = rows used; tokens_per_rank = rows per rank.
 *   bal        seg_offset [R*(E/R+B)+1]: first row of each (rank, segment),
 *              segments per rank = its E/R experts then its B slots;
 *              slot_expert [R*B]: expert copied in each slot, -1 if unused
 *              (the weights a rank must hold in that slot).
 *   workspace  at least moe_layout_balanced_workspace_bytes, 256-byte aligned;
 *              that is 0 for S*K <= 32768 (one launch, no scratch), and
 *              workspace may then be NULL.
 * pos/src are ordinary maps, so moe_dispatch and moe_combine take this
 * layout unchanged. */
enum { MOE_FLAG_UNBALANCED = 4 };
typedef struct {
    int32_t *seg_offset;  /* [R*(E/R+B)+1] */
    int32_t *slot_expert; /* [R*B] */
} moe_balance_bufs;
size_t moe_layout_balanced_workspace_bytes(const moe_layout_desc *desc, int32_t slots_per_rank);
moe_status moe_layout_balanced(const moe_layout_desc *desc, int32_t slots_per_rank,
                               const int32_t *topk_idx, const moe_layout_bufs *out,
                               const moe_balance_bufs *bal, void *workspace, size_t workspace_bytes,
                               void *stream);

/* CU budget for overlap: a new stream whose kernels may run only on
 * `num_cus` compute units, num_cus / (number of XCDs) on every XCD (default
 * priority).  Launching layout / dispatch / combine on it leaves
 * the other CUs to concurrent work, the AMD form of DeepEP's control of the
 * number of SMs its kernels occupy (DeepEP analysis, feature list and the
 * "normal kernels" paragraph; MoonEP basic usage, num_sms=32).  Results do not
 * depend on the budget.  Host call: touches the HIP runtime of the current
 * device, allocates the stream; release it with moe_stream_destroy.
 * MOE_ERR_SHAPE if num_cus is outside [1, CU count] or not a multiple of the
 * XCD count (8 on MI355X). */
moe_status moe_stream_create_cu_limited(int32_t num_cus, void **stream_out);

/* The same with the CU set placed: CUs [first_cu, first_cu + num_cus) in the
 * queue-mask numbering (CU i is on XCD i % XCD count), so two streams with
 * disjoint ranges split the chip -- e.g. layout / dispatch / combine on one
 * half and expert compute on the other.  first_cu and num_cus must be
 * multiples of the XCD count, the range within the CU count; else
 * MOE_ERR_SHAPE.  moe_stream_create_cu_limited(n) is the range [0, n). */
moe_status moe_stream_create_cu_range(int32_t first_cu, int32_t num_cus, void **stream_out);
moe_status moe_stream_destroy(void *stream);

/* ---------------------------------------------------------------------------
 * Router: logits -> top-k routing, load-balance loss, gradients
 * ------------------------------------------------------------------------- */

/* Types of the router's logits and of their gradient. */
typedef enum {
    MOE_F32 = 0,
    MOE_BF16 = 1
} moe_dtype;

/* A router's shape and rule (host struct). */
typedef struct {
    int32_t S;           /* tokens */
    int32_t E;           /* experts */
    int32_t K;           /* experts per token, K <= E */
    int32_t n_groups;    /* experts form n_groups groups of E/n_groups consecutive ids (1..64, divides E) */
    int32_t topk_groups; /* a token's picks come from its topk_groups best groups (n_groups: from all) */
    int32_t renorm;      /* 0: weights are the picks' probabilities; 1: the softmax over the picks alone */
    int32_t seq_len;     /* tokens per sequence of the balance loss (divides S); 0: the whole batch is one */
    float alpha;         /* factor of the balance loss */
} moe_router_desc;

/* What moe_router and moe_balance_loss write (host struct of device pointers).
 * G = number of sequences: S/seq_len, 1 for seq_len = 0.  expert_count,
 * balance_coef and balance_loss go together: all three, or none of them (a
 * serving call of moe_router, which then needs no workspace). */
typedef struct {
    int32_t *topk_idx;     /* [S,K] expert of each pick, descending logit; -1 where there is none */
    float *topk_w;         /* [S,K] route weights; 0 where there is no pick */
    int32_t *expert_count; /* [G,E] picks of each expert, per sequence */
    float *balance_coef;   /* [G,E] d balance_loss / d (a token's probability of e) */
    float *balance_loss;   /* [1] */
} moe_router_bufs;

/* Device workspace bytes of moe_router (when it writes the loss) and of
 * moe_balance_loss.  Host only; 0 for an invalid shape.  Its contents carry
 * nothing from call to call, but calls (or graph replays) that may overlap in
 * time need a workspace, and outputs, each. */
size_t moe_router_workspace_bytes(const moe_router_desc *desc);

/* Router: top-k routing of one batch (the gate in front of the layout), in the
 * group-limited form of the DeepEP analysis, "normal kernels" set-up (a
 * token's experts come from its best groups), and optionally the balance loss.
 *   logits      [S,E] fp32 or bf16 (logits_type); computed in fp32.
 *   token_mask  [S] bytes or NULL: 0 = the token does not count (padding of the
 *               batch); what its logits hold is not looked at.
 * A token counts if its mask lets it and some logit is above -inf (a logit of
 * -inf marks an expert that cannot be picked).  With p = softmax of a counting
 * token's logits (0 for other tokens):
 *   picks    the group score is the group's highest logit; of the topk_groups
 *            best groups' experts the K highest logits, in descending order;
 *            ties go to the lower index throughout.  Experts at -inf are never
 *            picked: entries left over are -1 with weight 0, as are all of a
 *            token that does not count (moe_layout places no row for them).
 *   weights  renorm != 0: softmax over the token's picks; else p of the pick.
 *   loss     per sequence, with n counting tokens and c_e picks of expert e:
 *            alpha * sum_e (E*c_e/(K*n)) * (sum_t p[t,e] / n), averaged over
 *            the sequences with n > 0 (0 if there is none).  coef_e =
 *            alpha*E*c_e/(K*n*n*sequences), 0 in a sequence with n = 0.
 * A counting token with a NaN or +inf logit is not routed (picks -1, weights
 * 0), and its probabilities are NaN: so is the loss, and its row of the
 * gradient.  The results do not depend on the order in which work runs.
 * No alignment beyond the element types' is needed; workspace 16 bytes.
 * MOE_ERR_SHAPE where a launch cannot number the work; it always can with fewer
 * than 2^26 - 4 tokens and, for the loss, sequences * ceil(E/32) and
 * sequences * min(ceil(T/16), 256) below 2^22, T tokens in a sequence. */
moe_status moe_router(const moe_router_desc *desc, const void *logits, int32_t logits_type, const uint8_t *token_mask,
                      const moe_router_bufs *out, void *workspace, size_t workspace_bytes, void *stream);

/* The balance loss and per-expert counts of a routing that the caller made:
 *   topk_idx  [S,K] int32; ids outside [0,E) count for nothing, an expert that
 *             a token names twice counts twice; picks of tokens that do not
 *             count are not counted.
 * Writes expert_count, balance_coef and balance_loss as moe_router does
 * (out->topk_idx and out->topk_w are not looked at); n_groups, topk_groups and
 * renorm are checked but change nothing, and K may exceed E.  Gradient:
 * moe_router_backward without d_topk_w. */
moe_status moe_balance_loss(const moe_router_desc *desc, const void *logits, int32_t logits_type,
                            const int32_t *topk_idx, const uint8_t *token_mask, const moe_router_bufs *out,
                            void *workspace, size_t workspace_bytes, void *stream);

/* Gradient with respect to the logits, in the logits' type; d_logits is
 * overwritten (0 for tokens that do not count) and may be the logits' own
 * buffer.  Two parts, at least one given:
 *   balance_coef, d_loss ([1] fp32)  d_loss * p * (coef - sum_j coef_j p_j)
 *   topk_idx, topk_w, d_topk_w ([S,K] fp32)  with inner = sum_k d_k w_k over
 *     the picks: renorm: w_k*(d_k - inner) at each pick; else
 *     p_e*(d of the pick of e, if any, - inner) at every expert.
 * logits, token_mask, topk_* and balance_coef as moe_router had and wrote
 * them; d_topk_w of an entry without a pick is not looked at. */
moe_status moe_router_backward(const moe_router_desc *desc, const void *logits, int32_t logits_type,
                               const uint8_t *token_mask, const int32_t *topk_idx, const float *topk_w,
                               const float *balance_coef, const float *d_topk_w, const float *d_loss, void *d_logits,
                               void *stream);

/* ---------------------------------------------------------------------------
 * MXFP4: rows in microscaled 4-bit floating point, and the experts' products
 * ------------------------------------------------------------------------- */

/* An MXFP4 row of H channels (H % 128 == 0; OCP microscaling formats, E2M1
 * elements with E8M0 scales for 32 channels):
 *   codes   H/2 bytes, channel 2i in the low half of byte i; sign bit, then
 *           magnitude 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *   scales  H/32 bytes, 2^(byte - 127) for 32 consecutive channels, 255 = NaN.
 * Rounding a bf16 row: per block, byte = floor(log2(amax)) - 2 + 127, at least
 * 0; code = x / 2^(byte - 127) to the nearest magnitude, ties to the even code,
 * saturating at 6, x's sign kept.  A block of zeros has byte 0 and codes that
 * are 0 but for the signs; a block with a NaN or an infinity has byte 255 and
 * codes 0. */

/* bf16 rows -> MXFP4 rows (an activation between two products, or an expert's
 * weights, laid out once).
 *   x       [rows,H] bf16, 16-byte aligned.
 *   src     [rows] or NULL: with a layout's src only the rows that hold an
 *           entry (src[r] >= 0) are read and written.
 *   codes   [rows,H/2], 16-byte aligned; scales [rows,H/32] (any alignment).
 * rows * H at most 2^37 - 8192. */
moe_status moe_quantize_mx4(const void *x, int64_t rows, int32_t H, const int32_t *src, void *codes, uint8_t *scales,
                            void *stream);

/* MXFP4 rows -> bf16.  Exact, but for the values past bf16's range, 2^128 and
 * more (scale byte 253 with 4 and 6, 254 with 2 and more; moe_quantize_mx4 writes
 * neither), which become infinities; a block of scale 255 gives NaN.  Arguments
 * and limit as in moe_quantize_mx4: rows with src[r] < 0 are neither read nor
 * written. */
moe_status moe_dequantize_mx4(const void *codes, const uint8_t *scales, int64_t rows, int32_t H, const int32_t *src,
                              void *out, void *stream);

/* moe_dispatch in MXFP4: row pos[t,k] of the receive buffer gets token t's row
 * as moe_quantize_mx4 rounds it: a little over half of the FP8 dispatch's
 * bytes per row.  H % 128 == 0; recv [max_recv,H/2] 16-byte aligned;
 * recv_scales [max_recv,H/32]; other arguments as in moe_dispatch.  Rows that
 * no entry maps to are not written. */
moe_status moe_dispatch_mx4(const moe_layout_desc *desc, const moe_layout_bufs *layout, const void *hidden, int32_t H,
                            const float *topk_w, void *recv, uint8_t *recv_scales, float *recv_w, void *stream);

/* What moe_expert_gemm_mx4 does with the products before it stores them. */
typedef enum {
    MOE_ACT_NONE = 0,
    MOE_ACT_SWIGLU = 1 /* silu(gate) * up */
} moe_act;

/* The experts' products: for every row r that holds an entry, of expert e,
 *   MOE_ACT_NONE    out[r,n] = bf16( sum_h x[r,h] * w[e,n,h] ),  n < N
 *   MOE_ACT_SWIGLU  out[r,n] = bf16( silu(g) * u ), g = sum_h x[r,h] * w[e,n,h],
 *                   u = sum_h x[r,h] * w[e,N+n,h];  silu(g) = g / (1 + exp(-g))
 * with fp32 sums and one rounding at the end (nearest even).
 *   layout    the layout that the rows were dispatched with.
 *   x         [max_recv,H/2] codes, x_scales [max_recv,H/32]; H % 128 == 0.
 *   w         [E,M,H/2] codes, w_scales [E,M,H/32], M = N or (SWIGLU) 2*N.
 *   N         N % 8 == 0.  H and N are at most 2^22.
 *   bal, slots_per_rank   NULL and 0 for a layout of moe_layout; for one of
 *             moe_layout_balanced its bal and slots: a replica slot's rows use
 *             the weights of the expert in slot_expert.
 *   out       [max_recv,N] bf16, 16-byte aligned, as are x and w; x_scales and
 *             w_scales 4 bytes.
 * Rows that hold no entry are neither read nor written: expert_offset,
 * tokens_per_expert, seg_offset and slot_expert say which rows hold one.  No
 * workspace; the grid depends on the shape alone, not on the routing:
 * MOE_ERR_SHAPE where a launch cannot number it; it always can with
 * (S*K/16 + segments that can hold a row) * ceil(M/32) at most 2^23 - 8. */
moe_status moe_expert_gemm_mx4(const moe_layout_desc *desc, const moe_layout_bufs *layout,
                               const moe_balance_bufs *bal, int32_t slots_per_rank, const void *x,
                               const uint8_t *x_scales, int32_t H, const void *w, const uint8_t *w_scales, int32_t N,
                               int32_t act, void *out, void *stream);

/* ---------------------------------------------------------------------------
 * The experts in bf16: products and their gradients
 * ------------------------------------------------------------------------- */

/* moe_expert_gemm_mx4's products in bf16: for every row r that holds an entry,
 * of expert e,
 *   MOE_ACT_NONE    out[r,n] = bf16( sum_h x[r,h] * w[e,n,h] ),  n < N
 *   MOE_ACT_SWIGLU  out[r,n] = bf16( silu(g) * u ), g = sum_h x[r,h] * w[e,n,h],
 *                   u = sum_h x[r,h] * w[e,N+n,h]
 * with fp32 sums; silu(g) is 0 from g = -87.4 on down, where it is below 10^-36 in
 * magnitude, and NaN at -inf.  The two make an expert's gated feed-forward block:
 * MOE_ACT_SWIGLU with its gate and up weights, MOE_ACT_NONE with its down weights.
 *   x         [max_recv,H], H % 8 == 0.
 *   w         [E,M,H], M = N or (SWIGLU) 2*N; N % 8 == 0.
 *   pre       [max_recv,2*N] or NULL, with SWIGLU only: g, then u of every row,
 *             as moe_expert_gemm_backward_x takes them; fp32 or bf16 (pre_type).
 *             With fp32 the gradients see the activation's own arguments; bf16
 *             takes half the bytes, and its rounding of them (2^-8) passes into
 *             the gradients.  N at most 2^20 with fp32.
 *   out       [max_recv,N].
 *   layout, bal, slots_per_rank as for moe_expert_gemm_mx4.
 * H and M are at most 2^22; all row arrays 16-byte aligned.  Rows that hold no
 * entry are neither read nor written.  No workspace; the grid depends on the
 * shape alone: MOE_ERR_SHAPE where a launch cannot number it (this holds for
 * the calls below too); it always can with (S*K/16 + segments that can hold a
 * row) * ceil(M/32) at most 2^23 - 8.
 * No output of this call or of those below may overlap an input (the arrays of the
 * layout that the call reads among them) or another output, unless it says so:
 * MOE_ERR_SHAPE where it is the same buffer, beginning at the same address. */
moe_status moe_expert_gemm(const moe_layout_desc *desc, const moe_layout_bufs *layout, const moe_balance_bufs *bal,
                           int32_t slots_per_rank, const void *x, int32_t H, const void *w, int32_t N, int32_t act, void *pre,
                           int32_t pre_type, void *out, void *stream);

/* Gradient of a product with respect to its rows, from d_out [max_recv,N] bf16
 * and the weights w [E,N,H] of the MOE_ACT_NONE product (of a SWIGLU one: N
 * counts gate and up rows, d_out is the gradient of its pre):
 *   pre NULL  dx[r,h] = bf16( sum_n d_out[r,n] * w[e,n,h] ),  dx [max_recv,H]
 *   pre given [max_recv,2*H], of the SWIGLU product that made the rows x: the
 *             gradient goes on through the activation to pre itself.  With d the
 *             sum above in fp32, g = pre[r,h], u = pre[r,H+h], s = 1/(1+exp(-g)):
 *             dx[r,h] = bf16( d*u*s*(1 + g*(1-s)) ), dx[r,H+h] = bf16( d*g*s ),
 *             dx [max_recv,2*H], H at most 2^21 (2^20 with fp32); it may be the
 *             buffer of a bf16 pre itself (pre_type), not of an fp32 one.
 * At g = -inf both values are NaN, at +inf the first is.  silu and its slope are as
 * in moe_expert_gemm where they are small.  Arguments otherwise as above. */
moe_status moe_expert_gemm_backward_x(const moe_layout_desc *desc, const moe_layout_bufs *layout, const moe_balance_bufs *bal,
                                      int32_t slots_per_rank, const void *d_out, int32_t N, const void *w, int32_t H,
                                      const void *pre, int32_t pre_type, void *dx, void *stream);

/* Gradient of a product with respect to its weights:
 *   dw[e,n,h] = sum over the rows r of expert e, replicas' rows too, of
 *               d_out[r,n] * x[r,h]
 * d_out [max_recv,N], x [max_recv,H], both bf16; dw [E,N,H], bf16 or fp32
 * (dw_type; then H at most 2^21), fp32 sums.  Every element is written, 0 for an expert without a
 * row.  The order of a sum is fixed by the layout.  Always taken:
 * E*ceil(N/64)*ceil(H/64) at most 2^24 - 16. */
moe_status moe_expert_gemm_backward_w(const moe_layout_desc *desc, const moe_layout_bufs *layout, const moe_balance_bufs *bal,
                                      int32_t slots_per_rank, const void *d_out, int32_t N, const void *x, int32_t H,
                                      int32_t dw_type, void *dw, void *stream);

/* Gradient of moe_combine, out[t] = sum_k w[t,k] * expert_out[pos[t,k]] (+ shared_out):
 *   d_expert_out  [max_recv,H] bf16 or NULL: row pos[t,k] gets bf16(w[t,k] * d_out[t]);
 *                 it may be expert_out's own buffer.
 *   d_w           [S,K] fp32 or NULL: sum_c d_out[t,c] * expert_out[pos[t,k],c] in
 *                 fp32, 0 where pos[t,k] is -1; needs expert_out.
 * At least one of the two, unless S = 0.  d_out [S,H] bf16 (it is shared_out's gradient too);
 * w [S,K] fp32 or NULL for weight 1; H % 8 == 0, at most 2^22; S below 2^23.  Rows that hold
 * no entry are neither read nor written.  (The gradient of moe_dispatch's rows
 * with respect to hidden is moe_combine of them with w = NULL.) */
moe_status moe_combine_backward(const moe_layout_desc *desc, const moe_layout_bufs *layout, const void *d_out, int32_t H,
                                const void *expert_out, const float *w, void *d_expert_out, float *d_w, void *stream);

/* ---------------------------------------------------------------------------
 * 8-bit integers: rows with one scale each, and the experts' products
 * ------------------------------------------------------------------------- */

/* An 8-bit row of H channels (H % 16 == 0, at most 2^22): H codes (int8) and one fp32 scale,
 * amax/127; code = round(x / scale), ties to the even code, both divisions
 * correctly rounded in fp32, within +-127.  A row of zeros has scale 0 and codes
 * 0, a row with a NaN or an infinity scale NaN and codes 0.
 *
 * bf16 rows -> 8-bit rows (activations with a scale per token, or weights with
 * a scale per output channel).
 *   x       [rows,H] bf16, codes [rows,H] int8, 16-byte aligned both.
 *   src     [rows] or NULL: with a layout's src only the rows that hold an
 *           entry (src[r] >= 0) are read and written.
 *   scales  [rows] fp32.
 * rows at most 2^23 - 8. */
moe_status moe_quantize_i8(const void *x, int64_t rows, int32_t H, const int32_t *src, void *codes, float *scales, void *stream);

/* 8-bit rows -> bf16: bf16(code * scale), the product in fp32.  Arguments and
 * limits as in moe_quantize_i8. */
moe_status moe_dequantize_i8(const void *codes, const float *scales, int64_t rows, int32_t H, const int32_t *src, void *out,
                             void *stream);

/* moe_dispatch in 8-bit integers: row pos[t,k] of the receive buffer gets
 * token t's row as moe_quantize_i8 rounds it.  recv [max_recv,H] int8, 16-byte
 * aligned; recv_scales [max_recv] fp32; other arguments as in moe_dispatch; S
 * at most 2^23 - 8.  Rows that no entry maps to are not written. */
moe_status moe_dispatch_i8(const moe_layout_desc *desc, const moe_layout_bufs *layout, const void *hidden, int32_t H,
                           const float *topk_w, void *recv, float *recv_scales, float *recv_w, void *stream);

/* moe_expert_gemm in 8-bit integers, with a scale for each row and each
 * channel: the sum over h of x[r,h] * w[e,n,h] is exact (32 bits, H at most
 * 131056), becomes fp32 and is multiplied by x_scales[r], then by w_scales[e,n];
 * SWIGLU as there, of two such values; one rounding to bf16.
 *   x [max_recv,H] int8, x_scales [max_recv] fp32; H % 16 == 0.
 *   w [E,M,H] int8, w_scales [E,M] fp32.
 * Arguments and limits otherwise as in moe_expert_gemm. */
moe_status moe_expert_gemm_i8(const moe_layout_desc *desc, const moe_layout_bufs *layout, const moe_balance_bufs *bal,
                              int32_t slots_per_rank, const void *x, const float *x_scales, int32_t H, const void *w,
                              const float *w_scales, int32_t N, int32_t act, void *out, void *stream);

/* Static string naming a moe_status value. */
const char *moe_status_str(int32_t status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EP_H */
