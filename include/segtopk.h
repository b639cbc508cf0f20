/*
 * segtopk.h -- segmented (batched) top-k on AMD Instinct MI355X (gfx950).
 *
 * One call, batched_topk(), selects for every segment of a batch the k
 * largest (or smallest) keys, optionally carrying a 32-bit value payload.
 * Selection is multi-pass most-significant-digit radix selection: each pass
 * builds a digit histogram over the surviving candidates, scans it to find the
 * bucket that holds the k-th key, narrows k and the candidate set to that
 * bucket and folds the digit into a running splitter; a final filter writes
 * every key beyond the splitter plus exactly enough splitter-equal keys.
 *   [PR "Implement Segmented TopK using Thread-Block-Clusters", §1.2 Radix
 *    (digit) top-k, §1.4 Early stop, §1.5 Final filter and output placement]
 *
 * The request model (determinism x tie-break x output ordering, their valid
 * pairings and defaults) follows the CCCL page "Top-K: Determinism,
 * Tie-Breaking, and Output Ordering".
 *
 * All pointers passed to batched_topk() are DEVICE pointers except the two
 * descriptor structs themselves, which live in host memory and are read
 * during the call only.  The library never frees or retains caller memory.
 */
#ifndef SEGTOPK_H
#define SEGTOPK_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---------------------------------------------------- */
#define SEGTOPK_OK 0
#define SEGTOPK_INVALID_ARGUMENT 1 /* bad pointer, enum, pairing or size      */
#define SEGTOPK_NOT_SUPPORTED 2    /* valid request this build does not serve */
#define SEGTOPK_HIP_ERROR 3        /* a HIP runtime call or launch failed     */
#define SEGTOPK_SCRATCH_TOO_SMALL 4 /* batched_topk_ex_noalloc: the request's
                                       plan needs more scratch than
                                       SEGTOPK_STATIC_SCRATCH_BYTES; operators
                                       with a workspace: it is too small     */

/* ---- key types ------------------------------------------------------- */
/* Keys are compared by numeric value.  Floating-point keys: -0.0 and +0.0
 * compare equal (either may be selected; the selected key is written with its
 * own original bit pattern, so a selected -0.0 comes back as -0.0); +inf and
 * -inf are the largest and smallest values.  NaN keys are outside the
 * contract (they are ordered above +inf / below -inf by sign, but no result is
 * promised for them).
 *   [PR "Fix BlockTopK +/-0.0 handling", Description: Cause / Fix] */
typedef enum segtopk_key_type {
    SEGTOPK_KEY_F32 = 0,  /* IEEE binary32                          */
    SEGTOPK_KEY_BF16 = 1, /* bfloat16 (upper half of a binary32)    */
    SEGTOPK_KEY_U32 = 2,  /* unsigned 32-bit integer                */
    SEGTOPK_KEY_I32 = 3,  /* signed 32-bit integer                  */
    SEGTOPK_KEY_F16 = 4,  /* IEEE binary16                          */
    SEGTOPK_KEY_U16 = 5,  /* unsigned 16-bit integer                */
    SEGTOPK_KEY_I16 = 6,  /* signed 16-bit integer                  */
    SEGTOPK_KEY_U64 = 7,  /* unsigned 64-bit integer                */
    SEGTOPK_KEY_I64 = 8,  /* signed 64-bit integer                  */
    SEGTOPK_KEY_F64 = 9,  /* IEEE binary64                          */
    SEGTOPK_KEY_U8 = 10,  /* unsigned 8-bit integer                 */
    SEGTOPK_KEY_I8 = 11   /* signed 8-bit integer                   */
} segtopk_key_type;

/* ---- request --------------------------------------------------------- */
/* Which end: the MaxKeys/MaxPairs vs MinKeys/MinPairs entry points. */
typedef enum segtopk_direction { SEGTOPK_MAX = 0, SEGTOPK_MIN = 1 } segtopk_direction;

/* Determinism of the result SET (not of positions).
 *   [docs "Top-K: Determinism ...", "Determinism (cuda::execution::determinism)"] */
typedef enum segtopk_determinism {
    SEGTOPK_NOT_GUARANTEED = 0, /* ties at the boundary: any valid subset      */
    SEGTOPK_RUN_TO_RUN = 1,     /* same set on every run on this GPU          */
    SEGTOPK_GPU_TO_GPU = 2      /* same set on every GPU of this architecture */
} segtopk_determinism;

/* Which tied boundary keys win.  prefer_smaller_index / prefer_larger_index
 * are valid only together with SEGTOPK_GPU_TO_GPU; unspecified is valid with
 * every determinism level.  With a deterministic level and unspecified, this
 * library resolves ties toward the smaller index.
 *   [docs "Top-K: Determinism ...", "Tie-break" and "Which items are
 *    selected?" tables] */
typedef enum segtopk_tie_break {
    SEGTOPK_TIE_UNSPECIFIED = 0,
    SEGTOPK_PREFER_SMALLER_INDEX = 1,
    SEGTOPK_PREFER_LARGER_INDEX = 2
} segtopk_tie_break;

/* How the selected set is laid out in each output row.
 *   unsorted       any permutation of the set
 *   sorted         by key, best first (descending for MAX, ascending for MIN);
 *                  this library writes the stable order
 *   stable_sorted  by key, best first; equal keys by source index ascending
 *   [docs "Top-K: Determinism ...", "Output ordering" table] */
typedef enum segtopk_ordering {
    SEGTOPK_UNSORTED = 0,
    SEGTOPK_SORTED = 1,
    SEGTOPK_STABLE_SORTED = 2
} segtopk_ordering;

/* Largest k served with SEGTOPK_SORTED / SEGTOPK_STABLE_SORTED (the sort runs
 * on-chip); larger k with a sorted ordering returns SEGTOPK_NOT_SUPPORTED.
 * Unsorted output has no such limit. */
#define SEGTOPK_MAX_SORTED_K 4096

/* ---- buffers ---------------------------------------------------------- */
/* Keys: `in` holds offsets[num_segments] elements of `type` (device memory,
 * aligned to the element size); `out` receives num_segments * k elements,
 * row-major with a fixed row stride of k. */
typedef struct segtopk_keys {
    const void *in;
    void *out;
    int32_t type; /* a segtopk_key_type */
} segtopk_keys;

/* Values: any 32-bit payload aligned with keys.in (batched_topk_ex also takes
 * 64-bit payloads), copied bit for bit; `out` has the same num_segments x k
 * shape as the key output.  Pass NULL (or in == NULL) for a keys-only
 * request. */
typedef struct segtopk_values {
    const void *in;
    void *out;
} segtopk_values;

/*
 * batched_topk -- top-k of every segment.
 *
 *   keys             key descriptor (host struct, device buffers), required
 *   values           value descriptor or NULL for keys only
 *   segment_offsets  device array of num_segments + 1 int64 offsets; segment
 *                    i is keys.in[segment_offsets[i] .. segment_offsets[i+1]).
 *                    A negative size (end < begin) is an empty segment.  Each
 *                    segment must hold fewer than 2^31 keys; the total may
 *                    exceed 2^31.
 *   num_segments     number of segments, >= 0
 *   k                keys kept per segment and the output row stride,
 *                    0 <= k <= 2^31 - 1.  Segment i writes k_i = min(k, n_i)
 *                    items to row i; slots k_i .. k-1 are left untouched.
 *                    k at or above the segment size selects the whole segment.
 *   direction        segtopk_direction
 *   determinism      segtopk_determinism
 *   tie_break        segtopk_tie_break (see the pairing rule above)
 *   ordering         segtopk_ordering
 *   stream           HIP stream the work is queued on (NULL: default stream)
 *
 * The call is asynchronous: it validates the request, queues kernels on
 * `stream` and returns without waiting.  It never copies data to the host.
 * Internal scratch (only for batches of fewer than 2048 segments) is one
 * buffer per (device, stream), taken from a memory pool the library creates
 * for the device (the device's default pool is not touched) on `stream` the
 * first time a call on that stream needs it, and grown (the old buffer freed
 * on `stream`) when a later call needs more.  Calls on one stream reuse it in
 * stream order.  The library keeps such buffers for at most 16 (device,
 * stream) pairs; the least recently used one is freed, in stream order, when
 * a seventeenth pair needs one.  A stream handle that is destroyed and
 * created again may inherit the buffer of its predecessor, which is safe
 * because every call first waits for the buffer's previous use.
 * Outputs must not overlap the inputs.  Calls on different streams are
 * independent.
 *
 * Returns SEGTOPK_OK, or SEGTOPK_INVALID_ARGUMENT for a NULL required pointer,
 * an out-of-range enum, k or num_segments, values.in without values.out, or a
 * (determinism, tie_break) pair outside the five valid ones; no work is queued
 * then.  k == 0 or num_segments == 0 returns SEGTOPK_OK with no work.
 * Offsets that decrease other than as empty segments, or a segment of 2^31 or
 * more keys, are precondition violations with undefined results.
 */
int batched_topk(const segtopk_keys *keys, const segtopk_values *values,
                 const int64_t *segment_offsets, int64_t num_segments, int64_t k,
                 int direction, int determinism, int tie_break, int ordering,
                 hipStream_t stream);

/*
 * batched_topk_ex -- batched_topk with per-segment k, a segment-size hint and
 * 64-bit payloads.   [PR "Implement Segmented TopK using
 * Thread-Block-Clusters", the review comment asking for deferred (per-segment)
 * k and for k and num_segments to be validated beyond their wrapper form;
 * §3.4 Single-CTA path and the runtime collapse; the static segment-size
 * bounds of the tuning discussion]
 *
 *   value_bytes       size of one payload item: 4 or 8 (ignored for a
 *                     keys-only request).  values.in / values.out must be
 *                     aligned to it.
 *   k                 output row stride and the largest k of any segment,
 *                     0 <= k <= 2^31 - 1
 *   k_per_segment     NULL (every segment uses k), or a DEVICE array of
 *                     num_segments int32 counts, aligned to 4 bytes: segment i
 *                     keeps k_i = min(max(k_per_segment[i], 0), k, n_i) items.
 *                     Slots k_i .. k-1 of row i are left untouched.  Read on
 *                     the device, in stream order, so it may be written by
 *                     earlier work on `stream`.
 *   max_segment_size  host-side hint: no segment holds more keys than this;
 *                     <= 0 means unknown.  It only steers the launch plan
 *                     (whether segments are split over several workgroups,
 *                     scratch and stash sizes, and, at 4096 keys or fewer for
 *                     4-byte keys and 8192 or fewer for 2-byte keys, a kernel
 *                     built only for segments that fit one load per lane);
 *                     a segment larger than the hint is still served
 *                     correctly, at the cost of a less suited plan.
 *   the other arguments are batched_topk's.
 *
 * With value_bytes == 8 the selection writes each winner's source index into
 * its output slot and a second kernel on `stream` replaces it with the
 * payload; no scratch is taken for that.
 * Returns what batched_topk returns; value_bytes other than 4 or 8, or a
 * misaligned k_per_segment, is SEGTOPK_INVALID_ARGUMENT.
 *
 * batched_topk(keys, values, off, S, k, ...) is
 * batched_topk_ex(keys, values, 4, off, S, k, NULL, 0, ...).
 *
 * Graph capture: a request whose plan needs internal scratch (fewer than
 * 2048 segments, unless max_segment_size shows that no segment needs more
 * than one workgroup) returns SEGTOPK_NOT_SUPPORTED while `stream` is being
 * captured; the other plans queue only kernel launches and may be captured.
 */
int batched_topk_ex(const segtopk_keys *keys, const segtopk_values *values, int32_t value_bytes,
                    const int64_t *segment_offsets, int64_t num_segments, int64_t k,
                    const int32_t *k_per_segment, int64_t max_segment_size, int direction,
                    int determinism, int tie_break, int ordering, hipStream_t stream);

/*
 * batched_topk_ex_noalloc -- batched_topk_ex that allocates nothing.
 *
 * For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  The
 * arguments, results and errors are batched_topk_ex's.  Instead of a
 * per-stream buffer from a memory pool, the scratch that plans for fewer than
 * 2048 segments use (the segment processing order; the per-segment histograms,
 * tickets and candidate slots when segments are split over workgroups) lives
 * in one file-scope device array of SEGTOPK_STATIC_SCRATCH_BYTES, which every
 * GPU the library runs on holds until the process ends.  The call makes no
 * hipMalloc / hipFree / pool call and no allocating library call; it queues
 * only kernels (a small fill kernel clears the words that must start at zero,
 * on every call that uses the array), so it may be captured into a graph.
 *
 * All calls on one device share that device's array and it keeps the last
 * call's contents: calls that can overlap on one device (on different
 * streams, or replays of graphs holding such calls) race and must be ordered
 * by the caller.  A request whose plan needs more than
 * SEGTOPK_STATIC_SCRATCH_BYTES returns SEGTOPK_SCRATCH_TOO_SMALL and queues
 * nothing (for instance 500 segments with k = 2048 of unknown sizes, split
 * two ways: about 41 MB of per-workgroup candidate slots; a max_segment_size
 * hint that rules out splitting avoids that scratch).  32 x 4 Mi keys with
 * k = 2048 (30.5 MiB) or one segment with k = 2048 (30.3 MiB) fit.
 */
#define SEGTOPK_STATIC_SCRATCH_BYTES (32u << 20)
int batched_topk_ex_noalloc(const segtopk_keys *keys, const segtopk_values *values,
                            int32_t value_bytes, const int64_t *segment_offsets,
                            int64_t num_segments, int64_t k, const int32_t *k_per_segment,
                            int64_t max_segment_size, int direction, int determinism,
                            int tie_break, int ordering, hipStream_t stream);

/* ======================================================================
 * Operators around the selection in a language model
 *
 * A router's top-k gives every token k experts: segtopk_sort_ids lists the
 * (token, expert) slots expert by expert, segtopk_dispatch_rows copies the
 * tokens into that order, segtopk_combine_rows brings the experts' results back
 * with the gate weights applied.  A sampler's top-k gives the next token:
 * segtopk_embedding_rows looks it up, and segtopk_policy_loss scores sampled
 * tokens under the model's logits.  The *_backward functions, and
 * segtopk_policy_loss with a gradient buffer, are their gradients.
 *
 * For all of them: pointers in the arguments are DEVICE pointers; the argument
 * structs are host memory read during the call only.  A call validates, queues
 * kernels on `stream` and returns without waiting; it allocates nothing, keeps
 * nothing, copies nothing to the host, and may be captured into a graph.
 * Element types are SEGTOPK_KEY_F32, _BF16 and _F16, id types SEGTOPK_KEY_I32
 * and _I64.  Sums are held in 32 bits or more, in one fixed order, and rounded
 * once: the same call gives the same bits every time.  Outputs must not overlap
 * inputs unless stated.  Workspaces hold at least what the *_workspace function
 * returns (bytes; 0 also for sizes that the call refuses), aligned to 256
 * bytes; a smaller one is SEGTOPK_SCRATCH_TOO_SMALL, and NULL is allowed for 0
 * bytes.  SEGTOPK_INVALID_ARGUMENT: a NULL or misaligned pointer, an unknown or
 * unmatched type, a negative or too large size, a stride below the width; no
 * work is queued then.
 * ====================================================================== */

/* Rows of a matrix: element c of row r is data[r * stride + c].  `stride` counts
 * elements; rows need the alignment of one element only. */
typedef struct segtopk_rows {
    void *data;
    int64_t stride;
    int32_t type; /* a segtopk_key_type */
} segtopk_rows;

/*
 * segtopk_sort_ids -- the stable sort of n ids into num_segments segments.
 *
 *   key_i = ids[i] if 0 <= ids[i] < num_segments, else num_segments (dropped)
 *   order     [n] the slots i by key, equal keys by slot; dropped ones last
 *   position  [n] its inverse: order[position[i]] = i
 *   offsets   [num_segments + 1] segment s is order[offsets[s] .. offsets[s+1]);
 *             offsets[num_segments] is the number of slots kept.  They serve as
 *             batched_topk's segment_offsets.
 * 0 <= n <= 2^31 - 1, 0 <= num_segments < 2^31 - 1.
 */
int64_t segtopk_sort_ids_workspace(int64_t n, int64_t num_segments);
int segtopk_sort_ids(const void *ids, int32_t id_type, int64_t n, int64_t num_segments,
                     int32_t *order, int32_t *position, int64_t *offsets, void *workspace,
                     int64_t workspace_bytes, hipStream_t stream);

/*
 * segtopk_dispatch_rows -- tokens copied into expert order:
 *   rows[position[t * k + j]] = x[t]
 * x has `tokens` rows, `rows` tokens * k; both are `width` wide and of one type.
 * A slot whose position is not below *kept is dropped and its row set to zero;
 * `kept` is a device pointer (&offsets[num_segments] of the sort) or NULL: all
 * are kept.  Slots whose position is outside [0, tokens * k) are skipped.
 * `position` is a permutation; tokens * k <= 2^31 - 1.
 */
int segtopk_dispatch_rows(const segtopk_rows *x, const segtopk_rows *rows, int64_t tokens,
                          int64_t k, int64_t width, const int32_t *position, const int64_t *kept,
                          hipStream_t stream);

/*
 * segtopk_combine_rows -- rows in expert order summed into their tokens:
 *   out[t] = sum_j weights[t * k + j] rows[position[t * k + j]]
 * over the slots kept.  Rows of dropped slots are not read, whatever they hold.
 * weights NULL: all one (the gradient of segtopk_dispatch_rows).  weight_type is
 * SEGTOPK_KEY_F32 or the rows' type.
 */
int segtopk_combine_rows(const segtopk_rows *rows, const segtopk_rows *out, const void *weights,
                         int32_t weight_type, int64_t tokens, int64_t k, int64_t width,
                         const int32_t *position, const int64_t *kept, hipStream_t stream);

/*
 * segtopk_combine_rows_backward -- the gradient of segtopk_combine_rows:
 *   drows[position[t * k + j]]  = weights[t * k + j] dout[t]
 *   dweights[t * k + j] = <dout[t], rows[position[t * k + j]]>
 * and zero for dropped slots.  dweights NULL: not wanted, and rows may be NULL.
 * weights NULL: all one.  dweights is of weight_type.
 */
int segtopk_combine_rows_backward(const segtopk_rows *dout, const segtopk_rows *rows,
                                  const segtopk_rows *drows, const void *weights, void *dweights,
                                  int32_t weight_type, int64_t tokens, int64_t k, int64_t width,
                                  const int32_t *position, const int64_t *kept,
                                  hipStream_t stream);

/*
 * segtopk_embedding_rows -- out[i] = scale * table[ids[i]], rounded once; the
 * row of an id outside [0, num_rows) is zero.
 */
int segtopk_embedding_rows(const segtopk_rows *table, const segtopk_rows *out, const void *ids,
                           int32_t id_type, int64_t n, int64_t num_rows, int64_t width,
                           float scale, hipStream_t stream);

/*
 * segtopk_embedding_backward -- the gradient of the table:
 *   dtable[v] = scale * sum over ids[i] = v of dout[i]
 * All num_rows rows are written, most of them zero.  Ids outside [0, num_rows)
 * add nothing, nor does padding_id (outside [0, num_rows): no padding).
 * accumulate != 0: the sums are added to what dtable holds, and rows of ids that
 * do not occur are neither read nor written.  dtable is of dout's type or
 * SEGTOPK_KEY_F32.  SEGTOPK_NOT_SUPPORTED: more work than one launch holds,
 * ceil(n / 64) * ceil(u / 256) >= 2^24 - 1, where u is the number of whole 16-byte
 * pieces in a row of dout and of elements past them.
 */
int64_t segtopk_embedding_backward_workspace(int64_t n, int64_t num_rows, int64_t width);
int segtopk_embedding_backward(const segtopk_rows *dout, const segtopk_rows *dtable,
                               const void *ids, int32_t id_type, int64_t n, int64_t num_rows,
                               int64_t width, float scale, int64_t padding_id, int32_t accumulate,
                               void *workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * segtopk_policy_loss -- the clipped policy loss of sampled tokens with a KL
 * term, and its gradient in the logits.
 *
 * Row t holds the logits that token_ids[t] was drawn from.  With
 * z = logits[t] / temperature:
 *   logp[t] = z[token] - log sum_c exp(z[c])
 *   r = exp(logp - old_logp),  A = advantages[t]
 *   term = -min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A)
 *          + kl_coef (exp(ref_logp - logp) - (ref_logp - logp) - 1)
 * Answer s is the rows segment_offsets[s] .. segment_offsets[s+1] (offsets do
 * not decrease).  loss is the mean over the answers of the mean over each
 * answer's live rows; an answer without one adds zero.  A row is live if its
 * token is in [0, vocab) and it lies in an answer; the others, and rows whose
 * logits are all -inf, have logp 0, no term and a gradient of zero, and what
 * else they hold does not matter.  A logit of -inf is a token ruled out.  NaN
 * in a live row (logits, old_logp, advantage; ref_logp if kl_coef is not 0) and
 * a logit of +inf make the loss and the row's gradient NaN.
 * A sampled token that is ruled out has logp -inf and r 0.  With kl_coef its
 * term, and the loss, are +inf, and so is the size of the row's gradient; that
 * of the other tokens ruled out is zero.
 *
 *   dlogits.data  NULL: no gradient.  Else grad_scale * d loss / d logits, of
 *                 the logits' type; it may be the logits themselves (same
 *                 data and stride).
 *   ref_logp      may be NULL when kl_coef is 0
 * 0 <= clip_low <= 1, clip_high >= 0, kl_coef >= 0, temperature > 0;
 * tokens < 2^22, num_segments < 2^24.
 */
typedef struct segtopk_policy_loss_args {
    segtopk_rows logits, dlogits;
    const void *token_ids;
    int32_t id_type;
    double clip_low, clip_high, kl_coef, temperature, grad_scale;
    int64_t tokens, vocab, num_segments;
    const int64_t *segment_offsets;
    const float *old_logp, *ref_logp, *advantages;
    float *loss; /* [1] */
    float *logp; /* [tokens] */
} segtopk_policy_loss_args;

int64_t segtopk_policy_loss_workspace(int64_t tokens, int64_t vocab, int64_t num_segments);
int segtopk_policy_loss(const segtopk_policy_loss_args *args, void *workspace,
                        int64_t workspace_bytes, hipStream_t stream);

/* Human-readable name of a status code (static storage). */
const char *segtopk_status_string(int status);

/* Library version as MAJOR * 10000 + MINOR * 100 + PATCH. */
int segtopk_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SEGTOPK_H */
