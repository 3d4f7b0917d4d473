/*
 * iso.h -- C ABI of the GB300 (sm_103a) isotonic-regression library libiso.so,
 * and of the training objectives beside it (token log-probabilities, policy,
 * preference and balance losses; see "Training objectives" below).
 *
 * The operation ("Merge Hulls Without Copying Vertices: GPU Isotonic Regression",
 * Section 2.1, eq. (1)): for every row y_1..y_n with weights w_i > 0, the unique
 * z with z_1 <= z_2 <= ... <= z_n that minimises sum_i w_i (z_i - y_i)^2.  The
 * decreasing problem is the increasing one for -y (same section).  z is taken,
 * as in eq. (3), as the slopes of the lower convex hull of the cumulative-sum
 * diagram P_k = (W_k, S_k), W_k = sum_{i<=k} w_i, S_k = sum_{i<=k} w_i y_i
 * (eq. (2)); the hull's vertices are the starts of the fit's blocks.
 *
 * Conventions shared by every entry point:
 *  - Layout: row-major, contiguous [rows, n] float32 arrays (row r starts at
 *    element r*n).  Any 4-byte alignment is accepted.
 *  - Memory: every array argument ("device" below) must be accessible from
 *    the device: device memory, or pinned (page-locked) host memory, which
 *    under unified addressing is device-accessible at its host address -- the
 *    kernels then read inputs and write outputs in place over the host link
 *    (NVLink-C2C on GB300), with no separate copy.  The workspace is best
 *    kept in device memory.
 *  - Ownership: the caller owns every buffer, the workspace and the stream.
 *    The fit and backward calls allocate no memory, keep no state between
 *    calls (beyond the device's SM count, read once), and never synchronise
 *    the stream: every call only enqueues kernels on `stream` (a cudaStream_t;
 *    NULL = the legacy default stream) and returns.  Only the optional
 *    benchmarking and debugging switches at the end of this file keep state.
 *  - Errors the host can see (NULL pointers, non-positive or oversized shapes,
 *    a workspace that is too small or misaligned) return a negative status and
 *    enqueue nothing.  A failed kernel launch returns ISO_ERR_CUDA.
 *  - Errors in the data (a non-finite y, a weight that is not finite and
 *    positive) never fail the call: that row's outputs are NaN, its block
 *    flags are 0, and its bit in `row_status` is set (the paper's per-row NaN
 *    flags, Section 6 "Blocks and memory", without its host synchronisation).
 *  - Limits: 1 <= n <= 2^31 - 1, 1 <= rows, rows * n <= 2^40.  An empty call
 *    (rows == 0 or n == 0, neither negative; for ragged batches segments == 0)
 *    does nothing and returns ISO_OK whatever the pointers; a ragged batch
 *    with total == 0 only writes the segments' statuses.
 *  - float64 I/O: every entry point that takes float32 arrays has an _f64
 *    twin taking float64 arrays (the paper supports both working types,
 *    Section 6 "Implementation"), with the same arguments, layout, workspace
 *    sizes, errors and status bits; only the element type differs.
 */
#ifndef ISO_H
#define ISO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ISO_OK = 0,
    ISO_ERR_INVALID_ARG = -1, /* NULL pointer, bad shape or flag                 */
    ISO_ERR_WORKSPACE = -2,   /* workspace NULL / too small / not 256-B aligned */
    ISO_ERR_CUDA = -3,        /* a CUDA call or kernel launch failed            */
    ISO_ERR_TIMEOUT = -4      /* reserved: a bounded device-side wait gave up   */
} iso_status;

/* Bits of a row's status word. */
#define ISO_ROW_BAD_Y 1u /* the row holds a NaN or infinite y                   */
#define ISO_ROW_BAD_W 2u /* the row holds a weight that is not finite and > 0   */
#define ISO_ROW_BAD_SHAPE 4u /* ragged batches: the segment's offsets are out of  */
                             /* order or range, or it is longer than max_len      */

/* Version of this ABI (major * 10000 + minor * 100 + patch). */
int iso_version(void);

/* Human-readable name of a status code (static string). */
const char *iso_status_string(int status);

/*
 * Bytes of device workspace that iso_fit needs for `rows` rows of `n` elements
 * (`weighted` != 0 when w is given).  0 means no workspace is needed.  Returns
 * 0 as well for invalid shapes (iso_fit then reports the error).
 */
size_t iso_fit_workspace_bytes(int64_t rows, int64_t n, int weighted);

/*
 * iso_fit -- forward fit.
 *
 * Defined by eq. (1)-(3) of the paper (Section 2.1); the method is the paper's
 * Section 3: lane hulls kept in register bit masks, lane and chunk merges by
 * walking to the bridge, and, for rows longer than one chunk, a merge tree
 * whose nodes are lists of segments of the chunk hulls (Section 3.3), followed
 * by reconstruction (Section 3.4).
 *
 *  y          [rows, n] float32, device, read only.
 *  w          [rows, n] float32, device, read only, or NULL for unit weights.
 *  rows, n    shape.
 *  increasing 1: non-decreasing fit; 0: non-increasing fit (fit of -y, negated).
 *  out        [rows, n] float32, device, written: the fit.  Every value is
 *             rounded to float32 once from the slope of its hull edge; the
 *             output is not forced to be monotone (no cumulative maximum),
 *             as in the paper's Section 6 "Output".
 *  blocks     [rows, n] uint8, device, written, or NULL: blocks[i] = 1 where
 *             element i starts a block (its left point is a hull vertex; the
 *             paper's block-start byte of Section 6 "Gradient"), else 0.
 *             blocks[0] of a valid row is always 1.  Needed by iso_backward.
 *  workspace  device scratch of at least iso_fit_workspace_bytes(rows, n, w != NULL)
 *             bytes, 256-byte aligned; may be NULL when that size is 0.  Its
 *             contents on entry do not matter.  Calls that share one workspace
 *             must not overlap in time (use one stream).
 *  row_status [rows] uint32, device, written, or NULL: 0 or ISO_ROW_BAD_* bits.
 *  stream     cudaStream_t to enqueue on.
 *
 * Accuracy: cumulative sums are exact integer sums of values rounded to a
 * fixed-point grid of 2^-50 of the largest |w*y| (and |w|) of each chunk; the
 * fit deviates from the exact one by about that amount plus one float32
 * rounding of each slope.
 */
iso_status iso_fit(const float *y, const float *w, int64_t rows, int64_t n, int increasing,
                   float *out, uint8_t *blocks, void *workspace, size_t workspace_bytes,
                   uint32_t *row_status, void *stream);

/*
 * iso_fit_f64 -- iso_fit on float64 arrays.  The same fixed-point arithmetic:
 * values are rounded to 2^-50 of their tile's largest magnitude (a float64
 * value keeps 50 of its 53 bits at the tile's top exponent), sums and turns
 * are exact, and each slope is one float64 quotient of two integers, so the
 * fit deviates from the exact fit of the input by about 2^-49 of the row's
 * largest |y| (times the weights' dynamic range for weighted rows) plus one
 * float64 rounding.
 */
iso_status iso_fit_f64(const double *y, const double *w, int64_t rows, int64_t n, int increasing,
                       double *out, uint8_t *blocks, void *workspace, size_t workspace_bytes,
                       uint32_t *row_status, void *stream);

/* Bytes of device workspace that iso_backward needs (0 = none). */
size_t iso_backward_workspace_bytes(int64_t rows, int64_t n, int weighted);

/*
 * iso_backward -- vector-Jacobian product of the fit with respect to y.
 *
 * The paper's Section 6 "Gradient": the fit is constant on blocks and equals
 * the block's weighted mean, so with G and W the sums of grad and of w over
 * element i's block, d/dy_i = w_i * G / W (G / |block| for unit weights).
 * The blocks are those that iso_fit wrote into `blocks`.
 *
 *  grad       [rows, n] float32, device: gradient with respect to the fit.
 *  blocks     [rows, n] uint8, device: block starts as written by iso_fit
 *             (element 0 of a row is treated as a start whatever its value).
 *  w          [rows, n] float32 or NULL, the weights given to iso_fit.
 *  out        [rows, n] float32, device, written.
 *  workspace  as for iso_fit, of iso_backward_workspace_bytes(rows, n, w != NULL) bytes.
 *  stream     cudaStream_t.
 */
iso_status iso_backward(const float *grad, const uint8_t *blocks, const float *w, int64_t rows,
                        int64_t n, float *out, void *workspace, size_t workspace_bytes,
                        void *stream);

/* iso_backward on float64 arrays (grad, w, out); the blocks are iso_fit_f64's. */
iso_status iso_backward_f64(const double *grad, const uint8_t *blocks, const double *w,
                            int64_t rows, int64_t n, double *out, void *workspace,
                            size_t workspace_bytes, void *stream);

/*
 * iso_backward_w -- the vector-Jacobian products of the fit with respect to y
 * and to the weights w.
 *
 * The paper's Section 6 "Gradient": on element i's block, with G and W the
 * sums of grad and of w over the block and z_i the block's weighted mean (the
 * fit), d/dy_i = w_i * G / W and d/dw_i = (y_i - z_i) * G / W.  The same
 * formulas hold for increasing and decreasing fits.
 *
 *  grad       [rows, n] float32, device: gradient with respect to the fit.
 *  blocks     [rows, n] uint8, device: block starts as written by iso_fit.
 *  w          [rows, n] float32 or NULL (unit weights), as given to iso_fit.
 *  y          [rows, n] float32, device: the input given to iso_fit.
 *  fit        [rows, n] float32, device: the fit iso_fit wrote.
 *  out_dy     [rows, n] float32, device, written; may be NULL (not wanted).
 *  out_dw     [rows, n] float32, device, written.
 *  workspace  as for iso_backward, of iso_backward_workspace_bytes(rows, n,
 *             w != NULL) bytes.
 *  stream     cudaStream_t.
 *
 * Errors: ISO_ERR_INVALID_ARG for a NULL grad, blocks, y, fit or out_dw or a
 * bad shape, ISO_ERR_WORKSPACE as for iso_backward, ISO_ERR_CUDA for a launch
 * failure.  A row whose forward pass was rejected (its fit is NaN) gets NaN.
 */
iso_status iso_backward_w(const float *grad, const uint8_t *blocks, const float *w,
                          const float *y, const float *fit, int64_t rows, int64_t n,
                          float *out_dy, float *out_dw, void *workspace, size_t workspace_bytes,
                          void *stream);

/*
 * Bytes of device workspace that iso_fit_ragged needs for `segments` segments
 * covering `total` elements, none longer than max_len (max_len <= 0: total).
 * Returns 0 for invalid arguments (iso_fit_ragged then reports the error).
 */
size_t iso_fit_ragged_workspace_bytes(int64_t segments, int64_t total, int64_t max_len,
                                      int weighted);

/*
 * iso_fit_ragged -- forward fit of a ragged batch: segments of their own
 * lengths laid end to end, each fitted as its own row (eq. (1)-(3), Section
 * 2.1).  The paper fits such batches (many per-segment calibration curves,
 * Section 7.7) by padding them to a rectangle or by laying them end to end in
 * one row with each segment's targets lifted above the previous segment's;
 * here the offsets are given to the library, and every segment gets exactly
 * the fit iso_fit would give it as a row of its own.
 *
 *  y          [total] float32, device, read only: the segments end to end.
 *  w          [total] float32, device, read only, or NULL for unit weights.
 *  offsets    [segments + 1] int64, device, read only: segment s holds elements
 *             offsets[s] .. offsets[s+1]-1.  The offsets are not read by the
 *             host.  Non-decreasing offsets within [0, total] give disjoint
 *             segments; elements outside every segment are not written.
 *  segments   number of segments, 0 <= segments <= 2^31 - 1 (0: nothing to do).
 *  total      length of y (and w, out, blocks), 0 <= total <= 2^40 (with 0, y and
 *             out may be NULL and every segment is empty or rejected).
 *  max_len    an upper bound on the segments' lengths that the caller knows,
 *             or <= 0 for none (total).  It only saves launches and workspace:
 *             a segment longer than it is rejected (ISO_ROW_BAD_SHAPE).  At
 *             most 2^31 - 1.
 *  increasing as for iso_fit.
 *  out        [total] float32, device, written: each segment's fit.
 *  blocks     [total] uint8, device, written, or NULL: block starts as for
 *             iso_fit.  The first element of every non-empty segment that was
 *             not rejected for its shape is flagged 1, also in a segment
 *             rejected for its values (whose other flags are 0), so that
 *             iso_backward / iso_backward_w over the whole array as ONE row
 *             (rows = 1, n = total) give each segment its own backward, when
 *             the segments cover the array end to end.
 *  workspace  device scratch of iso_fit_ragged_workspace_bytes(segments,
 *             total, max_len, w != NULL) bytes, 256-byte aligned.
 *  row_status [segments] uint32, device, written, or NULL: per segment, 0 or
 *             ISO_ROW_BAD_* bits (an empty segment: 0).
 *  stream     cudaStream_t.
 *
 * The segments are sorted on the device into lists by length: up to 8,192
 * elements by the whole-row kernels (by lane class), longer ones by the
 * long-row path; no host synchronisation.  Accuracy as for iso_fit.
 */
iso_status iso_fit_ragged(const float *y, const float *w, const int64_t *offsets,
                          int64_t segments, int64_t total, int64_t max_len, int increasing,
                          float *out, uint8_t *blocks, void *workspace, size_t workspace_bytes,
                          uint32_t *row_status, void *stream);

/* iso_fit_ragged on float64 arrays (y, w, out); offsets and statuses as iso_fit_ragged. */
iso_status iso_fit_ragged_f64(const double *y, const double *w, const int64_t *offsets,
                              int64_t segments, int64_t total, int64_t max_len, int increasing,
                              double *out, uint8_t *blocks, void *workspace,
                              size_t workspace_bytes, uint32_t *row_status, void *stream);

/*
 * iso_fit_copy_control -- a measurement control, not a faster fit: the same
 * fit as iso_fit (bit for bit), with the merge levels of rows longer than
 * 8,192 elements run on materialised hulls instead of segment lists -- the
 * paper's "grid copying" control of Section 7.3: after every level's bridges
 * are found (the same search), every merged hull's surviving vertices are
 * copied into a second flat array by the whole grid.  It measures what the
 * segment lists save; rows of up to 8,192 elements (no merge tree) take the
 * whole-row kernels as in iso_fit.
 *
 * Arguments, results and errors as iso_fit, with a workspace of
 * iso_fit_copy_control_workspace_bytes(rows, n, weighted) bytes (about four
 * times iso_fit's: two flat buffers of C + 1 vertex records per chunk);
 * n <= 2^30.
 */
size_t iso_fit_copy_control_workspace_bytes(int64_t rows, int64_t n, int weighted);
iso_status iso_fit_copy_control(const float *y, const float *w, int64_t rows, int64_t n,
                                int increasing, float *out, uint8_t *blocks, void *workspace,
                                size_t workspace_bytes, uint32_t *row_status, void *stream);

/* iso_backward_w on float64 arrays. */
iso_status iso_backward_w_f64(const double *grad, const uint8_t *blocks, const double *w,
                              const double *y, const double *fit, int64_t rows, int64_t n,
                              double *out_dy, double *out_dw, void *workspace,
                              size_t workspace_bytes, void *stream);

/*
 * iso_backward_noalloc -- iso_backward for callers that cannot allocate device
 * memory (no counterpart in the paper: it is an interface addition).
 *
 * Same arguments, results and errors as iso_backward, without the workspace:
 * the per-tile records that rows longer than 8,192 elements need live in a
 * fixed 2 MiB array inside the library (device memory that every GPU which
 * loads the library holds until the process exits), which limits such calls to
 * rows * ceil(n / 8192) <= 21,845 tiles; larger calls return ISO_ERR_WORKSPACE
 * and enqueue nothing.  Rows of at most 8,192 elements need no scratch and have
 * no such limit.
 *  - The first call on a device looks up the array's device address (once per
 *    device, on the calling thread's current device); make that first call
 *    before any stream capture.
 *  - Every call shares the one array: calls whose work may overlap on the GPU
 *    (different streams, several host threads) race on it and must be
 *    serialised by the caller.  Each call writes every record it reads, so
 *    nothing needs clearing between calls.
 *  - It calls no allocating function (no cudaMalloc, no cudaFree).
 */
iso_status iso_backward_noalloc(const float *grad, const uint8_t *blocks, const float *w,
                                int64_t rows, int64_t n, float *out, void *stream);

/* ------------------------------------------------------------------------
 * Training objectives over rows of scores.
 *
 * What a model trained on ranks and preferences needs beside the fit: rewards
 * that iso_fit calibrates, or their soft ranks, enter a policy or a preference
 * loss over the log-probabilities of a model's tokens; a router of experts
 * adds its balance loss.  With x [rows, n] a row's scores (logits), T > 0 the
 * temperature and l_r the row's label,
 *
 *   lp_r = x[r, l_r] / T - log sum_j exp(x[r, j] / T)
 *   d lp_r / d x[r, j] = ([j == l_r] - p[r, j]) / T,
 *   p[r, j] = exp(x[r, j] / T) / sum_i exp(x[r, i] / T).
 *
 * Conventions, beside those at the top of this file:
 *  - Scores and their gradients are float32, bfloat16 or float16 (`dtype`);
 *    everything else is float32 unless said otherwise.  Sums and softmax
 *    statistics are float32 within a row (and over up to 64 tokens of a router);
 *    sums over rows, tokens and pairs are two float32 each, of which the second
 *    holds what the first has rounded off.  A gradient is rounded once, to the
 *    scores' type.  Results do not depend on timing: the same call gives the
 *    same bits.
 *  - Row r of the scores starts at element r * stride, of the gradient at
 *    r * out_stride (strides in elements; the gradient's at least n).  1 <= n <=
 *    2^31 - 1, 0 <= rows <= 2^31 - 1, rows * stride <= 2^40.  Element alignment is enough.
 *  - labels [rows] int64: a negative label marks a row that takes no part; its
 *    scores (and its other inputs) are not used, its log-probability is 0 and
 *    its gradient 0.  A label >= n is an error in the data: the row's
 *    log-probability and gradient are NaN and its row_status has ISO_ROW_BAD_LABEL.
 *  - A score of -inf is a closed entry of probability 0.  The type's lowest
 *    value is an ordinary, very small score.  A row with a NaN or +inf, or
 *    with nothing but -inf, has no probabilities: its log-probability and
 *    gradient are NaN and its row_status has ISO_ROW_BAD_Y.
 *  - temperature > 0, with 1 / T and log2(e) / T in float32's range.
 *  - norm [rows, 2], 8-byte aligned: the row's softmax statistics (its largest score and the sum
 *    of exponentials against it), from which the backward forms p without another pass.
 *  - The gradient may be written over the scores (dlogits == logits, out_stride == stride).
 * ------------------------------------------------------------------------ */
typedef enum { ISO_F32 = 0, ISO_BF16 = 1, ISO_F16 = 2 } iso_dtype;
#define ISO_ROW_BAD_LABEL 8u /* the row's label is not below n                   */
#define ISO_ROW_TIMEOUT 16u  /* a bounded wait of the row's CTAs for one another */
                             /* gave up (a fault of the GPU); the row is NaN     */

/*
 * iso_token_logp -- the labels' log-probabilities.
 *
 *  logp       [rows], written: lp_r, or 0 for a row without a label.
 *  norm       [rows, 2], written.
 *  workspace  iso_token_logp_workspace_bytes(rows) bytes, 256-byte aligned; may be NULL when that
 *             is 0 (few rows).
 *  row_status [rows] uint32, written, or NULL.
 */
size_t iso_token_logp_workspace_bytes(int64_t rows);
iso_status iso_token_logp(const void *logits, int dtype, int64_t rows, int64_t n, int64_t stride,
                          const int64_t *labels, float temperature, float *logp, float *norm,
                          void *workspace, size_t workspace_bytes, uint32_t *row_status,
                          void *stream);

/*
 * iso_token_logp_backward -- dlogits[r, j] = g_r / T ([j == l_r] - p[r, j]) with
 * g_r = grad_logp[r] * grad_scale * (*grad_scale_dev).
 *
 *  norm            what the forward wrote for the same logits and temperature.
 *  grad_logp       [rows].
 *  grad_scale_dev  one float on the device, or NULL for 1.
 *  changed_only    0 or 1.  1: when *grad_scale_dev is 1, nothing is written
 *                  (dlogits already holds the gradient for a scale of 1, as
 *                  iso_policy_loss and iso_preference_loss leave it).
 */
iso_status iso_token_logp_backward(const void *logits, int dtype, int64_t rows, int64_t n,
                                   int64_t stride, const int64_t *labels, float temperature,
                                   const float *norm, const float *grad_logp, float grad_scale,
                                   const float *grad_scale_dev, int changed_only, void *dlogits,
                                   int64_t out_stride, void *stream);

/*
 * iso_policy_loss -- clipped policy loss with a KL term to a reference, and its
 * gradient in the scores.  Over the labelled rows, with q_r = exp(lp_r - old_logp[r])
 * and d_r = ref_logp[r] - lp_r,
 *
 *   policy_r = max(-A_r q_r, -A_r clip(q_r, 1 - clip_low, 1 + clip_high))
 *   kl_r     = exp(d_r) - 1 - d_r
 *   loss     = sum_r w_r (policy_r + kl_coef kl_r)
 *
 *  old_logp, advantages  [rows]: log-probabilities when the labels were drawn; A.
 *  ref_logp   [rows], or NULL: no KL term (kl_coef is then not used).
 *  weights    [rows]: w, or NULL: 1 / (number of labelled rows).
 *  clip_low, clip_high   0 <= clip_low <= 1, 0 <= clip_high.
 *  grad_scale multiplies the gradient only (loss scaling).
 *  loss       one float, written (0 when no row has a label).
 *  stats      three floats, written: sum w policy, sum w kl, sum of w over the
 *             rows whose policy term the clip holds (their policy gradient is 0).
 *  logp, norm [rows], [rows, 2], written.
 *  coef       [rows], written: d loss / d lp_r (without grad_scale).
 *  dlogits    [rows, n] of dtype, written, or NULL: not wanted.
 *  workspace  iso_policy_loss_workspace_bytes(rows) bytes, 256-byte aligned.
 */
size_t iso_policy_loss_workspace_bytes(int64_t rows);
iso_status iso_policy_loss(const void *logits, int dtype, int64_t rows, int64_t n, int64_t stride,
                           const int64_t *labels, float temperature, const float *old_logp,
                           const float *advantages, const float *ref_logp, const float *weights,
                           float clip_low, float clip_high, float kl_coef, float grad_scale,
                           float *loss, float *stats, float *logp, float *norm, float *coef,
                           void *dlogits, int64_t out_stride, void *workspace,
                           size_t workspace_bytes, uint32_t *row_status, void *stream);

/*
 * iso_preference_loss -- preference loss over pairs of token sequences, and its
 * gradient in the scores.  Sequence s holds rows offsets[s] .. offsets[s+1]-1;
 * pair q's chosen sequence is 2q, its rejected one 2q + 1.  With S_s the sum (or,
 * average != 0, the mean) of lp over s's labelled rows and R_s the same of ref_logp,
 *
 *   h_q = (S_2q - R_2q) - (S_2q+1 - R_2q+1),   z_q = beta h_q
 *   sigmoid: -(1 - label_smoothing) log sigmoid(z) - label_smoothing log sigmoid(-z)
 *            (a term of weight 0 is 0, also where z is infinite: a closed label)
 *   hinge:   max(0, 1 - z)
 *   squared: (h - 1 / (2 beta))^2
 *   loss = mean over the pairs.
 *
 *  offsets    [2 pairs + 1] int64, not read by the host.  A pair with offsets
 *             out of order or out of [0, rows], or that has rows and starts before
 *             the end of an earlier such pair in order, gets ISO_ROW_BAD_SHAPE in
 *             pair_status, a margin and sums of NaN, and adds nothing to a gradient;
 *             the loss is NaN.  Rows of no other sequence get a gradient of 0.
 *  ref_logp   [rows], or NULL: R = 0.
 *  loss       one float, written (0 for no pairs).
 *  margins    [pairs], written: z.       seq_logp [2 pairs], written: S.
 *  logp, norm, coef   [rows], [rows, 2], [rows], written; coef = d loss / d lp_r.
 *  dlogits    [rows, n], written, or NULL.
 *  workspace  iso_preference_loss_workspace_bytes(rows, pairs) bytes, 256-byte aligned.
 *  row_status, pair_status  [rows], [pairs] uint32, written, or NULL.
 */
#define ISO_PREFERENCE_SIGMOID 0
#define ISO_PREFERENCE_HINGE 1
#define ISO_PREFERENCE_SQUARED 2
size_t iso_preference_loss_workspace_bytes(int64_t rows, int64_t pairs);
iso_status iso_preference_loss(const void *logits, int dtype, int64_t rows, int64_t n,
                               int64_t stride, const int64_t *labels, const int64_t *offsets,
                               int64_t pairs, const float *ref_logp, int kind, float beta,
                               float label_smoothing, int average, float grad_scale, float *loss,
                               float *margins, float *seq_logp, float *logp, float *norm,
                               float *coef, void *dlogits, int64_t out_stride, void *workspace,
                               size_t workspace_bytes, uint32_t *row_status,
                               uint32_t *pair_status, void *stream);

/*
 * iso_balance_loss -- a router's choice of top_k experts for each token, its
 * balance loss and the tokens of each expert.  With p the softmax of a token's
 * scores, T the live tokens and n_e the tokens that chose e,
 *
 *   loss = experts / (top_k T^2) sum_e n_e sum_t p[t, e]     (1 when even)
 *
 *  logits     [tokens, experts] of dtype, row t at element t * stride;
 *             1 <= experts <= ISO_MAX_EXPERTS.
 *  top_k      1 <= top_k <= min(experts, ISO_MAX_TOP_K).
 *  mask       [tokens] uint8, or NULL: 0 marks a token that takes no part.  A
 *             token with nothing but -inf takes no part either.
 *  renormalize  0: gates are p at the chosen experts; 1: divided by their sum.
 *  loss       one float, written (0 for no live token).
 *  counts     [experts] int64, written: n.
 *  chosen     [tokens, top_k] int32, written: the experts by decreasing score,
 *             equal scores by increasing index; -1 where no open expert is left (a
 *             score of -inf or NaN is never chosen) or the token takes no part.
 *  gates      [tokens, top_k] float32, written: 0 where chosen is -1.
 *  live       one int64, written: T.
 *             A NaN or +inf among the scores of a token that takes part makes its
 *             gates, its gradient and the loss NaN.
 *  workspace  iso_balance_loss_workspace_bytes(tokens, experts) bytes, 256-byte aligned.
 *
 * iso_balance_loss_backward -- the gradient of grad_loss * (*grad_loss_dev) * loss
 * + sum grad_gates * gates in the scores (the counts carry none).
 *
 *  counts, chosen, gates, live   as the forward wrote them.
 *  grad_gates    [tokens, top_k], or NULL: 0.
 *  grad_loss_dev one float on the device, or NULL for 1.
 *  dlogits       [tokens, experts] of dtype, row t at t * out_stride, written.
 */
#define ISO_MAX_EXPERTS 1024
#define ISO_MAX_TOP_K 32
size_t iso_balance_loss_workspace_bytes(int64_t tokens, int64_t experts);
iso_status iso_balance_loss(const void *logits, int dtype, int64_t tokens, int64_t experts,
                            int64_t stride, int top_k, const uint8_t *mask, int renormalize,
                            float *loss, int64_t *counts, int32_t *chosen, float *gates,
                            int64_t *live, void *workspace, size_t workspace_bytes, void *stream);
iso_status iso_balance_loss_backward(const void *logits, int dtype, int64_t tokens,
                                     int64_t experts, int64_t stride, int top_k,
                                     const uint8_t *mask, int renormalize, const int64_t *counts,
                                     const int32_t *chosen, const float *gates,
                                     const int64_t *live, const float *grad_gates,
                                     float grad_loss, const float *grad_loss_dev, void *dlogits,
                                     int64_t out_stride, void *stream);

/*
 * Optional per-kernel timing for benchmarks (not part of the fit).
 * iso_profile_enable(1) makes the library create a few CUDA events (once, on
 * first use; the only state the library keeps) and record one before the first
 * kernel of every later call of a computing entry point and one after each of
 * its kernels, on the call's stream.  iso_profile_enable(0) stops the recording.
 * iso_profile_read waits for the events of the most recent call and writes the
 * duration of each of its kernels in launch order (milliseconds, into ms[0..])
 * and a static name for each (names may be NULL); it returns the number of
 * kernels, or a negative iso_status.  Calls must not run concurrently from
 * several host threads while profiling is enabled.
 */
int iso_profile_enable(int on);
int iso_profile_read(float *ms, const char **names, int max_kernels);

/*
 * Depth of the long-row path's bridge searches (the paper's Section 5.2,
 * Theorem 5.2: the merge depth is bounded by a capped walk followed by a
 * nested bisection over the left hull's vertices, each tested against its
 * tangent point on the right hull).
 *
 * A merge of two segment lists (hull vertices in global memory) moves the
 * bridge's ends alternately to each other's tangent points; after
 * ISO_BRIDGE_MAX_PASSES passes (a pass moves both ends) it finishes with the
 * nested bisection, so no merge takes more than that many passes.  A merge of
 * two flat hulls in shared memory uses the nested bisection from the start,
 * 32 candidates per round, at most ISO_BRIDGE_MAX_ROUNDS rounds after the
 * first window of 32 vertices next to the shared point.
 *
 * iso_bridge_stats_mode (a debugging aid, off by default) makes later long-row
 * fits on the current device count their bridge searches:
 *   mode 0: off;
 *   mode 1: count;
 *   mode 2: count, with every segment-list bridge search taking the nested
 *           bisection from its first pass (to test that path on any input).
 * Switching on allocates the device's eight counters once (cudaMalloc) and
 * zeroes them.  Returns ISO_OK, ISO_ERR_INVALID_ARG for another mode, or
 * ISO_ERR_CUDA.  Calls on several host threads must not change the mode
 * concurrently.
 *
 * iso_bridge_stats_read synchronises the current device and copies its
 * counters into out[0..7] (host memory):
 *   [0] segment-list merges
 *   [1] of those, bridge searches (the chain is not convex at the shared point)
 *   [2] passes, summed over those searches
 *   [3] the most passes of one search (at most ISO_BRIDGE_MAX_PASSES)
 *   [4] searches that ended in the nested bisection
 *   [5] flat merges with a bridge search
 *   [6] the most narrowing rounds of one flat search (at most ISO_BRIDGE_MAX_ROUNDS)
 *   [7] flat searches whose rounds ran out before the bridge was found (0 with
 *       exactly convex hulls; nonzero would mean a wrong merge)
 * It returns ISO_OK, ISO_ERR_INVALID_ARG for a NULL out or counting that was
 * never switched on for the device, or ISO_ERR_CUDA.
 */
#define ISO_BRIDGE_MAX_PASSES 6
#define ISO_BRIDGE_MAX_ROUNDS 8
iso_status iso_bridge_stats_mode(int mode);
iso_status iso_bridge_stats_read(uint64_t *out);

#ifdef __cplusplus
}
#endif

#endif /* ISO_H */
