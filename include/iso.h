/*
 * iso.h - C ABI of the MI355X (gfx950) batched weighted isotonic-regression
 * library, libiso.so.
 *
 * The operation (paper "Merge Hulls Without Copying Vertices: GPU Isotonic
 * Regression", section 2.1, equations (1)-(3)): for every row y[0..n) with
 * weights w[0..n) > 0, compute the weighted least-squares non-decreasing fit
 *
 *     z* = argmin_{z_0 <= ... <= z_{n-1}}  sum_i w_i (z_i - y_i)^2 ,
 *
 * as the slope sequence of the lower convex hull of the cumulative sum diagram
 * P_k = (W_k, S_k), W_k = sum_{i<k} w_i, S_k = sum_{i<k} w_i y_i, P_0 = (0, 0):
 * z*_i is the slope of the hull edge above [W_i, W_{i+1}].  Rows are
 * independent problems of one common length (paper section 3, first paragraph;
 * rectangular batches only, section 6).
 *
 * Conventions shared by every entry point
 *   - y, w, out, block_id are DEVICE pointers (hipMalloc'd or torch CUDA
 *     tensors), row-major and contiguous: element (r, i) is at r*n + i.  They
 *     are caller-owned; the library never frees or retains them.
 *   - y, w, out are float32 and must be 4-byte aligned (the _f64 entry points:
 *     float64, 8-byte aligned); block_id is int32.
 *   - w == NULL means unit weights.
 *   - The fit is accumulated in f64 and each output value is rounded once to
 *     the output type (round to nearest even), as the paper's section 6
 *     ("Output") asks.  The output is not forced to be monotone (same
 *     section).
 *   - block_id (optional, NULL = not written): for each element, the 0-based
 *     index of its block (hull edge) within its row; non-decreasing along the
 *     row, +1 at every block start.  The paper's one-byte block-start flag
 *     (section 6, "Gradient") is block_id[i] != block_id[i-1].  Where adjacent
 *     blocks have equal means the library may split or pool them (a point on
 *     a hull edge changes no slope, section 4, after Corollary 4.5).
 *
 * Errors (return value; also see iso_status_str)
 *   ISO_OK               success.
 *   ISO_WARN_NONFINITE   some rows hold a NaN or infinity in y: those rows'
 *                        out is NaN and their block_id is -1; other rows are
 *                        exact.  (The paper keeps per-row NaN flags, section 6.)
 *   ISO_ERR_ARG          a NULL y or out, rows < 0 or n < 0, rows*n too large,
 *                        an output overlapping an input, or bad flags.
 *                        Nothing is launched.
 *   ISO_ERR_WEIGHT       some w_i <= 0 or non-finite (the problem needs
 *                        w_i > 0, section 2.1).  out is unspecified.
 *   ISO_ERR_NOMEM        iso_fit could not allocate its cached workspace.
 *                        Nothing launched; the HIP runtime's last-error
 *                        state that the failed hipMalloc set is cleared.
 *   ISO_ERR_HIP          a HIP runtime call or kernel launch failed.
 *   ISO_ERR_WORKSPACE    iso_fit_ex got a workspace smaller than
 *                        iso_workspace_bytes() asks for, or the shape needs
 *                        more than iso_fit_noalloc's ISO_NOALLOC_BYTES.
 *                        Nothing launched.
 *   ISO_ERR_DATA         iso_calib_fit got a non-finite score or outcome, or
 *                        (with segments) a negative score or segment id.
 *   ISO_ERR_INVARIANT    (ISO_F_DEBUG_INVARIANTS) a segment list of the merge
 *                        broke Definition 4.3 / Theorem 4.4 or the root
 *                        chain was not convex.
 *   rows == 0 or n == 0 is a no-op that returns ISO_OK.
 *
 * The two warning/error statuses that depend on the data (NONFINITE, WEIGHT)
 * are only reported when the call checks: iso_fit always does; iso_fit_ex
 * does unless ISO_F_NOCHECK is set (then it only enqueues work and returns
 * ISO_OK; NaN rows still come out NaN).
 */
#ifndef ISO_H
#define ISO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    ISO_OK = 0,
    ISO_WARN_NONFINITE = 1,
    ISO_ERR_ARG = -1,
    ISO_ERR_WEIGHT = -2,
    ISO_ERR_NOMEM = -3,
    ISO_ERR_HIP = -4,
    ISO_ERR_WORKSPACE = -5,
    ISO_ERR_DATA = -6,
    ISO_ERR_INVARIANT = -7
};

enum {
    /* Enqueue only: no device-to-host wait for the data checks. */
    ISO_F_NOCHECK = 1u,
    /* Non-increasing fit instead: the increasing fit of -y, negated (paper
     * section 2.1: the decreasing problem is the increasing one for -y). */
    ISO_F_DECREASING = 2u,
    /* Measurement control: merge the chunk hulls of long rows by copying the
     * surviving vertices at every level of the merge tree (the paper's
     * "grid copy" control, sections 7.3-7.4) instead of segment lists.  Same
     * result; more memory traffic.  Needs the larger workspace that
     * iso_workspace_bytes reports for this flag. */
    ISO_F_COPY_CONTROL = 4u,
    /* Tests: check the merge's segment lists on the device (paper section 4,
     * Definition 4.3, Theorem 4.4): after every segment-list merge level, each
     * list holds at most one segment per chunk of its range, in strictly
     * increasing chunk order, with lo <= hi; each row's root list starts at
     * the row's first point, ends at its last, keeps every segment inside its
     * chunk hull, and its vertices form a convex chain (no right turn beyond
     * rounding).  Also counts which merge paths ran.  The counters, 8 uint64,
     * sit at the end of the workspace (pass the flag to iso_workspace_bytes),
     * after any phase stamps: [0] violations, [1] chunk hulls rebuilt after
     * the chunk kernel gave up, [2] thread walks handed to a wave, [3] nested
     * bisections, [4] three-case searches, [5] levels checked, [6] root
     * vertices checked, [7] rounds of the second stage's bridges between
     * neighbouring groups that dropped a group.  A checked call returns
     * ISO_ERR_INVARIANT when [0] is not zero.  Long rows only; slower. */
    ISO_F_DEBUG_INVARIANTS = 8u,
    /* For iso_workspace_bytes only: size the workspace for a weighted call
     * (w != NULL).  Ignored by the fitting calls. */
    ISO_F_WEIGHTED_HINT = 0x100u,
    /* Measurement: on long rows, thread 0 of every workgroup of the chunk,
     * first-merge-stage, second-merge-stage and expansion kernels records the
     * device's 100 MHz real-time counter at its phase boundaries.  The stamps
     * take 64 bytes per workgroup at the end of the workspace (pass the flag to
     * iso_workspace_bytes too), from byte iso_workspace_bytes(rows, n, flags
     * without this bit) on: rows*m rows of 16 uint64 for the chunk kernel, then
     * rows*ng for the first merge stage (ng = ceil(m / 64)), rows for the
     * second stage, rows*m for the expansion (m = ceil(n / iso_chunk_size(n))).
     * Slots: chunk 0 start, 1 loads/sums/scan, 5 first quickhull level, 2 hull
     * built, 4 end; merge stages 0 start, 1 prelude, 2 merge tree, 3 lists and
     * windows written, 4 end, 5 + l node 0 through level l of a compact
     * merge tree; expansion 0 start, 1 record ready, 4 end.  Rows beyond the
 * two-stage merge use the second-stage row for the row merge: 0 start, 1
 * prelude done, 3 start of the levels left to one workgroup, 5 + (r - 6)
 * through tree level r, 2 tree done, 4 end. */
    ISO_F_PHASE_STAMPS = 0x200u,
    /* Merge-schedule variants (measurement and stress; paper section 7.4 and
     * appendix A).  Same result.  WAVE_MERGES: every merge of a segment-list
     * level is run by a wave (default: a thread per merge when a level has more
     * merges than the workgroup has waves, with walks that reach their cap
     * handed to waves).  THREE_CASE: at the levels with a thread per merge,
     * walks are capped at 8 (r + log2 C) steps (r the tree level, C the chunk
     * size) and finished by the three-case bridge search of Lemma A.1.  The
     * compact-array merges of short hulls are not affected.  TREE_MERGES: the
     * second stage merges short group hulls by the merge tree (default: the
     * bridges between neighbouring groups, all at once, with groups that keep
     * no vertex dropped round by round, and the tree after 8 such rounds). */
    ISO_F_WAVE_MERGES = 0x400u,
    ISO_F_THREE_CASE = 0x800u,
    ISO_F_TREE_MERGES = 0x1000u
};

/*
 * iso_fit - blocking fit on the null stream of the current device.
 *   y    [rows*n] f32, device.          w   [rows*n] f32 or NULL, device.
 *   out  [rows*n] f32, device, written.  May not overlap y or w.
 * Uses a workspace the library allocates once per device and grows on demand
 * (freed by iso_release).  Waits for the GPU and always runs the data checks.
 * Not safe to call concurrently from several host threads on one device.
 */
int iso_fit(const float* y, const float* w, int64_t rows, int64_t n, float* out);

/*
 * iso_fit_ex - the fit on a caller stream with a caller workspace.
 *   block_id        [rows*n] int32, device, or NULL.
 *   workspace       device buffer of at least iso_workspace_bytes(rows, n,
 *                   flags) bytes, 256-byte aligned; may be NULL only when
 *                   that size is 0.  Owned by the caller; its contents need
 *                   no initialisation and are scratch after the call.
 *   workspace_bytes its size.
 *   stream          a hipStream_t (NULL = the null stream).
 *   flags           ISO_F_* bits.
 * Without ISO_F_NOCHECK the call synchronises with `stream` to read the
 * device's per-row data flags.  Calls that share one workspace must not
 * overlap in time.
 */
int iso_fit_ex(const float* y, const float* w, int64_t rows, int64_t n, float* out,
               int32_t* block_id, void* workspace, size_t workspace_bytes, void* stream,
               uint32_t flags);

/*
 * iso_fit_ex_f64, iso_fit_f64 - the same fits with f64 y, w and out (8-byte
 * aligned), through the same kernels (the paper's operator takes f32 and f64
 * in one code path, section 6).  Every sum and predicate is f64 either way;
 * with f64 input the products w_i y_i are rounded in f64, and each output is
 * the f64 slope itself.  The workspace is the same as for f32
 * (iso_workspace_bytes).  Statuses and flags as for iso_fit_ex / iso_fit.
 */
int iso_fit_ex_f64(const double* y, const double* w, int64_t rows, int64_t n, double* out,
                   int32_t* block_id, void* workspace, size_t workspace_bytes, void* stream,
                   uint32_t flags);
int iso_fit_f64(const double* y, const double* w, int64_t rows, int64_t n, double* out);

/*
 * iso_fit_noalloc - iso_fit_ex without a caller workspace and without any
 * allocation, for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc).
 *   y, w, out, block_id, stream, flags as for iso_fit_ex.
 * The workspace is a fixed device array of ISO_NOALLOC_BYTES that the library
 * holds on every device it runs on until the process ends; shapes whose
 * iso_workspace_bytes exceeds it return ISO_ERR_WORKSPACE with nothing
 * launched.  The call never calls hipMalloc, hipFree or any other allocating
 * routine (host or device); its first call on a device looks up the array's
 * device address once.  Every call on one device shares that array and leaves
 * its contents in it (the kernels need no initialised workspace), so calls on
 * one device must not overlap in time: overlapping calls race on it.  Without
 * ISO_F_NOCHECK the call synchronises with `stream` (not capturable then);
 * with it the call only enqueues work.
 */
#define ISO_NOALLOC_BYTES (64u << 20)
int iso_fit_noalloc(const float* y, const float* w, int64_t rows, int64_t n, float* out,
                    int32_t* block_id, void* stream, uint32_t flags);

/*
 * iso_vjp - the backward pass: the vector-Jacobian product of the fit (paper
 * section 6, paragraph "Gradient"; validated as its appendix C describes).
 * The fit is constant on its blocks, each block's value the weighted mean z of
 * y over the block, so for an element i with G and W the sums of g and of w
 * over its block:
 *     grad_y[i] = w_i G / W ,        grad_w[i] = (y_i - z) G / W
 * (wherever the blocks do not change; at a boundary between equal means the
 * fit is not differentiable and the blocks of the forward call are used).
 *   g         [rows*n] f32, device: the gradient with respect to the fit.
 *   y         [rows*n] f32, device: the forward call's y; needed only for
 *             grad_w (may be NULL when grad_w is NULL).
 *   w         [rows*n] f32, device: the forward call's weights, or NULL for
 *             unit weights.
 *   block_id  [rows*n] int32, device: the block ids the forward call wrote
 *             (iso_fit_ex or iso_fit_noalloc with a block_id buffer), for the
 *             same y, w and flags.  A block starts at a row's first element
 *             and wherever the id changes.  A row whose ids are negative (a
 *             non-finite row of the forward call) gets NaN gradients.
 *   grad_y    [rows*n] f32, device, written, or NULL.
 *   grad_w    [rows*n] f32, device, written, or NULL (needs y and w).
 *   workspace device buffer of iso_vjp_workspace_bytes(rows, n) bytes,
 *             256-byte aligned, contents need no initialisation (NULL when
 *             that size is 0: rows of at most 2048 elements).
 *   stream    hipStream_t (NULL = the null stream).  The call only enqueues.
 * A decreasing fit (ISO_F_DECREASING) has the same gradient formulas in y and
 * w, so the same call serves it.  Sums are f64, without atomics (the result
 * does not depend on scheduling); each output is rounded once to f32.
 * Returns ISO_OK, ISO_ERR_ARG (NULL g or block_id, no output, grad_w without y
 * or w, misaligned or overlapping buffers, bad sizes), ISO_ERR_WORKSPACE or
 * ISO_ERR_HIP; nothing is launched on an error.
 */
int iso_vjp(const float* g, const float* y, const float* w, const int32_t* block_id, int64_t rows,
            int64_t n, float* grad_y, float* grad_w, void* workspace, size_t workspace_bytes,
            void* stream);

/* The same with f64 g, y, w and gradients (8-byte aligned). */
int iso_vjp_f64(const double* g, const double* y, const double* w, const int32_t* block_id,
                int64_t rows, int64_t n, double* grad_y, double* grad_w, void* workspace,
                size_t workspace_bytes, void* stream);

/* Bytes of device workspace iso_vjp and iso_vjp_f64 need for this shape (0 for
 * rows of at most 2048 elements, or an empty or invalid shape). */
size_t iso_vjp_workspace_bytes(int64_t rows, int64_t n);

/*
 * Calibration front end (paper section 7.7, "Case study: calibrating a click
 * model"; the blog note's lab notebook, calibration cells), all f64.
 *
 * iso_calib_fit - an isotonic calibration curve from n scores and outcomes:
 *   1. each score is keyed: the score itself, or with segments
 *      segment[i] + min(score, 1 - 1e-12) (one curve per segment, all fitted
 *      as one problem laid end to end);
 *   2. the keys are sorted with their outcomes;
 *   3. equal keys are pooled: xp[r] is the r-th distinct key, with the count
 *      and the mean of the outcomes of its scores;
 *   4. with segments, each mean is lifted by twice its segment index, so that
 *      no block of the fit reaches across a segment boundary;
 *   5. the means are fitted, the counts as weights, by the f64 fit;
 *   6. the lift is dropped again: fp[r] is the curve at xp[r].
 *   scores, outcomes [n] f64, device.  segment [n] int32 >= 0, device, or NULL.
 *   xp, fp   [n] f64, device, written: the first *k_out entries are the curve.
 *   k_out    host pointer: the number of distinct keys.
 *   workspace device buffer of iso_calib_workspace_bytes(n) bytes, 256-byte
 *            aligned, contents need no initialisation.
 *   stream   hipStream_t (NULL = the null stream).
 * The call waits for the GPU once (for the number of distinct keys).  Returns
 * ISO_OK, ISO_ERR_ARG, ISO_ERR_DATA (non-finite score or outcome; with
 * segments a negative score or segment id), ISO_ERR_WORKSPACE or ISO_ERR_HIP.
 *
 * iso_calib_apply - the curve (xp, fp) of k distinct keys at m new scores:
 * the key of each score (as above; with segment != NULL the search stays in
 * that segment's keys), linear interpolation between the two keys around it,
 * held at the end values outside them.  A query whose segment has no keys, or
 * whose score is NaN, gets NaN.  Only enqueues.  Returns ISO_OK, ISO_ERR_ARG
 * or ISO_ERR_HIP.
 *
 * iso_calib_workspace_bytes - workspace of iso_calib_fit for n scores (0 for
 * an invalid n); queries the current device's sort configuration.
 */
int iso_calib_fit(const double* scores, const double* outcomes, const int32_t* segment, int64_t n,
                  double* xp, double* fp, int64_t* k_out, void* workspace, size_t workspace_bytes,
                  void* stream);
int iso_calib_apply(const double* xp, const double* fp, int64_t k, const double* scores,
                    const int32_t* segment, int64_t m, double* out, void* stream);
size_t iso_calib_workspace_bytes(int64_t n);

/*
 * Post-training losses: what turns calibrated rewards or preferences into
 * gradients of a language model (calibrated scores: iso_calib_apply above).
 * Token log-probabilities from logits with their backward pass, a paired
 * preference loss, a clipped policy loss with a KL term, and the policy loss
 * taken from the logits.  Logits are f32, f16 or bf16 (ISO_DT_*); every other
 * real array is f32.  The terms of softmax sums are f32, the sums f64 (an
 * entropy's are f32 over at most 32 terms of a thread, f64 beyond); the losses'
 * sums are f64; each output is rounded once.  No atomics on values: results do
 * not depend on scheduling.  The calls only enqueue work on `stream` (they may be captured
 * into a graph), allocate nothing, and use a caller workspace (256-byte
 * aligned, no initialisation) of the size the matching *_workspace_bytes
 * gives.  Statuses: ISO_OK, ISO_ERR_ARG, ISO_ERR_WORKSPACE, ISO_ERR_HIP;
 * nothing is launched on an error.
 *
 * iso_token_logp - for each row t of logits, with x = logits[t] / temperature
 * and target j = target[t]:
 *     lse[t]     = log sum_k exp(x_k) ,       logp[t] = x_j - lse[t] ,
 *     entropy[t] = lse[t] - sum_k p_k x_k ,   p_k = exp(x_k - lse[t]) .
 *   logits  [rows][vocab] of `dtype`, device, row r at r*ld elements, aligned
 *           to its element size; ld >= vocab (>= 1; at most 2^30).
 *   target  [rows] int32, device.  A negative target marks an ignored row: the
 *           row is not read and its outputs are 0.  A target >= vocab gives
 *           NaN logp.
 *   logp, lse [rows] f32, written.  entropy [rows] f32, written, or NULL.
 *   temperature from 1e-28 to 1e28.
 * A logit of -infinity (or far below the row's maximum) is a masked entry and
 * adds nothing.  A row with a NaN or +infinity, or of -infinity alone, has no
 * distribution: its outputs are NaN.
 *
 * iso_token_logp_vjp - the gradient of the logits, for gradients g_logp of
 * logp and g_entropy of the entropy (NULL: none):
 *     grad_k = ( g_logp ([k = j] - p_k) - g_entropy p_k (x_k - lse + entropy) ) / temperature .
 *   lse     [rows] f32: the forward call's.  entropy [rows] f32: the forward
 *           call's (needed with g_entropy only).  p is taken at this lse: its
 *           rounding to f32 is a relative |lse| 2^-24 of p, much at a small
 *           temperature (iso_policy_loss_logits does not round it).
 *   grad    [rows][vocab] of `dtype`, row r at r*ld_grad, written.  It may be
 *           the logits themselves (same pointer and ld): the gradient then
 *           takes the logits' place; any other overlap is an error.  Columns
 *           past vocab are not touched.
 * Ignored rows get zeros.  A row whose target is >= vocab gets NaN.  A masked
 * entry's gradient is 0 while g_logp and 200 g_entropy over temperature are
 * inside f32.
 */
enum { ISO_DT_F32 = 0, ISO_DT_F16 = 1, ISO_DT_BF16 = 2 };
size_t iso_token_logp_workspace_bytes(int64_t rows, int64_t vocab, int dtype);
int iso_token_logp(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                   const int32_t* target, double temperature, float* logp, float* lse,
                   float* entropy, void* workspace, size_t workspace_bytes, void* stream);
int iso_token_logp_vjp(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                       const int32_t* target, double temperature, const float* lse,
                       const float* entropy, const float* g_logp, const float* g_entropy,
                       void* grad, int64_t ld_grad, void* stream);

/*
 * Sequences of tokens, in both losses: packed one after another, sequence q
 * the tokens seq_off[q] .. seq_off[q+1]-1 (seq_off [seqs+1] int32, device,
 * non-decreasing, from 0 to `tokens`); with seq_off NULL all have the length
 * tokens / seqs (which must divide).  Offsets that break this are held inside
 * [0, tokens]: nothing outside the arrays is touched, the outputs are then
 * unspecified.  mask [tokens] bytes, device, or NULL: a token with mask 0
 * takes no part, whatever its values (NaN included), and its gradient is 0.
 * A sequence may be empty or wholly masked.  Tokens without a sequence are an
 * error.  tokens is at most 2^31 - 1.
 *
 * iso_pref_loss - the paired preference loss.  Sequence 2i is pair i's chosen
 * answer, 2i+1 its rejected one.  With s_q the sum over q's tokens of
 * logp - ref_logp (ISO_PREF_MEAN: divided by the number of unmasked tokens),
 * D = s_2i - s_2i+1 and e = label_smoothing:
 *     l_i = -(1-e) log sigma(beta D) - e log sigma(-beta D) ,
 *     ISO_PREF_SQUARED:  l_i = (D - 1 / (2 beta))^2 ,
 *     loss = (1 / pairs) sum_i l_i .
 *   logp, ref_logp [tokens] f32 (ref_logp NULL: no reference, zeros).
 *   beta > 0; label_smoothing in [0, 1/2] (0 with ISO_PREF_SQUARED).
 *   loss      [1], written (0 when pairs is 0).  pair_loss [pairs] = l_i,
 *             written.  reward [2 pairs] = beta s_q, written.
 *   grad      [tokens], written, or NULL: grad_scale times the gradient of
 *             loss with respect to logp.
 *
 * iso_policy_loss - the clipped policy loss.  Per token, with A its advantage,
 * d = logp - old_logp, r = exp(d), u = ref_logp - logp:
 *     pg = -min(r A, clip(r, 1 - clip_lo, 1 + clip_hi) A) ,
 *     kl = exp(u) - u - 1      (0 without ref_logp) ,
 *     loss = sum_t w_t (pg_t + kl_coef kl_t) ,
 *   w_t = 1 / (unmasked tokens), or with ISO_POLICY_SEQ_MEAN
 *   1 / (seqs * unmasked tokens of its sequence); a norm > 0 takes the place of
 *   the count of tokens, or of seqs (for sums over several calls).
 *   adv       [seqs] f32, or [tokens] with ISO_POLICY_ADV_TOKEN.
 *   clip_lo in [0, 1], clip_hi >= 0 (may be infinite), kl_coef finite (0
 *   without ref_logp; 0 with it: the reference is only watched, kl is summed into
 *   loss[2] and reaches neither the loss nor its gradient, whatever it is).
 *   loss      [3] f32, written: the loss, its part sum w pg, and sum w kl.
 *   counts    [2] int32, written: unmasked tokens, and those the clip holds
 *             (A > 0 and d > log(1 + clip_hi), or A < 0 and
 *             d < log(1 - clip_lo)): their pg has gradient 0.
 *   grad      [tokens], written, or NULL: grad_scale times the gradient of
 *             loss with respect to logp.
 *
 * iso_policy_loss_logits - token_logp, the policy loss and the gradient of the
 * logits in one call: rows of logits are the tokens, ignored rows (target < 0)
 * the masked ones.  Arguments as above; logp [rows] f32 is written (0 on
 * ignored rows), grad as in iso_token_logp_vjp (may be the logits; NULL for
 * the loss alone).
 */
enum { ISO_PREF_MEAN = 1u, ISO_PREF_SQUARED = 2u };
enum { ISO_POLICY_SEQ_MEAN = 1u, ISO_POLICY_ADV_TOKEN = 2u };
size_t iso_pref_loss_workspace_bytes(int64_t tokens, int64_t pairs);
int iso_pref_loss(const float* logp, const float* ref_logp, const uint8_t* mask,
                  const int32_t* seq_off, int64_t pairs, int64_t tokens, double beta,
                  double label_smoothing, float* loss, float* pair_loss, float* reward, float* grad,
                  double grad_scale, void* workspace, size_t workspace_bytes, void* stream,
                  uint32_t flags);
size_t iso_policy_loss_workspace_bytes(int64_t tokens, int64_t seqs);
int iso_policy_loss(const float* logp, const float* old_logp, const float* ref_logp,
                    const float* adv, const uint8_t* mask, const int32_t* seq_off, int64_t seqs,
                    int64_t tokens, double clip_lo, double clip_hi, double kl_coef, double norm,
                    float* loss, int32_t* counts, float* grad, double grad_scale, void* workspace,
                    size_t workspace_bytes, void* stream, uint32_t flags);
size_t iso_policy_loss_logits_workspace_bytes(int64_t rows, int64_t vocab, int64_t seqs, int dtype);
int iso_policy_loss_logits(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                           const int32_t* target, double temperature, const float* old_logp,
                           const float* ref_logp, const float* adv, const int32_t* seq_off,
                           int64_t seqs, double clip_lo, double clip_hi, double kl_coef, double norm,
                           float* loss, int32_t* counts, float* logp, void* grad, int64_t ld_grad,
                           double grad_scale, void* workspace, size_t workspace_bytes, void* stream,
                           uint32_t flags);

/*
 * Decoding steps: what makes the answers that the losses above compare, and
 * keeps their states apart while they are made.  Beam search's selection from
 * logits, the states of beams brought into the order of their parents, a paged
 * cache's sequences forked, grown and freed, and its live pages moved together.
 * The calls only enqueue work on `stream` (they may be captured into a graph),
 * allocate nothing, and results do not depend on scheduling.  Statuses: ISO_OK,
 * ISO_ERR_ARG, ISO_ERR_WORKSPACE, ISO_ERR_HIP; nothing is launched on an error.
 * Workspaces as for the losses (256-byte aligned, no initialisation).
 *
 * iso_beam_select - the best continuations of each batch item's beams.  Row
 * r = b * beams + k of logits is beam k of item b.  With z = logits[r] /
 * temperature and lse = log sum_v exp(z_v), the candidates of a beam are
 *     token v:   logp = z_v - lse ,   s = score[r] + logp      (logits[r][v] > -infinity) ,
 * and of an ended beam (ended[r] != 0) itself alone: end_token, logp = 0,
 * s = score[r].  They are ranked by s * weight[r], rounded to f32; equal ranks
 * by the lower beam, then the higher logit, then the lower token.  The first
 * `take` of each item are written in this order.
 *   logits   as for iso_token_logp, batch * beams rows.  The rows of ended
 *            beams are not read.
 *   score    [batch*beams] f32.  A beam whose score is not finite has no
 *            candidates and is not read (-infinity for all beams but one: the
 *            first step, where all are alike).
 *   weight   [batch*beams] f32, or NULL (1): the rank's factor, as 1 / length^a.
 *            A beam whose weight is not positive and finite has no candidates.
 *   ended    [batch*beams] bytes, or NULL.
 *   beams, take  from 1 to 128.
 *   out_score, out_logp [batch*take] f32, written: s and logp.  out_parent
 *            [batch*take] int32: the candidate's row, b * beams + k (what
 *            iso_beam_reorder and iso_pages_fork take).  out_token
 *            [batch*take] int32.  Places past an item's last candidate hold
 *            -infinity, -infinity, -1 and -1.
 * A row with a NaN or +infinity, or of -infinity alone, has no candidates, nor
 * has what ranks at -infinity (below f32).  Terms of sums are f32, the sums f64,
 * but that up to eight terms below half of the largest are added in f32 first;
 * the score and the rank are f64 until they are rounded.  How a row's terms are
 * grouped goes by its address modulo 16.  Tokens are masked by -infinity: a finite
 * value gives the same answers, but where stretches of some thousand tokens hold
 * nothing else, `take` passes over each of them.
 *
 * Arrays of states.  An iso_blocks describes, for rows (beams) or pages, the
 * blocks row r holds: `inner` bytes each, block (o, m) at
 *     base + o * outer_stride + r * row_stride + m * mid_stride ,
 * o < outer, m < mid, strides in bytes (not negative; of a count of 1 they are
 * not used).  A cache [layers][rows][heads][room][dim] whose first t tokens
 * count has outer = layers, mid = heads, inner = t * dim * element size.
 * Blocks may not overlap; arrays of one call may not either, from the first to
 * the last byte each (two interleaved arrays are one, with a larger outer or
 * mid).  At most ISO_MAX_BLOCKS arrays a call (a launch for every 16); any element
 * type and alignment.
 *
 * iso_beam_reorder - row r of every array becomes what row parent[r] was, in
 * place.  parent [batch*beams] int32: a row of the same item (r / beams); any
 * other value, and r itself, leaves the row as it is.  beams from 1 to 128.
 * Rows that stay are not written, those nobody comes from not read.
 *
 * iso_pages_fork - one step of a paged cache.  A page holds page_size tokens.
 * Sequence s has length[s] tokens, in the pages table[s][0 ..
 * ceil(length[s] / page_size)); refs[p] counts the entries, in this table or
 * outside it, that hold page p; a page of 0 is free.  Child i goes on from
 * sequence parent[i] (any value outside [0, seqs): a new sequence of length 0)
 * and has room for grow[i] more tokens:
 *     new_length[i] = length[parent[i]] + grow[i]
 * (a negative grow counts as 0).  A sequence with several children is forked,
 * one with none is freed.  Pages are shared, but for the one that a growing
 * child goes on to write, where its parent's tokens end inside a page: the
 * first such child (in order) keeps it if nobody but such children holds it,
 * the others have copies of its tokens.  Pages for copies and growth are the
 * lowest free ones (pages this call frees among them), in the children's order.
 *   table [seqs][max_pages] int32, length [seqs] int32, refs [pages] int32: the
 *            cache before the step, left as they are.
 *   parent [children] int32.  grow [children] int32, or NULL: grow_all each.
 *   pools    the arrays that hold the pages' tokens: rows are pages, a block's
 *            inner bytes are page_size tokens (inner a multiple of page_size).
 *            Copied tokens are written, nothing else.  May be NULL with count 0.
 *   new_table [children][max_pages], new_length [children], new_refs [pages],
 *            written: the cache after the step (entries without a page: -1).
 *   status [5] int32, written: pages lacking, children longer than max_pages
 *            allow, pages copied, pages taken, pages left free.
 * If one of the first two is not 0 nothing is done: new_length is 0, new_table
 * -1, new_refs is refs, the other statuses are 0, no token is copied, and the old
 * cache stands.
 * What breaks the above is held inside the arrays: lengths to [0, max_pages *
 * page_size], negative refs to 0, an entry outside [0, pages) holds no page.  Where
 * refs are below what the tables hold, a page that children go on to write has
 * them as holders at least, and other counts end at 0: such a page is free, also
 * where a table still holds it.  Counts stay below 2^31, after the step too.
 * seqs and children at most 2^20.
 *
 * iso_pages_compact - the live pages (refs > 0) moved together: with n of them,
 * those at n and beyond go, in order, to the free ones below n.
 *   table [entries] int32, any shape; entries outside [0, pages) become -1.
 *   new_table [entries], new_refs [pages], written.  moved [pages] int32,
 *            written: where each page is now, -1 for the free ones.
 *   pools    as above; whole pages are moved, in place.
 *   status [2] int32, written: live pages, pages moved.
 */
#define ISO_MAX_BLOCKS 512
typedef struct iso_blocks {
    void* base;
    int64_t outer, outer_stride, row_stride, mid, mid_stride, inner;
} iso_blocks;
size_t iso_beam_select_workspace_bytes(int64_t batch, int64_t beams, int64_t vocab, int64_t take,
                                       int dtype);
int iso_beam_select(const void* logits, int dtype, int64_t batch, int64_t beams, int64_t vocab,
                    int64_t ld, const float* score, const float* weight, const uint8_t* ended,
                    int32_t end_token, double temperature, int64_t take, float* out_score,
                    float* out_logp, int32_t* out_parent, int32_t* out_token, void* workspace,
                    size_t workspace_bytes, void* stream);
int iso_beam_reorder(const iso_blocks* states, int count, const int32_t* parent, int64_t batch,
                     int64_t beams, void* stream);
size_t iso_pages_fork_workspace_bytes(int64_t seqs, int64_t children, int64_t pages);
int iso_pages_fork(const int32_t* table, const int32_t* length, int64_t seqs, int64_t max_pages,
                   const int32_t* refs, int64_t pages, int64_t page_size, const int32_t* parent,
                   const int32_t* grow, int32_t grow_all, int64_t children, const iso_blocks* pools,
                   int count, int32_t* new_table, int32_t* new_length, int32_t* new_refs,
                   int32_t* status, void* workspace, size_t workspace_bytes, void* stream);
size_t iso_pages_compact_workspace_bytes(int64_t pages);
int iso_pages_compact(const int32_t* table, int64_t entries, const int32_t* refs, int64_t pages,
                      const iso_blocks* pools, int count, int32_t* new_table, int32_t* new_refs,
                      int32_t* moved, int32_t* status, void* workspace, size_t workspace_bytes,
                      void* stream);

/* Bytes of device workspace iso_fit_ex needs for this shape and these flags
 * (weighted or not is part of the shape: pass ISO_F_WEIGHTED_HINT in flags
 * when w will be non-NULL).  Returns 0 for an empty or invalid shape. */
size_t iso_workspace_bytes(int64_t rows, int64_t n, uint32_t flags);

/* A static English description of a status code. */
const char* iso_status_str(int status);

/* Frees the workspace that iso_fit caches on each device it has used. */
void iso_release(void);

/* Chunk size (points per chunk hull) that long rows of length n use; rows
 * with n at most iso_short_row_max() are fitted whole by one workgroup. */
int64_t iso_chunk_size(int64_t n);
int64_t iso_short_row_max(void);

/*
 * Measurement hooks (for benchmarks; not needed to fit).  After
 * iso_timing_enable(1), every fitting call made from any host thread records a
 * HIP event on its stream before each of its kernel launches and after the
 * last, so each launch's device duration can be read.  iso_timing_read waits
 * for the recorded events, adds each launch's duration (ms) to
 * ms[phase] and 1 to launches[phase] for its phase (ISO_PHASE_*), for phase <
 * nphase, clears the record and returns the number of launches read (or
 * ISO_ERR_HIP).  Enabling adds the event records to the stream and so may
 * widen the gaps between launches; iso_timing_enable(0) stops recording.
 */
enum {
    ISO_PHASE_SHORT_ROWS = 0,  /* whole short rows in one kernel          */
    ISO_PHASE_CHUNK_HULLS = 1, /* prefix sums, chunk hulls, chunk slots   */
    ISO_PHASE_MERGE = 2,       /* segment-list merge (first stage) or its control's set-up */
    ISO_PHASE_EXPAND = 3,      /* slope expansion (the fit)               */
    ISO_PHASE_COPY_BRIDGE = 4, /* copy control: bridges of one level      */
    ISO_PHASE_COPY_MOVE = 5,   /* copy control: vertex rewrite of a level */
    ISO_PHASE_MERGE_TOP = 6,   /* second merge stage (group hulls of a row) */
    ISO_PHASE_CHUNK_REDO = 7,  /* chunk hulls the first chunk kernel left over */
    ISO_PHASE_COUNT = 8
};
int iso_timing_enable(int on);

/* Measurement probe: a plain streaming copy of `bytes` (a multiple of 16;
 * src and dst 16-byte aligned device buffers that do not overlap) on `stream`,
 * the practical HBM bandwidth ceiling the fit's kernels are measured against.
 * Only enqueues.  Returns ISO_OK, ISO_ERR_ARG or ISO_ERR_HIP. */
int iso_copy_probe(const void* src, void* dst, size_t bytes, void* stream);
int iso_timing_read(double* ms, int64_t* launches, int nphase);

#ifdef __cplusplus
}
#endif

#endif /* ISO_H */
