/*
 * rk.h -- device-wide mapreduce for AMD Instinct MI355X (gfx950).
 *
 * A C ABI over hand-written HIP kernels.  It computes the mapped reductions
 * described on the AcceleratedKernels.jl pull-request pages:
 *
 *   - PR #139, "Finish whole-array reductions on the device": a whole array
 *     is reduced in at most two launches (a grid-capped first pass whose
 *     blocks stride over tiles, then a one-block second pass); the last pass
 *     applies `init`, or folds into the output's previous value, or leaves a
 *     bare partial that the host finishes (sections "What changes" and
 *     "Compatibility").
 *   - PR #176, strided reductions along dims: one selector picks among one
 *     thread per output, a tiled 2-d block and a split columns kernel, and
 *     the columns kernel also takes runs of contiguous outputs such as the
 *     middle dim of a 3-d array (section "This PR").
 *   - a two-input source f(a_i, b_i) on the whole-array passes
 *     (rk_reduce_all2), and scans, the prefix folds of PR #202 (rk_scan,
 *     rk_scan_dims).
 *
 * Beside them stand the reductions and scans that a language model's serving
 * step makes around its model: softmax of lines (rk_softmax), verification of
 * drafted tokens (rk_draft_verify), block tables and slot maps
 * (rk_block_tables, rk_slot_map); their arguments are described with them.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Arrays are column-major (Julia semantics).  `shape[d]` is the extent of
 * dim d and `strides[d]` its stride in ELEMENTS (>= 0); a contiguous
 * (d1, d2, d3) array has strides (1, d1, d1*d2).  Bit d of `reduce_mask`
 * marks dim d (0-based) as reduced, so Julia's `dims=k` is bit k-1.  The
 * outputs are the kept dims, stored contiguously in column-major order (the
 * reduced dims behave as extent 1).
 *
 * The result for each output is  R = s (+) f(x_0) (+) f(x_1) (+) ...  where
 * (+) is the op, f the map applied after widening an element to the
 * accumulator type, and s the starting value chosen by the mode:
 *   RK_MODE_OVERWRITE  s = *init (the op's identity when init is NULL); the
 *                      result is stored into the device array `out`;
 *   RK_MODE_FOLD       s = the previous value of out[o], read back into the
 *                      accumulator type; `init` is ignored, so an init that
 *                      was applied by an earlier call is not applied again;
 *   RK_MODE_HOST       s = *init (or identity); the GPU leaves a bare
 *                      accumulator-typed partial in a small pinned host
 *                      buffer the library keeps per host thread (or, without
 *                      one, in the workspace, copied back), and the host
 *                      finishes it; `out` is a HOST pointer and the call
 *                      returns after the stream has drained.  Valid only when
 *                      there is a single output.  Setting the environment
 *                      variable RK_HOST_COPY before the first host-mode call
 *                      of a thread selects the copy.
 * `init` is applied exactly once.  Partial results keep the accumulator type
 * until the final store, which converts once to the output type (round to
 * nearest even for floating point, two's-complement wrap for integers).  The
 * output is never used to hold intermediate values.  The association order
 * is the library's own, so floating-point results may differ from a
 * sequential loop by rounding.  Identities: 0 for sum, -inf / the
 * accumulator's minimum integer for max, +inf / its maximum for min.  max
 * and min propagate NaN.
 *
 * Dtype combinations: the input and accumulator are both floating point or
 * both integer, and the accumulator is at least as wide as the input
 * (f32 -> f32|f64, bf16 -> f32|f64, f16 -> f32|f64, f64 -> f64,
 * i32 -> i32|i64, i64 -> i64).  The output has the accumulator's kind and any
 * width of that kind; it may be narrower than the accumulator.
 *
 * Ownership: the caller owns every buffer (`ptr`, `out`, `workspace`).  The
 * library allocates and frees no device memory; its per-stream slots are
 * static device memory of its code objects (about 42 MB per device, loaded
 * with the library).  Kernels are enqueued on
 * `stream` (a hipStream_t; NULL is the null stream) of the current device.
 * OVERWRITE and FOLD calls are asynchronous: buffers must stay alive until
 * the stream's work has completed.  Between calls the library keeps only
 * cached device properties and, per (device, stream), a slot of state in its
 * own device memory, so a reduction split across blocks finishes inside its
 * one launch: a whole-array pass's blocks store their partials tagged with
 * the call's number and block 0 collects them; split dims reductions count
 * arrivals on counters that return to zero by themselves.  Calls from several host threads are
 * safe; two calls that share a workspace must be ordered by the caller.
 *
 * Graph capture: OVERWRITE and FOLD calls enqueue kernels only (no memset,
 * no copy, no allocation), so they may be captured into a HIP graph and the
 * graph replayed.  Captured kernels keep the slot of the stream they were
 * captured on: replays of one graph must not overlap each other or calls on
 * that capture stream.  HOST mode waits on the stream and cannot be captured.
 *
 * Errors: every argument is validated before any launch; a rejected call
 * returns a non-zero rk_status and writes nothing.  A HIP launch failure is
 * reported as RK_ERR_HIP.  The library prints nothing unless the environment
 * variable RK_DEBUG is set.
 *
 * Waits inside a launch: block 0 of a whole-array pass waits for the other
 * blocks' partials, and a scan tile waits for its predecessors' prefixes.  No
 * block waits on the block that waits for it, so these waits end; as a
 * safety net each is bounded (about a second).  A wait that gives up stores
 * no result (out keeps its previous contents; a scan's outputs after that
 * tile are wrong) and is counted: HOST mode then returns RK_ERR_HIP, and
 * rk_stream_timeouts reports the count for OVERWRITE, FOLD and scan calls.
 */
#ifndef RK_H
#define RK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    RK_OK = 0,
    RK_ERR_INVALID_ARGUMENT = 1, /* bad pointer, size, shape, mask, mode or alignment */
    RK_ERR_UNSUPPORTED = 2,      /* dtype combination outside the table above */
    RK_ERR_HIP = 3,              /* the HIP runtime reported an error */
    RK_ERR_TOO_LARGE = 4         /* rk_reduce_dims_no_workspace: the call needs more than the scratch */
} rk_status;

typedef enum { RK_OP_SUM = 0, RK_OP_MAX = 1, RK_OP_MIN = 2 } rk_op;

/* Element map f, applied after widening to the accumulator type (the `f` of
 * mapreduce(f, op, A); PR #139, opening section).  Integer maps wrap in the
 * accumulator type. */
typedef enum { RK_MAP_IDENTITY = 0, RK_MAP_SQUARE = 1, RK_MAP_ABS = 2 } rk_map;

/* Two-input map f(a, b) of a fused source (rk_reduce_all2), applied after
 * widening both elements to the accumulator type; integer forms wrap in the
 * accumulator type. */
typedef enum { RK_MAP2_MUL = 0, RK_MAP2_SQDIFF = 1, RK_MAP2_ABSDIFF = 2 } rk_map2;

typedef enum {
    RK_F32 = 0, RK_BF16 = 1, RK_F16 = 2, RK_F64 = 3, RK_I32 = 4, RK_I64 = 5
} rk_dtype;

typedef enum { RK_MODE_OVERWRITE = 0, RK_MODE_FOLD = 1, RK_MODE_HOST = 2 } rk_mode;

/*
 * Bytes of device workspace that rk_reduce_all (ndim = 1, reduce_mask = 1,
 * strides[0] = 1, shape[0] = n) or rk_reduce_dims needs for this layout on the
 * current device.  For a whole array this is one accumulator per first-pass
 * block plus one for the bare final partial (PR #139, "What changes": the
 * workspace holds target_blocks + 1 partial results) and a 4-byte word for
 * host mode's copied-back result, rounded up to 256
 * bytes; for a dims reduction split across blocks it is split * n_out
 * accumulators; otherwise 0.  The contents need not be initialised and the
 * same workspace may be reused by later calls of any shape and type.
 * Returns 0 for invalid arguments as well.
 */
size_t rk_workspace_size(int in_dtype, int acc_dtype, int ndim, const int64_t *shape,
                         const int64_t *strides, uint32_t reduce_mask);

/*
 * Whole-array mapped reduction of n contiguous elements at `ptr` (device
 * pointer, aligned to its element size; it need not be 16-byte aligned, so
 * offset views work).  PR #139, "What changes": at most two launches, one
 * launch when the input fits one block.  Here a larger input also takes one
 * launch: the last first-pass block to arrive folds the partials (it falls
 * back to the one-block second launch when its stream has no counter slot).
 *   init      host pointer to one accumulator-typed value, or NULL.
 *   mode      RK_MODE_OVERWRITE / RK_MODE_FOLD: `out` is a device pointer to
 *             one out-typed element; RK_MODE_HOST: `out` is a host pointer to
 *             one out-typed element, written before the call returns.
 *   workspace device pointer to >= rk_workspace_size bytes, aligned to 8
 *             bytes (may be NULL only if that size is 0).
 *   stream    hipStream_t or NULL.
 * n = 0 gives the starting value s.  Returns an rk_status.
 */
int rk_reduce_all(int op, int map, int in_dtype, int acc_dtype, int out_dtype,
                  const void *ptr, int64_t n, const void *init, int mode, void *out,
                  void *workspace, void *stream);

/*
 * Whole-array reduction of a fused two-input source: R = s (+) f(a_0, b_0)
 * (+) f(a_1, b_1) (+) ..., f one of rk_map2 -- a dot product, a squared or an
 * absolute distance.  PR #139, "What changes": the whole-array path takes a
 * lazy broadcast as its source, and the page's test list covers fused
 * sources; this is the broadcast of two arrays through f, read in one pass
 * with nothing materialised.
 *   a, b      device pointers to n contiguous in_dtype elements each, aligned
 *             to the element size; they may be the same array.  When both sit
 *             at the same offset from a 16-byte boundary the pass uses 16-byte
 *             loads, otherwise element loads (slower; rk_plan_all2 reports
 *             vec = 1).
 *   workspace >= rk_workspace_size(in_dtype, acc_dtype, 1, &n, &one, 1) bytes
 *             (the one-input whole-array size for n elements), aligned to 8.
 * op, dtypes, init, mode, out and stream as for rk_reduce_all; `out` must not
 * alias a or b.  n = 0 gives s.  Returns an rk_status.
 */
int rk_reduce_all2(int op, int map2, int in_dtype, int acc_dtype, int out_dtype,
                   const void *a, const void *b, int64_t n, const void *init, int mode,
                   void *out, void *workspace, void *stream);

/*
 * Mapped reduction along the dims in `reduce_mask` of a strided column-major
 * view with 1 <= ndim <= 4 dims (PR #176, section "This PR"; a single output
 * with a contiguous source takes the whole-array path, PR #139 "What
 * changes").  `ptr` is the device address of element (0,...,0), aligned to
 * its element size; `out` holds prod(kept extents) out-typed elements,
 * contiguous, column-major over the kept dims (device pointer; a host pointer
 * to one element in RK_MODE_HOST, which requires a single output).  `out`
 * must not alias the input.  Other arguments as for rk_reduce_all.
 */
int rk_reduce_dims(int op, int map, int in_dtype, int acc_dtype, int out_dtype,
                   const void *ptr, int ndim, const int64_t *shape, const int64_t *strides,
                   uint32_t reduce_mask, const void *init, int mode, void *out,
                   void *workspace, void *stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation):
 * rk_reduce_dims without the workspace argument.  Same arguments, results
 * and errors as rk_reduce_dims, and the same kernels, but the partials go to
 * a scratch array of the library's own (static device memory of 2 MiB per
 * GPU, held until the process ends) instead of a workspace; the call
 * allocates nothing (HOST mode copies its result back from that scratch
 * rather than using the pinned host buffer).  Every call on one GPU shares
 * that GPU's scratch: calls on one stream are ordered and safe, but calls
 * that may overlap on one GPU (different streams, or host threads without
 * ordering) race on it and must be ordered by the caller.  The scratch keeps
 * the last call's contents; no call reads what it did not write.  Returns
 * RK_ERR_TOO_LARGE, before any launch, when the call's plan needs more
 * workspace than the scratch holds (rk_workspace_size above 2 MiB; no plan
 * on a 256-CU GPU does).
 */
int rk_reduce_dims_no_workspace(int op, int map, int in_dtype, int acc_dtype, int out_dtype,
                                const void *ptr, int ndim, const int64_t *shape,
                                const int64_t *strides, uint32_t reduce_mask, const void *init,
                                int mode, void *out, void *stream);

/* ------------------------------------------------------------------------
 * Scans (prefix folds).  PR #202 (tile scans), opening paragraph:
 * accumulate! over a whole array or along one dim.  Every line -- the
 * elements whose indices differ only along the scan dim -- is scanned on its
 * own: with x_0, x_1, ... its elements in order and s = *init (the op's
 * identity when init is NULL), output k of the line is
 *   inclusive = 1:  s (+) x_0 (+) ... (+) x_k
 *   inclusive = 0:  s (+) x_0 (+) ... (+) x_(k-1)   (output 0 is s)
 * with elements widened to the accumulator type, running values kept in it,
 * and each output converted once to out_dtype (nearest even / wrap).  The
 * association order is the library's own, so floating-point outputs may
 * differ from a sequential loop by rounding.  The dtype table, ops and
 * identities are those of the reductions; there is no map.
 * ---------------------------------------------------------------------- */

/*
 * Bytes of device workspace rk_scan_dims (or rk_scan: ndim = 1, strides[0] =
 * 1, dim = 0) needs for this layout on the current device: the tile state of
 * a look-back scan (a 256-byte header; per tile a flag and two accumulators,
 * or two per line of a tile for a strided scan dim; neighbouring tiles'
 * state in different 128-byte lines), rounded up to 256 bytes; 0 when the
 * layout takes a kernel without tiles.  Contents need not be
 * initialised; the call clears what it uses.  After a look-back scan the
 * first two 32-bit words hold the number of tiles and a timeout word, which
 * is nonzero only if a bounded wait between tiles ever gave up (then the
 * outputs are not valid).  Returns 0 for invalid arguments as well.
 */
size_t rk_scan_workspace_size(int in_dtype, int acc_dtype, int ndim, const int64_t *shape,
                              const int64_t *strides, int dim);

/*
 * Scan along dim `dim` (0-based: Julia's dims=k is dim = k-1) of a strided
 * column-major view with 1 <= ndim <= 4 dims.  `ptr` is the device address
 * of element (0,...,0), aligned to its element size; `out` is a device
 * pointer to prod(shape) out-typed elements, the view's shape stored
 * contiguously in column-major order.  `out` may be `ptr` itself when the
 * view is contiguous and the two dtypes have the same size (an in-place
 * scan); any other overlap is rejected.  init: host pointer to one
 * accumulator-typed value, or NULL.  inclusive: 1 or 0.  workspace: device
 * pointer to >= rk_scan_workspace_size bytes, aligned to 8 (NULL allowed
 * when that size is 0); a workspace must not be shared by calls that may run
 * at the same time.  stream: hipStream_t or NULL; asynchronous.  A line
 * contiguous along the scan dim and at least one tile long (or contiguous on
 * one side only, input or output, the other side's elements then moved one
 * by one; or a strided scan dim over runs of contiguous lines; or a view
 * whose input and output are contiguous along different axes) is scanned in
 * one pass with decoupled look-back between tiles.  The tiles' counter and flags (along contiguous
 * lines: all of the per-tile state) live in the library's per-stream slot
 * when they fit one (4096 tiles along contiguous lines, 8192 for a strided
 * scan dim; the last block of the call zeroes them again), otherwise in the
 * workspace, cleared by a small launch first.  Returns an rk_status.
 */
int rk_scan_dims(int op, int in_dtype, int acc_dtype, int out_dtype, const void *ptr, int ndim,
                 const int64_t *shape, const int64_t *strides, int dim, const void *init,
                 int inclusive, void *out, void *workspace, void *stream);

/* Scan of n contiguous elements: rk_scan_dims with ndim = 1, shape = {n},
 * strides = {1}, dim = 0. */
int rk_scan(int op, int in_dtype, int acc_dtype, int out_dtype, const void *ptr, int64_t n,
            const void *init, int inclusive, void *out, void *workspace, void *stream);

/* ------------------------------------------------------------------------
 * Serving operators.  The reductions and scans around a language model's step:
 * logits to probabilities, drafted tokens verified, and the lengths that
 * result turned into block tables and slots, with no host in between.  Lines
 * are contiguous, line l at base + l * stride (elements; a line may start at
 * any element).  They are asynchronous, enqueue kernels only (so they may be
 * captured into a HIP graph; captured calls use no per-stream slot, and a
 * graph may be replayed on any stream, replays that share buffers ordered by
 * the caller), and take the size of their workspace, which is checked.
 * Device data that a host cannot check (offsets, token and block ids) is
 * clamped or ignored where it is out of range, as said with each call; nothing
 * outside the given buffers is read or written.
 * ---------------------------------------------------------------------- */

/* Bytes of device workspace rk_softmax needs on the current device (0 when
 * the call takes one launch, and for invalid arguments). */
size_t rk_softmax_workspace_size(int in_dtype, int out_dtype, int64_t n, int64_t lines);

/*
 * Softmax of `lines` lines of n entries:
 *   out_i = exp((x_i - m) / t) / sum_j exp((x_j - m) / t),   m = max_j x_j
 * with the line's temperature t = temperature[line] (device array; NULL: 1).
 * Statistics are float32 and the result is rounded once to out_dtype; both
 * dtypes are f32, bf16 or f16.  An entry of -inf is masked: 0 at every
 * temperature; a line of nothing else gives zeros.  t <= 0 puts 1 on the
 * first largest entry, 0 elsewhere.  A NaN in the line, a NaN temperature
 * (masked entries or not), or +inf with t > 0, makes the whole line NaN.
 * Exponentials below 2^-126 count as 0, temperatures between 0 and 4.24e-39
 * as that (1 / t is a float32).
 *   x_stride    elements between lines (>= 0; 0 reads one line for all)
 *   out         device pointer; may be x itself with the same stride and
 *               element size, or other columns of the same rows; any other
 *               overlap is rejected.  Entries between lines are left alone.
 *   workspace   device pointer to workspace_bytes >= rk_softmax_workspace_size
 *               bytes, aligned to 8 (may be NULL only if that size is 0).
 * Returns an rk_status.
 */
int rk_softmax(int in_dtype, int out_dtype, const void *x, int64_t n, int64_t lines, int64_t x_stride,
               const float *temperature, void *out, int64_t out_stride, void *workspace, size_t workspace_bytes,
               void *stream);

/* Bytes of device workspace rk_draft_verify needs (0 for invalid arguments
 * and for no requests). */
size_t rk_draft_verify_workspace_size(int prob_dtype, int64_t vocab, int64_t n_req);

/*
 * Verification of drafted tokens.  Request b has drafts i in [starts[b],
 * starts[b + 1]) (starts: n_req + 1 device int32; NULL: max_draft for every
 * request, n_draft = n_req * max_draft), draft i the token drafted[i] with
 * the draft's probabilities in line i of q, and the target's probabilities for
 * it in line i + b of p; line starts[b + 1] + b of p is the target's for the
 * token after the last draft.  In order, token x is kept while
 *   u[i] * q_i(x) < p_i(x)          (evaluated exactly)
 * At the first that is not, the next token is drawn from max(p_i - q_i, 0)
 * (from p_i where that leaves nothing), after the last kept one from p: the
 * first index whose running sum, in float64, passes r[b] times the whole sum
 * (the last index of positive weight where rounding lets none pass).
 *   q           NULL: the drafts have no probabilities (q_i is 1 at the token)
 *   u, r        device float32, n_draft and n_req uniform numbers of [0, 1)
 *   tokens      n_req lines of max_draft + 1: the kept tokens, the drawn one
 *               (-1 where the target's line weighs nothing), -1 behind it
 *   accepted    n_req int32: how many drafts each request kept
 * prob_dtype: f32, bf16 or f16, of p and q; they need not sum to 1.  A weight,
 * p_i or p_i - q_i, that is not a positive finite number counts as 0, also
 * p_i(x) in the comparison above.  token_dtype: i32 or i64, of drafted and
 * tokens.  A drafted token outside [0, vocab) is turned down.  starts is
 * clamped into [0, n_draft], and drafts beyond max_draft are ignored.  No
 * output may overlap an input.  vocab >= 1.  workspace: workspace_bytes >=
 * rk_draft_verify_workspace_size bytes, aligned to 8; calls that may overlap
 * need one each.  Returns an rk_status.
 */
int rk_draft_verify(int prob_dtype, int token_dtype, const void *p, int64_t p_stride, const void *q, int64_t q_stride,
                    int64_t vocab, int64_t n_req, int64_t n_draft, int max_draft, const int32_t *starts,
                    const void *drafted, const float *u, const float *r, void *tokens, int32_t *accepted,
                    void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device workspace rk_block_tables needs (0 for invalid arguments). */
size_t rk_block_tables_workspace_size(int64_t n_req);

/*
 * Brings block tables to the requests' lengths.  A request of len tokens needs
 * ceil(len / block_size) blocks (at most max_blocks); table line b names the
 * held[b] it has.  Free blocks wait in a ring of ring_size places, at places
 * head .. tail - 1 (modulo ring_size).  Blocks a request has too many go, in
 * order of request and position, to the ring's end; those it lacks are taken
 * in the same order from the ring's front, blocks given back in this call
 * last.  Where the free blocks run out, later ones are missing: held_out says
 * what every request has, and a later call goes on from there.
 *   lens        n_req int32 (negative: 0; 0 gives all blocks back)
 *   held        n_req int32 (clamped into [0, max_blocks]); held_out may be held
 *   table       n_req lines of max_blocks int32, in place; entries that are
 *               not newly taken are left as they were
 *   ring        ring_size int32, in place
 *   state       2 int64: head, tail (0 <= tail - head <= ring_size).
 *   state_out   4 int64: head and tail afterwards, blocks missing, and blocks
 *               given back that found no place in the ring; may be state
 * Everything else that is written may not overlap anything.  workspace:
 * workspace_bytes >= rk_block_tables_workspace_size bytes, aligned to 8;
 * calls that may overlap need one each.  Returns an rk_status.
 */
int rk_block_tables(const int32_t *lens, int64_t n_req, int block_size, const int32_t *held, int32_t *held_out,
                    int32_t *table, int64_t table_stride, int max_blocks, int32_t *ring, int64_t ring_size,
                    const int64_t *state, int64_t *state_out, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Slots of the new tokens of a batch.  Request b has lens[b] tokens, the last
 * fresh[b] of them new (clamped into [0, max(lens[b], 0)]); the batch is the
 * requests' new tokens one after the other.  For token t of it, number i of
 * request b:
 *   requests[t]  = b
 *   positions[t] = lens[b] - fresh[b] + i
 *   slots[t]     = table[b][positions[t] / block_size] * block_size
 *                  + positions[t] % block_size
 * and starts[b] is the batch's tokens before request b (starts[n_req]: all;
 * sums past 2^31 - 1 stay there).  A slot is -1 where the block lies behind
 * held[b] or max_blocks, or its id outside [0, n_blocks).  Entries behind the
 * batch, up to `capacity`, hold slot -1, position 0, request -1; tokens beyond
 * capacity are left out.
 *   slots        capacity elements of slot_dtype, i32 (n_blocks * block_size
 *                <= 2^31) or i64
 *   positions, requests  capacity int32 each, or NULL
 *   starts       n_req + 1 int32
 * No output may overlap an input or another.  Returns an rk_status.
 */
int rk_slot_map(const int32_t *lens, const int32_t *fresh, int64_t n_req, int block_size, const int32_t *table,
                int64_t table_stride, int max_blocks, const int32_t *held, int64_t n_blocks, int slot_dtype,
                int64_t capacity, void *slots, int32_t *positions, int32_t *requests, int32_t *starts, void *stream);

/* Bytes of device workspace rk_beam_select needs on the current device (0 for
 * invalid arguments and for no requests). */
size_t rk_beam_select_workspace_size(int dtype, int64_t vocab, int64_t n_req, int beams, int count);

/*
 * Beam search's selection.  Request b has `beams` lines of logits, b * beams and
 * on, and a score for each.  Token v of line l is a candidate with
 *   s = scores[l] + x_v - log sum_w exp(x_w)        (over the line's vocabulary)
 * and the `count` candidates with the largest s are kept, largest first; of equal
 * ones (s in float64) the one of the lower line, then of the larger logit, then
 * the lower token comes first.  Logits of -inf are masked, and a line of nothing
 * else, or of score -inf, has no candidate.
 *   logits      n_req * beams lines of vocab entries, f32, bf16 or f16
 *   scores      a float32 for every line
 *   ended       a byte for every line, or NULL: where it is not 0 the line is not
 *               read; its one candidate is end_token (0 <= end_token < vocab) at
 *               the line's score as it is
 *   best        n_req * count float32: the kept candidates' s, rounded once (to
 *               -inf below float32's range)
 *   tokens      n_req * count of token_dtype, i32 or i64
 *   parents     n_req * count int32: their lines (rows of rk_fork_blocks' table,
 *               sources of rk_linear_recurrence)
 * Behind a request's last candidate: -inf, -1, -1.  A request with a score of NaN
 * or +inf, or with a NaN or +inf among the logits of a line that is read, gets
 * NaN, -1, -1 throughout.  The sum's exponentials are float32 and its terms of
 * 2^-126 of the largest and less count as 0.  count <= 64, beams <= 4096.  No
 * output may overlap an input or another.  workspace: workspace_bytes >=
 * rk_beam_select_workspace_size bytes, aligned to 8; calls that may overlap need
 * one each.  Returns an rk_status.
 */
int rk_beam_select(int dtype, int token_dtype, const void *logits, int64_t stride, int64_t vocab, int64_t n_req, int beams,
                   const float *scores, const uint8_t *ended, int64_t end_token, int count, float *best, void *tokens,
                   int32_t *parents, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device workspace rk_fork_blocks needs (0 for invalid arguments). */
size_t rk_fork_blocks_workspace_size(int64_t n_rows, int64_t n_out, int max_blocks, int64_t n_blocks);

/*
 * Makes the rows of a block table those of other rows: row r of the new table is
 * what row parents[r] was, and rows that no row goes on from are given up.  Rows
 * may share blocks.  A row that goes on in several keeps its blocks in the first
 * of them, r the lowest.  The others share with it the lens / block_size blocks
 * that are full; of the next one, partly filled, each takes a block of its own
 * from the front of the ring of free blocks (as in rk_block_tables), in the order
 * of r, and pairs[r] says what is to be copied (rk_copy_blocks); blocks behind it
 * they do not have.  Blocks that no new row names go, in order of the old rows
 * that first name them and of position, to the ring's end; fresh blocks come from
 * these last.  Where free blocks run out a row is left without its partly filled
 * block, and is counted as missing: its tokens there are lost.
 *   parents     n_out int32; -1, or anything outside [0, n_rows): an empty row
 *   lens        n_rows int32: tokens of the old rows (negative: 0)
 *   held        n_rows int32: blocks of the old rows (clamped into [0, max_blocks])
 *   table       n_rows lines of max_blocks int32.  Ids outside [0, n_blocks) are
 *               passed on, but never given back.  No free block may be among them.
 *   ring, state, state_out  as in rk_block_tables: ring in place; state_out (4
 *               int64: head, tail, rows left without a block, blocks that found no
 *               place in the ring) may be state
 *   table_out   n_out lines of max_blocks int32; entries behind held_out are left
 *               as they were
 *   held_out, lens_out  n_out int32: blocks and tokens of the new rows
 *   pairs       n_out pairs of int32: (source, fresh block), or (-1, -1)
 * n_rows and n_out times max_blocks < 2^31 - 1.  What is written may not overlap
 * anything else.  workspace: workspace_bytes >= rk_fork_blocks_workspace_size
 * bytes, aligned to 8; calls that may overlap need one each.  Returns an
 * rk_status.
 */
int rk_fork_blocks(const int32_t *parents, int64_t n_out, const int32_t *lens, int64_t n_rows, int block_size,
                   const int32_t *held, const int32_t *table, int64_t table_stride, int max_blocks, int32_t *ring,
                   int64_t ring_size, const int64_t *state, int64_t n_blocks, int32_t *table_out, int64_t table_out_stride,
                   int32_t *held_out, int32_t *lens_out, int32_t *pairs, int64_t *state_out, void *workspace,
                   size_t workspace_bytes, void *stream);

/* Bytes of device workspace rk_compact_blocks needs (0 for invalid arguments). */
size_t rk_compact_blocks_workspace_size(int64_t n_blocks);

/*
 * Brings the blocks in use to the lowest ids.  With u different blocks of
 * [0, n_blocks) named by the table's lines (the held[b] first entries of line b),
 * the k-th lowest id of them that is >= u is moved to the k-th lowest id below u
 * that is not named.  Blocks that no line names are free afterwards, whatever
 * held them before: the ring is made anew, u .. n_blocks - 1 at its places 0 and
 * on (places behind them are left as they were).
 *   table       n_rows lines of max_blocks int32; ids outside [0, n_blocks) are
 *               passed on
 *   table_out   the same lines with the new ids; entries behind held are left as
 *               they were.  May be table itself.
 *   ring        ring_size >= n_blocks int32
 *   pairs       max_pairs >= n_blocks / 2 pairs of int32: (id before, id
 *               afterwards) of each move, in order, then (-1, -1): what
 *               rk_copy_blocks is to copy
 *   state_out   4 int64: head (0), tail (n_blocks - u), moves, 0
 * Everything else that is written may not overlap anything.  workspace:
 * workspace_bytes >= rk_compact_blocks_workspace_size bytes, aligned to 16; calls
 * that may overlap need one each.  Returns an rk_status.
 */
int rk_compact_blocks(const int32_t *held, int64_t n_rows, const int32_t *table, int64_t table_stride, int max_blocks,
                      int64_t n_blocks, int32_t *table_out, int64_t table_out_stride, int32_t *ring, int64_t ring_size,
                      int32_t *pairs, int64_t max_pairs, int64_t *state_out, void *workspace, size_t workspace_bytes,
                      void *stream);

/* A cache: n_blocks blocks of block_bytes bytes, block_stride bytes apart. */
typedef struct {
    void *data;
    int64_t block_stride, block_bytes, n_blocks;
} rk_block_cache;

/*
 * Copies blocks inside caches: for every pair (source, destination) of n_pairs
 * (device int32), block `destination` of each cache becomes what block `source`
 * is.  A pair with an id outside [0, n_blocks) of a cache is left out there.  No
 * block may be the destination of one pair and named by another; a block may be
 * the source of several.  (rk_fork_blocks and rk_compact_blocks leave such pairs.)
 * Blocks may start and end at any byte.  caches: host memory, read during the
 * call; they must not overlap each other or pairs (what they hold between blocks
 * is left alone, and may be another cache's).  Returns an rk_status.
 */
int rk_copy_blocks(const rk_block_cache *caches, int n_caches, const int32_t *pairs, int64_t n_pairs, void *stream);

/* ------------------------------------------------------------------------
 * Gated linear recurrence: the scan of a recurrent layer, and its gradient.
 * Tokens of `channels` contiguous elements; asynchronous, kernels only, so
 * the calls may be captured (they use no per-stream slot).
 * ---------------------------------------------------------------------- */

/* What is taken for the gate a of a token and channel: the value itself, its
 * exponential, or its logistic function 1 / (1 + exp(-gate)). */
typedef enum { RK_GATE_VALUE = 0, RK_GATE_LOG = 1, RK_GATE_SIGMOID = 2 } rk_gate;

/* Tokens of one or several sequences: token t of sequence b is the channels
 * from data + b * seq_stride + t * token_stride on (elements).  The strides of
 * what is only read may be 0.  `data` is written only where a call says so. */
typedef struct {
    void *data;
    int64_t seq_stride, token_stride;
} rk_rows;

/* Bytes of device workspace rk_linear_recurrence and its backward pass need for
 * tensors of any strides (0 where a call takes one launch, and for invalid
 * arguments).  packed: whether `starts` is given. */
size_t rk_linear_recurrence_workspace_size(int x_dtype, int gate_dtype, int64_t n_seq, int64_t tokens, int64_t channels,
                                           int packed);

/*
 * For every sequence and channel, from the sequence's own state h_0,
 *   h_t = a_t h_(t-1) + w_t x_t        w = 1, or 1 - a with `blend`
 * Token t's h goes to `out`, the last one's, in float32, to state_out.
 *   x_dtype     f32, bf16 or f16, of x and out; gate_dtype: the same or f32
 *   kind        rk_gate: a is the gate, exp(gate) or the logistic function of it
 *   state       n_states lines of channels float32, or NULL (zeros)
 *   sources     n_seq int32: the line of state each sequence starts from (zeros
 *               where it names none), or NULL: line b for sequence b, n_seq lines
 *   starts      n_seq + 1 device int32: the sequences are the tokens [starts[b],
 *               starts[b + 1]) of `tokens` in all (seq_stride is not used).  They
 *               must not fall, and are clamped into [0, tokens].  Tokens of no
 *               sequence are left as they were in out.  NULL: n_seq sequences of
 *               `tokens` tokens each.
 *   out         may be x or gate itself, or other columns of the same rows; no
 *               other overlap
 *   state_out   n_seq lines of channels float32: the last state, or the first one
 *               of a sequence without tokens.  May be state, without sources
 *               (first states that are still to be read are then kept in the
 *               workspace).
 * States, gates and their products are float32 and h is rounded once.  Nothing
 * passes from one sequence to another.  (Runs of up to 2048 tokens are folded
 * into one factor: a product of that many gates that leaves float32's range
 * makes a state infinite or NaN that need not be, unless the state before the
 * run is 0.)  Equal inputs give equal bits.  workspace: workspace_bytes >=
 * rk_linear_recurrence_workspace_size bytes, aligned to 8 (may be NULL only if
 * that size is 0); calls that may overlap need one each.  Returns an rk_status.
 */
int rk_linear_recurrence(int x_dtype, int gate_dtype, int kind, int blend, const rk_rows *gate, const rk_rows *x,
                         const float *state, int64_t n_states, const int32_t *sources, const int32_t *starts,
                         int64_t n_seq, int64_t tokens, int64_t channels, const rk_rows *out, float *state_out,
                         void *workspace, size_t workspace_bytes, void *stream);

/*
 * Gradients of rk_linear_recurrence (without sources).  With d_t the gradient of
 * token t's output and, after the last token, u = dstate_out (NULL: zeros),
 *   g_t = d_t + u_(t+1)      u_t = a_t g_t      dx_t = w_t g_t
 *   da_t = g_t h_(t-1), or g_t (h_(t-1) - x_t) with blend
 *   dgate_t = da_t, da_t a_t or da_t a_t (1 - a_t) by kind
 * and dstate = u of the first token (of a sequence without tokens: dstate_out).
 *   x           read with blend only, else it may be NULL
 *   out         what the forward pass returned (h_(t-1) is taken from it, the
 *               first token's from state)
 *   dgate, dx   of gate_dtype and x_dtype; either may be an input but `out` itself,
 *               or other columns of the same rows.  Tokens of no sequence are
 *               left as they were.
 *   dstate      n_seq lines of channels float32, or NULL; apart from all else
 * The rest is as with rk_linear_recurrence.  Returns an rk_status.
 */
int rk_linear_recurrence_backward(int x_dtype, int gate_dtype, int kind, int blend, const rk_rows *gate, const rk_rows *x,
                                  const rk_rows *out, const rk_rows *dout, const float *state, const float *dstate_out,
                                  const int32_t *starts, int64_t n_seq, int64_t tokens, int64_t channels,
                                  const rk_rows *dgate, const rk_rows *dx, float *dstate, void *workspace,
                                  size_t workspace_bytes, void *stream);

/* Static, human-readable name of an rk_status value. */
const char *rk_status_string(int status);

/* ------------------------------------------------------------------------
 * Diagnostics and hooks for tests and benchmarks: which kernel a call takes
 * and its plan (these launch nothing), timing of a call's first pass, the
 * device's read ceiling, and the finishing tags of a stream's slot.
 * ---------------------------------------------------------------------- */

/* Kernels a call can take.  The dims selector (PR #176, "This PR" item 1)
 * chooses among THREAD, TILED and COLUMNS for a strided reduced dim with
 * contiguous runs of outputs (in the output's order, or else in storage
 * order, each output then stored at its own place); ROW serves a contiguous
 * reduced dim, GENERIC any other layout, and a single output takes the
 * whole-array path. */
typedef enum {
    RK_KERNEL_NONE = 0,         /* nothing to compute (no outputs) */
    RK_KERNEL_ALL = 1,          /* whole-array first pass (+ one-block second pass) */
    RK_KERNEL_ALL_STRIDED = 2,  /* whole-array passes over a non-contiguous single-output view */
    RK_KERNEL_THREAD = 3,       /* one thread per output (or per 16-byte group of outputs) */
    RK_KERNEL_TILED = 4,        /* 2-d block over a narrow tile of outputs, one pass */
    RK_KERNEL_COLUMNS = 5,      /* 2-d block over a wide tile of outputs, split along the reduced dim */
    RK_KERNEL_ROW = 6,          /* one wave per output over a contiguous reduced dim */
    RK_KERNEL_GENERIC = 7,      /* one block per output, any layout */
    RK_KERNEL_ALL2 = 8,         /* whole-array passes over a two-input source (rk_reduce_all2) */
    RK_KERNEL_SCAN_TILE = 9,    /* scan: tiles of lines contiguous along the scan dim (in input and output,
                                   or on one side for a few lines), decoupled look-back (+ a clearing launch) */
    RK_KERNEL_SCAN_ROWWAVE = 10,/* scan: one wave per contiguous line shorter than a tile */
    RK_KERNEL_SCAN_LINES = 11,  /* scan: one thread per line along a strided scan dim */
    RK_KERNEL_SCAN_COLUMNS = 12,/* scan: tiles of contiguous lines x scan positions, look-back along
                                   a strided scan dim (+ a clearing launch) */
    RK_KERNEL_SCAN_TRANSPOSE = 13, /* scan: input and output contiguous along different axes (a
                                   transposed or permuted view): tiles of lines x scan positions
                                   staged through LDS, look-back along the scan dim (+ a clearing
                                   launch) */
    RK_KERNEL_SOFTMAX_LINE = 14, /* softmax: a line in the registers of a quarter wave, a wave or a block, one launch */
    RK_KERNEL_SOFTMAX_SPLIT = 15, /* softmax: tiles of a line, statistics first, then the line (two launches,
                                    three beyond 2^20 entries) */
    RK_KERNEL_DRAFT_VERIFY = 16   /* draft verification: a wave per tile of a request's line */
} rk_kernel;

typedef struct {
    int kernel;               /* rk_kernel */
    int launches;             /* kernel launches the call makes: 0, 1 or 2 (1 when a split
                                 reduction finishes inside its first launch) */
    int64_t grid;             /* blocks of the first launch */
    int block;                /* threads per block of the first launch */
    int split;                /* blocks sharing one output's reduction (1 = no second pass) */
    int vec;                  /* elements per load in the first launch */
    int tile_outputs;         /* outputs per block tile (tile kernels) */
    int64_t n_out;            /* number of outputs */
    int64_t reduce_len;       /* elements folded into each output */
    size_t workspace_bytes;   /* what rk_workspace_size returns for this layout */
} rk_plan_info;

/* Plan of rk_reduce_all / rk_reduce_all2 / rk_reduce_dims for `num_cus` compute units (0 =
 * the current device), without launching.  `ptr` only matters through its
 * alignment.  Returns an rk_status. */
int rk_plan_all(int in_dtype, int acc_dtype, const void *ptr, int64_t n, int num_cus,
                rk_plan_info *info);
int rk_plan_all2(int in_dtype, int acc_dtype, const void *a, const void *b, int64_t n, int num_cus,
                 rk_plan_info *info);
int rk_plan_dims(int in_dtype, int acc_dtype, const void *ptr, int ndim, const int64_t *shape,
                 const int64_t *strides, uint32_t reduce_mask, int num_cus,
                 rk_plan_info *info);
/* Plan of rk_scan_dims: kernel is one of the RK_KERNEL_SCAN_* values (NONE
 * for an empty view), split is the tiles along each line, tile_outputs the
 * elements per tile, n_out the number of outputs and reduce_len the line
 * length. */
int rk_plan_scan(int in_dtype, int acc_dtype, int out_dtype, const void *ptr, const void *out, int ndim,
                 const int64_t *shape, const int64_t *strides, int dim, int num_cus,
                 rk_plan_info *info);

/* Plans of rk_softmax (split: tiles per line) and rk_draft_verify (split:
 * blocks per request; tile_outputs: vocabulary entries a wave sums; launches as
 * outside a capture). */
int rk_plan_softmax(int in_dtype, int out_dtype, int64_t n, int64_t lines, rk_plan_info *info);
int rk_plan_draft_verify(int prob_dtype, int64_t vocab, int64_t n_req, int num_cus, rk_plan_info *info);

/* Whether a split reduction may finish inside its first launch (block 0
 * collecting tagged partials, or the last block to arrive; the default)
 * instead of a second launch.  Both give the same
 * results; tests switch it off to cover the second-launch path.  Process-
 * wide.  Returns the previous setting (1 or 0). */
int rk_debug_set_fused_finish(int enable);

/* Benchmark hook: while both are non-NULL, every later rk_reduce_*, rk_scan*,
 * serving and rk_debug_stream_read call made by this host thread records hipEvent_t
 * `begin` when its first kernel starts and `end` when it ends, on the call's
 * stream (the events ride on that kernel's dispatch packet).  Pass NULLs to
 * stop.  Returns an rk_status. */
int rk_debug_set_launch_events(void *begin, void *end);

/* Test hook: make the last whole-array finishing tag of `stream`'s slot `e`
 * (every kernel translation unit), so a test can run calls across the wrap
 * of the tags: e = 2^32 - 2 makes the next call the one that wraps.  Enqueued
 * on `stream`.  Returns an rk_status: RK_ERR_INVALID_ARGUMENT for e above
 * 2^32 - 2, RK_ERR_UNSUPPORTED when the stream gets no slot. */
int rk_debug_set_finish_tag(void *stream, uint32_t e);

/* Benchmark hook: the device's read-bandwidth ceiling.  Enqueues on `stream`
 * one kernel that loads each of the nbytes / 16 vectors at `ptr` once
 * (16-byte non-temporal loads, `grid` blocks of 256 threads, 0 = 2048) and
 * does one integer operation per word; it computes nothing a caller can use.
 * `ptr`: device memory, 16-byte aligned; nbytes: a multiple of 16.  `sink`:
 * one 4-byte device word that the kernel may overwrite with an unspecified
 * value.  Asynchronous.  Honours rk_debug_set_launch_events like the
 * reductions, so both are timed on their own dispatch packets.  Returns an
 * rk_status. */
int rk_debug_stream_read(const void *ptr, int64_t nbytes, int grid, void *sink, void *stream);

/* The current device's compute units, memory clock (kHz) and memory bus
 * width (bits), as the HIP runtime reports them.  Returns an rk_status
 * (RK_ERR_HIP without a usable device). */
int rk_debug_device_info(int64_t *num_cus, int64_t *mem_clock_khz, int64_t *mem_bus_bits);

/* How many waits inside launches gave up (see "Waits inside a launch" above)
 * in calls on `stream` since the last query, plus those of calls on streams
 * that have no library slot; the counts are cleared.  It waits for `stream`
 * to drain (hipStreamSynchronize), then reads the library's counts with
 * synchronous copies, so it must not be called during graph capture.  After
 * a whole-array wait gave up it also clears the stream's tagged partials,
 * so a block of that call that had not even started when the wait gave up
 * cannot be taken for one of a later call.  `*count` receives the number
 * (0 in every normal run).  Returns an rk_status: RK_ERR_INVALID_ARGUMENT
 * for a NULL count, RK_ERR_HIP when the stream or a copy fails. */
int rk_stream_timeouts(void *stream, uint64_t *count);

/* Test hook: with polls >= 0, every later whole-array collection (split
 * whole-array calls that finish in one launch) and scan look-back waits for
 * a tag or flag that never comes and gives up after `polls` polls, as a real
 * wait would after its bound; polls < 0 restores normal waits.  Every kernel
 * still ends; the calls store no result or wrong scan outputs, and count
 * their waits for rk_stream_timeouts.  (Linear recurrences, whose blocks do the
 * work of one they wait for in vain, do so once in every look-back, and their
 * results stay.)  Process-wide.  Returns an rk_status. */
int rk_debug_force_wait_timeout(int64_t polls);

/* Test hook: the next `count` reduction, scan or serving calls that pass validation
 * return RK_ERR_HIP where they would launch their first kernel, and launch
 * nothing (out and workspace untouched), as after a launch the runtime
 * rejected.  Process-wide; 0 switches it off.  Returns an rk_status. */
int rk_debug_fail_launches(int count);

#ifdef __cplusplus
}
#endif

#endif /* RK_H */
