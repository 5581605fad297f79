/*
 * sx_scan.h: C ABI of the MI355X (gfx950) scan library, libsx_scan.so.
 *
 * The scans of the SexpGPU documentation pages:
 *
 *   element-scan  "Nonlinear element scans": a nonlinear recurrence along
 *                 one axis, one independent lane per index of the other axes,
 *                 with one of three fixed bodies (tanh-affine, norm-capped
 *                 vector state, max-plus), forward or reverse.
 *   element-scan gradient  the chain rule through those bodies, trips last
 *                 to first.
 *   matrix-scan   "Tensor operations", Operations table (matrix-scan row) and
 *                 the "matrix-scan" section: h[t] = a[t] @ h[t-1] + b[t] from
 *                 h = 0, n <= 16, computed in f32, with :axis, :reverse and
 *                 broadcast leading dims.
 *   matrix-scan gradient  the same section and "gradient": the adjoint scan
 *                 in the other direction on a's transposes, then grad_a.
 *   table-scan    "Tensor operations", the "table-scan" section: a
 *                 deterministic automaton over int32 symbols.
 *   linear-scan   the same section: matrix-scan over one-by-one matrices,
 *                 a and b broadcast to one shape (cumsum: a = 1).
 *
 * and the operators of a linear-attention layer, whose state is a matrix-scan
 * with a scalar step and a rank-one input, read out by a query:
 *
 *   decay-attention  linear attention with a decay for each head, over prompts,
 *                 with its gradient, and for single tokens.
 *   head-norm-rotate  the norm of each head of queries and keys and the
 *                 rotation by position, with its gradient.
 *
 * Conventions shared by every entry point:
 *
 *  - Pointers to tensor data are DEVICE pointers on the device that is
 *    current on the calling thread. Shapes and strides are HOST arrays of
 *    int64_t, read during the call only. Strides count elements (not bytes),
 *    may be zero (a broadcast dimension) and may be passed as NULL to mean
 *    row-major contiguous. Layouts are row-major, as PyTorch's default.
 *  - The caller owns every buffer. The library keeps no pointer after it
 *    returns and allocates no device memory. Where a workspace is needed,
 *    the caller passes one of at least the queried size. Element-scan
 *    workspaces may hold anything on entry. A matrix-scan workspace (also
 *    those of its gradient and :projective) must be zero-filled once before
 *    its first use; every call then leaves it ready for the next one, on any
 *    later shape, with nothing to clear in between (no extra kernel per
 *    call). Keep it for matrix-scan calls only: other writes to its first
 *    256 bytes invalidate it until it is zero-filled again.
 *  - Work is enqueued on `stream` (a hipStream_t; NULL is the null stream)
 *    and the call returns without waiting. Results follow stream order.
 *    Concurrent calls that share one workspace race.
 *  - Every argument is checked on the host before anything is enqueued. On
 *    an error status nothing is launched and `out` is untouched;
 *    sx_last_error() then returns a message that names the operands with
 *    their shapes and dtypes, as the pages' error notes do.
 *  - Status codes mirror the pages' error table ("Tensor operations",
 *    Errors): E-DIM-001 for a shape mismatch, E-DIM-002 for mismatched or
 *    unsupported dtypes, E-DIM-003 for a missing tensor.
 */
#ifndef SX_SCAN_H
#define SX_SCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Largest tensor rank the library accepts. */
#define SX_MAX_RANK 8
/* Largest matrix size n of matrix-scan ("n at most 16") and largest state
 * width of a vector-state element scan ("vectors of 1 to 16 values"). */
#define SX_MAX_N 16
/* `state_axis` value that selects a scalar state (no :state-axis). */
#define SX_STATE_SCALAR INT32_MIN

typedef enum sx_status {
  SX_OK = 0,
  SX_E_DIM_001 = 1,     /* shapes do not fit, axis out of range, n > 16, empty element-scan axis */
  SX_E_DIM_002 = 2,     /* dtypes differ, or a dtype the operand does not allow */
  SX_E_DIM_003 = 3,     /* a tensor was expected: a required pointer is NULL */
  SX_E_UNSUPPORTED = 4, /* well-formed but not provided: rank > 8, strided matrix dims */
  SX_E_ALIAS = 5,       /* `out` overlaps an input */
  SX_E_WORKSPACE = 6,   /* workspace NULL or smaller than the queried size */
  SX_E_DEVICE = 7       /* a HIP call failed; sx_last_error() carries hipGetErrorString */
} sx_status;

typedef enum sx_dtype { SX_F32 = 0, SX_BF16 = 1 } sx_dtype;

/* The three element-scan bodies ("Nonlinear element scans", introduction),
 * each taking (state h, sequence x, sequence s) in the page's order:
 *   SX_BODY_TANH_AFFINE  h' = tanh(x + s * h)              s = decay
 *   SX_BODY_NORM_CAP     y = s * h + x; h' = y / max(1, |y|)  s = decay, |y| over the state vector
 *   SX_BODY_MAX_PLUS     h' = max(h - s, x)                s = cost
 * NORM_CAP reduces over the state vector and so needs a vector state; the
 * other two act on each state component on its own and accept either. */
typedef enum sx_body {
  SX_BODY_TANH_AFFINE = 0,
  SX_BODY_NORM_CAP = 1,
  SX_BODY_MAX_PLUS = 2
} sx_body;

/*
 * sx_element_scan: "Nonlinear element scans", introduction and "Arguments
 * and body".
 *
 * For every lane (every index outside `axis`, and outside the state axis for
 * a vector state) the state starts at `initial` and each trip applies the
 * body: forward h[t] = f(h[t-1], x[t], s[t]) from h[-1] = initial, reverse
 * h[t] = f(h[t+1], x[t], s[t]) from h[T] = initial. out[t] holds the state
 * after trip t. Computation is f32.
 *
 *  body          one of sx_body.
 *  rank, shape   the OUTPUT shape, rank 1..SX_MAX_RANK: the sequences' shape,
 *                whose last axis, for a vector state, is the state width n.
 *  axis          the sequence axis; negative counts from the end. Its length
 *                must be at least one (E-DIM-001 otherwise).
 *  state_axis    SX_STATE_SCALAR for a scalar state; -1 or rank-1 for a state
 *                vector along the last axis (1 <= n <= 16, axis != last);
 *                anything else is E-DIM-001.
 *  reverse       0 forward, nonzero reverse.
 *  initial       f32, shape = `shape` without `axis`; `initial_strides` has
 *                rank-1 entries (or NULL for contiguous).
 *  x, s          f32 sequences. Scalar state: shape = `shape`, widths
 *                ignored. Vector state: shape = `shape` with the last axis
 *                replaced by the sequence's own width, `x_width`/`s_width`,
 *                each 1 (broadcast over the state, a per-trip gate) or n.
 *                Strides have `rank` entries; a width-1 axis's stride is
 *                ignored.
 *  out           f32, contiguous, shape `shape`. Must not overlap an input.
 *  workspace     may be NULL when sx_element_scan_workspace_bytes() is 0.
 *  stream        hipStream_t.
 *
 * A shape with zero lanes returns SX_OK without launching.
 */
sx_status sx_element_scan(sx_body body, int rank, const int64_t* shape, int axis, int state_axis,
                          int reverse, const float* initial, const int64_t* initial_strides,
                          const float* x, int64_t x_width, const int64_t* x_strides, const float* s,
                          int64_t s_width, const int64_t* s_strides, float* out, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Workspace bytes sx_element_scan needs for these arguments (0 when none);
 * returns 0 as well for arguments sx_element_scan would reject. */
size_t sx_element_scan_workspace_bytes(sx_body body, int rank, const int64_t* shape, int axis,
                                       int state_axis);

/*
 * sx_element_scan_backward: gradients of an element scan. The chain rule
 * through the bodies of "Nonlinear element scans" (introduction), with each
 * gradient in its tensor's shape ("Tensor operations", "gradient" section).
 *
 * Given the forward call's arguments, its result h and the gradient g of a
 * loss with respect to h, writes the loss's gradients with respect to
 * initial, x and the second sequence s. The trips are taken last to first in
 * scan order; with lam the adjoint of the state a trip produced (g there plus
 * what the trip after passed back) and hp the state it started from:
 *   tanh-affine  dz = lam (1 - h^2); grad_x = dz; grad_s = dz hp; to hp: s dz
 *   norm-cap     y = s hp + x; when |y| > 1, u = y / |y| and
 *                dy = (lam - u (u . lam)) / |y|, else dy = lam;
 *                grad_x = dy; grad_s = dy hp; to hp: s dy
 *   max-plus     x won (x >= hp - c; ties to x): grad_x = lam, grad_c = 0,
 *                to hp 0; else grad_x = 0, grad_c = -lam, to hp lam
 * grad_initial is what the first trip passes back. A width-one sequence under
 * a vector state gets the sum over the state of its broadcast gradient. The
 * branch decisions use f32 values computed as the forward pass does.
 *
 *  body .. s_strides  as for sx_element_scan, except that initial must be
 *                contiguous (no strides argument).
 *  h, g          the forward result and its gradient: contiguous, `shape`.
 *  grad_initial, grad_x, grad_s
 *                contiguous, the shapes of initial, x and s. Must not overlap
 *                any input or each other (SX_E_ALIAS).
 *  workspace     at least sx_element_scan_backward_workspace_bytes() bytes
 *                (nonzero for width-one sequences under a vector state with
 *                tanh-affine or max-plus, and for norm-cap with fewer than
 *                8192 state vectors and at least 32 trips, which splits the
 *                axis), 256-byte aligned; may be NULL when that is 0. The
 *                call overwrites it.
 *
 * Errors as sx_element_scan; E-DIM-003 for any NULL tensor.
 */
sx_status sx_element_scan_backward(sx_body body, int rank, const int64_t* shape, int axis, int state_axis,
                                   int reverse, const float* initial, const float* x, int64_t x_width,
                                   const int64_t* x_strides, const float* s, int64_t s_width,
                                   const int64_t* s_strides, const float* h, const float* g, float* grad_initial,
                                   float* grad_x, float* grad_s, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* Workspace bytes sx_element_scan_backward needs (0 when none or for invalid arguments). */
size_t sx_element_scan_backward_workspace_bytes(sx_body body, int rank, const int64_t* shape, int axis,
                                                int state_axis, int64_t x_width, int64_t s_width);

/*
 * sx_matrix_scan: "Tensor operations", Operations table (matrix-scan row)
 * and the "matrix-scan" section.
 *
 * a is [lead_a..., n, n] and b [lead_b..., n, m], n <= 16, one float dtype.
 * The leading dims broadcast (NumPy: right-aligned, each equal or 1) to one
 * shape `lead`, and `axis` indexes them (-1: the last leading dim, next to
 * the matrix dims). For every other leading index the n-by-m state runs
 *   forward  h[t] = a[t] @ h[t-1] + b[t]  from h[-1] = 0  (h[0] = b[0]),
 *   reverse  h[t] = a[t] @ h[t+1] + b[t]  from h[T] = 0  (h[T-1] = b[T-1]),
 * and out[t] = h[t]. Computation is f32 for f32 and bf16 operands alike:
 * bf16 widens to f32 exactly, and with bf16 a each product a[t] @ h is
 * formed exactly (h split into three bf16 parts that sum to it) and summed in
 * f32, as with f32 operands.
 *
 *  dtype         SX_F32 or SX_BF16, shared by a and b.
 *  a_*, b_*      rank (>= 2), shape, strides (NULL = contiguous) and data.
 *                The two matrix dims must be row-major contiguous (strides
 *                [n, 1] and [m, 1] where those dims exceed 1); leading dims may
 *                have any stride, including 0. Otherwise SX_E_UNSUPPORTED.
 *  axis          the scan axis among the broadcast leading dims.
 *  reverse       0 forward, nonzero reverse.
 *  projective    nonzero: the :projective variant of the same section,
 *                meant for chains of projective maps whose plain product
 *                would leave f32's range. Each step multiplies a running
 *                product P (starting at the identity) by that step's a,
 *                P = a[t] @ P, then rescales: with m the entry of P of
 *                largest magnitude (m = 1 for a zero P), both P and the new
 *                state are divided by m, h[t] = (a[t] @ h[prev] + b[t]) / m.
 *                When b vanishes after its first step, every state then
 *                equals the plain scan's state times a positive number of
 *                its own. With n = 16, on the shapes the chunked scan
 *                takes, it runs in parallel in the workspace (passes that
 *                compute every step's factor, then the scan); on other
 *                shapes it runs serially in time.
 *  out_dtype     SX_F32 or SX_BF16. The result is rounded to bf16 to nearest
 *                even on store when SX_BF16.
 *  out           contiguous, shape lead + [n, m] (see sx_matrix_scan_out_shape).
 *  workspace     at least sx_matrix_scan_workspace_bytes() bytes, 256-byte
 *                aligned, zero-filled before its first use (see above); may
 *                be NULL when that size is 0.
 *
 * Time-parallel kernels hand each chunk's entering state on through the
 * workspace; every wait for an earlier chunk is bounded, and one that reaches
 * its bound is recorded in the workspace, not returned here (the call is
 * asynchronous): sx_matrix_scan_workspace_status reports it.
 *
 * An axis of length 0 (or m = 0) returns SX_OK with nothing to write.
 */
sx_status sx_matrix_scan(sx_dtype dtype, int a_rank, const int64_t* a_shape, const int64_t* a_strides,
                         const void* a, int b_rank, const int64_t* b_shape, const int64_t* b_strides,
                         const void* b, int axis, int reverse, int projective, sx_dtype out_dtype,
                         void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device memory sx_matrix_scan_noalloc keeps, per device, for its
 * look-back state. */
#define SX_MATRIX_SCAN_SCRATCH_BYTES (16u << 20)

/*
 * sx_matrix_scan_noalloc: sx_matrix_scan (the same arguments, the same result)
 * for callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc. It takes no
 * workspace: the look-back state lives in a fixed array of
 * SX_MATRIX_SCAN_SCRATCH_BYTES bytes in device memory, one per device the
 * library runs on, kept until the process ends. It calls no allocation
 * routine. The first call on a device sets the array up (its address, and a
 * synchronous zero-fill): make that first call outside graph capture.
 *
 * Shapes whose look-back state is larger than the array (sx_matrix_scan_workspace_bytes
 * above SX_MATRIX_SCAN_SCRATCH_BYTES: about 5000 units of 96 steps of one
 * 16-column tile, e.g. 32 x 8192 and 16 x 16384 fit) return SX_E_WORKSPACE
 * before anything is launched. Every call on a device shares that device's
 * array and leaves it ready for the next call: calls that overlap on one
 * device (concurrent streams, host threads) race. A look-back give-up is
 * recorded in the array, which sx_matrix_scan_workspace_status cannot reach.
 */
sx_status sx_matrix_scan_noalloc(sx_dtype dtype, int a_rank, const int64_t* a_shape, const int64_t* a_strides,
                                 const void* a, int b_rank, const int64_t* b_shape, const int64_t* b_strides,
                                 const void* b, int axis, int reverse, int projective, sx_dtype out_dtype, void* out,
                                 void* stream);

/* Workspace bytes sx_matrix_scan needs for these shapes (0 for invalid ones),
 * with or without :projective (the size covers both). */
size_t sx_matrix_scan_workspace_bytes(int a_rank, const int64_t* a_shape, int b_rank,
                                      const int64_t* b_shape, int axis);

/* Waits for `stream`, then reads and clears the status a matrix-scan
 * workspace carries ("Tensor operations", Errors: every failure is a reported
 * code). SX_OK when every look-back of the calls on this workspace since the
 * last check completed; SX_E_DEVICE when one gave up waiting for an earlier
 * chunk's published state (its results are then not valid), with the reason
 * in sx_last_error(). SX_E_DIM_003 for a NULL workspace, SX_E_WORKSPACE for
 * one of fewer than 256 bytes. Synchronous: not for use under graph capture. */
sx_status sx_matrix_scan_workspace_status(void* workspace, size_t workspace_bytes, void* stream);

/* Bound on the polls a matrix-scan look-back makes before it gives up and
 * records it (see sx_matrix_scan_workspace_status); 0 restores the default
 * (2^22 polls, about a tenth of a second). Process-wide, for calls launched
 * after it. A diagnostic: a small bound forces give-ups, so that the report
 * path can be tested with every kernel still running to its end. */
void sx_set_lookback_spin_limit(uint32_t limit);

/* Writes the matrix-scan result shape to out_shape (room for SX_MAX_RANK + 2
 * entries) and returns its rank, or -1 for shapes that do not fit. */
int sx_matrix_scan_out_shape(int a_rank, const int64_t* a_shape, int b_rank, const int64_t* b_shape,
                             int64_t* out_shape);

/*
 * sx_matrix_scan_backward: "Tensor operations", the "matrix-scan" section (its
 * gradient is a scan in the opposite direction over transposed a) and the
 * "gradient" section (a gradient has its operand's shape and dtype).
 *
 * Given the forward call's a and b shapes, its result h and the gradient g of
 * a loss with respect to h, writes the gradients of that loss with respect to
 * a and b. With lam[t] the adjoint of h[t] and s / p the steps after / before
 * t in the forward scan order,
 *   lam[t]    = g[t] + a[s]^T @ lam[s]   (no second term at the last step)
 *   grad_b[t] = lam[t]
 *   grad_a[t] = lam[t] @ h[p]^T        (zero at the first step, whose a
 *                                      multiplies the zero state)
 * summed over the dims along which a (or b) was broadcast. lam is computed in
 * f32 by the matrix-scan kernels in the other direction. With bf16 gradients
 * and b of the result's shape, lam is stored rounded into grad_b and grad_a
 * is formed from that rounded lam (a relative change of at most 2^-9 per
 * element of lam, inside bf16's own rounding of the result).
 *
 *  dtype         SX_F32 or SX_BF16: the dtype of a, h and g alike.
 *  a_*           a as passed to sx_matrix_scan (strides as there).
 *  b_rank/shape  b's shape (b's values are not needed).
 *  h             the forward result: contiguous, the shape
 *                sx_matrix_scan_out_shape gives, dtype `dtype`.
 *  g_strides, g  gradient of the result: that shape, dtype `dtype`; strides
 *                NULL for contiguous; its two matrix dims row-major
 *                contiguous (else SX_E_UNSUPPORTED).
 *  axis, reverse those of the forward call.
 *  grad_dtype    SX_F32 or SX_BF16 for grad_a and grad_b (rounded to nearest
 *                even on store).
 *  grad_a/grad_b contiguous, the shapes of a and b. Must not overlap any
 *                input or each other (SX_E_ALIAS).
 *  workspace     at least sx_matrix_scan_backward_workspace_bytes() bytes,
 *                256-byte aligned; may be NULL when that is 0.
 *
 * Errors as sx_matrix_scan (E-DIM-001 shapes, E-DIM-002 dtypes, E-DIM-003 a
 * NULL tensor that has elements). Empty operands return SX_OK; gradients of
 * operands that have elements are written even when the result is empty
 * (they are zero then).
 */
sx_status sx_matrix_scan_backward(sx_dtype dtype, int a_rank, const int64_t* a_shape, const int64_t* a_strides,
                                  const void* a, int b_rank, const int64_t* b_shape, const void* h,
                                  const int64_t* g_strides, const void* g, int axis, int reverse, sx_dtype grad_dtype,
                                  void* grad_a, void* grad_b, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes sx_matrix_scan_backward needs (0 for invalid shapes). */
size_t sx_matrix_scan_backward_workspace_bytes(int a_rank, const int64_t* a_shape, int b_rank,
                                               const int64_t* b_shape, int axis, sx_dtype grad_dtype);

/*
 * sx_linear_scan: "Tensor operations", the "matrix-scan" section, on the
 * prelude's linear-scan: matrix-scan over one-by-one matrices, with a and b
 * (tensors or plain numbers) broadcast together. cumsum is linear-scan with
 * a = 1 (a rank-0 a holding 1).
 *
 * For every index outside `axis` of the broadcast shape the scalar state runs
 *   forward  h[t] = a[t] * h[t-1] + b[t]  from h[-1] = 0  (h[0] = b[0]),
 *   reverse  h[t] = a[t] * h[t+1] + b[t]  from h[T] = 0  (h[T-1] = b[T-1]),
 * and out[t] = h[t]. a[0] (forward) or a[T-1] (reverse) multiplies the zero
 * state, so any finite value there gives the same result (the kernels do form
 * that product: an infinite or NaN entry there gives NaN). Computation is f32
 * for f32 and bf16 operands alike.
 *
 *  dtype         SX_F32 or SX_BF16, shared by a and b (else E-DIM-002).
 *  a_*, b_*      rank (0..SX_MAX_RANK; 0 is a number, its shape may be
 *                NULL), shape, strides (NULL = contiguous; any value,
 *                including 0 and negative) and data. The shapes broadcast
 *                NumPy-style (right-aligned, each dim equal or 1) to the
 *                result shape, of rank max(a_rank, b_rank) >= 1; otherwise
 *                E-DIM-001.
 *  axis          the scan axis of the result shape; negative counts from the
 *                end; out of range is E-DIM-001.
 *  reverse       0 forward, nonzero reverse.
 *  out_dtype     SX_F32 or SX_BF16 (rounded to nearest even on store).
 *  out           contiguous, the broadcast shape (see sx_linear_scan_out_shape);
 *                must not overlap a or b (SX_E_ALIAS).
 *
 * No workspace. A result with no elements returns SX_OK without launching.
 */
sx_status sx_linear_scan(sx_dtype dtype, int a_rank, const int64_t* a_shape, const int64_t* a_strides,
                         const void* a, int b_rank, const int64_t* b_shape, const int64_t* b_strides,
                         const void* b, int axis, int reverse, sx_dtype out_dtype, void* out, void* stream);

/* Writes the broadcast shape of a and b to out_shape (room for SX_MAX_RANK
 * entries) and returns its rank, or -1 for shapes that do not fit. */
int sx_linear_scan_out_shape(int a_rank, const int64_t* a_shape, int b_rank, const int64_t* b_shape,
                             int64_t* out_shape);

/*
 * sx_table_scan: "Tensor operations", the "table-scan" section.
 *
 * Runs a deterministic automaton along `axis` of `symbols`: each symbol
 * moves the state to table[previous, symbol], starting at `start`; out holds every
 * state, in symbols' shape. A symbol outside [0, nsym) is clamped into that
 * range, and so is any table value the run lands on outside [0, states), as the
 * pages' GPU backend does (their CPU backend refuses them instead). States
 * have no gradient.
 *
 *  states, nsym  the table's shape [states, nsym], each at least 1 (E-DIM-001).
 *  table         int32, row-major contiguous [states, nsym], device memory.
 *  rank, shape, strides, symbols
 *                int32 symbols, rank 1..SX_MAX_RANK; strides in elements (NULL
 *                for contiguous).
 *  axis          the scan axis; negative counts from the end (the pages'
 *                default is -1). Out of range: E-DIM-001.
 *  start         the first state; outside [0, states): E-DIM-001.
 *  out           int32, contiguous, symbols' shape; must not overlap symbols
 *                or the table (SX_E_ALIAS).
 *
 * No workspace. Symbols with no elements return SX_OK without launching.
 */
sx_status sx_table_scan(int states, int nsym, const int32_t* table, int rank, const int64_t* shape,
                        const int64_t* strides, const int32_t* symbols, int axis, int32_t start, int32_t* out,
                        void* stream);

/*
 * sx_decay_attention: linear attention with a decay for each head. With S a
 * dk-by-dv state for every batch row and head, from `initial` (or zero),
 *   S[t] = exp(g[t]) S[t-1] + k[t] v[t]^T,   out[t] = scale * S[t]^T q[t].
 * States, running sums and products are f32 (and finer) for f32 and bf16
 * operands alike; out is rounded to bf16 to nearest even once, on store. With
 * bf16 operands f32 values enter a product as bf16 parts: three that carry all
 * 24 bits into the state, two that carry 17 (the scores q[t] . k[s], and the
 * state where it is read for out).
 *
 *  dtype         SX_F32 or SX_BF16, shared by q, k, v and out.
 *  q, k, v       [B, T, heads, width]: shape (4 entries), strides (NULL for
 *                contiguous; any value) and data. q and k share their width dk,
 *                v has dv, each 1..256. The number of heads of each divides H;
 *                head h of the call uses head h / (H / heads) of it.
 *  g_*, log_decay  g, the natural log of the decay, f32: [H] (g_rank 1, one
 *                value a head) or [B, T, H] (g_rank 3), with strides. H is the
 *                number of heads of out. -INFINITY cuts: nothing of what came
 *                before is left. Values are taken into [-200, 200], where exp is
 *                0 and infinite in f32.
 *  initial       f32, contiguous [B, H, dk, dv], or NULL for zero.
 *  lengths       int32 [B], or NULL. Tokens of row b from lengths[b] on do not
 *                exist: they are not read, their rows of out are zero and the
 *                state ends before them. Taken into [0, T].
 *  out           contiguous [B, T, H, dv].
 *  final_state   f32, contiguous [B, H, dk, dv]: the state after the last token,
 *                or NULL.
 *  workspace     at least sx_decay_attention_workspace_bytes() bytes, 256-byte
 *                aligned; may hold anything; may be NULL when that is 0.
 *
 * An infinity or NaN of one token reaches that token's own row and later ones of
 * its head (it may past a cut as well), never earlier ones; an infinity may come
 * out as NaN. One of `initial` reaches no row from a cut on (a token whose decay is
 * zero in f32); where the decays of several tokens multiply to zero it may be left
 * behind too. out and final_state are 16-byte aligned (else SX_E_UNSUPPORTED) and
 * overlap no input and not each other (SX_E_ALIAS). Errors otherwise as the scans:
 * E-DIM-001 shapes, E-DIM-002 dtypes, E-DIM-003 a NULL tensor that has elements,
 * SX_E_UNSUPPORTED heads wider than 256.
 */
sx_status sx_decay_attention(sx_dtype dtype, const int64_t* q_shape, const int64_t* q_strides, const void* q,
                             const int64_t* k_shape, const int64_t* k_strides, const void* k, const int64_t* v_shape,
                             const int64_t* v_strides, const void* v, int g_rank, const int64_t* g_shape,
                             const int64_t* g_strides, const float* log_decay, const float* initial,
                             const int32_t* lengths, float scale, void* out, float* final_state, void* workspace,
                             size_t workspace_bytes, void* stream);

/* Workspace bytes sx_decay_attention needs for H = heads (0 when none, or for shapes it would reject). */
size_t sx_decay_attention_workspace_bytes(sx_dtype dtype, const int64_t* q_shape, const int64_t* v_shape,
                                          int64_t heads);

/*
 * sx_decay_attention_backward: gradients of sx_decay_attention. With A[t] the
 * adjoint of S[t],
 *   A[t] = exp(g[t+1]) A[t+1] + scale q[t] grad_out[t]^T   (grad_state after the last token)
 *   grad_q[t] = scale S[t] grad_out[t],  grad_k[t] = A[t] v[t],  grad_v[t] = A[t]^T k[t],
 *   grad_log_decay[t] = exp(g[t]) <A[t], S[t-1]>,  grad_initial = exp(g[0]) A[0].
 *
 *  dtype .. log_decay, initial, lengths, scale   as for the forward call.
 *  grad_out      [B, T, H, dv], dtype `dtype`, with strides (NULL for contiguous).
 *  grad_state    f32, contiguous [B, H, dk, dv]: the gradient of final_state, or
 *                NULL for none.
 *  grad_q/k/v    contiguous, the shapes of q, k and v, dtype `dtype`. A head that
 *                several heads of the call share gets the sum of their
 *                gradients, summed in f32 and rounded once.
 *  grad_log_decay  f32, contiguous, the shape of log_decay ([H]: summed over rows
 *                and tokens). Zero where the decay is.
 *  grad_initial  f32, contiguous [B, H, dk, dv]; may be NULL when initial is.
 *  workspace     at least sx_decay_attention_backward_workspace_bytes() bytes,
 *                256-byte aligned; may hold anything.
 *
 * Gradients of tokens that do not exist are zero. The outputs are 16-byte
 * aligned and overlap nothing. Results do not change from call to call (no
 * atomics). Errors as sx_decay_attention.
 */
sx_status sx_decay_attention_backward(sx_dtype dtype, const int64_t* q_shape, const int64_t* q_strides, const void* q,
                                      const int64_t* k_shape, const int64_t* k_strides, const void* k,
                                      const int64_t* v_shape, const int64_t* v_strides, const void* v, int g_rank,
                                      const int64_t* g_shape, const int64_t* g_strides, const float* log_decay,
                                      const int64_t* grad_out_strides, const void* grad_out, const float* grad_state,
                                      const float* initial, const int32_t* lengths, float scale, void* grad_q,
                                      void* grad_k, void* grad_v, float* grad_log_decay, float* grad_initial,
                                      void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes sx_decay_attention_backward needs for H = heads (0 for shapes it would reject). */
size_t sx_decay_attention_backward_workspace_bytes(sx_dtype dtype, const int64_t* q_shape, const int64_t* k_shape,
                                                   const int64_t* v_shape, int64_t heads);

/*
 * sx_decay_attention_step: one token of every request of a batch, the states
 * updated in place: S = exp(g) S + k v^T, out = scale * S^T q.
 *
 *  q, k, v       [B, heads, width] (3 entries of shape and strides), heads and
 *                widths as for sx_decay_attention.
 *  g_*, log_decay  [H] (g_rank 1) or [B, H] (g_rank 2), f32.
 *  pool, state_strides, state
 *                f32 states [pool, H, dk, dv]; each head's dk-by-dv block
 *                row-major contiguous (else SX_E_UNSUPPORTED), no two blocks
 *                overlapping; any strides and start otherwise (on 16-byte borders
 *                throughout they are read and written in larger pieces).
 *  slots         int32 [B]: the state of each row, or NULL (row b uses state b;
 *                pool >= B then). A row whose slot lies outside [0, pool) is
 *                idle: its row of out is zero and no state changes. Two rows with
 *                the same slot race: that state and those rows of out are then
 *                undefined. A token whose decay is zero in f32 starts from a state
 *                of zeros, whatever the slot holds.
 *  out           contiguous [B, H, dv], 16-byte aligned.
 *
 * No workspace. Errors as sx_decay_attention.
 */
sx_status sx_decay_attention_step(sx_dtype dtype, const int64_t* q_shape, const int64_t* q_strides, const void* q,
                                  const int64_t* k_shape, const int64_t* k_strides, const void* k,
                                  const int64_t* v_shape, const int64_t* v_strides, const void* v, int g_rank,
                                  const int64_t* g_shape, const int64_t* g_strides, const float* log_decay,
                                  int64_t pool, const int64_t* state_strides, float* state, const int32_t* slots,
                                  float scale, void* out, void* stream);

/*
 * sx_head_norm_rotate: the root-mean-square norm of each head of the queries and
 * keys, and the rotation by position, in one pass. For each row x of width d,
 *   u = x / sqrt(mean(x^2) + eps) * weight,
 *   y = u with the pairs of its first `rotated` components turned by
 *       2 pi position turns[i]:  (a, b) -> (a cos - b sin, a sin + b cos).
 * Pair i is (i, i + rotated/2), or (2i, 2i+1) when `neighbours` is nonzero; the
 * components behind `rotated` are not turned. Angles are reduced in 64 bits, so
 * far positions lose nothing; the rest is f32, rounded to `dtype` once.
 *
 *  dtype         SX_F32 or SX_BF16: q, k and the results.
 *  q, k          [B, T, heads, d] with strides (NULL for contiguous; any value),
 *                the same B, T and d (1..256); the numbers of heads are free.
 *  positions     [B, T], int64 (positions_i64 nonzero) or int32, with strides
 *                (NULL for contiguous; 0 for one row or one value for all).
 *  rotated, turns  an even number up to d, and f64 [rotated/2]: turns (of 2 pi)
 *                of pair i for each position.
 *  q_weight, k_weight  f32 [d], or NULL for ones.
 *  out_q, out_k  contiguous, the shapes of q and k, 16-byte aligned; overlap
 *                nothing.
 */
sx_status sx_head_norm_rotate(sx_dtype dtype, const int64_t* q_shape, const int64_t* q_strides, const void* q,
                              const int64_t* k_shape, const int64_t* k_strides, const void* k, int positions_i64,
                              const int64_t* position_strides, const void* positions, int64_t rotated,
                              const double* turns, const float* q_weight, const float* k_weight, float eps,
                              int neighbours, void* out_q, void* out_k, void* stream);

/*
 * sx_head_norm_rotate_backward: gradients of sx_head_norm_rotate. With r = 1 /
 * sqrt(mean(x^2) + eps) and gu the gradient of a row turned back,
 *   grad_weight = sum over rows of gu x r,
 *   grad_x = r (gu weight - x r^2 mean(gu weight x)).
 *
 *  dtype .. neighbours  as for the forward call; grad_out_q and grad_out_k have
 *                the shapes of q and k, with strides (NULL for contiguous).
 *  grad_q, grad_k  contiguous, the shapes of q and k, dtype `dtype`.
 *  grad_q_weight, grad_k_weight  f32 [d], or NULL where not wanted. Summed in a
 *                fixed order (no atomics).
 *  workspace     at least sx_head_norm_rotate_backward_workspace_bytes() bytes,
 *                256-byte aligned, when a weight's gradient is wanted; may hold
 *                anything.
 */
sx_status sx_head_norm_rotate_backward(sx_dtype dtype, const int64_t* q_shape, const int64_t* q_strides,
                                       const void* q, const int64_t* k_shape, const int64_t* k_strides, const void* k,
                                       int positions_i64, const int64_t* position_strides, const void* positions,
                                       int64_t rotated, const double* turns, const int64_t* gq_strides,
                                       const void* grad_out_q, const int64_t* gk_strides, const void* grad_out_k,
                                       const float* q_weight, const float* k_weight, float eps, int neighbours,
                                       void* grad_q, void* grad_k, float* grad_q_weight, float* grad_k_weight,
                                       void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes sx_head_norm_rotate_backward needs for the weights' gradients. */
size_t sx_head_norm_rotate_backward_workspace_bytes(const int64_t* q_shape, const int64_t* k_shape);

/* What an operator's result goes through: nothing, or u / (1 + exp(-u)). */
typedef enum sx_activation { SX_ACT_NONE = 0, SX_ACT_SILU = 1 } sx_activation;

/* Most taps of sx_causal_conv and most states a channel of sx_selective_scan. */
#define SX_MAX_TAPS 8
#define SX_MAX_STATES 32

/*
 * sx_causal_conv: a short causal convolution of each channel along the tokens,
 *   u[t] = bias + sum over j of weight[j] x[t - (taps - 1) + j],  out[t] = act(u[t]),
 * where the inputs before the first are `initial` (or zero). f32 sums, rounded to
 * `dtype` once.
 *
 *  dtype         SX_F32 or SX_BF16: x, initial, out and final_state.
 *  x             [B, T, D]: shape (3 entries), strides (NULL for contiguous; any
 *                value) and data.
 *  taps, weight  1..SX_MAX_TAPS (else SX_E_UNSUPPORTED), and f32, contiguous [D, taps].
 *  bias          f32 [D], or NULL for zero.
 *  initial       contiguous [B, taps - 1, D], oldest first, or NULL for zero.
 *  lengths       int32 [B], or NULL. Tokens of row b from lengths[b] on do not
 *                exist: they are not read, their rows of out are zero and the
 *                state ends before them. Taken into [0, T].
 *  activation    one of sx_activation.
 *  out           contiguous [B, T, D], 16-byte aligned.
 *  final_state   contiguous [B, taps - 1, D], 16-byte aligned: the last taps - 1
 *                inputs, of `initial` too where there are fewer tokens; or NULL.
 *
 * No workspace. Outputs overlap no input and not each other (SX_E_ALIAS). Errors
 * otherwise as sx_decay_attention.
 */
sx_status sx_causal_conv(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x, int64_t taps,
                         const float* weight, const float* bias, const void* initial, const int32_t* lengths,
                         sx_activation activation, void* out, void* final_state, void* stream);

/*
 * sx_causal_conv_backward: gradients of sx_causal_conv. With gu[t] = grad_out[t] act'(u[t]),
 *   grad_x[s] = sum over j of weight[j] gu[s + (taps - 1) - j], and grad_state's row where x[s] is one of the last,
 *   grad_weight[j] = sum over rows and tokens of gu[t] x[t - (taps - 1) + j],  grad_bias = sum of gu.
 *
 *  dtype .. activation   as for the forward call.
 *  grad_out      [B, T, D], dtype `dtype`, with strides (NULL for contiguous).
 *  grad_state    contiguous [B, taps - 1, D], dtype `dtype`: the gradient of
 *                final_state, or NULL for none.
 *  grad_x        contiguous [B, T, D], dtype `dtype`. Zero for tokens that do not exist.
 *  grad_weight   f32, contiguous [D, taps].
 *  grad_bias     f32 [D], or NULL where not wanted.
 *  grad_initial  contiguous [B, taps - 1, D], dtype `dtype`, or NULL where not wanted.
 *  workspace     at least sx_causal_conv_backward_workspace_bytes() bytes,
 *                256-byte aligned; may hold anything.
 *
 * Summed in a fixed order (no atomics). Errors as sx_causal_conv.
 */
sx_status sx_causal_conv_backward(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x,
                                  int64_t taps, const float* weight, const float* bias, const void* initial,
                                  const int32_t* lengths, sx_activation activation, const int64_t* grad_out_strides,
                                  const void* grad_out, const void* grad_state, void* grad_x, float* grad_weight,
                                  float* grad_bias, void* grad_initial, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* Workspace bytes sx_causal_conv_backward needs, whatever the strides (0 for shapes it would reject). */
size_t sx_causal_conv_backward_workspace_bytes(sx_dtype dtype, const int64_t* x_shape, int64_t taps);

/*
 * sx_causal_conv_step: one token of every request of a batch. The state of a
 * request is its last taps - 1 inputs; they are read and moved up by one in place.
 *
 *  x             [B, D] with strides (NULL for contiguous).
 *  pool, state_stride, state
 *                dtype `dtype`, [pool, taps - 1, D]; each state contiguous,
 *                `state_stride` elements from one to the next, none overlapping
 *                (else SX_E_UNSUPPORTED).
 *  slots         int32 [B]: the state of each row, or NULL (row b uses state b;
 *                pool >= B then). A row whose slot lies outside [0, pool) is
 *                idle: its row of out is zero and no state changes. Two rows with
 *                the same slot race.
 *  out           contiguous [B, D], 16-byte aligned.
 *
 * No workspace. Errors as sx_causal_conv.
 */
sx_status sx_causal_conv_step(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x,
                              int64_t taps, const float* weight, const float* bias, sx_activation activation,
                              int64_t pool, int64_t state_stride, void* state, const int32_t* slots, void* out,
                              void* stream);

/*
 * sx_selective_scan: the scan of a selective state space. With N states h a
 * channel from `initial` (or zero), for each token
 *   dt = softplus(delta + delta_bias)   (delta + delta_bias where `softplus` is zero)
 *   h[n] = exp(dt a[n]) h[n] + dt x b[n],   y = sum over n of c[n] h[n] + skip x,
 *   out = y z / (1 + exp(-z))           (y where z is NULL).
 * Steps, states and sums are f32 for f32 and bf16 operands alike; out is rounded
 * to `dtype` once. Rates and steps have any sign: a state may grow, and one of
 * zero stays zero while no token's own decay exp(dt a) passes f32's range. A step of
 * zero keeps a state whatever its rate.
 *
 *  dtype         SX_F32 or SX_BF16: x, delta, b, c, z and out.
 *  x, delta, z   [B, T, D] (x's shape), each with strides (NULL for contiguous; any
 *                value). z and its strides may be NULL.
 *  a             f32, contiguous [D, N], 1 <= N <= SX_MAX_STATES (else SX_E_UNSUPPORTED).
 *  b, c          [B, T, G, N] (b's shape, 4 entries), each with strides; G divides
 *                D, and channel d reads row d / (D / G).
 *  skip, delta_bias  f32 [D], or NULL for zero.
 *  initial       f32, contiguous [B, D, N], or NULL for zero.
 *  lengths       int32 [B], or NULL. Tokens of row b from lengths[b] on do not
 *                exist: they are not read, their rows of out are zero and the
 *                state ends before them. Taken into [0, T].
 *  out           contiguous [B, T, D], 16-byte aligned.
 *  final_state   f32, contiguous [B, D, N], 16-byte aligned: the state after the
 *                last token; or NULL.
 *  workspace     at least sx_selective_scan_workspace_bytes() bytes, 256-byte
 *                aligned; may hold anything; may be NULL when that is 0.
 *
 * An infinity or NaN of one token's x, delta or z stays in its channel, one of b
 * or c in its group (an infinity may come out as NaN); of x, delta and b it
 * reaches later tokens too, earlier ones never. Outputs overlap no input and not each other (SX_E_ALIAS). Errors
 * otherwise as sx_decay_attention.
 */
sx_status sx_selective_scan(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x,
                            const int64_t* delta_strides, const void* delta, const float* a, const int64_t* b_shape,
                            const int64_t* b_strides, const void* b, const int64_t* c_strides, const void* c,
                            const float* skip, const int64_t* z_strides, const void* z, const float* delta_bias,
                            int softplus, const float* initial, const int32_t* lengths, void* out, float* final_state,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes sx_selective_scan needs (0 when none, or for shapes it would reject). */
size_t sx_selective_scan_workspace_bytes(sx_dtype dtype, const int64_t* x_shape, const int64_t* b_shape);

/*
 * sx_selective_scan_backward: gradients of sx_selective_scan. With gy = grad_out
 * z / (1 + exp(-z)) and lam the adjoint of h (grad_state after the last token),
 *   lam = c gy + mu,  mu = exp(dt a) lam  (what is passed back),  q = mu h of the token before,
 *   grad_c = sum over a group's channels of gy h,  grad_b = the same of dt x lam,
 *   grad_a = sum over rows and tokens of dt q,  grad_x = dt sum over n of (lam b) + skip gy,
 *   grad_delta = (sum over n of (a q) + x sum over n of (lam b)) softplus'(delta + delta_bias),
 *   grad_z = grad_out y silu'(z),  grad_skip and grad_delta_bias sums of gy x and grad_delta.
 *
 *  dtype .. lengths  as for the forward call.
 *  grad_out      [B, T, D], dtype `dtype`, with strides (NULL for contiguous).
 *  grad_state    f32, contiguous [B, D, N]: the gradient of final_state, or NULL.
 *  grad_x, grad_delta, grad_z  contiguous [B, T, D], dtype `dtype`; grad_z may be
 *                NULL where z is.
 *  grad_a        f32, contiguous [D, N].
 *  grad_b, grad_c  contiguous [B, T, G, N], dtype `dtype`, summed in f32 and rounded once.
 *  grad_skip, grad_delta_bias  f32 [D], or NULL where not wanted.
 *  grad_initial  f32, contiguous [B, D, N], or NULL where not wanted.
 *  workspace     at least sx_selective_scan_backward_workspace_bytes() bytes,
 *                256-byte aligned; may hold anything. It holds the states of
 *                every eighth token, 0.125 B T D N floats for N of 4, 8, 12, 16
 *                or 32 (others take those of the next), and sums: 0.15 to 0.16
 *                B T D N in all for many tokens of 16 or 32 states.
 *
 * Gradients of tokens that do not exist are zero. The outputs are 16-byte
 * aligned and overlap nothing. Results do not change from call to call (no
 * atomics). Errors as sx_selective_scan.
 */
sx_status sx_selective_scan_backward(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x,
                                     const int64_t* delta_strides, const void* delta, const float* a,
                                     const int64_t* b_shape, const int64_t* b_strides, const void* b,
                                     const int64_t* c_strides, const void* c, const float* skip,
                                     const int64_t* z_strides, const void* z, const float* delta_bias, int softplus,
                                     const float* initial, const int32_t* lengths, const int64_t* grad_out_strides,
                                     const void* grad_out, const float* grad_state, void* grad_x, void* grad_delta,
                                     float* grad_a, void* grad_b, void* grad_c, float* grad_skip, void* grad_z,
                                     float* grad_delta_bias, float* grad_initial, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* Workspace bytes sx_selective_scan_backward needs (0 for shapes it would reject). */
size_t sx_selective_scan_backward_workspace_bytes(sx_dtype dtype, const int64_t* x_shape, const int64_t* b_shape);

/*
 * sx_selective_scan_step: one token of every request of a batch, the states
 * updated in place.
 *
 *  x, delta, z   [B, D] (x's shape), b, c [B, G, N] (b's shape), each with strides.
 *  a .. softplus  as for sx_selective_scan.
 *  pool, state_stride, state
 *                f32 [pool, D, N]; each state contiguous, `state_stride` elements
 *                from one to the next, none overlapping (else SX_E_UNSUPPORTED).
 *                On 16-byte borders throughout it is read and written in larger pieces.
 *  slots         as for sx_causal_conv_step.
 *  out           contiguous [B, D], 16-byte aligned.
 *
 * No workspace. Errors as sx_selective_scan.
 */
sx_status sx_selective_scan_step(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x,
                                 const int64_t* delta_strides, const void* delta, const float* a,
                                 const int64_t* b_shape, const int64_t* b_strides, const void* b,
                                 const int64_t* c_strides, const void* c, const float* skip, const int64_t* z_strides,
                                 const void* z, const float* delta_bias, int softplus, int64_t pool,
                                 int64_t state_stride, float* state, const int32_t* slots, void* out, void* stream);

/*
 * sx_group_norm: the norm of groups of channels, channels last. Over the
 * positions of a sample and the channels of a group,
 *   u = (x - mean) / sqrt(variance + eps) weight + bias,  out = act(u).
 * f32, the variance from differences to a mean; rounded to `dtype` once.
 *
 *  dtype         SX_F32 or SX_BF16: x and out.
 *  x             [samples, positions, channels]: shape, strides (NULL for
 *                contiguous; the channels next to each other, else SX_E_UNSUPPORTED)
 *                and data.
 *  groups        divides the channels.
 *  weight, bias  f32 [channels], or NULL for ones and zeros.
 *  out           contiguous, x's shape, 16-byte aligned.
 *  workspace     at least sx_group_norm_workspace_bytes() bytes, 256-byte aligned;
 *                may hold anything; may be NULL when that is 0.
 *
 * An infinity or NaN turns its sample's group to NaN and no other. A variance
 * past f32's range counts as infinite: u is the bias then. Errors as
 * sx_decay_attention.
 */
sx_status sx_group_norm(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x, int64_t groups,
                        const float* weight, const float* bias, float eps, sx_activation activation, void* out,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes sx_group_norm needs (0 when none, or for shapes it would reject). */
size_t sx_group_norm_workspace_bytes(sx_dtype dtype, const int64_t* x_shape, int64_t groups);

/*
 * sx_group_norm_backward: gradients of sx_group_norm. With n = (x - mean) r,
 * r = 1 / sqrt(variance + eps) and gu = grad_out act'(u),
 *   grad_weight = sum of gu n,  grad_bias = sum of gu,
 *   grad_x = r (gu weight - mean(gu weight) - n mean(gu weight n)).
 *
 *  dtype .. activation   as for the forward call.
 *  grad_out      x's shape, with strides as x has them.
 *  grad_x        contiguous, x's shape, dtype `dtype`.
 *  grad_weight, grad_bias  f32 [channels], or NULL where not wanted. Summed in a
 *                fixed order (no atomics).
 *  workspace     at least sx_group_norm_backward_workspace_bytes() bytes,
 *                256-byte aligned; may hold anything.
 */
sx_status sx_group_norm_backward(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x,
                                 int64_t groups, const float* weight, const float* bias, float eps,
                                 sx_activation activation, const int64_t* grad_out_strides, const void* grad_out,
                                 void* grad_x, float* grad_weight, float* grad_bias, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Workspace bytes sx_group_norm_backward needs (0 for shapes it would reject). */
size_t sx_group_norm_backward_workspace_bytes(sx_dtype dtype, const int64_t* x_shape, int64_t groups);

/* "E-DIM-001" etc. for a status; "OK" for SX_OK. Static storage. */
const char* sx_status_name(sx_status status);

/* Message of the last failed call on this thread (thread-local storage,
 * valid until the next call on the thread); "" after a success. */
const char* sx_last_error(void);

/* Library version string, e.g. "sx_scan 0.1 gfx950". Static storage. */
const char* sx_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SX_SCAN_H */
