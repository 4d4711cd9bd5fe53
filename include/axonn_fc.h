/*
 * axonn_fc.h -- C ABI of the GB300 FC-layer GEMM library (libaxonn_fc.so).
 *
 * What it computes.  The three matrix products of a fully-connected layer's
 * training step, either on the whole layer or on one local block of
 * Agarwal's 3D parallel matrix multiplication.  Figure 1 of "Democratizing
 * AI: Open-source Scalable LLM Training on GPU-based Supercomputers" shows
 * one FC layer's matmul split this way over a virtual grid whose three
 * extents are G_x, G_y and G_z; the pith.science review of arXiv
 * 2502.08145 ("What carries the argument") places that grid inside a 4D
 * one, G_data x G_x x G_y x G_z, joined by collectives:
 *
 *   forward          Y[T x N]  = X[T x K] . W[K x N]
 *   data gradient    dX[T x K] = dY[T x N] . W^T
 *   weight gradient  dW[K x N] = X^T . dY
 *
 * Inputs and outputs are bf16; products accumulate in fp32 on the tensor
 * cores and are rounded once, to nearest even, when written as bf16.
 *
 * 3D grid.  T is split by G_z, K by G_x and N by G_y.  Block (x, y, z) owns
 * X[Tz, Kx], W[Kx, Ny] and dY[Tz, Ny] and computes
 *   fwd    Y^(x)_{z,y}  = X[Tz,Kx] . W[Kx,Ny]      (partials summed over x)
 *   dgrad  dX^(y)_{z,x} = dY[Tz,Ny] . W[Kx,Ny]^T   (summed over y)
 *   wgrad  dW^(z)_{x,y} = X[Tz,Kx]^T . dY[Tz,Ny]   (summed over z)
 * A dimension D is cut into units of 8 elements: with U = ceil(D/8), block b
 * of G gets floor(U/G) units plus one if b < U mod G, blocks are contiguous
 * in order, and the last block is clipped at D (see axonn_block_range).
 *
 * Virtual grid (AXONN_VGRID).  All G_x*G_y*G_z block products run on this
 * GPU, and an on-device sum over the reduced axis (G = G_x for fwd, G_y for
 * dgrad, G_z for wgrad) stands in for the grid's all-reduce /
 * reduce-scatter.  Three forms:
 *  - default (chained): each output tile runs the G block products of its
 *    output block one after another, in order g = 0..G-1, into one fp32
 *    accumulator on the tensor cores, each block product read from its own
 *    block (its own tensor maps, zero-filled at the block's edges).  One
 *    launch, no workspace, no partial in memory; results are the same on
 *    every run.
 *  - AXONN_VGRID_PARTIALS: one launch writes the partials 0..G-2 in fp32 to
 *    the caller's workspace, and a second computes partial G-1, whose
 *    epilogue adds partials 0..G-1 in that order and writes the output
 *    (the partials as the grid's ranks would hold them); results are the
 *    same on every run, and may differ from the chained form in the last
 *    bits (another summation order).
 *  - AXONN_REDUCE_ADD (fp32 accumulating output only): all blocks run in
 *    one launch and each adds its tile into the output with fp32 reduction
 *    adds (PTX red.global.add: rounded to nearest even, subnormal inputs
 *    and results flushed to zero): no workspace, and a summation order that
 *    can change from run to run (every order stays within the same error
 *    bound; integer-valued sums below 2^24 are exact in any order).
 *
 * Conventions for every entry point below.
 *  - Pointers are DEVICE pointers; the caller owns every buffer and the
 *    stream.  The library never allocates device memory on a call; scratch
 *    comes from the caller's workspace (axonn_fc_workspace_size).
 *  - Layout: matrices are row-major with a leading dimension (row stride) in
 *    elements.  Flag AXONN_A_T says the op's first operand (X for fwd and
 *    wgrad, dY for dgrad) is stored transposed, i.e. as [K x T] / [N x T];
 *    AXONN_B_T says the second operand (W for fwd and dgrad, dY for wgrad) is
 *    stored transposed ([N x K] for W -- PyTorch's Linear layout -- or
 *    [N x T] for dY).  Outputs are always row-major in their logical shape.
 *  - Alignment: every base pointer 16-byte aligned; bf16 leading dimensions
 *    multiples of 8, fp32 ones multiples of 4.  Otherwise AXONN_ERR_ALIGNMENT.
 *  - Calls are asynchronous on `stream`.  A device-side timeout (a bounded
 *    wait inside a kernel that expired) is reported by axonn_sync_status.
 *  - Errors are status codes; axonn_last_error() gives a thread-local message.
 *    No C++ exception crosses this boundary.
 *  - Threads: every entry point may be called from several host threads at
 *    once (on different streams); the tuning table and per-device set-up are
 *    guarded by locks.  The kernel-configuration override and the wait
 *    timeout are process-wide.
 *  - Empty outputs (an extent of 0) return AXONN_OK and touch nothing; an
 *    empty reduction range writes zeros (leaves C bit for bit unchanged
 *    with AXONN_ACCUM_F32).
 */
#ifndef AXONN_FC_H_
#define AXONN_FC_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  AXONN_OK = 0,
  AXONN_ERR_INVALID_ARG = 1,  /* bad size, grid, coordinate, flag or pointer */
  AXONN_ERR_ALIGNMENT = 2,    /* pointer or leading dimension misaligned */
  AXONN_ERR_UNSUPPORTED = 3,  /* valid request the library cannot run */
  AXONN_ERR_WORKSPACE = 4,    /* workspace missing or too small */
  AXONN_ERR_CUDA = 5,         /* a CUDA runtime/driver call failed */
  AXONN_ERR_TIMEOUT = 6       /* a bounded device-side wait expired */
} axonn_status_t;

typedef enum { AXONN_OP_FWD = 0, AXONN_OP_DGRAD = 1, AXONN_OP_WGRAD = 2 } axonn_op_t;

/* Layer sizes, grid and block coordinate.  A full-layer product is the grid
 * 1x1x1 at (0,0,0).  gx, gy, gz >= 1; 0 <= x < gx etc. */
typedef struct {
  int64_t T, K, N;
  int32_t gx, gy, gz;
  int32_t x, y, z;
} axonn_fc_shape_t;

/* Flags (bitwise or). */
#define AXONN_A_T 0x1u            /* first operand stored transposed */
#define AXONN_B_T 0x2u            /* second operand stored transposed */
#define AXONN_ACCUM_F32 0x4u      /* output is fp32 and the result is added (one fp32
                                     reduction add per element: round to nearest even,
                                     subnormals flushed to zero) */
#define AXONN_VGRID 0x8u          /* all blocks + on-device partial sum */
#define AXONN_FULL_OPERANDS 0x10u /* block mode: pointers are full matrices */
#define AXONN_OUT_F32 0x20u       /* output is fp32, overwritten */
#define AXONN_ZSHARDED 0x40u      /* axonn_fc_workspace_size of axonn_fc_wgrad_zsharded */
#define AXONN_REDUCE_ADD 0x80u    /* with AXONN_VGRID | AXONN_ACCUM_F32: every block added
                                     into the output by fp32 reduction adds, in no fixed
                                     order; one launch, no workspace */
#define AXONN_VGRID_PARTIALS 0x100u /* with AXONN_VGRID: the two-launch form, fp32 partials
                                     of blocks 0..G-2 in the workspace, summed in order in
                                     the last block's epilogue */

/*
 * Forward product Y = X . W of the layer, of block (x,y,z), or of the whole
 * virtual grid.
 *   X   first operand, [T x K] (or [K x T] with AXONN_A_T), leading dim ldx
 *   W   second operand, [K x N] (or [N x K] with AXONN_B_T), leading dim ldw
 *   Y   output [T x N], leading dim ldy; bf16 unless AXONN_ACCUM_F32 /
 *       AXONN_OUT_F32 make it fp32
 *   Block mode (no AXONN_VGRID, grid larger than 1): without
 *   AXONN_FULL_OPERANDS the pointers address the block's own shards
 *   (X_blk [Tz x Kx], W_blk [Kx x Ny], Y_blk [Tz x Ny], each with its ld);
 *   with it they address the full matrices and the block is located by its
 *   offsets, its partial written at Y[Tz, Ny].
 *   ws / ws_bytes: device workspace, needed with AXONN_VGRID |
 *   AXONN_VGRID_PARTIALS when G_x > 1 (size from
 *   axonn_fc_workspace_size).  Otherwise optional: a full-size one enables
 *   the stream-K tail of large products; NULL / 0 runs without it.
 *   Reduction split: a single product (no AXONN_VGRID) whose tiles leave
 *   SMs idle may have its reduction range cut into S = 2, 4 or 8 pieces of
 *   whole 64-deep stages, computed by the S CTAs of a thread-block cluster
 *   and added in fixed order (pieces 0, 1, ..., S-1) inside it, with no
 *   workspace and no extra launch.  Without a tuning entry it is chosen
 *   for reductions of 32 stages or more; the tuner times S = 2, 4, 8.
 */
axonn_status_t axonn_fc_fwd(const void* X, const void* W, void* Y, int64_t ldx, int64_t ldw,
                            int64_t ldy, const axonn_fc_shape_t* shape, uint32_t flags,
                            void* ws, size_t ws_bytes, cudaStream_t stream);

/* Data gradient dX = dY . W^T.  dY [T x N] (AXONN_A_T: [N x T]), W [K x N]
 * (AXONN_B_T: [N x K]), dX [T x K].  Block (x,y,z) yields dX^(y)_{z,x};
 * the virtual grid sums over y.  Other arguments as for axonn_fc_fwd. */
axonn_status_t axonn_fc_dgrad(const void* dY, const void* W, void* dX, int64_t lddy,
                              int64_t ldw, int64_t lddx, const axonn_fc_shape_t* shape,
                              uint32_t flags, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Weight gradient dW = X^T . dY.  X [T x K] (AXONN_A_T: [K x T]), dY
 * [T x N] (AXONN_B_T: [N x T]), dW [K x N].  Block (x,y,z) yields
 * dW^(z)_{x,y}; the virtual grid sums over z.  AXONN_ACCUM_F32 gives the
 * fp32 main-gradient update dW += X^T . dY. */
axonn_status_t axonn_fc_wgrad(const void* X, const void* dY, void* dW, int64_t ldx,
                              int64_t lddy, int64_t lddw, const axonn_fc_shape_t* shape,
                              uint32_t flags, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * Z-sharded weights of the 3D grid.  Each rank (x, y, z) keeps only shard z
 * of its weight block W_{x,y}; the grid all-gathers the block over the Z
 * group before using it and reduce-scatters the weight-gradient partials
 * over the Z group into shards (the review of arXiv 2502.08145, "What
 * carries the argument", has the weights split over the Z axis and data
 * moved by all-gather, reduce-scatter and all-reduce).  Shards are row
 * blocks of W_{x,y} cut by the grid's split rule (units of 8 rows, leading
 * shards take the extra unit; see axonn_block_range).
 *
 * axonn_shards_gather -- the all-gather, on one GPU: copies g bf16 row
 * shards, shard z = rows [split(rows, g, z)) stored row-major with leading
 * dimension ld_shard at shards[z] (a HOST array of g DEVICE pointers), into
 * `out` [rows x cols] (leading dimension ld_out).  cols, ld_shard and ld_out
 * must be multiples of 8 and every pointer 16-byte aligned
 * (AXONN_ERR_ALIGNMENT); 1 <= g <= 64.
 *
 * axonn_fc_wgrad_zsharded -- the Z-group weight gradient with its
 * reduce-scatter, on one GPU: for block (shape->x, shape->y) it computes
 * every partial dW^(z)_{x,y} = X[Tz,Kx]^T . dY[Tz,Ny], z = 0..G_z-1, sums
 * them in fixed order z = 0..G_z-1 and writes row shard z' of the sum to
 * dW_shards[z'] (a HOST array of G_z DEVICE pointers; each [rows of shard z'
 * x Ny], leading dimension ld_shard; bf16, or fp32 with AXONN_OUT_F32 /
 * AXONN_ACCUM_F32).  X and dY are the full [T x K] and [T x N] matrices (or
 * transposed with AXONN_A_T / AXONN_B_T); shape->z is ignored.  Partials
 * 0..G_z-2 go to `ws`: axonn_fc_workspace_size(AXONN_OP_WGRAD, shape,
 * AXONN_ZSHARDED) bytes.
 */
axonn_status_t axonn_shards_gather(const void* const* shards, int32_t g, int64_t rows, int64_t cols,
                                   int64_t ld_shard, void* out, int64_t ld_out, cudaStream_t stream);
axonn_status_t axonn_fc_wgrad_zsharded(const void* X, const void* dY, void* const* dW_shards,
                                       int64_t ldx, int64_t lddy, int64_t ld_shard,
                                       const axonn_fc_shape_t* shape, uint32_t flags, void* ws,
                                       size_t ws_bytes, cudaStream_t stream);

/*
 * Virtual-grid product (as the entry points above with AXONN_VGRID) that
 * allocates nothing and needs no workspace argument.  The pages have no
 * counterpart: this exists for callers that cannot call cudaMalloc, such as
 * code that runs inside a host framework that owns all device memory, or
 * code that must not allocate once it is running.
 *   op        axonn_op_t; P, Q, C and ld* as for that op's entry point
 *   flags     as for the entry points; AXONN_VGRID is implied
 * The fp32 partials of the two-launch form (AXONN_VGRID_PARTIALS) live in
 * a fixed 64 MiB scratch array inside the library, which every GPU that
 * loads the library holds until the process exits.  A product whose
 * partials need more ((G-1) * M * ceil8(N) * 4 bytes, G the reduced grid
 * extent, M x N the output) returns AXONN_ERR_WORKSPACE with a message.
 * The default chained form, AXONN_REDUCE_ADD and products whose reduced
 * axis has one block need no scratch.  The first call
 * on each device looks up the scratch's device address (once, with that
 * device current); make that first call before any stream capture.  Every
 * call uses the same scratch and the kernels overwrite every partial they
 * later read, so no clearing is needed -- but calls that overlap on the GPU
 * (on different streams, or from different threads) race on it and must be
 * serialised by the caller.
 */
axonn_status_t axonn_fc_vgrid_static(int op, const void* P, const void* Q, void* C, int64_t ldp,
                                     int64_t ldq, int64_t ldc, const axonn_fc_shape_t* shape,
                                     uint32_t flags, cudaStream_t stream);

/*
 * Goldfish-loss masked cross-entropy over bf16 logits, with its gradient.
 * Against memorisation the paper trains with Goldfish Loss, which leaves
 * tokens out of the cross-entropy at random (pith.science review of arXiv
 * 2502.08145, "What carries the argument"), with mask parameters k = 2 and
 * h = 13 ("Assumptions & free parameters").  The rule, read from the
 * method's own paper that the pages cite (Hans et al., arXiv 2406.10209):
 *   label (b, t) is dropped when FNV-1a-64 of input_ids[b, t-h+1 .. t] (each
 *   id as 4 little-endian bytes, oldest first) is 0 mod k; labels with
 *   fewer than h tokens before them in their row are kept; k = 0 keeps all;
 *   labels outside [0, vocab) are padding (neither kept nor counted).
 *   CE_t = logsumexp(z_t) - z_t[y_t] (natural log, fp32 arithmetic)
 *   loss = sum over kept t of CE_t / n, n = number kept (0 when n = 0)
 *   dlogits_t = G_t (softmax(z_t) - e_{y_t}) / n  (zero rows where dropped)
 * Arguments (DEVICE pointers, caller-owned; T = batch * seq positions in
 * row-major (b, t) order):
 *   logits      bf16 [T x vocab], leading dimension ld_logits (multiple of
 *               8, 16-byte aligned base); rows of dropped labels are not read
 *   input_ids   int32 [batch x seq], the tokens the windows are hashed from
 *   labels      int32 [batch x seq], the token each position predicts
 *   keep        out, uint8 [T]: 1 where the label counts
 *   token_loss  out, fp32 [T]: CE_t where kept, 0 elsewhere
 *   loss        out, fp32 [1]: the mean over kept labels (a fixed-order sum);
 *               during the call its word is the kernels' row counter
 *   kept        out, int32 [1]: n
 *   dlogits     out, bf16 [T x vocab] with ld_dlogits (same alignment), or
 *               NULL for the loss alone
 * 1 <= h <= 4096, k >= 0, vocab up to 8 x 49152.  Three kernel launches on
 * `stream`, no workspace, no allocation.  A wait that expires is reported
 * by axonn_sync_status.  AXONN_ERR_INVALID_ARG / _ALIGNMENT / _UNSUPPORTED
 * as for the products.
 */
axonn_status_t axonn_goldfish_ce(const void* logits, int64_t ld_logits, const int32_t* input_ids,
                                 const int32_t* labels, int64_t batch, int64_t seq, int64_t vocab,
                                 int32_t k, int32_t h, uint8_t* keep, float* token_loss,
                                 float* loss, int32_t* kept, void* dlogits, int64_t ld_dlogits,
                                 cudaStream_t stream);

/*
 * Epilogues of an FC layer: bias, activation, dropout and residual.
 *
 *   forward    Z = X . W + b;   Y = R + D(act(Z))
 *   backward   d = act'(Z) D(G);  dZ = d + R;  db = column sums of d
 *
 * where G is the gradient of Y, either a matrix (axonn_epi_bwd) or the data
 * gradient dY . W^T of the layer after it (axonn_fc_dgrad_epi, in whose
 * epilogue it is then never written out).  dW and dX of the layer itself are
 * the products above on dZ.  Every part is optional.  All arithmetic is fp32,
 * and Y, Z and dZ are rounded once.  Exponentials and reciprocals come from
 * the special function units (relative errors near 2^-22, and 0 for results
 * below 2^-126): an activation is within 2^-20 of itself plus 2^-21, a slope
 * within 2^-20.  GELU's negative tail, z <= -2, is within 1.5 z^2 2^-24 + 2^-19
 * of itself, its slope there within 1.6 times that.
 *
 * Activations: relu (slope 0 at 0; NaN stays), gelu z (1 + erf(z/sqrt 2))/2,
 * gelu_tanh z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))/2, silu z/(1+e^-z).
 *
 * Dropout D drops an element with probability p and scales the others.  Its
 * mask is computed where it is needed, forward and backward, and never
 * stored: 16 random bits for each element from Philox4x32-10 (Salmon,
 * Moraes, Dror and Shaw, SC'11), the key the seed's two 32-bit halves (low
 * first), the counter (col >> 3, row, offset low, offset high), and the bits
 * word col & 7 of the output's eight 16-bit words, lowest first.  With
 * thr = floor(65536 p + 1/2) an element is dropped (set to 0, whatever it
 * is) where its bits are below thr and is multiplied by the fp32 number
 * nearest 65536/(65536 - thr) elsewhere; thr = 65536 drops all.
 * (seed, offset) are two 64-bit words on the DEVICE, so that a captured graph
 * draws a new mask when they are changed between replays; the library only
 * reads them.  Calls that must
 * draw alike, as a forward and its backward, get the same words and rows.
 */
#define AXONN_BIAS_F32 0x200u     /* axonn_fc_fwd_epi: the bias is fp32 (else bf16) */
#define AXONN_IN_F32 0x400u       /* axonn_epi_bwd: dY is fp32 (else bf16); axonn_dropout: X,
                                     residual and Y are fp32 (else bf16); operators over rows
                                     of logits: logits and dlogits are fp32 (else bf16) */
#define AXONN_LSE_PARTS 0x800u    /* axonn_token_logprobs and its backward: lse is [T x 2], the
                                     row's largest logit and ln sum_v e^(z_v - max z) */
typedef enum {
  AXONN_ACT_NONE = 0,
  AXONN_ACT_RELU = 1,
  AXONN_ACT_GELU = 2,
  AXONN_ACT_GELU_TANH = 3,
  AXONN_ACT_SILU = 4
} axonn_act_t;

typedef struct {
  const void* bias;      /* forward: [N] or NULL; bf16, or fp32 with AXONN_BIAS_F32 */
  void* pre;             /* bf16 Z: written by the forward where not NULL, read by the
                            backward (NULL only with AXONN_ACT_NONE) */
  int64_t ld_pre;
  const void* residual;  /* R or NULL, of the output's type; may be the output itself */
  int64_t ld_residual;
  float* dbias;          /* backward: db, fp32 [columns], overwritten; or NULL */
  const uint64_t* rng;   /* seed and offset (device); may be NULL with p = 0 */
  int32_t act;           /* axonn_act_t */
  float p;               /* dropout probability, 0 <= p <= 1 */
} axonn_epilogue_t;

/* Y = R + D(act(X . W + b)) of the whole layer (grid 1x1x1, else
 * AXONN_ERR_UNSUPPORTED) in one launch.  X, W, Y and their leading
 * dimensions as for axonn_fc_fwd; flags AXONN_A_T, AXONN_B_T, AXONN_OUT_F32
 * (Y and R fp32) and AXONN_BIAS_F32.  bias is 16-byte aligned like every
 * matrix.  No workspace. */
axonn_status_t axonn_fc_fwd_epi(const void* X, const void* W, void* Y, int64_t ldx, int64_t ldw,
                                int64_t ldy, const axonn_fc_shape_t* shape, uint32_t flags,
                                const axonn_epilogue_t* epi, cudaStream_t stream);

/* dZ = act'(Z) D(dY . W^T) + R, [T x K], and db [K]: the data gradient of
 * the layer `shape`, turned into the gradient of the pre-activation Z of the
 * layer before it.  dY, W, dX (here dZ) as for axonn_fc_dgrad; flags
 * AXONN_A_T, AXONN_B_T and AXONN_OUT_F32 (dZ and R fp32).  dX may be pre
 * itself (bf16) or R.  db is summed in a fixed order from fp32 values; it
 * needs a workspace of axonn_epi_workspace_size(T, K) bytes and a second
 * launch. */
axonn_status_t axonn_fc_dgrad_epi(const void* dY, const void* W, void* dX, int64_t lddy, int64_t ldw,
                                  int64_t lddx, const axonn_fc_shape_t* shape, uint32_t flags,
                                  const axonn_epilogue_t* epi, void* ws, size_t ws_bytes,
                                  cudaStream_t stream);

/* dZ = act'(Z) D(dY), bf16 [rows x cols], and db [cols], from a gradient
 * that is already there (bf16, or fp32 with AXONN_IN_F32).  dZ may be dY
 * (bf16) or pre.  db as for axonn_fc_dgrad_epi.  bias and residual of the
 * epilogue must be NULL. */
axonn_status_t axonn_epi_bwd(const void* dY, int64_t lddy, void* dZ, int64_t lddz, int64_t rows,
                             int64_t cols, uint32_t flags, const axonn_epilogue_t* epi, void* ws,
                             size_t ws_bytes, cudaStream_t stream);

/* Workspace bytes of the bias gradient over a [rows x cols] matrix:
 * ceil(rows / 32) * ceil8(cols) * 4.  Host-only. */
axonn_status_t axonn_epi_workspace_size(int64_t rows, int64_t cols, size_t* bytes);

/* Y = R + D(X) over [rows x cols] (residual NULL: no R), bf16, or fp32 with
 * AXONN_IN_F32; Y may be X or R.  The backward is the same call on the
 * gradient.  One launch. */
axonn_status_t axonn_dropout(const void* X, int64_t ldx, const void* residual, int64_t ld_residual,
                             void* Y, int64_t ldy, int64_t rows, int64_t cols, float p,
                             const uint64_t* rng, uint32_t flags, cudaStream_t stream);

/*
 * Softmax cross-entropy of the logits X . W over a vocabulary, with its
 * gradients, without the logits ever being written out.
 *   z_t = X_t . W (fp32);  CE_t = ln sum_v e^(z_tv) - z_t[y_t]
 *   loss = sum over counted t of CE_t / n, n = number counted (0 when n = 0)
 *   P_tv = softmax(z_t)_v - [v = y_t] for counted t, g = grad_scale / n
 *   dX = g P . W^T (rows that do not count: zeros);  dW = g X^T . P
 * A position counts when its label is in [0, V) and keep (uint8 [T], may be
 * NULL) is not 0 there; the mask of axonn_goldfish_ce fits.  The others cost
 * no products and their rows of X are not read: the counted rows are packed
 * first, and their number stays on the device.
 *   X        bf16 [T x K];  W bf16 [K x V], or [V x K] with AXONN_B_T (an
 *            embedding tied to the head)
 *   token_loss  out, fp32 [T]: CE_t where counted, 0 elsewhere
 *   lse      out, fp32 [T]: the logsumexp, 0 elsewhere; or NULL
 *   loss, kept  out, fp32 [1] and int32 [1] (n)
 *   dX       out, bf16 [T x K], or NULL
 *   dW       out, in W's layout, or NULL; bf16, fp32 with AXONN_OUT_F32, or
 *            added into fp32 with AXONN_ACCUM_F32
 * With dX and dW NULL it is the loss alone.  dX must not overlap X.
 * The vocabulary is taken in pieces.  The softmax's statistics come from
 * each piece's product, in fp32, in its epilogue; P is held for one piece at
 * a time, in bf16 (each entry rounded once), and the products dX and dW read
 * it from there.  The last piece of the forward sweep stays, each logit as
 * its distance below a maximum of its row in 16 bits (which changes an entry
 * of P by at most 2^-12 of itself, and by 2^-32 of that maximum's), and
 * opens the backward one; the others are computed again (the last one too
 * where the features are so few that this is sooner).  The piece is as large
 * as the workspace allows: with one that holds the whole vocabulary
 * nothing is computed twice.  A NaN logit shows in its whole row's gradient.
 *   ws       256-byte aligned; axonn_linear_ce_workspace_size gives its
 *            bytes for pieces of `piece` columns (rounded up to 256; 0: at
 *            most 2 GiB of P at a time).  Anything from the size for
 *            piece = 1 up will do (AXONN_ERR_WORKSPACE below).
 * All sums are in a fixed order: results are the same on every run.
 */
axonn_status_t axonn_linear_ce(const void* X, int64_t ldx, const void* W, int64_t ldw,
                               const int32_t* labels, const uint8_t* keep, int64_t T, int64_t K,
                               int64_t V, float grad_scale, uint32_t flags, float* token_loss,
                               float* lse, float* loss, int32_t* kept, void* dX, int64_t lddx,
                               void* dW, int64_t lddw, void* ws, size_t ws_bytes,
                               cudaStream_t stream);

/* Workspace bytes of axonn_linear_ce; grad != 0 when dX or dW is asked for.
 * They include room for dX as fp32 parts where its few tiles leave SMs idle
 * over a long vocabulary, which depends on the current device (without one:
 * none, and the call then runs without them).  Launches nothing. */
axonn_status_t axonn_linear_ce_workspace_size(int64_t T, int64_t K, int64_t V, uint32_t flags,
                                              int grad, int64_t piece, size_t* bytes);

/*
 * Rows of vocabulary logits: log probabilities of given tokens with their
 * entropy and top alternatives, the way back through them, and distillation
 * from a teacher's lists.  With x a row of logits [V], tau the temperature,
 *   z = x / tau;  lse = ln sum_v e^(z_v);  ln p_v = z_v - lse
 *   H = -sum_v p_v ln p_v
 * Common to the three calls:
 *   logits   bf16, or fp32 with AXONN_IN_F32, [T x V] (ld_logits).  Columns
 *            behind V are neither read nor written.
 *   keep     uint8 [T] or NULL: a row whose byte is 0 counts for nothing and
 *            is not read
 *   temperature  in [1e-4, 1e4]
 * A logit of -inf has probability 0.  In a row of nothing else every
 * probability is 0: ln p = lse = -inf, H = 0, and no gradient of either (the
 * distillation's is p - q with p = 0 there, below).  A NaN or +inf among the
 * logits makes the row's numbers NaN.  Arithmetic and sums are fp32,
 * sums in an order that depends on the sizes alone, exponentials the special
 * function units' (2^-22; 0 below 2^-126); differences are taken from the row's
 * maximum before they are scaled, so a row of finite logits of any size gives
 * its own probabilities (in the way back with AXONN_LSE_PARTS).  No workspace.
 *
 * axonn_token_logprobs -- scoring, answering and a teacher's lists, in one
 * launch that reads the logits once (what a list may come from, again).  Each
 * output may be NULL:
 *   tokens   int32 [T], given with logprob: a token outside [0, V) (padding)
 *            has logprob 0; the row's other outputs are as for any row
 *   logprob  out, fp32 [T]: ln p of the row's token
 *   entropy  out, fp32 [T]: H;   lse  out, fp32 [T], or [T x 2] with
 *            AXONN_LSE_PARTS: m = max_v x_v and ln S = lse - m / tau
 *   top_index, top_logprob  out, int32 and fp32 [T x k] (ld_top >= k, 4-byte
 *            aligned): the row's k largest logits, best first, equal ones by
 *            index, and their ln p.  0 <= k <= min(V, 128).  -0 equals 0, and
 *            a NaN comes before every number.
 * Rows that keep leaves out get 0, and -1 as indices.
 *
 * axonn_token_logprobs_bwd -- with g and h the gradients of logprob and
 * entropy (a policy loss and its entropy bonus),
 *   dlogits_v = (g ([v = token] - p_v) - h p_v (ln p_v + H)) / tau
 *   tokens, dlogprob   int32 and fp32 [T], or both NULL; a token outside
 *                      [0, V) has no gradient
 *   lse                as the forward left it for these logits and this
 *                      temperature.  [T x 2] with AXONN_LSE_PARTS: p =
 *                      e^((x - m) / tau - ln S), right for logits of any size.
 *                      [T]: p = e^(x / tau - lse), which is off by 2^-23 |lse|
 *                      of itself; where |lse| is above 65536 a gradient cannot
 *                      be had from it and is NaN (0 at logits of -inf where lse
 *                      is -inf: a row of nothing else has no gradient)
 *   entropy, dentropy  fp32 [T], H as the forward left it, and h; or both NULL
 *   dlogits            out, of the logits' type, rounded once; may be the
 *                      logits themselves (same ld), else must not overlap them
 * Rows left out are written as zeros, and so are rows with g = h = 0, whatever
 * is in them.
 *
 * axonn_distill -- a student's loss against a teacher's lists of k logits
 * (or log probabilities: a list may be shifted by any number), renormalised:
 *   q = softmax(top_logit / tau) over the list
 *   KL_t = sum_j q_j (ln q_j - ln p[top_index_j]);  token_loss_t = tau^2 KL_t
 *   loss = sum over counted t of token_loss_t / n, n = number counted
 *   dlogits_v = grad_scale tau (p_v - sum of q_j with top_index_j = v) / n
 *   top_index, top_logit  int32 and fp32 [T x k] (ld_top >= k, 4-byte aligned),
 *              1 <= k <= 1024; a list ends at its first index outside [0, V).
 *              An index given twice teaches twice.  Entries of -inf have q = 0;
 *              a list of nothing else has loss and gradient 0, but counts.
 *   A row counts when keep does not leave it out and its list is not empty.
 *   token_loss out, fp32 [T]: 0 where not counted; +inf where q > 0 at p = 0.
 *              The gradient stays p - q there, and -q in a row of logits that are
 *              all -inf: finite beside an infinite loss
 *   loss, kept out, fp32 [1] and int32 [1] (n); loss is 0 for n = 0, and its
 *              word is the kernels' counter during the call
 *   dlogits    out, of the logits' type, or NULL for the loss alone; rows not
 *              counted get zeros; in place as above
 * Two launches; the logits are read from memory once, as far as a row fits the
 * shared memory of the CTAs that share it, and what does not again from L2.  A long
 * list costs as its square (4096 x 128256 bf16: 332 us with lists of 64, 464 of 256,
 * 664 of 257, 3.8 ms of 1024).
 */
typedef struct {
  const void* logits;
  int64_t ld_logits;
  const int32_t* tokens;
  const uint8_t* keep;
  int64_t T, V;
  float temperature;
  uint32_t flags;      /* AXONN_IN_F32, AXONN_LSE_PARTS */
  float* logprob;
  float* entropy;
  float* lse;
  int32_t* top_index;
  float* top_logprob;
  int64_t ld_top;
  int32_t k;
} axonn_token_logprobs_t;

typedef struct {
  const void* logits;
  int64_t ld_logits;
  const int32_t* tokens;
  const uint8_t* keep;
  int64_t T, V;
  float temperature;
  uint32_t flags;
  const float* lse;
  const float* dlogprob;
  const float* entropy;
  const float* dentropy;
  void* dlogits;
  int64_t ld_dlogits;
} axonn_token_logprobs_bwd_t;

typedef struct {
  const void* logits;
  int64_t ld_logits;
  const int32_t* top_index;
  const float* top_logit;
  int64_t ld_top;
  const uint8_t* keep;
  int64_t T, V;
  float temperature;
  uint32_t flags;
  float* token_loss;
  float* loss;
  int32_t* kept;
  void* dlogits;
  int64_t ld_dlogits;
  float grad_scale;
  int32_t k;
} axonn_distill_t;

/* The arguments are read during the call and not kept. */
axonn_status_t axonn_token_logprobs(const axonn_token_logprobs_t* args, cudaStream_t stream);
axonn_status_t axonn_token_logprobs_bwd(const axonn_token_logprobs_bwd_t* args, cudaStream_t stream);
axonn_status_t axonn_distill(const axonn_distill_t* args, cudaStream_t stream);

/*
 * Per-shape tuning -- the GB300 counterpart of the automatic tuning of BLAS
 * kernels that the pages credit (TL;DR of the sciencestack.ai page; "The
 * reading", review of arXiv 2502.08145).  Runs this call once per candidate -- kernel
 * configuration x rasterisation group {8, 16 tile rows; 8, 16 tile columns,
 * written -8, -16}, every configuration for products that leave SMs idle
 * (with reduction splits {2, 4, 8} of the 128x128 and 128x64
 * configurations, each piece
 * at least 128 deep), the 128x256 and 256-row configurations otherwise,
 * and the two best of them again with the
 * operand roles exchanged (see axonn_set_swap) -- and times each (through a captured
 * CUDA graph of 3 calls, 20 for products under 2e10 FLOP, where the stream
 * allows it) relative to the default choice run just before and after it,
 * so clock drift under the power cap cancels.  For products of 2e11 FLOP or
 * more, a candidate within 2 % of the fastest that loads fewer operand
 * bytes from L2 per multiply-add is kept instead (under the power cap those
 * bytes cost clock in a long run, which short timings do not show).  The
 * call synchronises `stream`.  It
 * records the fastest for later calls with the same op, sizes, grid, block
 * and flags on a GPU with the same SM count.  Arguments are those of the
 * op's entry point (op is an axonn_op_t); the caller's output is
 * overwritten (with AXONN_ACCUM_F32 the runs overwrite instead of adding;
 * with AXONN_REDUCE_ADD as well they add, once per run: tune on a scratch
 * output).  Not for use during stream capture.  Any
 * of the result pointers may be NULL.
 */
axonn_status_t axonn_fc_tune(int op, const void* P, const void* Q, void* C, int64_t ldp,
                             int64_t ldq, int64_t ldc, const axonn_fc_shape_t* shape,
                             uint32_t flags, void* ws, size_t ws_bytes, cudaStream_t stream,
                             int* best_config, int* best_split, int* best_group_m,
                             float* best_us);

/* The tuning table as text, one JSON object per line:
 *   {"key": "...", "config": "<name>", "split": S, "group_m": G,
 *    "streamk": 0 | 1 | 2, "swap": 0 | 1, "us": t}
 * (S a whole number 1..8, run as the largest power of two not above it
 * or the product's stage count, and only on the 128x128 and 128x64
 * configurations;
 * G a whole number in -64..-1 or 1..64, tile rows
 * per rasterisation group, negative for tile columns; streamk: off, on for
 * a partial round at most a quarter full, on wherever it applies; a line
 * without it loads as 1; swap: operand roles exchanged, see axonn_set_swap;
 * a line without it loads as 0).
 * save writes every entry; load merges a file's entries into the table
 * (AXONN_ERR_INVALID_ARG on an unreadable file or a malformed line, leaving
 * the table unchanged).  Host-only. */
axonn_status_t axonn_tune_cache_save(const char* path);
axonn_status_t axonn_tune_cache_load(const char* path);
void axonn_tune_cache_clear(void);
int axonn_tune_cache_size(void);

/* Whether the tuning table holds an entry that a call of op `op` (an
 * axonn_op_t) with this shape and these flags would run on the current
 * device (same SM count): *found = 1, else 0 (the call runs the default
 * choice).  AXONN_ERR_INVALID_ARG for a bad shape or flag or a NULL
 * `found`; AXONN_ERR_CUDA without a usable device.  Launches nothing. */
axonn_status_t axonn_tune_lookup(int op, const axonn_fc_shape_t* shape, uint32_t flags,
                                 int* found);

/* How the last call on this thread ran: kernel configuration, reduction
 * split and rasterisation group. */
void axonn_last_choice(int* config, int* split, int* group_m);

/* Workspace bytes an op needs with these flags (0 when none).  `op` is an
 * axonn_op_t.  With AXONN_VGRID | AXONN_VGRID_PARTIALS it is the fp32
 * partials 0..G-2 of the reduced grid axis ((G-1) * M * ceil8(N) * 4); the
 * other virtual-grid forms need none.  Without AXONN_VGRID it is nonzero
 * for products of more than one wave of 128x128 tiles, which may run a
 * stream-K tail (see axonn_set_streamk; up to about 80 MB on a 152-SM GPU);
 * the reduction split needs none.  Passing less workspace just disables
 * the tail.
 * Returns AXONN_ERR_INVALID_ARG for a bad shape or flag. */
axonn_status_t axonn_fc_workspace_size(int op, const axonn_fc_shape_t* shape, uint32_t flags,
                                       size_t* bytes);

/* Rows [*start, *stop) of block b when a dimension D is cut into G blocks by
 * the 8-element-unit rule above.  Host-only, no GPU needed. */
axonn_status_t axonn_block_range(int64_t D, int32_t G, int32_t b, int64_t* start, int64_t* stop);

/* Logical ranges of block (shape->x, shape->y, shape->z) of op `op` (an
 * axonn_op_t), as the product entry points resolve them: rows[2] = its
 * output rows, red[2] = its reduced range, cols[2] = its output columns,
 * each [start, stop) in the full matrices (forward: Tz, Kx, Ny; data
 * gradient: Tz, Ny, Kx; weight gradient: Kx, Tz, Ny -- the block products
 * of Figure 1 of the sciencestack.ai page under the reading T by G_z, K by
 * G_x, N by G_y).  AXONN_ERR_INVALID_ARG for a bad op, shape or
 * coordinate or a NULL output.  Host-only, no GPU needed. */
axonn_status_t axonn_fc_block_extents(int op, const axonn_fc_shape_t* shape, int64_t* rows,
                                      int64_t* red, int64_t* cols);

/* Waits for `stream`, then reports (and clears) a device-side timeout
 * recorded by any kernel of this library on the current device since the
 * last call: AXONN_ERR_TIMEOUT, AXONN_ERR_CUDA if the stream failed, else
 * AXONN_OK.  *detail (may be NULL) receives the raw error word. */
axonn_status_t axonn_sync_status(cudaStream_t stream, uint64_t* detail);

/* Upper bound, in nanoseconds, on any single wait inside the kernels
 * (default 4e9).  Process-wide; applies to launches made afterwards. */
void axonn_set_wait_timeout_ns(uint64_t ns);

/* Test hook: 1 makes the next launches' producer withhold all operand
 * loads (the GEMM kernels' tiles, the Goldfish loss's kept rows, the rows of a
 * distillation of many long ones), so the bounded waits expire and
 * AXONN_ERR_TIMEOUT is reported; 2 makes the latter two hold back the first
 * load of each CTA for two limits (2 s at most), so that it lands after the wait
 * for it has expired; 0 restores normal operation.  Never needed in production. */
void axonn_debug_set_inject(int mode);

/* Kernel configurations.  The library chooses one per call from the
 * problem's tile counts (the pages' automatic BLAS kernel tuning: review of
 * arXiv 2502.08145, "The reading"); these calls expose the choice.
 *   0  1cta_128x128      one CTA per 128x128 output tile, 64-deep stages
 *   1  1cta_128x256      one CTA per 128x256 output tile, 64-deep stages
 *   2  pair_256x256      a CTA pair (cluster of 2, cta_group::2 MMA) per
 *                        256x256 output tile, 64-deep stages
 *   3  1cta_256x256      one CTA per 256x256 output tile (two M=128 MMAs
 *                        per B slice), 3 stages, single-buffered TMEM
 *   4  1cta_128x192      one CTA per 128x192 output tile, 5 stages
 *   5  1cta_256x192      one CTA per 256x192 output tile, 4 stages
 *   6  pair_512x256      a CTA pair per 512x256 output tile (each CTA two
 *                        M=128 halves of 256 columns), 4 stages, 12 warps
 *   7  1cta_128x64       one CTA per 128x64 output tile, 8 stages (for
 *                        products with too few larger tiles)
 * (the N=192 tiles trade a little operand reuse for fewer idle SMs in the
 * last wave on shapes such as 8192 x 6144; configurations 0 and 7 also run
 * the reduction split inside a cluster)
 * axonn_set_kernel_config(c) forces configuration c for all later calls in
 * the process (-1 restores automatic choice); AXONN_ERR_INVALID_ARG if c is
 * out of range.  The products with an epilogue and those of the linear
 * cross-entropy have the tiles 0, 2, 6 and 7 and choose among them when
 * another is forced; while any is forced, their forms for one or two rows and
 * for a reduction cut over a cluster are not used.
 * axonn_last_kernel_config() is the configuration the last
 * GEMM launch on this thread used (-1 before any, and after a product with an
 * epilogue that ran without tiles, for one or two rows). */
axonn_status_t axonn_set_kernel_config(int config);
/* SM count of the current device and how many CTA pairs (clusters of 2
 * running configuration 2) it keeps resident at once. */
axonn_status_t axonn_device_info(int* sms, int* max_pairs);
int axonn_num_kernel_configs(void);

/* Stream-K tail for later calls in this process: -1 = as tuned, 0 = off,
 * 1 = on wherever it applies.  It applies to a single-product call that is
 * given the workspace axonn_fc_workspace_size reports and whose output
 * tiles do not fill a whole number of rounds of the persistent grid: the
 * last partial round plus one full round are cut into equal ranges of
 * 64-deep reduction steps, one per CTA (or CTA pair).  Untuned calls use it
 * only when the partial round is at most a quarter full; the tuner times
 * off, that default and always-on, and keeps the fastest.  Each such tile
 * is computed in at most two pieces; the second to finish adds the other's
 * fp32 partial (two terms, the same sum in either order), so results are
 * deterministic for a given shape and GPU but may differ in the last bit
 * from a call with it off.  No CTA waits for another, so concurrent
 * launches cannot stall each other.
 * Not part of the source pages: it removes the idle SMs of the last wave.
 * AXONN_ERR_INVALID_ARG for another mode.  Host-only. */
axonn_status_t axonn_set_streamk(int mode);

/* Operand roles for later calls in this process: -1 = as tuned (default
 * off), 0 = never exchanged, 1 = exchanged wherever it applies.  Exchanged,
 * a call computes the transpose of its product, C^T = B^T . A^T: the second
 * operand is read in the first operand's role (output rows) and the first
 * in the second's, and the epilogue writes each tile back transposed, so
 * the caller's output is the same matrix.  The tuner times the swap for the
 * two best configurations of each call, the row-major BLAS counterpart of
 * choosing among NN, NT and TN operand orders (the pages' automatic BLAS
 * kernel tuning: TL;DR of the sciencestack.ai page; review of arXiv
 * 2502.08145, "The reading").  It does not apply with AXONN_VGRID_PARTIALS.
 * Results may differ from the unswapped call in the
 * last bit (another tile order of the same fp32 sums).  Host-only;
 * AXONN_ERR_INVALID_ARG for another mode. */
axonn_status_t axonn_set_swap(int mode);

/* Programmatic dependent launch of the GEMM kernels (1, the default): each
 * launch may start while the previous kernel in the stream finishes, so its
 * barrier set-up, TMEM allocation and tensor-map prefetch overlap that
 * kernel's last tiles; it reads and writes global memory only after the
 * previous kernel has completed (griddepcontrol.wait), so stream order is
 * kept.  0 launches them plainly.  Process-wide, host-only;
 * AXONN_ERR_INVALID_ARG for another value. */
axonn_status_t axonn_set_pdl(int on);

/* L2 priorities of the GEMM operand loads.  A rasterisation group walks its
 * tile rows (or columns) across the whole product, so each later wave of
 * the group reads the group's panel of that operand again, while the other
 * operand's panels pass through once.  With a budget of `bytes` > 0 the
 * kept operand's loads mark their lines evict-last (the fraction
 * min(1, bytes / panel bytes) of them, panel = group x tile edge x
 * reduction x 2; createpolicy and the .L2::cache_hint form of the tensor
 * copies); the other operand's keep the default priority.  0 issues all
 * loads with the default priority.  Default 64 MiB.  Results are unchanged
 * either way.
 * Process-wide, host-only; AXONN_ERR_INVALID_ARG for a negative value. */
axonn_status_t axonn_set_l2_budget(int64_t bytes);
int64_t axonn_l2_budget(void);

/* 1 if the last call on this thread ran with exchanged operand roles. */
int axonn_last_swap(void);

/* Output tiles the last GEMM launch on this thread computed as stream-K
 * pieces (0: none).  Host-only. */
int axonn_last_streamk_tiles(void);
const char* axonn_kernel_config_name(int config);
int axonn_last_kernel_config(void);

/* Thread-local description of the last error returned on this thread. */
const char* axonn_last_error(void);

/* Library version string. */
const char* axonn_version(void);

#ifdef __cplusplus
}
#endif
#endif /* AXONN_FC_H_ */
