/*
 * vmscan: Vision Mamba bidirectional selective scan and VMamba SS2D cross-scan for MI355X
 * (gfx950).  C ABI: plain pointers and sizes; no C++ or framework types cross this boundary.
 *
 * Pages cited (short keys):
 *   [P1] "状态空间模型如何重塑视觉序列处理 Vision Mamba的技术突破与应用价值" (sumeiyu.com/news/203653),
 *        section "选择性扫描机制的计算效率优势": h_t = A h_{t-1} + B x_t, y_t = C h_t + D x_t.
 *   [P3] "Vision Mamba的双向SSM 计算机视觉模型架构的下一代突破" (aitangshan.cn/news/1404048),
 *        §2.1 (A/A_b, v1/v2 parameter sets), §2.2 (reverse, scan, reverse back; average fusion),
 *        §4.3 (v2 fast path: (out + out_b.flip) / 2).
 *   [P4] "VMamba的SS2D模块 状态空间模型在视觉领域的革新设计" (lpnh.cn/news/670717),
 *        §2.1 (y * act(z) after the core), §2.2 (four cross-scan orders), §3.1 (Δ = softplus of a
 *        projection; per-direction projections), §3.2 (A = -exp(A_log)).
 *   [P5] "Vision Mamba实战 双向SSM Encoder核心代码解析与实现" (lpnh.cn/news/710454),
 *        §1 table (A/A_b [d_inner, d_state], B/C [batch, d_state, seq_len], D/D_b [d_inner]),
 *        §2.2 (bidirectional scan = forward scan + reversed scan of the reversed input),
 *        §4 (delta = softplus(.)).
 *
 * Per direction and per (batch b, channel d) both entry points compute, in fp32:
 *   Δ_t   = softplus(Δ_raw[t] + delta_bias[d])                     [P4] §3.1, [P5] §4
 *   a_t,n = exp(Δ_t A_n),  A_n = -exp(A_log[d, n])                  [P4] §3.2 (zero-order hold)
 *   h_t,n = a_t,n h_{t-1},n + Δ_t B_t,n u_t,  h_{-1} = 0           [P1]
 *   y_t   = Σ_n C_t,n h_t,n + D[d] u_t                              [P1]
 *
 * Conventions shared by every entry point:
 *   - Ownership: every pointer is caller-owned DEVICE memory (except `stream`).  The library never
 *     allocates or frees memory.  Its only state is a thread-local last HIP error and, for
 *     vmscan_fwd_bidir_noalloc, the address of its fixed device scratch buffer on each device.
 *   - Layout: all tensors are dense, row-major, with the shapes stated per argument.  Every
 *     pointer must be 16-byte aligned (else VMSCAN_ERR_ALIGN).  `out` must not alias an input.
 *   - Activation dtype: VMSCAN_F32 (float) or VMSCAN_BF16 (bfloat16 bit patterns, 2 bytes) for
 *     u/x, delta_raw, z, B, C and out.  A_log, D and delta_bias are always float32.  The state
 *     and all arithmetic are float32; bf16 outputs are rounded to nearest even once, at the store.
 *   - d_state: every scan entry point, forward and backward, takes 16 or 32 (else
 *     VMSCAN_ERR_UNSUPPORTED; the workspace and chunk-length queries return 0).  The pages use
 *     16 and suggest a larger state for high-resolution inputs ([P3] §4.1; [P4] §4.2 gives the
 *     16-32 range).  The workspace size depends on d_state.
 *   - Errors: arguments are validated synchronously and a status is returned before anything is
 *     enqueued; on success the kernels are enqueued on `stream` (NULL = the default stream) and the
 *     call returns without waiting.  A failed launch returns VMSCAN_ERR_HIP and the hipError_t
 *     is kept for vmscan_last_hip_error().  No entry point throws or aborts.
 *   - Workspace: caller-provided device scratch of at least the queried size.  When the query
 *     returns 0 none is needed and `workspace` may be NULL (if given, it must still be 16-byte
 *     aligned).  Its contents on entry are ignored.
 *   - Wait status: the waves that hold different state parts of one direction wait for each other
 *     through LDS counters.  Every such wait ends by construction; it is also bounded, and a wait
 *     that runs out of its bound stores 1 into the first int32 of the workspace (the call's status
 *     word, which the call's first kernel sets to 0).  So after the call's kernels have finished,
 *     that word reads 0 unless the results are unspecified.  A library built with
 *     -DVMSCAN_CHECK_WAITS checks the word itself: each scan entry point then waits for its kernels
 *     and returns VMSCAN_ERR_WAIT if it is set.  (A stage-2-only call leaves the word of its stage 1.)
 */
#ifndef VMSCAN_H
#define VMSCAN_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  VMSCAN_OK = 0,
  VMSCAN_ERR_NULL = 1,        /* a required pointer is NULL                                  */
  VMSCAN_ERR_SHAPE = 2,       /* a size is < 1, or too large for the index types               */
  VMSCAN_ERR_UNSUPPORTED = 3, /* d_state, dtype or another option not supported                */
  VMSCAN_ERR_ALIGN = 4,       /* a pointer (a stride, where one is taken) is not 16-byte aligned */
  VMSCAN_ERR_WORKSPACE = 5,   /* workspace NULL or smaller than the queried size               */
  VMSCAN_ERR_HIP = 6,         /* a HIP call failed; see vmscan_last_hip_error()                */
  VMSCAN_ERR_SCRATCH = 7,     /* the call needs more than VMSCAN_SCRATCH_BYTES (no-alloc entry) */
  VMSCAN_ERR_WAIT = 8         /* a bounded wait gave up (builds with VMSCAN_CHECK_WAITS only)   */
} vmscan_status;

typedef enum { VMSCAN_F32 = 0, VMSCAN_BF16 = 1 } vmscan_dtype;

/* Human-readable name of a status (static string, never NULL). */
const char *vmscan_status_string(vmscan_status s);

/* hipError_t (as int) behind the last VMSCAN_ERR_HIP returned on the calling thread; 0 if none. */
int vmscan_last_hip_error(void);

/* Chunk length (tokens) the library uses for a bidirectional scan of this shape when
 * chunk_len = 0 is passed to the _ex entry points; a value >= seqlen means one chunk. */
/* chunk_len = VMSCAN_CHUNK_LANE_SCAN selects, for seqlen <= 8192, the scan that spreads each
 * sequence over the lanes instead of splitting it into chunks: one workgroup per (batch, channel),
 * a run of 16 positions per lane, and the state carried between lanes by an associative scan of
 * (decay, state) pairs within each 1024-position wave segment ([P4] §3.2, the parallel cumulative
 * form; [P3] §3, the selective-scan kernel's block scan), so no chunk end state is recomputed.
 * Same results as the other paths up to rounding order; its workspace is the status word only.
 * Longer sequences return VMSCAN_ERR_UNSUPPORTED. */
#define VMSCAN_CHUNK_LANE_SCAN (-1)
int64_t vmscan_fwd_bidir_chunk_len(int64_t batch, int64_t dim, int64_t seqlen, int d_state);

/* Workspace bytes for vmscan_fwd_bidir / vmscan_fwd_bidir_ex (chunk_len 0 = library choice).
 * Returns 0 for invalid arguments. */
size_t vmscan_fwd_bidir_workspace_bytes(int64_t batch, int64_t dim, int64_t seqlen, int d_state,
                                        vmscan_dtype dtype);
size_t vmscan_fwd_bidir_workspace_bytes_ex(int64_t batch, int64_t dim, int64_t seqlen, int d_state,
                                           vmscan_dtype dtype, int64_t chunk_len);

/*
 * Vision Mamba bidirectional (v2 scan inputs) selective scan, fused with the SiLU gate.
 *   out = ( y_f + flip(y_b') ) / 2 * silu(z)                       [P3] §2.2, §4.3; [P5] §2.2
 * where y_f is the scan above over t = 0..L-1 with (A_log, B, C, D) and y_b' is the same scan of
 * the reversed sequence (reversed u, Δ_raw) with (A_b_log, reversed B_b, reversed C_b, D_b).
 * The backward direction shares u, delta_raw, z and delta_bias with the forward one; B_b and C_b
 * are given in ORIGINAL token order.  No reversed copy is materialised.  The v1 variant of [P3]
 * §2.1 is obtained by passing B_b = B, C_b = C and D_b = D.
 *
 *   u, delta_raw, z : [batch, dim, seqlen]     activation dtype
 *   A_log, A_b_log  : [dim, d_state]           float32
 *   B, C, B_b, C_b  : [batch, d_state, seqlen] activation dtype, original token order
 *   D, D_b          : [dim]                    float32
 *   delta_bias      : [dim]                    float32 (shared by both directions)
 *   out             : [batch, dim, seqlen]     activation dtype
 * Long sequences are split into chunks whose boundary states are carried across workgroups
 * (chunk_len 0 = library choice; otherwise the given length, clamped to [1, min(seqlen, 206)]).
 * The workspace (size from vmscan_fwd_bidir_workspace_bytes[_ex]) holds a float32 copy of
 * B/C/B_b/C_b in position-major order and, for split sequences, the chunk end states.
 */
vmscan_status vmscan_fwd_bidir(const void *u, const void *delta_raw, const void *z,
                               const float *A_log, const float *A_b_log,
                               const void *B, const void *C, const void *B_b, const void *C_b,
                               const float *D, const float *D_b, const float *delta_bias,
                               void *out, int64_t batch, int64_t dim, int64_t seqlen, int d_state,
                               vmscan_dtype dtype, void *workspace, size_t workspace_bytes,
                               hipStream_t stream);
vmscan_status vmscan_fwd_bidir_ex(const void *u, const void *delta_raw, const void *z,
                                  const float *A_log, const float *A_b_log,
                                  const void *B, const void *C, const void *B_b, const void *C_b,
                                  const float *D, const float *D_b, const float *delta_bias,
                                  void *out, int64_t batch, int64_t dim, int64_t seqlen, int d_state,
                                  vmscan_dtype dtype, void *workspace, size_t workspace_bytes,
                                  int64_t chunk_len, hipStream_t stream);

/*
 * vmscan_fwd_bidir for callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation): the same computation, kernels and
 * results as vmscan_fwd_bidir (bit for bit), with the workspace taken from a fixed scratch
 * buffer of VMSCAN_SCRATCH_BYTES that the library holds in device memory (a file-scope device
 * array, one per GPU, loaded with the library's code object and kept until the process ends)
 * instead of a caller's workspace.  The caller still passes every input and the output, with
 * the layouts, validation and error codes of vmscan_fwd_bidir.  The call allocates nothing
 * (no hipMalloc/hipFree or allocating library routine); on its first call on a device it looks
 * up that device's copy of the buffer (hipGetSymbolAddress, with that device current).
 * A shape whose workspace (vmscan_fwd_bidir_workspace_bytes) exceeds VMSCAN_SCRATCH_BYTES
 * returns VMSCAN_ERR_SCRATCH before anything is enqueued; the other entry points take such shapes.
 * Every call on one GPU uses that GPU's one buffer: calls that overlap on one GPU (on different
 * streams or from different threads) race and give unspecified results; calls ordered on one
 * stream are safe.  The buffer keeps the last call's contents; the forward scan needs none of
 * them cleared.
 */
#define VMSCAN_SCRATCH_BYTES ((size_t)64 << 20)
vmscan_status vmscan_fwd_bidir_noalloc(const void *u, const void *delta_raw, const void *z,
                                       const float *A_log, const float *A_b_log,
                                       const void *B, const void *C, const void *B_b, const void *C_b,
                                       const float *D, const float *D_b, const float *delta_bias,
                                       void *out, int64_t batch, int64_t dim, int64_t seqlen,
                                       int d_state, vmscan_dtype dtype, hipStream_t stream);

/*
 * The two stages of vmscan_fwd_bidir_ex, for callers that time or overlap them separately:
 *   stage 1: preparation: the float32 position-major copy of B/C/B_b/C_b and, for a split
 *            sequence, each chunk's end state (scanned from zero) and Δ sum, in the workspace;
 *   stage 2: the fused bidirectional scan, which reads that copy and folds the carries into
 *            each chunk's initial state; it requires a completed stage 1 with the same inputs,
 *            shapes, chunk_len and workspace, else the output is unspecified;
 *   stage 3: both (= vmscan_fwd_bidir_ex).
 * Other stage values return VMSCAN_ERR_UNSUPPORTED.  Arguments as for vmscan_fwd_bidir_ex.
 */
vmscan_status vmscan_fwd_bidir_stage(const void *u, const void *delta_raw, const void *z,
                                     const float *A_log, const float *A_b_log,
                                     const void *B, const void *C, const void *B_b, const void *C_b,
                                     const float *D, const float *D_b, const float *delta_bias,
                                     void *out, int64_t batch, int64_t dim, int64_t seqlen,
                                     int d_state, vmscan_dtype dtype, void *workspace,
                                     size_t workspace_bytes, int64_t chunk_len, int stage,
                                     hipStream_t stream);

/*
 * The same bidirectional scan with a separate backward branch: in Vim's v2 parameter sets the
 * backward branch has its own convolution, input projection and Δ projection ([P3] §2.1), so
 * its scan input u_b, Δ input delta_raw_b and Δ bias delta_bias_b differ from the forward
 * branch's.  With y_f the scan of (u, delta_raw, delta_bias; A_log, B, C, D) and y_b' that of
 * the reversed (u_b, delta_raw_b; A_b_log, B_b, C_b, D_b) with delta_bias_b:
 *   out = ( y_f + flip(y_b') ) / 2 * silu(z)                       [P3] §2.2, §4.3
 *   u_b, delta_raw_b : [batch, dim, seqlen] activation dtype, ORIGINAL token order (the library
 *                      walks them backwards; no flipped copy is made)
 *   delta_bias_b     : [dim] float32
 * Any of u_b, delta_raw_b, delta_bias_b may alias the forward branch's tensor;
 * vmscan_fwd_bidir_stage(...) equals vmscan_fwd_bidir_v2_stage with u_b = u,
 * delta_raw_b = delta_raw and delta_bias_b = delta_bias.  All other arguments, the workspace
 * (same size query as vmscan_fwd_bidir_workspace_bytes[_ex]), chunk_len, stage, validation and
 * error codes are as for vmscan_fwd_bidir_ex / vmscan_fwd_bidir_stage; out must not alias any
 * input.
 */
vmscan_status vmscan_fwd_bidir_v2(const void *u, const void *delta_raw, const float *delta_bias,
                                  const void *u_b, const void *delta_raw_b, const float *delta_bias_b,
                                  const void *z, const float *A_log, const float *A_b_log,
                                  const void *B, const void *C, const void *B_b, const void *C_b,
                                  const float *D, const float *D_b, void *out,
                                  int64_t batch, int64_t dim, int64_t seqlen, int d_state,
                                  vmscan_dtype dtype, void *workspace, size_t workspace_bytes,
                                  int64_t chunk_len, hipStream_t stream);
vmscan_status vmscan_fwd_bidir_v2_stage(const void *u, const void *delta_raw, const float *delta_bias,
                                        const void *u_b, const void *delta_raw_b,
                                        const float *delta_bias_b, const void *z,
                                        const float *A_log, const float *A_b_log,
                                        const void *B, const void *C, const void *B_b, const void *C_b,
                                        const float *D, const float *D_b, void *out,
                                        int64_t batch, int64_t dim, int64_t seqlen, int d_state,
                                        vmscan_dtype dtype, void *workspace, size_t workspace_bytes,
                                        int64_t chunk_len, int stage, hipStream_t stream);

/*
 * Gradients of vmscan_fwd_bidir_v2 (the backward pass, for training).  The pages define the
 * forward and check its gradient numerically ([P5] §4 gradcheck); these are its exact
 * derivatives.  Given the forward's inputs and dout = dL/dout [batch, dim, seqlen]:
 *   du, ddelta_raw, du_b, ddelta_raw_b, dz   : [batch, dim, seqlen]  activation dtype
 *   dB, dC, dB_b, dC_b                       : [batch, 16, seqlen]   activation dtype
 *   dA_log, dA_b_log                         : [dim, 16]             float32
 *   dD, dD_b, ddelta_bias, ddelta_bias_b     : [dim]                 float32
 * Every gradient is written (not accumulated), summed over batch where the tensor has no batch
 * dimension, in float32 and rounded once.  du_b, ddelta_raw_b and ddelta_bias_b may each be
 * NULL: the backward branch's gradient for that input is then ADDED to the forward branch's
 * output (du, ddelta_raw, ddelta_bias), which is the gradient of vmscan_fwd_bidir, whose two
 * branches share u, delta_raw and delta_bias (pass the same tensor as u_b etc. then).
 * The library recomputes the forward: it runs the forward scan, which turns the un-gated sum into
 * dz and the scan's output gradient at once (the sum itself is not stored), and it stores the
 * state at window boundaries (in that scan when the sequence is not split, else in a second
 * forward pass per direction), then walks backwards over the sequence with the adjoint
 * recurrence, window by window from those states.  A long sequence with few (batch, channel-group) tiles
 * is split into chunks, the adjoint carry between them coming from a reverse carry pass; the
 * result does not depend on the split beyond float32 rounding order.  Workspace:
 * vmscan_bwd_bidir_v2_workspace_bytes.
 * Gradient outputs must not alias each other or any input.  Validation and error codes as for
 * vmscan_fwd_bidir_v2 (all pointers but the three optional ones are required, all 16-byte
 * aligned); launches are asynchronous on `stream`.  d_state 16 or 32 (B, C, dB, dC are then
 * [batch, d_state, seqlen]; A_log, dA_log [dim, d_state]).
 */
size_t vmscan_bwd_bidir_v2_workspace_bytes(int64_t batch, int64_t dim, int64_t seqlen, int d_state,
                                           vmscan_dtype dtype);
vmscan_status vmscan_bwd_bidir_v2(const void *u, const void *delta_raw, const float *delta_bias,
                                  const void *u_b, const void *delta_raw_b, const float *delta_bias_b,
                                  const void *z, const float *A_log, const float *A_b_log,
                                  const void *B, const void *C, const void *B_b, const void *C_b,
                                  const float *D, const float *D_b, const void *dout,
                                  void *du, void *ddelta_raw, float *ddelta_bias,
                                  void *du_b, void *ddelta_raw_b, float *ddelta_bias_b,
                                  void *dz, float *dA_log, float *dA_b_log,
                                  void *dB, void *dC, void *dB_b, void *dC_b, float *dD, float *dD_b,
                                  int64_t batch, int64_t dim, int64_t seqlen, int d_state,
                                  vmscan_dtype dtype, void *workspace, size_t workspace_bytes,
                                  hipStream_t stream);

/*
 * Gradients of ss2d_cross_scan_fwd (the SS2D backward pass).  Given the forward's inputs and
 * dout = dL/dout [batch, dim, H, W]:
 *   dx                 : [batch, dim, H, W]          activation dtype
 *   ddelta_raw         : [batch, 4, dim, H*W]        activation dtype, each direction's scan order
 *   dB, dC             : [batch, 4, N, H*W]          activation dtype, each direction's scan order
 *   dA_log             : [4, dim, N]                 float32  (N = d_state, 16 or 32)
 *   dD, ddelta_bias    : [4, dim]                    float32
 *   dz                 : [batch, dim, H, W]          activation dtype; NULL exactly when z is NULL
 * Every gradient is written (not accumulated), batch-summed where the tensor has no batch
 * dimension, in float32 and rounded once.  The gradient reaching direction k is dout silu(z)
 * (or dout) in that direction's scan order; each direction's adjoint is walked as in
 * vmscan_bwd_bidir_v2 and its du is mapped back to pixels and summed into dx.  With a gate the
 * library first recomputes the un-gated forward sum for dz.  Workspace:
 * ss2d_cross_scan_bwd_workspace_bytes.  Outputs must not alias each other or any input.
 * Validation and error codes as for ss2d_cross_scan_fwd (z and dz must both be given or both be
 * NULL, else VMSCAN_ERR_NULL); launches are asynchronous on `stream`.  d_state 16 or 32.
 */
size_t ss2d_cross_scan_bwd_workspace_bytes(int64_t batch, int64_t dim, int64_t H, int64_t W, int d_state,
                                           vmscan_dtype dtype);
vmscan_status ss2d_cross_scan_bwd(const void *x, const void *delta_raw, const float *A_log,
                                  const void *B, const void *C, const float *D, const float *delta_bias,
                                  const void *z, const void *dout, void *dx, void *ddelta_raw,
                                  float *dA_log, void *dB, void *dC, float *dD, float *ddelta_bias,
                                  void *dz, int64_t batch, int64_t dim, int64_t H, int64_t W,
                                  int d_state, vmscan_dtype dtype, void *workspace,
                                  size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes for ss2d_cross_scan_fwd / _ex (chunk_len 0 = library choice); 0 if invalid. */
size_t ss2d_cross_scan_workspace_bytes(int64_t batch, int64_t dim, int64_t H, int64_t W, int d_state,
                                       vmscan_dtype dtype);
size_t ss2d_cross_scan_workspace_bytes_ex(int64_t batch, int64_t dim, int64_t H, int64_t W,
                                          int d_state, vmscan_dtype dtype, int64_t chunk_len);

/*
 * VMamba SS2D cross-scan and cross-merge ([P4] §2.2, §3.1).  Direction k scans x in order
 *   k=0 row-major, k=1 column-major, k=2 reversed row-major, k=3 reversed column-major,
 * each with its own delta_raw[:,k], B[:,k], C[:,k] (stored in THAT direction's scan order),
 * A_log[k], D[k] and delta_bias[k], without a gate.  The four outputs are mapped back to
 * row-major pixels and summed in fp32:  out = Σ_k y_k  (times silu(z) when z is not NULL).
 *
 *   x          : [batch, dim, H, W]          activation dtype
 *   delta_raw  : [batch, 4, dim, H*W]        activation dtype, scan order of each direction
 *   A_log      : [4, dim, d_state]           float32
 *   B, C       : [batch, 4, d_state, H*W]    activation dtype, scan order of each direction
 *   D          : [4, dim]                    float32
 *   delta_bias : [4, dim]                    float32
 *   z          : [batch, dim, H, W] or NULL  activation dtype
 *   out        : [batch, dim, H, W]          activation dtype
 * H*W must be < 2^31.  Sequences are either cut into chunks of at most 206 positions (an LDS row),
 * whose entering states come from a chunk pass and a carry prefix, or walked whole, each pair's
 * two directions meeting in float32 rows in the workspace that a merge kernel then sums per
 * pixel.  The library walks whole when H*W > 206 and batch * ceil(dim / 64) >= 256 (enough
 * (batch, channel-group) tiles to fill the GPU without chunks); chunk_len >= H*W asks for the
 * whole walk, 0 < chunk_len < H*W for chunks of that length (at most 206).
 */
vmscan_status ss2d_cross_scan_fwd(const void *x, const void *delta_raw, const float *A_log,
                                  const void *B, const void *C, const float *D,
                                  const float *delta_bias, const void *z, void *out,
                                  int64_t batch, int64_t dim, int64_t H, int64_t W, int d_state,
                                  vmscan_dtype dtype, void *workspace, size_t workspace_bytes,
                                  hipStream_t stream);
vmscan_status ss2d_cross_scan_fwd_ex(const void *x, const void *delta_raw, const float *A_log,
                                     const void *B, const void *C, const float *D,
                                     const float *delta_bias, const void *z, void *out,
                                     int64_t batch, int64_t dim, int64_t H, int64_t W, int d_state,
                                     vmscan_dtype dtype, void *workspace, size_t workspace_bytes,
                                     int64_t chunk_len, hipStream_t stream);

/*
 * ss2d_cross_scan_fwd_ex with x's transposed copy supplied by the caller (for instance the xT_out
 * of ss2d_conv2d_silu_fwd): xT [batch, dim, W, H], activation dtype, must equal x transposed in
 * its last two dimensions; the column-major scans read it instead of a copy made here.  xT NULL
 * gives VMSCAN_ERR_NULL; the rest (arguments, workspace query, errors) as ss2d_cross_scan_fwd_ex.
 */
vmscan_status ss2d_cross_scan_fwd_xt(const void *x, const void *xT, const void *delta_raw,
                                     const float *A_log, const void *B, const void *C, const float *D,
                                     const float *delta_bias, const void *z, void *out,
                                     int64_t batch, int64_t dim, int64_t H, int64_t W, int d_state,
                                     vmscan_dtype dtype, void *workspace, size_t workspace_bytes,
                                     int64_t chunk_len, hipStream_t stream);

/*
 * Front of the Vim scan: the depthwise convolution + SiLU that produces the scan input u
 * ([P3] §2.1: each branch's Conv1d of width d_conv over the d_inner channels, v2's conv1d_b for
 * the backward branch; §2.2: the backward branch works on the flipped sequence).  Per
 * (batch b, channel d, position t), with K = d_conv:
 *   u[b,d,t]   = silu(conv_b[d]   + Σ_k conv_w[d,k]   x[b,d,t-(K-1)+k])      (causal)
 *   u_b[b,d,t] = silu(conv_b_b[d] + Σ_k conv_w_b[d,k] x[b,d,t+(K-1)-k])      (the flipped branch's
 *                causal convolution, stored in original token order as vmscan_fwd_bidir_v2's u_b)
 * with x = 0 outside [0, seqlen).  v1 (shared convolution): pass conv_w and conv_b again as
 * conv_w_b and conv_b_b.
 *   x, u, u_b            : [batch, dim, seqlen]   activation dtype
 *   conv_w, conv_w_b     : [dim, d_conv]          float32, d_conv in 1..4
 *   conv_b, conv_b_b     : [dim]                  float32
 * conv_w_b, conv_b_b and u_b are all NULL (forward branch only) or all set (else
 * VMSCAN_ERR_NULL).  x is read once; u and u_b are written once, rounded once.  Outputs must not
 * alias x.  No workspace.  Errors as for the other entry points.
 */
vmscan_status vmscan_conv1d_silu_fwd(const void *x, const float *conv_w, const float *conv_b,
                                     const float *conv_w_b, const float *conv_b_b, void *u, void *u_b,
                                     int64_t batch, int64_t dim, int64_t seqlen, int d_conv,
                                     vmscan_dtype dtype, hipStream_t stream);

/*
 * Front of SS2D: the depthwise 3 x 3 convolution ([P4] §2.1, d_conv = 3 in its table), optionally
 * followed by SiLU, written in the two layouts the cross-scan reads:
 *   pre[b,d,i,j] = conv_b[d] + Σ_{a,c} conv_w[d,a,c] x[b,d,i-1+a,j-1+c]   (zero padding)
 *   x_out[b,d,i,j] = xT_out[b,d,j,i] = act ? silu(pre) : pre
 *   x, x_out             : [batch, dim, H, W]     activation dtype
 *   xT_out               : [batch, dim, W, H]     activation dtype, or NULL (row-major only)
 *   conv_w               : [dim, 3, 3]            float32
 *   conv_b               : [dim]                  float32
 * d_conv must be 3 and act 0 or 1 (else VMSCAN_ERR_UNSUPPORTED).  x is read once, each output
 * written once; both hold the same rounded values.  Outputs must not alias x.  No workspace.
 */
vmscan_status ss2d_conv2d_silu_fwd(const void *x, const float *conv_w, const float *conv_b, int act,
                                   void *x_out, void *xT_out, int64_t batch, int64_t dim, int64_t H,
                                   int64_t W, int d_conv, vmscan_dtype dtype, hipStream_t stream);

/* ------------------------------------------------------------------------------------------------
 * Operators of a linear-attention block over the same tokens: the residual addition with its norm,
 * the rotary positions, and the attention whose state is a matrix per head.  Their activations are
 * token-major.  Ownership, errors, streams and the workspace follow the conventions above (no wait
 * status word: none of these kernels waits for another).
 */

/*
 * Root-mean-square norm with the residual's addition.  Per row, in float32:
 *   r = x + residual;   rstd = 1 / sqrt(mean(r^2) + eps);   y = r * rstd * weight
 *   x            : [rows, dim] with a row stride of x_stride >= dim elements, activation dtype
 *   residual     : [rows, dim] residual_dtype, or NULL (r = x; then residual_out is NULL too)
 *   weight       : [dim] float32
 *   y            : [rows, dim] activation dtype, or with out_fp8 = 1 8-bit codes (OCP e4m3)
 *   scale        : out_fp8 = 0: NULL.  out_fp8 = 1: float32, [rows] (group 0) or
 *                  [rows, ceil(dim / 128)] (group 128, the last group may be short)
 *   residual_out : [rows, dim] residual_dtype, r rounded once; NULL with residual.  May be residual.
 *   rstd         : [rows] float32, for the gradient, or NULL
 * y is computed from r before its rounding.  8 bits: y = code * scale, scale = max|y| / 448 over the
 * row or group (1 where that maximum is 0; at least the smallest normal float32), the code the value
 * nearest to y / scale.  A NaN in a row makes its rstd, scale and codes NaN.
 * dtype F32 takes residual_dtype F32; BF16 takes F32 or BF16.  1 <= dim <= 32768, any value.
 * No workspace.
 */
vmscan_status vmscan_rmsnorm_fwd(const void *x, int64_t x_stride, const void *residual,
                                 const float *weight, void *y, float *scale, void *residual_out,
                                 float *rstd, int64_t rows, int64_t dim, float eps,
                                 vmscan_dtype dtype, vmscan_dtype residual_dtype, int out_fp8,
                                 int group, hipStream_t stream);

/*
 * Gradient of vmscan_rmsnorm_fwd (activation output).  With n = r * rstd:
 *   dr = rstd * (weight * dy - n * mean(weight * dy * n)) + dresidual_out;   dweight = sum_rows dy * n
 *   dy             : [rows, dim] activation dtype
 *   r              : [rows, dim] residual_dtype: the forward's residual_out (x when it had no residual)
 *   rstd           : [rows] float32, the forward's
 *   dresidual_out  : [rows, dim] residual_dtype, the gradient of residual_out, or NULL
 *   dx             : [rows, dim] activation dtype: dr rounded
 *   dresidual      : [rows, dim] residual_dtype: dr rounded to that type, or NULL; must be NULL when the
 *                    two types are the same (dx is it)
 *   dweight        : [dim] float32, summed in a fixed order
 * Outputs must not alias inputs, except dx = dy and dresidual = dresidual_out.
 */
size_t vmscan_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t dim);
vmscan_status vmscan_rmsnorm_bwd(const void *dy, const void *r, const float *weight,
                                 const float *rstd, const void *dresidual_out, void *dx,
                                 void *dresidual, float *dweight, int64_t rows, int64_t dim,
                                 vmscan_dtype dtype, vmscan_dtype residual_dtype, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream);
/* The same for an r whose rows are r_stride >= dim elements apart: the forward's x, when that was so
 * and had no residual. */
vmscan_status vmscan_rmsnorm_bwd_ex(const void *dy, const void *r, int64_t r_stride, const float *weight,
                                    const float *rstd, const void *dresidual_out, void *dx,
                                    void *dresidual, float *dweight, int64_t rows, int64_t dim,
                                    vmscan_dtype dtype, vmscan_dtype residual_dtype, void *workspace,
                                    size_t workspace_bytes, hipStream_t stream);

/*
 * Rotary positions with several axes (rows and columns of an image; time, rows and columns of a
 * video).  Pair p of every head turns by the angle  positions[b, t, axis[p]] * inv_freq[p]:
 *   y1 = x1 cos - x2 sin,   y2 = x1 sin + x2 cos        (inverse = 1: by the negative angle, which is
 *                                                        also the gradient of the forward turn)
 * Pair p of the rot/2 pairs is the channels (p, p + rot/2), or with interleaved = 1 (2p, 2p + 1);
 * the channels from rot on pass through unchanged.
 *   q, q_out   : [batch, seqlen, heads, dim]  activation dtype; *_strides: batch, token and head
 *   k, k_out   : [batch, seqlen, kheads, dim]  stride in elements, channels contiguous.  kheads = 0:
 *                no k (its four arguments are not looked at).  An output may be its own input (same
 *                strides); otherwise they must not overlap.  Pointers: aligned to one element.  An
 *                output whose own elements overlap (a stride of 0, say) is refused (VMSCAN_ERR_SHAPE).
 *   positions  : [seqlen, axes] float32 per batch, positions_stride elements apart (0: shared)
 *   inv_freq   : [rot / 2] float32
 *   axis       : [rot / 2] int32; a pair whose axis is not in 0 .. axes - 1 is not turned
 * The angle is reduced from the exact product, so large positions lose nothing.  No workspace.
 */
vmscan_status vmscan_rope_axes(const void *q, const int64_t *q_strides, void *q_out,
                               const int64_t *q_out_strides, const void *k,
                               const int64_t *k_strides, void *k_out,
                               const int64_t *k_out_strides, const float *positions,
                               int64_t positions_stride, const float *inv_freq, const int32_t *axis,
                               int64_t batch, int64_t seqlen, int heads, int kheads, int dim,
                               int rot, int axes, int interleaved, int inverse,
                               vmscan_dtype dtype, hipStream_t stream);

/*
 * Linear attention with a decay for each head.  Per (batch b, head h), with hk = h / (heads / kheads)
 * and a float32 state S [dk, dv], S_{-1} = initial_state (NULL: 0):
 *   S_t = exp(log_decay[b, t, h]) S_{t-1} + k[b, t, hk] v[b, t, h]^T;   out[b, t, h] = scale S_t^T q[b, t, hk]
 *   q, k          : [batch, seqlen, kheads, dk]  activation dtype; *_strides: batch, token and head
 *   v             : [batch, seqlen, heads, dv]   stride in elements, channels contiguous.  Pointers
 *                   and strides must be multiples of 16 bytes (else VMSCAN_ERR_ALIGN),
 *                   token strides below 2^24 elements.
 *   log_decay     : float32; decay_strides (batch, token, head; 0 broadcasts) or NULL for one value
 *                   per head, [heads].  -inf clears the state; values above 0 are taken as they are.
 *   initial_state, final_state : [batch, heads, dk, dv] float32 or NULL; they may be one buffer, whose
 *                   states then go on in place, and must not overlap otherwise (VMSCAN_ERR_UNSUPPORTED)
 *   lengths       : [batch] int32 or NULL: row b has lengths[b] tokens (clamped to 0 .. seqlen).  What
 *                   lies past them is never read (it may be NaN), `out` is 0 there and the
 *                   final state is the one after the last token.
 *   out           : [batch, seqlen, heads, dv]   activation dtype, dense
 * heads must be a multiple of kheads; dk and dv multiples of 8 up to 128 (else
 * VMSCAN_ERR_UNSUPPORTED).  The masked scores are multiplied, as zeros, within a block (64 tokens; see
 * vmscan_linattn_plan), so a NaN or infinity in a token's v can reach the outputs of earlier tokens of its
 * block, but no others before it; one in its q, k or decay reaches no earlier output.
 */
/* How a call of vmscan_linattn_fwd (gradient 0) or _bwd (1) is cut up, which is the library's choice by sizes:
 * cut[0] tokens of a block, [1] value channels of a workgroup, [2] segments of a sequence, each walked by a
 * workgroup, [3] parts of a segment in the gradient's passes, [4] how the states of segments or parts are joined. */
enum { VMSCAN_JOIN_NONE = 0, VMSCAN_JOIN_WALK = 1, VMSCAN_JOIN_LAUNCH = 2 };
vmscan_status vmscan_linattn_plan(int64_t batch, int64_t seqlen, int heads, int dk, int dv,
                                  vmscan_dtype dtype, int gradient, int32_t *cut);

size_t vmscan_linattn_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int heads, int dk, int dv,
                                          vmscan_dtype dtype);
vmscan_status vmscan_linattn_fwd(const void *q, const int64_t *q_strides, const void *k,
                                 const int64_t *k_strides, const void *v, const int64_t *v_strides,
                                 const float *log_decay, const int64_t *decay_strides,
                                 const float *initial_state, const int32_t *lengths, void *out,
                                 float *final_state, int64_t batch, int64_t seqlen, int heads,
                                 int kheads, int dk, int dv, float scale, vmscan_dtype dtype,
                                 void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of vmscan_linattn_fwd.  Inputs as there, and
 *   dout           : [batch, seqlen, heads, dv]  activation dtype, dout_strides as q's
 *   dfinal_state   : [batch, heads, dk, dv] float32 or NULL (0)
 * Outputs, dense: dq, dk_out [batch, seqlen, kheads, dk] (summed over the heads that share them) and
 * dv_out [batch, seqlen, heads, dv], activation dtype; dlog_decay float32, [batch, seqlen, heads] or,
 * when decay_strides is NULL, [heads]; dinitial_state [batch, heads, dk, dv] float32 or NULL.  Zero
 * past a row's length.  No atomics: the same inputs give the same bits.  dinitial_state may be the buffer
 * of dfinal_state or of initial_state and must not overlap them otherwise (VMSCAN_ERR_UNSUPPORTED).  A NaN
 * or infinity in a token's k can reach dq of earlier tokens of its block, one in its q or dout dk and dv of
 * later ones, and those of other blocks where the formula has it.
 * per_head of the workspace query: 1 when decay_strides will be NULL.
 */
size_t vmscan_linattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int heads, int kheads,
                                          int dk, int dv, int per_head, vmscan_dtype dtype);
vmscan_status vmscan_linattn_bwd(const void *q, const int64_t *q_strides, const void *k,
                                 const int64_t *k_strides, const void *v, const int64_t *v_strides,
                                 const float *log_decay, const int64_t *decay_strides,
                                 const float *initial_state, const int32_t *lengths,
                                 const void *dout, const int64_t *dout_strides,
                                 const float *dfinal_state, void *dq, void *dk_out, void *dv_out,
                                 float *dlog_decay, float *dinitial_state, int64_t batch,
                                 int64_t seqlen, int heads, int kheads, int dk, int dv, float scale,
                                 vmscan_dtype dtype, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/*
 * One token of each of `batch` sequences: the recurrence of vmscan_linattn_fwd once, the states
 * updated in place.
 *   q, k      : [batch, kheads, dk], v : [batch, heads, dv]  activation dtype; *_strides: batch, head
 *   log_decay : float32, decay_strides (batch, head) or NULL for [heads]
 *   state     : [pool, heads, dk, dv] float32
 *   slots     : [batch] int32: the state of each sequence, all different; a row whose slot is not in
 *               0 .. pool - 1 has no state: its out is 0.  NULL: row b has state b, pool = batch.
 *   out       : [batch, heads, dv]  activation dtype, dense
 * q, k and v may start at any element.  No workspace.
 */
vmscan_status vmscan_linattn_step(const void *q, const int64_t *q_strides, const void *k,
                                  const int64_t *k_strides, const void *v, const int64_t *v_strides,
                                  const float *log_decay, const int64_t *decay_strides,
                                  float *state, const int32_t *slots, void *out, int64_t batch,
                                  int64_t pool, int heads, int kheads, int dk, int dv, float scale,
                                  vmscan_dtype dtype, hipStream_t stream);

/*
 * The operators below are those of a gated recurrence block over image tokens, for training that keeps its
 * activations in 8 bits: the 8-bit form itself, the group norm with its activation and the gated linear
 * recurrence.  Activations are token-major, [batch, seqlen, dim] (channels last); *_strides are batch and token
 * stride in elements, channels contiguous, and such inputs may start at any element.  Outputs are dense.
 * Ownership, errors, streams and the workspace follow the conventions above; only the recurrence over a sequence of
 * several chunks has a wait status word.
 */

/*
 * Activations in 8 bits: OCP e4m3 codes and a float32 scale for each 128 channels of a row (the last group may
 * be short): x ~ code * scale, scale = max|x| / 448 over the group (1 where that is 0; at least the smallest normal
 * float32), the code the value nearest to x / scale, ties to even, both quotients in float32: the 8-bit form of
 * vmscan_rmsnorm_fwd with group 128.  A NaN or an infinity makes its group's values NaN.  (Operators that leave this form
 * as or beside their output multiply by 1 / scale, and those that keep it by 1 / 448: a kept scale may differ by a unit in
 * the last place, a code where x / scale lies half-way between two.)
 *   x     : [rows, dim] activation dtype; pack: rows x_stride >= dim elements apart; unpack: dense
 *   codes : [rows, dim] bytes
 *   scale : [rows, ceil(dim / 128)] float32
 * 1 <= dim <= 2^30; rows * ceil(dim / 128) at most 2^28 - 16 (else VMSCAN_ERR_SHAPE).  No workspace.
 */
vmscan_status vmscan_act8_pack(const void *x, int64_t x_stride, void *codes, float *scale,
                               int64_t rows, int64_t dim, vmscan_dtype dtype, hipStream_t stream);
vmscan_status vmscan_act8_unpack(const void *codes, const float *scale, void *x, int64_t rows,
                                 int64_t dim, vmscan_dtype dtype, hipStream_t stream);

/*
 * Group norm with an optional activation.  Over the tokens and the dim / groups neighbouring channels of each
 * group of a batch row:
 *   mean, var = E[x], E[(x - mean)^2];   rstd = 1 / sqrt(var + eps)
 *   u = (x - mean) * rstd * weight + bias;   y = act ? u * sigmoid(u) : u
 *   x          : [batch, seqlen, dim] activation dtype, x_strides
 *   weight, bias : [dim] float32
 *   lengths    : [batch] int32 or NULL: row b has lengths[b] tokens (clamped to 0 .. seqlen).  What lies past
 *                them is never read, y is 0 there; a row without tokens has mean 0 and var 0.
 *   y          : [batch, seqlen, dim] activation dtype
 *   mean, rstd : [batch, groups] float32, for the gradient
 *   keep_codes, keep_scale : NULL, or x's 8-bit form (as vmscan_act8_pack; zeros past a row's length)
 * dim <= 4096 and a multiple of groups, batch < 65536 (else VMSCAN_ERR_SHAPE).  y must not alias x.  `keep` of the
 * workspace query: 1 when the 8-bit form will be kept.
 */
size_t vmscan_groupnorm_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim,
                                            int64_t groups, int keep);
vmscan_status vmscan_groupnorm_fwd(const void *x, const int64_t *x_strides, const float *weight,
                                   const float *bias, const int32_t *lengths, void *y, float *mean,
                                   float *rstd, void *keep_codes, float *keep_scale, int64_t batch,
                                   int64_t seqlen, int64_t dim, int64_t groups, float eps, int act,
                                   vmscan_dtype dtype, void *workspace, size_t workspace_bytes,
                                   hipStream_t stream);

/*
 * Gradient of vmscan_groupnorm_fwd.  With n = (x - mean) * rstd, u = n * weight + bias and
 * g = dy * (act ? sigmoid(u) (1 + u (1 - sigmoid(u))) : 1):
 *   dx = rstd * (weight g - E[weight g] - n E[weight g n])  (E over the group),  dweight = sum g n,  dbias = sum g
 *   dy            : [batch, seqlen, dim] activation dtype, dy_strides
 *   x, x_strides  : as in the forward; or NULL, and codes, codes_scale the 8-bit form that it kept
 *   mean, rstd    : the forward's
 *   dx            : [batch, seqlen, dim] activation dtype, 0 past a row's length
 *   dweight, dbias : [dim] float32, summed in a fixed order
 */
size_t vmscan_groupnorm_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim,
                                            int64_t groups);
vmscan_status vmscan_groupnorm_bwd(const void *dy, const int64_t *dy_strides, const void *x,
                                   const int64_t *x_strides, const void *codes,
                                   const float *codes_scale, const float *weight, const float *bias,
                                   const float *mean, const float *rstd, const int32_t *lengths,
                                   void *dx, float *dweight, float *dbias, int64_t batch,
                                   int64_t seqlen, int64_t dim, int64_t groups, int act,
                                   vmscan_dtype dtype, void *workspace, size_t workspace_bytes,
                                   hipStream_t stream);

/*
 * Gated linear recurrence with one state per channel.  Per (batch b, channel d), in float32:
 *   a_t = exp(A sigmoid(r_t)),  A = -exp(A_log[d]);   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t
 * from h_{-1} = initial_state (NULL: 0), over t = 0 .. n - 1, or with reverse = 1 from t = n - 1 down to 0.
 * (Rates exp(A_log[d]) over 2^125, infinite ones too, count as 2^125.)
 *   x, r, i    : [batch, seqlen, dim] activation dtype; the scan input and its two gates before their
 *                sigmoids; token strides below 2^24 elements
 *   A_log      : [dim] float32
 *   initial_state, final_state : [batch, dim] float32 or NULL; they may be one buffer, whose states then go on
 *                in place, and must not overlap otherwise (VMSCAN_ERR_UNSUPPORTED)
 *   lengths    : [batch] int32 or NULL: n = lengths[b] (clamped to 0 .. seqlen).  What lies past them is never
 *                read, `out` is 0 there and the final state is the one after the last token of the walk.
 *   out        : [batch, seqlen, dim] activation dtype: h
 *   keep_codes, keep_scale : NULL, or the 8-bit form (as vmscan_act8_pack) of what the gradient needs:
 *                [4, batch, seqlen, dim] and [4, batch, seqlen, ceil(dim / 128)], planes x, r, i and h (before
 *                its rounding to `out`), zeros past a row's length
 * A NaN or infinity reaches the later states of its own channel only (kept in 8 bits: that token's copies of its
 * 128 channels too), as either of the two.
 * A sequence is walked in chunks of 128 tokens (the gradient: of 64) by workgroups of their own; a chunk waits for what
 * those before it publish.  If there are several, the workspace's first int32 is the call's status word.
 * ceil(dim / 128) * batch * chunks must be below 2^23, seqlen below 2^30, dim below 2^20 (else VMSCAN_ERR_SHAPE).
 */
size_t vmscan_gated_scan_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim);
vmscan_status vmscan_gated_scan_fwd(const void *x, const int64_t *x_strides, const void *r,
                                    const int64_t *r_strides, const void *i,
                                    const int64_t *i_strides, const float *A_log,
                                    const float *initial_state, const int32_t *lengths, int reverse,
                                    void *out, float *final_state, void *keep_codes,
                                    float *keep_scale, int64_t batch, int64_t seqlen, int64_t dim,
                                    vmscan_dtype dtype, void *workspace, size_t workspace_bytes,
                                    hipStream_t stream);

/*
 * Gradients of vmscan_gated_scan_fwd.  x, r, i (and their strides) as there and h [batch, seqlen, dim] its `out`;
 * or these seven NULL, and codes, codes_scale what it kept in 8 bits.  And
 *   dout           : [batch, seqlen, dim] activation dtype, dout_strides
 *   dfinal_state   : [batch, dim] float32 or NULL (0)
 * Outputs: dx, dr, di [batch, seqlen, dim] activation dtype, 0 past a row's length; dA_log [dim] float32;
 * dinitial_state [batch, dim] float32 or NULL; it may be the buffer of dfinal_state, and must not overlap that
 * one otherwise, nor initial_state (VMSCAN_ERR_UNSUPPORTED).  At a_t = 1, where sqrt(1 - a^2) has no slope, the
 * gradient of r is its limit.  Sums and joins are in a fixed order: the same inputs give the same bits.
 */
size_t vmscan_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim);
vmscan_status vmscan_gated_scan_bwd(const void *x, const int64_t *x_strides, const void *r,
                                    const int64_t *r_strides, const void *i,
                                    const int64_t *i_strides, const void *h, const void *codes,
                                    const float *codes_scale, const float *A_log,
                                    const float *initial_state, const int32_t *lengths, int reverse,
                                    const void *dout, const int64_t *dout_strides,
                                    const float *dfinal_state, void *dx, void *dr, void *di,
                                    float *dA_log, float *dinitial_state, int64_t batch,
                                    int64_t seqlen, int64_t dim, vmscan_dtype dtype,
                                    void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One token of each of `batch` sequences: the recurrence once, the states updated in place.
 *   x, r, i : [batch, dim] activation dtype, rows *_stride elements apart
 *   state   : [pool, dim] float32
 *   slots   : [batch] int32: the state of each sequence, all different; a row whose slot is not in
 *             0 .. pool - 1 has no state: its out is 0.  NULL: row b has state b, pool = batch.
 *   out     : [batch, dim] activation dtype, dense
 * batch < 65536, dim < 2^20 (else VMSCAN_ERR_SHAPE).  No workspace.
 */
vmscan_status vmscan_gated_scan_step(const void *x, int64_t x_stride, const void *r,
                                     int64_t r_stride, const void *i, int64_t i_stride,
                                     const float *A_log, float *state, const int32_t *slots,
                                     void *out, int64_t batch, int64_t pool, int64_t dim,
                                     vmscan_dtype dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* VMSCAN_H */
