/*
 * libscan.h -- C ABI of libscan, the GB300 (sm_103a) associative affine scan.
 *
 * The library computes the first-order affine recurrence
 *
 *     h_t = A_t h_{t-1} + B_t
 *
 * forward and backward on one GPU, in three forms:
 *   - scalar, channel-wise: h[t] = a[t] * h[t-1] + x[t] over [B, C, T], with
 *     packed variable-length sequences (cu_seqlens), resets (a_t = 0), a
 *     nonzero initial state and two opposite-direction branches;
 *   - block matrix: A_t is k x k and B_t, h_t are k x v;
 *   - log space: the scalar recurrence carried as l_t = log h_t.
 *
 * Sources (page titles and sections of the pages that define the operation):
 *   [TSK]  "Triton scan kernels" (minGRU docs): One associative-scan family
 *          (the recurrence, its monoid and the four scan ops), Kernel design
 *          ((b, n) lanes, channel tiles, (k, v) blocks), The TF32 / IEEE
 *          precision guard (envelope k, v in {1, 2, 4, 8, 16}), Autograd
 *          integration and the reversed-scan backward.
 *   [AST]  "associative_scan_triton" README: quick start (scan_causal,
 *          scan_bidirectional_branched, cu_seqlens), how it works (chunked
 *          scan, no cross-document leakage, backward by a reverse scan on
 *          shifted gates with d_gates = shifted_states * d_tokens).
 *   [GDN]  "Operations & Triton Kernels" (HyMo): The chunked GDN algorithm;
 *          Mathematical Derivation of the Reverse-Time Backward Pass.
 *   [RGA]  "Our RG-LRU GPU audit": Strengthened fused path (resets, nonzero
 *          initial state and its gradient, partial final chunks), Exact real
 *          chunk algebra (h_out = P h_in + Q).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers to contiguous row-major arrays;
 *     scalars are passed by value. The caller owns every buffer. The library
 *     never allocates device memory and never synchronises the stream except
 *     in scan_get_device_status().
 *   - Every call is asynchronous on `stream`; it returns after validating its
 *     arguments on the host and enqueueing its kernel(s). No exception crosses
 *     the ABI and there is no fallback: an input outside what the kernels
 *     support returns an error status and computes nothing.
 *   - Time index t is 0-based and h_{-1} = h0 (zero when h0 is NULL).
 *   - Accumulation is always fp32. `a`, `x`, `da`, `dx` may be fp32 or bf16
 *     (scan_dtype); h, h0, dh, dh0 are always fp32 ([TSK] Kernel design:
 *     "Accumulation is fp32 regardless of input dtype").
 *   - Dense layout: a, x, h, dh, da, dx are [B, C, T]; h0, dh0 are [B, C].
 *     Packed layout (cu_seqlens != NULL): B must be 1, tensors are [C, T]
 *     with T the total packed length, cu_seqlens is a device int32 array of
 *     n_seqs + 1 non-decreasing offsets from 0 to T ([AST] quick start,
 *     flash-attn convention), h0/dh0 are [n_seqs, C]. Empty sequences are
 *     allowed; their dh0 rows are written as 0.
 *   - A reset is simply a_t = 0: it erases the prefix ([RGA] Exact real chunk
 *     algebra). No separate reset mask exists.
 *   - Workspace: a device buffer of scan_workspace_bytes() bytes that the
 *     caller allocates once and zeroes once with scan_workspace_init(). After
 *     that it may be reused by any number of calls on one stream without
 *     clearing; calls that run concurrently on the GPU need separate
 *     workspaces. It also holds the sticky device status word read by
 *     scan_get_device_status().
 *   - Scalar and log forms accept any base pointer; 16-byte aligned fp32
 *     tensors and 8-byte aligned bf16 tensors (torch allocations are) take
 *     the vectorised path. The block form needs 16-byte aligned tensors.
 */
#ifndef LIBSCAN_H
#define LIBSCAN_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LIBSCAN_VERSION 1

typedef enum scan_status {
  SCAN_OK = 0,
  SCAN_ERR_INVALID_ARG = 1, /* null pointer, negative size, bad enum, malformed host cu_seqlens */
  SCAN_ERR_UNSUPPORTED = 2, /* outside the kernels' envelope (e.g. k, v not in {1,2,4,8,16}) */
  SCAN_ERR_ALIGNMENT = 3,   /* affine tensors must be 16-byte aligned */
  SCAN_ERR_WORKSPACE = 4,   /* workspace missing or smaller than scan_workspace_bytes() */
  SCAN_ERR_CUDA = 5,        /* a CUDA runtime call or launch failed */
  SCAN_ERR_TIMEOUT = 6,     /* device: a look-back wait ran past opts.wait_limit_s */
  SCAN_ERR_SEQLENS = 7      /* device: cu_seqlens not 0 = cu[0] <= ... <= cu[n] = T */
} scan_status;

typedef enum scan_dtype {
  SCAN_F32 = 0,
  SCAN_BF16 = 1
} scan_dtype;

/* How T is split across thread blocks. STATIONARY: a block walks a row
 * group in order with the running state in registers ([TSK] Kernel design;
 * [RGA] state-stationary serial path); long rows may be cut into a few
 * segments, each block waiting once for the end state of the previous
 * segment. LOOKBACK: T is cut into chunks handled by independent blocks; each
 * block publishes its chunk summary (P, Q) ([RGA] Exact real chunk algebra)
 * and reads its predecessors' summaries (decoupled look-back). STREAM: a
 * persistent grid sized by occupancy; each warp walks a contiguous share of
 * whole rows with the running state in registers, its chunks arriving in a
 * ring of shared-memory stages by 2-D tensor copies (TMA) several chunks
 * ahead, and leaving through tensor stores; needs every tensor 16-byte
 * aligned and at least 64 elements (else it runs as STATIONARY). AUTO picks
 * per shape. */
typedef enum scan_variant {
  SCAN_VARIANT_AUTO = 0,
  SCAN_VARIANT_STATIONARY = 1,
  SCAN_VARIANT_LOOKBACK = 2,
  SCAN_VARIANT_STREAM = 3
} scan_variant;

typedef enum scan_op {
  SCAN_OP_FWD = 0,
  SCAN_OP_BWD = 1,
  SCAN_OP_BIDIR_FWD = 2,
  SCAN_OP_BIDIR_BWD = 3,
  SCAN_OP_LOG_FWD = 4,
  SCAN_OP_AFFINE_FWD = 5,
  SCAN_OP_AFFINE_BWD = 6,
  SCAN_OP_LOG_BWD = 7
} scan_op;

/* Optional tuning and test controls; pass NULL for the defaults (all zero). */
typedef struct scan_opts {
  int32_t variant;       /* scan_variant; 0 = AUTO */
  int32_t chunk;         /* scalar/log: elements of T per block row, one of 128, 256, 512;
                            affine: time steps per block, one of 64, 128, 256; 0 = planner */
  int32_t rows_per_cta;  /* scalar/log: rows (channels) per block, 1..8 (blocks of 32 x
                            rows_per_cta threads); 0 = planner */
  int32_t test_stall;    /* test hook: 1 makes one look-back wait on a summary that is
                            never published, so the wait limit expires (SCAN_ERR_TIMEOUT) */
  double wait_limit_s;   /* bound on every look-back wait; <= 0 means 1.0 second */
  const int32_t* cu_seqlens_host; /* optional host copy of cu_seqlens, validated before launch */
  int32_t segments;      /* stationary: segments each row is cut into (>= 1); 0 = planner */
  int32_t stages;        /* stream: chunks in flight per warp, 2..16; 0 = planner */
} scan_opts;

/* Human-readable name of a status code (static string, never NULL). */
const char* scan_status_string(scan_status status);

/* LIBSCAN_VERSION of the loaded library. */
int32_t scan_version(void);

/* Bytes of workspace a call of `op` with these sizes needs under `opts`
 * (NULL = defaults). Scalar/log ops: (B, C, T) as in the call, k = v = 0.
 * Affine ops: B = batch, C = N (state blocks), T = time, and k, v.
 * Returns 0 for arguments the call itself would reject. */
size_t scan_workspace_bytes(scan_op op, int64_t B, int64_t C, int64_t T,
                            int32_t k, int32_t v, const scan_opts* opts);

/* Zero a freshly allocated workspace (asynchronous on `stream`). */
scan_status scan_workspace_init(void* workspace, size_t workspace_bytes,
                                cudaStream_t stream);

/* Synchronise `stream`, read the workspace's sticky device status
 * (SCAN_ERR_TIMEOUT, SCAN_ERR_SEQLENS or SCAN_OK), reset it to SCAN_OK and
 * return it. */
scan_status scan_get_device_status(void* workspace, cudaStream_t stream);

/* Scalar forward ([AST] quick start, scan_causal; [TSK] linear_scan):
 *   reverse == 0: h_t = a_t h_{t-1} + x_t, h_{-1} = h0;
 *   reverse != 0: h_t = a_t h_{t+1} + x_t, h_T = h0 (per row or sequence).
 * a, x: [B,C,T] or packed [C,T] of `dt`; h0: nullable fp32 [B,C] or
 * [n_seqs,C]; h: fp32 output. */
scan_status scan_fwd(const void* a, const void* x, const float* h0,
                     const int32_t* cu_seqlens, int32_t n_seqs, float* h,
                     int64_t B, int64_t C, int64_t T, scan_dtype dt,
                     int32_t reverse, const scan_opts* opts, void* workspace,
                     size_t workspace_bytes, cudaStream_t stream);

/* Scalar backward of L = sum_t <dh_t, h_t> ([AST] how it works: d_tokens by a
 * reverse scan on shifted gates, d_gates = shifted_states * d_tokens):
 *   g_t = dh_t + a_{t+1} g_{t+1} (a_{t+1} = 0 past the sequence end),
 *   dx_t = g_t, da_t = g_t h_{t-1} (h_{-1} = h0), dh0 = a_0 g_0
 * (mirrored when reverse != 0). `h` is the forward output, used as the
 * shifted state so no forward state is recomputed or stored ([TSK]
 * Autograd integration: the backward reads only the forward's inputs and
 * outputs). h0 is needed for da at a sequence start (nullable = 0). da, dx
 * have dtype `dt`; dh0 is a nullable fp32 output. */
scan_status scan_bwd(const void* a, const float* h, const float* dh,
                     const float* h0, const int32_t* cu_seqlens, int32_t n_seqs,
                     void* da, void* dx, float* dh0, int64_t B, int64_t C,
                     int64_t T, scan_dtype dt, int32_t reverse,
                     const scan_opts* opts, void* workspace,
                     size_t workspace_bytes, cudaStream_t stream);

/* Two independent branches in one launch ([AST] quick start,
 * scan_bidirectional_branched): branch f is causal over (af, xf), branch r
 * runs from each sequence's end over (ar, xr). Same result as scan_fwd with
 * reverse = 0 and reverse = 1; the outputs are separate, not summed. */
scan_status scan_bidir_fwd(const void* af, const void* xf, const void* ar,
                           const void* xr, const float* h0f, const float* h0r,
                           const int32_t* cu_seqlens, int32_t n_seqs,
                           float* hf, float* hr, int64_t B, int64_t C,
                           int64_t T, scan_dtype dt, const scan_opts* opts,
                           void* workspace, size_t workspace_bytes,
                           cudaStream_t stream);

/* Backward of both branches in one launch; equal to scan_bwd with
 * reverse = 0 on branch f and reverse = 1 on branch r. */
scan_status scan_bidir_bwd(const void* af, const float* hf, const float* dhf,
                           const float* h0f, const void* ar, const float* hr,
                           const float* dhr, const float* h0r,
                           const int32_t* cu_seqlens, int32_t n_seqs,
                           void* daf, void* dxf, float* dh0f, void* dar,
                           void* dxr, float* dh0r, int64_t B, int64_t C,
                           int64_t T, scan_dtype dt, const scan_opts* opts,
                           void* workspace, size_t workspace_bytes,
                           cudaStream_t stream);

/* Log-space forward ([TSK] One associative-scan family, parallel_scan_log):
 *   l_t = log(exp(l_{t-1} + log_a_t) + exp(log_x_t)), l_{-1} = log_h0
 *   (-inf when log_h0 is NULL), output h_t = exp(l_t) in linear space.
 * log_a may be -inf (a reset). All fp32; layouts as scan_fwd. */
scan_status scan_log_fwd(const float* log_a, const float* log_x,
                         const float* log_h0, const int32_t* cu_seqlens,
                         int32_t n_seqs, float* h, int64_t B, int64_t C,
                         int64_t T, int32_t reverse, const scan_opts* opts,
                         void* workspace, size_t workspace_bytes,
                         cudaStream_t stream);

/* Log-space backward of L = sum_t dh_t h_t with h = scan_log_fwd(...). The
 * adjoint is the linear one on a = exp(log_a), x = exp(log_x)
 * ([TSK] One associative-scan family; the chain rule through exp):
 *   g_t = dh_t + a_{t+1} g_{t+1} (a_{t+1} = 0 past a sequence end),
 *   dlog_x_t = g_t x_t, dlog_a_t = g_t a_t h_{t-1} (h_{-1} = exp(log_h0)),
 *   dlog_h0 = a_0 g_0 exp(log_h0) per row or sequence (0 without log_h0).
 * reverse mirrors the shifts as scan_bwd does. Inputs: log_a, log_x as given
 * to scan_log_fwd, h its output, dh fp32; all outputs fp32 in the same
 * layouts; dlog_h0 nullable. Runs STATIONARY or LOOKBACK (a STREAM request
 * runs STATIONARY). */
scan_status scan_log_bwd(const float* log_a, const float* log_x, const float* h,
                         const float* dh, const float* log_h0,
                         const int32_t* cu_seqlens, int32_t n_seqs,
                         float* dlog_a, float* dlog_x, float* dlog_h0, int64_t B,
                         int64_t C, int64_t T, int32_t reverse,
                         const scan_opts* opts, void* workspace,
                         size_t workspace_bytes, cudaStream_t stream);

/* Block-matrix forward ([TSK] One associative-scan family, matrix_affine_scan;
 * Kernel design): H_t = A_t H_{t-1} + B_t per (b, n) lane, H_{-1} = h0.
 * A: [B,T,N,k,k], Bm and H: [B,T,N,k,v], h0: nullable [B,N,k,v]; row-major
 * matrices; fp32, 16-byte aligned (else SCAN_ERR_ALIGNMENT). Supported
 * (k, v): k and v each in {1, 2, 4, 8, 16} ([TSK] Conformance envelope);
 * others return SCAN_ERR_UNSUPPORTED. (4, 4) and (2, 2) run a kernel that
 * keeps whole blocks in registers, every other shape one that streams A. */
scan_status affine_scan_fwd(const float* A, const float* Bm, const float* h0,
                            float* H, int64_t B, int64_t T, int64_t N,
                            int32_t k, int32_t v, const scan_opts* opts,
                            void* workspace, size_t workspace_bytes,
                            cudaStream_t stream);

/* Block-matrix backward of L = sum_t <dH_t, H_t> ([TSK] Autograd integration
 * and the reversed-scan backward): G_t = dH_t + A_{t+1}^T G_{t+1},
 * dB_t = G_t, dA_t = G_t H_{t-1}^T (H_{-1} = h0), dh0 = A_0^T G_0.
 * H is the forward output; dh0 is nullable. Same envelope as the forward. */
scan_status affine_scan_bwd(const float* A, const float* H, const float* dH,
                            const float* h0, float* dA, float* dB, float* dh0,
                            int64_t B, int64_t T, int64_t N, int32_t k,
                            int32_t v, const scan_opts* opts, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream);

/* Coefficient prefix of the block scan ([TSK] One associative-scan family:
 * matrix_affine_scan composes the pairs (A, B) and returns the composed
 * coefficient as well): Abar_t = A_t A_{t-1} ... A_0 per (b, n) lane, i.e. the
 * block scan with v = k, B_t = 0 and h0 = I. A, Abar: [B,T,N,k,k] fp32,
 * 16-byte aligned; k in {1, 2, 4, 8, 16}; workspace as affine_scan_fwd with
 * v = k. */
scan_status affine_prefix_fwd(const float* A, float* Abar, int64_t B, int64_t T,
                              int64_t N, int32_t k, const scan_opts* opts,
                              void* workspace, size_t workspace_bytes,
                              cudaStream_t stream);

/* Backward of L = sum_t <dAbar_t, Abar_t>: G_t = dAbar_t + A_{t+1}^T G_{t+1},
 * dA_t = G_t Abar_{t-1}^T (Abar_{-1} = I). Abar is affine_prefix_fwd's output.
 * accumulate != 0 adds into dA (so a dA already written by affine_scan_bwd
 * receives both gradient terms); otherwise dA is overwritten. */
scan_status affine_prefix_bwd(const float* A, const float* Abar,
                              const float* dAbar, float* dA, int32_t accumulate,
                              int64_t B, int64_t T, int64_t N, int32_t k,
                              const scan_opts* opts, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream);

/* Scalar-gated outer-product state ([GDN] The chunked GDN algorithm), per
 * (batch, head):  h_t = alpha_t h_{t-1} + b_t v_t^T (S x D),  h_{-1} = h0,
 *                 o_t = h_t^T c_t (a D-vector).
 * Layouts (fp32, T-major within a head): alpha [B,H,T]; b, c [B,H,T,S];
 * v, o [B,H,T,D]; h0 nullable [B,H,S,D] (0 when NULL). S, D in {16, 32}
 * (else SCAN_ERR_UNSUPPORTED); b, c, v, o, h0, ckpt 16-byte aligned (else
 * SCAN_ERR_ALIGNMENT). ckpt (nullable): gdn_checkpoint_bytes() bytes, filled
 * with the state before every 32nd step, [B,H,ceil(T/32),S,D]; the backward
 * starts from it. Computed in 64-step chunks run in parallel, from the state
 * between chunks carried by a short serial pass per head.
 * workspace: gdn_workspace_bytes() bytes of device memory, 16-byte aligned,
 * owned by the caller (else SCAN_ERR_WORKSPACE); no state is kept in it
 * between calls. Asynchronous on `stream`. */
size_t gdn_checkpoint_bytes(int64_t B, int64_t H, int64_t T, int64_t S,
                            int64_t D);
size_t gdn_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t S,
                           int64_t D);
scan_status gdn_fwd(const float* alpha, const float* b, const float* v,
                    const float* c, const float* h0, float* o, float* ckpt,
                    int64_t B, int64_t H, int64_t T, int64_t S, int64_t D,
                    void* workspace, size_t workspace_bytes,
                    cudaStream_t stream);

/* Its backward for L = sum_t <dout_t, o_t> ([GDN] Mathematical Derivation of
 * the Reverse-Time Backward Pass, with alpha itself as the gate input):
 *   dh_t = c_t dout_t^T + alpha_{t+1} dh_{t+1},   dc_t = h_t dout_t,
 *   dv_t = dh_t^T b_t,  db_t = dh_t v_t,  dalpha_t = <dh_t, h_{t-1}>,
 *   dh0 = alpha_0 dh_0 (nullable).
 * Computed chunk by chunk over T ([GDN] The chunked GDN algorithm): within a
 * 32-step chunk the products above become small matrix products; only the
 * adjoint of the state between chunks runs serially. ckpt is the forward's
 * checkpoint buffer (for the same inputs and h0); no state is stored besides
 * it. workspace: as for gdn_fwd. Outputs in the layouts of the corresponding
 * inputs. */
scan_status gdn_bwd(const float* alpha, const float* b, const float* v,
                    const float* c, const float* ckpt, const float* dout,
                    float* dalpha, float* db, float* dv, float* dc, float* dh0,
                    int64_t B, int64_t H, int64_t T, int64_t S, int64_t D,
                    void* workspace, size_t workspace_bytes,
                    cudaStream_t stream);

/* RG-LRU gate preparation fused in front of the scalar scan ("Our RG-LRU GPU
 * audit", Strengthened fused path: the recurrent input, two gate logits,
 * a_param, optional segment_pos and initial state, with the gate activations,
 * log_a, transition, square-root multiplier and write formed in registers and
 * never stored; Exact real chunk algebra: a reset is a_t = 0 with the
 * canonical write). The gate formulas are the method's own (the pages name
 * these tensors but do not print them):
 *   r_t = sigmoid(gate_a_t), i_t = sigmoid(gate_x_t),
 *   log_a_t = 8 r_t log(sigmoid(a_param[c])), a_t = exp(log_a_t),
 *   write_t = sqrt(1 - a_t^2) i_t x_t;
 *   where segment_pos[b, t] == 0 (a reset): a_t = 0, write_t = i_t x_t;
 *   h_t = a_t h_{t-1} + write_t, h_{-1} = h0 (zero when h0 is NULL).
 *   x, gate_a, gate_x: [B, C, T] of dtype dt (SCAN_F32, or SCAN_BF16: the
 *     page's BF16 boundaries, read into fp32 registers), T contiguous (the
 *     scalar scan's dense layout); h: fp32 [B, C, T] (the state is carried in
 *     fp32 either way); a_param: fp32 [C]; segment_pos: int32 [B, T], shared
 *     by the channels of a batch row, or NULL (no resets); h0: fp32 [B, C] or
 *     NULL. All device pointers; any alignment (rows of T % 4 == 0 elements
 *     from pointers aligned to four elements take the vector path).
 * Returns SCAN_ERR_INVALID_ARG for negative sizes, a bad dtype or a NULL
 * required pointer,
 * SCAN_ERR_UNSUPPORTED for C > 2^31 - 1, SCAN_ERR_CUDA if the launch fails.
 * Asynchronous on `stream`; no workspace, no allocation. */
scan_status rglru_fwd(const void* x, const void* gate_a, const void* gate_x,
                      const float* a_param, const int32_t* segment_pos, const float* h0,
                      float* h, int64_t B, int64_t C, int64_t T, scan_dtype dt,
                      cudaStream_t stream);

/* Its backward for L = sum_t dh_t h_t, recomputing the gate terms from the
 * logits (the same page: backward recomputation of the pointwise terms, the
 * clipped square-root backward, partial a_param gradients followed by a
 * reduction): the adjoint g_t = dh_t + a_{t+1} g_{t+1} (a_T = 0), then
 *   dx_t = g_t m_t i_t, dgate_x_t = g_t m_t x_t i_t (1 - i_t)   (m = sqrt(1 - a^2)),
 *   dL/da_t = g_t h_{t-1} + g_t i_t x_t (d sqrt(u)/du) (-2 a_t), u = 1 - a_t^2,
 *     with d sqrt(u)/du taken at max(u, 1e-6) (the clip),
 *   dgate_a_t = a_t dL/da_t 8 log(sigmoid(a_param)) r_t (1 - r_t),
 *   da_param[c] = sigmoid(-a_param[c]) sum_{b,t} a_t dL/da_t 8 r_t,
 *   dh0 = a_0 g_0; a reset step has dgate_a = 0 and m = 1.
 *   h: the forward's output for the same inputs; dh: fp32 [B, C, T];
 *   dx, dgate_a, dgate_x: [B, C, T] of dtype dt (bf16 rounded to nearest from
 *   the fp32 results); da_param: fp32 [C], written (not
 *   accumulated), summed over b and t in a fixed order; dh0: [B, C] or NULL.
 * Errors as for rglru_fwd. Asynchronous on `stream`; no workspace. */
scan_status rglru_bwd(const void* x, const void* gate_a, const void* gate_x,
                      const float* a_param, const int32_t* segment_pos, const float* h0,
                      const float* h, const float* dh, void* dx, void* dgate_a,
                      void* dgate_x, float* da_param, float* dh0, int64_t B, int64_t C,
                      int64_t T, scan_dtype dt, cudaStream_t stream);

/* One training step of dense rows (scan_fwd then scan_bwd, reverse = 0) whose
 * inputs and results are in host memory ([AST] the scan and its reversed-scan
 * backward; the rows of [B,C,T] are independent, so cutting between rows is
 * exact). The B*C rows are cut into `pieces` pieces (0: 8; at most 64): each
 * piece's inputs are copied to the device buffers on one internal stream, the
 * piece is scanned forward and backward on `stream`, and its results are copied
 * back on a second internal stream, so the copies of neighbouring pieces run
 * under the scans and both copy directions run together. Results equal those
 * of scan_fwd and scan_bwd on the whole problem with the same variant, bit for
 * bit when T is a multiple of 4; otherwise a piece's rows start at another
 * 4-element memory phase, which moves the kernels' run boundaries and so the
 * rounding (within the forms' usual tolerance).
 * host: a, x (dt), dh [B,C,T] and h0 [B,C] (nullable) in; h [B,C,T] fp32, da,
 *       dx (dt) and dh0 [B,C] (nullable, with h0 and the device's h0/dh0 on
 *       the same footing) out. Page-locked host memory is needed for the
 *       copies to overlap (pageable memory works, without overlap).
 * dev:  device buffers of the same shapes, owned by the caller; their
 *       contents are overwritten.
 * Host and device pointers must all be given except h0/dh0 (else
 * SCAN_ERR_INVALID_ARG). opts: as for scan_fwd, except that the variant
 * defaults to SCAN_VARIANT_STATIONARY (a piece has fewer rows than the GPU has
 * warp slots). workspace: scan_workspace_bytes(SCAN_OP_BWD, 1, C', T, ...) for
 * the largest piece of C' = ceil(B*C / pieces) rows, shared by the pieces'
 * scans (they run in order on `stream`). The options and shape of the
 * largest piece (SCAN_ERR_INVALID_ARG / SCAN_ERR_UNSUPPORTED) and the
 * workspace (missing, not 16-byte aligned or too small: SCAN_ERR_WORKSPACE)
 * are checked before anything is queued; a CUDA error after that returns
 * SCAN_ERR_CUDA with `stream` made to wait for the copies already queued.
 * Asynchronous: on return the whole step is queued and `stream` waits for its
 * last copy; calls on one device are serialised on the host. */
typedef struct {
  const void* a;
  const void* x;
  const float* h0;
  const float* dh;
  float* h;
  void* da;
  void* dx;
  float* dh0;
} scan_host_io;
typedef struct {
  void* a;
  void* x;
  float* h0;
  float* dh;
  float* h;
  void* da;
  void* dx;
  float* dh0;
} scan_device_io;
scan_status scan_step_host(const scan_host_io* host, const scan_device_io* dev,
                           int64_t B, int64_t C, int64_t T, scan_dtype dt,
                           int32_t pieces, const scan_opts* opts,
                           void* workspace, size_t workspace_bytes,
                           cudaStream_t stream);

/* scan_copy modes. */
typedef enum scan_copy_mode {
  SCAN_COPY_VEC = 0, /* 128-bit streaming loads and stores, grid-stride */
  SCAN_COPY_TMA = 1  /* 32 KB 2-D tensor-copy tiles through a shared-memory ring */
} scan_copy_mode;

/* Copies `bytes` from src to dst on the device: the achievable read + write
 * bandwidth that the scan kernels' roofline fractions are reported against.
 * No counterpart in the source pages (they time their kernels alone): it
 * exists so that the ceiling is measured on the same GPU, launch path and
 * stream as the kernels it bounds, by copies written the way those kernels
 * move data (SCAN_COPY_VEC: the register path's 16-byte vector accesses;
 * SCAN_COPY_TMA: the stream variant's tensor copies).
 *   src, dst: device pointers, 16-byte aligned, not overlapping.
 *   bytes: a multiple of 16 (VEC) or of 128 (TMA); 0 does nothing.
 *   status: nullable device word; a TMA wait that expires (1 s) sets it to
 *     SCAN_ERR_TIMEOUT (the call itself has already returned).
 * Returns SCAN_ERR_INVALID_ARG for a bad mode, null pointer or size,
 * SCAN_ERR_ALIGNMENT for misaligned pointers, SCAN_ERR_CUDA if the launch or
 * the tensor-map encoding fails. Asynchronous on `stream`; allocates nothing. */
scan_status scan_copy(const void* src, void* dst, size_t bytes, int32_t mode, uint32_t* status,
                      cudaStream_t stream);

/* Bytes of the library's own scratch used by scan_fwd_noalloc (16 MiB). */
#define SCAN_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

/* scan_fwd without a caller-provided workspace and without any allocation.
 * No counterpart in the source pages: it exists for callers that cannot
 * allocate device memory -- code running inside a memory-capped or
 * pre-partitioned arena, real-time paths that forbid allocation after
 * start-up, plugin hosts that hand over only the tensors they own. The
 * caller still passes a, x, h0, cu_seqlens and h exactly as for scan_fwd
 * (same layouts and meaning); the look-back chunk summaries go to a fixed
 * scratch array of SCAN_NOALLOC_SCRATCH_BYTES compiled into the library,
 * which every GPU that loads the library keeps until the process exits.
 *   - Limit: the call needs 256 + 16 * rows * chunks bytes (rows = B*C, or C
 *     when packed; chunks = ceil((T + 3) / 512) for T > 256). Larger problems
 *     return SCAN_ERR_WORKSPACE and compute nothing; use scan_fwd for them.
 *   - The first call on each device sets the scratch up: it looks up the
 *     array's device address (cudaGetSymbolAddress, which may load the
 *     library's device code) and writes nothing; the array is zero when the
 *     module loads. Make that first call before any stream capture on that
 *     device.
 *   - a, x, h (and h0, cu_seqlens) must be device memory of the current
 *     device, whose scratch the call uses; other pointers return
 *     SCAN_ERR_INVALID_ARG.
 *   - Every call on a device shares the same scratch and leaves its contents
 *     behind; the kernel resets what the next call needs. Calls whose kernels
 *     overlap on the GPU (different streams, or threads) race on it and give
 *     undefined results: serialise them.
 *   - Device-side findings (a malformed cu_seqlens, an expired wait) are kept
 *     in that scratch; scan_noalloc_device_status reads them back. Host-side
 *     checks return their status as usual. Never calls cudaMalloc, cudaFree
 *     or any allocating routine. */
scan_status scan_fwd_noalloc(const void* a, const void* x, const float* h0,
                             const int32_t* cu_seqlens, int32_t n_seqs, float* h,
                             int64_t B, int64_t C, int64_t T, scan_dtype dt,
                             int32_t reverse, cudaStream_t stream);

/* The sticky device status of the current device's scan_fwd_noalloc scratch,
 * read and cleared: scan_get_device_status (synchronises `stream`, reads the
 * status word, resets it to 0) applied to the library's own scratch, which
 * the caller has no pointer to. Returns SCAN_OK, the finding of a call since
 * the last read (SCAN_ERR_TIMEOUT for an expired look-back wait,
 * SCAN_ERR_SEQLENS for a malformed device cu_seqlens), or SCAN_ERR_CUDA
 * when the synchronisation or copies fail. Like scan_fwd_noalloc, it
 * allocates nothing; the copies are synchronous. */
scan_status scan_noalloc_device_status(cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Token mixers that language models run next to the scans: the norm and
 * rotation of queries and keys, linear attention with a decay for each head
 * (the outer-product state above at the head sizes and types of such models)
 * and attention with a sliding window and first tokens that stay visible. They
 * have no counterpart in the source pages. The scans' conventions hold
 * (asynchronous, no allocation, no fallback); the operands are
 * [B, T, H, D] with a unit stride along D and any strides along the others, so
 * that they may be slices of a fused projection. */

/* A [B, T, H, D] device operand: element (b, t, h, d) is at
 * ptr + b stride_b + t stride_t + h stride_h + d (strides in elements). */
typedef struct scan_view4 {
  void* ptr;
  int64_t stride_b, stride_t, stride_h;
} scan_view4;

/* RMS norm of every query and key head, then the rotation of its position:
 *   z = w x (mean(x^2) + eps)^(-1/2),  y = z with each pair (a, b) of its first
 *   R elements replaced by (a cos - b sin, a sin + b cos).
 * Pair i is elements (i, R/2 + i), or (2i, 2i + 1) when interleaved != 0; its
 * cosine and sine are entry [position][i] of the fp32 tables [P, R/2].
 *   q, q_out: [B, T, Hq, D], k, k_out: [B, T, Hk, D] of dtype dt; an output may
 *   be its own input. Hq or Hk may be 0 (its pointers are not used).
 *   q_weight, k_weight: fp32 [D] or NULL (ones). positions: int32 [B, T]
 *   contiguous, or NULL (position t). A position outside [0, P) gives NaN in
 *   the rotated elements. R = 0: no rotation (tables may be NULL).
 * The norm and products are fp32; the result is rounded once. With eps = 0 a row
 * of zeros has no norm and gives NaN.
 * SCAN_ERR_UNSUPPORTED unless D % 8 == 0, D <= 256 and R % 8 == 0;
 * SCAN_ERR_ALIGNMENT unless every pointer is 16-byte aligned and every stride
 * a multiple of 16 bytes; SCAN_ERR_INVALID_ARG for negative sizes, R > D,
 * a negative or NaN eps, an empty table with R > 0 or a missing pointer. */
scan_status qk_norm_rope_fwd(const scan_view4* q, const scan_view4* k, const float* q_weight,
                             const float* k_weight, const float* cos_table, const float* sin_table,
                             const int32_t* positions, const scan_view4* q_out,
                             const scan_view4* k_out, int64_t B, int64_t T, int64_t Hq, int64_t Hk,
                             int64_t D, int64_t R, int64_t P, int32_t interleaved, float eps,
                             scan_dtype dt, cudaStream_t stream);

/* Its backward: with n = x (mean(x^2) + eps)^(-1/2), dz the gradient turned
 * back by the same angle and g = w dz,
 *   dx = (mean(x^2) + eps)^(-1/2) (g - n mean(g n)),  dw = sum over b, t, h of dz n.
 * q, k: the forward's inputs; dq_out, dk_out: the gradients of its outputs;
 * dq, dk: written, of dtype dt; dq_weight, dk_weight: fp32 [D], written, or
 * NULL. The sums over rows are fp32 in a fixed order. workspace:
 * qk_norm_rope_workspace_bytes(D) bytes, 16-byte aligned, nothing kept between
 * calls (else SCAN_ERR_WORKSPACE). Other errors as the forward's. */
size_t qk_norm_rope_workspace_bytes(int64_t D);
scan_status qk_norm_rope_bwd(const scan_view4* q, const scan_view4* k, const float* q_weight,
                             const float* k_weight, const float* cos_table, const float* sin_table,
                             const int32_t* positions, const scan_view4* dq_out,
                             const scan_view4* dk_out, const scan_view4* dq, const scan_view4* dk,
                             float* dq_weight, float* dk_weight, int64_t B, int64_t T, int64_t Hq,
                             int64_t Hk, int64_t D, int64_t R, int64_t P, int32_t interleaved,
                             float eps, scan_dtype dt, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream);

/* Linear attention with a decay for each head, per (sequence, head):
 *   S_t = lambda_h S_{t-1} + k_t v_t^T  (Dk x Dv, fp32),  S_{-1} = h0,
 *   o_t = scale q_t S_t,   lambda_h = exp(log_decay[h]).
 *   q, k: [B, T, H, Dk], v, o: [B, T, H, Dv] of dtype dt; log_decay: fp32 [H]
 *   (a constant of the model: no gradient; -inf: no memory); h0 (nullable) and
 *   hT (nullable, written): fp32 [B, H, Dk, Dv] contiguous.
 * Packed (cu_seqlens != NULL): B = 1, int32 [n_seqs + 1] offsets from 0 to T
 * on the device as for scan_fwd, h0 and hT [n_seqs, H, Dk, Dv]; empty sequences
 * are allowed (their hT is h0, or 0). Malformed offsets set the workspace's
 * device status to SCAN_ERR_SEQLENS.
 * bf16 operands on 16-byte boundaries run chunk by chunk on the tensor cores:
 * products of bf16 operands summed in fp32, the within-chunk weights and the
 * state as read by a query rounded to bf16, the state itself carried and
 * updated to fp32 accuracy. Other operands and short rows run the recurrence in
 * fp32. A row takes the chunks from 16 steps on (32 for many rows of heads up to
 * 32 x 32); packed rows go by the mean length of their sequences, so that a long
 * one among many of a few steps is walked step by step as well. Operands off 16
 * bytes, or broadcast over an axis by a stride of 0, take the recurrence too: it
 * costs 0.35 to 0.9 us a step.
 * Values within a sequence must be finite: in chunks, a value that is not makes
 * earlier results of its chunk NaN too. Values outside the sequences are never
 * used. An output must not overlap an input or another output.
 * workspace: linattn_workspace_bytes() bytes, zeroed once with
 * scan_workspace_init (it starts with the device status word), for forward and
 * backward; n_seqs = 0 when dense. SCAN_ERR_UNSUPPORTED unless Dk and Dv are
 * multiples of 8 up to 128; SCAN_ERR_INVALID_ARG unless scale > 0 and finite. */
size_t linattn_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv,
                               int64_t n_seqs);
scan_status linattn_fwd(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                        const float* log_decay, const float* h0, const int32_t* cu_seqlens,
                        int32_t n_seqs, const scan_view4* o, float* hT, int64_t B, int64_t T,
                        int64_t H, int64_t Dk, int64_t Dv, float scale, scan_dtype dt,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Its backward for L = sum <dout, o> + <dhT, hT>: three passes of the same
 * recurrence, since each gradient is linear attention over the other operands:
 *   dq: forward over (dout, v, k) from h0^T,
 *   dk: reversed over (v, dout, q), dv: reversed over (k, q, dout), from dhT,
 * dh0 = lambda (the state that the reversed pass ends in). dhT (nullable: 0),
 * dh0 (nullable): fp32 in h0's layout; dq, dk, dv: dtype dt, written. Nothing
 * of the forward is stored. Errors and workspace as the forward's. */
scan_status linattn_bwd(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                        const float* log_decay, const float* h0, const int32_t* cu_seqlens,
                        int32_t n_seqs, const scan_view4* dout, const float* dhT,
                        const scan_view4* dq, const scan_view4* dk, const scan_view4* dv, float* dh0,
                        int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, float scale,
                        scan_dtype dt, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream);

/* One token of each of B requests: S = lambda_h S + k v^T in place, o = scale q S.
 *   q, k: [B, H, Dk], v, o: [B, H, Dv] of dtype dt (views with stride_t unused);
 *   state: fp32 [n_slots, H, Dk, Dv] contiguous, 16-byte aligned; slots: int32
 *   [B], the state of each request, or NULL (request b has state b). Two requests
 *   must not share a state. A slot outside [0, n_slots) marks an idle request:
 *   o = 0 and no state is touched. */
scan_status linattn_step(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                         const float* log_decay, float* state, const int32_t* slots, int64_t n_slots,
                         const scan_view4* o, int64_t B, int64_t H, int64_t Dk, int64_t Dv,
                         float scale, scan_dtype dt, cudaStream_t stream);

/* Causal attention with a sliding window and first tokens that stay visible:
 * the query at position i sees key j where j <= i and (i - j < window or
 * j < sinks);  o_i = sum_j softmax_j(scale q_i k_j) v_j.
 *   q, o: [B, Tq, Hq, D]; k, v: [B, Tk, Hk, D] of dtype dt, Hq a multiple of Hk
 *   (query heads h Hq/Hk .. share key head h). The queries are the last Tq of
 *   the Tk positions. A query that sees no key (Tq > Tk) has o = 0, lse = -inf.
 *   lse: fp32 [B, Hq, Tq], the log of each row's sum of exponentials, written.
 * Packed (cu_seqlens): B = 1, Tq = Tk, positions count from each sequence's
 * start; device status as for linattn_fwd.
 * bf16 operands on 16-byte boundaries run on the tensor cores, weights rounded
 * to bf16 for the second product; statistics and sums are fp32. Other operands,
 * those broadcast over an axis by a stride of 0 among them, take general kernels
 * that are some twenty-five times slower.
 * Values within a sequence must be finite; what lies outside is never used. An
 * output must not overlap an input or another output.
 * workspace: window_attn_workspace_bytes() (backward != 0 for the backward's),
 * zeroed once with scan_workspace_init. SCAN_ERR_UNSUPPORTED unless D is a
 * multiple of 8 up to 128 and B Hq <= 65535; SCAN_ERR_INVALID_ARG unless
 * window >= 1, sinks >= 0, Hq % Hk == 0 and scale > 0 and finite. */
size_t window_attn_workspace_bytes(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk,
                                   int64_t D, int64_t window, int64_t sinks, int64_t n_seqs,
                                   int32_t backward);
scan_status window_attn_fwd(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                            const int32_t* cu_seqlens, int32_t n_seqs, const scan_view4* o,
                            float* lse, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk,
                            int64_t D, int64_t window, int64_t sinks, float scale, scan_dtype dt,
                            void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Its backward from the forward's o and lse:
 *   p_ij = exp(scale q_i k_j - lse_i), ds_ij = scale p_ij (dout_i v_j - dout_i o_i),
 *   dq_i = sum_j ds_ij k_j, dk_j = sum_i ds_ij q_i, dv_j = sum_i p_ij dout_i,
 * the last two over the query heads that share the key head as well. (bf16 on
 * the tensor cores: rows that see one tile of 128 keys form dout_i o_i anew, as
 * the sum of p_ij dout_i v_j in fp32, since o is rounded.) dq, dk, dv: dtype dt,
 * written. No sum depends on the order in which blocks run.
 * Errors and workspace as the forward's. */
scan_status window_attn_bwd(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                            const scan_view4* o, const float* lse, const scan_view4* dout,
                            const int32_t* cu_seqlens, int32_t n_seqs, const scan_view4* dq,
                            const scan_view4* dk, const scan_view4* dv, int64_t B, int64_t Tq,
                            int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int64_t window,
                            int64_t sinks, float scale, scan_dtype dt, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream);

/* One token of each of B requests over cached keys and values, which it joins.
 *   q, o: [B, Hq, D], k, v: [B, Hk, D] of dtype dt (views with stride_t unused);
 *   k_cache, v_cache: [n_slots, sinks + window, Hk, D] of dtype dt, contiguous,
 *   16-byte aligned: position p of a request is row p while p < sinks, then row
 *   sinks + (p - sinks) % window, so a token takes the place of the one that
 *   leaves the window. positions: int32 [B], the new token's position; the rows
 *   of the min(positions, sinks + window) positions before it are filled.
 *   slots: int32 [B], the cache of each request, or NULL (request b has cache
 *   b); two requests must not share a cache. A slot outside [0, n_slots) or a
 *   negative position marks an idle request: o = 0 and no cache is touched.
 *   Rows that are not filled are never used. */
scan_status window_attn_step(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                             void* k_cache, void* v_cache, const int32_t* positions,
                             const int32_t* slots, int64_t n_slots, const scan_view4* o, int64_t B,
                             int64_t Hq, int64_t Hk, int64_t D, int64_t window, int64_t sinks,
                             float scale, scan_dtype dt, cudaStream_t stream);

/* Attention to the states of another sequence, of another length (an encoder's):
 *   o_i = sum_j softmax_j(scale q_i k_j) v_j over the keys of the query's sequence.
 *   q, o: [B, Tq, Hq, D]; k, v: [B, Tk, Hk, D] of dtype dt, Hq a multiple of Hk
 *   (query heads h Hq/Hk .. share key head h).
 *   k_lens (nullable): int32 [B] on the device; batch row b's queries see its first
 *   k_lens[b] keys (a padded batch), else all Tk.
 *   Packed (cu_seqlens_q and cu_seqlens_k, no k_lens): B = 1, int32 [n_seqs + 1]
 *   offsets each, from 0 to Tq and to Tk; the queries of sequence i see the keys of
 *   sequence i. Malformed offsets and lengths outside [0, Tk] set the workspace's
 *   device status to SCAN_ERR_SEQLENS (and are clamped).
 *   A query that has no key has o = 0, lse = -inf. lse: fp32 [B, Hq, Tq], the log of
 *   each row's sum of exponentials, written.
 * Statistics and sums are fp32. bf16 operands on 16-byte boundaries with strides of
 * whole 16 bytes (and none of 0) take the tensor cores: the weights, and in the backward
 * their gradients, are rounded to bf16 before the second product, each by half a step at
 * most (2^-8 of itself; the gradients in two parts, 2^-16, for a sequence or batch row of
 * 512 keys or fewer, by its own length, where that takes little time). All other operands
 * take the general kernels, whose products are of fp32 accuracy (each factor as the sum of
 * two tf32 numbers); bf16 operands, those broadcast over an axis by a stride of 0 among
 * them, are some thirty-five times slower there.
 * Keys and values past a row's length are never used, whatever they hold; values within
 * have to be finite: v 2^80 in magnitude at most, since its sums are divided by the sum of
 * weights at the end (up to 2^16 for 128 keys, before the reference of a row's softmax
 * moves), and other fp32 operands 2^127, since they are rounded to 11 bits on the way. With
 * larger ones a result that is finite by its formula may come out infinite or NaN. An
 * output must not overlap an input or another output.
 * workspace: cross_attn_workspace_bytes() (n_seqs = 0 unless packed, backward != 0 for
 * the backward's), zeroed once with scan_workspace_init. SCAN_ERR_UNSUPPORTED unless D
 * is a multiple of 8 up to 128 and B Hq <= 65535; SCAN_ERR_INVALID_ARG unless Hq % Hk
 * == 0 and scale > 0 and finite. */
size_t cross_attn_workspace_bytes(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk,
                                  int64_t D, int64_t n_seqs, int32_t backward);
scan_status cross_attn_fwd(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                           const int32_t* k_lens, const int32_t* cu_seqlens_q,
                           const int32_t* cu_seqlens_k, int32_t n_seqs, const scan_view4* o,
                           float* lse, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk,
                           int64_t D, float scale, scan_dtype dt, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream);

/* Its backward from the forward's o and lse, by the formulas of window_attn_bwd over
 * the same pairs. dq, dk, dv: dtype dt, written; the rows of dk and dv past a length
 * are zeros. No sum depends on the order in which blocks run. Errors and workspace as
 * the forward's. */
scan_status cross_attn_bwd(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                           const scan_view4* o, const float* lse, const scan_view4* dout,
                           const int32_t* k_lens, const int32_t* cu_seqlens_q,
                           const int32_t* cu_seqlens_k, int32_t n_seqs, const scan_view4* dq,
                           const scan_view4* dk, const scan_view4* dv, int64_t B, int64_t Tq,
                           int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, float scale,
                           scan_dtype dt, void* workspace, size_t workspace_bytes,
                           cudaStream_t stream);

/* One query token of each of B requests over a pool of encoders' keys and values,
 * which are only read.
 *   q, o: [B, Hq, D] of dtype dt (views with stride_t unused); k_cache, v_cache:
 *   [n_slots, Tk, Hk, D] of dtype dt, any strides but along D; lens (nullable): int32
 *   [n_slots], the keys that each cache holds (forced into [0, Tk]), else Tk; slots:
 *   int32 [B], the cache of each request, or NULL (request b has cache b). Requests may
 *   share a cache. A slot outside [0, n_slots) marks an idle request, which gets o = 0,
 *   as one without keys does. Rows past a length are never used; values are as large as the
 *   forward's may be. bf16 caches on 16-byte boundaries are read by tensor copies, the
 *   weights of their values the sum of two bf16 numbers each (2^-16 of themselves).
 * workspace: cross_attn_step_workspace_bytes(), zeroed once with scan_workspace_init;
 * nothing is kept in it between calls but its status word. Errors as the forward's, but
 * B Hq may be up to 2^31 - 1. */
size_t cross_attn_step_workspace_bytes(int64_t B, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D);
scan_status cross_attn_step(const scan_view4* q, const scan_view4* k_cache,
                            const scan_view4* v_cache, const int32_t* lens, const int32_t* slots,
                            int64_t n_slots, const scan_view4* o, int64_t B, int64_t Tk, int64_t Hq,
                            int64_t Hk, int64_t D, float scale, scan_dtype dt, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * What a network runs around its blocks. Operands are [B, T, C] with a unit stride
 * along C (scan_view4 with stride_h unused). */

/* Dropout whose mask is never stored: y = x / (1 - p) where an element is kept, else 0
 * (whatever x holds there).
 * Element i (counted over [B, T, C] in order) has 16 bits of block i / 8 of Philox 4x32
 * with ten rounds (Salmon, Moraes, Dror and Shaw, SC 2011): key = seed, counter =
 * (block, call), number i % 8 counted from the low half of the first word. It is dropped
 * where they are below 65536 p, rounded to a whole number (p is taken in steps of 2^-16,
 * also in the factor 1 / (1 - p)). The mask depends on nothing else: not on types, strides
 * or the GPU. Other values of `call` are independent masks of the same seed.
 *   x, y: dtype dt, any strides; y may be x. rng (nullable): int64 {seed, call} on the
 *   device, read instead of seed and call when the kernel runs, so that a captured graph
 *   draws anew as its owner changes them.
 * SCAN_ERR_INVALID_ARG unless 0 <= p <= 1; SCAN_ERR_UNSUPPORTED past 2^41 elements;
 * SCAN_ERR_ALIGNMENT unless rng is 8-byte aligned. */
scan_status dropout_fwd(const scan_view4* x, const scan_view4* y, int64_t B, int64_t T, int64_t C,
                        double p, uint64_t seed, uint64_t call, const int64_t* rng, scan_dtype dt,
                        cudaStream_t stream);
/* Its backward, the same pass over the gradient: dx = dy / (1 - p) where kept, else 0. */
scan_status dropout_bwd(const scan_view4* dy, const scan_view4* dx, int64_t B, int64_t T, int64_t C,
                        double p, uint64_t seed, uint64_t call, const int64_t* rng, scan_dtype dt,
                        cudaStream_t stream);

/* The norms after and before a block, with its gate, dropout and residual scale:
 *   z = post_weight y (mean(y^2) + eps)^(-1/2)          (y itself without post_weight)
 *   x_out = alpha x + drop(gate z)
 *   n = next_weight x_out (mean(x_out^2) + eps)^(-1/2)  (not formed without next_weight)
 * y is what the block gave, x the residual stream before it, n what the next block reads;
 * n is the norm of x_out as it is stored.
 *   x, x_out: [B, T, C] of dtype stream_dt; y, n: of dtype dt (stream_dt fp32 with either
 *   dt, or bf16 with bf16). post_weight, next_weight: fp32 [C] or NULL; gate: fp32 [C], or
 *   [B, C] with row_gate != 0, or NULL (ones). p, seed, call, rng: as for dropout_fwd, over
 *   the elements of [B, T, C] (without post_weight, what y holds at a dropped element leaves no
 *   trace, forward or backward; with it, y's norm has it in).
 *   y NULL: only the norm of x (no post_weight and gate, alpha =
 *   1, p = 0; x_out is not written). x_out may be x, n may be y.
 * Norms and sums are fp32, each result is rounded once. With eps = 0 a row of zeros has no
 * norm and gives NaN.
 * SCAN_ERR_UNSUPPORTED unless C % 8 == 0, C <= 8192 and B T < 2^31; SCAN_ERR_ALIGNMENT
 * unless every pointer is 16-byte aligned and every stride a multiple of 16 bytes;
 * SCAN_ERR_INVALID_ARG for negative sizes, a NaN or negative eps, an alpha that is not
 * finite, p outside [0, 1] or a missing pointer. */
size_t residual_norm_workspace_bytes(int64_t B, int64_t T, int64_t C, int32_t row_gate);
scan_status residual_norm_fwd(const scan_view4* x, const scan_view4* y, const float* post_weight,
                              const float* gate, const float* next_weight, const scan_view4* x_out,
                              const scan_view4* n, int64_t B, int64_t T, int64_t C, int32_t row_gate,
                              float alpha, float eps, double p, uint64_t seed, uint64_t call,
                              const int64_t* rng, scan_dtype stream_dt, scan_dtype dt,
                              cudaStream_t stream);

/* Its backward for L = sum <dx_out, x_out> + <dn, n>, from x_out and y; the same mask is
 * drawn again. dx_out may be NULL (0) where next_weight is given; x_out and dn are not used
 * without it. dx: stream_dt, dy: dt, written (dx may be dx_out, dy may be dn); dpost_weight,
 * dgate, dnext_weight: fp32 in their inputs' shapes, written, or NULL. The sums over rows are
 * fp32 in a fixed order. workspace: residual_norm_workspace_bytes() bytes, 16-byte aligned,
 * zeroed once with scan_workspace_init. Other errors as the forward's. */
scan_status residual_norm_bwd(const scan_view4* x_out, const scan_view4* y, const scan_view4* dx_out,
                              const scan_view4* dn, const float* post_weight, const float* gate,
                              const float* next_weight, const scan_view4* dx, const scan_view4* dy,
                              float* dpost_weight, float* dgate, float* dnext_weight, int64_t B,
                              int64_t T, int64_t C, int32_t row_gate, float alpha, float eps,
                              double p, uint64_t seed, uint64_t call, const int64_t* rng,
                              scan_dtype stream_dt, scan_dtype dt, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBSCAN_H */
