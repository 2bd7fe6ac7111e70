/*
 * pb.h — C ABI of the GB300 (sm_103a) forward pass of the parallel transformer block
 *
 *     y = x + MLP(LN(x)) + Attention(LN(x))
 *
 * (MegaScale reading notes, section 1.1 "Parallel Transformer Block", eq. (4)), where
 *   LN         = LayerNorm with gamma/beta, computed ONCE and shared by both branches;
 *   MLP(z)     = GeLU(z W1) W2               (Megatron-LM notes, section 2.1, Y = GeLU(XA)B);
 *   Attention  = multi-head attention on the [q | k | v] = z Wqkv projection (Megatron-LM
 *                notes, section 2.2), each query attending to the most recent `window`
 *                tokens of its own sequence, itself included (MegaScale reading notes,
 *                section 1.1 "Sliding Window Attention", eqs. (5)-(6)), followed by Wo.
 *
 * The library fuses the two branches: one GEMM against [Wqkv | W1] (GeLU in its
 * epilogue), one sliding-window flash attention kernel, and one GEMM of
 * [attn | GeLU(h)] against [Wo ; W2] with the residual added in its epilogue.
 *
 * Conventions for every entry point:
 *  - Tensors are bf16 (IEEE bfloat16 bit patterns), row-major, on the CURRENT CUDA
 *    device unless stated. Weights use the pages' Y = X W convention: [in, out].
 *  - Token rows are ordered (batch, position): x and y are [batch*seq, hidden].
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream). All work is
 *    enqueued asynchronously on it; no call synchronises the host, except
 *    pb_get_status, which reads a word the kernels write.
 *  - The library allocates NO device memory. The caller owns every buffer: inputs,
 *    outputs, the per-handle weight workspace and the per-call scratch.
 *  - Every function returns pb_status; no C++ exception crosses the ABI. Argument
 *    errors are detected before anything is enqueued. pb_last_error_message() returns
 *    a thread-local description of the last failure on the calling thread.
 *  - Device-side failures (a bounded wait inside a kernel that ran out) do not fault the
 *    GPU: the kernel records PB_ERR_DEVICE_TIMEOUT in the handle's status word and
 *    returns; pb_get_status reports it.
 */
#ifndef PB_H_
#define PB_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pb_status {
  PB_OK = 0,
  PB_ERR_INVALID_ARG = 1,     /* NULL/misaligned pointer, bad size, partial aliasing   */
  PB_ERR_UNSUPPORTED = 2,     /* shape outside the supported set (see pb_dims)         */
  PB_ERR_WORKSPACE = 3,       /* workspace or scratch smaller than required            */
  PB_ERR_CUDA = 4,            /* a CUDA runtime/driver call failed (message has why)   */
  PB_ERR_DEVICE_TIMEOUT = 5,  /* a kernel's bounded wait expired; results are invalid  */
  PB_ERR_BAD_HANDLE = 6,      /* NULL, destroyed or foreign handle, or wrong device    */
  PB_ERR_RANGE = 7            /* PB_OPERANDS_FP16 only: a weight or an activation that */
                              /* feeds a GEMM exceeded the fp16 range (|v| > 65504)    */
} pb_status;

/*
 * Shape of one block. Supported (else PB_ERR_UNSUPPORTED):
 *   batch, seq >= 1; window >= 1 (window >= seq is full causal attention);
 *   head_dim in {64, 128}; hidden = heads * head_dim; hidden % 64 == 0; ffn % 64 == 0;
 *   batch * seq < 2^31; ln_eps > 0.
 */
typedef struct pb_dims {
  int32_t batch;
  int32_t seq;
  int32_t hidden;    /* H */
  int32_t heads;     /* nh */
  int32_t head_dim;  /* dh, H = nh * dh */
  int32_t ffn;       /* F, width of the MLP (4H on the pages) */
  int32_t window;    /* w: key k is visible to query i iff 0 <= i - k < w */
  float ln_eps;      /* LayerNorm epsilon, inside the square root */
  int32_t variant;   /* PB_BLOCK_LN_GELU (eq. (4) as written) or PB_BLOCK_RMS_SWIGLU */
} pb_dims;

/* Block variants. PB_BLOCK_RMS_SWIGLU replaces the LayerNorm by RMSNorm
 * (x / sqrt(mean x^2 + eps) * gamma; ln_beta unused) and the GeLU MLP by SwiGLU,
 * silu(z W_gate) * (z W_up) then W2: the fused "RMSNorm" and "SiLU + elementwise
 * multiply" kernels of the MegaScale reading notes, section 1.3 (named there without a
 * definition; the standard forms are used). */
typedef enum pb_block_variant { PB_BLOCK_LN_GELU = 0, PB_BLOCK_RMS_SWIGLU = 1 } pb_block_variant;

/*
 * Parameters of one block (device pointers, bf16). They are read only by pb_create,
 * which packs them into the workspace; they may be freed once the stream has passed
 * pb_create's work.
 *   ln_gamma, ln_beta : [H]     (ln_beta unused, may be NULL, for PB_BLOCK_RMS_SWIGLU)
 *   wqkv              : [H, 3H]; columns [Q | K | V], head j of each owns columns
 *                       [j*dh, (j+1)*dh) of its H-wide block
 *   w1                : [H, F]    (first MLP linear, "A" of Y = GeLU(XA)B); for
 *                       PB_BLOCK_RMS_SWIGLU [H, 2F] = [W_gate | W_up], and b1 is [2F]
 *   wo                : [H, H]    (attention output projection)
 *   w2                : [F, H]    (second MLP linear, "B")
 *   b_qkv [3H], b1 [F], b_o [H], b2 [H] : optional biases, NULL = none.
 */
typedef struct pb_weights {
  const void* ln_gamma;
  const void* ln_beta;
  const void* wqkv;
  const void* w1;
  const void* wo;
  const void* w2;
  const void* b_qkv;
  const void* b1;
  const void* b_o;
  const void* b2;
} pb_weights;

/* Byte offsets of the intermediates inside the scratch buffer of a forward call, valid
 * after the stream passes it (for inspection and tests):
 *   xn   [T, H]          LN(x)                      (bf16, fp16 with PB_OPERANDS_FP16)
 *   qk   [T, 2H]         [q | k], head-major columns (bf16)
 *   vt   [batch, heads, dh, seq_pad] v transposed per head, seq_pad = seq rounded up to 8
 *   act  [T, H + F]      [attention output (before Wo) | GeLU(h)]  (bf16 / fp16)
 *   q8, qscale           the FP8 operands of PB_OPERANDS_FP8 (see the fields)
 *   io, io2 [T, H]       bf16 staging of the host-buffer entry points
 *   res0, res1 [T, H]    fp32 residual stream between the layers of a stack
 *   sk                   stream-K partial tiles (fp32) and flags of the two GEMMs
 * T = batch * seq, F' = F (GeLU) or 2F (SwiGLU).
 * A training scratch (pb_forward_train / pb_backward, train_total bytes) has the same
 * regions up to `total`, then:
 *   hpre   [T, F']       h before the activation (bf16; SwiGLU: W1cat's interleaved order)
 *   lse    [batch * heads, seq64]  fp32 log2-sum-exp of each attention row's scores x
 *                        log2(e) / sqrt(dh); seq64 = seq rounded up to 64
 *   d_attn [T, H]        dL/d(attention output) (bf16)
 *   delta  [batch * heads, seq64]  fp32 dO . O per row
 *   dq_acc [T, H]        fp32 dq accumulator
 *   dz     [T, 3H + F']  [dq | dk | dv | dh], dL/d[q | k | v | h] (bf16, W1cat order)
 *   dxn    [T, H]        fp32 dL/dLN(x)
 *   stats  [T]           fp32 (mean, rstd) per row
 *   partials             fp32 partial column sums of the parameter gradients */
typedef struct pb_scratch_layout {
  size_t xn;
  size_t qk;
  size_t vt;
  size_t act;
  size_t io;
  size_t io2;
  size_t res0;
  size_t res1;
  size_t sk;  /* stream-K partial tiles and flags of the GEMMs */
  size_t q8;      /* PB_OPERANDS_FP8: [T, H + F] E4M3 codes of act (xn holds LN(x)'s codes) */
  size_t qscale;  /* PB_OPERANDS_FP8: [2T] fp32 row scales of LN(x), then of act */
  size_t seq_pad;
  size_t total;
  size_t hpre;
  size_t lse;
  size_t d_attn;
  size_t delta;
  size_t dq_acc;
  size_t dz;
  size_t dxn;
  size_t stats;
  size_t partials;
  size_t train_total;
} pb_scratch_layout;

/* Precision of the two GEMMs' operands. The pages' mixed-precision recipe computes in
 * bf16 with fp32 accumulation (Megatron-LM notes, section 5.4-5.5; performance notes,
 * "BF16 / FP16 / FP8"), which is the default. PB_OPERANDS_FP16 stores LN(x), the packed
 * weights, the attention output and GeLU(h) as fp16 instead: the same 16 bits and the
 * same tensor-core rate, 3 more mantissa bits, and a range limit of 65504 that the
 * kernels check (PB_ERR_RANGE). Attention (q, k, v, P) stays bf16 in both modes.
 * PB_OPERANDS_FP8 runs both GEMMs on FP8 E4M3 operands (the performance notes' FP8
 * recipe: E4M3 for the forward pass, only the GEMMs in FP8, LayerNorm, softmax and the
 * residual in bf16 / fp32) with current scaling per row: each row of LN(x) and of
 * [attention output | GeLU(h)], and each output channel of the packed weights, is scaled
 * by 448 / its largest magnitude; the GEMM epilogue multiplies the fp32 sum back by both
 * scales. Needs H and H + F to be multiples of 128; pb_forward_serial does not support it.
 * Not the reference precision: its results differ from the bf16 path by the E4M3 rounding
 * (3 mantissa bits). */
typedef enum pb_operand_precision {
  PB_OPERANDS_BF16 = 0,
  PB_OPERANDS_FP16 = 1,
  PB_OPERANDS_FP8 = 2
} pb_operand_precision;

typedef struct pb_options {
  int32_t operand_precision; /* pb_operand_precision */
  uint64_t wait_limit_ns;    /* limit of every bounded wait in the kernels; 0 = 2e9 */
} pb_options;

typedef struct pb_handle pb_handle;

/* Guard gaps (a debugging aid for out-of-bounds writes; the pages have no counterpart).
 * pb_set_guard_bytes(g) makes every workspace and scratch layout computed afterwards leave
 * g unused bytes after each of its regions (before the next region's 1024-byte alignment):
 * pb_weight_workspace_bytes, pb_create, pb_scratch_bytes, pb_train_scratch_bytes,
 * pb_get_scratch_layout and every call that takes a scratch buffer. No kernel reads or
 * writes those bytes, so a caller that fills the buffers with a known pattern can check
 * after its calls that nothing ran past the end of a region. g <= 1 MiB (else
 * PB_ERR_INVALID_ARG); default 0. It is process-wide: set it before sizing the buffers and
 * creating the handles that use them, and keep it until they are released (a handle keeps
 * the workspace layout of its pb_create; a scratch sized under another setting is too small
 * or laid out differently, and too small is reported as PB_ERR_WORKSPACE). */
pb_status pb_set_guard_bytes(size_t bytes);
pb_status pb_get_guard_bytes(size_t* bytes);

/* Bytes of the per-handle weight workspace (packed [Wqkv | W1] and [Wo ; W2] in the
 * K-major layout the tensor cores read, biases, LN parameters and the status word). */
pb_status pb_weight_workspace_bytes(const pb_dims* dims, size_t* bytes);

/* Bytes of the scratch one forward call needs (shared by all layers of a stack), and
 * its layout. */
pb_status pb_scratch_bytes(const pb_dims* dims, size_t* bytes);
pb_status pb_get_scratch_layout(const pb_dims* dims, pb_scratch_layout* layout);

/* Creates a handle for one block on the current device. `workspace` (device, 256-byte
 * aligned, >= pb_weight_workspace_bytes) is owned by the caller and must outlive the
 * handle. Enqueues the weight packing on `stream`. */
pb_status pb_create(const pb_dims* dims, const pb_weights* weights, void* workspace,
                    size_t workspace_bytes, void* stream, pb_handle** out);

/* pb_create with options (NULL = defaults: bf16 operands, 2 s wait limit). */
pb_status pb_create_ex(const pb_dims* dims, const pb_weights* weights, const pb_options* options,
                       void* workspace, size_t workspace_bytes, void* stream, pb_handle** out);

/* One block: y = x + MLP(LN(x)) + Attention(LN(x)). x, y: [batch*seq, hidden] bf16,
 * 16-byte aligned; y may equal x (in place), partial overlap is PB_ERR_INVALID_ARG.
 * `scratch` (device, 256-byte aligned, >= pb_scratch_bytes) must not be used by another
 * call that may run concurrently. */
pb_status pb_forward(pb_handle* h, const void* x, void* y, void* scratch, size_t scratch_bytes,
                     void* stream);

/* ------------------------------------------------------------------------------------
 * Training: the block's backward pass (the pages' subject is training: MFU counts the
 * forward's 2 and the backward's 4 FLOPs per weight and token, performance notes "MFU").
 * pb_forward_train is pb_forward that also keeps, in a training scratch, what the
 * backward reads: h before its activation and each attention row's log-sum-exp. The
 * attention probabilities are not kept; pb_backward recomputes them (the selective
 * recomputation of the MegaScale reading notes, section 1.3). Supported: bf16 operands
 * (PB_OPERANDS_BF16), head_dim 64 or 128; other operand precisions give
 * PB_ERR_UNSUPPORTED.
 * ---------------------------------------------------------------------------------- */

/* Bytes of the training scratch of pb_forward_train / pb_backward (train_total). */
pb_status pb_train_scratch_bytes(const pb_dims* dims, size_t* bytes);

/* pb_forward, keeping hpre and lse in `scratch` (>= pb_train_scratch_bytes) for a
 * following pb_backward on the same handle, x and scratch. */
pb_status pb_forward_train(pb_handle* h, const void* x, void* y, void* scratch,
                           size_t scratch_bytes, void* stream);

/* Gradients of the block, all device pointers: dx bf16 [T, H] (dL/dx, the residual path
 * included); every parameter gradient fp32 in the layout of its pb_weights entry
 * (dwqkv [H, 3H], dw1 [H, F'] = [gate | up] for SwiGLU, dwo [H, H], dw2 [F, H], biases
 * [3H], [F'], [H], [H], dgamma and dbeta [H]). NULL skips a bias gradient or dbeta. */
typedef struct pb_grads {
  void* dx;
  float* dgamma;
  float* dbeta;
  float* dwqkv;
  float* dw1;
  float* dwo;
  float* dw2;
  float* db_qkv;
  float* db1;
  float* db_o;
  float* db2;
} pb_grads;

/* The backward pass for upstream gradient dy (bf16 [T, H]) after pb_forward_train(h, x,
 * ...) with the same scratch: d_attn and dh from one GEMM against W2cat, the attention
 * backward (P recomputed from q, k and lse), dLN(x) from one GEMM against W1cat, the
 * normalisation backward plus dy (dx), and the weight gradients as two GEMMs over the
 * tokens ([dWo ; dW2] = act^T dy, [dWqkv | dW1] = LN(x)^T dz). accumulate != 0 adds the
 * fp32 parameter gradients to what the buffers hold (dx is always overwritten). */
pb_status pb_backward(pb_handle* h, const void* x, const void* dy, const pb_grads* grads,
                      int32_t accumulate, void* scratch, size_t scratch_bytes, void* stream);

/* The serial (standard) transformer block of eq. (3) (MegaScale reading notes, section 1.1,
 * "Parallel Transformer Block") on the handle's weights, for comparison with pb_forward:
 *   h = x + Attn(LN(x)),   y = h + MLP(LN'(h)),   MLP(z) = GeLU(z W1 + b1) W2 + b2,
 * with Attn(.) W_o + b_o as in pb_forward. The printed eq. (3) omits the attention term from
 * the outer sum; the derivation beside it (the parallel block replaces LN(x + h2) by LN(x))
 * requires it, so it is included. LN' has parameters ln2_gamma / ln2_beta (device bf16
 * [H], 16-byte aligned), or the handle's LayerNorm when both are NULL (eq. (3) writes the
 * same LN twice). x, y, scratch as in pb_forward (x == y allowed); h is kept in fp32 in
 * scratch res0. Seven kernel launches instead of four: the MLP waits for the attention
 * output. */
pb_status pb_forward_serial(pb_handle* h, const void* x, void* y, const void* ln2_gamma,
                            const void* ln2_beta, void* scratch, size_t scratch_bytes,
                            void* stream);

/* A stack of residual blocks (MegaScale reading notes, section 1.1: L layers give a
 * receptive field of L*w), x_{l+1} = block_l(x_l). All handles must have the same
 * dims. Between layers the residual stream stays in fp32 (scratch res0/res1; the pages
 * keep residual accumulation in BF16/FP32, performance notes, "BF16 / FP16 / FP8"): only
 * x and the final y are bf16. */
pb_status pb_forward_stack(pb_handle* const* layers, int32_t n_layers, const void* x, void* y,
                           void* scratch, size_t scratch_bytes, void* stream);

/* As pb_forward_stack, with y in fp32 (float [batch*seq, hidden], 16-byte aligned, not
 * overlapping x): the residual stream the stack carries between its layers, returned
 * without the final rounding to bf16 (the same stream as pb_forward_stack's y before that
 * rounding). For callers that keep the residual stream in fp32 across stacks. */
pb_status pb_forward_stack_f32(pb_handle* const* layers, int32_t n_layers, const void* x,
                               float* y, void* scratch, size_t scratch_bytes, void* stream);

/* As pb_forward_stack, with x and y in HOST memory (pinned memory gives asynchronous
 * copies): copies x to the device, runs the stack, copies y back, all on `stream`.
 * The caller synchronises the stream before reading y. */
pb_status pb_forward_stack_host(pb_handle* const* layers, int32_t n_layers, const void* x_host,
                                void* y_host, void* scratch, size_t scratch_bytes, void* stream);

/* A sequence of n_steps independent passes of the stack over host inputs, the loop of a
 * resident model serving a stream of batches: step s copies x_host[s] in, runs the stack,
 * copies y_host[s] out. Two device staging buffers (scratch io and io2) alternate and the
 * copies run on a copy stream the library creates in layers[0] on first use (released by
 * pb_destroy), so the input of step s + 1 and the output of step s - 1 move while step s
 * computes on `stream`. When `stream` reaches the point after this call, every y_host[s]
 * is written. x_host, y_host: arrays of n_steps host pointers (pinned memory for
 * asynchronous copies); a y_host[s] may equal an x_host[t] only if t <= s. The handles
 * must not be used by another host thread meanwhile. */
pb_status pb_forward_stack_host_steps(pb_handle* const* layers, int32_t n_layers,
                                      int32_t n_steps, const void* const* x_host,
                                      void* const* y_host, void* scratch, size_t scratch_bytes,
                                      void* stream);

/* Reads the handle's device status word (blocks until the word can be read on the
 * handle's device) and returns PB_OK or the first device-side error recorded since
 * the last pb_clear_status. */
pb_status pb_get_status(pb_handle* h);
pb_status pb_clear_status(pb_handle* h, void* stream);

/* Sets the limit, in nanoseconds, of every bounded wait inside this handle's kernels
 * (default 2e9). A wait that reaches it records PB_ERR_DEVICE_TIMEOUT and the kernel
 * returns. */
pb_status pb_set_wait_limit_ns(pb_handle* h, uint64_t limit_ns);

/* Per-kernel timing of this handle's forward calls. pb_trace_enable(h, n) makes the
 * next n forward calls record CUDA events (host-side event objects, no device memory)
 * around each of the block's four kernels on the call's stream; n = 0 turns tracing off.
 * pb_trace_read waits for the recorded events and returns in ms[4] the summed
 * milliseconds of [LayerNorm, first GEMM, attention, second GEMM] over the traced calls,
 * and their number in *calls. */
pb_status pb_trace_enable(pb_handle* h, int32_t n_calls);
pb_status pb_trace_read(pb_handle* h, float* ms, int32_t* calls);

/* Destroys the handle (host memory only; the caller frees the workspace). */
pb_status pb_destroy(pb_handle* h);

const char* pb_status_string(pb_status s);
const char* pb_last_error_message(void);

/* ------------------------------------------------------------------------------------
 * Single steps of the block, exported for testing and reuse. Same conventions.
 * ---------------------------------------------------------------------------------- */

/* Per-row current scaling of a bf16 [rows, cols] matrix to FP8 E4M3, the quantizer of
 * PB_OPERANDS_FP8 (performance notes, "BF16 / FP16 / FP8"), in fixed fp32 steps:
 * amax = max |x[r,:]|, inv = 448 / amax (0 if amax = 0), scales[r] = amax / 448,
 * codes[r,c] = E4M3(x[r,c] * inv) rounded to nearest even and saturated at +-448.
 * x: device bf16 [rows, cols], codes: device [rows, cols] bytes, scales: device fp32
 * [rows]; cols % 8 == 0, pointers 16-byte aligned. */
pb_status pb_quantize_rows_e4m3(int64_t rows, int32_t cols, const void* x, void* codes,
                                void* scales, void* stream);

/* LayerNorm (the LN of eq. (4)): out[r,:] = (x[r,:] - mean) / sqrt(var + eps) * gamma
 * + beta, biased variance, fp32 statistics. x, out: [rows, H] bf16; gamma, beta: [H]
 * bf16. H % 8 == 0, H <= 16384. beta == NULL gives RMSNorm instead (the fused kernel of
 * section 1.3): out[r,:] = x[r,:] / sqrt(mean x^2 + eps) * gamma. */
pb_status pb_layernorm(int64_t rows, int32_t H, const void* x, const void* gamma,
                       const void* beta, float eps, void* out, void* stream);

/* C[M, N] = A[M, K] * B[N, K]^T on the tensor cores (bf16 inputs, fp32 accumulation,
 * bf16 output rounded to nearest even): the contraction of every linear layer of the
 * block with the weight stored K-major. A, B, C 16-byte aligned; K % 64 == 0,
 * N % 32 == 0. `scratch` (device, 256-byte aligned, >= pb_gemm_scratch_bytes, or NULL)
 * lets the last waves of tiles be split along K across the SMs (stream-K); with NULL every
 * tile is computed whole. Calls that share a scratch buffer must not overlap on the GPU.
 * `status` (device int, may be NULL) receives PB_ERR_DEVICE_TIMEOUT if a bounded wait
 * runs out. */
pb_status pb_gemm_scratch_bytes(size_t* bytes);
pb_status pb_gemm_bf16(int32_t M, int32_t N, int32_t K, const void* A, const void* B, void* C,
                       void* scratch, size_t scratch_bytes, int* status, void* stream);

/* pb_gemm_bf16 with either operand stored MN-major, the layouts of the backward pass's
 * GEMMs (activations stored token-major are MN-major when the contraction runs over
 * tokens): a_mn = 0: A is [M, K] (K contiguous), a_mn = 1: A is [K, M] (M contiguous);
 * b_mn = 0: B is [N, K], b_mn = 1: B is [K, N]. C[m, n] = sum_k A(m, k) B(n, k), bf16.
 * N % 32 == 0; a K-major operand needs K % 8 == 0, an MN-major one M (or N) % 8 == 0;
 * a ragged last block of K is zero filled. Otherwise as pb_gemm_bf16. */
pb_status pb_gemm_bf16_layout(int32_t M, int32_t N, int32_t K, const void* A, int32_t a_mn,
                              const void* B, int32_t b_mn, void* C, void* scratch,
                              size_t scratch_bytes, int* status, void* stream);

/* pb_gemm_bf16 for callers that cannot allocate device memory: plugins inside an engine or
 * framework whose device memory all belongs to the host program's allocator (they are
 * handed inputs and outputs, nothing more), and latency-bound paths where a cudaMalloc
 * could synchronise the device or block. The pages have no counterpart; it is a
 * convenience of this library. It computes the same product with the same stream-K
 * schedule as pb_gemm_bf16 with scratch, so its output is bit-identical to that call's,
 * with the scratch in a fixed array of the library's own device memory (25,171,968 bytes
 * per GPU, held until the process exits) instead of a caller buffer. It allocates nothing
 * and calls no allocating routine. Limits: GPUs with at most 192 SMs (96 CTA pairs);
 * otherwise PB_ERR_UNSUPPORTED, before anything is enqueued. The first call on each device
 * looks up the array's address (cudaGetSymbolAddress) in the device's primary context,
 * which must stay alive for the rest of the process; make that first call before any
 * stream capture. All calls share the one array, which keeps the last call's contents
 * (each call leaves its flags cleared): calls that can overlap on the GPU (other streams,
 * other host threads) race on it and must be serialised by the caller. */
pb_status pb_gemm_bf16_static(int32_t M, int32_t N, int32_t K, const void* A, const void* B,
                              void* C, int* status, void* stream);

/* Sliding-window causal attention alone (section 1.1, eqs. (5)-(6)) from the scratch
 * layout's qk and vt buffers into columns [0, H) of `act` ([T, act_ld] bf16). */
pb_status pb_swa_attention(const pb_dims* dims, const void* qk, const void* vt, void* act,
                           int64_t act_ld, int* status, void* stream);

/* ------------------------------------------------------------------------------------
 * Positions: the norm of every query and key head and its rotation, in one pass between a
 * projection and pb_swa_attention, and its backward pass. For a head x of head_dim values,
 *   n = x / sqrt(mean x^2 + eps) * gamma               (skipped where gamma is NULL)
 *   (a, b) -> (a cos t - b sin t, a sin t + b cos t)   for every rotated pair of n,
 * t = position on the pair's axis x the pair's frequency. Computed in fp32, rounded once to
 * bf16; with frequencies up to 1 the angle is off by 2^-24 of a turn at most, at any position.
 * A normed head whose sum of squares passes fp32's range (values of 1e18 and more) comes out as
 * zero.
 * ---------------------------------------------------------------------------------- */

#define PB_ROPE_MAX_AXES 4

/* Pair i of the rot_dim / 2: values (i, i + rot_dim / 2), or (2i, 2i + 1). */
typedef enum pb_rope_pairing { PB_ROPE_HALVES = 0, PB_ROPE_ADJACENT = 1 } pb_rope_pairing;
/* Frequency of pair i: theta^(-2i / rot_dim) over all pairs, or on each axis from 1 on,
 * theta^(-j / n) for pair j of the axis's n. */
typedef enum pb_rope_ladder { PB_ROPE_SHARED = 0, PB_ROPE_PER_AXIS = 1 } pb_rope_ladder;

/* A rotation's plan, filled by pb_rope_init and only read by the calls: a plain value in
 * host memory that may be copied and shared between threads. */
typedef struct pb_rope {
  uint32_t magic;
  int32_t head_dim;
  int32_t rot_dim;
  int32_t pairing;
  int32_t axes;
  int32_t section_end[PB_ROPE_MAX_AXES];
  uint64_t turns[128]; /* frequency of each pair, 2^-64 turns a position */
} pb_rope;

/* head_dim: a multiple of 16, 16 to 256 (else PB_ERR_UNSUPPORTED). rot_dim: how many leading
 * values of a head are rotated, a multiple of 16, 0 to head_dim; the others only take the
 * norm. axes: 1 to 4; the first sections[0] pairs turn with the position on axis 0, the next
 * sections[1] with axis 1, ... (their sum is rot_dim / 2; NULL for one axis). inv_freq: host
 * array of rot_dim / 2 frequencies (radians a position), or NULL for theta's ladder. */
pb_status pb_rope_init(int32_t head_dim, int32_t rot_dim, int32_t pairing, int32_t axes,
                       const int32_t* sections, int32_t ladder, double theta,
                       const double* inv_freq, pb_rope* out);

/* The heads of every token, bf16: value d of head h at (b, s) is ptr[b batch_stride + s
 * seq_stride + h head_stride + d]. Strides in elements, multiples of 8, >= 0; ptr 16-byte
 * aligned; 2^48 values at most from the first to the last. [B, S, heads, dh], [B, heads, S, dh]
 * and the q or k columns of a [q | k | v] or of the scratch layout's [q | k] buffer are such
 * views. */
typedef struct pb_heads {
  void* ptr;
  int32_t heads;
  int64_t batch_stride;
  int64_t seq_stride;
  int64_t head_stride;
} pb_heads;

/* q_out = R(norm(q)), k_out = R(norm(k)). Either may be left out (input and result NULL).
 * gamma_q, gamma_k: [head_dim] bf16, or NULL for no norm. positions: int32 [axes, batch,
 * seq], any value (negative ones turn backwards); NULL is position s of each sequence, for
 * one axis. A result may be its own input (in place); otherwise results overlap neither
 * inputs nor one another (PB_ERR_INVALID_ARG where the strides do not show that). batch or
 * seq 0 does nothing; batch * seq < 2^31. */
pb_status pb_qk_norm_rope(const pb_rope* rope, int32_t batch, int32_t seq, const pb_heads* q,
                          const pb_heads* k, const void* gamma_q, const void* gamma_k, float eps,
                          const int32_t* positions, const pb_heads* q_out,
                          const pb_heads* k_out, void* stream);

/* Backward: from the inputs q, k of the forward call (read only where there is a gamma, else
 * they may be NULL) and the gradients dq, dk of its results, the gradients dq_out, dk_out of
 * its inputs (bf16) and of gamma_q, gamma_k (fp32 [head_dim]; NULL skips one; accumulate != 0
 * adds to what is there). A result may be its own dq (dk) or q (k). `scratch` (device,
 * 256-byte aligned, >= pb_qk_norm_rope_scratch_bytes) is needed where there is a gamma and
 * must not be used by another call that may run concurrently. dgamma_q, dgamma_k and scratch
 * overlap nothing else (one gamma for both: two gradients, added by the caller). Sums over
 * tokens and heads are taken in a fixed order. batch or seq 0 gives zero sums. With a gamma eps is
 * 2^-80 at least (rstd^3 has to stay in fp32's range for a head of zeros). */
pb_status pb_qk_norm_rope_scratch_bytes(size_t* bytes);
pb_status pb_qk_norm_rope_backward(const pb_rope* rope, int32_t batch, int32_t seq,
                                   const pb_heads* q, const pb_heads* k, const void* gamma_q,
                                   const void* gamma_k, float eps, const int32_t* positions,
                                   const pb_heads* dq, const pb_heads* dk,
                                   const pb_heads* dq_out, const pb_heads* dk_out,
                                   float* dgamma_q, float* dgamma_k, int32_t accumulate,
                                   void* scratch, size_t scratch_bytes, void* stream);

/* The step inside the block: every forward entry point on the handle then norms and rotates
 * the q and k heads of its projection before the attention (one launch more), pb_backward takes
 * their gradients back through it. dims.head_dim must be the plan's. gamma_q, gamma_k: bf16
 * [head_dim] device pointers, read by each call, or NULL; positions: int32 [axes, batch, seq]
 * device pointer, read by each call, or NULL for one axis. For training with a gamma, `saved`
 * (device, 256-byte aligned, batch * seq * 2 * hidden * 2 bytes) keeps the projection's q and k
 * between pb_forward_train and pb_backward, as their scratch does the rest; dgamma_q and
 * dgamma_k (fp32 [head_dim], or NULL) receive the gammas' gradients, by pb_backward's
 * accumulate. These three overlap nothing else of a training step. `saved` belongs to one
 * forward at a time. The handle remembers which `saved` and which scratch every forward filled,
 * whatever is set afterwards, and pb_backward through a norm is refused where the current
 * `saved` holds no forward, one with another scratch, or one of which a later forward has
 * overwritten either (two forwards in flight: two handles, or this call with another `saved`
 * before each forward and each backward; a captured forward counts when it is captured). The
 * struct is copied; what it points to must stay valid until the calls are done, and the same
 * from pb_forward_train to its pb_backward. NULL takes the step out again. In pb_trace_read its
 * time counts with the attention. */
typedef struct pb_block_rope {
  pb_rope rope;
  const void* gamma_q;
  const void* gamma_k;
  float eps;
  const int32_t* positions;
  void* saved;
  size_t saved_bytes;
  float* dgamma_q;
  float* dgamma_k;
} pb_block_rope;
pb_status pb_set_qk_norm_rope(pb_handle* h, const pb_block_rope* r);

/* ------------------------------------------------------------------------------------
 * A linear layer outside the block (an embedding's or a head's projection, an adapter, a
 * projection around pb_qk_norm_rope): bias, activation and residual in the product's epilogue,
 * any number of tokens from one on, and its backward pass.
 * ---------------------------------------------------------------------------------- */

typedef enum pb_dtype { PB_DTYPE_BF16 = 0, PB_DTYPE_FP16 = 1, PB_DTYPE_FP32 = 2 } pb_dtype;

/* w as [k, n] (the pages' Y = X W, as in pb_weights) or as [n, k]. */
typedef enum pb_weight_layout { PB_WEIGHT_IN_OUT = 0, PB_WEIGHT_OUT_IN = 1 } pb_weight_layout;

/* GELU: z Phi(z). GELU_TANH: z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2. SILU: z / (1 +
 * e^-z). RELU: max(z, 0), with derivative 0 at 0. Computed in fp32. GELU: Phi(z) is off by (1.5 z^2
 * + 24) 2^-24 of itself at most, in its left tail too; by 5e-7 where the result is bf16 and has
 * more than 32 rows (of GELU's value 5e-4 at z = -4, an eighth of its rounding, 1.6e-3 at -5).
 * GELU_TANH and SILU: off by (8 |s| + 9) 2^-24 and (1.5 |z| + 9) 2^-24 of the value at most, s =
 * 2 sqrt(2/pi) (z + 0.044715 z^3). */
typedef enum pb_activation {
  PB_ACT_NONE = 0,
  PB_ACT_GELU = 1,
  PB_ACT_GELU_TANH = 2,
  PB_ACT_SILU = 3,
  PB_ACT_RELU = 4
} pb_activation;

/* pre = x w + bias, y = activation(pre) + residual: x [m, k], w [k, n] or [n, k], bias [n],
 * residual and y [m, n]. x, w, bias and pre have dtype (PB_DTYPE_BF16 or _FP16), residual and
 * y either dtype or PB_DTYPE_FP32. Sums in fp32; pre (optional, for the backward pass) and y
 * are each rounded once from the fp32 value. bias, residual and pre may be NULL. Any m >= 0
 * (0 does nothing), n and k >= 1; ld*: row strides in elements, at least the row's length, a
 * multiple of 8 (of 4 for an fp32 matrix); pointers 16-byte aligned. Bytes between the rows are
 * neither used nor written. y may be the residual (same pointer, stride and type); no other
 * overlap of y or pre. */
typedef struct pb_linear_args {
  int32_t m, n, k;
  int32_t dtype;
  int32_t w_layout;
  int32_t activation;
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  const void* bias;
  const void* residual;
  int64_t ldr;
  int32_t residual_dtype;
  void* pre;
  int64_t ldp;
  void* y;
  int64_t ldy;
  int32_t y_dtype;
} pb_linear_args;

/* `scratch` (device, 256-byte aligned, >= pb_linear_scratch_bytes, or NULL) lets products be
 * split along k where their tiles do not fill the GPU; with NULL every tile is computed whole.
 * It needs no preparation; no operand or result may lie in it. Calls that share one must not
 * overlap on the GPU. `status` as in
 * pb_gemm_bf16. */
pb_status pb_linear_scratch_bytes(size_t* bytes);
pb_status pb_linear(const pb_linear_args* args, void* scratch, size_t scratch_bytes, int* status,
                    void* stream);

/* Backward of y = x w + bias for dy [m, n], the gradient of x w + bias: dx = dy w^T [m, k]
 * (dtype), dw = x^T dy in w's layout (fp32), db [n] = the sum of dy's rows (fp32, in a fixed
 * order); NULL skips one. Where x is activation(pre) of the layer before, give its pre [m, k]:
 * dx is then the gradient of pre, dy w^T * activation'(pre), ready as that layer's dy.
 * accumulate != 0 adds dw and db to what is there (dx is always overwritten; a value below
 * 2^-126 may count as zero in dw's addition); with m = 0 they are zero. The gradient of the
 * residual is dy itself. ld*, pointers, scratch and status as in pb_linear. Results overlap
 * nothing else. */
typedef struct pb_linear_grads {
  int32_t m, n, k;
  int32_t dtype;
  int32_t w_layout;
  int32_t activation; /* of pre; PB_ACT_NONE: pre is not read */
  int32_t accumulate;
  const void* dy;
  int64_t lddy;
  const void* x; /* read for dw */
  int64_t ldx;
  const void* w; /* read for dx */
  int64_t ldw;
  const void* pre;
  int64_t ldp;
  void* dx;
  int64_t lddx;
  float* dw;
  int64_t lddw;
  float* db;
} pb_linear_grads;
pb_status pb_linear_backward(const pb_linear_grads* args, void* scratch, size_t scratch_bytes,
                             int* status, void* stream);

/* out = dy * activation'(pre), [rows, cols] of dtype (PB_DTYPE_BF16 or _FP16), for an
 * activation whose result goes elsewhere than into a pb_linear. Row strides in elements,
 * multiples of 8; pointers 16-byte aligned; out may be dy or pre (same stride). */
pb_status pb_activation_backward(int64_t rows, int64_t cols, int32_t dtype, int32_t activation,
                                 const void* dy, int64_t lddy, const void* pre, int64_t ldp,
                                 void* out, int64_t ldo, void* stream);

/* ------------------------------------------------------------------------------------
 * Optimiser: what follows pb_backward in a training step.
 * ---------------------------------------------------------------------------------- */

/* Values of a tensor that share a scale in an 8-bit state. */
#define PB_ADAMW_BLOCK 256

/* One tensor of n values (contiguous; n = 0 is skipped), device pointers, 16-byte aligned:
 *   param       updated in place (pb_adamw_args.param_dtype)
 *   param_copy  bf16 copy of an fp32 param, written with it (pb_weights' type), or NULL
 *   grad        read (pb_adamw_args.grad_dtype)
 *   m, v        states, zero before the first step. 32 bits: fp32 m and v. 8 bits: E4M3 codes
 *               of m and of sqrt(v); value = code x scale of its PB_ADAMW_BLOCK values
 *   m_scale, v_scale  8 bits: fp32 [ceil(n / PB_ADAMW_BLOCK)], zero before the first step;
 *               32 bits: NULL */
typedef struct pb_adamw_tensor {
  int64_t n;
  void* param;
  void* param_copy;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float weight_decay;
} pb_adamw_tensor;

/* d_lr, d_step, d_grad_scale: device scalars read when the step runs, or NULL. d_lr and
 * d_step stand in for lr and step (a captured graph is replayed with other values);
 * every gradient is multiplied by *d_grad_scale, and where that is not finite the step
 * changes nothing. */
typedef struct pb_adamw_args {
  double lr;
  double beta1;
  double beta2;
  double eps;
  int64_t step; /* counts from 1 */
  int32_t param_dtype; /* PB_DTYPE_FP32 or PB_DTYPE_BF16 */
  int32_t grad_dtype;  /* PB_DTYPE_FP32 or PB_DTYPE_BF16 */
  int32_t state_bits;  /* 32 or 8 */
  const float* d_lr;
  const int32_t* d_step;
  const float* d_grad_scale;
} pb_adamw_args;

/* One AdamW step over all tensors (host array, read before the call returns):
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,
 *   param -= lr (weight_decay param + (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps))
 * in fp32, with m and v unrounded in the step that computes them. A gradient that is not finite, or
 * whose square is not (beyond 1.8e19), spoils its own value; the 8-bit states of the 255 that share
 * its scale then lose their smaller magnitudes, as next to any large value. No buffer that is written
 * may overlap another one (PB_ERR_INVALID_ARG: a tensor listed twice, too). */
pb_status pb_adamw(const pb_adamw_args* args, int32_t n_tensors, const pb_adamw_tensor* tensors,
                   void* stream);

/* The 2-norm of all tensors' gradients together (n and grad of each are read): out (device
 * fp32 [2]) = {norm, min(1, max_norm / (norm + 1e-6))}; the second is NaN where the norm is
 * not finite, so that as d_grad_scale it clips the step, or leaves it out. Squares are taken
 * in fp32 (gradients beyond 1e19 give an infinite norm), sums in a fixed order. `scratch`:
 * device, 256-byte aligned, >= pb_grad_norm_scratch_bytes, not shared with a call that may
 * run concurrently. */
pb_status pb_grad_norm_scratch_bytes(int32_t n_tensors, size_t* bytes);
pb_status pb_grad_norm(int32_t n_tensors, const pb_adamw_tensor* tensors, int32_t grad_dtype,
                       float max_norm, float* out, void* scratch, size_t scratch_bytes,
                       void* stream);

/* Failure-detection self-test: one thread waits, with the kernels' bounded-wait
 * routine, on an mbarrier that nothing arrives at. After `limit_ns` it records
 * PB_ERR_DEVICE_TIMEOUT in *status (a device int) and the kernel returns; no copy, MMA
 * or tensor memory is involved, so the context stays usable. */
pb_status pb_wait_probe(uint64_t limit_ns, int* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PB_H_ */
