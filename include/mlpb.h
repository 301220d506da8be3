/*
 * mlpb.h -- C ABI of libmlpb: the tensor-parallel transformer MLP block and
 * the sequence-parallel LayerNorm on one GB300 (sm_103a).
 *
 * What the library computes.  "Megatron-LM" source tour (pyshine.com/megatron-lm),
 * section "The Tensor-Parallel Primitives": fc1 is a ColumnParallelLinear (its
 * weight split along the output dimension; every rank sees the full input),
 * fc2 a RowParallelLinear (weight split along the input dimension, partial
 * sums all-reduced at the end), so the block needs one all-reduce.  Section
 * "The Transformer Stack": a fused bias-GELU sits between them; gated
 * variants (SwiGLU) multiply a gate by an up projection.  "Megatron-LM /
 * Megatron-Core" concept note, section "Key math / How it works": the
 * conjugate operators f (identity forward, all-reduce backward) and g
 * (all-reduce forward, identity backward), and sequence parallelism (LN split
 * along the sequence, gathers and reduce-scatters at the GEMM boundaries).
 *
 * The t tensor-parallel ranks are emulated on one device as partitions of the
 * weights.  The g all-reduce is the accumulation of all t shards' K-blocks
 * into one tensor-memory accumulator in the fc2 GEMM; the f all-reduce of the
 * backward is the same accumulation in the dX GEMM.  Sequence shards are
 * contiguous row blocks, so the SP gather / reduce-scatter are index ranges.
 *
 *   GELU:   Z = X W1^T + b1, A = gelu_tanh(Z), Y = A W2^T + b2
 *   SwiGLU: G = X Wg^T, U = X Wu^T, A = silu(G) * U, Y = A W2^T   (no biases)
 *
 * Conventions for every entry point
 *   - Pointers named as tensors are DEVICE pointers, 16-byte aligned, owned by
 *     the caller; the library never frees or retains them past the call.
 *   - bf16 means IEEE bfloat16 (2 bytes); all matrices are row-major.
 *   - Layouts (shard-major, as each tensor-parallel rank stores its slice):
 *       X, Xn, dY           [T][H] bf16
 *       W1 (GELU)           [t][Fs][H] bf16        W1 (SwiGLU) [t][2][Fs][H] (gate, up)
 *       b1                  [F] bf16 (shard i owns b1[i*Fs .. (i+1)*Fs))
 *       W2                  [t][H][Fs] bf16        b2 [H] bf16
 *       Z saved (GELU)      [T][F]  bf16, column i*Fs+j = shard i, feature j
 *       Z saved (SwiGLU)    [T][t][2][Fs] bf16 (G then U of each shard)
 *                           (both 8-bit codes and scales under MLPB_FLAG_CHECKPOINT8)
 *       A saved             [T][F]  bf16
 *       Y, dX               [T][H] fp32 (bf16 under MLPB_FLAG_BF16_OUT)
 *       dW1, dW2            fp32 in the layouts of W1, W2;  db1 [F], db2 [H] fp32
 *     where T = tokens, H = hidden, F = ffn, t = tp, Fs = F / t.
 *   - With T = 0 the per-row pointers (X, Y, Z/A saved, dY, dX, Xn, mean, rstd, dXn,
 *     workspace) may be NULL; forwards do nothing and backwards write zero parameter
 *     grads (weights, biases, gamma, beta), or leave them as they are when accumulating.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream).  Argument errors are returned synchronously and launch
 *     nothing.  Outputs are overwritten, except the parameter gradients of a handle
 *     created with MLPB_FLAG_ACCUMULATE_GRADS, which are added into.
 *   - A device-side bounded wait that expires (about one second) is recorded in
 *     a per-handle error word and reported by mlpb_last_device_error().
 *   - A handle may be used from one host thread at a time, and its calls must not
 *     overlap on the GPU (issue them on one stream, or order the streams).
 *     mlpb_backward runs part of its work on a second stream that the handle owns,
 *     forked from and joined back into `stream` with events, so all of its work is
 *     ordered before later work on `stream`.
 */
#ifndef MLPB_H_
#define MLPB_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *mlpb_stream_t; /* identical to cudaStream_t */

typedef enum {
  MLPB_OK = 0,
  MLPB_EINVAL = -1,       /* null / misaligned pointer, bad config value          */
  MLPB_EUNSUPPORTED = -2, /* shape outside the supported set (see mlpb_create)    */
  MLPB_ECUDA = -3,        /* a CUDA runtime call or launch failed                 */
  MLPB_ETIMEOUT = -4,     /* a device-side bounded wait expired (kernel bailed)   */
  MLPB_ENOMEM = -5        /* host allocation failed                               */
} mlpb_status;

typedef enum { MLPB_ACT_GELU_TANH = 0, MLPB_ACT_SWIGLU = 1 } mlpb_act;

/* mlpb_config.flags */
#define MLPB_FLAG_FAULT_INJECT 0x1u    /* test only: the first GEMM launch of the  \
                                          next forward skips one producer arrive, so \
                                          its consumers' bounded wait expires        */
/* Gradient-accumulation fusion ("The Tensor-Parallel Primitives": the linear layers'
 * shared autograd function accumulates weight gradients).  With this flag the parameter
 * gradients of mlpb_backward (dW1, dW2, db1, db2) and mlpb_layernorm_sp_bwd (dgamma,
 * dbeta) are ADDED to what their fp32 buffers hold (main-grad buffers carried across
 * micro-batches) instead of overwriting them; the weight-gradient GEMM epilogues read,
 * add and write each fp32 element once, the bias/LN parameter reductions add their final
 * sums.  The caller zeroes the buffers before the first micro-batch.  With T = 0 the
 * buffers are left as they are.  dX (an activation gradient) is always overwritten. */
#define MLPB_FLAG_ACCUMULATE_GRADS 0x2u
/* Selective activation recomputation (the concept note's "Key math": activation
 * recomputation, selective granularity).  With this flag mlpb_backward does not read
 * the forward's A: the dgrad GEMM's epilogue, which already reads the saved Z (or G, U)
 * for the activation derivative, also rewrites A = act(Z) into the Asaved buffer, and
 * the dW2 GEMM runs after it on that A.  Only Z (G, U) must survive from the forward to
 * the backward; the T*F bf16 A buffer can be scratch shared with other work (the
 * forward writes it for fc2, the backward rewrites it).  A is recomputed from the
 * bf16-rounded Z, so dW2 can differ from the stored-A path by bf16 rounding. */
#define MLPB_FLAG_RECOMPUTE_ACT 0x4u
/* FP8 GEMMs ("Why Megatron-LM Matters" / "Key Features" of the onegen.ai page: mixed
 * precision down to FP8; the concept note's "Key math": FP8 through Transformer Engine).
 * All six GEMMs of mlpb_forward / mlpb_backward run on E4M3 operands (tcgen05
 * kind::f8f6f4, fp32 accumulation) with per-tensor current scaling: each operand tensor
 * (X, W1, W2, A, dY, dZ; every shard at once) gets the power-of-two scale of
 * mlpb_quantize_e4m3 from its own absolute maximum, and each GEMM rescales its sums by
 * the inverse of its two operands' scales.  Everything else keeps the bf16 path's
 * precision: Z (G, U), A and dZ are bf16, Y, dX and the parameter gradients fp32, the
 * bias sums and the LayerNorm unchanged.  The workspace (mlpb_workspace_size) then also
 * holds the E4M3 copies and is required by mlpb_forward too.  Requires F/tp % 16 == 0;
 * not combined with MLPB_FLAG_RECOMPUTE_ACT. */
#define MLPB_FLAG_FP8 0x8u
/* bf16 outputs (the mixed precision of the parallel linears in "The Tensor-Parallel
 * Primitives": activations and their gradients travel in bf16).  With this flag Y
 * (mlpb_forward, mlpb_branch_forward) and dX (mlpb_backward, mlpb_layernorm_sp_bwd,
 * mlpb_branch_backward) are bf16 [T][H] instead of fp32, and mlpb_layernorm_sp_bwd reads
 * its dXn as bf16 (what mlpb_backward then writes).  The sums are the same fp32 values
 * as without the flag, rounded once to bf16 (nearest, ties to even) when stored; the
 * parameter gradients stay fp32.  Halves those tensors' bytes, at the cost of one bf16
 * rounding of Y and dX (up to 2^-9 of each value). */
#define MLPB_FLAG_BF16_OUT 0x10u
/* Emulated sequence-parallel exchange as copies (requires seq_parallel_ln; "The
 * Tensor-Parallel Primitives": with sequence parallelism the linear layers all-gather the
 * sequence-sharded activations in front of the column-parallel GEMM and reduce-scatter
 * after the row-parallel one, and the conjugates in the backward).  Without the flag the
 * gathered tensor is the row-block layout itself (shard s owns rows [s T/t, (s+1) T/t))
 * and no byte moves.  With it, mlpb_forward first copies the input X into a gathered
 * buffer in the workspace and writes fc2's output there before copying its rows out to Y
 * (the scatter; the reduction over shards happened in the accumulator); mlpb_backward
 * gathers X and dY and scatters dX the same way.  Results are bit for bit those of the
 * view; the copies' bytes are reported apart from the algorithmic bytes (timing records
 * "sp_gather_x", "sp_gather_dy", "sp_scatter_y", "sp_scatter_dx").  mlpb_forward then
 * needs the workspace; the workspace holds 8*T*H more bytes. */
#define MLPB_FLAG_EMULATE_COPIES 0x20u
/* 8-bit activation checkpoints ("Key math" of the concept note: activation memory is what
 * recomputation saves).  With this flag the forward saves Z (G, U) for the backward as
 * 8-bit codes with one power-of-two scale for each 32 features of a row (the format of
 * mlpb_act8_save, of the bf16-rounded Z), written in fc1's epilogue and read in the dgrad
 * GEMM's: Zsaved is T*F1 code bytes [T][F1] followed by T*F1/32 scale bytes [T][F1/32]
 * (F1 = F for GELU, 2F for SwiGLU; mlpb_saved_size gives the sum), 0.52 times the bf16 Z.
 * As under MLPB_FLAG_RECOMPUTE_ACT, which it implies, A is rewritten by the backward, here
 * from the decoded Z, and only Zsaved must survive between the passes.  The forward's Y is bit
 * for bit that of the block without the flag; the gradients are those of the decoded Z.
 * Requires F/tp % 32 == 0; not combined with MLPB_FLAG_FP8. */
#define MLPB_FLAG_CHECKPOINT8 0x100u

typedef struct {
  int64_t tokens;          /* T: rows of X; multiple of 128 (0 allowed)           */
  int64_t hidden;          /* H: multiple of 64, >= 64                            */
  int64_t ffn;             /* F: divisible by tp, with F/tp a multiple of 8       */
  int32_t tp;              /* t: emulated tensor-parallel degree, 1..1024         */
  int32_t act;             /* mlpb_act                                            */
  int32_t has_bias;        /* GELU only: b1, b2 present (SwiGLU requires 0)       */
  int32_t seq_parallel_ln; /* LN entry points enabled; requires T % t == 0        */
  float ln_eps;            /* LayerNorm epsilon (inside the square root)          */
  uint32_t flags;          /* MLPB_FLAG_*                                         */
} mlpb_config;

typedef struct mlpb_handle mlpb_handle; /* opaque; owns no tensors */

/* Per-kernel timing record (filled when timing is enabled). */
typedef struct {
  char name[32];  /* kernel name, e.g. "fc1_gelu", "colsum_db2"                  */
  float ms;       /* device time between CUDA events recorded around the launch   */
  double flops;   /* algorithmic GEMM flops of the launch (0 for memory kernels)  */
  double bytes;   /* algorithmic HBM bytes of the launch (minimum reads + writes) */
  int32_t kernels; /* CUDA kernels launched inside this record (e.g. 2 for a       \
                      two-pass reduction)                                          */
} mlpb_kernel_time;

/* Validates *cfg, queries the current device and allocates the 4-byte device
 * error word.  Returns EINVAL for a null argument or an out-of-range field,
 * EUNSUPPORTED for shapes outside: T % 128 == 0, H % 64 == 0 and H >= 64,
 * F % tp == 0 and (F/tp) % 8 == 0, SwiGLU without bias, SP with T % tp == 0
 * and H <= 16384.  On success *out owns host state only. */
mlpb_status mlpb_create(const mlpb_config *cfg, mlpb_handle **out);

/* Frees the handle and its error word.  NULL is ignored. */
void mlpb_destroy(mlpb_handle *h);

/* Bytes of device scratch the caller passes as `workspace` to mlpb_forward,
 * mlpb_backward and mlpb_layernorm_sp_bwd (it holds dZ [T][F1] bf16, with a bias the
 * db1 column sums of each 32-row group of dZ that the dgrad epilogue writes, two regions
 * of fp32 partial tiles for the K-range split of a GEMM's last wave -- dX and dW1 run at
 * once on two streams -- a transposed copy of W2 ([F][H] bf16, the dgrad GEMM's operand)
 * (not under MLPB_FLAG_FP8), with a bias db2's column sums over row ranges of dY, and,
 * under MLPB_FLAG_FP8, the E4M3 operand copies and their amax words). */
mlpb_status mlpb_workspace_size(const mlpb_handle *h, size_t *bytes);

/* Bytes of the saved activations: z_bytes for Z (GELU, T*F*2) or G|U (SwiGLU,
 * T*2F*2), the codes and scales under MLPB_FLAG_CHECKPOINT8 (T*F1 + T*F1/32); a_bytes
 * for A (T*F*2). */
mlpb_status mlpb_saved_size(const mlpb_handle *h, size_t *z_bytes, size_t *a_bytes);

/* Forward of the block ("The Tensor-Parallel Primitives" and "The Transformer
 * Stack" of the source tour; f and g of "Key math").  fc1 over all t column
 * shards with the fused bias+GELU or SwiGLU epilogue writes Zsaved and Asaved;
 * fc2 accumulates all t row shards into one accumulator per output tile (the
 * emulated g all-reduce) and adds b2 once, writing Y [T][H] fp32.  b1 and b2
 * must be NULL when has_bias is 0.  `workspace` is NULL or mlpb_workspace_size() bytes:
 * when given, fc2 uses it to split the K range of the tiles of its last, partly filled
 * wave across idle SM pairs (their partial sums are added by a fixup kernel, in a fixed
 * order); it is required under MLPB_FLAG_FP8. */
mlpb_status mlpb_forward(mlpb_handle *h, const void *X, const void *W1, const void *b1,
                         const void *W2, const void *b2, void *Y, void *Zsaved,
                         void *Asaved, void *workspace, mlpb_stream_t stream);

/* Backward of the block for an upstream gradient dY [T][H] bf16.  g backward is
 * the identity (every shard reads the same dY); dZ = (dY W2_i) * act'(.) per
 * shard; dW2_i = dY^T A_i; dW1_i = dZ_i^T X; db1 = sum_t dZ (column sums of the bf16
 * dZ taken in the dgrad epilogue, then added in row order); db2 = sum_t dY (column sums
 * over row ranges taken in the launch that transposes W2 -- under MLPB_FLAG_FP8 in one of
 * its own -- then added in row-range order);
 * dX = sum_i dZ_i W1_i with the sum over shards accumulated in one tensor-memory
 * accumulator (the emulated f all-reduce).  db1/db2 must be NULL without bias.
 * `workspace` must hold mlpb_workspace_size() bytes.  Asaved is read only (the
 * forward's A), except under MLPB_FLAG_RECOMPUTE_ACT, where it is scratch that the
 * backward writes before reading. */
mlpb_status mlpb_backward(mlpb_handle *h, const void *X, const void *W1, const void *W2,
                          const void *Zsaved, void *Asaved, const void *dY,
                          void *dX, float *dW1, float *dW2, float *db1, float *db2,
                          void *workspace, mlpb_stream_t stream);

/* Sequence-parallel LayerNorm forward ("The Tensor-Parallel Primitives": norms
 * run on sequence-sharded activations).  Shard s owns rows [s*T/t, (s+1)*T/t);
 * each row r gets mean[r], rstd[r] = 1/sqrt(var + eps) (biased variance) and
 * Xn[r] = (X[r]-mean)*rstd*gamma + beta in bf16.  The emulated all-gather is
 * the row-block layout of Xn itself: shard s writes rows s*T/t.. of the gathered
 * tensor that fc1 reads, so no copy is made.
 * X, gamma, beta bf16; mean, rstd [T] fp32.  Requires seq_parallel_ln. */
mlpb_status mlpb_layernorm_sp_fwd(mlpb_handle *h, const void *X, const void *gamma,
                                  const void *beta, void *Xn, float *mean, float *rstd,
                                  mlpb_stream_t stream);

/* Sequence-parallel LayerNorm backward for dXn [T][H] fp32 (the dX output of
 * mlpb_backward run on Xn; bf16 under MLPB_FLAG_BF16_OUT).  dX [T][H] fp32 (bf16 under
 * MLPB_FLAG_BF16_OUT; it may be the dXn buffer itself); dgamma, dbeta [H] fp32 are the sum
 * over shards of each shard's partials (the all-reduce the SP layout implies).
 * `workspace` must hold mlpb_workspace_size() bytes. */
mlpb_status mlpb_layernorm_sp_bwd(mlpb_handle *h, const void *X, const void *gamma,
                                  const float *mean, const float *rstd, const void *dXn,
                                  void *dX, float *dgamma, float *dbeta, void *workspace,
                                  mlpb_stream_t stream);

/* Pre-norm MLP branch of a transformer layer ("The Transformer Stack": the layer runs
 * its MLP branch on the layer-normalised input and adds the branch input back through a
 * residual connection; dropout is left out), sequence-parallel:
 *     Y = X + MLP(LN(X))        (Y [T][H] fp32, bf16 under MLPB_FLAG_BF16_OUT; X, gamma,
 *                                beta bf16)
 * Runs mlpb_layernorm_sp_fwd (writes Xn, mean, rstd, kept for the backward) and the
 * forward of mlpb_forward on Xn, with X added to every output element in fc2's epilogue
 * after b2 (the residual of a row lives on the sequence shard that owns the row).
 * Requires seq_parallel_ln.  Arguments as in the two calls it combines. */
mlpb_status mlpb_branch_forward(mlpb_handle *h, const void *X, const void *gamma,
                                const void *beta, const void *W1, const void *b1,
                                const void *W2, const void *b2, void *Y, void *Xn,
                                float *mean, float *rstd, void *Zsaved, void *Asaved,
                                void *workspace, mlpb_stream_t stream);

/* Backward of mlpb_branch_forward for an upstream gradient dY [T][H] bf16:
 *     dX = dY + LN'(dXn),  dXn = the MLP backward's input gradient on Xn
 * plus dW1, dW2, db1, db2 (as mlpb_backward, on Xn) and dgamma, dbeta (as
 * mlpb_layernorm_sp_bwd).  dXn is formed in the dX buffer and the LayerNorm backward
 * rewrites it in place with the residual gradient dY added in its epilogue, so the call
 * needs no [T][H] buffer beyond dX.  `workspace` holds mlpb_workspace_size() bytes.
 * Honours MLPB_FLAG_ACCUMULATE_GRADS for the parameter gradients. */
mlpb_status mlpb_branch_backward(mlpb_handle *h, const void *X, const void *gamma,
                                 const void *W1, const void *W2, const void *Xn,
                                 const float *mean, const float *rstd, const void *Zsaved,
                                 void *Asaved, const void *dY, void *dX, float *dW1,
                                 float *dW2, float *db1, float *db2, float *dgamma,
                                 float *dbeta, void *workspace, mlpb_stream_t stream);

/* Synchronises `stream`, reads and clears the device error word.  Returns
 * MLPB_ETIMEOUT if a bounded wait expired since the last call, MLPB_ECUDA if
 * the stream reported an error, else MLPB_OK. */
mlpb_status mlpb_last_device_error(mlpb_handle *h, mlpb_stream_t stream);

/* Enables (1) or disables (0) per-kernel CUDA-event timing on the handle.  While it is
 * on, mlpb_backward issues all of its kernels on the caller's stream, one after the other,
 * so that every recorded interval belongs to one kernel. */
mlpb_status mlpb_enable_timing(mlpb_handle *h, int enable);

/* Copies up to `capacity` timing records of the launches since the last read
 * (waiting on their events), sets *count, and clears the list. */
mlpb_status mlpb_read_timings(mlpb_handle *h, mlpb_kernel_time *out, int capacity, int *count);

/* Column sums out[c] = sum_r in[r][c] of a bf16 [rows][cols] matrix into fp32 -- the
 * bias-gradient reduction of mlpb_backward (db2 = sum_t dY, db1 = sum_t dZ) -- for
 * callers that cannot allocate device memory where they need it (code under a memory
 * manager that owns all of the GPU's memory, or inside that manager's own callbacks).
 * The pages have no counterpart: this is an allocation-free variant of the same kernels.
 * It needs no handle and no workspace: its scratch is a fixed 4 MiB device array inside
 * the library (held by every GPU that loads the library until the process exits).
 * Each call looks up that array's device address on the current device (a host-side
 * lookup, so a device reset or a re-created context cannot leave a stale address); the
 * first call on a device also loads the library's device code there, so make it before
 * any stream capture.  Every call shares the one array and the array keeps the last
 * call's partial sums; each call writes every partial it reads before reading it, so
 * nothing needs clearing.  Calls whose kernels overlap on the GPU (other streams, other
 * host threads) race on the array and must be serialised by the caller.
 * Requires cols % 8 == 0 and cols <= 1048576 (one split of fp32 partials must fit the
 * scratch; larger widths return MLPB_EUNSUPPORTED), 16-byte aligned `in` and `out`;
 * rows may be 0 (out becomes zeros, `in` may then be NULL).  Allocates nothing. */
mlpb_status mlpb_bias_grad_noalloc(const void *in, int64_t rows, int64_t cols, float *out,
                                   mlpb_stream_t stream);

/* E4M3 quantization of a bf16 tensor [batches][rows][cols] with one power-of-two scale
 * for the whole tensor (the FP8 recipe of MLPB_FLAG_FP8; "Why Megatron-LM Matters" and
 * "Key Features" of the onegen.ai page name FP8 mixed precision, the concept note's "Key
 * math" FP8 through Transformer Engine).  With amax the largest |x| and k the largest
 * integer such that amax * 2^k <= 448, each code is e4m3(x * 2^k), round to nearest even
 * (x * 2^k is exact).  Writes q [batches][rows][cols] and/or qt [batches][cols][rows]
 * (the transposed codes; either may be NULL, not both), *amax = the fp32 bit pattern of
 * the tensor's largest magnitude (device word, overwritten), and *scale_exp = k (device
 * int, may be NULL).  rows % 16 == 0, cols % 16 == 0, 16-byte aligned tensors, 4-byte
 * aligned words.  Allocates nothing; no handle. */
mlpb_status mlpb_quantize_e4m3(const void *in, int64_t batches, int64_t rows, int64_t cols,
                               void *q, void *qt, uint32_t *amax, int32_t *scale_exp,
                               mlpb_stream_t stream);

/* 8-bit activation checkpoints: fc1's output saved as 8-bit codes, and the activation's
 * backward from them -- the format and arithmetic of MLPB_FLAG_CHECKPOINT8 for callers whose
 * GEMMs are their own.
 *   act = MLPB_ACT_GELU_TANH: Z [T][F], A = gelu_tanh(Z); tp only has to divide F.
 *   act = MLPB_ACT_SWIGLU: Z [T][tp][2][Fs] (G then U of each shard), A = silu(G) * U [T][F].
 * Blocks of 32 consecutive features of a row's segment -- all F for GELU, each shard's Fs
 * gate and Fs up features for SwiGLU; a segment's last block may be shorter -- share one
 * scale byte.  With amax the block's largest magnitude and k the largest integer, at most
 * 126, with amax 2^k <= 127 (k = 0 for zeros), each code is z 2^k rounded to the nearest
 * integer, ties to even, and the scale byte is 127 - k: a code c stands for c 2^(byte - 127),
 * exactly.  (bf16's largest value would become 64 2^122, past the range: the block that holds
 * it has k = -121 and ties towards zero, 127 for that value.)  A block that holds an infinity or
 * a NaN has the byte 255 and stands for NaN throughout (its codes mean nothing).
 *
 * mlpb_act8_scales: *per_row = scale bytes of a row (ceil(F / 32) for GELU,
 * 2 tp ceil(Fs / 32) for SwiGLU).
 * mlpb_act8_save: writes codes [T][F1] (layout of Z), scales [T][per_row] and, unless A is
 * NULL, A = act(Z) in bf16, from the bf16 Z itself.
 * mlpb_act8_grad: with z the values the codes stand for, writes dZ = dA act'(z) (layout of Z,
 * bf16) and, unless A is NULL, A = act(z), for an upstream gradient dA [T][F] bf16.
 * F % tp == 0 and (F/tp) % 8 == 0 (else MLPB_EUNSUPPORTED); tensors 16-byte aligned, scales
 * of any alignment; outputs overlap no input.  tokens = 0 does nothing.  No handle, no
 * workspace; allocate nothing. */
mlpb_status mlpb_act8_scales(int32_t act, int64_t ffn, int32_t tp, int64_t *per_row);
mlpb_status mlpb_act8_save(int32_t act, int64_t tokens, int64_t ffn, int32_t tp, const void *Z,
                           void *A, void *codes, void *scales, mlpb_stream_t stream);
mlpb_status mlpb_act8_grad(int32_t act, int64_t tokens, int64_t ffn, int32_t tp, const void *dA,
                           const void *codes, const void *scales, void *dZ, void *A,
                           mlpb_stream_t stream);

/* The join between two blocks of a transformer's residual stream, in one pass each way: the
 * norm after a block, its gate, the residual scale, the sum, and the norm before the next
 * block ("The Transformer Stack": norms, residual connections around each branch).
 *     P    = norm_post(Y)                          (P = Y with MLPB_NORM_NONE)
 *     Xout = res_scale * X + gate[group] * P       (gate, res_scale: 1 where absent)
 *     Xn   = norm_pre(Xout)                        (not written with MLPB_NORM_NONE)
 * LAYER: (x - mean) / sqrt(var + eps) * gamma + beta, biased variance;  RMS: x / sqrt(mean x^2
 * + eps) * gamma, no beta.  norm_pre is that of Xout as stored.  A gate is one [hidden] row
 * for each of gate_groups contiguous row blocks of tokens / gate_groups rows (1: one gate for
 * all; the number of sequences: one for each; tokens: one for each token).
 * Without a block (has_block 0) the call is norm_pre alone, Xn = norm_pre(X): the norm in front
 * of a first block. */
typedef enum { MLPB_NORM_NONE = 0, MLPB_NORM_LAYER = 1, MLPB_NORM_RMS = 2 } mlpb_norm;

/* mlpb_join_config.flags */
#define MLPB_JOIN_STREAM_F32 0x1u       /* X, Xout, dXout, dX are fp32 (else bf16)           */
#define MLPB_JOIN_BLOCK_F32 0x2u        /* Y, dXn are fp32 (else bf16)                       */
#define MLPB_JOIN_ACCUMULATE_GRADS 0x4u /* parameter gradients are added into, as under      \
                                           MLPB_FLAG_ACCUMULATE_GRADS                        */

typedef struct {
  int64_t tokens;      /* rows (0 allowed), below 2^31                                       */
  int64_t hidden;      /* a multiple of 8, at most 16384                                     */
  int64_t gate_groups; /* 0: no gate; else a divisor of tokens                               */
  int32_t has_block;   /* 0: norm_pre alone (no post norm, gate or residual scale then)      */
  int32_t post_norm;   /* mlpb_norm                                                          */
  int32_t pre_norm;    /* mlpb_norm                                                          */
  float eps;           /* of both norms, inside the root                                     */
  uint32_t flags;      /* MLPB_JOIN_*                                                        */
} mlpb_join_config;

/* Bytes of the workspace of mlpb_join_bwd on the current device (the parameter gradients'
 * partial sums). */
mlpb_status mlpb_join_workspace_size(const mlpb_join_config *cfg, size_t *bytes);

/* Forward.  X, Y [tokens][hidden]; res_scale one fp32 on the device, or NULL; gate
 * [gate_groups][hidden], gamma_* and beta_* [hidden] bf16, given exactly where the
 * configuration has them; Xout like X; Xn bf16; stats [tokens][4] fp32: mean and 1/sqrt(...)
 * of Y's row, then of Xout's (zeros where there is no norm; the mean of an RMS norm is 0), for
 * the backward.  Xout may be X's buffer; no other output may overlap an input.  Without a
 * block Y, Xout and res_scale are NULL.  No workspace; 16-byte aligned tensors. */
mlpb_status mlpb_join_fwd(const mlpb_join_config *cfg, const void *X, const void *Y,
                          const float *res_scale, const void *gate, const void *gamma_post,
                          const void *beta_post, const void *gamma_pre, const void *beta_pre,
                          void *Xout, void *Xn, float *stats, mlpb_stream_t stream);

/* Backward, for the gradients dXout of Xout (NULL: zero, with a pre norm) and dXn of Xn (NULL
 * without a pre norm):
 *     dh = dXout + norm_pre'(dXn),  dX = res_scale dh,  dY = norm_post'(gate dh)  (dY bf16)
 * and, in fp32, dres_scale (one value), dgate [gate_groups][hidden], dgamma_*, dbeta_*
 * [hidden], each given exactly where its parameter is.  Sums run in a fixed order: the same
 * bits every run.  Xout and stats are the forward's (without a block Xout is X itself, and X,
 * Y, dY are NULL).  Y is read with a post norm or a gate, X with a res_scale; either may be
 * NULL otherwise.  dX may be dXout's buffer; no other output may overlap an input.  tokens =
 * 0 writes zero parameter gradients.  `workspace`: mlpb_join_workspace_size() bytes, not
 * shared by calls that overlap. */
mlpb_status mlpb_join_bwd(const mlpb_join_config *cfg, const void *X, const void *Y,
                          const void *Xout, const float *stats, const float *res_scale,
                          const void *gate, const void *gamma_post, const void *beta_post,
                          const void *gamma_pre, const void *dXout, const void *dXn, void *dX,
                          void *dY, float *dres_scale, float *dgate, float *dgamma_post,
                          float *dbeta_post, float *dgamma_pre, float *dbeta_pre,
                          void *workspace, mlpb_stream_t stream);

/* A mixture-of-experts MLP for a few tokens (decoding), in one launch: the block's MLP with
 * `experts` experts in the place of its shards, of which every token takes `topk`.
 *     l   = X Wr^T                                  (to about 2^-40 of sum |x||wr|)
 *     ids = the topk experts of largest l, descending, equal ones by index (NaN last)
 *     w   = softmax(l) at ids, over all experts; divided by its sum over ids with `normalize`
 *     Y   = sum over a token's experts of w W2_e act(W1_e x)       (no biases)
 * Every routed expert's weights are read once for all of its tokens.  act(W1_e x) is rounded to
 * bf16 (the second product's operand); every other sum is fp32. */
#define MLPB_MOE_FAULT_INJECT 0x2u /* mlpb_moe_config.flags, test only: the handle's first launch \
                                      never fills one stage of a ring, its second leaves out an \
                                      arrival at a barrier of the grid; both end by their waits' \
                                      limit (MLPB_ETIMEOUT), and the third is an ordinary one    */

typedef struct {
  int32_t max_tokens; /* most tokens of a call, 1..64                                         */
  int32_t hidden;     /* a multiple of 8                                                      */
  int32_t ffn;        /* features of one expert, a multiple of 8                              */
  int32_t experts;    /* 1..256                                                               */
  int32_t topk;       /* 1..16, at most experts                                               */
  int32_t act;        /* mlpb_act                                                             */
  int32_t normalize;  /* 1: the weights of a token sum to 1                                   */
  uint32_t flags;     /* 0, or MLPB_MOE_FAULT_INJECT                                          */
} mlpb_moe_config;

typedef struct mlpb_moe mlpb_moe; /* opaque; owns a few device words and no tensors */

/* Validates *cfg and allocates the handle on the current device; EINVAL for null arguments or
 * values out of range, EUNSUPPORTED for sizes outside those above (or hidden, ffn > 2^20). */
mlpb_status mlpb_moe_create(const mlpb_moe_config *cfg, mlpb_moe **out);
void mlpb_moe_destroy(mlpb_moe *h);

/* Bytes of the workspace of mlpb_moe_forward (logits, activations and unweighted outputs of
 * max_tokens). */
mlpb_status mlpb_moe_workspace_size(const mlpb_moe *h, size_t *bytes);

/* Forward of `tokens` <= max_tokens rows (0 does nothing).  X [tokens][hidden]; Wr
 * [experts][hidden]; W1 [experts][2][ffn][hidden] (gate, up) for SwiGLU, [experts][ffn][hidden]
 * for GELU; W2 [experts][hidden][ffn]; Y [tokens][hidden]: all bf16, 16-byte aligned.  ids
 * [tokens][topk] int32 and weights [tokens][topk] fp32 receive the routing.  The launch is
 * cooperative (one CTA on every SM, which synchronise).  The current device must be the
 * handle's.  Calls of one handle, or with one workspace, must not overlap on the GPU (use one
 * stream, or a handle and a workspace for each; a captured graph counts as its call, and the
 * handle has to outlive it). */
mlpb_status mlpb_moe_forward(mlpb_moe *h, int64_t tokens, const void *X, const void *Wr,
                             const void *W1, const void *W2, void *Y, int32_t *ids,
                             float *weights, void *workspace, mlpb_stream_t stream);

/* As mlpb_last_device_error, for a mixture-of-experts handle: MLPB_ETIMEOUT if a bounded wait
 * of its launches on `stream` so far expired since the last call.  The current device must be
 * the handle's (EINVAL). */
mlpb_status mlpb_moe_last_device_error(mlpb_moe *h, mlpb_stream_t stream);

/* Block-scaled E4M3: one power-of-two scale for each 128 consecutive columns of a row, or for each
 * 128 x 128 block (`square`, for weights, whose codes and transposed codes then are the same).
 * With amax the block's largest magnitude and k the largest integer, at most 126, with amax 2^k
 * <= 448 (k = 0 for zeros), a code is e4m3(x 2^k), nearest, ties to even, and the scale byte is
 * 127 - k: a code c stands for c 2^(byte - 127), exactly.  A block that holds an infinity or a NaN
 * has the byte 255 and stands for NaN throughout.
 *   codes   [rows][ld] bytes, ld = columns rounded up to 16 (mlpb_b128_sizes); the pad holds 0 (NaN
 *           in a block that holds one)
 *   scales  byte of (row, kb = column / 128) at
 *             ((kb / 4) * ceil(rows / 128) + row / 128) * 512
 *               + (row % 32) * 16 + (row % 128) / 32 * 4 + kb % 4,
 *           the order in which the tensor cores take them; bytes past the end hold 127
 *
 * mlpb_b128_sizes: *ld and the bytes of the scales of a [rows][cols] matrix.
 * mlpb_b128_quantize: x [rows][cols], bf16 or (x_f32 = 1) fp32, to codes q and scales qs of x
 * and/or codes qt and scales qts of its transpose [cols][rows] (blocks along its own columns);
 * either pair may be NULL, not both.  cols % 8 == 0, both at most 2^20 (else MLPB_EUNSUPPORTED);
 * tensors 16-byte aligned; outputs overlap no input.  rows = 0 does nothing.  No handle, no
 * workspace; allocates nothing. */
mlpb_status mlpb_b128_sizes(int64_t rows, int64_t cols, int64_t *ld, size_t *scale_bytes);
mlpb_status mlpb_b128_quantize(const void *x, int32_t x_f32, int64_t rows, int64_t cols,
                               int32_t square, void *q, void *qs, void *qt, void *qts,
                               mlpb_stream_t stream);

/* A linear layer on block-scaled E4M3 operands, forward and backward ("Why Megatron-LM Matters" /
 * "Key Features": mixed precision down to FP8; finer than the one scale for a tensor of
 * MLPB_FLAG_FP8, at the same rate: the tensor cores apply the scales):
 *     Y = Xq Wq^T,   dX = dYq Wq,   dW = (dY^T)q ((X^T)q)^T
 * where (.)q rounds blocks of 128 along the axis that is summed over, and W blocks of 128 x 128.
 * Products of codes are exact, sums fp32, which the tensor cores cut off instead of rounding: by
 * 6e-7 of a sum of 8192 products, in chunks of which an fp32 result is summed, and in proportion in
 * a longer sum of a bf16 result. */
#define MLPB_LINEAR8_OUT_F32 0x1u      /* Y and dX are fp32 (else bf16)                       */
#define MLPB_LINEAR8_FAULT_INJECT 0x2u /* test only, as MLPB_FLAG_FAULT_INJECT: the first     \
                                          product's first stage is never filled               */

typedef struct {
  int64_t max_tokens; /* most rows of a call, 1..2^20                  */
  int64_t inputs;     /* K: a multiple of 8, at most 2^20              */
  int64_t outputs;    /* N: a multiple of 8, at most 2^20              */
  uint32_t flags;     /* MLPB_LINEAR8_*                                */
} mlpb_linear8_config;

typedef struct mlpb_linear8 mlpb_linear8; /* opaque; owns a device word and no tensors */

/* Validates *cfg and allocates the handle on the current device; EINVAL for null arguments or
 * values out of range, EUNSUPPORTED for sizes outside those above. */
mlpb_status mlpb_linear8_create(const mlpb_linear8_config *cfg, mlpb_linear8 **out);
void mlpb_linear8_destroy(mlpb_linear8 *h);

/* Bytes of the workspace of the calls below (codes and scales of X, or of dY and dY^T). */
mlpb_status mlpb_linear8_workspace_size(const mlpb_linear8 *h, size_t *bytes);

/* Forward of `tokens` <= max_tokens rows (0 does nothing): X [tokens][inputs] bf16; Wq, Ws the
 * codes and scales of W [outputs][inputs] (mlpb_b128_quantize, square); Y [tokens][outputs].
 * Xt, Xts, NULL in serving, receive codes and scales of X^T [inputs][tokens] for the backward.
 * Outputs overlap no input, here and in the backward.
 * The current device must be the handle's.  Calls that share a workspace must not overlap on the
 * GPU (a captured graph counts as its call, and the handle has to outlive it). */
mlpb_status mlpb_linear8_forward(mlpb_linear8 *h, int64_t tokens, const void *X, const void *Wq,
                                 const void *Ws, void *Y, void *Xt, void *Xts, void *workspace,
                                 mlpb_stream_t stream);

/* Backward for dY [tokens][outputs] bf16, with as many tokens as the forward that wrote Xt and
 * Xts; Wt, Wts the codes and scales of W^T [inputs][outputs] of the same quantization.  dX
 * [tokens][inputs] or dW [outputs][inputs] fp32 may be NULL, not both (nor are their operands
 * read then).  accumulate: dW is added into (by additions that take subnormal values as zeros).
 * tokens = 0 writes a zero dW, or leaves it as it is
 * when accumulating. */
mlpb_status mlpb_linear8_backward(mlpb_linear8 *h, int64_t tokens, const void *dY, const void *Wt,
                                  const void *Wts, const void *Xt, const void *Xts, void *dX,
                                  float *dW, int32_t accumulate, void *workspace,
                                  mlpb_stream_t stream);

/* As mlpb_moe_last_device_error, for a linear layer's handle. */
mlpb_status mlpb_linear8_last_device_error(mlpb_linear8 *h, mlpb_stream_t stream);

/* Orthogonalised updates of weights, by Newton-Schulz products ("From Install to Your First
 * Model" and the sharded optimizer's section of the source tour name the optimizer's step, which
 * this library's weight gradients feed): for `batch` matrices [rows][cols], each by itself,
 *     X_0 = U / |U|_F,  X <- a X + (b A + c A A) X, A = X X^T   (`steps` times),  O = X
 * (X <- a X + X (b A + c A A), A = X^T X, with more rows than columns), and, in
 * mlpb_muon_step,
 *     M <- momentum M + G,   U = G + momentum M (nesterov) or M
 *     W <- (1 - lr weight_decay) W - lr scale O
 * A zero matrix stays zero; one with an infinity or a NaN becomes NaN, alone.
 * The shards of dW1 and dW2 can be taken as they lie, as a batch: that is the blockwise update, in
 * which every shard is orthogonalised by itself, not the update of the whole weight.  For that one
 * the matrices are whole: dW1 [t][Fs][H] is [F][H] as it lies, and so is dW2 with t = 1; else
 * dW2's shards are put side by side first, and a gated dW1's apart into gate and up.
 * Products take fp16 operands with fixed scales, sums and both products' diagonals are fp32, X
 * keeps 22 bits between the steps.  With five steps of the usual coefficients O is off by 3e-4 to
 * 1.4e-3 of its size, by up to 4e-3 where the smaller side is below 32 or one singular value
 * dominates the others.  What U holds below 2^-22 of its size is rounding, which grows a times a
 * step like the rest: many steps of a large a bring it up (12 of 3.4: to 0.1 of O where U has rank
 * one). */
#define MLPB_MUON_FAULT_INJECT 0x1u /* test only, as MLPB_FLAG_FAULT_INJECT: the first product's \
                                       first stage is never filled (no effect on matrices that \
                                       lie in shared memory, where nothing waits for a copy)    */

typedef struct {
  int64_t batch;      /* matrices, 1..65535                                                     */
  int64_t rows, cols; /* of each, 1..65536                                                      */
  int32_t steps;      /* 1..64                                                                  */
  int32_t nesterov;   /* mlpb_muon_step: 1 U = G + momentum M, 0 U = M                           */
  float coef[3];      /* a, b, c: singular values from [0, 1] have to stay below 2               */
  float momentum;     /* [0, 1)                                                                 */
  float weight_decay;
  float scale;        /* of the update, such as 0.2 sqrt(max(rows, cols))                       */
  uint32_t flags;     /* 0, or MLPB_MUON_FAULT_INJECT                                           */
} mlpb_muon_config;

typedef struct mlpb_muon mlpb_muon; /* opaque; owns a device word and no tensors */

/* Validates *cfg and allocates the handle on the current device; EINVAL for null arguments or
 * values out of range, EUNSUPPORTED for sizes and coefficients outside those above. */
mlpb_status mlpb_muon_create(const mlpb_muon_config *cfg, mlpb_muon **out);
void mlpb_muon_destroy(mlpb_muon *h);

/* Bytes of the workspace of the calls below: three fp16 copies of X, two symmetric fp16 matrices of
 * the smaller side, and where few tiles are cut into ranges their fp32 sums; 256 bytes where
 * matrices lie in shared memory (a few with a smaller side of at most 128 and a longer one of some
 * thousands). */
mlpb_status mlpb_muon_workspace_size(const mlpb_muon *h, size_t *bytes);

/* O [batch][rows][cols] bf16 from U, bf16 or (u_f32 = 1) fp32 (O may not overlap U).  16-byte
 * aligned tensors.  The current device must be the handle's.  Calls that share a workspace must
 * not overlap on the GPU (a captured graph counts as its call; the handle has to outlive it). */
mlpb_status mlpb_muon_orthogonalize(mlpb_muon *h, const void *U, int32_t u_f32, void *O,
                                    void *workspace, mlpb_stream_t stream);

/* One step: G, M, W [batch][rows][cols] fp32, M and W updated in place; Wb, unless NULL, receives
 * the new W in bf16; lr one fp32 on the device (a captured graph then takes any schedule).  No two
 * of the tensors overlap. */
mlpb_status mlpb_muon_step(mlpb_muon *h, const float *G, float *M, float *W, void *Wb,
                           const float *lr, void *workspace, mlpb_stream_t stream);

/* As mlpb_moe_last_device_error, for an update's handle. */
mlpb_status mlpb_muon_last_device_error(mlpb_muon *h, mlpb_stream_t stream);

/* Static English text of a status code. */
const char *mlpb_status_str(mlpb_status s);

#ifdef __cplusplus
}
#endif
#endif /* MLPB_H_ */
