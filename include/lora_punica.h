/*
 * lora_punica.h -- C ABI of the GB300 (sm_103a) multi-LoRA shrink/expand
 * library (liblora_punica.so).
 *
 * The three core entry points are the three steps of the Punica-style
 * batched LoRA apply described by vLLM's API pages:
 *
 *   lora_meta_prepare  page "vllm.lora.ops.triton_ops.lora_kernel_metadata",
 *                      class LoRAKernelMeta, methods make / _reset /
 *                      prepare_tensors / meta_args.
 *   lora_shrink        page "vllm.lora.punica_wrapper.punica_gpu", method
 *                      PunicaWrapperGPU.add_shrink and its lora_shrink call
 *                      (argument order x, lora_a_stacked, y, meta, scale).
 *   lora_expand        same page, method PunicaWrapperGPU.add_expand and its
 *                      lora_expand call (x, lora_b_stacked, y, meta,
 *                      offset_start, add_inputs); the bias step of
 *                      PunicaWrapperTPU._apply_bias (page
 *                      "vllm.lora.punica_wrapper.punica_tpu") is fused into
 *                      it.
 *
 * Conventions shared by every call:
 *   - Every data pointer is a DEVICE pointer owned by the caller; the
 *     library allocates nothing and keeps no pointer after a call returns.
 *     Arrays of per-slice pointers (lora_a, lora_b, lora_bias) and
 *     slice_sizes are HOST arrays, read during the call only.
 *   - bf16 tensors are passed as pointers to their raw 16-bit patterns
 *     (lora_bf16_t).  All tensors are row-major and dense unless a leading
 *     dimension argument says otherwise.
 *   - Calls are asynchronous and ordered on `stream` (a cudaStream_t passed
 *     as void*; NULL is the legacy default stream).  Nothing is
 *     synchronised and nothing is read back to the host.
 *   - The device that owns `stream` and every tensor of a call must be the
 *     calling thread's current CUDA device (per-device launch settings are
 *     looked up for the current device).
 *   - Return value: 0 on success; a negative LORA_ERR_* code when an
 *     argument is rejected on the host (nothing is launched); a positive
 *     cudaError_t when a launch fails.  lora_status_string() names both.
 *   - Invalid LoRA ids (outside [-1, max_loras)) are not host errors: the
 *     metadata kernel counts them into meta->error_word and treats those
 *     tokens as having no LoRA, so shrink/expand skip them.
 *   - The no-LoRA early exit is taken on the device: shrink and expand read
 *     *meta->no_lora_flag and return at once when it is set, so a whole
 *     forward pass stays capturable in a CUDA graph with no host sync.
 */
#ifndef LORA_PUNICA_H
#define LORA_PUNICA_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Raw bit pattern of one bfloat16 value. */
typedef uint16_t lora_bf16_t;

#define LORA_PUNICA_VERSION 1
#define LORA_MAX_SLICES 8      /* slices per shrink/expand call          */
#define LORA_MAX_LORAS 1024    /* max_loras accepted by the metadata step */
#define LORA_MAX_RANK 128      /* rank r: a multiple of 8, 8 <= r <= 128 */
#define LORA_NOALLOC_MAX_FLOATS (1 << 20)  /* lora_linear_noalloc buffer: 4 MiB */

enum lora_status {
    LORA_OK = 0,
    LORA_ERR_NULL = -1,        /* a required pointer is NULL               */
    LORA_ERR_SIZE = -2,        /* a size is negative or out of range       */
    LORA_ERR_ALIGN = -3,       /* a pointer / stride breaks an alignment rule */
    LORA_ERR_RANK = -4,        /* rank not a multiple of 8 in [8, 128]      */
    LORA_ERR_SLICES = -5,      /* num_slices not in [1, LORA_MAX_SLICES]    */
    LORA_ERR_TOKENS = -6,      /* num_tokens > meta->max_num_tokens         */
    LORA_ERR_WIDTH = -7,       /* offset_start + sum(slice_sizes) > y_ld    */
    LORA_ERR_DEVICE = -8,      /* no usable CUDA device / wrong architecture */
    LORA_ERR_SCRATCH = -9,     /* num_slices * num_tokens * rank exceeds
                                  LORA_NOALLOC_MAX_FLOATS (lora_linear_noalloc) */
    LORA_ERR_WORKSPACE = -10   /* the workspace is smaller than the call's
                                  *_workspace function says                 */
};

/*
 * Per-forward metadata, the device-side counterpart of LoRAKernelMeta
 * (page "vllm.lora.ops.triton_ops.lora_kernel_metadata", LoRAKernelMeta.make
 * gives the buffer sizes).  The caller allocates every buffer once (int32,
 * device memory) and may reuse them for every forward pass:
 *   token_lora_mapping                [max_num_tokens]  copy of the id map
 *   token_indices_sorted_by_lora_ids  [max_num_tokens]  stable argsort
 *   num_tokens_per_lora               [max_loras + 1]   tokens per active id
 *   lora_token_start_loc              [max_loras + 2]   0, running sums
 *   active_lora_ids                   [max_loras + 1]   ascending, pad -1
 *   no_lora_flag                      [1]               1 = every id is -1
 *   error_word                        [1]               invalid ids counted
 *   grid_sync                         [2]               zero-filled once by
 *       the caller; the grid barrier of lora_linear's single-kernel path
 *       (every call leaves it zero again).  May be NULL, which turns that
 *       path off.  Calls that share a struct must be stream-ordered.
 * The same struct (by pointer) is then handed to lora_shrink/lora_expand;
 * they read it on the device.  The struct itself is host memory and is only
 * read during each call.
 */
typedef struct lora_meta {
    int32_t *token_lora_mapping;
    int32_t *token_indices_sorted_by_lora_ids;
    int32_t *num_tokens_per_lora;
    int32_t *lora_token_start_loc;
    int32_t *active_lora_ids;
    int32_t *no_lora_flag;
    int32_t *error_word;
    int32_t max_loras;
    int32_t max_num_tokens;
    int32_t *grid_sync;
} lora_meta_t;

/*
 * lora_meta_prepare -- LoRAKernelMeta.prepare_tensors on the device.
 *
 *   token_lora_mapping  device int32 [num_tokens], LoRA id per token, -1 =
 *                       no LoRA.
 *   num_tokens          0 <= num_tokens <= meta->max_num_tokens.
 *   meta                buffers as described above; 1 <= max_loras <=
 *                       LORA_MAX_LORAS.
 *
 * Writes, in one kernel: the reset values (active ids -1, counts 0,
 * start_loc 0); no_lora_flag = all(ids == -1) (true for num_tokens == 0);
 * and, only when the flag is false: the mapping copy, the stable permutation
 * of tokens sorted by id (ties keep token order, so id -1 tokens come
 * first), the distinct ids in ascending order with their counts, and
 * start_loc[k + 1] = counts[0] + ... + counts[k].  error_word receives the
 * number of ids outside [-1, max_loras); those tokens are sorted as -1.
 * Result: bit-exact, deterministic.
 */
int lora_meta_prepare(const int32_t *token_lora_mapping, int32_t num_tokens,
                      const lora_meta_t *meta, void *stream);

/*
 * lora_meta_read_no_lora -- the host copy of the no-LoRA flag (page
 * "vllm.lora.ops.triton_ops.lora_kernel_metadata", LoRAKernelMeta field
 * no_lora_flag_cpu, set by prepare_tensors).
 *
 *   meta      the metadata a preceding lora_meta_prepare on `stream` wrote;
 *             only meta->no_lora_flag is read.
 *   stream    the stream that call was ordered on.
 *   no_lora   HOST int32, receives 1 when every id of that batch is -1 (or
 *             it had no tokens), else 0.
 *
 * Copies the 4-byte device flag to the host and synchronises `stream`, so
 * it cannot be captured in a CUDA graph.  No other call needs it: every
 * kernel reads the device flag itself and returns early.
 * Errors: LORA_ERR_NULL for a NULL meta, meta->no_lora_flag or no_lora (on
 * the host, before any CUDA call); a positive cudaError_t if the copy or the
 * synchronisation fails (then *no_lora is left unchanged).
 */
int lora_meta_read_no_lora(const lora_meta_t *meta, void *stream, int32_t *no_lora);

/*
 * lora_shrink -- y[s][t, :] += scale * x[t, :] @ lora_a[s][id(t)]^T for
 * every slice s and every token t whose id is not -1 (page
 * "vllm.lora.punica_wrapper.punica_gpu", PunicaWrapperGPU.add_shrink,
 * "Semantics").  Rows of tokens without a LoRA are not touched.
 *
 *   x           device bf16 [num_tokens, x_ld]; the first `hidden` values of
 *               each row are used.  16-byte aligned, x_ld % 8 == 0.
 *   num_tokens  rows of x, <= meta->max_num_tokens; the metadata must have
 *               been prepared for exactly these tokens.
 *   hidden      H, a multiple of 8.
 *   lora_a      host array of num_slices device pointers, each bf16
 *               [max_loras, rank, hidden] (a leading singleton layer
 *               dimension is the same layout), 16-byte aligned.
 *   rank        r, a multiple of 8 in [8, LORA_MAX_RANK].
 *   y           device fp32 [num_slices, num_tokens, rank], 16-byte
 *               aligned; accumulated into (the caller zeroes it first to
 *               get a plain product).
 *   scale       multiplies the product before it is added.
 *
 * Accumulation is fp32 on the tensor cores (mma.sync; tcgen05 with TMEM
 * accumulators for batches of >= 1024 tokens with num_slices * rank >=
 * 256, LORA_PUNICA_UMMA* in the environment); when the hidden dimension is
 * split across CTAs the partial sums are added with fp32 atomics, so the
 * rounding order is not fixed from run to run.  A bounded wait of the
 * tcgen05 path that runs out sets bit 30 of meta->error_word.
 */
int lora_shrink(const lora_bf16_t *x, int32_t num_tokens, int32_t hidden,
                int64_t x_ld, const lora_bf16_t *const *lora_a,
                int32_t num_slices, int32_t rank, float *y,
                const lora_meta_t *meta, float scale, void *stream);

/*
 * lora_expand -- for every slice s and token t whose id is not -1:
 *   v = x[s][t, :] @ lora_b[s][id(t)]^T + (bias ? lora_bias[s][id(t)] : 0)
 *   y[t, off_s : off_s + n_s] = (add_inputs ? y[t, off_s : off_s + n_s] : 0) + v
 * with off_s = offset_start + n_0 + ... + n_{s-1} (page
 * "vllm.lora.punica_wrapper.punica_gpu", PunicaWrapperGPU.add_expand,
 * "Semantics"; bias as PunicaWrapperTPU._apply_bias).  Rows of tokens
 * without a LoRA, and columns outside the slices, are not touched.
 *
 *   x            device fp32 [num_slices, num_tokens, rank], 16-byte aligned
 *                (the shrink output).
 *   lora_b       host array of num_slices device pointers, each bf16
 *                [max_loras, n_s, rank], 16-byte aligned.
 *   lora_bias    NULL, or a host array of num_slices entries, each NULL or
 *                a device pointer to bf16 [max_loras, n_s].
 *   slice_sizes  host int32 [num_slices], n_s >= 1.
 *   y            device bf16 [num_tokens, y_ld],
 *                offset_start + sum(n_s) <= y_ld.
 *   add_inputs   nonzero: add to y; zero: overwrite the slice columns.
 *
 * x is rounded to bf16 for the tensor cores (as the Triton kernel does when
 * it casts its input to the weight type); products accumulate in fp32
 * (tcgen05 with TMEM accumulators at rank >= 64 when y, y_ld and
 * offset_start are 32-byte aligned and every slice width is a multiple of
 * 64; mma.sync otherwise; LORA_PUNICA_EXPAND_TC* in the environment move
 * the boundary, and with LORA_PUNICA_EXPAND_TC=2 a call the tcgen05 path
 * does not take fails with LORA_ERR_ALIGN or LORA_ERR_SIZE); y, the bias
 * and the product are summed in fp32 and
 * rounded to bf16 once (round to nearest even).  Output: deterministic.  A
 * bounded wait of the tcgen05 path that runs out sets bit 30 of
 * meta->error_word.
 */
int lora_expand(const float *x, const lora_bf16_t *const *lora_b,
                const lora_bf16_t *const *lora_bias,
                const int32_t *slice_sizes, int32_t num_slices, int32_t rank,
                lora_bf16_t *y, int64_t y_ld, int32_t num_tokens,
                int32_t offset_start, int32_t add_inputs,
                const lora_meta_t *meta, void *stream);

/*
 * lora_expand_bf16 -- lora_expand over a bf16 input, for the embedding LoRA
 * (page "vllm.lora.punica_wrapper.punica_gpu",
 * PunicaWrapperGPU.add_lora_embedding: y (+)= x @ lora_b, where x holds the
 * rows of the embedding LoRA's A looked up for each token, and add_inputs
 * is passed through from the caller).
 *
 *   x   device bf16 [num_slices, num_tokens, rank], 16-byte aligned; the
 *       tensor cores take it as it is (no rounding of the input).
 * Every other argument, the results and the errors are those of
 * lora_expand.
 */
int lora_expand_bf16(const lora_bf16_t *x, const lora_bf16_t *const *lora_b,
                     const lora_bf16_t *const *lora_bias,
                     const int32_t *slice_sizes, int32_t num_slices, int32_t rank,
                     lora_bf16_t *y, int64_t y_ld, int32_t num_tokens,
                     int32_t offset_start, int32_t add_inputs,
                     const lora_meta_t *meta, void *stream);

/*
 * lora_linear -- one LoRA layer applied to a batch, metadata included: the
 * result of lora_meta_prepare(token_lora_mapping), then lora_shrink(x ->
 * buf, scale), then lora_expand(buf -> y, lora_bias, offset_start = 0,
 * add_inputs = 1) (page "vllm.lora.punica_wrapper.punica_gpu",
 * PunicaWrapperGPU.update_metadata + add_lora_linear: add_shrink into the
 * fp32 buffer, then add_expand).  Arguments mean what they mean in those
 * three calls; `buf` is accumulated into like lora_shrink's y, and every
 * metadata buffer of `meta` is written as lora_meta_prepare writes it.
 *
 * How the layer runs (every form gives the three calls' results; the
 * shrink's partial sums may be added in a different order):
 *   - one cooperative kernel, by default when num_tokens * num_slices <=
 *     256 (and num_tokens <= 512, max_loras <= 256, rank <= 64, 16-byte
 *     aligned rows): every CTA sorts the ids in shared memory, the shrink
 *     is spread over the grid, a grid barrier (meta->grid_sync; bounded,
 *     bit 30 of the error word on expiry) separates it from the expand;
 *   - one thread-block-cluster kernel for other batches of at most 128
 *     tokens (max_loras <= 256, num_slices * padded rank <= 128);
 *   - rank 128, at most three slices, slice widths multiples of 64, y
 *     32-byte aligned with y_ld a multiple of 16, x and buf 16-byte
 *     aligned, batches of at least 72 tokens per SM of the device
 *     (LORA_PUNICA_LINEAR_TC_MIN_TOKENS sets another threshold): the
 *     metadata kernel, then one tensor-core kernel that runs
 *     the shrink of a 128-token tile, adds its result into that tile's
 *     buffer rows and runs the tile's expand (one CTA per SM, tiles of one
 *     LoRA in turn);
 *   - otherwise three kernels with programmatic dependent launch: the
 *     metadata kernel, the shrink (sorting the ids itself and loading
 *     before its dependency wait, for <= 512 tokens) and the expand
 *     (fetching the metadata, y and B before its wait).
 * Environment (read once, see lora_reload_options): LORA_PUNICA_COOP=0/1
 * never / always (when the batch fits) the cooperative kernel;
 * LORA_PUNICA_FUSED=0/1 and LORA_PUNICA_FUSED_MAX_TOKENS the cluster
 * kernel; LORA_PUNICA_LINEAR_TC=0/1 never / for every call that fits (any
 * batch size) the rank-128 tensor-core kernel (=2 requires it: a call it
 * does not fit fails with LORA_ERR_SIZE), and
 * LORA_PUNICA_LINEAR_TC_MIN_TOKENS its threshold; LORA_PUNICA_SELF_META=1 two
 * kernels (the shrink writes the metadata), =0 the plain three calls.
 */
int lora_linear(const int32_t *token_lora_mapping, int32_t num_tokens,
                const lora_bf16_t *x, int32_t hidden, int64_t x_ld,
                const lora_bf16_t *const *lora_a, const lora_bf16_t *const *lora_b,
                const lora_bf16_t *const *lora_bias, const int32_t *slice_sizes,
                int32_t num_slices, int32_t rank, float scale, float *buf,
                lora_bf16_t *y, int64_t y_ld, const lora_meta_t *meta, void *stream);

/*
 * lora_linear_noalloc -- lora_linear for callers that cannot allocate
 * device memory (code running where cudaMalloc is unavailable or forbidden:
 * inside an allocator or memory-pool callback, a plugin whose host owns
 * every allocation, a process that must not grow after start-up).  The
 * pages have no counterpart: this is an addition of this library.
 *
 * Same arguments and results as lora_linear, without `buf`: the fp32
 * buffer between shrink and expand lives in a fixed array of
 * LORA_NOALLOC_MAX_FLOATS floats (4 MiB) that the library holds on every
 * GPU that loads it, until the process exits.  Each call clears the
 * num_slices * num_tokens * rank floats it uses, so the shrink starts from
 * zero (as add_lora_linear's own zeroed buffer does); larger calls return
 * LORA_ERR_SCRATCH.  No cudaMalloc, cudaFree or allocating library routine
 * is called.
 *
 * The first call on a device looks up the array's device address (with that
 * device current); make it before any stream capture.  `stream` must belong
 * to the current device, else LORA_ERR_DEVICE is returned before anything
 * runs.  All calls on a device share the array: calls that may overlap on
 * the GPU (other streams or threads) race on it and must be serialised by
 * the caller.
 */
int lora_linear_noalloc(const int32_t *token_lora_mapping, int32_t num_tokens,
                        const lora_bf16_t *x, int32_t hidden, int64_t x_ld,
                        const lora_bf16_t *const *lora_a, const lora_bf16_t *const *lora_b,
                        const lora_bf16_t *const *lora_bias, const int32_t *slice_sizes,
                        int32_t num_slices, int32_t rank, float scale, lora_bf16_t *y,
                        int64_t y_ld, const lora_meta_t *meta, void *stream);

/* ------------------------------------------------------------------------
 * Training the adapters: the loss over the vocabulary, the gradients of one
 * layer's adapters, and the orthogonalised update of stacked adapters.  The
 * pages have no counterpart (they serve adapters); these are additions.
 * Every call takes a workspace of at least the bytes that its *_workspace
 * function returns (device memory, 256-byte aligned, contents of no matter
 * before and after); calls that may overlap need a workspace each.  The bytes
 * for a number of tokens (or matrices) hold any smaller call of the same
 * sizes, with fewer gradients too.
 * ------------------------------------------------------------------------ */

/*
 * lora_cross_entropy -- softmax cross entropy of the logits hidden x weight^T
 * and its gradients, without keeping the logits (at most about 2^27 of them,
 * a piece of the vocabulary, exist at a time, in the workspace):
 *   loss[t] = w_t (log sum_v exp S[t, v] - S[t, y_t]),  S = hidden weight^T
 *   hidden_grad[t] = w_t (sum_v p[t, v] weight[v] - weight[y_t])
 *   weight_grad[v] = sum_t w_t (p[t, v] - (v == y_t)) hidden[t]
 *
 *   hidden       device bf16 [num_tokens, hidden_ld]; the first hidden_size
 *                values of each row are used.  Any alignment.
 *   hidden_size  a multiple of 8.
 *   weight       device bf16 [vocab, hidden_size], dense, 16-byte aligned.
 *   targets      device int32 [num_tokens].  A token whose target lies
 *                outside [0, vocab) has none: its loss, log-sum and gradient
 *                are zero, its row of hidden is not read, and it costs no
 *                products.
 *   token_weight NULL (all ones) or device fp32 [num_tokens]: w_t (a mean
 *                over an adapter's tokens, a loss scale).
 *   loss         device fp32 [num_tokens].
 *   logsumexp    NULL or device fp32 [num_tokens]: log sum_v exp S[t, v].
 *   hidden_grad  NULL or device bf16 [num_tokens, hidden_grad_ld], written;
 *                may be hidden itself.  No other output may overlap an input
 *                or another output.
 *   weight_grad  NULL or device bf16 [vocab, hidden_size], dense, 16-byte
 *                aligned, written.
 *   error_word   NULL or device int32 [1]: receives the number of targets
 *                >= vocab; bit 30 is set if a bounded wait ran out (the
 *                outputs are then not valid).
 *
 * Products run on the tensor cores (tcgen05) in bf16 with fp32 sums; the
 * softmax's terms are rounded to bf16 once for the gradient products (for
 * weight_grad of up to 128 tokens they are two bf16 terms, 16 bits),
 * its sums and the accumulated gradients are fp32, and each gradient is
 * rounded to bf16 once.  A NaN logit of a token with a target makes its loss
 * and gradient NaN, and infinite logits give what the formulas give.
 * Deterministic.  Errors: LORA_ERR_NULL,
 * LORA_ERR_SIZE, LORA_ERR_ALIGN (weight, weight_grad, workspace,
 * hidden_size), LORA_ERR_WORKSPACE, LORA_ERR_DEVICE.
 */
int lora_cross_entropy(const lora_bf16_t *hidden, int32_t num_tokens, int32_t hidden_size,
                       int64_t hidden_ld, const lora_bf16_t *weight, int32_t vocab,
                       const int32_t *targets, const float *token_weight, float *loss,
                       float *logsumexp, lora_bf16_t *hidden_grad, int64_t hidden_grad_ld,
                       lora_bf16_t *weight_grad, int32_t *error_word, void *workspace,
                       int64_t workspace_bytes, void *stream);

/* Bytes of workspace of lora_cross_entropy on the current device, by whether
 * the gradients are asked for; LORA_ERR_SIZE for sizes that it refuses. */
int64_t lora_cross_entropy_workspace(int32_t num_tokens, int32_t hidden_size, int32_t vocab,
                                     int32_t hidden_grad, int32_t weight_grad);

/*
 * lora_linear_backward -- the gradients of one linear layer's adapters:
 * with u = buf (what lora_shrink left: scale * x @ A^T) and a = id(t), for
 * every slice s and every token t with an adapter
 *   g[s][t]  = lora_b[s][a]^T dy[t, off_s : off_s + n_s]
 *   dx[t]    (+)= scale * sum_s lora_a[s][a]^T g[s][t]
 *   d_lora_a[s][a] = scale * sum_t g[s][t] x[t]^T
 *   d_lora_b[s][a] = sum_t dy[t, slice s] buf[s][t]^T
 *   d_lora_bias[s][a] = sum_t dy[t, slice s]
 * with off_s = n_0 + ... + n_{s-1}.
 *
 *   dy           device bf16 [num_tokens, dy_ld], dy_ld >= sum of the
 *                slices: the gradient of the layer's output.  Any alignment
 *                (16-byte aligned rows are read faster); a slice may begin
 *                at any column.
 *   x            device bf16 [num_tokens, x_ld]: the layer's input.  Any
 *                alignment.  hidden is a multiple of 8.
 *   buf          device fp32 [num_slices, num_tokens, rank], 16-byte
 *                aligned: the buffer the forward pass left.
 *   lora_a, lora_b, slice_sizes, num_slices, rank, scale, meta: those of
 *                the forward pass; `meta` prepared for these tokens.
 *   dx           NULL or device bf16 [num_tokens, dx_ld], any alignment.
 *                May be dy or x, or overlap them (a residual layer's gradient
 *                in place: dy is read before dx is written).  No other output
 *                may overlap an input or another output.
 *   add_inputs   nonzero: the adapters' part is added to dx (rows of tokens
 *                without an adapter are not touched); zero: dx is
 *                overwritten (those rows with zeros).
 *   d_lora_a, d_lora_b, d_lora_bias  NULL, or host arrays of num_slices
 *                entries, each NULL or a device pointer to bf16
 *                [max_loras, rank, hidden], [max_loras, n_s, rank] (16-byte
 *                aligned) and [max_loras, n_s].  Overwritten for all
 *                max_loras adapters: zero for those without tokens.
 *
 * g and buf enter the products that follow as bf16 (rounded once; as two bf16
 * terms, 16 bits, in batches of up to 64 tokens, whose few terms would show
 * it); sums are fp32 and every output is rounded to bf16 once.  Deterministic.  Invalid
 * ids were mapped to -1 by the metadata.  Errors: as lora_shrink and
 * lora_expand, LORA_ERR_WIDTH for dy_ld, LORA_ERR_WORKSPACE.
 */
int lora_linear_backward(const lora_bf16_t *dy, int64_t dy_ld, int32_t num_tokens,
                         const lora_bf16_t *x, int32_t hidden, int64_t x_ld, const float *buf,
                         const lora_bf16_t *const *lora_a, const lora_bf16_t *const *lora_b,
                         const int32_t *slice_sizes, int32_t num_slices, int32_t rank,
                         float scale, lora_bf16_t *dx, int64_t dx_ld, int32_t add_inputs,
                         lora_bf16_t *const *d_lora_a, lora_bf16_t *const *d_lora_b,
                         lora_bf16_t *const *d_lora_bias, const lora_meta_t *meta,
                         void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace of lora_linear_backward; a negative status for sizes
 * that it refuses. */
int64_t lora_linear_backward_workspace(int32_t num_tokens, int32_t hidden,
                                       const int32_t *slice_sizes, int32_t num_slices,
                                       int32_t rank, int32_t max_loras);

/*
 * lora_orthogonalize -- Newton-Schulz steps on `count` (>= 0) stacked matrices, as
 * the Muon optimiser takes them on an update: for each matrix
 *   X = U / (|U|_F + eps);  steps times: X <- a X + (b G + c G^2) X, G = X X^T
 * (on the short side), out = scale X.  With a = 3.4445, b = -4.7750,
 * c = 2.0315 and five steps the singular values that U has end near 1.
 *
 *   update       device [count, rows, cols], dense, 16-byte aligned: bf16
 *                (update_f32 == 0) or fp32.  Stacked adapter gradients or
 *                momenta: A [.., rank, hidden], B [.., n, rank].
 *   rows, cols   min(rows, cols) <= 128 (an adapter's rank), cols a
 *                multiple of 8.
 *   steps        >= 1.
 *   out          device bf16 [count, rows, cols], dense, 16-byte aligned;
 *                may be `update` itself where that is bf16.
 *   error_word   NULL or device int32 [1]: bit 30 is set in it if a bounded
 *                wait ran out (the output is then not valid); otherwise it is
 *                left as it is.
 *
 * A zero matrix gives zeros (with eps > 0); a matrix with a NaN or an infinity
 * gives NaN in its own place only; one whose norm is below about 1e-17 is
 * divided by eps.  |U|_F^2 and the products U U^T are summed in fp32 and
 * must be finite there (entries up to about 1e17).  Up to |coef_a|^steps =
 * 512 (five steps with 3.4445) all steps run on r x r matrices in fp32 (every
 * factor is a polynomial in U U^T); the error is within 2% of the result's
 * norm for updates of rank one, the worst, and below bf16's rounding for
 * updates that lack no direction.  Longer runs form X and sum X X^T afresh
 * every few steps, in fp32: many times slower, a group of matrices at a time
 * (as many as the workspace holds in fp32 beside their sums; give more than
 * asked for larger groups).  There a rounding grows by coef_a a step in
 * directions that U lacks, as in any 32-bit iteration.  `out` is rounded to
 * bf16 once.  Deterministic.  Errors: LORA_ERR_NULL,
 * LORA_ERR_SIZE, LORA_ERR_ALIGN, LORA_ERR_WORKSPACE.
 */
int lora_orthogonalize(const void *update, int32_t update_f32, int32_t count, int32_t rows,
                       int32_t cols, int32_t steps, float coef_a, float coef_b, float coef_c,
                       float eps, float scale, lora_bf16_t *out, int32_t *error_word,
                       void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace of lora_orthogonalize on the current device;
 * LORA_ERR_SIZE for sizes that it refuses. */
int64_t lora_orthogonalize_workspace(int32_t count, int32_t rows, int32_t cols);

/*
 * lora_expert_linear -- the product of a mixture of experts, grouped by the
 * ids of the metadata (an expert per row): the layer that adapters are added
 * to.  With one expert it is one frozen layer.
 *   y[i] (+)= weight[id(i)] x[i / fan_out]        for every row i with an id
 * Rows without an id are not touched.
 *
 *   x            device bf16 [num_rows / fan_out, x_ld], any alignment: the
 *                tokens.  Token t has rows t * fan_out ... of y and of the
 *                metadata (a router's choices), each with an id of its own;
 *                num_rows is a multiple of fan_out >= 1.
 *   hidden       a multiple of 8 (of 32 with weight_scale).
 *   weight       device, 16-byte aligned: bf16 [max_loras, out_features,
 *                hidden] (weight_scale NULL), or the codes of
 *                lora_quantize_mxfp4, uint8 [max_loras, out_features,
 *                hidden / 2].
 *   weight_scale NULL, or the scales of the codes, 16-byte aligned uint8
 *                [max_loras, out_features, hidden / 32].
 *   y            device bf16 [num_rows, y_ld], any alignment.  Must not overlap an
 *                input.
 *   add_inputs   nonzero: added to y; zero: y is overwritten.
 *   meta         prepared for these num_rows ids; max_loras is the number of
 *                experts.  (Metadata of a larger batch write nothing beyond
 *                num_rows, and leave rows out.)
 *   workspace    256-byte aligned, at least lora_expert_linear_workspace
 *                bytes; a workspace for a batch holds every smaller one.
 *
 * Products run in bf16 on the tensor cores with fp32 sums, and each value of y
 * is rounded to bf16 once; 4-bit weights are bf16 values, so their products
 * lose nothing beside that (a scale of 2^127 times 6 is an infinity there).
 * Deterministic.  Bit 30 of meta->error_word: a bounded wait ran out (the
 * output is then not valid).  Errors: LORA_ERR_NULL, LORA_ERR_SIZE,
 * LORA_ERR_ALIGN, LORA_ERR_TOKENS, LORA_ERR_WORKSPACE, LORA_ERR_DEVICE.
 */
int lora_expert_linear(const lora_bf16_t *x, int64_t x_ld, int32_t num_rows, int32_t fan_out,
                       int32_t hidden, const void *weight, const uint8_t *weight_scale,
                       int32_t out_features, lora_bf16_t *y, int64_t y_ld, int32_t add_inputs,
                       const lora_meta_t *meta, void *workspace, int64_t workspace_bytes,
                       void *stream);

/* Bytes of workspace of lora_expert_linear on the current device; a negative
 * status for sizes that it refuses. */
int64_t lora_expert_linear_workspace(int32_t num_rows, int32_t hidden, int32_t out_features,
                                     int32_t max_loras, int32_t quantized);

/*
 * lora_expert_linear_backward -- the gradients of lora_expert_linear:
 *   dx[t] (+)= sum over the token's rows i with an id of weight[id(i)]^T dy[i]
 *   d_weight[e] = sum over the rows i with id e of dy[i] x[i / fan_out]^T
 *
 *   dy           device bf16 [num_rows, dy_ld], any alignment.
 *   x, fan_out, hidden, weight, weight_scale, out_features, meta: those of
 *                the forward pass.
 *   dx           NULL or device bf16 [num_rows / fan_out, dx_ld], any
 *                alignment.  The sum over a token's rows is fp32, in their
 *                order, and rounded once.  No output may overlap an input or
 *                another output.
 *   add_inputs   nonzero: added to dx (tokens without any id are not
 *                touched); zero: dx is overwritten (those with zeros).
 *   d_weight     NULL or device bf16 [max_loras, out_features, hidden],
 *                16-byte aligned, overwritten: zeros for experts without
 *                rows.  With 4-bit weights it is the gradient of the values
 *                that they stand for.
 *
 * Deterministic.  Errors as lora_expert_linear.
 */
int lora_expert_linear_backward(const lora_bf16_t *dy, int64_t dy_ld, int32_t num_rows,
                                int32_t fan_out, const lora_bf16_t *x, int64_t x_ld,
                                int32_t hidden, const void *weight, const uint8_t *weight_scale,
                                int32_t out_features, lora_bf16_t *dx, int64_t dx_ld,
                                int32_t add_inputs, lora_bf16_t *d_weight,
                                const lora_meta_t *meta, void *workspace,
                                int64_t workspace_bytes, void *stream);

/* Bytes of workspace of lora_expert_linear_backward, by whether dx and
 * d_weight are asked for; a negative status for sizes that it refuses. */
int64_t lora_expert_linear_backward_workspace(int32_t num_rows, int32_t fan_out, int32_t hidden,
                                              int32_t out_features, int32_t max_loras,
                                              int32_t hidden_grad, int32_t weight_grad,
                                              int32_t quantized);

/*
 * lora_quantize_mxfp4 / lora_dequantize_mxfp4 -- weights in microscaled 4 bits
 * (OCP MXFP4) and back.  Every 32 elements that follow one another share a
 * scale, a power of two: s = floor(log2 max|v|) - 2, at least -127, stored as
 * the byte s + 127.  An element is v / 2^s rounded to 0, 0.5, 1, 1.5, 2, 3, 4
 * or 6 with its sign (ties to the even code; beyond 6 to 6), as four bits,
 * two to a byte, the first in the low half.  A block with a NaN or an
 * infinity has scale byte 255 and is NaN as a whole.
 *
 *   weight     device bf16 (weight_f32 == 0) or fp32 [elements], dense,
 *              16-byte aligned; elements is a multiple of 32 (rows of a
 *              multiple of 32 keep blocks within a row).
 *   codes      device uint8 [elements / 2], 16-byte aligned.
 *   scales     device uint8 [elements / 32].
 *   out        device bf16 (out_f32 == 0) or fp32 [elements], 16-byte
 *              aligned.  Exact in both (6 x 2^127 is an infinity).
 *
 * What is written overlaps nothing that is read.
 *
 * Errors: LORA_ERR_NULL, LORA_ERR_SIZE, LORA_ERR_ALIGN.
 */
int lora_quantize_mxfp4(const void *weight, int32_t weight_f32, int64_t elements, uint8_t *codes,
                        uint8_t *scales, void *stream);
int lora_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t elements, void *out,
                          int32_t out_f32, void *stream);

/*
 * lora_clip_gradients -- the norm of many tensors' gradients, and the
 * gradients scaled down to a largest norm.  Every tensor is a stack of
 * `groups` equal slices (one per adapter; groups = 1: one norm over all):
 *   norms[g] = sqrt(sum over the tensors and the elements of slice g of v^2)
 *   out = v * min(1, max_norm / (norms[g] + eps))
 *
 *   grads        host array of num_tensors device pointers, each to groups *
 *                slice_sizes[i] dense elements, bf16 or (grads_f32[i]) fp32,
 *                aligned to an element.
 *   out          NULL (in place) or as grads; a tensor may be its own out, no
 *                others may overlap.
 *   slice_sizes  host int64 [num_tensors], >= 0.
 *   grads_f32    host int32 [num_tensors].
 *   max_norm     >= 0; infinite: the norms only (out then receives copies).
 *   eps          >= 0.
 *   norms        device fp32 [groups].
 *   workspace    256-byte aligned, lora_clip_gradients_workspace bytes.
 *
 * Sums of squares are fp64 beyond an fp32 sum of a few dozen each, and do not
 * overflow or underflow for any fp32 values.  The factor keeps fp32's digits
 * however far the norm lies above max_norm; its product with a gradient is
 * rounded to fp32, and then to bf16 where the gradient is.
 * A NaN norm makes its group's gradients NaN, an infinite one makes finite
 * gradients zero.  Deterministic.  Any number of tensors (1024 a launch).
 * The host arrays are read during the call only.  Errors: LORA_ERR_NULL,
 * LORA_ERR_SIZE, LORA_ERR_ALIGN, LORA_ERR_WORKSPACE.
 */
int lora_clip_gradients(const void *const *grads, void *const *out, const int64_t *slice_sizes,
                        const int32_t *grads_f32, int32_t num_tensors, int32_t groups,
                        float max_norm, float eps, float *norms, void *workspace,
                        int64_t workspace_bytes, void *stream);

/* Bytes of workspace of lora_clip_gradients on the current device;
 * LORA_ERR_SIZE for groups < 1. */
int64_t lora_clip_gradients_workspace(int32_t groups);

/*
 * lora_reload_options -- re-reads the library's tuning variables
 * (LORA_PUNICA_*: which of lora_linear's launch paths a batch takes, which
 * batches the tensor-core kernels take, programmatic dependent launch).
 * The library reads them once, at its first call; no later call reads the
 * environment unless this is called.  It must not run while another thread
 * is inside the library.  The pages have no counterpart: this is a control
 * of this library's own launch choices.
 */
void lora_reload_options(void);

/* Human-readable name of a status (negative LORA_ERR_* or cudaError_t). */
const char *lora_status_string(int status);

/* LORA_PUNICA_VERSION of the loaded library. */
int lora_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LORA_PUNICA_H */
