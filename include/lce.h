/*
 * lce.h — C ABI of the fused output-projection + cross-entropy library
 * (liblce.so, sm_103a).
 *
 * Operation. For hidden states H[N,d], a vocabulary matrix W[V,d] (tied to the
 * input embedding or not) and integer targets t[N] in which ignore_index marks
 * padding, with I = { i : t_i != ignore_index } and Nv = |I|:
 *
 *   loss    = (1/Nv) * sum_{i in I} ( logsumexp_v(h_i . w_v) - h_i . w_{t_i} )
 *   dH[i,:] = sum_v g_iv W[v,:]  for i in I, and 0 for ignored rows
 *   dW[v,:] = sum_{i in I} g_iv H[i,:]
 *   g_iv    = ( softmax_v(h_i . W^T)_v - [v == t_i] ) / Nv
 *
 * This is the output projection and loss computed in streamed chunks with
 * padding tokens skipped, so that no N x V logits buffer ever exists
 * ("OjasX 0.6.1: Training a 1B-Parameter LLM in 6.35GB of RAM", section
 * "Core Technology", the zero-byte vocabulary logits item), with the logits
 * recomputed in backward rather than kept ("6GB显卡预训练11亿参数模型：全是已发表
 * 技术，实测需375天", section "关键参数说明", --chunked-loss 512, and section
 * "内存实际花在哪里"). The row normaliser is the streaming (online) softmax
 * recurrence, which reaches the same value as the two-pass one (OjasX page,
 * "Online Softmax" note). Padding is removed by an on-device compaction into a
 * dense index list ("为什么26万词表会卡死16GB显卡", section 2.3 稀疏索引引擎).
 *
 * Conventions shared by every entry point.
 *  - All tensor arguments are DEVICE pointers owned by the caller, row-major
 *    and contiguous; the library never frees or retains them after the call.
 *  - H, W (and dH) are bf16 for lce_forward / lce_forward_backward, or the
 *    dtype given in lce_args_t; dW, loss and lse are fp32.
 *  - H, W, dH, dW base pointers must be 16-byte aligned and d % 8 == 0:
 *    W and the compacted H are read by the Tensor Memory Accelerator in rows
 *    of 16-byte multiples.
 *  - bf16 inputs run on bf16 tensor cores with fp32 accumulation. fp32
 *    inputs are split into bf16 pairs x = hi + lo and every product is formed
 *    as hi.hi + hi.lo + lo.hi (three times the tensor work, relative error
 *    about 2^-16); that path also holds a bf16 split copy of W (4*V*d bytes)
 *    in its workspace.
 *  - 1 <= N < 2^31, 1 <= d <= 65536, 1 <= V < 2^31.
 *  - Work is enqueued on `stream` (NULL = the legacy default stream) and the
 *    call returns without synchronising. Scratch memory is stream-ordered
 *    (cudaMallocAsync/cudaFreeAsync) unless a workspace is passed.
 *  - Host-detectable problems (null pointers, shapes, alignment, device)
 *    return an error code synchronously and enqueue nothing. Problems only the
 *    device can see (a non-ignored target outside [0, V), a bounded wait that
 *    gave up) never trap: they set bits in a per-device status word that
 *    lce_get_device_status reads; the loss is then NaN and the gradients are
 *    unspecified.
 *  - Nv == 0 gives loss = NaN (a mean over no tokens) and zero dH and dW.
 *  - Results are deterministic: the same inputs give bitwise-identical
 *    outputs (no floating-point atomics).
 *  - The library runs on sm_103 devices only (LCE_ERR_DEVICE otherwise).
 */
#ifndef LCE_H
#define LCE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream. */
typedef struct CUstream_st *lce_stream_t;

typedef enum {
    LCE_OK = 0,
    LCE_ERR_NULL = 1,         /* a required pointer is NULL */
    LCE_ERR_SHAPE = 2,        /* N, d, V or vocab_chunk out of range */
    LCE_ERR_ALIGN = 3,        /* base pointer or row stride not 16-byte aligned */
    LCE_ERR_DTYPE = 4,        /* unknown dtype */
    LCE_ERR_CUDA = 5,         /* a CUDA call failed; see lce_last_cuda_error() */
    LCE_ERR_WORKSPACE = 6,    /* workspace_bytes below lce_workspace_size() */
    LCE_ERR_TARGET_RANGE = 7, /* device: a non-ignored target outside [0, V) */
    LCE_ERR_TIMEOUT = 8,      /* device: a bounded wait inside a kernel gave up */
    LCE_ERR_DEVICE = 9,       /* current device is not sm_103 */
    LCE_ERR_ARG = 10          /* an option value or combination that is not supported */
} lce_status_t;

typedef enum { LCE_BF16 = 0, LCE_FP32 = 1 } lce_dtype_t;

/* Bits of the device status word (lce_get_device_status). */
#define LCE_DEV_TARGET_RANGE 0x1  /* a non-ignored target was outside [0, V) */
#define LCE_DEV_TIMEOUT      0x2  /* a pipeline wait gave up; that kernel returned early */
#define LCE_DEV_SEQLENS      0x4  /* sequence offsets of an attention call that are not ascending within the tokens */

/*
 * Forward only: writes the mean loss to the device scalar `loss`.
 * H [N,d] bf16, W [V,d] bf16, targets [N] int64.
 */
lce_status_t lce_forward(const void *H, const void *W, const int64_t *targets,
                         int64_t ignore_index, int64_t N, int64_t d, int64_t V,
                         float *loss, lce_stream_t stream);

/*
 * Forward and backward in one call: loss (device fp32 scalar), dH [N,d] bf16
 * (overwritten; ignored rows are zero) and dW [V,d] fp32 (overwritten).
 * H, W and targets as in lce_forward. dW is fp32 so a tied W's gradient can be
 * added to the input-embedding gradient without a rounding step.
 */
lce_status_t lce_forward_backward(const void *H, const void *W, const int64_t *targets,
                                  int64_t ignore_index, int64_t N, int64_t d, int64_t V,
                                  float *loss, void *dH, float *dW, lce_stream_t stream);

/*
 * Valid-token compaction alone (the first step of every call): idx[0..Nv)
 * receives the ascending positions whose target is not ignore_index, inv[i]
 * the compacted row of position i or -1, counts[0] = Nv and counts[1] = the
 * number of non-ignored targets outside [0, V). idx and inv hold N int32
 * each, counts 2 int32; all device pointers. One CTA sweeps the targets with
 * warp ballots and a block scan; the list is exact (integer) and ascending.
 * Padding-aware valid mask of "为什么26万词表会卡死16GB显卡", section 2.3
 * 稀疏索引引擎.
 */
lce_status_t lce_compact(const int64_t *targets, int64_t N, int64_t ignore_index, int64_t V,
                         int32_t *idx, int32_t *inv, int32_t *counts, lce_stream_t stream);

/*
 * Optimizer step on W fused into the backward (lce_args_t.optim): the
 * gradient of W is consumed where it is produced, in the epilogue of each dW
 * tile, and never stored — no V x d gradient buffer exists, the "zero-byte
 * persistent .grad buffers" item of "OjasX 0.6.1: Training a 1B-Parameter LLM
 * in 6.35GB of RAM" (section "Core Technology"; its usage listing attaches an
 * "adamw" or "sgd" optimizer that updates weights in place during backward).
 * The pages do not define the two rules; these follow PyTorch's SGD and AdamW
 * (no dampening, no Nesterov, no amsgrad), with g the gradient of W
 * (grad_scale and grad_loss applied):
 *   SGD:   g += weight_decay * w; with momentum != 0: b = g on step 1, else
 *          b = momentum * b + g, and g = b (b in exp_avg); w -= lr * g.
 *   AdamW: w *= 1 - lr * weight_decay; m = beta1*m + (1-beta1)*g;
 *          v = beta2*v + (1-beta2)*g^2;
 *          w -= lr/(1-beta1^step) * m / (sqrt(v)/sqrt(1-beta2^step) + eps)
 *          (m in exp_avg, v in exp_avg_sq).
 * W is updated in place in its own dtype (bf16 rounded to nearest), or, for
 * bf16 W with master_W given, the fp32 master copy is updated and W is
 * rewritten as its bf16 rounding. Every W row is updated exactly once per
 * call, after the last read of its old value (loss, lse and dH are those of
 * the old W). State arrays are fp32 [V,d], device, 16-byte aligned, owned by
 * the caller; with state_bf16 they are bf16 [V,d] instead, as torch.optim
 * keeps them for a bf16 parameter: each is read, updated in fp32 (the update
 * of w uses the fp32 values) and stored rounded to the nearest bf16, which
 * halves their memory and traffic (12 instead of 20 bytes moved per W
 * element for AdamW on a bf16 W). Requirements (else LCE_ERR_ARG /
 * LCE_ERR_NULL): dH given and
 * dW NULL, accumulate_dW 0, one token chunk, step >= 1, lr >= 0,
 * weight_decay >= 0, 0 <= beta1, beta2 < 1, eps > 0, master_W only for bf16.
 */
typedef enum { LCE_OPT_NONE = 0, LCE_OPT_SGD = 1, LCE_OPT_ADAMW = 2 } lce_optim_kind_t;
typedef struct {
    lce_optim_kind_t kind;
    float lr;
    float weight_decay;
    float momentum;           /* SGD */
    float beta1, beta2, eps;  /* AdamW */
    int64_t step;             /* 1-based number of this update */
    float *master_W;          /* optional fp32 [V,d] master weights of a bf16 W */
    void *exp_avg;            /* [V,d] fp32 (bf16 with state_bf16): AdamW first moment, SGD momentum buffer */
    void *exp_avg_sq;         /* [V,d] fp32 (bf16 with state_bf16): AdamW second moment */
    int state_bf16;           /* nonzero: exp_avg / exp_avg_sq are bf16 */
} lce_optim_t;

/* Full argument set for lce_run. Zero-initialise, then fill. */
typedef struct {
    lce_dtype_t dtype;        /* element type of H, W and dH */
    const void *H;            /* [N,d] */
    const void *W;            /* [V,d]; written only by a fused optimizer step (optim) */
    const int64_t *targets;   /* [N] */
    int64_t ignore_index;
    int64_t N, d, V;
    float *loss;              /* device fp32 scalar; required unless lse_in is given */
    void *dH;                 /* [N,d] of dtype, or NULL for forward only */
    void *dW;                 /* [V,d] fp32 (bf16 with dW_bf16), or NULL for forward only (NULL iff dH
                                 is NULL, except that dW is NULL with a fused optimizer) */
    int accumulate_dW;        /* nonzero: dW += gradient; zero: dW = gradient */
    float grad_scale;         /* multiplies dH and dW (0 is read as 1) */
    float *lse;               /* optional [N] fp32: per-row logsumexp (natural log), NaN on ignored rows */
    void *workspace;          /* optional device scratch; NULL = stream-ordered allocation */
    size_t workspace_bytes;   /* size of `workspace` */
    int64_t vocab_chunk;      /* vocab rows per backward chunk; 0 = default (6144-row chunks, evened out over V); else a multiple of 256 */
    lce_stream_t stream;
    const float *lse_in;      /* optional [N] fp32 per-row logsumexp from an earlier forward (the `lse`
                                 output of lce_run): the forward pass is skipped, only dH/dW are
                                 computed (dH and dW required, loss may be NULL) */
    const float *grad_loss;   /* optional device fp32 scalar: upstream gradient of the loss,
                                 multiplies dH and dW (read on the device, no host sync) */
    int64_t token_chunk;      /* 0 = all N rows at once; else the rows are processed token_chunk
                                 positions at a time (scratch O(token_chunk*(d + vocab_chunk)),
                                 dW accumulated across chunks in a fixed order): the chunked loss
                                 of "6GB显卡预训练11亿参数模型", section "关键参数说明" (--chunked-loss 512) */
    const lce_optim_t *optim; /* optional: optimizer step on W fused into the backward (W is written) */
    int row_gather;           /* nonzero: the GEMMs read H's valid rows through the compaction index
                                 with TMA gather4 loads instead of from a compacted copy (no
                                 N*d*2-byte copy in the workspace; bf16 and d % 256 == 0 only, else
                                 LCE_ERR_ARG). Same results; slower on sm_103 (32 gather4 of 512
                                 bytes per pipeline stage against one tiled load). The dense index
                                 list of "为什么26万词表会卡死16GB显卡", section 2.3 稀疏索引引擎,
                                 used directly as the operand's row map. */
    int dW_bf16;              /* nonzero: dW is bf16 [V,d] (the fp32 accumulator of each element
                                 rounded to nearest once), for a bf16 W whose gradient is kept in
                                 its own dtype; half the dW bytes. bf16 inputs only, not with
                                 accumulate_dW or token chunks (else LCE_ERR_ARG). */
} lce_args_t;

/* Forward, or forward + backward when dH/dW are given, or backward alone
 * from a stored lse (lse_in), with every option. */
lce_status_t lce_run(const lce_args_t *args);

/*
 * Backward alone, for a training loop that runs the forward and backward
 * passes at different times: dH [N,d] bf16 and dW [V,d] fp32 (overwritten)
 * from the per-row lse [N] fp32 that a forward stored (lce_run with
 * args.lse), times the device scalar *grad_loss (NULL = 1). The logits are
 * recomputed from H and W ("6GB显卡预训练11亿参数模型", section "关键参数说明":
 * the chunked loss recomputes logits in backward instead of keeping them).
 * H, W, targets and ignore_index must be those of the forward.
 */
lce_status_t lce_backward(const void *H, const void *W, const int64_t *targets, int64_t ignore_index,
                          int64_t N, int64_t d, int64_t V, const float *lse, const float *grad_loss,
                          void *dH, float *dW, lce_stream_t stream);

/*
 * Bytes of scratch lce_run needs for these sizes (what the library allocates
 * itself when no workspace is passed). Grows as O(N*(d + vocab_chunk)), never
 * with N*V. Returns 0 for invalid arguments.
 */
size_t lce_workspace_size(int64_t N, int64_t d, int64_t V, lce_dtype_t dtype, int64_t vocab_chunk);

/* Bytes of scratch lce_run needs for exactly these arguments (all options,
 * token_chunk included); 0 for invalid arguments. Pointers are not read. */
size_t lce_workspace_size_args(const lce_args_t *args);

/*
 * Synchronises `stream`, then returns in *bits the current device's status
 * word (LCE_DEV_* bits accumulated since the last read) and clears it.
 * Returns LCE_ERR_TARGET_RANGE, LCE_ERR_TIMEOUT or (LCE_DEV_SEQLENS)
 * LCE_ERR_SHAPE when the matching bit is set, LCE_OK when the word is clear.
 */
lce_status_t lce_get_device_status(lce_stream_t stream, int32_t *bits);

/* Static string naming a status code. */
const char *lce_status_string(lce_status_t status);

/* cudaError_t value of the last CUDA failure seen by this thread (0 = none). */
int lce_last_cuda_error(void);

/* Number of kernels this library has launched in this process. */
int64_t lce_launch_count(void);

/*
 * Phase timing for profiling. While enabled (on the calling thread), every
 * call records CUDA events on its stream around each phase:
 *   0 compaction + gather of valid rows, 1 logits + online log-sum-exp,
 *   2 log-sum-exp merge + loss, 3 backward (recomputed logits -> G, dW = G^T H,
 *   dH += G W, one launch per vocab chunk), 4 scatter of dH to the caller's rows.
 * lce_profile_end synchronises those events and returns, per phase, the summed
 * milliseconds and the number of kernel launches; it then disables timing.
 * n is the length of both output arrays (at most LCE_PROFILE_PHASES used).
 */
#define LCE_PROFILE_PHASES 5
lce_status_t lce_profile_begin(void);
lce_status_t lce_profile_end(double *ms, int64_t *launches, int n);

/*
 * Forward loss like lce_forward, for callers that must not allocate device
 * memory: real-time or long-running loops whose memory budget is fixed up
 * front (an allocation can stall the device or fail from fragmentation at an
 * arbitrary point), and hosts that forbid device allocation after start-up.
 * It calls no cudaMalloc, cudaFree or other allocating routine; the pages
 * have no counterpart of this entry point.
 *
 * Scratch lives in one fixed 21 MiB device array inside the library, which
 * every GPU that loads liblce.so holds until the process exits. Limits:
 * N <= 4096 and d <= 2048 (LCE_ERR_SHAPE beyond them); bf16 H and W; other
 * arguments, layout and errors as in lce_forward. The first call on each
 * device looks up the array's device address (with that device current); make
 * that first call before any stream capture. All calls share the one array:
 * calls that overlap on the GPU (different streams, or different host threads
 * on one device) race and corrupt each other's results; serialise them.
 */
lce_status_t lce_forward_noalloc(const void *H, const void *W, const int64_t *targets,
                                 int64_t ignore_index, int64_t N, int64_t d, int64_t V,
                                 float *loss, lce_stream_t stream);

/*
 * Failure-path self-test: launches one thread that waits on a pipeline
 * barrier nothing completes, using the same bounded wait as the GEMM kernels
 * but with a limit of `cycles` SM clocks (1 .. 2^34). The wait gives up,
 * sets LCE_DEV_TIMEOUT in the device status word and the kernel returns, so
 * the context stays usable; *gave_up (device int32) receives 1. Read the
 * status with lce_get_device_status.
 */
lce_status_t lce_selftest_wait_timeout(int64_t cycles, int32_t *gave_up, lce_stream_t stream);

/*
 * Input-embedding lookup that skips padding, for a vocabulary matrix W shared
 * by the input lookup and the output projection ("6GB显卡预训练11亿参数模型",
 * section "关键参数说明", --tie-embeddings):
 *   E[i,:] = W[tokens[i],:] where tokens[i] != pad_id, a zero row where it is.
 * The valid mask and the lookup run in one kernel with no host
 * synchronisation ("为什么26万词表会卡死16GB显卡", section 2.3 稀疏索引引擎).
 * W [V,d] and E [N,d] are device arrays of `dtype`; tokens [N] int64.
 * A non-padding token outside [0, V) gets a zero row and sets
 * LCE_DEV_TARGET_RANGE in the device status word. Same shape, alignment and
 * error rules as lce_run (d % 8 == 0, 16-byte aligned W and E).
 */
lce_status_t lce_embedding_forward(lce_dtype_t dtype, const void *W, const int64_t *tokens, int64_t pad_id,
                                   int64_t N, int64_t d, int64_t V, void *E, lce_stream_t stream);

/*
 * Gradient of lce_embedding_forward with respect to W:
 *   dW[v,:] (+)= sum of dE[i,:] over the positions i with tokens[i] == v,
 * for tokens that are not pad_id and lie in [0, V) (others are skipped and
 * flagged as in the forward). dE [N,d] of `dtype`, dW [V,d] fp32 (device).
 * accumulate = 0 overwrites dW (rows of tokens that do not occur become 0);
 * nonzero adds into it, so for a tied W the output projection's dW (lce_run)
 * and this gradient sum into one buffer. The positions are grouped by token
 * on the device and each row's sum is taken in ascending position order (the
 * batch's per-token gradients aggregated after backward, same page, section
 * 2.2, without atomics): results are reproducible bit for bit.
 * The grouping is a stable radix sort of the valid positions by token over
 * several CTAs; the sorted list is cut into fixed chunks of 32, each token's
 * rows in a chunk are summed in order and a token whose rows span chunks
 * gets its chunk sums added in chunk order. Scratch: lce_embedding_workspace_size(N, d) bytes of
 * `workspace` (device, 16-byte aligned), or NULL for a stream-ordered
 * allocation.
 */
size_t lce_embedding_workspace_size(int64_t N, int64_t d);
lce_status_t lce_embedding_backward(lce_dtype_t dtype, const void *dE, const int64_t *tokens, int64_t pad_id,
                                    int64_t N, int64_t d, int64_t V, float *dW, int accumulate, void *workspace,
                                    size_t workspace_bytes, lce_stream_t stream);

/*
 * The same gradient written as bf16 [V,d] (dW, device, 16-byte aligned):
 * every row sum is taken in fp32 exactly as above and rounded to nearest once
 * when it is stored, so the result equals lce_embedding_backward's fp32 dW
 * rounded to bf16. For a bf16 W whose gradient is kept in its own dtype; dW
 * is overwritten (no accumulation: a second rounding would follow).
 */
lce_status_t lce_embedding_backward_bf16(lce_dtype_t dtype, const void *dE, const int64_t *tokens, int64_t pad_id,
                                         int64_t N, int64_t d, int64_t V, void *dW, void *workspace,
                                         size_t workspace_bytes, lce_stream_t stream);

/*
 * Attention over packed sequences, and its backward pass: the mixing layer of
 * a block between the embedding lookup and the head loss. For query token i
 * and key token j of the same sequence,
 *   s_ij  = scale * q_i . k_j,  allowed where not causal, or
 *           pos(j) <= pos(i) + Lk - Lq   (causal, aligned at the ends),
 *   lse_i = log sum_j exp(s_ij),   o_i = sum_j exp(s_ij - lse_i) v_j,
 * and from (q, k, v, o, lse, dO), with the probabilities recomputed,
 *   p_ij = exp(s_ij - lse_i),  delta_i = dO_i . o_i,
 *   ds_ij = p_ij (dO_i . v_j - delta_i),
 *   dq_i = scale * sum_j ds_ij k_j,  dk_j = scale * sum_i ds_ij q_i,
 *   dv_j = sum_i p_ij dO_i,
 * dk and dv summed over the query heads that share a key head. A row with no
 * allowed key has o = 0, lse = -inf and no gradient.
 *
 * Layout. Token-major [tokens][heads][D]: element (t, h, c) of q lies at
 * q + t*q_ts + h*q_hs + c, strides in elements, so q, k and v may be slices of
 * one projection's output and dq, dk, dv slices of its gradient. lse is fp32
 * [Hq][Tq], contiguous. cu_q and cu_k hold the B+1 ascending token offsets of
 * the sequences (device int32, cu[0] = 0, cu[B] <= tokens); tokens after
 * cu[B] belong to no sequence (o = 0, lse = -inf, zero gradients). NULL: B
 * sequences of equal length. Either side of a sequence may be empty. Values of
 * one sequence, infinities and NaN among them, never reach another sequence;
 * inside a sequence a non-finite masked key or value may reach the rows that
 * share its 128-token tile.
 *
 * dtype LCE_BF16 runs on the bf16 tensor cores with fp32 accumulation (the
 * probabilities and their gradient are rounded to bf16 once, as operands; to
 * two bf16 parts where Tq*Hq*D <= 2^18 and sequences average at most 512, so a
 * sequence's last bits depend on what it is packed with; probabilities below
 * 2^-126 count as zero); LCE_FP32 runs in fp32 arithmetic throughout.
 * Requirements: 1 <= D <= 128, D % 8 == 0, Hq a multiple of Hk, 0 <= Tq, Tk <
 * 2^30, 1 <= B < 2^30, Tq and Tk multiples of B without offsets; bases 16-byte
 * aligned, strides multiples of 16 bytes, positive (but for a single head or
 * token). The rows of an output must be apart from one another (checked), and
 * outputs apart from each other and from every input (not checked).
 * Results are deterministic. Scratch: lce_attention_forward_workspace_size bytes
 * (0 but for few rows over long keys, whose keys are taken in ranges) or
 * lce_attention_workspace_size bytes (backward), device, 16-byte aligned, or
 * NULL for a stream-ordered allocation. Offsets that are not ascending within the tokens set
 * LCE_DEV_SEQLENS; the outputs are then unspecified.
 */
typedef struct {
    lce_dtype_t dtype;
    int causal;
    float scale;
    int64_t B, Tq, Tk, Hq, Hk, D;
    const int32_t *cu_q, *cu_k;      /* [B+1] device, or both NULL */
    const void *q, *k, *v;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
    void *o;                         /* [Tq][Hq][D]: written by the forward, read by the backward */
    int64_t o_ts, o_hs;
    float *lse;                      /* [Hq][Tq]: written by the forward, read by the backward */
    const void *dO;                  /* backward only, as are the rest */
    int64_t dO_ts, dO_hs;
    void *dq, *dk, *dv;
    int64_t dq_ts, dq_hs, dk_ts, dk_hs, dv_ts, dv_hs;
    void *workspace;
    size_t workspace_bytes;
    lce_stream_t stream;
} lce_attn_t;
lce_status_t lce_attention_forward(const lce_attn_t *args);
lce_status_t lce_attention_backward(const lce_attn_t *args);
size_t lce_attention_workspace_size(const lce_attn_t *args);
size_t lce_attention_forward_workspace_size(const lce_attn_t *args);

/*
 * The norms before and after a block, fused with the block's gate and
 * residual scale. For the residual stream x, the block's output b and
 * rms(t) = sqrt(mean(t^2) + eps) over the d channels of a row:
 *   y = b / rms(b) * w_post     (y = b without w_post)
 *   r = x + scale * gate * y    (gate: none, [d], or [N,d] with gate_full)
 *   n = r / rms(r) * w_pre      (the next block's input; absent without w_pre)
 * The forward writes r, n and the fp32 rows rstd_post = 1/rms(b) and
 * rstd_pre = 1/rms(r); r may be x (updated in place). Without b, r is x itself
 * and only n and rstd_pre are written (r NULL). n and rstd_pre are formed from r
 * before r is rounded to its type. The backward takes r as it was rounded, b and
 * the stored rstd, the gradients dr (of r, or NULL for zero) and dn (of n), and
 * writes
 *   dx = dr + rstd_pre * (u - rhat * mean(u * rhat)),   u = w_pre * dn,
 *   dy = scale * gate * dx,  dgate = scale * dx * y (summed over rows for [d]),
 *   db = rstd_post * (t - bhat * mean(t * bhat)),       t = w_post * dy,
 *   dw_post = sum over rows of dy * bhat,  dw_pre = sum of dn * rhat,
 * each rounded once to its own type. All tensors are of `dtype` (statistics
 * fp32), rows of d contiguous elements, ld_* apart (0 stands for d: rows that
 * all lie in one place have to be copied first); outputs are contiguous.
 * d % 8 == 0, 8 <= d <= 16384, 0 <= N < 2^31, bases and row strides 16-byte
 * aligned. Sums are fp32 in a fixed order (deterministic).
 * Scratch (backward): lce_block_norm_workspace_size bytes or NULL.
 */
typedef struct {
    lce_dtype_t dtype;
    int64_t N, d;
    float scale, eps;
    const void *x, *b;
    const void *w_post, *gate, *w_pre;
    int gate_full;                   /* nonzero: gate is [N,d] */
    int64_t ld_x, ld_b, ld_gate;
    void *r, *n;                     /* r: written by the forward, read by the backward */
    float *rstd_post, *rstd_pre;     /* [N]: written by the forward, read by the backward */
    const void *dr, *dn;             /* backward only, as are the rest */
    int64_t ld_r, ld_dr, ld_dn;
    void *dx, *db, *dw_post, *dgate, *dw_pre;
    void *workspace;
    size_t workspace_bytes;
    lce_stream_t stream;
} lce_norm_t;
lce_status_t lce_block_norm_forward(const lce_norm_t *args);
lce_status_t lce_block_norm_backward(const lce_norm_t *args);
size_t lce_block_norm_workspace_size(const lce_norm_t *args);

/*
 * Global gradient norm over `count` tensors and clipping by it:
 *   norm = sqrt( sum over all elements of g^2 ),
 *   factor = min(1, max_norm / (norm + eps)),   out = g * factor.
 * grads, outs, sizes and dtypes are HOST arrays of `count` entries (device
 * tensor addresses, element counts, lce_dtype_t); tensors are contiguous, of
 * any size (zero included) and aligned to their element. outs NULL clips in
 * place, and then writes nothing where the factor is 1; an out may be its own
 * grad and must not overlap any other tensor. A norm that is not finite gives
 * factor 0 (infinite) or NaN, as the formulas say. norm is a device fp32
 * scalar; factor an optional one. The squares are summed in fp32 over short
 * runs and in fp64 across them, in a fixed order (deterministic); a run whose
 * squares overflow fp32 is summed in fp64, so the norm is infinite only where
 * fp32 cannot hold it. Elements below 1.1e-19, whose squares are subnormal,
 * lose bits; below 2.6e-23 they count as zero. Scratch: lce_clip_workspace_size
 * bytes of device memory (16-byte aligned) or NULL (a stream-ordered
 * allocation; none for up to 1 MB of gradients, whose sums need no memory).
 */
size_t lce_clip_workspace_size(int64_t count);
lce_status_t lce_grad_norm(int64_t count, const void *const *grads, const int64_t *sizes, const int32_t *dtypes,
                           float *norm, void *workspace, size_t workspace_bytes, lce_stream_t stream);
lce_status_t lce_clip_grads(int64_t count, const void *const *grads, void *const *outs, const int64_t *sizes,
                            const int32_t *dtypes, float max_norm, float eps, float *norm, float *factor,
                            void *workspace, size_t workspace_bytes, lce_stream_t stream);

/*
 * Layer norm with the residual sum before it: for the stream x and a block's
 * output b (or none), row by row over d channels,
 *   r = x + b   (rounded to its type; x itself without b),
 *   mean = sum r / d,   rstd = 1 / sqrt(sum (r - mean)^2 / d + eps),
 *   n = (r - mean) * rstd * weight + bias   (bias may be NULL).
 * n and the statistics are those of r as it is stored; the sum of squares is
 * taken after the mean is known. The forward writes r (with b; it may be x or
 * b), n, mean and rstd (fp32 [N]) and, where `codes` is given, r packed to 8
 * bits (lce_pack8 below, in the same pass). The backward takes r, or its 8-bit
 * form where `codes` is given (r is then not read), the gradients dr (of r, or
 * NULL for zero) and dn (of n), and writes
 *   dx = dr + rstd * (u - mean(u) - rhat * mean(u * rhat)),  u = weight * dn,
 *   rhat = (r - mean) * rstd   (the gradient of x and of b alike),
 *   dweight = sum over rows of dn * rhat,  dbias = sum of dn (NULL: not wanted),
 * each rounded once to its own type. All tensors are of `dtype`, rows of d
 * contiguous elements, ld_* apart (0 stands for d); outputs are contiguous.
 * d % 8 == 0, 8 <= d <= 16384, 0 <= N < 2^31, bases and row strides 16-byte
 * aligned. Sums are fp32 in a fixed order (deterministic): a row whose sum, or
 * sum of squares around its mean, leaves fp32 (values of 1e19 and more) has no
 * finite mean or an rstd of 0.
 * Scratch (backward): lce_layer_norm_workspace_size bytes or NULL.
 */
typedef struct {
    lce_dtype_t dtype;
    int64_t N, d;
    float eps;
    const void *x, *b;               /* forward only */
    const void *weight, *bias;       /* [d] */
    int64_t ld_x, ld_b;
    void *r, *n;                     /* r: written by the forward (with b), read by the backward */
    float *mean, *rstd;              /* [N]: written by the forward, read by the backward */
    uint8_t *codes;                  /* r in 8 bits, or NULL: written by the forward, read by the backward */
    int8_t *exps;
    int64_t ld_codes, ld_exps;
    const void *dr, *dn;             /* backward only, as are the rest */
    int64_t ld_r, ld_dr, ld_dn;
    void *dx, *dweight, *dbias;
    void *workspace;
    size_t workspace_bytes;
    lce_stream_t stream;
} lce_layer_norm_t;
lce_status_t lce_layer_norm_forward(const lce_layer_norm_t *args);
lce_status_t lce_layer_norm_backward(const lce_layer_norm_t *args);
size_t lce_layer_norm_workspace_size(const lce_layer_norm_t *args);

/*
 * Activations in 8 bits, for what a backward pass needs of them. A row's
 * channels are taken in blocks of 128 (the last may be shorter); a block has
 * one exponent e and a code for each value x:
 *   e    = the least integer in [-100, 119] with max |x| <= 448 * 2^e,
 *   code = x * 2^-e rounded to the nearest e4m3 value (ties to even, at most
 *          448 in magnitude), standing for code * 2^e.
 * A value is off by at most 2^-4 of itself, or 2^-10 * 2^e where that is more.
 * The scale is a power of two so that what a code stands for is exact in bf16
 * (and in fp32): the products that read codes round nothing further. A block
 * with an infinity or NaN in it gets e = -128 and stands for NaNs throughout.
 * Magnitudes beyond 448 * 2^119 = 2.98e38 come back as that.
 * codes: [N] rows of d bytes, ld_codes apart (a multiple of 16, at least d);
 * exps: int8 [ceil(d/128)][N], rows ld_exps apart (a multiple of 16, at least
 * N). Of every row, the last too, d and N rounded up to 16 bytes may be read.
 * Whatever reads codes and exponents takes them to be lce_pack8's, unchecked:
 * exponents of -128 or -100 to 119, and the codes 0x7f and 0xff (NaN) only under
 * -128; others give other values, and not the same in every operator.
 * x and out are of `dtype`, rows ld_x and ld_out elements apart (0 stands for
 * d). d % 8 == 0, 8 <= d < 2^24, 0 <= N < 2^31, bases 16-byte aligned, row
 * strides multiples of 16 bytes.
 */
lce_status_t lce_pack8(lce_dtype_t dtype, const void *x, int64_t ld_x, int64_t N, int64_t d, uint8_t *codes,
                       int64_t ld_codes, int8_t *exps, int64_t ld_exps, lce_stream_t stream);
lce_status_t lce_unpack8(lce_dtype_t dtype, const uint8_t *codes, int64_t ld_codes, const int8_t *exps,
                         int64_t ld_exps, int64_t N, int64_t d, void *out, int64_t ld_out, lce_stream_t stream);

/*
 * The gradient of a linear layer's weight [n][k] from the gradient dy [T][n] of
 * its output and its input packed to 8 bits (T rows of k channels):
 *   dw[i][j] = sum over t of dy[t][i] * x[t][j],
 * x being what the codes stand for. dy is of `dtype`, dw of `dw_dtype` (fp32,
 * or bf16 with a bf16 dy), contiguous, rounded once from fp32 sums. bf16 dy
 * runs on the bf16 tensor cores with the codes widened on the way to them; an
 * fp32 dy is taken as three bf16 parts, which hold it exactly (but for parts
 * below 1.2e-38, that is values below 2^-109). The tensor cores truncate their
 * fp32 sums, so they take no more than 1024 tokens (fp32 dw; 512 of an fp32 dy)
 * or 32768 (bf16 dw) at a time, and what they make of those is added up in fp32.
 * Sums are in a fixed order (deterministic). n % 8 == 0, k % 8 == 0, n and k >= 8 and
 * < 2^24, 0 <= T < 2^30, bases and row strides of dy 16-byte aligned (ld_dy 0
 * stands for n). T = 0 writes zeros.
 * Scratch: lce_packed_wgrad_workspace_size bytes or NULL.
 */
typedef struct {
    lce_dtype_t dtype, dw_dtype;
    int64_t T, n, k;
    const void *dy;
    int64_t ld_dy;
    const uint8_t *codes;
    const int8_t *exps;
    int64_t ld_codes, ld_exps;
    void *dw;
    void *workspace;
    size_t workspace_bytes;
    lce_stream_t stream;
} lce_wgrad_t;
lce_status_t lce_packed_wgrad(const lce_wgrad_t *args);
size_t lce_packed_wgrad_workspace_size(const lce_wgrad_t *args);

/*
 * Gated recurrence over packed sequences, channel by channel, and its backward
 * pass: a token mixer whose memory is one state a sequence. With the gate's
 * logit g,
 *   a_t = 1 / (1 + exp(-g_t)),   h_t = a_t * h_{t-1} + (1 - a_t) * x_t,
 * h before a sequence's first token being its `state` (fp32 [B][d], NULL for
 * zeros) and `final` (fp32 [B][d], may be NULL, may be `state`) receiving h
 * after its last (the state itself for an empty sequence). Logits, not gates,
 * are the input, since gates near 1 have no neighbours in bf16 that would tell
 * a memory of 1000 tokens from an endless one. From the gradients dh of h and
 * dfinal of `final` (NULL for zeros) the backward goes through the tokens from
 * the last, with m after a sequence's last token being its dfinal:
 *   l_t = dh_t + m_{t+1},   m_t = a_t * l_t,
 *   dx_t = (1 - a_t) * l_t,   dg_t = l_t * (h_{t-1} - x_t) * a_t * (1 - a_t),
 *   dstate = m of the first token (dfinal itself for an empty sequence).
 * h is not read: the forward may leave `kept`, the fp32 state after every 128
 * tokens (fp32 [ceil(T/128)][d]; row c is h of token 128 c - 1, zeros for c =
 * 0), from which the backward forms h again.
 *
 * x and g are of `dtype`, T rows of d contiguous elements, ld_* apart, so they
 * may be slices of one projection's output, and dx and dg slices of its
 * gradient. cu: B+1 ascending token offsets (device int32, cu[0] = 0, cu[B] <=
 * T), NULL for B sequences of equal length; tokens after cu[B] belong to no
 * sequence (h = 0, zero gradients, kept = 0 behind them). Sequences may be empty. Values of one
 * sequence, infinities and NaN among them, never reach another. States and all
 * arithmetic are fp32; h, dx and dg are rounded once. a_t and 1 - a_t are off by
 * at most 9 units of 2^-24 of themselves (bf16 logits: 9 + |g_t|). Logits below -87 count
 * as -87, and above 87 1 - a_t is 0. d % 8 == 0, 8 <= d < 2^24, 0 <= T < 2^30, 1 <= B < 2^30, T a multiple
 * of B without offsets; bases 16-byte aligned, strides multiples of 16 bytes,
 * at least d (0 stands for d). Outputs must not overlap one another or, but for
 * `final`, any input. Deterministic. Offsets that are not ascending within the
 * tokens set LCE_DEV_SEQLENS; the outputs are then unspecified.
 */
typedef struct {
    lce_dtype_t dtype;
    int64_t B, T, d;
    const int32_t *cu;               /* [B+1] device, or NULL */
    const void *x, *g;
    int64_t ld_x, ld_g;
    const float *state;              /* [B][d], or NULL */
    float *kept;                     /* written by the forward (may be NULL), read by the backward */
    void *h;                         /* forward only, as is final */
    int64_t ld_h;
    float *final;
    const void *dh;                  /* backward only, as are the rest */
    int64_t ld_dh;
    const float *dfinal;             /* [B][d], or NULL */
    void *dx, *dg;
    int64_t ld_dx, ld_dg;
    float *dstate;                   /* [B][d], may be NULL */
    lce_stream_t stream;
} lce_recurrence_t;
lce_status_t lce_recurrence_forward(const lce_recurrence_t *args);
lce_status_t lce_recurrence_backward(const lce_recurrence_t *args);

/* ABI version: major*10000 + minor*100 + patch. */
int lce_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LCE_H */
