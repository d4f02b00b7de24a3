/*
 * chunk_dr.h -- C interface of the chunked gated delta-rule forward for MI355X (gfx950).
 *
 * The operation (page "PyPTO-Gym 的 chunk_kda 算子实战", sections 算子定位与算法背景
 * and M1-M4): for every sequence n and head h, starting from a K x V state S
 * (the transpose of initial_state[n, h], or zero), and for every token t in order,
 *
 *     S   <- diag(exp(g_t)) S                  per-dimension gate (g_t in R^K), or the
 *                                              scalar per-head gate g_t times the identity
 *     S   <- S + beta_t k_t (v_t - S^T k_t)^T
 *     o_t <- scale * S^T q_t
 *
 * evaluated chunk by chunk (chunk_size tokens; chunks restart at every sequence
 * start): an in-chunk prefix sum of g, the decayed strictly lower-triangular
 * A = beta k k^T, the inverse of (I + A), the w/u projections, and an fp32 state
 * carried from one chunk to the next.  The final state is returned as
 * [N, H, V, K], the transpose of the internal K x V matrix, as on that page
 * (section 算子签名与 I/O 规格).
 *
 * Two variants of the inputs are supported.  Grouped value heads: HV value heads (v, g,
 * beta, o, state) share H query/key heads in groups of HV / H, value head hv reading key
 * head hv / (HV / H), as in the workloads of the page "flash-linear-attention 中的
 * G_T_CONTIG" (H = 4, HV = 8).  In-kernel normalisation (the wrapper switch
 * use_qk_l2norm_in_kernel of the chunk_kda page, section 测试与验证体系): q_t and k_t are
 * replaced by x / sqrt(|x|^2 + 1e-6) over K before anything else.
 *
 * Conventions shared by every entry point:
 *  - Tensor pointers are DEVICE pointers to contiguous row-major buffers.
 *  - Tokens are packed: fixed-length batches are addressed as B*T consecutive tokens
 *    (sequence b owns tokens [b*T, (b+1)*T)); a varlen batch has B == 1 and its
 *    sequences are given by cu_seqlens.
 *  - The caller owns every buffer.  The library never allocates, frees, copies
 *    to the host or synchronises; kernels are queued on the given stream and the
 *    call returns immediately.
 *  - Errors are returned as cdr_status values; nothing is printed or thrown.
 *
 * Beside the operator stand the parts of a block and of a serving step that touch it: the norms,
 * gate and residual at a block's boundary (cdr_block_norm_*), the offsets, page tables and slots
 * of a step from its request lengths (cdr_build_page_tables), and latent attention, the softmax
 * attention of hybrid stacks: over a paged cache in the absorbed form (cdr_latent_decode_*), and
 * over packed sequences in the expanded form, with its gradients (cdr_latent_attn_*).
 */
#ifndef CHUNK_DR_H
#define CHUNK_DR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CDR_VERSION 10

typedef enum {
    CDR_OK = 0,
    CDR_ERR_NULL_ARG = 1,      /* a required pointer is NULL */
    CDR_ERR_BAD_SHAPE = 2,     /* non-positive or inconsistent sizes */
    CDR_ERR_UNSUPPORTED = 3,   /* K or V != 128, chunk_size not 64 or 128, unknown gate, type or
                                  activation, a width the entry point does not take */
    CDR_ERR_VARLEN_BATCH = 4,  /* cu_seqlens given with B != 1 */
    CDR_ERR_WORKSPACE = 5,     /* workspace NULL or smaller than cdr_workspace_bytes() */
    CDR_ERR_HIP = 6,           /* a kernel launch failed (hipGetLastError) */
    CDR_ERR_SCRATCH_LIMIT = 7  /* chunk_dr_fwd_noalloc: the problem needs more workspace than its
                                  static array holds (CDR_NOALLOC_SCRATCH_BYTES) */
} cdr_status;

typedef enum {
    CDR_GATE_PER_DIM = 0,      /* g [B*T, HV, K] fp32: per-key-dimension log gate (KDA) */
    CDR_GATE_PER_HEAD = 1      /* g [B*T, HV] fp32: one log gate per token and head (Gated DeltaNet) */
} cdr_gate;

/* Problem description.  All fields are plain host values. */
typedef struct {
    int32_t B;                  /* batch rows; must be 1 when varlen != 0 */
    int32_t T;                  /* tokens per batch row (total packed tokens when varlen) */
    int32_t H;                  /* query/key heads */
    int32_t K;                  /* key dimension; must be 128 */
    int32_t V;                  /* value dimension; must be 128 */
    int32_t N;                  /* sequences: B when varlen == 0, else len(cu_seqlens) - 1 */
    int32_t gate;               /* cdr_gate */
    int32_t chunk_size;         /* 64 or 128 */
    float scale;                /* multiplies q; the usual choice is K^-0.5 */
    int32_t has_initial_state;  /* initial_state is read when non-zero, else S starts at 0 */
    int32_t output_final_state; /* final_state is written when non-zero */
    int32_t varlen;             /* cu_seqlens is read when non-zero */
    int32_t HV;                 /* value heads (v, g, beta, o and the state); 0 means H.  Must be a
                                   multiple of H: value head hv uses query/key head hv / (HV / H) */
    int32_t qk_l2norm;          /* when non-zero, q and k are L2-normalised over K per token inside
                                   the kernels, x / sqrt(|x|^2 + 1e-6) */
} cdr_problem;

/*
 * Host-only validation of a problem description; never touches the device.  The rules are the
 * input checks of the chunk_kda page's host wrapper (section 主机侧 wrapper 与输入校验: K = V =
 * 128, a batch of one with cu_seqlens, shapes that agree), with the page's fixed-length
 * T % 128 == 0 relaxed: any T is accepted, a short last chunk being zero-filled as the page does
 * for varlen tails.  Dtypes are not described here (the interface is untyped); the Python
 * binding checks them.  Returns CDR_OK or the first violated rule (see cdr_status).
 */
cdr_status cdr_check(const cdr_problem* p);

/*
 * Bytes of device workspace chunk_dr_fwd needs for problem p (0 if p is invalid).  The
 * workspace replaces the intermediate tensors of the page's wrapper (section 主机侧 wrapper 与
 * 输入校验 allocates them per call); here the caller owns it.  The size depends only on the
 * shape fields (B, T, H, HV, K, V, N, chunk_size): per chunk and value head the factors of the
 * chunk step (-P split in two bf16 parts, B in fp32, Q, U, exp(gamma_C)) and the chunk-entry
 * state, 224.5 KiB at chunk_size 128 and 192.5 KiB at 64, plus up to 512 per-workgroup scratch
 * slots of 36 KiB (20 KiB at 64).
 */
size_t cdr_workspace_bytes(const cdr_problem* p);

/*
 * Chunked gated delta-rule forward.
 *
 *   q, k          bf16 [B*T, H, K]   queries and keys
 *   v             bf16 [B*T, HV, V]  values (HV value heads, see cdr_problem)
 *   g             fp32 [B*T, HV, K] (CDR_GATE_PER_DIM) or [B*T, HV] (CDR_GATE_PER_HEAD);
 *                 log-domain forget gate.  Supported: every finite g <= 0 (the page's gates
 *                 are logsigmoid values); the in-chunk sums of g must be finite in fp32.
 *                 A key dimension whose gate sums to more than 32 in magnitude over half a
 *                 16-token tile takes, in that tile, pivots that bound every factor by 1 and
 *                 an exact sum over the tile's own pairs (one exponential per pair); the
 *                 other dimensions and tiles are unaffected.  With every dimension that
 *                 strong, the forward takes about 40 % longer than with ordinary gates; with
 *                 a few strong dimensions, about 8 %.  g > 0 is outside the contract (the
 *                 state can then grow without bound).
 *   beta          fp32 [B*T, HV]     delta-rule step size
 *   initial_state fp32 [N, HV, V, K] read when p->has_initial_state, else may be NULL
 *   cu_seqlens    int32 [N + 1]      device array of sequence offsets into the packed token
 *                                    axis (0 = cu[0] <= cu[1] <= ... <= cu[N] = T); read when
 *                                    p->varlen, else may be NULL.  Its contents are not
 *                                    validated; offsets outside [0, T] are undefined behaviour.
 *   o             bf16 [B*T, HV, V]  output, written for every token of every sequence
 *   final_state   fp32 [N, HV, V, K] written when p->output_final_state, else may be NULL.
 *                                    An empty sequence returns its initial state (or zeros).
 *   workspace     device buffer of at least cdr_workspace_bytes(p) bytes, 256-byte aligned;
 *                 its contents on entry do not matter.  It must not be used by another call
 *                 until the kernels of this call have finished on `stream`.
 *   stream        hipStream_t to launch on (NULL = the default stream)
 *
 * The result does not depend on the contents of the workspace or on previous calls:
 * repeated calls on the same inputs give bit-identical o and final_state.
 * Returns CDR_OK after queueing the kernels, or an error status without launching
 * anything (CDR_ERR_HIP if a launch failed).
 */
cdr_status chunk_dr_fwd(const cdr_problem* p,
                        const void* q, const void* k, const void* v,
                        const float* g, const float* beta,
                        const float* initial_state, const int32_t* cu_seqlens,
                        void* o, float* final_state,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * Device-side check of the contents of cu_seqlens, which chunk_dr_fwd does not read on the
 * host and does not validate.  The rules are the varlen input checks of the chunk_kda page's
 * host wrapper (section 主机侧 wrapper 与输入校验) and of the G_T_CONTIG page's varlen checklist
 * (section 3): the offsets start at 0, never decrease, and end at the total token count.
 *
 *   cu_seqlens  int32 [N + 1] device array
 *   N           sequences, >= 1
 *   T           total packed tokens, >= 0 (the problem's T)
 *   result      device int32, written by the check: 0 when every rule holds, else i + 1 for
 *               the first index i in 0..N where one fails (cu[0] != 0; cu[i] < cu[i - 1];
 *               cu[i] outside 0..T; cu[N] != T)
 *   stream      hipStream_t to launch on (NULL = the default stream)
 *
 * Queues one small kernel and returns without waiting; read *result after the stream has
 * finished it.  The kernel writes *result on every call, so no clearing is needed and the call
 * can be captured in a graph.  Returns CDR_ERR_NULL_ARG for a NULL array or result,
 * CDR_ERR_BAD_SHAPE for N < 1 or T < 0, CDR_ERR_HIP if the launch failed, else CDR_OK.
 */
cdr_status cdr_check_cu_seqlens(const int32_t* cu_seqlens, int32_t N, int32_t T, int32_t* result, void* stream);

/*
 * The same forward, split into its three kernel stages so that each can be timed or
 * profiled on its own.  `stages` is a bit mask of
 *   CDR_STAGE_INTRA  (1)  per-chunk work independent of the carried state: gate prefix sum,
 *                         decayed A and its inverse, w, u (page sections M1-M3), and the
 *                         factors of the chunk step of section M4 re-associated, P = kg^T w,
 *                         B = kg^T u, Q = qg - A2 w, U = A2 u
 *   CDR_STAGE_CHAIN  (2)  the sequential chunk-to-chunk state recurrence
 *                         S <- exp(gamma_C) S - P S + B, the chunk-entry states and the final
 *                         state (section M4; the same sums as u - w S carried through v_new)
 *   CDR_STAGE_OUTPUT (4)  o = Q S_entry + U for every chunk (= qg S + A2 v_new, section M4)
 * Stages run in this order.  A stage reads what earlier stages left in the workspace, so a
 * call with a stage whose predecessors are not in `stages` is only meaningful after a call
 * with the same problem, inputs and workspace that ran them.  chunk_dr_fwd(...) is
 * chunk_dr_fwd_stages(..., CDR_STAGE_ALL, stream).  Arguments and errors as chunk_dr_fwd;
 * a mask outside 1..7 returns CDR_ERR_UNSUPPORTED.
 */
#define CDR_STAGE_INTRA 1
#define CDR_STAGE_CHAIN 2
#define CDR_STAGE_OUTPUT 4
#define CDR_STAGE_ALL 7
cdr_status chunk_dr_fwd_stages(const cdr_problem* p,
                               const void* q, const void* k, const void* v,
                               const float* g, const float* beta,
                               const float* initial_state, const int32_t* cu_seqlens,
                               void* o, float* final_state,
                               void* workspace, size_t workspace_bytes,
                               int32_t stages, void* stream);

/* ------------------------------------------------------------------------------------------
 * The forward for callers that cannot allocate device memory: code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation.
 *
 * chunk_dr_fwd_noalloc is chunk_dr_fwd (same arguments, same kernels, same bits) with its
 * workspace in a static device array of CDR_NOALLOC_SCRATCH_BYTES owned by the library: one such
 * array per device the entry point runs on, taken when the library's code for it is first used
 * on that device and held until the process ends.  It allocates and frees nothing.  Problems
 * whose cdr_workspace_bytes() exceeds CDR_NOALLOC_SCRATCH_BYTES are rejected with
 * CDR_ERR_SCRATCH_LIMIT before anything is launched; the limit holds the workspace of 8192
 * tokens x 16 heads at chunk_size 128.  The caller still passes (and owns) inputs and outputs.
 *
 * Every call on one device uses that device's one array: two calls whose kernels overlap in time
 * on the same device (different streams, or different threads without ordering) race on it and
 * give undefined results.  Calls ordered on one stream are safe.  The forward reads nothing of
 * the workspace that the same call has not written, so what a previous call left there does not
 * matter and nothing is cleared.
 * ------------------------------------------------------------------------------------------ */
#define CDR_NOALLOC_SCRATCH_BYTES (256u * 1024u * 1024u)
cdr_status chunk_dr_fwd_noalloc(const cdr_problem* p,
                                const void* q, const void* k, const void* v,
                                const float* g, const float* beta,
                                const float* initial_state, const int32_t* cu_seqlens,
                                void* o, float* final_state, void* stream);

/* ------------------------------------------------------------------------------------------
 * Context parallelism, the part one device computes (page "flash-linear-attention KCP 精度失效
 * 根因排查手册": a sequence split over ranks, each rank summarising its segment, the summaries
 * exchanged and merged so that each rank learns the state entering its segment).
 *
 * The forward of a segment is affine in its initial state: in the [V, K] layout of the states,
 * final = initial M + X, where X is the final state from a zero start and M ([K, K]) is the
 * product of the segment's chunk maps (exp(gamma_C) - P per chunk, transposed to this layout).
 *
 * chunk_dr_segment_map: M [N, HV, K, K] and X [N, HV, V, K] of every sequence of problem p
 *   (each sequence is one segment).  Arguments as chunk_dr_fwd; p->has_initial_state and
 *   p->output_final_state are ignored.  Uses the forward workspace (cdr_workspace_bytes(p)).
 * chunk_dr_merge_states: given the maps of R consecutive segments of one sequence (M
 *   [R, HV, K, K], X [R, HV, V, K], in order) and the state entering the first (initial_state
 *   [HV, V, K], or NULL for zeros), writes s_in [R + 1, HV, V, K]: s_in[0] = initial_state,
 *   s_in[r + 1] = s_in[r] M[r] + X[r], the state entering segment r + 1; s_in[R] is the final
 *   state.  Running segment r's forward from s_in[r] gives the outputs of the unsplit sequence.
 * On several devices the (M, X) pairs would be all-gathered between the two calls; here they are
 * in one device's memory.
 * ------------------------------------------------------------------------------------------ */
cdr_status chunk_dr_segment_map(const cdr_problem* p,
                                const void* q, const void* k, const void* v,
                                const float* g, const float* beta, const int32_t* cu_seqlens,
                                float* M, float* X,
                                void* workspace, size_t workspace_bytes, void* stream);

cdr_status chunk_dr_merge_states(int32_t R, int32_t HV, int32_t K, int32_t V,
                                 const float* M, const float* X, const float* initial_state,
                                 float* s_in, void* stream);

/* ------------------------------------------------------------------------------------------
 * Backward of the chunked forward.
 *
 * The gradients of L = sum(o * do) + sum(final_state * dht) with respect to q, k, v, g, beta and
 * initial_state, for the forward chunk_dr_fwd computes with the same problem p (the vector-
 * Jacobian products of the per-token rule of the chunk_kda page, section 算子定位与算法背景).
 * The backward recomputes what it needs from the inputs (nothing is kept from the forward call):
 * per chunk the decayed blocks, the inverse of (I + A) and the chunk's affine state map, the
 * chunk entry states by a forward chain, the gradients of the chunk exit states by a reverse
 * chain, then all input gradients chunk by chunk.  Storage and the serial chains are fp32; the
 * products run on split-bf16 MFMA (about 16 mantissa bits per operand).
 *
 *   q, k, v, g, beta, initial_state, cu_seqlens  as chunk_dr_fwd
 *   d_o     bf16 [B*T, HV, V]      gradient of o
 *   dht     fp32 [N, HV, V, K]     gradient of the final state, or NULL (zero)
 *   dq, dk  fp32 [B*T, H, K]       written (summed over the value heads of a group)
 *   dv      fp32 [B*T, HV, V]      written
 *   dg      fp32, the shape of g   written
 *   dbeta   fp32 [B*T, HV]         written
 *   dh0     fp32 [N, HV, V, K]     written when p->has_initial_state, else may be NULL
 *   workspace  at least cdr_bwd_workspace_bytes(p) bytes, 256-byte aligned, contents irrelevant
 * Rows of padded or empty chunks are not written; every token of every sequence is.
 * p->output_final_state is ignored.  Errors as chunk_dr_fwd.
 * ------------------------------------------------------------------------------------------ */
size_t cdr_bwd_workspace_bytes(const cdr_problem* p);

cdr_status chunk_dr_bwd(const cdr_problem* p,
                        const void* q, const void* k, const void* v,
                        const float* g, const float* beta,
                        const float* initial_state, const int32_t* cu_seqlens,
                        const void* d_o, const float* dht,
                        float* dq, float* dk, float* dv, float* dg, float* dbeta, float* dh0,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same backward split into its stages, for timing and profiling.  `stages` is a bit mask of
 *   CDR_BWD_PREP   (1)  per chunk: decayed blocks, (I + A)^-1, w, u, the chunk's state map P, B
 *                       and Q^T do
 *   CDR_BWD_CHAINS (2)  the forward chain (chunk entry states) and the reverse chain (gradients
 *                       of the chunk exit states, dh0)
 *   CDR_BWD_LOCAL  (4)  per chunk: dq, dk, dv, dg, dbeta (and the sum over grouped value heads)
 * Stages run in this order and read what earlier stages left in the workspace, as for
 * chunk_dr_fwd_stages.  chunk_dr_bwd(...) is chunk_dr_bwd_stages(..., CDR_BWD_ALL, stream).
 */
#define CDR_BWD_PREP 1
#define CDR_BWD_CHAINS 2
#define CDR_BWD_LOCAL 4
#define CDR_BWD_ALL 7
cdr_status chunk_dr_bwd_stages(const cdr_problem* p,
                               const void* q, const void* k, const void* v,
                               const float* g, const float* beta,
                               const float* initial_state, const int32_t* cu_seqlens,
                               const void* d_o, const float* dht,
                               float* dq, float* dk, float* dv, float* dg, float* dbeta, float* dh0,
                               void* workspace, size_t workspace_bytes, int32_t stages, void* stream);

/* ------------------------------------------------------------------------------------------
 * Per-token (recurrent) forward: the decode path.
 *
 * The decode-side companion of the chunked operator (page "PyPTO-Gym 的 chunk_kda 算子实战",
 * section 与其他 KDA 算子的关系): the same update rule as above, applied token by token to an
 * fp32 [HV, V, K] state per sequence, which may be kept in place in a pool of states addressed
 * by slot indices (ssm_state_indices) and may keep one state per draft token for speculative
 * decoding (num_accepted_tokens).  The page names these arguments without defining them; the
 * reading implemented here:
 *
 *  CDR_STATE_SEPARATE  initial_state [N, HV, V, K] (or zeros) in, final_state [N, HV, V, K]
 *                      out, exactly as chunk_dr_fwd.  initial_state and final_state may be the
 *                      same buffer (the update is then in place).
 *  CDR_STATE_POOL      state_pool [num_slots, HV, V, K] fp32, read and written in place;
 *                      ssm_state_indices int32 [N]: sequence n starts from slot idx[n] and its
 *                      state after its last token is written back to slot idx[n].
 *  CDR_STATE_POOL_SPEC ssm_state_indices int32 [N, index_cols]: draft position t of sequence n
 *                      owns slot idx[n, t].  The sequence starts from slot idx[n, a_n - 1], with
 *                      a_n = num_accepted_tokens[n] (int32 [N]; NULL means a_n = 1), and its
 *                      state after its own token t is written to slot idx[n, t] for every
 *                      t < index_cols (later positions have no slot and are not stored).
 *
 * In both pool modes a slot index outside [0, num_slots) marks padding: a start index outside
 * it (or a_n outside 1..index_cols) makes the sequence a padding entry, whose o rows are set to
 * zero and which reads and writes no state; a write index outside it skips that one write.
 * Indices are read on the device and never cause an access outside the pool.  Every start
 * state is read before any state of the same sequence is written, so a sequence may write the
 * slot it starts from; two sequences writing the same slot, or one writing a slot that another
 * starts from, give an undefined result.
 *
 * No workspace: the kernels keep each state row in registers for the whole sequence.
 * ------------------------------------------------------------------------------------------ */
typedef enum {
    CDR_STATE_SEPARATE = 0,
    CDR_STATE_POOL = 1,
    CDR_STATE_POOL_SPEC = 2
} cdr_state_mode;

typedef struct {
    int32_t B;                  /* batch rows; must be 1 when varlen != 0 */
    int32_t T;                  /* tokens per batch row (total packed tokens when varlen) */
    int32_t H;                  /* query/key heads */
    int32_t HV;                 /* value heads, a multiple of H; 0 means H */
    int32_t K;                  /* must be 128 */
    int32_t V;                  /* must be 128 */
    int32_t N;                  /* sequences: B when varlen == 0, else len(cu_seqlens) - 1 */
    int32_t gate;               /* cdr_gate */
    float scale;                /* multiplies q */
    int32_t varlen;             /* cu_seqlens is read when non-zero */
    int32_t qk_l2norm;          /* normalise q and k per token inside the kernel, as chunk_dr_fwd */
    int32_t state_mode;         /* cdr_state_mode */
    int32_t has_initial_state;  /* CDR_STATE_SEPARATE: initial_state is read, else zeros */
    int32_t output_final_state; /* CDR_STATE_SEPARATE: final_state is written */
    int32_t num_slots;          /* pool modes: entries of state_pool (> 0) */
    int32_t index_cols;         /* CDR_STATE_POOL_SPEC: columns of ssm_state_indices (> 0) */
} cdr_recurrent_problem;

/* Host-only validation of a recurrent problem description. */
cdr_status cdr_recurrent_check(const cdr_recurrent_problem* p);

/*
 * Per-token forward.
 *
 *   q, k, v, g, beta, cu_seqlens, o   as chunk_dr_fwd (device pointers, same layouts)
 *   initial_state, final_state        CDR_STATE_SEPARATE only (NULL allowed when the matching
 *                                     flag is 0); ignored in the pool modes
 *   state_pool                        pool modes: fp32 [num_slots, HV, V, K], updated in place
 *   ssm_state_indices                 pool modes: int32 [N] (CDR_STATE_POOL) or
 *                                     [N, index_cols] (CDR_STATE_POOL_SPEC), device
 *   num_accepted_tokens               CDR_STATE_POOL_SPEC: int32 [N], device, or NULL
 *   stream                            hipStream_t (NULL = default stream)
 *
 * One kernel is queued; nothing is allocated, copied to the host or synchronised.  Repeated
 * calls on the same inputs give bit-identical results.  Returns CDR_OK after queueing, or an
 * error status without launching anything (CDR_ERR_HIP if the launch failed).
 */
cdr_status chunk_dr_recurrent_fwd(const cdr_recurrent_problem* p,
                                  const void* q, const void* k, const void* v,
                                  const float* g, const float* beta, const int32_t* cu_seqlens,
                                  const float* initial_state, float* final_state,
                                  float* state_pool, const int32_t* ssm_state_indices,
                                  const int32_t* num_accepted_tokens,
                                  void* o, void* stream);

/* ------------------------------------------------------------------------------------------
 * The block boundary: the norm after a token mixer, its gate, the residual and the norm before the
 * next block, in one pass over the data.  For every row (a token, or a token and head), with
 * rstd(x) = 1 / sqrt(mean x^2 + eps) over the row's D elements:
 *
 *     n = y * rstd(y) * weight                      (has_weight; else n = y)
 *     r = residual + alpha * res_scale * a(gate) * n
 *                                                   a(z) = sigmoid(z) or z * sigmoid(z); residual,
 *                                                   res_scale and gate each optional
 *     h = r * rstd(r) * next_weight                 (has_next)
 *
 * `out` receives r and `next_out` h.  Arithmetic is fp32 whatever the types (squares beyond 3e38
 * overflow); h is formed from the fp32 r and each output is rounded once.  With D = 128, a gate, a
 * weight and nothing else this is the gated norm of o [.., HV, V] per head; with everything it is a
 * whole block boundary.
 *
 *   y, gate      dtype, rows of D contiguous elements (strides below)
 *   residual     res_dtype, likewise
 *   weight, res_scale, next_weight   fp32 [D]
 *   out          res_dtype with a residual, else dtype; dense [rows, D]
 *   next_out     dtype, dense [rows, D]
 * out may be residual itself, and next_out y itself, when those are dense (every element is read
 * before it is written, by the same thread); any other overlap of inputs and outputs is undefined.
 *
 * Strides: row i of an operand starts at element (i / inner) * stride[0] + (i % inner) * stride[1]
 * (inner 0 or 1: i * stride[0]), so a slice [T, HV, 128] of a wider projection is read in place.
 * D is 1 to 8192.  Rows of 16-byte aligned operands with D and strides divisible by 8 are read and
 * written 16 bytes at a time, others element by element.
 * ------------------------------------------------------------------------------------------ */
typedef enum {
    CDR_BF16 = 0,
    CDR_F32 = 1
} cdr_dtype;

typedef enum {
    CDR_ACT_NONE = 0,          /* no gate */
    CDR_ACT_SIGMOID = 1,
    CDR_ACT_SILU = 2
} cdr_act;

typedef struct {
    int32_t rows;
    int32_t D;
    int32_t dtype;              /* cdr_dtype of y, gate, next_out and their gradients */
    int32_t res_dtype;          /* cdr_dtype of residual, out and their gradients (has_residual) */
    int32_t gate_act;           /* cdr_act */
    int32_t has_weight;
    int32_t has_residual;
    int32_t has_scale;
    int32_t has_next;
    int32_t inner;              /* rows of one outer step, a divisor of rows; 0 means 1 */
    float alpha;
    float eps;                  /* >= 0 */
    int64_t y_stride[2];        /* elements: outer, inner */
    int64_t gate_stride[2];
    int64_t residual_stride[2];
} cdr_block_norm_problem;

/* Host-only validation of a block norm problem. */
cdr_status cdr_block_norm_check(const cdr_block_norm_problem* p);

/* One kernel on `stream`; nothing for rows == 0.  Pointers whose flag is 0 may be NULL. */
cdr_status cdr_block_norm_fwd(const cdr_block_norm_problem* p, const void* y, const void* gate, const void* residual,
                              const float* weight, const float* res_scale, const float* next_weight, void* out,
                              void* next_out, void* stream);

/*
 * Gradients of L = sum(out * d_out) + sum(next_out * d_next).  Inputs as the forward, which is
 * recomputed (nothing is kept from it).
 *
 *   d_out    type of out, dense; NULL means zero, allowed with has_next
 *   d_next   dtype, dense (has_next)
 *   dy, dgate (dtype), dresidual (res_dtype)      dense [rows, D], written where their input is given
 *   dweight, dres_scale, dnext_weight             fp32 [D], sums over the rows (zeros for rows == 0)
 *   workspace  at least cdr_block_norm_bwd_workspace_bytes(p) bytes, 16-byte aligned, contents
 *              irrelevant, not to be used by another call until this one's kernels have finished
 * No output may overlap an input.  Column sums are added in a fixed order: repeated calls give the
 * same bits.
 */
size_t cdr_block_norm_bwd_workspace_bytes(const cdr_block_norm_problem* p);

cdr_status cdr_block_norm_bwd(const cdr_block_norm_problem* p, const void* y, const void* gate, const void* residual,
                              const float* weight, const float* res_scale, const float* next_weight, const void* d_out,
                              const void* d_next, void* dy, void* dgate, void* dresidual, float* dweight,
                              float* dres_scale, float* dnext_weight, void* workspace, size_t workspace_bytes,
                              void* stream);

/* ------------------------------------------------------------------------------------------
 * Bookkeeping of a serving step on the device, from the lengths of its requests: the offsets of its
 * packed tokens (cu_seqlens), positions, the page table and the slots of a paged cache, with new pages
 * taken from a list of free ones.  Latent attention takes the offsets as they are, also in a step padded
 * to a captured size, where cu_seqlens[N] < max_tokens; the chunked and the per-token forward of the delta
 * rule need offsets that end at their T, so there max_tokens is the step's own number of tokens.  All arrays are int32 on the device;
 * with q_n = max(query_lens[n], 0), c_n = max(context_lens[n], 0), P = page_size, W = table_cols:
 *
 *     cu_seqlens[0] = 0, cu_seqlens[n + 1] = min(cu_seqlens[n] + q_n, max_tokens)
 *     len_n   = c_n + (cu_seqlens[n + 1] - cu_seqlens[n])       -> seq_lens[n]
 *     held_n  = min(ceil(c_n / P), W)       pages that the request holds already
 *     upto_n  = min(ceil(len_n / P), W)     pages that it holds after the step
 *     head    = clip(free_head[0], 0, num_free);  first_n = head + sum of (upto_m - held_m), m < n
 *     block_table[n, held_n + j] = free_pages[first_n + j], -1 behind the list's end
 *     free_head_out[0] = min(first_N, num_free)
 *     shortage[0] = max(first_N - num_free, 0) + sum of (ceil(len_n / P) - upto_n)
 *
 * and for token t of request n (cu_seqlens[n] <= t < cu_seqlens[n + 1]), p = c_n + t - cu_seqlens[n]:
 *
 *     positions[t] = p,   slot_map[t] = block_table[n, p / P] * P + p % P
 *
 * slot_map[t] = -1 where that page is missing (p / P >= W, a negative entry, or a slot beyond
 * int32), which the cache writers skip.  Tokens behind the last request (t >= cu_seqlens[N]) get
 * position 0 and slot -1, so that a step padded to a captured size writes nothing for them.  Table
 * entries other than the new pages' are left as they were.  free_pages[free_head:] is the stack of
 * free pages: a caller gives pages back by writing them below the head and lowering it.
 * shortage[0] counts the pages that were wanted and are not there; a step with a shortage is still
 * well defined (no access leaves the arrays).  free_head_out may be free_head (in place); no other
 * output may overlap an input.
 *
 *   query_lens, context_lens [N];  block_table [N, table_cols], updated in place
 *   free_pages [num_free];  free_head, free_head_out, shortage [1]
 *   cu_seqlens [N + 1];  seq_lens [N];  positions, slot_map [max_tokens]
 *   workspace  at least cdr_page_tables_workspace_bytes(N) bytes
 * One kernel is queued for up to 2048 tokens, two beyond.
 * ------------------------------------------------------------------------------------------ */
size_t cdr_page_tables_workspace_bytes(int32_t N);

cdr_status cdr_build_page_tables(int32_t N, int32_t table_cols, int32_t num_free, int32_t page_size, int32_t max_tokens,
                                 const int32_t* query_lens, const int32_t* context_lens, int32_t* block_table,
                                 const int32_t* free_pages, const int32_t* free_head, int32_t* free_head_out,
                                 int32_t* cu_seqlens, int32_t* seq_lens, int32_t* positions, int32_t* slot_map,
                                 int32_t* shortage, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------------
 * Latent attention, absorbed form, over a paged cache (decode and a few draft tokens).
 *
 * A cached key is CDR_LATENT_DIM + CDR_LATENT_ROPE = 512 + 64 bf16, one for all heads: the latent
 * c_j, which is the value too, and the rope part r_j.  q_latent is the query with the key's
 * up-projection absorbed.  For token i of sequence n's L_n new tokens and every head,
 *
 *     o = sum_j p_j c_j,   p = softmax over j < seq_lens[n] - L_n + i + 1 of
 *                              scale (q_latent . c_j + q_rope . r_j)
 *     lse = log of the sum of exp of those scores (natural)
 *
 * so seq_lens counts the new tokens, whose keys are written first (cdr_latent_cache_write).  Key j
 * of sequence n is row block_table[n, j / page_size] * page_size + j % page_size of the cache.
 * Keys beyond table_cols * page_size or 2^31 - 256 and keys whose page lies outside [0, num_pages) do not
 * exist: they are masked and not read; seq_lens may count them, and the rows' limits count from it all the
 * same.  A row left without keys gives o = 0 and lse = -inf.  What lies behind a sequence's last key,
 * in its last page or elsewhere, does not affect it, whatever it holds; keys below seq_lens[n] must be
 * finite, those that a row's causal limit hides from it too (they meet a weight of zero).
 *
 *   q_latent   bf16 [tokens, H, 512], q_rope bf16 [tokens, H, 64]: strides (token, head) in
 *              elements, multiples of 8; tokens = N * T, or T in all when varlen
 *   cache      bf16 [num_pages, page_size, 576], page_size a power of two
 *   block_table int32 [N, table_cols], seq_lens int32 [N], cu_seqlens int32 [N + 1] (varlen;
 *              offsets do not fall and are clipped to [0, T])
 *   o          bf16 [tokens, H, 512], lse fp32 [tokens, H] or NULL; rows that no sequence holds (in
 *              front of the first offset, behind the last) are left as they were, or become 0 and
 *              -inf with varlen CDR_VARLEN_FILL
 *   workspace  at least cdr_latent_decode_workspace_bytes(p) bytes, 16-byte aligned, contents
 *              irrelevant, not to be used by another call until this one's kernels have finished
 * q, cache, o and the workspace are 16-byte aligned; no output may overlap an input.  Scores and
 * sums are fp32; the weights p_j
 * enter the second product as bf16 (the first product's sum of them does not).  Lengths are read on
 * the device, so a captured call serves any lengths.  Repeated calls give the same bits.
 * ------------------------------------------------------------------------------------------ */
#define CDR_VARLEN_FILL 2      /* varlen of latent attention: packed, and rows and keys that no sequence
                                  holds are written too */
#define CDR_LATENT_DIM 512
#define CDR_LATENT_ROPE 64

typedef struct {
    int32_t N;                  /* sequences */
    int32_t T;                  /* new tokens of each sequence (all packed tokens when varlen) */
    int32_t H;                  /* heads */
    int32_t varlen;             /* cu_seqlens is read when non-zero */
    int32_t num_pages;
    int32_t page_size;          /* a power of two; num_pages * page_size < 2^31 */
    int32_t table_cols;         /* columns of block_table */
    float scale;
    int64_t qc_stride[2];       /* q_latent: token, head */
    int64_t qr_stride[2];       /* q_rope: token, head */
} cdr_latent_decode_problem;

/* Host-only validation of a latent decode problem. */
cdr_status cdr_latent_decode_check(const cdr_latent_decode_problem* p);

size_t cdr_latent_decode_workspace_bytes(const cdr_latent_decode_problem* p);

/* Two kernels on `stream`. */
cdr_status cdr_latent_decode_fwd(const cdr_latent_decode_problem* p, const void* q_latent, const void* q_rope,
                                 const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                                 const int32_t* cu_seqlens, void* o, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * Writes T tokens' latents into the cache: row slot_map[t] of cache [num_pages * page_size, 576]
 * becomes (c[t], k_rope[t]).  Slots outside the cache are skipped (padding, as
 * cdr_build_page_tables marks it with -1); two tokens with one slot give an undefined row.  c and k_rope
 * may be rows of the cache itself where no slot names one of them.
 *   c bf16 [T, 512], k_rope bf16 [T, 64]: token strides in elements, multiples of 8; c, k_rope
 *   and cache 16-byte aligned; slot_map int32 [T]
 */
cdr_status cdr_latent_cache_write(int32_t T, int32_t num_pages, int32_t page_size, const void* c, const void* k_rope,
                                  int64_t c_stride, int64_t k_rope_stride, void* cache, const int32_t* slot_map,
                                  void* stream);

/* ------------------------------------------------------------------------------------------
 * Latent attention, expanded form, over packed or equal-length sequences: prefill and training.
 *
 * Every head has its own keys and values, expanded from the latents, and all heads share the rope
 * part of the key.  For row i of sequence n's L_q rows and its L_k keys (causal; the last row sees
 * all keys, so L_k - L_q earlier keys are a context),
 *
 *     o_i = sum_j p_ij v_j,  p_i = softmax over j < L_k - L_q + i + 1 of
 *                                  scale (q_i[:128] . k_nope_j + q_i[128:] . k_rope_j)
 *     lse_i = log of the sum of exp of those scores (natural)
 *
 * A row without keys (L_q > L_k) gives o = 0 and lse = -inf, and no gradient.
 *
 *   q        bf16 [tokens, H, 192]: nope, then rope part     strides (token, head)
 *   k_nope   bf16 [keys, H, 128]                             strides (token, head)
 *   k_rope   bf16 [keys, 64]                                 stride of a token
 *   v        bf16 [keys, H, 128]                             strides (token, head)
 *   cu_seqlens, cu_seqlens_k  int32 [N + 1], varlen: rows' and keys' offsets, which do not fall and are
 *            clipped to [0, T] and [0, Tk]; may be the same array.  Else every sequence has T rows and Tk keys.
 *   o        bf16 [tokens, H, 128], lse fp32 [tokens, H]; dense.  Rows that no sequence holds (in front
 *            of the first offset, behind the last) are left as they were, or become 0 and -inf with
 *            varlen CDR_VARLEN_FILL.
 * Strides are in elements, multiples of 8, not negative and below 2^23, so k_nope and v may be the
 * two halves of one projection [keys, H, 256]; all but lse are 16-byte aligned.  scale is positive.
 * Values of a sequence must be finite, also those that the causal limit hides from a row (they meet
 * weights of zero); those of other sequences do not matter.  No output may overlap an input.
 * Scores and sums are fp32, the weights enter the second product as bf16.  Repeated calls give the
 * same bits.
 * ------------------------------------------------------------------------------------------ */
#define CDR_LATENT_NOPE 128
#define CDR_LATENT_VALUE 128

typedef struct {
    int32_t N;                  /* sequences */
    int32_t T;                  /* rows of each sequence (all packed rows when varlen) */
    int32_t Tk;                 /* keys of each sequence (all packed keys when varlen) */
    int32_t H;                  /* heads, at most 32768 */
    int32_t varlen;             /* cu_seqlens and cu_seqlens_k are read when non-zero */
    float scale;
    int64_t q_stride[2];        /* token, head */
    int64_t k_stride[2];
    int64_t v_stride[2];
    int64_t k_rope_stride;      /* token */
} cdr_latent_attn_problem;

/* Host-only validation of a latent attention problem. */
cdr_status cdr_latent_attn_check(const cdr_latent_attn_problem* p);

/* One kernel on `stream`, no workspace. */
cdr_status cdr_latent_attn_fwd(const cdr_latent_attn_problem* p, const void* q, const void* k_nope, const void* k_rope,
                               const void* v, const int32_t* cu_seqlens, const int32_t* cu_seqlens_k, void* o, float* lse,
                               void* stream);

/*
 * Gradients of L = sum(o * d_o), from the forward's o and lse.
 *
 *   o, lse    as the forward wrote them;  d_o bf16 [tokens, H, 128] dense
 *   dq        bf16 [tokens, H, 192], dk_nope bf16 [keys, H, 128], dk_rope bf16 [keys, 64] (the sum
 *             over the heads, added in fp32), dv bf16 [keys, H, 128]; dense.  Rows and keys that no
 *             sequence holds (in front of the first offset, behind the last) are left as they were,
 *             or set to zero with varlen CDR_VARLEN_FILL.
 *   workspace at least cdr_latent_attn_bwd_workspace_bytes(p) bytes, 16-byte aligned, contents
 *             irrelevant, not to be used by another call until this one's kernels have finished
 * No output may overlap an input.  No atomics: repeated calls give the same bits.
 */
size_t cdr_latent_attn_bwd_workspace_bytes(const cdr_latent_attn_problem* p);

cdr_status cdr_latent_attn_bwd(const cdr_latent_attn_problem* p, const void* q, const void* k_nope, const void* k_rope,
                               const void* v, const int32_t* cu_seqlens, const int32_t* cu_seqlens_k, const void* o,
                               const float* lse, const void* d_o, void* dq, void* dk_nope, void* dk_rope, void* dv,
                               void* workspace, size_t workspace_bytes, void* stream);

/* Human-readable name of a status code (static storage). */
const char* cdr_status_str(cdr_status s);

/* CDR_VERSION of the built library. */
int32_t cdr_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CHUNK_DR_H */
