/*
 * gdn_cp.h -- C ABI of the context-parallel Gated DeltaNet forward for one
 * NVIDIA GB300 (sm_103a).
 *
 * What it computes (sources are two public web pages):
 *   [FLA-CP] flash-linear-attention, fla/ops/cp/context.py: get_cp_cu_seqlens
 *            and build_cp_context (the per-shard cu_seqlens plan).
 *   [HP-CP]  hyper-parallel, linear_attention_context_parallel.py: the causal
 *            conv1d + SiLU with the previous shard's halo
 *            (_causal_conv1d_with_cp_halo), the chunked gated delta rule in
 *            WY/UT form (_prepare_gdn_chunks_for_summary,
 *            _run_prepared_gdn_chunks), the shard state summary
 *            (_compute_gdn_state_summary_from_prepared) and its prefix merge
 *            (_merge_gdn_prefix_state_summaries_torch).
 *
 * The gated delta rule, per sequence and value head, with S a [dk, dv] fp32
 * state:   S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T
 *          o_t = S_t^T (scale q_t)
 * A long sequence may be cut into P contiguous "virtual shards" of one
 * device's memory; each shard's state map S_out = M S_in + N is combined by
 * a prefix scan so that the sharded result equals the unsharded one.
 *
 * Conventions shared by every entry point
 *   - Pointers marked "device" must be CUDA device (or managed) memory; the
 *     caller allocates and owns every buffer.  Scratch memory is the
 *     workspace argument of the entry points that have one (required but in
 *     gdn_chunk_fwd); none allocates.
 *   - All work is enqueued on `stream` (a cudaStream_t passed as void*; NULL
 *     = the legacy default stream) of the current device, which has to be the
 *     one that the buffers are on.  No entry point synchronises the host.
 *   - Tokens are packed, batch 1: a token-major [T, ...] layout with
 *     sequence boundaries in cu_seqlens (int32, device, [num_seqs + 1],
 *     cu_seqlens[0] = 0, non-decreasing, cu_seqlens[num_seqs] = T).
 *     Empty sequences are allowed.
 *   - Head layout: Hk query/key heads, Hv value heads, Hv % Hk == 0; value
 *     head h reads query/key head h / (Hv / Hk) (repeat_interleave on the
 *     head dimension, [HP-CP] the P2P wrapper's forward).
 *   - Supported: dk, dv in {32, 64, 128}; conv kernel size 1..4; chunk 64.
 *     (The entry points from the selective scan layer on state their own.)
 *   - dtype GDN_BF16: q/k/v/x/beta/o/conv weights in bf16, arithmetic and
 *     the state in fp32.  GDN_F32: everything fp32.  g is always fp32.
 *   - Errors detectable on the host return a non-OK status before anything
 *     is enqueued; gdn_last_error() then describes the first failing check.
 *     Errors that depend on device data (a malformed cu_seqlens) are written
 *     to a device status word (see gdn_cp_plan) and never trap.
 */
#ifndef GDN_CP_H
#define GDN_CP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1,       /* null pointer, negative size, misaligned buffer */
    GDN_ERR_UNSUPPORTED_SHAPE = 2, /* dk/dv/conv_k/channels outside the supported set */
    GDN_ERR_DTYPE = 3,             /* unknown gdn_dtype */
    GDN_ERR_NOT_DIVISIBLE = 4,     /* T % n_shards != 0 ([HP-CP] _slice_local_cp) */
    GDN_ERR_SHARD_TOO_SHORT = 5,   /* T / n_shards < conv_k - 1 ([HP-CP] conv halo check) */
    GDN_ERR_BAD_CU_SEQLENS = 6,    /* device status only: cu_seqlens malformed */
    GDN_ERR_TIMEOUT = 7,           /* device status only: a bounded wait expired */
    GDN_ERR_CUDA = 8,              /* a CUDA launch failed; see gdn_last_error() */
    GDN_ERR_WORKSPACE = 9          /* workspace missing or smaller than required */
} gdn_status;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype;

/* flags for gdn_chunk_fwd / gdn_chunk_summary / gdn_shard_fwd */
enum {
    /* replace q and k by x * rsqrt(sum(x^2) + 1e-6) per head before use
       ([HP-CP] _l2norm_torch, use_qk_l2norm_in_kernel) */
    GDN_QK_L2NORM = 1u
};

/* Human-readable name of a status code (static string). */
const char *gdn_status_string(gdn_status s);

/* Thread-local description of the last non-OK status returned on this
   thread ("" if none). */
const char *gdn_last_error(void);

/* Number of bounded device-side waits (on the tensor core) that expired on
   the current device since load or the last reset; such a wait makes its
   kernel stop early and leave its outputs incomplete.  Synchronises the
   device (a copy from device memory).  reset != 0 zeroes the counter. */
gdn_status gdn_device_timeouts(int32_t *count, int reset);

/* Testing hook (no counterpart on the source pages): settings of the
   split-item hand-over of the tensor-core chunk kernel, used by the launches
   that follow on any thread.  wait_ns bounds the wait of a second half for
   its first half's final state (default 1e9 ns); publish == 0 makes first
   halves skip publishing it, so that every second half's wait expires:
   the kernel then stops early, counts a timeout (gdn_device_timeouts) and
   writes GDN_ERR_TIMEOUT to the launch's status word (the plan's word for
   gdn_shard_fwd, word 2 of the gdn_chunk_fwd workspace).  Restore with
   gdn_debug_set_handover(1000000000, 1).  Not for production use. */
gdn_status gdn_debug_set_handover(int64_t wait_ns, int publish);

/* Testing hook (no counterpart on the source pages): enable = 0 turns off the
   splitting of work-queue items into two parts handed over through a final
   state (single-segment launches: long items in halves; shard passes: short
   tail parts), so that a test can compare split and unsplit runs, which give
   bit-identical results.  enable = 1 (the default) restores it.  Applies to
   launches made after the call from any thread.  Not for production use. */
gdn_status gdn_debug_set_split(int32_t enable);

/* Profiling hook (no counterpart on the source pages): while n > 0, every
   gdn_shard_fwd call on this host thread records events[i] (cudaEvent_t
   handles, created by the caller) on its stream: [0] at entry, [1] after the
   plan and the conv, [2] after chunk pass 1, [3] after the merge, [4] after
   pass 2, [5] at exit (as far as n reaches).  n = 0 turns it off. */
gdn_status gdn_debug_set_phase_events(void *const *events, int32_t n);

/* ------------------------------------------------------------------------
 * Shard plan  ([FLA-CP] get_cp_cu_seqlens, steps 1-5)
 *
 * For each shard r < n_shards (part = T / n_shards, rs = r * part,
 * re = rs + part, cu = cu_seqlens):
 *   s = #{i : cu[i+1] <= rs}            start_seq_idx (searchsorted right)
 *   e = #{i < num_seqs : cu[i] < re}    end_seq_idx   (searchsorted left)
 *   local_cu = dedupe(clamp(cu[s..e], rs, re) - rs)   (unique_consecutive)
 *   pre_num_conv_tokens = max(0, rs - cu[s])
 *   pre_num_ranks  = r - cu[s] / part;        is_first_rank = (pre == 0)
 *   post_num_ranks = (cu[e] - 1) / part - r;  is_last_rank  = (post == 0)
 *
 * `plan` is a device int32 buffer of gdn_cp_plan_words(num_seqs, n_shards)
 * words, laid out as:
 *   plan[0]                                  status word (0 = OK, else a
 *                                            gdn_status: BAD_CU_SEQLENS when
 *                                            cu[0] != 0, cu decreases, or
 *                                            cu[num_seqs] % n_shards != 0)
 *   plan[GDN_PLAN_REC(r) + GDN_PLAN_*]       the fields below for shard r
 *   plan[GDN_PLAN_CU(num_seqs, n_shards, r) + i], 0 <= i <= local_num_seqs
 *                                            local cu_seqlens of shard r
 *   plan[GDN_PLAN_SEQ(num_seqs, n_shards, r) + j], 0 <= j < local_num_seqs
 *                                            global index of the sequence that
 *                                            local segment j belongs to (the one
 *                                            holding the segment's first token;
 *                                            empty sequences, which the dedupe
 *                                            of step 4 removes, own no segment)
 * Needs 1 <= n_shards <= 65536 and num_seqs >= 1.  The whole plan is
 * computed on the device: no device-to-host copy of cu_seqlens.
 * ---------------------------------------------------------------------- */
enum {
    GDN_PLAN_LOCAL_NUM_SEQS = 0,
    GDN_PLAN_START_SEQ_IDX = 1,
    GDN_PLAN_END_SEQ_IDX = 2,
    GDN_PLAN_PRE_NUM_RANKS = 3,
    GDN_PLAN_POST_NUM_RANKS = 4,
    GDN_PLAN_IS_FIRST_RANK = 5,
    GDN_PLAN_IS_LAST_RANK = 6,
    GDN_PLAN_PRE_NUM_CONV_TOKENS = 7,
    GDN_PLAN_SEG_OFFSET = 8, /* sum of local_num_seqs over shards < r */
    GDN_PLAN_NFIELDS = 9
};
#define GDN_PLAN_REC(r) (1 + (int64_t)(r) * GDN_PLAN_NFIELDS)
#define GDN_PLAN_CU(num_seqs, n_shards, r) \
    (1 + (int64_t)(n_shards) * GDN_PLAN_NFIELDS + (int64_t)(r) * ((num_seqs) + 1))
#define GDN_PLAN_SEQ(num_seqs, n_shards, r) \
    (GDN_PLAN_CU(num_seqs, n_shards, n_shards) + (int64_t)(r) * ((num_seqs) + 1))

int64_t gdn_cp_plan_words(int32_t num_seqs, int32_t n_shards);

gdn_status gdn_cp_plan(const int32_t *cu_seqlens, int32_t num_seqs, int32_t n_shards,
                       int32_t *plan, void *stream);

/* ------------------------------------------------------------------------
 * Causal depthwise conv1d + SiLU with a halo
 * ([HP-CP] _causal_conv1d_with_cp_halo; zero history before each sequence
 * start, as the varlen plan's pre_num_conv_tokens implies)
 *
 *   y[t, c] = silu(bias[c] + sum_{j < conv_k} w[c, j] * x'[t - conv_k + 1 + j, c])
 *
 * x' is x within the token's own sequence and 0 before its start, except
 * that the FIRST sequence continues from `halo`: halo is [conv_k - 1,
 * channels] (row stride `channels`), its last row being the token just
 * before x[0]; only its last `halo_len` rows are history (0 <= halo_len <=
 * conv_k - 1; halo may be NULL when halo_len == 0).
 *   x     device [T, channels] dtype, row stride ldx (elements)
 *   w     device [channels, conv_k] dtype;  bias device [channels] or NULL
 *   y     device [T, channels] dtype, row stride ldy; must not overlap x
 * Needs channels % 8 == 0, ldx and ldy multiples of 8, and 16-byte aligned
 * x, y and halo.  Accumulates in fp32; bf16 output rounds to nearest even
 * (its SiLU uses a hardware tanh, error about 5e-4, below bf16 rounding;
 * fp32 output uses a / (1 + e^-a)).
 * ---------------------------------------------------------------------- */
gdn_status gdn_conv_silu(const void *x, int64_t ldx, gdn_dtype dtype, int32_t T,
                         int32_t channels, const void *w, const void *bias, int32_t conv_k,
                         const int32_t *cu_seqlens, int32_t num_seqs, const void *halo,
                         int32_t halo_len, void *y, int64_t ldy, void *stream);

/* ------------------------------------------------------------------------
 * Chunked (C = 64) gated delta rule forward, WY/UT form
 * ([HP-CP] _prepare_gdn_chunks_for_summary + _run_prepared_gdn_chunks)
 *
 *   q, k  device [T, Hk, dk] dtype at q + t*ldq + h*dk + i (same for k)
 *   v     device [T, Hv, dv] dtype at v + t*ldv + h*dv + j
 *   g     device [T, Hv] fp32 log-gates (per-token decay exp(g))
 *   beta  device [T, Hv] dtype
 *   h0    device [num_seqs, Hv, dk, dv] fp32 initial states, or NULL (= 0)
 *   o     device [T, Hv, dv] dtype (dense)
 *   h_final device [num_seqs, Hv, dk, dv] fp32 state after each sequence's
 *         last token (h0 or 0 for an empty sequence), or NULL
 *   scale multiplies q (1/sqrt(dk) in the pages)
 *   workspace, workspace_bytes  optional device scratch of at least
 *         gdn_chunk_fwd_workspace_size(...) bytes, 16-byte aligned (the work
 *         queue described there), or NULL, 0
 * Chunks restart at every sequence start; a sequence's last chunk is padded
 * with beta = 0, g = 0 rows that are never stored.  Row strides must be
 * multiples of 8 elements and q/k/v 16-byte aligned.  o may not alias the
 * inputs.
 * ---------------------------------------------------------------------- */
gdn_status gdn_chunk_fwd(const void *q, const void *k, const void *v, int64_t ldq,
                         int64_t ldk, int64_t ldv, gdn_dtype dtype, const float *g,
                         const void *beta, const float *h0, const int32_t *cu_seqlens,
                         int32_t num_seqs, int32_t T, int32_t Hk, int32_t Hv, int32_t dk,
                         int32_t dv, float scale, uint32_t flags, void *o, float *h_final,
                         void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of the optional gdn_chunk_fwd workspace (device, 16-byte aligned,
 * contents on entry irrelevant; the call rewrites it on its stream).  With a
 * workspace, the bf16 d=128 kernel takes its (sequence, head) jobs from a
 * work queue sorted longest-first, one persistent block per SM; with h_final
 * as well it may split a long sequence's token range into two halves run one
 * after the other (the second starts from the first's final state, handed
 * over through h_final), so that the work packs more evenly onto the SMs.
 * Results are bit-identical with and without a workspace.  Without one every
 * block runs one job, longest first.  A workspace smaller than this size is
 * an error (GDN_ERR_WORKSPACE). */
size_t gdn_chunk_fwd_workspace_size(int32_t num_seqs, int32_t Hv, int32_t dk, int32_t dv,
                                    gdn_dtype dtype);

/* ------------------------------------------------------------------------
 * Head-major layout ([HP-CP] LinearAttentionUlyssesCPWrapper: after its
 * seq-to-heads all-to-all every rank holds whole sequences of a subset of the
 * heads; on one device that exchange is a re-layout of whole d-element rows)
 *   gdn_to_head_major   x device [T, H, d] dtype with token stride ldx
 *                       (elements, ldx >= H*d, 16-byte rows) -> y device
 *                       [H, T, d] dense
 *   gdn_to_token_major  the inverse: y [H, T, d] -> x [T, H, d] (stride ldx)
 *   gdn_chunk_fwd_heads gdn_chunk_fwd on dense head-major q, k [Hk, T, dk],
 *                       v [Hv, T, dv] -> o [Hv, T, dv]; g, beta [T, Hv], h0,
 *                       h_final, cu_seqlens, scale, flags and the optional
 *                       workspace as in gdn_chunk_fwd (same size); q, k, v, o
 *                       16-byte aligned.  Same arithmetic as the token-major
 *                       call, so the results are bit-identical.
 * ---------------------------------------------------------------------- */
gdn_status gdn_to_head_major(const void *x, int64_t ldx, gdn_dtype dtype, int32_t T, int32_t H,
                             int32_t d, void *y, void *stream);
gdn_status gdn_to_token_major(const void *y, gdn_dtype dtype, int32_t T, int32_t H, int32_t d,
                              void *x, int64_t ldx, void *stream);
gdn_status gdn_chunk_fwd_heads(const void *q, const void *k, const void *v, gdn_dtype dtype,
                               const float *g, const void *beta, const float *h0,
                               const int32_t *cu_seqlens, int32_t num_seqs, int32_t T, int32_t Hk,
                               int32_t Hv, int32_t dk, int32_t dv, float scale, uint32_t flags,
                               void *o, float *h_final, void *workspace, size_t workspace_bytes,
                               void *stream);

/* ------------------------------------------------------------------------
 * State summary of each sequence ([HP-CP]
 * _compute_gdn_state_summary_from_prepared): the affine map of the state
 * across the sequence,  S_end = M S_start + N, with
 *   M = prod_t exp(g_t) (I - beta_t k_t k_t^T)   device [num_seqs, Hv, dk, dk] fp32
 *   N = the state reached from S_start = 0       device [num_seqs, Hv, dk, dv] fp32
 * computed chunk by chunk on the augmented state [N | M] from [0 | I].
 * Inputs as in gdn_chunk_fwd (q is not needed).
 * ---------------------------------------------------------------------- */
gdn_status gdn_chunk_summary(const void *k, const void *v, int64_t ldk, int64_t ldv,
                             gdn_dtype dtype, const float *g, const void *beta,
                             const int32_t *cu_seqlens, int32_t num_seqs, int32_t T, int32_t Hk,
                             int32_t Hv, int32_t dk, int32_t dv, uint32_t flags, float *M,
                             float *N, void *stream);

/* ------------------------------------------------------------------------
 * Prefix merge of shard summaries ([HP-CP]
 * _merge_gdn_prefix_state_summaries_torch), for every value head h:
 *   S_in[0] = S0 (or 0);   S_in[r] = M[r-1] S_in[r-1] + N[r-1],  r = 1..P-1
 *   M device [P, Hv, dk, dk] (16-byte aligned), N device [P, Hv, dk, dv],
 *   S0 device [Hv, dk, dv] or NULL, S_in device [P, Hv, dk, dv]; all fp32.
 *   M[P-1], N[P-1] unused.
 * Sequential over r in fp32, parallel over heads and 32-column tiles of the
 * state; each M is staged in shared memory while the previous one is applied.
 * ---------------------------------------------------------------------- */
gdn_status gdn_state_combine(const float *M, const float *N, const float *S0, int32_t P,
                             int32_t Hv, int32_t dk, int32_t dv, float *S_in, void *stream);

/* ------------------------------------------------------------------------
 * The whole path on P virtual shards of one device:
 *   plan -> conv + SiLU (halo = previous shard's rows) -> q/k/v views of the
 *   conv output -> chunked gated delta rule per shard (pass 1; shards that
 *   continue a sequence from an earlier shard run the [N | M] summary) ->
 *   prefix merge -> pass 2 for the continuing shards.
 *   x       device [T, Cch] dtype, Cch = 2*Hk*dk + Hv*dv, fused channel order
 *           [Q (Hk*dk) | K (Hk*dk) | V (Hv*dv)] ([HP-CP] torch.split of
 *           mixed_qkv); row stride Cch
 *   conv_w  device [Cch, conv_k] dtype; conv_b device [Cch] dtype or NULL
 *   g, beta, h0, o, h_final as in gdn_chunk_fwd
 *   plan_out  device int32 [gdn_cp_plan_words(num_seqs, n_shards)] or NULL:
 *           receives a copy of the plan (incl. its status word)
 *   workspace device, >= gdn_shard_fwd_workspace_size(...) bytes, 256-byte
 *           aligned; its contents on entry do not matter.  For bf16 with
 *           dk = dv = 128 and n_shards > 1 that size includes room in which
 *           the summaries' N halves store their chunks' W rows, K~ tiles and
 *           e^{G_last} (about T * Hv * 512 bytes), so that the M halves run apart on
 *           the tensor cores (with few long shards each M chain is cut into
 *           up to 8 segments, whose fp32 products take n_shards * Hv * 64 KiB
 *           per segment more); a workspace down to
 *           gdn_shard_fwd_workspace_min_size(...) bytes is accepted as well,
 *           with the M halves run in the chunk kernel (the same results up to
 *           rounding; bit for bit where the chains are not cut; slower).  The
 *           size depends on the current device's SM count.
 * With n_shards == 1 this is the ordinary (unsharded) forward.  Checks on
 * the host: T % n_shards == 0 and T / n_shards >= conv_k - 1.  A malformed
 * cu_seqlens sets the plan status word and every later kernel returns
 * without touching o / h_final.
 * ---------------------------------------------------------------------- */
size_t gdn_shard_fwd_workspace_size(int32_t T, int32_t num_seqs, int32_t n_shards, int32_t Hk,
                                    int32_t Hv, int32_t dk, int32_t dv, gdn_dtype dtype);
/* the smallest workspace gdn_shard_fwd accepts (see its workspace argument);
 * 0 for invalid arguments */
size_t gdn_shard_fwd_workspace_min_size(int32_t T, int32_t num_seqs, int32_t n_shards, int32_t Hk,
                                        int32_t Hv, int32_t dk, int32_t dv, gdn_dtype dtype);

gdn_status gdn_shard_fwd(const void *x, const void *conv_w, const void *conv_b, int32_t conv_k,
                         const float *g, const void *beta, const float *h0,
                         const int32_t *cu_seqlens, int32_t num_seqs, int32_t T, int32_t Hk,
                         int32_t Hv, int32_t dk, int32_t dv, float scale, uint32_t flags,
                         int32_t n_shards, gdn_dtype dtype, void *workspace,
                         size_t workspace_bytes, void *o, float *h_final, int32_t *plan_out,
                         void *stream);

/* ------------------------------------------------------------------------
 * The layer between its projections ([HP-CP] LinearAttentionP2PCPWrapper /
 * LinearAttentionAllGatherCPWrapper forward, from the projection outputs to
 * the input of the output projection):
 *   beta = sigmoid(b),  g = -exp(A_log) * softplus(a + dt_bias)   (per v-head)
 *   o    = the path of gdn_shard_fwd on n_shards virtual shards
 *   y    = norm_w * o / sqrt(mean(o^2) + norm_eps) * silu(z)   per (token,
 *          v-head) row of dv values (the wrappers' norm(core_attn_out, z))
 *   x, conv_w, conv_b, h0, cu_seqlens, workspace, h_final, plan_out: as in
 *           gdn_shard_fwd (same workspace size)
 *   a, b    device [T, Hv] dtype (the raw gate projections)
 *   A_log, dt_bias  device [Hv] fp32
 *   z       device [T, Hv, dv] dtype with token row stride ldz (a multiple of
 *           8, >= Hv*dv), 16-byte aligned; or NULL: no norm (y = o)
 *   norm_w  device [dv] dtype, 16-byte aligned (with z)
 *   y       device [T, Hv, dv] dtype
 * The gates are computed where g and beta are read (inside the chunk
 * kernels): g in fp32 (softplus(x) = x for x > 20), beta rounded to dtype.
 * The norm is the tensor-core chunk kernel's output epilogue for bf16 with
 * dk = dv = 128 (on the bf16-rounded o); other shapes run it as one more
 * pass over y.
 * ---------------------------------------------------------------------- */
gdn_status gdn_layer_fwd(const void *x, const void *conv_w, const void *conv_b, int32_t conv_k,
                         const void *a, const void *b, const float *A_log, const float *dt_bias,
                         const void *z, int64_t ldz, const void *norm_w, float norm_eps,
                         const float *h0, const int32_t *cu_seqlens, int32_t num_seqs, int32_t T,
                         int32_t Hk, int32_t Hv, int32_t dk, int32_t dv, float scale, uint32_t flags,
                         int32_t n_shards, gdn_dtype dtype, void *workspace, size_t workspace_bytes,
                         void *y, float *h_final, int32_t *plan_out, void *stream);

/* ------------------------------------------------------------------------
 * Backward of the gated delta rule ([HP-CP] the custom autograd functions
 * _RecvInitialStateP2PFunction / _SendFinalStateP2PFunction, whose backward
 * sends the state gradient the other way; the forward is gdn_chunk_fwd's).
 * Given the loss gradients dout (w.r.t. o) and dh_final (w.r.t. the final
 * states), computes the gradients w.r.t. every input of gdn_chunk_fwd:
 *   per token, with a = e^g, P = a S_prev, u = v - P^T k, S = P + beta k u^T,
 *   o = S^T (scale q), walked backwards with the state gradient dS:
 *     dq = scale S do,  dS += scale q do^T,  dbeta = k . (dS u),
 *     du = beta dS^T k = dv,  dk = beta dS u - P du,  dP = dS - k du^T,
 *     dg = <P, dP>,  dS_prev = a dP;   dh0 = dS before the first token.
 *   q, k, v, ldq, ldk, ldv, dtype, g, beta, h0, cu_seqlens, num_seqs, T, Hk,
 *           Hv, dk, dv, scale, flags: as in gdn_chunk_fwd (the same forward)
 *   dout    device [T, Hv, dv] dtype, dense
 *   dh_final device [num_seqs, Hv, dk, dv] fp32, or NULL (zero)
 *   dq, dk_ device [T, Hk, dk] fp32 (summed over the Hv/Hk value heads that
 *           read the q/k head; gradients of the stored q, k, through the L2
 *           norm when flags has GDN_QK_L2NORM)
 *   dv_     device [T, Hv, dv] fp32;  dg, dbeta device [T, Hv] fp32
 *   dh0     device [num_seqs, Hv, dk, dv] fp32 (also when h0 is NULL)
 *   workspace device, >= gdn_chunk_bwd_workspace_size(...) bytes, 256-byte
 *           aligned, contents on entry irrelevant (8-token block-start states of every
 *           sequence and a per-(sequence, head) replay scratch)
 * dk, dv in {32, 64, 128}.  One block of 512 threads per (sequence, value
 * head); the states before each token are recomputed from block-start
 * checkpoints, so the cost grows with the longest sequence.
 * ---------------------------------------------------------------------- */
size_t gdn_chunk_bwd_workspace_size(int32_t T, int32_t num_seqs, int32_t Hk, int32_t Hv, int32_t dk,
                                    int32_t dv);
gdn_status gdn_chunk_bwd(const void *q, const void *k, const void *v, int64_t ldq, int64_t ldk,
                         int64_t ldv, gdn_dtype dtype, const float *g, const void *beta,
                         const float *h0, const void *dout, const float *dh_final,
                         const int32_t *cu_seqlens, int32_t num_seqs, int32_t T, int32_t Hk,
                         int32_t Hv, int32_t dk, int32_t dv, float scale, uint32_t flags, float *dq,
                         float *dk_, float *dv_, float *dg, float *dbeta, float *dh0,
                         void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * gdn_chunk_bwd with every sequence cut into its pieces on n_shards virtual
 * shards ([HP-CP] the backward of _RecvInitialStateP2PFunction /
 * _SendFinalStateP2PFunction: the state gradient travels from a shard to the
 * one before it).  The pieces (the shard plan's local segments) run in
 * parallel: each piece's state map S_end = M S_start + N comes from its
 * summary, the start states from a forward merge over each sequence's pieces,
 * each piece's start-state gradient from its own outputs (b) from a first
 * backward pass, the end-state gradients from the reverse merge
 * dS_end(j - 1) = M_j^T dS_end(j) + b_j (dS_end of a sequence's last piece =
 * dh_final), and the input gradients from a second backward pass.
 * Arguments and results as in gdn_chunk_bwd, plus:
 *   n_shards  1..65536, T % n_shards == 0
 *   workspace device, >= gdn_shard_bwd_workspace_size(...) bytes, 256-byte
 *             aligned, contents on entry irrelevant
 *   plan_out  device int32 [gdn_cp_plan_words(num_seqs, n_shards)] or NULL:
 *             receives the shard plan; its status word is
 *             GDN_ERR_BAD_CU_SEQLENS when cu_seqlens is malformed, in which
 *             case no gradient beyond zeroed dq / dk is written
 * Results equal gdn_chunk_bwd's up to rounding.
 * ---------------------------------------------------------------------- */
size_t gdn_shard_bwd_workspace_size(int32_t T, int32_t num_seqs, int32_t n_shards, int32_t Hk,
                                    int32_t Hv, int32_t dk, int32_t dv);
gdn_status gdn_shard_bwd(const void *q, const void *k, const void *v, int64_t ldq, int64_t ldk,
                         int64_t ldv, gdn_dtype dtype, const float *g, const void *beta,
                         const float *h0, const void *dout, const float *dh_final,
                         const int32_t *cu_seqlens, int32_t num_seqs, int32_t T, int32_t Hk,
                         int32_t Hv, int32_t dk, int32_t dv, float scale, uint32_t flags,
                         int32_t n_shards, float *dq, float *dk_, float *dv_, float *dg,
                         float *dbeta, float *dh0, void *workspace, size_t workspace_bytes,
                         int32_t *plan_out, void *stream);

/* ------------------------------------------------------------------------
 * gdn_shard_fwd without a caller workspace.  The source pages have no
 * counterpart: this entry point exists for callers that cannot allocate
 * device memory -- a plugin whose host application owns all device buffers
 * and passes it only inputs and outputs, or a latency-critical loop that may
 * not call cudaMalloc (which can synchronise the device).
 *
 * Same arguments and results as gdn_shard_fwd, minus the workspace.  The
 * scratch is one file-scope device array of GDN_NOALLOC_SCRATCH_BYTES
 * (32 MiB) that every device loading the library holds until the process
 * exits.  A problem whose gdn_shard_fwd_workspace_min_size(...) exceeds it is
 * rejected with GDN_ERR_WORKSPACE before anything is enqueued.  The entry
 * point never calls cudaMalloc/cudaFree or any allocating routine.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current) and caches it with
 *     the device's current CUDA context; a call under a new context (after
 *     cudaDeviceReset) looks it up again.  Make the first call on a device,
 *     and the first after a reset, before any stream capture.
 *   - All calls share the one array and it keeps the previous call's
 *     contents; nothing in it needs to start at zero.  Calls whose work
 *     overlaps on the GPU (other streams, other host threads) race on it:
 *     serialise them, e.g. on one stream.
 * ---------------------------------------------------------------------- */
#define GDN_NOALLOC_SCRATCH_BYTES (32u << 20)

gdn_status gdn_shard_fwd_noalloc(const void *x, const void *conv_w, const void *conv_b,
                                 int32_t conv_k, const float *g, const void *beta, const float *h0,
                                 const int32_t *cu_seqlens, int32_t num_seqs, int32_t T,
                                 int32_t Hk, int32_t Hv, int32_t dk, int32_t dv, float scale,
                                 uint32_t flags, int32_t n_shards, gdn_dtype dtype, void *o,
                                 float *h_final, int32_t *plan_out, void *stream);

/* ------------------------------------------------------------------------
 * Selective scan layer.  The entry points below have no counterpart on the
 * source pages: they are the other recurrent layer that a stack of gated
 * linear-attention layers holds, over the same packed tokens (cu_seqlens) and
 * with the same conventions, and the norms between two blocks of such a stack.
 *
 * Causal depthwise conv1d + SiLU with a state per sequence
 *
 *   y[t, c] = silu(bias[c] + sum_{j < conv_k} w[c, j] * x'[t - conv_k + 1 + j, c])
 *
 * x' is x within the token's own sequence n and state[n] before its start:
 * row conv_k - 2 of state[n] is the token just before the sequence's first.
 *   x, y      device [T, channels] dtype, row strides ldx, ldy; no overlap
 *   w         device [channels, conv_k] dtype;  bias device [channels] or NULL
 *   state     device [num_seqs, conv_k - 1, channels] dtype, or NULL (zeros)
 *   state_out device, as state, or NULL: the last conv_k - 1 rows of
 *             (state[n], x of sequence n), so that a prompt may be fed in
 *             pieces; must not overlap state
 * Needs channels % 8 == 0, conv_k 1..4, row strides multiples of 8 and
 * 16-byte aligned x, y, state and state_out.  fp32 accumulation.  The SiLU is
 * a / (1 + e^-a) for both types (gdn_conv_silu takes a hardware tanh for
 * bf16).  The sizes of the workspaces from here on do not fall with T: one
 * for the longest call serves shorter ones.  T is at most 2^31 - 1 - 2^20, and a
 * malformed cu_seqlens gives unspecified results, never an access outside the
 * arrays (both hold for every entry point below).
 *
 * gdn_ssm_conv_bwd: gradients of the above for dy and dstate_out
 *   dy         device [T, channels] dtype, row stride lddy
 *   dstate_out device [num_seqs, conv_k - 1, channels] fp32, or NULL (zero)
 *   dx         device [T, channels] dtype, row stride lddx
 *              (dy, dx, dstate_out and dstate 16-byte aligned; dx overlaps
 *              neither x nor dy)
 *   dw         device [channels, conv_k] fp32;  dbias device [channels] fp32
 *              or NULL;  dstate device [num_seqs, conv_k - 1, channels] fp32
 *              or NULL
 *   workspace  device, >= gdn_ssm_conv_bwd_workspace_size(...) bytes, 256-byte
 *              aligned, contents on entry irrelevant
 * Sums are taken in a fixed order: equal calls give equal bits.
 *
 * gdn_ssm_conv_step: one token of `batch` requests over a cache of states
 *   x, y    device [batch, channels] dtype, row strides ldx, ldy
 *   states  device [num_slots, conv_k - 1, channels] dtype
 *   src, dst device int32 [batch] or NULL (slot i for request i): request i
 *           reads slot src[i] and writes the state after its token to slot
 *           dst[i] (equal for an update in place).  src[i] < 0: a zero state
 *           (a new request).  dst[i] < 0: a padded row, for which nothing is
 *           read or written but zeros to y.  A slot number >= num_slots is
 *           taken as negative.  No slot may be the dst of two requests, nor
 *           the dst of one and the src of another.
 * ---------------------------------------------------------------------- */
gdn_status gdn_ssm_conv_fwd(const void *x, int64_t ldx, gdn_dtype dtype, int32_t T,
                            int32_t channels, const void *w, const void *bias, int32_t conv_k,
                            const int32_t *cu_seqlens, int32_t num_seqs, const void *state,
                            void *state_out, void *y, int64_t ldy, void *stream);
size_t gdn_ssm_conv_bwd_workspace_size(int32_t T, int32_t channels, int32_t conv_k);
gdn_status gdn_ssm_conv_bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                            gdn_dtype dtype, int32_t T, int32_t channels, const void *w,
                            const void *bias, int32_t conv_k, const int32_t *cu_seqlens,
                            int32_t num_seqs, const void *state, const float *dstate_out, void *dx,
                            int64_t lddx, float *dw, float *dbias, float *dstate, void *workspace,
                            size_t workspace_bytes, void *stream);
gdn_status gdn_ssm_conv_step(const void *x, int64_t ldx, gdn_dtype dtype, int32_t batch,
                             int32_t channels, const void *w, const void *bias, int32_t conv_k,
                             void *states, int32_t num_slots, const int32_t *src,
                             const int32_t *dst, void *y, int64_t ldy, void *stream);

/* ------------------------------------------------------------------------
 * Selective state space scan: per sequence and channel c (group
 * q = c / (channels / groups)), with N = d_state diagonal states in fp32,
 *
 *   delta_t = softplus(dt_t + dt_bias)         (softplus(v) = v for v > 20)
 *   h_n    <- exp(-exp(A_log[c, n]) delta_t) h_n + delta_t x_t B_t[q, n]
 *   y_t     = (sum_n C_t[q, n] h_n + D x_t) * silu(z_t)
 *
 *   x, dt   device [T, channels] dtype, row strides ldx, lddt
 *   z       as x with row stride ldz, or NULL (no gate)
 *   B, C    device [T, groups, N] dtype at B + t * ldb + q * N + n (C: ldc);
 *           any alignment and row stride
 *   A_log   device [channels, N] fp32;  D, dt_bias device [channels] fp32 or
 *           NULL (zero)
 *   h0      device [num_seqs, channels, N] fp32 or NULL (zero)
 *   y       device [T, channels] dtype, row stride ldy
 *   h_final device [num_seqs, channels, N] fp32, or NULL: the state after each
 *           sequence's last token (h0 or 0 for an empty sequence); must not
 *           overlap h0
 *   ckpt    device fp32 [gdn_ssm_scan_ckpt_floats(...)], or NULL: the states
 *           before every 8th packed token, for gdn_ssm_scan_bwd
 *   workspace device, >= gdn_ssm_scan_workspace_size(...) bytes, 256-byte
 *           aligned, contents on entry irrelevant
 * Needs channels / groups a multiple of 8, N in 1..64, row strides of x, dt,
 * z, y multiples of 8 and those arrays, h_final and ckpt 16-byte aligned (here
 * and below; A_log, D, dt_bias, h0 and dh_final: as their type).  All arithmetic in
 * fp32 whatever the dtype; y is rounded once.  The packed tokens are cut into
 * segments that run at the same time; a first pass gives each segment's own
 * end state where the next one continues its sequence.
 *
 * gdn_ssm_scan_bwd: gradients for dy (w.r.t. y) and dh_final (fp32
 * [num_seqs, channels, N] or NULL = zero), with the forward's inputs and ckpt
 *   dx, ddt, dz  device [T, channels] dtype, dense (dz NULL iff z is)
 *   dB, dC       device [T, groups, N] dtype, dense
 *   dA_log       device [channels, N] fp32;  dD, ddt_bias device [channels]
 *                fp32 or NULL;  dh0 device [num_seqs, channels, N] fp32 or NULL
 *                (dy, dx, ddt, dz 16-byte aligned)
 *   workspace    device, >= gdn_ssm_scan_bwd_workspace_size(...) bytes,
 *                256-byte aligned, contents on entry irrelevant
 * Sums are taken in a fixed order: equal calls give equal bits.
 *
 * gdn_ssm_scan_step: one token of `batch` requests over a cache of states
 *   x, dt, z, B, C, y  as above with batch rows in place of T
 *   states  device [num_slots, channels, N] fp32, 16-byte aligned
 *   src, dst           as in gdn_ssm_conv_step
 * ---------------------------------------------------------------------- */
size_t gdn_ssm_scan_ckpt_floats(int32_t T, int32_t channels, int32_t d_state);
size_t gdn_ssm_scan_workspace_size(int32_t T, int32_t channels, int32_t d_state, int32_t groups);
gdn_status gdn_ssm_scan_fwd(const void *x, int64_t ldx, const void *dt, int64_t lddt, const void *z,
                            int64_t ldz, const void *B, int64_t ldb, const void *C, int64_t ldc,
                            gdn_dtype dtype, const float *A_log, const float *D,
                            const float *dt_bias, const float *h0, const int32_t *cu_seqlens,
                            int32_t num_seqs, int32_t T, int32_t channels, int32_t d_state,
                            int32_t groups, void *y, int64_t ldy, float *h_final, float *ckpt,
                            void *workspace, size_t workspace_bytes, void *stream);
size_t gdn_ssm_scan_bwd_workspace_size(int32_t T, int32_t channels, int32_t d_state,
                                       int32_t groups);
gdn_status gdn_ssm_scan_bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                            const void *dt, int64_t lddt, const void *z, int64_t ldz, const void *B,
                            int64_t ldb, const void *C, int64_t ldc, gdn_dtype dtype,
                            const float *A_log, const float *D, const float *dt_bias,
                            const float *h0, const float *ckpt, const float *dh_final,
                            const int32_t *cu_seqlens, int32_t num_seqs, int32_t T,
                            int32_t channels, int32_t d_state, int32_t groups, void *dx, void *ddt,
                            void *dz, void *dB, void *dC, float *dA_log, float *dD, float *ddt_bias,
                            float *dh0, void *workspace, size_t workspace_bytes, void *stream);
gdn_status gdn_ssm_scan_step(const void *x, int64_t ldx, const void *dt, int64_t lddt,
                             const void *z, int64_t ldz, const void *B, int64_t ldb, const void *C,
                             int64_t ldc, gdn_dtype dtype, const float *A_log, const float *D,
                             const float *dt_bias, int32_t batch, int32_t channels,
                             int32_t d_state, int32_t groups, float *states, int32_t num_slots,
                             const int32_t *src, const int32_t *dst, void *y, int64_t ldy,
                             void *stream);

/* ------------------------------------------------------------------------
 * Block norm: what stands between two blocks of a stack, in one pass.  Per
 * token row of `width` values, rms(v) = sqrt(mean(v^2) + eps):
 *
 *   p       = w_post * o / rms(o)                   (w_post NULL: p = o)
 *   res_out = res + scale * sigmoid(gate) * p       (gate, scale NULL: 1)
 *   y       = w_pre * res_out / rms(res_out)        (res_out before rounding)
 *
 *   o       device [T, width] dtype: the block's output;  gate as o (raw), or
 *           NULL;  y as o: the next block's input
 *   res, res_out device [T, width] res_dtype (dtype or GDN_F32): the residual
 *           stream; res_out may be res
 *   w_post, w_pre device [width] dtype;  scale device [width] fp32
 * All arrays dense but for the token row strides ldo, ldgate (multiples of
 * 8); 16-byte aligned; width % 8 == 0, width <= 16384.
 *
 * gdn_block_norm_bwd: gradients for dy and dres_out (res_dtype, or NULL =
 * zero).  res_out is the stored stream; the pre norm is taken at it.
 *   d_o, dgate device [T, width] dtype (dgate NULL iff gate is)
 *   dres       device [T, width] res_dtype; may be dres_out
 *   dw_pre, dw_post, dscale device [width] fp32 (the latter two NULL iff
 *              w_post / scale is)
 *   workspace  device, >= gdn_block_norm_bwd_workspace_size(...) bytes,
 *              256-byte aligned, contents on entry irrelevant
 * Sums are taken in a fixed order: equal calls give equal bits.
 * ---------------------------------------------------------------------- */
gdn_status gdn_block_norm_fwd(const void *o, int64_t ldo, const void *gate, int64_t ldgate,
                              gdn_dtype dtype, const void *res, gdn_dtype res_dtype,
                              const void *w_post, const void *w_pre, const float *scale, float eps,
                              int32_t T, int32_t width, void *res_out, void *y, void *stream);
size_t gdn_block_norm_bwd_workspace_size(int32_t T, int32_t width);
gdn_status gdn_block_norm_bwd(const void *dy, const void *dres_out, const void *o, int64_t ldo,
                              const void *gate, int64_t ldgate, gdn_dtype dtype,
                              const void *res_out, gdn_dtype res_dtype, const void *w_post,
                              const void *w_pre, const float *scale, float eps, int32_t T,
                              int32_t width, void *d_o, void *dgate, void *dres, float *dw_pre,
                              float *dw_post, float *dscale, void *workspace,
                              size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * The gated delta rule for one token of `batch` requests over a cache of
 * states, per value head h (query/key head h / (Hv / Hk)):
 *
 *   S' = e^g S[src],  u = v - S'^T k,  S = S' + beta k u^T,
 *   o = S^T (scale q),  S[dst] = S
 *
 *   q, k    device [batch, Hk, dk] dtype, row strides ldq, ldk
 *   v       device [batch, Hv, dv] dtype, row stride ldv
 *   g       device [batch, Hv] fp32;  beta device [batch, Hv] dtype
 *   states  device [num_slots, Hv, dk, dv] fp32, 16-byte aligned
 *   src, dst  as for gdn_ssm_conv_step
 *   o       device [batch, Hv, dv] dtype
 * flags: GDN_QK_L2NORM as for gdn_chunk_fwd.  dk, dv in {32, 64, 128}; batch *
 * Hv below 2^31; every array but states at any alignment of its type.  fp32
 * arithmetic; o is rounded once.
 *
 * gdn_layer_step: the same behind the short conv of a layer, as gdn_layer_fwd
 *   x       device [batch, 2 Hk dk + Hv dv] dtype, row stride ldx: the conv's
 *           output (gdn_ssm_conv_step), channels [Q | K | V]; q and k are
 *           divided by their norms
 *   a, b    device [batch, Hv] dtype, row strides lda, ldb: g = -exp(A_log)
 *           softplus(a + dt_bias), beta = sigmoid(b), both in fp32
 *   z       device [batch, Hv, dv] dtype, row stride ldz, or NULL: then
 *           y = norm_w * o / sqrt(mean(o^2) + norm_eps) * silu(z), of the
 *           unrounded o;  norm_w device [dv] dtype
 * ---------------------------------------------------------------------- */
gdn_status gdn_chunk_step(const void *q, const void *k, const void *v, int64_t ldq, int64_t ldk,
                          int64_t ldv, gdn_dtype dtype, const float *g, const void *beta,
                          int32_t batch, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv,
                          float scale, uint32_t flags, float *states, int32_t num_slots,
                          const int32_t *src, const int32_t *dst, void *o, void *stream);
gdn_status gdn_layer_step(const void *x, int64_t ldx, const void *a, int64_t lda, const void *b,
                          int64_t ldb, gdn_dtype dtype, const float *A_log, const float *dt_bias,
                          const void *z, int64_t ldz, const void *norm_w, float norm_eps,
                          int32_t batch, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv,
                          float scale, float *states, int32_t num_slots, const int32_t *src,
                          const int32_t *dst, void *y, void *stream);

/* ------------------------------------------------------------------------
 * Embedding:  y_t = scale table[token_t]
 *
 *   tokens  device [T] int32 or int64 (index_bits 32 or 64); a token outside
 *           [0, vocab) is a padded one: a row of zeros, no gradient
 *   table   device [vocab, width] dtype, row stride ldt
 *   y       device [T, width] dtype, row stride ldy; must not overlap table
 * Any width up to 2^20 and any alignment; 16-byte accesses where the width, the
 * strides and the arrays allow them.
 *
 * gdn_embed_bwd: dtable[v] = scale * (sum of dy_t over the tokens v, in the
 * tokens' order), added in fp32 and rounded once; with accumulate != 0 it is
 * added to what dtable holds, and only the rows of tokens that occur are
 * touched.  Equal calls give equal bits.
 *   dy      device [T, width] dtype, row stride lddy
 *   dtable  device [vocab, width] dtype, row stride ldd; must not overlap dy
 *   workspace  device, >= gdn_embed_bwd_workspace_size(...) bytes, 256-byte
 *           aligned, contents on entry irrelevant
 * ---------------------------------------------------------------------- */
gdn_status gdn_embed_fwd(const void *tokens, int32_t index_bits, const void *table, int64_t ldt,
                         gdn_dtype dtype, int32_t vocab, int32_t T, int32_t width, float scale,
                         void *y, int64_t ldy, void *stream);
size_t gdn_embed_bwd_workspace_size(int32_t T, int32_t vocab, int32_t width);
gdn_status gdn_embed_bwd(const void *dy, int64_t lddy, gdn_dtype dtype, const void *tokens,
                         int32_t index_bits, int32_t vocab, int32_t T, int32_t width, float scale,
                         int32_t accumulate, void *dtable, int64_t ldd, void *workspace,
                         size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Softmax cross entropy over a vocabulary from hidden states and output
 * weights; the logits x_tv = scale h_t . w_v never exist as an array:
 *
 *   lse_t = log sum_v e^{x_tv},  loss_t = lse_t - x_{t, target_t}
 *
 *   h       device [T, width] dtype, row stride ldh
 *   w       device [vocab, width] dtype, row stride ldw
 *   targets device [T] int32 or int64 (index_bits 32 or 64).  Negative: the
 *           token is left out (loss 0, no gradient, whatever its h holds).
 *           vocab or more: loss NaN, and NaN in what its gradient reaches.
 *   loss, lse  device [T] fp32
 * Any width up to 2^20, T and vocab up to 2^28.  bf16 rows of a multiple of 8
 * elements are read in place, so that h and w then have to be 16-byte aligned
 * with row strides that are multiples of 8; other widths and fp32 are read at
 * any alignment, into a copy in the workspace.  Products of bf16 inputs are
 * exact and added in fp32: by the tensor cores, which cut, in chunks of up to 768
 * terms for logits and 16384 for gradients (there by 2^-11 of the sum at most).
 * fp32 inputs are scaled by powers of two and split into two fp16 parts, of
 * whose four products three are added in fp32: a value is off by 2^-23 of itself
 * down to 2^-16 of the largest under its scaling (its row's for h, and for w in
 * the forward; one for all of w in the backward, its token's dloss for P, there
 * down to 2^-15), below that by 2^-39 of the largest (2^-38 of dloss).  An
 * infinite element of fp32 inputs gives NaN.
 * Calls of few tokens (16 of fp32, 4 of bf16, 8 at widths that are no multiple
 * of 8; at widths up to 6400, up to 4 tokens 12800, one 51200; vocab 64 or
 * more) form products, sums and P in fp32, of infinite elements too.
 * An expired wait (gdn_device_timeouts) leaves the outputs incomplete.
 *
 * gdn_vocab_loss_bwd_from_loss: gradients of the above for dloss, from the
 * forward's loss and lse
 *   dloss   device [T] fp32
 *   dh      device [T, width] dtype, row stride lddh;  dw device [vocab,
 *           width] dtype, row stride lddw; neither overlaps an input
 * dh and dw are products with P_tv = scale dloss_t (softmax - one hot), which
 * is rounded to bf16 for bf16 inputs (what that takes from the entry at the
 * target is given back where the token is the only one with it, to dh always:
 * dh is off by its own rounding, 1.7e-3 in norm, dw by 1.7e-3 to 2.3e-3)
 * and split like them for fp32.  A token whose dloss is 0 has no gradient,
 * whatever its h holds.  The vocabulary is taken in pieces; the workspace holds
 * one piece's P (half a gigabyte at most, or 1024 columns), and dh in fp32.
 *   workspace  device, >= the _workspace_size(...) bytes of the call, 256-byte
 *           aligned, contents on entry irrelevant; sizes do not fall with T, so
 *           that the longest call's serves all
 * Equal calls give equal bits.
 *
 * gdn_vocab_loss_bwd: the same without the loss.  P at a target, softmax - 1, then
 * comes from the rounded lse, as a difference that is off by 2^-24 of lse: fine for
 * tokens whose softmax is away from 1, but where 1 - softmax is 1e-5 the
 * gradients are off by 3e-2 of themselves beside an lse of 15 and by all of
 * themselves beside one of 300 (with the loss by 9e-6 and 3e-4, of fp32).
 * ---------------------------------------------------------------------- */
size_t gdn_vocab_loss_fwd_workspace_size(int32_t T, int32_t vocab, int32_t width, gdn_dtype dtype);
gdn_status gdn_vocab_loss_fwd(const void *h, int64_t ldh, const void *w, int64_t ldw,
                              gdn_dtype dtype, const void *targets, int32_t index_bits, int32_t T,
                              int32_t vocab, int32_t width, float scale, float *loss, float *lse,
                              void *workspace, size_t workspace_bytes, void *stream);
size_t gdn_vocab_loss_bwd_workspace_size(int32_t T, int32_t vocab, int32_t width, gdn_dtype dtype);
gdn_status gdn_vocab_loss_bwd(const float *dloss, const void *h, int64_t ldh, const void *w,
                              int64_t ldw, gdn_dtype dtype, const void *targets,
                              int32_t index_bits, const float *lse, int32_t T, int32_t vocab,
                              int32_t width, float scale, void *dh, int64_t lddh, void *dw,
                              int64_t lddw, void *workspace, size_t workspace_bytes,
                              void *stream);
gdn_status gdn_vocab_loss_bwd_from_loss(const float *dloss, const void *h, int64_t ldh,
                                        const void *w, int64_t ldw, gdn_dtype dtype,
                                        const void *targets, int32_t index_bits,
                                        const float *loss, const float *lse, int32_t T,
                                        int32_t vocab, int32_t width, float scale, void *dh,
                                        int64_t lddh, void *dw, int64_t lddw, void *workspace,
                                        size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_CP_H */
