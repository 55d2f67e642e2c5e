/*
 * sinkattn.h — C ABI of the GB300 (sm_103a) sink-aware attention library.
 *
 * The operation is exact softmax attention under the mask of the SinkFlex-RL
 * paper ("Efficient Reinforcement Learning for Long-Horizon Tool-Use Agentic
 * Tasks", summary page, paragraph on the sink-aware FlexAttention path):
 *
 *     M[q, k] = [k <= q]  and  ( [q - k <= w]  or  [k < p] )
 *
 * with w the local window (inclusive; w + 1 keys including the query) and p
 * the number of always-visible prefix positions, the same mask for every
 * sequence and head.  Scores are s_qk = scale * <Q_q, K_k>.  The attention
 * call returns the output together with the natural-log log-sum-exp
 * l_q = log sum_{k visible} exp(s_qk) (sink excluded), and the output is
 * scaled by alpha_q = sigmoid(l_q - sink[h]), which is the same as appending
 * one more softmax column with logit sink[h] and a zero value vector
 * (section 5, "zero-value sink equivalence").  The backward returns dQ, dK,
 * dV and the per-head sink gradient dL/dS_h ("GPT-OSS agentic RL training"
 * page, FlashAttention v3 implementation), recomputing probabilities from l
 * so that no S x S matrix is ever stored.
 *
 * Layouts (all contiguous, row-major, head_dim innermost):
 *   q, o, dout, dq : bf16 [T, Hq, D]
 *   k, v, dk, dv   : bf16 [T, Hkv, D]
 *   lse            : fp32 [Hq, T]
 *   sink, dsink    : fp32 [Hq]
 * T is the number of tokens of all packed sequences.  Query head h reads
 * key/value head h / (Hq / Hkv) (contiguous GQA groups).  Positions inside
 * the mask are positions inside each packed sequence.
 *
 * Ownership: the caller allocates every buffer, including the workspace,
 * and keeps it alive until the stream has run the work.  The library
 * allocates no device memory and keeps no per-call state.  All device
 * pointers must be 16-byte aligned.  Every call is asynchronous on `stream`
 * (a cudaStream_t passed as void*; NULL = legacy default stream).
 * Outputs are overwritten, never accumulated (dsink included).  No output
 * may alias an input or another output.
 *
 * Errors: argument checks run on the host before anything is launched; a
 * failing check returns its status and launches nothing.  A failed launch
 * returns SINKATTN_ERR_CUDA.  Nothing aborts, exits or traps on the device.
 *
 * First call on a device: the calls whose kernels wait (fwd, bwd, decode,
 * kv4 decode, GRPO, the wait self-test) look up the device address of the library's
 * status word once per device, with that device current, through
 * cudaGetSymbolAddress (thread-safe).  Make the first such call on each
 * device outside any stream capture; later calls only launch kernels.
 */
#ifndef SINKATTN_H
#define SINKATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SINKATTN_OK = 0,
  SINKATTN_ERR_INVALID_ARG = 1,  /* null pointer, bad size, bad mask parameter, bad cu_seqlens */
  SINKATTN_ERR_UNSUPPORTED = 2,  /* head_dim other than 64, or sizes beyond the int32 index range */
  SINKATTN_ERR_ALIGNMENT = 3,    /* a device pointer that is not 16-byte aligned */
  SINKATTN_ERR_WORKSPACE = 4,    /* workspace smaller than the matching *_workspace_size() */
  SINKATTN_ERR_CUDA = 5,         /* a CUDA runtime call or launch failed */
  SINKATTN_ERR_TIMEOUT = 6       /* a kernel gave up a bounded wait (see sinkattn_get_device_status) */
} sinkattn_status;

/* One attention problem.  Uniform batch: cu_seqlens == NULL, num_seqs = B,
 * seqlen = S, total_tokens = B * S.  Packed variable-length sequences:
 * cu_seqlens (device) and cu_seqlens_host (host) hold the same num_seqs + 1
 * offsets, cu[0] = 0, nondecreasing, cu[num_seqs] = total_tokens, and
 * seqlen is the largest cu[i+1] - cu[i]. */
typedef struct {
  int32_t num_seqs;
  int32_t seqlen;
  const int32_t* cu_seqlens;       /* device, [num_seqs + 1], or NULL */
  const int32_t* cu_seqlens_host;  /* host copy of cu_seqlens (NULL iff cu_seqlens is NULL) */
  int32_t total_tokens;
  int32_t num_heads_q;             /* Hq, a multiple of num_heads_kv */
  int32_t num_heads_kv;            /* Hkv >= 1 */
  int32_t head_dim;                /* must be 64 */
  int64_t window;                  /* w >= 0 (inclusive), or -1 for unbounded */
  int64_t prefix;                  /* p >= 0 */
  int32_t causal;                  /* 1: keep [k <= q]; 0: drop that term */
  float scale;                     /* softmax scale, finite and > 0 (1/sqrt(64) usually) */
} sinkattn_problem;

/* Bytes of device workspace that sinkattn_fwd / sinkattn_bwd need for
 * `prob` (0 when the problem is invalid). */
size_t sinkattn_fwd_workspace_size(const sinkattn_problem* prob);
size_t sinkattn_bwd_workspace_size(const sinkattn_problem* prob);

/* Number of kernel launches sinkattn_fwd (which = 1) or sinkattn_bwd /
 * sinkattn_bwd_noalloc (which = 2) make for this problem, from host
 * arithmetic alone (the same work lists the calls build); -1 for an invalid
 * problem or `which`.  Lets a caller count the library's launches without a
 * profiler.  The calls make no other stream operation, except the backward
 * of a problem without tokens, which sets dsink to zero with one memset. */
int32_t sinkattn_kernel_launches(const sinkattn_problem* prob, int32_t which);

/* Forward.  Reads q, k, v (bf16) and sink (fp32 [Hq]); writes
 * o = alpha * softmax_M(s) V (bf16 [T, Hq, 64]) and lse = l (fp32 [Hq, T]).
 * Rows of a sequence are never mixed with rows of another sequence. */
sinkattn_status sinkattn_fwd(const sinkattn_problem* prob,
                             const void* q, const void* k, const void* v, const float* sink,
                             void* o, float* lse,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Backward.  Reads the forward's inputs, its outputs o and lse, and dout;
 * writes dq, dk, dv (bf16) and dsink (fp32 [Hq]), where
 * dsink[h] = -sum over all rows of (1 - alpha_q) * <dout_q, o_q>.
 * The workspace holds an fp32 dQ accumulator [T, Hq, 64], one 16-byte row
 * per (head, token) with the per-row terms -D and -l'/scale, where
 * l' = l + softplus(sink - l), as three bf16 summands each ([Hq, T]),
 * partial sums of dsink per 8-token group and head, and, when key tiles are split over
 * several work items, per-chunk dK/dV partial sums.
 * Its contents on entry do not matter (the call clears what it accumulates
 * into).  dK, dV and dsink are bitwise reproducible run to run; dQ is summed
 * in arrival order and reproducible to fp32 rounding. */
sinkattn_status sinkattn_bwd(const sinkattn_problem* prob,
                             const void* q, const void* k, const void* v, const void* o,
                             const float* lse, const void* dout, const float* sink,
                             void* dq, void* dk, void* dv, float* dsink,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Backward without a caller-provided workspace, for callers that cannot
 * allocate device memory (a host program with no device allocator of its
 * own, a runtime whose memory pool is fixed at start-up, a hot loop where an
 * allocation is not acceptable).  The paper has no counterpart: this is a
 * deployment variant of sinkattn_bwd, same arguments minus the workspace,
 * same results.  It uses a 32 MiB workspace compiled into the library as a
 * device array (held by every GPU that loads the library until the process
 * ends) and allocates nothing.  Problems whose sinkattn_bwd_workspace_size()
 * exceeds 32 MiB return SINKATTN_ERR_WORKSPACE and launch nothing.  The
 * first call on each device looks up the array's device address while that
 * device is current; make it before any stream capture.  All calls share
 * the array: calls whose kernels overlap on the GPU race and must be
 * serialised by the caller.  Nothing in the array needs clearing between
 * calls (the kernels clear what they accumulate into). */
sinkattn_status sinkattn_bwd_noalloc(const sinkattn_problem* prob,
                                     const void* q, const void* k, const void* v, const void* o,
                                     const float* lse, const void* dout, const float* sink,
                                     void* dq, void* dk, void* dv, float* dsink, void* stream);

/* Decode forward: the rollout side of the same attention (SinkFlex-RL,
 * rollout worker: the policy samples turn by turn; GPT-OSS agentic RL page:
 * the sink-aware forward of an inference FlashAttention fork).  `kv`
 * describes the cached sequences exactly as `prob` does for sinkattn_fwd:
 * k, v bf16 [kv->total_tokens, Hkv, 64] hold every position of each
 * sequence.  q bf16 [num_seqs * q_per_seq, Hq, 64] holds, for sequence b,
 * the queries of its last q_per_seq positions L_b - q_per_seq ... L_b - 1
 * in that order (rows b * q_per_seq ...).  Writes o bf16 [num_seqs *
 * q_per_seq, Hq, 64] and lse fp32 [Hq, num_seqs * q_per_seq], each row equal
 * to the same row of sinkattn_fwd over the whole sequence (same mask, sink
 * and lse).  Limits: 1 <= q_per_seq <= every sequence length,
 * (Hq / Hkv) * q_per_seq <= 128 and num_seqs <= 4096, else
 * SINKATTN_ERR_INVALID_ARG / SINKATTN_ERR_UNSUPPORTED.  The workspace
 * (sinkattn_decode_workspace_size bytes, 16-byte aligned) holds the partial
 * results of the key chunks and one counter per (sequence, kv head); its
 * size depends on the device's SM count.  Its first 4 * num_seqs * Hkv bytes
 * (the counters) must be zero before the first call; every completed call
 * leaves them zero, so a workspace zero-filled once can be reused by later
 * calls (not by calls that overlap on the GPU).  After SINKATTN_ERR_TIMEOUT,
 * zero the workspace again. */
size_t sinkattn_decode_workspace_size(const sinkattn_problem* kv, int32_t q_per_seq);
sinkattn_status sinkattn_decode_fwd(const sinkattn_problem* kv, int32_t q_per_seq,
                                    const void* q, const void* k, const void* v, const float* sink,
                                    void* o, float* lse,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* GRPO token loss and its gradient (SinkFlex-RL, zh page, "Policy update",
 * equations (3)-(7)), the memory-bound step of the same training loop.
 * Rollouts are consecutive groups of group_size (the G rollouts of one
 * prompt); rollout i owns tokens [cu_tokens[i], cu_tokens[i + 1]) of the
 * fp32 arrays logp (current policy), logp_old (sampling policy) and
 * logp_ref (reference policy; may be NULL when kl_beta == 0); mask (uint8,
 * nonzero = optimised token); rewards fp32 [num_rollouts].
 *   A_i = (R_i - mean_group) / (population std of the group + adv_eps)
 *   rho = exp(logp - logp_old),  J = min(rho A_i, clip(rho, 1 -+ clip_eps) A_i)
 *   loss = -(1/N) sum J + kl_beta (1/N) sum (e^r - r - 1),  r = logp_ref - logp
 * with both sums over optimised tokens and N their count.  Writes stats fp32
 * [4] = {loss, -(1/N) sum J, (1/N) sum (e^r - r - 1), fraction of optimised
 * tokens whose gradient the clip removes}, dlogp fp32 [total_tokens] =
 * dloss/dlogp (0 on tokens that are not optimised) and, if non-NULL,
 * advantages fp32 [num_rollouts].  With N = 0 everything is 0.  logp,
 * logp_old, logp_ref, mask and dlogp must be 16-byte aligned.  Workspace:
 * sinkattn_grpo_workspace_size bytes, 16-byte aligned, zero-filled before
 * its first use; every completed call leaves it reusable (its barrier words
 * zero again).  The kernel is one cooperative launch whose CTAs meet at a
 * grid-wide barrier with a bounded wait: if that wait runs out of time the
 * outputs are not written, sinkattn_get_device_status reports TIMEOUT and
 * the workspace must be zero-filled again.
 * Checks: group_size >= 1 dividing num_rollouts, clip_eps > 0, adv_eps >= 0,
 * kl_beta >= 0 (all finite), offsets as for sinkattn_problem. */
typedef struct {
  int32_t num_rollouts;
  int32_t group_size;
  const int32_t* cu_tokens;       /* device [num_rollouts + 1] */
  const int32_t* cu_tokens_host;  /* host copy */
  int32_t total_tokens;
  float clip_eps;
  float adv_eps;
  float kl_beta;
} sinkattn_grpo_problem;
size_t sinkattn_grpo_workspace_size(const sinkattn_grpo_problem* g);
sinkattn_status sinkattn_grpo_loss(const sinkattn_grpo_problem* g, const float* logp, const float* logp_old,
                                   const float* logp_ref, const uint8_t* mask, const float* rewards,
                                   float* stats, float* dlogp, float* advantages,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- rollout
 * The 4-bit paged key/value cache and what a rollout does with it.  One
 * prompt's pages are shared by the rollouts of its GRPO group; every new
 * token attends to the cache and is sampled with the log-probability that
 * sinkattn_grpo_loss takes as logp_old.  A cache is one layer's: a model keeps
 * one per layer, each with its own tables and counts, and reserves, forks,
 * frees and compacts each of them.
 *
 * All state is on the device and every call is asynchronous, so a step can be
 * captured into a CUDA graph and replayed while the sequences grow (make the
 * first call of each kind on a device outside any capture: it asks once for
 * the kernel's shared memory).
 *
 * Format.  pages is [num_pages][num_heads_kv][page_size / 16] blocks of 16
 * tokens, 1152 bytes each.  With g = 0..7, t = 0..3, lane = 4 g + t:
 *   [0, 512)      keys' codes: per lane 8 bytes of token g, then 8 of token
 *                 g + 8, dims 16 t .. 16 t + 15
 *   [512, 1024)   values' codes: per lane 4 bytes each of tokens 2t, 2t + 1,
 *                 2t + 8, 2t + 9, dims 8 g .. 8 g + 7
 *   [1024, 1088)  keys' scales: per lane of tokens g and g + 8, those dims
 *   [1088, 1152)  values' scales: per (16 dims, t) of the four tokens
 * A byte holds two e2m1 codes, the lower dim in the low nibble (0, 0.5, 1,
 * 1.5, 2, 3, 4, 6 and a sign); a scale is e4m3 and serves 16 dims of a token.
 * A value is code * scale * (the head's fp32 factor k_scale or v_scale, which
 * lies between 2^-100 and 2^100); what is below 2^-126 counts as 0.
 *
 * Pages.  Slot s holds seqlens[s] tokens in the pages page_table[s][0 ..
 * ceil(seqlens[s] / page_size) - 1]; the other entries mean nothing.
 * refcount[p] says how many slots hold page p; 0 is free.  Calls that need
 * pages take the lowest-numbered free ones, request after request.  A new
 * cache is page_table all -1, seqlens and refcount all 0.
 *
 * Entries of `slots` outside [0, num_slots) are idle: nothing is written for
 * them, they read as an empty sequence.  A page number outside
 * [0, num_pages), or a position beyond the table, is never accessed: tokens
 * there are not written and read as NaN.  Limits: page_size 16, 32, 64, 128
 * or 256; max_pages * page_size <= 2^30; 4096 entries per call; head_dim 64.
 * All pointers of the cache are 16-byte aligned; int32 and fp32 lists
 * elsewhere 4-byte aligned.  Calls that change a cache must not overlap on the
 * GPU with other calls on it. */
typedef struct {
  void* pages;            /* uint8 [num_pages][num_heads_kv][page_size * 72] */
  int32_t* page_table;    /* [num_slots][max_pages] */
  int32_t* seqlens;       /* [num_slots] */
  int32_t* refcount;      /* [num_pages] */
  const float* k_scale;   /* [num_heads_kv] */
  const float* v_scale;   /* [num_heads_kv] */
  int32_t num_pages;
  int32_t page_size;
  int32_t num_heads_kv;
  int32_t num_slots;
  int32_t max_pages;
} sinkattn_kv4_cache;

/* reserve: slot slots[i] grows by new_tokens[i] tokens and gets the pages
 * they need; done[i] = 1.  Pages are given in the order of the requests; one
 * that does not fit, and every later one that needs a page, gets none and
 * done[i] = 0.  done[i] = 0 also for a slot out of range, a slot named
 * earlier in the call, a negative count or a length beyond the table.  The
 * last page of a slot is never shared (see fork), so a grown slot can be
 * written at once. */
sinkattn_status sinkattn_kv4_reserve(const sinkattn_kv4_cache* cache, const int32_t* slots, const int32_t* new_tokens,
                                     int32_t n, int32_t* done, void* stream);

/* fork: the empty slot dst[i] becomes a copy of src[i]: full pages are shared
 * (refcount + 1), of a page that is not full the blocks that hold tokens are
 * copied to a new page.  Several entries may name one source; all sources are
 * read as they were before the call.  done[i] = 0, and nothing changes for
 * the entry, where a slot is out of range, dst[i] is not empty or is named
 * earlier in the call, or the pages run out (then every later entry that
 * needs one gets none either).  Where the source's open page is not in the
 * pool, the copy's is -1.  A `done` that shares memory with src or dst is
 * refused (INVALID_ARG). */
sinkattn_status sinkattn_kv4_fork(const sinkattn_kv4_cache* cache, const int32_t* src, const int32_t* dst, int32_t n,
                                  int32_t* done, void* stream);

/* free: the slots give their pages back (refcount - 1) and are empty; their
 * used table entries become -1.  Naming a slot again, or an empty one, does
 * nothing. */
sinkattn_status sinkattn_kv4_free(const sinkattn_kv4_cache* cache, const int32_t* slots, int32_t n, void* stream);

/* compact: writes the live pages of `from` (refcount > 0), in the order of
 * their numbers, to pages 0 .. live - 1 of `to`, with refcount, page_table
 * (entries not in use -1) and seqlens to match; *count (device) = live.  If
 * live > to->num_pages, `to` is left as it was and only count is written.
 * `from` is not changed.  Both have the same page_size, num_heads_kv,
 * num_slots and max_pages, and share no memory except, if the caller likes,
 * the scales (`to` keeps its own, which must be equal). */
size_t sinkattn_kv4_compact_workspace_size(const sinkattn_kv4_cache* from);
sinkattn_status sinkattn_kv4_compact(const sinkattn_kv4_cache* from, const sinkattn_kv4_cache* to, int32_t* count,
                                     void* workspace, size_t workspace_bytes, void* stream);

/* append: quantises k and v (bf16 [total, num_heads_kv, 64]) into the cache.
 * Rows cu_new[b] .. cu_new[b + 1] - 1 are the last positions of slot
 * slots[b], whose length already counts them (reserve first); cu_new is int32
 * [num_seqs + 1] on the device, nondecreasing, or NULL for total / num_seqs
 * rows each.  Rows behind the last offset are not read.  Per 16 dims with
 * y = x / factor: scale = e4m3(min(max|y| / 6, 448)), code = e2m1(y / scale),
 * both rounded to nearest even, codes saturating, 0 where the scale is 0.  16
 * dims with a y that is a NaN or an infinity in fp32 read back as NaN.  A slot
 * may be named once per call. */
sinkattn_status sinkattn_kv4_append(const sinkattn_kv4_cache* cache, const int32_t* slots, int32_t num_seqs,
                                    const int32_t* cu_new, int32_t total, const void* k, const void* v, void* stream);

/* read: the same rows back as bf16 (rounded once from the fp32 product), for
 * instance the whole prefix for sinkattn_fwd.  A slot may be named more than
 * once.  Rows before a sequence's begin are zero; rows behind the last offset
 * are left as they were. */
sinkattn_status sinkattn_kv4_read(const sinkattn_kv4_cache* cache, const int32_t* slots, int32_t num_seqs,
                                  const int32_t* cu, int32_t total, void* k, void* v, void* stream);

/* Decode forward over the cache: as sinkattn_decode_fwd (causal) with slots
 * for sequences.  q and o bf16 [num_seqs * q_per_seq, num_heads_q, 64], lse
 * fp32 [num_heads_q, num_seqs * q_per_seq]; row b * q_per_seq + i is position
 * seqlens[slots[b]] - q_per_seq + i.  Rows at negative positions (an idle
 * entry, a sequence shorter than q_per_seq) get o = 0, lse = -inf.  Scores are
 * fp32: a row that sees one beyond fp32's range in log2 units may read as NaN.
 * The lengths are read on the device.  (num_heads_q / num_heads_kv) * q_per_seq
 * <= 128.  The workspace (sinkattn_kv4_decode_workspace_size bytes for
 * num_rows = num_seqs * q_per_seq, 16-byte aligned, its size depends on the
 * device's SM count) is zero-filled once; every call leaves it usable for
 * later calls of any shape it is large enough for, not for calls that overlap
 * on the GPU.  Results do not depend on the order in which the GPU runs the
 * parts of the work. */
size_t sinkattn_kv4_decode_workspace_size(int64_t num_rows, int32_t num_heads_q);
sinkattn_status sinkattn_kv4_decode_fwd(const sinkattn_kv4_cache* cache, const int32_t* slots, int32_t num_seqs,
                                        int32_t q_per_seq, int32_t num_heads_q, int64_t window, int64_t prefix,
                                        float scale, const void* q, const float* sink, void* o, float* lse,
                                        void* workspace, size_t workspace_bytes, void* stream);

/* Token sampling from logits [rows][row_stride] (the first `vocab` of each
 * row; dtype 0 fp32, 1 bf16, 2 fp16) and one random number u[r] in [0, 1) per
 * row, with temperature, top_k, top_p and min_p per row (device, [rows]):
 *   e_i = exp((x_i - max x) / temperature), order: larger x first, of equal
 *   ones the lower index; top_k keeps the first top_k (<= 0 or >= vocab: all);
 *   top_p the shortest run of those whose mass is at least top_p of theirs
 *   (>= 1: all, <= 0: the first one); min_p those with e_i >= min_p (>= 1:
 *   those that equal the largest).
 *   The token is the first index whose kept mass up to and including it
 *   exceeds u times the kept mass.  temperature 0: the first in the order,
 *   with e at temperature 1.
 * tokens int32; logp = log(e / sum of all e), what sinkattn_grpo_loss takes
 * as logp_old; logq = log(e / kept mass) (0 where one token is kept).  Logits
 * of -inf are never chosen; a row of nothing else gives token -1 and -inf.  A
 * row with a NaN or +inf logit, a NaN parameter or a temperature that is
 * negative or above 1e36 gives token -1 and NaN.  u outside [0, 1) is clamped,
 * fp32 subnormals count as 0.  vocab <= 2^18, row_stride >= vocab, any
 * alignment of the rows. */
sinkattn_status sinkattn_sample_tokens(const void* logits, int32_t dtype, int32_t rows, int32_t vocab,
                                       int64_t row_stride, const float* u, const float* temperature,
                                       const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens,
                                       float* logp, float* logq, void* stream);

/* Packed-sequence front end (multi-turn trajectories of different lengths,
 * SinkFlex-RL section 3).  seqlens: device int32 [num_seqs];
 * cu_seqlens_out: device int32 [num_seqs + 1] receives the exclusive prefix
 * sum (cu[0] = 0).  Fails with INVALID_ARG for num_seqs < 0 or null pointers.
 * A negative length is clamped to 0 on the device. */
sinkattn_status sinkattn_varlen_plan(const int32_t* seqlens, int32_t num_seqs, int32_t* cu_seqlens_out,
                                     void* stream);

/* Padded <-> packed copies of a bf16 [*, H, D] tensor.
 * pack:   padded [B, Smax, H, D] -> packed [cu[B], H, D] (rows past each length are skipped).
 * unpack: packed -> padded; padding rows of `padded` are written with zeros.
 * cu_seqlens is the device copy of the offsets; each length must be <= Smax
 * (rows beyond Smax are not copied).  H * D * 2 bytes must be a multiple of 16. */
sinkattn_status sinkattn_pack(const void* padded, const int32_t* cu_seqlens, int32_t B, int32_t Smax,
                              int32_t H, int32_t D, void* packed, void* stream);
sinkattn_status sinkattn_unpack(const void* packed, const int32_t* cu_seqlens, int32_t B, int32_t Smax,
                                int32_t H, int32_t D, void* padded, void* stream);

/* Synchronises `stream`, then reads and clears the library's device status
 * word: SINKATTN_OK, or SINKATTN_ERR_TIMEOUT when a kernel gave up a bounded
 * wait since the last call (its outputs are then undefined). */
sinkattn_status sinkattn_get_device_status(void* stream);

/* Measurement hook.  kind 1 selects the forward attention kernel, kind 2
 * the backward main kernel, kind 3 the key-chunk kernel of the decode
 * forward (the warp-MMA kernel for at most 16 rows per (sequence, kv head),
 * the tensor-core kernel above).  With non-NULL `start` and `stop` (cudaEvent_t handles passed as
 * void*), every later sinkattn_fwd / sinkattn_bwd / sinkattn_decode_fwd call
 * records `start` on its stream immediately before that kernel's launch and
 * `stop` immediately after it, so the caller can time the kernel alone with
 * cudaEventElapsedTime.  NULL for both clears the hook.  The setting is
 * process-wide and not thread-safe; the events must outlive the calls.
 * Returns INVALID_ARG for an unknown kind or a half-NULL pair. */
sinkattn_status sinkattn_set_profile_events(int32_t kind, void* start, void* stop);

/* Self-test of the bounded waits the kernels use: launches one CTA that
 * waits on an mbarrier nothing ever arrives on, giving up after
 * `limit_cycles` SM cycles (1 .. 2e9) exactly as a kernel's wait does on a
 * timeout.  Afterwards sinkattn_get_device_status() reports
 * SINKATTN_ERR_TIMEOUT once.  Nothing faults or hangs; the context stays
 * usable.  INVALID_ARG for a limit out of range. */
sinkattn_status sinkattn_selftest_wait_timeout(int64_t limit_cycles, void* stream);

/* Static, human-readable name of a status. */
const char* sinkattn_status_string(sinkattn_status s);

/* Library version, major * 10000 + minor * 100 + patch. */
int32_t sinkattn_version(void);

#ifdef __cplusplus
}
#endif
#endif /* SINKATTN_H */
