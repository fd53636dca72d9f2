/*
 * mi355emb, the dense side of a step -- what the looked-up rows feed, on MI355X (gfx950):
 *   - attn_window_*: attention over ragged event sequences in which an event sees the last `window`
 *     events of its sequence, itself among them, and the sequence's first `sinks` events; forward,
 *     backward, and the serving form of one new event per sequence against a cache.
 *   - attn_shared_*: attention of the many candidates of a request to its one history and their own tokens;
 *     forward, backward, and the serving form against caches.
 *   - cache_q8_*: caches of keys and values in 8 bits, written as events come in and read back;
 *     attn_shared_cache_q8 and attn_window_decode_q8 read them as they are.
 *   - norm_gate_residual_*: the norm after a block, its gate, the scaled residual and the norm
 *     before the next block in one pass; forward and backward.
 *   - adamw_step, adamw_step_q8: an AdamW step over many weight tensors at once, with fp32 states
 *     or states held in 8 bits.
 *
 * Conventions are those of emb.h: 0 (EMB_OK) or a negative emb_status, emb_last_error() for the
 * message, nothing throws, device pointers are the caller's, device work goes to the caller's stream and
 * returns at once, and no call allocates device memory.  Workspaces may be reused by the next call
 * on the same stream.  Every result is the same from run to run (no atomics on values).  Every call
 * may be captured into a HIP graph.
 */
#ifndef MI355EMB_DENSE_H
#define MI355EMB_DENSE_H

#include "emb.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A third element type, of this header's calls only. */
#define EMB_BF16 2

/* ------------------------------------------------------------------ attention
 *
 * Query i of a sequence sees key j of the same sequence when j <= i and (i - j < window or
 * j < sinks).  With s_ij = scale * q_i . k_j over the keys seen, p_i = softmax(s_i) and
 *   out_i = sum_j p_ij v_j,   lse_i = log sum_j exp(s_ij).
 * Query head h reads key/value head h / (q_heads / kv_heads).
 */
typedef struct {
  int32_t dtype;    /* EMB_F16 or EMB_BF16: q, k, v, out and their gradients */
  int32_t q_heads;  /* a multiple of kv_heads */
  int32_t kv_heads;
  int32_t dim;      /* of a head: a multiple of 8, 8 to 128 */
  int32_t window;   /* at least 1; any value beyond the longest sequence makes it plain causal */
  int32_t sinks;    /* 0 to EMB_ATTN_MAX_SINKS */
  float scale;
} EmbAttn;

#define EMB_ATTN_MAX_SINKS 32

/*
 * Heads of tokens in device memory: element (s, t, h, d) at p + s * seq + t * tok + h * head + d,
 * strides in elements.  p must be 16-byte aligned and the strides multiples of 8 (EMB_EINVAL), so
 * views of one projection's output may be passed as they are.  `seq` is read for a cache only.  Inputs may
 * repeat (a stride of 0); tokens or heads of an output less than dim apart are refused (EMB_EINVAL).
 */
typedef struct {
  void* p;
  int64_t seq, tok, head;
} EmbHeads;

/*
 * Attention over the n_seq sequences of a ragged batch: sequence s holds tokens d_offsets[s] to
 * d_offsets[s + 1] - 1 of n_tok, as the bags of lookup_pool_fwd hold keys (offsets int32,
 * ascending from 0 to n_tok; empty sequences are fine).  Softmax statistics and sums are fp32.
 *   d_lse : nullable; fp32 [q_heads][n_tok], what the backward reads.
 * A key or value that is not finite reaches only the queries that see it (and in the backward, a
 * query or gradient only the keys it sees).  Sums that are not finite, in EMB_F16 also those of score gradients
 * over 65504, are computed once more: such a call takes a few times as long.  In EMB_F16 score gradients, and the
 * backward's probabilities, keep the bits that type has for them: fewer below 2^-14.
 * EMB_VALIDATE=1 checks the offsets first (it synchronises the stream); without it malformed
 * offsets give wrong results but no access outside the n_tok tokens.
 * Errors: EMB_EINVAL for a null pointer, a bad descriptor, alignment or stride; EMB_ERANGE for
 * n_tok or n_seq (or a cache's capacity) over 2^30, or more tiles than a launch can hold.
 */
int attn_window_fwd(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v,
                    const int32_t* d_offsets, int64_t n_seq, int64_t n_tok, const EmbHeads* out,
                    float* d_lse, emb_stream_t stream);

/* Workspace of attn_window_bwd (host only). */
int attn_window_bwd_workspace_bytes(const EmbAttn* a, int64_t n_seq, int64_t n_tok, size_t* bytes);

/*
 * Gradients of attn_window_fwd with respect to q, k and v, from its inputs, out and lse and the
 * gradient of out; dk and dv are summed over the query heads that share them.
 * d_ws (16-byte aligned): at least attn_window_bwd_workspace_bytes (EMB_ENOSPACE otherwise).
 */
int attn_window_bwd(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v,
                    const int32_t* d_offsets, int64_t n_seq, int64_t n_tok, const EmbHeads* out,
                    const float* d_lse, const EmbHeads* dout, const EmbHeads* dq,
                    const EmbHeads* dk, const EmbHeads* dv, void* d_ws, size_t ws_bytes,
                    emb_stream_t stream);

/*
 * Workspace of attn_window_decode for n_seq sequences with caches of `capacity` tokens (host only).  Fewer
 * sequences may need more: the keys of each are split over more of the GPU.
 */
int attn_window_decode_workspace_bytes(const EmbAttn* a, int64_t n_seq, int64_t capacity,
                                       size_t* bytes);

/*
 * The newest event of each of n_seq users against the cached keys and values of their sequences:
 * d_lens[s] (int32) events are cached, the newest included; its query is q's token s (q and out:
 * stride `tok` from one sequence to the next).  A length of 0 gives zeros; lengths are clamped to
 * [0, capacity].  Cache places at and past the length are not read.
 */
int attn_window_decode(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k_cache,
                       const EmbHeads* v_cache, const int32_t* d_lens, int64_t n_seq,
                       int64_t capacity, const EmbHeads* out, void* d_ws, size_t ws_bytes,
                       emb_stream_t stream);

/* ------------------------------------------------------------------ caches in 8 bits
 *
 * A cache holds the keys and values of n_seq sequences of up to `capacity` events as e4m3 codes (OCP, uint8) with
 * one power of two for each event's head: codes at (s, t, h, d) as EmbHeads says, exponents, a byte each, at
 * p + s * seq + t * tok + h * head of an EmbHeads of their own, in any order of dimensions (tok = 1 is read fastest).
 * The value of a code is code * 2^(exponent - 127).  The power of two brings the row's largest finite value into
 * [128, 256); a value becomes the nearest code, halfway the even one, but no code past the largest number of the
 * type that it came in.  What is not finite is held as NaN; a row of zeros has exponent 0.  An exponent of 255,
 * which no write makes, stands for NaN.
 * Codes are 8-byte aligned, their strides multiples of 8.  dim: a multiple of 8, 8 to 128.  kv_heads: 1 to 4096.
 */

/*
 * Writes keys and values of new events: sequence s's are tokens d_offsets[s] to d_offsets[s + 1] - 1 of n_tok (or
 * token s alone, without offsets: n_tok == n_seq), and go to places d_start[s] (0 without it) and on.  Places
 * outside [0, capacity) are left out.  dtype: EMB_F32, EMB_F16 or EMB_BF16, of k and v.  Nothing else of the
 * cache is touched.  Errors: EMB_EINVAL for a bad argument, alignment or stride, or places that overlap.
 */
int cache_q8_write(int32_t kv_heads, int32_t dim, int32_t dtype, const EmbHeads* k, const EmbHeads* v,
                   const int32_t* d_offsets, const int32_t* d_start, int64_t n_seq, int64_t n_tok,
                   const EmbHeads* k_cache, const EmbHeads* k_exp, const EmbHeads* v_cache,
                   const EmbHeads* v_exp, int64_t capacity, emb_stream_t stream);

/*
 * The way back: the values of places d_start[s] and on to tokens of k and v in dtype (exact but in EMB_F16 past
 * its range: infinities, and below its smallest numbers).  A place outside the cache gives zeros.
 */
int cache_q8_read(int32_t kv_heads, int32_t dim, int32_t dtype, const EmbHeads* k_cache, const EmbHeads* k_exp,
                  const EmbHeads* v_cache, const EmbHeads* v_exp, int64_t capacity, const int32_t* d_offsets,
                  const int32_t* d_start, int64_t n_seq, int64_t n_tok, const EmbHeads* k, const EmbHeads* v,
                  emb_stream_t stream);

/* attn_window_decode against a cache in 8 bits, whose values it reads as a->dtype. */
int attn_window_decode_q8_workspace_bytes(const EmbAttn* a, int64_t n_seq, int64_t capacity, size_t* bytes);
int attn_window_decode_q8(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k_cache, const EmbHeads* k_exp,
                          const EmbHeads* v_cache, const EmbHeads* v_exp, const int32_t* d_lens, int64_t n_seq,
                          int64_t capacity, const EmbHeads* out, void* d_ws, size_t ws_bytes, emb_stream_t stream);

/* ------------------------------------------------------------------ attention of candidates
 *
 * A request has a history of events and any number of candidates, each of one or more tokens.  Token i of a
 * candidate sees the history and its candidate's tokens up to itself; no candidate sees another.  A candidate
 * stands at the place after the history's n events: event j is seen when n - j < window or j < sinks, as the next
 * event of that sequence would see it in attn_window_fwd.  window and sinks say nothing about a candidate's own
 * tokens: all of them see the same events, so under a window shorter than the history the later tokens of a candidate see
 * a few events more than they would if the earlier ones had been appended to the sequence.  Otherwise as there: scores, softmax, heads that share keys, EmbAttn and its limits.  A score of minus
 * infinity weighs nothing beside others, and 0 times a value that is not finite is NaN; where all that a row sees are such
 * scores, its out is NaN and its lse minus infinity, however many workgroups share the keys.
 *
 * Requests are ragged: request s holds tokens d_offsets[s] to d_offsets[s + 1] - 1 of q, k and v (int32, ascending
 * from 0 to at most n_tok).  d_first (nullable: every token is a candidate of its own): int32 [n_tok], for each token the
 * first token of its candidate; a candidate's tokens stand together.  Rows of tokens, or events of a packed
 * history, past the last offset belong to no request: nothing is written there.
 */

/*
 * Training: histories are packed, request s's are events d_hist_offsets[s] to d_hist_offsets[s + 1] - 1 of hist_k
 * and hist_v (int32, ascending from 0 to at most n_hist).
 *   d_lse : nullable; fp32 [q_heads][n_tok], what the backward reads.
 *   d_ws  : 16-byte aligned, at least attn_shared_fwd_workspace_bytes (EMB_ENOSPACE otherwise); null where that is 0.
 * What is not finite reaches only the tokens that see it.  EMB_VALIDATE=1 checks offsets and first (it synchronises
 * the stream); without it malformed ones give wrong results but no access outside the tokens and events.
 * Errors: as attn_window_fwd's.
 */
int attn_shared_fwd_workspace_bytes(const EmbAttn* a, int64_t n_seq, int64_t n_tok, int64_t n_hist, size_t* bytes);
int attn_shared_fwd(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v,
                    const EmbHeads* hist_k, const EmbHeads* hist_v, const int32_t* d_offsets, const int32_t* d_first,
                    const int32_t* d_hist_offsets, int64_t n_seq, int64_t n_tok, int64_t n_hist,
                    const EmbHeads* out, float* d_lse, void* d_ws, size_t ws_bytes, emb_stream_t stream);

/*
 * The backward: gradients with respect to q, k, v and the history, from the forward's inputs, out and lse and the
 * gradient of out.  The history's are summed over the request's tokens and the query heads that share a head; events
 * that no token sees get zeros.  In EMB_F16 score gradients are brought to where 16 bits hold them, so that neither those
 * over 65504 nor small ones (of a small dout, or many events) cost the results bits that these have.
 * d_ws (16-byte aligned): at least attn_shared_bwd_workspace_bytes (EMB_ENOSPACE otherwise).
 */
int attn_shared_bwd_workspace_bytes(const EmbAttn* a, int64_t n_seq, int64_t n_tok, int64_t n_hist, size_t* bytes);
int attn_shared_bwd(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v,
                    const EmbHeads* hist_k, const EmbHeads* hist_v, const int32_t* d_offsets, const int32_t* d_first,
                    const int32_t* d_hist_offsets, int64_t n_seq, int64_t n_tok, int64_t n_hist,
                    const EmbHeads* out, const float* d_lse, const EmbHeads* dout, const EmbHeads* dq,
                    const EmbHeads* dk, const EmbHeads* dv, const EmbHeads* dhist_k, const EmbHeads* dhist_v,
                    void* d_ws, size_t ws_bytes, emb_stream_t stream);

/*
 * Serving: the history of request s is the first d_lens[s] (int32, clamped to [0, capacity]) events of its cache.
 * Cache places at and past the length are not read.  The workspace is enough for any window.
 */
int attn_shared_cache_workspace_bytes(const EmbAttn* a, int64_t n_seq, int64_t n_tok, int64_t capacity,
                                      size_t* bytes);
int attn_shared_cache(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v,
                      const EmbHeads* k_cache, const EmbHeads* v_cache, const int32_t* d_offsets,
                      const int32_t* d_first, const int32_t* d_lens, int64_t n_seq, int64_t n_tok,
                      int64_t capacity, const EmbHeads* out, void* d_ws, size_t ws_bytes, emb_stream_t stream);
/* The same against a cache in 8 bits (q, k and v have a->dtype), with the same workspace. */
int attn_shared_cache_q8(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v,
                         const EmbHeads* k_cache, const EmbHeads* k_exp, const EmbHeads* v_cache,
                         const EmbHeads* v_exp, const int32_t* d_offsets, const int32_t* d_first,
                         const int32_t* d_lens, int64_t n_seq, int64_t n_tok, int64_t capacity, const EmbHeads* out,
                         void* d_ws, size_t ws_bytes, emb_stream_t stream);

/* ------------------------------------------------------------------ norms, gate, residual
 *
 * Row by row over `dim` columns, rms(z) = z * rsqrt(mean(z^2) + eps):
 *   n = w_post * rms(y)                 (n = y without w_post)
 *   r = alpha * x + gate * n            (the residual stream; alpha * x without y)
 *   h = w_pre * rms(r)                  (the next block's input)
 * gate: none, one row for all (EMB_GATE_VECTOR), or a row of its own for each (EMB_GATE_ROWS).
 * x, y, gate, r, h and their gradients have `dtype` (EMB_F32, EMB_F16 or EMB_BF16) and are contiguous
 * [rows][dim]; w_post, w_pre and the gradients of them and of a gate vector are fp32 [dim].
 * Arithmetic is fp32.  dim: 1 to 8192.
 */
typedef enum { EMB_GATE_NONE = 0, EMB_GATE_VECTOR = 1, EMB_GATE_ROWS = 2 } emb_gate;

/*
 * Nullable: y with w_post and gate (the norm before the first block), w_post, w_pre with h (the last
 * block), r.  r may be x's buffer and h may be y's.  h is computed from r before r is rounded.
 */
int norm_gate_residual_fwd(const void* x, const void* y, const void* gate, int32_t gate_kind,
                           const float* w_post, const float* w_pre, int64_t rows, int32_t dim,
                           int32_t dtype, float alpha, float eps, void* r, void* h,
                           emb_stream_t stream);

/* Workspace of norm_gate_residual_bwd (host only). */
int norm_gate_residual_bwd_workspace_bytes(int64_t rows, int32_t dim, size_t* bytes);

/*
 * The backward: from r as stored, y, gate and the weights, and the gradients dr of r (nullable: 0)
 * and dh of h (null exactly where w_pre is), to dx, dy, dgate, dw_post and dw_pre (each output
 * nullable).  dgate: dtype [rows][dim] for EMB_GATE_ROWS, fp32 [dim] for EMB_GATE_VECTOR.  Column
 * sums are fp32 over a block's rows, then over the blocks.  dx may be dr's buffer, dy may be y's or
 * dh's.  rows == 0 gives zero dw_post, dw_pre and gate vector gradient.
 */
int norm_gate_residual_bwd(const void* r, const void* y, const void* gate, int32_t gate_kind,
                           const float* w_post, const float* w_pre, int64_t rows, int32_t dim,
                           int32_t dtype, float alpha, float eps, const void* dr, const void* dh,
                           void* dx, void* dy, void* dgate, float* dw_post, float* dw_pre,
                           void* d_ws, size_t ws_bytes, emb_stream_t stream);

/* ------------------------------------------------------------------ AdamW
 *
 * For every element of n_tensors weight tensors, g' = g * *d_grad_scale (1 without it), step t >= 1:
 *   m = beta1 m + (1 - beta1) g'        v = beta2 v + (1 - beta2) g'^2
 *   w = w - lr (m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps) + weight_decay w)
 * Weights are fp32; copies (nullable as a whole) receive the new weights in copy_dtype.
 *   n            : elements of each tensor, 0 to 2^32 - 1
 *   w, grads, copies : host arrays of n_tensors device pointers, aligned to their elements
 *   weight_decay : host array of n_tensors
 * The states of all tensors lie in one array each: tensor i's elements start where those of i - 1,
 * rounded up to a multiple of EMB_ADAMW_BLOCK, end; adamw_state_elems gives the total.  State arrays
 * are 16-byte aligned.  What pads a tensor is written as zero.  lr, the betas and eps come in 64 bits, so
 * that 1 - beta and the corrections are rounded to fp32 once; elements are computed in fp32.
 */
#define EMB_ADAMW_BLOCK 128

int adamw_state_elems(const int64_t* n, int32_t n_tensors, int64_t* elems);

int adamw_step(int32_t n_tensors, const int64_t* n, void* const* w, const void* const* grads,
               int32_t grad_dtype, void* const* copies, int32_t copy_dtype, float* d_m, float* d_v,
               int64_t state_elems, int64_t step, double lr, double beta1, double beta2, double eps,
               const float* weight_decay, const float* d_grad_scale, emb_stream_t stream);

/*
 * The same with states in 8 bits: m and the root of v, each as e4m3 codes (OCP, uint8) with one
 * power of two per EMB_ADAMW_BLOCK elements (d_m_exp, d_v_exp: its exponent + 127, uint8; a zeroed
 * state is all zeros).  The power of two brings a block's largest finite value into [128, 256).
 * A value becomes one of the two codes beside it, the upper one with the probability that keeps the
 * mean, by 16 bits of a hash of `seed` and the element's index in the state array: with rounding to
 * the nearest a second moment would never move, since a step changes its root by less than half a code.
 * Exactly: at a place p in [0, 1) between the two, with bits b, the upper one where p + (b + 0.5) / 65536 > 1.
 * `seed` is to differ from step to step.  A root that is not zero does not become zero.  What is
 * not finite is held as NaN.  The weights are updated from the states before they are rounded.
 */
int adamw_step_q8(int32_t n_tensors, const int64_t* n, void* const* w, const void* const* grads,
                  int32_t grad_dtype, void* const* copies, int32_t copy_dtype, uint8_t* d_m,
                  uint8_t* d_m_exp, uint8_t* d_v, uint8_t* d_v_exp, int64_t state_elems,
                  int64_t step, double lr, double beta1, double beta2, double eps,
                  const float* weight_decay, const float* d_grad_scale, uint64_t seed,
                  emb_stream_t stream);

/* The values that elems (a multiple of EMB_ADAMW_BLOCK) codes stand for, in EMB_BF16 (exact except
 * below its smallest numbers) or EMB_F32. */
int adamw_q8_values(const uint8_t* d_codes, const uint8_t* d_exp, int64_t elems, void* d_out,
                    int32_t out_dtype, emb_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MI355EMB_DENSE_H */
