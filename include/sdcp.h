/*
 * sdcp.h - C ABI of libsdcp, the batched acceptance step of a speculative-decoding
 * verifier, for NVIDIA GB300 (sm_103a).
 *
 * The operation is the verifier's "Acceptance" step of the Speculative Decoding
 * Coordination Protocol (IETF draft-li-mlc-inference-acceleration-00, "Speculative
 * Decoding Coordination Protocol (SDCP) for Distributed Inference with Multi-Level
 * Caches"):
 *   - the sampling profile of Section 4.1 (temperature, then top-k, then top-p; a
 *     temperature of zero selects the most probable token, ties to the smallest id)
 *     turns logits into the distributions p (target) and q (draft);
 *   - Section 6.4, Rule 1 (greedy) and Rule 2 (speculative sampling) decide how many
 *     of the M proposed tokens are accepted and which one additional token is emitted;
 *   - Section 6.3, "Preconditions of the rule": q[i](x[i]) must be non-zero at every
 *     proposed position before any random value is drawn;
 *   - Section 6.3, "Scoring": the verifier may batch the proposals of many sessions;
 *   - Section 5.2, "verdict": the results are the accepted count a (0 <= a <= M) and
 *     the emitted tokens;
 *   - Table 2 (Section 6.9), problem types: a per-session status mirrors the ones that
 *     can arise inside this call.
 *
 * Random values are Philox4x32-10 uniforms (Salmon, Moraes, Dror and Shaw,
 * "Parallel random numbers: as easy as 1, 2, 3", SC'11), keyed by the session's
 * 64-bit seed (key word 0 = low 32 bits, key word 1 = high 32 bits), with counter
 * (position, purpose, round, session_tag); purpose 0 is the acceptance test and 1 the
 * additional token, as in SDCP Section 6.4.  The uniform is
 * ((w0 << 21) | (w1 >> 11)) * 2^-53, the first 53 bits of the output, like the
 * 53-bit value of Section 6.4.
 *
 * Ragged batch layout (all device memory, row-major, row stride V elements):
 *   B sessions; session b proposes M_b = m_offsets[b+1] - m_offsets[b] tokens.
 *   target row of session b at position i (i = 0..M_b):  T[m_offsets[b] + b + i]
 *   draft row of session b at position i (i = 0..M_b-1): D[m_offsets[b] + i]
 *   draft token of session b at position i:               draft_tokens[m_offsets[b] + i]
 *   output tokens of session b:                           out_tokens[m_offsets[b] + b + j],
 *                                                         j = 0..n_out[b]-1; the slots
 *                                                         j = n_out[b]..M_b hold -1.
 *
 * Ownership: the caller owns every buffer and the stream.  The library allocates
 * nothing, never synchronises the stream and keeps no state between calls, so calls on
 * different streams with different workspaces may run concurrently.  Results are a
 * pure function of the inputs: re-running a call reproduces every output bit for bit.
 *
 * Errors: a non-zero return code (SDCP_E_*) means nothing was launched (argument
 * errors) or a launch failed (SDCP_E_LAUNCH).  Errors that depend on values stored in
 * device memory are reported per session in status[] (SDCP_S_*); such a session gets
 * accepted = 0, n_out = 0 and all its output slots -1, and so commits nothing.
 */
#ifndef SDCP_H
#define SDCP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types of the logits ------------------------------------------------ */
#define SDCP_F32  0   /* IEEE binary32 */
#define SDCP_BF16 1   /* bfloat16 (upper half of a binary32) */

/* ---- acceptance rules: SDCP Section 10.2.2 registry ------------------------------ */
#define SDCP_RULE_GREEDY 1              /* Rule 1 */
#define SDCP_RULE_SPECULATIVE_SAMPLING 2 /* Rule 2 */
/* A private-use rule (Section 10.2 keeps ids 192-255 for private use): the relaxed rule of
 * "Inference: KV Cache, Batching, Speculative Decoding" (section on variants of the
 * acceptance rule: accept if the token is in the target's top-k).  Acceptance test: x[i]
 * lies in the kept set of p[i], the target distribution after the session's sampling profile
 * (top_k = k makes it "in the target's top-k"), with a finite logit.  Additional token: a
 * draw from p[a] (purpose 1) at the first rejection, or from p[M+1] when all M are accepted;
 * argmax at temperature 0.  The proposal carries tokens only: draft rows are never read.  It
 * does NOT preserve the target distribution, and needs no trust in a drafter's q. */
#define SDCP_RULE_RELAXED_TOP_K 192

/* ---- return codes ---------------------------------------------------------------- */
#define SDCP_OK           0
#define SDCP_E_INVALID    1  /* null pointer, B < 0, V < 1, unknown dtype, sizes overflow */
#define SDCP_E_WORKSPACE  2  /* workspace null, too small or not 256-byte aligned */
#define SDCP_E_ALIGN      3  /* a logits pointer is not aligned to its element size, a pointer or
                                stride of the cache calls not to 16 bytes, or another array of
                                the serving calls not to the 4 bytes of its words */
#define SDCP_E_TOO_LARGE  4  /* V above SDCP_MAX_VOCAB or a row count above INT32_MAX */
#define SDCP_E_LAUNCH     5  /* a CUDA launch failed (cudaGetLastError after launch) */
#define SDCP_E_DEVICE     6  /* no usable CUDA device / device query failed */
#define SDCP_E_SCRATCH_LIMIT 7 /* batch needs more scratch than SDCP_NOALLOC_SCRATCH_BYTES */

/* ---- per-session status (mirrors SDCP Table 2 problem types) ---------------------- */
#define SDCP_S_OK             0
#define SDCP_S_BAD_PROPOSAL   1  /* "sdcp-bad-proposal": a token outside [0,V), or, under
                                    Rule 2, q[i](x[i]) = 0 at some position (Section 6.4) */
#define SDCP_S_LIMIT          2  /* "sdcp-limit": M outside [1, SDCP_MAX_M] (m_max <= 64,
                                    Section 4.1; 1 <= M, Section 6.2) */
#define SDCP_S_BAD_PARAMS     3  /* unknown rule id, top_p_milli > 1000, inconsistent
                                    m_offsets, or a scored row holding NaN, +inf or only
                                    -inf (no distribution can be formed) */
#define SDCP_S_Q_UNAVAILABLE  4  /* "sdcp-q-unavailable": Rule 2 without draft logits */
#define SDCP_S_INTERNAL       5  /* the call gave up a bounded wait on the GPU (a bulk copy
                                    that never completed); no output of the call is valid */

#define SDCP_MAX_M      64          /* m_max upper bound, SDCP Section 4.1 contract */
#define SDCP_MAX_VOCAB  (1 << 24)   /* ids and ranks are int32; 16 Mi keeps all sums exact */

/* One per session, device memory, 32 bytes, naturally aligned. */
typedef struct sdcp_session_params {
  uint32_t rule_id;           /* SDCP_RULE_*; anything else -> SDCP_S_BAD_PARAMS */
  uint32_t temperature_milli; /* temperature x 1000 (Section 4.1); 0 selects the argmax */
  uint32_t top_k;             /* keep the top_k most probable; 0 or >= V disables */
  uint32_t top_p_milli;       /* nucleus mass x 1000, <= 1000; 1000 disables */
  uint64_t seed;              /* Philox key of the verifier's random values */
  uint32_t round;             /* protocol round of this proposal */
  uint32_t session_tag;       /* 32 bits that name the session (e.g. the first four
                                 octets of its 16-octet identifier), not the batch slot */
} sdcp_session_params;

/*
 * Bytes of device workspace sdcp_verify_batch and sdcp_row_stats need for a batch of
 * B sessions with total_drafts = sum of M_b proposed tokens.  Returns 0 for invalid
 * sizes (B < 0, total_drafts < 0, V < 1 or V > SDCP_MAX_VOCAB).
 */
size_t sdcp_workspace_bytes(int64_t V, int32_t B, int64_t total_drafts);

/*
 * Verify one ragged batch (SDCP Sections 4.1, 6.3 and 6.4).
 *
 * target_logits  device, [total_drafts + B][V] of dtype; the scores p[1..M+1] of each
 *                session (Section 6.3 "Scoring"), laid out as described above.
 * draft_logits   device, [total_drafts][V] of dtype, or NULL when no session uses Rule 2
 *                (a Rule 2 session then gets SDCP_S_Q_UNAVAILABLE).  Rows of Rule 1
 *                sessions are never read.  The profile of the session is applied to these
 *                logits to form q (the draft distribution the tokens were sampled from).
 * dtype          SDCP_F32 or SDCP_BF16, for both logits arrays.
 * V              vocabulary size, 1..SDCP_MAX_VOCAB.  Any V is accepted; rows whose start
 *                is not 16-byte aligned are read with narrower loads at their ends.
 * B              number of sessions, >= 0 (B = 0 launches nothing).
 * m_offsets      device, [B+1] int32, m_offsets[0] = 0, non-decreasing,
 *                m_offsets[B] = total_drafts.  A session whose own pair m_offsets[b],
 *                m_offsets[b+1] is out of order or out of range gets SDCP_S_BAD_PARAMS;
 *                offsets out of order elsewhere leave the results of the sessions they
 *                overlap unspecified.  Never an out-of-range access.
 * total_drafts   host copy of m_offsets[B] (sizes the launch without a device read).
 * draft_tokens   device, [total_drafts] int32, the proposed tokens x[i].
 * params         device, [B] sdcp_session_params.
 * accepted       device out, [B] int32: a, the number of accepted draft tokens.
 * n_out          device out, [B] int32: a + 1 emitted tokens (0 for a failed session).
 * out_tokens     device out, [total_drafts + B] int32 (layout above).
 * status         device out, [B] int32 SDCP_S_*.
 * workspace      device scratch of at least sdcp_workspace_bytes(V, B, total_drafts)
 *                bytes, 256-byte aligned; its contents need no initialisation and are
 *                garbage afterwards.
 * stream         the cudaStream_t (as void*) all work is enqueued on; NULL = legacy stream.
 *
 * Returns SDCP_OK or SDCP_E_*.  Asynchronous: results are ready when the stream reaches
 * this point.
 */
int sdcp_verify_batch(const void* target_logits, const void* draft_logits, int dtype,
                      int64_t V, int32_t B, const int32_t* m_offsets, int64_t total_drafts,
                      const int32_t* draft_tokens, const sdcp_session_params* params,
                      int32_t* accepted, int32_t* n_out, int32_t* out_tokens,
                      int32_t* status, void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * The two phases of sdcp_verify_batch as separate calls (same arguments, same workspace):
 * phase 1 (sdcp_verify_rows) computes the statistics of every scored row of the sampling
 * profile (Section 4.1) into the workspace; phase 2 (sdcp_verify_sessions) runs the
 * precondition, the acceptance tests, the first-rejection scan and the draw of the
 * additional token (Sections 6.3, 6.4) and writes the outputs.  Calling phase 1 then
 * phase 2 on one stream is exactly sdcp_verify_batch; a profiler or a scheduler can put an
 * event between them.  Return codes as for sdcp_verify_batch.
 */
int sdcp_verify_rows(const void* target_logits, const void* draft_logits, int dtype,
                     int64_t V, int32_t B, const int32_t* m_offsets, int64_t total_drafts,
                     const int32_t* draft_tokens, const sdcp_session_params* params,
                     void* workspace, size_t workspace_bytes, void* stream);
int sdcp_verify_sessions(const void* target_logits, const void* draft_logits, int dtype,
                         int64_t V, int32_t B, const int32_t* m_offsets, int64_t total_drafts,
                         const int32_t* draft_tokens, const sdcp_session_params* params,
                         int32_t* accepted, int32_t* n_out, int32_t* out_tokens,
                         int32_t* status, void* workspace, size_t workspace_bytes,
                         void* stream);

/*
 * Per-row statistics of the sampling profile (parity hook for the first phase).
 *
 * Same inputs as sdcp_verify_batch.  For every target row r (0 <= r < total_drafts + B)
 * and then every draft row (total_drafts of them) it writes one sdcp_row_stat to
 * stats_out (device, [2 * total_drafts + B]), target rows first.  All rows are given the
 * full statistics regardless of the session's rule (draft rows of a session with an
 * invalid rule or M get flags = SDCP_ROW_SKIPPED).  Row statistics follow Section 4.1:
 *   lmax    the largest logit of the row (before temperature);
 *   log_s   natural log of S = sum over the kept set of exp((l_j - lmax) * 1000/T);
 *   lp_x    natural log of the probability of the row's draft token x (target row i < M
 *           and draft row i carry x[i]); -inf when x is outside the kept set or its
 *           logit is -inf; NaN for rows without a draft token (target row M) or x out
 *           of range;
 *   argmax  smallest id among the largest logits;
 *   kept    number of tokens in the kept set (1 when the temperature is 0);
 *   flags   SDCP_ROW_* bits.
 */
typedef struct sdcp_row_stat {
  float lmax;
  float log_s;
  float lp_x;
  int32_t argmax;
  int32_t kept;
  uint32_t thr_key;   /* internal: order key of the lowest kept value */
  int32_t thr_n;      /* internal: how many tokens with that value are kept, the first ones
                         in id order (INT32_MAX: all) */
  uint32_t flags;
} sdcp_row_stat;

#define SDCP_ROW_INVALID   1u  /* NaN, +inf, or no finite logit: no distribution */
#define SDCP_ROW_X_KEPT    2u  /* the draft token is in the kept set with a finite logit */
#define SDCP_ROW_SKIPPED   4u  /* row not processed */
#define SDCP_ROW_FALLBACK  8u  /* the threshold needed the generic multi-pass search */

int sdcp_row_stats(const void* target_logits, const void* draft_logits, int dtype,
                   int64_t V, int32_t B, const int32_t* m_offsets, int64_t total_drafts,
                   const int32_t* draft_tokens, const sdcp_session_params* params,
                   sdcp_row_stat* stats_out, void* workspace, size_t workspace_bytes,
                   void* stream);

/*
 * sdcp_verify_batch for callers that cannot allocate device memory.
 *
 * The SDCP draft has no counterpart to this entry point: it exists for callers that must not
 * call cudaMalloc, such as code running inside a CUDA graph being built by someone else,
 * an allocator-less runtime, or a plugin whose host forbids device allocations.  Instead
 * of a caller-provided workspace it uses a scratch array of SDCP_NOALLOC_SCRATCH_BYTES that
 * lives in the library itself (a file-scope __device__ array): every GPU that loads the
 * library holds that memory until the process exits.  The caller still passes the inputs
 * and outputs, exactly as for sdcp_verify_batch, and gets identical results.
 *
 * Limit: sdcp_workspace_bytes(V, B, total_drafts) must not exceed
 * SDCP_NOALLOC_SCRATCH_BYTES; larger batches are rejected with SDCP_E_SCRATCH_LIMIT before
 * anything is launched.  The function calls no cudaMalloc, cudaFree or other allocating
 * routine.
 * Set-up: the first call on a device looks up the array's device address on the current
 * device (cudaGetSymbolAddress) and caches it; make that first call outside any stream
 * capture.  The current device must be the one the stream and the buffers belong to.
 * Sharing: all calls on a device share the one array and it keeps whatever the last call
 * left in it; nothing in it needs to start at zero.  Calls whose work overlaps on the GPU
 * (different streams, or host threads without ordering) race on the array: serialise them.
 * Returns as sdcp_verify_batch, plus SDCP_E_DEVICE if the device or the array's address
 * cannot be obtained.
 */
#define SDCP_NOALLOC_SCRATCH_BYTES ((size_t)2 << 20)
int sdcp_verify_batch_noalloc(const void* target_logits, const void* draft_logits, int dtype,
                              int64_t V, int32_t B, const int32_t* m_offsets,
                              int64_t total_drafts, const int32_t* draft_tokens,
                              const sdcp_session_params* params, int32_t* accepted,
                              int32_t* n_out, int32_t* out_tokens, int32_t* status,
                              void* stream);

/* ---- random values of the acceptance step --------------------------------------- */
#define SDCP_RNG_PHILOX4X32_10 0  /* counter-based Philox (the default, described above) */
#define SDCP_RNG_HMAC_SHA256   1  /* the draft's own derivation (Section 6.4, last
                                     paragraph): HMAC-SHA-256 keyed with the seed as eight
                                     octets in network order, over "SDCP-VERIFY-1" || 0x00
                                     || session (16 octets) || uint32(round) || uint32(i) ||
                                     uint8(purpose), the first 53 bits / 2^53; i is the
                                     1-based position of the pages (the acceptance test of
                                     0-based position k uses i = k + 1, the additional token
                                     after a accepted tokens i = a + 1) */

/* Options of sdcp_verify_batch_ex (host struct). */
typedef struct sdcp_verify_options {
  uint32_t struct_size;         /* sizeof(sdcp_verify_options) */
  uint32_t rng_id;              /* SDCP_RNG_* */
  const uint8_t* session_ids;   /* device, [B][16]: each session's 16-octet identifier
                                   (Section 5.2 session-id); needed by SDCP_RNG_HMAC_SHA256,
                                   ignored by Philox (which uses params[b].session_tag) */
  const float* q_rows;          /* device, [total_drafts][V] binary32, or NULL: q given as the
                                   drafter's rows of probabilities (Section 5.2 q_rows; q[i]
                                   is row i of the session, Section 6.4 Rule 2), used as given
                                   (no sampling profile).  Draft logits are then not read (they
                                   may be NULL) and the first phase reads target rows only.
                                   q(x) = 0 gives SDCP_S_BAD_PROPOSAL; a q(x) that is NaN,
                                   infinite or negative gives SDCP_S_BAD_PARAMS; other values
                                   of a row are used as given. */
} sdcp_verify_options;

/*
 * sdcp_verify_batch with options: the same arguments, layout and results, with the random
 * values chosen by opts->rng_id and q from the draft logits or from opts->q_rows.
 * opts = NULL is sdcp_verify_batch.  Returns SDCP_E_INVALID for an unknown rng_id, a
 * struct_size below sizeof(sdcp_verify_options), or the HMAC generator without session_ids;
 * SDCP_E_ALIGN for q_rows not aligned to 4 bytes.
 */
int sdcp_verify_batch_ex(const void* target_logits, const void* draft_logits, int dtype,
                         int64_t V, int32_t B, const int32_t* m_offsets, int64_t total_drafts,
                         const int32_t* draft_tokens, const sdcp_session_params* params,
                         int32_t* accepted, int32_t* n_out, int32_t* out_tokens,
                         int32_t* status, void* workspace, size_t workspace_bytes,
                         const sdcp_verify_options* opts, void* stream);

/* ---- the commit step after acceptance (Sections 4.2, 6.3, 6.5) ------------------- */
/* actions of a verdict (Section 4.1 "action"; Section 6.5.2) */
#define SDCP_ACTION_NONE        (-1) /* the session's status was not SDCP_S_OK: nothing
                                        committed, its state unchanged */
#define SDCP_ACTION_CONTINUE    0
#define SDCP_ACTION_REDUCE      1
#define SDCP_ACTION_SWITCH      2
#define SDCP_ACTION_SELF_DECODE 3
#define SDCP_ACTION_FINISH      4
#define SDCP_ACTION_FAIL        5
#define SDCP_NO_SELF_LOAD  0xFFFFFFFFu  /* the contract has no self_load member */

/* The contract terms of one session the commit step uses (Section 4.1), 48 bytes, device. */
typedef struct sdcp_commit_params {
  uint32_t max_new;       /* maximum output tokens of the session */
  uint32_t stop_offset;   /* its stop tokens are stop_tokens[stop_offset .. +stop_count) */
  uint32_t stop_count;
  uint32_t m_max;         /* upper bound on M (<= SDCP_MAX_M); caps m_cap */
  uint32_t low_rounds;    /* R >= 1, the escalation period */
  uint32_t low_ratio;     /* percent 0..100; 0 = absent (a round is low iff a = 0) */
  uint32_t self_load;     /* percent 0..100, or SDCP_NO_SELF_LOAD */
  uint32_t fallback_len;  /* 1..8 entries of fallback[] */
  uint8_t fallback[8];    /* the ladder: SDCP_ACTION_REDUCE, _SWITCH, _SELF_DECODE, _FAIL */
  uint32_t m_restore;     /* after a round that is not low, m_cap grows by this, up to m_max
                             (Section 6.5.1: "restore gradually"; 0 = never) */
  uint32_t reserved;
} sdcp_commit_params;

/* The verifier's per-session state between rounds, 64 bytes, device; read and updated. */
typedef struct sdcp_session_state {
  uint8_t digest[32];     /* d[n], the committed-prefix digest (Section 4.2) */
  uint32_t committed;     /* n, the committed length */
  uint32_t c, g, j;       /* consecutive low rounds, consecutive rounds not low, position in
                             the fallback list (Section 6.5.2) */
  uint32_t m_cap;         /* the largest M of the next round (Section 6.5.1); set it to
                             m_init before the first round */
  uint32_t reserved[3];
} sdcp_session_state;

/*
 * The commit step of one batch, after sdcp_verify_batch on the same stream (Section 6.3,
 * steps "Acceptance" (its truncation), "Commit" and "Control"; Sections 4.2 and 6.5).  For
 * each session b whose status is SDCP_S_OK:
 *   - truncation: the emitted tokens out_tokens[m_offsets[b] + b ..][0 .. n_out[b]) are
 *     cut after the first stop token of the session (the stop token itself is emitted)
 *     and to at most max_new - committed tokens; n_out[b] is lowered in place and the
 *     dropped slots set to -1;
 *   - commit: state.digest becomes d[n + m] by d[k] = SHA-256(d[k-1] || uint32(o[k])) over
 *     the m tokens kept, and state.committed grows by m;
 *   - control: the round is low if 100 a < low_ratio M (or, with low_ratio 0, if a = 0),
 *     with a = accepted[b] and M = m_offsets[b+1] - m_offsets[b]; the counters c, g, j and
 *     m_cap follow Section 6.5.2 (the ladder entry j applies when c reaches R, skipping
 *     self_decode unless self_load is present and load_percent <= self_load; "fail" when no
 *     entry remains; reduce halves m_cap, at least 1); a round that emitted a stop token or
 *     reached max_new gets SDCP_ACTION_FINISH instead (its counters are still updated, no
 *     ladder entry is applied).
 *   action[b] receives the SDCP_ACTION_* of the round (SDCP_ACTION_NONE for a session whose
 *   status is not SDCP_S_OK; its state, n_out and tokens are left as they are).
 * All pointers are device memory: m_offsets, accepted, status [B] / [B+1] as written by
 * sdcp_verify_batch; n_out, out_tokens in/out; cparams [B]; stop_tokens [sum of
 * stop_count] (may be NULL when every stop_count is 0); state [B] in/out; action [B] out.
 * Asynchronous on `stream`; allocates nothing.  Returns SDCP_OK, SDCP_E_INVALID (null
 * pointer, B < 0) or SDCP_E_LAUNCH.  Contract terms out of range (low_rounds 0,
 * fallback_len > 8) are read as the nearest valid value (1, 8).
 */
int sdcp_commit_batch(int32_t B, const int32_t* m_offsets, const int32_t* accepted,
                      int32_t* n_out, int32_t* out_tokens, const int32_t* status,
                      const sdcp_commit_params* cparams, const uint32_t* stop_tokens,
                      sdcp_session_state* state, uint32_t load_percent, int32_t* action,
                      void* stream);

/* ---- before a verify call: penalties, biases and grammar masks on logits ---------- */
/* Which rows of a batch an array of logits holds: target rows (M_b + 1 of each session,
 * session b's first row is m_offsets[b] + b) or draft rows (M_b of each, first row
 * m_offsets[b]).  Row i of a session is the distribution after its first i drafts. */
#define SDCP_ROWS_TARGET 0
#define SDCP_ROWS_DRAFT  1

/* The logit controls of one session, 32 bytes, device memory, naturally aligned. */
typedef struct sdcp_logit_controls {
  float repetition;       /* > 0 and finite; 1 = none: a seen token's positive logit is divided
                             by it, any other multiplied */
  float frequency;        /* finite; taken off a logit times the token's number of outputs */
  float presence;         /* finite; taken off once for a token with at least one output */
  uint32_t history_len;   /* tokens of the session's history row: prompt, then outputs */
  uint32_t prompt_len;    /* the first prompt_len of them are the prompt */
  uint32_t bias_offset;   /* its biases are entries bias_offset .. bias_offset + bias_count - 1 */
  uint32_t bias_count;    /*   of bias_tokens / bias_values, token ids strictly rising */
  uint32_t reserved;
} sdcp_logit_controls;

/*
 * Penalties for repeated tokens, biases and grammar masks on the target or the draft rows of
 * a ragged batch, before sdcp_verify_batch reads them.  For token t of row i of session b, with
 *   c = the number of t among the session's outputs (history[prompt_len .. history_len)) and
 *       its drafts x[0 .. i-1],
 *   seen = t is in the prompt, or c > 0,
 * the logit l becomes, in binary32 arithmetic and in this order,
 *   seen:  l = l > 0 ? l / repetition : l * repetition;
 *   l = l - frequency * c;   c > 0:  l = l - presence;   biased:  l = l + bias(t);
 *   masked:  l = -inf (whatever it was, NaN included)
 * and is rounded once to dtype.  A logit nothing applies to is copied bit for bit.
 *
 * logits        device, [rows][V] of dtype; rows = total_drafts + B (SDCP_ROWS_TARGET) or
 *               total_drafts (SDCP_ROWS_DRAFT).
 * out           device out, [rows][V] of dtype.  May be logits itself (in place: logits that
 *               nothing applies to are then neither read nor written), else must not overlap.
 * m_offsets, total_drafts, draft_tokens   as for sdcp_verify_batch; M_b in 0..SDCP_MAX_M.
 *               draft_tokens may be NULL when total_drafts is 0.
 * controls      device, [B].
 * history       device, [B][history_stride] int32 token ids, the prompt first; may be NULL when
 *               history_stride is 0.  Ids outside [0, V), here and among the drafts, count for
 *               nothing.
 * bias_tokens, bias_values   device, [n_bias] int32 / float; NULL when n_bias is 0.
 * masks         device, [n_masks][mask_stride] uint32, mask_stride >= ceil(V / 32): bit t % 32 of
 *               word t / 32 set = token t may be chosen.  NULL when n_masks is 0.
 * mask_rows     device, [rows] int32: the mask of each row, -1 = none.  NULL: no row has one.
 * status        device out, [B] int32: SDCP_S_OK; SDCP_S_LIMIT (M_b above SDCP_MAX_M);
 *               SDCP_S_BAD_PARAMS (controls out of range, history_len above history_stride,
 *               prompt_len above history_len, biases out of the arrays' range or not strictly
 *               rising ids of [0, V), a mask index outside -1 .. n_masks - 1, or inconsistent
 *               offsets: its own pair out of range, or any of the batch's out of order, which
 *               refuses every session).  The rows of such a session are filled with NaN, so that
 *               sdcp_verify_batch commits nothing for it (with inconsistent offsets no row is
 *               known to be the session's own, and none is written).
 * A row whose mask leaves no token holds only -inf; sdcp_verify_batch reports it as
 * SDCP_S_BAD_PARAMS.  No workspace; deterministic.  Returns SDCP_OK or SDCP_E_*.
 */
int sdcp_adjust_logits(const void* logits, void* out, int dtype, int64_t V, int32_t B, int rows,
                       const int32_t* m_offsets, int64_t total_drafts, const int32_t* draft_tokens,
                       const sdcp_logit_controls* controls, const int32_t* history,
                       int64_t history_stride, const int32_t* bias_tokens, const float* bias_values,
                       int64_t n_bias, const uint32_t* masks, int64_t mask_stride, int64_t n_masks,
                       const int32_t* mask_rows, int32_t* status, void* stream);

/* ---- scoring a round: a paged cache of keys and values in 4 bits ------------------ */
/*
 * A session's keys and values live in pages of page_tokens tokens; token t of session b is slot
 * t % page_tokens of page page_table[b][t / page_tokens].  One array holds all pages:
 *   pages[n_pages][kv_heads][2][block]   (uint8; 0 = keys, 1 = values)
 * and a block, of P = page_tokens tokens and D = head_dim channels, is
 *   codes  [D / 32][P][16 bytes]  then  scales [P][D / 32 bytes],
 * so block = P (D / 2 + D / 32) bytes: 4.25 bits a channel.  The 16 bytes of a group of 32
 * channels are four little-endian 32-bit words of 8 channels; channel e of a word is the four
 * bits from 4 (e / 2 + 4 (e % 2)), holding n + 8 with n in -7..7.  A scale byte 8 e + m in
 * 8..167 is s = (1 + m / 8) 2^(e - 15); the channel's value is n s (exact in bfloat16).
 * Quantisation: s is the smallest scale >= (the group's largest magnitude) / 7 (the nearest end
 * of the range where there is none: magnitudes above 420 saturate), n = x / s rounded to nearest
 * even, clamped to -7..7; a NaN becomes 0.
 */
typedef struct sdcp_kv_cache {   /* host struct */
  uint32_t struct_size;          /* sizeof(sdcp_kv_cache) */
  int32_t n_pages;
  int32_t page_tokens;           /* a power of two, 16..1024 */
  int32_t kv_heads;              /* 1..256 */
  int32_t head_dim;              /* 64 or 128 */
  int32_t max_pages;             /* row length of page_table */
  const int32_t* page_table;     /* device, [B][max_pages]; entries past a session's last token
                                    are not read */
  uint8_t* pages;                /* device, 16-byte aligned, n_pages * sdcp_kv_page_bytes bytes */
} sdcp_kv_cache;

/* Bytes of one page (all heads, keys and values); 0 for a geometry that is not supported. */
size_t sdcp_kv_page_bytes(int32_t page_tokens, int32_t kv_heads, int32_t head_dim);

#define SDCP_ROTARY_HALF        0  /* channel j turns with channel j + rot_dim / 2 */
#define SDCP_ROTARY_INTERLEAVED 1  /* channel 2 j turns with channel 2 j + 1 */

/* The position rotation: the first rot_dim channels of a head turn, the others stay.  Pair j at
 * position t becomes (x1 cos - x2 sin, x2 cos + x1 sin), each product and sum rounded to binary32;
 * the table carries the base, its scaling for long contexts and any factor on cos and sin. */
typedef struct sdcp_rotary {     /* host struct */
  uint32_t struct_size;          /* sizeof(sdcp_rotary) */
  int32_t layout;                /* SDCP_ROTARY_* */
  int32_t rot_dim;               /* even, 2..head_dim */
  int32_t n_positions;           /* rows of the table */
  const float* table;            /* device, [n_positions][rot_dim]: rot_dim / 2 cosines, then sines */
} sdcp_rotary;

/*
 * Appends the keys and values of one round to the cache, turned by their positions on the way,
 * and turns the queries with them.  The round of session b is its M_b + 1 target rows
 * (m_offsets[b] + b + i); row i is the token at position kv_len[b] + i.  M_b = 0 is a single
 * token, and M_b has no upper limit here (a prompt is one long round).  After the verdict the
 * caller adds n_out[b] to kv_len[b]; what was rejected is overwritten by the next round.
 *
 * cache         the cache (host struct); sessions of one batch share no page they write to.
 * m_offsets, total_drafts   as for sdcp_verify_batch.
 * kv_len        device, [B] int32: tokens cached before the round.
 * k, v          device, [total_drafts + B] rows of kv_heads * head_dim elements of dtype, rows
 *               k_stride / v_stride elements apart; q (or NULL) likewise with q_heads heads.
 *               16-byte aligned, strides a multiple of 16 bytes.
 * rotary        host struct, or NULL: no rotation.
 * q_out         device out, [total_drafts + B][q_heads][head_dim] of dtype, contiguous, 16-byte
 *               aligned; NULL exactly when q is.  Must not overlap q.
 * status        device out, [B] int32: SDCP_S_OK; SDCP_S_LIMIT (a position past the page table's
 *               row or the rotary table); SDCP_S_BAD_PARAMS (a negative kv_len, a page outside
 *               [0, n_pages) or inconsistent offsets, as for sdcp_adjust_logits).  A session
 *               that is not SDCP_S_OK writes nothing to the cache; its rows of q_out are
 *               unspecified.
 * A refusal is this call's alone: sdcp_attend_kv knows no rotary table and would attend what the
 * cache held before.  Keep the calls' statuses apart and give sdcp_commit_batch, for each
 * session, one that is not SDCP_S_OK where any call's is not (the largest will do); n_out of such
 * a session is not added to kv_len.
 */
int sdcp_append_kv(const sdcp_kv_cache* cache, int32_t B, const int32_t* m_offsets,
                   int64_t total_drafts, const int32_t* kv_len, int dtype, const void* k,
                   int64_t k_stride, const void* v, int64_t v_stride, const sdcp_rotary* rotary,
                   const void* q, int64_t q_stride, int32_t q_heads, void* q_out, int32_t* status,
                   void* stream);

/*
 * Stretches of cached tokens as values (a session that moves to another verifier, a check of a
 * cache): tokens start[b] .. start[b] + n_b - 1 of session b, n_b = offsets[b+1] - offsets[b],
 * become rows offsets[b] .. of k_out and v_out, [n_tokens][kv_heads][head_dim] of dtype (either
 * may be NULL), 16-byte aligned.  offsets is device, [B+1] int32, offsets[0] = 0, non-decreasing,
 * offsets[B] = n_tokens (given by the host as well); start is device, [B] int32.  status as for
 * sdcp_append_kv; the rows of a session that is not SDCP_S_OK are zero.
 */
int sdcp_read_kv(const sdcp_kv_cache* cache, int32_t B, const int32_t* offsets, int64_t n_tokens,
                 const int32_t* start, int dtype, void* k_out, void* v_out, int32_t* status,
                 void* stream);

/* ---- the pages between rounds: fork, reserve, copy, release, compact --------------- */
/*
 * A pool keeps who holds which page, in three device arrays that these calls alone change: slot b (a
 * session, or a place for one) has row b of page_table, whose first held[b] entries are pages; refs[p]
 * is the number of rows that hold page p, 0 for a free one, never negative.  An empty pool is held = 0,
 * refs = 0.  Rows may share pages (sdcp_fork_kv); a page is written only while one row holds it
 * (sdcp_reserve_kv).  The arrays serve all layers of a model: each layer's cache has the same n_pages and
 * page_tokens, its batch rows are rows of page_table, and only sdcp_copy_pages, the bytes themselves, runs
 * once for each.
 *
 * The calls work on all slots at once; arrays of one entry a slot say what is to happen to it.  No call
 * reads a number back: counts stay on the device (n_copies), and a slot whose request is refused is left
 * as it was.  A round of a program that branches:
 *   sdcp_fork_kv (new continuations), sdcp_reserve_kv (room for the round), for each layer
 *   sdcp_copy_pages and the layer itself, the verdict, sdcp_release_kv (what was rejected or has ended).
 * All are deterministic and asynchronous on `stream`; free pages are taken lowest first.  Calls on one
 * pool must not overlap, nor calls with one workspace.
 */
typedef struct sdcp_kv_pool {    /* host struct */
  uint32_t struct_size;          /* sizeof(sdcp_kv_pool) */
  int32_t n_pages;               /* 1..2^30 */
  int32_t page_tokens;           /* a power of two, 16..1024 */
  int32_t n_slots;               /* rows of page_table, 0..2^30 */
  int32_t max_pages;             /* entries of a row; max_pages * page_tokens below 2^31 */
  int32_t* page_table;           /* device, [n_slots][max_pages] */
  int32_t* held;                 /* device, [n_slots] */
  int32_t* refs;                 /* device, [n_pages] */
} sdcp_kv_pool;

/* One page to copy, 16 bytes, device memory: the first `tokens` tokens of every head's keys and values. */
typedef struct sdcp_page_copy {
  int32_t from, to;
  int32_t tokens;                /* 0..page_tokens */
  int32_t reserved;
} sdcp_page_copy;

/*
 * Forks sessions: slot b with parent[b] = a takes the pages of a's first length[b] tokens as its own,
 * shared with a (no page is taken, no byte copied: a page that either will write is replaced by
 * sdcp_reserve_kv).
 *
 * parent        device, [n_slots] int32: a slot, or -1: b is not forked.
 * length        device, [n_slots] int32: tokens, looked at where parent[b] is not -1.
 * status        device out, [n_slots] int32: SDCP_S_OK; SDCP_S_LIMIT (length beyond the parent's pages);
 *               SDCP_S_BAD_PARAMS (parent outside the slots, b itself or forked in this call too, b holds
 *               pages, a negative length, a row that is not in order: held[] outside 0..max_pages or an
 *               entry outside the pool).
 */
int sdcp_fork_kv(const sdcp_kv_pool* pool, const int32_t* parent, const int32_t* length, int32_t* status,
                 void* stream);

/* Bytes of device workspace sdcp_reserve_kv and sdcp_compact_kv need; 0 for invalid sizes. */
size_t sdcp_pool_workspace_bytes(int32_t n_pages, int32_t n_slots);

/*
 * Pages for what slots are to write: positions kv_len[b] .. upto[b] - 1 (upto[b] <= kv_len[b]: nothing).
 * Of the entries that these positions lie in, those past held[b] get new pages, and those whose page
 * other rows hold too get a new page in its stead (copy on write); where the first of them already holds
 * tokens (kv_len[b] is inside a page), they are to be copied.  New pages are the lowest free ones (free
 * when the call began), in the order of the slots and of their entries.  If all holders of a shared page
 * write it in one call, each gets a page and the shared one becomes free.
 *
 * kv_len, upto  device, [n_slots] int32.
 * copies        device out, [max_copies], 16-byte aligned, max_copies >= n_slots: the copies to make
 *               before the round (sdcp_copy_pages), at most one a slot, in the order of the slots.
 * n_copies      device out, [1] int32.
 * status        device out, [n_slots] int32: SDCP_S_OK; SDCP_S_LIMIT (the row has no entry for upto[b], or
 *               too few pages are free: more than there are, counted over the needs of the slots up to and
 *               with b); SDCP_S_BAD_PARAMS (kv_len[b] is negative or beyond the pages held, held[b] is
 *               outside 0..max_pages, or one of these entries is outside the pool).
 * workspace     device scratch of sdcp_pool_workspace_bytes bytes, 256-byte aligned, no initialisation
 *               needed.
 * A refused session may still hold shared pages where it was to write: keep it out of sdcp_append_kv (a
 * kv_len of -1 there refuses it and writes nothing).
 */
int sdcp_reserve_kv(const sdcp_kv_pool* pool, const int32_t* kv_len, const int32_t* upto,
                    sdcp_page_copy* copies, int32_t max_copies, int32_t* n_copies, int32_t* status,
                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * Executes a list of page copies on one cache (of one layer).  The destination's other tokens stay as they
 * are.  cache->page_table and max_pages are not looked at.
 *
 * copies        device, [max_copies], 16-byte aligned; n_copies is device, [1] int32, the number of them
 *               that are there.  No page may be the destination of two copies, or the source of one and
 *               the destination of another (the lists of sdcp_reserve_kv and sdcp_compact_kv are so).
 * status        device out, [1] int32: SDCP_S_OK, or SDCP_S_BAD_PARAMS: a record is not usable (a page
 *               outside [0, n_pages), from equal to to, tokens outside 0..page_tokens) and was left out, or
 *               n_copies is outside 0..max_copies and nothing was copied.
 */
int sdcp_copy_pages(const sdcp_kv_cache* cache, const sdcp_page_copy* copies, int32_t max_copies,
                    const int32_t* n_copies, int32_t* status, void* stream);

/*
 * Gives pages back: slot b keeps the pages of its first keep[b] tokens (keep[b] < 0: all of them, 0: none;
 * beyond what it holds: all), the entries past them become -1, and a page that no row holds any more is
 * free.  Usual values: the committed length after a verdict, and 0 for a session that has ended.
 *
 * keep          device, [n_slots] int32.
 * status        device out, [n_slots] int32: SDCP_S_OK; SDCP_S_BAD_PARAMS (a row that is not in order, as
 *               for sdcp_fork_kv).
 */
int sdcp_release_kv(const sdcp_kv_pool* pool, const int32_t* keep, int32_t* status, void* stream);

/*
 * Moves live pages to the front of the pool, so that its end can be given to something else: of L live
 * pages, the k-th highest of those at or past L goes to the k-th lowest free page.  Rows and counts are
 * changed by this call; the bytes move with sdcp_copy_pages, of each layer, behind it.
 *
 * copies        device out, [max_copies], 16-byte aligned: the moves, whole pages.  With max_copies below
 *               their number (at most n_pages / 2) the first max_copies are made, highest pages first; call
 *               again for the others.
 * n_copies      device out, [1] int32: the moves made.
 * n_live        device out, [1] int32: L.
 * workspace     as for sdcp_reserve_kv.
 * Entries outside the pool, and those that name a free page, stay as they are; rows are looked at up to held[b]
 * (at most max_pages) entries.
 */
int sdcp_compact_kv(const sdcp_kv_pool* pool, sdcp_page_copy* copies, int32_t max_copies,
                    int32_t* n_copies, int32_t* n_live, void* workspace, size_t workspace_bytes,
                    void* stream);

/* Bytes of device workspace sdcp_attend_kv needs; 0 for invalid sizes.  What suffices for a batch does
 * for any with no more sessions and no more drafts (and the same heads). */
size_t sdcp_attend_workspace_bytes(int32_t B, int64_t total_drafts, int32_t q_heads,
                                   int32_t kv_heads, int32_t head_dim);

/*
 * Attention of one round's rows over the cache.  Row i of session b attends the positions
 *   max(0, kv_len[b] + i + 1 - window) .. kv_len[b] + i      (window 0: from 0)
 * so each row sees the cached context, the round's earlier rows and itself (sdcp_append_kv has
 * put them there).  Query head h reads cached head h / (q_heads / kv_heads):
 *   out[row][h] = sum_t softmax_t(scale * q[row][h] . key_t) value_t.
 * Scores, the softmax's statistics and the sums are binary32.  A weight is rounded to binary16
 * for the product with the values (11 significant bits down to 2^-21 of the row's largest weight,
 * a spacing of 2^-31 of it below), and the sum is of the weights so rounded; exponentials and the last division are the
 * hardware's approximate ones (2 units in the last place); out is rounded once.
 *
 * q             device, [total_drafts + B] rows of q_heads * head_dim bfloat16, q_stride elements
 *               apart (16-byte aligned, stride a multiple of 8); q_heads a multiple of kv_heads.
 * scale         finite; usually 1 / sqrt(head_dim).
 * window        0 = none, else the number of positions a row sees, itself included.
 * out           device out, [total_drafts + B][q_heads][head_dim] bfloat16, contiguous, 16-byte
 *               aligned.  Must not overlap q.
 * status        device out, [B] int32, as for sdcp_append_kv (only the pages a row attends are
 *               looked at; there is no rotary table's limit here); the rows of a session that
 *               is not SDCP_S_OK are zero, which a model turns into ordinary logits: see
 *               sdcp_append_kv on what to do with a refusal.
 * workspace     device scratch of sdcp_attend_workspace_bytes bytes, 256-byte aligned, no
 *               initialisation needed.
 * M_b has no upper limit here.  A query row holding NaN or infinities gives NaN in its own
 * output row alone.  Deterministic.  SDCP_S_INTERNAL for every session: the call gave up a
 * bounded wait on the GPU, and no output of it is valid.
 */
int sdcp_attend_kv(const sdcp_kv_cache* cache, int32_t B, const int32_t* m_offsets,
                   int64_t total_drafts, const int32_t* kv_len, const void* q, int64_t q_stride,
                   int32_t q_heads, float scale, int32_t window, void* out, int32_t* status,
                   void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace sdcp_attend_shared_kv needs (n_groups 0: as 1); 0 for invalid sizes.  What
 * suffices for a batch does for any with no more sessions, drafts and groups (and the same heads).  Four
 * times the bytes of out (two sums in binary32 for each row and head, whether or not anything is shared),
 * 16 bytes for each row and head, some 60 for each session and group, and 43 MB (22 MB for 64 channels). */
size_t sdcp_attend_shared_workspace_bytes(int32_t B, int64_t total_drafts, int32_t n_groups,
                                          int32_t q_heads, int32_t kv_heads, int32_t head_dim);

/*
 * sdcp_attend_kv without a window, for a batch in which sessions have their first pages in common (a
 * system prompt, branches of one session: sdcp_fork_kv).  The sessions of a group are neighbours in the
 * batch, and the call finds what they share from the page table: the leading entries on which all rows of
 * the group agree, as far as every one of them has cached whole pages.  These pages are read and turned
 * once for the group's rows together; the rest of each session for its own rows.  Where that would save
 * less than joining the two costs (few sessions, short stretches), the group's sessions are attended by
 * themselves, as this call does it.  What a group is only decides how the sum is cut: the output is sdcp_attend_kv's up to rounding
 * for any grouping.  (A batch that shares little is faster with sdcp_attend_kv: eight sessions of a row each
 * gain from about 2000 shared tokens on, two from about 10000.)
 *
 * group_offsets device, [n_groups + 1] int32: group g is sessions group_offsets[g] ..
 *               group_offsets[g+1] - 1; from 0, non-decreasing, to B.  NULL with n_groups 0: all sessions
 *               are one group.
 * workspace     device scratch of sdcp_attend_shared_workspace_bytes bytes, 256-byte aligned, no
 *               initialisation needed; calls that may run at once (streams, graphs) need one each.
 * Everything else, the arithmetic and the statuses among it, as for sdcp_attend_kv; group offsets that are
 * not in order refuse every session with SDCP_S_BAD_PARAMS, and a session that is refused leaves its
 * group.  (total_drafts + B) * q_heads is below 2^31, and n_groups + B at most 2^30.  A row's sum of
 * weights is of the weights before their rounding to binary16.
 */
int sdcp_attend_shared_kv(const sdcp_kv_cache* cache, int32_t B, const int32_t* m_offsets,
                          int64_t total_drafts, const int32_t* kv_len, int32_t n_groups,
                          const int32_t* group_offsets, const void* q, int64_t q_stride,
                          int32_t q_heads, float scale, void* out, int32_t* status, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * Host-side split of one ragged batch into n_parts contiguous blocks of sessions for
 * n_parts GPUs (one process per GPU).  Sessions are independent (Section 6.3 "Scoring":
 * a verifier may batch the proposals of many sessions), so block k can be verified on its
 * own GPU, and concatenating the blocks' outputs in order gives the whole batch's outputs:
 * no collective is needed on the data path.
 *
 * m_offsets  host, [B+1] int32 (as for sdcp_verify_batch).
 * params     host, [B] sdcp_session_params, or NULL (every session counted as Rule 2).
 * bounds     host out, [n_parts+1] int32: block k holds sessions bounds[k] .. bounds[k+1]-1;
 *            bounds[0] = 0, bounds[n_parts] = B, non-decreasing.
 * The blocks are balanced by the rows each session makes the first phase read: M_b + 1
 * target rows, plus M_b draft rows under Rule 2.  Boundary k is the first session index
 * (not before boundary k-1) whose prefix of rows comes closest to k/n_parts of the total;
 * the split is a pure function of its inputs.
 * Returns SDCP_OK, or SDCP_E_INVALID for null pointers, B < 0, n_parts < 1 or offsets that
 * are not non-decreasing from 0.  Touches no device.
 */
int sdcp_split_sessions(const int32_t* m_offsets, const sdcp_session_params* params, int32_t B,
                        int32_t n_parts, int32_t* bounds);

/* Human-readable text for an SDCP_E_* code (static storage, never NULL). */
const char* sdcp_strerror(int code);

/* ABI version of this header; bumps on any incompatible change. */
#define SDCP_ABI_VERSION 2
int sdcp_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SDCP_H */
