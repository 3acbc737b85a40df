/* specverify.h - C ABI of the MI355X (gfx950) speculative-sampling verification library.
 *
 * The library computes, on one GPU, the data-parallel hot path of lossless speculative sampling
 * and of Saguaro's outcome cache:
 *
 *   spec_verify          - per request: temperature / top-k / nucleus processing of draft and
 *                          target rows, optional Saguaro downweight sigma_{F,C} of the draft, the
 *                          min(1, q/p) acceptance scan with first-rejection cutoff, and the
 *                          correction token from the normalised residual (q - p)+ (or the bonus
 *                          token from the target's extra position when every draft token is
 *                          accepted).  Outputs the verification outcome (k, t*).
 *   saguaro_downweight   - sigma_{F,C} of the processed draft rows (the downweighted set, its
 *                          normaliser and, optionally, the full distribution).
 *   saguaro_cache_build  - the geometric fan-out F_k (Theorem 12) and, per verify depth k, the
 *                          F_k guessed outcome tokens.
 *   saguaro_cache_lookup - hit / miss of the verified outcome (k, t*) against the cache, or the
 *                          branch-reuse test of a branch-complete tree.
 *   saguaro_verify_cache - spec_verify and saguaro_cache_build fused: one pass over the draft
 *                          rows serves both (the cache's token sets are the leading tokens of
 *                          the same rows the verification reads).
 *   saguaro_backup_plan  - the batch-aware fallback on a cache miss: which requests take the
 *                          random-token backup speculator this round (verified by spec_verify
 *                          with SPEC_UNIFORM_DRAFT).
 *   mirror_signposts     - Mirror-SD early-exit signposts: the kappa most likely tokens of a
 *                          logit row with their log-probabilities (the draft's token-channel
 *                          message).
 *   mirror_tree_lookup   - reuse of the committed prefix against a draft tree that may branch
 *                          below its roots.
 *   pyramid_verify       - PyramidSD fuzzy acceptance (lossy, behind its own entry point):
 *                          spec_verify where a position whose distributions are within a
 *                          divergence threshold keeps its drafted token outright.
 *   spec_verify_probs    - the verification for callers that hold processed probabilities and
 *                          draw their own random numbers.
 *
 * and the model-side steps of a round that scores drafted tokens, guessed outcomes and tree
 * branches on top of one shared context:
 *
 *   spec_tree_rows        - the rows of draft trees: each node's position and the cache slots of
 *                           the nodes above it.
 *   spec_rope_frequencies - host helper: rotary inverse frequencies, scaled for long contexts.
 *   spec_kv_append        - rotary positions for queries and keys, and the append of the keys and
 *                           values to a paged cache.
 *   spec_prefix_attention - attention of rows that share a long prefix of the paged cache and see
 *                           tokens of their own behind it.
 *
 * Sources (notation p = draft, q = target, as on the DeepMind page):
 *   [SpS]   "Accelerating LLM Decoding with Speculative Sampling" (DeepMind, arXiv 2302.01318),
 *           knowledge-base reading, sections 1, 3 and 6.
 *   [SSD]   "Speculative Speculative Decoding" reading notes, sections 1.3, 2.2, 4.3, 4.4, 5.1, 7.1.
 *   [SSD-H] hyper.ai summary of arXiv 2603.03251, "Method" (fan-out closed form, sigma_{F,C}).
 *   [MSD]   "Mirror Speculative Decoding" reading notes, sections 2, 3.1, 3.2 and 3.3.
 *   [PSD]   "3-Model Speculative Decoding (PyramidSD)" notes, method, key designs 1 and 2.
 *
 * Conventions for every entry point:
 *   - Array pointers are HIP device memory owned by the caller (unless marked "host"); the
 *     library never allocates, frees or retains them, and keeps no state between calls.
 *   - Every call is asynchronous on `stream` (0 = the default stream); outputs are valid once
 *     the stream has reached them.  Calls on different streams with disjoint outputs and
 *     workspaces may run concurrently.
 *   - Host-detectable argument errors return a negative SPEC_E* code and launch nothing.
 *     Data-dependent conditions are reported per request in status bits (a kernel cannot
 *     return an error code).
 *   - Logits are row-major and contiguous with the vocabulary fastest: draft [B][Kd][V],
 *     target [B][K+1][V]; element type SPEC_FP32 (float) or SPEC_BF16 (bfloat16 bits).
 *   - Token order used by every selection (top-k, nucleus, the downweighted set, cache ranks,
 *     greedy argmax): logit descending, then token id ascending on equal logits.
 */
#ifndef SPECVERIFY_H
#define SPECVERIFY_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* return codes */
enum {
    SPEC_OK = 0,
    SPEC_EINVAL = -1,      /* null pointer, size < 1, F outside [0, SPEC_MAX_F], C outside [0, 1], ... */
    SPEC_EDTYPE = -2,      /* dtype is none of those the entry point takes */
    SPEC_EWORKSPACE = -3,  /* workspace null or smaller than its ..._workspace_bytes() */
    SPEC_EHIP = -4         /* a kernel launch failed (hipGetLastError after the launch) */
};

/* Element types.  The logit entry points take SPEC_FP32 and SPEC_BF16; the others say theirs.
 * SPEC_E4M3: 8-bit floats of 4 exponent and 3 mantissa bits with no infinities (OCP e4m3fn). */
enum { SPEC_FP32 = 0, SPEC_BF16 = 1, SPEC_FP16 = 2, SPEC_E4M3 = 3, SPEC_FP64 = 4 };

#define SPEC_MAX_F 64          /* largest downweighted set */
#define SPEC_MAX_FANOUT 1024   /* largest cache width for one depth */
#define SPEC_MAX_KAPPA 16      /* most signposts per request */
#define SPEC_NOALLOC_SCRATCH_BYTES (32u << 20)  /* static scratch of saguaro_verify_cache_noalloc, per GPU */

/* Per-request processing, applied to the draft AND the target rows of that request ([SpS]
 * section 6: temperature, top-k and nucleus act on both distributions before the correction).
 * Order: temperature, then top-k, then softmax, then nucleus.
 *   temperature  > 0, or 0 for greedy verification (argmax match, [MSD] section 2)
 *   top_k        <= 0 or >= V: off; else keep exactly top_k tokens (ties by lower id)
 *   top_p        in (0, 1): keep the smallest prefix of the token order whose mass reaches
 *                top_p; >= 1: off.  temperature < 0, NaN or top_p <= 0 sets SPEC_ST_BAD_PARAM. */
typedef struct {
    float temperature;
    int32_t top_k;
    float top_p;
} spec_params;

/* flags for spec_verify (and pyramid_verify) */
enum {
    SPEC_SAMPLE_DRAFT = 1, /* draft_tokens is an output: s_j is drawn from the processed (and
                              downweighted) draft row j by inverse CDF in token-id order with
                              Philox lane 2, or is the draft argmax when temperature is 0 */
    SPEC_UNIFORM_DRAFT = 2,/* the draft distribution of every position is uniform on [0, V):
                              the random-token backup speculator ([SSD] section 7.1).  No draft
                              row is read (draft_logits may be NULL), F and C do not apply, and
                              temperature, top-k and top-p act on the target rows only; with
                              SPEC_SAMPLE_DRAFT, s_j = floor(u V) for the Philox lane-2 uniform u
                              (the inverse CDF of the uniform law, taken exactly) */
    SPEC_ASSISTED = 4,     /* pyramid_verify only: a rejected position draws its correction from
                              the verifier's processed distribution q_j itself, not from the
                              residual ([PSD] key design 2, the assisted variant) */
    SPEC_POINT_DRAFT = 8   /* spec_verify_probs only: every drafted token had probability 1 (a
                              drafter that looks tokens up or takes its argmax) */
};

/* per-request status bits (out_status) */
enum {
    SPEC_ST_EMPTY_RESIDUAL = 8,            /* rejection with no residual mass: t* drawn from q_k */
    SPEC_ST_OUTSIDE_DRAFT_SUPPORT = 16,    /* an evaluated draft token has p'(s) = 0; it is
                                              accepted iff q(s) > 0 */
    SPEC_ST_BAD_LOGIT = 32,                /* NaN / +inf logit, or a row with no finite logit:
                                              k = 0, t* = -1 */
    SPEC_ST_BAD_TOKEN = 64,                /* a draft token outside [0, V): k = 0, t* = -1 */
    SPEC_ST_DEGENERATE_DOWNWEIGHT = 128,   /* C = 0 and the set holds all the draft mass: the
                                              row is left undownweighted */
    SPEC_ST_BAD_PARAM = 256,               /* invalid spec_params: k = 0, t* = -1 */
    SPEC_ST_PLACEMENT = 512,               /* the exact-count path found the workgroups of one
                                              position on different XCDs (its slices meet in one
                                              XCD's L2): the request was redone by the general
                                              path.  Never expected; a guard on the launch map */
    SPEC_ST_BAD_PROB = 1024,               /* spec_verify_probs: a negative, infinite or NaN
                                              probability where one was read, or a target row
                                              without mass: k = 0, t* = -1 */
    SPEC_ST_BAD_SLOT = 2048                /* spec_kv_append: a slot past the cache (nothing of
                                              that token was stored) */
};

/* Uniforms.  Counter-based Philox4x64-10 (Salmon et al., SC'11) with key (seed, 0) and counter
 * (round, b, j, 0) gives the block of request b and position j = 0..K; word w of the block
 * becomes the uniform ((w >> 12) + 0.5) * 2^-52 in (0, 1).  Word 0: acceptance u_j; word 1:
 * residual / bonus v_j; word 2: draft sampling (SPEC_SAMPLE_DRAFT). */

/* Bytes of scratch spec_verify needs for B requests of K draft positions over V tokens (pure
 * host function).  The workspace must be zero-filled before its first use; every call that
 * completes leaves its arrival counters at zero again, so it can be reused without clearing
 * for the same (B, K, V); the counters' places depend on the shape, so a workspace taken over
 * for another shape is zero-filled again first.  It carries no results between calls.  One
 * workspace serves one call at a time. */
size_t spec_workspace_bytes(int B, int K, int V);

/* spec_verify - batched speculative-sampling verification ([SpS] sections 1 and 3; [SSD]
 * section 2.2; outcome (k, t*) as in [SSD] section 1.3).
 *
 * For each request b, with p_j the processed draft row j after sigma_{F,C} (F > 0 and C < 1;
 * [SSD-H] Method, [SSD] section 4.4) and q_j the processed target row j:
 *   for j = 0..K-1: accept s_j iff u_j * p_j(s_j) < q_j(s_j); stop at the first rejection.
 *   k = number of accepted tokens.  k < K: t* ~ (q_k - p_k)+ / sum (q_k - p_k)+ with v_k;
 *   k = K: t* ~ q_K with v_K.  Sampling is the inverse CDF in token-id order: the first token
 *   whose running mass exceeds v times the total.  Greedy requests (temperature 0) accept s_j
 *   iff it is the argmax of q_j and take t* = argmax q_k.
 *
 *   draft_logits    [B][draft_rows][V]; draft_rows = K or K+1 (row K, used by the cache, is
 *                   ignored here); not read with SPEC_UNIFORM_DRAFT
 *   target_logits   [B][K+1][V]
 *   params          [B] spec_params (device)
 *   F, C            downweighted set size (0 = off) and factor in [0, 1] (1 = off)
 *   draft_tokens    [B][K] int32: read, or written when flags has SPEC_SAMPLE_DRAFT
 *   seed, round     Philox key and first counter word
 *   out_k           [B] int32 in [0, K]
 *   out_tstar       [B] int32 correction / bonus token, -1 for bad requests
 *   out_resid_mass  [B] float: sum (q_k - p_k)+ when k < K, else 0 (nullable)
 *   out_status      [B] uint32 status bits (nullable)
 *   workspace       >= spec_workspace_bytes(B, K, V) bytes of device memory
 * Paths: bf16 logits with V % 8 == 0, 2048 <= V <= 262144, 16-byte aligned rows and K <= 63
 * take the exact-count path (two launches); every other shape takes the general path (one
 * workgroup per position).  Both give the same outputs.
 * Returns SPEC_OK or a negative SPEC_E* code. */
int spec_verify(const void* draft_logits, int draft_rows, const void* target_logits, int dtype, int B, int K,
                int V, const spec_params* params, int F, float C, int32_t* draft_tokens, uint64_t seed,
                uint64_t round, uint32_t flags, int32_t* out_k, int32_t* out_tstar, float* out_resid_mass,
                uint32_t* out_status, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* saguaro_downweight - Saguaro sampling sigma_{F,C} ([SSD-H] Method; [SSD] section 4.4 with the
 * Theorem 19 example): on each processed draft row j < K the first F tokens of the token order
 * that carry mass form the set S; with P_S their mass, Z = 1 - (1 - C) P_S and
 * p'_i = p_i C / Z on S, p_i / Z elsewhere.
 *   out_ids    [B][K][F] int32, S in rank order, -1 past its end
 *   out_Z      [B][K] float (nullable)
 *   out_probs  [B][K][V] float, the full p' (nullable; for tests)
 *   out_status [B][K] uint32 (nullable): SPEC_ST_BAD_LOGIT / _BAD_PARAM / _DEGENERATE_DOWNWEIGHT */
int saguaro_downweight(const void* draft_logits, int draft_rows, int dtype, int B, int K, int V,
                       const spec_params* params, int F, float C, int32_t* out_ids, float* out_Z, float* out_probs,
                       uint32_t* out_status, hipStream_t stream);

/* Host helper: the Theorem 12 fan-out ([SSD] section 4.3; [SSD-H] Method).  Real values
 * F_k = F0 a^{k/(1+r)} (k < K) and F_K = F0 a^{K/(1+r)} (1 - a)^{-1/(1+r)} with F0 such that
 * they sum to `budget`; integers by largest remainder (ties to the smaller k) so that they
 * sum to the budget exactly.  a in (0, 1), r > -1.  out_fanout [K+1] host. */
int saguaro_fanout(int K, int budget, double a, double r, int32_t* out_fanout);

/* saguaro_cache_build - the outcome cache's token sets ([SSD] section 5.1; [SSD-H] Method).
 * For depth k < K: the first F_k tokens of draft row k in token order other than the drafted
 * token s_k; for depth K: the first F_K tokens of draft row K.  NaN logits rank last.
 *   draft_logits     [B][K+1][V]
 *   draft_tokens     [B][K]
 *   out_fanout_host  [K+1] host, the fan-out used (nullable)
 *   out_cache        [B][budget] int32, depth-major, rank order, -1 past a row's end */
int saguaro_cache_build(const void* draft_logits, int dtype, int B, int K, int V, const int32_t* draft_tokens,
                        int budget, double a, double r, int32_t* out_fanout_host, int32_t* out_cache,
                        hipStream_t stream);

/* saguaro_verify_cache - spec_verify followed by saguaro_cache_build on the same inputs, in
 * one pass over the logits ([SSD] sections 4.3 and 5.1: the cache is built from the draft
 * distributions the verification reads).  Outputs are exactly those of
 *   spec_verify(draft_logits, K + 1, target_logits, dtype, B, K, V, params, F, C, draft_tokens,
 *               seed, round, flags, out_k, out_tstar, out_resid_mass, out_status, workspace, ...)
 *   saguaro_cache_build(draft_logits, dtype, B, K, V, draft_tokens, budget, a, r,
 *                       out_fanout_host, out_cache, stream)
 * (with SPEC_SAMPLE_DRAFT the cache leaves out the drafted tokens this call samples).
 *   draft_logits  [B][K+1][V] (draft row K feeds the cache only)
 *   workspace     spec_workspace_bytes(B, K, V) bytes, same contract as spec_verify
 * Return codes: as spec_verify and saguaro_cache_build (SPEC_EINVAL also for a null out_cache
 * or an invalid fan-out). */
int saguaro_verify_cache(const void* draft_logits, const void* target_logits, int dtype, int B, int K, int V,
                         const spec_params* params, int F, float C, int32_t* draft_tokens, uint64_t seed,
                         uint64_t round, uint32_t flags, int budget, double a, double r, int32_t* out_fanout_host,
                         int32_t* out_k, int32_t* out_tstar, float* out_resid_mass, uint32_t* out_status,
                         int32_t* out_cache, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* saguaro_backup_plan - the batch-aware fallback on a cache miss ([SSD] section 7.1; [SSD-H]
 * Method, fallback).  Any miss makes the whole batch wait for the fallback, so from a critical
 * batch size b_star on, the missed requests switch to the fast random-token backup speculator
 * (verified with SPEC_UNIFORM_DRAFT) while requests that hit keep their cached speculation;
 * below b_star the primary drafter serves the misses.  The text does not give b_star's formula,
 * so it is an argument.
 *   hit             [B] uint8, the lookup's per-request hit flags
 *   batch           [2] int32, the lookup's {hit count, all-hit flag}
 *   out_use_backup  [B] int32: 1 where request b takes random tokens this round
 *   out_switch      [1] int32: 1 when the backup serves this round (a miss and B >= b_star)
 * Returns SPEC_EINVAL for a null pointer or B < 1. */
int saguaro_backup_plan(int B, const uint8_t* hit, const int32_t* batch, int b_star, int32_t* out_use_backup,
                        int32_t* out_switch, hipStream_t stream);

/* saguaro_cache_lookup - hit / miss of the verified outcome.
 * mode 0 ([SSD-H] Method: cache lookup; [SSD] section 7.1): cache [B][sum F] from
 *   saguaro_cache_build, fanout_or_shape = the [K+1] fan-out (host), k / tstar [B];
 *   out_slot[b] = offset(k_b) + rank of t*_b in C_{k_b}, or -1 on a miss.
 * mode 1 ([MSD] sections 3.2-3.3, branch-complete tree): cache = branch tokens [B][kappa][gamma],
 *   fanout_or_shape = {kappa, gamma} (host), k / tstar [B][kappa] per chain, chain 0 of each
 *   request being the verified path; out_slot[b] = lowest branch whose first k+1 tokens equal
 *   (accepted tokens, t*), -1 if none, -2 when all gamma tokens were accepted.
 *   out_hit [B] uint8 (slot >= 0); out_batch [2] int32 = {hits, 1 if every request hit}. */
int saguaro_cache_lookup(int mode, const int32_t* cache, const int32_t* fanout_or_shape, int K, int B,
                         const int32_t* k, const int32_t* tstar, int32_t* out_slot, uint8_t* out_hit,
                         int32_t* out_batch, hipStream_t stream);

/* mirror_signpost_workspace_bytes - device workspace mirror_signposts needs for (B, V, kappa);
 * 0 for sizes it rejects.  Same contract as the verification workspace: zero-filled before its
 * first use; every completed call leaves its arrival counters at zero again (the rest is
 * scratch each call writes before reading), so it is reused without clearing; one call at a
 * time per workspace. */
size_t mirror_signpost_workspace_bytes(int B, int V, int kappa);

/* mirror_signposts - early-exit signposts ([MSD] sections 3.1 and 3.3: the LM head at the
 * early-exit layer gives a distribution p~; its top kappa tokens with log p~ form the message to
 * the draft).  p~ is read as the softmax of the given logits at temperature 1; tokens are
 * ranked by logit descending, ties to the lower id (-0 ties +0), and
 * log p~(v) = z_v - m - log sum_i exp(z_i - m), m the row maximum.
 *   logits         [B][V] device, dtype SPEC_FP32 or SPEC_BF16 (V <= 2^19)
 *   kappa          1..SPEC_MAX_KAPPA signposts per request
 *   out_ids        [B][kappa] int32, rank order; -1 past the vocabulary
 *   out_logp       [B][kappa] float32 log p~ (-inf past the vocabulary or for a -inf logit)
 *   out_logp_bf16  [B][kappa] bf16 bits, round-to-nearest-even of out_logp (nullable): the
 *                  message's compact form
 *   out_status     [B] (nullable): SPEC_ST_BAD_LOGIT for a row with a NaN or +inf logit or no
 *                  finite one (its ids are -1 and its log-probabilities NaN), else 0
 *   workspace      mirror_signpost_workspace_bytes(B, V, kappa) bytes
 * Return codes: SPEC_EINVAL (null pointer, sizes out of range), SPEC_EDTYPE, SPEC_EWORKSPACE,
 * SPEC_EHIP. */
int mirror_signposts(const void* logits, int dtype, int B, int V, int kappa, int32_t* out_ids, float* out_logp,
                     uint16_t* out_logp_bf16, uint32_t* out_status, void* workspace, size_t workspace_bytes,
                     hipStream_t stream);

/* mirror_tree_lookup - reuse against a draft tree ([MSD] sections 3.2-3.3: the committed
 * prefix, accepted tokens then the correction, is reused when it is one of the paths the draft
 * precomputed; the worked example forks below a root).  Per request the tree is N nodes listed
 * parents first: tree_tokens[b][n] and tree_parents[b][n] (-1 for a root, i.e. a signpost the
 * draft expanded).  A node with a negative token or a parent outside [-1, n) is not part of the
 * tree, nor is anything below it.
 *   path_tokens  [B][gamma] the verified chain's draft tokens (gamma <= 1024)
 *   k, tstar     [B] accepted count and correction token (spec_verify's outputs for the chain)
 *   out_node     [B] the lowest node whose root path equals (path[0..k-1], t*), so at depth
 *                k + 1; -1 when there is none (or k, t* out of range), -2 when k == gamma
 *   out_hit      [B] uint8 (out_node >= 0)
 *   out_batch    [2] int32 {hits, 1 if every request hit} (nullable)
 * Returns SPEC_EINVAL for a null pointer or sizes out of range. */
int mirror_tree_lookup(const int32_t* tree_tokens, const int32_t* tree_parents, int B, int N, int gamma,
                       const int32_t* path_tokens, const int32_t* k, const int32_t* tstar, int32_t* out_node,
                       uint8_t* out_hit, int32_t* out_batch, hipStream_t stream);

/* pyramid_verify - fuzzy acceptance ([PSD] key design 1: a drafted token passes when
 * Div(P_verifier, P_drafter) <= tau; one call per stage, drafter -> qualifier with tau_Q and
 * qualifier -> target with tau_T).  Div is read as the Jensen-Shannon divergence in bits
 * (in [0, 1]) of the processed verifier row q_j and the processed, downweighted drafter row
 * p'_j.  Where Div_j <= tau[b], s_j is kept outright; elsewhere the lossless test of
 * spec_verify decides and a rejection draws the correction from the residual, or from q_j with
 * SPEC_ASSISTED.  A threshold below every divergence (e.g. a negative one) is exactly
 * spec_verify.  The output distribution is NOT the verifier's: this is a lossy variant.
 * Arguments as spec_verify (verifier_logits in the place of target_logits), plus
 *   tau        [B] float32 device, per-request thresholds
 *   flags      SPEC_SAMPLE_DRAFT | SPEC_UNIFORM_DRAFT | SPEC_ASSISTED
 *   out_div    [B][K] float32 device (nullable): Div_j of every position whose drafted token
 *              is valid, whether or not the scan reached it
 * bf16 rows with V a multiple of 8, 2048 <= V <= 262144 and 16-byte aligned logits, given (or
 * uniform) drafted tokens, no SPEC_ASSISTED and K < 64 take the register-resident path: a
 * divergence pass runs between its count and resolve kernels.  Everything else runs on the
 * general path (one workgroup per position).  Both sum the divergence in fp64; the decision
 * Div_j <= tau[b] is taken on that sum.  Return codes as spec_verify (SPEC_EINVAL also for a
 * null tau). */
int pyramid_verify(const void* draft_logits, int draft_rows, const void* verifier_logits, int dtype, int B, int K,
                   int V, const spec_params* params, int F, float C, const float* tau, int32_t* draft_tokens,
                   uint64_t seed, uint64_t round, uint32_t flags, int32_t* out_k, int32_t* out_tstar,
                   float* out_resid_mass, uint32_t* out_status, float* out_div, void* workspace,
                   size_t workspace_bytes, hipStream_t stream);

/* saguaro_verify_cache_lookup - one round of Saguaro's verification and outcome cache in one
 * call: saguaro_verify_cache followed by the lookup of the verified outcomes in the cache just
 * built ([SSD] sections 5.1 and 7.1).  Outputs are exactly those of
 *   saguaro_verify_cache(..., out_cache, workspace, workspace_bytes, stream)
 *   saguaro_cache_lookup(0, out_cache, fanout, K, B, out_k, out_tstar, out_slot, out_hit, out_batch, stream)
 * where fanout is the call's fan-out (returned in out_fanout_host).  On the bf16 path the lookup
 * runs inside the verification's last kernel, as each request's outcome is settled (one kernel
 * launch fewer); elsewhere the two calls run one after the other.
 *   out_slot [B] int32, out_hit [B] uint8, out_batch [2] int32 (nullable): as saguaro_cache_lookup
 *   workspace  spec_workspace_bytes(B, K, V) bytes, same contract as spec_verify
 * Return codes: as saguaro_verify_cache (SPEC_EINVAL also for a null out_slot or out_hit). */
int saguaro_verify_cache_lookup(const void* draft_logits, const void* target_logits, int dtype, int B, int K, int V,
                                const spec_params* params, int F, float C, int32_t* draft_tokens, uint64_t seed,
                                uint64_t round, uint32_t flags, int budget, double a, double r, int32_t* out_fanout_host,
                                int32_t* out_k, int32_t* out_tstar, float* out_resid_mass, uint32_t* out_status,
                                int32_t* out_cache, int32_t* out_slot, uint8_t* out_hit, int32_t* out_batch,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

/* saguaro_verify_cache_noalloc - saguaro_verify_cache for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments and outputs without the workspace: a static device array of
 * SPEC_NOALLOC_SCRATCH_BYTES inside the library takes its place (each GPU the library runs on
 * holds one until the process ends; the call allocates nothing).  Calls on one GPU share that
 * scratch: the call clears what must start at zero with a fill kernel on `stream` (so shapes
 * may change between calls), and calls that overlap on one GPU (e.g. on two streams) race.
 * Returns SPEC_EWORKSPACE when spec_workspace_bytes(B, K, V) exceeds the scratch (e.g. B = 16,
 * K = 5, V = 128256 needs 18.5 MiB and fits; B = 32 at that K and V does not), SPEC_EHIP when
 * the scratch's device address cannot be had, otherwise the codes of saguaro_verify_cache. */
int saguaro_verify_cache_noalloc(const void* draft_logits, const void* target_logits, int dtype, int B, int K, int V,
                                 const spec_params* params, int F, float C, int32_t* draft_tokens, uint64_t seed,
                                 uint64_t round, uint32_t flags, int budget, double a, double r,
                                 int32_t* out_fanout_host, int32_t* out_k, int32_t* out_tstar, float* out_resid_mass,
                                 uint32_t* out_status, int32_t* out_cache, hipStream_t stream);

/* saguaro_verify_cache_lookup_timed - measurement helper, not part of the method:
 * saguaro_verify_cache_lookup with the same arguments and outputs, plus two HIP events
 * (created by the caller, with timing enabled) that bound the execution of the kernel that reads
 * every logit: the start and stop events of the bf16 path's count kernel launch (elsewhere,
 * events recorded on `stream` before and after the verification, ahead of the lookup).
 * hipEventElapsedTime of the pair gives that kernel's duration; the call's outputs and the work
 * done are unchanged.
 * Return codes as saguaro_verify_cache_lookup, SPEC_EINVAL also for a null event, SPEC_EHIP
 * when an event cannot be recorded. */
int saguaro_verify_cache_lookup_timed(const void* draft_logits, const void* target_logits, int dtype, int B, int K,
                                      int V, const spec_params* params, int F, float C, int32_t* draft_tokens,
                                      uint64_t seed, uint64_t round, uint32_t flags, int budget, double a, double r,
                                      int32_t* out_fanout_host, int32_t* out_k, int32_t* out_tstar,
                                      float* out_resid_mass, uint32_t* out_status, int32_t* out_cache,
                                      int32_t* out_slot, uint8_t* out_hit, int32_t* out_batch, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream, hipEvent_t count_before,
                                      hipEvent_t count_after);

/* ---------------------------------------------------------------------------------------------
 * Verification from given probabilities
 * ------------------------------------------------------------------------------------------- */

/* Bytes of scratch spec_verify_probs needs for B requests over V tokens (pure host function); 0 where
 * it needs none (V up to 8192; the workspace may then be null), and for sizes it rejects.  Every call
 * writes what it reads of it, so it needs no clearing; one workspace serves one call at a time (two
 * captured graphs that may run at once need two). */
size_t spec_verify_probs_workspace_bytes(int B, int V);

/* spec_verify_probs - the acceptance scan and the correction token of spec_verify ([SpS]
 * sections 1 and 3) for callers that hold processed probabilities and draw their own random
 * numbers.  For each request b with L = draft_lens[b] drafted tokens (K where draft_lens is null):
 *   for j = 0..L-1: accept s_j iff u_j * p_j(s_j) < q_j(s_j) (in fp64); stop at the first
 *   rejection; k = number of accepted tokens.  k < L: t* ~ (q_k - p_k)+ ; k = L: t* ~ q_L.
 *   t* is the first token whose running mass exceeds v times the row's total, and the last one
 *   that has mass where none does (v = 1).  Rows need not sum to 1: each is taken over its own
 *   total.  Masses are summed in fp64.  A rejection that leaves no residual draws from q_k.
 *   draft_probs   [B][K][V], or null with SPEC_UNIFORM_DRAFT (p = 1/V everywhere) or
 *                 SPEC_POINT_DRAFT (p = 1 at the drafted token)
 *   target_probs  [B][K+1][V] (rows past L are not read)
 *   dtype         SPEC_FP32, SPEC_BF16 or SPEC_FP16, of both
 *   *_request_stride, *_row_stride   in elements; V is contiguous.  No alignment is needed
 *                 beyond the element's
 *   draft_tokens  [B][K] int32; entries past L are not read
 *   draft_lens    [B] int32 in [0, K] (nullable)
 *   accept_u      [B][K], sample_v [B], in [0, 1]; uniform_dtype SPEC_FP32 or SPEC_FP64
 *   flags         0, SPEC_UNIFORM_DRAFT or SPEC_POINT_DRAFT
 *   out_k, out_tstar [B] int32; out_emitted [B][K+1] int32 (nullable): the accepted tokens, then
 *                 t*, then -1; out_resid_mass [B] float (nullable); out_status [B] (nullable)
 * Status: SPEC_ST_EMPTY_RESIDUAL, _OUTSIDE_DRAFT_SUPPORT, and with k = 0, t* = -1: _BAD_PROB
 * (among the probabilities read), _BAD_TOKEN (a drafted token that the scan reached), _BAD_PARAM
 * (a length outside [0, K], a random number that was used and is outside [0, 1] or NaN).
 * One launch for up to 8192 tokens, otherwise two. */
int spec_verify_probs(const void* draft_probs, int64_t draft_request_stride, int64_t draft_row_stride,
                      const void* target_probs, int64_t target_request_stride, int64_t target_row_stride, int dtype,
                      int B, int K, int V, const int32_t* draft_tokens, const int32_t* draft_lens, const void* accept_u,
                      const void* sample_v, int uniform_dtype, uint32_t flags, int32_t* out_k, int32_t* out_tstar,
                      int32_t* out_emitted, float* out_resid_mass, uint32_t* out_status, void* workspace,
                      size_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------------------------
 * Draft-tree rows, the paged cache and attention over a shared prefix
 * ------------------------------------------------------------------------------------------- */

/* spec_tree_rows - the rows that score a draft tree in one pass of a model ([MSD] section 3.1:
 * the branches hang off one context; [SSD] section 5.1: guessed outcomes hang off the drafted
 * chain).  Trees as in mirror_tree_lookup: N nodes per request, parents first,
 * tree_parents[b][n] in [-1, n) (-1: it follows the context), a node with a negative token or
 * another parent is not part of the tree, nor is anything below it, nor is a node deeper than
 * max_depth.  A chain is the tree with parents n - 1.
 *   node_slots        [B][N] int32: the cache slot each node's key and value go to
 *   ctx_len           [B] int32: tokens already in the context
 *   max_depth         entries per list (>= 1)
 *   out_positions     [B][N] int32: ctx_len + depth - 1 for a node of depth 1 (a root), 2, ...;
 *                     -1 for a node outside the tree
 *   out_append_slots  [B][N] int32: node_slots, -1 for a node outside the tree
 *   out_suffix_slots  [B][N][max_depth] int32: the slots from the root to the node, then -1
 *   out_suffix_len    [B][N] int32: the depth; 0 for a node outside the tree
 * positions and append_slots feed spec_kv_append, the lists spec_prefix_attention. */
int spec_tree_rows(const int32_t* tree_tokens, const int32_t* tree_parents, const int32_t* node_slots,
                   const int32_t* ctx_len, int B, int N, int max_depth, int32_t* out_positions,
                   int32_t* out_append_slots, int32_t* out_suffix_slots, int32_t* out_suffix_len, hipStream_t stream);

/* A paged cache of keys and values: k and v are [num_pages][page_size][heads][head_dim] with
 * head_dim contiguous and the other strides in elements, not negative and the same for both (so a
 * cache with heads outside tokens, or keys and values side by side in one buffer, is described as well).  Slot s is
 * token s % page_size of page s / page_size; num_pages * page_size < 2^31.
 * dtype SPEC_BF16, SPEC_FP16, or SPEC_E4M3 with k_scale and v_scale [heads] float (null: 1): the
 * key of head h is its 8-bit value times k_scale[h]. */
typedef struct {
    void* k;
    void* v;
    int32_t dtype;
    int32_t num_pages;
    int32_t page_size;
    int32_t heads;
    int32_t head_dim;
    int64_t page_stride;
    int64_t token_stride;
    int64_t head_stride;
    const float* k_scale;
    const float* v_scale;
} spec_kv_cache;

/* Host helper: rotary inverse frequencies f_i = base^(-2i / rot_dim), i < rot_dim / 2, with those
 * that turn slowly stretched for a context `factor` times the original one: with
 * n_i = original_len f_i / 2 pi turns over the original context and
 * g_i = clamp((n_i - low) / (high - low), 0, 1), f_i becomes f_i (g_i + (1 - g_i) / factor).
 * factor = 1 leaves all as they are; low = high takes g_i = (n_i >= low) (+inf: all stretched,
 * linear interpolation of positions).  rot_dim even and >= 2, base > 0, factor >= 1, low <= high,
 * original_len >= 1; low and high may be +inf.  out [rot_dim / 2] host. */
int spec_rope_frequencies(int rot_dim, double base, double factor, double low, double high, int original_len,
                          double* out);

enum { SPEC_ROPE_INTERLEAVED = 1 }; /* pairs (2i, 2i + 1); without it pairs (i, i + rot_dim / 2) */

/* spec_kv_append - rotary positions and the append to the paged cache in one pass: queries are
 * rotated into q_out, keys are rotated on their way into the cache, values go along.
 * The pair (x, y) of index i becomes rope_scale * (x cos - y sin, y cos + x sin) with the angle
 * position * freqs[i] taken in fp64; elements from rot_dim on pass through.  Sums are in fp32 and
 * rounded once, to the output's type; an 8-bit cache holds (value / scale), clamped to its range.
 *   q        [T][q_heads][head_dim] (null: no queries), q_out likewise: q itself (in place, the
 *            same strides) or memory apart from it
 *   k, v     [T][heads][head_dim], apart from the cache (both null with a null cache: queries only)
 *   dtype    SPEC_BF16 or SPEC_FP16, of q, q_out, k and v; a cache of that type or SPEC_E4M3
 *   strides  in elements, per token and per head; head_dim is contiguous
 *   positions [T] int32;  freqs [rot_dim / 2] double, device; rot_dim even, 0 (no rotation, freqs
 *            and positions may be null) to head_dim;  rope_scale: a factor on cos and sin (1: none)
 *   slots    [T] int32: -1 stores nothing for that token (its query is rotated all the same).
 *            Slots of one call differ; where two are the same, which of the values stays is open
 *   out_status [T] (nullable): SPEC_ST_BAD_SLOT for a slot outside [-1, num_pages * page_size),
 *            which stores nothing, else 0
 * T = 0 launches nothing.  Rows of eight elements that start 16-byte aligned move as vectors;
 * other strides and sizes are taken element by element. */
int spec_kv_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out, int64_t q_out_token_stride,
                   int64_t q_out_head_stride, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                   const void* v, int64_t v_token_stride, int64_t v_head_stride, int dtype, int T, int q_heads,
                   int heads, int head_dim, const int32_t* positions, const int32_t* slots, const double* freqs,
                   int rot_dim, float rope_scale, uint32_t rope_flags, const spec_kv_cache* cache, uint32_t* out_status,
                   hipStream_t stream);

/* Bytes of scratch spec_prefix_attention needs (pure host function; 0 for sizes it rejects):
 * rows R, groups G, query heads, cache heads, head_dim, the longest prefix the page table can hold
 * (max_pages * page_size), and the entries of a suffix list.  Every call writes what it reads of it, so it needs no clearing;
 * one workspace serves one call at a time (two captured graphs that may run at once need two). */
size_t spec_prefix_attention_workspace_bytes(int R, int G, int q_heads, int heads, int head_dim,
                                             int64_t max_prefix, int max_suffix);

/* spec_prefix_attention - attention of R rows (one query token each) in G groups: the rows of a
 * group share a prefix of the cache and see tokens of their own behind it ([SSD] section 8.2,
 * [MSD] section 3.1: all branches of a request are scored on one context).  The keys and values of
 * a prefix are read once for all rows of its group.  For row r of group g and query head h, with
 * cache head h / (q_heads / heads):
 *   out[r][h] = sum_t softmax_t(scale * q[r][h] . k_t) v_t
 * over the prefix tokens t < prefix_len[g] (slot page_table[g][t / page_size] * page_size +
 * t % page_size) and the tokens at the slots suffix_slots[r][i], i < suffix_len[r].
 * Rows verify, decode and roll out alike: a chain's token j lists the chain's slots 0..j, a tree
 * node the slots from its root (spec_tree_rows), a plain decoding step its own slot or none.
 *   q, out       [R][q_heads][head_dim], dtype SPEC_BF16 or SPEC_FP16; strides in elements per row
 *                and per head, head_dim contiguous
 *   cache        of q's dtype or SPEC_E4M3; q_heads a multiple of cache heads
 *   row_start    [G+1] int32, not decreasing, in [0, R]: group g holds rows row_start[g] to
 *                row_start[g+1] - 1.  Rows outside every group (padding) are left as they were
 *   page_table   [G][max_pages] int32;  prefix_len [G] int32 (taken within [0, max_pages *
 *                page_size]).  max_pages may be 0 (then both may be null)
 *   suffix_slots [R][max_suffix] int32, suffix_len [R] int32 (taken within [0, max_suffix]);
 *                max_suffix may be 0 (then both may be null)
 *   out_lse      [R][q_heads] float (nullable): log of the sum of exp of the scaled scores
 * A page outside [0, num_pages) and a slot outside the cache hold no token: they are left out, as
 * holes of a mask.  A row that sees nothing (or only scores of -inf) gives zeros and lse = -inf.
 * What lies in the cache outside the tokens named does not matter, NaN and infinities included.
 * Scores, softmax statistics and sums are in fp32; the weights are rounded to q's type for the
 * product with the values.
 * R = 0 launches nothing.  head_dim: a multiple of 8, up to 256.  out is apart from q.  q, out, k and v 16-byte aligned (k and v of an 8-bit
 * cache 8-byte), strides multiples of 8 elements: otherwise SPEC_EINVAL. */
int spec_prefix_attention(const void* q, int64_t q_row_stride, int64_t q_head_stride, int dtype, int R, int q_heads,
                          const spec_kv_cache* cache, int G, const int32_t* row_start, const int32_t* page_table,
                          int max_pages, const int32_t* prefix_len, const int32_t* suffix_slots, int max_suffix,
                          const int32_t* suffix_len, float scale, void* out, int64_t out_row_stride,
                          int64_t out_head_stride, float* out_lse, void* workspace, size_t workspace_bytes,
                          hipStream_t stream);

/* spec_read_ceiling - measurement helper, not part of the method: one plain streaming read of
 * `bytes` bytes of device memory at `data` (16-byte aligned, bytes a multiple of 16), the
 * bandwidth ceiling a verification call that reads the same number of logit bytes is compared
 * against.  sink: [1] uint32 device word, written only if the xor of the data equals a fixed
 * value (never in practice).  Returns SPEC_EINVAL for a null pointer, zero or unaligned sizes. */
int spec_read_ceiling(const void* data, size_t bytes, uint32_t* sink, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_H */
