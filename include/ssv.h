/*
 * ssv.h -- C ABI of libssv: the target-model verification pass of
 * speculative decoding for block-diffusion language models, on one GB300
 * (sm_103a).
 *
 * The pass (SimSD, "Simple Speculative Decoding in Diffusion Language
 * Models", summary sections 1-4): after the prompt the target sees a data
 * section D (B reference tokens) and a mask section D~ (B [MASK] slots);
 * the pair (D_k, D~_k) occupies one response position.  A stage map tau,
 * a permutation of 1..B, orders the positions in time and gates attention.
 * One forward pass under that mask yields logits for every drafted
 * position; acceptance then keeps the longest accepted prefix in stage
 * order (SimSD section 4; state equality and the coupled Gumbel-noise match
 * of the SPOT review, section "How it is used").
 *
 * Conventions for every entry point
 *  - All pointers named "device" are CUDA device (or managed) addresses on
 *    the current device; "host" pointers are ordinary CPU memory.  The
 *    caller owns every buffer; the library allocates nothing on these
 *    paths.  Scratch space is caller-provided ("workspace"), sized by the
 *    matching *_workspace query, 256-byte aligned, and must be all-zero
 *    when first used: each call leaves the zero-initialised counter area
 *    zero again on exit.  The attention entry points (ssv_verify_attn,
 *    ssv_tree_verify_attn, ssv_verify_attn_fp8) keep their counters at a
 *    place and in an extent that no argument changes, the same for the three:
 *    one workspace, at least as large as each call asks for, serves them with
 *    any sizes, one after the other.  ssv_accept and ssv_lmhead_accept lay
 *    theirs out by the call: clear a workspace before calls of another batch,
 *    total_slots, V, hidden or mode, or of another entry point, use it.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls are
 *    asynchronous on it.  Host-side validation errors return synchronously
 *    and launch nothing.
 *  - Errors found on the device (a stage map that is not a permutation, a
 *    bounded wait that ran out, a non-finite temperature) are written to
 *    `dev_status` (device int32, may be NULL; first error wins) and read
 *    back with ssv_get_status().  Affected outputs are then unspecified,
 *    and after SSV_ERR_TIMEOUT the workspace's counter area may be left
 *    non-zero: clear the workspace before its next use.
 *  - Nothing is thread-local; calls from several host threads on different
 *    streams are safe.  Two calls whose workspaces overlap must not run
 *    concurrently.
 */
#ifndef SSV_H_
#define SSV_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SSV_API __attribute__((visibility("default")))
#else
#define SSV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SSV_OK = 0,
  SSV_ERR_INVALID = 1,      /* bad argument (null pointer, shape, alignment) */
  SSV_ERR_UNSUPPORTED = 2,  /* valid but not implemented (e.g. head_dim 96) */
  SSV_ERR_CUDA = 3,         /* a CUDA runtime call failed */
  SSV_ERR_TIMEOUT = 4,      /* a bounded on-device wait ran out */
  SSV_ERR_BAD_TAU = 5,      /* stage map of some sequence is not a permutation of 1..B */
  SSV_ERR_WORKSPACE = 6,    /* workspace null, misaligned or smaller than the query */
  SSV_ERR_NOT_FINITE = 7,   /* temperature not finite / negative */
  SSV_ERR_NO_PAGES = 8      /* the free stack holds fewer pages than the pass needs (ssv_page_plan) */
} ssv_status;

typedef enum { SSV_F32 = 0, SSV_BF16 = 1 } ssv_dtype;

typedef enum {
  SSV_ACCEPT_ARGMAX = 0,    /* T = 0 state equality: accept iff draft == argmax(l) */
  SSV_ACCEPT_GUMBEL = 1,    /* coupled noise: accept iff draft == argmax(fl(l/T) + G[row]) */
  SSV_ACCEPT_REJECT = 2,    /* standard rejection sampling, accept iff u < p(d)/q(d) */
  SSV_ACCEPT_GUMBEL_GEN = 3 /* coupled noise generated on the device: accept iff
                               draft == argmax(fl(l/T) + G(noise_seed, noise_row[k], v)) */
} ssv_accept_mode;

/*
 * One sequence of a packed batch.  Query rows of a sequence are its N fresh
 * prompt rows followed by 2B tail rows (D_1..D_B, then D~_1..D~_B); they sit
 * at rows [q_off, q_off + N + 2B) of Q, K_new, V_new and O.  Its C cached
 * prompt keys sit at rows [kv_off, kv_off + C) of K_cache / V_cache.  Its
 * stage map occupies tau[tau_off .. tau_off + B).  Sequences are packed in
 * increasing q_off order without overlap (q_off[b] + N_b + 2B_b <=
 * q_off[b+1]): kernels find a row's sequence by binary search on q_off.
 * Every kernel checks each sequence's extents on the device before it
 * touches the sequence's rows (q_off + N + 2B <= total_rows, kv_off + C <=
 * the cache rows, tau_off + B <= total_slots, all offsets >= 0, 1 <= B <=
 * 64, and for the attention C, N, B within max_cache, max_new, max_block):
 * a sequence that fails is skipped -- nothing of it is read or written --
 * and SSV_ERR_INVALID is reported through dev_status.  Overlapping or
 * unsorted sequences are not detected (their rows may be processed twice or
 * under the wrong sequence, still inside the buffers).
 */
typedef struct {
  int32_t cache_len;  /* C >= 0 */
  int32_t new_len;    /* N >= 0 */
  int32_t block;      /* B, 1 <= B <= 64 */
  int32_t q_off;
  int32_t kv_off;
  int32_t tau_off;
} ssv_seq;

/* ------------------------------------------------------------------------
 * ssv_rope_copy -- rotary embedding with the RoPE-copy index.
 * SimSD summary, section 3 "Position Encoding Alignment": each mask slot
 * D~_k reuses the RoPE index of its data token D_k.
 *
 * Positions, without a position table (positions == NULL): fresh prompt row
 * i is at C + i; tail row r (0 <= r < 2B) at P + (r mod B), P = C + N.
 * With a table (device int32 [total_rows], entries >= 0): fresh prompt row
 * i of a sequence is at positions[q_off + i], data row D_k at
 * positions[q_off + N + k - 1], and mask row D~_k at D_k's entry (entries
 * at mask rows are not read).  The table serves passes whose positions are
 * not contiguous: after a commit (ssv_commit) the accepted data rows keep
 * the positions of their slots, so the next pass over the same block gives
 * its remaining slots, and the emitted token entering as a fresh prompt
 * row, the positions of their own slots (a reading: the pages do not
 * describe the loop).  Rotate-half pairing (x_i, x_{i+d/2}) with
 * theta_i = base^(-2i/d); angles are formed and reduced in fp64, the
 * rotation is done in fp32 and stored in `dtype`.
 *
 * q_in  [total_rows, Hq, d]  device, dtype     q_out same shape (may equal q_in)
 * k_in  [total_rows, Hkv, d] device, dtype     k_out same shape (may equal k_in)
 * seqs  [batch] device ssv_seq.  Every row of [0, total_rows) must belong to
 *       exactly one sequence (rows outside all sequences are left untouched).
 * d in {64, 128}; pointers 16-byte aligned.
 * Errors: SSV_ERR_INVALID (null, non-positive sizes, misalignment),
 *         SSV_ERR_UNSUPPORTED (d), SSV_ERR_CUDA (launch); on device
 *         SSV_ERR_INVALID for a sequence whose rows leave [0, total_rows)
 *         (or B outside 1..64, or C + N + B beyond int range; its rows are
 *         left untouched) and for a negative table entry (that row is left
 *         untouched).
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* q_in;
  const void* k_in;
  void* q_out;
  void* k_out;
  ssv_dtype dtype;
  int32_t Hq, Hkv, d;
  double base;                 /* RoPE base, e.g. 10000 */
  const ssv_seq* seqs;         /* device */
  int32_t batch;
  int32_t total_rows;
  const int32_t* positions;    /* device [total_rows] or NULL (see above) */
  int32_t* dev_status;         /* device, may be NULL */
} ssv_rope_args;

SSV_API ssv_status ssv_rope_copy(const ssv_rope_args* a, void* stream);

/* ------------------------------------------------------------------------
 * ssv_verify_attn -- attention of the verification pass.
 * SimSD summary, section 2 "Temporal Attention Mask" and section 4
 * "Verification".  For every query row and query head h (kv head h / G,
 * G = Hq / Hkv):  O = softmax(scale * q K^T restricted to allowed keys) V.
 * Keys of a sequence, in order: cache (C), fresh prompt (N), D_1..D_B,
 * D~_1..D~_B.  Allowed keys:
 *   fresh prompt row i : cache and fresh prompt keys 0 .. C+i (causal)
 *   data row D_j       : whole prompt, D_k with tau(k) <= tau(j)  (reading;
 *                        the pages fix only the mask-slot rule)
 *   mask row D~_i      : whole prompt, D_j with tau(j) < tau(i),
 *                        D~_j with tau(j) >= tau(i)
 * The mask is derived on the device from tau; it is never stored.
 *
 * q       [total_rows, Hq, d]   device, in_dtype, post-RoPE
 * k_cache [total_cache, Hkv, d] device, in_dtype, already rotated
 * v_cache [total_cache, Hkv, d] device
 * k_new   [total_rows, Hkv, d]  device, post-RoPE
 * v_new   [total_rows, Hkv, d]  device
 * o       [total_rows, Hq, d]   device, out_dtype (written for every row of
 *                               every sequence)
 * tau     [sum B] int32 device
 * in_dtype: SSV_F32 (exact fp32 SIMT path) or SSV_BF16 (tensor-core path,
 * fp32 accumulation).  out_dtype: SSV_F32 or SSV_BF16 (bf16 input only).
 * d in {64, 128}; Hq % Hkv == 0; 1 <= B <= 64; pointers 16-byte aligned.
 * max_cache / max_new / max_block bound every sequence's C / N / B (used to
 * size grids and workspace).  scale 0 means 1/sqrt(d).
 * Errors: SSV_ERR_INVALID, SSV_ERR_UNSUPPORTED, SSV_ERR_WORKSPACE,
 *         SSV_ERR_CUDA; on device SSV_ERR_BAD_TAU, SSV_ERR_TIMEOUT, and
 *         SSV_ERR_INVALID for a sequence outside the buffers (skipped: its
 *         rows of o are not written).
 * Scheduling: the bf16 path launches one CTA per SM; where a unit of work is
 * split across CTAs, the CTA holding its first key block waits (bounded, about
 * one second of SM clock) for the others' partial results.  Before launching,
 * the host checks that the kernel's resources let one CTA reside on every SM
 * at once (else SSV_ERR_CUDA, nothing launched).  Work on other streams that
 * keeps SMs busy for longer than that second while this kernel runs can
 * still end the call with SSV_ERR_TIMEOUT (never a hang).
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const void* k_new;
  const void* v_new;
  void* o;
  ssv_dtype in_dtype;
  ssv_dtype out_dtype;
  int32_t Hq, Hkv, d;
  float scale;
  const ssv_seq* seqs;         /* device [batch] */
  int32_t batch;
  const int32_t* tau;          /* device [total_slots] */
  int32_t total_rows;          /* sum of N + 2B */
  int32_t total_cache;         /* sum of C */
  int32_t total_slots;         /* sum of B */
  int32_t max_cache, max_new, max_block;
  int32_t* dev_status;         /* device, may be NULL */
} ssv_attn_args;

SSV_API ssv_status ssv_verify_attn_workspace(const ssv_attn_args* a, size_t* bytes);
SSV_API ssv_status ssv_verify_attn(const ssv_attn_args* a, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * ssv_accept -- acceptance in temporal order, longest accepted prefix.
 * SimSD summary section 4 "Acceptance" (rejection sampling in the draft's
 * temporal order); SPOT review "How it is used" (state equality, exact at
 * T = 0; coupled-noise match with one Gumbel table per absolute output
 * position, which recovers the target distribution, Proposition 2).
 *
 * Per sequence b with block B, verified stages 1..gamma (0 <= gamma <= B):
 * stage s is slot k = tau^{-1}(s).  Walk s = 1..gamma and accept while
 *   ARGMAX : draft_tokens[k] == argmax_v l_k[v]            (ties: lowest v)
 *   GUMBEL : draft_tokens[k] == argmax_v fl32(fl32(l_k[v]/T) + noise[noise_row[k]][v])
 *            (IEEE fp32, no contraction; T = 0 means ARGMAX)
 *   REJECT : u_accept[k] < p(d)/q(d), p = softmax(l_k/T), q = softmax(draft_logits_k/T)
 *   GUMBEL_GEN : as GUMBEL with the table value replaced by one generated on
 *            the device, G(seed, pos, v) = -L(-L(U)), U = (floor(x / 2^9) + 1/2)
 *            2^-23, x = word (v mod 4) of Philox4x32-10 at counter
 *            (floor(v / 4), pos, 0, 0) under key (low, high word of noise_seed),
 *            pos = noise_row[k] (any 32-bit value the caller assigns to the
 *            slot's absolute output position; drafter and target use the same),
 *            L the natural logarithm by one fixed sequence of fp32 operations:
 *            reduction to m in [sqrt(1/2), sqrt 2], s = (m - 1) / (m + 1),
 *            ln m = 2 s + s z (2/3 + z (2/5 + z (2/7 + z 2/9))), z = s^2
 *            (Horner from the inside, every operation rounded to nearest), plus
 *            e ln 2.  Nothing but the logits is read; T = 0 means ARGMAX.
 * n_acc = leading accepted stages.  If c = n_acc + 1 <= B one target token
 * is emitted at stage c: the ARGMAX/GUMBEL decision; for REJECT a sample of
 * (p - q)_+ if c <= gamma, else of p, by inverse CDF with u_sample[b]
 * (smallest v whose cumulative mass exceeds u_sample * total).
 *
 * logits       [total_slots, V] device, logits_dtype, row = slot (slot order);
 *              only rows of stages <= min(gamma + 1, B) are read.
 * draft_logits [total_slots, V] device, logits_dtype (REJECT only, else NULL)
 * draft_tokens, tau, noise_row, u_accept: [total_slots] device
 * block, gamma, slot_off, u_sample: [batch] device; slot_off[b] = first slot;
 *              sequences in increasing slot order without overlap
 *              (slot_off[b] + block[b] <= slot_off[b+1])
 * noise [n_noise_rows, V] fp32 device (GUMBEL with T > 0 only)
 * noise_seed: GUMBEL_GEN only (noise_row then holds positions, not rows)
 * Outputs: n_acc[batch], n_out[batch] (= n_acc + 1 if a token is emitted),
 *          tokens[total_slots]: per sequence, the accepted drafts in stage
 *          order then the emitted token, rest -1.
 * V >= 1; T >= 0 (REJECT needs T > 0); 1 <= block <= 64.
 * Workspace: ssv_accept_workspace bytes.  Under REJECT it includes
 *   16 * batch * 8192 * ceil(V / 8192) bytes in which the first emission
 *   pass keeps the double-float exponentials of each sequence's emitted row
 *   for the second (about 2.4 MB per sequence at V = 151936).
 * Errors: SSV_ERR_INVALID, SSV_ERR_WORKSPACE, SSV_ERR_NOT_FINITE,
 *         SSV_ERR_CUDA; on device SSV_ERR_BAD_TAU.
 * ---------------------------------------------------------------------- */
typedef struct {
  ssv_accept_mode mode;
  float T;
  int32_t V;
  int32_t batch;
  int32_t total_slots;
  int32_t max_block;
  ssv_dtype logits_dtype;
  const void* logits;
  const void* draft_logits;
  const int32_t* draft_tokens;
  const int32_t* tau;
  const int32_t* block;
  const int32_t* gamma;
  const int32_t* slot_off;
  const float* noise;
  int32_t n_noise_rows;
  const int32_t* noise_row;
  const float* u_accept;
  const float* u_sample;
  int32_t* n_acc;
  int32_t* n_out;
  int32_t* tokens;
  int32_t* dev_status;         /* device, may be NULL */
  uint64_t noise_seed;         /* GUMBEL_GEN: key of the noise generator */
} ssv_accept_args;

SSV_API ssv_status ssv_accept_workspace(const ssv_accept_args* a, size_t* bytes);
SSV_API ssv_status ssv_accept(const ssv_accept_args* a, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * ssv_verify_step -- the whole verification step in one call: ssv_rope_copy
 * (rope, may be NULL when Q and K_new are already rotated), ssv_verify_attn
 * (attn), then ssv_accept (acc, may be NULL), in that order on `stream`, with
 * the same arguments, results and workspaces as the three separate calls.
 * SimSD summary sections 2-4 (one verification pass: rotation with the
 * RoPE-copy index, temporal attention, acceptance in temporal order).
 *
 * The difference is overlap: each kernel is launched with programmatic
 * dependent launch and may begin its input-independent set-up while the one
 * before it finishes.  When the rotation's outputs (rope->q_out, k_out)
 * overlap none of attn->seqs, tau, k_cache, v_cache, the attention kernel
 * plans and starts streaming the KV cache before the rotation completes;
 * when neither the rotation's outputs nor attn->o or the attention
 * workspace overlap acc->tau, block, gamma, slot_off, noise_row, the
 * acceptance kernel builds its row list before the attention completes.
 * Everything else is read only after the preceding kernel has completed.
 * Kernels that ran before the call must be complete or ordered by the stream
 * as usual; nothing here relaxes that.
 * All arguments are validated before anything is launched.
 * Errors: those of the three calls.
 * ---------------------------------------------------------------------- */
SSV_API ssv_status ssv_verify_step(const ssv_rope_args* rope, const ssv_attn_args* attn, void* attn_workspace,
                                   size_t attn_workspace_bytes, const ssv_accept_args* acc, void* acc_workspace,
                                   size_t acc_workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * ssv_accept_noalloc -- ssv_accept for callers that cannot allocate.
 * The pages have no counterpart: this is an interface addition of the
 * library.  Some callers have no way to obtain device memory of their own:
 * a host runtime that owns every byte of the GPU and hands its plugins no
 * allocator, or a latency-critical path where cudaMalloc (which can
 * synchronise the device) and allocating library routines are not allowed.
 * They pass inputs and outputs exactly as for ssv_accept but no workspace;
 * the scratch lives in a fixed 4 MiB array inside the library, which every
 * GPU that loads libssv holds until the process exits.
 *  - Same arguments, semantics and results as ssv_accept.
 *  - Calls whose scratch would exceed 4 MiB (roughly total_slots *
 *    ceil(V / 8192) > 120000 chunk records, e.g. more than ~6000 slots at
 *    V = 151936) return SSV_ERR_WORKSPACE and launch nothing.  Under REJECT
 *    the stored exponentials of the emitted rows (see ssv_accept) are kept
 *    only when they fit too; otherwise the second emission pass forms them
 *    again from the logits, with identical results.
 *  - Calls nothing that allocates: no cudaMalloc/cudaFree, no allocating
 *    library routine.  It clears its arrival counters with a memset on
 *    `stream` at every call.
 *  - The first call in each CUDA context looks up the array's device
 *    address (cudaGetSymbolAddress with that context current) and caches it
 *    per device together with the context; a later call from another
 *    context on that device (after cudaDeviceReset, or a context the caller
 *    made current) looks it up again.  Make the first call in a context
 *    before any stream capture.  Device ordinals of 64 and above are refused
 *    with SSV_ERR_INVALID.
 *  - All calls share the one array and it keeps the last call's contents:
 *    calls that overlap on the GPU (different streams or host threads)
 *    race and must be serialised by the caller.
 * ---------------------------------------------------------------------- */
SSV_API ssv_status ssv_accept_noalloc(const ssv_accept_args* a, void* stream);

/* ------------------------------------------------------------------------
 * ssv_commit -- commit of a verification pass into the KV cache.
 * SimSD summary, section 4 "Speculative decoding pipeline" (Acceptance: the
 * longest accepted prefix, in the temporal order the draft induces, is
 * committed and the loop repeats) and "Main contributions" 3 (composes with
 * a KV cache).  The pages give no cache layout; the reading taken: after
 * sequence b's pass (C cached rows, N fresh prompt rows, block B, stage map
 * tau, n_acc[b] accepted stages) its cache gains, appended after row C,
 *   - the keys / values of the N fresh prompt rows, in row order, then
 *   - those of the data rows of stages 1..n_acc, in stage order (stage s is
 *     slot k = tau^{-1}(s), fresh row N + k).
 * Mask rows are never committed.  Rows are copied as they are (keys keep the
 * rotation ssv_rope_copy gave them).  new_len[b] = C + N + n_acc[b].
 *
 * k_new, v_new [total_rows, Hkv, d]  device, dtype: the pass's fresh rows
 *                                     (post-RoPE keys), packed per sequence at
 *                                     seqs[b].q_off as for ssv_verify_attn
 * k_dst, v_dst [dst_rows, Hkv, d]    device, dtype: destination caches;
 *                                     sequence b's cache starts at row
 *                                     dst_off[b] and has dst_cap[b] rows of
 *                                     room (rows C .. C + N + n_acc - 1 of it
 *                                     are written, nothing else).  May be the
 *                                     k_cache / v_cache of ssv_verify_attn
 *                                     when its sequences were laid out with
 *                                     room (dst_off = kv_off).
 * seqs, tau, batch, total_rows as for ssv_verify_attn; n_acc [batch] device
 * (as written by ssv_accept); dst_off, dst_cap [batch] device; new_len
 * [batch] device, written (-1 for a sequence rejected on the device).
 * dtype SSV_F32 or SSV_BF16; d in {64, 128}; pointers 16-byte aligned.
 * k_new / v_new must not overlap k_dst / v_dst (checked), and the
 * destination ranges [dst_off[b], dst_off[b] + dst_cap[b]) of different
 * sequences must not overlap (not checked: overlapping ones race).
 * Errors: SSV_ERR_INVALID, SSV_ERR_CUDA; on device SSV_ERR_BAD_TAU (stage
 * map not a permutation of 1..B) and SSV_ERR_INVALID (B outside 1..64, a
 * stage map outside tau[0, total_slots), n_acc outside 0..B, or the
 * appended rows do not fit dst_cap / dst_rows): that sequence's rows are not
 * written and its new_len is -1.  No workspace; asynchronous on `stream`.
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* k_new;
  const void* v_new;
  void* k_dst;
  void* v_dst;
  ssv_dtype dtype;
  int32_t Hkv, d;
  const ssv_seq* seqs;         /* device [batch] */
  int32_t batch;
  const int32_t* tau;          /* device [total_slots] */
  const int32_t* n_acc;        /* device [batch] */
  const int32_t* dst_off;      /* device [batch] */
  const int32_t* dst_cap;      /* device [batch] */
  int32_t* new_len;            /* device [batch], out */
  int32_t total_rows;          /* rows of k_new / v_new */
  int32_t total_slots;         /* entries of tau (sum of B) */
  int32_t dst_rows;            /* rows of k_dst / v_dst */
  int32_t* dev_status;         /* device, may be NULL */
} ssv_commit_args;

SSV_API ssv_status ssv_commit(const ssv_commit_args* a, void* stream);

/* ------------------------------------------------------------------------
 * ssv_lmhead_accept -- LM head over the mask slots fused with acceptance.
 * SimSD summary section 4 (the target scores every drafted position in one
 * pass; acceptance in the temporal order the draft induces); SPOT review
 * "How it is used" (state equality; coupled-noise match).  The pages do not
 * say how the logits are formed; the reading taken: the logits of mask slot
 * k are l_k = W h_k for the LM head W [V, hidden] and the slot's final
 * hidden state h_k.  This call computes, for every verified row (stage
 * <= min(gamma + 1, B)), the decision score over the whole vocabulary
 * without writing logits anywhere:
 *   ARGMAX : argmax_v l_k[v]                                   (ties: lowest v)
 *   GUMBEL : argmax_v fl32(fl32(l_k[v] / T) + noise[noise_row[k]][v])
 *            (IEEE fp32, no contraction; T = 0 means ARGMAX)
 * and then walks the stages exactly as ssv_accept (same n_acc, n_out,
 * tokens).  l_k is accumulated in fp32 on the tensor cores from the bf16
 * operands (exact products, fp32 sums in an unspecified order), so a
 * decision between two tokens whose scores differ by less than that
 * accumulation error may fall either way.  Rejection sampling is not
 * offered here (it needs the draft model's logits as well).
 *
 * hidden_states [total_slots, hidden] bf16 device, row = slot (slot order);
 *               only rows of verified stages are read (when some stages
 *               are not verified, a first kernel copies the verified rows
 *               into the workspace and the GEMM runs over those).
 * lm_head       [V, hidden] bf16 device, row-major.
 * draft_tokens, tau, noise_row: [total_slots] int32 device
 * block, gamma, slot_off: [batch] int32 device (as for ssv_accept)
 * noise [n_noise_rows, V] fp32 device (GUMBEL with T > 0 only, else NULL)
 * Outputs n_acc, n_out [batch], tokens [total_slots] as for ssv_accept.
 * Sizes: hidden % 64 == 0 and >= 64; 1 <= V; 1 <= total_slots <= 2048;
 *        batch <= 2048; pointers 16-byte aligned.
 * Workspace: ssv_lmhead_accept_workspace bytes, zero before first use.
 * Errors: SSV_ERR_INVALID (mode REJECT, sizes, null, alignment),
 *         SSV_ERR_NOT_FINITE (T), SSV_ERR_UNSUPPORTED (total_slots or batch
 *         above 2048), SSV_ERR_WORKSPACE, SSV_ERR_CUDA; on device
 *         SSV_ERR_BAD_TAU (that sequence's outputs are not written),
 *         SSV_ERR_INVALID (a verified slot's noise_row outside the table;
 *         likewise), SSV_ERR_TIMEOUT (a bounded wait ran out).
 * Scheduling: two kernels chained by programmatic dependent launch (a
 * gather of the verified rows, then the GEMM with one CTA per SM); the CTA
 * that finishes an M-tile last merges its rows; no CTA waits on another.
 * ---------------------------------------------------------------------- */
typedef struct {
  ssv_accept_mode mode;        /* SSV_ACCEPT_ARGMAX or SSV_ACCEPT_GUMBEL */
  float T;
  int32_t V;
  int32_t hidden;
  int32_t batch;
  int32_t total_slots;
  const void* hidden_states;   /* bf16 [total_slots, hidden] */
  const void* lm_head;         /* bf16 [V, hidden] */
  const int32_t* draft_tokens;
  const int32_t* tau;
  const int32_t* block;
  const int32_t* gamma;
  const int32_t* slot_off;
  const float* noise;
  int32_t n_noise_rows;
  const int32_t* noise_row;
  int32_t* n_acc;
  int32_t* n_out;
  int32_t* tokens;
  int32_t* dev_status;         /* device, may be NULL */
} ssv_lmhead_accept_args;

SSV_API ssv_status ssv_lmhead_accept_workspace(const ssv_lmhead_accept_args* a, size_t* bytes);
SSV_API ssv_status ssv_lmhead_accept(const ssv_lmhead_accept_args* a, void* workspace, size_t workspace_bytes,
                                     void* stream);

/* ------------------------------------------------------------------------
 * Tree (state-set) verification -- the verification pass over a draft tree
 * of block states and the acceptance by state equality.
 * SPOT review, "How it works" (the drafter grows a tree of candidate block
 * states, each edge committing one position with one token) and "How it is
 * used" (an edge (y, z) is accepted only if z is the target's next state
 * from y, so the accepted set is one path; coupled noise at T > 0); SimSD
 * summary section 2 (in a block state, the mask slot of an undecided
 * position sees the committed data tokens and the undecided mask slots).
 * Readings (the pages give neither a layout nor the target's choice of
 * position):
 *  - Tree of a sequence: E edges (0 <= E <= 63) over B positions
 *    (1 <= B <= 64); edge e hangs under node parent[e] + 1 (parent[e] = -1:
 *    the root, the block state before the pass; parent[e] < e) and commits
 *    position pos[e] (undecided there) with token token[e].  Node 0 is the
 *    root, node e + 1 the child of edge e.
 *  - Query rows at q_off: the N fresh prompt rows, then one mask-slot row per
 *    position p (its query is the same in every state).  New key / value rows
 *    at k_off: the N fresh rows, one data row per edge, one mask row per
 *    position.  Output rows at o_off: the N fresh rows (causal over cache and
 *    fresh prompt), then node-major rows (n, p), n = 0..E, p = 0..B-1: row
 *    (n, p), for p undecided at node n, is mask slot p attending the whole
 *    prompt, the data rows of the edges on the path root -> n and the mask
 *    rows of the positions undecided at n.  Rows of committed positions are
 *    not written.  A chain of edges in stage order gives SimSD's mask rows.
 *  - Target transition from node n: for each undecided p the decision token
 *    dec(n, p) of logits row (n, p) (argmax, or coupled-noise argmax with the
 *    noise row of position p) and its confidence l[dec] - logsumexp(l)
 *    (log-probability under softmax(l)); the most confident position wins
 *    (ties: the lowest).  The walk from the root follows the child edge
 *    carrying that (position, token) (the lowest such edge) while there is
 *    one, and emits the transition where there is none; a node with no
 *    undecided position ends the walk with nothing emitted.
 * Every kernel checks each sequence's extents and tree on the device; a
 * sequence that fails is skipped (its outputs are not written; the
 * acceptance sets n_acc = -1) and SSV_ERR_INVALID is reported.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t cache_len;  /* C >= 0 */
  int32_t new_len;    /* N >= 0 */
  int32_t block;      /* B, 1 <= B <= 64 */
  int32_t n_edges;    /* E, 0 <= E <= 63 */
  int32_t q_off;      /* N + B query rows */
  int32_t k_off;      /* N + E + B new key / value rows */
  int32_t kv_off;     /* C cache rows */
  int32_t edge_off;   /* E entries of parent / pos / token */
  int32_t o_off;      /* N + (E + 1) B output rows (and logits rows) */
} ssv_tree_seq;

/* ssv_tree_verify_attn -- the attention of the tree pass.
 * q [total_q, Hq, d], k_new / v_new [total_k, Hkv, d], k_cache / v_cache
 * [total_cache, Hkv, d] device, in_dtype (post-RoPE); o [total_out, Hq, d]
 * device, out_dtype.  parent, pos [total_edges] int32 device.  Sequences in
 * increasing q_off order.  d in {64, 128}, Hq % Hkv == 0, pointers 16-byte
 * aligned; max_cache bounds every C.
 * The part every row shares -- the prompt (cache + fresh rows), the same keys
 * for a mask slot at every node -- is computed once per query row: for bf16
 * inputs with d = 128 on the tensor cores (the verify attention's schedule
 * in a prompt-only form, bf16 P and fp32 accumulation as there), which then
 * leaves each row's normalised output and log-sum-exp in the workspace; a
 * node kernel (fp32) continues that softmax over each node's tail keys.
 * Other inputs run the prompt part in the node kernel itself (fp32 SIMT).
 * Workspace: ssv_tree_verify_attn_workspace bytes (0 when the prompt part
 * runs in fp32), 256-byte aligned, all-zero before its first use and left
 * reusable (as for ssv_verify_attn).
 * Errors: SSV_ERR_INVALID, SSV_ERR_UNSUPPORTED, SSV_ERR_WORKSPACE,
 * SSV_ERR_CUDA; on device SSV_ERR_INVALID (see above). */
typedef struct {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const void* k_new;
  const void* v_new;
  void* o;
  ssv_dtype in_dtype;
  ssv_dtype out_dtype;
  int32_t Hq, Hkv, d;
  float scale;                 /* 0 => 1/sqrt(d) */
  const ssv_tree_seq* seqs;    /* device [batch] */
  int32_t batch;
  const int32_t* parent;       /* device [total_edges] */
  const int32_t* pos;          /* device [total_edges] */
  int32_t total_q, total_k, total_cache, total_edges, total_out;
  int32_t max_cache;
  int32_t* dev_status;         /* device, may be NULL */
} ssv_tree_attn_args;

SSV_API ssv_status ssv_tree_verify_attn_workspace(const ssv_tree_attn_args* a, size_t* bytes);
SSV_API ssv_status ssv_tree_verify_attn(const ssv_tree_attn_args* a, void* workspace, size_t workspace_bytes,
                                        void* stream);

/* ssv_tree_accept -- acceptance of the tree by state equality.
 * logits [total_out, V] device (row (n, p) of sequence b at o_off + N + n B + p,
 * the numbering of the attention's output rows; fresh rows are not read).
 * mode SSV_ACCEPT_ARGMAX or SSV_ACCEPT_GUMBEL (coupled noise: the table row of
 * position p of sequence b is noise_row[pos_off[b] + p]; T = 0 means argmax).
 * parent, pos, token [total_edges] int32 device.
 * Outputs (device): n_acc [batch] (accepted edges, -1 for a rejected
 * sequence); path [batch * 64] (the accepted edges' ids within the sequence,
 * root first, -1 padded); emit_pos, emit_tok [batch] (the target's
 * transition where the walk stopped, -1 if none).
 * Workspace: ssv_tree_accept_workspace bytes, 256-byte aligned (no state is
 * kept between calls).  Errors: SSV_ERR_INVALID, SSV_ERR_NOT_FINITE,
 * SSV_ERR_WORKSPACE, SSV_ERR_CUDA; on device SSV_ERR_INVALID. */
typedef struct {
  ssv_accept_mode mode;
  float T;
  int32_t V;
  const ssv_tree_seq* seqs;    /* device [batch] */
  int32_t batch;
  ssv_dtype logits_dtype;
  const void* logits;
  const int32_t* parent;
  const int32_t* pos;
  const int32_t* token;
  int32_t total_edges;
  int32_t total_out;
  const float* noise;          /* [n_noise_rows, V] fp32 (GUMBEL, T > 0) */
  int32_t n_noise_rows;
  const int32_t* noise_row;    /* [total_positions] */
  const int32_t* pos_off;      /* [batch] */
  int32_t total_positions;
  int32_t* n_acc;
  int32_t* path;
  int32_t* emit_pos;
  int32_t* emit_tok;
  int32_t* dev_status;         /* device, may be NULL */
} ssv_tree_accept_args;

SSV_API ssv_status ssv_tree_accept_workspace(const ssv_tree_accept_args* a, size_t* bytes);
SSV_API ssv_status ssv_tree_accept(const ssv_tree_accept_args* a, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* ------------------------------------------------------------------------
 * The paged 8-bit KV cache: four operators of a serving loop whose cache is
 * held in e4m3 pages, in the order a pass calls them (SimSD summary, "Main
 * contributions" 3: the method composes with a KV cache; the pages give no
 * cache layout, so the layout is this library's own):
 *   ssv_page_plan       lengths of the requests -> page table, sequence table, slot map
 *   ssv_norm_rope_copy  RMS norm of every query / key head and ssv_rope_copy in one pass
 *   ssv_verify_attn_fp8 ssv_verify_attn with the cached keys read from the pages
 *   ssv_commit_fp8      ssv_commit into the pages, quantising
 *
 * Cache: k_cache, v_cache [n_pages, Hkv, page_size, d] device, e4m3 codes
 * (one byte each); k_scale, v_scale [n_pages, Hkv] device fp32.  A code c of
 * (page, head) stands for c * scale[page][head].  page_size in {16, 32, 64,
 * 128}.  Page table: pages [table_len] device int32; token t of sequence b
 * sits in row t mod page_size of page pages[seqs[b].kv_off + t / page_size].
 * An all-zero-length record (new_len = block = 0, as ssv_page_plan writes for
 * an ended or refused request) is idle: ssv_norm_rope_copy,
 * ssv_verify_attn_fp8 and ssv_commit_fp8 skip it without an error.
 * ---------------------------------------------------------------------- */

/* ------------------------------------------------------------------------
 * ssv_page_plan -- the tables of a pass from the lengths of its requests,
 * built on the device (lengths known only there, such as ssv_commit_fp8's
 * new_len, never travel to the host; ssv_commit_fp8 is then given cache_len,
 * from which the requests that this call leaves idle keep their lengths).
 * Per request b, in batch order (all arrays device int32):
 *   cache_len[b] < 0: the request has ended.  The held[b] pages at the front
 *     of its table row go back to the free stack (table order), held_out = 0,
 *     no rows, an idle record.
 *   otherwise C = cache_len, N = new_len, B = block: it needs
 *     ceil((C + N + B) / page_size) pages, enough for every row the pass may
 *     commit, and wants those beyond the held[b] it has.  Rows of requests
 *     are packed: q_off and tau_off (also slot_off) are the sums of N + 2B
 *     and B over the earlier requests that have not ended.
 * The free stack is free_list[0 .. n_free) with the released pages pushed on
 * top; wanted pages are taken from its top in (request, page) order and
 * entered in the table row.  A request whose wanted pages, with those wanted
 * before it, exceed the stack is refused (SSV_ERR_NO_PAGES; so is every later
 * one that wants pages): it keeps its place in the packing and its held
 * pages, takes none, and gets an idle record.
 * Outputs: seqs [batch] (kv_off = b * max_pages); slot_map [total_rows]: for
 * row q_off + j, j < N + B, of a granted request the cache row page *
 * page_size + offset of token C + j, -1 at mask rows and at every row of
 * [0, total_rows) that is no granted request's (tokens are appended in stage
 * order: the entry at j = N + s - 1 is where ssv_commit_fp8 puts the data row
 * of stage s, not that of slot s; a caller that stores rows itself looks up
 * slot k at j = N + tau(k) - 1); slot_off [batch]; held_out [batch];
 * n_free_out [1].  pages and free_list are updated in place, at
 * entries that the call does not read otherwise; held and n_free are not
 * written, so a pass that fails can be planned again from them.
 * pages [batch, max_pages]; free_list [n_pages]; 1 <= batch <= 4096 (a call
 * with batch 0 writes nothing);
 * n_pages * page_size < 2^31; page_size in {16, 32, 64, 128}.  held_out and
 * n_free_out must not overlap any input.  held[b] of an ended request and
 * the table's entries are trusted to name distinct pages.
 * Errors: SSV_ERR_INVALID, SSV_ERR_UNSUPPORTED (batch), SSV_ERR_CUDA; on
 * device SSV_ERR_INVALID for a request with N < 0, B outside 1..64, held
 * outside 0..max_pages, more than max_pages pages needed, or rows beyond
 * total_rows (it takes no pages and gets an idle record; unless only its
 * rows do not fit, it takes no rows either), for n_free outside 0..n_pages
 * (taken as 0), and for a released stack that outgrows n_pages (the excess is
 * dropped); SSV_ERR_NO_PAGES.
 * ---------------------------------------------------------------------- */
typedef struct {
  const int32_t* cache_len;    /* device [batch]; < 0: ended */
  const int32_t* new_len;      /* device [batch] */
  const int32_t* block;        /* device [batch] */
  const int32_t* held;         /* device [batch] */
  int32_t* pages;              /* device [batch, max_pages], in and out */
  int32_t* free_list;          /* device [n_pages], in and out */
  const int32_t* n_free;       /* device [1] */
  int32_t batch, max_pages, page_size, n_pages, total_rows;
  ssv_seq* seqs;               /* device [batch], out */
  int32_t* slot_map;           /* device [total_rows], out */
  int32_t* slot_off;           /* device [batch], out */
  int32_t* held_out;           /* device [batch], out */
  int32_t* n_free_out;         /* device [1], out */
  int32_t* dev_status;         /* device, may be NULL */
} ssv_page_plan_args;

SSV_API ssv_status ssv_page_plan(const ssv_page_plan_args* a, void* stream);

/* ------------------------------------------------------------------------
 * ssv_norm_rope_copy -- RMS norm of each query and key head and the rotation
 * of ssv_rope_copy, in one pass over the rows.  For head row x of width d:
 *   y = x / sqrt(mean(x_i^2) + eps) * weight      (weight: q_weight or k_weight)
 * then the rotation of y at the row's position, as ssv_rope_copy (same
 * positions, same optional table).  Computed in fp32, rounded once, to dtype;
 * angles are formed mod one turn in 64-bit fixed point.
 * q_in, q_out [total_rows, Hq, d], k_in, k_out [total_rows, Hkv, d] device,
 * dtype; the heads of a row are contiguous, consecutive rows *_stride
 * elements apart (0: Hq * d or Hkv * d), so that the inputs may be parts of a
 * fused projection's output.  An output may be its own input (same address
 * and stride), and overlaps no other argument.
 * q_weight, k_weight [d] device, dtype.  eps >= 0 finite.  d in {64, 128};
 * pointers 16-byte aligned, strides a multiple of 16 bytes.
 * Errors and device checks as ssv_rope_copy (idle records are skipped).
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* q_in;
  const void* k_in;
  void* q_out;
  void* k_out;
  const void* q_weight;
  const void* k_weight;
  int64_t q_in_stride, k_in_stride, q_out_stride, k_out_stride;  /* elements; 0: packed */
  ssv_dtype dtype;
  int32_t Hq, Hkv, d;
  float eps;
  double base;                 /* RoPE base, e.g. 10000 */
  const ssv_seq* seqs;         /* device */
  int32_t batch;
  int32_t total_rows;
  const int32_t* positions;    /* device [total_rows] or NULL, as ssv_rope_copy */
  int32_t* dev_status;         /* device, may be NULL */
} ssv_norm_rope_args;

SSV_API ssv_status ssv_norm_rope_copy(const ssv_norm_rope_args* a, void* stream);

/* ------------------------------------------------------------------------
 * ssv_verify_attn_fp8 -- ssv_verify_attn (same rows, same mask, same
 * grouped heads) with the C cached keys and values of a sequence read from
 * e4m3 pages; the fresh rows k_new, v_new stay bf16.
 * q, o [total_rows, Hq, d] bf16 device, packed; k_new, v_new [total_rows,
 * Hkv, d] bf16 device, rows k_stride / v_stride elements apart (0: Hkv * d).
 * Scores, softmax statistics and the accumulation of O are fp32.  Rounded to
 * fewer bits on the way: the queries of cached keys, to two e4m3 parts (2^-18
 * of a row's largest element); the weights, to fp16 over cached keys (2^-11,
 * or 2^-32 of the row's largest where that is more) and bf16 over fresh ones
 * (2^-8), the sum that divides them being that of the unrounded ones; a cached
 * value times its scale, to fp16 (below).
 * A sequence's own fresh rows must be finite (a masked non-finite value row
 * still meets a zero weight).  A query (row, head) with an infinity or NaN
 * gives NaN in its own row of o alone.  Rows of other sequences, rows of a
 * page behind token C - 1 and pages that are not a sequence's own never
 * influence it, whatever they hold.  scales: positive and finite.  A cached
 * value times its scale enters as a 16-bit float beside the largest scale met
 * so far in its unit of work, or beside 2^-59 where that is larger: exactly
 * for scales that are powers of two, as ssv_commit_fp8 writes them, down to
 * 2^-20 of it, within 2^-30 of it below.  Beside value scales above 2^96,
 * weights of fresh keys below 2^-42 of the row's largest count as none (below
 * 2^-11 at the largest scale, 2^127).  Sums of weights times fresh values beside
 * cached values of less than 2^-59 have to stay below 2^48.
 * d = 128; Hq % Hkv == 0, Hq / Hkv <= 128; 1 <= B <= 64; n_pages * Hkv *
 * page_size < 2^31; pointers 16-byte aligned, strides multiples of 8.
 * max_cache / max_new / max_block as ssv_verify_attn.  scale 0 means
 * 1/sqrt(d).  o overlaps no input (checked for q, k_new and v_new).
 * Workspace: ssv_verify_attn_fp8_workspace bytes, 256-byte aligned, zero
 * before its first use; it serves calls of any sizes that ask for no more
 * (see the conventions).
 * Errors: SSV_ERR_INVALID, SSV_ERR_UNSUPPORTED (d, heads), SSV_ERR_WORKSPACE,
 * SSV_ERR_CUDA; on device SSV_ERR_BAD_TAU, SSV_ERR_TIMEOUT, and
 * SSV_ERR_INVALID for a sequence outside the buffers or with a page outside
 * [0, n_pages) among its first ceil(C / page_size) (skipped: its rows of o
 * are unspecified).  SSV_ERR_UNSUPPORTED also where the plan could pass 32
 * bits: more than 2^30 / 12 blocks for total_rows / 64 + batch tiles of rows (64
 * at a group of four) of the longest sequence that max_cache, max_new and
 * max_block allow.  Where batch such sequences would pass it, sequences have
 * to be in order without shared rows, which is then checked on the device.
 * Scheduling as ssv_verify_attn: one CTA per SM, and where a unit of work is
 * split the CTA with its first key block waits (bounded) for the others.
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* q;
  const void* k_cache;         /* e4m3 [n_pages, Hkv, page_size, d] */
  const void* v_cache;
  const float* k_scale;        /* [n_pages, Hkv] */
  const float* v_scale;
  const int32_t* pages;        /* [table_len] */
  const void* k_new;
  const void* v_new;
  void* o;
  int64_t k_stride, v_stride;  /* elements; 0: packed */
  int32_t Hq, Hkv, d, page_size, n_pages, table_len;
  float scale;
  const ssv_seq* seqs;         /* device [batch]; kv_off: first entry in pages */
  int32_t batch;
  const int32_t* tau;          /* device [total_slots] */
  int32_t total_rows, total_slots;
  int32_t max_cache, max_new, max_block;
  int32_t* dev_status;         /* device, may be NULL */
} ssv_attn_fp8_args;

SSV_API ssv_status ssv_verify_attn_fp8_workspace(const ssv_attn_fp8_args* a, size_t* bytes);
SSV_API ssv_status ssv_verify_attn_fp8(const ssv_attn_fp8_args* a, void* workspace, size_t workspace_bytes,
                                       void* stream);

/* ------------------------------------------------------------------------
 * ssv_commit_fp8 -- ssv_commit into the pages: tokens C .. C + N + n_acc - 1
 * (the fresh prompt rows, then the data rows of stages 1..n_acc in stage
 * order) are quantised and appended.  For each touched (page, head), K and V
 * apart:
 *   s_new = 2^e, e the smallest integer >= -100 with max |x| <= 448 * 2^e over
 *           the finite x appended to the page
 *   s     = max(s_old, s_new) where the page already holds tokens of the
 *           sequence (its first page, C mod page_size > 0), else s_new
 *   codes of appended rows: x / s rounded to the nearest e4m3 (ties to even),
 *           NaN and infinities stored as NaN
 *   codes of rows already there: code * s_old / s rounded likewise, when s grew
 * A power-of-two scale costs an 8-bit float no precision, makes x / s exact
 * and a later rescale exact but for values that fall below 2^-6 s.  Where the
 * caller has left another positive scale, x * (1 / s) and code * (s_old / s)
 * are formed in fp32 before they are rounded.  Rows behind the last appended
 * token are left as they were.
 * k_new, v_new [total_rows, Hkv, d] device, dtype (SSV_F32 or SSV_BF16), rows
 * k_stride / v_stride elements apart (0: Hkv * d).  seqs, tau, n_acc, new_len
 * and their checks as ssv_commit; kv_off is the sequence's first entry in
 * pages [table_len].  d in {64, 128} (ssv_verify_attn_fp8 reads 128 alone); 1 <= max_new + max_block bounds every
 * N + B (sizes the grid); pointers 16-byte aligned, strides a multiple of 16
 * bytes.  No two touched pages may be the same page (not checked).
 * Errors: SSV_ERR_INVALID, SSV_ERR_UNSUPPORTED (d), SSV_ERR_CUDA; on device
 * SSV_ERR_BAD_TAU and SSV_ERR_INVALID as ssv_commit, also for a sequence
 * whose rows leave [0, total_rows), whose N or B exceeds max_new or max_block,
 * whose touched pages leave the table or name a page outside [0, n_pages):
 * nothing of that sequence is written.
 * new_len[b]: C + N + n_acc of a sequence that was appended to.  Of any other
 * -- an idle record, a rejected sequence -- cache_len[b] where the lengths
 * that ssv_page_plan was given are passed on (device [batch], may be new_len
 * itself): a request that got no pages keeps its length, an ended one stays
 * ended, and a rejected one keeps its tokens (dev_status tells).  Without
 * them: the record's cache_len (0 in ssv_page_plan's idle records) and -1; a
 * loop that feeds new_len to its next ssv_page_plan has to pass them.
 * No workspace; asynchronous on `stream`.
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* k_new;
  const void* v_new;
  void* k_cache;               /* e4m3 [n_pages, Hkv, page_size, d], in and out */
  void* v_cache;
  float* k_scale;              /* [n_pages, Hkv], in and out */
  float* v_scale;
  const int32_t* pages;        /* [table_len] */
  int64_t k_stride, v_stride;  /* elements; 0: packed */
  ssv_dtype dtype;
  int32_t Hkv, d, page_size, n_pages, table_len;
  const ssv_seq* seqs;         /* device [batch] */
  int32_t batch;
  const int32_t* tau;          /* device [total_slots] */
  const int32_t* n_acc;        /* device [batch] */
  int32_t* new_len;            /* device [batch], out */
  int32_t total_rows, total_slots;
  int32_t max_new, max_block;
  int32_t* dev_status;         /* device, may be NULL */
  const int32_t* cache_len;    /* device [batch], may be NULL: lengths before the pass */
} ssv_commit_fp8_args;

SSV_API ssv_status ssv_commit_fp8(const ssv_commit_fp8_args* a, void* stream);

/* ------------------------------------------------------------------------
 * What else a pass's logits give.  ssv_accept decides on the target's rows;
 * the three entry points below return the log-probabilities that a server
 * reports beside the tokens, and train a drafter on the target's answers (the
 * SPOT review's order predictor reads the top 32 probabilities and summary
 * statistics per slot; the DFlash review weighs a draft position's loss by
 * exp(-(k - 1) / gamma), section 3.1; neither page gives an interface).
 * Rows: logits [rows, V] device, SSV_F32 or SSV_BF16, rows logits_stride
 * elements apart (0: V; at least V), at any element-aligned address; rows that
 * start on 16-byte boundaries are fastest.  1 <= V <= 524288.  T: positive
 * and finite.  No workspace; sums and results are the same from call to call.
 * -inf marks a token that cannot be: it has probability 0.  A result beyond
 * fp32's range (the lse of a row at the type's lowest number, T < 1) is infinite,
 * and so is a difference of two logits of a row beyond it, whatever T: the lower
 * one then has probability 0 and log-probability -inf, as one of -inf.
 * ---------------------------------------------------------------------- */

/* ------------------------------------------------------------------------
 * ssv_logprobs -- log-probabilities of given tokens under softmax(l / T), their
 * ranks, each row's entropy and its top alternatives.
 * Entry i (0 <= i < n) has the logits row rows[i] (NULL: i) and the token
 * tokens[i] (NULL: none is asked for).  An entry with token -1 (as ssv_accept
 * leaves behind the last emitted token) or row -1 is idle: its row is not read,
 * and logprob, rank, entropy, lse are 0, its alternatives absent.
 *   lse[i]     = ln sum_v exp(l_v / T)
 *   logprob[i] = l_t / T - lse
 *   rank[i]    = 1 + number of tokens before t in the order of the logits
 *                (descending, equal ones by index)
 *   entropy[i] = - sum_v p_v ln p_v (nats; tokens of probability 0 add nothing)
 *   top_token[i][0..top_k), top_logprob[i][..]: the first top_k tokens of that
 *                order with logits above -inf, and their log-probabilities;
 *                where there are fewer, -1 and -inf.
 * Tokens in the order of the stages, as ssv_accept writes them, have the row
 * of slot k at entry slot_off + tau(k) - 1.
 * Sums are fp32, per thread and joined in a fixed order; logprob, lse and entropy
 * are formed from them in 48 bits and rounded once, top_logprob in fp32.
 * A row with a NaN or +inf gives NaN in logprob, entropy, lse and top_logprob;
 * NaN logits are in no order (never listed, never before another; the rank of
 * such a token is 0).  A row of nothing but -inf gives lse = logprob = -inf,
 * entropy 0 and no alternatives.
 * Mask with -inf where alternatives are asked for: where a row has more than 512
 * elements equal to its top_k-th largest (masked with a number, with fewer tokens
 * left than top_k; or all equal), that one is searched for by reading the row some
 * fifty times (milliseconds for 151936 tokens instead of microseconds).
 * tokens given: logprob is not NULL; not given: logprob and rank are NULL.
 * rank, entropy, lse may be NULL.  0 <= top_k <= 128; top_logprob, top_token
 * [n, top_k] (NULL for 0).  Outputs overlap no input
 * (checked for the logits).
 * Errors: SSV_ERR_INVALID, SSV_ERR_NOT_FINITE (T), SSV_ERR_UNSUPPORTED (V,
 * top_k), SSV_ERR_CUDA; on device SSV_ERR_INVALID for a row outside
 * [-1, total_rows) or a token outside [-1, V) (that entry is taken as idle).
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* logits;          /* [total_rows, V] */
  int64_t logits_stride;       /* elements; 0: V */
  ssv_dtype dtype;
  int32_t V;
  int32_t total_rows;
  const int32_t* rows;         /* device [n] or NULL */
  const int32_t* tokens;       /* device [n] or NULL */
  int32_t n;
  int32_t top_k;
  float T;
  float* logprob;              /* device [n] */
  int32_t* rank;               /* device [n] or NULL */
  float* entropy;              /* device [n] or NULL */
  float* lse;                  /* device [n] or NULL */
  float* top_logprob;          /* device [n, top_k] */
  int32_t* top_token;          /* device [n, top_k] */
  int32_t* dev_status;         /* device, may be NULL */
} ssv_logprobs_args;

SSV_API ssv_status ssv_logprobs(const ssv_logprobs_args* a, void* stream);

/* ------------------------------------------------------------------------
 * ssv_distill, ssv_distill_backward -- distillation of a drafter from the
 * target's top alternatives: the loss, or the loss and its gradient in one
 * call, and the gradient for given upstream gradients.
 * Row i: drafter logits z [V], weight w = weight[i] (NULL: 1), and K listed
 * tokens teacher_token[i][j] with values t_j = teacher_logprob[i][j], as
 * ssv_logprobs writes them (at the same T).  Token -1 is absent; one listed
 * more than once counts with the sum of its probabilities.
 *   SSV_DISTILL_RENORM: p_j = exp(t_j) / sum exp(t), r = 0 (so that logits
 *                       divided by T serve as well as log-probabilities)
 *   SSV_DISTILL_REST:   p_j = exp(t_j), r = max(0, 1 - sum p): the target's
 *                       probability of all other tokens together (where the drafter
 *                       leaves them nothing, each being -inf or more than 100 T below
 *                       the row's largest logit as a masked one is, an r below 2^-20,
 *                       left by the roundings of t, counts as 0)
 *   q = softmax(z / T), u = sum of q over the tokens that are not listed
 *   loss[i] = w [ sum_j p_j (ln p_j - ln q_j) + r (ln r - ln u) ]
 * (terms of probability 0 add nothing), the divergence of q from p with the
 * other tokens as one; its gradient with P = sum p + r:
 *   d loss / d z_v = (w / T) (P q_v - p_v)            v listed
 *                    (w / T) (P q_v - r q_v / u)      v not listed
 * ssv_distill: writes loss [n]; stats [n, 4] (may be NULL), each row's
 * (m, S, m', S'): m = max z, S = sum exp((z - m) / T), and the same over the
 * tokens that are not listed (lse = m / T + ln S; -inf and 0 where there is
 * nothing above -inf); and, where grad is given, the gradient of
 * sum_i loss[i].  grad_loss is NULL.
 * ssv_distill_backward: takes stats as written by ssv_distill on the same
 * arguments and grad_loss [n] (NULL: 1), writes grad, row i times grad_loss[i].
 * loss is not used (may be NULL).
 * grad [n, V] device in the logits' dtype, rows grad_stride elements apart
 * (0: V).  It may be the logits themselves (same address and stride), and
 * overlaps no other argument; fastest where its rows lie to 16-byte boundaries
 * as the logits' do.  Elements between rows are not written.
 * A row of weight 0 is not read: its loss, statistics and gradient are 0.
 * A row with a NaN (or +inf) in its logits, or a NaN in its target, gives NaN in
 * its loss and gradient.  A listed token with p > 0 and logit -inf, or r > 0 with
 * u = 0, gives the loss +inf (the gradient stays finite); so does a row of nothing
 * but -inf, whose gradient is 0 whatever its target.  Any other row whose listed
 * tokens are all absent has the loss and gradient 0.
 * Sums over a row are fp32 per thread and joined in 48 bits; u is summed from the
 * tokens that are not listed; the loss, a small difference of logarithms, is
 * formed in 48 bits and rounded once.  The gradient is formed in fp32, from r and
 * the exponent of u to 48 bits, and rounded once.
 * 1 <= K <= 128.
 * Errors: SSV_ERR_INVALID, SSV_ERR_NOT_FINITE (T), SSV_ERR_UNSUPPORTED (V, K),
 * SSV_ERR_CUDA; on device SSV_ERR_INVALID for a listed token outside [-1, V)
 * (taken as absent).
 * ---------------------------------------------------------------------- */
typedef enum { SSV_DISTILL_RENORM = 0, SSV_DISTILL_REST = 1 } ssv_distill_mode;

typedef struct {
  const void* logits;          /* [n, V] */
  int64_t logits_stride;       /* elements; 0: V */
  ssv_dtype dtype;
  int32_t V;
  int32_t n;
  int32_t K;
  const int32_t* teacher_token;    /* device [n, K] */
  const float* teacher_logprob;    /* device [n, K] */
  float T;
  ssv_distill_mode mode;
  const float* weight;         /* device [n] or NULL */
  float* loss;                 /* device [n] */
  float* stats;                /* device [n, 4] */
  const float* grad_loss;      /* device [n] or NULL (ssv_distill_backward) */
  void* grad;                  /* [n, V], dtype */
  int64_t grad_stride;         /* elements; 0: V */
  int32_t* dev_status;         /* device, may be NULL */
} ssv_distill_args;

SSV_API ssv_status ssv_distill(const ssv_distill_args* a, void* stream);
SSV_API ssv_status ssv_distill_backward(const ssv_distill_args* a, void* stream);

/* ------------------------------------------------------------------------
 * ssv_set_fault_injection -- test support for failure detection.
 * The pages have no counterpart: this lets a test make a bounded device wait
 * run out without faulting, trapping or hanging the GPU.  For the chosen
 * kernel -- the tensor-core attentions (SSV_FAULT_ATTN: ssv_verify_attn and
 * ssv_verify_attn_fp8, where the copy is that of a key block), the streaming
 * acceptance reduce (SSV_FAULT_ACCEPT) or the fused LM head's GEMM
 * (SSV_FAULT_LMHEAD) -- every bounded wait gives up after
 * wait_budget_cycles SM cycles instead of about one second, and, if
 * skip >= 0, CTA 0 leaves out one asynchronous copy: its skip-th key block
 * (attention), its skip-th vocabulary chunk (acceptance) or its skip-th
 * operand stage (LM head), so that the wait for that copy runs out.  The
 * kernel then drains every copy and MMA it issued (bounded), releases its
 * tensor memory, writes SSV_ERR_TIMEOUT to dev_status and returns; its
 * outputs are unspecified and its workspace counters must be cleared before
 * the workspace is used again (as after any SSV_ERR_TIMEOUT).
 * The setting is process-wide and applies to every later launch of that
 * kernel from every host thread, until reset with NULL.  For tests only.
 * f: kernel in SSV_FAULT_NONE..SSV_FAULT_LMHEAD, skip >= -1,
 *    1000 <= wait_budget_cycles <= 2^31.  Errors: SSV_ERR_INVALID.
 * ---------------------------------------------------------------------- */
typedef enum {
  SSV_FAULT_NONE = 0,
  SSV_FAULT_ATTN = 1,
  SSV_FAULT_ACCEPT = 2,
  SSV_FAULT_LMHEAD = 3
} ssv_fault_kernel;

typedef struct {
  ssv_fault_kernel kernel;
  int32_t skip;                /* index of the copy CTA 0 leaves out, or -1 */
  int64_t wait_budget_cycles;  /* budget of every bounded wait of that kernel */
} ssv_fault_injection;

SSV_API ssv_status ssv_set_fault_injection(const ssv_fault_injection* f);

/* ------------------------------------------------------------------------
 * Status and utilities
 * ---------------------------------------------------------------------- */
/* Waits for `stream`, reads the device status word, resets it to 0 and
 * returns it (SSV_OK if dev_status is NULL). */
SSV_API ssv_status ssv_get_status(int32_t* dev_status, void* stream);

SSV_API const char* ssv_status_string(ssv_status s);

/* Library build identification, e.g. "ssv 0.2 sm_103a". */
SSV_API const char* ssv_version(void);

/* ------------------------------------------------------------------------
 * ssv_bench -- native timing of the library on a named synthetic workload
 * ("tiny", "gqa1p7b", "gqa8b", "prefill", "sweep").  Allocates its own
 * device buffers (this is not a hot-path call), fills them with a
 * counter-hash generator, runs `iters` timed iterations per op with an L2
 * flush between them and writes one JSON object (median/p10/p90 times,
 * algorithmic bytes and FLOPs) into json_out.  The DFlash review's latency
 * model L = (T_draft + T_verify) / tau needs T_verify; this reports it.
 * Errors: SSV_ERR_INVALID (unknown config, short buffer), SSV_ERR_CUDA.
 * ---------------------------------------------------------------------- */
SSV_API ssv_status ssv_bench(const char* config, int32_t iters, char* json_out, size_t json_len);

/* ------------------------------------------------------------------------
 * ssv_stream_read -- the measurement reference for a memory-bound kernel
 * of the path: reads `bytes` at device address `buf` once (16-byte loads,
 * two CTAs per SM, each a contiguous range) and XORs every word read into
 * *out (device address; a checksum that keeps the loads live, not a result
 * of the method).  Timed like the kernel it is compared with (same L2
 * flush, same launch mode), it gives the achievable time for reading those
 * bytes, launch and first-byte latency included; on small workloads that is
 * well above bytes / peak bandwidth.  Not a hot-path call.  buf must be
 * 16-byte aligned and bytes a multiple of 16.  Asynchronous on `stream`.
 * Errors: SSV_ERR_INVALID (null or misaligned arguments), SSV_ERR_CUDA.
 * ---------------------------------------------------------------------- */
SSV_API ssv_status ssv_stream_read(const void* buf, size_t bytes, uint32_t* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSV_H_ */
