/*
 * msa.h -- C ABI of libmsa.so: MiniMax-M3 MSA block-sparse attention on one
 * NVIDIA GB300 (sm_103a).
 *
 * What the library computes is defined on these pages:
 *   "MiniMax-M3.1-Flash" (miles docs), section 1 "Model Introduction":
 *       a 4-head indexer (dim 128, its own gemma q/k norm and RoPE) scores every
 *       causal 128-token key block by its maximum logit; each query attends to
 *       the 16 best blocks, its own block always included; index head h picks
 *       the blocks of KV head h.  Attention is GQA, 64 query / 4 KV heads of
 *       dim 128, with per-head gemma q/k norm and RoPE on the first 64 dims
 *       (base 1e7).
 *   same page, section 5.1 "Parallelism": the sparse attention runs on
 *       THD-packed sequences (cu_seqlens).
 *   same page, section 5.4 "Notable quirks": the indexer is frozen, so the
 *       block selection gets no gradient.
 *   "[1/4] Add MiniMax-M3 support - #4581" (radixark/miles), "Kernel tuning":
 *       per-block max-logit scores, top-k select, forward and dQ/dK/dV
 *       backward of the block-sparse attention kernel.
 *   "MiniMax-M3" (Megatron-Bridge docs), "Architecture Notes": Gemma-style
 *       RMSNorm x * (1 + w); "Known Limitations": 16 x 128 = 2048 keys per
 *       query, so the method equals full causal attention up to that length.
 *
 * Conventions shared by every call
 *   - Every pointer argument is a DEVICE pointer (cudaMalloc / torch CUDA
 *     tensor memory), 16-byte aligned, contiguous in the stated layout, on
 *     the device that is current when the call is made.
 *   - bf16 means IEEE bfloat16 (2 bytes); compute is fp32 inside the kernels.
 *   - D (head dim) is 128, the key block is 128 tokens, top-k is 16, the
 *     rotated part is the first 64 channels: the library rejects other values,
 *     except where a call states its own.
 *   - Packed (THD) inputs: token t of the pack belongs to sequence s with
 *     cu_seqlens[s] <= t < cu_seqlens[s+1]; its position is t - cu_seqlens[s].
 *     Key block b of sequence s covers positions [128 b, 128 b + 128); the last
 *     block of a sequence may be partial.  cu_seqlens is int32 [S + 1] on the
 *     device, cu_seqlens[0] = 0, non-decreasing, cu_seqlens[S] = T, and no
 *     sequence longer than max_seqlen.  The library does not read device
 *     memory on the host, so it cannot verify these contents: kernels clamp
 *     indices and set MSA_STATUS_BOUNDS in the device status word instead of
 *     reading or writing out of range.
 *   - Selected block ids (sel) are int32 [T, H, 16], relative to the start of
 *     the token's sequence, sorted ascending, padded with -1.
 *   - GQA: query head i uses KV head i / (Hq / Hkv).
 *   - Ownership: the caller allocates every buffer, including the workspace
 *     (size from the matching *_workspace_size call, 256-byte aligned).  The
 *     library never allocates or frees device memory and never synchronizes
 *     the stream.  Outputs are fully overwritten.  Two calls that may run at
 *     the same time need distinct workspaces.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default).
 *   - Errors: argument checks run on the host before any launch and return
 *     MSA_ERR_INVALID_ARG / MSA_ERR_UNSUPPORTED with nothing enqueued; a
 *     failed launch returns MSA_ERR_CUDA.  msa_last_error() gives the message
 *     of the calling thread's last failure.  Kernels never trap: a wait that
 *     runs out or an index out of range sets a bit in the device status word,
 *     read (and cleared) by msa_check_status().
 */
#ifndef MSA_H_
#define MSA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MSA_API __attribute__((visibility("default")))
#else
#define MSA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MSA_OK = 0,
  MSA_ERR_INVALID_ARG = 1,  /* bad pointer, size, alignment or workspace */
  MSA_ERR_UNSUPPORTED = 2,  /* a shape the library does not implement */
  MSA_ERR_CUDA = 3,         /* a CUDA runtime call or launch failed */
  MSA_ERR_TIMEOUT = 4,      /* msa_check_status: a kernel wait ran out */
  MSA_ERR_BOUNDS = 5        /* msa_check_status: an index was out of range */
} msa_status_t;

/* A cudaStream_t passed through as an opaque handle. */
typedef void* msa_stream_t;

#define MSA_ABI_VERSION 1

MSA_API int msa_abi_version(void);

/* Message of the calling thread's most recent failed call ("" if none). */
MSA_API const char* msa_last_error(void);

/* Synchronizes `stream`, then reads and clears the device status word of the
 * current device.  MSA_OK if no kernel reported a problem since the last
 * check, MSA_ERR_TIMEOUT or MSA_ERR_BOUNDS otherwise.  Meant for tests and
 * debugging; it blocks the host. */
MSA_API msa_status_t msa_check_status(msa_stream_t stream);

/* Diagnostic of the failure-detection path: launches one kernel on `stream`
 * whose bounded wait on an mbarrier that nothing completes runs out (after the
 * library's wait limit, about 2 s) and sets the timeout bit of the status word,
 * then returns.  No fault is raised and the context stays usable; the next
 * msa_check_status returns MSA_ERR_TIMEOUT (wait site 65535). */
MSA_API msa_status_t msa_selftest_wait(msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Prologue ("MiniMax-M3.1-Flash", 1 "Model Introduction"; "MiniMax-M3",
 * "Architecture Notes").  x bf16 [T, H, 128] -> y bf16 [T, H, 128] (y may be
 * x itself, for an in-place update):
 *   y = x / sqrt(mean(x^2) + eps) * (1 + w)        per (token, head), w bf16 [128]
 *   then channels i and i + rope_dim/2 (i < rope_dim/2) are rotated by the
 *   angle pos * rope_base^(-2 i / rope_dim), pos = the token's in-sequence
 *   position; channels >= rope_dim pass through.  rope_dim must be 64.
 * The four-tensor form runs q [T,Hq,128], k [T,Hkv,128], q_idx and k_idx
 * [T,Hi,128] with their own weights in one launch; same result as four calls.
 * Head counts: 1 <= H <= 256 per tensor (MSA_ERR_INVALID_ARG below,
 * MSA_ERR_UNSUPPORTED above; nothing is enqueued).
 */
MSA_API msa_status_t msa_qk_norm_rope(const void* x, void* y, int T, int H, const void* w,
                                      const int32_t* cu_seqlens, int S, int rope_dim,
                                      float rope_base, float eps, msa_stream_t stream);

MSA_API msa_status_t msa_qk_norm_rope4(const void* q, void* q_out, int Hq, const void* k,
                                       void* k_out, int Hkv, const void* q_idx,
                                       void* q_idx_out, const void* k_idx, void* k_idx_out,
                                       int Hi, const void* w_q, const void* w_k,
                                       const void* w_qi, const void* w_ki,
                                       const int32_t* cu_seqlens, int S, int T, int rope_dim,
                                       float rope_base, float eps, msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Prologue backward (the gradients of msa_qk_norm_rope for one tensor; the
 * indexer's prologue needs none: "MiniMax-M3.1-Flash", 5.4 "Notable quirks").
 * x: the prologue's input, bf16 [T, H, 128]; dy = dL/dy for its output (same
 * shape, e.g. dq or dk from msa_sparse_attn_bwd).  With z = gemma_norm(x, w)
 * and y = RoPE(z):  dz = R^T dy (the rotation turned back), r =
 * 1/sqrt(mean(x^2) + eps), xh = x r, g = dz (1 + w):
 *   dx = r (g - xh mean(g xh))          bf16 [T, H, 128]  (dx may be dy)
 *   dw = sum over tokens and heads of dz * xh     fp32 [128] (overwritten)
 * dw is summed in a fixed order (run to run identical).  Workspace from
 * msa_qk_norm_rope_bwd_workspace_size; other arguments (and the head-count
 * limit 1 <= H <= 256) as for msa_qk_norm_rope.
 */
MSA_API size_t msa_qk_norm_rope_bwd_workspace_size(int T, int H);

MSA_API msa_status_t msa_qk_norm_rope_bwd(const void* x, const void* dy, void* dx, float* dw,
                                          int T, int H, const void* w,
                                          const int32_t* cu_seqlens, int S, int rope_dim,
                                          float rope_base, float eps, void* workspace,
                                          size_t workspace_bytes, msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Prologue for any rotary layout: the norm and the rotation of
 * msa_qk_norm_rope with the head dim (64, 128 or 256, e.g. the narrow-block
 * layers'), the rotated part, the pairing and the frequencies as arguments.
 * Frequencies scaled for contexts beyond the trained length come from
 * msa_rope_init (host only; a rope may also be filled in by hand):
 *   PLAIN   f_i = base^(-2 i / dim), i < dim / 2
 *   LINEAR  f_i / factor                       (positions interpolated)
 *   NTK     base * factor^(dim / (dim - 2)) in place of base
 *   YARN    by parts ("YaRN: Efficient Context Window Extension of Large
 *           Language Models", Peng et al. 2023, 3.2 and 3.3): with t_i = orig_len
 *           f_i / (2 pi) turns over the trained length and k = clamp((t_i -
 *           beta_slow) / (beta_fast - beta_slow), 0, 1): f_i k + f_i / factor (1 - k);
 *           gain 0.1 ln(factor) + 1
 * gain multiplies the rotated channels; 0 in msa_rope_init takes the scaling's
 * own (1 except for YARN).  dim: a multiple of 16, 16 .. 256, at most the head
 * dim.  Layout HALF pairs channels (i, i + dim/2), INTERLEAVED (2i, 2i + 1).
 */
enum { MSA_ROPE_HALF = 0, MSA_ROPE_INTERLEAVED = 1 };
enum { MSA_ROPE_PLAIN = 0, MSA_ROPE_LINEAR = 1, MSA_ROPE_NTK = 2, MSA_ROPE_YARN = 3 };

typedef struct {
  int32_t dim;        /* rotated channels */
  int32_t layout;     /* MSA_ROPE_HALF or MSA_ROPE_INTERLEAVED */
  float gain;         /* factor of the rotated channels */
  float reserved;
  double freqs[128];  /* angle per position of pair i < dim / 2, in radians */
} msa_rope_t;

MSA_API msa_status_t msa_rope_init(msa_rope_t* rope, int dim, double base, int layout,
                                   int scaling, double factor, double orig_len,
                                   double beta_fast, double beta_slow, double gain);

/* x bf16 [T, H, D] -> y bf16 [T, H, D] (y may be x).  w bf16 [D], or NULL for
 * the rotation alone (z = x).  The position of token t is positions[t] (int32
 * [T], any value) or, with positions NULL, its place in cu_seqlens' sequence;
 * tokens outside [cu_seqlens[0], cu_seqlens[S]) are then left alone.  Channels
 * behind the rotated part take nothing from other channels, whatever those hold, and
 * with w NULL they keep their bits (so does their dx).
 * `rope` is read on the host during the call.  1 <= H <= 256.
 */
MSA_API msa_status_t msa_qk_norm_rope_ex(const void* x, void* y, int T, int H, int D,
                                         const void* w, const int32_t* positions,
                                         const int32_t* cu_seqlens, int S,
                                         const msa_rope_t* rope, float eps,
                                         msa_stream_t stream);

/* Its gradients, as msa_qk_norm_rope_bwd: dx bf16 [T, H, D] (may be dy) and dw
 * fp32 [D] (overwritten; fixed summation order).  With w NULL only dx = the
 * gradient turned back is formed; x, dw and the workspace may then be NULL.
 * Tokens outside the sequences add nothing to dw and have no dx written.
 */
MSA_API size_t msa_qk_norm_rope_bwd_ex_workspace_size(int T, int H, int D);

MSA_API msa_status_t msa_qk_norm_rope_bwd_ex(const void* x, const void* dy, void* dx, float* dw,
                                             int T, int H, int D, const void* w,
                                             const int32_t* positions,
                                             const int32_t* cu_seqlens, int S,
                                             const msa_rope_t* rope, float eps,
                                             void* workspace, size_t workspace_bytes,
                                             msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Index select ("MiniMax-M3.1-Flash", 1 "Model Introduction"; "#4581",
 * "Kernel tuning").  q_idx, k_idx: post-prologue bf16 [T, Hi, 128].
 * For token t at position p and index head h the own block is p / 128; every
 * earlier block b of the sequence is scored by max_j q_idx[t,h] . k_idx[j,h]
 * over its keys (fp32 accumulation); the own block plus the best
 * min(15, own) earlier blocks (equal scores: lower id) are written to
 * sel [T, Hi, 16] (ascending, -1 padded).  topk must be 16.
 */
MSA_API size_t msa_index_select_workspace_size(int T, int S, int Hi, int max_seqlen);

MSA_API msa_status_t msa_index_select(const void* q_idx, const void* k_idx,
                              const int32_t* cu_seqlens, int S, int T, int Hi,
                              int max_seqlen, int topk, int32_t* sel, void* workspace,
                              size_t workspace_bytes, msa_stream_t stream);

/* The same selection with the "init" rule that "#4581" (Kernel tuning) names
 * beside the local and causal rules but does not define.  Read here as: the
 * first n_init blocks of every sequence (those before the token's own block)
 * are always kept; the best of the other earlier blocks fill the remaining
 * 15 - min(n_init, own) slots.  0 <= n_init <= 15; n_init = 0 is
 * msa_index_select.  Workspace: msa_index_select_workspace_size.
 */
MSA_API msa_status_t msa_index_select_ex(const void* q_idx, const void* k_idx,
                                 const int32_t* cu_seqlens, int S, int T, int Hi,
                                 int max_seqlen, int topk, int n_init, int32_t* sel,
                                 void* workspace, size_t workspace_bytes,
                                 msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Block-sparse attention forward ("MiniMax-M3.1-Flash", 1; "#4581").
 * q bf16 [T, Hq, 128]; k, v bf16 [T, Hkv, 128]; sel int32 [T, Hkv, 16].
 * For query head i of token t (KV head g = i / (Hq/Hkv)) the keys are those
 * of the blocks in sel[t, g] at positions <= the query's position:
 *   o[t, i]   = softmax(scale * q k_j) v_j            bf16 [T, Hq, 128]
 *   lse[t, i] = log sum_j exp(scale * q k_j)         fp32 [T, Hq] (natural log)
 * Hq / Hkv must divide 128.
 */
MSA_API size_t msa_sparse_attn_fwd_workspace_size(int T, int S, int Hq, int Hkv, int max_seqlen);

MSA_API msa_status_t msa_sparse_attn_fwd(const void* q, const void* k, const void* v,
                                 const int32_t* sel, const int32_t* cu_seqlens, int S,
                                 int T, int Hq, int Hkv, int max_seqlen, float scale,
                                 void* o, float* lse, void* workspace,
                                 size_t workspace_bytes, msa_stream_t stream);

/* The forward of a training step: msa_sparse_attn_fwd that also zeroes the
 * fp32 accumulators and item counters of `bwd_workspace` (sized by
 * msa_sparse_attn_bwd_workspace_size for the same T, S, Hq, Hkv, max_seqlen)
 * while it runs, by bulk copies from the forward's otherwise idle memory
 * bandwidth.  It stands in for msa_sparse_attn_bwd_prepare: follow it with
 * msa_sparse_attn_bwd_prepared on that workspace (same stream, or an event),
 * writing nothing into the workspace in between. */
MSA_API msa_status_t msa_sparse_attn_fwd_train(const void* q, const void* k, const void* v,
                                               const int32_t* sel, const int32_t* cu_seqlens,
                                               int S, int T, int Hq, int Hkv, int max_seqlen,
                                               float scale, void* o, float* lse,
                                               void* workspace, size_t workspace_bytes,
                                               void* bwd_workspace, size_t bwd_workspace_bytes,
                                               msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Block-sparse attention backward ("#4581", "Kernel tuning"; the selection
 * is constant: "MiniMax-M3.1-Flash", 5.4 "Notable quirks").
 * Inputs as for the forward plus o (bf16, the forward's output), dout (bf16
 * [T, Hq, 128], gradient of the loss w.r.t. o) and lse (fp32 [T, Hq]).
 * With P = exp(scale q k^T - lse) over the attended keys, dP = dout v^T and
 * Delta = rowsum(dout * o):  dS = P * (dP - Delta);
 *   dq = scale dS k  (bf16 [T,Hq,128]),  dk = scale dS^T q,  dv = P^T dout
 *   (bf16 [T,Hkv,128]; sums over all query heads and tokens using the key).
 */
MSA_API size_t msa_sparse_attn_bwd_workspace_size(int T, int S, int Hq, int Hkv, int max_seqlen);

MSA_API msa_status_t msa_sparse_attn_bwd(const void* q, const void* k, const void* v,
                                 const void* o, const void* dout, const float* lse,
                                 const int32_t* sel, const int32_t* cu_seqlens, int S,
                                 int T, int Hq, int Hkv, int max_seqlen, float scale,
                                 void* dq, void* dk, void* dv, void* workspace,
                                 size_t workspace_bytes, msa_stream_t stream);

/* The backward in two parts, so that a caller can clear the workspace's fp32
 * accumulators (about T * (Hq + 2 Hkv) * 512 bytes, one memset) while other
 * work runs, e.g. on a second stream during the forward:
 *   msa_sparse_attn_bwd_prepare  clears them on `stream` (same sizes as the
 *                                backward that follows);
 *   msa_sparse_attn_bwd_prepared is msa_sparse_attn_bwd without the clear.
 * The caller orders the prepare before the prepared call (same stream, or an
 * event) and writes nothing into the workspace in between; the prepared call
 * leaves the accumulators dirty, so every call needs its own prepare.
 * msa_sparse_attn_bwd equals prepare + prepared on one stream.
 */
MSA_API msa_status_t msa_sparse_attn_bwd_prepare(int T, int S, int Hq, int Hkv, int max_seqlen,
                                                 void* workspace, size_t workspace_bytes,
                                                 msa_stream_t stream);

MSA_API msa_status_t msa_sparse_attn_bwd_prepared(const void* q, const void* k, const void* v,
                                                  const void* o, const void* dout,
                                                  const float* lse, const int32_t* sel,
                                                  const int32_t* cu_seqlens, int S, int T,
                                                  int Hq, int Hkv, int max_seqlen, float scale,
                                                  void* dq, void* dk, void* dv, void* workspace,
                                                  size_t workspace_bytes, msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Narrow-block sparse attention ("[1/4] Add MiniMax-M3 support - #4581",
 * Kernel tuning: the QSA layers of qwen3.8-next, 12 query heads per KV head,
 * head dim 256, 4-token key blocks, timed fwd+bwd on 16k-token packs).
 * Same definition as msa_sparse_attn_fwd / _bwd with blocks of 4 tokens:
 *   q bf16 [T, Hq, 256]; k, v bf16 [T, Hkv, 256]; Hq must equal 12 Hkv;
 *   sel int32 [T, Hkv, topk], 1 <= topk <= 1024: block ids relative to the
 *   sequence start (block b = positions 4b .. 4b+3), distinct, each at most
 *   the token's own block p / 4 (larger ids set MSA_STATUS_BOUNDS and are
 *   dropped), -1 for unused slots.  A token attends to the keys j <= p of its
 *   listed blocks; the own block should be listed (a row with no key gets
 *   o = 0, lse = -inf).  max_seqlen <= 32768.
 *   o bf16 [T, Hq, 256], lse fp32 [T, Hq] (natural log);
 *   dq bf16 [T, Hq, 256], dk, dv bf16 [T, Hkv, 256].
 * Ownership, alignment, streams and errors as for the 128-token calls.
 */
MSA_API size_t msa_qsa_attn_fwd_workspace_size(int T, int S, int Hq, int Hkv, int max_seqlen);

MSA_API msa_status_t msa_qsa_attn_fwd(const void* q, const void* k, const void* v,
                              const int32_t* sel, const int32_t* cu_seqlens, int S, int T,
                              int Hq, int Hkv, int topk, int max_seqlen, float scale,
                              void* o, float* lse, void* workspace, size_t workspace_bytes,
                              msa_stream_t stream);

MSA_API size_t msa_qsa_attn_bwd_workspace_size(int T, int S, int Hq, int Hkv, int max_seqlen);

MSA_API msa_status_t msa_qsa_attn_bwd(const void* q, const void* k, const void* v,
                              const void* o, const void* dout, const float* lse,
                              const int32_t* sel, const int32_t* cu_seqlens, int S, int T,
                              int Hq, int Hkv, int topk, int max_seqlen, float scale,
                              void* dq, void* dk, void* dv, void* workspace,
                              size_t workspace_bytes, msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Decode step against a paged cache (scoring and selection rule of
 * "MiniMax-M3.1-Flash", 1 "Model Introduction", applied to one new token).
 * A page holds one 128-token block: k_cache, v_cache bf16 [num_pages, Hkv,
 * 128, 128] and kidx_cache bf16 [num_pages, Hkv, 128, 128] (index head h =
 * KV head h), post-prologue values.  block_table int32 [B, max_pages] maps
 * block c of sequence b to a page; cache_lens int32 [B] counts the cached
 * tokens INCLUDING the new one, whose position is cache_lens[b] - 1.
 * q bf16 [B, Hq, 128] and q_idx bf16 [B, Hkv, 128] are the new token's
 * post-prologue query and index query.  Per (b, h): every block up to the
 * own block is scored by its max logit, the own block plus the best 15
 * earlier ones are selected (sel_out int32 [B, Hkv, 16], may be NULL), and
 * o bf16 [B, Hq, 128] is the attention of the 16 query heads of KV head h
 * over the selected keys.
 */
MSA_API size_t msa_decode_step_workspace_size(int B, int Hq, int Hkv, int max_pages);

MSA_API msa_status_t msa_decode_step(const void* q, const void* q_idx, const void* k_cache,
                             const void* v_cache, const void* kidx_cache,
                             const int32_t* block_table, const int32_t* cache_lens, int B,
                             int Hq, int Hkv, int num_pages, int max_pages, float scale,
                             void* o, int32_t* sel_out, void* workspace,
                             size_t workspace_bytes, msa_stream_t stream);

/* msa_decode_step with the init rule of msa_index_select_ex: blocks
 * 0 .. min(n_init, own) - 1 of every sequence are always selected
 * (0 <= n_init <= 15; n_init = 0 is msa_decode_step).  Same workspace.
 */
MSA_API msa_status_t msa_decode_step_ex(const void* q, const void* q_idx, const void* k_cache,
                                const void* v_cache, const void* kidx_cache,
                                const int32_t* block_table, const int32_t* cache_lens,
                                int B, int Hq, int Hkv, int num_pages, int max_pages,
                                float scale, int n_init, void* o, int32_t* sel_out,
                                void* workspace, size_t workspace_bytes,
                                msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Decode append (the prologue of one new token per sequence, written into its
 * page; "MiniMax-M3.1-Flash", 1 "Model Introduction"; "MiniMax-M3",
 * "Architecture Notes").  Sequence b's new token is at position
 * p = cache_lens[b] - 1 (the length counts it).  q [B,Hq,128], q_idx, k, v,
 * k_idx [B,Hkv,128] are its pre-norm projections (bf16).  Then:
 *   q_out, q_idx_out = prologue(q, w_q), prologue(q_idx, w_qi) at p
 *                      (may be q / q_idx themselves, for an in-place update)
 *   k_cache[page, h, p % 128]    = prologue(k, w_k)[h]
 *   kidx_cache[page, h, p % 128] = prologue(k_idx, w_ki)[h]
 *   v_cache[page, h, p % 128]    = v[h]
 * with page = block_table[b, p / 128] and prologue = gemma norm + partial RoPE
 * as in msa_qk_norm_rope.  Caches as in msa_decode_step, which can follow on
 * the same stream.  A length outside [1, 128 max_pages] or a page outside
 * [0, num_pages) sets MSA_STATUS_BOUNDS and leaves that sequence untouched.
 */
MSA_API msa_status_t msa_decode_append(const void* q, const void* q_idx, const void* k,
                                       const void* v, const void* k_idx, const void* w_q,
                                       const void* w_qi, const void* w_k, const void* w_ki,
                                       void* k_cache, void* v_cache, void* kidx_cache,
                                       const int32_t* block_table, const int32_t* cache_lens,
                                       int B, int Hq, int Hkv, int num_pages, int max_pages,
                                       int rope_dim, float rope_base, float eps, void* q_out,
                                       void* q_idx_out, msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Append to a 16-bit paged cache: msa_decode_append for any number of new
 * tokens per row and any rotation.  A pack of T tokens, those of row s at cu_seqlens[s] ..
 * cu_seqlens[s + 1] - 1, is the end of the row: cache_lens[s] counts them, so that
 * token t is at position cache_lens[s] - cu_seqlens[s + 1] + t (a prompt, a chunk of
 * one, drafted tokens; one token per row in a decode step).  q bf16 [T, Hq, 128], k and v
 * bf16 [T, Hkv, 128]; optionally (all four or none) index q and k bf16 [T, Hkv, 128] with
 * kidx_cache and q_idx_out.  Then, with the prologue of msa_qk_norm_rope_ex at the token's
 * position (each weight bf16 [128], or NULL: no norm):
 *   q_out, q_idx_out = prologue(q, w_q), prologue(q_idx, w_qi)   (may be q / q_idx)
 *   k_cache[page, h, p % 128]    = prologue(k, w_k)[h]
 *   kidx_cache[page, h, p % 128] = prologue(k_idx, w_ki)[h]
 *   v_cache[page, h, p % 128]    = v[h]             with page = block_table[s, p / 128]
 * q_out and q_idx_out must not overlap the inputs otherwise.  Caches as in msa_decode_step; Hq
 * is any multiple of Hkv up to 256.  Tokens outside [cu_seqlens[0], cu_seqlens[S]) and those
 * of rows with cache_lens[s] = 0 (padding) are left alone.  Positions outside [0, 128
 * max_pages) and pages outside [0, num_pages) set MSA_STATUS_BOUNDS and leave the token's
 * outputs untouched.  A page that rows share has to be made the row's own first
 * (msa_pages_extend).
 */
MSA_API msa_status_t msa_cache_append(const void* q, const void* k, const void* v,
                                      const void* q_idx, const void* k_idx, const void* w_q,
                                      const void* w_k, const void* w_qi, const void* w_ki,
                                      void* k_cache, void* v_cache, void* kidx_cache,
                                      const int32_t* block_table, const int32_t* cu_seqlens,
                                      const int32_t* cache_lens, int S, int T, int Hq, int Hkv,
                                      int num_pages, int max_pages, const msa_rope_t* rope,
                                      float eps, void* q_out, void* q_idx_out,
                                      msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Full attention of one new token per row over the 16-bit paged cache (the
 * model's layers without an indexer), computed once where rows share pages.
 *   o[b, i]   = softmax(scale * q[b, i] k_j) v_j over the row's cache_lens[b] tokens
 *   lse[b, i] = log sum_j exp(scale * q[b, i] k_j)         fp32 [B, Hq] (may be NULL)
 * q, o bf16 [B, Hq, 128], Hq = G Hkv with 1 <= G <= 128; caches, block_table and
 * cache_lens as in msa_decode_step (the new token included).  The result is that of every
 * row by itself, whatever the tables hold.  Where neighbouring rows (those of length 0
 * not counted) begin with the same pages, as rows that were forked or reordered do, the
 * full pages that they have in common are read once for all of them, at up to 6
 * levels (a system prompt, behind it a prompt of each user, behind that its samples); so
 * put rows that share next to each other.  This is found out on the device in each call; calls
 * with G <= 16 whose tables are small (max_pages <= 128, few pages in all) read every row by itself,
 * which then takes less time.
 * A row with cache_lens[b] = 0 gets o = 0 and lse = -infinity, and so does a head whose
 * products are all -infinity; lengths outside [0, 128 max_pages] set MSA_STATUS_BOUNDS and are
 * treated so too.  A page outside [0, num_pages) sets MSA_STATUS_BOUNDS and has no keys.  o
 * may be q; o and lse must not overlap the inputs otherwise.  Slots of a row's last page
 * behind its end may hold anything.  B <= 2048, Hq <= 1024, Hkv <= 256, max_pages <= 1024; scale
 * from 2^-64 to 2^64.  Small calls as above need no workspace to speak of (256 bytes).
 */
MSA_API size_t msa_decode_shared_workspace_size(int B, int Hq, int Hkv, int max_pages);

MSA_API msa_status_t msa_decode_shared(const void* q, const void* k_cache, const void* v_cache,
                                       const int32_t* block_table, const int32_t* cache_lens,
                                       int B, int Hq, int Hkv, int num_pages, int max_pages,
                                       float scale, void* o, float* lse, void* workspace,
                                       size_t workspace_bytes, msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Beam search's selection.  Row n W + w is beam w of prompt n; logits of row r at
 * logits + r * row_stride (elements; row_stride >= V, any alignment of the type),
 * scores fp32 [N W] the beams' log probabilities.  Of the continuations
 *   score(w, v) = scores[w] + logits[w, v] - log sum_u exp(logits[w, u])
 * of a prompt the K best, best first: scores_out fp32 [N, K], parents int32 [N, K] (the row
 * n W + w), tokens int32 [N, K].  Scores are compared before they are rounded to fp32, as
 * 64-bit values over a log-sum-exp of fp32 exponentials; equal ones go to the lower w, then to
 * the larger logit, then to the lower v.  A beam with finished[r] != 0 (uint8 [N W], NULL:
 * none) goes on by pad_token alone, with its score unchanged; its logits are not read.  A NaN
 * among the logits counts as -infinity, what lies above 2^28 as 2^28 (and, where a beam has
 * nothing else, what lies below -2^28 as -2^28); a beam whose score is -infinity or NaN is
 * dead.  Continuations of probability zero are never chosen: where fewer than K are left, the
 * last places get score -infinity, parent -1, token -1 (msa_pages_reorder empties such rows).
 * scores_out may be scores where K = W; the outputs must not overlap scores or finished
 * otherwise, nor each other.  W, K <= 64, K <= W V, V <= 2^24, N W <= 65535.
 */
enum { MSA_F32 = 0, MSA_BF16 = 1 };

MSA_API size_t msa_beam_select_workspace_size(int N, int W, int V, int K);

MSA_API msa_status_t msa_beam_select(const void* logits, int dtype, int64_t row_stride,
                                     const float* scores, const uint8_t* finished, int N, int W,
                                     int V, int K, int pad_token, float* scores_out,
                                     int32_t* parents, int32_t* tokens, void* workspace,
                                     size_t workspace_bytes, msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Paged cache held in 4 bits.  A page of one head (a "slab") is 9216 bytes:
 * 128 tokens x 64 bytes of e2m1 codes (low nibble = even channel), then 128
 * tokens x 8 bytes of e4m3 scales, one for 16 consecutive channels.  A cache is
 * uint8 [num_pages, Hkv, 9216]; pages, block tables and positions are those of
 * msa_decode_step, so a cache takes 72 bytes per (token, head) instead of 256.
 * Per 16 channels with values x (bf16) and the cache's gain g:
 *   scale = e4m3(min(max|x| / g / 6, 448)),  code = e2m1(x / g / scale)
 * both rounded to nearest even (magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6, larger
 * ones saturate; scale 0 gives codes 0).  A code stands for code * scale * g,
 * exact in bf16.  Sixteen channels that hold an infinity or NaN get the scale
 * NaN, so they read back as NaN.  Gains (one per cache, finite, > 0, a power
 * of two from 2^-64 to 2^64) place values far from 1 in e4m3's range [2^-9, 448].
 *
 * msa_cache4_store writes a pack: token t of sequence s (cu_seqlens) goes to
 * position start[s] + t - cu_seqlens[s] of block table row s (start int32 [S],
 * NULL = 0); k, v, k_idx bf16 [T, Hkv, 128].  msa_cache4_load is its inverse:
 * the held values of those positions as bf16 [T, Hkv, 128].  Either may leave
 * out tensors: a NULL tensor with its cache NULL is skipped (one at least is
 * needed).  Tokens outside [0, max_pages * 128) or on pages outside
 * [0, num_pages) set MSA_STATUS_BOUNDS; they are not stored, and load as zeros.
 * Rows of the pack outside [cu_seqlens[0], cu_seqlens[S]) are left alone.
 * Store and append write where the table says: a page that rows share has to
 * be made the row's own first (msa_pages_extend), and no position may be written twice
 * in one call.
 */
MSA_API msa_status_t msa_cache4_store(const void* k, const void* v, const void* k_idx,
                                      void* k_cache, void* v_cache, void* kidx_cache,
                                      const int32_t* block_table, const int32_t* cu_seqlens,
                                      const int32_t* start, int S, int T, int Hkv,
                                      int num_pages, int max_pages, float k_gain, float v_gain,
                                      float kidx_gain, msa_stream_t stream);

MSA_API msa_status_t msa_cache4_load(const void* k_cache, const void* v_cache,
                                     const void* kidx_cache, const int32_t* block_table,
                                     const int32_t* cu_seqlens, const int32_t* start, int S,
                                     int T, int Hkv, int num_pages, int max_pages, float k_gain,
                                     float v_gain, float kidx_gain, void* k, void* v,
                                     void* k_idx, msa_stream_t stream);

/* msa_decode_append into a 4-bit cache, with the rotation of `rope` (dim <=
 * 128): q_out and q_idx_out as there, and k, k_idx (normed, rotated, rounded to
 * bf16) and v held in 4 bits at position cache_lens[b] - 1.  Hq is any multiple
 * of Hkv up to 256 heads.  A row with cache_lens[b] = 0 is padding: nothing of
 * it is read or written.  Other lengths outside [1, 128 max_pages] and pages
 * outside [0, num_pages) set MSA_STATUS_BOUNDS and leave the row untouched.
 */
MSA_API msa_status_t msa_decode4_append(const void* q, const void* q_idx, const void* k,
                                        const void* v, const void* k_idx, const void* w_q,
                                        const void* w_qi, const void* w_k, const void* w_ki,
                                        void* k_cache, void* v_cache, void* kidx_cache,
                                        const int32_t* block_table, const int32_t* cache_lens,
                                        int B, int Hq, int Hkv, int num_pages, int max_pages,
                                        const msa_rope_t* rope, float k_gain, float v_gain,
                                        float kidx_gain, float eps, void* q_out,
                                        void* q_idx_out, msa_stream_t stream);

/* msa_decode_step_ex over 4-bit caches.  Selection and attention are those of
 * the held values: blocks are scored by their largest index logit (the own
 * block and the first n_init blocks are kept without a score, and sequences of
 * at most 16 blocks keep all), equal scores go to the lower block.  Hq = G Hkv
 * with 1 <= G <= 16.  A row with cache_lens[b] = 0 gets o = 0 and sel = -1;
 * lengths outside [0, 128 max_pages] set MSA_STATUS_BOUNDS and are treated
 * so too.  A page outside [0, num_pages) sets MSA_STATUS_BOUNDS; its block scores
 * -infinity and, if it is selected all the same, has no keys.  Slots of the
 * own page behind the sequence's end may hold anything.  scale > 0 and its product
 * with k_gain have to be finite.  kidx_gain scales all
 * scores of a call alike and is not needed.
 */
MSA_API size_t msa_decode4_step_workspace_size(int B, int Hq, int Hkv, int max_pages);

MSA_API msa_status_t msa_decode4_step(const void* q, const void* q_idx, const void* k_cache,
                                      const void* v_cache, const void* kidx_cache,
                                      const int32_t* block_table, const int32_t* cache_lens,
                                      int B, int Hq, int Hkv, int num_pages, int max_pages,
                                      float scale, float k_gain, float v_gain, int n_init,
                                      void* o, int32_t* sel_out, void* workspace,
                                      size_t workspace_bytes, msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Pages of a paged cache: block_table int32 [B, max_pages], cache_lens int32
 * [B] and ref_count int32 [num_pages] (rows that hold the page; 0 = free) on the
 * device are changed in place, with no host synchronisation, and what is
 * chosen depends on their contents alone (the same calls give the same tables).
 * Row b holds ceil(cache_lens[b] / 128) pages; entries behind those are not
 * read.  `caches` is a HOST array of n_caches (0 .. 8) device pointers, page p of
 * cache c at caches[c] + p * page_bytes[c] (host array, multiples of 16): any
 * format, 16 or 4 bits.  Contents that contradict each other (rows or pages out
 * of range, a reference count below what the tables hold) set
 * MSA_STATUS_BOUNDS and are skipped.  Calls on one set of tables are ordered by
 * the caller (one stream, or events).
 *
 * fork: row dst[i] (empty before: length 0) becomes the first keep[i] tokens
 * (keep NULL = all) of row src[i]; the pages are shared.  Sources are read as
 * they were before the call.  forked[i] (int32 [n], output) is the length given, -1
 * where the pair is refused (dst not empty or equal to src, a row out of range,
 * or an earlier pair with the same dst); keep outside [0, length] is clamped and
 * sets MSA_STATUS_BOUNDS.
 */
MSA_API msa_status_t msa_pages_fork(const int32_t* src, const int32_t* dst, const int32_t* keep,
                                    int n, int32_t* block_table, int32_t* cache_lens,
                                    int32_t* ref_count, int B, int num_pages, int max_pages,
                                    int32_t* forked, msa_stream_t stream);

/* free: row rows[i] keeps its first keep[i] tokens (keep NULL = none): the
 * pages behind lose one reference, their table entries become -1 and the length
 * becomes keep[i] (a keep above the length changes nothing).  dropped[i] (int32
 * [n], output) is the number of tokens dropped, -1 where refused (a row out of range,
 * keep < 0, or a row that an earlier entry already shortens).
 */
MSA_API msa_status_t msa_pages_free(const int32_t* rows, const int32_t* keep, int n,
                                    int32_t* block_table, int32_t* cache_lens,
                                    int32_t* ref_count, int B, int num_pages, int max_pages,
                                    int32_t* dropped, msa_stream_t stream);

/* extend: row b grows by add[b] >= 0 tokens (int32 [B]), so that they can be
 * appended: it gets the pages it lacks, and if its last page is partly filled
 * and shared, a copy of that page for itself first (copy on write, the page's
 * bytes of every cache).  Free pages go out in ascending order, to the rows in order,
 * the copy before the new pages.  done[b] (int32 [B], output) is 1 where the row
 * has grown; 0 where it is left as it was: what rows 0 .. b want together is more than
 * the pages that were free before the call, or the row would exceed max_pages,
 * or add[b] < 0 (which sets MSA_STATUS_BOUNDS); rows of the last two kinds want
 * nothing.  Rows with add[b] = 0 are done.  A page that loses its last row here (all
 * its sharers copied it) is free after the call.
 */
MSA_API size_t msa_pages_extend_workspace_size(int B, int num_pages);

MSA_API msa_status_t msa_pages_extend(const int32_t* add, int32_t* block_table,
                                      int32_t* cache_lens, int32_t* ref_count, int B,
                                      int num_pages, int max_pages, void* const* caches,
                                      const int64_t* page_bytes, int n_caches, int32_t* done,
                                      void* workspace, size_t workspace_bytes,
                                      msa_stream_t stream);

/* compact: the pages in use (ref_count > 0) move to the front of the pool: of
 * n of them, those at n and behind go, in ascending order, to the free places
 * below n, in ascending order; tables and reference counts follow.  page_map int32
 * [num_pages] (output): the new place of each page, -1 for free ones; n_live
 * int32 [1] (output): n.  Bytes of the places that become free are left as they were.
 */
MSA_API size_t msa_pages_compact_workspace_size(int num_pages);

MSA_API msa_status_t msa_pages_compact(int32_t* block_table, const int32_t* cache_lens,
                                       int32_t* ref_count, int B, int num_pages, int max_pages,
                                       void* const* caches, const int64_t* page_bytes,
                                       int n_caches, int32_t* page_map, int32_t* n_live,
                                       void* workspace, size_t workspace_bytes,
                                       msa_stream_t stream);

/* reorder: row r becomes what row parents[r] (int32 [B]) was before the call: its table
 * entries, its length and, from now on, its pages, which rows with the same parent share
 * (a partly filled last page too: msa_pages_extend gives each its own copy before it is
 * written).  parents[r] = r keeps the row, -1 empties it; rows that are nobody's
 * parent lose their pages, and entries that a row no longer needs become -1.  kept[r]
 * (int32 [B], output) is the row's length after the call, -1 where it is refused and left
 * as it was: a parent outside [-1, B), or one whose length is out of range (both set
 * MSA_STATUS_BOUNDS).  parents, kept, the tables and ref_count must not overlap.
 */
MSA_API size_t msa_pages_reorder_workspace_size(int B, int max_pages);

MSA_API msa_status_t msa_pages_reorder(const int32_t* parents, int32_t* block_table,
                                       int32_t* cache_lens, int32_t* ref_count, int B,
                                       int num_pages, int max_pages, int32_t* kept,
                                       void* workspace, size_t workspace_bytes,
                                       msa_stream_t stream);

/* copy: the bytes of page src[i] become those of page dst[i], i < n, in every
 * cache (a page must not be a dst twice, nor both a dst and another pair's src;
 * src[i] = dst[i] does nothing).  Pairs with a page out of range set
 * MSA_STATUS_BOUNDS and are skipped.
 */
MSA_API msa_status_t msa_pages_copy(const int32_t* src, const int32_t* dst, int n, int num_pages,
                                    void* const* caches, const int64_t* page_bytes, int n_caches,
                                    msa_stream_t stream);

/* ------------------------------------------------------------------------
 * msa_decode_step_static: the decode step above for callers that cannot
 * allocate device memory.  The pages have no counterpart of this call; it
 * exists for integration.  Some callers of a decode step own no allocator:
 * a serving engine that hands out a fixed pool of GPU memory at start-up and
 * forbids later cudaMalloc / cudaFree (which synchronize the device and
 * fragment the pool), or a plugin whose host framework gives it only the
 * tensors it computes on.  Such a caller cannot provide the workspace that
 * msa_decode_step needs.
 *
 * Same arguments, layouts and results as msa_decode_step, minus the
 * workspace: the scratch (per-block scores and per-split partial outputs)
 * lives in one fixed array in the library's device memory, sized for
 *   B * Hkv <= 256   and   max_pages <= 1024   (128K cached tokens),
 * about 9.6 MB, which every GPU that loads the library keeps until the
 * process exits.  Larger calls return MSA_ERR_UNSUPPORTED and enqueue nothing.
 * The call allocates nothing: no cudaMalloc, no cudaFree, no allocating
 * library routine.  Its first call on a device looks up that device's copy
 * of the array (a host-side query, done with the device current); make that
 * first call before any stream capture.  The address is kept per CUDA
 * context (keyed by the context's process-unique id), so after
 * cudaDeviceReset the first call in the new context looks it up again, and
 * that call too should come before any capture.  All calls share the one array, so
 * two calls whose kernels may overlap on the GPU (different streams, no
 * ordering between them) race and corrupt each other's results; calls on one
 * stream are safe.  Every scratch element a call reads is written earlier in
 * the same call, so leftovers of a previous call do not matter.
 */
MSA_API msa_status_t msa_decode_step_static(const void* q, const void* q_idx,
                                            const void* k_cache, const void* v_cache,
                                            const void* kidx_cache, const int32_t* block_table,
                                            const int32_t* cache_lens, int B, int Hq, int Hkv,
                                            int num_pages, int max_pages, float scale, void* o,
                                            int32_t* sel_out, msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Launch tracing (no counterpart on the pages: measurement plumbing).
 * msa_trace_begin() clears the record and turns tracing on: from then on the
 * library brackets each of its kernel launches with a pair of CUDA events on
 * the launch stream (host-side objects, created on first use and kept).
 * msa_trace_end() waits for the recorded events, turns tracing off and writes
 * a JSON object {"<kernel>": {"launches": n, "ms": total}, ...} (NUL
 * terminated, truncated to `cap` bytes) into `json`.  Not for use inside
 * stream capture.  Tracing is process-wide and off by default.
 */
MSA_API msa_status_t msa_trace_begin(void);
MSA_API msa_status_t msa_trace_end(char* json, size_t cap);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H_ */
