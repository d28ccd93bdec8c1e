/*
 * mla.h -- C ABI of the GB300 (sm_103a) multi-head latent attention sublayer.
 *
 * The operation is the MLA sublayer of a Kimi K2 / DeepSeek-V3 style block:
 *   Kimi K2 "Dense transformer block" page, equation list (x_attn = RMSNorm(x),
 *     c^Q, c^KV, q^C/q^pe, k^C/k^pe, v, RoPE, Q = [Q^C; Q^R], K_i = [K^C_i; k^R],
 *     x' = x + Delta_attn);
 *   "Mix and project" page (decode, P = 1,000), code excerpt: scores scaled and
 *     masked, float32 softmax, P.V, heads merged head-major, o_proj;
 *   "Key-value compression" page: kv_a_proj_with_mqa gives a 512-wide latent
 *     and one 64-wide rotary key (576 features, split after the product); the
 *     latent alone is normalised; 576 cached values per position for the
 *     latent form versus 20,480 for rebuilt per-head keys and values.
 *
 * Fixed sizes (checked against the pages' 101,124,096 MLA parameters):
 *   d = 7168, H = 64 heads, q_lora = 1536, kv_lora = 512,
 *   qk = 128 (nope) + 64 (rope, 32 pairs) = 192, v = 128, no biases.
 * Other sizes are not supported.
 *
 * Conventions for every entry point
 *   - All tensors are bf16, row-major, in device memory, owned by the caller.
 *     Weights use the nn.Linear layout [out, in].
 *   - Every pointer must be 16-byte aligned (MLA_ERR_ALIGNMENT otherwise).
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream).  The library never synchronises and allocates no
 *     device memory: all scratch lives in the caller's workspace, sized by
 *     mla_workspace_size().  A workspace must not be shared by calls that may
 *     run concurrently.
 *   - Decode and prefill calls of at most 4096 rows run the kv_b product on a
 *     second stream of the library's own, beside q_b (neither fills the GPU
 *     alone, or its last wave of tiles), forked from and joined back into
 *     `stream` with events: the call is still ordered on `stream` as a whole.
 *     mla_prefill_paged, mla_prefill_chunk_latent and a prefill that only fills
 *     caches (out NULL) stay on `stream`.
 *     That stream and its two events are created by the first such call of
 *     each host thread on each device (not during a stream capture: a call
 *     captured before any uncaptured call of its thread stays on `stream`)
 *     and destroyed when the thread exits.
 *   - Positions are implicit: prefill tokens sit at positions 0..T-1 with a
 *     causal mask (key j visible to query i iff j <= i); a decode token sits
 *     at position P and attends to all P + 1 keys.
 *   - RoPE is rotate-half on pairs (i, i+32), theta_i = rope_base^(-2i/64).
 *   - `out` may be the same buffer as `x` (in-place residual); any other
 *     overlap between out and x is rejected.
 *   - Arguments are checked on the host before anything is enqueued; a
 *     failed check returns a negative status and enqueues nothing.  This
 *     mirrors the shape checks (ValueError / assert) of the pages' code.
 */
#ifndef MLA_H_
#define MLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define MLA_OK 0
#define MLA_ERR_INVALID_ARG (-1)  /* null pointer, B/T/P out of range, cap too small, overlap */
#define MLA_ERR_ALIGNMENT (-2)    /* a pointer is not 16-byte aligned */
#define MLA_ERR_WORKSPACE (-3)    /* workspace NULL or smaller than mla_workspace_size() */
#define MLA_ERR_UNSUPPORTED (-4)  /* a size or mode the library does not implement */
#define MLA_ERR_CUDA (-5)         /* a CUDA call or kernel launch failed */
#define MLA_ERR_TIMEOUT (-6)      /* a bounded device-side wait gave up (see mla_device_status) */
#define MLA_ERR_NO_PAGES (-7)     /* fewer free pages than a call takes (see mla_device_status) */

/* ---- fixed sizes -------------------------------------------------------- */
#define MLA_D 7168
#define MLA_HEADS 64
#define MLA_Q_LORA 1536
#define MLA_KV_LORA 512
#define MLA_QK_NOPE 128
#define MLA_QK_ROPE 64
#define MLA_QK 192
#define MLA_V 128
#define MLA_FFN_INTER 18432  /* SwiGLU MLP width: 396,361,728 parameters / (3 x 7168) */

/* ---- modes for mla_workspace_size ---------------------------------------- */
#define MLA_MODE_PREFILL 0
#define MLA_MODE_DECODE 1
#define MLA_MODE_DECODE_LATENT 2
#define MLA_MODE_FFN 3
#define MLA_MODE_CHUNK_LATENT 4
#define MLA_MODE_CHUNK_ABSORBED 5
#define MLA_MODE_FOLD 6
#define MLA_MODE_PAGED_APPEND 8
#define MLA_MODE_PAGED_ATTN 9
#define MLA_MODE_WINDOW_ATTN 10
#define MLA_MODE_DECODE_PAGED 11
#define MLA_MODE_PREFILL_PAGED 12
#define MLA_MODE_PAGES 13
#define MLA_MODE_DOCUMENTS 14

/* Weights of one MLA sublayer: device pointers to bf16, nn.Linear [out, in].
 * Key-value compression page, MLA __init__ excerpt, for the projections;
 * w_in_norm is the block's input RMSNorm gain (dense-block page). */
typedef struct {
  const void* w_in_norm;   /* [7168]          input RMSNorm gain            */
  const void* w_q_a;       /* [1536, 7168]    q_a_proj (W_DQ)               */
  const void* w_q_a_norm;  /* [1536]          q_a_layernorm gain            */
  const void* w_q_b;       /* [12288, 1536]   q_b_proj; per head [128 nope | 64 pe] */
  const void* w_kv_a;      /* [576, 7168]     kv_a_proj_with_mqa (W_DKV ; W_KR) */
  const void* w_kv_a_norm; /* [512]           kv_a_layernorm gain           */
  const void* w_kv_b;      /* [16384, 512]    kv_b_proj; per head [128 k_nope | 128 v] */
  const void* w_o;         /* [7168, 8192]    o_proj                        */
} mla_weights_t;

/* Stage ids for optional per-stage timing. */
#define MLA_STAGE_INPUT_NORM 0   /* RMSNorm(x)                               */
#define MLA_STAGE_A_PROJ 1       /* x_attn . [W_DQ ; W_DKV ; W_KR]^T          */
#define MLA_STAGE_LATENT 2       /* split, q/kv latent RMSNorm, RoPE table and RoPE(k), latent cache write */
#define MLA_STAGE_Q_B 3          /* q_b_proj + RoPE(q)                       */
#define MLA_STAGE_KV_B 4         /* kv_b_proj + per-head K/V cache write     */
#define MLA_STAGE_ATTN 5         /* attention (prefill, decode or latent decode) */
#define MLA_STAGE_COMBINE 6      /* split-KV combine                         */
#define MLA_STAGE_ABSORB_Q 7     /* latent decode: q_nope . W_UK             */
#define MLA_STAGE_ABSORB_O 8     /* latent decode: o_latent . W_UV^T         */
#define MLA_STAGE_O_PROJ 9       /* o_proj + residual                        */
#define MLA_STAGE_FFN_NORM 10    /* mla_ffn: RMSNorm(x')                     */
#define MLA_STAGE_FFN_GATE_UP 11 /* mla_ffn: [W_1 ; W_3] product + SiLU(g) * u */
#define MLA_STAGE_FFN_DOWN 12    /* mla_ffn: W_2 product + residual          */
#define MLA_MAX_STAGES 13

/* Optional per-stage timing.  start[s] / stop[s] are cudaEvent_t handles
 * created by the caller (or NULL to skip stage s); the library records them
 * on `stream` around stage s.  n_launches is written with the number of
 * kernels the call enqueued. */
typedef struct {
  void* start[MLA_MAX_STAGES];
  void* stop[MLA_MAX_STAGES];
  int n_launches;
} mla_timing_t;

/* Runtime parameters.  Passing NULL for the whole struct selects
 * eps = 1e-6, rope_base = 10000, softmax_scale = 1/sqrt(192). */
typedef struct {
  float eps;            /* RMSNorm epsilon, used by all three norms        */
  float rope_base;      /* RoPE base                                       */
  float softmax_scale;  /* multiplies Q.K before the softmax               */
  float* delta_out;     /* optional: float32 [N_tok, 7168] receives Delta_attn
                           (o_proj output before the residual); NULL = off */
  mla_timing_t* timing; /* optional per-stage events; NULL = off            */
} mla_params_t;

/* Bytes of workspace an entry point needs.
 *   mode = MLA_MODE_PREFILL:       B sequences of T = t_or_p tokens; `cap` is
 *                                  ignored (pass the cache capacity or 0).
 *   mode = MLA_MODE_DECODE / _LATENT: B sequences, P = t_or_p cached positions.
 *   mode = MLA_MODE_FFN:           B * t_or_p token rows (mla_ffn).
 *   mode = MLA_MODE_CHUNK_LATENT:  B sequences, chunks of T = t_or_p tokens,
 *                                  latent caches of `cap` positions
 *                                  (mla_prefill_chunk_latent; the size grows
 *                                  with cap: it holds the rebuilt keys and
 *                                  values of every position, 40 KB each).
 *   mode = MLA_MODE_CHUNK_ABSORBED: B sequences, chunks of T = t_or_p
 *                                  tokens, latent caches of `cap` positions
 *                                  (mla_prefill_chunk_absorbed; the size grows
 *                                  with B * T only).
 *   mode = MLA_MODE_FOLD:          mla_fold_wuv_into_wo (B, t_or_p, cap
 *                                  ignored: a status region only).
 *   mode = MLA_MODE_PAGED_APPEND:  mla_paged_append, B sequences of at most
 *                                  t_or_p new tokens (`cap` ignored).
 *   mode = MLA_MODE_PAGED_ATTN:    mla_paged_attention, B sequences of
 *                                  t_or_p new tokens (`cap` ignored).
 *   mode = MLA_MODE_WINDOW_ATTN:   mla_window_attention, B sequences of
 *                                  t_or_p queries (`cap` ignored).
 *   mode = MLA_MODE_DECODE_PAGED:  mla_decode_paged, B sequences, P_max = t_or_p.
 *   mode = MLA_MODE_PREFILL_PAGED: mla_prefill_paged, B sequences of T = t_or_p
 *                                  tokens, cap = P0 + T (or more): it holds
 *                                  those positions' keys and values in bf16.
 *   mode = MLA_MODE_PAGES:         the mla_pages_ calls on lists of B entries,
 *                                  t_or_p = n_pages (of the destination cache
 *                                  in a copy), cap = the table's rows (0 for a
 *                                  copy).
 *   mode = MLA_MODE_DOCUMENTS:     mla_document_attention, B documents, t_or_p =
 *                                  N rows of q (`cap` ignored).
 * Returns 0 when the arguments are out of range. */
size_t mla_workspace_size(int mode, int B, int t_or_p, int cap);

/* Causal prefill of x [B, T, 7168] at positions 0..T-1.
 *   out       [B, T, 7168]        x + Delta_attn (may alias x exactly); or NULL:
 *                                 the call then only fills the caches it is
 *                                 given (a prompt-cache fill: the query path,
 *                                 attention and o_proj are skipped)
 *   k_cache   [B, 64, cap, 192]   optional (NULL): receives K rows 0..T-1, post-RoPE
 *   v_cache   [B, 64, cap, 128]   optional, given together with k_cache
 *   ckv_cache [B, cap, 512]       optional (NULL): receives the normalised latent c^KV-hat
 *   kpe_cache [B, cap, 64]        optional, given together with ckv_cache: rotated k^R
 *   cap       cache capacity in positions; must be >= T when a cache is given
 * Errors: INVALID_ARG (B < 1, T < 1, null x or weights, out NULL with no
 * cache, only one of a cache pair, cap < T, partial x/out overlap),
 * ALIGNMENT, WORKSPACE, CUDA. */
int mla_prefill(const mla_weights_t* w, const mla_params_t* params, const void* x, int B, int T,
                void* out, void* k_cache, void* v_cache, void* ckv_cache, void* kpe_cache, int cap,
                void* workspace, size_t workspace_bytes, void* stream);

/* Chunked prefill: T new tokens per sequence at positions P0..P0+T-1, after
 * P0 tokens already in the rebuilt cache ("Mix and project" page: the cache
 * update appends the new keys and values after the cached ones, and the
 * additive mask of shape (B, 1, q_len, kv_seq_len), kv_seq_len = P0 + T,
 * keeps the causal order: token t sees keys 0..P0+t).
 *   x         [B, T, 7168]        the chunk's tokens
 *   out       [B, T, 7168]        x + Delta_attn (may alias x exactly)
 *   k_cache   [B, 64, cap, 192]   rows 0..P0-1 are read, rows P0..P0+T-1 written
 *   v_cache   [B, 64, cap, 128]   same (both required)
 *   ckv_cache, kpe_cache          optional latent cache, rows P0..P0+T-1 written
 * Requires P0 >= 0 and P0 + T <= cap; the workspace is that of
 * mla_workspace_size(MLA_MODE_PREFILL, B, T, cap).  P0 = 0 computes what
 * mla_prefill computes with caches.
 * Errors: INVALID_ARG (null or missing K/V cache, P0 < 0, P0 + T > cap),
 * ALIGNMENT, WORKSPACE, CUDA. */
int mla_prefill_chunk(const mla_weights_t* w, const mla_params_t* params, const void* x, int B, int T,
                      int P0, void* out, void* k_cache, void* v_cache, void* ckv_cache, void* kpe_cache,
                      int cap, void* workspace, size_t workspace_bytes, void* stream);

/* Chunked prefill against the 576-value latent cache (latent-cache serving:
 * "Key-value compression" page, the per-head keys and values of every
 * position are rebuilt from its one latent).  T new tokens per sequence at
 * positions P0..P0+T-1; their latent rows are written to the cache, then the
 * keys and values of positions 0..P0+T-1 are rebuilt from the cache into the
 * workspace (kv_b product, rotary key appended) and the chunk attends to them
 * with the causal mask offset by P0, as mla_prefill_chunk.
 *   x, out          [B, T, 7168]   (out may alias x exactly; required)
 *   ckv_cache       [B, cap, 512]  rows 0..P0-1 read, rows P0..P0+T-1 written
 *   kpe_cache       [B, cap, 64]   same
 * Requires P0 >= 0, P0 + T <= cap; workspace
 * mla_workspace_size(MLA_MODE_CHUNK_LATENT, B, T, cap).
 * Errors: INVALID_ARG (null pointer, P0 < 0, P0 + T > cap), ALIGNMENT,
 * WORKSPACE, CUDA. */
int mla_prefill_chunk_latent(const mla_weights_t* w, const mla_params_t* params, const void* x, int B, int T,
                             int P0, void* out, void* ckv_cache, void* kpe_cache, int cap, void* workspace,
                             size_t workspace_bytes, void* stream);

/* W_UV folded into the output projection (latent-cache serving, "Key-value
 * compression" page: the value up-projection moves past the attention, and
 * here on into W_o): for every head h,
 *   W_fold[:, h*512 .. h*512+511] = W_o[:, h*128 .. h*128+127] W_UV[h],
 * W_UV[h] = rows h*256+128 .. h*256+255 of W_kv_b ([128, 512]).
 *   w_fold     [7168, 32768] bf16, caller-allocated (470 MB), written
 *   workspace  mla_workspace_size(MLA_MODE_FOLD, 1, 1, 0) bytes
 * Errors: INVALID_ARG (null weight or w_fold), ALIGNMENT, WORKSPACE, CUDA. */
int mla_fold_wuv_into_wo(const mla_weights_t* w, void* w_fold, void* workspace, size_t workspace_bytes,
                         void* stream);

/* mla_decode_latent with the output projection through W_fold: the latent
 * attention output of all heads, o_lat [B, 64*512], times W_fold^T plus the
 * residual, one GEMM in place of W_UV and o_proj.  Arguments, workspace
 * (MLA_MODE_DECODE_LATENT) and errors as mla_decode_latent; w_fold from
 * mla_fold_wuv_into_wo (16-byte aligned).  It streams 470 MB of weights where
 * W_UV and W_o are 125 MB, so a weight-bound decode step is slower; kept for
 * comparison. */
int mla_decode_latent_folded(const mla_weights_t* w, const void* w_fold, const mla_params_t* params, const void* x,
                             int B, int P, void* ckv_cache, void* kpe_cache, int cap, void* out, void* workspace,
                             size_t workspace_bytes, void* stream);

/* The same chunk in the absorbed form (latent-cache serving, "Key-value
 * compression" page: W_UK folded into the query, W_UV applied after the
 * attention, so the cached latent is never expanded).  Every new token
 * (b, t) is one latent decode step at position P0 + t that attends to cache
 * rows 0..P0+t of sequence b: scores q_lat . [k^R ; c^KV], o_lat = P c^KV,
 * then W_UV and o_proj.  Results, arguments and errors as
 * mla_prefill_chunk_latent; the chunk's latent rows are written first.
 * Cost: the cache is read once per new token (B T (P0 + T) 1152 bytes)
 * instead of rebuilding the keys and values of every cached position (a
 * 16384 x 512 product per position), so it is the form for short chunks.
 * Requires P0 >= 0, P0 + T <= cap; workspace
 * mla_workspace_size(MLA_MODE_CHUNK_ABSORBED, B, T, cap).
 * Errors: INVALID_ARG (null pointer, P0 < 0, P0 + T > cap), ALIGNMENT,
 * WORKSPACE, CUDA. */
int mla_prefill_chunk_absorbed(const mla_weights_t* w, const mla_params_t* params, const void* x, int B, int T,
                               int P0, void* out, void* ckv_cache, void* kpe_cache, int cap, void* workspace,
                               size_t workspace_bytes, void* stream);

/* One decode step against the rebuilt per-head cache (the pinned
 * implementation's cache, "Mix and project" page at P = 1,000).
 *   x        [B, 7168]           the new token of each sequence, at position P
 *   k_cache  [B, 64, cap, 192]   positions 0..P-1 are read; row P is written
 *   v_cache  [B, 64, cap, 128]   same
 *   out      [B, 7168]           x + Delta_attn (may alias x exactly)
 * Requires 0 <= P and P + 1 <= cap.
 * Errors: INVALID_ARG, ALIGNMENT, WORKSPACE, CUDA. */
int mla_decode(const mla_weights_t* w, const mla_params_t* params, const void* x, int B, int P,
               void* k_cache, void* v_cache, int cap, void* out,
               void* workspace, size_t workspace_bytes, void* stream);

/* One decode step against the 576-value latent cache, with W_UK absorbed
 * into the query and W_UV applied after attention (the latent-caching design
 * the key-value compression page describes).
 *   ckv_cache [B, cap, 512]  normalised latent; positions 0..P-1 read, row P written
 *   kpe_cache [B, cap, 64]   rotated rotary key; same
 * Other arguments as mla_decode. */
int mla_decode_latent(const mla_weights_t* w, const mla_params_t* params, const void* x, int B,
                      int P, void* ckv_cache, void* kpe_cache, int cap, void* out,
                      void* workspace, size_t workspace_bytes, void* stream);

/* The same two decode steps for a batch of sequences of different lengths
 * (a ragged batch: "Mix and project" page, each sequence its own cache update
 * and score row).  Sequence b's new token sits at position P[b] and attends
 * to its P[b] + 1 keys; its cache row P[b] is written.
 *   P      int [B] in DEVICE memory (4-byte aligned), read by the kernels, so
 *          a captured CUDA graph can be replayed with new lengths
 *   P_max  an upper bound of every P[b]; it sizes the launch and the
 *          workspace: mla_workspace_size(MLA_MODE_DECODE or
 *          MLA_MODE_DECODE_LATENT, B, P_max, cap); requires P_max + 1 <= cap
 * A P[b] outside [0, P_max] cannot be checked on the host: the kernels clamp
 * it into that range (no access leaves the caches) and record it, and
 * mla_device_status then returns MLA_ERR_INVALID_ARG.
 * Other arguments, results and errors as mla_decode / mla_decode_latent. */
int mla_decode_varlen(const mla_weights_t* w, const mla_params_t* params, const void* x, int B, const int* P,
                      int P_max, void* k_cache, void* v_cache, int cap, void* out, void* workspace,
                      size_t workspace_bytes, void* stream);
int mla_decode_latent_varlen(const mla_weights_t* w, const mla_params_t* params, const void* x, int B,
                             const int* P, int P_max, void* ckv_cache, void* kpe_cache, int cap, void* out,
                             void* workspace, size_t workspace_bytes, void* stream);

/* mla_decode without a workspace argument.  The pages have no counterpart
 * to this entry point: it exists for callers that cannot allocate device
 * memory (code running under a host framework that owns all device memory
 * and allows no allocation of its own, such as inference-server plugins or
 * runtimes with a fixed memory budget, and latency-critical loops that cannot
 * afford the device synchronisation an allocation may cause).
 *   Scratch: a 64 MiB static device array inside the library, held by every
 *   GPU that loads the library until the process exits.  Batches whose
 *   mla_workspace_size(MLA_MODE_DECODE, B, P, cap) exceeds 64 MiB (more than
 *   455 sequences) are rejected with MLA_ERR_WORKSPACE; nothing is allocated.
 *   The first call on each device looks up the array's device address (with
 *   that device current); make that first call before any stream capture.
 *   Every call on a device shares the one array and it keeps the last call's
 *   contents: calls that may overlap on the GPU (different streams without
 *   ordering between them) race.  A device-side timeout is recorded only in
 *   the array, not returned.
 * Arguments, checks and results otherwise as mla_decode. */
int mla_decode_noalloc(const mla_weights_t* w, const mla_params_t* params, const void* x, int B, int P,
                       void* k_cache, void* v_cache, int cap, void* out, void* stream);

/* ---- FP8 block-scaled weights ---------------------------------------------
 * The dense-block page counts the checkpoint's tensors with its "FP8 block
 * scales" left out: the released weights are FP8 with one scale per block.
 * Block size and scale format are not printed; this library's format:
 * E4M3 codes (the OCP FP8 E4M3 encoding, largest finite 448) of the [out, in]
 * matrix, and one float scale per 128 x 128 block, always a power of two:
 * the smallest 2^k with amax(block) <= 448 * 2^k.  The weight used is
 * code * scale, exact in bfloat16, so the FP8 decode computes with exactly
 * the quantized weights (on the bf16 tensor-core path: the codes are
 * dequantized in shared memory; the bytes read from HBM halve).
 *   cols   a multiple of 128
 *   codes  uint8, block-major: block (i, j) (rows 128i.., columns 128j..) is
 *          16,384 contiguous bytes at offset (i * cols/128 + j) * 16384,
 *          row-major inside; ceil(rows/128) * cols/128 * 16384 bytes in all,
 *          the rows past the matrix zero
 *   scales [ceil(rows/128), cols/128] float */
int mla_quantize_fp8(const void* w_bf16, int rows, int cols, void* codes, float* scales, void* stream);

/* The MLA weights with the five projection matrices in that format (gains
 * stay bf16). */
typedef struct {
  const void* w_in_norm;   /* [7168] bf16                                       */
  const void* w_q_a_norm;  /* [1536] bf16                                       */
  const void* w_kv_a_norm; /* [512]  bf16                                       */
  const void* w_q_a;       /* [1536, 7168]   E4M3 codes, block-major; scales [12, 56] */
  const void* w_q_b;       /* [12288, 1536]  E4M3 codes, block-major; scales [96, 12] */
  const void* w_kv_a;      /* [576, 7168]    E4M3 codes, block-major (640 rows); scales [5, 56] */
  const void* w_kv_b;      /* [16384, 512]   E4M3 codes, block-major; scales [128, 4] */
  const void* w_o;         /* [7168, 8192]   E4M3 codes, block-major; scales [56, 64] */
  const float* s_q_a;
  const float* s_q_b;
  const float* s_kv_a;
  const float* s_kv_b;
  const float* s_o;
} mla_weights_fp8_t;

/* mla_decode with FP8 block-scaled weights: the same step, arguments,
 * workspace (MLA_MODE_DECODE) and errors; every projection reads its E4M3
 * codes and scales (codes 16-byte aligned, scales 4-byte aligned, else
 * MLA_ERR_ALIGNMENT). */
int mla_decode_fp8(const mla_weights_fp8_t* w, const mla_params_t* params, const void* x, int B, int P,
                   void* k_cache, void* v_cache, int cap, void* out, void* workspace, size_t workspace_bytes,
                   void* stream);

/* ---- the block's second half ---------------------------------------------
 * Kimi K2 "Dense transformer block" page, equation list after
 * x'_n = x_n + Delta_attn, and its DecoderLayer forward excerpt: the dense
 * block applies the MLA sublayer (mla_prefill / mla_decode /
 * mla_decode_latent: x -> x'), then
 *   x_ffn = RMSNorm(x'); g = x_ffn W_1; u = x_ffn W_3; a = g sigma(g);
 *   h = a (.) u; Delta_ffn = h W_2; x_{n+1} = x' + Delta_ffn.
 * The intermediate width is not printed; the page's parameter table gives
 * the SwiGLU MLP 396,361,728 parameters = 3 x 7168 x 18,432 (no biases). */
typedef struct {
  const void* w_post_norm; /* [7168]          post-attention RMSNorm gain   */
  const void* w_1;         /* [18432, 7168]   gate projection (g)           */
  const void* w_3;         /* [18432, 7168]   up projection (u)             */
  const void* w_2;         /* [7168, 18432]   down projection               */
} mla_ffn_weights_t;

/* x_{n+1} = x' + Delta_ffn for n_tok token rows (any mix of prefill and
 * decode rows: every row is independent).
 *   x    [n_tok, 7168]   x' (the MLA sublayer's output)
 *   out  [n_tok, 7168]   x_{n+1} (may alias x exactly)
 *   params: eps (the MLP RMSNorm's), delta_out (optional float32
 *   [n_tok, 7168] receiving Delta_ffn) and timing (stages
 *   MLA_STAGE_FFN_*); rope_base and softmax_scale are not used.  NULL
 *   selects eps = 1e-6.
 *   workspace: mla_workspace_size(MLA_MODE_FFN, 1, n_tok, 0) bytes (it holds
 *   RMSNorm(x') and h, n_tok x (7168 + 18432) bf16 values).
 * g and u accumulate in float32; SiLU(g) u is rounded once to bf16 (h), the
 * input of the down projection, whose float32 sum is added to x' in float32
 * and rounded once.
 * Errors: INVALID_ARG (null pointer, n_tok < 1, partial x/out overlap),
 * ALIGNMENT, WORKSPACE, CUDA. */
int mla_ffn(const mla_ffn_weights_t* w, const mla_params_t* params, const void* x, int n_tok, void* out,
            void* workspace, size_t workspace_bytes, void* stream);

/* ---- paged 8-bit cache ------------------------------------------------------
 * The rebuilt per-head cache ("Mix and project" page: keys and values of every
 * head, 20,480 values per position) in pages of a few tokens, with the 128
 * unrotated key values and the 128 values of a head as E4M3 codes and one
 * scale per page and head, and the rotary key, which all heads share, once
 * per token in bf16: heads * 256 + 128 bytes a position (16.5 KB at 64 heads)
 * where the bf16 cache takes 40 KB.
 *   k_codes, v_codes  uint8 [n_pages, heads, page, 128], E4M3 (the OCP FP8
 *                     encoding, largest finite 448)
 *   k_pe              bf16 [n_pages, page, 64], rotated
 *   k_scales, v_scales float [n_pages, heads], positive and finite;
 *                     mla_paged_append writes powers of two, 2^-60 .. 2^60,
 *                     except that a partly filled page keeps a larger scale
 *                     that it came with
 *   table             int [B, max_pages] in DEVICE memory: the pages of each
 *                     sequence in order, position p in page table[b][p / page],
 *                     slot p % page.  Read by the kernels: a captured graph
 *                     can be replayed with a new table.
 * A key is code * scale.  A page that receives tokens belongs to one sequence;
 * pages that are only read may be shared.  Codes, scales and rotary keys are
 * 16-byte aligned, the table 4-byte aligned.
 *   page   16, 32, 64 or 128
 *   heads  a multiple of 4, at most 128 (the sublayer's entry points need 64;
 *          a shard of the heads has fewer)
 * n_pages * heads and n_pages * page must fit a 31-bit int, and a sequence has
 * at most 2^30 positions (max_pages * page). */
typedef struct {
  void* k_codes;
  void* v_codes;
  void* k_pe;
  float* k_scales;
  float* v_scales;
  const int* table;
  int n_pages, max_pages, page, heads;
} mla_paged_cache_t;

/* Appends new tokens to the paged cache, rotating their rotary keys on the
 * way.  Sequence b's T_b new tokens take positions P[b] .. P[b] + T_b - 1.
 *   k, v     bf16: the 128 key / value numbers of (token row n, head h) are
 *            contiguous at k + n * k_token + h * k_head (strides in elements,
 *            multiples of 8: e.g. both halves of a kv_b product [N, heads, 256])
 *   k_pe     bf16, the 64 unrotated values of row n at k_pe + n * pe_token
 *            (a multiple of 8); rotated as RoPE above, angle formed in double
 *   P        int [B] in DEVICE memory; -1 marks an idle sequence: nothing is
 *            appended for it
 *   T, cu    cu NULL: T tokens each, row n = b * T + t, N = B * T.  Else cu is
 *            int [B + 1] in DEVICE memory, sequence b's rows are cu[b] ..
 *            cu[b + 1] - 1, at most T of them (0 is allowed), N >= cu[B].
 *            The launch covers B times the pages that min(T, N) tokens touch:
 *            one very long prompt among hundreds of short ones (600 with one
 *            of 32,768: 20 ms at 64 heads) is better in a call of its own
 *   params   rope_base (eps, softmax_scale, delta_out, timing: not used)
 *   workspace mla_workspace_size(MLA_MODE_PAGED_APPEND, B, T, 0)
 * Scales: with k the smallest integer in [-60, 60] for which the new tokens
 * of a page and head have amax <= 448 * 2^k, the page's scale becomes 2^k; in
 * a page that already holds tokens (P[b] not on a page's start) it only grows:
 * the larger of that and the old scale (any positive number), and where it
 * grows the codes already there are re-expressed at the new scale (rounded
 * again).  Code = x / scale rounded to
 * nearest even, saturating at +-448 (an infinity gives the page 2^60); NaN
 * stays NaN and does not count for amax.  Slots behind the last token, and
 * every other page, are left as they were.
 * A P[b] below -1, T_b outside [0, T], rows outside [0, N), positions past
 * max_pages * page or a page number outside [0, n_pages) cannot be checked on
 * the host: the kernel skips that sequence (or page) and mla_device_status
 * then returns MLA_ERR_INVALID_ARG.
 * Errors: INVALID_ARG (null pointer, B, T or N < 1, B or N > 2^24, T > 2^30,
 * N < B * T without cu, B times the pages that min(T, N) tokens touch > 2^22
 * where B * T > 2^24, a stride not a multiple of 8 or below 0), UNSUPPORTED (page, heads), ALIGNMENT,
 * WORKSPACE, CUDA. */
int mla_paged_append(const mla_paged_cache_t* cache, const mla_params_t* params, const void* k, long long k_token,
                     long long k_head, const void* v, long long v_token, long long v_head, const void* k_pe,
                     long long pe_token, const int* P, const int* cu, int B, int T, int N, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Attention of T new tokens per sequence (1 for a decode step, up to 8 to
 * verify drafted tokens) over the paged cache, which already holds them.
 * Query t of sequence b sits at position i = P[b] + t and sees key j iff
 * j <= i and, with window > 0, i - j < window or j < sinks (the first `sinks`
 * positions stay visible).
 *   q        bf16, row b * T + t at q + row * q_row: heads x [128 nope | 64 pe],
 *            pe rotated (the q_b product after RoPE); q_row a multiple of 8,
 *            >= heads * 192
 *   out      bf16, row b * T + t at out + row * out_row: heads x 128; out_row a
 *            multiple of 8, >= heads * 128
 *   P        int [B] in DEVICE memory, -1 .. P_max; P[b] = -1 marks an idle
 *            sequence (its output rows are zeros).  P_max sizes the launch;
 *            P_max + T <= max_pages * page.  A query sees at most 2^24 keys:
 *            P_max + T, or window + T - 1 + sinks, is at most that
 *   window   0 = every key; sinks is then ignored
 *   params   softmax_scale (the others are not used)
 *   workspace mla_workspace_size(MLA_MODE_PAGED_ATTN, B, T, 0); not shared by
 *            calls that may run concurrently, or by two captured graphs that may
 * Keys that no query of the sequence sees are not used, whatever their pages
 * hold (table entries of pages without a visible key are not looked at, so
 * pages that a window has passed can be given back).  A key that one query
 * sees has weight zero for the others; a NaN among its values reaches those
 * of its call too.  Scores, softmax statistics and sums are float32.  For the
 * product with V the weights of the up to 32 keys that a page holds of a tile
 * are rounded to float16, relative to the largest of them: by 2^-11 of the
 * weight, or 2^-40 of that largest one where it is below 2^-29 of it.  Query
 * values of the nope part that are below 2^-17 of the largest one of their row
 * and head are rounded to 2^-24 of the power of two below that one.
 * A P[b] outside [-1, P_max] is taken as idle, a page number outside
 * [0, n_pages) is clamped, and mla_device_status then returns
 * MLA_ERR_INVALID_ARG.
 * Errors: INVALID_ARG (null pointer, B < 1 or > 2^24, T < 1, P_max < 0, P_max +
 * T > max_pages * page, more than 2^24 keys, B times the tiles of 64 keys that
 * a sequence may take >= 2^31, window or sinks < 0, row strides), UNSUPPORTED
 * (T > 8, page, heads), ALIGNMENT, WORKSPACE, CUDA. */
int mla_paged_attention(const mla_paged_cache_t* cache, const mla_params_t* params, const void* q, long long q_row,
                        int B, int T, const int* P, int P_max, int window, int sinks, void* out, long long out_row,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Causal prefill attention under a sliding window with sinks, over the dense
 * rebuilt cache: query t of sequence b at position i = P0 + t sees key j iff
 * j <= i and (i - j < window or j < sinks).
 *   q        [B, T, 64 * 192]  per head [128 nope | 64 pe], pe rotated
 *   k_cache  [B, 64, cap, 192], v_cache [B, 64, cap, 128]: positions that some
 *            query sees are read
 *   out      [B, T, 64 * 128]
 *   window   >= 1;  sinks >= 0;  P0 >= 0, P0 + T <= cap
 *   params   softmax_scale (the others are not used)
 *   workspace mla_workspace_size(MLA_MODE_WINDOW_ATTN, B, T, 0)
 * Probabilities are rounded to bf16 for the product with V, as in mla_prefill.
 * A NaN or an infinity among a key's values may also reach queries that do not see
 * the key but share a tile with one that does (weight zero times it): those less than
 * 256 positions short of it, or past the end of its window.
 * Errors: INVALID_ARG (null pointer, sizes, B * T > 2^24), ALIGNMENT,
 * WORKSPACE, CUDA. */
int mla_window_attention(const mla_params_t* params, const void* q, int B, int T, int P0, const void* k_cache,
                         const void* v_cache, int cap, int window, int sinks, void* out, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Attention of several documents (ragged prompts, pieces of prompts behind
 * cached tokens, single new tokens) packed one after the other: rows cu_q[d] ..
 * cu_q[d + 1] - 1 of q are the n new tokens of document d, rows cu_k[d] ..
 * cu_k[d + 1] - 1 of the caches its L keys, the last n of which are the new
 * tokens' own.  Query t of a document sits at position i = L - n + t and sees
 * key j of its document (0 <= j < L), and no other document's, iff
 *   j < prefix[d], or j <= i and (window = 0, or i - j < window, or j < sinks).
 * A row that sees no key (a document with fewer keys than queries) is zeros.
 *   q        bf16, row n at q + n * q_row: 64 heads x [128 nope | 64 pe], pe
 *            rotated; q_row a multiple of 8, >= 64 * 192
 *   k_cache  bf16 [64, cap, 192], v_cache [64, cap, 128]: the layout of
 *            mla_prefill's caches at B = 1 (a score depends on the distance of
 *            its positions only, so keys and queries may be rotated by their
 *            place in the pack or in the document alike)
 *   out      bf16, row n at out + n * out_row: 64 x 128; out_row a multiple of
 *            8, >= 64 * 128.  Rows outside cu_q[0] .. cu_q[n_docs] are left as
 *            they were.  Must not overlap q, k_cache or v_cache
 *   cu_q, cu_k  int [n_docs + 1] in DEVICE memory, 0 <= cu[0] <= cu[1] <= ..,
 *            cu_q[n_docs] <= N, cu_k[n_docs] <= cap; empty documents are
 *            allowed; cu_k NULL: cu_q
 *   prefix   int [n_docs] in DEVICE memory, or NULL: none.  Tokens of the
 *            document that all its queries see (a prompt read from both sides);
 *            taken as at least 0 and at most L
 *   window   0 = no window; sinks is then ignored
 *   params   softmax_scale (the others are not used)
 *   workspace mla_workspace_size(MLA_MODE_DOCUMENTS, n_docs, N, 0)
 * Offsets out of range or order cannot be checked on the host: the kernel then
 * writes nothing and mla_device_status returns MLA_ERR_INVALID_ARG.
 * N and n_docs, all of the pack that the host knows, also choose the kernel: rows
 * for long documents (2,816 each on average; no window, or one of 2,048 keys) are
 * taken 256 at a time, which suits these and costs shorter ones up to a quarter, so
 * a captured call is best sized for the packs that it gets.  Results are within the
 * same bounds either way.
 * Probabilities are rounded to bf16 for the product with V, as in mla_prefill.
 * Keys behind the last one that a query of its tile of up to 256 sees are not used,
 * whatever the caches hold; a NaN or an infinity among the values of another key
 * may also reach queries of its document that do not see the key (weight zero
 * times it), but no other document.
 * Errors: INVALID_ARG (null pointer, N, cap < 1 or > 2^24, n_docs < 1 or > 2^20,
 * window or sinks < 0, row strides), ALIGNMENT (cu_q, cu_k, prefix: 4 bytes),
 * WORKSPACE, CUDA. */
int mla_document_attention(const mla_params_t* params, const void* q, long long q_row, int N, const int* cu_q,
                           const void* k_cache, const void* v_cache, int cap, const int* cu_k, const int* prefix,
                           int n_docs, int window, int sinks, void* out, long long out_row, void* workspace,
                           size_t workspace_bytes, void* stream);

/* One decode step of the sublayer against the paged 8-bit cache (64 heads):
 * sequence b's new token at position P[b] is appended to its pages (as
 * mla_paged_append) and attends to keys 0..P[b] (as mla_paged_attention with
 * T = 1, its own key as the cache holds it), window and sinks as there.
 *   x, out   [B, 7168]      (out may alias x exactly); idle rows (P[b] = -1)
 *                           append nothing and get out = x
 *   P        int [B] in DEVICE memory, -1 .. P_max; P_max + 1 <= max_pages * page,
 *            and the bounds on keys and tiles of mla_paged_attention
 *   workspace mla_workspace_size(MLA_MODE_DECODE_PAGED, B, P_max, 0)
 * The kv_b product is rounded to bf16 before it is quantized.
 * Errors: those of mla_decode_varlen and of the cache (UNSUPPORTED unless
 * heads = 64); device-side reports as mla_paged_attention. */
int mla_decode_paged(const mla_weights_t* w, const mla_params_t* params, const void* x, int B, const int* P,
                     int P_max, const mla_paged_cache_t* cache, int window, int sinks, void* out, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Prefill of T new tokens per sequence at positions P0..P0+T-1 into the paged
 * 8-bit cache (64 heads): their keys and values are appended to the pages, and
 * the tokens attend to the P0 cached positions (as the pages hold them, code *
 * scale rounded to bf16: exact for a power of two) and to
 * each other (as computed, not quantized), causally, with window > 0 only to
 * the last `window` keys and the first `sinks`.  P0 = 0, window = 0 computes
 * the out of mla_prefill.
 *   x, out   [B, T, 7168]  (out may alias x exactly)
 *   workspace mla_workspace_size(MLA_MODE_PREFILL_PAGED, B, T, P0 + T)
 * Requires P0 >= 0, P0 + T <= max_pages * page, B * T <= 2^24 and
 * B * (P0 + T) <= 2^26 (the workspace holds those positions in bf16).
 * Errors: INVALID_ARG, UNSUPPORTED (cache), ALIGNMENT, WORKSPACE, CUDA. */
int mla_prefill_paged(const mla_weights_t* w, const mla_params_t* params, const void* x, int B, int T, int P0,
                      const mla_paged_cache_t* cache, int window, int sinks, void* out, void* workspace,
                      size_t workspace_bytes, void* stream);

/* ---- pages of the paged cache -------------------------------------------------
 * Who holds a page, kept on the device: a pool is the cache's table with one
 * row per sequence, and the number of holds on each page.  The calls below
 * change both on `stream`, without a word from the host, so a captured serving
 * step can take, share and give back pages on every replay.
 *   table    int [rows, max_pages], the same memory as the cache's table: the
 *            pages of each sequence in order, -1 where there is none
 *   refs     int [n_pages]: table entries that hold the page (and holds of the
 *            user's own, e.g. of a stored prefix); 0 = the page is free
 * All -1 and all 0 is an empty pool.  Pages are taken lowest number first, in
 * the order of the list and then of the positions, so a call has one result.
 * Lists are int [n] in DEVICE memory (4-byte aligned), 1 <= n <= 2^20; P[i]
 * counts positions, ceil(P[i] / page) entries of a row hold P[i] of them.
 * Calls on one pool are ordered by their stream; two calls, or a call and one
 * that reads the cache, must not overlap.  All entries of a list see the pool as
 * it was before the call.
 * An entry that cannot be carried out (a row outside [0, rows), P[i] outside
 * [0, max_pages * page], what the calls name below) is skipped, and
 * mla_device_status then returns MLA_ERR_INVALID_ARG. */
typedef struct {
  int* table;
  int* refs;
  int rows, max_pages, n_pages, page;
} mla_page_pool_t;

/* Gives back the pages of rows[i] behind its first P[i] positions (0: all of
 * them; a rejected draft: the positions that stay): entry e >= ceil(P[i] / page)
 * becomes -1 and its page loses one hold.  A row may be listed more than once
 * (the smallest P counts); P[i] past the row's end gives nothing back.  Reported:
 * entries that are no page (they become -1), pages held by nobody (they stay free).
 * A row may be cut inside a page that others hold too (refs above 1: whole pages
 * that a fork shares, the parent's as well as the child's, or a hold of the user's
 * own).  It can then be read and forked, but must not be appended to as it is: its
 * next token would go into the others' page, and neither this call nor the reserve
 * or the append looks at that (a row that keeps what it had at its forks, as with
 * drafts that came after them, never ends in such a page).  mla_pages_fork of its
 * P[i] positions into an empty row gives that row a copy of the page of its own.
 *   workspace mla_workspace_size(MLA_MODE_PAGES, n, n_pages, rows), as in the
 *            calls below; not shared by calls that may run concurrently
 * Errors: INVALID_ARG (null pointer, n < 1 or > 2^20, rows < 1 or > 2^24,
 * max_pages < 1, n_pages < 1), UNSUPPORTED (page not 16, 32, 64 or 128,
 * n_pages * page above 31 bits, max_pages * page > 2^30), ALIGNMENT, WORKSPACE,
 * CUDA. */
int mla_pages_free(const mla_page_pool_t* pool, const int* rows, const int* P, int n, void* workspace,
                   size_t workspace_bytes, void* stream);

/* Takes free pages so that rows[i] holds its first P[i] positions: every entry
 * e < ceil(P[i] / page) that holds none gets one (its contents are what they
 * were), with one hold.  With too few free pages for the whole list nothing is
 * changed and mla_device_status returns MLA_ERR_NO_PAGES.  A row that is listed
 * again is skipped from the second time on and reported, entries past n_pages
 * are left and reported.  Errors as mla_pages_free. */
int mla_pages_reserve(const mla_page_pool_t* pool, const int* rows, const int* P, int n, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Row children[i] becomes a sequence that has the first P[i] positions of row
 * parents[i]: the whole pages are shared (one more hold each), and where P[i]
 * ends inside a page, its first P[i] % page tokens, in all heads and with the
 * page's scales, are copied into a new page, so that both sequences can go on
 * appending behind what they hold then (cut back further, into a page that they
 * share, see mla_pages_free).  The other slots of the new page are left as they were.  With too
 * few free pages nothing is changed (MLA_ERR_NO_PAGES, as mla_pages_reserve).
 * Skipped and reported: a child whose first ceil(P[i] / page) entries are not
 * all -1 or that an earlier entry of the list names, a parent that does not
 * hold P[i] positions in pages that somebody holds.  P[i] = 0 changes nothing.
 * Errors as mla_pages_free, and those of the cache (INVALID_ARG where its table,
 * n_pages, max_pages or page are not the pool's). */
int mla_pages_fork(const mla_paged_cache_t* cache, const mla_page_pool_t* pool, const int* parents, const int* children,
                   const int* P, int n, void* workspace, size_t workspace_bytes, void* stream);

/* Moves the pages that are held to the numbers 0 .. n_live - 1: those from
 * n_live on, in order, into the free ones below, in order; refs and the table
 * follow.  Pages from n_live on are free afterwards, their contents as before.
 *   moved    int [n_pages] in DEVICE memory: receives the new number of every
 *            page (its own where it stays, -1 where it was free), for what the
 *            user keeps page numbers in
 *   n_live   int [1] in DEVICE memory: receives the number of pages held
 * Reported: table entries that are no page, or a page held by nobody (they
 * become -1).
 *   workspace mla_workspace_size(MLA_MODE_PAGES, 1, n_pages, rows)
 * Errors as mla_pages_fork. */
int mla_pages_compact(const mla_paged_cache_t* cache, const mla_page_pool_t* pool, int* moved, int* n_live,
                      void* workspace, size_t workspace_bytes, void* stream);

/* Copies page src[i] of one cache (codes, scales, rotary keys) to page dst[i]
 * of another of the same page and heads, or of the same one; tables and holds
 * are the caller's.  Where a destination is named more than once, the last
 * entry counts; in one cache an entry whose source is written by another entry
 * is skipped; page numbers outside a cache are skipped; all three are reported
 * (MLA_ERR_INVALID_ARG from mla_device_status).  The tables of the caches are
 * not looked at.
 *   workspace mla_workspace_size(MLA_MODE_PAGES, n, to->n_pages, 0)
 * Errors: INVALID_ARG (null pointer, n < 1 or > 2^20, caches that overlap
 * without being one), UNSUPPORTED (page, heads, or different ones), ALIGNMENT,
 * WORKSPACE, CUDA. */
int mla_pages_copy(const mla_paged_cache_t* from, const mla_paged_cache_t* to, const int* src, const int* dst, int n,
                   void* workspace, size_t workspace_bytes, void* stream);

/* Synchronises `stream` and reads the device status word the last call on
 * this workspace left: MLA_OK, MLA_ERR_TIMEOUT if a bounded device wait
 * gave up (the kernel then skipped its remaining work and returned),
 * MLA_ERR_NO_PAGES (see the mla_pages_ calls), or
 * MLA_ERR_INVALID_ARG if numbers in device memory were outside the ranges
 * that the call states (positions, lengths, offsets, rows, pages).
 * The word describes one call only: every entry point clears it (and the
 * rest of the status region) on its stream before its first kernel, so a
 * caller that needs the status of a call must read it before enqueueing the
 * next call on the same workspace.
 * MLA_ERR_CUDA if the synchronisation itself fails. */
int mla_device_status(const void* workspace, void* stream);

/* Human-readable name of a status code (static string). */
const char* mla_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* MLA_H_ */
