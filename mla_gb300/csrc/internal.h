// Host-side declarations shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <utility>

#include "per_device.h"

namespace mla {

// Lets `kern` take `smem` bytes of dynamic shared memory on the current
// device: set by the kernel's first launch on each device.
template <typename... KArgs>
cudaError_t allow_smem(PerDevice<bool>& allowed, void (*kern)(KArgs...), size_t smem) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  bool done = false;
  return e != cudaSuccess ? e : allowed.get(dev, done, [&](bool&) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
}

// The same, and *n = clusters of two CTAs that fit on the current device at once.
template <typename... KArgs>
cudaError_t allow_smem_cluster2(PerDevice<int>& known, void (*kern)(KArgs...), size_t smem, int threads, int num_sms,
                                int* n) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : known.get(dev, *n, [&](int& max_clusters) {
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * num_sms);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t asked = cudaOccupancyMaxActiveClusters(&max_clusters, kern, &cfg);
    return asked == cudaSuccess && max_clusters < 1 ? cudaErrorInvalidConfiguration : asked;
  });
}

// Launch with programmatic stream serialization (see pdl_wait in common.cuh).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The same launch as clusters of `cluster` consecutive CTAs (grid.x a multiple of it).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kern)(KArgs...), int cluster, dim3 grid, dim3 block, size_t smem,
                               cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster2(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                Args&&... args) {
  return launch_pdl_cluster(kern, 2, grid, block, smem, stream, std::forward<Args>(args)...);
}

struct DevStatusHost {
  uint32_t* word;
  uint64_t wait_limit_ns;
};
// Words of the status region (256 bytes before the split-K counters, zeroed
// before every call): 0 = the status word, kWorkCounterWord = the persistent
// prefill attention's work counter.
constexpr int kWorkCounterWord = 16;

// ---- tensor maps ------------------------------------------------------------
// 2D bf16 tensor map over a row-major [rows, cols] matrix with row stride
// `ld` elements, box {box_cols, box_rows}, 128-byte swizzle (box_cols * 2
// must be 128).  Returns false if the driver rejects it.
bool make_tmap_bf16_2d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t ld,
                       uint32_t box_rows, uint32_t box_cols);

// Tensor maps for epilogue stores: 32 x 32 chunks of bf16 with 64-byte
// swizzle (64-byte chunk rows) and of float32 with 128-byte swizzle; the 3D
// bf16 map (the per-head K/V caches) stores 32 x 64 chunks with 128-byte
// swizzle, one whole 128-byte line of a cache row per chunk row.
bool make_tmap_store_bf16_2d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t ld);
bool make_tmap_store_f32_2d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t ld);
bool make_tmap_store_bf16_3d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t mid, uint64_t outer,
                             uint64_t mid_stride_bytes, uint64_t outer_stride_bytes);

// 3D bf16 tensor map over [outer][mid][inner] with byte strides for mid and
// outer, box {box_inner, box_mid, 1}, 128-byte swizzle.
bool make_tmap_bf16_3d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t mid, uint64_t outer,
                       uint64_t mid_stride_bytes, uint64_t outer_stride_bytes, uint32_t box_inner, uint32_t box_mid);
// bf16 rows of `atoms` x 64 numbers, `outer` of them; a box of box_rows rows and
// box_atoms of their atoms arrives atom after atom, each box_rows x 128 bytes
bool make_tmap_bf16_atoms(CUtensorMap* map, const void* base, uint64_t rows, uint64_t atoms, uint64_t outer,
                          uint64_t row_stride_bytes, uint64_t outer_stride_bytes, uint32_t box_rows, uint32_t box_atoms);

// 3D view of [outer][rows][128 bytes] (contiguous), box {128 bytes, box_rows,
// box_outer}, 128-byte swizzle: the paged cache's codes and rotary keys.
bool make_tmap_rows128_3d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t outer, uint32_t box_rows,
                          uint32_t box_outer);

// ---- GEMM (tcgen05, TMA, persistent) --------------------------------------
// D[b][m, n] = sum_k A[m, a_col0 + b*a_col_step + k] * Bmat(b)[n, k]
// A is K-major.  B is either K-major ([N, K] rows, weight layout) taken from
// B0 for n < n_split and from B1 (rows n - n_split) otherwise, or MN-major
// ([K, N] rows, N contiguous).  Row offset b_row0 + b*b_row_step selects the
// batch's slice of B (along N for K-major, along K for MN-major).
struct GemmShape {
  int M, N, K;
  int batches;
  int a_col0, a_col_step;
  int b_row0, b_row_step;
  int n_split;
  int ksplit;   // set by launch_gemm: K slices per tile (1 = no split)
  int kb_per;   // set by launch_gemm: 64-wide K blocks per slice
  int raster_g; // set by launch_gemm: tiles walk groups of raster_g row blocks,
                // row block fastest inside a group (1 = column block fastest)
};

// Split-K (used when a GEMM has too few output tiles to fill the GPU, as
// the decode projections with M <= 128 do): each CTA of a tile's K slice
// writes its float32 partial to its own slot; the last warp to finish a
// 32-row slice of the tile (counter per tile and quarter) sums the slots in
// slice order and runs the epilogue.  Units = tiles x slices <= kMaxSplitUnits.
// A slot holds a whole BM x BN tile (BM = 64 for M <= 64, else 128).
constexpr int kMaxSplitUnits = 160;
constexpr int kMaxSplitCounters = 960;
inline size_t split_part_bytes(int M) { return (size_t)kMaxSplitUnits * (M <= 64 ? 64 : 128) * 256 * sizeof(float); }

struct GemmOperands {
  const __nv_bfloat16* A;
  int lda;
  int a_rows;  // rows of the A tensor (>= M)
  const __nv_bfloat16* B0;
  int ldb0;
  int b0_rows;
  const __nv_bfloat16* B1;  // may be null
  int ldb1;
  int b1_rows;
  bool b_mn_major;
};

enum class Epi { kStoreBf16, kStoreF32, kQRope, kKVCache, kResidual, kSwiGLU };

struct EpiArgs {
  // kStoreBf16: out[row, c_col0 + batch*c_col_step + n]; kStoreF32: out_f32[row, n]
  __nv_bfloat16* out;
  float* out_f32;
  int ldo;
  int c_col0, c_col_step;
  // kQRope: q[row, n] with RoPE on columns 128..191 of each 192 block;
  //         position index of a row = row % t_mod into cs (float2 [.., 32])
  const float2* cs;
  int t_mod;
  // kQRope, register epilogue only (decode sizes): when set, the rotated pe
  // columns of row r, head h are also written to qpe_out[(r*64 + h)*576 + 512 ..]
  __nv_bfloat16* qpe_out;
  // kKVCache: K[b, h, t, 0:128] / V[b, h, t, 0:128] / K[b, h, t, 128:192] = kpe[row]
  //           b = row / t_mod, t = t_off + row % t_mod
  __nv_bfloat16* kc;
  __nv_bfloat16* vc;
  const __nv_bfloat16* kpe;
  int t_off;
  int cap;
  // kResidual: out[row, n] = x[row, n] + acc; delta[row, n] = acc (optional)
  // kSwiGLU: out[row, j] = SiLU(g) * u for j < N / 2, g from B0 (gate) row j,
  //          u from B1 (up) row j: each BN-wide tile holds BN / 2 gate columns
  //          then the BN / 2 up columns of the same j (B0, B1 both [N / 2, K])
  const __nv_bfloat16* x;
  float* delta;
  // split-K scratch (null: no split): partial slots and zeroed counters
  float* part;
  size_t part_bytes;
  int* counters;
  // rows of the K/V caches the kv_b epilogue may write (t < t_off + t_mod)
  int B;
  // kKVCache, decode with per-sequence lengths: row b's position pos[b]
  // (clamped into [0, pos_max]) replaces t_off; null otherwise
  const int* pos;
  int pos_max;
};

cudaError_t launch_gemm(const GemmShape& s, const GemmOperands& op, Epi epi, const EpiArgs& ea,
                        const DevStatusHost& st, int num_sms, cudaStream_t stream);

// The same product with B stored as FP8 (E4M3) codes and one power-of-two
// scale per 128 x 128 block (scales [rows / 128 rounded up, K / 128]); B is
// K-major ([N, K]), K a multiple of 128, one batch; the codes are stored
// block-major: block (i, j) = rows 128i.., columns 128j.. is 16 KB at
// ((i * K/128 + j) * 128) * 128, row-major inside (rows past the matrix are
// zero).  The codes are bulk-copied and dequantized to bf16 in shared memory
// (exact: the scales are powers of two); the product runs on the bf16
// tensor-core path.  Decode-size M: the weight bytes halve.
struct GemmW8Operands {
  const __nv_bfloat16* A;
  int lda;
  int a_rows;
  const uint8_t* B0;  // rows n < n_split
  int b0_rows;
  const float* s0;
  const uint8_t* B1;  // rows n - n_split (may be null)
  int b1_rows;
  const float* s1;
};
cudaError_t launch_gemm_w8(const GemmShape& s, const GemmW8Operands& op, Epi epi, const EpiArgs& ea,
                           const DevStatusHost& st, int num_sms, cudaStream_t stream);

// bf16 [rows, cols] (cols a multiple of 128) -> E4M3 codes, block-major with
// the row count padded to 128 (zeros), and scales [ceil(rows/128), cols/128]
cudaError_t launch_fp8_quantize(const __nv_bfloat16* w, int rows, int cols, uint8_t* codes, float* scales,
                                cudaStream_t stream);

// ---- row kernels --------------------------------------------------------------
cudaError_t launch_rmsnorm_rows(const __nv_bfloat16* x, const __nv_bfloat16* g, __nv_bfloat16* y, int rows,
                                float eps, cudaStream_t stream);
// Split the A-projection output ca [rows, 2112] (float32) into RMSNorm(c^Q) [rows,1536],
// RMSNorm(c^KV) [rows,512] and RoPE(k_pe) [rows,64]; optional latent cache
// copies at ckv_cache[b, t_off + t] / kpe_cache[b, t_off + t]; also writes the
// RoPE table cs[t] = (cos, sin)((pos0 + t) theta_i) that the q_b epilogue reads.
struct LatentArgs {
  const float* ca;
  const __nv_bfloat16* g_qa;
  const __nv_bfloat16* g_kva;
  float2* cs;              // RoPE table [t_mod, 32] written here (rows of batch 0)
  double inv_freq[32];     // theta_i = base^(-2i/64), computed on the host in double
  int pos0;                // position of t = 0
  __nv_bfloat16* cq;
  __nv_bfloat16* ckv;
  __nv_bfloat16* kpe;
  __nv_bfloat16* ckv_cache;
  __nv_bfloat16* kpe_cache;
  int rows, t_mod, t_off, cap;
  float eps;
  // decode with per-sequence lengths: row r sits at position pos[r] (cache
  // row and RoPE angle; cs then holds one entry per row); positions outside
  // [0, pos_max] set kStatusBadLength in *status and are clamped
  const int* pos;
  int pos_max;
  uint32_t* status;
  bool idle_ok;            // pos[r] = -1 marks an idle row (taken as position 0, not reported)
};
cudaError_t launch_latent_split(const LatentArgs& a, cudaStream_t stream);

// ---- attention ----------------------------------------------------------------
struct PrefillAttnArgs {
  const __nv_bfloat16* q;   // [B*T, 64*192], queries at positions past..past+T-1
  const __nv_bfloat16* k;   // [B, 64, cap, 192], keys 0..past+T-1
  const __nv_bfloat16* v;   // [B, 64, cap, 128]
  __nv_bfloat16* o;         // [B*T, 64*128]
  int B, T, cap;
  float scale;
  int past;                 // keys before the first query (chunked prefill), 0 otherwise
  // sliding window (0 = none): the query at position i sees key j <= i iff
  // i - j < window or j < sinks
  int window = 0, sinks = 0;
};
cudaError_t launch_prefill_attention(const PrefillAttnArgs& a, const DevStatusHost& st, int num_sms,
                                     cudaStream_t stream);

// Attention over packed documents: rows cu_q[d] .. cu_q[d + 1] - 1 of q against
// rows cu_k[d] .. of every head's keys and values (cu_k null: cu_q); see
// mla_document_attention for the mask.
struct DocAttnArgs {
  const __nv_bfloat16* q;   // row n at q + n * q_row: 64 x 192
  const __nv_bfloat16* k;   // [64, cap, 192]
  const __nv_bfloat16* v;   // [64, cap, 128]
  __nv_bfloat16* o;         // row n at o + n * o_row: 64 x 128
  long long q_row, o_row;
  const int* cu_q;
  const int* cu_k;
  const int* prefix;        // [n_docs] or null
  int N, cap, n_docs, window, sinks;
  float scale;
  uint8_t* plan;            // kDocTileBytes for its head and for each of doc_tiles_at_most() tiles
  int* first_tile;          // [n_docs] of many documents
};
constexpr int kDocTileBytes = 48;
constexpr int kNoWindow = 1 << 29;
inline long long doc_tiles_at_most(int N, int n_docs) {
  const long long n = (long long)N / 128 + n_docs;  // whole tiles, and a partial one a document
  return n < N ? n : N;
}
cudaError_t launch_document_attention(const DocAttnArgs& a, const DevStatusHost& st, int num_sms, cudaStream_t stream);

struct DecodeAttnArgs {
  const __nv_bfloat16* q;   // [B, 64*192]
  const __nv_bfloat16* k;   // [B, 64, cap, 192]
  const __nv_bfloat16* v;   // [B, 64, cap, 128]
  __nv_bfloat16* o;         // [B, 64*128]
  float* part_o;            // [B*64*splits, 128] split partials
  float2* part_ml;          // [B*64*splits] (max, sum)
  int B, L, cap, splits;    // L = keys attended (P + 1); with lens_pos: the largest P_b + 1
  float scale;
  const int* lens_pos;      // optional per-sequence P_b (keys 0..P_b), clamped into [0, L - 1]
};
int decode_splits(int B, int L, int num_sms);
cudaError_t launch_decode_attention(const DecodeAttnArgs& a, const DevStatusHost& st, cudaStream_t stream,
                                    int* launches);

struct LatentAttnArgs {
  const __nv_bfloat16* qlat;  // [B, 64, 576] (absorbed q_nope | rotated q_pe)
  const __nv_bfloat16* ckv;   // [B, cap, 512]
  const __nv_bfloat16* kpe;   // [B, cap, 64]
  __nv_bfloat16* olat;        // [B, 64, 512]
  float* part_o;              // [2*ctas, 64, 512]: two partial slots per CTA
  float2* part_ml;            // [2*ctas, 64]
  int B, L, cap, ctas;        // ctas = latent_ctas(B, L, SMs); with pos: L = the largest P_b + 1
  float scale;
  // decode with per-sequence lengths: P_b = pos[b] (clamped into [0, L - 1])
  // and the work plan that latent_plan_kernel writes (null: every sequence L keys)
  const int* pos;
  int* plan;                  // [latent_plan_ints(B, ctas)] workspace, written by the launch
  // sequences per cache plane: sequence b reads plane b / kv_div of the
  // caches (absorbed chunked prefill: each new token is a sequence of its own)
  int kv_div = 1;
};
int latent_ctas(int B, int L, int num_sms);
// Work plan of the latent decode for per-sequence lengths: plan[0..B] =
// first flattened 64-key tile of each sequence (plan[B] = total), then per
// CTA g: (first sequence, first tile within it, tile count).  Written by a
// one-CTA kernel that launch_latent_attention runs first when pos is set.
inline size_t latent_plan_ints(int B, int ctas) { return (size_t)B + 1 + 3 * (size_t)ctas; }
cudaError_t launch_latent_attention(const LatentAttnArgs& a, const DevStatusHost& st, cudaStream_t stream,
                                    int* launches);
// pos[i] = p0 + i % t for i < n (the positions of a chunk's tokens, row-major
// over (sequence, token)).
cudaError_t launch_chunk_positions(int* pos, int n, int t, int p0, cudaStream_t stream);

// ---- paged 8-bit cache ---------------------------------------------------------
// Pages of `page` (a power of two, 16..128) tokens; codes E4M3 [n_pages, heads,
// page, 128], one scale per page and head, rotary keys bf16 [n_pages, page, 64],
// table [B, max_pages].
struct PagedCache {
  uint8_t* k_codes;
  uint8_t* v_codes;
  __nv_bfloat16* k_pe;
  float* k_scales;
  float* v_scales;
  const int* table;
  int n_pages, max_pages, page, heads;
};

// Status words of the paged operators.  They start no memset: word 0 is
// written by their first CTA and word kStatusExtraWord is the number of
// further words, from word kStatusExtraFirst on, that the host ORs in (one
// per CTA, each CTA storing its own).  Entry points that clear the region
// leave that number zero.
constexpr int kStatusExtraWord = 1;
constexpr int kStatusExtraFirst = 64;
constexpr int kPagedMaxCtas = 256;
constexpr int kMaxStatusExtra = kPagedMaxCtas;

struct PagedAppendArgs {
  PagedCache c;
  // source row of sequence b's token t: (cu ? cu[b] : b * T) + t; keys at
  // k + b * k_seq + row_or_t * k_token + h * k_head, where row_or_t is the
  // row if k_seq == 0 and t otherwise (values alike)
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long k_seq, k_token, k_head, v_seq, v_token, v_head;
  const __nv_bfloat16* pe;     // unrotated rotary keys, row n at n * pe_token ...
  const float* pe_f32;         // ... or in float32 (the A-projection's output); one of the two
  long long pe_token;
  const int* P;                // per-sequence first position (-1: idle, at most p_max), or null: p0 for all
  int p0, p_max;
  const int* cu;               // row offsets [B + 1], or null: T rows each
  int B, T, N;
  double inv_freq[32];
  uint32_t* status;
  bool status_cleared;         // the caller cleared the status region: OR into it
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream);
// Pages that T tokens of one sequence may touch, wherever they begin; times B at most 2^24.
inline int paged_append_pages(int T, int page) { return (T - 1 + page - 1) / page + 1; }

// Positions of the dense caches K [B, heads, cap, 192], V [B, heads, cap, 128]
// filled with the paged ones' values (code * scale in bf16, exact where the
// scale is a power of two): positions j < P with j >= from or j < first, of
// every sequence.
struct PagedGatherArgs {
  PagedCache c;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  int B, P, cap, from, first;
  uint32_t* status;            // cleared by the caller
};
cudaError_t launch_paged_gather(const PagedGatherArgs& a, cudaStream_t stream);

struct PagedAttnArgs {
  PagedCache c;
  const __nv_bfloat16* q;      // row b*T + t at q + row * q_row: heads x 192
  __nv_bfloat16* o;            // row b*T + t at o + row * o_row: heads x 128
  long long q_row, o_row;
  const int* P;
  int B, T, P_max, window, sinks;
  float scale;
  uint32_t* status;
  bool status_cleared;
  float* part_o;               // [2 * kPagedMaxCtas][T][4 heads][128]
  float2* part_ml;             // [2 * kPagedMaxCtas][T][4 heads]
  int* first_unit;             // [B + 1]: units of work of the sequences before b, one head group
};
constexpr int kPagedMaxT = 8;
// The most tiles of 64 keys that a sequence can have, plus one times B at most INT32_MAX.
inline long long paged_attention_tiles(int P_max, int T, int window, int sinks) {
  const long long all = ((long long)P_max + T + 63) / 64;
  if (!window) return all;
  const long long seen = ((long long)window + T - 2) / 64 + 2 + ((long long)sinks + 63) / 64;
  return seen < all ? seen : all;
}
cudaError_t launch_paged_attention(const PagedAttnArgs& a, const DevStatusHost& st, int num_sms, cudaStream_t stream,
                                   int* launches);

// ---- pages of the paged cache -----------------------------------------------------
// table [rows, max_pages] (below 0: no page) and refs [n_pages], the holds on
// each page (0: free).
struct PagePool {
  int* table;
  int* refs;
  int rows, max_pages, n_pages, page;
};
// Scratch of the plan; all but status is written before it is read.
struct PagePlanArgs {
  PagePool pool;
  const int* rows;             // the list: rows of the table (fork: the children) ...
  const int* parents;          // ... fork: the rows that they follow ...
  const int* P;                // ... and positions
  int n;
  int* need;                   // [n] pages that an entry takes, -1: it is skipped
  int* first;                  // [n] pages taken by the entries before, -1: skipped
  int* claims;                 // [rows] of large tables: the first entry that names the row
  uint32_t* bits;              // [n_pages / 32, whole segments] free pages
  int* seg;                    // free pages before each segment of 1,024
  int* fresh;                  // [n_pages] free pages by rank: those to take, or to move to
  int* from;                   // [n_pages] compact: the pages to move
  int* moved;                  // [n_pages] compact: every page's new number, -1: free
  int* n_live;                 // [1] compact
  int* head;                   // [2] {whether the pages suffice, pages taken} or {live pages, moves}
  uint32_t* status;
};
cudaError_t launch_pages_free(const PagePool& p, const int* rows, const int* P, int n, uint32_t* status,
                              cudaStream_t stream);
cudaError_t launch_pages_reserve(const PagePlanArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_pages_fork(const PagedCache& c, const PagePlanArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_pages_compact(const PagedCache& c, const PagePlanArgs& a, int num_sms, cudaStream_t stream);
struct PageCopyArgs {
  PagedCache from, to;         // of one page and head count
  bool same;                   // from and to are one cache
  const int* src;
  const int* dst;
  int n;
  int* claims;                 // [to.n_pages]
  uint32_t* status;
};
cudaError_t launch_pages_copy(const PageCopyArgs& a, int num_sms, cudaStream_t stream);

// qlat[b, h, 512:576] = q[b, h*192 + 128 : h*192 + 192]
cudaError_t launch_copy_qpe(const __nv_bfloat16* q, __nv_bfloat16* qlat, int B, cudaStream_t stream);

}  // namespace mla
