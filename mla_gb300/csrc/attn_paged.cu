// Attention of a few new tokens per sequence over the paged 8-bit cache.
//
// Scores s_j = scale * (kscale * (q_nope . code_j) + q_pe . kpe_j), softmax in
// float32 over the visible keys, o = sum_j p_j vscale * code_j: 256 bytes of
// codes per (head, key) and 128 bytes of rotary key per key for all heads,
// read once; about 5 flop per byte and query, so HBM bounds it as long as the
// arithmetic on the codes keeps up.  On CUDA cores it would not (two flops a
// code and a conversion at 6.8 TB/s are near the issue limit), so both
// products run on mma.sync m16n8k16 with keys (then value dimensions) as the
// 16 rows and the queries as the 8 columns: tcgen05 needs its operands in
// shared memory in 16 bits, i.e. a written copy of every converted tile, where
// mma.sync takes the converted codes from registers, and the tensor work is
// small either way.
//
// Work: tiles of 64 keys of a group of 4 heads, flattened in (sequence, head
// group, tile) order and cut into equal ranges, one per CTA (one CTA per SM).
// A sequence and head group counts kPieceCost units more than its tiles, for
// loading its queries and writing its rows (without it the CTAs with many
// short sequences ended last: 16 sequences of 100 to 4000 keys, four queries
// each, 42.0 us against 37.5).
// The lengths are device data: every CTA scans them for its own range.  A
// piece of a sequence and head group that lies in one CTA is written
// directly; pieces that a cut separates are left as partials (at most two per
// CTA) and merged by paged_combine_kernel, in order.  (Merging in the last of
// the CTAs to arrive instead, counted by atomics, took as long: 93 against 95
// us at one sequence of 32,818 keys, 391 against 381 at 32 ragged ones.)
//
// CTA, 384 threads: warps 8..11 fill a 3-stage ring (72 KB a stage) with tiles,
// page by page from the table, whose entries they read ahead: warp 8 the key
// codes (4 x 64 x 128 bytes), 9 the value codes, 10 the 64 rotary keys (TMA),
// 11 the scales (plain loads).  One thread issuing all of a tile's copies was
// the limit with 16-token pages, 20 copies a tile: 32 sequences of up to 8192
// keys 463 us, with four warps 382 us.  Warps 2h and 2h + 1 take the first and
// last 32 keys of each tile for head h of the group (against every second tile
// each, which holds a stage for longer: 64 x 1001 keys 169 us against 177 us):
//   * S^T = K Q^T: a thread's 16-byte loads hold 16 consecutive dimensions of
//     one key, which are taken as the k index of four MMAs in the order in
//     which they come (Q's fragments are laid out in the same order).  Loads
//     hit distinct banks: rows are 128 bytes, 16-byte chunk c of row r sits at
//     c ^ (r & 7) (TMA's 128-byte swizzle), a quad reads chunks 2t + i.
//   * codes become float16 exactly (cvt e4m3x2 -> f16x2); q_nope is scaled by
//     a power of two per row so that its largest element is in [1, 2) (bf16's
//     8 bits fit float16's 11; elements below 2^-14 of the largest lose bits
//     below 2^-24 of it).  The rotary part is a bf16 MMA with its own sum.
//   * softmax on the accumulator fragments, in float32: a running maximum per
//     query, moved only when it grows by more than 2^8, and the sum of p.
//   * O^T = V^T P^T: the weights of the 32 keys (16 with 16-token pages) that
//     share a value scale, over the largest of them and times 2^15, are rounded
//     to float16: relative 2^-11, an eighth of the output's own bf16 rounding,
//     down to 2^-29 of the largest, and 2^-40 of it below.  They are transposed
//     8 x 8 (movmatrix) into the B operand; V codes of two keys are interleaved by
//     byte permutes into A fragments, a thread's 16 bytes being 16 rows.  The
//     sum of those keys enters the accumulators in float32, times the value
//     scale and the largest weight: neither a page whose scale is far above
//     its visible values nor a key that outweighs a long context by far takes
//     bits from the other pages.  (With weight times scale rounded against one
//     running maximum, a page whose scale was 2^24 times what its visible
//     values need took a third of the output.  It costs nothing at 64-token
//     pages, 64 x 1001 keys 170 us; with 16-token ones, two maxima a tile, 32
//     ragged sequences take 379 us for 370, four drafts on 32-token ones 39.6
//     for 37.3.)
// Keys that no query sees give weight zero and their value codes are cleared
// (they may decode to NaN).
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mla {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kWeightScale = 32768.f;    // of the float16 weights: the largest one, 2^15

constexpr int kTile = 64, kStages = 3, kGroup = 4;
constexpr int kThreads = 384;
constexpr int kPieceCost = 1;
constexpr uint32_t kCodeBytes = kGroup * kTile * 128;
constexpr uint32_t kVOff = kCodeBytes, kPeOff = 2 * kCodeBytes;
constexpr uint32_t kStageBytes = 2 * kCodeBytes + kTile * 128;
constexpr uint32_t kMergeOff = kStages * kStageBytes;
constexpr int kMergeRows = 4;
constexpr uint32_t kBarOff = kMergeOff + kGroup * kMergeRows * 128 * 4;
constexpr uint32_t kSmemBytes = kBarOff + 1024 + 1024;
static_assert(kSmemBytes <= 232448, "paged attention shared memory");

struct Bars {
  uint64_t full[kStages], empty[kStages];
  float scales[kStages][2][kTile / 16][kGroup];  // [k, v][page of the tile][head]
  float2 ml[kGroup][kMergeRows];
  int scan[kThreads / 32];
  int first_b, first_g, first_t;
  long long tiles[2];  // tiles before this CTA's range, and before the next one's
  int abort;
};
static_assert(sizeof(Bars) <= 1024, "barrier block");

// A sequence's keys: positions p .. p + T - 1 are its queries, keys j < len
// with j >= w0 or j < n_first are seen by at least one of them.  Its tiles:
// n_sink over the sinks, then those from w0 on; an idle sequence has one tile
// without visible keys (which writes its zeros).
struct Seq {
  int p, len, w0, n_first, n_sink, t0, nt;
  bool bad;
  __device__ __forceinline__ void read(const PagedAttnArgs& a, int b) {
    const int x = b < a.B ? a.P[b] : -1;
    bad = x < -1 || x > a.P_max;
    p = bad ? -1 : x;
    len = p < 0 ? 0 : p + a.T;
    w0 = a.window ? max(0, p - a.window + 1) : 0;
    n_first = min(a.sinks, w0);
    t0 = w0 / kTile;
    n_sink = min((n_first + kTile - 1) / kTile, t0);
    nt = p < 0 ? 1 : n_sink + (len - 1) / kTile - t0 + 1;
  }
  __device__ __forceinline__ int key0(int ti) const { return (ti < n_sink ? ti : ti - n_sink + t0) * kTile; }
  // whether a query sees one of the keys j .. j + n - 1
  __device__ __forceinline__ bool sees(int j, int n) const { return j < len && (j + n > w0 || j < n_first); }
};

struct Walk {
  int b, grp, ti;
  Seq s;
  __device__ __forceinline__ void start(const PagedAttnArgs& a, const Bars* bar) {
    b = bar->first_b;
    grp = bar->first_g;
    ti = bar->first_t;
    s.read(a, b);
  }
  __device__ __forceinline__ void next(const PagedAttnArgs& a, int groups) {
    if (++ti < s.nt) return;
    ti = 0;
    if (++grp < groups) return;
    grp = 0;
    s.read(a, ++b);
  }
};

__device__ __forceinline__ long long range_start(int g, long long total, int C) {
  const long long x = g * total;
  return x <= UINT32_MAX ? (long long)((uint32_t)x / (uint32_t)C) : x / C;  // (a 64-bit division is a few hundred cycles)
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// four E4M3 codes -> two pairs of float16 (exact)
__device__ __forceinline__ void decode4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void lds128(uint4& v, uint32_t addr) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
}
// 8 x 8 matrix of 16-bit elements, row r = lane / 4, columns 2 * (lane % 4) and + 1, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The merge of a pair's halves: the second warp fills the pair's buffer, the
// first one reads it.  Named barriers 1 + head (filled) and 5 + head (read);
// each has 32 arrivals that do not wait and 32 that do.
template <int ID>
__device__ __forceinline__ void bar_arrive64() { asm volatile("bar.arrive %0, 64;" ::"n"(ID) : "memory"); }
template <int ID>
__device__ __forceinline__ void bar_sync64() { asm volatile("bar.sync %0, 64;" ::"n"(ID) : "memory"); }
__device__ __forceinline__ void pair_arrive(int k) {
  switch (k) {
    case 0: bar_arrive64<1>(); break;
    case 1: bar_arrive64<2>(); break;
    case 2: bar_arrive64<3>(); break;
    case 3: bar_arrive64<4>(); break;
    case 4: bar_arrive64<5>(); break;
    case 5: bar_arrive64<6>(); break;
    case 6: bar_arrive64<7>(); break;
    default: bar_arrive64<8>(); break;
  }
}
__device__ __forceinline__ void pair_wait(int k) {
  switch (k) {
    case 0: bar_sync64<1>(); break;
    case 1: bar_sync64<2>(); break;
    case 2: bar_sync64<3>(); break;
    case 3: bar_sync64<4>(); break;
    case 4: bar_sync64<5>(); break;
    case 5: bar_sync64<6>(); break;
    case 6: bar_sync64<7>(); break;
    default: bar_sync64<8>(); break;
  }
}

// ONE: one query per sequence (a fragment's second column is not there).
// TWO_PAGES: pages of 16 tokens, i.e. a warp's 32 keys of a tile lie in two.
template <bool ONE, bool TWO_PAGES>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmPe, const PagedAttnArgs a, uint64_t wait_limit_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bar = reinterpret_cast<Bars*>(smem + kBarOff);
  volatile int* abort_flag = &bar->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, C = gridDim.x;
  const int groups = a.c.heads / kGroup;
  const int tp = min(a.c.page, kTile);  // tokens of one page in a tile

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar->full[i], 4);
      mbar_init(&bar->empty[i], 2 * kGroup);
    }
    bar->abort = 0;
    bar->first_b = bar->first_g = bar->first_t = 0;
    bar->tiles[0] = bar->tiles[1] = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmPe);
  }
  pdl_launch_dependents();
  pdl_wait();
  const DevStatus st{a.status_cleared ? a.status : a.status + kStatusExtraFirst + cta, wait_limit_ns};
  if (tid == 0 && !a.status_cleared) {
    *st.word = 0u;
    if (cta == 0) {
      a.status[0] = 0u;
      a.status[kStatusExtraWord] = (uint32_t)C;
    }
  }

  // This CTA's range of the flattened units: per sequence and head group
  // kPieceCost units, then one per tile.
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  int sum = 0;  // units of sequences b0 .. b1 - 1, for one head group
  Seq sq;
  for (int b = b0; b < b1; ++b) {
    sq.read(a, b);
    sum += sq.nt + kPieceCost;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) bar->scan[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += bar->scan[i];
    all += bar->scan[i];
  }
  const long long total = (long long)all * groups;
  {
    const int e0 = before + incl - sum;  // units before b0
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long x = range_start(cta + k, total, C);
      const bool mine = x >= (long long)e0 * groups && x < (long long)(e0 + sum) * groups;
      int e = e0;
      for (int b = b0; b < b1 && (mine || (cta == 0 && k == 0)); ++b) {
        sq.read(a, b);
        const int u = sq.nt + kPieceCost;
        if (cta == 0 && k == 0) a.first_unit[b] = e;
        if (x >= (long long)e * groups && x < (long long)(e + u) * groups) {
          const int r = (int)(x - (long long)e * groups);
          const int grp = r / u, t = max(0, r - grp * u - kPieceCost);
          if (k == 0) {
            bar->first_b = b;
            bar->first_g = grp;
            bar->first_t = t;
          }
          // units before x that are tiles
          bar->tiles[k] = (long long)(e - b * kPieceCost) * groups + (long long)grp * sq.nt + t;
        }
        e += u;
      }
      if (tid == 0 && x == total) bar->tiles[k] = (long long)(all - a.B * kPieceCost) * groups;
    }
    if (cta == 0 && tid == 0) a.first_unit[a.B] = all;
  }
  __syncthreads();
  const int R = (int)(bar->tiles[1] - bar->tiles[0]);
  Walk w;
  if (R > 0) w.start(a, bar);
  const int first_b = bar->first_b, first_g = bar->first_g;

  const int n_sub = kTile / tp;  // pages in a tile
  constexpr int kNone = INT_MIN;
  const int page_log = 31 - __clz(a.c.page);
  // page number of part `sub` of the walk's tile (kNone: no visible key there)
  auto entry = [&](int sub) {
    const int j = w.s.key0(w.ti) + sub * tp;
    return sub < n_sub && w.s.sees(j, tp) ? a.c.table[(size_t)w.b * a.c.max_pages + (j >> page_log)] : kNone;
  };
  auto page_of = [&](int ent) { return ent == kNone ? 0 : min(max(ent, 0), a.c.n_pages - 1); };

  if (warp >= 8 && warp < 11) {
    // ---- TMA: key codes, value codes, rotary keys ----
    if (R == 0) return;
    const CUtensorMap* map = warp == 8 ? &tmK : warp == 9 ? &tmV : &tmPe;
    const bool codes = warp < 10;
    const uint32_t at = warp == 8 ? 0 : warp == 9 ? kVOff : kPeOff;
    const uint32_t bytes = codes ? kCodeBytes : kTile * 128;
    bool bad = false;
    int ent = entry(lane);  // lane i: part i of the tile
    int issued = 0;
    for (int i = 0; i < R; ++i) {
      const int k0 = w.s.key0(w.ti), grp = w.grp, e = ent;
      bad |= w.s.bad || (e != kNone && (e < 0 || e >= a.c.n_pages));
      const int pid = page_of(e);
      if (i + 1 < R) {
        w.next(a, groups);
        ent = entry(lane);
      }
      const int stg = i % kStages;
      if (i >= kStages &&
          !__all_sync(0xffffffffu, mbar_wait(&bar->empty[stg], (i / kStages - 1) & 1, st, abort_flag, 81)))
        break;
      if (lane == 0) mbar_arrive_expect_tx(&bar->full[stg], bytes);
      uint8_t* dst = smem + stg * kStageBytes + at;
      for (int sub = 0; sub < n_sub; ++sub) {
        const int id = __shfl_sync(0xffffffffu, pid, sub);
        const int row = (k0 + sub * tp) & (a.c.page - 1);
        if (lane == 0) {
          if (codes)
            tma_load_3d(dst + sub * tp * 128 * kGroup, map, &bar->full[stg], 0, row, id * a.c.heads + grp * kGroup);
          else
            tma_load_3d(dst + sub * tp * 128, map, &bar->full[stg], 0, row, id);
        }
      }
      ++issued;
    }
    // no copy may still be in flight into shared memory
    for (int i = max(0, issued - kStages); i < issued; ++i)
      mbar_wait(&bar->full[i % kStages], (i / kStages) & 1, st, nullptr, 82);
    if (warp == 8 && __any_sync(0xffffffffu, bad) && lane == 0) atomicOr(st.word, kStatusBadLength);
    return;
  }
  if (warp == 11) {
    // ---- scales: lane = (part of the tile, key or value, head); entries two tiles ahead, scales one ----
    if (R == 0) return;
    const int sub = lane >> 3;
    const float* src = (lane & 4) ? a.c.v_scales : a.c.k_scales;
    auto scale_of = [&](int ent, int grp) {
      return ent == kNone ? 1.f : src[(size_t)page_of(ent) * a.c.heads + grp * kGroup + (lane & 3)];
    };
    // The queries of the walk's next piece into L1 (its rows are not read for
    // anything else, so the warps that need them would wait for HBM).
    auto touch_q = [&]() {
      if (w.ti != 0 || w.s.p < 0) return;
      for (int k = lane; k < a.T * 12; k += 32) {  // 4 heads x 384 bytes a row
        const int row = k / 12;
        const char* at = reinterpret_cast<const char*>(a.q + ((long long)w.b * a.T + row) * a.q_row +
                                                       w.grp * kGroup * 192) + (k - row * 12) * 128;
        uint32_t sink;
        asm volatile("ld.global.b32 %0, [%1];" : "=r"(sink) : "l"(at));
      }
    };
    float val = scale_of(entry(sub), w.grp);  // of tile i
    int ent = kNone, grp = 0;                 // of tile i + 1
    if (R > 1) {
      w.next(a, groups);
      ent = entry(sub);
      grp = w.grp;
      touch_q();
    }
    for (int i = 0; i < R; ++i) {
      const float cur = val;
      if (i + 1 < R) val = scale_of(ent, grp);
      if (i + 2 < R) {
        w.next(a, groups);
        ent = entry(sub);
        grp = w.grp;
        touch_q();
      }
      const int stg = i % kStages;
      if (i >= kStages &&
          !__all_sync(0xffffffffu, mbar_wait(&bar->empty[stg], (i / kStages - 1) & 1, st, abort_flag, 84)))
        break;
      (&bar->scales[stg][0][0][0])[(lane & 4 ? kTile / 16 * kGroup : 0) + sub * kGroup + (lane & 3)] = cur;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->full[stg]);
    }
    return;
  }

  // ---- warps 0..7: head hh of the group, keys half * 32 .. + 31 of each tile ----
  const int hh = warp >> 1, half = warp & 1;
  const int g = lane >> 2, t = lane & 3;
  const float sl2 = a.scale * kLog2e;
  float* merge = reinterpret_cast<float*>(smem + kMergeOff) + hh * kMergeRows * 128;
  constexpr int kKeys = kTile / 2, kBlocks = kKeys / 16, NE = ONE ? 1 : 2, kRefs = TWO_PAGES ? kBlocks : 1;
  uint32_t off16[kBlocks];  // byte offset of this head's 16-key blocks in the tile's K and V
  int sub16[kBlocks];       // and their page of the tile
#pragma unroll
  for (int ks = 0; ks < kBlocks; ++ks) {
    const int tok = half * kKeys + ks * 16;
    sub16[ks] = tok / tp;
    off16[ks] = (uint32_t)((sub16[ks] * kGroup + hh) * tp + (tok & (tp - 1))) * 128;
  }
  uint32_t qa[8][2], qp[4][2];  // Q's row g (B operand)
  float acc[8][4];              // O^T: dimensions 16g + 2i (+ 1 in [2], [3]), queries 2t and 2t + 1
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, qs[2] = {0.f, 0.f};  // of queries 2t and 2t + 1
  bool ok = true;
  if (R > 0 && half == 0) pair_arrive(4 + hh);  // the pair's buffer is free

  for (int i = 0; i < R; ++i) {
    const int stg = i % kStages;
    const bool seg_first = i == 0 || w.ti == 0;
    const bool seg_last = i == R - 1 || w.ti == w.s.nt - 1;
    const int head = w.grp * kGroup + hh;
    if (seg_first) {
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.f;
      // Q: dimensions 32t .. 32t+31 of the nope part, 16t .. 16t+15 of the rotary part of row g
      uint4 u[4], r[2];
      const bool row = g < a.T && w.s.p >= 0;
      const __nv_bfloat16* q = a.q + ((long long)w.b * a.T + g) * a.q_row + head * 192;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        u[c] = row ? reinterpret_cast<const uint4*>(q + 32 * t)[c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        r[c] = row ? reinterpret_cast<const uint4*>(q + 128 + 16 * t)[c] : make_uint4(0u, 0u, 0u, 0u);
      float top = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t x[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_bf16x2(x[e]);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = min(126, max(-126, (int)(__float_as_uint(top) >> 23) - 127));
      const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
      const float up = __uint_as_float((uint32_t)(127 + ex) << 23) * sl2;
      qs[0] = __shfl_sync(0xffffffffu, up, 8 * t);
      qs[1] = __shfl_sync(0xffffffffu, up, 8 * t + 4);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t x[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_bf16x2(x[e]);
          qa[c * 2 + (e >> 1)][e & 1] = pack_f16x2(f.x * down, f.y * down);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        qp[2 * c][0] = r[c].x;
        qp[2 * c][1] = r[c].y;
        qp[2 * c + 1][0] = r[c].z;
        qp[2 * c + 1][1] = r[c].w;
      }
    }
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&bar->full[stg], (i / kStages) & 1, st, abort_flag, 83));
    {
      const int a0 = w.s.key0(w.ti) + half * kKeys;  // this warp's first key
      if (ok && w.s.sees(a0, kKeys)) {
        const uint8_t* kb = smem + stg * kStageBytes;
        const uint8_t* vb = kb + kVOff;
        const uint8_t* pb = kb + kPeOff;
        // every query of the sequence sees all of these keys
        const bool full = a0 + kKeys - 1 <= w.s.p &&
                          (a.window == 0 || a0 > w.s.p + a.T - 1 - a.window || a0 + kKeys - 1 < a.sinks);
        float vsc[kBlocks];
        // scores of 16 keys at a time: keys g ([0], [1]) and g + 8 ([2], [3]) of queries 2t and 2t + 1
        float s[kBlocks][4];
#pragma unroll
        for (int ks = 0; ks < kBlocks; ++ks) {
          // a chain of dependent MMAs for each 64 dimensions of the nope part and each 32 of the rotary one
          float c[2][4] = {}, d[2][4] = {};
          const float ksc = bar->scales[stg][0][sub16[ks]][hh];
          vsc[ks] = bar->scales[stg][1][sub16[ks]][hh];
          const uint8_t* kr = kb + off16[ks] + (uint32_t)g * 128;
          const uint8_t* pr = pb + (uint32_t)(half * kKeys + ks * 16 + g) * 128;
          uint4 x[2], x8[2], y[2], y8[2];
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
            const uint32_t chunk = (uint32_t)(((2 * t + h2) ^ g) << 4);
            x[h2] = *reinterpret_cast<const uint4*>(kr + chunk);
            x8[h2] = *reinterpret_cast<const uint4*>(kr + 1024 + chunk);
            y[h2] = *reinterpret_cast<const uint4*>(pr + chunk);
            y8[h2] = *reinterpret_cast<const uint4*>(pr + 1024 + chunk);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              const uint32_t cw = e == 0 ? x[h2].x : e == 1 ? x[h2].y : e == 2 ? x[h2].z : x[h2].w;
              const uint32_t cw8 = e == 0 ? x8[h2].x : e == 1 ? x8[h2].y : e == 2 ? x8[h2].z : x8[h2].w;
              uint32_t b0, b1, b2, b3;
              decode4(cw, b0, b2);
              decode4(cw8, b1, b3);
              mma_f16(c[h2], b0, b1, b2, b3, qa[h2 * 4 + e][0], qa[h2 * 4 + e][1]);
              if (e == 0) mma_bf16(d[h2], y[h2].x, y8[h2].x, y[h2].y, y8[h2].y, qp[h2 * 2][0], qp[h2 * 2][1]);
              if (e == 2) mma_bf16(d[h2], y[h2].z, y8[h2].z, y[h2].w, y8[h2].w, qp[h2 * 2 + 1][0], qp[h2 * 2 + 1][1]);
            }
          }
          const float kq[2] = {ksc * qs[0], ksc * qs[1]};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if ((e & 1) < NE) s[ks][e] = fmaf(c[0][e] + c[1][e], kq[e & 1], (d[0][e] + d[1][e]) * sl2);
        }
        // V: keys 2t, 2t+1, 2t+8, 2t+9 of each 16, dimensions 16g .. 16g+15, loaded
        // ahead of the softmax (its shuffles would hold the loads back: 190 -> 184
        // us at 64 sequences under a window of 1,024)
        uint4 xv[kBlocks][4];
        {
          const uint32_t ce = (uint32_t)((g ^ (2 * t)) << 4), co = (uint32_t)((g ^ (2 * t + 1)) << 4);
#pragma unroll
          for (int ks = 0; ks < kBlocks; ++ks) {
            const uint32_t vr = smem_u32(vb) + off16[ks] + (uint32_t)(2 * t) * 128;
            lds128(xv[ks][0], vr + ce);
            lds128(xv[ks][1], vr + 128 + co);
            lds128(xv[ks][2], vr + 1024 + ce);
            lds128(xv[ks][3], vr + 1152 + co);
            if (!full) {
              const int j = a0 + ks * 16 + 2 * t;
              const uint4 z = make_uint4(0u, 0u, 0u, 0u);
              if (!w.s.sees(j, 1)) xv[ks][0] = z;
              if (!w.s.sees(j + 1, 1)) xv[ks][1] = z;
              if (!w.s.sees(j + 8, 1)) xv[ks][2] = z;
              if (!w.s.sees(j + 9, 1)) xv[ks][3] = z;
            }
          }
        }
        if (!full) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if ((e & 1) >= NE) continue;
            const int qi = w.s.p + min(2 * t + (e & 1), a.T - 1);  // the query's position
            const int lo = a.window ? qi - a.window : -1;
#pragma unroll
            for (int ks = 0; ks < kBlocks; ++ks) {
              const int j = a0 + ks * 16 + (e >> 1) * 8 + g;
              if (j > qi || (j <= lo && j >= a.sinks)) s[ks][e] = -INFINITY;
            }
          }
        }
        // maximum score per query and page, over the 8 lanes of its column
        float mx[2] = {-INFINITY, -INFINITY}, top[kRefs][2];
        bool need[2] = {false, false};
#pragma unroll
        for (int e = 0; e < NE; ++e) {
#pragma unroll
          for (int r = 0; r < kRefs; ++r) {
            float x = fmaxf(s[r][e], s[r][e + 2]);
            if (kRefs == 1) x = fmaxf(x, fmaxf(s[kBlocks - 1][e], s[kBlocks - 1][e + 2]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            top[r][e] = x;
            mx[e] = fmaxf(mx[e], x);
          }
          need[e] = mx[e] > m[e] + kRescaleThreshold;
        }
        if (__any_sync(0xffffffffu, need[0] | need[1])) {
          float alpha[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (e >= NE) {
              alpha[e] = 1.f;
              continue;
            }
            alpha[e] = need[e] ? ex2_approx(m[e] - mx[e]) : 1.f;
            if (need[e]) m[e] = mx[e];
            l[e] *= alpha[e];
          }
#pragma unroll
          for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][e] *= alpha[e & 1];
        }
        uint32_t pw[kBlocks][2];  // weights of keys 2t, 2t+1 (and 8 further) of query g
        float to_acc[kRefs][2];   // largest weight * value scale
#pragma unroll
        for (int ks = 0; ks < kBlocks; ++ks) {
          const int r = ks < kRefs ? ks : kRefs - 1;
          float p[4] = {0.f, 0.f, 0.f, 0.f};
          to_acc[r][1] = 0.f;
#pragma unroll
          for (int e = 0; e < NE; ++e) {
            const bool none = top[r][e] == -INFINITY;
            const float ref = none ? 0.f : top[r][e], f = none ? 0.f : ex2_approx(ref - m[e]);
            p[e] = ex2_approx(s[ks][e] - ref);
            p[e + 2] = ex2_approx(s[ks][e + 2] - ref);
            l[e] = fmaf(f, p[e] + p[e + 2], l[e]);
            to_acc[r][e] = f * (vsc[ks] * (1.f / kWeightScale));
          }
          pw[ks][0] = transpose8(pack_f16x2(p[0] * kWeightScale, p[1] * kWeightScale));
          pw[ks][1] = transpose8(pack_f16x2(p[2] * kWeightScale, p[3] * kWeightScale));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int r = 0; r < kRefs; ++r) {
            float c0[4] = {}, c1[4] = {};
#pragma unroll
            for (int ks = r; ks < kBlocks; ks += kRefs) {
              const uint4 (&x)[4] = xv[ks];
              uint32_t w4[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) w4[i] = e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w;
              uint32_t b0, b1, b2, b3;
              decode4(__byte_perm(w4[0], w4[1], 0x5140), b0, b1);
              decode4(__byte_perm(w4[2], w4[3], 0x5140), b2, b3);
              mma_f16(c0, b0, b1, b2, b3, pw[ks][0], pw[ks][1]);
              decode4(__byte_perm(w4[0], w4[1], 0x7362), b0, b1);
              decode4(__byte_perm(w4[2], w4[3], 0x7362), b2, b3);
              mma_f16(c1, b0, b1, b2, b3, pw[ks][0], pw[ks][1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if ((i & 1) >= NE) continue;
              acc[2 * e][i] = fmaf(c0[i], to_acc[r][i & 1], acc[2 * e][i]);
              acc[2 * e + 1][i] = fmaf(c1[i], to_acc[r][i & 1], acc[2 * e + 1][i]);
            }
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar->empty[stg]);

    if (seg_last) {
      // the pair's two halves become one, then the rows are written
#pragma unroll
      for (int e = 0; e < NE; ++e)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], o);
      for (int r0 = 0; r0 < a.T; r0 += kMergeRows) {
        if (half == 1) {
          pair_wait(4 + hh);  // the partner has read what was there
#pragma unroll
          for (int e = 0; e < NE; ++e) {
            const int row = 2 * t + e;
            if (row >= r0 && row < r0 + kMergeRows && row < a.T) {
              float* at = merge + (row - r0) * 128 + 16 * g;
#pragma unroll
              for (int c = 0; c < 4; ++c)
                reinterpret_cast<float4*>(at)[(c + (g >> 1)) & 3] =
                    make_float4(acc[2 * c][e], acc[2 * c][e + 2], acc[2 * c + 1][e], acc[2 * c + 1][e + 2]);
              if (g == 0) bar->ml[hh][row - r0] = make_float2(m[e], l[e]);
            }
          }
          pair_arrive(hh);
        } else {
          pair_wait(hh);
#pragma unroll
          for (int e = 0; e < NE; ++e) {
            const int row = 2 * t + e;
            if (row >= r0 && row < r0 + kMergeRows && row < a.T) {
              const float2 ml = bar->ml[hh][row - r0];
              const float mm = fmaxf(m[e], ml.x), ref = mm == -INFINITY ? 0.f : mm;
              const float f0 = ex2_approx(m[e] - ref), f1 = ex2_approx(ml.x - ref);
              m[e] = mm;
              l[e] = l[e] * f0 + ml.y * f1;
              const float* at = merge + (row - r0) * 128 + 16 * g;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float4 x = reinterpret_cast<const float4*>(at)[(c + (g >> 1)) & 3];
                acc[2 * c][e] = acc[2 * c][e] * f0 + x.x * f1;
                acc[2 * c][e + 2] = acc[2 * c][e + 2] * f0 + x.y * f1;
                acc[2 * c + 1][e] = acc[2 * c + 1][e] * f0 + x.z * f1;
                acc[2 * c + 1][e + 2] = acc[2 * c + 1][e + 2] * f0 + x.w * f1;
              }
            }
          }
          pair_arrive(4 + hh);
        }
      }
      if (ok && half == 0) {
        const bool whole = w.ti == w.s.nt - 1 && i >= w.ti;  // its first tile is in this CTA too
        const int slot = 2 * cta + (w.b == first_b && w.grp == first_g ? 0 : 1);
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          const int row = 2 * t + e;
          if (row >= a.T) continue;
          if (whole) {
            const float inv = l[e] > 0.f ? 1.f / l[e] : 0.f;
            uint4* d = reinterpret_cast<uint4*>(a.o + ((long long)w.b * a.T + row) * a.o_row + head * 128 + 16 * g);
#pragma unroll
            for (int c = 0; c < 2; ++c)
              d[c] = make_uint4(pack_bf16x2(acc[4 * c][e] * inv, acc[4 * c][e + 2] * inv),
                                pack_bf16x2(acc[4 * c + 1][e] * inv, acc[4 * c + 1][e + 2] * inv),
                                pack_bf16x2(acc[4 * c + 2][e] * inv, acc[4 * c + 2][e + 2] * inv),
                                pack_bf16x2(acc[4 * c + 3][e] * inv, acc[4 * c + 3][e + 2] * inv));
          } else {
            const size_t at = ((size_t)slot * a.T + row) * kGroup + hh;
            float4* d = reinterpret_cast<float4*>(a.part_o + at * 128 + 16 * g);
#pragma unroll
            for (int c = 0; c < 4; ++c)
              d[c] = make_float4(acc[2 * c][e], acc[2 * c][e + 2], acc[2 * c + 1][e], acc[2 * c + 1][e + 2]);
            if (g == 0) a.part_ml[at] = make_float2(m[e], l[e]);
          }
        }
      }
    }
    if (i + 1 < R) w.next(a, groups);
  }
  if (R > 0 && half == 1) pair_wait(4 + hh);  // the last arrival
}

// Merges the pieces of the (sequence, head group) pairs that a cut between
// CTAs separates; the others were written by paged_attn_kernel.  One warp per
// head and query, 4 dimensions a lane; pieces eight at a time, in order.
__global__ void __launch_bounds__(32 * kGroup) paged_combine_kernel(const PagedAttnArgs a, int C) {
  pdl_launch_dependents();
  pdl_wait();
  const int groups = a.c.heads / kGroup;
  const int t = blockIdx.y, b = blockIdx.x / groups, grp = blockIdx.x - b * groups;
  const int hh = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = a.first_unit[b], u = a.first_unit[b + 1] - e, all = a.first_unit[a.B];
  const long long total = (long long)all * groups;
  const long long xa = (long long)e * groups + (long long)grp * u;  // the pair's first unit
  // the CTA that holds unit x: the largest g with range_start(g) <= x
  auto cta_of = [&](long long x) {
    const long long n = (x + 1) * C - 1;
    return total * C <= INT_MAX ? (int)((uint32_t)n / (uint32_t)total) : (int)(n / total);
  };
  const int g0 = cta_of(xa + kPieceCost), g1 = cta_of(xa + u - 1);  // of the first and the last tile
  if (g0 == g1) return;
  // a CTA's first piece is in its slot 0; only g0 can have begun before this pair
  const int slot0 = 2 * g0 + (range_start(g0, total, C) >= xa ? 0 : 1);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = g0; k0 <= g1; k0 += 8) {
    float2 ml[8];
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int gg = k0 + k;
      ml[k] = make_float2(-INFINITY, 0.f);
      x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (gg > g1) continue;
      // with fewer units than CTAs some of them have none
      if (total < C && range_start(gg, total, C) == range_start(gg + 1, total, C)) continue;
      const size_t at = ((size_t)(gg == g0 ? slot0 : 2 * gg) * a.T + t) * kGroup + hh;
      ml[k] = a.part_ml[at];
      x[k] = reinterpret_cast<const float4*>(a.part_o + at * 128)[lane];
    }
    float mm = m;
#pragma unroll
    for (int k = 0; k < 8; ++k) mm = fmaxf(mm, ml[k].x);
    const float ref = mm == -INFINITY ? 0.f : mm;
    const float f = exp2f(m - ref);
    m = mm;
    l *= f;
    o.x *= f;
    o.y *= f;
    o.z *= f;
    o.w *= f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float wk = exp2f(ml[k].x - ref);
      l = fmaf(wk, ml[k].y, l);
      o.x = fmaf(wk, x[k].x, o.x);
      o.y = fmaf(wk, x[k].y, o.y);
      o.z = fmaf(wk, x[k].z, o.z);
      o.w = fmaf(wk, x[k].w, o.w);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint2 r;
  r.x = pack_bf16x2(o.x * inv, o.y * inv);
  r.y = pack_bf16x2(o.z * inv, o.w * inv);
  reinterpret_cast<uint2*>(a.o + ((long long)b * a.T + t) * a.o_row + (grp * kGroup + hh) * 128)[lane] = r;
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnArgs& a, const DevStatusHost& st, int num_sms, cudaStream_t stream,
                                   int* launches) {
  const int tp = std::min(a.c.page, kTile);
  CUtensorMap tk, tv, tpe;
  const uint64_t planes = (uint64_t)a.c.n_pages * a.c.heads;
  if (!make_tmap_rows128_3d(&tk, a.c.k_codes, a.c.page, planes, tp, kGroup) ||
      !make_tmap_rows128_3d(&tv, a.c.v_codes, a.c.page, planes, tp, kGroup) ||
      !make_tmap_rows128_3d(&tpe, a.c.k_pe, a.c.page, a.c.n_pages, tp, 1))
    return cudaErrorInvalidValue;
  const bool one = a.T == 1, two_pages = a.c.page < kTile / 2;
  auto kern = one ? (two_pages ? paged_attn_kernel<true, true> : paged_attn_kernel<true, false>)
                  : (two_pages ? paged_attn_kernel<false, true> : paged_attn_kernel<false, false>);
  static PerDevice<bool> allowed[2][2];
  cudaError_t e = allow_smem(allowed[one][two_pages], kern, kSmemBytes);
  if (e != cudaSuccess) return e;
  const long long nt = paged_attention_tiles(a.P_max, a.T, a.window, a.sinks);
  const long long most = nt * a.B * (a.c.heads / kGroup);
  static_assert(kTile == 64 && kPieceCost == 1, "the host's count of tiles");
  if ((nt + kPieceCost) * a.B > INT32_MAX || (long long)a.B * (a.c.heads / kGroup) > INT32_MAX) return cudaErrorInvalidValue;
  const int C = (int)std::min<long long>(most, std::min(num_sms, kPagedMaxCtas));
  e = launch_pdl(kern, dim3(C), dim3(kThreads), kSmemBytes, stream, tk, tv, tpe, a, st.wait_limit_ns);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (nt > 1) {  // with one tile per sequence nothing is cut
    e = launch_pdl(paged_combine_kernel, dim3((unsigned)(a.B * (a.c.heads / kGroup)), a.T), dim3(32 * kGroup), 0, stream, a,
                   C);
    ++*launches;
  }
  return e;
}

}  // namespace mla
