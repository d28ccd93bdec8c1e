// The pages of the paged cache: who holds them, and their copies.
//
// A pool is a table [rows, max_pages] of page numbers (below 0: none) and
// refs [n_pages], the number of table entries (and of a user's own holds) on
// each page; a page without any is free.  New pages are the lowest-numbered
// free ones, in the order of the call's list and of the positions, so that a
// call has one answer however its thread blocks run.
//
// mla_pages_free is one launch: an entry is exchanged for -1 and the page that
// came out of it loses one hold (a row that is listed twice loses each page
// once).  The others are two launches:
//   1. a plan by one cluster of 8 CTAs, which meet at the cluster's barrier
//      between its steps: the free pages as a bitmap with their number before
//      each 1,024 pages, what every list entry needs and whether it can be
//      carried out; then sums over both, by one CTA; then the list of the
//      pages that the call takes.  (One cluster, because its steps depend on
//      each other: its barrier takes a fraction of a microsecond, a launch two
//      to three.)
//   2. the changes themselves, over the whole GPU.  Nothing is changed before
//      the plan has found enough free pages, so a call without them changes
//      nothing.
// Bounds: free and reserve move a few bytes and take the launches' time; fork,
// compact and copy move pages, and HBM bounds them from a few hundred pages on.
#include "common.cuh"
#include "internal.h"

namespace mla {

namespace {

constexpr int kPlanCtas = 8;         // (the largest cluster that every GPU of the kind takes)
constexpr int kPlanThreads = 1024;
constexpr int kSeg = 1024;           // pages whose bitmap a warp reads at once, 32 bits a lane
constexpr int kClaimsInSmem = 8192;  // rows

__device__ __forceinline__ int pages_of(int P, int page) { return (P + page - 1) / page; }

// Status of a call: word 0 is zero, each CTA stores its own further word.
__device__ __forceinline__ void store_status(uint32_t* status, int cta, int ctas, uint32_t word) {
  if (cta == 0) {
    status[0] = 0u;
    status[kStatusExtraWord] = (uint32_t)ctas;
  }
  status[kStatusExtraFirst + cta] = word;
}

// Exclusive sum over the block's threads (all of kPlanThreads), and the total.
__device__ __forceinline__ long long block_sum(long long v, long long& total, long long* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long w = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    sh[lane] = w;
  }
  __syncthreads();
  total = sh[kPlanThreads / 32 - 1];
  const long long before = x - v + (warp > 0 ? sh[warp - 1] : 0);
  __syncthreads();
  return before;
}

// ---- giving pages back --------------------------------------------------------
// Grid: items (list entry, 1,024 entries of its row) in turn.
__global__ void __launch_bounds__(256) pages_free_kernel(const PagePool p, const int* __restrict__ rows,
                                                         const int* __restrict__ P, int n, int per_row,
                                                         uint32_t* status) {
  pdl_launch_dependents();
  pdl_wait();
  bool bad = false;
  for (long long item = blockIdx.x; item < (long long)n * per_row; item += gridDim.x) {
    const int i = (int)(item / per_row), part = (int)(item - (long long)i * per_row);
    const int r = rows[i], pos = P[i];
    if (r < 0 || r >= p.rows || pos < 0) {
      bad = true;
      continue;
    }
    const int keep = (int)min((long long)p.max_pages, ((long long)pos + p.page - 1) / p.page);
    int* row = p.table + (size_t)r * p.max_pages;
    const int end = min(p.max_pages, (part + 1) * 1024);
    int held[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int e = part * 1024 + c * 256 + (int)threadIdx.x;
      held[c] = e >= keep && e < end ? row[e] : -1;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (held[c] == -1) continue;
      const int was = atomicExch(row + part * 1024 + c * 256 + threadIdx.x, -1);
      if (was == -1) continue;  // (another list entry of this row has taken it)
      if (was < 0 || was >= p.n_pages) {
        bad = true;
        continue;
      }
      if (atomicSub(p.refs + was, 1) <= 0) {  // held by nobody: stays free
        atomicAdd(p.refs + was, 1);
        bad = true;
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) store_status(status, blockIdx.x, gridDim.x, bad ? kStatusBadLength : 0u);
}

// ---- the plan -------------------------------------------------------------------
enum class PageOp { kReserve, kFork, kCompact };

// What list entry i of a reservation or fork needs: pages, or -1 if it cannot
// be carried out.  One warp.
template <PageOp OP>
__device__ __forceinline__ int pages_needed(const PagePlanArgs& a, int i, bool& bad) {
  const PagePool& p = a.pool;
  const int lane = threadIdx.x & 31;
  const int r = a.rows[i], pos = a.P[i];
  int parent = 0;
  bool ok = r >= 0 && r < p.rows && pos >= 0 && pos <= p.max_pages * p.page;
  if (OP == PageOp::kFork) {
    parent = a.parents[i];
    ok = ok && parent >= 0 && parent < p.rows;
  }
  if (!ok) {
    bad = true;
    return -1;
  }
  const int want = pages_of(pos, p.page);
  const int* row = p.table + (size_t)r * p.max_pages;
  int missing = 0;
  if (OP == PageOp::kReserve) {
#pragma unroll 4
    for (int e0 = 0; e0 < want; e0 += 32) {
      const int x = e0 + lane < want ? row[e0 + lane] : 0;
      missing += __popc(__ballot_sync(0xffffffffu, x < 0));
      bad |= x >= p.n_pages;
    }
    return missing;
  }
  // fork: the child's entries are empty, the parent's pages are held
  const int* from = p.table + (size_t)parent * p.max_pages;
#pragma unroll 4
  for (int e0 = 0; e0 < want; e0 += 32) {
    if (e0 + lane < want) {
      const int x = from[e0 + lane];
      ok = ok && row[e0 + lane] < 0 && x >= 0 && x < p.n_pages && p.refs[x] > 0;
    }
  }
  if (!__all_sync(0xffffffffu, ok)) {
    bad = true;
    return -1;
  }
  return pos % p.page ? 1 : 0;
}

template <PageOp OP>
__global__ void __launch_bounds__(kPlanThreads, 1) pages_plan_kernel(const PagePlanArgs a) {
  __shared__ long long sums[32];
  __shared__ int claims_smem[OP == PageOp::kCompact ? 1 : kClaimsInSmem];
  pdl_launch_dependents();
  pdl_wait();
  const PagePool& p = a.pool;
  const int rank = (int)cluster_ctarank(), tid = threadIdx.x, lane = tid & 31;
  const int warp = rank * (kPlanThreads / 32) + (tid >> 5), warps = kPlanCtas * (kPlanThreads / 32);
  const int n_seg = (p.n_pages + kSeg - 1) / kSeg;
  bool bad = false;

  // 1. free pages as bits, their number in each segment; what the list needs
  for (int s = warp; s < n_seg; s += warps) {
    uint32_t mine = 0;
    int count = 0;
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
      const int at = s * kSeg + j * 32 + lane;
      const uint32_t b = __ballot_sync(0xffffffffu, at < p.n_pages && p.refs[at] <= 0);
      count += __popc(b);
      if (lane == j) mine = b;
    }
    a.bits[(size_t)s * 32 + lane] = mine;
    if (lane == 0) a.seg[s] = count;
  }
  if (OP != PageOp::kCompact) {
    for (int i = warp; i < a.n; i += warps) {
      const int need = pages_needed<OP>(a, i, bad);
      if (lane == 0) a.need[i] = need;
    }
  }
  cluster_sync();

  // 2. one CTA: list entries whose row an earlier one has taken; sums
  if (rank == 0) {
    if (OP != PageOp::kCompact && a.n > 1) {
      int* claim = p.rows <= kClaimsInSmem ? claims_smem : a.claims;
      for (int i = tid; i < a.n; i += kPlanThreads)
        if (__ldcg(a.need + i) >= 0) claim[a.rows[i]] = INT32_MAX;
      __syncthreads();
      for (int i = tid; i < a.n; i += kPlanThreads)
        if (__ldcg(a.need + i) >= 0) atomicMin(claim + a.rows[i], i);
      __syncthreads();
      for (int i = tid; i < a.n; i += kPlanThreads)
        if (__ldcg(a.need + i) >= 0 && *(volatile int*)(claim + a.rows[i]) != i) {
          a.need[i] = -1;
          bad = true;
        }
      __syncthreads();
    }
    long long free_pages = 0, taken = 0, total = 0;
    for (int s0 = 0; s0 < n_seg; s0 += kPlanThreads) {
      const int s = s0 + tid;
      const long long before = block_sum(s < n_seg ? __ldcg(a.seg + s) : 0, total, sums);
      if (s < n_seg) a.seg[s] = (int)(free_pages + before);
      free_pages += total;
    }
    if (OP != PageOp::kCompact) {
      for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
        const int i = i0 + tid, need = i < a.n ? __ldcg(a.need + i) : 0;
        const long long before = block_sum(need > 0 ? need : 0, total, sums);
        if (i < a.n) a.first[i] = need < 0 ? -1 : (int)min((long long)INT32_MAX, taken + before);
        taken += total;
      }
      if (tid == 0) {
        a.head[0] = taken <= free_pages;
        a.head[1] = taken <= free_pages ? (int)taken : 0;
      }
      if (taken > free_pages) {
        if (tid == 0) store_status(a.status, 0, kPlanCtas, kStatusNoPages);
        bad = false;
      }
    } else {
      const int n_live = p.n_pages - (int)free_pages;
      __syncthreads();
      if (tid < 32) {  // free pages below n_live: as many as there are live ones from it on
        const int s = n_live / kSeg, in_seg = n_live - s * kSeg;
        int below = 0;
        if (s < n_seg) {
          const uint32_t b = __ldcg(a.bits + (size_t)s * 32 + lane);
          const int k = in_seg - lane * 32;  // bits of this word that lie below
          below = __popc(k >= 32 ? b : k <= 0 ? 0u : b & ((1u << k) - 1u));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
        }
        if (lane == 0) {
          const int moves = s < n_seg ? *(volatile int*)(a.seg + s) + below : (int)free_pages;
          a.head[0] = n_live;
          a.head[1] = moves;
          *a.n_live = n_live;
        }
      }
    }
  }
  cluster_sync();

  // 3. the pages in question, by rank
  const int h0 = __ldcg(a.head), h1 = __ldcg(a.head + 1);
  for (int s = warp; s < n_seg; s += warps) {
    const int before = __ldcg(a.seg + s);
    if (OP != PageOp::kCompact && before >= h1) break;  // (the sums grow)
    const uint32_t mine = __ldcg(a.bits + (size_t)s * 32 + lane);
    int at = __popc(mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    at += before - __popc(mine);  // free pages before this lane's word
    for (int j = 0; j < 32; ++j) {
      const uint32_t b = __shfl_sync(0xffffffffu, mine, j);
      const int k = __shfl_sync(0xffffffffu, at, j) + __popc(b & ((1u << lane) - 1u));  // free pages before page q
      const int q = s * kSeg + j * 32 + lane;
      const bool is_free = (b >> lane) & 1u;
      if (OP != PageOp::kCompact) {
        if (is_free && k < h1) a.fresh[k] = q;
      } else if (q < p.n_pages) {
        if (is_free && q < h0) a.fresh[k] = q;
        if (!is_free && q >= h0) a.from[q - k - (h0 - h1)] = q;
        a.moved[q] = is_free ? -1 : q;
      }
    }
  }
  if (OP == PageOp::kCompact) {
    // 4. the moved pages' holds and new numbers
    cluster_sync();
    for (int i = rank * kPlanThreads + tid; i < h1; i += kPlanCtas * kPlanThreads) {
      const int src = __ldcg(a.from + i), dst = __ldcg(a.fresh + i);
      a.moved[src] = dst;
      p.refs[dst] = p.refs[src];
      p.refs[src] = 0;
    }
    // (the launch that follows reports on the table)
  } else {
    bad = __syncthreads_or(bad);
    if (tid == 0 && (rank != 0 || h0)) store_status(a.status, rank, kPlanCtas, bad ? kStatusBadLength : 0u);
  }
}

// ---- the changes ----------------------------------------------------------------
// A CTA a list entry in turn: 1,024 entries of the row at a time.
__global__ void __launch_bounds__(256) pages_reserve_kernel(const PagePlanArgs a) {
  __shared__ int counts[2][8];
  pdl_launch_dependents();
  pdl_wait();
  if (!a.head[0]) return;
  const PagePool& p = a.pool;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int turn = 0;
  for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
    int at = a.first[i];
    if (at < 0) continue;
    const int want = pages_of(a.P[i], p.page);
    int* row = p.table + (size_t)a.rows[i] * p.max_pages;
    for (int e0 = 0; e0 < want; e0 += 1024, turn ^= 1) {
      // thread t: entries e0 + 4 t .. + 3
      bool none[4];
      int mine = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int e = e0 + tid * 4 + c;
        none[c] = e < want && row[e] < 0;
        mine += none[c];
      }
      int before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      if (lane == 31) counts[turn][warp] = before;
      __syncthreads();
      before -= mine;
      int all = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const int c = counts[turn][w];
        if (w < warp) before += c;
        all += c;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (none[c]) {
          const int page = a.fresh[at + before++];
          row[e0 + tid * 4 + c] = page;
          p.refs[page] = 1;
        }
      at += all;
    }
  }
}

// Grid: x = list entries in turn, y = part of the row's entries and of the tail's heads.
__global__ void __launch_bounds__(256) pages_fork_kernel(const PagedCache c, const PagePlanArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  if (!a.head[0]) return;
  const PagePool& p = a.pool;
  const int tid = threadIdx.x, part = blockIdx.y, parts = gridDim.y;
  for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
    const int at = a.first[i];
    if (at < 0) continue;
    const int pos = a.P[i], full = pos / p.page, rest = pos - full * p.page;
    const int* from = p.table + (size_t)a.parents[i] * p.max_pages;
    int* row = p.table + (size_t)a.rows[i] * p.max_pages;
    for (int e = part * 256 + tid; e < full; e += parts * 256) {
      const int page = from[e];
      row[e] = page;
      atomicAdd(p.refs + page, 1);
    }
    if (rest == 0) continue;
    const int src = from[full], dst = a.fresh[at];
    if (part == 0) {
      if (tid == 0) {
        row[full] = dst;
        p.refs[dst] = 1;
      }
      for (int h = tid; h < c.heads; h += 256) {
        c.k_scales[(size_t)dst * c.heads + h] = c.k_scales[(size_t)src * c.heads + h];
        c.v_scales[(size_t)dst * c.heads + h] = c.v_scales[(size_t)src * c.heads + h];
      }
      const uint4* ps = reinterpret_cast<const uint4*>(c.k_pe + (size_t)src * c.page * 64);
      uint4* pd = reinterpret_cast<uint4*>(c.k_pe + (size_t)dst * c.page * 64);
      for (int u = tid; u < rest * 8; u += 256) pd[u] = ps[u];
    }
    // the first `rest` slots of this part's heads, keys then values
    const int h0 = (int)((long long)c.heads * part / parts), nh = (int)((long long)c.heads * (part + 1) / parts) - h0;
    const int per = rest * 8, step = c.page * 8;  // units of 16 bytes
    const size_t so = ((size_t)src * c.heads + h0) * step, to = ((size_t)dst * c.heads + h0) * step;
    const uint4 *ks = reinterpret_cast<const uint4*>(c.k_codes) + so, *vs = reinterpret_cast<const uint4*>(c.v_codes) + so;
    uint4 *kd = reinterpret_cast<uint4*>(c.k_codes) + to, *vd = reinterpret_cast<uint4*>(c.v_codes) + to;
    for (int u0 = tid; u0 < nh * per; u0 += 1024) {
      uint4 x[4], y[4];
      int where[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int u = u0 + k * 256, h = u / per;
        where[k] = u < nh * per ? h * step + (u - h * per) : -1;
        if (where[k] >= 0) {
          x[k] = ks[where[k]];
          y[k] = vs[where[k]];
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (where[k] >= 0) {
          kd[where[k]] = x[k];
          vd[where[k]] = y[k];
        }
    }
  }
}

// Whole pages, in pieces of 2,048 units of 16 bytes (32 KB, all of whose loads
// are in flight at once): the pieces of a page's keys, those of its values, and
// one more with its rotary keys and scales.
constexpr int kPiece = 2048;
constexpr int kCopyCtas = 4;  // an SM

struct PagePieces {
  int page_units, per, total;  // units of a page's keys, pieces of them, pieces of a page
  __host__ __device__ explicit PagePieces(const PagedCache& c)
      : page_units(c.heads * c.page * 8), per((page_units + kPiece - 1) / kPiece), total(2 * per + 1) {}
  // piece k of page `src` of s into page `dst` of d
  __device__ __forceinline__ void copy(const PagedCache& s, int src, const PagedCache& d, int dst, int k) const {
    const int tid = threadIdx.x;
    const uint4* from;
    uint4* to;
    int units;
    if (k == 2 * per) {
      units = s.page * 8;
      from = reinterpret_cast<const uint4*>(s.k_pe) + (size_t)src * units;
      to = reinterpret_cast<uint4*>(d.k_pe) + (size_t)dst * units;
      if (tid < s.heads) {
        d.k_scales[(size_t)dst * s.heads + tid] = s.k_scales[(size_t)src * s.heads + tid];
        d.v_scales[(size_t)dst * s.heads + tid] = s.v_scales[(size_t)src * s.heads + tid];
      }
    } else {
      const bool v = k >= per;
      const int u = (v ? k - per : k) * kPiece;
      units = min(kPiece, page_units - u);
      from = reinterpret_cast<const uint4*>(v ? s.v_codes : s.k_codes) + (size_t)src * page_units + u;
      to = reinterpret_cast<uint4*>(v ? d.v_codes : d.k_codes) + (size_t)dst * page_units + u;
    }
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * 256 + tid < units) x[i] = __ldcs(from + i * 256 + tid);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * 256 + tid < units) __stcs(to + i * 256 + tid, x[i]);
  }
};

__global__ void __launch_bounds__(256, 4) pages_compact_kernel(const PagedCache c, const PagePlanArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const PagePool& p = a.pool;
  const PagePieces pieces(c);
  const int moves = a.head[1];
  bool bad = false;
  // the table, by the CTAs that have a status word
  const int tables = min((int)gridDim.x, kMaxStatusExtra);
  const long long entries = (long long)blockIdx.x < tables ? (long long)p.rows * p.max_pages : 0;
  for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < entries; e += (long long)tables * 256) {
    const int page = p.table[e];
    if (page == -1) continue;
    const int to = page >= 0 && page < p.n_pages ? a.moved[page] : -1;
    bad |= to < 0;  // no page, or one that is held by nobody
    if (to != page) p.table[e] = to;
  }
  for (long long item = blockIdx.x; item < (long long)moves * pieces.total; item += gridDim.x) {
    const int i = (int)(item / pieces.total), k = (int)(item - (long long)i * pieces.total);
    pieces.copy(c, a.from[i], c, a.fresh[i], k);
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0 && (int)blockIdx.x < tables)
    store_status(a.status, blockIdx.x, tables, bad ? kStatusBadLength : 0u);
}

// Whether pair i of a copy is carried out: its pages exist, it is the last pair
// that writes its destination, and none writes its source (but itself, when a
// page is copied onto itself).
__device__ __forceinline__ bool carried_out(const PageCopyArgs& a, int i, int s, int d) {
  if (s < 0 || s >= a.from.n_pages || d < 0 || d >= a.to.n_pages) return false;
  return __ldcg(a.claims + d) == i && (!a.same || s == d || __ldcg(a.claims + s) < 0);
}

// claim[page] = the last pair that
// writes the page, -1 for a source that none writes.
__global__ void __launch_bounds__(kPlanThreads, 1) pages_claim_kernel(const PageCopyArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int step = kPlanCtas * kPlanThreads, first = (int)cluster_ctarank() * kPlanThreads + threadIdx.x;
  for (int i = first; i < a.n; i += step) {
    const int s = a.src[i], d = a.dst[i];
    if (d >= 0 && d < a.to.n_pages) a.claims[d] = -1;
    if (a.same && s >= 0 && s < a.to.n_pages) a.claims[s] = -1;
  }
  cluster_sync();
  for (int i = first; i < a.n; i += step) {
    const int d = a.dst[i];
    if (d >= 0 && d < a.to.n_pages) atomicMax(a.claims + d, i);
  }
  cluster_sync();
  bool bad = false;
  for (int i = first; i < a.n; i += step) bad |= !carried_out(a, i, a.src[i], a.dst[i]);
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0)
    store_status(a.status, (int)cluster_ctarank(), kPlanCtas, bad ? kStatusBadLength : 0u);
}

__global__ void __launch_bounds__(256, 4) pages_copy_kernel(const PageCopyArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const PagePieces pieces(a.from);
  for (long long item = blockIdx.x; item < (long long)a.n * pieces.total; item += gridDim.x) {
    const int i = (int)(item / pieces.total), k = (int)(item - (long long)i * pieces.total);
    const int s = a.src[i], d = a.dst[i];
    if (carried_out(a, i, s, d) && !(a.same && s == d)) pieces.copy(a.from, s, a.to, d, k);
  }
}

template <PageOp OP>
cudaError_t launch_plan(const PagePlanArgs& a, cudaStream_t stream) {
  return launch_pdl_cluster(pages_plan_kernel<OP>, kPlanCtas, dim3(kPlanCtas), dim3(kPlanThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_pages_free(const PagePool& p, const int* rows, const int* P, int n, uint32_t* status,
                              cudaStream_t stream) {
  const int per_row = (p.max_pages + 1023) / 1024;
  const long long items = (long long)n * per_row;
  const int grid = items < kMaxStatusExtra ? (int)items : kMaxStatusExtra;
  return launch_pdl(pages_free_kernel, dim3(grid), dim3(256), 0, stream, p, rows, P, n, per_row, status);
}

cudaError_t launch_pages_reserve(const PagePlanArgs& a, int num_sms, cudaStream_t stream) {
  const cudaError_t e = launch_plan<PageOp::kReserve>(a, stream);
  if (e != cudaSuccess) return e;
  const int grid = a.n < 4 * num_sms ? a.n : 4 * num_sms;
  return launch_pdl(pages_reserve_kernel, dim3(grid), dim3(256), 0, stream, a);
}

cudaError_t launch_pages_fork(const PagedCache& c, const PagePlanArgs& a, int num_sms, cudaStream_t stream) {
  const cudaError_t e = launch_plan<PageOp::kFork>(a, stream);
  if (e != cudaSuccess) return e;
  // two CTAs an SM where the pairs are few: a part is at least one head
  const int grid = a.n < 4 * num_sms ? a.n : 4 * num_sms;
  int parts = (2 * num_sms + grid - 1) / grid;
  if (parts > c.heads) parts = c.heads;
  return launch_pdl(pages_fork_kernel, dim3(grid, parts), dim3(256), 0, stream, c, a);
}

cudaError_t launch_pages_compact(const PagedCache& c, const PagePlanArgs& a, int num_sms, cudaStream_t stream) {
  const cudaError_t e = launch_plan<PageOp::kCompact>(a, stream);
  if (e != cudaSuccess) return e;
  return launch_pdl(pages_compact_kernel, dim3(kCopyCtas * num_sms), dim3(256), 0, stream, c, a);
}

cudaError_t launch_pages_copy(const PageCopyArgs& a, int num_sms, cudaStream_t stream) {
  const cudaError_t e =
      launch_pdl_cluster(pages_claim_kernel, kPlanCtas, dim3(kPlanCtas), dim3(kPlanThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  const long long items = (long long)a.n * PagePieces(a.from).total;
  const int grid = items < kCopyCtas * num_sms ? (int)items : kCopyCtas * num_sms;
  return launch_pdl(pages_copy_kernel, dim3(grid), dim3(256), 0, stream, a);
}

}  // namespace mla
