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
// once).  The others begin with a plan by one cluster of 8 CTAs, which meet at the
// cluster's barrier between its steps: the free pages as a bitmap with their
// number before each 1,024 pages, what every list entry needs and whether it can
// be carried out; then sums over both, by one CTA, in its shared memory; then the
// list of the pages that the call takes.  (One cluster, because its steps depend
// on each other: its barrier takes a fraction of a microsecond, a launch two to
// three.  Handing the numbers over through global memory took 1 to 2 us more.)
// Nothing is changed before the plan has found enough free pages, so a call
// without them changes nothing.  The changes follow in a second launch over the
// whole GPU; those of a short reservation end in the plan's own.
// A copy has no plan but its pairs' claims on their destinations, for up to 32 pairs none.
//
// Bounds and figures: free, reserve and fork move little and take their launches,
// each 2 to 3 us, and the plan's chain of dependent reads: 64 rows given back and
// taken again 9.8 us on the GPU, 600 rows of up to 2,048 more tokens 21.9, 1 row
// forked into 4 and given back 12.2.  compact and copy move pages, and HBM bounds
// them from a few hundred pages on: 1,531 pages of 32 tokens of 64 heads copied in
// 258 us (6.28 TB/s, 0.93 of the measured copy rate), the 2,048 of 8,192 pages of
// 16 tokens that a half-full pool has to move in 186 us (5.8 TB/s).
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

// Exclusive sums over the block's threads (all of kPlanThreads) of two numbers,
// and the totals.
__device__ __forceinline__ void block_sums(int& u, int& u_total, long long& v, long long& v_total, int* shu, long long* shv) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = u;
  long long y = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int p = __shfl_up_sync(0xffffffffu, x, o);
    const long long q = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += p;
      y += q;
    }
  }
  if (lane == 31) {
    shu[warp] = x;
    shv[warp] = y;
  }
  __syncthreads();
  int wx = shu[lane];  // (as many warps as lanes)
  long long wy = shv[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int p = __shfl_up_sync(0xffffffffu, wx, o);
    const long long q = __shfl_up_sync(0xffffffffu, wy, o);
    if (lane >= o) {
      wx += p;
      wy += q;
    }
  }
  u_total = __shfl_sync(0xffffffffu, wx, 31);
  v_total = __shfl_sync(0xffffffffu, wy, 31);
  const int bx = __shfl_sync(0xffffffffu, wx, max(warp - 1, 0));
  const long long by = __shfl_sync(0xffffffffu, wy, max(warp - 1, 0));
  u = x - u + (warp > 0 ? bx : 0);
  v = y - v + (warp > 0 ? by : 0);
  __syncthreads();
}
static_assert(kPlanThreads == 32 * 32, "a lane for each warp");

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
// A variable of the cluster's first CTA, this CTA's of which is at `local`.
__device__ __forceinline__ void put_first(int* local, int x) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(mapa_rank(smem_u32(local), 0)), "r"(x) : "memory");
}
__device__ __forceinline__ int get_first(const int* local) {
  int x;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(mapa_rank(smem_u32(local), 0)) : "memory");
  return x;
}

enum class PageOp { kReserve, kFork, kCompact };

// What a list entry of a reservation or fork needs: pages, or -1 if it cannot be
// carried out.  One warp.
template <PageOp OP>
__device__ __forceinline__ int pages_needed(const PagePool& p, int r, int parent, int pos, bool& bad) {
  const int lane = threadIdx.x & 31;
  bool ok = r >= 0 && r < p.rows && pos >= 0 && pos <= p.max_pages * p.page;
  if (OP == PageOp::kFork) ok = ok && parent >= 0 && parent < p.rows;
  if (!ok) {
    bad = true;
    return -1;
  }
  const int want = pages_of(pos, p.page);
  const int* row = p.table + (size_t)r * p.max_pages;
  int missing = 0;
  if (OP == PageOp::kReserve) {
#pragma unroll 8
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
  constexpr bool kList = OP != PageOp::kCompact;
  __shared__ int sums_seg[32];
  __shared__ long long sums_need[32];
  __shared__ int claims_smem[kList ? kClaimsInSmem : 1];
  // the first CTA's: what the others tell it and what it tells them, of lists and pools that
  // are not larger (else in the workspace)
  __shared__ int need_smem[kList ? kPlanThreads : 1];
  __shared__ int seg_smem[kPlanThreads];
  __shared__ int head[2];
  pdl_launch_dependents();
  cluster_sync();  // (the first CTA's shared memory may be written from here on; ahead of the
                   // wait for the launch before: 64 rows 9.8 us on the GPU, behind it 10.1)
  pdl_wait();
  const PagePool& p = a.pool;
  const int rank = (int)cluster_ctarank(), tid = threadIdx.x, lane = tid & 31;
  const int warp = (tid >> 5) * kPlanCtas + rank, warps = kPlanCtas * (kPlanThreads / 32);  // (the first few: one a CTA)
  const int n_seg = (p.n_pages + kSeg - 1) / kSeg;
  const bool list_near = a.n <= kPlanThreads, seg_near = n_seg <= kPlanThreads;
  bool bad = false;

  // 1. free pages as bits, their number in each segment; what the list needs (by the last
  // warps first: the segments are the first ones')
  uint32_t bits0 = 0;  // this warp's first segment
  for (int s = warp; s < n_seg; s += warps) {
    uint32_t mine = 0;
    int count = 0;
    bool free_at[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int at = s * kSeg + j * 32 + lane;
      free_at[j] = at < p.n_pages && p.refs[at] <= 0;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const uint32_t b = __ballot_sync(0xffffffffu, free_at[j]);
      count += __popc(b);
      if (lane == j) mine = b;
    }
    a.bits[(size_t)s * 32 + lane] = mine;
    if (s == warp) bits0 = mine;
    if (lane == 0) {
      if (seg_near)
        put_first(&seg_smem[s], count);
      else
        a.seg[s] = count;
    }
  }
  if (kList) {
    // (a warp's next 32 entries at once, one a lane)
    for (int i0 = warps - 1 - warp; i0 < a.n; i0 += 32 * warps) {
      const int mine = i0 + lane * warps;
      const bool in = mine < a.n;
      const int row = in ? a.rows[mine] : 0, pos = in ? a.P[mine] : 0;
      const int parent = OP == PageOp::kFork && in ? a.parents[mine] : 0;
      int need = 0;
      for (int k = 0; k < 32 && i0 + k * warps < a.n; ++k) {
        const int x = pages_needed<OP>(p, __shfl_sync(0xffffffffu, row, k), __shfl_sync(0xffffffffu, parent, k),
                                       __shfl_sync(0xffffffffu, pos, k), bad);
        if (lane == k) need = x;
      }
      if (in) {
        if (list_near)
          put_first(&need_smem[mine], need);
        else
          a.need[mine] = need;
      }
    }
  }
  cluster_sync();

  // 2. one CTA: list entries whose row an earlier one has taken; sums
  if (rank == 0) {
    if (kList && a.n > 1) {
      int* claim = p.rows <= kClaimsInSmem ? claims_smem : a.claims;
      for (int i = tid; i < a.n; i += kPlanThreads)
        if ((list_near ? need_smem[i] : __ldcg(a.need + i)) >= 0) claim[a.rows[i]] = INT32_MAX;
      __syncthreads();
      for (int i = tid; i < a.n; i += kPlanThreads)
        if ((list_near ? need_smem[i] : __ldcg(a.need + i)) >= 0) atomicMin(claim + a.rows[i], i);
      __syncthreads();
      for (int i = tid; i < a.n; i += kPlanThreads)
        if ((list_near ? need_smem[i] : __ldcg(a.need + i)) >= 0 && *(volatile int*)(claim + a.rows[i]) != i) {
          if (list_near)
            need_smem[i] = -1;
          else
            a.need[i] = -1;
          bad = true;
        }
    }
    int free_pages = 0, seg_total;
    long long taken = 0, need_total;
    for (int i0 = 0; i0 < max(n_seg, kList ? a.n : 0); i0 += kPlanThreads) {
      const int i = i0 + tid;
      int seg = i < n_seg ? (seg_near ? seg_smem[i] : __ldcg(a.seg + i)) : 0;
      const int need = kList && i < a.n ? (list_near ? need_smem[i] : __ldcg(a.need + i)) : 0;
      long long before = max(need, 0);
      block_sums(seg, seg_total, before, need_total, sums_seg, sums_need);
      if (i < n_seg) {
        if (seg_near)
          seg_smem[i] = free_pages + seg;
        else
          a.seg[i] = free_pages + seg;
      }
      if (kList && i < a.n) a.first[i] = need < 0 ? -1 : (int)min((long long)INT32_MAX, taken + before);
      free_pages += seg_total;
      taken += need_total;
    }
    __syncthreads();
    if (kList) {
      if (tid == 0) {
        head[0] = taken <= free_pages;
        head[1] = taken <= free_pages ? (int)taken : 0;
      }
      if (taken > free_pages) {
        if (tid == 0) store_status(a.status, 0, kPlanCtas, kStatusNoPages);
        bad = false;
      }
    } else if (tid < 32) {  // free pages below n_live: as many as there are live ones from it on
      const int n_live = p.n_pages - free_pages;
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
        head[0] = n_live;
        head[1] = s < n_seg ? (seg_near ? seg_smem[s] : *(volatile int*)(a.seg + s)) + below : free_pages;
        *a.n_live = n_live;
      }
    }
    if (tid == 0) {
      a.head[0] = head[0];
      a.head[1] = head[1];
    }
  }
  cluster_sync();

  // 3. the pages in question, by rank
  const int h0 = get_first(&head[0]), h1 = get_first(&head[1]);
  for (int s = warp; s < n_seg; s += warps) {
    const int before = seg_near ? get_first(&seg_smem[s]) : __ldcg(a.seg + s);
    const uint32_t mine = s == warp ? bits0 : __ldcg(a.bits + (size_t)s * 32 + lane);
    if (kList && before >= h1) break;  // (the sums grow)
    int at = __popc(mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    at += before - __popc(mine);  // free pages before this lane's word
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
      const uint32_t b = __shfl_sync(0xffffffffu, mine, j);
      const int k = __shfl_sync(0xffffffffu, at, j) + __popc(b & ((1u << lane) - 1u));  // free pages before page q
      const int q = s * kSeg + j * 32 + lane;
      const bool is_free = (b >> lane) & 1u;
      if (kList) {
        if (is_free && k < h1) a.fresh[k] = q;
      } else if (q < p.n_pages) {
        if (is_free && q < h0) a.fresh[k] = q;
        if (!is_free && q >= h0) a.from[q - k - (h0 - h1)] = q;
        a.moved[q] = is_free ? -1 : q;
      }
    }
  }
  cluster_sync();  // (the first CTA's shared memory is read no more)
  if (OP == PageOp::kCompact) {
    // 4. the moved pages' holds and new numbers
    for (int i = rank * kPlanThreads + tid; i < h1; i += kPlanCtas * kPlanThreads) {
      const int src = __ldcg(a.from + i), dst = __ldcg(a.fresh + i);
      a.moved[src] = dst;
      p.refs[dst] = p.refs[src];
      p.refs[src] = 0;
    }
    // (the launch that follows reports on the table)
  } else {
    if (OP == PageOp::kReserve && h0 && a.n <= kPlanCtas * (kPlanThreads / 32)) {
      // 4. the rows of a short list, a warp each
      const int i = warps - 1 - warp;
      int at = i < a.n ? __ldcg(a.first + i) : -1;
      if (at >= 0) {
        const int want = pages_of(a.P[i], p.page);
        int* row = p.table + (size_t)a.rows[i] * p.max_pages;
        for (int e0 = 0; e0 < want; e0 += 256) {
          bool none[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int e = e0 + c * 32 + lane;
            none[c] = e < want && row[e] < 0;
          }
          int page[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint32_t b = __ballot_sync(0xffffffffu, none[c]);
            page[c] = none[c] ? __ldcg(a.fresh + at + __popc(b & ((1u << lane) - 1u))) : 0;
            at += __popc(b);
          }
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (none[c]) {
              row[e0 + c * 32 + lane] = page[c];
              p.refs[page[c]] = 1;
            }
        }
      }
    }
    bad = __syncthreads_or(bad);
    if (tid == 0 && (rank != 0 || h0)) store_status(a.status, rank, kPlanCtas, bad ? kStatusBadLength : 0u);
  }
}

// ---- the changes ----------------------------------------------------------------
// The rows of a long list: a CTA each in turn, 1,024 entries at a time.
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

// claim[page] = the last pair that writes the page, -1 for a source that none writes.
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

// The same for at most as many pairs as a warp has lanes: each warp holds the list and
// finds out by itself which pairs are carried out.
__global__ void __launch_bounds__(256, 4) pages_copy_few_kernel(const PageCopyArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const PagePieces pieces(a.from);
  const int lane = threadIdx.x & 31;
  const int src = lane < a.n ? a.src[lane] : -1, dst = lane < a.n ? a.dst[lane] : -1;
  bool ok = src >= 0 && src < a.from.n_pages && dst >= 0 && dst < a.to.n_pages;
  for (int j = 0; j < a.n; ++j) {
    const int d = __shfl_sync(0xffffffffu, dst, j);
    if ((j > lane && d == dst) || (a.same && src != dst && d == src)) ok = false;
  }
  const uint32_t done = __ballot_sync(0xffffffffu, ok);
  if (blockIdx.x == 0 && threadIdx.x == 0) store_status(a.status, 0, 1, __popc(done) == a.n ? 0u : kStatusBadLength);
  for (int item = blockIdx.x; item < a.n * pieces.total; item += gridDim.x) {
    const int i = item / pieces.total, k = item - i * pieces.total;
    const int s = __shfl_sync(0xffffffffu, src, i), d = __shfl_sync(0xffffffffu, dst, i);
    if ((done >> i & 1u) && !(a.same && s == d)) pieces.copy(a.from, s, a.to, d, k);
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
  // (a list of at most one row for each of the plan's warps is done: 64 rows, given back and
  // taken again, 12.9 us with a second launch, 10.6 without; 600 rows 27.0 without, 22.0 with)
  if (e != cudaSuccess || a.n <= kPlanCtas * (kPlanThreads / 32)) return e;
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
  const long long items = (long long)a.n * PagePieces(a.from).total;
  const int grid = items < kCopyCtas * num_sms ? (int)items : kCopyCtas * num_sms;
  // (3 pages of 64 tokens of 64 heads: 5.7 us on the GPU with the claims' launch, 2.8 without)
  if (a.n <= 32) return launch_pdl(pages_copy_few_kernel, dim3(grid), dim3(256), 0, stream, a);
  const cudaError_t e =
      launch_pdl_cluster(pages_claim_kernel, kPlanCtas, dim3(kPlanCtas), dim3(kPlanThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(pages_copy_kernel, dim3(grid), dim3(256), 0, stream, a);
}

}  // namespace mla
