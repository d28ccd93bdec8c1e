// Attention over packed documents for MLA heads (qk = 192, v = 128) on tcgen05.
//
// "Mix and project" page, code excerpt: scores = Q K^T * softmax_scale plus
// the mask, softmax in float32, then P V; here for several sequences packed one
// after the other, each seeing its own keys only (mla_document_attention).
// Computed in the flash form: online softmax over tiles of 96 keys.
//
// A plan kernel (or, for a few tiles, one warp of each CTA) lists the documents'
// query tiles of up to 128 rows, a tile never holding rows of two documents,
// heaviest first.  Persistent: one CTA per SM takes items (tile, head) from an
// atomic counter, in groups of heads whose K/V stay in L2.  An item's key tiles begin at the document's (or the window's)
// first key.  V rows behind the last key that the tile's queries see would be
// another document's: the P.V product takes only the 16-key steps up to that
// key, and the V producer's warp clears the rows behind it in the last step, so
// that nothing of a neighbour (a NaN times zero among it) reaches the sum.  Rows
// of the next document in the Q tile are computed and not stored; a row that
// sees no key has the sum zero and is stored as zeros.
//
// Warp roles (512 threads):
//   warp 0   TMA: K tiles, 64 dimensions at a time, into a ring of 7 such thirds (TMA
//            takes 1,900 cycles under load: with a ring of two whole tiles, each
//            slot idle for that long, a tile took 160 cycles more)
//   warp 1   TMEM allocation; an item's Q into tensor memory (tcgen05.cp), then
//            S_x = Q K_x^T (M=128 N=96 K=192) into score buffer x & 1, x
//            counting this CTA's key tiles
//   warp 2   TMA: V, half a tile at a time, into a ring of 5 halves, and their cut
//   warp 3   O += P_x V_x (M=128 N=128 K=96), P from tensor memory
//   warps 4..7, 8..11   two softmax groups, one thread a query row.  Group g takes
//            the key tiles with x & 1 = g, half a tile's time apart, so that one's
//            waits, maximum and stores lie beside the other's exponentials.  Both
//            express P and O in one reference a row, the running maximum with
//            lazy rescaling (it moves only when the maximum grows by more than
//            2^8, so P stays <= 256): the tile before hands its reference on
//            through shared memory.  Each group sums its own tiles' rows.  At an
//            item's end the group without the last tile hands over its sums and
//            goes on to the next item's first tile, which is its own; the other
//            one writes O / l.
//   warp 12  work scheduler (counter -> a 4-slot ring of items), then TMA: the item's Q
//            tile.  (Beside the K tiles in warp 0, with items taken three ahead: 8
//            documents with a prefix 150 us where they take 128, 16 of up to 1,531
//            tokens 240 where 232.  An SM then sat on up to 80 key tiles while others
//            had none, and warp 0's own instructions held the K tiles up.)
//   warp 13  watches that the roles get on: no key tile for the call's time limit ends
//            every wait, and the call reports it
//   (warps 14 and 15 give their registers to the softmax groups)
// 96 keys: two score buffers, two of P (so that a P is stored while the product of
// the one before runs), O and all of Q take the 512 tensor-memory columns exactly,
// and products of N = 96 from tensor memory run at the full rate (4,080 MAC a clock
// measured; N = 64: 2,906).
// What bounds it: the SM's shared memory.  A key tile is 60 KB, written once by
// TMA and read once by the products, 960 cycles at 128 bytes a clock, which is
// also what its products take (960 at 4,096 MAC a clock); an item adds Q and O,
// 160 KB.  Measured about 1,200 cycles a tile and 1,100 an item.  With the K and V
// copies left out (wrong results) 16 documents of up to 1,531 tokens took 185 us
// where they took 241, 5 of up to 4,096 tokens 523 where they took 720.
//
// Pairs of CTAs (PAIR): for long documents a cluster of two takes two query tiles of a
// document with one product of 256 rows (cta_group::2), of whose keys and values each
// CTA holds half, so that a key tile costs an SM 30 KB in and 30 KB out: 5 documents
// of up to 4,096 tokens take 678 us instead of 697 (back to back, at the power limit),
// one of 16,384 tokens 2,733 instead of 2,902 (one cold launch).  The even CTA schedules
// and issues; each CTA loads its half and does the softmax of its own
// 128 rows.  What it costs: the first tile's products over the keys that only the second
// sees, and a tile of nothing behind an odd number of them, 4% more tiles in the first
// case, 22% for 16 documents of up to 1,531 tokens (307 us instead of 277).
// Measured on the way, GPU time: the windowed prefill's two threads a row on the same
// tile 309 and 820 us; this form 248 and 745 with lane-0 loops and Q through
// registers.  Two CTAs sharing K/V tiles by multicast, with products of their own, 263
// and 749 (the copies' writes stay); warps of their own for the output 260 and 771;
// pairs with a third of a K tile a copy 295 and 703; O stored without staging 266 and
// 753, and with its 32 KB as a third whole slot of K 253 and 737.  (All of them graphs of
// a few passes; a second of them runs into the power limit, 1.36 kW at 1.47 GHz, and takes
// 277 and 711 us where a single launch takes 237 and 611.)
//
// Code size: the roles' loops share one instruction cache.  At 81 KB of code (every
// wait inlined with its clock) 5.4 of the stalls per instruction were for
// instructions and the second case took 1,290 us; at 35 KB, before few documents were
// planned here, it took 720, and as much at the 51 of now.  Hence waits of a try and a
// flag, with the clock in a warp of its own (the same times as waits that counted their
// tries, at 48 KB), loops that are not unrolled, and the plan's own numbers of key tiles.
#include "common.cuh"
#include "internal.h"

namespace mla {

namespace {

constexpr int kKeys = 96;                        // of a key tile
constexpr uint32_t kAtom = 128 * 128;            // 128 rows x 64 bf16
constexpr uint32_t kKeyAtom = kKeys * 128;       // 96 rows x 64 bf16
constexpr uint32_t kQOff = 0;                    // Q: 3 atoms (staging)
constexpr uint32_t kOOff = 3 * kAtom;            // O: 2 atoms (staging)
constexpr int kHalf = kKeys / 2;
constexpr uint32_t kHalfAtom = kHalf * 128;      // 48 rows x 64 bf16
constexpr uint32_t kKOff = 5 * kAtom;            // K slots, then V slots
// The rings' slots: a third of a K tile (64 dimensions) and half a V tile (48 keys).  In a
// pair of CTAs: a whole tile, of which each CTA holds half, 48 keys of K and 64 dimensions of V.
template <bool PAIR>
struct Rings {
  static constexpr int kKSlots = PAIR ? 4 : 7, kVSlots = PAIR ? 6 : 5;
  static constexpr int kKTiles = PAIR ? kKSlots : 3;  // in flight at most
  static constexpr uint32_t kKSlotBytes = PAIR ? 3 * kHalfAtom : kKeyAtom;
  static constexpr uint32_t kVSlotBytes = PAIR ? kKeyAtom : 2 * kHalfAtom;
  static constexpr uint32_t kVOff = kKOff + kKSlots * kKSlotBytes, kEnd = kVOff + kVSlots * kVSlotBytes;
};
constexpr uint32_t kBarOff = Rings<false>::kEnd;
static_assert(Rings<true>::kEnd <= kBarOff, "rings");
constexpr uint32_t kRefOff = kBarOff + 768;      // references by tile parity, 2 x 128 fp32
constexpr uint32_t kSumOff = kRefOff + 1024;     // sums and references handed over, 128 x 2 fp32
constexpr uint32_t kTileOff = kSumOff + 1024;    // the query tiles of the item ring
constexpr uint32_t kSmemBytes = kTileOff + 256;
static_assert(kSmemBytes <= 232448, "document attention shared memory");
// tensor memory columns: S_0, S_1 (fp32), O (fp32), P_0, P_1 (bf16 pairs), Q (bf16 pairs)
constexpr uint32_t kTmS = 0, kTmO = 2 * kKeys, kTmP = kTmO + 128, kTmQ = kTmP + kKeys;
static_assert(kTmQ + 96 == 512, "tensor memory columns");
constexpr int kThreads = 512;
constexpr int kRoles = 13;                       // warps 0..12; warp 13 watches that they get on
constexpr long long kGroupBytes = 64ll << 20;    // K/V of the heads worked on at a time (at 16 MB 8 documents with a
                                                 // prefix take 144 us, at 64 140, at 160 141; 5 of up to 4,096 tokens
                                                 // 698, 696, 705)
constexpr float kRescaleThreshold = 8.0f;        // log2 units
constexpr int kItemRing = 4;
constexpr uint64_t kSettleNs = 10000000;         // a copy or a product takes microseconds
constexpr int kAhead = 4;                        // key tiles left of an item when the next is asked for (3 to 12 alike)
// Pairs from this many rows of q a document on (8 documents of random lengths around a mean,
// two draws, back to back in us: 1,536 tokens 384 and 405 as single tiles, 391 and 431 in
// pairs; 2,048: 624 and 667, 652 and 671; 2,500: 885 and 958, 908 and 980; 3,000: 1,216 and
// 1,337, 1,204 and 1,304; 4,000: 2,055 and 2,224, 1,999 and 2,198; one of 16,384: 3,257,
// 3,048), where a document's odd last tile of 128, a whole one of 256 here, counts less (8 of
// 2,176: 582, 624; of 2,304: 640, 638).  N and n_docs are what the host knows: cached keys
// gain from pairs with fewer rows too (8 of 512 tokens behind 4,096 517, 493, not taken).
constexpr int kPairRows = 2816;
// ... and under a window of this many keys on (the pair's keys are its window's and 256, a
// tile's 128: 5 documents of 4,000 tokens under 512 keys 414, 433; 1,024: 615, 648; 1,536:
// 786, 788; 2,048: 917, 892).
constexpr int kPairWindow = 2048;
// Up to this many query tiles each CTA makes the plan itself and takes every so many-th item,
// which saves the plan's launch (4 documents of a token 14.3 us, 11.8 without; one of 900
// tokens 26.5, 23.0) and costs balance where an SM's turns are few and long (1,000 tokens
// behind 8,000 231, 238).  Up to 32: 8 documents of 300 tokens 46.5 -> 43.7 and 3 of 600
// 47.9 -> 44.3, but one of 1,900 61.1 -> 62.9 and 2 of 1,000 behind 8,000 469 -> 471.
constexpr int kFewTiles = 16;

// A role's place in a ring of N slots.
template <int N>
struct Place {
  int slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
    }
  }
};

template <bool PAIR>
struct Bars {
  static constexpr int kKTiles = Rings<PAIR>::kKTiles, kKSlots = Rings<PAIR>::kKSlots, kVSlots = Rings<PAIR>::kVSlots;
  uint64_t q_full, q_empty, q_free;
  uint64_t item_full[kItemRing], item_empty[kItemRing];
  uint64_t k_full[kKTiles], k_empty[kKSlots];  // full: a whole tile, of those in flight; empty: a slot
  uint64_t v_full[kVSlots], v_empty[kVSlots], v_cut[kVSlots];  // full and cut: a whole tile, by its first half's slot
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[2], pv_done[2];
  // per quarter of the rows (a warp of each group): every phase is one that a warp has
  // waited for or completed itself, so that its parity cannot be mistaken
  uint64_t ref[2][4], sum[4], o_free[4], o_stored[4];
  uint64_t near_end, drain_s, drain_pv;
  uint64_t ended;  // the roles' warps
  uint32_t tmem_slot;
  int progress;    // key tiles of the first softmax group
  int abort;       // set: every role gives up (the watching warp, or a drain that gave up)

  // A role's wait.  After giving up a role issues nothing more and waits (`drain`) for its own
  // copies and products in flight.  A tile whose copies were issued in part never completes
  // its barrier, and the even CTA of a pair counts the odd one's copies, so a CTA that gives
  // up also stays for kSettleNs, which any copy is long done in.
  // CLUSTER: for what the other CTA of a pair wrote to shared memory.
  template <bool CLUSTER = false>
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    return mbar_wait_or<CLUSTER>(bar, parity, &abort);
  }
};
static_assert(sizeof(Bars<false>) <= 768 && sizeof(Bars<true>) <= 768, "barrier block");

// What differs in a pair of CTAs (cta_group::2): the even one issues the products of
// both, so that a role's signal goes to it, and a product's completion to both, or to it.
// A signal that hands over tensor memory has the tcgen05 fences for its order and is a
// plain arrival; one that hands over shared memory is released to the cluster.  (With
// such releases for all, two a tile and warp, the softmax groups took twice as long a
// tile: 5 documents of up to 4,096 tokens 1,138 us where they take 700.)
template <bool PAIR>
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
  if (PAIR)
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapa_rank(smem_u32(bar), 0)) : "memory");
  else
    mbar_arrive(bar);
}
template <bool PAIR>
__device__ __forceinline__ void release_leader(uint64_t* bar) {
  if (PAIR)
    mbar_arrive_cluster(mapa_rank(smem_u32(bar), 0));
  else
    mbar_arrive(bar);
}
template <bool PAIR>
__device__ __forceinline__ void commit_both(uint64_t* bar) {
  if (PAIR)
    umma_commit_pair(bar, 3);
  else
    umma_commit(bar);
}
template <bool PAIR>
__device__ __forceinline__ void commit_leader(uint64_t* bar) {
  if (PAIR)
    umma_commit_pair(bar, 1);
  else
    umma_commit(bar);
}
// A box of rows and 64-number atoms, counted on the even CTA's barrier.
template <bool PAIR>
__device__ __forceinline__ void load_leader(void* dst, const CUtensorMap* map, uint64_t* bar, int row, int atom,
                                            int outer) {
  if (PAIR)
    tma_load_4d_pair(dst, map, mapa_rank(smem_u32(bar), 0), 0, row, atom, outer);
  else
    tma_load_4d(dst, map, bar, 0, row, atom, outer);
}
template <bool PAIR>
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if (PAIR)
    umma_bf16_ts_pair(d, a, b, idesc, accumulate);
  else
    umma_bf16_ts(d, a, b, idesc, accumulate);
}

// A document's query tile, as the plan lists it: its rows q_row .. q_row + rows
// - 1 sit at positions pos .. (below 0: before the document's first key), its
// keys begin at row k_row; the first `prefix` are seen by every query.  Its key
// tiles: first n_sink tiles over keys 0 .. n_first - 1, which are seen however far
// back they are (the prefix, the sinks), then tiles from w0 on, the window's first
// key; where the former reach the window, the tiles run from key 0.  `end` is the
// key behind the last one that the tile's queries see.
struct __align__(16) DocTile {
  int q_row, rows, k_row, pos, prefix, head;
  int n_kv, w0, n_first, n_sink, end, pad;
  __device__ __forceinline__ void set_keys(int window, int sinks) {
    const int last = pos + rows;  // behind the last query's position
    w0 = max(0, pos - window + 1);
    end = max(last, prefix);
    n_first = max(prefix, min(sinks, last));
    if (n_first >= w0) w0 = n_first = 0;
    n_first = max(n_first, 0);
    n_sink = (n_first + kKeys - 1) / kKeys;
    // (one tile of nothing where no key is seen: its item stores zeros)
    n_kv = max(1, n_sink + max(0, end - w0 + kKeys - 1) / kKeys);
  }
  // first key of key tile j
  __device__ __forceinline__ int key0(int j) const { return j < n_sink ? j * kKeys : w0 + (j - n_sink) * kKeys; }
  // its keys that some query may see: those behind them are not the document's, or nobody's
  __device__ __forceinline__ int keys(int j) const {
    return max(0, min(kKeys, (j < n_sink ? n_first : end) - key0(j)));
  }
};
static_assert(sizeof(DocTile) == kDocTileBytes && kItemRing * sizeof(DocTile) <= 256, "tiles of the item ring");
// The plan: this, then the tiles, heaviest first.
struct DocPlan {
  int n_tiles, group_log, pad[10];
};
static_assert(sizeof(DocPlan) == kDocTileBytes, "the plan's head is as long as a tile");

// A document's rows and keys.
struct Doc {
  int q0, n, k0, keys, prefix;
  __device__ __forceinline__ Doc() {}
  __device__ __forceinline__ Doc(const DocAttnArgs& a, int d) {
    const int* ck = a.cu_k ? a.cu_k : a.cu_q;
    const int q1 = a.cu_q[d + 1], k1 = ck[d + 1], p = a.prefix ? a.prefix[d] : 0;
    q0 = a.cu_q[d];
    k0 = ck[d];
    n = q1 - q0;
    keys = k1 - k0;
    prefix = max(0, min(p, keys));
  }
  __device__ __forceinline__ bool bad(const DocAttnArgs& a) const {
    // (differences of numbers in range do not overflow; of others any answer but "in order" will do)
    return q0 < 0 || q0 > a.N || n < 0 || n > a.N - q0 || k0 < 0 || k0 > a.cap || keys < 0 || keys > a.cap - k0;
  }
};

// The query tile of `rows` at most that begins at row `at` of a document.
__device__ __forceinline__ DocTile tile_at(const Doc& d, int at, int rows, int window, int sinks) {
  DocTile tile{};
  tile.q_row = d.q0 + at;
  tile.rows = min(rows, d.n - at);
  tile.k_row = d.k0;
  tile.pos = d.keys - d.n + at;
  tile.prefix = d.prefix;
  tile.set_keys(window, sinks);
  return tile;
}

// Heads a group, a power of two: the smallest whose work is at least 1.5 times the
// workers times the heaviest item (the heavy tiles of the last group then start early
// enough), halved while its heads' K/V exceed kGroupBytes of L2.
__device__ __forceinline__ int group_log_of(const DocAttnArgs& a, unsigned long long key_tiles, int heaviest,
                                            int workers) {
  const unsigned long long need = (3ull * workers * heaviest + 2 * key_tiles - 1) / (2 * key_tiles);
  const int* ck = a.cu_k ? a.cu_k : a.cu_q;
  const long long kv_head_bytes = ((long long)ck[a.n_docs] - ck[0]) * (192 + 128) * 2;
  int log = 0;
  while ((1ull << log) < need && log < 6) ++log;
  while (log > 0 && (kv_head_bytes << log) > kGroupBytes) --log;
  return log;
}

// The query tile and head of work item w: groups of 2^log heads, in a group tile
// after tile, in a tile head after head.
__device__ __forceinline__ void doc_item(int w, int n_tiles, int log, int& tile, int& head) {
  const int per = n_tiles << log, g = w / per, r = w - g * per;
  tile = r >> log;
  head = (g << log) + (r & ((1 << log) - 1));
}

// A warpgroup's registers a thread, from those of the launch (65,536 / 512 threads = 128).
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// One lane of a whole warp.  The control warps run their loops as warps and let one
// lane issue, so that the operands of the copies and products are uniform values:
// with the loops in lane 0 alone the twelve products of a tile's scores took 1,255
// cycles to issue (with three waits), so 661.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

// A warp reads item `it` from the ring, then releases the slot.  False: a wait gave up.
template <bool PAIR>
__device__ __forceinline__ bool read_item(uint8_t* smem, Bars<PAIR>* bar, int it, DocTile& tile) {
  const int slot = it % kItemRing;
  if (!bar->template wait<PAIR>(&bar->item_full[slot], (it / kItemRing) & 1)) return false;
  tile = reinterpret_cast<const DocTile*>(smem + kTileOff)[slot];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&bar->item_empty[slot]);
  return true;
}

__device__ __forceinline__ void st_cluster(uint32_t addr, int x) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void copy_q(uint32_t taddr, uint64_t desc) {
  if (PAIR)
    tmem_copy_128x256b_pair(taddr, desc);
  else
    tmem_copy_128x256b(taddr, desc);
}

// the lowest n bits of 32 (none for n < 0, all for n > 32)
__device__ __forceinline__ uint32_t first_bits(int n) {
  uint32_t m;
  asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(m) : "r"(max(n, 0)));
  return m;
}

// Word `lane` of the tile that lane `from` holds.
__device__ __forceinline__ int word_of(const DocTile& mine, int from) {
  int word = 0;
#pragma unroll
  for (int i = 0; i < (int)sizeof(DocTile) / 4; ++i) {
    const int x = __shfl_sync(0xffffffffu, reinterpret_cast<const int*>(&mine)[i], from);
    if ((int)(threadIdx.x & 31) == i) word = x;
  }
  return word;
}

// The plan of a few documents by one warp of every CTA, a tile a lane: `mine`, of the
// place-th most key tiles (-1: none).  Offsets out of order or range leave no tiles.
__device__ __forceinline__ void few_tiles(const DocAttnArgs& a, int window, int sinks, int& n_tiles, int& group_log,
                                       DocTile& mine, int& place, const DevStatus& st) {
  const int lane = threadIdx.x & 31;
  Doc doc;
  doc.q0 = doc.n = doc.k0 = doc.keys = doc.prefix = 0;
  if (lane < a.n_docs) doc = Doc(a, lane);
  const bool bad = __any_sync(0xffffffffu, doc.bad(a));
  if (blockIdx.x == 0 && lane == 0) {
    st.word[0] = bad ? kStatusBadLength : 0u;
    st.word[kStatusExtraWord] = 0u;
  }
  const int count = bad ? 0 : (doc.n + 127) / 128;
  int behind = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, behind, o);
    if (lane >= o) behind += y;
  }
  n_tiles = __shfl_sync(0xffffffffu, behind, 31);
  int d = 0;  // this lane's tile's document: the first one that ends behind it
  for (int k = 0; k < a.n_docs; ++k) d += __shfl_sync(0xffffffffu, behind, k) <= lane;
  d = min(d, 31);
  const int first = __shfl_sync(0xffffffffu, behind - count, d);
  Doc of;
  of.q0 = __shfl_sync(0xffffffffu, doc.q0, d);
  of.n = __shfl_sync(0xffffffffu, doc.n, d);
  of.k0 = __shfl_sync(0xffffffffu, doc.k0, d);
  of.keys = __shfl_sync(0xffffffffu, doc.keys, d);
  of.prefix = __shfl_sync(0xffffffffu, doc.prefix, d);
  const bool some = lane < n_tiles;
  if (some) mine = tile_at(of, (lane - first) * 128, 128, window, sinks);
  const int n_kv = some ? mine.n_kv : 0;
  int heaviest = n_kv, before = 0;
  unsigned long long key_tiles = n_kv;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    heaviest = max(heaviest, __shfl_xor_sync(0xffffffffu, heaviest, o));
    key_tiles += __shfl_xor_sync(0xffffffffu, key_tiles, o);
  }
#pragma unroll 1
  for (int k = 0; k < n_tiles; ++k) {
    const int y = __shfl_sync(0xffffffffu, n_kv, k);
    before += y > n_kv || (y == n_kv && k < lane);
  }
  place = some ? before : -1;
  group_log = n_tiles ? group_log_of(a, key_tiles, heaviest, gridDim.x) : 0;
}

template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    document_attn_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, float sl2,
                     int window, int sinks, int* __restrict__ work, const uint8_t* __restrict__ plan, const DocAttnArgs a,
                     const DevStatus st) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using R = Rings<PAIR>;
  constexpr int kKSlots = R::kKSlots, kVSlots = R::kVSlots, kKTiles = R::kKTiles;
  Bars<PAIR>* bar = reinterpret_cast<Bars<PAIR>*>(smem + kBarOff);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);  // (uniform to the compiler)
  const int lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_ctarank() : 0;
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    mbar_init(&bar->q_full, 1);
    mbar_init(&bar->q_empty, 1);
    mbar_init(&bar->q_free, 1);
    for (int i = 0; i < kItemRing; ++i) {
      mbar_init(&bar->item_full[i], 1);
      // producers, issuers and softmax warps; in a pair the odd CTA's scheduler for its own
      mbar_init(&bar->item_empty[i], leader ? 12 + PAIR : 10);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->p_full[i], PAIR ? 8 : 4);  // the group's warps, of both CTAs
      mbar_init(&bar->s_full[i], 1);
      mbar_init(&bar->s_free[i], PAIR ? 8 : 4);
      mbar_init(&bar->pv_done[i], 1);
      for (int q = 0; q < 4; ++q) mbar_init(&bar->ref[i][q], 32);
    }
#pragma unroll 1
    for (int i = 0; i < kKSlots; ++i) mbar_init(&bar->k_empty[i], 1);
    for (int i = 0; i < kKTiles; ++i) mbar_init(&bar->k_full[i], 1);
#pragma unroll 1
    for (int i = 0; i < kVSlots; ++i) {
      mbar_init(&bar->v_full[i], 1);
      mbar_init(&bar->v_empty[i], 1);
      mbar_init(&bar->v_cut[i], PAIR ? 2 : 1);
    }
    for (int q = 0; q < 4; ++q) {
      mbar_init(&bar->sum[q], 32);
      mbar_init(&bar->o_free[q], 32);
      mbar_init(&bar->o_stored[q], 1);
    }
    mbar_init(&bar->near_end, 1);
    mbar_init(&bar->drain_s, 1);
    mbar_init(&bar->drain_pv, 1);
    mbar_init(&bar->ended, kRoles);
    bar->progress = 0;
    bar->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(&bar->tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&bar->tmem_slot, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // both CTAs' barriers exist before any signal from the other
  tc_fence_after();
  const uint32_t tmem = bar->tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  bool ok = true;
  auto drain = [&](uint64_t& b, uint32_t parity) {
    const bool done = mbar_drain(&b, parity, max(st.wait_limit_ns, kSettleNs));
    if (!done && lane == 0) *static_cast<volatile int*>(&bar->abort) = warp + 1;
    return done;
  };
  if (warp < 4) {
    registers_down<96>();
    if (warp == 0) {
      // ---- K producer ----
      if (elected()) tma_prefetch_desc(&tmK);
      Place<kKSlots> k;
      Place<kKTiles> full;
#pragma unroll 1
      for (int it = 0; ok; ++it) {
        DocTile tile;
        if (!(ok = read_item<PAIR>(smem, bar, it, tile)) || tile.rows == 0) break;
#pragma unroll 1
        for (int j = 0; ok && j < tile.n_kv; ++j) {
          if (leader && j > 0 && j == tile.n_kv - kAhead) {
            if (elected()) mbar_arrive(&bar->near_end);
            __syncwarp();
          }
          const int key = tile.k_row + tile.key0(j);
          if (PAIR) {
            if (!(ok = bar->wait(&bar->k_empty[k.slot], k.phase ^ 1))) break;
            if (elected()) {
              if (leader) mbar_arrive_expect_tx(&bar->k_full[k.slot], 3 * kKeyAtom);
              load_leader<PAIR>(smem + kKOff + k.slot * R::kKSlotBytes, &tmK, &bar->k_full[k.slot],
                                key + rank * kHalf, 0, tile.head);
            }
            __syncwarp();
            k.next();
          } else {
#pragma unroll 1
            for (int c = 0; c < 3; ++c, k.next()) {
              if (!(ok = bar->wait(&bar->k_empty[k.slot], k.phase ^ 1))) break;
              if (elected()) {
                if (c == 0) mbar_arrive_expect_tx(&bar->k_full[full.slot], 3 * kKeyAtom);
                load_leader<PAIR>(smem + kKOff + k.slot * R::kKSlotBytes, &tmK, &bar->k_full[full.slot], key, c,
                                  tile.head);
              }
              __syncwarp();
            }
          }
          full.next();
        }
      }
      // no copy may still be in flight into shared memory
#pragma unroll 1
      for (int i = 0; leader && i < kKTiles; ++i, full.next())
        if (!drain(bar->k_full[full.slot], full.phase ^ 1)) break;
    } else if (warp == 1) {
      if (leader) {
        // ---- S issuer: S_x = Q K_x^T into score buffer x & 1 ----
        constexpr uint32_t idesc_s = idesc_bf16(PAIR ? 256 : 128, kKeys, false, false);
        const uint32_t k_addr = smem_u32(smem + kKOff);
        int x = 0;
        Place<kKSlots> k;
        Place<kKTiles> full;
#pragma unroll 1
        for (int it = 0; ok; ++it) {
          DocTile tile;
          if (!(ok = read_item<PAIR>(smem, bar, it, tile)) || tile.rows == 0) break;
          // the item's Q rows (three 128-byte-swizzled 64-column atoms) into tensor memory as bf16
          // pairs, the A operand of every S, once the S of the item before are done
          if (!(ok = bar->wait(&bar->q_full, it & 1) && (it == 0 || bar->wait(&bar->q_free, (it - 1) & 1)))) break;
          tc_fence_after();
          if (elected()) {
#pragma unroll
            for (int kk = 0; kk < 12; ++kk)
              copy_q<PAIR>(tmem + kTmQ + kk * 8,
                           sdesc_sw128(smem_u32(smem + kQOff) + (kk >> 2) * kAtom + (kk & 3) * 32, 16, 1024));
            commit_both<PAIR>(&bar->q_empty);  // the staging atoms may take the Q after it
          }
          __syncwarp();
#pragma unroll 1
          for (int j = 0; ok && j < tile.n_kv; ++j, ++x) {
            const int sb = x & 1, keys = tile.keys(j);
            // (a tile's last columns, behind the last key, are masked whatever they hold: a shorter
            // product takes as long and less power, 16 documents of up to 1,531 tokens 270 us, so 267)
            const uint32_t idesc = PAIR || keys > 64 ? idesc_s : idesc_bf16(128, 64, false, false);
            // the tile is there, and the group has read the buffer's previous scores (tile x - 2)
            if (!(ok = bar->wait(&bar->k_full[full.slot], full.phase) &&
                       (x < 2 || bar->wait(&bar->s_free[sb], ((x - 2) >> 1) & 1))))
              break;
            full.next();
            tc_fence_after();
            if (PAIR) {
              const uint64_t kb = sdesc_sw128(k_addr + k.slot * R::kKSlotBytes, 16, 1024);
              if (elected()) {
#pragma unroll
                for (int kk = 0; kk < 12; ++kk)
                  product<PAIR>(tmem + kTmS + sb * kKeys, tmem + kTmQ + kk * 8,
                                kb + (kk >> 2) * (kHalfAtom >> 4) + (kk & 3) * 2, idesc, kk > 0 ? 1u : 0u);
                commit_both<PAIR>(&bar->k_empty[k.slot]);
                commit_both<PAIR>(&bar->s_full[sb]);
              }
              __syncwarp();
              k.next();
            } else {
#pragma unroll
              for (int c = 0; c < 3; ++c, k.next()) {
                const uint64_t kb = sdesc_sw128(k_addr + k.slot * R::kKSlotBytes, 16, 1024);
                if (elected()) {
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk)
                    product<PAIR>(tmem + kTmS + sb * kKeys, tmem + kTmQ + c * 32 + kk * 8, kb + kk * 2, idesc,
                                  c > 0 || kk > 0 ? 1u : 0u);
                  commit_both<PAIR>(&bar->k_empty[k.slot]);
                  if (c == 2) commit_both<PAIR>(&bar->s_full[sb]);
                }
                __syncwarp();
              }
            }
          }
          if (!ok) break;
          if (elected()) commit_leader<PAIR>(&bar->q_free);  // the item's S are done: its Q may be replaced
          __syncwarp();
        }
        if (elected()) commit_leader<PAIR>(&bar->drain_s);
        __syncwarp();
        drain(bar->drain_s, 0);
      }
    } else if (warp == 2) {
      // ---- V producer: half tiles, and clears what lies behind the last key ----
      Place<kVSlots> v;
      uint32_t phases = 0;  // of each slot's full barrier
      if (elected()) tma_prefetch_desc(&tmV);
#pragma unroll 1
      for (int it = 0; ok; ++it) {
        DocTile tile;
        if (!(ok = read_item<PAIR>(smem, bar, it, tile)) || tile.rows == 0) break;
#pragma unroll 1
        for (int j = 0; ok && j < tile.n_kv; ++j) {
          // (a second half that no query sees is left out)
          const int keys = tile.keys(j), halves = PAIR || keys <= kHalf ? 1 : 2, first = v.slot;
          const int key = tile.k_row + tile.key0(j);
          const bool cut = keys == 0 || (keys & 15);
#pragma unroll 1
          for (int h = 0; h < halves; ++h, v.next()) {
            if (!(ok = bar->wait(&bar->v_empty[v.slot], v.phase ^ 1))) break;
            if (elected()) {
              uint8_t* const at = smem + R::kVOff + v.slot * R::kVSlotBytes;
              // (in a pair, a tile that is to be cut arrives on each CTA's own barrier)
              if (h == 0 && (cut || leader))
                mbar_arrive_expect_tx(&bar->v_full[first], PAIR ? (cut ? 1 : 2) * kKeyAtom : halves * R::kVSlotBytes);
              if (PAIR && cut)
                tma_load_4d(at, &tmV, &bar->v_full[first], 0, key, rank, tile.head);
              else
                load_leader<PAIR>(at, &tmV, &bar->v_full[first], key + h * kHalf, rank, tile.head);
            }
            __syncwarp();
          }
          if (ok && cut) {  // rows `keys` .. of the last 16-key step: eight lanes a row and atom
            if (!(ok = bar->wait(&bar->v_full[first], (phases >> first) & 1))) break;
            const int last = halves == 1 ? first : (first + 1) % kVSlots, from = keys - (halves - 1) * kHalf;
            uint8_t* const mine =
                smem + R::kVOff + last * R::kVSlotBytes + (PAIR ? 0 : ((lane >> 3) & 1) * kHalfAtom) + (lane & 7) * 16;
#pragma unroll 1
            for (int r = from + (PAIR ? lane >> 3 : lane >> 4); r < max(16, (from + 15) & ~15); r += PAIR ? 4 : 2)
              *reinterpret_cast<uint4*>(mine + r * 128) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (elected()) release_leader<PAIR>(&bar->v_cut[first]);
            __syncwarp();
          }
          if (leader || cut) phases ^= 1u << first;
        }
      }
      // (every tile has arrived: its slot's barrier has left the phase before its next one)
#pragma unroll 1
      for (int i = 0; i < kVSlots; ++i)
        if (!drain(bar->v_full[i], ((phases >> i) & 1) ^ 1)) break;
    } else if (warp == 3) {
      if (leader) {
        // ---- P.V issuer: O += P_x V_x ----
        constexpr uint32_t idesc_pv = idesc_bf16(PAIR ? 256 : 128, 128, false, true);
        const uint32_t v_addr = smem_u32(smem + R::kVOff);
        int x = 0;
        Place<kVSlots> v;
        uint32_t phases = 0, cuts = 0;  // of each slot's full and cut barriers
#pragma unroll 1
        for (int it = 0; ok; ++it) {
          DocTile tile;
          if (!(ok = read_item<PAIR>(smem, bar, it, tile)) || tile.rows == 0) break;
#pragma unroll 1
          for (int j = 0; j < tile.n_kv; ++j, ++x) {
            const int sb = x & 1, first = v.slot;
            // the 16-key steps that hold a key (one where there is none: O becomes zeros), the
            // last one's other rows cleared
            const int keys = tile.keys(j), steps = max(1, (keys + 15) >> 4);
            if (!(ok = bar->wait(&bar->v_full[first], (phases >> first) & 1))) break;
            phases ^= 1u << first;
            if (keys == 0 || (keys & 15)) {
              if (!(ok = bar->template wait<PAIR>(&bar->v_cut[first], (cuts >> first) & 1))) break;
              cuts ^= 1u << first;
            }
            // P_x is written (and, for an item's first tile, the previous item's O read)
            if (!(ok = bar->wait(&bar->p_full[sb], (x >> 1) & 1))) break;
            tc_fence_after();
            constexpr int kSlotsOfTile = PAIR ? 1 : 2, kSteps = kKeys / 16 / kSlotsOfTile;
#pragma unroll
            for (int h = 0; h < kSlotsOfTile; ++h) {
              if (h && keys <= kHalf) break;
              const uint64_t vb = sdesc_sw128(v_addr + v.slot * R::kVSlotBytes, kHalfAtom, 1024);
              if (elected()) {
#pragma unroll
                for (int kk = 0; kk < kSteps; ++kk)
                  if (h * kSteps + kk < steps)
                    product<PAIR>(tmem + kTmO, tmem + kTmP + sb * kHalf + (h * kSteps + kk) * 8, vb + kk * 128, idesc_pv,
                                  (j > 0 || h > 0 || kk > 0) ? 1u : 0u);
                commit_both<PAIR>(&bar->v_empty[v.slot]);
              }
              __syncwarp();
              v.next();
            }
            if (elected()) commit_both<PAIR>(&bar->pv_done[sb]);
            __syncwarp();
          }
        }
        if (elected()) commit_leader<PAIR>(&bar->drain_pv);
        __syncwarp();
        drain(bar->drain_pv, 0);
      }
    }
  } else if (warp >= 12) {
    registers_down<64>();
    if (warp == 12) {
      // ---- work scheduler and Q producer ----
      const DocPlan* head = reinterpret_cast<const DocPlan*>(plan);
      const int* tiles = reinterpret_cast<const int*>(plan + sizeof(DocPlan)) + min(lane, (int)sizeof(DocTile) / 4 - 1);
      int n_tiles, group_log, place = -1;  // (few: this lane's tile is the place-th heaviest)
      DocTile mine{};
      const bool few = !PAIR && !plan;
      if (few)
        few_tiles(a, window, sinks, n_tiles, group_log, mine, place, st);
      else
        n_tiles = head->n_tiles, group_log = head->group_log;
      const int n_items = 64 * n_tiles;
      DocTile* const ring = reinterpret_cast<DocTile*>(smem + kTileOff);
      if (elected()) tma_prefetch_desc(&tmQ);
      // the next item: the counter's, or of few tiles every CTA's in turn, there and back
      auto ask = [&](int it) {
        if (few) return it * (int)gridDim.x + (it & 1 ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x);
        return lane == 0 ? atomicAdd(work, 1) : 0;
      };
      int index = leader ? ask(0) : 0, it = 0, n_long = 0;
#pragma unroll 1
      for (; ok; ++it) {
        // the item's tile (a word a lane) into the ring, where every role finds it
        const int slot = it % kItemRing, turn = it / kItemRing;
        if (leader) {
          index = __shfl_sync(0xffffffffu, index, 0);
          int word = 0;  // (no rows: the end)
          if (index < n_items) {
            int at, of;
            doc_item(index, n_tiles, group_log, at, of);
            if (few)
              word = word_of(mine, __ffs(__ballot_sync(0xffffffffu, place == at)) - 1);
            else
              word = tiles[at * (int)(sizeof(DocTile) / 4)];
            if (lane == (int)offsetof(DocTile, head) / 4) word = of;
          }
          if (turn > 0 && !(ok = bar->wait(&bar->item_empty[slot], (turn - 1) & 1))) break;
          if (lane < (int)sizeof(DocTile) / 4) {
            int* const at = reinterpret_cast<int*>(&ring[slot]) + lane;
            *at = word;
            if (PAIR) st_cluster(mapa_rank(smem_u32(at), 1), word);
          }
          __syncwarp();
          if (elected()) {  // release
            mbar_arrive(&bar->item_full[slot]);
            if (PAIR) mbar_arrive_cluster(mapa_rank(smem_u32(&bar->item_full[slot]), 1));
          }
          __syncwarp();
        } else if (!(ok = bar->template wait<PAIR>(&bar->item_full[slot], turn & 1))) {
          break;
        }
        const int rows = ring[slot].rows, n_kv = ring[slot].n_kv, q_row = ring[slot].q_row, of = ring[slot].head;
        if (rows == 0) break;
        // A long item's successor is asked for when its last key tiles are being loaded, so that
        // no SM sits on work while others have none; a short one's at once, for its latency
        const bool is_long = n_kv > kAhead;
        if (leader && !is_long) index = ask(it + 1);
        // its Q, into the staging atoms once the one before has been copied into tensor memory
        if (it > 0 && !(ok = bar->wait(&bar->q_empty, (it - 1) & 1))) break;
        if (elected()) {
          if (leader) mbar_arrive_expect_tx(&bar->q_full, (PAIR ? 6 : 3) * kAtom);
          load_leader<PAIR>(smem + kQOff, &tmQ, &bar->q_full, q_row + rank * 128, of * 3, 0);
        }
        __syncwarp();
        if (leader && is_long) {
          if (!(ok = bar->wait(&bar->near_end, n_long++ & 1))) {
            ++it;  // (its Q is on the way)
            break;
          }
          index = ask(it + 1);
        }
        if (!leader && it >= 2) {  // two items back: it has been read by now
          if (!(ok = bar->wait(&bar->item_empty[(it - 2) % kItemRing], ((it - 2) / kItemRing) & 1))) break;
          if (elected()) release_leader<PAIR>(&bar->item_empty[(it - 2) % kItemRing]);
          __syncwarp();
        }
      }
      if (leader && it > 0) drain(bar->q_full, (it - 1) & 1);
    }
    if (warp == kRoles) mbar_watch(&bar->ended, &bar->progress, st.wait_limit_ns, &bar->abort, kRoles + 1);
  } else {
    registers_up<168>();
    // ---- softmax groups, one thread a query row ----
    const int g = (warp >> 2) - 1;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    float* const refs = reinterpret_cast<float*>(smem + kRefOff) + row;    // + 128 x parity of the tile
    float2* const sums = reinterpret_cast<float2*>(smem + kSumOff) + row;
    auto wait = [&](uint64_t& b, int phase) { return bar->wait(&b, phase & 1); };
    auto rows_done = [&](uint64_t& b) {
      __syncwarp();
      if (lane == 0) arrive_leader<PAIR>(&b);
    };
    // Item by item, this group's tiles of each.  At an item's end the group with the
    // last tile `ends` it: it writes O / l.  The other group goes on to the next item's
    // first tile, which is its own.
    int x0 = 0;    // this CTA's key tiles before the item
    bool stored = false;  // the staging atoms of O are still being read
#pragma unroll 1
    for (int it = 0;; ++it) {
      DocTile tile;
      if (!(ok = read_item<PAIR>(smem, bar, it, tile)) || tile.rows == 0) break;
      if (PAIR) {  // this CTA's tile of the two (the odd one may have no rows)
        tile.q_row += rank * 128;
        tile.pos += rank * 128;
        tile.rows -= rank * 128;
      }
      const int last = x0 + tile.n_kv - 1;
      const bool ends = (last & 1) == g;
      float m = -INFINITY, l = 0.f;  // this group's sum, relative to 2^m
#pragma unroll 1
      for (int x = x0 + ((x0 ^ g) & 1);; x += 2) {
        const bool here = x <= last;
        const int j = x - x0;
        float m_old = 0.f, m_new = 0.f;
        bool need = false;
        uint32_t pk[kKeys / 2];
        if (here) {
          if (!(ok = wait(bar->s_full[g], x >> 1))) break;
          if (warp == 4 && lane == 0) *static_cast<volatile int*>(&bar->progress) = x;
          tc_fence_after();
          uint32_t s[kKeys];
#pragma unroll
          for (int c = 0; c < kKeys; c += 32)
            tmem_ld32(tmem + lanes + kTmS + g * kKeys + c, *reinterpret_cast<uint32_t(*)[32]>(&s[c]));
          tmem_wait_ld();
          tc_fence_before();
          rows_done(bar->s_free[g]);  // the score buffer may take S_{x+2}
          // where some row of the warp sees a part of the tile: the keys that this thread's
          // row sees, lo .. hi - 1 of the window and 0 .. near - 1 however far back, as bits
          const int k0 = tile.key0(j), first = tile.pos + quarter * 32;
          const bool in_sinks = j < tile.n_sink;
          if (in_sinks ? k0 + kKeys > tile.n_first
                       : k0 + kKeys > tile.prefix && (first + 31 - k0 >= window || k0 + kKeys - 1 > first)) {
            const int i = first + lane;
            const int hi = in_sinks ? 0 : i + 1 - k0, lo = i + 1 - window - k0;
            const int near = max(tile.prefix, min(sinks, i + 1)) - k0;
#pragma unroll
            for (int c0 = 0; c0 < kKeys; c0 += 32) {
              const uint32_t seen = (first_bits(hi - c0) & ~first_bits(lo - c0)) | first_bits(near - c0);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(seen & (1u << c))) s[c0 + c] = __float_as_uint(-INFINITY);
            }
          }
          // max of the raw scores (the scale is positive): eight partial maxima and
          // sums, three-input maxima, two-lane FMA and add
          float mp[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mp[i] = fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 8]));
#pragma unroll
          for (int c = 16; c < kKeys; c += 16)
#pragma unroll
            for (int i = 0; i < 8; ++i) mp[i] = fmax3(mp[i], __uint_as_float(s[c + i]), __uint_as_float(s[c + 8 + i]));
          const float mx = sl2 * fmaxf(fmax3(mp[0], mp[1], mp[2]), fmax3(mp[3], mp[4], fmax3(mp[5], mp[6], mp[7])));
          // the reference after the tile before, and after this one
          if (x > 0 && !(ok = wait(bar->ref[g ^ 1][quarter], (x - 1) >> 1))) break;
          m_old = j > 0 ? refs[(g ^ 1) * 128] : -INFINITY;
          need = mx > m_old + kRescaleThreshold;
          m_new = need ? mx : m_old;
          refs[g * 128] = m_new;
          mbar_arrive(&bar->ref[g][quarter]);
          if (m != m_new) l *= ex2_approx(m - m_new);
          m = m_new;
          const float ref = m_new == -INFINITY ? 0.f : m_new;  // (all that a row sees so far may score -infinity)
          // P as bf16 pairs (low half = even key; 2^-8 of each, both operands of an MMA
          // have one type and V is bf16; the sum takes the float32 values)
          float sp[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < kKeys; c += 2) {
            float y0, y1;
            fma_x2(y0, y1, __uint_as_float(s[c]), __uint_as_float(s[c + 1]), sl2, sl2, -ref, -ref);
            const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
            add_x2(sp[c & 7], sp[(c & 7) + 1], sp[c & 7], sp[(c & 7) + 1], p0, p1);
            pk[c / 2] = pack_bf16x2(p0, p1);
          }
          l += ((sp[0] + sp[1]) + (sp[2] + sp[3])) + ((sp[4] + sp[5]) + (sp[6] + sp[7]));
        }
        if (stored) {
          if (lane == 0) {
            bulk_wait_read<0>();
            mbar_arrive(&bar->o_stored[quarter]);
          }
          stored = false;
        }
        if (!here) break;
        // this group's tile before has been read: its P may be replaced
        if (x > 1 && !(ok = wait(bar->pv_done[g], (x - 2) >> 1))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kHalf; c += 16) tmem_st16(tmem + lanes + kTmP + g * kHalf + c, &pk[c]);
        // an item's first tile replaces O, which must have been read
        if (j == 0 && it > 0 && !(ok = wait(bar->o_free[quarter], it - 1))) break;
        if (j > 0 && __any_sync(0xffffffffu, need)) {
          // O in the new reference, once the tile before has been added
          if (!(ok = wait(bar->pv_done[g ^ 1], (x - 1) >> 1))) break;
          tc_fence_after();
          const float alpha = need ? ex2_approx(m_old - m_new) : 1.f;
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            uint32_t r[16];
            tmem_ld16(tmem + lanes + kTmO + c, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
            tmem_st16(tmem + lanes + kTmO + c, r);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        rows_done(bar->p_full[g]);
      }
      if (!ok) break;
      if (!ends) {
        *sums = make_float2(l, m);
        mbar_arrive(&bar->sum[quarter]);
      } else {
        // O / l through this row of the staging atoms, once the O before has left them, and a
        // TMA store; where the document ends among this warp's rows, each row that it has is
        // stored by itself
        if (!(ok = wait(bar->sum[quarter], it) && (it == 0 || wait(bar->o_stored[quarter], it - 1)) &&
                   wait(bar->pv_done[g], last >> 1)))
          break;
        tc_fence_after();
        const float2 other = *sums;
        if (other.x != 0.f) l += other.x * ex2_approx(other.y - m);
        const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);  // (a row that saw no key: its O is zeros)
        const bool whole = quarter * 32 + 32 <= tile.rows, mine = row < tile.rows;
        // 16-byte unit u of the row: base + (u / 8) * atom + ((u % 8) ^ flip) * 16
        uint8_t* base = whole ? smem + kOOff + row * 128
                              : reinterpret_cast<uint8_t*>(a.o + (long long)(tile.q_row + row) * a.o_row + tile.head * 128);
        const int atom = whole ? (int)kAtom : 128, flip = whole ? row & 7 : 0;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t r[64];
          tmem_ld32(tmem + lanes + kTmO + c * 64, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
          tmem_ld32(tmem + lanes + kTmO + c * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
          tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float y0, y1;
              fma_x2(y0, y1, __uint_as_float(r[8 * u + 2 * i]), __uint_as_float(r[8 * u + 2 * i + 1]), inv, inv, 0.f, 0.f);
              w[i] = pack_bf16x2(y0, y1);
            }
            if (mine) *reinterpret_cast<uint4*>(base + ((u ^ flip) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          base += atom;
        }
        tc_fence_before();
        mbar_arrive(&bar->o_free[quarter]);
        fence_proxy_async_smem();
        __syncwarp();
        if (whole && lane == 0) {
          const uint8_t* rows = smem + kOOff + quarter * 32 * 128;
          for (int c = 0; c < 2; ++c)
            tma_store_3d(&tmO, rows + c * kAtom, tile.head * 128 + 64 * c, tile.q_row + quarter * 32, 0);
          bulk_commit();
        }
        stored = true;
      }
      x0 = last + 1;
    }
    if (lane == 0) bulk_wait_all();
  }
  if (warp < kRoles && lane == 0) mbar_arrive(&bar->ended);

  tc_fence_before();
  __syncthreads();
  if (*static_cast<volatile int*>(&bar->abort)) {
    const uint64_t since = globaltimer_ns();
#pragma unroll 1
    while (globaltimer_ns() - since < kSettleNs) __nanosleep(100000);
    if (threadIdx.x == 0) report_timeout(st, bar->abort);
  }
  __syncwarp();
  if (PAIR) cluster_sync();  // (the other CTA's products, copies and signals are done)
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

// ---- the documents' query tiles ------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kBuckets = kPlanThreads;  // tiles are ordered by their number of key tiles, up to this many
constexpr int kDocsInSmem = 1024;

// Exclusive sums over the block, and the total (sh: one int a warp).
__device__ __forceinline__ int block_before(int v, int& total, int* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  int w = sh[lane];  // (as many warps as lanes)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
  __syncthreads();
  return before + x - v;
}
static_assert(kPlanThreads == 32 * 32, "a lane for each warp");

// One CTA: the documents' numbers of query tiles, the tiles' numbers of key
// tiles counted by value, and the tiles in that order, the heaviest first (the
// order among equals is any: an item's result does not depend on it).  An
// offset that is out of order or out of range leaves the plan empty.
__global__ void __launch_bounds__(kPlanThreads, 1)
    doc_plan_kernel(const DocAttnArgs a, int tile_rows, int window, int sinks, int workers, int* work, uint32_t* status) {
  __shared__ Doc doc_smem[kDocsInSmem];
  __shared__ int first_smem[kDocsInSmem];
  __shared__ int bucket[kBuckets];
  __shared__ int sh[32];
  __shared__ unsigned long long key_tiles;
  __shared__ int heaviest;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x;
  const bool in_smem = a.n_docs <= kDocsInSmem;
  int* first = in_smem ? first_smem : a.first_tile;
  bucket[tid] = 0;
  if (tid == 0) {
    key_tiles = 0;
    heaviest = 1;
  }
  bool bad = false;
  int n_tiles = 0;
  for (int d0 = 0; d0 < a.n_docs; d0 += kPlanThreads) {
    const int d = d0 + tid;
    int mine = 0, total;
    if (d < a.n_docs) {
      const Doc doc(a, d);
      bad |= doc.bad(a);
      mine = bad ? 0 : (doc.n + tile_rows - 1) / tile_rows;
      if (in_smem) doc_smem[d] = doc;
    }
    const int before = block_before(mine, total, sh);
    if (d < a.n_docs) first[d] = n_tiles + before;
    n_tiles += total;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    status[0] = bad ? kStatusBadLength : 0u;
    status[kStatusExtraWord] = 0u;
    *work = 0;
  }
  DocPlan* head = reinterpret_cast<DocPlan*>(a.plan);
  DocTile* tiles = reinterpret_cast<DocTile*>(a.plan + sizeof(DocPlan));
  if (bad || n_tiles == 0) {
    if (tid == 0) {
      head->n_tiles = 0;
      head->group_log = 0;
    }
    return;
  }
  // tile t: its document is the last one that begins at or before it
  auto tile_of = [&](int t) {
    int lo = 0, hi = a.n_docs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= t)
        lo = mid;
      else
        hi = mid - 1;
    }
    Doc d;
    if (in_smem)
      d = doc_smem[lo];
    else
      d = Doc(a, lo);
    const int at = (t - first[lo]) * tile_rows;
    return tile_at(d, at, tile_rows, window, sinks);
  };
  auto bucket_of = [&](const DocTile& t) { return &bucket[kBuckets - 1 - min(t.n_kv, kBuckets - 1)]; };
  unsigned long long sum = 0;
  int most = 0;
  DocTile kept{};  // this thread's first tile
  for (int t = tid; t < n_tiles; t += kPlanThreads) {
    const DocTile tile = tile_of(t);
    if (t == tid) kept = tile;
    atomicAdd(bucket_of(tile), 1);
    sum += tile.n_kv;
    most = max(most, tile.n_kv);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  if ((tid & 31) == 0 && most > 0) {
    atomicAdd(&key_tiles, sum);
    atomicMax(&heaviest, most);
  }
  __syncthreads();
  {
    int total;
    bucket[tid] = block_before(bucket[tid], total, sh);
  }
  __syncthreads();
  for (int t = tid; t < n_tiles; t += kPlanThreads) {
    const DocTile tile = t == tid ? kept : tile_of(t);
    tiles[atomicAdd(bucket_of(tile), 1)] = tile;
  }
  if (tid == 0) {
    head->n_tiles = n_tiles;
    head->group_log = group_log_of(a, key_tiles, heaviest, workers);
  }
}

template <bool PAIR>
cudaError_t launch_tiles(const DocAttnArgs& a, const DevStatusHost& st, int num_sms, cudaStream_t stream) {
  CUtensorMap tq, tk, tv, to;
  if (!make_tmap_bf16_atoms(&tq, a.q, a.N, 192, 1, (uint64_t)a.q_row * 2, (uint64_t)a.q_row * 2, 128, 3) ||
      !make_tmap_bf16_atoms(&tk, a.k, a.cap, 3, 64, 384, (uint64_t)a.cap * 384, PAIR ? kHalf : kKeys, PAIR ? 3 : 1) ||
      !make_tmap_bf16_atoms(&tv, a.v, a.cap, 2, 64, 256, (uint64_t)a.cap * 256, PAIR ? kKeys : kHalf, PAIR ? 1 : 2) ||
      !make_tmap_store_bf16_3d(&to, a.o, 8192, a.N, 1, (uint64_t)a.o_row * 2, (uint64_t)a.o_row * 2))
    return cudaErrorInvalidValue;
  static PerDevice<bool> allowed;
  const cudaError_t attr_err = allow_smem(allowed, document_attn_tc<PAIR>, kSmemBytes);
  if (attr_err != cudaSuccess) return attr_err;
  // no window: one that reaches behind every key (positions minus it stay in range)
  const int window = a.window > 0 && a.window < kNoWindow ? a.window : kNoWindow;
  const int sinks = a.window > 0 ? a.sinks : 0;
  int* work = reinterpret_cast<int*>(st.word) + kWorkCounterWord;
  const long long items = 64 * doc_tiles_at_most(a.N, a.n_docs);
  constexpr int kCtas = PAIR ? 2 : 1;  // that work on an item together
  const int workers = items < num_sms / kCtas ? (int)items : num_sms / kCtas;
  const bool few = !PAIR && a.n_docs <= 32 && doc_tiles_at_most(a.N, a.n_docs) <= kFewTiles;
  if (!few) {
    const cudaError_t e = launch_pdl(doc_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a, kCtas * 128, window,
                                     sinks, workers, work, st.word);
    if (e != cudaSuccess) return e;
  }
  const uint8_t* plan = few ? nullptr : a.plan;
  DevStatus dst{st.word, st.wait_limit_ns};
  const float sl2 = a.scale * 1.4426950408889634f;
  if (PAIR)
    return launch_pdl_cluster2(document_attn_tc<PAIR>, dim3(2 * workers), dim3(kThreads), kSmemBytes, stream, tq, tk,
                               tv, to, sl2, window, sinks, work, plan, a, dst);
  return launch_pdl(document_attn_tc<PAIR>, dim3(workers), dim3(kThreads), kSmemBytes, stream, tq, tk, tv, to, sl2,
                    window, sinks, work, plan, a, dst);
}
}  // namespace

cudaError_t launch_document_attention(const DocAttnArgs& a, const DevStatusHost& st, int num_sms, cudaStream_t stream) {
  const bool pairs = a.N >= kPairRows * (long long)a.n_docs && (a.window == 0 || a.window >= kPairWindow);
  return pairs ? launch_tiles<true>(a, st, num_sms, stream) : launch_tiles<false>(a, st, num_sms, stream);
}

}  // namespace mla
