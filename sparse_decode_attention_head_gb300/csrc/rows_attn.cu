// Attention of packed rows over the paged cache: prompts (causal) and trees of
// drafted tokens (ancestor words).
//
// For query row i of a sequence and a head, with z_t = scale q.k_t over the
// positions t that the row sees,
//   out = sum_t e^{z_t - m} v_t / sum_t e^{z_t - m},   lse = m + log sum_t e^{z_t - m}
// in one pass over t with a running maximum m, tile after tile of 128 tokens.
//
// Work: an item is one KV head of one sequence with up to 256 rows, a row
// being one of the G query heads of a token (so the G heads share every K and
// V byte): two query tiles of 128 rows, or one.  The items of all sequences
// are laid end to end, weighted by the KV tokens they see, and cut into one
// equal run for each block (one block an SM, persistent): many rows give
// whole items, few rows over a long cache split an item's KV range over
// blocks.  With little work a block takes no more than one item (16 us in
// place of 21 for four prompts of at most 200 rows).  A cut item leaves
// (maximum, sum, unnormalised output) for each row, and the merge kernel joins
// the pieces in order with the log-sum-exp identity; blocks never wait on one
// another and nothing is added atomically, so results do not depend on timing.
//
// Block: 12 warps.
//   warps 0-3, 4-7  softmax of query tile 0 and 1, a thread a row
//   warp 8          issues the matrix instructions (one thread)
//   warp 9          loads: Q tiles once an item, K and V tiles into a ring of
//                   five 32 KB slots, one TMA box of 4 KB a page
//   warps 10, 11    clean the V tiles at the edge of what rows see
// S = Q K^T and O += P V run on tcgen05, accumulators in TMEM (S0 S1 O0 O1,
// 128 columns each); P overwrites the first half of its S as packed bf16 and
// is the product's left operand there.  While one tile's softmax runs, the
// tensor core works on the other's.  An item with one query tile instead
// gives every other KV tile to the second softmax group, with a maximum, sum
// and output of its own, joined at the item's end.
//
// The running maximum is let lag: O and the sum are rescaled only when a row
// maximum has grown by more than 2^8, which the fp32 sums and the bf16 of P
// (whose relative precision does not depend on its size) hold with ease.  A row
// is rescaled by its own growth alone, so its bits depend on the tiles and cuts
// it is given, not on the values of other rows.
//
// The weights are rounded to bf16, the operand type of the tensor core, and
// the sum beneath them is of the unrounded ones.  A second product with what
// the rounding leaves (the decode step does that) would add half of the
// kernel's matrix work; the rounding errors of thousands of weights average
// out ahead of the one rounding of the result, which is to bf16 as well: the
// error against 64 bits is 0.0017 of the norm with it and with fp32 weights
// (16384 causal rows; trees at 32K).
//
// Masked places: a weight of zero times a non-finite V would be NaN, so in the
// tiles that hold positions some row of the item does not see, V rows behind
// the item's last position become zero and non-finite values become zero in
// shared memory; rows that do see such a value add it at the end.
//
// What bounds it, measured on one GB300 (1868 TFLOP/s bf16, 6.78 TB/s): with
// two query tiles a KV tile takes 1.55 us, of which the tensor core works two
// thirds; S reads 8 KB of shared memory an instruction and runs slower than O,
// and a group's softmax (0.8 us) and its matrix products do not overlap with
// each other, only with the other group's.  The issuing warp stands between
// them, so what it waits for is looked at once a step (1.49 ms in place of
// 1.56).  16384 causal rows of 32 / 8 heads: 1.43 ms, 1.54 PFLOP/s, for the first
// 50 ms of a run (SM clock 2070 MHz), 1.50 ms, 1.46 PFLOP/s, under the power cap
// of a longer one (1900 MHz); the same in calls and in graph replays.  2048 rows
// behind 30K others: 0.68 ms, 1.56 PFLOP/s, and 0.72 ms, 1.48 PFLOP/s.  With one
// query tile the cache's bytes bound it: 32 drafted tokens for each of 8
// sequences of 32K: 177 us, 6.1 TB/s.
// Slower for the 16384 rows: two issuing warps, one a group (1.94 ms: the groups'
// instructions interleave and both finish late); one barrier for all of a tile's
// weights in place of one for each half (2 %); two threads a row (1.90 ms: 104
// registers do not hold what they need, and they meet once a tile).
//
// Two more instances of the kernel (Kind below).  With shared prefixes the rows of
// a group's sequences are one item's over the prefix, which is so read once, and
// each sequence's own tokens are items of their own; the two parts are joined
// as 32-bit sums.  128 single tokens behind 32K, 32 / 8 heads: 178 us for 616 MB
// (3.5 TB/s): prefix tiles of 256 rows are bound by the tensor core's chain, the
// sequences' own by HBM, and an item's start and end cost 3.4 us.  With selected
// blocks an item's tiles are the pages that some of its rows see, and each row
// finds its own in them: 32768 rows, 16 blocks of 64 each and a window of 512,
// 3.1 ms; a tile of 256 rows takes 1.9 us, of which the tensor core's chain alone
// is 1.54, and the items see five times what a row does.
#include <algorithm>
#include <type_traits>

#include "rows.cuh"
#include "tcgen.cuh"

namespace sa {
namespace {

constexpr int kRows = 128;               // rows of a query tile, tokens of a KV tile
constexpr int kTileBytes = kRows * kD * 2;
constexpr int kSlots = 5;                // K and V tiles in flight: what 227 KB leave beside two query tiles
constexpr int kThreads = 384;
// Registers a thread, out of the 168 the block is launched with: a row's 128
// scores stay in the softmax threads' registers.  The compiler reports 80 bytes
// of spill stores and 184 of loads, in the other warps at their 72 (fewer with
// more there: none at 200 and 104; what that takes from the softmax is not
// measured yet).
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "registers");
// What the kernel attends to, an instance each.
enum Kind {
  kPlain,     // prompts and trees, each sequence over all of its cache
  kShared,    // the same, with the prefix of a group of sequences as an item of its own
  kSparse,    // causal rows over sinks, window and the blocks of their lists
};
template <int KIND>
using Args = std::conditional_t<KIND == kPlain, RowsAttnArgs, RowsMoreArgs>;
// What work weighs: a KV token of an item with one query tile (bound by the
// loads: measured 1.45 us a tile of them) and with two (1.6 us), and an item's
// query load, first tile and epilogue (3.4 us).
// With shared prefixes items with one query tile run beside others with two, which leave them more of the
// memory's rate, and most items are a sequence's few own tokens (128 sequences behind 32K: 179 us at the others' costs,
// 173 at these, both with all own tokens as items).
template <int KIND>
constexpr int kOneCost = KIND == kShared ? 5 : 6;
template <int KIND>
constexpr int kItemCost = KIND == kShared ? 2400 : 2000;
constexpr int kTwoCost = 7;
constexpr float kLag = 8.f;              // log2 of the growth of a row maximum that makes a rescale

enum { kDescValid = 1, kDescFirst = 2, kDescLast = 4, kDescDual = 8 };

// A piece of a block's run: KV tiles [k0, k1) of one item.  The loading warp
// walks the run and hands the pieces to the other roles through a ring.
struct Piece {
  int b, kvh, i;
  int k0, k1, nt;     // of the item's nt tiles; k0 < 0: the run is over
  int row0;           // first packed row of the item
  int tokens;         // of the item
  int end, edge;      // item_end, item_edge
  int a;              // tokens of the sequence ahead of its rows
  int first;          // the item's first row in the sequence
  bool dual;          // one query tile, KV tiles taken in turn by both softmax groups
};
struct MorePiece : Piece {
  int to;             // Part: where the result goes
  int u;              // kSparse: the item,
  int out;            // and how many halves of pages, ahead of its window's, are not in its list
  long long pt;       // entry of the page table with the item's position 0
};
template <int KIND>
using PieceOf = std::conditional_t<KIND == kPlain, Piece, MorePiece>;
// The entry of the page table with an item's position 0.
__device__ __forceinline__ long long table_at(const RowsAttnArgs& A, const Piece& p) { return (long long)p.b * A.mpp; }
__device__ __forceinline__ long long table_at(const RowsAttnArgs&, const MorePiece& p) { return p.pt; }

constexpr int kPieces = 4;
constexpr int kPieceReaders = 11;        // warps: softmax, matrix instructions, edge

template <int KIND>
struct alignas(16) Ctl {
  PieceOf<KIND> piece[kPieces];
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t full[kSlots], empty[kSlots];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2][2], o_done[2];
  uint64_t edge_go[kSlots], clean[kSlots];   // a V tile at the edge: its load is under way, it is clean
  uint64_t ml_full, ml_free;
  uint64_t drain;
  uint32_t tmem;
  int abort;
  int4 range[2];             // (sequence, KV head, item, KV tile) at which this block begins and ends
  uint32_t bad[16];          // pages outside the pool, a bit each, of the last tiles loaded
  int poison[4];             // 1 + the piece that met a non-finite V at its edge
  float2 ml[kRows];          // (maximum, sum) of the second softmax group
};

// kSparse: the pages of the last tiles loaded, ascending, -1 behind an item's
// last.  K and V slots let the loads run at most four tiles ahead of the softmax.
constexpr int kPageDepth = 8;
struct alignas(16) PageRing {
  int page[kPageDepth][8];
};
template <int KIND>
constexpr size_t kSmemBytes = 1024 + (2 + kSlots) * kTileBytes + sizeof(Ctl<KIND>) + (KIND == kSparse ? sizeof(PageRing) : 0);
static_assert(kSmemBytes<kSparse> <= 227 * 1024, "shared memory");
constexpr uint32_t kCut = 256;           // beside a tile's bad pages: some row's view begins or ends inside 8 tokens

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// Waits with a limit of kWaitNs; a wait that runs out, here or elsewhere in the
// block, ends the block's work.
constexpr unsigned long long kWaitNs = 2000000000ull;
template <typename C>
[[nodiscard]] __device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, C* c, int* status) {
  unsigned long long t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 63u) != 0) continue;
    if (*(volatile int*)&c->abort) return false;
    const unsigned long long t = now_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > kWaitNs) {
      set_status(status, SA_ERR_TIMEOUT);
      *(volatile int*)&c->abort = 1;
      return false;
    }
  }
  return true;
}

// For what is in flight when a block ends: not cut short by an abort.
__device__ __forceinline__ void wait_out(uint64_t* bar, uint32_t parity, int* status) {
  const unsigned long long t0 = now_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (now_ns() - t0 > kWaitNs) {
      set_status(status, SA_ERR_TIMEOUT);
      return;
    }
  }
}

// wait_bar by a whole warp: all lanes see the same answer.
template <typename C>
[[nodiscard]] __device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, C* c, int* status) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, c, status));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// A place in the ring of K and V tiles and the parity of its use.
struct Ring {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void advance(int n) {
    slot += n;
    if (slot >= kSlots) {
      slot -= kSlots;
      parity ^= 1;
    }
  }
};

// ---------------------------------------------------------------- the items

// What a sequence's rows are over: all they see, or one of two parts that
// rows_join_kernel puts together.
enum Part { kAll, kPrefix, kOwn };

struct Seq : RowSeq {
  int items;      // of one KV head
  int T;          // tokens of an item
  int to;         // Part
  long long pt;   // entry of the page table with position 0
};

// A sequence whose own tokens the joining kernel attends: few of them, for few
// rows.  Each would take an item of the attention kernel, whose start and end
// cost more than two tiles.
constexpr int kJoinTokens = 160, kJoinRows = 4;
__device__ __forceinline__ bool own_in_join(const RowsMoreArgs& A, const Seq& s) {
  return A.join_own && s.to == kOwn && s.n <= kJoinRows && s.L <= kJoinTokens;
}

// Sequence v.  With prefixes of groups (kShared) there are two for each of the
// batch: 2 b, the rows of the group that b leads over its prefix (all of them
// see all of it), and 2 b + 1, b's rows over what is behind the prefix; both
// count positions from their own first token.
template <int KIND>
__device__ __forceinline__ int sequences(const RowsAttnArgs& A) {
  return KIND == kShared ? 2 * A.B : A.B;
}
template <int KIND>
__device__ __forceinline__ Seq load_seq(const Args<KIND>& A, int v, int* status) {
  const int b = KIND == kShared ? v >> 1 : v;
  Seq s;
  s.T = 2 * A.tpt;
  s.to = kAll;
  s.pt = (long long)b * A.mpp;
  if constexpr (KIND == kShared) {
    if ((v & 1) == 0) {
      static_cast<RowSeq&>(s) = shared_rows(A.row_offsets, A.members, A.prefix_lens, A.B, b, A.n_rows, A.mpp);
      s.to = kPrefix;
      s.items = (s.n + s.T - 1) / s.T;
      return s;
    }
  }
  static_cast<RowSeq&>(s) = row_seq(A.row_offsets, A.seq_lens, b, A.n_rows, A.mpp, status);
  s.items = (s.n + s.T - 1) / s.T;
  if constexpr (KIND == kShared) {
    const int x = shared_prefix(A.prefix_lens, b, s, A.mpp, status);
    if (x > 0) {
      s.to = kOwn;
      s.pt += x / kP;
      s.a -= x;
      s.L -= x;
    }
    if (own_in_join(A, s)) s.items = 0;
  }
  if (A.tree != nullptr && s.n > kMaxTree) {
    if (status != nullptr) set_status(status, SA_ERR_CAPACITY);
    s.items = 0;
  }
  return s;
}
// The first position that no row of item i sees.
__device__ __forceinline__ int item_end(const RowsAttnArgs& A, const Seq& s, int i) {
  if (A.tree != nullptr) return s.L;
  return max(0, min(s.L, s.a + min(s.n, (i + 1) * s.T)));
}
// The first position that some row of item i does not see (positions of a
// tree's drafts included); at most item_end, behind which nobody sees any.
__device__ __forceinline__ int item_edge(const RowsAttnArgs& A, const Seq& s, int i) {
  return max(0, min(A.tree != nullptr ? s.a : s.a + i * s.T + 1, item_end(A, s, i)));
}
__device__ __forceinline__ int tiles_of(int end) { return (end + kRows - 1) / kRows; }

// Weight of a KV head's first k items, in closed form: KV tokens seen, times
// what a tile of them takes with one query tile or with two, and a fixed cost
// each.  All items but a sequence's last have two query tiles.
template <int KIND>
__device__ __forceinline__ long long weight_before(const RowsAttnArgs& A, const Seq& s, int k) {
  if (k == 0) return 0;
  const int full = min(k, s.items - 1);
  const bool flat = A.tree != nullptr || s.to == kPrefix;     // all rows see about the same
  const long long before = max(flat ? s.L : s.a, 0);
  long long w = (before * full + (flat ? 0 : (long long)s.T * full * (full + 1) / 2)) * kTwoCost +
                (long long)k * kItemCost<KIND>;
  if (k == s.items) {
    const int tokens = s.n - full * s.T;
    w += (before + (flat ? 0 : s.n)) * (tokens <= A.tpt ? kOneCost<KIND> : kTwoCost);
  }
  return w;
}

// One warp: the total weight of all items.  `s` and `mine` are the lane's own
// sequence, of the first 32, and its weight.
template <int KIND>
__device__ __forceinline__ long long total_weight(const Args<KIND>& A, int* status, Seq& s, long long& mine) {
  const int lane = threadIdx.x & 31;
  long long w = 0;
  mine = 0;
  s = Seq{};
  for (int b = lane; b < sequences<KIND>(A); b += 32) {
    const Seq x = load_seq<KIND>(A, b, status);
    const long long m = weight_before<KIND>(A, x, x.items) * A.Hk;
    w += m;
    if (b < 32) {
      s = x;
      mine = m;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  return w;
}

// The KV head, item and KV tile at weight `rem` of a sequence, all of whose heads weigh `mine`.
template <int KIND, typename T>
__device__ __forceinline__ void locate_in(const RowsAttnArgs& A, T rem, const Seq& s, T mine, int4& r) {
  const T each = mine / (T)A.Hk;
  r.y = (int)(rem / each);
  rem -= each * r.y;
  int lo = 0, hi = s.items;     // the item: weight_before(lo) <= rem < weight_before(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((T)weight_before<KIND>(A, s, mid) <= rem) lo = mid; else hi = mid;
  }
  const T w0 = (T)weight_before<KIND>(A, s, lo), w1 = (T)weight_before<KIND>(A, s, lo + 1);
  r.z = lo;
  r.w = (int)((unsigned long long)(rem - w0) * tiles_of(item_end(A, s, lo)) / (w1 - w0));
}

// One warp: the item and KV tile at weight w (the end: a sequence behind the last).
template <int KIND, typename T>
__device__ __forceinline__ int4 locate(const Args<KIND>& A, T w, Seq s, T mine) {
  const int lane = threadIdx.x & 31, n_seq = sequences<KIND>(A);
  T before = 0;
  for (int b0 = 0; b0 < n_seq; b0 += 32) {
    const int b = b0 + lane;
    if (b0 > 0) {
      mine = 0;
      if (b < n_seq) {
        s = load_seq<KIND>(A, b, nullptr);
        mine = (T)weight_before<KIND>(A, s, s.items) * A.Hk;
      }
    }
    T upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, w < before + upto);
    if (hit == 0) {
      before += __shfl_sync(0xffffffffu, upto, 31);
      continue;
    }
    const int src = __ffs(hit) - 1;
    int4 r = make_int4(b, 0, 0, 0);
    if (lane == src) locate_in<KIND, T>(A, w - (before + upto - mine), s, mine, r);
    r.x = __shfl_sync(0xffffffffu, r.x, src);
    r.y = __shfl_sync(0xffffffffu, r.y, src);
    r.z = __shfl_sync(0xffffffffu, r.z, src);
    r.w = __shfl_sync(0xffffffffu, r.w, src);
    return r;
  }
  return make_int4(n_seq, 0, 0, 0);
}

// Little work: every block takes one item or an equal part of one, of two KV
// tiles or four, and none takes two.  `s` as above (at most 32 sequences).  Answers false
// where the blocks do not suffice for that.
__device__ __forceinline__ int runs_of(const RowsAttnArgs& A, const Seq& s, int i, int tiles) {
  return max(1, (tiles_of(item_end(A, s, i)) + tiles - 1) / tiles);
}
template <int KIND>
__device__ __forceinline__ bool locate_small(const RowsAttnArgs& A, int run, int blocks, const Seq& s, int4& r) {
  const int lane = threadIdx.x & 31;
  if (sequences<KIND>(A) > 32) return false;
  auto sum = [](int x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  };
  const int some = s.items > blocks ? blocks + 1 : s.items;
  if ((long long)sum(some) * A.Hk > blocks) return false;
  int tiles = 2, mine;
  while (true) {
    mine = 0;
    for (int i = 0; i < s.items; ++i) mine += min(runs_of(A, s, i, tiles), blocks + 1);
    mine = min(mine, blocks + 1) * A.Hk;
    if (sum(mine) <= blocks) break;
    if (tiles == 4) return false;
    tiles = 4;
  }
  r = make_int4(sequences<KIND>(A), 0, 0, 0);
  const int upto = warp_incl_scan(mine);
  const unsigned hit = __ballot_sync(0xffffffffu, run < upto);
  if (hit == 0) return true;
  const int src = __ffs(hit) - 1;
  if (lane == src) {
    int rem = run - (upto - mine);
    const int each = mine / A.Hk;
    r = make_int4(lane, rem / each, 0, 0);
    rem -= each * r.y;
    int n = runs_of(A, s, 0, tiles);
    while (rem >= n) {
      rem -= n;
      n = runs_of(A, s, ++r.z, tiles);
    }
    r.w = rem * tiles_of(item_end(A, s, r.z)) / n;
  }
  r.x = __shfl_sync(0xffffffffu, r.x, src);
  r.y = __shfl_sync(0xffffffffu, r.y, src);
  r.z = __shfl_sync(0xffffffffu, r.z, src);
  r.w = __shfl_sync(0xffffffffu, r.w, src);
  return true;
}

// Many sequences, by the whole block: the weight ahead of each goes to `ahead`
// [sequences + 1] in shared memory, and warps 0 and 1 look up where the block's
// run begins and ends.  (Warp by warp, 32 sequences a round of loads: 1000
// sequences in groups of 50 took 183 us in place of 119.)
constexpr int kMaxAhead = kSlots * kTileBytes / (int)sizeof(long long) - 1;
template <int KIND>
__device__ __forceinline__ int4 locate_many(const Args<KIND>& A, long long* ahead, long long* s_sum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = sequences<KIND>(A);
  for (int v = tid; v < n; v += kThreads) {
    const Seq s = load_seq<KIND>(A, v, blockIdx.x == 0 ? A.status : nullptr);
    ahead[v] = weight_before<KIND>(A, s, s.items) * A.Hk;
  }
  __syncthreads();
  const int each = (n + kThreads - 1) / kThreads, v0 = min(tid * each, n), v1 = min(v0 + each, n);
  long long sum = 0;
  for (int v = v0; v < v1; ++v) sum += ahead[v];
  long long upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) s_sum[warp] = upto;
  __syncthreads();
  long long at = upto - sum;
  for (int w = 0; w < warp; ++w) at += s_sum[w];
  for (int v = v0; v < v1; ++v) {
    const long long x = ahead[v];
    ahead[v] = at;
    at += x;
  }
  if (tid == kThreads - 1) ahead[n] = at;      // the last thread's share ends at n
  __syncthreads();
  int4 r = make_int4(n, 0, 0, 0);
  if (warp < 2) {
    const long long w = ahead[n] * (blockIdx.x + warp) / gridDim.x;
    if (w < ahead[n]) {
      int lo = 0, hi = n;                      // ahead[lo] <= w < ahead[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ahead[mid] <= w) lo = mid; else hi = mid;
      }
      const Seq s = load_seq<KIND>(A, lo, nullptr);
      r.x = lo;
      locate_in<KIND, long long>(A, w - ahead[lo], s, ahead[lo + 1] - ahead[lo], r);
    }
  }
  return r;
}

// One thread walks a block's run, piece by piece.
template <int KIND>
struct Walk {
  const Args<KIND>& A;
  int b, kvh, i, kt;
  int4 end;
  bool done;
  Seq s;
  __device__ Walk(const Args<KIND>& a, const Ctl<KIND>* c) : A(a) {
    const int4 r = c->range[0];
    b = r.x; kvh = r.y; i = r.z; kt = r.w;
    end = c->range[1];
    done = b >= sequences<KIND>(A);
    if (!done) s = load_seq<KIND>(A, b, nullptr);
  }
  // The next sequence with items, looked for by a whole warp, 32 at once: every
  // other one may be the prefix of a sequence that leads no group.
  __device__ __forceinline__ void next_shared() {
    const int lane = threadIdx.x & 31;
    for (++b; b < sequences<KIND>(A); b += 32) {
      Seq x{};
      if (b + lane < sequences<KIND>(A)) x = load_seq<KIND>(A, b + lane, nullptr);
      const unsigned hit = __ballot_sync(0xffffffffu, x.items > 0);
      if (hit == 0) continue;
      const int src = __ffs(hit) - 1;
      b += src;
      s.row0 = __shfl_sync(0xffffffffu, x.row0, src);
      s.n = __shfl_sync(0xffffffffu, x.n, src);
      s.L = __shfl_sync(0xffffffffu, x.L, src);
      s.a = __shfl_sync(0xffffffffu, x.a, src);
      s.items = __shfl_sync(0xffffffffu, x.items, src);
      s.to = __shfl_sync(0xffffffffu, x.to, src);
      s.pt = __shfl_sync(0xffffffffu, x.pt, src);
      return;
    }
    done = true;
  }
  __device__ bool next(PieceOf<KIND>& p) {
    while (!done) {
      const bool at_end = b == end.x && kvh == end.y && i == end.z;
      p.b = b; p.kvh = kvh; p.i = i;
      p.end = item_end(A, s, i);
      p.edge = item_edge(A, s, i);
      p.nt = tiles_of(p.end);
      p.k0 = kt;
      p.k1 = at_end ? end.w : p.nt;
      p.a = s.a;
      if constexpr (KIND != kPlain) {
        p.to = s.to;
        p.pt = s.pt;
      }
      p.first = i * s.T;
      p.row0 = s.row0 + i * s.T;
      p.tokens = min(s.T, s.n - i * s.T);
      p.dual = p.tokens <= A.tpt;
      const bool some = p.k0 < p.k1 || (p.nt == 0 && !at_end);
      kt = 0;
      if (at_end) {
        done = true;
      } else if (++i == s.items) {
        i = 0;
        if (++kvh == A.Hk) {
          kvh = 0;
          if (KIND == kShared) {
            next_shared();
          } else {
            do {
              if (++b >= sequences<KIND>(A)) { done = true; break; }
              s = load_seq<KIND>(A, b, nullptr);
            } while (s.items == 0);
          }
        }
      }
      if (some) return true;
    }
    return false;
  }
};

// With selected blocks: the items lie one behind the other.  Where they are
// many, a block takes whole ones, the next when it is done with the last: the
// items under way at a time are neighbours, whose pages L2 holds.  Else each
// block has its share of their weight, and cuts items.
constexpr int kWholeItems = 8;       // a block, from which they are taken whole (5.7 a block: 426 us cut, 443 whole)
__device__ __forceinline__ bool whole_items(const RowsMoreArgs& A) {
  return __ldg(A.ticket + 1) >= kWholeItems * (int)gridDim.x;
}
template <>
struct Walk<kSparse> {
  const RowsMoreArgs& A;
  int u, kt, ahead;
  int4 end;
  SparseItem it;
  bool whole;
  __device__ Walk(const RowsMoreArgs& a, const Ctl<kSparse>* c) : A(a) {
    whole = whole_items(A);
    if (whole) {
      u = blockIdx.x;
      kt = 0;
      end = make_int4(__ldg(A.ticket + 1), 0, 0, 0);
      ahead = take();
    } else {
      u = c->range[0].x;
      kt = c->range[0].y;
      end = c->range[1];
    }
    load();
  }
  __device__ int take() {      // a whole warp
    int x = 0;
    if ((threadIdx.x & 31) == 0) x = (int)gridDim.x + atomicAdd(A.ticket, 1);
    return __shfl_sync(0xffffffffu, x, 0);
  }
  __device__ void load() {
    if (u < A.n_items) {
      const int4* x = reinterpret_cast<const int4*>(A.items + u);
      const int4 a = __ldg(x), b = __ldg(x + 1);
      it = SparseItem{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    }
  }
  __device__ bool next(MorePiece& p) {
    while (u < end.x || (u == end.x && kt < end.y)) {
      const bool at_end = u == end.x;
      p.b = it.b; p.kvh = it.kvh; p.i = it.i;
      p.nt = (it.pages + 7) / 8;
      p.k0 = kt;
      p.k1 = at_end ? end.y : p.nt;
      p.row0 = it.row0;
      p.tokens = it.tokens;
      p.end = it.end;
      p.edge = (p.nt - 1) * kRows + 1;           // the last tile alone holds positions that no row sees
      p.a = it.pos0;
      p.first = 0;
      p.to = kAll;
      p.pt = (long long)it.b * A.mpp;
      p.u = u;
      p.out = 2 * ((it.end + kP - 1) / kP - it.pages);
      p.dual = it.tokens <= A.tpt;
      const bool some = p.k0 < p.k1 || (p.nt == 0 && p.tokens > 0 && !at_end);
      kt = 0;
      if (at_end) {
        end.y = 0;
      } else {
        u = whole ? ahead : u + 1;
        if (whole && u < end.x) ahead = take();
        load();
      }
      if (some) return true;
    }
    return false;
  }
};

// One warp: the item and tile at weight w of all items (w = total: behind the
// last that there is; there is room for one more a sequence and KV head, and the
// last block would walk over those).
__device__ __forceinline__ int4 locate_item(const RowsMoreArgs& A, long long w) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = __ldg(A.ticket + 1);      // before[lo] <= w < before[hi]
  if (w >= __ldg(A.before + hi)) return make_int4(hi, 0, 0, 0);
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + step * (lane + 1);
    const int n = __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(A.before + at) <= w));
    hi = min(hi, lo + step * (n + 1));
    lo += step * n;
  }
  const long long w0 = __ldg(A.before + lo), w1 = __ldg(A.before + lo + 1);
  return make_int4(lo, (int)((w - w0) * ((A.items[lo].pages + 7) / 8) / (w1 - w0)), 0, 0);
}

// ---------------------------------------------------------------- what a row sees of selected blocks

// The pages of an item's bitmap, eight at a time, by a whole warp, which looks up
// those of four tiles at once.
template <int KIND>
struct PageWalk {
  __device__ __forceinline__ PageWalk(const RowsAttnArgs&, const Piece&, int) {}
};
template <>
struct PageWalk<kSparse> {
  const uint32_t* bits;
  int words, base;       // base: the first of the 32 words that the lanes hold
  uint32_t mine;
  int upto, total;       // pages up to and with the lane's word, of all 32
  int given;             // of these
  int batch, place;      // a page a lane; the next of them
  __device__ __forceinline__ void load() {
    const int w = base + (threadIdx.x & 31);
    mine = w < words ? __ldg(bits + w) : 0u;
    upto = warp_incl_scan(__popc(mine));
    total = __shfl_sync(0xffffffffu, upto, 31);
    given = 0;
  }
  // ahead: pages to pass over
  __device__ __forceinline__ PageWalk(const RowsMoreArgs& A, const MorePiece& p, int ahead)
      : bits(A.pages + (size_t)p.u * A.words), words((p.end + 32 * kP - 1) / (32 * kP)), base(0), place(32) {
    load();
    while (ahead >= total && base + 32 < words) {
      ahead -= total;
      base += 32;
      load();
    }
    given = min(ahead, total);
  }
  __device__ __forceinline__ void refill() {
    const int lane = threadIdx.x & 31;
    batch = -1;
    for (int got = 0;;) {
      // the word with page `want`: behind all that hold fewer
      const int want = given + lane - got;
      int owner = 0;
#pragma unroll
      for (int step = 16; step > 0; step >>= 1)
        if (__shfl_sync(0xffffffffu, upto, owner + step - 1) <= want) owner += step;
      uint32_t x = __shfl_sync(0xffffffffu, mine, owner);
      int k = want - (__shfl_sync(0xffffffffu, upto, owner) - __popc(x));     // of the word's
      if (lane >= got && want < total) {
        batch = (base + owner) * 32;
#pragma unroll
        for (int half = 16; half > 0; half >>= 1) {
          const int n = __popc(x & ((1u << half) - 1u));
          if (k >= n) {
            k -= n;
            x >>= half;
            batch += half;
          }
        }
      }
      const int take = min(32 - got, total - given);
      got += take;
      given += take;
      if (got == 32 || base + 32 >= words) break;
      base += 32;
      load();
    }
    place = 0;
  }
  // Lane j < 8: the j-th of the next eight, -1 where there are no more.
  __device__ __forceinline__ int next() {
    if (place == 32) refill();
    const int page = __shfl_sync(0xffffffffu, batch, place + (threadIdx.x & 7));
    place += 8;
    return (threadIdx.x & 31) < 8 ? page : -1;
  }
};

// A row's blocks as places in the item's list of pages, in halves of pages,
// ascending (sparse_items_kernel writes them), along ascending tiles of 16
// halves.  Four at a time, the next four on their way.
struct RankWalk {
  const int4* list;
  int groups, at;          // of four; the next to load
  int4 now, next;
  int used;                // of `now`
  uint32_t acc;            // halves from the last tile's first on
  __device__ __forceinline__ int4 get(int j) const {
    constexpr int kNone = 0x7fffffff;
    return j < groups ? __ldg(list + j) : make_int4(kNone, kNone, kNone, kNone);
  }
  // blocks of `len` halves, those ahead of tile t0 passed over
  __device__ __forceinline__ void start(const int* l, int n_groups, int len, int t0) {
    list = reinterpret_cast<const int4*>(l);
    groups = n_groups;
    int lo = 0, hi = groups;          // the first group whose last block reaches into the tile
    if (t0 > 0) {
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(l + 4 * mid + 3) <= 16 * t0 - len) lo = mid + 1; else hi = mid;
      }
    }
    now = get(lo);
    next = get(lo + 1);
    at = lo + 2;
    used = 0;
    acc = 0;
  }
  // A bit for each half of tile t that the row's blocks hold; `by` tiles on from the last one asked for.
  __device__ __forceinline__ uint32_t mask(int t, int by, int len) {
    acc = by == 1 ? acc >> 16 : 0;    // a block is at most 8 halves: it reaches into one more tile
    while (now.x < 16 * t + 16) {
      const int sh = now.x - 16 * t;
      const uint32_t ones = (1u << len) - 1u;
      if (sh > -8) acc |= sh >= 0 ? ones << sh : ones >> -sh;
      now.x = now.y;
      now.y = now.z;
      now.z = now.w;
      if (++used == 4) {
        now = next;
        next = get(at++);
        used = 0;
      }
    }
    return acc & 0xffffu;
  }
};
// Bits [a, b) of 16, from `base` on.
__device__ __forceinline__ uint32_t bits16(int a, int b, int base) {
  const uint32_t lo = (1u << min(max(a - base, 0), 16)) - 1u, hi = (1u << min(max(b - base, 0), 16)) - 1u;
  return hi & ~lo;
}

// The sums of one row over one piece from its definition, by a whole warp:
// dims 4 lane on.  Taken where the product of a tile with V is not finite: a
// weight of zero times such a value is NaN for rows that do not see it.
struct SeenRow {
  size_t row;           // packed row and head
  int kvh, pos;
  float M;
};
__device__ __noinline__ float4 sums_of_row(const RowsMoreArgs& A, const MorePiece& p, SeenRow s) {
  const int lane = threadIdx.x & 31;
  const int shift = A.bs_shift[s.kvh];
  const int n = min(max(__ldg(A.sel_cnt + s.row), 0), A.kcap);
  const int* list = A.sel_idx + s.row * A.kcap;
  const uint32_t* bits = A.pages + (size_t)p.u * A.words;
  const int words = (p.end + 32 * kP - 1) / (32 * kP);
  const int half = lane >> 4, tk = lane & 15;      // a token's dims 64 half on
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  int rank = 0;
  for (int w = 0; w < words && rank < 8 * p.k1; ++w) {
    uint32_t x = __ldg(bits + w);
    if (rank + __popc(x) <= 8 * p.k0) {
      rank += __popc(x);
      continue;
    }
    for (; x != 0; x &= x - 1, ++rank) {
      if (rank < 8 * p.k0 || rank >= 8 * p.k1) continue;
      const int page = w * 32 + __ffs(x) - 1;
      const int phys = __ldg(A.page_table + p.pt + page);
      if (phys < 0 || phys >= A.num_pages) continue;
      const int t = page * kP + tk, e = t >> shift;
      int lo = 0, hi = n;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(list + mid) < e) lo = mid + 1; else hi = mid;
      }
      const bool seen = t <= s.pos && (t < A.S || t > s.pos - A.W || (lo < n && __ldg(list + lo) == e));
      const size_t at = (((size_t)phys * A.Hk + s.kvh) * kP + tk) * kD;
      float z = 0.f;
      if (seen)
        for (int d = 64 * half; d < 64 * half + 64; ++d)
          z = fmaf(__bfloat162float(A.q[s.row * kD + d]), __bfloat162float(A.k_pool[at + d]), z);
      z += __shfl_xor_sync(0xffffffffu, z, 16);
      const float weight = __bfloat162float(__float2bfloat16_rn(ex2(fmaf(z, A.scale_log2, -s.M))));
      unsigned who = __ballot_sync(0xffffffffu, seen) & 0xffffu;
      for (; who != 0; who &= who - 1) {
        const int j = __ffs(who) - 1;
        const float f = __shfl_sync(0xffffffffu, weight, j);
        const uint2 q = *reinterpret_cast<const uint2*>(
            A.v_pool + (((size_t)phys * A.Hk + s.kvh) * kP + j) * kD + 4 * lane);
        auto add = [f](float& o, float v) { o = isfinite(v) ? fmaf(f, v, o) : o + v; };
        add(acc.x, bf16_lo(q.x));
        add(acc.y, bf16_hi(q.x));
        add(acc.z, bf16_lo(q.y));
        add(acc.w, bf16_hi(q.y));
      }
    }
  }
  return acc;
}

// ---------------------------------------------------------------- epilogue

__device__ __forceinline__ bool bf16_pair_nonfinite(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// The non-finite values of V at the edge positions [t0, t1) that a row sees
// are added to its stored result (the product with them was taken as zero).
// Rare, and kept out of the kernel's registers.
struct EdgeRow {
  const int* pages;             // the sequence's row of the page table
  unsigned long long word;
  int t0, t1, lim, a;           // sees t < lim, and bit t - a of word
};
__device__ __noinline__ void add_poison(const RowsAttnArgs& A, EdgeRow e, int kvh, __nv_bfloat16* out, float* part,
                                        int step) {   // part: dims in fours, `step` values apart
  for (int t = e.t0; t < e.t1; ++t) {
    const int bit = t - e.a;
    if (!(t < e.lim || (bit >= 0 && bit < 64 && ((e.word >> bit) & 1ull)))) continue;
    const int phys = __ldg(e.pages + t / kP);
    if (phys < 0 || phys >= A.num_pages) continue;
    const __nv_bfloat16* v = A.v_pool + (((size_t)phys * A.Hk + kvh) * kP + t % kP) * kD;
    for (int d = 0; d < kD; ++d) {
      const float x = __bfloat162float(v[d]);
      if (isfinite(x)) continue;
      if (out != nullptr) out[d] = __float2bfloat16_rn(__bfloat162float(out[d]) + x);
      else part[(d >> 2) * step + (d & 3)] += x;
    }
  }
}

// Four neighbouring lanes exchange 16-byte pieces: lane l's piece j for lane
// j's piece l, so that each row's pieces lie in four lanes.
__device__ __forceinline__ void swap_rows4(uint32_t (&x)[4][4], int lane) {
#pragma unroll
  for (int step = 1; step <= 2; step <<= 1) {
    const bool upper = lane & step;
#pragma unroll
    for (int a0 = 0; a0 < 4; ++a0) {
      if (a0 & step) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? x[a0][j] : x[a0 + step][j], step);
        if (upper) x[a0][j] = got; else x[a0 + step][j] = got;
      }
    }
  }
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// ---------------------------------------------------------------- the kernel

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1)
rows_attention_kernel(Args<KIND> A, const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = smem;                                  // two tiles: [half of the dims][128 rows][64]
  uint8_t* s_kv = smem + 2 * kTileBytes;                // kSlots tiles: [16 groups of 8 tokens][half][8][64]
  auto* c = reinterpret_cast<Ctl<KIND>*>(s_kv + kSlots * kTileBytes);
  PageRing* ring = reinterpret_cast<PageRing*>(c + 1);  // kSparse
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&c->full[i], 1);
      mbar_init(&c->empty[i], 1);
      mbar_init(&c->edge_go[i], 1);
      mbar_init(&c->clean[i], 2);
    }
    mbar_init(&c->q_full, 1);
    mbar_init(&c->q_empty, 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&c->s_full[h], 1);
      mbar_init(&c->p_full[h][0], kRows);
      mbar_init(&c->p_full[h][1], kRows);
      mbar_init(&c->o_done[h], 1);
    }
    mbar_init(&c->ml_full, kRows);
    mbar_init(&c->ml_free, kRows);
    mbar_init(&c->drain, 1);
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&c->piece_full[i], 1);
      mbar_init(&c->piece_empty[i], kPieceReaders);
    }
    c->abort = 0;
    for (int i = 0; i < 4; ++i) c->poison[i] = 0;
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(&c->tmem, 512);
  if (tid == 288) {
    prefetch_map(&tmQ);
    prefetch_map(&tmK);
    prefetch_map(&tmV);
  }
  pdl_wait();
  pdl_trigger();
  if constexpr (KIND == kSparse) {
    if (warp < 2 && !whole_items(A)) {
      const int4 r = locate_item(A, __ldg(A.before + A.n_items) * (blockIdx.x + warp) / gridDim.x);
      if (lane == 0) c->range[warp] = r;
    }
  } else if (KIND == kShared && sequences<KIND>(A) > 32 && sequences<KIND>(A) <= kMaxAhead) {
    const int4 r = locate_many<KIND>(A, reinterpret_cast<long long*>(s_kv), reinterpret_cast<long long*>(c->ml));
    if (warp < 2 && lane == 0) c->range[warp] = r;
    fence_proxy_async_smem();      // copies come to where the weights were
  } else if (warp < 2) {   // where this block's run begins (warp 0) and ends (warp 1)
    Seq s;
    long long mine;
    const long long W = total_weight<KIND>(A, blockIdx.x == 0 && warp == 0 ? A.status : nullptr, s, mine);
    int4 r;
    if (locate_small<KIND>(A, blockIdx.x + warp, gridDim.x, s, r)) {
    } else if (W < (1ll << 32) / kRowsMaxCtas) {     // in 32 bits, whose divisions are short
      r = locate<KIND, uint32_t>(A, (uint32_t)W * (blockIdx.x + warp) / gridDim.x, s, (uint32_t)mine);
    } else {
      r = locate<KIND, long long>(A, W * (blockIdx.x + warp) / gridDim.x, s, mine);
    }
    if (lane == 0) c->range[warp] = r;
  }
  if (tid < 2) A.desc[blockIdx.x * 2 + tid] = make_int4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;

  if (warp < 8) {
    regs_inc<kSoftmaxRegs>();
    // ------------------------------------------------------------ softmax: a thread a row
    const int h = warp >> 2;
    const int r = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // 32 lanes a warp, in the address' upper half
    const uint32_t tS = tmem + lanes + h * 128, tO = tmem + lanes + 256 + h * 128;
    const int t_row = r / A.G, g = r - t_row * A.G;
    uint32_t steps_done = 0, items_done = 0, duals = 0, tiles = 0;
    bool ok = true;
    for (int piece = 0;; ++piece) {
      if (!(ok = wait_warp(&c->piece_full[piece % kPieces], (piece / kPieces) & 1, c, A.status))) break;
      const PieceOf<KIND>& p = c->piece[piece % kPieces];
      const int k0 = p.k0, ntp = p.k1 - k0, edge = p.edge;
      const bool dual = p.dual;
      if (k0 < 0) break;
      const int N = dual ? ntp : 2 * ntp;
      const int tok = t_row + (dual || h == 0 ? 0 : A.tpt);
      const bool valid = t_row < A.tpt && tok < p.tokens;
      // what the row sees: positions below lim, and bit j of its word for position p.a + j
      int lim = 0;
      unsigned long long word = 0;
      if (KIND == kSparse) {
        lim = valid ? max(p.a + tok + 1, 0) : 0;      // and of those what its mask has
      } else if (valid) {
        if (A.tree != nullptr) {
          lim = p.a;
          word = __ldg(A.tree + p.row0 + tok);
        } else {
          lim = p.a + p.first + tok + 1;
        }
      }
      const float lag = valid ? kLag : INFINITY;   // a lane without a row never grows
      float m = -INFINITY, l = 0.f;
      RankWalk walk;
      int sink = 0, win0 = 0, win1 = 0, len = 0;     // kSparse: whole halves of sinks and window, of a block
      if constexpr (KIND == kSparse) {
        len = (1 << A.bs_shift[p.kvh]) / 8;
        const size_t row = (size_t)(p.row0 + tok) * A.Hq + p.kvh * A.G + g;
        walk.start(A.ranks + (valid ? row * A.rank_stride : 0), valid && lim > 0 ? A.rank_stride / 4 : 0, len, k0);
        sink = min(A.S, min(lim, p.end)) >> 3;
        win0 = ((max(lim - A.W, 0) + 7) >> 3) - p.out;
        win1 = (min(lim, p.end) >> 3) - p.out;
      }
      for (int s = h; s < N; s += 2) {
        const int t = dual ? s : s >> 1;
        const int kt = k0 + t;
        uint32_t mask = 0;
        if constexpr (KIND == kSparse) {     // while the product is under way
          mask = walk.mask(kt, dual ? 2 : 1, len) | bits16(0, sink, 16 * kt) | bits16(win0, win1, 16 * kt);
          if (lim <= 0) mask = 0;
        }
        if (!(ok = wait_warp(&c->s_full[h], steps_done & 1, c, A.status))) break;
        ++steps_done;
        tc_fence_after();
        float v[128];
        const uint32_t bad = *(volatile uint32_t*)&c->bad[(tiles + t) & 15];
        if constexpr (KIND == kSparse) if (bad != 0) {
          // halves of which a row sees some tokens, where its sinks end, its window begins and the row itself is: those
          // tokens are taken out in TMEM, and the half counts as seen.  Few columns of a tile, by a short loop.
          for (uint32_t x = bad & 255u; x != 0; x &= x - 1) mask &= ~(3u << (2 * (__ffs(x) - 1)));
          mask &= bits16(16 * kt, ((min(lim, p.end) + 7) >> 3) - p.out, 16 * kt);      // a block reaches behind row or table
          const int s0 = (A.S >> 3) - 16 * kt, w0 = ((lim - A.W) >> 3) - p.out - 16 * kt, c0 = (lim >> 3) - p.out - 16 * kt;
          uint32_t cut = 0;
          if ((A.S & 7) != 0 && A.S < lim && (unsigned)s0 < 16u) cut |= 1u << s0;
          if (lim > A.W && lim - A.W < p.end && ((lim - A.W) & 7) != 0 && (unsigned)w0 < 16u) cut |= 1u << w0;
          cut &= ~mask;              // a selected block's are seen in full, up to the row
          if (lim > 0 && lim <= p.end && (lim & 7) != 0 && (unsigned)c0 < 16u) cut |= 1u << c0;
          for (uint32_t x = bad & 255u; x != 0; x &= x - 1) cut &= ~(3u << (2 * (__ffs(x) - 1)));
          const int* page = ring->page[(tiles + t) % kPageDepth];
#pragma unroll 1
          for (uint32_t x = __reduce_or_sync(0xffffffffu, cut); x != 0; x &= x - 1) {
            const int e = __ffs(x) - 1, t0 = page[e >> 1] * kP + 8 * (e & 1);
            auto below = [t0](int y) { return (1u << min(max(y - t0, 0), 8)) - 1u; };   // of 8 tokens, those before y
            uint32_t see = (mask >> e) & 1u ? 0xffu : below(A.S) | (~below(max(lim - A.W, 0)) & 0xffu);
            see &= below(lim);
            if (!((cut >> e) & 1u)) see = 0xffu;     // this row's half is whole, or not seen at all
            uint32_t y[8];
            tmem_ld8(tS + 8 * e, y);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = (see >> j) & 1u ? y[j] : 0xff800000u;
            tmem_st8(tS + 8 * e, y);
          }
          mask |= cut;
          tmem_wait_st();
        }
        tmem_ld64_start<0>(tS, v);
        tmem_ld64_finish<0>(v);
        if constexpr (KIND == kSparse) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (!((mask >> (j >> 3)) & 1u)) v[j] = -INFINITY;
        } else if ((kt + 1) * kRows > edge || bad != 0) {
          // masked in TMEM, 32 columns at a time: once or twice an item, and
          // a long piece of straight code would cost its instruction fetches
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {
            const int c0 = kt * kRows + 32 * w;
            const int nlim = lim - c0, nend = p.end - c0;
            uint32_t see = nlim >= 32 ? 0xffffffffu : nlim <= 0 ? 0u : (1u << nlim) - 1u;   // bit j: column c0 + j
            const int sh = c0 - p.a;     // column c0 is bit sh of the word
            if (sh > -32 && sh < 64) see |= sh >= 0 ? (uint32_t)(word >> sh) : (uint32_t)(word << -sh);
            see &= nend >= 32 ? 0xffffffffu : nend <= 0 ? 0u : (1u << nend) - 1u;
            if ((bad >> (2 * w)) & 1u) see &= 0xffff0000u;
            if ((bad >> (2 * w + 1)) & 1u) see &= 0x0000ffffu;
            float x[32];
            uint32_t y[32];
            tmem_ld32(tS + 32 * w, x);
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = (see >> j) & 1u ? __float_as_uint(x[j]) : 0xff800000u;
            tmem_st32(tS + 32 * w, y);
          }
          tmem_wait_st();
          tmem_ld64_start<0>(tS, v);
          tmem_ld64_finish<0>(v);
        }
        tmem_ld64_start<64>(tS + 64, v);
        // the maximum of the first half while the second is on its way
        float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int j = 4; j < 60; j += 8) {
#pragma unroll
          for (int x = 0; x < 4; ++x) top[x] = fmaxf(fmaxf(top[x], v[j + x]), v[j + 4 + x]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) top[x] = fmaxf(top[x], v[60 + x]);
        tmem_ld64_finish<64>(v);
        if constexpr (KIND == kSparse) {
#pragma unroll
          for (int j = 64; j < 128; ++j)
            if (!((mask >> (j >> 3)) & 1u)) v[j] = -INFINITY;
        }
#pragma unroll
        for (int j = 64; j < 128; j += 8) {
#pragma unroll
          for (int x = 0; x < 4; ++x) top[x] = fmaxf(fmaxf(top[x], v[j + x]), v[j + 4 + x]);
        }
        float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        mx *= A.scale_log2;
        if (m == -INFINITY) m = mx;   // all zeros so far: nothing to rescale
        // a warp rescales together, each row by what it grew itself: a factor of one
        // for the others, whose bits depend on no neighbour, and no vote for lanes
        // without a row, which hold another sequence's queries or an earlier call's
        const bool grow = mx > m + lag;
        if (__any_sync(0xffffffffu, grow)) {
          const float alpha = grow ? ex2(m - mx) : 1.f;
          m = grow ? mx : m;
          l *= alpha;
          if (s >= 2) {
#pragma unroll 1
            for (int q4 = 0; q4 < 4; ++q4) {
              float o[32];
              uint32_t ow[32];
              tmem_ld32(tO + 32 * q4, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) ow[j] = __float_as_uint(o[j] * alpha);
              tmem_st32(tO + 32 * q4, ow);
            }
          }
        }
        const float mu = m == -INFINITY ? 0.f : m;
        const uint64_t scale2 = pack2(A.scale_log2, A.scale_log2), shift2 = pack2(-mu, -mu);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          uint32_t pw[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float p0, p1;
            unpack2(fma2(pack2(v[32 * q4 + 2 * j], v[32 * q4 + 2 * j + 1]), scale2, shift2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            sum[j & 1] = add2(sum[j & 1], pack2(p0, p1));
            pw[j] = pack_bf16(p0, p1);      // half a step, 2^-9 to 2^-8, of each weight
          }
          tmem_st16(tS + 16 * q4, pw);
          if (q4 & 1) {   // half of the weights are there: their product may begin
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&c->p_full[h][q4 >> 1]);
          }
        }
        float sum0, sum1;
        unpack2(add2(sum[0], sum[1]), sum0, sum1);
        l += sum0 + sum1;
      }
      if (!ok) break;
      const bool mine = N > h;     // this group had a tile
      if (mine) {
        if (!(ok = wait_warp(&c->o_done[h], items_done & 1, c, A.status))) break;
        ++items_done;
        tc_fence_after();
      }
      const bool whole = p.k0 == 0 && p.k1 == p.nt;
      float m1 = -INFINITY, l1 = 0.f;
      if (p.dual) {
        if (h == 1) {
          c->ml[r] = make_float2(m, l);
          tc_fence_before();
          mbar_arrive(&c->ml_full);
        } else {
          if (!(ok = wait_warp(&c->ml_full, duals & 1, c, A.status))) break;
          tc_fence_after();
          const float2 x = c->ml[r];
          m1 = x.x;
          l1 = x.y;
        }
      }
      // every tile of the piece has been multiplied by now, so its edge is clean and known
      const bool poisoned = *(volatile int*)&c->poison[piece & 3] == piece + 1;
      if (!(p.dual && h == 1)) {
        // the two groups' states of a row joined; a group without a tile, or without a position seen, has l = 0
        const bool two = p.dual && N > 1;
        const float M = two ? fmaxf(m, m1) : m;
        const float w0 = l == 0.f ? 0.f : two ? ex2(m - M) : 1.f, w1 = two && l1 != 0.f ? ex2(m1 - M) : 0.f;
        const float lt = l * w0 + (two ? l1 * w1 : 0.f);
        // a whole item's rows are done; those of a part of two wait for the other, as 32-bit sums
        const long long row = (long long)(p.row0 + tok) * A.Hq + p.kvh * A.G + g;
        bool final_out = whole;
        float* half = nullptr;
        float2* half_ml = nullptr;
        if constexpr (KIND == kShared) {
          final_out = whole && p.to == kAll;
          const long long at = (p.to == kOwn ? (long long)A.n_rows * A.Hq : 0) + row;
          half = A.half + at * kD;
          half_ml = A.half_ml + at;
        }
        const float inv = final_out ? (lt == 0.f ? 0.f : 1.f / lt) : 1.f;
        const int which = p.k0 > 0 ? 0 : 1;
        const size_t slot = ((size_t)blockIdx.x * 2 + which) * 2 + h;
        float* part = A.part + slot * kRows * kD + 4 * r;     // [dims / 4][row][4]
        // a row's result lies in one lane: four lanes exchange theirs, so that
        // a store covers 64 bytes of each of 8 rows and not 16 of 32
        long long rows4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) rows4[j] = __shfl_sync(0xffffffffu, valid ? row : -1ll, (lane & 28) + j);
        const float f0 = w0 * inv, f1 = w1 * inv;
        float zero = 0.f;     // kSparse: NaN where a sum is not finite
        // kept short (a loop over 32 columns): it runs once an item, and the
        // fetch of its instructions costs more than the work
#pragma unroll 1
        for (int q4 = 0; q4 < 4; ++q4) {
          float o[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0.f;
          if (mine) {
            tmem_ld32(tO + 32 * q4, o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= f0;     // zeros where the row saw nothing
          }
          if (two) {
            float o1[32];
            tmem_ld32(tO + 128 + 32 * q4, o1);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = fmaf(o1[j], f1, o[j]);
          }
          if constexpr (KIND == kSparse) {
#pragma unroll
            for (int j = 0; j < 32; ++j) zero = fmaf(o[j], 0.f, zero);
          }
          if (final_out) {
            uint32_t x[4][4];
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j >> 2][j & 3] = pack_bf16(o[2 * j], o[2 * j + 1]);
            swap_rows4(x, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (rows4[j] >= 0)
                reinterpret_cast<uint4*>(A.out + rows4[j] * kD + 32 * q4)[lane & 3] =
                    make_uint4(x[j][0], x[j][1], x[j][2], x[j][3]);
          } else if (KIND == kShared && whole) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t x[4][4];
#pragma unroll
              for (int j = 0; j < 16; ++j) x[j >> 2][j & 3] = __float_as_uint(o[16 * e + j]);
              swap_rows4(x, lane);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (rows4[j] >= 0)
                  reinterpret_cast<uint4*>(half + (rows4[j] - row) * kD + 32 * q4 + 16 * e)[lane & 3] =
                      make_uint4(x[j][0], x[j][1], x[j][2], x[j][3]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(part + (8 * q4 + j) * (4 * kRows)) =
                  make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        }
        if constexpr (KIND == kSparse) {
          unsigned again = __ballot_sync(0xffffffffu, valid && zero != 0.f);
          for (; again != 0; again &= again - 1) {
            const int src = __ffs(again) - 1;
            __syncwarp();     // the row was stored by its neighbours too
            SeenRow s;
            s.row = (size_t)__shfl_sync(0xffffffffu, row, src);
            s.kvh = p.kvh;
            s.pos = __shfl_sync(0xffffffffu, lim, src) - 1;
            s.M = __shfl_sync(0xffffffffu, M == -INFINITY ? 0.f : M, src);
            const float f = __shfl_sync(0xffffffffu, inv, src);
            const float4 x = sums_of_row(A, p, s);
            if (whole)
              reinterpret_cast<uint2*>(A.out + s.row * kD)[lane] =
                  make_uint2(pack_bf16(x.x * f, x.y * f), pack_bf16(x.z * f, x.w * f));
            else
              *reinterpret_cast<float4*>(part + 4 * (src - lane) + lane * (4 * kRows)) = x;
          }
        } else if (poisoned) {
          __syncwarp();     // the row was stored by its neighbours too
          if (valid)
            add_poison(A, EdgeRow{A.page_table + table_at(A, p), word, max(p.edge, p.k0 * kRows),
                                  min(p.end, p.k1 * kRows), lim, p.a},
                       p.kvh, final_out ? A.out + row * kD : nullptr, whole ? half : part, whole ? 4 : 4 * kRows);
        }
        if (KIND == kShared && whole && !final_out) {
          if (valid) *half_ml = make_float2(M, lt);
        } else if (whole) {
          if (valid && A.lse != nullptr) A.lse[row] = lt == 0.f ? -INFINITY : (M + log2f(lt)) * 0.693147180559945309f;
        } else {
          if (valid) A.part_ml[slot * kRows + r] = make_float2(M, lt);
          if (tid == 0)
            A.desc[blockIdx.x * 2 + which] =
                make_int4(p.b, p.kvh, p.i, kDescValid | (p.k0 == 0 ? kDescFirst : 0) | (p.k1 == p.nt ? kDescLast : 0) |
                                               (p.dual ? kDescDual : 0));
        }
      }
      if (p.dual) {   // the second group's O may be written again
        if (h == 0) {
          tc_fence_before();
          mbar_arrive(&c->ml_free);
        } else if (!(ok = wait_warp(&c->ml_free, duals & 1, c, A.status))) {
          break;
        }
        ++duals;
      }
      tiles += ntp;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->piece_empty[piece % kPieces]);
    }
  } else {
    regs_dec<kOtherRegs>();
    if (warp == 8) {
      // ------------------------------------------------------------ matrix instructions
      // The whole warp runs the loop and one elected lane issues; the others
      // wait for it at the end of each group (spinning ahead at the next
      // barrier they would take its issue slots).
      constexpr uint32_t idS = bf16_idesc(128, 128, false), idO = bf16_idesc(128, 128, true);
      const uint64_t dQ = smem_desc(smem_u32(s_q), 16, 1024);
      const uint64_t dK = smem_desc(smem_u32(s_kv), 16, 2048), dV = smem_desc(smem_u32(s_kv), 1024, 2048);
      Ring kr, vr;               // the next K and the next V tile
      vr.advance(1);
      uint32_t pieces = 0, cleaned = 0, p_par[2] = {0, 0};   // cleaned: a parity bit a slot
      bool ok = true;
      for (int piece = 0; wait_warp(&c->piece_full[piece % kPieces], (piece / kPieces) & 1, c, A.status); ++piece) {
        const Piece* pp = &c->piece[piece % kPieces];
        const int k0 = pp->k0, ntp = pp->k1 - k0, edge = pp->edge;
        const bool dual = pp->dual;
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->piece_empty[piece % kPieces]);
        if (k0 < 0) break;
        if (ntp == 0) continue;
        if (!(ok = wait_warp(&c->q_full, pieces & 1, c, A.status))) break;
        ++pieces;
        auto mma_s = [&](int h) {      // S of group h from the tile at kr
          const uint64_t q = dQ + (dual ? 0 : h * (kTileBytes / 16)), k = dK + kr.slot * (kTileBytes / 16);
          const uint32_t d = tmem + h * 128;
#pragma unroll
          for (int x = 0; x < 8; ++x)
            tc_mma_ss(d, q + (x >> 2) * (kTileBytes / 2 / 16) + (x & 3) * 2,
                      k + (x >> 2) * (1024 / 16) + (x & 3) * 2, idS, x != 0);
        };
        // O of group h from the tile at vr: the tokens of one half of the weights
        auto mma_o = [&](int h, int part, bool first) {
          const uint64_t v = dV + vr.slot * (kTileBytes / 16);
          const uint32_t d = tmem + 256 + h * 128, w = tmem + h * 128;
#pragma unroll
          for (int x = 4 * part; x < 4 * part + 4; ++x)
            tc_mma_ts(d, w + x * 8, v + x * (4096 / 16), idO, x != 0 || !first);
        };
        auto issue_s = [&](int h, bool k_done, bool q_done) {
          mma_s(h);
          tc_commit(&c->s_full[h]);
          if (k_done) tc_commit(&c->empty[kr.slot]);
          if (q_done) tc_commit(&c->q_empty);
        };
        auto wait_k = [&]() -> bool { return wait_warp(&c->full[kr.slot], kr.parity, c, A.status); };
        auto wait_v = [&](int kt) -> bool {
          if (!wait_warp(&c->full[vr.slot], vr.parity, c, A.status)) return false;
          if ((kt + 1) * kRows > edge) {
            if (!wait_warp(&c->clean[vr.slot], (cleaned >> vr.slot) & 1, c, A.status)) return false;
            cleaned ^= 1u << vr.slot;
          }
          return true;
        };
        // A step of group h: O from the tile at vr, then S from the tile at kr
        // (`more`: there is one).  What it needs is there as a rule: one look at
        // all of it, and nothing stands between the instructions.  What is late
        // is waited for in the order of its use, a K tile behind O, whose V
        // slot comes free.
        // seen: the other group has waited for both tiles; done: they have no
        // other reader; q_done: nor has Q.
        auto step = [&](int h, int kt, bool first, bool more, bool seen, bool done, bool q_done) -> bool {
          const bool clean = (kt + 1) * kRows <= edge;
          const bool v_there = seen || mbar_test_wait(&c->full[vr.slot], vr.parity);
          const bool k_there = !more || seen || mbar_test_wait(&c->full[kr.slot], kr.parity);
          const bool p_there = mbar_test_wait(&c->p_full[h][1], p_par[h]);
          if (__all_sync(0xffffffffu, v_there && k_there && p_there && (seen || clean))) {
            tc_fence_after();
            if (elect_one()) {
              mma_o(h, 0, first);
              mma_o(h, 1, first);
              if (done) tc_commit(&c->empty[vr.slot]);
              if (more) issue_s(h, done, q_done);
              else tc_commit(&c->o_done[h]);
            }
          } else {
            if (!seen && !wait_v(kt)) return false;
            if (!wait_warp(&c->p_full[h][0], p_par[h], c, A.status)) return false;   // half of the weights
            tc_fence_after();
            if (elect_one()) mma_o(h, 0, first);
            __syncwarp();
            if (!wait_warp(&c->p_full[h][1], p_par[h], c, A.status)) return false;
            tc_fence_after();
            if (elect_one()) {
              mma_o(h, 1, first);
              if (done) tc_commit(&c->empty[vr.slot]);
              if (!more) tc_commit(&c->o_done[h]);
            }
            __syncwarp();
            if (more) {
              if (!seen && !wait_k()) return false;
              if (elect_one()) issue_s(h, done, q_done);
            }
          }
          __syncwarp();
          p_par[h] ^= 1;
          if (done) {
            vr.advance(2);
            if (more) kr.advance(2);
          }
          return true;
        };
        auto first_s = [&](int h, bool k_done, bool q_done) {
          if (elect_one()) issue_s(h, k_done, q_done);
          __syncwarp();
          if (k_done) kr.advance(2);
        };
        if (!(ok = wait_k())) break;
        if (dual) {      // a tile a step, the groups in turn
          first_s(0, true, ntp == 1);
          if (ntp > 1) {
            if (!(ok = wait_k())) break;
            first_s(1, true, ntp == 2);
          }
#pragma unroll 1
          for (int s = 0; s < ntp; ++s) {
            const bool more = s + 2 < ntp;
            if (!(ok = step(s & 1, k0 + s, s < 2, more, false, true, s + 3 == ntp))) break;
          }
        } else {         // a tile two steps
          first_s(0, false, false);
          first_s(1, true, ntp == 1);
#pragma unroll 1
          for (int t = 0; t < ntp; ++t) {
            const bool first = t == 0, more = t + 1 < ntp;
            if (!(ok = step(0, k0 + t, first, more, false, false, false))) break;
            if (!(ok = step(1, k0 + t, first, more, true, true, t + 2 == ntp))) break;
          }
        }
        if (!ok) break;
      }
      // nothing of this block is in flight when it frees its TMEM and ends
      __syncwarp();
      if (elect_one()) {
        tc_commit(&c->drain);
        wait_out(&c->drain, 0, A.status);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ------------------------------------------------------------ loads
      uint32_t tile = 0, pieces = 0, loads = 0;
      const uint32_t q_bytes = (uint32_t)(A.tpt * A.G) * kD * 2;
      bool ok = true;
      Walk<KIND> walk(A, c);
      for (int piece = 0;; ++piece) {
        PieceOf<KIND> p;
        if (!walk.next(p)) p.k0 = p.k1 = -1;
        if (piece >= kPieces &&
            !(ok = wait_warp(&c->piece_empty[piece % kPieces], (piece / kPieces - 1) & 1, c, A.status)))
          break;
        if (lane == 0) {
          c->piece[piece % kPieces] = p;
          mbar_arrive(&c->piece_full[piece % kPieces]);
        }
        if (p.k0 < 0) break;
        const int ntp = p.k1 - p.k0;
        if (ntp == 0) continue;
        if (pieces > 0 && !(ok = wait_warp(&c->q_empty, (pieces - 1) & 1, c, A.status))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&c->q_full, p.dual ? q_bytes : 2 * q_bytes);
          for (int x = 0; x < (p.dual ? 2 : 4); ++x)
            tma_load_3d(s_q + x * (kTileBytes / 2), &tmQ, (x & 1) * 64, p.kvh * A.G, p.row0 + (x >> 1) * A.tpt,
                        &c->q_full);
        }
        ++pieces;
        // a lane a page of the tile; the next tile's pages are looked up while this one's are copied
        const int* pt = A.page_table + table_at(A, p);
        PageWalk<KIND> pages(A, p, 8 * p.k0);
        bool next_there = false;
        uint32_t next_cut = 0;
        auto page_of = [&](int t) {
          int page;
          if constexpr (KIND == kSparse) {
            if (t == ntp) return -1;
            int* place = ring->page[(tile + t) % kPageDepth];
            page = pages.next();
            if (lane < kRows / kP) place[lane] = page;
            // views begin or end inside 8 tokens where the sinks do, and where rows' windows and the rows themselves are;
            // on an item's last page a block may go on behind it (rows behind a table that ends inside a block)
            const int t0 = page * kP, w0 = max(p.a + 1, 0) - A.W, w1 = w0 + p.tokens - 1;
            const bool in = ((A.S & 7) != 0 && t0 == (A.S & ~(kP - 1))) || (t0 + kP > w0 && t0 <= w1) ||
                            t0 + kP > min(p.a, p.end - 1);
            next_cut = __any_sync(0xffffffffu, page >= 0 && in) ? kCut : 0;
            next_there = page >= 0;
          } else {
            page = (p.k0 + t) * (kRows / kP) + lane;
            next_there = lane < kRows / kP && page * kP < p.end;
          }
          return next_there ? __ldg(pt + page) : -1;
        };
        int next_phys = page_of(0);
        for (int t = 0; t < ntp; ++t) {
          const bool there = next_there;
          const uint32_t cut = next_cut;
          const int phys = next_phys;
          next_phys = page_of(t + 1);
          const bool good = phys >= 0 && phys < A.num_pages;
          const unsigned goods = __ballot_sync(0xffffffffu, good), bads = __ballot_sync(0xffffffffu, there && !good);
          if (bads != 0 && lane == 0) set_status(A.status, SA_ERR_BAD_PAGE);
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t idx = 2 * (tile + t) + kv, slot = idx % kSlots;
            if (idx >= kSlots && !(ok = wait_warp(&c->empty[slot], (idx / kSlots - 1) & 1, c, A.status))) break;
            uint8_t* dst = s_kv + slot * kTileBytes;
            if (kv == 0) {
              if (lane == 0) *(volatile uint32_t*)&c->bad[(tile + t) & 15] = bads | cut;
            } else if (bads != 0) {   // V of a page that is not there: zeros
              for (int x = lane; x < kTileBytes / 16; x += 32)
                if ((bads >> (x >> 8)) & 1u) reinterpret_cast<uint4*>(dst)[x] = make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_expect_tx(&c->full[slot], __popc(goods) * 4096);
              if (kv == 1 && (p.k0 + t + 1) * kRows > p.edge) mbar_arrive(&c->edge_go[slot]);
            }
            ++loads;
            __syncwarp();
            if (good)
              tma_load_4d(dst + lane * 4096, kv == 0 ? (const void*)&tmK : (const void*)&tmV, 0, 0, 0,
                          (phys * A.Hk + p.kvh) * 2, &c->full[slot]);
          }
          if (!ok) break;
        }
        if (!ok) break;
        tile += ntp;
      }
      // copies in flight land before the block ends
      for (uint32_t j = loads > kSlots ? loads - kSlots : 0; j < loads; ++j)
        wait_out(&c->full[j % kSlots], (j / kSlots) & 1, A.status);
      if (pieces > 0) wait_out(&c->q_full, (pieces - 1) & 1, A.status);
    } else {
      // ------------------------------------------------------------ the edge of V
      const int w = warp - 10;
      // edge_go orders these warps behind the loads: they skip most uses of a
      // slot, so the parity of its full barrier alone would not tell which one
      uint32_t tile = 0, gone = 0;   // gone: a parity bit a slot
      bool ok = true;
      for (int piece = 0; wait_warp(&c->piece_full[piece % kPieces], (piece / kPieces) & 1, c, A.status); ++piece) {
        const PieceOf<KIND> p = c->piece[piece % kPieces];
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->piece_empty[piece % kPieces]);
        if (p.k0 < 0) break;
        const int ntp = p.k1 - p.k0;
        for (int t = max(0, (p.edge >> 7) - p.k0); t < ntp; ++t) {
          const uint32_t idx = 2 * (tile + t) + 1, slot = idx % kSlots;
          if (!(ok = wait_warp(&c->edge_go[slot], (gone >> slot) & 1, c, A.status))) break;
          gone ^= 1u << slot;
          if (!(ok = wait_warp(&c->full[slot], (idx / kSlots) & 1, c, A.status))) break;
          const int base = (p.k0 + t) * kRows;
          // 16-byte chunk x: token group x / 128, row (x / 8) % 8
          uint4* sv = reinterpret_cast<uint4*>(s_kv + slot * kTileBytes);
          if constexpr (KIND == kSparse) {
            const int* page = ring->page[(tile + t) % kPageDepth];
            for (int x = w * 32 + lane; x < kTileBytes / 16; x += 64) {
              const int at = page[x >> 8];
              if (at < 0 || at * kP + ((x >> 7) & 1) * 8 + ((x >> 3) & 7) >= p.end) sv[x] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->clean[slot]);
            continue;
          }
          bool found = false;
          for (int x = (max(0, p.edge - base) >> 3) * 128 + w * 32 + lane; x < kTileBytes / 16; x += 64) {
            const int pos = base + (x >> 7) * 8 + ((x >> 3) & 7);
            if (pos >= p.end) {
              sv[x] = make_uint4(0, 0, 0, 0);
            } else if (pos >= p.edge) {
              uint4 q = sv[x];
              uint32_t* e = reinterpret_cast<uint32_t*>(&q);
              bool hit = false;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (!bf16_pair_nonfinite(e[j])) continue;
                hit = true;
                if ((e[j] & 0x7f80u) == 0x7f80u) e[j] &= 0xffff0000u;
                if ((e[j] & 0x7f800000u) == 0x7f800000u) e[j] &= 0x0000ffffu;
              }
              if (hit) sv[x] = q;
              found |= hit;
            }
          }
          if (found) *(volatile int*)&c->poison[piece & 3] = piece + 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c->clean[slot]);
        }
        if (!ok) break;
        tile += ntp;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_free(tmem, 512);
}

// Joins the pieces of a cut item, in the order of the cache.  Block (c, y)
// takes rows 16 y on of the item that begins in block c of the attention
// kernel and does not end there (the others leave at once); a warp takes 4
// rows, eight lanes a row.  Bound by latency: what the pieces are is one look
// at all of them, and no load waits for another's value after that.
constexpr int kMergeWarps = 4, kMergeRows = 4 * kMergeWarps, kMergeBatch = 4;
template <int KIND>
__global__ void __launch_bounds__(kMergeWarps * 32) rows_merge_kernel(Args<KIND> A) {
  __shared__ int s_last;
  __shared__ unsigned s_there[kRowsMaxCtas / 32 + 1];
  __shared__ float2 s_ml[kMergeWarps][kRowsMaxCtas][4];   // (maximum, sum) of piece i, then (weight, -)
  pdl_wait();
  pdl_trigger();
  const int ctas = gridDim.x, c = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int4 d = A.desc[2 * c + 1];
  int4 e[kRowsMaxCtas / (kMergeWarps * 32) + 1];
#pragma unroll
  for (int k = 0; k < kRowsMaxCtas / (kMergeWarps * 32) + 1; ++k) {
    const int i = c + k * (kMergeWarps * 32) + tid;        // piece i - c
    e[k] = i < ctas ? A.desc[2 * i + (i == c ? 1 : 0)] : make_int4(0, 0, 0, 0);
  }
  if (!(d.w & kDescValid)) return;
  const bool dual = d.w & kDescDual;
  if (dual && (int)blockIdx.y >= kRows / kMergeRows) return;
  if (tid == 0) s_last = ctas;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kRowsMaxCtas / (kMergeWarps * 32) + 1; ++k) {
    const int i = k * (kMergeWarps * 32) + tid;
    const bool there = e[k].w & kDescValid;
    const unsigned m = __ballot_sync(0xffffffffu, there);
    if (lane == 0 && i / 32 <= kRowsMaxCtas / 32) s_there[i / 32] = m;
    if (there && (e[k].w & kDescLast) && i > 0) atomicMin(&s_last, c + i);
  }
  __syncthreads();
  const int n = min(s_last, ctas - 1) - c + 1;     // pieces: block c's second, then the first of the blocks behind
  const int j4 = lane & 3, part = lane >> 2;
  const int R = blockIdx.y * kMergeRows + warp * 4 + j4, half = R >> 7, r = R & 127;
  const float4* sums = reinterpret_cast<const float4*>(A.part) +
                       ((((size_t)c * 2 + 1) * 2 + half) * (kD / 4) + part) * kRows + r;   // piece 0's
  auto sums_of = [&](int i) { return sums + (i == 0 ? 0ll : (long long)(4 * i - 2) * (kD / 4) * kRows); };
  auto there = [&](int i) { return (s_there[i >> 5] >> (i & 31)) & 1u; };
  float4 v[kMergeBatch][4];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kMergeBatch; ++k) {
      const bool on = i0 + k < n && there(i0 + k);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        v[k][x] = on ? __ldcs(sums_of(i0 + k) + 8 * x * kRows) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  load(0);
  const Seq s = load_seq<KIND>(A, d.x, nullptr);
  float M = -INFINITY;
  for (int i = part; i < n; i += 8) {
    const size_t slot = ((size_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * 2 + half;
    const float2 ml = there(i) ? A.part_ml[slot * kRows + r] : make_float2(0.f, 0.f);
    s_ml[warp][i][j4] = ml;
    if (ml.y != 0.f) M = fmaxf(M, ml.x);
  }
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  float l = 0.f;
  for (int i = part; i < n; i += 8) {
    const float2 ml = s_ml[warp][i][j4];
    const float w = ml.y == 0.f ? 0.f : ex2(ml.x - M);
    s_ml[warp][i][j4].x = w;
    l += ml.y == 0.f ? 0.f : w * ml.y;
  }
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  __syncwarp();
  float4 o[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += kMergeBatch) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int k = 0; k < kMergeBatch; ++k) {
      // a piece without weight is added too (its sums are zeros where the row saw
      // nothing of it): a weight that underflows does not hide an infinite sum
      const float w = i0 + k < n ? s_ml[warp][i0 + k][j4].x : 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        o[x].x = fmaf(v[k][x].x, w, o[x].x);
        o[x].y = fmaf(v[k][x].y, w, o[x].y);
        o[x].z = fmaf(v[k][x].z, w, o[x].z);
        o[x].w = fmaf(v[k][x].w, w, o[x].w);
      }
    }
  }
  const int t_row = r / A.G, g = r - t_row * A.G;
  const int tok = d.z * s.T + half * A.tpt + t_row;    // the row in its sequence
  if (t_row >= A.tpt || tok >= s.n) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const size_t row = (size_t)(s.row0 + tok) * A.Hq + (size_t)d.y * A.G + g;
  if constexpr (KIND == kShared) if (s.to != kAll) {
    const size_t half_row = (s.to == kOwn ? (size_t)A.n_rows * A.Hq : 0) + row;
#pragma unroll
    for (int x = 0; x < 4; ++x) reinterpret_cast<float4*>(A.half + half_row * kD)[8 * x + part] = o[x];
    if (part == 0) A.half_ml[half_row] = make_float2(M, l);
    return;
  }
#pragma unroll
  for (int x = 0; x < 4; ++x)
    reinterpret_cast<uint2*>(A.out + row * kD)[8 * x + part] =
        make_uint2(pack_bf16(o[x].x * inv, o[x].y * inv), pack_bf16(o[x].z * inv, o[x].w * inv));
  if (part == 0 && A.lse != nullptr) A.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.693147180559945309f;
}

constexpr int kJoinWarps = 8;
// Joins the two parts of rows behind a shared prefix.  A block takes a packed
// row, a warp each of its heads in turn; rows that had no prefix are done.
__global__ void __launch_bounds__(kJoinWarps * 32) rows_join_kernel(RowsMoreArgs A) {
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the row's sequence: the last whose rows begin at or ahead of it
  int lo = 0, hi = A.B;      // row_offsets[lo] <= row < row_offsets[hi]
  if (row < __ldg(A.row_offsets) || row >= __ldg(A.row_offsets + A.B)) return;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + step * (lane + 1);
    const unsigned up = __ballot_sync(0xffffffffu, at < hi && __ldg(A.row_offsets + at) <= row);
    const int n = __popc(up);
    hi = min(hi, lo + step * (n + 1));
    lo += step * n;
  }
  const RowSeq s = row_seq(A.row_offsets, A.seq_lens, lo, A.n_rows, A.mpp, nullptr);
  if (row < s.row0 || row >= s.row0 + s.n || shared_prefix(A.prefix_lens, lo, s, A.mpp, nullptr) == 0) return;
  if (A.tree != nullptr && s.n > kMaxTree) return;
  const size_t own = (size_t)A.n_rows * A.Hq;
  for (int h = warp; h < A.Hq; h += kJoinWarps) {
    const size_t r = (size_t)row * A.Hq + h;
    const float4 a = reinterpret_cast<const float4*>(A.half + r * kD)[lane];
    const float4 b = reinterpret_cast<const float4*>(A.half + (own + r) * kD)[lane];
    const float2 ma = A.half_ml[r], mb = A.half_ml[own + r];
    const float M = ma.y == 0.f ? mb.x : mb.y == 0.f ? ma.x : fmaxf(ma.x, mb.x);
    const float wa = ma.y == 0.f ? 0.f : ex2(ma.x - M), wb = mb.y == 0.f ? 0.f : ex2(mb.x - M);
    const float l = wa * ma.y + wb * mb.y;
    const float inv = l == 0.f ? 0.f : 1.f / l, fa = wa * inv, fb = wb * inv;
    reinterpret_cast<uint2*>(A.out + r * kD)[lane] =
        make_uint2(pack_bf16(fmaf(a.x, fa, b.x * fb), fmaf(a.y, fa, b.y * fb)),
                   pack_bf16(fmaf(a.z, fa, b.z * fb), fmaf(a.w, fa, b.w * fb)));
    if (lane == 0 && A.lse != nullptr) A.lse[r] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.693147180559945309f;
  }
}

// The same, and the own tokens of rows that have few (A.join_own).  A block takes
// a KV head of a packed row, a warp every fourth head of its group, and to attend
// them a warp a page: K in pairs of lanes a token, V in four dims a lane, in 32 bits
// throughout.  Bound by the latency of its reads: the row's sequence, the page,
// then K and V at once (a warp a row and KV head, page after page: 91 us in
// place of 72 for 8 x 8 beams).  Four blocks of four warps an SM: rows of few
// pages leave eight warps idle (1000 rows of 10..60 tokens: 79 us with eight, 69
// with four; 2000 rows of 64 heads: 631 and 505; three blocks without the spills
// of groups of five heads and more: 524).
constexpr int kOwnWarps = 4;
template <int G>
__global__ void __launch_bounds__(kOwnWarps * 32, 4) rows_own_join_kernel(RowsMoreArgs A) {
  __shared__ __align__(16) float4 s_o[kOwnWarps][G][32];
  __shared__ float2 s_ml[kOwnWarps][G];
  __shared__ __align__(16) uint4 s_q[G][kD / 8];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x / A.Hk, kvh = blockIdx.x - row * A.Hk;
  // the row's sequence: the last whose rows begin at or ahead of it
  int lo = 0, hi = A.B;      // row_offsets[lo] <= row < row_offsets[hi]
  if (row < __ldg(A.row_offsets) || row >= __ldg(A.row_offsets + A.B)) return;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + step * (lane + 1);
    const unsigned up = __ballot_sync(0xffffffffu, at < hi && __ldg(A.row_offsets + at) <= row);
    const int n = __popc(up);
    hi = min(hi, lo + step * (n + 1));
    lo += step * n;
  }
  const Seq s = load_seq<kShared>(A, 2 * lo + 1, nullptr);
  if (s.to != kOwn || row < s.row0 || row >= s.row0 + s.n) return;
  if (A.tree != nullptr && s.n > kMaxTree) return;
  const size_t own = (size_t)A.n_rows * A.Hq, r = (size_t)row * A.Hq + (size_t)kvh * G;
  const bool here = own_in_join(A, s);
  constexpr int kHeads = (G + kOwnWarps - 1) / kOwnWarps;
  float4 a[kHeads], o[kHeads];           // of heads warp, warp + 4: the prefix's part and the sequence's own
  float2 ma[kHeads], mb[kHeads];
#pragma unroll
  for (int x = 0; x < kHeads; ++x) {
    const int g = warp + x * kOwnWarps;
    if (g >= G) continue;
    a[x] = reinterpret_cast<const float4*>(A.half + (r + g) * kD)[lane];
    ma[x] = A.half_ml[r + g];
    if (!here) {
      o[x] = reinterpret_cast<const float4*>(A.half + (own + r + g) * kD)[lane];
      mb[x] = A.half_ml[own + r + g];
    }
  }
  if (here) {
    for (int x = threadIdx.x; x < G * (kD / 8); x += kOwnWarps * 32)
      (&s_q[0][0])[x] = __ldg(reinterpret_cast<const uint4*>(A.q + r * kD) + x);
    const int lim = A.tree != nullptr ? s.a : s.a + row - s.row0 + 1;   // sees positions below, and the drafts of its word
    const unsigned long long word = A.tree != nullptr ? __ldg(A.tree + row) : 0ull;
    auto sees = [&](int t) {
      const int bit = t - s.a;
      return t < s.L && (t < lim || (bit >= 0 && bit < 64 && ((word >> bit) & 1ull)));
    };
    const int t2 = lane >> 1, half = lane & 1;                  // a lane's token of a page, and half of its dims
    float4 part[G];
    float m[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      part[g] = make_float4(0.f, 0.f, 0.f, 0.f);
      m[g] = -INFINITY;
      l[g] = 0.f;
    }
    __syncthreads();
    for (int page = warp; page * kP < s.L; page += kOwnWarps) {
      const int phys = __ldg(A.page_table + s.pt + page);
      if (phys < 0 || phys >= A.num_pages) {
        if (lane == 0) set_status(A.status, SA_ERR_BAD_PAGE);
        continue;
      }
      const size_t slab = ((size_t)phys * A.Hk + kvh) * kP * kD;
      const uint4* k = reinterpret_cast<const uint4*>(A.k_pool + slab + t2 * kD) + 8 * half;
      const uint2* v = reinterpret_cast<const uint2*>(A.v_pool + slab) + lane;
      uint4 kv[8];
      uint2 x[kP];
#pragma unroll
      for (int d = 0; d < 8; ++d) kv[d] = __ldg(k + d);
#pragma unroll
      for (int e = 0; e < kP; ++e) x[e] = __ldg(v + e * (kD / 4));
      const bool seen = sees(page * kP + t2);
      float z[G];
#pragma unroll
      for (int g = 0; g < G; ++g) z[g] = 0.f;
#pragma unroll
      for (int d = 0; d < 8; ++d) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint4 q = s_q[g][8 * half + d];
          z[g] = fma_bf16_lo(q.x, kv[d].x, z[g]);
          z[g] = fma_bf16_hi(q.x, kv[d].x, z[g]);
          z[g] = fma_bf16_lo(q.y, kv[d].y, z[g]);
          z[g] = fma_bf16_hi(q.y, kv[d].y, z[g]);
          z[g] = fma_bf16_lo(q.z, kv[d].z, z[g]);
          z[g] = fma_bf16_hi(q.z, kv[d].z, z[g]);
          z[g] = fma_bf16_lo(q.w, kv[d].w, z[g]);
          z[g] = fma_bf16_hi(q.w, kv[d].w, z[g]);
        }
      }
      const unsigned who = __ballot_sync(0xffffffffu, seen);      // bits 2 e and 2 e + 1: token e
#pragma unroll
      for (int g = 0; g < G; ++g) {
        z[g] += __shfl_xor_sync(0xffffffffu, z[g], 1);
        z[g] = seen ? z[g] * A.scale_log2 : -INFINITY;
        float top = z[g];
#pragma unroll
        for (int y = 2; y < 32; y <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
        const float M = fmaxf(m[g], top), mu = M == -INFINITY ? 0.f : M;
        const float alpha = m[g] == -INFINITY ? 0.f : ex2(m[g] - mu);
        m[g] = M;
        z[g] = seen ? ex2(z[g] - mu) : 0.f;
        float sum = z[g];
#pragma unroll
        for (int y = 2; y < 32; y <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
        l[g] = fmaf(l[g], alpha, sum);
        part[g].x *= alpha;
        part[g].y *= alpha;
        part[g].z *= alpha;
        part[g].w *= alpha;
      }
#pragma unroll
      for (int e = 0; e < kP; ++e) {
        // what the row does not see is not multiplied: a weight of zero times infinity is NaN
        if (!((who >> (2 * e)) & 1u)) continue;
        const float v0 = bf16_lo(x[e].x), v1 = bf16_hi(x[e].x), v2 = bf16_lo(x[e].y), v3 = bf16_hi(x[e].y);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float p = __shfl_sync(0xffffffffu, z[g], 2 * e);
          part[g].x = fmaf(p, v0, part[g].x);
          part[g].y = fmaf(p, v1, part[g].y);
          part[g].z = fmaf(p, v2, part[g].z);
          part[g].w = fmaf(p, v3, part[g].w);
        }
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      s_o[warp][g][lane] = part[g];
      if (lane == 0) s_ml[warp][g] = make_float2(m[g], l[g]);
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kHeads; ++x) {
      const int g = warp + x * kOwnWarps;
      if (g >= G) continue;
      o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      mb[x] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int w = 0; w < kOwnWarps; ++w) mb[x].x = fmaxf(mb[x].x, s_ml[w][g].x);
#pragma unroll
      for (int w = 0; w < kOwnWarps; ++w) {
        const float2 z = s_ml[w][g];
        if (z.y == 0.f) continue;                // no page of it, or nothing seen
        const float f = ex2(z.x - mb[x].x);
        const float4 y = s_o[w][g][lane];
        mb[x].y = fmaf(z.y, f, mb[x].y);
        o[x].x = fmaf(y.x, f, o[x].x);
        o[x].y = fmaf(y.y, f, o[x].y);
        o[x].z = fmaf(y.z, f, o[x].z);
        o[x].w = fmaf(y.w, f, o[x].w);
      }
    }
  }
#pragma unroll
  for (int x = 0; x < kHeads; ++x) {
    const int g = warp + x * kOwnWarps;
    if (g >= G) continue;
    const float M = ma[x].y == 0.f ? mb[x].x : mb[x].y == 0.f ? ma[x].x : fmaxf(ma[x].x, mb[x].x);
    const float wa = ma[x].y == 0.f ? 0.f : ex2(ma[x].x - M), wb = mb[x].y == 0.f ? 0.f : ex2(mb[x].x - M);
    const float sum = wa * ma[x].y + wb * mb[x].y;
    const float inv = sum == 0.f ? 0.f : 1.f / sum, fa = wa * inv, fb = wb * inv;
    reinterpret_cast<uint2*>(A.out + (r + g) * kD)[lane] =
        make_uint2(pack_bf16(fmaf(a[x].x, fa, o[x].x * fb), fmaf(a[x].y, fa, o[x].y * fb)),
                   pack_bf16(fmaf(a[x].z, fa, o[x].z * fb), fmaf(a[x].w, fa, o[x].w * fb)));
    if (lane == 0 && A.lse != nullptr) A.lse[r + g] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.693147180559945309f;
  }
}

template <int KIND>
int launch(const Args<KIND>& A, const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV, int num_sms,
           cudaStream_t stream) {
  const int ctas = std::min(num_sms, kRowsMaxCtas);
  if (smem_limit_at_least(reinterpret_cast<const void*>(rows_attention_kernel<KIND>), (int)kSmemBytes<KIND>) != cudaSuccess)
    return SA_ERR_CUDA;
  cudaError_t e =
      launch_pdl(rows_attention_kernel<KIND>, dim3(ctas), dim3(kThreads), kSmemBytes<KIND>, stream, A, tmQ, tmK, tmV);
  if (e != cudaSuccess) return SA_ERR_CUDA;
  e = launch_pdl(rows_merge_kernel<KIND>, dim3(ctas, 2 * kRows / kMergeRows), dim3(kMergeWarps * 32), 0, stream, A);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace

int launch_rows_attention(const RowsAttnArgs& A, const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                          int num_sms, cudaStream_t stream) {
  return launch<kPlain>(A, tmQ, tmK, tmV, num_sms, stream);
}

int launch_shared_attention(const RowsMoreArgs& args, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                            const CUtensorMap& tmV, int num_sms, cudaStream_t stream) {
  RowsMoreArgs A = args;
  // few rows a sequence, and more sequences and KV heads than twice the blocks: a block would have items of one or two
  // tiles one behind the other (1000 single tokens in groups of 50: 120 us without, 78 with; four beams: 19.5 and 21.9)
  A.join_own = (long long)A.n_rows <= (long long)kJoinRows * A.B && (long long)A.B * A.Hk >= 2ll * num_sms &&
               (long long)A.n_rows * A.Hk < (1ll << 31);
  const int rc = launch<kShared>(A, tmQ, tmK, tmV, num_sms, stream);
  if (rc != SA_OK) return rc;
  cudaError_t e;
  if (!A.join_own) {
    e = launch_pdl(rows_join_kernel, dim3(A.n_rows), dim3(kJoinWarps * 32), 0, stream, A);
  } else {
    void (*const join[kMaxG])(RowsMoreArgs) = {rows_own_join_kernel<1>, rows_own_join_kernel<2>, rows_own_join_kernel<3>,
                                               rows_own_join_kernel<4>, rows_own_join_kernel<5>, rows_own_join_kernel<6>,
                                               rows_own_join_kernel<7>, rows_own_join_kernel<8>};
    e = launch_pdl(join[A.G - 1], dim3(A.n_rows * A.Hk), dim3(kOwnWarps * 32), 0, stream, A);
  }
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

int launch_sparse_attention(const RowsMoreArgs& A, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                            const CUtensorMap& tmV, int num_sms, cudaStream_t stream) {
  const int rc = launch_sparse_items(A, stream);
  return rc == SA_OK ? launch<kSparse>(A, tmQ, tmK, tmV, num_sms, stream) : rc;
}

}  // namespace sa
