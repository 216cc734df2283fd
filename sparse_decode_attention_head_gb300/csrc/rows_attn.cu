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
// Slower: two issuing warps, one a group (1.94 ms: the groups' instructions
// interleave and both finish late); one barrier for all of a tile's weights
// in place of one for each half (2 %); two threads a row (1.90 ms: 104
// registers do not hold what they need, and they meet once a tile).
#include <algorithm>

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
// What work weighs: a KV token of an item with one query tile (bound by the
// loads: measured 1.45 us a tile of them) and with two (1.6 us), and an item's
// query load, first tile and epilogue (3.4 us).
constexpr int kOneCost = 6, kTwoCost = 7, kItemCost = 2000;
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

constexpr int kPieces = 4;
constexpr int kPieceReaders = 11;        // warps: softmax, matrix instructions, edge

struct Ctl {
  Piece piece[kPieces];
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
constexpr size_t kSmemBytes = 1024 + 2 * kTileBytes + kSlots * kTileBytes + sizeof(Ctl);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// Waits with a limit of kWaitNs; a wait that runs out, here or elsewhere in the
// block, ends the block's work.
constexpr unsigned long long kWaitNs = 2000000000ull;
[[nodiscard]] __device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Ctl* c, int* status) {
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
[[nodiscard]] __device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Ctl* c, int* status) {
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

struct Seq : RowSeq {
  int items;      // of one KV head
  int T;          // tokens of an item
};

__device__ __forceinline__ Seq load_seq(const RowsAttnArgs& A, int b, int* status) {
  Seq s;
  static_cast<RowSeq&>(s) = row_seq(A.row_offsets, A.seq_lens, b, A.n_rows, A.mpp, status);
  s.T = 2 * A.tpt;
  s.items = (s.n + s.T - 1) / s.T;
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
__device__ __forceinline__ long long weight_before(const RowsAttnArgs& A, const Seq& s, int k) {
  if (k == 0) return 0;
  const int full = min(k, s.items - 1);
  const long long before = max(A.tree != nullptr ? s.L : s.a, 0);
  long long w = (before * full + (A.tree != nullptr ? 0 : (long long)s.T * full * (full + 1) / 2)) * kTwoCost +
                (long long)k * kItemCost;
  if (k == s.items) {
    const int tokens = s.n - full * s.T;
    w += (before + (A.tree != nullptr ? 0 : s.n)) * (tokens <= A.tpt ? kOneCost : kTwoCost);
  }
  return w;
}

// One warp: the total weight of all items.  `s` and `mine` are the lane's own
// sequence, of the first 32, and its weight.
__device__ __forceinline__ long long total_weight(const RowsAttnArgs& A, int* status, Seq& s, long long& mine) {
  const int lane = threadIdx.x & 31;
  long long w = 0;
  mine = 0;
  s = Seq{};
  for (int b = lane; b < A.B; b += 32) {
    const Seq x = load_seq(A, b, status);
    const long long m = weight_before(A, x, x.items) * A.Hk;
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

// One warp: the item and KV tile at weight w (the end: sequence B).
template <typename T>
__device__ __forceinline__ int4 locate(const RowsAttnArgs& A, T w, Seq s, T mine) {
  const int lane = threadIdx.x & 31;
  T before = 0;
  for (int b0 = 0; b0 < A.B; b0 += 32) {
    const int b = b0 + lane;
    if (b0 > 0) {
      mine = 0;
      if (b < A.B) {
        s = load_seq(A, b, nullptr);
        mine = (T)weight_before(A, s, s.items) * A.Hk;
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
    if (lane == src) {
      T rem = w - (before + upto - mine);
      const T each = mine / (T)A.Hk;
      r.y = (int)(rem / each);
      rem -= each * r.y;
      int lo = 0, hi = s.items;     // the item: weight_before(lo) <= rem < weight_before(hi)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((T)weight_before(A, s, mid) <= rem) lo = mid; else hi = mid;
      }
      const T w0 = (T)weight_before(A, s, lo), w1 = (T)weight_before(A, s, lo + 1);
      r.z = lo;
      r.w = (int)((unsigned long long)(rem - w0) * tiles_of(item_end(A, s, lo)) / (w1 - w0));
    }
    r.x = __shfl_sync(0xffffffffu, r.x, src);
    r.y = __shfl_sync(0xffffffffu, r.y, src);
    r.z = __shfl_sync(0xffffffffu, r.z, src);
    r.w = __shfl_sync(0xffffffffu, r.w, src);
    return r;
  }
  return make_int4(A.B, 0, 0, 0);
}

// Little work: every block takes one item or an equal part of one, of two KV
// tiles or four, and none takes two.  `s` as above (B <= 32).  Answers false
// where the blocks do not suffice for that.
__device__ __forceinline__ int runs_of(const RowsAttnArgs& A, const Seq& s, int i, int tiles) {
  return max(1, (tiles_of(item_end(A, s, i)) + tiles - 1) / tiles);
}
__device__ __forceinline__ bool locate_small(const RowsAttnArgs& A, int run, int blocks, const Seq& s, int4& r) {
  const int lane = threadIdx.x & 31;
  if (A.B > 32) return false;
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
  r = make_int4(A.B, 0, 0, 0);
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

// One thread walks a block's run, piece by piece.
struct Walk {
  const RowsAttnArgs& A;
  int b, kvh, i, kt;
  int4 end;
  bool done;
  Seq s;
  __device__ Walk(const RowsAttnArgs& a, const Ctl* c) : A(a) {
    const int4 r = c->range[0];
    b = r.x; kvh = r.y; i = r.z; kt = r.w;
    end = c->range[1];
    done = b >= A.B;
    if (!done) s = load_seq(A, b, nullptr);
  }
  __device__ bool next(Piece& p) {
    while (!done) {
      const bool at_end = b == end.x && kvh == end.y && i == end.z;
      p.b = b; p.kvh = kvh; p.i = i;
      p.end = item_end(A, s, i);
      p.edge = item_edge(A, s, i);
      p.nt = tiles_of(p.end);
      p.k0 = kt;
      p.k1 = at_end ? end.w : p.nt;
      p.a = s.a;
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
          do {
            if (++b >= A.B) { done = true; break; }
            s = load_seq(A, b, nullptr);
          } while (s.items == 0);
        }
      }
      if (some) return true;
    }
    return false;
  }
};

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
__device__ __noinline__ void add_poison(const RowsAttnArgs& A, EdgeRow e, int kvh, __nv_bfloat16* out, float* part) {
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
      else part[(d >> 2) * (4 * kRows) + (d & 3)] += x;
    }
  }
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// ---------------------------------------------------------------- the kernel

__global__ void __launch_bounds__(kThreads, 1)
rows_attention_kernel(RowsAttnArgs A, const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = smem;                                  // two tiles: [half of the dims][128 rows][64]
  uint8_t* s_kv = smem + 2 * kTileBytes;                // kSlots tiles: [16 groups of 8 tokens][half][8][64]
  Ctl* c = reinterpret_cast<Ctl*>(s_kv + kSlots * kTileBytes);
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
  if (warp < 2) {   // where this block's run begins (warp 0) and ends (warp 1)
    Seq s;
    long long mine;
    const long long W = total_weight(A, blockIdx.x == 0 && warp == 0 ? A.status : nullptr, s, mine);
    int4 r;
    if (locate_small(A, blockIdx.x + warp, gridDim.x, s, r)) {
    } else if (W < (1ll << 32) / kRowsMaxCtas) {     // in 32 bits, whose divisions are short
      r = locate<uint32_t>(A, (uint32_t)W * (blockIdx.x + warp) / gridDim.x, s, (uint32_t)mine);
    } else {
      r = locate<long long>(A, W * (blockIdx.x + warp) / gridDim.x, s, mine);
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
      const Piece& p = c->piece[piece % kPieces];
      const int k0 = p.k0, ntp = p.k1 - k0, edge = p.edge;
      const bool dual = p.dual;
      if (k0 < 0) break;
      const int N = dual ? ntp : 2 * ntp;
      const int tok = t_row + (dual || h == 0 ? 0 : A.tpt);
      const bool valid = t_row < A.tpt && tok < p.tokens;
      // what the row sees: positions below lim, and bit j of its word for position p.a + j
      int lim = 0;
      unsigned long long word = 0;
      if (valid) {
        if (A.tree != nullptr) {
          lim = p.a;
          word = __ldg(A.tree + p.row0 + tok);
        } else {
          lim = p.a + p.first + tok + 1;
        }
      }
      const float lag = valid ? kLag : INFINITY;   // a lane without a row never grows
      float m = -INFINITY, l = 0.f;
      for (int s = h; s < N; s += 2) {
        const int t = dual ? s : s >> 1;
        const int kt = k0 + t;
        if (!(ok = wait_warp(&c->s_full[h], steps_done & 1, c, A.status))) break;
        ++steps_done;
        tc_fence_after();
        float v[128];
        tmem_ld64_start<0>(tS, v);
        const uint32_t bad = *(volatile uint32_t*)&c->bad[(tiles + t) & 15];
        tmem_ld64_finish<0>(v);
        if ((kt + 1) * kRows > edge || bad != 0) {
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
        const float inv = whole ? (lt == 0.f ? 0.f : 1.f / lt) : 1.f;
        const int which = p.k0 > 0 ? 0 : 1;
        const size_t slot = ((size_t)blockIdx.x * 2 + which) * 2 + h;
        float* part = A.part + slot * kRows * kD + 4 * r;     // [dims / 4][row][4]
        const long long row = (long long)(p.row0 + tok) * A.Hq + p.kvh * A.G + g;
        // a row's result lies in one lane: four lanes exchange theirs, so that
        // a store covers 64 bytes of each of 8 rows and not 16 of 32
        long long rows4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) rows4[j] = __shfl_sync(0xffffffffu, valid ? row : -1ll, (lane & 28) + j);
        const float f0 = w0 * inv, f1 = w1 * inv;
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
          if (whole) {
            uint32_t x[4][4];     // pieces of 16 bytes; then row j's piece lane % 4
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j >> 2][j & 3] = pack_bf16(o[2 * j], o[2 * j + 1]);
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
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (rows4[j] >= 0)
                reinterpret_cast<uint4*>(A.out + rows4[j] * kD + 32 * q4)[lane & 3] =
                    make_uint4(x[j][0], x[j][1], x[j][2], x[j][3]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(part + (8 * q4 + j) * (4 * kRows)) =
                  make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        }
        if (poisoned) {
          __syncwarp();     // the row was stored by its neighbours too
          if (valid)
            add_poison(A, EdgeRow{A.page_table + (size_t)p.b * A.mpp, word, max(p.edge, p.k0 * kRows),
                                  min(p.end, p.k1 * kRows), lim, p.a},
                       p.kvh, whole ? A.out + row * kD : nullptr, whole ? nullptr : part);
        }
        if (whole) {
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
      Walk walk(A, c);
      for (int piece = 0;; ++piece) {
        Piece p;
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
        const int* pt = A.page_table + (size_t)p.b * A.mpp;
        auto page_of = [&](int t) {
          const int page = (p.k0 + t) * (kRows / kP) + lane;
          return lane < kRows / kP && page * kP < p.end ? __ldg(pt + page) : -1;
        };
        int next_phys = page_of(0);
        for (int t = 0; t < ntp; ++t) {
          const bool there = lane < kRows / kP && ((p.k0 + t) * (kRows / kP) + lane) * kP < p.end;
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
              if (lane == 0) *(volatile uint32_t*)&c->bad[(tile + t) & 15] = bads;
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
        const Piece p = c->piece[piece % kPieces];
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
__global__ void __launch_bounds__(kMergeWarps * 32) rows_merge_kernel(RowsAttnArgs A) {
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
  const Seq s = load_seq(A, d.x, nullptr);
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
#pragma unroll
  for (int x = 0; x < 4; ++x)
    reinterpret_cast<uint2*>(A.out + row * kD)[8 * x + part] =
        make_uint2(pack_bf16(o[x].x * inv, o[x].y * inv), pack_bf16(o[x].z * inv, o[x].w * inv));
  if (part == 0 && A.lse != nullptr) A.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.693147180559945309f;
}

}  // namespace

int launch_rows_attention(const RowsAttnArgs& A, const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                          int num_sms, cudaStream_t stream) {
  const int ctas = std::min(num_sms, kRowsMaxCtas);
  if (smem_limit_at_least(reinterpret_cast<const void*>(rows_attention_kernel), (int)kSmemBytes) != cudaSuccess)
    return SA_ERR_CUDA;
  cudaError_t e = launch_pdl(rows_attention_kernel, dim3(ctas), dim3(kThreads), kSmemBytes, stream, A, tmQ, tmK, tmV);
  if (e != cudaSuccess) return SA_ERR_CUDA;
  e = launch_pdl(rows_merge_kernel, dim3(ctas, 2 * kRows / kMergeRows), dim3(kMergeWarps * 32), 0, stream, A);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace sa
