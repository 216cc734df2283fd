// The work of sa_sparse_row_attention: which pages the rows of an item see, and
// where each row's blocks lie among them.
//
// An item is one KV head of a sequence with up to 256 / G neighbouring rows.
// The pages that some row sees (sinks, windows, blocks of the rows' lists) are
// a bitmap, L / 128 bytes an item; the attention reads eight of them a tile.
// A row's list is written again with places in that list of pages for blocks:
// a row then finds what it sees of a tile by one comparison a tile and a few
// instructions an entry (looking every page of a tile up in the list took the
// attention three times as long).
//
// A block an item: bits are set in shared memory, so lists of any length give
// the same bitmap whatever the order of the threads.  Bound by the latency of
// its reads (offsets, then counts and entries, four rows' at once) and the
// lists' bytes: a row a warp at a time, counts first, took 375 us of a 32K
// prompt's 3.7 ms.  The last block to finish sums the items' weights up for the
// attention's blocks.
#include "rows.cuh"

namespace sa {
namespace {

constexpr int kItemThreads = 256, kAtOnce = 4, kScanEach = 4;
constexpr int kNone = 0x7fffffff;

// before[u + 1]: item u's weight becomes the sum up to and with it.  A whole block.
__device__ void sum_weights(const RowsMoreArgs& A, long long* s_sum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long carry = 0;
  int real = 0;
  for (int u0 = 0; u0 < A.n_items; u0 += kItemThreads * kScanEach) {
    long long x[kScanEach], sum = 0;
#pragma unroll
    for (int e = 0; e < kScanEach; ++e) {
      const int u = u0 + tid * kScanEach + e;
      x[e] = u < A.n_items ? *(volatile long long*)(A.before + u + 1) : 0;
      sum += x[e];
      real += x[e] > 0;
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    long long at = carry + incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kItemThreads / 32; ++w) {
      if (w < warp) at += s_sum[w];
      total += s_sum[w];
    }
    __syncthreads();
    carry += total;
#pragma unroll
    for (int e = 0; e < kScanEach; ++e) {
      const int u = u0 + tid * kScanEach + e;
      at += x[e];
      if (u < A.n_items) A.before[u + 1] = at;
    }
  }
  if (tid == 0) {
    A.before[0] = 0;
    A.ticket[0] = A.ticket[1] = 0;
  }
  __syncthreads();
  real = __reduce_add_sync(0xffffffffu, real);
  if (lane == 0 && real > 0) atomicAdd(A.ticket + 1, real);
}

// f(row's token, row and head ahead of it from the item's first, entry's index
// j, entry) for all places j < rank_stride of the lists of an item's rows;
// entries behind a row's count are kNone.  No divisions: they were most of the
// kernel's instructions.
template <typename F>
__device__ __forceinline__ void each_entry(const RowsMoreArgs& A, const SparseItem& it, F f) {
  int log = 2;                                       // of the lanes a row
  while ((1 << log) < A.rank_stride && log < 5) ++log;
  const int tid = threadIdx.x, sub = tid & ((1 << log) - 1), groups = kItemThreads >> log;
  const int rows = it.tokens * A.G;
  const unsigned by_g = 65536u / A.G + 1;            // r / G for r < 256, G <= 8
  const size_t first = (size_t)it.row0 * A.Hq + it.kvh * A.G;
  const int* counts = A.sel_cnt + first;
  const int* lists = A.sel_idx + first * A.kcap;
  for (int j = sub; j < A.rank_stride; j += 1 << log) {
    for (int r0 = tid >> log; r0 < rows; r0 += groups * kAtOnce) {
      int n[kAtOnce], e[kAtOnce];
      unsigned tok[kAtOnce], at[kAtOnce];
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {
        const unsigned r = r0 + x * groups;
        n[x] = 0;
        e[x] = 0;
        if (r < rows) {
          tok[x] = r * by_g >> 16;
          at[x] = tok[x] * (A.Hq - A.G) + r;         // tok * Hq + head
          n[x] = __ldg(counts + at[x]);
          if (j < A.kcap) e[x] = __ldg(lists + (size_t)at[x] * A.kcap + j);
        }
      }
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x)
        if (r0 + x * groups < rows) f((int)tok[x], first + at[x], j, j < min(n[x], A.kcap) ? e[x] : kNone);
    }
  }
}

__global__ void __launch_bounds__(kItemThreads) sparse_items_kernel(RowsMoreArgs A) {
  extern __shared__ uint32_t s_bits[];
  __shared__ ItemPlace s_place;
  __shared__ long long s_sum[kItemThreads / 32];
  __shared__ bool s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u = blockIdx.x, T = 2 * A.tpt;
  pdl_wait();
  pdl_trigger();
  find_item<kItemThreads>(A.row_offsets, A.seq_lens, A.B, A.n_rows, A.mpp, A.Hk, T, u, A.status, &s_place);
  const int b = s_place.b;
  SparseItem it{};
  long long weight = 0;
  if (b >= 0) {
    const RowSeq s = row_seq(A.row_offsets, A.seq_lens, b, A.n_rows, A.mpp, nullptr);
    it.b = b;
    it.kvh = s_place.kvh;
    it.i = (s.n + T - 1) / T - 1 - s_place.i;      // those that see most first: the last ones taken are short
    it.tokens = min(T, s.n - it.i * T);
    it.row0 = s.row0 + it.i * T;
    it.pos0 = s.a + it.i * T;
    it.end = max(0, min(s.L, it.pos0 + it.tokens));
    const int n_pages = (it.end + kP - 1) / kP, words = (n_pages + 31) / 32;
    for (int w = tid; w < words; w += kItemThreads) s_bits[w] = 0;
    __syncthreads();
    auto set = [&](int w, uint32_t m) {
      if ((*(volatile uint32_t*)&s_bits[w] & m) != m) atomicOr(&s_bits[w], m);
    };
    const int shift = A.bs_shift[it.kvh];
    // a row's last position that is there (rows behind the table see what lies in it); negative: it sees nothing
    auto last_pos = [&](int tok) {
      const int pos = it.pos0 + tok;
      return pos < 0 ? pos : min(pos, it.end - 1);
    };
    if (it.end > 0) {
      const int sinks = (min(A.S, it.end) + kP - 1) / kP;
      for (int page = tid; page < sinks; page += kItemThreads) set(page >> 5, 1u << (page & 31));
      const int first = max(it.pos0, 0);                    // the first row that sees anything
      const int window = first + 1 > A.W ? first + 1 - A.W : 0;
      for (int page = window / kP + tid; page < n_pages; page += kItemThreads) set(page >> 5, 1u << (page & 31));
      each_entry(A, it, [&](int tok, size_t, int, int e) {
        const int pos = last_pos(tok);
        if (pos < 0 || e < 0 || e > pos >> shift) return;
        const int page = (e << shift) / kP, end = min(((e + 1) << shift) - 1, pos) / kP;   // in one word: aligned
        set(page >> 5, ((2u << (end - page)) - 1u) << (page & 31));
      });
    }
    __syncthreads();
    // pages ahead of each word
    int* s_ahead = reinterpret_cast<int*>(s_bits + A.words);
    int* s_warp = reinterpret_cast<int*>(s_sum);
    int carry = 0;
    for (int w0 = 0; w0 < words; w0 += kItemThreads) {
      const int w = w0 + tid;
      const uint32_t x = w < words ? s_bits[w] : 0u;
      if (w < words) A.pages[(size_t)u * A.words + w] = x;
      const int n = __popc(x), incl = warp_incl_scan(n);
      if (lane == 31) s_warp[warp] = incl;
      __syncthreads();
      int at = carry + incl - n, total = 0;
#pragma unroll
      for (int y = 0; y < kItemThreads / 32; ++y) {
        if (y < warp) at += s_warp[y];
        total += s_warp[y];
      }
      if (w < words) s_ahead[w] = at;
      __syncthreads();
      carry += total;
    }
    // the lists again: the place of a block's first half page.  Entries below zero are ahead of all of them,
    // those behind the row or its count are behind, so that lists stay ascending.
    each_entry(A, it, [&](int tok, size_t row, int j, int e) {
      const int pos = last_pos(tok);
      int rank = e < 0 ? -64 : kNone;
      if (e >= 0 && pos >= 0 && e <= pos >> shift) {
        const int page = (e << shift) / kP, w = page >> 5;
        rank = 2 * (s_ahead[w] + __popc(s_bits[w] & ((1u << (page & 31)) - 1u))) + (shift == 3 ? e & 1 : 0);
      }
      A.ranks[row * A.rank_stride + j] = rank;
    });
    it.pages = carry;
    weight = (long long)((carry + 7) / 8) * kSparseTileCost + kSparseItemCost;
  }
  if (tid == 0) {
    A.items[u] = it;
    A.before[u + 1] = weight;
    __threadfence();
    s_last = atomicAdd(A.arrived, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  sum_weights(A, s_sum);
  if (tid == 0) *A.arrived = 0;      // as the next call finds it
}

}  // namespace

int launch_sparse_items(const RowsMoreArgs& A, cudaStream_t stream) {
  const int smem = 2 * A.words * (int)sizeof(uint32_t);
  if (smem_limit_at_least(reinterpret_cast<const void*>(sparse_items_kernel), smem) != cudaSuccess) return SA_ERR_CUDA;
  const cudaError_t e = launch_pdl(sparse_items_kernel, dim3(A.n_items), dim3(kItemThreads), (size_t)smem, stream, A);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace sa
