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
// A block an item: bits are set in shared memory, so lists of any length and
// order give the same bitmap.  Bound by the latency of its reads (offsets,
// counts, lists) and the lists' bytes.  A second kernel sums the items' weights
// up for the attention's blocks.
#include "rows.cuh"

namespace sa {
namespace {

constexpr int kItemThreads = 128, kScanThreads = 1024, kScanEach = 4;

__global__ void __launch_bounds__(kItemThreads) sparse_items_kernel(RowsAttnArgs A) {
  extern __shared__ uint32_t s_bits[];
  __shared__ ItemPlace s_place;
  __shared__ int s_sum[kItemThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u = blockIdx.x, T = 2 * A.tpt;
  pdl_wait();
  pdl_trigger();
  find_item<kItemThreads>(A.row_offsets, A.seq_lens, A.B, A.n_rows, A.mpp, A.Hk, T, u, A.status, &s_place);
  const int b = s_place.b;
  SparseItem it{};
  if (b < 0) {
    if (tid == 0) {
      A.items[u] = it;
      A.before[u + 1] = 0;
    }
    return;
  }
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
  auto set = [&](int page) {
    const uint32_t bit = 1u << (page & 31);
    if (!(*(volatile uint32_t*)&s_bits[page >> 5] & bit)) atomicOr(&s_bits[page >> 5], bit);
  };
  if (it.end > 0) {
    const int sinks = (min(A.S, it.end) + kP - 1) / kP;
    for (int page = tid; page < sinks; page += kItemThreads) set(page);
    const int first = max(it.pos0, 0);                    // the first row that sees anything
    const int window = first + 1 > A.W ? first + 1 - A.W : 0;
    for (int page = window / kP + tid; page < n_pages; page += kItemThreads) set(page);
    const int shift = A.bs_shift[it.kvh];
    for (int r = warp; r < it.tokens * A.G; r += kItemThreads / 32) {
      const int tok = r / A.G, pos = min(it.pos0 + tok, it.end - 1);   // rows behind the table see what lies in it
      if (it.pos0 + tok < 0) continue;
      const size_t row = (size_t)(it.row0 + tok) * A.Hq + it.kvh * A.G + (r - tok * A.G);
      const int n = min(max(__ldg(A.sel_cnt + row), 0), A.kcap);
      const int* list = A.sel_idx + row * A.kcap;
      for (int j = lane; j < n; j += 32) {
        const int e = __ldg(list + j);
        if (e < 0 || e > pos >> shift) continue;
        const int t0 = e << shift, last = min(t0 + (1 << shift) - 1, pos) / kP;
        for (int page = t0 / kP; page <= last; ++page) set(page);
      }
    }
  }
  __syncthreads();
  // pages ahead of each word
  int* s_ahead = reinterpret_cast<int*>(s_bits + A.words);
  int carry = 0;
  for (int w0 = 0; w0 < words; w0 += kItemThreads) {
    const int w = w0 + tid;
    const uint32_t x = w < words ? s_bits[w] : 0u;
    if (w < words) A.pages[(size_t)u * A.words + w] = x;
    const int n = __popc(x), incl = warp_incl_scan(n);
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int at = carry + incl - n, total = 0;
#pragma unroll
    for (int y = 0; y < kItemThreads / 32; ++y) {
      if (y < warp) at += s_sum[y];
      total += s_sum[y];
    }
    if (w < words) s_ahead[w] = at;
    __syncthreads();
    carry += total;
  }
  // the lists again, entries that count alone: the place of a block's first half page
  const int shift = A.bs_shift[it.kvh];
  for (int r = warp; r < it.tokens * A.G; r += kItemThreads / 32) {
    const int tok = r / A.G, pos = min(it.pos0 + tok, it.end - 1);
    if (it.pos0 + tok < 0) continue;
    const size_t row = (size_t)(it.row0 + tok) * A.Hq + it.kvh * A.G + (r - tok * A.G);
    const int n = min(max(__ldg(A.sel_cnt + row), 0), A.kcap);
    const int* list = A.sel_idx + row * A.kcap;
    int* ranks = A.ranks + row * A.rank_stride;
    int m = 0;
    for (int j0 = 0; j0 < n; j0 += 32) {
      const int e = j0 + lane < n ? __ldg(list + j0 + lane) : -1;
      const bool on = e >= 0 && pos >= 0 && e <= pos >> shift;
      const unsigned all = __ballot_sync(0xffffffffu, on);
      if (on) {
        const int page = (e << shift) / kP, w = page >> 5;
        const int rank = s_ahead[w] + __popc(s_bits[w] & ((1u << (page & 31)) - 1u));
        ranks[m + __popc(all & ((1u << lane) - 1u))] = 2 * rank + (shift == 3 ? e & 1 : 0);
      }
      m += __popc(all);
    }
    for (int j = m + lane; j < A.rank_stride; j += 32) ranks[j] = 0x7fffffff;
  }
  if (tid == 0) {
    it.pages = carry;
    A.items[u] = it;
    A.before[u + 1] = (long long)((carry + 7) / 8) * kSparseTileCost + kSparseItemCost;
  }
}

// before[u + 1]: item u's weight becomes the sum up to and with it.
__global__ void __launch_bounds__(kScanThreads) sparse_scan_kernel(RowsAttnArgs A) {
  __shared__ long long s_sum[kScanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  long long carry = 0;
  int real = 0;
  for (int u0 = 0; u0 < A.n_items; u0 += kScanThreads * kScanEach) {
    long long x[kScanEach], sum = 0;
#pragma unroll
    for (int e = 0; e < kScanEach; ++e) {
      const int u = u0 + tid * kScanEach + e;
      x[e] = u < A.n_items ? A.before[u + 1] : 0;
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
    for (int w = 0; w < kScanThreads / 32; ++w) {
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

}  // namespace

int launch_sparse_items(const RowsAttnArgs& A, cudaStream_t stream) {
  const int smem = 2 * A.words * (int)sizeof(uint32_t);
  if (smem_limit_at_least(reinterpret_cast<const void*>(sparse_items_kernel), smem) != cudaSuccess) return SA_ERR_CUDA;
  cudaError_t e = launch_pdl(sparse_items_kernel, dim3(A.n_items), dim3(kItemThreads), (size_t)smem, stream, A);
  if (e == cudaSuccess) e = launch_pdl(sparse_scan_kernel, dim3(1), dim3(kScanThreads), 0, stream, A);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace sa
