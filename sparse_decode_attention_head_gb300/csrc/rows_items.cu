// The work of sa_sparse_row_attention: which pages the rows of an item see.
//
// An item is one KV head of a sequence with up to 128 / G neighbouring rows.
// The pages that some row sees (sinks, windows, blocks of the rows' lists) are
// a bitmap; the attention reads eight of them a tile and finds what each row
// sees of a page from the row's own list.  A bitmap takes L / 128 bytes an
// item, where a mask of a bit for each row would take 128 times that.
//
// A block an item: bits are set in shared memory, so lists of any length and
// order give the same bitmap.  Bound by the latency of its reads (offsets, counts, lists)
// and the lists' bytes.  A second kernel sums the items' weights up for the
// attention's blocks.
#include "rows.cuh"

namespace sa {
namespace {

constexpr int kItemThreads = 128, kScanThreads = 1024, kScanEach = 4;

__global__ void __launch_bounds__(kItemThreads) sparse_items_kernel(RowsAttnArgs A) {
  extern __shared__ uint32_t s_bits[];
  __shared__ ItemPlace s_place;
  __shared__ int s_pages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u = blockIdx.x, T = A.tpt;
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
  it.i = s_place.i;
  if (tid == 0) s_pages = 0;
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
  int n = 0;
  for (int w = tid; w < words; w += kItemThreads) {
    const uint32_t x = s_bits[w];
    A.pages[(size_t)u * A.words + w] = x;
    n += __popc(x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if (lane == 0) atomicAdd(&s_pages, n);
  __syncthreads();
  if (tid == 0) {
    it.tiles = (s_pages + 7) / 8;
    A.items[u] = it;
    A.before[u + 1] = (long long)it.tiles * kSparseTileCost + kSparseItemCost;
  }
}

// before[u + 1]: item u's weight becomes the sum up to and with it.
__global__ void __launch_bounds__(kScanThreads) sparse_scan_kernel(RowsAttnArgs A) {
  __shared__ long long s_sum[kScanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  long long carry = 0;
  for (int u0 = 0; u0 < A.n_items; u0 += kScanThreads * kScanEach) {
    long long x[kScanEach], sum = 0;
#pragma unroll
    for (int e = 0; e < kScanEach; ++e) {
      const int u = u0 + tid * kScanEach + e;
      x[e] = u < A.n_items ? A.before[u + 1] : 0;
      sum += x[e];
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
  if (tid == 0) A.before[0] = 0;
}

}  // namespace

int launch_sparse_items(const RowsAttnArgs& A, cudaStream_t stream) {
  const int smem = A.words * (int)sizeof(uint32_t);
  if (smem_limit_at_least(reinterpret_cast<const void*>(sparse_items_kernel), smem) != cudaSuccess) return SA_ERR_CUDA;
  cudaError_t e = launch_pdl(sparse_items_kernel, dim3(A.n_items), dim3(kItemThreads), (size_t)smem, stream, A);
  if (e == cudaSuccess) e = launch_pdl(sparse_scan_kernel, dim3(1), dim3(kScanThreads), 0, stream, A);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace sa
