// The pages of the cache: the next table of a batch (fork, free, truncate,
// grow), packing the pool, copying pages, taking over a tree's accepted rows.
//
// Who holds a page is counted afresh from the table each time (integer
// counts, so the order of the atomics leaves no trace); there is no state of
// its own that could disagree with it.  Ranks of free, live and moved pages
// come from a count of each chunk of 1024 pages and a sum over the chunks
// before.  The steps hang on one another, so the whole of it runs in one
// cluster of 16 blocks with a cluster barrier between them: bound by latency
// (12 us for a table of 64 rows of 510 pages, 19 us for packing a pool of 64K
// pages; 13 and 28 with 8 blocks).  The copies are bound by HBM: a page is
// read and written once, a warp moving a 4 KB slab (one head of one page) with
// eight 16-byte loads a lane in flight.
#include <algorithm>
#include <atomic>

#include "rows.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kP - 1) / kP; }

// A row of the next table: the old row it goes on from, the tokens it keeps
// and has room for.  Impossible ones are empty (and recorded by the count).
struct PlanRow {
  int parent, keep, room;
  bool writes;     // will write inside the last page that it keeps
};

template <bool PLAN>
__device__ __forceinline__ PlanRow plan_row(const PageArgs& A, int b, int* status) {
  PlanRow r;
  const int cap = A.mpp * kP;
  r.keep = A.keep[b];
  if (PLAN) {
    r.parent = A.parent[b];
    r.room = A.lens[b];
    const bool ok = r.parent >= -1 && r.parent < A.B && r.keep >= 0 && r.keep <= cap && r.room <= cap;
    if (!ok) {
      if (status != nullptr) set_status(status, SA_ERR_INVALID_ARG);
      r.parent = -1;
      r.room = 0;
    }
    if (r.parent < 0) r.keep = 0;
    r.room = max(r.room, r.keep);
    r.writes = r.keep % kP != 0 && r.room > r.keep;
  } else {
    if (r.keep < 0 || r.keep > cap) {
      if (status != nullptr) set_status(status, SA_ERR_INVALID_ARG);
      r.keep = 0;
    }
    r.parent = b;
    r.room = r.keep;
    r.writes = false;
  }
  return r;
}

constexpr int kCluster = 16, kTableThreads = kPageChunk;

// What one block of the cluster wrote is seen by the others behind this.
__device__ __forceinline__ void cluster_sync() {
  __threadfence();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Inclusive sum over a block of 1024 threads.
__device__ __forceinline__ int block_scan(int x, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = warp_incl_scan(x);
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) s_warp[lane] = warp_incl_scan(s_warp[lane]);
  __syncthreads();
  return x + (warp > 0 ? s_warp[warp - 1] : 0);
}
// The sum, for every thread.
__device__ __forceinline__ int block_sum(int x, int* s_warp) {
  block_scan(x, s_warp);
  return s_warp[31];
}

// PLAN: the next table of a batch; else the packing of the pool.
template <bool PLAN>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kTableThreads) table_kernel(PageArgs A) {
  __shared__ int s_warp[32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, cta = blockIdx.x;
  const int chunks = (A.num_pages + kPageChunk - 1) / kPageChunk;
  // a warp takes 128 entries of a table row at a time, four a lane, so that
  // their loads do not wait on one another
  const int lane = tid & 31, cols = (A.mpp + 127) / 128;
  const long long pieces = (long long)A.B * cols, warps = kCluster * (kTableThreads / 32);
  const long long piece0 = (long long)(tid >> 5) * kCluster + cta;

  // no holders
  const long long words = (long long)A.num_pages * (PLAN ? 3 : 1);   // refs, writers, lowest lie together
  for (long long i = (long long)cta * kTableThreads + tid; i < words; i += kCluster * kTableThreads) A.refs[i] = 0;
  cluster_sync();

  // holders of every page; for a plan also the rows that will write inside it and the lowest of them
  for (long long x = piece0; x < pieces; x += warps) {
    const int b = (int)(x / cols), j0 = (int)(x % cols) * 128 + lane;
    const PlanRow r = plan_row<PLAN>(A, b, j0 == 0 ? A.status : nullptr);
    const int held = pages_of(r.keep);
    int page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      page[k] = j0 + 32 * k < held ? __ldg(A.table_in + (size_t)r.parent * A.mpp + j0 + 32 * k) : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (j0 + 32 * k >= held) continue;
      if (page[k] < 0 || page[k] >= A.num_pages) {
        set_status(A.status, SA_ERR_BAD_PAGE);
        continue;
      }
      atomicAdd(A.refs + page[k], 1);
      if (PLAN && r.writes && j0 + 32 * k == held - 1) {
        atomicAdd(A.writers + page[k], 1);
        atomicMax(A.lowest + page[k], kMaxPlanRows - b);
      }
    }
  }
  cluster_sync();

  // free (plan) or live (compact) pages of each chunk
  for (int c = cta; c < chunks; c += kCluster) {
    const int page = c * kPageChunk + tid;
    const int n = __syncthreads_count(page < A.num_pages && (__ldcg(A.refs + page) == 0) == PLAN);
    if (tid == 0) A.chunk[c] = n;
  }
  if (PLAN && cta == kCluster - 1) {   // what the rows need, lined up
    int need = 0, copy = 0;
    if (tid < A.B) {
      const PlanRow r = plan_row<true>(A, tid, nullptr);
      const int held = pages_of(r.keep);
      if (r.writes) {
        const int page = A.table_in[(size_t)r.parent * A.mpp + held - 1];
        if (page >= 0 && page < A.num_pages)
          copy = !(__ldcg(A.writers + page) == __ldcg(A.refs + page) && __ldcg(A.lowest + page) == kMaxPlanRows - tid);
      }
      need = copy + pages_of(r.room) - held;
    }
    const int upto = block_scan(need, s_warp);
    const int copies = block_scan(copy, s_warp);
    if (tid < A.B) {
      A.need[2 * tid] = upto - need;
      A.need[2 * tid + 1] = 2 * (copies - copy) + copy;
    }
    if (tid == kTableThreads - 1) {
      A.need[2 * A.B] = upto;
      A.need[2 * A.B + 1] = 2 * copies;
    }
  }
  cluster_sync();

  // ranks: the first free pages that the plan takes; or source and target of every move
  int all = 0;
  for (int i = tid; i < chunks; i += kTableThreads) all += __ldcg(A.chunk + i);
  all = block_sum(all, s_warp);
  const int take = PLAN ? __ldcg(A.need + 2 * A.B) : 0;
  int low = 0;                       // compact: live pages below index `all`, the number of live pages
  if (!PLAN) {
    for (int i = tid; i < min(chunks, all / kPageChunk); i += kTableThreads) low += __ldcg(A.chunk + i);
    const int edge = all / kPageChunk * kPageChunk + tid;
    low += edge < all && edge < A.num_pages && __ldcg(A.refs + edge) != 0;
    low = block_sum(low, s_warp);
  }
  const int moves = all - low;
  int before = 0;                    // in the chunks before this block's next one
  for (int c = cta, seen = 0; c < chunks; c += kCluster) {
    int sum = 0;
    for (int i = seen + tid; i < c; i += kTableThreads) sum += __ldcg(A.chunk + i);
    before += block_sum(sum, s_warp);
    seen = c;
    const int page = c * kPageChunk + tid;
    const bool in = page < A.num_pages;
    const bool hit = in && (__ldcg(A.refs + page) == 0) == PLAN;
    const int rank = before + block_scan(hit, s_warp) - hit;      // hits below this page
    if (PLAN) {
      if (hit && rank < take) A.list[rank] = page;
    } else if (in) {
      if (hit && page >= all) {
        A.src[rank - low] = page;
        A.list[page] = rank - low;
      }
      if (!hit && page < all) A.dst[page - rank] = page;
      if (page >= moves) A.src[page] = A.dst[page] = -1;
    }
  }
  if (cta == 0 && tid == 0) {
    A.counts[0] = PLAN ? __ldcg(A.need + 2 * A.B + 1) >> 1 : moves;
    A.counts[1] = PLAN ? all - take : all;
    if (PLAN && all < take) set_status(A.status, SA_ERR_CAPACITY);
  }
  cluster_sync();

  // the next table, and a plan's list of copies
  const int copies = PLAN ? __ldcg(A.need + 2 * A.B + 1) >> 1 : 0;
  for (long long x = piece0; x < pieces; x += warps) {
    const int b = (int)(x / cols), j0 = (int)(x % cols) * 128 + lane;
    const PlanRow r = plan_row<PLAN>(A, b, nullptr);
    const int held = pages_of(r.keep), room = pages_of(r.room);
    const int start = PLAN ? __ldcg(A.need + 2 * b) : 0, mark = PLAN ? __ldcg(A.need + 2 * b + 1) : 0, copy = mark & 1;
    int page[4], to[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + 32 * k;
      page[k] = j < held ? __ldg(A.table_in + (size_t)r.parent * A.mpp + j) : -1;
      if (page[k] < 0 || page[k] >= A.num_pages) page[k] = -1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {      // a fresh page of the plan, the place of a page that moves
      const int j = j0 + 32 * k;
      to[k] = page[k];
      if (PLAN) {
        const bool copied = copy && j == held - 1;
        if (copied || (j >= held && j < room)) {
          const int at = start + (copied ? 0 : copy + j - held);
          to[k] = at < all ? __ldcg(A.list + at) : -1;
        }
      } else if (page[k] >= all) {
        to[k] = __ldcg(A.dst + __ldcg(A.list + page[k]));
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + 32 * k;
      if (PLAN && copy && j == held - 1) {
        A.src[mark >> 1] = page[k];
        A.dst[mark >> 1] = to[k];
      }
      if (j < A.mpp) A.table_out[(size_t)b * A.mpp + j] = to[k];
    }
    // rows behind the number of copies clear its entries
    if (PLAN && j0 == 0 && b >= copies) A.src[b] = A.dst[b] = -1;
  }
}

template <bool PLAN>
int launch_table(const PageArgs& A, cudaStream_t stream) {
  // clusters of more than 8 blocks are an opt-in, once a device
  static std::atomic<bool> allowed[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SA_ERR_CUDA;
  if (dev >= 64 || !allowed[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(table_kernel<PLAN>),
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return SA_ERR_CUDA;
    if (dev < 64) allowed[dev].store(true, std::memory_order_release);
  }
  const cudaError_t e = launch_pdl(table_kernel<PLAN>, dim3(kCluster), dim3(kTableThreads), 0, stream, A);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

// ---------------------------------------------------------------- copies

__global__ void __launch_bounds__(kThreads)
copy_pages_kernel(uint4* __restrict__ k_pool, uint4* __restrict__ v_pool, const int* __restrict__ src,
                  const int* __restrict__ dst, const int* __restrict__ count, int max_pages, int num_pages, int Hk,
                  int* status) {
  pdl_wait();
  pdl_trigger();
  constexpr int kSlab = kP * kD * 2 / 16;    // 16-byte chunks of one head of one page
  const int lane = threadIdx.x & 31;
  const int n = min(max(__ldg(count), 0), max_pages);
  const long long units = (long long)n * 2 * Hk;
  for (long long u = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units;
       u += (long long)gridDim.x * (kThreads / 32)) {
    const int i = (int)(u / (2 * Hk)), rest = (int)(u - (long long)i * 2 * Hk);
    const int s = __ldg(src + i), d = __ldg(dst + i);
    if (s < 0 || s >= num_pages || d < 0 || d >= num_pages) {
      if (lane == 0) set_status(status, SA_ERR_BAD_PAGE);
      continue;
    }
    uint4* pool = rest < Hk ? k_pool : v_pool;
    const int h = rest < Hk ? rest : rest - Hk;
    const uint4* from = pool + ((size_t)s * Hk + h) * kSlab + lane;
    uint4* to = pool + ((size_t)d * Hk + h) * kSlab + lane;
    uint4 x[kSlab / 32];
#pragma unroll
    for (int k = 0; k < kSlab / 32; ++k) x[k] = __ldcs(from + 32 * k);
#pragma unroll
    for (int k = 0; k < kSlab / 32; ++k) __stcs(to + 32 * k, x[k]);
  }
}

// One block a (KV head, sequence): all rows of the path are in registers
// before the first is written.
__global__ void __launch_bounds__(kThreads)
accept_rows_kernel(uint4* k_pool, uint4* v_pool, const int* __restrict__ page_table, const int* __restrict__ base_lens,
                   const int* __restrict__ path, int max_path, const int* __restrict__ path_cnt, int Hk, int mpp,
                   int num_pages, int* status) {
  constexpr int kChunks = kD * 2 / 16;                              // of a row
  constexpr int kEach = kMaxTree * kChunks * 2 / kThreads;          // of a thread, K and V
  pdl_wait();
  pdl_trigger();
  const int kvh = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int base = base_lens[b], cnt = path_cnt[b];
  const int* pt = page_table + (size_t)b * mpp;
  int error = SA_OK;
  if (cnt < 0 || cnt > max_path || base < 0 || base > mpp * kP - cnt) error = SA_ERR_INVALID_ARG;
  if (cnt == 0 || error != SA_OK) {
    if (error != SA_OK && tid == 0) set_status(status, error);
    return;
  }
  // row offsets in the pools, in 16-byte chunks
  __shared__ long long s_from[kMaxTree], s_to[kMaxTree];
  if (tid < cnt) {
    const int node = path[(size_t)b * max_path + tid];
    const int to = base + tid;
    if (node < 0 || node >= mpp * kP - base) {
      error = SA_ERR_INVALID_ARG;
    } else {
      const int from = base + node;
      const int pf = __ldg(pt + from / kP), pd = __ldg(pt + to / kP);
      if (pf < 0 || pf >= num_pages || pd < 0 || pd >= num_pages) error = SA_ERR_BAD_PAGE;
      s_from[tid] = (((long long)pf * Hk + kvh) * kP + from % kP) * kChunks;
      s_to[tid] = (((long long)pd * Hk + kvh) * kP + to % kP) * kChunks;
    }
    if (error != SA_OK) set_status(status, error);
  }
  if (__syncthreads_or(error != SA_OK)) return;
  uint4 x[kEach];
  const int rows = 2 * cnt;       // K rows, then V rows
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = e * (kThreads / kChunks) + tid / kChunks;
    if (i < rows) x[e] = (i < cnt ? k_pool : v_pool)[s_from[i < cnt ? i : i - cnt] + tid % kChunks];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = e * (kThreads / kChunks) + tid / kChunks;
    if (i < rows) (i < cnt ? k_pool : v_pool)[s_to[i < cnt ? i : i - cnt] + tid % kChunks] = x[e];
  }
}

}  // namespace

int launch_plan_pages(const PageArgs& A, cudaStream_t stream) { return launch_table<true>(A, stream); }
int launch_compact_pages(const PageArgs& A, cudaStream_t stream) { return launch_table<false>(A, stream); }

int launch_copy_pages(void* k_pool, void* v_pool, const int* src, const int* dst, const int* count, int max_pages,
                      int num_pages, int Hk, int* status, int num_sms, cudaStream_t stream) {
  const long long units = (long long)max_pages * 2 * Hk;
  const int grid = (int)std::min<long long>((units + kThreads / 32 - 1) / (kThreads / 32), (long long)num_sms * 8);
  const cudaError_t e =
      launch_pdl(copy_pages_kernel, dim3(grid), dim3(kThreads), 0, stream, static_cast<uint4*>(k_pool),
                 static_cast<uint4*>(v_pool), src, dst, count, max_pages, num_pages, Hk, status);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

int launch_accept_rows(void* k_pool, void* v_pool, const int* page_table, const int* base_lens, const int* path,
                       int max_path, const int* path_cnt, int B, int Hk, int mpp, int num_pages, int* status,
                       cudaStream_t stream) {
  const cudaError_t e = launch_pdl(accept_rows_kernel, dim3(Hk, B), dim3(kThreads), 0, stream,
                                   static_cast<uint4*>(k_pool), static_cast<uint4*>(v_pool), page_table, base_lens,
                                   path, max_path, path_cnt, Hk, mpp, num_pages, status);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace sa
