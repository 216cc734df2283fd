// What neighbouring sequences hold in the same pages (sa_shared_prefixes).
//
// A group's prefix is the longest run of leading table entries that every
// member with rows has in common, in whole pages ahead of all their rows.  It
// is found from the table alone: pages have no other owner than its rows, so
// equal entries are the same tokens.
//
// A cluster of eight blocks takes a group: each block compares some members'
// entries with the first member's, a stretch of pages at a time, and keeps the
// first place where one differs; the eight answers are joined through
// distributed shared memory.  A stretch behind a difference is not read.
// Bound by the latency of its reads: offsets and lengths, then entries, then
// the exchange.
#include <cooperative_groups.h>

#include <climits>

#include "rows.cuh"

namespace sa {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8, kThreads = 256, kStretch = 8;   // entries a thread has in flight

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
shared_prefixes_kernel(const int* table, const int* seq_lens, const int* row_offsets, const int* group_offsets,
                       int n_groups, int min_tokens, int* members, int* prefix_lens, int B, int mpp, int num_pages,
                       int* status) {
  __shared__ int s_first, s_with, s_pages, s_answer, s_begin, s_end;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = (int)cluster.block_rank(), g = blockIdx.x / kCluster;
  pdl_wait();
  pdl_trigger();
  if (tid == 0) {
    s_first = INT_MAX;
    s_with = 0;
    s_pages = mpp;
    s_begin = s_end = 0;
  }
  __syncthreads();
  // A group begins where those before it have ended, whatever its offset says: a
  // sequence has one group, and one cluster that writes its answer.
  auto offset = [&](int i) { return min(max(__ldg(group_offsets + i), 0), B); };
  if (g < n_groups) {
    for (int i = tid; i <= g + 1; i += kThreads) {
      const int x = offset(i);
      if (i <= g) atomicMax(&s_begin, x);
      else s_end = x;
    }
  } else {   // the cluster behind the last group: sequences of none, before and behind all groups
    for (int i = tid; i <= n_groups; i += kThreads) atomicMax(&s_end, offset(i));
    __syncthreads();
    const int lo = n_groups > 0 ? offset(0) : B, hi = n_groups > 0 ? s_end : B;
    for (int b = rank * kThreads + tid; b < B; b += kCluster * kThreads) {
      if (b >= lo && b < hi) continue;
      // its errors are recorded too, by plain comparisons: of row_seq with a constant number of rows and no other use,
      // nvcc 13.0 makes a test that is always true (max(y, max(x, 0)) != y alone does it)
      const int o0 = __ldg(row_offsets + b), o1 = __ldg(row_offsets + b + 1);
      if (o0 < 0 || o1 < o0) set_status(status, SA_ERR_INVALID_ARG);
      if (__ldg(seq_lens + b) > mpp * kP) set_status(status, SA_ERR_CAPACITY);
      members[b] = 0;
      prefix_lens[b] = 0;
    }
    return;   // all of the cluster
  }
  __syncthreads();
  const int b0 = s_begin, b1 = max(s_end, b0);
  if (rank == 0 && tid == 0 && (b0 != __ldg(group_offsets + g) || b1 != __ldg(group_offsets + g + 1)))
    set_status(status, SA_ERR_INVALID_ARG);
  // the first member with rows, how many have some, and the whole pages ahead of all their rows
  for (int b = b0 + tid; b < b1; b += kThreads) {
    const RowSeq s = row_seq(row_offsets, seq_lens, b, INT_MAX, mpp, rank == 0 ? status : nullptr);
    if (s.n == 0) continue;
    atomicMin(&s_first, b);
    atomicAdd(&s_with, 1);
    atomicMin(&s_pages, max(s.a, 0) / kP);
  }
  __syncthreads();
  const int first = s_first;
  const int most = s_with > 1 ? s_pages : 0;
  __syncthreads();
  // s_pages becomes the first place at which a member of this block differs
  if (first < b1) {
    const int* mine = table + (size_t)first * mpp;
    for (int b = first + rank; b < b1; b += kCluster) {
      if (__ldg(row_offsets + b + 1) <= max(__ldg(row_offsets + b), 0)) continue;
      const int* theirs = table + (size_t)b * mpp;
      for (int j0 = 0; j0 < most; j0 += kStretch * kThreads) {
        if (j0 >= *(volatile int*)&s_pages) break;
        int x[kStretch], y[kStretch];
#pragma unroll
        for (int e = 0; e < kStretch; ++e) {
          const int j = j0 + e * kThreads + tid;
          x[e] = j < most ? __ldg(mine + j) : 0;
          y[e] = j < most ? __ldg(theirs + j) : 0;
        }
#pragma unroll
        for (int e = kStretch - 1; e >= 0; --e)
          if (x[e] != y[e] || x[e] < 0 || x[e] >= num_pages) atomicMin(&s_pages, j0 + e * kThreads + tid);
      }
    }
  }
  __syncthreads();
  if (tid == 0) s_answer = min(most, s_pages);
  cluster.sync();
  int pages = most;
#pragma unroll
  for (int r = 0; r < kCluster; ++r) pages = min(pages, *cluster.map_shared_rank(&s_answer, r));
  const int prefix = pages * kP >= min_tokens ? pages * kP : 0;
  for (int b = b0 + rank * kThreads + tid; b < b1; b += kCluster * kThreads) {
    members[b] = b == first && prefix > 0 ? b1 - first : 0;
    prefix_lens[b] = prefix;
  }
  cluster.sync();   // the others' answers are there until all have read them
}

}  // namespace

int launch_shared_prefixes(const int* table, const int* seq_lens, const int* row_offsets, const int* group_offsets,
                           int n_groups, int min_tokens, int* members, int* prefix_lens, int B, int mpp, int num_pages,
                           int* status, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(shared_prefixes_kernel, dim3((n_groups + 1) * kCluster), dim3(kThreads), 0, stream,
                                   table, seq_lens, row_offsets, group_offsets, n_groups, min_tokens, members,
                                   prefix_lens, B, mpp, num_pages, status);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace sa
