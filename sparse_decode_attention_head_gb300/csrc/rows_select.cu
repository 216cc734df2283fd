// Selected blocks of packed rows (sa_select_rows): what sa_select_topk selects
// for a sequence, for each of its newest rows as if the cache ended there.
//
// Scores are in the canonical fp32 order (8 lanes of 16 dims, each lane summed
// upwards, lanes joined 4, 2 and 1 apart), so a row's list is the one that a
// decode step of its length writes, bit for bit.
//
// This form scores on the CUDA cores: drafts and single tokens, whose few rows
// under a KV head leave the summaries' bytes as the bound, and caches with more
// candidates than rows_select_tc.cu takes.  A block scores 32 rows and heads
// (an item) against a stretch of blocks, 64 at a time from shared memory, four
// rows by two blocks a thread; a second kernel has a block a list for the top-k.
// Scores go through a scratch; items are taken in runs that fit it.
#include "rows_select.cuh"

namespace sa {
namespace {

constexpr int kSelThreads = 256, kSelRows = 32, kSelBlocks = 64, kSelStretch = 256;
constexpr int kPad = 16;                              // bytes behind a row in shared memory: no bank is hit twice
constexpr int kRowStride = kD * 2 + kPad;
constexpr size_t kScratchBytes = 256u << 20;          // at least one item

// Byte selectors of two dims for max where q >= 0 and min elsewhere, as __byte_perm(max, min, .) takes them.
__device__ __forceinline__ uint32_t selectors(uint32_t q) {
  return (bf16_lo(q) >= 0.f ? 0x10u : 0x54u) | (bf16_hi(q) >= 0.f ? 0x3200u : 0x7600u);
}

// Four rows against two blocks, the sums of 128 products in the canonical
// order.  The loop over lanes is kept a loop: all of it at once is 48 KB of
// instructions.
template <bool MINMAX>
__device__ __forceinline__ void score_tile(const uint8_t* s_q, const uint8_t* s_sel, const uint8_t* s_lo,
                                           const uint8_t* s_hi, int r0, int c0, float (&out)[4][2]) {
  auto lane_sum = [&](int part, float (&acc)[4][2]) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int at = part * 32 + half * 16;
      uint4 q[4], sel[4], lo[2], hi[2];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        q[r] = *reinterpret_cast<const uint4*>(s_q + (r0 + r) * kRowStride + at);
        if (MINMAX) sel[r] = *reinterpret_cast<const uint4*>(s_sel + (r0 + r) * kRowStride + at);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        hi[c] = *reinterpret_cast<const uint4*>(s_hi + (c0 + 32 * c) * kRowStride + at);
        if (MINMAX) lo[c] = *reinterpret_cast<const uint4*>(s_lo + (c0 + 32 * c) * kRowStride + at);
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t x = (&q[r].x)[w];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t y = MINMAX ? __byte_perm((&hi[c].x)[w], (&lo[c].x)[w], (&sel[r].x)[w]) : (&hi[c].x)[w];
            const float a = fma_bf16_lo(x, y, half == 0 && w == 0 ? -0.0f : acc[r][c]);
            acc[r][c] = fma_bf16_hi(x, y, a);
          }
        }
      }
    }
  };
  float first[4][2], quad[4][2];
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {        // lanes 0 and 4, 2 and 6; 1 and 5, 3 and 7
    const int part = (i & 1) * 2 + (i >> 1);
    float a[4][2], b[4][2];
    lane_sum(part, a);
    lane_sum(part + 4, b);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float x = __fadd_rn(a[r][c], b[r][c]);
        if ((i & 1) == 0) {
          first[r][c] = x;
        } else {
          const float four = __fadd_rn(first[r][c], x);
          if (i == 1) quad[r][c] = four;
          else out[r][c] = __fadd_rn(__fadd_rn(quad[r][c], four), 0.0f);
        }
      }
    }
  }
}

template <bool MINMAX>
__global__ void __launch_bounds__(kSelThreads, 2) score_rows_kernel(SelectArgs A, int u0) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* s_q = smem;
  uint8_t* s_sel = s_q + kSelRows * kRowStride;
  uint8_t* s_hi = s_sel + (MINMAX ? kSelRows * kRowStride : 0);
  uint8_t* s_lo = s_hi + kSelBlocks * kRowStride;
  __shared__ ItemPlace s_place;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  SelectItem it;
  if (!select_item<kSelThreads>(A, kSelRows / A.G, u0 + blockIdx.x, &s_place, it)) return;
  int j0, j1;
  if (item_candidates(A, it.kvh, it.pos0 + it.tokens - 1, j0, j1)) return;
  const int from = j0 + blockIdx.y * kSelStretch, to = min(j1, from + kSelStretch);
  if (from >= to) return;
  const int h0 = it.kvh * A.G;
  for (int x = tid; x < kSelRows * (kD / 8); x += kSelThreads) {
    const int r = x / (kD / 8), d = x % (kD / 8);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < it.tokens * A.G)
      v = reinterpret_cast<const uint4*>(A.q + ((size_t)(it.row0 + r / A.G) * A.Hq + h0 + r % A.G) * kD)[d];
    *reinterpret_cast<uint4*>(s_q + r * kRowStride + d * 16) = v;
    if (MINMAX)
      *reinterpret_cast<uint4*>(s_sel + r * kRowStride + d * 16) =
          make_uint4(selectors(v.x), selectors(v.y), selectors(v.z), selectors(v.w));
  }
  constexpr int kVecs = (MINMAX ? 2 : 1) * (kD / 8);     // 16-byte pieces of a block's summary
  const uint4* summ = reinterpret_cast<const uint4*>(A.summaries) + ((size_t)it.b * A.Hk + it.kvh) * A.slots * kVecs;
  float* scratch = A.scores + (size_t)blockIdx.x * kSelRows * A.slots;
  // a tile's summaries while the one before is scored
  constexpr int kEach = kSelBlocks * kVecs / kSelThreads;
  uint4 next[kEach];
  auto fetch = [&](int c0) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int x = e * kSelThreads + tid;
      next[e] = c0 + x / kVecs < to ? __ldg(summ + (size_t)c0 * kVecs + x) : make_uint4(0, 0, 0, 0);
    }
  };
  fetch(from);
  for (int c0 = from; c0 < to; c0 += kSelBlocks) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int x = e * kSelThreads + tid, d = x % (kD / 8), y = x / (kD / 8), c = MINMAX ? y >> 1 : y;
      *reinterpret_cast<uint4*>((MINMAX && (y & 1) == 0 ? s_lo : s_hi) + c * kRowStride + d * 16) = next[e];
    }
    __syncthreads();
    if (c0 + kSelBlocks < to) fetch(c0 + kSelBlocks);
    float z[4][2];
    score_tile<MINMAX>(s_q, s_sel, s_lo, s_hi, 4 * warp, lane, z);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (c0 + lane + 32 * c < to) scratch[(size_t)(4 * warp + r) * A.slots + c0 + lane + 32 * c] = z[r][c];
    }
  }
}

// A block a row and head (of a group that selects together: a row).
template <int THREADS, int KEYS>
__global__ void __launch_bounds__(THREADS) topk_rows_kernel(SelectArgs A, int u0) {
  __shared__ TopkScratch S;
  __shared__ ItemPlace s_place;
  pdl_wait();
  pdl_trigger();
  SelectItem it;
  if (!select_item<THREADS>(A, kSelRows / A.G, u0 + blockIdx.x, &s_place, it)) return;
  const int tok = A.group ? blockIdx.y : blockIdx.y / A.G, g = A.group ? 0 : blockIdx.y % A.G;
  if (tok >= it.tokens) return;
  int c0, c1;
  row_candidates(A, it.pos0 + tok, A.bs[it.kvh], c0, c1);
  const int h = it.kvh * A.G + g;
  const size_t row = (size_t)(it.row0 + tok) * A.Hq + h;
  const float* z = A.scores + ((size_t)blockIdx.x * kSelRows + tok * A.G + g) * A.slots + c0;
  int *list = A.sel_idx + row * A.kcap, *cnt = A.sel_cnt + row;
  if (!A.group) {
    group_topk<THREADS, KEYS>(z, c1 - c0, A.k[h], c0, list, cnt, 0, S);
    return;
  }
  group_topk<THREADS, KEYS, true>(z, c1 - c0, A.k[h], c0, list, cnt, 0, S, A.G, (size_t)A.slots);
  __syncthreads();
  const int n = *cnt;
  for (int y = 1; y < A.G; ++y) {
    for (int i = threadIdx.x; i < n; i += THREADS) list[(size_t)y * A.kcap + i] = list[i];
    if (threadIdx.x == 0) cnt[y] = n;
  }
}

long long items_at_a_time(int slots, int n_items) {
  const long long fit = (long long)(kScratchBytes / ((size_t)kSelRows * slots * sizeof(float)));
  return std::max(1ll, std::min({fit, (long long)n_items, 65535ll}));
}

}  // namespace

size_t score_rows_scratch(int slots, long long n_items) {
  return (size_t)items_at_a_time(slots, (int)std::min(n_items, 1ll << 30)) * kSelRows * slots * sizeof(float);
}

int launch_score_rows(const SelectArgs& A, int max_candidates, cudaStream_t stream) {
  const int smem = (A.minmax ? 2 : 1) * (kSelRows + kSelBlocks) * kRowStride;
  auto* score = A.minmax ? score_rows_kernel<true> : score_rows_kernel<false>;
  if (smem_limit_at_least(reinterpret_cast<const void*>(score), smem) != cudaSuccess) return SA_ERR_CUDA;
  const int at_a_time = (int)items_at_a_time(A.slots, A.n_items), T = kSelRows / A.G;
  const int stretches = std::max(1, (max_candidates + kSelStretch - 1) / kSelStretch);
  for (int u0 = 0; u0 < A.n_items; u0 += at_a_time) {
    const int n = std::min(at_a_time, A.n_items - u0);
    cudaError_t e =
        launch_pdl(score, dim3(n, stretches), dim3(kSelThreads), (size_t)smem, stream, A, u0);
    if (e != cudaSuccess) return SA_ERR_CUDA;
    const dim3 lists(n, A.group ? T : T * A.G);
    // the smallest block that holds every candidate
    if (max_candidates <= 128 * 8)
      e = launch_pdl(topk_rows_kernel<128, 8>, lists, dim3(128), 0, stream, A, u0);
    else if (max_candidates <= 256 * 8)
      e = launch_pdl(topk_rows_kernel<256, 8>, lists, dim3(256), 0, stream, A, u0);
    else if (max_candidates <= 256 * 16)
      e = launch_pdl(topk_rows_kernel<256, 16>, lists, dim3(256), 0, stream, A, u0);
    else if (max_candidates <= 1024 * 16)
      e = launch_pdl(topk_rows_kernel<1024, 16>, lists, dim3(1024), 0, stream, A, u0);
    else
      e = launch_pdl(topk_rows_kernel<1024, 64>, lists, dim3(1024), 0, stream, A, u0);
    if (e != cudaSuccess) return SA_ERR_CUDA;
  }
  return SA_OK;
}

}  // namespace sa
