// Selected blocks of packed rows (sa_select_rows): what sa_select_topk selects
// for a sequence, for each of its newest rows as if the cache ended there.
//
// Scores are in the canonical fp32 order (8 lanes of 16 dims, each lane summed
// upwards, lanes joined 4, 2 and 1 apart), so a row's list is the one that a
// decode step of its length writes, bit for bit.
//
// A block takes an item, one KV head with 32 / G neighbouring rows of a
// sequence (up to 32 rows and heads), scores 64 candidate blocks at a time
// from shared memory, four rows by two blocks a thread, and leaves the scores
// in a scratch of its own; then a warp a row finds the k-th score by halving
// the range of keys and writes the list in order.
#include "rows.cuh"
#include "topk.cuh"

namespace sa {
namespace {

constexpr int kSelThreads = 256, kSelRows = 32, kSelBlocks = 64;
constexpr int kPad = 16;                              // bytes behind a row in shared memory: no bank is hit twice
constexpr int kRowStride = kD * 2 + kPad;

// Candidate blocks [j0, j1) of a row at position pos.
__device__ __forceinline__ void row_candidates(const SelectArgs& A, int pos, int size, int& j0, int& j1) {
  candidate_range(pos + 1, A.S, A.W, size, j0, j1);
  j1 = min(j1, (A.mpp * kP + size - 1) / size);
}

// The sum of 128 products in the canonical order.
template <bool MINMAX>
__device__ __forceinline__ void score_tile(const uint8_t* s_q, const uint8_t* s_lo, const uint8_t* s_hi, int r0, int c0,
                                           float (&out)[4][2]) {
  float quad[4][2], pair[4][2];
#pragma unroll
  for (int step = 0; step < 8; ++step) {
    // lanes 0 4 2 6 1 5 3 7: (0 + 4) + (2 + 6), then (1 + 5) + (3 + 7)
    constexpr int kOrder[8] = {0, 4, 2, 6, 1, 5, 3, 7};
    const int part = kOrder[step];
    float acc[4][2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint4 q[4], lo[2], hi[2];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        q[r] = *reinterpret_cast<const uint4*>(s_q + (r0 + r) * kRowStride + part * 32 + half * 16);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        hi[c] = *reinterpret_cast<const uint4*>(s_hi + (c0 + 32 * c) * kRowStride + part * 32 + half * 16);
        if (MINMAX) lo[c] = *reinterpret_cast<const uint4*>(s_lo + (c0 + 32 * c) * kRowStride + part * 32 + half * 16);
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t x = reinterpret_cast<const uint32_t*>(&q[r])[w];
          uint32_t sel = 0;
          if (MINMAX)
            sel = (bf16_lo(x) >= 0.f ? 0x10u : 0x54u) | (bf16_hi(x) >= 0.f ? 0x3200u : 0x7600u);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t y = reinterpret_cast<const uint32_t*>(&hi[c])[w];
            if (MINMAX) y = __byte_perm(y, reinterpret_cast<const uint32_t*>(&lo[c])[w], sel);
            float a = half == 0 && w == 0 ? -0.0f : acc[r][c];
            a = fma_bf16_lo(x, y, a);
            acc[r][c] = fma_bf16_hi(x, y, a);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float a = acc[r][c];
        if (step == 0 || step == 2 || step == 4 || step == 6) {
          if (step == 0 || step == 4) pair[r][c] = a;
          else out[r][c] = a;
        } else if (step == 1 || step == 5) {
          pair[r][c] = __fadd_rn(pair[r][c], a);
        } else {
          const float four = __fadd_rn(pair[r][c], __fadd_rn(out[r][c], a));
          if (step == 3) quad[r][c] = four;
          else out[r][c] = __fadd_rn(__fadd_rn(quad[r][c], four), 0.0f);
        }
      }
    }
  }
}

template <bool MINMAX>
__global__ void __launch_bounds__(kSelThreads) select_rows_kernel(SelectArgs A) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* s_q = smem;
  uint8_t* s_hi = smem + kSelRows * kRowStride;
  uint8_t* s_lo = s_hi + kSelBlocks * kRowStride;
  __shared__ ItemPlace s_place;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  float* scratch = A.scores + (size_t)blockIdx.x * kSelRows * A.slots;
  const int T = kSelRows / A.G;
  for (int u = blockIdx.x; u < A.n_items; u += gridDim.x) {
    find_item<kSelThreads>(A.row_offsets, A.seq_lens, A.B, A.n_rows, A.mpp, A.Hk, T, u, A.status, &s_place);
    const ItemPlace at = s_place;
    if (at.b < 0) return;
    const RowSeq s = row_seq(A.row_offsets, A.seq_lens, at.b, A.n_rows, A.mpp, nullptr);
    const int tokens = min(T, s.n - at.i * T), row0 = s.row0 + at.i * T, pos0 = s.a + at.i * T, rows = tokens * A.G;
    const int size = A.bs[at.kvh], h0 = at.kvh * A.G;
    int j0, j1, first0, first1;
    row_candidates(A, pos0 + tokens - 1, size, j0, j1);       // the last row has the most, and the first ones
    row_candidates(A, pos0, size, first0, first1);
    if (first1 > first0) j0 = min(j0, first0);
    bool all = true;                                          // every head keeps every candidate
    for (int g = 0; g < A.G; ++g) all &= A.k[h0 + g] >= j1 - j0;
    if (!all) {
      for (int x = tid; x < kSelRows * (kD / 8); x += kSelThreads) {
        const int r = x / (kD / 8), d = x % (kD / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < rows)
          v = reinterpret_cast<const uint4*>(A.q + ((size_t)(row0 + r / A.G) * A.Hq + h0 + r % A.G) * kD)[d];
        *reinterpret_cast<uint4*>(s_q + r * kRowStride + d * 16) = v;
      }
      const uint4* summ = reinterpret_cast<const uint4*>(A.summaries) +
                          ((size_t)at.b * A.Hk + at.kvh) * A.slots * (MINMAX ? 2 : 1) * (kD / 8);
      for (int c0 = j0; c0 < j1; c0 += kSelBlocks) {
        __syncthreads();
        for (int x = tid; x < kSelBlocks * (MINMAX ? 2 : 1) * (kD / 8); x += kSelThreads) {
          const int d = x % (kD / 8), y = x / (kD / 8), c = MINMAX ? y >> 1 : y;
          const bool low = MINMAX && (y & 1) == 0;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (c0 + c < j1) v = __ldg(summ + ((size_t)(c0 + c) * (MINMAX ? 2 : 1) + (MINMAX ? y & 1 : 0)) * (kD / 8) + d);
          *reinterpret_cast<uint4*>((low ? s_lo : s_hi) + c * kRowStride + d * 16) = v;
        }
        __syncthreads();
        float z[4][2];
        score_tile<MINMAX>(s_q, s_lo, s_hi, 4 * warp, lane, z);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (c0 + lane + 32 * c < j1) scratch[(size_t)(4 * warp + r) * A.slots + c0 + lane + 32 * c] = z[r][c];
        }
      }
      __syncthreads();
    }
    // a warp a row and head (of a group that selects together: a row)
    const int lists = A.group ? tokens : rows;
    for (int x = warp; x < lists; x += kSelThreads / 32) {
      const int tok = A.group ? x : x / A.G, g = A.group ? 0 : x % A.G;
      int c0, c1;
      row_candidates(A, pos0 + tok, size, c0, c1);
      const int n = c1 - c0, k = min(A.k[h0 + g], n), copies = A.group ? A.G : 1;
      const size_t row = (size_t)(row0 + tok) * A.Hq + h0 + g;
      int* list = A.sel_idx + row * A.kcap;
      if (lane < copies) A.sel_cnt[row + lane] = k;
      if (k == 0) continue;
      if (k == n) {
        for (int j = lane; j < n; j += 32)
          for (int y = 0; y < copies; ++y) list[(size_t)y * A.kcap + j] = c0 + j;
        continue;
      }
      const float* z = scratch + (size_t)(tok * A.G + g) * A.slots + c0;
      auto key = [&](int j) -> uint32_t {
        float v = z[j];
        for (int y = 1; y < copies; ++y) v = __fadd_rn(v, z[(size_t)y * A.slots + j]);
        return order_key(v);
      };
      // the largest key that at least k candidates reach
      uint32_t top = 0;
      int reach = n;
      for (int bit = 31; bit >= 0 && reach != k; --bit) {
        const uint32_t t = top | 1u << bit;
        int m = 0;
        for (int j = lane; j < n; j += 32) m += key(j) >= t;
        m = __reduce_add_sync(0xffffffffu, m);
        if (m >= k) {
          top = t;
          reach = m;
        }
      }
      // those above it, and as many equal to it as there is room for (reach == k: all of them)
      int above = 0;
      if (reach != k) {
        for (int j = lane; j < n; j += 32) above += key(j) > top;
        above = __reduce_add_sync(0xffffffffu, above);
      }
      int ties = reach == k ? n : k - above, out = 0;
      for (int j = lane; j - lane < n; j += 32) {
        const uint32_t v = j < n ? key(j) : 0;
        const bool more = j < n && v > top, even = j < n && v == top;
        const unsigned tie = __ballot_sync(0xffffffffu, even), below = (1u << lane) - 1u;
        const bool take = more || (even && __popc(tie & below) < ties);
        ties -= min(ties, __popc(tie));
        const unsigned m = __ballot_sync(0xffffffffu, take);
        if (take)
          for (int y = 0; y < copies; ++y) list[(size_t)y * A.kcap + out + __popc(m & below)] = c0 + j;
        out += __popc(m);
      }
    }
    __syncthreads();
  }
}

}  // namespace

int select_rows_blocks(int num_sms) { return 2 * num_sms; }
int select_rows_scratch_rows() { return kSelRows; }

int launch_select_rows(const SelectArgs& A, int num_sms, cudaStream_t stream) {
  const int smem = (kSelRows + (A.minmax ? 2 : 1) * kSelBlocks) * kRowStride;
  auto* kernel = A.minmax ? select_rows_kernel<true> : select_rows_kernel<false>;
  if (smem_limit_at_least(reinterpret_cast<const void*>(kernel), smem) != cudaSuccess) return SA_ERR_CUDA;
  const int grid = A.n_items < select_rows_blocks(num_sms) ? A.n_items : select_rows_blocks(num_sms);
  const cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(kSelThreads), (size_t)smem, stream, A);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace sa
