// What the two forms of the selection of packed rows share: candidates, the
// canonical score of one block, and a warp's top-k from scores in memory.
#pragma once

#include "rows.cuh"
#include "topk.cuh"

namespace sa {

// Candidate blocks [j0, j1) of a row at position pos, j0 <= j1.  Every row with
// some has the same j0.  A row ahead of the cache (pos < 0) has none: its length
// less a window near 2^31 would be no int32.  Nor has one whose sinks reach
// behind the table.
__device__ __forceinline__ void row_candidates(const SelectArgs& A, int pos, int size, int& j0, int& j1) {
  candidate_range(max(pos + 1, 0), A.S, A.W, size, j0, j1);
  j1 = max(j0, min(j1, (A.mpp * kP + size - 1) / size));
}

// Candidates [j0, j1) of an item's rows together, the last of them at position
// last; `all`: every head keeps every one.
__device__ __forceinline__ bool item_candidates(const SelectArgs& A, int kvh, int last, int& j0, int& j1) {
  row_candidates(A, last, A.bs[kvh], j0, j1);
  bool all = true;
  for (int g = 0; g < A.G; ++g) all &= A.k[kvh * A.G + g] >= j1 - j0;
  return all;
}

// An item's rows: T of a sequence's rows, under one KV head.
struct SelectItem {
  int b, kvh, tokens, row0, pos0;
};
template <int THREADS>
__device__ __forceinline__ bool select_item(const SelectArgs& A, int T, int u, ItemPlace* place, SelectItem& it) {
  find_item<THREADS>(A.row_offsets, A.seq_lens, A.B, A.n_rows, A.mpp, A.Hk, T, u, A.status, place);
  const ItemPlace at = *place;
  if (at.b < 0) return false;
  const RowSeq s = row_seq(A.row_offsets, A.seq_lens, at.b, A.n_rows, A.mpp, nullptr);
  it.b = at.b;
  it.kvh = at.kvh;
  it.tokens = min(T, s.n - at.i * T);
  it.row0 = s.row0 + at.i * T;
  it.pos0 = s.a + at.i * T;
  return true;
}

// The canonical score of one summary by eight lanes (part 0 .. 7 of them), the
// same in all eight.
template <bool MINMAX>
__device__ __forceinline__ float canonical_score(const __nv_bfloat16* q, const __nv_bfloat16* summary, int part) {
  const uint4* qp = reinterpret_cast<const uint4*>(q) + 2 * part;
  const uint4* lo = reinterpret_cast<const uint4*>(summary) + 2 * part;      // min (or mean)
  const uint4* hi = lo + (MINMAX ? kD / 8 : 0);
  float acc = -0.0f;       // fma with c = -0 is the plain product
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 x = __ldg(qp + h), a = MINMAX ? __ldg(lo + h) : make_uint4(0, 0, 0, 0), b = __ldg(hi + h);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t xw = (&x.x)[w];
      uint32_t y = (&b.x)[w];
      if (MINMAX)
        y = __byte_perm(y, (&a.x)[w], (bf16_lo(xw) >= 0.f ? 0x10u : 0x54u) | (bf16_hi(xw) >= 0.f ? 0x3200u : 0x7600u));
      acc = fma_bf16_lo(xw, y, acc);
      acc = fma_bf16_hi(xw, y, acc);
    }
  }
  acc = __fadd_rn(acc, __shfl_xor_sync(0xffffffffu, acc, 4));
  acc = __fadd_rn(acc, __shfl_xor_sync(0xffffffffu, acc, 2));
  acc = __fadd_rn(acc, __shfl_xor_sync(0xffffffffu, acc, 1));
  return __fadd_rn(acc, 0.0f);
}

// A warp: the k of n keys (0 < k < n) that are largest, the lowest index first
// among equals; their indices, base added, ascending to `copies` lists kcap apart.
template <typename Key>
__device__ __forceinline__ void warp_topk(Key key, int n, int k, int base, int* list, int copies, int kcap) {
  const int lane = threadIdx.x & 31;
  uint32_t top = 0;            // the largest key that at least k reach
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
  int ties = n;                // of those equal to it, as many as there is room for
  if (reach != k) {
    int above = 0;
    for (int j = lane; j < n; j += 32) above += key(j) > top;
    ties = k - __reduce_add_sync(0xffffffffu, above);
  }
  int out = 0;
  for (int j = lane; j - lane < n; j += 32) {
    const uint32_t v = j < n ? key(j) : 0;
    const bool more = j < n && v > top, even = j < n && v == top;
    const unsigned tie = __ballot_sync(0xffffffffu, even), below = (1u << lane) - 1u;
    const bool take = more || (even && __popc(tie & below) < ties);
    ties -= min(ties, __popc(tie));
    const unsigned m = __ballot_sync(0xffffffffu, take);
    if (take)
      for (int y = 0; y < copies; ++y) list[(size_t)y * kcap + out + __popc(m & below)] = base + j;
    out += __popc(m);
  }
}

}  // namespace sa
