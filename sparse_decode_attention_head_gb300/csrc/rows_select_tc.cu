// Selected blocks of many rows (sa_select_rows): scores on the tensor cores
// find the selection, scores in the canonical order decide where they are close.
//
// The canonical fp32 order of a score is no order that a matrix instruction
// has, so what the tensor cores give is taken as a value a with
//   |a - s| <= E = 2^-14 |q| max_j |k_j|      (norms of q and of max(|min|, |max|))
// of the canonical s.  A matrix product of 256 terms in steps of 16 adds, a
// step, 17 numbers cut to 24 bits of the largest (2^-23 of it each at most);
// none is above sum |q k| <= |q| |k|, so 16 steps are off by at most
// 16 * 17 * 2^-23 |q| |k| < 2^-14.9 |q| |k|, and the canonical sum by less than
// 2^-19.  A candidate that is more than 2 E above the best one left out is
// selected whatever the order; one that is more than 2 E below the worst one
// taken is not; those between (in one row out of six or so) are scored again in
// the canonical order, and the best of them, lowest index first among equals,
// fill the list.  So lists are the canonical ones, entry for entry.  A row with
// more close ones than kClose, or without a bound (infinities), is scored
// again as a whole.
//
// q . min/max summary: sum over d of q+_d kmax_d + q-_d kmin_d with q+ and q-
// the positive and negative part, a product of twice the length.
// Heads that select together: a row is a token and the product runs over the
// group's heads too; E is G times that of the sum of their norms.
//
// A block (four warps, two blocks an SM) takes an item: one KV head with 128
// rows (tokens and heads; tokens, for heads that select together) of a sequence, a thread a row.  Scores stay in
// TMEM (up to 256 candidates; more go through a scratch, [candidate][row]).
// The k-th score is found by counting against a threshold that starts where a
// normal distribution has it and follows its density (three to five passes).
// Bound by the passes' instructions: about 20 a candidate and row.
#include <cfloat>

#include "rows_select.cuh"
#include "tcgen.cuh"

namespace sa {
namespace {

constexpr int kThreads = 128, kRows = 128, kCols = 256, kTile = 64;
constexpr int kHalfTile = kRows * 64 * 2, kSummHalf = kTile * 64 * 2;     // 64 dims of q's rows, of a tile of summaries
constexpr int kClose = 8;                                                   // of a row, scored again one by one

template <bool MINMAX>
constexpr size_t kOperands = (MINMAX ? 2 : 1) * (2 * kHalfTile + 2 * kSummHalf);

struct Warp {
  uint16_t close[32][kClose];
  uint16_t task[32 * kClose];
  float score[32 * kClose];
};
struct Ctl {
  Warp warp[kThreads / 32];
  uint64_t q_full, s_full, done;
  uint32_t tmem;
  ItemPlace place;
};
template <bool MINMAX>
constexpr size_t kSmem = 1024 + kOperands<MINMAX> + sizeof(Ctl);
static_assert(2 * (kSmem<true> + 1024) <= 228 * 1024, "two blocks an SM");

// The largest norm of max(|min|, |max|) (of the mean) among a KV head's summaries, as the bits of its square.
template <bool MINMAX>
__global__ void __launch_bounds__(256) summary_norms_kernel(SelectArgs A) {
  pdl_wait();
  pdl_trigger();
  const int unit = blockIdx.x, b = unit / A.Hk, kvh = unit % A.Hk, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const RowSeq s = row_seq(A.row_offsets, A.seq_lens, b, A.n_rows, A.mpp, nullptr);
  if (s.n == 0) return;
  int j0, j1;
  row_candidates(A, s.a + s.n - 1, A.bs[kvh], j0, j1);
  constexpr int kVecs = (MINMAX ? 2 : 1) * (kD / 8);
  const uint4* summ = reinterpret_cast<const uint4*>(A.summaries) + (size_t)unit * A.slots * kVecs;
  float most = 0.f;
  // half a warp a block
  const int part = lane & 15;
  for (int j = j0 + (blockIdx.y * 8 + warp) * 2 + (lane >> 4); j - (lane >> 4) < j1; j += gridDim.y * 16) {
    float sum = 0.f;
    if (j < j1) {
      const uint4 a = __ldg(summ + (size_t)j * kVecs + part);
      const uint4 c = MINMAX ? __ldg(summ + (size_t)j * kVecs + kD / 8 + part) : a;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x = (&a.x)[w], y = (&c.x)[w];
        // of NaN and a number fmaxf takes the number: their sum does not
        const float l0 = fabsf(bf16_lo(x)), l1 = fabsf(bf16_lo(y)), h0 = fabsf(bf16_hi(x)), h1 = fabsf(bf16_hi(y));
        const float lo = l0 > l1 ? l0 : l1, hi = h0 > h1 ? h0 : h1;
        sum = fmaf(lo, lo, sum) + 0.f * l0;
        sum = fmaf(hi, hi, sum) + 0.f * h0;
      }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (!(sum <= most)) most = sum;
    if (isnan(sum)) most = INFINITY;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) atomicMax(A.norms + unit, __float_as_int(most));     // not negative: ordered like its bits
}

// 32 scores of a row from column 32 c on.
template <bool MEMORY>
__device__ __forceinline__ void load32(uint32_t tmem, const float* scratch, int c, float (&v)[32]) {
  if (MEMORY) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = scratch[(size_t)(32 * c + i) * kRows];
  } else {
    tmem_ld32(tmem + 32 * c, v);
  }
}

// A row's list.  Everything is converged by warp; lanes without work pass along.
struct RowTask {
  bool valid;            // has candidates to choose from: 0 < k < n
  int n, k, base;        // candidates, how many to keep, the first one's block
  float E;
  size_t row;            // of the lists
  const __nv_bfloat16* q;
  const __nv_bfloat16* summ;      // of the first candidate
};

template <bool MINMAX>
__device__ __forceinline__ float row_score(const SelectArgs& A, const __nv_bfloat16* q, const __nv_bfloat16* summary,
                                           int part) {
  float v = canonical_score<MINMAX>(q, summary, part);
  if (A.group)
    for (int g = 1; g < A.G; ++g) v = __fadd_rn(v, canonical_score<MINMAX>(q + g * kD, summary, part));
  return v;
}

template <bool MINMAX, bool MEMORY>
__device__ void select_list(const SelectArgs& A, const RowTask& t, uint32_t tmem, const float* scratch, float* keys,
                            Warp* w) {
  constexpr int kSummary = (MINMAX ? 2 : 1) * kD;
  const int lane = threadIdx.x & 31;
  int most = t.valid ? t.n : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (most == 0) return;
  const int chunks = (most + 31) / 32, n = t.valid ? t.n : 0;
  float v[32];
  auto load = [&](int c) {      // columns behind the row's last are -infinity
    load32<MEMORY>(tmem, scratch, c, v);
    if (__any_sync(0xffffffffu, 32 * c + 32 > n)) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 32 * c + i < n ? v[i] : -INFINITY;
    }
  };
  // range, mean and spread
  float lo = INFINITY, hi = -INFINITY, sum = 0.f, sq = 0.f;
  for (int c = 0; c < chunks; ++c) {
    load(c);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float x = v[i] == -INFINITY ? 0.f : v[i];
      sum += x;
      sq = fmaf(x, x, sq);
      hi = fmaxf(hi, v[i]);
      lo = fminf(lo, v[i] == -INFINITY ? INFINITY : v[i]);
    }
  }
  bool whole = t.valid && !(t.E < 1e30f && hi < 1e30f && lo > -1e30f);   // no bound: scored again as a whole
  bool active = t.valid && !whole;
  const float mean = sum / n, sigma = sqrtf(fmaxf(sq / n - mean * mean, 1e-30f));
  hi += fmaxf(t.E, fabsf(hi) * 1e-6f) + 1e-30f;       // none reaches it
  // where a normal distribution has the k-th (Hastings' approximation of its quantile)
  float at;
  {
    const float p = (float)t.k / n, tail = sqrtf(-2.f * logf(fminf(p, 1.f - p)));
    const float z = tail - (2.30753f + 0.27061f * tail) / (1.f + tail * (0.99229f + 0.04481f * tail));
    at = mean + sigma * (p < 0.5f ? z : -z);
    if (!(at > lo && at < hi)) at = 0.5f * (lo + hi);
  }
  // count(>= lo) >= k > count(>= hi)
  bool found = false, search = active;
  for (int step = 0; step < 40 && __any_sync(0xffffffffu, search); ++step) {
    int cnt = 0;
    for (int c = 0; c < chunks; ++c) {
      load(c);
#pragma unroll
      for (int i = 0; i < 32; ++i) cnt += v[i] >= at;
    }
    if (search) {
      if (cnt == t.k) {
        found = true;
        search = false;
      } else {
        if (cnt > t.k) lo = at; else hi = at;
        const float z = (at - mean) / sigma, density = n * 0.3989f * __expf(-0.5f * z * z) / sigma;
        float next = at + (cnt - t.k) / fmaxf(density, 1e-6f / sigma);
        if (step % 3 == 2 || !(next > lo && next < hi)) next = 0.5f * (lo + hi);
        search = hi - lo > t.E && next > lo && next < hi;
        at = next;
      }
    }
  }
  // taken without a look: above `sure`.  Close: from `close_lo` to `sure`.
  float sure = hi + 2.f * t.E, close_lo = lo - 2.f * t.E;
  if (__any_sync(0xffffffffu, found)) {
    float least = INFINITY, best = -INFINITY;          // of those taken, of those left
    for (int c = 0; c < chunks; ++c) {
      load(c);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const bool in = v[i] >= at;
        least = fminf(least, in ? v[i] : INFINITY);
        best = fmaxf(best, in ? -INFINITY : v[i]);
      }
    }
    if (found) {
      const bool apart = least - best > 2.f * t.E;
      sure = apart ? best : best + 2.f * t.E;
      close_lo = apart ? INFINITY : least - 2.f * t.E;
    }
  }
  unsigned chosen = 0;     // of the close ones, in their order
  bool some = active && close_lo < INFINITY;
  if (__any_sync(0xffffffffu, some)) {
    int taken = 0, n_close = 0;
    for (int c = 0; c < chunks; ++c) {
      load(c);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        taken += v[i] > sure;
        if (some && v[i] <= sure && v[i] >= close_lo) {
          if (n_close < kClose) w->close[lane][n_close] = (uint16_t)(32 * c + i);
          ++n_close;
        }
      }
    }
    if (some && n_close > kClose) {
      whole = true;
      some = active = false;
    }
    if (!some) n_close = 0;
    const int upto = warp_incl_scan(n_close), total = __shfl_sync(0xffffffffu, upto, 31), first = upto - n_close;
    for (int i = 0; i < n_close; ++i) w->task[first + i] = (uint16_t)(lane * kClose + i);
    __syncwarp();
    const int part = lane & 7;
    for (int x0 = 0; x0 < total; x0 += 4) {
      const int x = min(x0 + (lane >> 3), total - 1), task = w->task[x], who = task / kClose;
      const size_t row = __shfl_sync(0xffffffffu, (unsigned long long)t.q, who);
      const size_t summ = __shfl_sync(0xffffffffu, (unsigned long long)t.summ, who);
      const float z = row_score<MINMAX>(A, reinterpret_cast<const __nv_bfloat16*>(row),
                                        reinterpret_cast<const __nv_bfloat16*>(summ) +
                                            (size_t)w->close[who][task % kClose] * kSummary, part);
      if (part == 0) w->score[x] = z;
    }
    __syncwarp();
    for (int i = 0; i < n_close; ++i) {
      const float z = w->score[first + i];
      int rank = 0;
      for (int j = 0; j < n_close; ++j) {
        const float o = w->score[first + j];
        rank += o > z || (o == z && j < i);
      }
      if (rank < t.k - taken) chosen |= 1u << i;
    }
  }
  // the list, ascending
  const int copies = A.group ? A.G : 1;
  if (__any_sync(0xffffffffu, active)) {
    int* list = A.sel_idx + t.row * A.kcap;
    int out = 0;
    unsigned left = chosen;
    for (int c = 0; c < chunks; ++c) {
      load(c);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        bool take = active && v[i] > sure;
        if (active && v[i] <= sure && v[i] >= close_lo) {
          take = left & 1u;
          left >>= 1;
        }
        if (take && out < t.k) {
          for (int y = 0; y < copies; ++y) list[(size_t)y * A.kcap + out] = t.base + 32 * c + i;
          ++out;
        }
      }
    }
  }
  // rows that are scored again as a whole, a warp a row
  for (unsigned m = __ballot_sync(0xffffffffu, whole); m != 0; m &= m - 1) {
    const int src = __ffs(m) - 1, nn = __shfl_sync(0xffffffffu, t.n, src), kk = __shfl_sync(0xffffffffu, t.k, src);
    const auto* q = reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(0xffffffffu, (unsigned long long)t.q, src));
    const auto* s = reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(0xffffffffu, (unsigned long long)t.summ, src));
    const size_t row = __shfl_sync(0xffffffffu, (unsigned long long)t.row, src);
    const int base = __shfl_sync(0xffffffffu, t.base, src), part = lane & 7;
    for (int j0 = 0; j0 < nn; j0 += 4) {
      const int j = min(j0 + (lane >> 3), nn - 1);
      const float z = row_score<MINMAX>(A, q, s + (size_t)j * kSummary, part);
      if (part == 0) keys[j] = z;
    }
    __syncwarp();
    warp_topk([&](int j) { return order_key(keys[j]); }, nn, kk, base, A.sel_idx + row * A.kcap, copies, A.kcap);
    __syncwarp();
  }
}

template <bool MINMAX>
__global__ void __launch_bounds__(kThreads, 2)
select_rows_tc_kernel(SelectArgs A, const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmS) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = smem;                                             // [q or q+, q-][half of the dims][128 rows][64]
  uint8_t* s_k = smem + (MINMAX ? 2 : 1) * 2 * kHalfTile;          // [max, min][half][64 blocks][64]
  Ctl* c = reinterpret_cast<Ctl*>(smem + kOperands<MINMAX>);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    mbar_init(&c->q_full, 1);
    mbar_init(&c->s_full, 1);
    mbar_init(&c->done, 1);
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&c->tmem, kCols);
  pdl_wait();
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem, mine = tmem + ((uint32_t)warp << 21);
  const uint64_t dQ = smem_desc(smem_u32(s_q), 16, 1024), dK = smem_desc(smem_u32(s_k), 16, 1024);
  constexpr uint32_t id = bf16_idesc(kRows, kTile, false);
  float* scratch = A.scores + (size_t)blockIdx.x * A.slots * (kRows + kThreads / 32);
  float* keys = scratch + (size_t)A.slots * kRows + (size_t)warp * A.slots;
  const int T = A.group ? kRows : kRows / A.G, heads = A.group ? A.G : 1;
  uint32_t q_phase = 0, s_phase = 0, d_phase = 0;
  bool ok = true;
  for (int u = blockIdx.x; u < A.n_items; u += gridDim.x) {
    SelectItem it;
    if (!select_item<kThreads>(A, T, u, &c->place, it)) break;
    const int h0 = it.kvh * A.G;
    int j0, j1;
    const bool all = item_candidates(A, it.kvh, it.pos0 + it.tokens - 1, j0, j1);
    const int n_item = all ? 0 : j1 - j0;
    // the thread's row
    const int tok = A.group ? tid : tid / A.G, g = A.group ? 0 : tid - tok * A.G;
    RowTask t{};
    {
      const bool there = tid < T * (A.group ? 1 : A.G) && tok < it.tokens;
      int c0 = 0, c1 = 0;
      if (there) row_candidates(A, it.pos0 + tok, A.bs[it.kvh], c0, c1);
      t.n = c1 - c0;
      t.k = min(A.k[h0 + g], t.n);
      t.base = c0;
      t.row = (size_t)(it.row0 + (there ? tok : 0)) * A.Hq + h0 + g;
      t.valid = there && t.k > 0 && t.k < t.n;
      t.q = A.q + t.row * kD;
      t.summ = A.summaries + (((size_t)it.b * A.Hk + it.kvh) * A.slots + c0) * (MINMAX ? 2 : 1) * kD;
      if (there) {
        const int copies = A.group ? A.G : 1;
        for (int y = 0; y < copies; ++y) {
          A.sel_cnt[t.row + y] = t.k;
          if (t.k == t.n)
            for (int j = 0; j < t.n; ++j) A.sel_idx[(t.row + y) * A.kcap + j] = c0 + j;
        }
      }
    }
    if (n_item == 0) {
      __syncthreads();
      continue;
    }
    float norm = 0.f;
    const bool memory = n_item > kCols;
    for (int w0 = 0; w0 < n_item && ok; w0 += kCols) {
      const int cols = min(kCols, n_item - w0);
      for (int head = 0; head < heads && ok; ++head) {
        if (w0 == 0 || heads > 1) {       // else q is there
          if (tid == 0) {
            const int rows = A.group ? kRows : T * A.G;
            mbar_arrive_expect_tx(&c->q_full, rows * kD * 2);
            for (int half = 0; half < 2; ++half)
              tma_load_3d(s_q + half * kHalfTile, &tmQ, half * 64, h0 + head, it.row0, &c->q_full);
          }
          ok = mbar_wait_bounded(&c->q_full, q_phase & 1, A.status);
          ++q_phase;
          // q+ and q- of the thread's row, and its norm
          float sq = 0.f;
          if (ok) {
#pragma unroll 4
            for (int x = 0; x < 16; ++x) {
              uint4* p = reinterpret_cast<uint4*>(s_q + (x >> 3) * kHalfTile + tid * 128 + (((x & 7) ^ (tid & 7)) << 4));
              uint4 y = *p, neg = make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t& a = (&y.x)[e];
                const float lo = bf16_lo(a), hi = bf16_hi(a);
                sq = fmaf(lo, lo, sq);
                sq = fmaf(hi, hi, sq);
                if (MINMAX) {
                  const uint32_t minus = (a & 0x8000u ? 0xffffu : 0u) | (a & 0x80000000u ? 0xffff0000u : 0u);
                  (&neg.x)[e] = a & minus;
                  a &= ~minus;
                }
              }
              if (MINMAX) {
                *p = y;
                *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p) + 2 * kHalfTile) = neg;
              }
            }
          }
          if (w0 == 0) norm += sqrtf(sq);
          fence_proxy_async_smem();
          ok = !__syncthreads_or(!ok);
        }
        for (int x = 0; x < cols && ok; x += kTile) {
          if (tid == 0) {
            // summaries behind the item's last come along; no row looks at them
            const int slot = ((it.b * A.Hk + it.kvh) * A.slots) + j0 + w0 + x;
            mbar_arrive_expect_tx(&c->s_full, (MINMAX ? 4 : 2) * kSummHalf);
            for (int y = 0; y < (MINMAX ? 4 : 2); ++y)
              tma_load_3d(s_k + y * kSummHalf, &tmS, (y & 1) * 64, MINMAX ? 1 - (y >> 1) : 0, slot, &c->s_full);
            ok = mbar_wait_bounded(&c->s_full, s_phase & 1, A.status);
            if (ok) {
              tc_fence_after();
#pragma unroll
              for (int y = 0; y < (MINMAX ? 16 : 8); ++y)
                tc_mma_ss(tmem + x, dQ + (y >> 2) * (kHalfTile / 16) + (y & 3) * 2,
                          dK + (y >> 2) * (kSummHalf / 16) + (y & 3) * 2, id, y != 0 || head != 0);
              tc_commit(&c->done);
            }
          }
          ++s_phase;
          if (ok) ok = mbar_wait_bounded(&c->done, d_phase & 1, A.status);
          ++d_phase;
          ok = !__syncthreads_or(!ok);
        }
      }
      if (!ok) break;
      tc_fence_after();
      if (memory) {
        for (int x = 0; x < cols; x += 32) {
          float v[32];
          tmem_ld32(mine + x, v);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (w0 + x + i < n_item) scratch[(size_t)(w0 + x + i) * kRows + tid] = v[i];
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
      }
    }
    if (!ok) break;
    const float k2 = __int_as_float(__ldg(A.norms + it.b * A.Hk + it.kvh));
    t.E = 6.103515625e-5f * heads * norm * sqrtf(k2) * 1.001f + 1e-35f;
    if (memory) select_list<MINMAX, true>(A, t, mine, scratch + tid, keys, &c->warp[warp]);
    else select_list<MINMAX, false>(A, t, mine, scratch + tid, keys, &c->warp[warp]);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tmem, kCols);
}

}  // namespace

size_t select_tc_scratch(int slots) {
  return (size_t)2 * kRowsMaxCtas * slots * (kRows + kThreads / 32) * sizeof(float);
}

template <bool MINMAX>
static int launch(const SelectArgs& A, const CUtensorMap& tmQ, const CUtensorMap& tmS, int num_sms, cudaStream_t stream) {
  if (smem_limit_at_least(reinterpret_cast<const void*>(select_rows_tc_kernel<MINMAX>), (int)kSmem<MINMAX>) != cudaSuccess)
    return SA_ERR_CUDA;
  if (cudaMemsetAsync(A.norms, 0, (size_t)A.B * A.Hk * sizeof(int), stream) != cudaSuccess) return SA_ERR_CUDA;
  cudaError_t e = launch_pdl(summary_norms_kernel<MINMAX>, dim3(A.B * A.Hk, std::min(16, (A.slots + 63) / 64)), dim3(256),
                             0, stream, A);
  if (e != cudaSuccess) return SA_ERR_CUDA;
  e = launch_pdl(select_rows_tc_kernel<MINMAX>, dim3(std::min(A.n_items, 2 * num_sms)), dim3(kThreads), kSmem<MINMAX>,
                 stream, A, tmQ, tmS);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

int launch_select_tc(const SelectArgs& A, const CUtensorMap& tmQ, const CUtensorMap& tmS, int num_sms,
                     cudaStream_t stream) {
  return A.minmax ? launch<true>(A, tmQ, tmS, num_sms, stream) : launch<false>(A, tmQ, tmS, num_sms, stream);
}

}  // namespace sa
