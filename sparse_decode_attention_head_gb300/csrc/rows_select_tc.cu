// Selected blocks of many rows (sa_select_rows): scores on the tensor cores
// find the selection, scores in the canonical order decide where they are close.
//
// The canonical fp32 order of a score is no order that a matrix instruction
// has, so what the tensor cores give is taken as a value a with
//   |a - s| <= E = 2^-15 |q| max_j |k_j|      (norms of q and of max(|min|, |max|))
// of the canonical s.  A matrix instruction adds 16 products and the sum so far,
// each cut to 24 bits of the largest of them (off by 2^-23 of it at most, the
// products of zeros not at all); none is above sum |q k| <= |q| |k|.  128
// products and at most 16 sums are off by 144 * 2^-23 |q| |k| < 2^-15.8 |q| |k|,
// the canonical sum by less than 2^-19.  A candidate that is more than 2 E above the best one left out is
// selected whatever the order; one that is more than 2 E below the worst one
// taken is not; those between (in one row out of seven or so) are scored again in
// the canonical order, and the best of them, lowest index first among equals,
// fill the list.  So lists are the canonical ones, entry for entry.  A row with
// more close ones than kClose, or without a bound (infinities), is scored
// again as a whole.
//
// q . min/max summary: sum over d of q+_d kmax_d + q-_d kmin_d with q+ and q-
// the positive and negative part, a product of twice the length, half of it zeros.
// Heads that select together: a row is a token, and what the product takes is
// the sum of the group's queries (of their positive and of their negative
// parts), as two bf16 that hold 2^-17 of it, one product behind the other.  In
// units of |Q| |K|, Q the sum over heads of |q| and K the largest of max_j |k_j|:
//   means: 256 products and 16 sums, 272 * 2^-23 < 2^-14.9;
//   min/max: with heads of both signs a dim has two products in each of the two,
//   512 products and 32 sums, 544 * 2^-23 < 2^-13.9;
//   the operand 2^-17 and its sums of eight 2^-21, the heads' canonical sums
//   (18 roundings each, 7 between them) 2^-19.
// Together below 2^-14.5 and 2^-13.7: E = 2^-14 |Q| |K| of means and 2^-13 of min/max.
//
// A block (four warps, two blocks an SM) takes an item: one KV head with 128
// rows (tokens and heads; tokens, for heads that select together) of a sequence, a thread a row.  Scores stay in
// TMEM (up to 256 candidates; more go through a scratch, [candidate][row]).
// A threshold that starts where a normal distribution has it and follows its
// density until a few more than k reach it (two to four passes that count)
// leaves a short list of each row, in the shared memory of the operands; the
// k-th is found there by a sorting network.
#include <algorithm>

#include <cuda_fp16.h>

#include "rows_select.cuh"
#include "tcgen.cuh"

namespace sa {
namespace {

constexpr int kThreads = 128, kRows = 128, kCols = 256, kTile = 64;
constexpr int kHalfTile = kRows * 64 * 2, kSummHalf = kTile * 64 * 2;     // 64 dims of q's rows, of a tile of summaries
constexpr int kClose = 8;                                                   // of a row, scored again one by one
// A row's short list: the candidates above a threshold, at least k of them and
// kShort at most, where k is at most kShortK; it lies where the operands were.
constexpr int kShort = 64, kShortRoom = kShort + 32, kShortK = 40;
constexpr size_t kShortBytes = (size_t)kRows * kShortRoom * sizeof(float2);     // (score, candidate)

// Tiles of summaries under way: what 96 KB, two blocks an SM, leave beside two
// tiles of q (its parts, or the two bf16 of a group's sum).
template <bool MINMAX>
constexpr int kStages = MINMAX ? 1 : 2;
template <bool MINMAX>
constexpr size_t kOperands = std::max<size_t>(4 * kHalfTile + kStages<MINMAX> * (MINMAX ? 4 : 2) * kSummHalf, kShortBytes);

struct Warp {
  uint16_t close[32][kClose];
  uint16_t task[32 * kClose];
  float score[32 * kClose];
};
struct Ctl {
  Warp warp[kThreads / 32];
  uint64_t q_full, s_full[4], free[4], done, drain;
  uint32_t loaded, q_loaded;      // tiles of summaries and of q asked for so far
  float norm[kRows];
  uint32_t tmem;
  ItemPlace place;
};
template <bool MINMAX>
constexpr size_t kSmem = 1024 + kOperands<MINMAX> + sizeof(Ctl);
static_assert(2 * (kSmem<true> + 1024) <= 228 * 1024, "two blocks an SM");

// Of a block's scratch: whole steps of candidates.
__host__ __device__ constexpr size_t scratch_columns(int slots) { return (size_t)(slots + 31) / 32 * 32; }

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

// Where a normal distribution has the share p of its values above.  (Hastings'
// approximation of the quantile: Abramowitz and Stegun 26.2.22.)
__device__ __forceinline__ float upper_quantile(float p) {
  const float tail = sqrtf(-2.f * logf(fminf(p, 1.f - p)));
  const float z = tail - (2.30753f + 0.27061f * tail) / (1.f + tail * (0.99229f + 0.04481f * tail));
  return p < 0.5f ? z : -z;
}

// The close candidates of a warp's rows, n_close of each in w->close, scored in
// the canonical order; a bit for each of the `need` best of the lane's row.
template <bool MINMAX>
__device__ __forceinline__ unsigned choose_close(const SelectArgs& A, const RowTask& t, int n_close, int need, Warp* w) {
  constexpr int kSummary = (MINMAX ? 2 : 1) * kD;
  const int lane = threadIdx.x & 31, part = lane & 7;
  const int upto = warp_incl_scan(n_close), total = __shfl_sync(0xffffffffu, upto, 31), first = upto - n_close;
  for (int i = 0; i < n_close; ++i) w->task[first + i] = (uint16_t)(lane * kClose + i);
  __syncwarp();
  for (int x0 = 0; x0 < total; x0 += 8) {      // two each eight lanes, their loads together
    float z[2];
    int x[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      x[y] = min(x0 + 4 * y + (lane >> 3), total - 1);
      const int task = w->task[x[y]], who = task / kClose;
      const size_t row = __shfl_sync(0xffffffffu, (unsigned long long)t.q, who);
      const size_t summ = __shfl_sync(0xffffffffu, (unsigned long long)t.summ, who);
      z[y] = row_score<MINMAX>(A, reinterpret_cast<const __nv_bfloat16*>(row),
                               reinterpret_cast<const __nv_bfloat16*>(summ) +
                                   (size_t)w->close[who][task % kClose] * kSummary, part);
    }
    if (part < 2) w->score[part == 0 ? x[0] : x[1]] = part == 0 ? z[0] : z[1];
  }
  __syncwarp();
  unsigned chosen = 0;
  for (int i = 0; i < n_close; ++i) {
    const float z = w->score[first + i];
    int rank = 0;
    for (int j = 0; j < n_close; ++j) {
      const float o = w->score[first + j];
      rank += o > z || (o == z && j < i);
    }
    if (rank < need) chosen |= 1u << i;
  }
  __syncwarp();
  return chosen;
}

// Rows (a bit a lane) that are scored again as a whole, a warp a row.
template <bool MINMAX>
__device__ __noinline__ void select_whole(const SelectArgs& A, const RowTask& t, unsigned rows, float* keys) {
  constexpr int kSummary = (MINMAX ? 2 : 1) * kD;
  const int lane = threadIdx.x & 31, part = lane & 7;
  for (; rows != 0; rows &= rows - 1) {
    const int src = __ffs(rows) - 1, n = __shfl_sync(0xffffffffu, t.n, src), k = __shfl_sync(0xffffffffu, t.k, src);
    const auto* q = reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(0xffffffffu, (unsigned long long)t.q, src));
    const auto* s = reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(0xffffffffu, (unsigned long long)t.summ, src));
    const size_t row = __shfl_sync(0xffffffffu, (unsigned long long)t.row, src);
    const int base = __shfl_sync(0xffffffffu, t.base, src);
    for (int j0 = 0; j0 < n; j0 += 4) {
      const int j = min(j0 + (lane >> 3), n - 1);
      const float z = row_score<MINMAX>(A, q, s + (size_t)j * kSummary, part);
      if (part == 0) keys[j] = z;
    }
    __syncwarp();
    warp_topk([&](int j) { return order_key(keys[j]); }, n, k, base, A.sel_idx + row * A.kcap, A.group ? A.G : 1, A.kcap);
    __syncwarp();
  }
}

// A row's candidates' approximate scores, kStep at a time; those behind the
// row's last are -infinity.
constexpr int kStep = 32;
template <bool MEMORY>
struct Scores {
  uint32_t tmem;
  const float* scratch;
  int n;
  __device__ __forceinline__ void load(int c, float (&v)[kStep]) const {
    if (MEMORY) {
#pragma unroll
      for (int i = 0; i < kStep; ++i) v[i] = scratch[(size_t)(kStep * c + i) * kRows];
    } else {
      tmem_ld32(tmem + kStep * c, v);
    }
    if (__any_sync(0xffffffffu, kStep * c + kStep > n)) {
#pragma unroll
      for (int i = 0; i < kStep; ++i) v[i] = kStep * c + i < n ? v[i] : -INFINITY;
    }
  }
  // f(first column, kStep scores) for every chunk, in order
  template <typename F>
  __device__ __forceinline__ void each(int chunks, F f) const {
    for (int c = 0; c < chunks; ++c) {
      float v[kStep];
      load(c, v);
      f(kStep * c, v);
    }
  }
  __device__ __forceinline__ int count(int chunks, float at) const {
    int a = 0, b = 0;
    for (int c = 0; c < chunks; ++c) {
      float v[kStep];
      load(c, v);
#pragma unroll
      for (int i = 0; i < kStep; i += 2) {
        a += v[i] >= at;
        b += v[i + 1] >= at;
      }
    }
    return a + b;
  }
};

// How many of a row's scores reach a threshold.  In TMEM a look at all of them
// is a load's round trip every 32 columns (200 cycles for 16 scores), so up to
// 256 are kept in registers, as pairs of fp16 in units of their spread about
// their mean: counts that are off by what lies within 2^-9 of the threshold
// change the length of a list, not what is selected.
template <bool MEMORY>
struct Counter {
  const Scores<MEMORY>& S;
  int chunks;
  float mean, sigma;
  __device__ __forceinline__ Counter(const Scores<MEMORY>& s, int c, float m, float d) : S(s), chunks(c), mean(m), sigma(d) {}
  __device__ __forceinline__ int count(float at) const { return S.count(chunks, at); }
};
template <>
struct Counter<false> {
  __half2 h[kCols / 2];
  float mean, inv;
  int used;      // chunks
  __device__ __forceinline__ Counter(const Scores<false>& S, int chunks, float m, float sigma)
      : mean(m), inv(fminf(1.f / sigma, 1e30f)), used(chunks) {
#pragma unroll
    for (int c = 0; c < kCols / kStep; ++c) {
      if (c < chunks) {
        float v[kStep];
        S.load(c, v);
#pragma unroll
        for (int i = 0; i < kStep / 2; ++i)
          h[c * (kStep / 2) + i] = __floats2half2_rn((v[2 * i] - mean) * inv, (v[2 * i + 1] - mean) * inv);
      }
    }
  }
  __device__ __forceinline__ int count(float at) const {
    const __half2 t = __float2half2_rn((at - mean) * inv);
    __half2 sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = __float2half2_rn(0.f);
#pragma unroll
    for (int c = 0; c < kCols / kStep; ++c) {
      if (c < used) {
#pragma unroll
        for (int i = 0; i < kStep / 2; ++i) sum[i & 3] = __hadd2(sum[i & 3], __hge2(h[c * (kStep / 2) + i], t));
      }
    }
    const __half2 all = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
    return (int)(__low2float(all) + __high2float(all));
  }
};

// N values in descending order (Batcher's odd-even merge sort): no branches, and
// comparators that do not wait for one another.  A step compares values K apart
// inside runs of 2 P.
template <int N, int P, int K>
__device__ __forceinline__ void sort_steps(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N - K; ++i) {
    if (i >= K % P && (i - K % P) % (2 * K) < K && i / (2 * P) == (i + K) / (2 * P)) {
      const float a = v[i], b = v[i + K];
      v[i] = fmaxf(a, b);
      v[i + K] = fminf(a, b);
    }
  }
  if constexpr (K > 1) sort_steps<N, P, K / 2>(v);
  else if constexpr (2 * P < N) sort_steps<N, 2 * P, 2 * P>(v);
}

// The k-th and the next largest of a short list of at most N (-infinity where it has no such).
template <int N>
__device__ __forceinline__ void kth_of_list(const float2* list, int len, int k, float& kth, float& next) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = i < len ? list[i * kRows].x : -INFINITY;
  sort_steps<N, 1, 1>(v);
  kth = next = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i == k - 1) kth = v[i];
    if (i == k) next = v[i];
  }
}

// The next threshold of a search for `want` values at or above it, where there
// are cnt at or above `at`: along the normal distribution's density, or the
// middle of what is left.
__device__ __forceinline__ float next_threshold(float at, int cnt, int want, int n, float mean, float sigma, float lo,
                                                float hi, bool halve) {
  const float z = (at - mean) / sigma, density = n * 0.3989f * __expf(-0.5f * z * z) / sigma;
  const float next = at + (cnt - want) / fmaxf(density, 1e-6f / sigma);
  return halve || !(next > lo && next < hi) ? 0.5f * (lo + hi) : next;
}

// Rows with many to keep: the k-th is looked for among all candidates.
template <bool MINMAX, bool MEMORY>
__device__ __noinline__ unsigned select_long(const SelectArgs& A, const RowTask& t, const Scores<MEMORY>& S, int chunks,
                                             bool active, float mean, float sigma, float bound, Warp* w) {
  const int lane = threadIdx.x & 31;
  float lo = -bound, hi = bound;
  bool whole = false;
  float at = mean + sigma * upper_quantile((float)t.k / t.n);
  if (!(at > lo && at < hi)) at = 0.f;
  // count(>= lo) >= k > count(>= hi)
  bool found = false, search = active;
  for (int step = 0; step < 60 && __any_sync(0xffffffffu, search); ++step) {
    const int cnt = S.count(chunks, at);
    if (search) {
      if (cnt == t.k) {
        found = true;
        search = false;
      } else {
        if (cnt > t.k) lo = at; else hi = at;
        const float next = next_threshold(at, cnt, t.k, t.n, mean, sigma, lo, hi, step % 3 == 2);
        search = hi - lo > t.E && next > lo && next < hi;
        at = next;
      }
    }
  }
  // taken without a look: above `sure`.  Close: from `close_lo` to `sure`.
  float sure = hi + 2.f * t.E, close_lo = lo - 2.f * t.E;
  if (__any_sync(0xffffffffu, found)) {
    float least = INFINITY, best = -INFINITY;          // of those taken, of those left
    S.each(chunks, [&](int, const float (&v)[kStep]) {
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const bool in = v[i] >= at;
        least = fminf(least, in ? v[i] : INFINITY);
        best = fmaxf(best, in ? -INFINITY : v[i]);
      }
    });
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
    S.each(chunks, [&](int first, const float (&v)[kStep]) {
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        taken += v[i] > sure;
        if (some && v[i] <= sure && v[i] >= close_lo) {
          if (n_close < kClose) w->close[lane][n_close] = (uint16_t)(first + i);
          ++n_close;
        }
      }
    });
    if (some && n_close > kClose) {
      whole = true;
      some = active = false;
    }
    chosen = choose_close<MINMAX>(A, t, some ? n_close : 0, t.k - taken, w);
  }
  // the list, ascending
  const int copies = A.group ? A.G : 1;
  if (__any_sync(0xffffffffu, active)) {
    int* list = A.sel_idx + t.row * A.kcap;
    int out = 0;
    unsigned left = chosen;
    S.each(chunks, [&](int first, const float (&v)[kStep]) {
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        bool take = active && v[i] > sure;
        if (active && v[i] <= sure && v[i] >= close_lo) {
          take = left & 1u;
          left >>= 1;
        }
        if (take && out < t.k) {
          for (int y = 0; y < copies; ++y) list[(size_t)y * A.kcap + out] = t.base + first + i;
          ++out;
        }
      }
    });
  }
  return __ballot_sync(0xffffffffu, whole);
}

// A row's list, a thread a row.  mine: the lane's own column of the short lists.
template <bool MINMAX, bool MEMORY>
__device__ __forceinline__ void select_list(const SelectArgs& A, const RowTask& t, const Scores<MEMORY>& S, float* keys,
                                            Warp* w, float2* mine) {
  const int lane = threadIdx.x & 31;
  const int most = __reduce_max_sync(0xffffffffu, t.valid ? t.n : 0);
  if (most == 0) return;
  const int chunks = (most + kStep - 1) / kStep;
  bool whole = t.valid && !(t.E < 1e30f);        // no bound
  bool active = t.valid && !whole;
  const float bound = t.E * 33000.f;             // |score| < |q| |k| + E
  // mean and spread of at most 128 of them
  float mean, sigma;
  {
    const int full = max(1, __reduce_min_sync(0xffffffffu, t.valid ? t.n : most) / kStep), step = (full + 3) / 4;
    float sum = 0.f, sq = 0.f;
    int cnt = 0;
    for (int c = 0; c < full; c += step) {
      float v[kStep];
      S.load(c, v);
      const int here = min(kStep, t.n - kStep * c);    // fewer where the row has no more
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const float x = i < here ? v[i] : 0.f;
        sum += x;
        sq = fmaf(x, x, sq);
      }
      cnt += here;
    }
    mean = active ? sum / cnt : 0.f;
    sigma = active ? sqrtf(fmaxf(sq / cnt - mean * mean, 1e-30f)) : 1.f;
  }
  if (__any_sync(0xffffffffu, active && t.k > kShortK)) {
    unsigned again = select_long<MINMAX, MEMORY>(A, t, S, chunks, active, mean, sigma, bound, w);
    again |= __ballot_sync(0xffffffffu, whole);
    if (again != 0) select_whole<MINMAX>(A, t, again, keys);
    return;
  }
  // a threshold that a few more than k reach: enough to be sure, as a rule, that
  // all that are close to the k-th are among them
  float lo = -bound, hi = bound;
  const int few = min(t.k + 2, t.n), many = t.k + 16;
  float at = t.n <= many ? lo : mean + sigma * upper_quantile((t.k + 8.f) / t.n);
  if (!(at >= lo && at < hi)) at = lo;
  int tries = 0;
  bool search = active && t.n > many;
  if (__any_sync(0xffffffffu, search)) {
  const Counter<MEMORY> C(S, chunks, mean, sigma);
  while (__any_sync(0xffffffffu, search)) {
    const int cnt = C.count(at);
    if (search) {
      if (cnt >= few && cnt <= many) {
        search = false;
      } else {
        if (cnt > many) lo = at; else hi = at;
        const float next = next_threshold(at, cnt, t.k + 8, t.n, mean, sigma, lo, hi, tries % 3 == 2);
        if (++tries < 30 && next > lo && next < hi) {
          at = next;
        } else {           // many equal or close ones: all of them, if the list holds them
          at = lo;
          search = false;
        }
      }
    }
  }
  }
  // the short list: everything at or above it
  int len = 0;
  float sure = INFINITY, close_lo = INFINITY;    // taken above; close from close_lo to sure
  search = active;
  for (int round = 0; __any_sync(0xffffffffu, search); ++round) {
    __syncwarp();
    const float from = search ? at : INFINITY;
    int got = 0;
    S.each(chunks, [&](int first, const float (&v)[kStep]) {
      // one that is too long already is only counted
      const uint32_t begin = smem_u32(mine + min(got, kShort) * kRows);
      uint32_t place = begin;
#pragma unroll
      for (int i = 0; i < kStep; ++i)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ge.f32 p, %1, %2;\n\t"
            "@p st.shared.v2.b32 [%0], {%3, %4};\n\t@p add.u32 %0, %0, %5;\n\t}"
            : "+r"(place)
            : "f"(v[i]), "f"(from), "r"(__float_as_int(v[i])), "r"(first + i), "n"(kRows * 8)
            : "memory");
      got += (place - begin) / (kRows * 8);
    });
    if (search) len = got;
    if (search && got > kShort) {
      whole = true;
      search = false;
    }
    const int longest = __reduce_max_sync(0xffffffffu, search ? got : 0);
    float least, best;                           // of those taken; of those left
    if (longest <= 32) kth_of_list<32>(mine, search ? len : 0, t.k, least, best);
    else kth_of_list<64>(mine, search ? len : 0, t.k, least, best);
    if (search) {
      if (len < t.n) best = fmaxf(best, at);     // not above: what the list does not hold
      const bool apart = least - best > 2.f * t.E;
      sure = apart ? best : best + 2.f * t.E;
      close_lo = apart ? INFINITY : least - 2.f * t.E;
      search = close_lo < at && len < t.n;       // some that are close may be missing: once more, from there
      whole = search && round > 0;
      search = search && round == 0;
      at = close_lo;
    }
  }
  active = active && !whole;
  bool some = active && close_lo < INFINITY;
  if (__any_sync(0xffffffffu, some)) {
    int taken = 0, n_close = 0;
    uint64_t at_place = 0;      // of the close ones, eight bits each
    if (some) {
      for (int i = 0; i < len; ++i) {
        const float2 x = mine[i * kRows];
        taken += x.x > sure;
        if (x.x <= sure && x.x >= close_lo) {
          if (n_close < kClose) {
            w->close[lane][n_close] = (uint16_t)__float_as_int(x.y);
            at_place |= (uint64_t)i << (8 * n_close);
          }
          ++n_close;
        }
      }
      if (n_close > kClose) {
        whole = true;
        some = active = false;
        n_close = 0;
      }
    }
    __syncwarp();
    const unsigned chosen = choose_close<MINMAX>(A, t, n_close, t.k - taken, w);
    for (int i = 0; i < n_close; ++i)
      mine[((at_place >> (8 * i)) & 255) * kRows].x = (chosen >> i) & 1u ? INFINITY : -INFINITY;
  }
  // the list, ascending
  const int copies = A.group ? A.G : 1, longest = __reduce_max_sync(0xffffffffu, active ? len : 0);
  int* list = A.sel_idx + t.row * A.kcap;
  int out = 0;
  for (int i0 = 0; i0 < longest; i0 += 8) {
    float2 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = mine[(i0 + i) * kRows];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (active && i0 + i < len && x[i].x > sure && out < t.k) {
        const int e = t.base + __float_as_int(x[i].y);
        list[out] = e;
        mine[out * kRows].y = __int_as_float(e);     // for the copies; its place has been read
        ++out;
      }
    }
  }
  if (copies > 1) {            // the group's other heads: a row at a time, its entries in turn by the lanes
    __syncwarp();
    for (unsigned m = __ballot_sync(0xffffffffu, active); m != 0; m &= m - 1) {
      const int src = __ffs(m) - 1, k = __shfl_sync(0xffffffffu, t.k, src);
      int* to = reinterpret_cast<int*>(__shfl_sync(0xffffffffu, (unsigned long long)list, src));
      for (int j = lane; j < k; j += 32) {
        const int e = __float_as_int(mine[src - lane + j * kRows].y);
        for (int y = 1; y < copies; ++y) to[(size_t)y * A.kcap + j] = e;
      }
    }
  }
  const unsigned rows = __ballot_sync(0xffffffffu, whole);
  if (rows != 0) select_whole<MINMAX>(A, t, rows, keys);
}

// A row of q in shared memory (128-byte swizzle) becomes q+, and q- a tile
// further on; its squared norm.
template <bool MINMAX>
__device__ __forceinline__ float split_row(uint8_t* s_q, int row) {
  float sq = 0.f;
#pragma unroll 4
  for (int x = 0; x < 16; ++x) {
    uint4* p = reinterpret_cast<uint4*>(s_q + (x >> 3) * kHalfTile + row * 128 + (((x & 7) ^ (row & 7)) << 4));
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
  return sq;
}

// The sums of a group's queries as the operand, rounded to bf16, and what that
// leaves, rounded too: of all at once in two tiles, or of the positive and of
// the negative parts in two tiles, the rounded ones in part 0 and the rest in
// part 1.  16 threads a row.  Answers the norm of the thread's row's sum of |q|.
template <bool MINMAX>
__device__ __forceinline__ float sum_of_heads(const SelectArgs& A, const SelectItem& it, uint8_t* s_q, int part,
                                              float* s_norm) {
  const int tid = threadIdx.x, x = tid & 15;
#pragma unroll 2
  for (int row = tid >> 4; row < kRows; row += kThreads / 16) {
    const uint4* q = reinterpret_cast<const uint4*>(
        A.q + ((size_t)min(it.row0 + row, A.n_rows - 1) * A.Hq + it.kvh * A.G) * kD) + x;
    uint4 y[kMaxG];
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) y[g] = g < A.G ? __ldg(q + g * (kD / 8)) : make_uint4(0, 0, 0, 0);
    float plus[8], minus[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      plus[e] = minus[e] = 0.f;
#pragma unroll
      for (int g = 0; g < kMaxG; ++g) {
        const uint32_t w = (&y[g].x)[e >> 1];
        const float v = e & 1 ? bf16_hi(w) : bf16_lo(w);
        plus[e] += v > 0.f ? v : 0.f;
        minus[e] += v > 0.f ? 0.f : v;            // NaN goes here
      }
    }
    float sq = 0.f;
    uint32_t a[4], b[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float both = plus[e] - minus[e];
      sq = fmaf(both, both, sq);
      if (!MINMAX) plus[e] += minus[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      auto rest = [](float v) { return v - __bfloat162float(__float2bfloat16_rn(v)); };
      const float p0 = plus[2 * e], p1 = plus[2 * e + 1], m0 = minus[2 * e], m1 = minus[2 * e + 1];
      if (MINMAX) {
        a[e] = part == 0 ? pack_bf16(p0, p1) : pack_bf16(rest(p0), rest(p1));
        b[e] = part == 0 ? pack_bf16(m0, m1) : pack_bf16(rest(m0), rest(m1));
      } else {
        a[e] = pack_bf16(p0, p1);
        b[e] = pack_bf16(rest(p0), rest(p1));
      }
    }
    uint8_t* p = s_q + (x >> 3) * kHalfTile + row * 128 + (((x & 7) ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(p) = make_uint4(a[0], a[1], a[2], a[3]);
    *reinterpret_cast<uint4*>(p + 2 * kHalfTile) = make_uint4(b[0], b[1], b[2], b[3]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (x == 0) s_norm[row] = sqrtf(sq);
  }
  __syncthreads();
  return s_norm[tid];
}

template <bool MINMAX>
__global__ void __launch_bounds__(kThreads, 2)
select_rows_tc_kernel(SelectArgs A, const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmS) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = smem;                         // [q+, q- or a sum's two bf16][half of the dims][128 rows][64]
  uint8_t* s_k = smem + 4 * kHalfTile;         // [stage][max, min][half][64 blocks][64]
  Ctl* c = reinterpret_cast<Ctl*>(smem + kOperands<MINMAX>);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    mbar_init(&c->q_full, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&c->s_full[i], 1);
      mbar_init(&c->free[i], 1);
    }
    mbar_init(&c->done, 1);
    mbar_init(&c->drain, 1);
    c->loaded = c->q_loaded = 0;
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
  const size_t columns = scratch_columns(A.slots);
  float* scratch = A.scores + blockIdx.x * columns * (kRows + kThreads / 32);
  float* keys = scratch + columns * (kRows + warp);
  const int T = A.group ? kRows : kRows / A.G, parts = MINMAX && A.group ? 2 : 1;
  uint32_t q_phase = 0, tile = 0, d_phase = 0;
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
      for (int part = 0; part < parts && ok; ++part) {
        constexpr int kPieces = MINMAX ? 4 : 2, kStageBytes = kPieces * kSummHalf, kS = kStages<MINMAX>;
        const int tiles = (cols + kTile - 1) / kTile, slot0 = (it.b * A.Hk + it.kvh) * A.slots + j0 + w0;
        auto load = [&](int i) {     // summaries behind the item's last come along; no row looks at them
          uint64_t* bar = &c->s_full[(tile + i) % kS];
          mbar_arrive_expect_tx(bar, kStageBytes);
          c->loaded = tile + i + 1;
          for (int y = 0; y < kPieces; ++y)
            tma_load_3d(s_k + (tile + i) % kS * kStageBytes + y * kSummHalf, &tmS, (y & 1) * 64, MINMAX ? 1 - (y >> 1) : 0,
                        slot0 + i * kTile, bar);
        };
        if (tid == 0) {
          if (!A.group && w0 == 0) {
            mbar_arrive_expect_tx(&c->q_full, T * A.G * kD * 2);
            c->q_loaded = q_phase + 1;
            for (int half = 0; half < 2; ++half)
              tma_load_3d(s_q + half * kHalfTile, &tmQ, half * 64, h0, it.row0, &c->q_full);
          }
          for (int i = 0; i < min(tiles, kS); ++i) load(i);
        }
        __syncwarp();
        if (!A.group) {
          if (w0 == 0) {
            ok = mbar_wait_bounded(&c->q_full, q_phase & 1, A.status);
            ++q_phase;
            if (ok) norm = sqrtf(split_row<MINMAX>(s_q, tid));
          }
        } else if (MINMAX || w0 == 0) {      // else both are there
          norm = sum_of_heads<MINMAX>(A, it, s_q, part, c->norm);
        }
        fence_proxy_async_smem();
        ok = !__syncthreads_or(!ok);
        if (ok && tid == 0) {
          const int steps = MINMAX || A.group ? 16 : 8;
          for (int i = 0; i < tiles; ++i) {
            const uint32_t stage = (tile + i) % kS, parity = ((tile + i) / kS) & 1;
            if (!(ok = mbar_wait_bounded(&c->s_full[stage], parity, A.status))) break;
            tc_fence_after();
            const uint64_t k = dK + stage * (kStageBytes / 16);
#pragma unroll
            for (int y = 0; y < 16; ++y)
              if (y < steps)
                tc_mma_ss(tmem + i * kTile, dQ + (y >> 2) * (kHalfTile / 16) + (y & 3) * 2,
                          k + (y >> 2) % kPieces * (kSummHalf / 16) + (y & 3) * 2, id, y != 0 || part != 0);
            tc_commit(&c->free[stage]);
            if (i + kS < tiles) {
              if (!(ok = mbar_wait_bounded(&c->free[stage], parity, A.status))) break;
              load(i + kS);
            }
          }
          tc_commit(&c->done);
        }
        __syncwarp();        // lanes that wait for `done` already would hold up the one that issues
        tile += tiles;
        if (ok) ok = mbar_wait_bounded(&c->done, d_phase & 1, A.status);
        ++d_phase;
        ok = !__syncthreads_or(!ok);
      }
      if (!ok) break;
      tc_fence_after();
      if (memory) {
        for (int x = 0; x < cols; x += kStep) {
          float v[kStep];
          tmem_ld32(mine + x, v);
#pragma unroll
          for (int i = 0; i < kStep; ++i)
            if (w0 + x + i < n_item) scratch[(size_t)(w0 + x + i) * kRows + tid] = v[i];
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
      }
    }
    if (!ok) break;
    // squares below the smallest fp32 are lost: together less than (5e-22)^2
    const float k_norm = sqrtf(__int_as_float(__ldg(A.norms + it.b * A.Hk + it.kvh))) + 5e-22f;
    t.E = (!A.group ? 0x1p-15f : MINMAX ? 0x1p-13f : 0x1p-14f) * (norm + 5e-22f) * k_norm * 1.001f + 1e-35f;
    float2* list = reinterpret_cast<float2*>(smem) + tid;      // the operands are done with
    const int n = t.valid ? t.n : 0;
    if (memory) select_list<MINMAX, true>(A, t, Scores<true>{mine, scratch + tid, n}, keys, &c->warp[warp], list);
    else select_list<MINMAX, false>(A, t, Scores<false>{mine, scratch + tid, n}, keys, &c->warp[warp], list);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (!ok && tid == 0) {      // a wait gave up: what is in flight ends before the block does
    constexpr uint32_t kS = kStages<MINMAX>;
    for (uint32_t x = c->loaded - min(c->loaded, kS); x < c->loaded; ++x)
      (void)mbar_wait_bounded(&c->s_full[x % kS], (x / kS) & 1, A.status);
    if (c->q_loaded > 0) (void)mbar_wait_bounded(&c->q_full, (c->q_loaded - 1) & 1, A.status);
    tc_commit(&c->drain);
    (void)mbar_wait_bounded(&c->drain, 0, A.status);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tmem, kCols);
}

}  // namespace

size_t select_tc_scratch(int slots, long long n_items) {
  const size_t blocks = (size_t)std::min<long long>(2 * kRowsMaxCtas, n_items);
  return blocks * scratch_columns(slots) * (kRows + kThreads / 32) * sizeof(float);
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
