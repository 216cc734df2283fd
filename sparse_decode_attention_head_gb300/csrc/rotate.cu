// Norm, rotation and append of packed rows (sa_qk_norm_rope).
//
//   x <- x / sqrt(mean(x^2) + eps) * w,   (x1, x2) <- (x1 cos - x2 sin, x2 cos + x1 sin)
// for every query and key head of a row, values copied; keys and values go to
// the row's place in the paged cache.  Every byte is read and written once:
// 2 (Hq + 2 Hk) 256 bytes a row, which bounds it.
//
// A warp takes a row and a run of its heads, half a warp a head at a time, 8
// dims a lane.  The heads come through shared memory by bulk copies, 24 heads
// ahead of the ones at work: what is in flight then costs no registers (held
// there, four heads a lane, it was 1.4 times as slow).  With s = 1 / sqrt(...), a
// lane's result is s (x (w cos) + x' (+-w' sin)) with x' its partner's values:
// the two factors are the same for all query (key) heads of the row and stay
// in registers, two values an instruction, and the partner's values come as
// the packed words that were read.
//
// The angle: a frequency in turns is a 64-bit fraction F = frac(f / 2 pi) 2^64,
// computed once a block in fp64, and position x F modulo 2^64 is the exact
// fraction of a turn of that product; the top 32 bits, signed, go to
// sincospi.  What is lost is F's own rounding: position x frequency x 2^-55 of a
// turn, 2^-24 at the farthest position with a frequency of one.  No fp64 stands
// in the loop over rows (its rate here is a fraction of fp32's).
//
// Measured on one GB300: 65536 rows of 32 + 8 + 8 heads, norm and rotation,
// 287 us, 5.6 TB/s (0.83 of a copy's rate; issue slots 59 % busy, which is what
// is left to shorten); a row for each of 8 sequences 4.7 us.
#include <algorithm>

#include "rows.cuh"
#include "tcgen.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kStage = 24;      // heads of a copy stage, of which a warp has two

// Sequence whose rows hold `row`, by a warp together: the last one that begins
// at or before it (a 32-way search, one look for B <= 32).
__device__ __forceinline__ int seq_of_row(const int* row_offsets, int B, int row, int lane) {
  int lo = 0, n = B;             // the answer is in [lo, lo + n)
  while (true) {
    const int step = (n + 31) / 32;
    const bool before = lane * step < n && (lane == 0 || __ldg(row_offsets + lo + lane * step) <= row);
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, before));
    lo += last * step;
    if (step == 1) return lo;
    n = min(step, n - last * step);
  }
}

__device__ __forceinline__ void unpack(const uint4& w, uint64_t (&x)[4]) {
  x[0] = pack2(bf16_lo(w.x), bf16_hi(w.x));
  x[1] = pack2(bf16_lo(w.y), bf16_hi(w.y));
  x[2] = pack2(bf16_lo(w.z), bf16_hi(w.z));
  x[3] = pack2(bf16_lo(w.w), bf16_hi(w.w));
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// HALVES: the pairing (sa_rope.layout), known to the inner loops.  WHOLE: the
// pairs are a multiple of 8, so a lane's 8 dims turn alike and with the 8 of
// one other lane.  Else (sections of several axes with another sum) each dim
// looks up its own part, and the partner's value of a rotation of halves comes
// from the head in shared memory, two bytes a look, eight looks a lane:
// 65536 rows with 20 + 30 pairs take 345 us, with 24 + 24 of the other form 296.
template <bool HALVES, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 2) rotate_kernel(RotateArgs A, int run, int runs) {
  extern __shared__ __align__(16) uint8_t s_heads[];            // [warp][2][kStage][kD] bf16
  __shared__ unsigned long long s_freq[kD / 2];
  __shared__ uint64_t s_full[kWarps][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hl = lane & 15, half = lane >> 4;
  const int heads = A.Hq + 2 * A.Hk, turned_heads = A.Hq + A.Hk;
  const long long items = (long long)A.n_rows * runs, stride = (long long)gridDim.x * kWarps;
  uint8_t* stage[2] = {s_heads + (size_t)(warp * 2) * kStage * kD * 2,
                       s_heads + (size_t)(warp * 2 + 1) * kStage * kD * 2};
  if (lane < 2) mbar_init(&s_full[warp][lane], 1);
  fence_mbar_init();
  __syncwarp();
  pdl_wait();
  pdl_trigger();

  // what is loaded next: heads [lh, lh + kStage) of item li's run
  long long li = (long long)blockIdx.x * kWarps + warp;
  int lh = li < items ? (int)(li % runs) * run : 0;
  uint32_t loads = 0;
  auto load = [&]() {
    if (li >= items) return;
    const int row = (int)(li / runs), end = min(heads, (int)(li % runs) * run + run);
    const int h1 = min(end, lh + kStage);
    if (lane == 0) {
      uint64_t* bar = &s_full[warp][loads & 1];
      uint8_t* dst = stage[loads & 1];
      mbar_arrive_expect_tx(bar, (h1 - lh) * kD * 2);
      for (int h = lh; h < h1;) {      // a copy for each of q, k and v that the stage meets
        const int e = min(h1, h < A.Hq ? A.Hq : h < turned_heads ? turned_heads : heads);
        const __nv_bfloat16* src = h < A.Hq           ? A.q + row * A.q_stride + h * kD
                                   : h < turned_heads ? A.k + row * A.k_stride + (h - A.Hq) * kD
                                                      : A.v + row * A.v_stride + (h - turned_heads) * kD;
        bulk_load_1d(dst + (h - lh) * kD * 2, src, (e - h) * kD * 2, bar);
        h = e;
      }
    }
    ++loads;
    lh = h1;
    if (lh == end) {
      li += stride;
      lh = li < items ? (int)(li % runs) * run : 0;
    }
  };
  load();
  // every sequence's offsets and length are looked at once, also of those that
  // no row leads to; by a warp that has nothing to do with the frequencies
  if (warp == kWarps - 1) {
    for (int b = (int)blockIdx.x * 32 + lane; b < A.B; b += (int)gridDim.x * 32)
      row_seq(A.row_offsets, A.seq_lens, b, A.n_rows, A.mpp, A.status);
  }
  if (tid < A.pairs) {
    const double turns = (double)A.inv_freq[tid] * 0.15915494309189533577;
    s_freq[tid] = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
  }
  __syncthreads();

  // the partner lane of a rotation of halves, and this lane's part in it
  const int half_lanes = A.pairs / 8;
  const bool turned = 8 * hl < 2 * A.pairs, all_turned = 2 * A.pairs == kD;
  const bool second = HALVES && hl >= half_lanes;
  const int partner = turned && HALVES ? (lane & 16) + (second ? hl - half_lanes : hl + half_lanes) : lane;
  const int pair0 = HALVES ? 8 * (second ? hl - half_lanes : hl) : 4 * hl;
  // the dim that a dim of halves turns with, -1: none
  auto partner_dim = [&](int d) { return d < A.pairs ? d + A.pairs : d < 2 * A.pairs ? d - A.pairs : -1; };

  uint32_t used = 0;
  for (long long item = (long long)blockIdx.x * kWarps + warp; item < items; item += stride) {
    const int row = (int)(item / runs), h0 = (int)(item % runs) * run, h1 = min(heads, h0 + run);
    int axis_pos[SA_MAX_AXES] = {0, 0, 0, 0};
    if (A.positions != nullptr) {
#pragma unroll
      for (int a = 0; a < SA_MAX_AXES; ++a)
        if (a == 0 || A.axis_end[a - 1] < A.pairs) axis_pos[a] = __ldg(A.positions + (size_t)a * A.n_rows + row);
    }
    const int b = seq_of_row(A.row_offsets, A.B, row, lane);
    const RowSeq s = row_seq(A.row_offsets, A.seq_lens, b, A.n_rows, A.mpp, nullptr);
    const bool mine = row >= s.row0 && row < s.row0 + s.n;
    const int pos = s.a + row - s.row0;
    bool place = false;
    size_t slab = 0;              // the row's offset in a pool, without its head
    if (mine && pos >= 0 && pos < A.mpp * kP && h1 > A.Hq) {
      const int phys = __ldg(A.page_table + (size_t)b * A.mpp + pos / kP);
      place = phys >= 0 && phys < A.num_pages;
      if (!place) set_status(A.status, SA_ERR_BAD_PAGE);
      slab = ((size_t)phys * A.Hk * kP + pos % kP) * kD;
    }
    // cos and sin of the lane's dims: 8 pairs of halves, or 4 neighbouring pairs
    float cs[8], sn[8];
    if (h0 < turned_heads) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
      }
      if (turned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!HALVES && (i & 1)) {          // the odd dim of a pair
            cs[i] = cs[i - 1];
            sn[i] = sn[i - 1];
            continue;
          }
          const int d = 8 * hl + i;
          if (!WHOLE && d >= 2 * A.pairs) continue;
          const int j = WHOLE ? pair0 + (HALVES ? i : i >> 1) : !HALVES ? d >> 1 : d < A.pairs ? d : d - A.pairs;
          const int at = A.positions == nullptr ? pos
                         : j < A.axis_end[0]    ? axis_pos[0]
                         : j < A.axis_end[1]    ? axis_pos[1]
                         : j < A.axis_end[2]    ? axis_pos[2]
                                                : axis_pos[3];
          const unsigned long long turn = (unsigned long long)(long long)at * s_freq[j];
          sincospif((float)(int)(turn >> 32) * 4.656612873077392578125e-10f, &sn[i], &cs[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!HALVES ? (i & 1) == 0 : WHOLE ? !second : 8 * hl + i < A.pairs) sn[i] = -sn[i];
      }
    }
    uint64_t own_f[4], other_f[4];     // factors of the lane's values and of its partner's
    int kind = -1;                     // that they are for: 0 queries, 1 keys
    auto factors = [&](int key, const __nv_bfloat16* wt) {
      kind = key;
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.f;
      if (wt != nullptr) {
        const uint4 w4 = __ldg(reinterpret_cast<const uint4*>(wt) + hl);
        const uint32_t ww[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[2 * i] = bf16_lo(ww[i]);
          w[2 * i + 1] = bf16_hi(ww[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // the partner's weights
        float w0 = w[2 * i + 1], w1 = w[2 * i];
        if (HALVES && WHOLE) {
          w0 = __shfl_sync(0xffffffffu, w[2 * i], partner);
          w1 = __shfl_sync(0xffffffffu, w[2 * i + 1], partner);
        } else if (HALVES) {
          const int p0 = partner_dim(8 * hl + 2 * i), p1 = partner_dim(8 * hl + 2 * i + 1);
          w0 = wt != nullptr && p0 >= 0 ? __bfloat162float(wt[p0]) : 1.f;
          w1 = wt != nullptr && p1 >= 0 ? __bfloat162float(wt[p1]) : 1.f;
        }
        own_f[i] = pack2(w[2 * i] * cs[2 * i], w[2 * i + 1] * cs[2 * i + 1]);
        other_f[i] = pack2(w0 * sn[2 * i], w1 * sn[2 * i + 1]);
      }
    };
    // one head: 8 values of the lane, and the head they are of
    auto turn = [&](uint4 y, const uint4* head, bool norm) -> uint4 {
      uint32_t z[4] = {y.x, y.y, y.z, y.w};      // the partner's values; none where nothing turns
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (HALVES && !WHOLE) {
          const unsigned short* x = reinterpret_cast<const unsigned short*>(head);
          const int p0 = partner_dim(8 * hl + 2 * i), p1 = partner_dim(8 * hl + 2 * i + 1);
          z[i] = (p0 >= 0 ? (uint32_t)x[p0] : 0u) | (p1 >= 0 ? (uint32_t)x[p1] << 16 : 0u);
        } else {
          z[i] = HALVES ? __shfl_sync(0xffffffffu, z[i], partner) : __funnelshift_l(z[i], z[i], 16);
          if (!WHOLE && 4 * hl + i >= A.pairs) z[i] = 0u;
        }
      }
      if (WHOLE && !all_turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = turned ? z[i] : 0u;
      }
      uint64_t own[4], other[4];
      unpack(y, own);
      unpack(make_uint4(z[0], z[1], z[2], z[3]), other);
#pragma unroll
      for (int i = 0; i < 4; ++i) other[i] = mul2(other[i], other_f[i]);
      if (norm) {
        uint64_t s2 = mul2(own[0], own[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) s2 = fma2(own[i], own[i], s2);
        float sa, sb;
        unpack2(s2, sa, sb);
        sa += sb;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sa += __shfl_xor_sync(0xffffffffu, sa, o);
        sa = rsqrtf(sa * (1.f / kD) + A.eps);
        const uint64_t scale = pack2(sa, sa);
#pragma unroll
        for (int i = 0; i < 4; ++i) own[i] = mul2(fma2(own[i], own_f[i], other[i]), scale);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) own[i] = fma2(own[i], own_f[i], other[i]);
      }
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack2(own[i], lo, hi);
        r[i] = pack_bf16(lo, hi);
      }
      return make_uint4(r[0], r[1], r[2], r[3]);
    };
    for (int hs = h0; hs < h1; hs += kStage) {
      __syncwarp();                    // the stage that is loaded next has been read
      load();
      const uint32_t st = used & 1;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&s_full[warp][st], (used >> 1) & 1, A.status))) {
        // nothing of a stage that did not arrive is stored; the copies that are
        // under way are waited for, with the same limit, and the warp ends
        for (; used < loads; ++used) (void)mbar_wait_bounded(&s_full[warp][used & 1], (used >> 1) & 1, A.status);
        return;
      }
      ++used;
      const uint4* src = reinterpret_cast<const uint4*>(stage[st]) + hl;      // head hs + i is src[16 i]
      const int he = min(h1, hs + kStage);
      // queries, then keys: a head a half-warp, two of them at a time
#pragma unroll 1
      for (int key = 0; key < 2; ++key) {
        const int a = max(hs, key ? A.Hq : 0), e = min(he, key ? turned_heads : A.Hq);
        if (a >= e) continue;
        const __nv_bfloat16* wt = key ? A.k_weight : A.q_weight;
        if (key != kind) factors(key, wt);
        uint4* dst = key ? reinterpret_cast<uint4*>(A.k_pool + slab) + hl + (ptrdiff_t)(a - A.Hq) * (kP * kD / 8)
                         : reinterpret_cast<uint4*>(A.q_out + ((size_t)row * A.Hq + a) * kD) + hl;
        const int step = key ? kP * kD / 8 : kD / 8;      // between heads, in 16-byte pieces
        const bool write = key ? place : mine;
        const uint4* from = src + (a - hs) * 16;
        const uint4* head = from - hl;
        int h = half;
        const int n = e - a;
#pragma unroll 1
        for (; h - half + 4 <= n; h += 4) {
          const uint4 y0 = turn(from[16 * h], head + 16 * h, wt != nullptr);
          const uint4 y1 = turn(from[16 * h + 32], head + 16 * h + 32, wt != nullptr);
          if (write) {
            dst[(ptrdiff_t)h * step] = y0;
            dst[(ptrdiff_t)(h + 2) * step] = y1;
          }
        }
        for (; h - half < n; h += 2) {
          const bool there = h < n;
          const uint4 y = turn(there ? from[16 * h] : make_uint4(0, 0, 0, 0), there ? head + 16 * h : head, wt != nullptr);
          if (write && there) dst[(ptrdiff_t)h * step] = y;
        }
      }
      if (place) {      // values as they are
        uint4* dst = reinterpret_cast<uint4*>(A.v_pool + slab) + hl;
        for (int h = max(hs, turned_heads) + half; h < he; h += 2)
          dst[(ptrdiff_t)(h - turned_heads) * (kP * kD / 8)] = src[(h - hs) * 16];
      }
    }
  }
}

}  // namespace

int launch_rotate(const RotateArgs& A, int num_sms, cudaStream_t stream) {
  constexpr size_t smem = (size_t)kWarps * 2 * kStage * kD * 2;
  const bool halves = A.layout == SA_ROPE_HALVES, eights = A.pairs % 8 == 0;
  const auto kern = eights ? (halves ? rotate_kernel<true, true> : rotate_kernel<false, true>)
                           : (halves ? rotate_kernel<true, false> : rotate_kernel<false, false>);
  const void* kernel = reinterpret_cast<const void*>(kern);
  if (smem_limit_at_least(kernel, (int)smem) != cudaSuccess) return SA_ERR_CUDA;
  const int heads = A.Hq + 2 * A.Hk;
  const int blocks_per_sm = ctas_per_sm(kernel, kThreads, smem);
  const long long warps = (long long)num_sms * blocks_per_sm * kWarps;
  // heads of a warp's run: all of them (a row's sines are then computed once),
  // unless that leaves the last round of warps mostly idle: with few rows, or
  // a little more than one round, the heads are spread over more warps
  int runs = 1, run = heads;
  for (int r = 1; r <= (heads + 3) / 4; ++r) {
    const int each = ((heads + r - 1) / r + 3) / 4 * 4;
    const long long items = (long long)A.n_rows * r, rounds = (items + warps - 1) / warps;
    runs = r;
    run = each;
    if (items * 4 >= rounds * warps * 3) break;
  }
  runs = (heads + run - 1) / run;
  const long long blocks = ((long long)A.n_rows * runs + kWarps - 1) / kWarps;
  const int grid = (int)std::min<long long>(blocks, (long long)num_sms * blocks_per_sm);
  const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(kThreads), smem, stream, A, run, runs);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace sa
