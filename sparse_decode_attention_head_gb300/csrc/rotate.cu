// Norm, rotation and append of packed rows (sa_qk_norm_rope).
//
//   x <- x / sqrt(mean(x^2) + eps) * w,   (x1, x2) <- (x1 cos - x2 sin, x2 cos + x1 sin)
// for every query and key head of a row, values copied; keys and values go to
// the row's place in the paged cache.  Every byte is read and written once:
// 2 (Hq + 2 Hk) 256 bytes a row, which bounds it.
//
// Half a warp takes a row and a run of its heads, 8 dims a lane (one 16-byte
// load and store a head), four heads in flight; a lane's sines and cosines
// are the same for all heads of the row and stay in registers.  Where rows
// are few the heads are spread over more warps.
//
// The angle: a frequency in turns is a 64-bit fraction F = frac(f / 2 pi) 2^64,
// computed once a block in fp64, and position x F modulo 2^64 is the exact
// fraction of a turn of that product; the top 32 bits, signed, go to
// sincospi.  A far position therefore loses nothing, and no fp64 stands in
// the loop over rows (its rate here is a fraction of fp32's).
#include <algorithm>

#include "rows.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;    // heads a lane has loaded ahead

// Sequence whose rows hold `row`: the last one that begins at or before it.
__device__ __forceinline__ int seq_of_row(const int* row_offsets, int B, int row) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(row_offsets + mid) <= row) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
  x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x);
  x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z);
  x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
}

__global__ void __launch_bounds__(kThreads)
rotate_kernel(RotateArgs A, int chunk, int chunks) {
  __shared__ unsigned long long s_freq[kD / 2];
  const int tid = threadIdx.x, lane = tid & 31, hl = lane & 15;
  pdl_wait();
  pdl_trigger();
  if (tid < A.pairs) {
    const double turns = (double)A.inv_freq[tid] * 0.15915494309189533577;
    s_freq[tid] = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
  }
  __syncthreads();
  const int heads = A.Hq + 2 * A.Hk;
  const long long items = (long long)((A.n_rows + 1) / 2) * chunks;
  // the partner lane of a rotation of halves, and this lane's part in it
  const int half_lanes = A.pairs / 8;
  const bool halves = A.layout == SA_ROPE_HALVES;
  const bool turned = 8 * hl < 2 * A.pairs;
  const bool second = halves && hl >= half_lanes;
  const int partner = turned && halves ? (lane & 16) + (second ? hl - half_lanes : hl + half_lanes) : lane;
  const int npair = halves ? 8 : 4, pair0 = halves ? 8 * (second ? hl - half_lanes : hl) : 4 * hl;

  for (long long item = (long long)blockIdx.x * (kThreads / 32) + (tid >> 5); item < items;
       item += (long long)gridDim.x * (kThreads / 32)) {
    const int row = (int)(item / chunks) * 2 + (lane >> 4);
    const int h0 = (int)(item % chunks) * chunk, h1 = min(heads, h0 + chunk);
    bool mine = row < A.n_rows, place = false;
    int pos = 0;
    size_t slab = 0;              // the row's offset in a pool, without its head
    if (mine) {
      const int b = seq_of_row(A.row_offsets, A.B, row);
      const RowSeq s = row_seq(A.row_offsets, A.seq_lens, b, A.n_rows, A.mpp, A.status);
      mine = row >= s.row0 && row < s.row0 + s.n;
      pos = s.a + row - s.row0;
      if (mine && pos >= 0 && pos < A.mpp * kP && h1 > A.Hq) {
        const int phys = __ldg(A.page_table + (size_t)b * A.mpp + pos / kP);
        place = phys >= 0 && phys < A.num_pages;
        if (!place) set_status(A.status, SA_ERR_BAD_PAGE);
        slab = ((size_t)phys * A.Hk * kP + pos % kP) * kD;
      }
    }
    float cs[8], sn[8];
    if (h0 < A.Hq + A.Hk) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
      }
      if (mine && turned) {
        int axis_pos[SA_MAX_AXES];
#pragma unroll
        for (int a = 0; a < SA_MAX_AXES; ++a) {
          const bool used = a == 0 || A.axis_end[a - 1] < A.pairs;
          axis_pos[a] = A.positions == nullptr ? pos : used ? __ldg(A.positions + (size_t)a * A.n_rows + row) : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= npair) break;
          const int j = pair0 + i;
          const int x = j < A.axis_end[0] ? axis_pos[0] : j < A.axis_end[1] ? axis_pos[1] : j < A.axis_end[2] ? axis_pos[2] : axis_pos[3];
          const unsigned long long turn = (unsigned long long)(long long)x * s_freq[j];
          sincospif((float)(int)(turn >> 32) * 4.656612873077392578125e-10f, &sn[i], &cs[i]);
        }
      }
    }
    for (int hb = h0; hb < h1; hb += kInFlight) {
      uint4 x[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int h = hb + u;
        x[u] = make_uint4(0, 0, 0, 0);
        if (h < h1 && mine) {
          const __nv_bfloat16* src = h < A.Hq           ? A.q + row * A.q_stride + h * kD
                                     : h < A.Hq + A.Hk ? A.k + row * A.k_stride + (h - A.Hq) * kD
                                                       : A.v + row * A.v_stride + (h - A.Hq - A.Hk) * kD;
          x[u] = reinterpret_cast<const uint4*>(src)[hl];
        }
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int h = hb + u;
        if (h >= h1) break;
        uint4 y = x[u];
        if (h < A.Hq + A.Hk) {
          const __nv_bfloat16* wt = h < A.Hq ? A.q_weight : A.k_weight;
          float own[8], scale = 1.f;
          unpack(x[u], own);
          uint4 w4 = make_uint4(0, 0, 0, 0);
          if (wt != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(own[i], own[i], ss);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            scale = rsqrtf(ss * (1.f / kD) + A.eps);
            w4 = __ldg(reinterpret_cast<const uint4*>(wt) + hl);
            float w[8];
            unpack(w4, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) own[i] = own[i] * scale * w[i];
          }
          if (halves) {
            float other[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(0xffffffffu, own[i], partner);
#pragma unroll
            for (int i = 0; i < 8; ++i) own[i] = own[i] * cs[i] + (second ? other[i] : -other[i]) * sn[i];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = own[2 * i], b = own[2 * i + 1];
              own[2 * i] = a * cs[i] - b * sn[i];
              own[2 * i + 1] = b * cs[i] + a * sn[i];
            }
          }
          y = make_uint4(pack_bf16(own[0], own[1]), pack_bf16(own[2], own[3]), pack_bf16(own[4], own[5]),
                         pack_bf16(own[6], own[7]));
        }
        if (h < A.Hq) {
          if (mine) reinterpret_cast<uint4*>(A.q_out + ((size_t)row * A.Hq + h) * kD)[hl] = y;
        } else if (place) {
          const bool key = h < A.Hq + A.Hk;
          const int kvh = h - A.Hq - (key ? 0 : A.Hk);
          reinterpret_cast<uint4*>((key ? A.k_pool : A.v_pool) + slab + (size_t)kvh * kP * kD)[hl] = y;
        }
      }
    }
  }
}

}  // namespace

int launch_rotate(const RotateArgs& A, int num_sms, cudaStream_t stream) {
  const int heads = A.Hq + 2 * A.Hk;
  const long long pairs = (A.n_rows + 1) / 2;
  // heads of a warp's run: all of them once the rows alone fill the device
  // (a row's sines are then computed once), else as few as fill it
  int chunk = heads;
  while (chunk > kInFlight && pairs * ((heads + chunk - 1) / chunk) < (long long)num_sms * 16) chunk = (chunk + 1) / 2;
  chunk = std::max(kInFlight, (chunk + kInFlight - 1) / kInFlight * kInFlight);
  const int chunks = (heads + chunk - 1) / chunk;
  const long long blocks = (pairs * chunks + kThreads / 32 - 1) / (kThreads / 32);
  const int grid = (int)std::min<long long>(blocks, (long long)num_sms * 8);
  const cudaError_t e = launch_pdl(rotate_kernel, dim3(grid), dim3(kThreads), 0, stream, A, chunk, chunks);
  return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace sa
