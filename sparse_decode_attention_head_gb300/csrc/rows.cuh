// Packed rows: what the rotation, the prompt and tree attention and their ABI
// share.  Sequence b has n rows from row_offsets[b] on; they are its newest n
// tokens, row i at position L - n + i of the paged cache.
#pragma once

#include <cuda.h>

#include "sa_common.cuh"

namespace sa {

constexpr int kMaxTree = SA_MAX_TREE;

// One sequence's rows.  a = L - n may be negative (rows that see nothing).
struct RowSeq {
  int row0, n, L, a;
};

// Offsets are cut to the rows there are, the length to the page table; either
// cut is recorded once, by the caller that passes a status word.
__device__ __forceinline__ RowSeq row_seq(const int* row_offsets, const int* seq_lens, int b, int n_rows, int mpp,
                                          int* status) {
  const int o0 = __ldg(row_offsets + b), o1 = __ldg(row_offsets + b + 1), len = __ldg(seq_lens + b);
  RowSeq s;
  s.row0 = min(max(o0, 0), n_rows);
  const int e = min(max(o1, s.row0), n_rows);
  s.n = e - s.row0;
  if ((s.row0 != o0 || e != o1) && status != nullptr) set_status(status, SA_ERR_INVALID_ARG);
  const int cap = mpp * kP;
  if (len > cap && status != nullptr) set_status(status, SA_ERR_CAPACITY);
  s.a = max(len, 0) - s.n;      // of the true length: a row's position does not move when the table ends early
  s.L = min(max(len, 0), cap);
  return s;
}

// Sequence b's tokens in the pages of its group's prefix: whole pages ahead of
// its rows, or none where the number is not that (a sequence without rows has
// none to give).
__device__ __forceinline__ int shared_prefix(const int* prefix_lens, int b, const RowSeq& s, int mpp, int* status) {
  if (s.n == 0) return 0;
  const int x = __ldg(prefix_lens + b);
  if (x >= 0 && x % kP == 0 && x <= s.a && x <= mpp * kP) return x;
  if (status != nullptr) set_status(status, SA_ERR_INVALID_ARG);
  return 0;
}

// The rows of the members[b] sequences from b on, over the first prefix_lens[b]
// tokens of b: all of them see all of these (a = L, as of rows behind them).
__device__ __forceinline__ RowSeq shared_rows(const int* row_offsets, const int* members, const int* prefix_lens,
                                              int B, int b, int n_rows, int mpp) {
  const int m = min(__ldg(members + b), B - b), x = __ldg(prefix_lens + b), o0 = __ldg(row_offsets + b);
  RowSeq s{0, 0, 0, 0};
  if (m <= 0 || x <= 0 || x % kP != 0 || x > mpp * kP) return s;
  s.row0 = min(max(o0, 0), n_rows);
  s.n = min(max(__ldg(row_offsets + b + m), s.row0), n_rows) - s.row0;
  s.a = s.L = x;
  return s;
}

// ---------------------------------------------------------------- attention

// One KV head of a sequence with up to two query tiles of its rows, and how
// many pages they see some of.
struct __align__(16) SparseItem {
  int b, kvh, i, pages;
  int row0, tokens, pos0, end;      // first packed row, rows, position of the first, first position that none sees
};
// What work weighs: a tile, and an item's query load, first tile and epilogue.
constexpr int kSparseTileCost = 3, kSparseItemCost = 8;

constexpr int kRowsMaxCtas = 192;   // one block an SM; bounds the workspace

struct RowsAttnArgs {
  const __nv_bfloat16* v_pool;
  const int* page_table;
  const int* seq_lens;
  const int* row_offsets;
  const unsigned long long* tree;   // [n_rows] words of a tree, NULL: causal
  __nv_bfloat16* out;               // [n_rows][Hq][kD]
  float* lse;                       // [n_rows][Hq] or NULL
  float* part;                      // split items: [cta][2][2][kD / 4][128][4] sums
  float2* part_ml;                  // [cta][2][2][128] (maximum, sum), base 2
  int4* desc;                       // [cta][2] what the partials are of
  int* status;
  int n_rows, B, Hq, Hk, G, mpp, num_pages;
  int tpt;                          // tokens of a query tile: 128 / G
  float scale_log2;                 // scale log2(e)
};
// With shared prefixes or selected blocks.  (Apart: with these fields the kernel
// of prompts keeps its arguments elsewhere and takes 1448 us in place of 1397 for
// 16384 rows.)
struct RowsMoreArgs : RowsAttnArgs {
  // shared prefixes only
  const int* members;               // [B] sequences of the group that b leads, 0 elsewhere
  const int* prefix_lens;           // [B] tokens of the group's prefix
  float* half;                      // [2][n_rows][Hq][kD] sums over the prefix and over a sequence's own tokens
  float2* half_ml;                  // [2][n_rows][Hq] (maximum, sum), base 2
  bool join_own;                    // few own tokens are attended where the two are joined
  // these two in both
  const __nv_bfloat16* q;           // [n_rows][Hq][kD]
  const __nv_bfloat16* k_pool;
  // selected blocks only
  const int* sel_idx;               // [n_rows][Hq][kcap] blocks, ascending
  const int* sel_cnt;               // [n_rows][Hq]
  SparseItem* items;                // [n_items]
  long long* before;                // [n_items + 1] weight of the items before
  uint32_t* pages;                  // [n_items][words] a bit for each page that some row of the item sees
  int* ranks;                       // [n_rows][Hq][rank_stride] a row's blocks as places in that list
  int* ticket;                      // the next item to take (of those behind one a block), items there are
  int* arrived;                     // in the workspace's header: blocks that are done, zero between calls
  int n_items, words;               // at most that many; ceil(mpp / 32)
  int kcap, rank_stride, S, W;      // rank_stride: kcap up to a multiple of four
  unsigned char bs_shift[SA_MAX_HK];
};

int launch_rows_attention(const RowsAttnArgs& A, const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                          int num_sms, cudaStream_t stream);
int launch_shared_attention(const RowsMoreArgs& A, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                            const CUtensorMap& tmV, int num_sms, cudaStream_t stream);

int launch_sparse_items(const RowsMoreArgs& A, cudaStream_t stream);
int launch_sparse_attention(const RowsMoreArgs& A, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                            const CUtensorMap& tmV, int num_sms, cudaStream_t stream);
int launch_shared_prefixes(const int* table, const int* seq_lens, const int* row_offsets, const int* group_offsets,
                           int n_groups, int min_tokens, int* members, int* prefix_lens, int B, int mpp, int num_pages,
                           int* status, cudaStream_t stream);

// ---------------------------------------------------------------- items

// Where item u lies when each KV head of a sequence's n rows is ceil(n / T)
// items: sequences in order, their KV heads in order, runs of T rows in order.
struct ItemPlace {
  int b, kvh, i;     // b < 0: there is no such item
};

// A whole block of THREADS; the answer is in *place behind the call.  Item 0's
// block looks at every sequence, for their errors.
template <int THREADS>
__device__ __forceinline__ void find_item(const int* row_offsets, const int* seq_lens, int B, int n_rows, int mpp,
                                          int Hk, int T, int u, int* status, ItemPlace* place) {
  __shared__ int s_sum[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) *place = ItemPlace{-1, 0, 0};
  __syncthreads();
  int carry = 0;
  for (int b0 = 0; b0 < B; b0 += THREADS) {
    const int b = b0 + tid;
    int runs = 0;
    if (b < B) {
      const RowSeq s = row_seq(row_offsets, seq_lens, b, n_rows, mpp, u == 0 ? status : nullptr);
      runs = (s.n + T - 1) / T;
    }
    const int mine = runs * Hk, incl = warp_incl_scan(mine);
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int upto = carry + incl, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) upto += s_sum[w];
      total += s_sum[w];
    }
    if (u >= upto - mine && u < upto) {
      const int rem = u - (upto - mine);
      *place = ItemPlace{b, rem / runs, rem % runs};
    }
    __syncthreads();
    carry += total;
    if (u > 0 && place->b >= 0) break;
  }
}

// ---------------------------------------------------------------- selection

struct SelectArgs {
  const __nv_bfloat16* q;           // [n_rows][Hq][kD]
  const __nv_bfloat16* summaries;   // [B][Hk][slots][2][kD] or [B][Hk][slots][kD]
  const int *row_offsets, *seq_lens;
  int* sel_idx;                     // [n_rows][Hq][kcap]
  int* sel_cnt;                     // [n_rows][Hq]
  float* scores;                    // scratch
  int* norms;                       // [B][Hk] the bits of the largest squared norm of a summary
  int* status;
  int n_rows, n_items, B, Hq, Hk, G, mpp, slots, kcap, S, W;
  bool minmax, group;
  int bs[SA_MAX_HK];
  int k[SA_MAX_HQ];
};

// rows_select.cu: any number of rows, up to 65536 candidates
int launch_score_rows(const SelectArgs& A, int max_candidates, cudaStream_t stream);
size_t score_rows_scratch(int slots, long long n_items);
// rows_select_tc.cu: many rows
constexpr int kTcMaxSlots = 4096;
int launch_select_tc(const SelectArgs& A, const CUtensorMap& tmQ, const CUtensorMap& tmS, int num_sms,
                     cudaStream_t stream);
size_t select_tc_scratch(int slots, long long n_items);

// ---------------------------------------------------------------- rotation

struct RotateArgs {
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, k_stride, v_stride;   // elements between rows
  const __nv_bfloat16 *q_weight, *k_weight;
  const float* inv_freq;                    // [pairs]
  const int* positions;                     // [axes][n_rows] or NULL
  const int *row_offsets, *seq_lens, *page_table;
  __nv_bfloat16 *q_out, *k_pool, *v_pool;
  int* status;
  float eps;
  int n_rows, B, Hq, Hk, mpp, num_pages;
  int pairs;       // R / 2; 0: no rotation
  int layout;
  int axis_end[SA_MAX_AXES];   // pairs up to and with axis a
};

int launch_rotate(const RotateArgs& A, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------- pages

struct PageArgs {
  const int* table_in;
  const int* parent;      // plan only
  const int* keep;        // tokens a row keeps (plan) or holds (compact)
  const int* lens;        // plan only: tokens a row gets room for
  int* table_out;
  int* src;               // plan: [B], compact: [num_pages]
  int* dst;
  int* counts;
  int* refs;              // [num_pages] rows that hold a page
  int* writers;           // [num_pages] rows that will write inside it (plan)
  int* lowest;            // [num_pages] kMaxPlanRows - the lowest of them (plan)
  int* list;              // [num_pages] plan: free pages; compact: a moved page's rank
  int* chunk;             // per chunk of pages: free (plan) or live (compact) ones
  int* need;              // [B + 1] plan: new pages of the rows before
  int* status;
  int B, mpp, num_pages;
};
constexpr int kMaxPlanRows = 1024;
constexpr int kPageChunk = 1024;

int launch_plan_pages(const PageArgs& A, cudaStream_t stream);
int launch_compact_pages(const PageArgs& A, cudaStream_t stream);
int launch_copy_pages(void* k_pool, void* v_pool, const int* src, const int* dst, const int* count, int max_pages,
                      int num_pages, int Hk, int* status, int num_sms, cudaStream_t stream);
int launch_accept_rows(void* k_pool, void* v_pool, const int* page_table, const int* base_lens, const int* path,
                       int max_path, const int* path_cnt, int B, int Hk, int mpp, int num_pages, int* status,
                       cudaStream_t stream);

}  // namespace sa
