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

// ---------------------------------------------------------------- attention

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

int launch_rows_attention(const RowsAttnArgs& A, const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                          int num_sms, cudaStream_t stream);

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
