// The C ABI of the packed-row and page calls (declared in include/sa.h):
// argument checks, workspace layout, TMA descriptors, launches.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "launch.cuh"
#include "rows.cuh"

using sa::Params;

namespace {

constexpr size_t kAlign = 256;
size_t up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }
bool aligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }
cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// Counts of table entries and loops over sequences are 32-bit on the device: a
// table of 2^30 entries or more (4 GB) is refused by every call here.
int make_params(const sa_problem* prob, Params* p) {
  const int rc = sa_host::make_params(prob, p);
  if (rc != SA_OK) return rc;
  return (long long)p->B * p->mpp < (1ll << 30) ? SA_OK : SA_ERR_UNSUPPORTED;
}

constexpr long long kMaxItems = 1 << 30;     // indices of items are 32-bit
constexpr int kMaxSparsePages = 100 * 1024 * 8;   // an item's bitmap of pages lies in shared memory: 13 M tokens

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x < y + nb && y < x + na;
}

// The attention's partials and the page calls' counts share the space behind
// the header: calls on one workspace are ordered on one stream.
struct AttnLayout {
  size_t desc, ml, part, total;
};
AttnLayout attn_layout() {
  constexpr size_t pieces = (size_t)sa::kRowsMaxCtas * 2;
  AttnLayout l;
  size_t off = up(sizeof(sa::WsHeader));
  l.desc = off;
  off = up(off + pieces * sizeof(int4));
  l.ml = off;
  off = up(off + pieces * 2 * 128 * sizeof(float2));
  l.part = off;
  off = up(off + pieces * 2 * 128 * sa::kD * sizeof(float));
  l.total = off;
  return l;
}

// The two parts of rows behind a shared prefix, behind the partials.
struct SharedLayout {
  size_t ml, half, total;
};
SharedLayout shared_layout(const Params& p, int n_rows) {
  const size_t rows = 2 * (size_t)n_rows * p.Hq;
  SharedLayout l;
  size_t off = attn_layout().total;
  l.ml = off;
  off = up(off + rows * sizeof(float2));
  l.half = off;
  off = up(off + rows * sa::kD * sizeof(float));
  l.total = off;
  return l;
}

// Items of the calls with selected blocks, `rows` rows and heads each.
long long max_items(const Params& p, int n_rows, int rows) {
  const int T = rows == 256 ? 2 * (128 / p.G) : rows / p.G;
  return ((long long)n_rows / T + std::min(p.B, n_rows)) * p.Hk;
}

// The sparse attention's items behind the partials.
struct SparseLayout {
  size_t items, before, ticket, pages, ranks, total;
  int words, rank_stride;
};
SparseLayout sparse_layout(const Params& p, int n_rows) {
  const size_t n = (size_t)max_items(p, n_rows, 256);
  SparseLayout l;
  l.words = (p.mpp + 31) / 32;
  l.rank_stride = (p.kcap + 3) & ~3;
  size_t off = attn_layout().total;
  l.items = off;
  off = up(off + n * sizeof(sa::SparseItem));
  l.before = off;
  off = up(off + (n + 1) * sizeof(long long));
  l.ticket = off;
  off = up(off + 2 * sizeof(int));
  l.pages = off;
  off = up(off + n * l.words * sizeof(uint32_t));
  l.ranks = off;
  off = up(off + (size_t)n_rows * p.Hq * l.rank_stride * sizeof(int));
  l.total = off;
  return l;
}

// The selection's scratch behind the norms.
constexpr int kSelectMaxSlots = 1024 * 64;      // candidates that a block's top-k holds
// Which form takes less, from what each measured (32 heads over 8): the tensor
// cores' one a round of two items an SM, 15 us and 0.16 us a candidate block;
// the canonical one 15 us and 1 us for 60000 scores.  At most 40 blocks kept:
// 8 x 64 rows of 8K, blocks of 64: 32 us against 100; 8 x 8 rows of 32K, blocks
// of 16: 330 us against 81.  Longer lists, whose k-th is looked for among all
// candidates, took the tensor form 1.4 to 4.6 times what lists of 40 did; they
// count seven times here, which leaves them to it in groups alone.  Per head: 41
// of 256 blocks for 16384 rows 1384 us against 2755 here, 41 of 512 for 32768
// 7865 against 7403, 100 of 2048 for 32768 26.1 ms against 20.9.
// Both are bounded by the table's width, not by lengths, which the host does not see.
// ctas: blocks that run at a time; 0: for a workspace, whether any number of rows
// up to n_rows takes the tensor form (a round is the least it needs).
bool select_by_tensor(const Params& p, int n_rows, int ctas) {
  if (p.slots > sa::kTcMaxSlots || (long long)p.B * p.Hk * p.slots >= (1ll << 31)) return false;
  const int T = p.sel_mode == SA_SELECT_GROUP ? 128 : 128 / p.G;
  const int k = *std::max_element(p.k, p.k + p.Hq);
  const long long items = ((long long)n_rows / T + std::min(p.B, n_rows)) * p.Hk;
  const long long rounds = ctas == 0 ? 1 : (items + ctas - 1) / ctas;
  const double tensor = rounds * (15.0 + 0.16 * p.slots) * (k > 40 ? 7.0 : 1.0);
  return tensor < 15.0 + (double)n_rows * p.Hq * p.slots / 60e3;
}
struct SelectLayout {
  size_t norms, scores, total;
};
SelectLayout select_layout(const Params& p, int n_rows) {
  SelectLayout l;
  size_t off = up(sizeof(sa::WsHeader));
  l.norms = off;
  off = up(off + (size_t)p.B * p.Hk * sizeof(int));
  l.scores = off;
  // a workspace for n_rows serves fewer too, in either form
  size_t scores = sa::score_rows_scratch(p.slots, max_items(p, n_rows, 32));
  if (select_by_tensor(p, n_rows, 0))
    scores = std::max(scores, sa::select_tc_scratch(p.slots, max_items(p, n_rows, 128)));
  off = up(off + scores);
  l.total = off;
  return l;
}

struct PageLayout {
  size_t refs, list, chunk, need, total;
};
PageLayout page_layout(const Params& p) {
  const size_t pages = (size_t)p.num_pages;
  PageLayout l;
  size_t off = up(sizeof(sa::WsHeader));
  l.refs = off;    // holders, writers and lowest writers, one behind the other
  off = up(off + 3 * pages * sizeof(int));
  l.list = off;
  off = up(off + pages * sizeof(int));
  l.chunk = off;
  off = up(off + (pages / sa::kPageChunk + 2) * sizeof(int));
  l.need = off;
  off = up(off + 2 * (sa::kMaxPlanRows + 1) * sizeof(int));
  l.total = off;
  return l;
}

// q [n_rows][Hq][D] as boxes of 64 dims x G heads x some tokens.
int make_q_map(CUtensorMap* m, const void* q, int n_rows, const Params& p, int tokens) {
  auto fn = sa_host::encode_fn();
  if (fn == nullptr) return SA_ERR_CUDA;
  cuuint64_t dims[3] = {SA_HEAD_DIM, (cuuint64_t)p.Hq, (cuuint64_t)n_rows};
  cuuint64_t strides[2] = {SA_HEAD_DIM * 2, (cuuint64_t)p.Hq * SA_HEAD_DIM * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SA_OK : SA_ERR_CUDA;
}

// Summaries [B][Hk][slots] as boxes of 64 dims of the minimum, the maximum or
// the mean of 64 blocks.
int make_summary_map(CUtensorMap* m, const void* summaries, const Params& p) {
  auto fn = sa_host::encode_fn();
  if (fn == nullptr) return SA_ERR_CUDA;
  const cuuint64_t kinds = p.mode == SA_SUMMARY_MINMAX ? 2 : 1;
  cuuint64_t dims[3] = {SA_HEAD_DIM, kinds, (cuuint64_t)p.B * p.Hk * p.slots};
  cuuint64_t strides[2] = {SA_HEAD_DIM * 2, kinds * SA_HEAD_DIM * 2};
  cuuint32_t box[3] = {64, 1, 64};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(summaries), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SA_OK : SA_ERR_CUDA;
}

// A pool as (64 dims, 8 tokens, 2 halves of a row, groups of 8 tokens): one
// box of 64 x 8 x 2 x 2 is a page's 4 KB slab of one head, landing as
// [group][half][8][64], so that groups of 8 tokens lie 2 KB apart throughout
// a tile of several pages, the one stride a matrix descriptor has.
int make_tile_map(CUtensorMap* m, const void* pool, const Params& p) {
  auto fn = sa_host::encode_fn();
  if (fn == nullptr) return SA_ERR_CUDA;
  cuuint64_t dims[4] = {64, 8, 2, (cuuint64_t)p.num_pages * p.Hk * (SA_PAGE_SIZE / 8)};
  cuuint64_t strides[3] = {SA_HEAD_DIM * 2, 128, 8 * SA_HEAD_DIM * 2};
  cuuint32_t box[4] = {64, 8, 2, 2};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SA_OK : SA_ERR_CUDA;
}

// The checks and arguments that the attention calls share; launch says whether
// there is anything to do, `rest` whether a call's other arguments are there.
struct AttnCall {
  Params p;
  sa::RowsMoreArgs A;
  CUtensorMap tmQ, tmK, tmV;
  int nsm;
  bool launch;
};
int attention_args(const sa_problem* prob, int32_t n_rows, const void* q, const void* k_pool, const void* v_pool,
                   const int32_t* page_table, const int32_t* seq_lens, const int32_t* row_offsets, void* out, float* lse,
                   void* ws, bool rest, AttnCall* c) {
  Params& p = c->p;
  c->launch = false;
  int rc = make_params(prob, &p);
  if (rc != SA_OK) return rc;
  if (n_rows < 0) return SA_ERR_INVALID_ARG;
  if (!k_pool || !v_pool || !page_table || !seq_lens || !row_offsets || !ws || !rest) return SA_ERR_INVALID_ARG;
  if (n_rows == 0) return SA_OK;
  if (!q || !out) return SA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out) || !aligned16(ws))
    return SA_ERR_INVALID_ARG;
  const size_t row_bytes = (size_t)n_rows * p.Hq * SA_HEAD_DIM * 2;
  if (overlap(q, row_bytes, out, row_bytes)) return SA_ERR_INVALID_ARG;
  c->nsm = sa_host::num_sms_current();
  if (c->nsm <= 0) return SA_ERR_CUDA;
  sa::RowsMoreArgs& A = c->A;
  A = sa::RowsMoreArgs{};
  A.tpt = 128 / p.G;
  if ((rc = make_q_map(&c->tmQ, q, n_rows, p, A.tpt)) != SA_OK) return rc;
  if ((rc = make_tile_map(&c->tmK, k_pool, p)) != SA_OK) return rc;
  if ((rc = make_tile_map(&c->tmV, v_pool, p)) != SA_OK) return rc;
  const AttnLayout l = attn_layout();
  A.v_pool = static_cast<const __nv_bfloat16*>(v_pool);
  A.page_table = page_table;
  A.seq_lens = seq_lens;
  A.row_offsets = row_offsets;
  A.out = static_cast<__nv_bfloat16*>(out);
  A.lse = lse;
  A.part = at<float>(ws, l.part);
  A.part_ml = at<float2>(ws, l.ml);
  A.desc = at<int4>(ws, l.desc);
  A.status = at<int>(ws, 0);
  A.n_rows = n_rows;
  A.B = p.B;
  A.Hq = p.Hq;
  A.Hk = p.Hk;
  A.G = p.G;
  A.mpp = p.mpp;
  A.num_pages = p.num_pages;
  A.scale_log2 = p.scale * 1.4426950408889634f;
  c->launch = true;
  return SA_OK;
}

int rows_attention(const sa_problem* prob, int32_t n_rows, const void* q, const void* k_pool, const void* v_pool,
                   const int32_t* page_table, const int32_t* seq_lens, const int32_t* row_offsets, const uint64_t* tree,
                   void* out, float* lse, void* ws, void* stream) {
  AttnCall c;
  const int rc =
      attention_args(prob, n_rows, q, k_pool, v_pool, page_table, seq_lens, row_offsets, out, lse, ws, true, &c);
  if (rc != SA_OK || !c.launch) return rc;
  c.A.tree = reinterpret_cast<const unsigned long long*>(tree);
  return sa::launch_rows_attention(c.A, c.tmQ, c.tmK, c.tmV, c.nsm, as_stream(stream));
}

int page_args(const sa_problem* prob, const int32_t* table_in, const int32_t* keep, int32_t* table_out, int32_t* src,
              int32_t* dst, int32_t* counts, void* ws, Params* p, sa::PageArgs* A) {
  const int rc = make_params(prob, p);
  if (rc != SA_OK) return rc;
  if (!table_in || !keep || !table_out || !src || !dst || !counts || !ws) return SA_ERR_INVALID_ARG;
  if (!aligned16(ws)) return SA_ERR_INVALID_ARG;
  const size_t bytes = (size_t)p->B * p->mpp * sizeof(int32_t);
  if (overlap(table_in, bytes, table_out, bytes)) return SA_ERR_INVALID_ARG;
  const PageLayout l = page_layout(*p);
  A->table_in = table_in;
  A->parent = nullptr;
  A->keep = keep;
  A->lens = nullptr;
  A->table_out = table_out;
  A->src = src;
  A->dst = dst;
  A->counts = counts;
  A->refs = at<int>(ws, l.refs);
  A->writers = A->refs + p->num_pages;
  A->lowest = A->writers + p->num_pages;
  A->list = at<int>(ws, l.list);
  A->chunk = at<int>(ws, l.chunk);
  A->need = at<int>(ws, l.need);
  A->status = at<int>(ws, 0);
  A->B = p->B;
  A->mpp = p->mpp;
  A->num_pages = p->num_pages;
  return SA_OK;
}

}  // namespace

extern "C" {

size_t sa_rows_workspace_size(const sa_problem* prob) {
  Params p;
  if (make_params(prob, &p) != SA_OK) return 0;
  return std::max(attn_layout().total, page_layout(p).total);
}

int sa_qk_norm_rope(const sa_problem* prob, int32_t n_rows, const void* q, int64_t q_stride, const void* k,
                    int64_t k_stride, const void* v, int64_t v_stride, const void* q_weight_or_null,
                    const void* k_weight_or_null, float eps, const sa_rope* rope_or_null, const float* inv_freq,
                    const int32_t* positions_or_null, const int32_t* row_offsets, const int32_t* seq_lens,
                    const int32_t* page_table, void* q_out, void* k_pool, void* v_pool, void* ws, void* stream) {
  Params p;
  int rc = make_params(prob, &p);
  if (rc != SA_OK) return rc;
  if (n_rows < 0 || !(eps >= 0.f) || !std::isfinite(eps)) return SA_ERR_INVALID_ARG;
  if (!row_offsets || !seq_lens || !page_table || !k_pool || !v_pool || !ws) return SA_ERR_INVALID_ARG;
  sa::RotateArgs A{};
  if (rope_or_null != nullptr) {
    const sa_rope& r = *rope_or_null;
    if (r.layout != SA_ROPE_HALVES && r.layout != SA_ROPE_PAIRS) return SA_ERR_INVALID_ARG;
    if (r.axes < 1 || r.axes > SA_MAX_AXES || inv_freq == nullptr) return SA_ERR_INVALID_ARG;
    long long pairs = 0;
    for (int a = 0; a < SA_MAX_AXES; ++a) {
      if (a < r.axes) {
        if (r.axis_pairs[a] < 0) return SA_ERR_INVALID_ARG;
        pairs += r.axis_pairs[a];
        if (pairs > SA_HEAD_DIM / 2) return SA_ERR_INVALID_ARG;
      }
      A.axis_end[a] = (int)pairs;
    }
    if (pairs < 1) return SA_ERR_INVALID_ARG;
    if (pairs % 8 != 0 && r.axes == 1) return SA_ERR_UNSUPPORTED;
    A.pairs = (int)pairs;
    A.layout = r.layout;
  }
  if (n_rows == 0) return SA_OK;
  if (!q || !k || !v || !q_out) return SA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_pool) ||
      !aligned16(v_pool) || !aligned16(ws))
    return SA_ERR_INVALID_ARG;
  if ((q_weight_or_null && !aligned16(q_weight_or_null)) || (k_weight_or_null && !aligned16(k_weight_or_null)))
    return SA_ERR_INVALID_ARG;
  const int64_t q_row = (int64_t)p.Hq * SA_HEAD_DIM, kv_row = (int64_t)p.Hk * SA_HEAD_DIM;
  if (q_stride % 8 || k_stride % 8 || v_stride % 8 || q_stride < q_row || k_stride < kv_row || v_stride < kv_row)
    return SA_ERR_INVALID_ARG;
  const size_t out_bytes = (size_t)n_rows * q_row * 2;
  auto span = [&](int64_t stride, int64_t row) { return (size_t)((n_rows - 1) * stride + row) * 2; };
  if (!(q_out == q && q_stride == q_row) && overlap(q, span(q_stride, q_row), q_out, out_bytes))
    return SA_ERR_INVALID_ARG;
  if (overlap(k, span(k_stride, kv_row), q_out, out_bytes) || overlap(v, span(v_stride, kv_row), q_out, out_bytes))
    return SA_ERR_INVALID_ARG;
  const int nsm = sa_host::num_sms_current();
  if (nsm <= 0) return SA_ERR_CUDA;
  A.q = static_cast<const __nv_bfloat16*>(q);
  A.k = static_cast<const __nv_bfloat16*>(k);
  A.v = static_cast<const __nv_bfloat16*>(v);
  A.q_stride = q_stride;
  A.k_stride = k_stride;
  A.v_stride = v_stride;
  A.q_weight = static_cast<const __nv_bfloat16*>(q_weight_or_null);
  A.k_weight = static_cast<const __nv_bfloat16*>(k_weight_or_null);
  A.inv_freq = inv_freq;
  A.positions = positions_or_null;
  A.row_offsets = row_offsets;
  A.seq_lens = seq_lens;
  A.page_table = page_table;
  A.q_out = static_cast<__nv_bfloat16*>(q_out);
  A.k_pool = static_cast<__nv_bfloat16*>(k_pool);
  A.v_pool = static_cast<__nv_bfloat16*>(v_pool);
  A.status = at<int>(ws, 0);
  A.eps = eps;
  A.n_rows = n_rows;
  A.B = p.B;
  A.Hq = p.Hq;
  A.Hk = p.Hk;
  A.mpp = p.mpp;
  A.num_pages = p.num_pages;
  return sa::launch_rotate(A, nsm, as_stream(stream));
}

int sa_prompt_attention(const sa_problem* prob, int32_t n_rows, const void* q, const void* k_pool, const void* v_pool,
                        const int32_t* page_table, const int32_t* seq_lens, const int32_t* row_offsets, void* out,
                        float* lse_or_null, void* ws, void* stream) {
  return rows_attention(prob, n_rows, q, k_pool, v_pool, page_table, seq_lens, row_offsets, nullptr, out, lse_or_null,
                        ws, stream);
}

int sa_tree_attention(const sa_problem* prob, int32_t n_rows, const void* q, const void* k_pool, const void* v_pool,
                      const int32_t* page_table, const int32_t* seq_lens, const int32_t* row_offsets,
                      const uint64_t* tree_mask, void* out, float* lse_or_null, void* ws, void* stream) {
  if (tree_mask == nullptr && n_rows != 0) return SA_ERR_INVALID_ARG;
  return rows_attention(prob, n_rows, q, k_pool, v_pool, page_table, seq_lens, row_offsets, tree_mask, out, lse_or_null,
                        ws, stream);
}

size_t sa_shared_workspace_size(const sa_problem* prob, int32_t max_rows) {
  Params p;
  if (make_params(prob, &p) != SA_OK || max_rows < 0) return 0;
  return std::max(sa_rows_workspace_size(prob), shared_layout(p, max_rows).total);
}

int sa_shared_prefixes(const sa_problem* prob, const int32_t* page_table, const int32_t* seq_lens,
                       const int32_t* row_offsets, const int32_t* group_offsets, int32_t n_groups, int32_t min_tokens,
                       int32_t* members, int32_t* prefix_lens, void* ws, void* stream) {
  Params p;
  const int rc = make_params(prob, &p);
  if (rc != SA_OK) return rc;
  if (!page_table || !seq_lens || !row_offsets || !group_offsets || !members || !prefix_lens || !ws)
    return SA_ERR_INVALID_ARG;
  if (!aligned16(ws) || n_groups < 0 || n_groups > p.B) return SA_ERR_INVALID_ARG;
  return sa::launch_shared_prefixes(page_table, seq_lens, row_offsets, group_offsets, n_groups, min_tokens, members,
                                    prefix_lens, p.B, p.mpp, p.num_pages, at<int>(ws, 0), as_stream(stream));
}

int sa_shared_attention(const sa_problem* prob, int32_t n_rows, const void* q, const void* k_pool, const void* v_pool,
                        const int32_t* page_table, const int32_t* seq_lens, const int32_t* row_offsets,
                        const uint64_t* tree_mask_or_null, const int32_t* members, const int32_t* prefix_lens, void* out,
                        float* lse_or_null, void* ws, void* stream) {
  AttnCall c;
  const int rc = attention_args(prob, n_rows, q, k_pool, v_pool, page_table, seq_lens, row_offsets, out, lse_or_null, ws,
                                members != nullptr && prefix_lens != nullptr, &c);
  if (rc != SA_OK || !c.launch) return rc;
  const SharedLayout l = shared_layout(c.p, n_rows);
  c.A.tree = reinterpret_cast<const unsigned long long*>(tree_mask_or_null);
  c.A.members = members;
  c.A.prefix_lens = prefix_lens;
  c.A.q = static_cast<const __nv_bfloat16*>(q);
  c.A.k_pool = static_cast<const __nv_bfloat16*>(k_pool);
  c.A.half = at<float>(ws, l.half);
  c.A.half_ml = at<float2>(ws, l.ml);
  return sa::launch_shared_attention(c.A, c.tmQ, c.tmK, c.tmV, c.nsm, as_stream(stream));
}

size_t sa_sparse_workspace_size(const sa_problem* prob, int32_t max_rows) {
  Params p;
  if (make_params(prob, &p) != SA_OK || max_rows < 0 || max_items(p, max_rows, 32) > kMaxItems) return 0;
  if (p.mpp > kMaxSparsePages) return 0;      // neither call takes it: that many pages are more slots than kSelectMaxSlots
  return std::max({sa_rows_workspace_size(prob), sparse_layout(p, max_rows).total,
                   p.slots <= kSelectMaxSlots ? select_layout(p, max_rows).total : 0});
}

int sa_select_rows(const sa_problem* prob, int32_t n_rows, const void* q, const void* summaries,
                   const int32_t* seq_lens, const int32_t* row_offsets, int32_t* sel_idx, int32_t* sel_cnt, void* ws,
                   void* stream) {
  Params p;
  const int rc = make_params(prob, &p);
  if (rc != SA_OK) return rc;
  if (n_rows < 0 || !summaries || !seq_lens || !row_offsets || !ws) return SA_ERR_INVALID_ARG;
  if (max_items(p, n_rows, 32) > kMaxItems || p.slots > kSelectMaxSlots) return SA_ERR_UNSUPPORTED;
  if (n_rows == 0) return SA_OK;
  if (!q || !sel_idx || !sel_cnt) return SA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(summaries) || !aligned16(ws)) return SA_ERR_INVALID_ARG;
  int nsm = sa_host::num_sms_current();
  if (nsm <= 0) return SA_ERR_CUDA;
  nsm = std::min(nsm, sa::kRowsMaxCtas);
  sa::SelectArgs A{};
  A.q = static_cast<const __nv_bfloat16*>(q);
  A.summaries = static_cast<const __nv_bfloat16*>(summaries);
  A.row_offsets = row_offsets;
  A.seq_lens = seq_lens;
  A.sel_idx = sel_idx;
  A.sel_cnt = sel_cnt;
  const SelectLayout l = select_layout(p, n_rows);
  A.scores = at<float>(ws, l.scores);
  A.norms = at<int>(ws, l.norms);
  A.status = at<int>(ws, 0);
  A.n_rows = n_rows;
  A.B = p.B;
  A.Hq = p.Hq;
  A.Hk = p.Hk;
  A.G = p.G;
  A.mpp = p.mpp;
  A.slots = p.slots;
  A.kcap = p.kcap;
  A.S = p.S;
  A.W = p.W;
  A.minmax = p.mode == SA_SUMMARY_MINMAX;
  A.group = p.sel_mode == SA_SELECT_GROUP;
  std::copy(p.bs, p.bs + p.Hk, A.bs);
  std::copy(p.k, p.k + p.Hq, A.k);
  if (!select_by_tensor(p, n_rows, 2 * nsm)) {
    A.n_items = (int)max_items(p, n_rows, 32);
    return sa::launch_score_rows(A, p.slots, as_stream(stream));
  }
  const int T = A.group ? 128 : 128 / p.G;
  A.n_items = (int)(((long long)n_rows / T + std::min(p.B, n_rows)) * p.Hk);
  CUtensorMap tmQ{}, tmS;
  int e = A.group ? SA_OK : make_q_map(&tmQ, q, n_rows, p, T);      // the sum of a group's queries is no copy of them
  if (e == SA_OK) e = make_summary_map(&tmS, summaries, p);
  return e == SA_OK ? sa::launch_select_tc(A, tmQ, tmS, nsm, as_stream(stream)) : e;
}

int sa_sparse_row_attention(const sa_problem* prob, int32_t n_rows, const void* q, const void* k_pool,
                            const void* v_pool, const int32_t* page_table, const int32_t* seq_lens,
                            const int32_t* row_offsets, const int32_t* sel_idx, const int32_t* sel_cnt, void* out,
                            float* lse_or_null, void* ws, void* stream) {
  AttnCall c;
  const int rc = attention_args(prob, n_rows, q, k_pool, v_pool, page_table, seq_lens, row_offsets, out, lse_or_null, ws,
                                sel_idx != nullptr && sel_cnt != nullptr, &c);
  if (rc != SA_OK) return rc;
  const Params& p = c.p;
  if (max_items(p, n_rows, 32) > kMaxItems || p.mpp > kMaxSparsePages) return SA_ERR_UNSUPPORTED;
  if (!c.launch) return SA_OK;
  const SparseLayout l = sparse_layout(p, n_rows);
  sa::RowsMoreArgs& A = c.A;
  A.q = static_cast<const __nv_bfloat16*>(q);
  A.k_pool = static_cast<const __nv_bfloat16*>(k_pool);
  A.sel_idx = sel_idx;
  A.sel_cnt = sel_cnt;
  A.items = at<sa::SparseItem>(ws, l.items);
  A.before = at<long long>(ws, l.before);
  A.ticket = at<int>(ws, l.ticket);
  A.arrived = at<sa::WsHeader>(ws, 0)->pad;
  A.pages = at<uint32_t>(ws, l.pages);
  A.n_items = (int)max_items(p, n_rows, 256);
  A.words = l.words;
  A.ranks = at<int>(ws, l.ranks);
  A.rank_stride = l.rank_stride;
  A.kcap = p.kcap;
  A.S = std::min(p.S, 1 << 30);
  A.W = p.W;      // of a row behind the table the window may begin in it however far that is
  for (int h = 0; h < p.Hk; ++h) A.bs_shift[h] = (unsigned char)(p.bs[h] == 8 ? 3 : p.bs[h] == 16 ? 4 : p.bs[h] == 32 ? 5 : 6);
  return sa::launch_sparse_attention(A, c.tmQ, c.tmK, c.tmV, c.nsm, as_stream(stream));
}

int sa_accept_rows(const sa_problem* prob, void* k_pool, void* v_pool, const int32_t* page_table,
                   const int32_t* base_lens, const int32_t* path, int32_t max_path, const int32_t* path_cnt, void* ws,
                   void* stream) {
  Params p;
  const int rc = make_params(prob, &p);
  if (rc != SA_OK) return rc;
  if (!k_pool || !v_pool || !page_table || !base_lens || !path || !path_cnt || !ws) return SA_ERR_INVALID_ARG;
  if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(ws)) return SA_ERR_INVALID_ARG;
  if (max_path < 1) return SA_ERR_INVALID_ARG;
  if (max_path > SA_MAX_TREE || p.B > 65535) return SA_ERR_UNSUPPORTED;
  return sa::launch_accept_rows(k_pool, v_pool, page_table, base_lens, path, max_path, path_cnt, p.B, p.Hk, p.mpp,
                                p.num_pages, at<int>(ws, 0), as_stream(stream));
}

int sa_plan_pages(const sa_problem* prob, const int32_t* table_in, const int32_t* parent, const int32_t* keep,
                  const int32_t* lens, int32_t* table_out, int32_t* copy_src, int32_t* copy_dst, int32_t* counts,
                  void* ws, void* stream) {
  Params p;
  sa::PageArgs A;
  const int rc = page_args(prob, table_in, keep, table_out, copy_src, copy_dst, counts, ws, &p, &A);
  if (rc != SA_OK) return rc;
  if (!parent || !lens) return SA_ERR_INVALID_ARG;
  if (p.B > sa::kMaxPlanRows) return SA_ERR_UNSUPPORTED;
  A.parent = parent;
  A.lens = lens;
  return sa::launch_plan_pages(A, as_stream(stream));
}

int sa_compact_pages(const sa_problem* prob, const int32_t* table_in, const int32_t* seq_lens, int32_t* table_out,
                     int32_t* move_src, int32_t* move_dst, int32_t* counts, void* ws, void* stream) {
  Params p;
  sa::PageArgs A;
  const int rc = page_args(prob, table_in, seq_lens, table_out, move_src, move_dst, counts, ws, &p, &A);
  if (rc != SA_OK) return rc;
  return sa::launch_compact_pages(A, as_stream(stream));
}

int sa_copy_pages(const sa_problem* prob, void* k_pool, void* v_pool, const int32_t* src, const int32_t* dst,
                  const int32_t* count, int32_t max_pages, void* ws, void* stream) {
  Params p;
  const int rc = make_params(prob, &p);
  if (rc != SA_OK) return rc;
  if (!k_pool || !v_pool || !src || !dst || !count || !ws) return SA_ERR_INVALID_ARG;
  if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(ws)) return SA_ERR_INVALID_ARG;
  if (max_pages < 0) return SA_ERR_INVALID_ARG;
  if (max_pages == 0) return SA_OK;
  const int nsm = sa_host::num_sms_current();
  if (nsm <= 0) return SA_ERR_CUDA;
  return sa::launch_copy_pages(k_pool, v_pool, src, dst, count, max_pages, p.num_pages, p.Hk, at<int>(ws, 0), nsm,
                               as_stream(stream));
}

}  // extern "C"
