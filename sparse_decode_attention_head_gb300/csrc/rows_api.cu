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

// q [n_rows][Hq][D] as boxes of 64 dims x G heads x 128 / G tokens.
int make_q_map(CUtensorMap* m, const void* q, int n_rows, const Params& p, int tpt) {
  auto fn = sa_host::encode_fn();
  if (fn == nullptr) return SA_ERR_CUDA;
  cuuint64_t dims[3] = {SA_HEAD_DIM, (cuuint64_t)p.Hq, (cuuint64_t)n_rows};
  cuuint64_t strides[2] = {SA_HEAD_DIM * 2, (cuuint64_t)p.Hq * SA_HEAD_DIM * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)tpt};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
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

int rows_attention(const sa_problem* prob, int32_t n_rows, const void* q, const void* k_pool, const void* v_pool,
                   const int32_t* page_table, const int32_t* seq_lens, const int32_t* row_offsets, const uint64_t* tree,
                   void* out, float* lse, void* ws, void* stream) {
  Params p;
  int rc = make_params(prob, &p);
  if (rc != SA_OK) return rc;
  if (n_rows < 0) return SA_ERR_INVALID_ARG;
  if (!k_pool || !v_pool || !page_table || !seq_lens || !row_offsets || !ws) return SA_ERR_INVALID_ARG;
  if (n_rows == 0) return SA_OK;
  if (!q || !out) return SA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out) || !aligned16(ws))
    return SA_ERR_INVALID_ARG;
  const size_t row_bytes = (size_t)n_rows * p.Hq * SA_HEAD_DIM * 2;
  if (overlap(q, row_bytes, out, row_bytes)) return SA_ERR_INVALID_ARG;
  const int nsm = sa_host::num_sms_current();
  if (nsm <= 0) return SA_ERR_CUDA;
  sa::RowsAttnArgs A{};
  A.tpt = 128 / p.G;
  CUtensorMap tmQ, tmK, tmV;
  if ((rc = make_q_map(&tmQ, q, n_rows, p, A.tpt)) != SA_OK) return rc;
  if ((rc = make_tile_map(&tmK, k_pool, p)) != SA_OK) return rc;
  if ((rc = make_tile_map(&tmV, v_pool, p)) != SA_OK) return rc;
  const AttnLayout l = attn_layout();
  A.v_pool = static_cast<const __nv_bfloat16*>(v_pool);
  A.page_table = page_table;
  A.seq_lens = seq_lens;
  A.row_offsets = row_offsets;
  A.tree = reinterpret_cast<const unsigned long long*>(tree);
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
  return sa::launch_rows_attention(A, tmQ, tmK, tmV, nsm, as_stream(stream));
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
