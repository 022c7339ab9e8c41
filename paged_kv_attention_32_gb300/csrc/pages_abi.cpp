// extern "C" entry points of the page pool: argument checks and launches.
#include <algorithm>
#include <climits>
#include <initializer_list>
#include <utility>

#include "host_common.h"
#include "pages.h"

using namespace pka;

namespace {

int64_t table_bytes(int32_t rows, int64_t row_stride, int32_t width) {
  return rows > 0 ? ((rows - 1) * row_stride + width) * 4 : 0;
}

bool aligned4(std::initializer_list<const void*> list) {
  for (const void* p : list)
    if (!aligned(p, 4)) return false;
  return true;
}

// No output shares a byte with an input or with another output.
int check_apart(std::initializer_list<Range> ins, std::initializer_list<Range> outs) {
  for (const Range& o : outs) {
    for (const Range& i : ins) PKA_CHECK_ARG(!overlap(o, i), "an output overlaps an input");
    for (const Range& u : outs) PKA_CHECK_ARG(&u == &o || !overlap(o, u), "two outputs overlap");
  }
  return PKA_OK;
}

Range array(const void* p, int64_t n) { return Range{p, p != nullptr && n > 0 ? (size_t)n * 4 : 0}; }

// What the table operations have in common.
int check_tables(int32_t batch_size, int32_t num_free, const int32_t* free_pages, int32_t page_size,
                 int64_t row_stride, int32_t width) {
  PKA_CHECK_ARG(batch_size >= 1, "batch_size must be >= 1 (got %d)", batch_size);
  if (batch_size > kPageOpRows)
    return fail(PKA_ERR_UNSUPPORTED, "batch_size %d is above %d", batch_size, kPageOpRows);
  PKA_CHECK_ARG(num_free >= 0 && (free_pages != nullptr || num_free == 0),
                "num_free must be >= 0 and free_pages not NULL");
  PKA_CHECK_ARG(page_size >= 1 && page_size <= 65536, "page_size must be in [1, 65536] (got %d)", page_size);
  PKA_CHECK_ARG(width >= 1 && row_stride >= width, "block_tables rows of %d entries, row stride %lld", width,
                (long long)row_stride);
  return PKA_OK;
}

int check_pool_pages(int64_t num_pages) {
  PKA_CHECK_ARG(num_pages >= 1, "num_pages must be >= 1 (got %lld)", (long long)num_pages);
  if (num_pages > kPageOpPages)
    return fail(PKA_ERR_UNSUPPORTED, "num_pages %lld is above %lld", (long long)num_pages, (long long)kPageOpPages);
  return PKA_OK;
}

// Whether at + i * step lies within (-row, row) for an i with |i| < n, not 0 where `other` is set.
bool step_hits(__int128 at, int64_t n, int64_t step, int64_t row, bool other) {
  const auto hits = [&](__int128 i) {
    i = std::max<__int128>(-(__int128)(n - 1), std::min<__int128>(i, n - 1));
    const __int128 d = at + i * step;
    return (i != 0 || !other) && d > -(__int128)row && d < row;
  };
  const __int128 q = step > 0 ? -at / step : 0;   // the sum is nearest to 0 at q or beside it
  return hits(q - 1) || hits(q) || hits(q + 1);
}

// Whether two of n x m rows of `row` elements, at i * outer + j * inner, share an element: at once where one
// stride has room for all of the other's rows, else in a step for each of the smaller count.
bool rows_meet(int64_t n, int64_t outer, int64_t m, int64_t inner, int64_t row) {
  if (n > m) {
    std::swap(n, m);
    std::swap(outer, inner);
  }
  if (n > 1 && m > 1 && inner >= row && outer >= (__int128)(m - 1) * inner + row) return false;
  if (n > 1 && m > 1 && outer >= row && inner >= (__int128)(n - 1) * outer + row) return false;
  for (int64_t i = 0; i < n; ++i)   // two rows that are i apart along the one, anything along the other
    if (step_hits((__int128)i * outer, m, inner, row, i == 0)) return true;
  return false;
}

// n x m rows of `row` units of 16 bits, at p + i * outer + j * inner.
struct Rows {
  const void* p;
  int64_t n, outer, m, inner, row;
};
__int128 apart(const Rows& x, const Rows& y) {
  return ((__int128)reinterpret_cast<uintptr_t>(y.p) - (__int128)reinterpret_cast<uintptr_t>(x.p)) / 2;
}
__int128 last(int64_t n, int64_t stride) { return (__int128)(n - 1) * stride; }   // where the last of n begins

// Whether rows of x and of y share a unit.
bool rows_meet(const Rows& x, const Rows& y) {
  const __int128 d = apart(x, y);
  const __int128 end_x = last(x.n, x.outer) + last(x.m, x.inner) + x.row;
  const __int128 end_y = last(y.n, y.outer) + last(y.m, y.inner) + y.row;
  if (d >= end_x || -d >= end_y) return false;
  // in turn along a stride that both have: y's between x's all along
  const auto between = [&](int64_t stride, __int128 size_x, __int128 size_y) {
    const int64_t at = (int64_t)((d % stride + stride) % stride);
    return at >= size_x && at + size_y <= stride;
  };
  if (x.outer == y.outer && x.outer > 0 && between(x.outer, last(x.m, x.inner) + x.row, last(y.m, y.inner) + y.row))
    return false;
  if (x.inner == y.inner && x.inner > 0 && between(x.inner, last(x.n, x.outer) + x.row, last(y.n, y.outer) + y.row))
    return false;
  if (x.n == y.n && x.outer == y.outer && x.m == y.m && x.inner == y.inner && x.row == y.row) {
    const bool few = x.n < x.m;   // in a step for each of the smaller count, and back
    const int64_t n = few ? x.n : x.m, far = few ? x.outer : x.inner;
    const int64_t m = few ? x.m : x.n, step = few ? x.inner : x.outer;
    for (int64_t i = 1 - n; i < n; ++i)
      if (step_hits(d + (__int128)i * far, m, step, x.row, false)) return true;
    return false;
  }
  // rows that lie in the other's gaps, or meet them: each of x with each of y's smaller count
  const bool few = y.m < y.n;
  const int64_t n = few ? y.m : y.n, far = few ? y.inner : y.outer;
  const int64_t m = few ? y.n : y.m, step = few ? y.outer : y.inner;
  for (int64_t i = 0; i < x.n; ++i)
    for (int64_t j = 0; j < x.m; ++j)
      for (int64_t k = 0; k < n; ++k) {
        // the first of m rows, `step` apart from 0 on, that ends behind where x's begins
        const __int128 at = (__int128)i * x.outer + (__int128)j * x.inner - d - (__int128)k * far;
        const __int128 first = at < y.row || step == 0 ? 0 : (at - y.row) / step + 1;
        if (first < m && first * step + y.row > at && first * step < at + x.row) return true;
      }
  return false;
}

}  // namespace

extern "C" {

int paged_rope_append(const void* q, int64_t q_stride_tok, int64_t q_stride_head, void* q_out,
                      int64_t q_out_stride_tok, int64_t q_out_stride_head, int32_t num_qo_heads,
                      const void* k, const void* v, int64_t kv_stride_tok, int64_t kv_stride_head,
                      int32_t num_kv_heads, int32_t head_dim, const int32_t* positions,
                      int64_t positions_stride, const double* inv_freq, int32_t rotary_dim,
                      int32_t num_axes, const int32_t* sections_host, int32_t pairs,
                      const int64_t* slot_map, int64_t num_tokens, void* k_pages, void* v_pages,
                      int64_t num_pages, int32_t page_size, int64_t stride_page, int64_t stride_head,
                      int32_t dtype, int32_t* status, void* stream) {
  NvtxRange nvtx_range("pka::paged_rope_append");
  clear_error();
  if (dtype != PKA_DTYPE_BF16 && dtype != PKA_DTYPE_F16)
    return fail(PKA_ERR_UNSUPPORTED, "q, k, v and the pools must be bf16 or f16 (dtype %d)", dtype);
  if (head_dim != 128) return fail(PKA_ERR_UNSUPPORTED, "head_dim must be 128 (got %d)", head_dim);
  PKA_CHECK_ARG(num_tokens >= 0 && num_tokens <= INT32_MAX, "num_tokens must be in [0, 2^31 - 1] (got %lld)",
                (long long)num_tokens);
  PKA_CHECK_ARG(num_kv_heads >= 1 && num_kv_heads <= 65536 && num_qo_heads >= 0 && num_qo_heads <= 65536,
                "head counts must be in [1, 65536], without queries 0 (got %d and %d)", num_qo_heads, num_kv_heads);
  PKA_CHECK_ARG((num_qo_heads > 0) == (q != nullptr) && (q != nullptr) == (q_out != nullptr),
                "q and q_out go together, with num_qo_heads > 0");
  PKA_CHECK_ARG(num_tokens == 0 || (k && v && slot_map && k_pages && v_pages),
                "k, v, slot_map and the pools must not be NULL");
  PKA_CHECK_ARG(num_pages >= 1 && num_pages <= INT32_MAX && page_size >= 1 && page_size <= 65536,
                "num_pages must be in [1, 2^31 - 1], page_size in [1, 65536]");
  PKA_CHECK_ARG(rotary_dim >= 0 && rotary_dim <= head_dim && rotary_dim % 16 == 0,
                "rotary_dim must be a multiple of 16 in [0, head_dim] (got %d)", rotary_dim);
  RopeArgs a{};
  if (rotary_dim > 0) {
    PKA_CHECK_ARG((num_tokens == 0 || positions != nullptr) && inv_freq != nullptr && sections_host != nullptr,
                  "a rotation needs positions, inv_freq and sections");
    PKA_CHECK_ARG(pairs == PKA_ROPE_HALVES || pairs == PKA_ROPE_NEIGHBOURS, "unknown pairs %d", pairs);
    PKA_CHECK_ARG(num_axes >= 1 && num_axes <= kRopeAxes, "num_axes must be in [1, %d] (got %d)", kRopeAxes, num_axes);
    int64_t end = 0;
    for (int x = 0; x < kRopeAxes; ++x) {
      if (x < num_axes) {
        PKA_CHECK_ARG(sections_host[x] >= 0, "section %d is negative", x);
        end += sections_host[x];
      }
      a.axis_end[x] = (int32_t)(end < 65536 ? end : 65536);
    }
    PKA_CHECK_ARG(end == rotary_dim / 2, "the sections cover %lld frequencies, rotary_dim has %d", (long long)end,
                  rotary_dim / 2);
    PKA_CHECK_ARG(num_axes == 1 || positions_stride == 0 || positions_stride >= num_tokens,
                  "positions rows of %lld entries, row stride %lld", (long long)num_tokens, (long long)positions_stride);
    PKA_CHECK_ARG(aligned(positions, 4) && aligned(inv_freq, 8), "positions or inv_freq is not aligned");
  }
  for (int64_t s : {q_stride_tok, q_stride_head, q_out_stride_tok, q_out_stride_head, kv_stride_tok, kv_stride_head,
                    stride_page, stride_head})
    PKA_CHECK_ARG(s >= 0 && s % 8 == 0, "strides must be non-negative multiples of 8 elements");
  PKA_CHECK_ARG(aligned(q, 16) && aligned(q_out, 16) && aligned(k, 16) && aligned(v, 16) && aligned(k_pages, 16) &&
                    aligned(v_pages, 16) && aligned(slot_map, 8) && aligned(status, 4),
                "q, k, v and the pools must be 16-byte aligned, slot_map 8-byte aligned");
  if (num_tokens == 0) return PKA_OK;
  // what is written: no element of it twice
  PKA_CHECK_ARG(!rows_meet(num_pages, stride_page, num_kv_heads, stride_head, (int64_t)page_size * head_dim),
                "pages of %d rows overlap: stride_page %lld, stride_head %lld", page_size, (long long)stride_page,
                (long long)stride_head);
  const auto pool = [&](const void* p) {
    return Rows{p, num_pages, stride_page, num_kv_heads, stride_head, (int64_t)page_size * head_dim};
  };
  const auto rows = [&](const void* p, int64_t tok, int64_t head, int32_t heads) {
    return Rows{p, num_tokens, tok, heads, head, head_dim};
  };
  const Rows k_pool = pool(k_pages), v_pool = pool(v_pages);
  const Rows out = rows(q_out, q_out_stride_tok, q_out_stride_head, num_qo_heads);
  PKA_CHECK_ARG(!rows_meet(k_pool, v_pool), "k_pages and v_pages overlap");
  const Rows ins[] = {rows(q, q_stride_tok, q_stride_head, num_qo_heads),
                      rows(k, kv_stride_tok, kv_stride_head, num_kv_heads),
                      rows(v, kv_stride_tok, kv_stride_head, num_kv_heads),
                      {slot_map, 1, 0, 1, 0, 4 * num_tokens},
                      {rotary_dim > 0 ? positions : nullptr, num_axes, num_axes > 1 ? 2 * positions_stride : 0, 1, 0,
                       2 * num_tokens},
                      {rotary_dim > 0 ? inv_freq : nullptr, 1, 0, 1, 0, 2 * (int64_t)rotary_dim},
                      {status, 1, 0, 1, 0, 2}};
  for (const Rows& in : ins)
    PKA_CHECK_ARG(in.p == nullptr || (!rows_meet(in, k_pool) && !rows_meet(in, v_pool)), "an input lies in a pool");
  if (q != nullptr) {
    PKA_CHECK_ARG(!rows_meet(num_tokens, q_out_stride_tok, num_qo_heads, q_out_stride_head, head_dim),
                  "rows of q_out overlap");
    PKA_CHECK_ARG(!rows_meet(out, k_pool) && !rows_meet(out, v_pool), "q_out lies in a pool");
    // q itself it may be, all of it
    const bool in_place = q_out == q && q_out_stride_tok == q_stride_tok && q_out_stride_head == q_stride_head;
    for (const Rows& in : ins)
      PKA_CHECK_ARG(in.p == nullptr || (in_place && &in == ins) || !rows_meet(in, out),
                    "q_out overlaps an input without being q");
  }
  a.q = q;
  a.q_stride_tok = q_stride_tok;
  a.q_stride_head = q_stride_head;
  a.q_out = q_out;
  a.qo_stride_tok = q_out_stride_tok;
  a.qo_stride_head = q_out_stride_head;
  a.k = k;
  a.v = v;
  a.kv_stride_tok = kv_stride_tok;
  a.kv_stride_head = kv_stride_head;
  a.positions = positions;
  a.pos_stride = positions_stride;
  a.inv_freq = inv_freq;
  a.slot_map = slot_map;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.stride_page = stride_page;
  a.stride_head = stride_head;
  a.num_slots = num_pages * page_size;
  a.status = status;
  a.num_tokens = (int32_t)num_tokens;
  a.num_qo_heads = num_qo_heads;
  a.num_kv_heads = num_kv_heads;
  a.page_size = page_size;
  a.rotary = rotary_dim;
  return launch_rope_append(a, dtype == PKA_DTYPE_F16, pairs == PKA_ROPE_HALVES, static_cast<cudaStream_t>(stream));
}

int paged_kv_fork(const int32_t* parents, const int32_t* children, int32_t num_forks, const int32_t* kv_lens,
                  int32_t batch_size, const int32_t* free_pages, int32_t num_free, const int32_t* free_head,
                  int32_t page_size, int32_t* block_tables, int64_t bt_row_stride, int32_t max_pages_per_seq,
                  int32_t* seq_lens, int32_t* src_pages, int32_t* dst_pages, int32_t* free_head_out, int32_t* status,
                  void* stream) {
  NvtxRange nvtx_range("pka::paged_kv_fork");
  clear_error();
  PKA_CHECK_ARG(kv_lens && free_head && block_tables && seq_lens && free_head_out,
                "only free_pages (with num_free 0), the fork arrays (with num_forks 0) and status may be NULL");
  int rc = check_tables(batch_size, num_free, free_pages, page_size, bt_row_stride, max_pages_per_seq);
  if (rc != PKA_OK) return rc;
  PKA_CHECK_ARG(num_forks >= 0 && num_forks <= batch_size, "num_forks must be in [0, batch_size] (got %d)", num_forks);
  PKA_CHECK_ARG(num_forks == 0 || (parents && children && src_pages && dst_pages), "a fork array is NULL");
  PKA_CHECK_ARG(aligned4({parents, children, kv_lens, free_pages, free_head, block_tables, seq_lens, src_pages,
                          dst_pages, free_head_out, status}),
                "int32 arrays must be 4-byte aligned");
  const Range tables{block_tables, (size_t)table_bytes(batch_size, bt_row_stride, max_pages_per_seq)};
  rc = check_apart({array(parents, num_forks), array(children, num_forks), array(kv_lens, batch_size),
                    array(free_pages, num_free), array(free_head, 1)},
                   {tables, array(seq_lens, batch_size), array(src_pages, num_forks), array(dst_pages, num_forks),
                    array(free_head_out, 1), array(status, 1)});
  if (rc != PKA_OK) return rc;
  return launch_kv_fork(ForkArgs{parents, children, num_forks, kv_lens, batch_size, free_pages, num_free, free_head,
                                 page_size, block_tables, bt_row_stride, max_pages_per_seq, seq_lens, src_pages,
                                 dst_pages, free_head_out, status},
                        static_cast<cudaStream_t>(stream));
}

int paged_kv_free(const int32_t* rows, int32_t num_rows, const int32_t* kv_lens, int32_t batch_size,
                  int32_t* free_pages, int32_t num_free, const int32_t* free_head, int32_t page_size,
                  const int32_t* block_tables, int64_t bt_row_stride, int32_t max_pages_per_seq, int64_t num_pages,
                  int32_t* seq_lens, int32_t* free_head_out, int32_t* status, void* stream) {
  NvtxRange nvtx_range("pka::paged_kv_free");
  clear_error();
  PKA_CHECK_ARG(kv_lens && free_head && block_tables && seq_lens && free_head_out,
                "only free_pages (with num_free 0), rows (with num_rows 0) and status may be NULL");
  int rc = check_tables(batch_size, num_free, free_pages, page_size, bt_row_stride, max_pages_per_seq);
  if (rc == PKA_OK) rc = check_pool_pages(num_pages);
  if (rc != PKA_OK) return rc;
  PKA_CHECK_ARG(num_rows >= 0 && num_rows <= batch_size && (rows != nullptr || num_rows == 0),
                "num_rows must be in [0, batch_size] (got %d) and rows not NULL", num_rows);
  PKA_CHECK_ARG(aligned4({rows, kv_lens, free_pages, free_head, block_tables, seq_lens, free_head_out, status}),
                "int32 arrays must be 4-byte aligned");
  const Range tables{block_tables, (size_t)table_bytes(batch_size, bt_row_stride, max_pages_per_seq)};
  rc = check_apart({array(rows, num_rows), array(kv_lens, batch_size), array(free_head, 1), tables},
                   {array(free_pages, num_free), array(seq_lens, batch_size), array(free_head_out, 1),
                    array(status, 1)});
  if (rc != PKA_OK) return rc;
  return launch_kv_free(ReleaseArgs{rows, num_rows, kv_lens, batch_size, free_pages, num_free, free_head, page_size,
                                    block_tables, bt_row_stride, max_pages_per_seq, (int32_t)num_pages, seq_lens,
                                    free_head_out, status},
                        static_cast<cudaStream_t>(stream));
}

int paged_kv_compact(const int32_t* kv_lens, int32_t batch_size, const int32_t* free_pages, int32_t num_free,
                     const int32_t* free_head, int32_t page_size, const int32_t* block_tables, int64_t bt_row_stride,
                     int32_t max_pages_per_seq, int64_t num_pages, int32_t* block_tables_out,
                     int64_t bt_out_row_stride, int32_t* free_pages_out, int32_t* src_pages, int32_t* dst_pages,
                     int32_t max_moves, int32_t* num_moves, int32_t* status, void* stream) {
  NvtxRange nvtx_range("pka::paged_kv_compact");
  clear_error();
  PKA_CHECK_ARG(kv_lens && free_head && block_tables && block_tables_out && num_moves,
                "only the free list (with num_free 0), the moves (with max_moves 0) and status may be NULL");
  int rc = check_tables(batch_size, num_free, free_pages, page_size, bt_row_stride, max_pages_per_seq);
  if (rc == PKA_OK) rc = check_pool_pages(num_pages);
  if (rc != PKA_OK) return rc;
  PKA_CHECK_ARG(bt_out_row_stride >= max_pages_per_seq, "block_tables_out rows of %d entries, row stride %lld",
                max_pages_per_seq, (long long)bt_out_row_stride);
  PKA_CHECK_ARG(num_free == 0 || free_pages_out != nullptr, "free_pages_out must not be NULL");
  PKA_CHECK_ARG(max_moves >= 0 && (max_moves == 0 || (src_pages && dst_pages)),
                "max_moves must be >= 0 and its arrays not NULL");
  PKA_CHECK_ARG(aligned4({kv_lens, free_pages, free_head, block_tables, block_tables_out, free_pages_out, src_pages,
                          dst_pages, num_moves, status}),
                "int32 arrays must be 4-byte aligned");
  const Range tables{block_tables, (size_t)table_bytes(batch_size, bt_row_stride, max_pages_per_seq)};
  const Range tables_out{block_tables_out, (size_t)table_bytes(batch_size, bt_out_row_stride, max_pages_per_seq)};
  const Range none{nullptr, 0};
  // the tables and the list may be written over themselves
  const bool same_tables = block_tables_out == block_tables && bt_out_row_stride == bt_row_stride;
  const bool same_list = free_pages_out == free_pages;
  rc = check_apart({array(kv_lens, batch_size), same_list ? none : array(free_pages, num_free), array(free_head, 1),
                    same_tables ? none : tables},
                   {tables_out, array(free_pages_out, num_free), array(src_pages, max_moves),
                    array(dst_pages, max_moves), array(num_moves, 1), array(status, 1)});
  if (rc != PKA_OK) return rc;
  return launch_kv_compact(CompactArgs{kv_lens, batch_size, free_pages, num_free, free_head, page_size, block_tables,
                                       bt_row_stride, max_pages_per_seq, (int32_t)num_pages, block_tables_out,
                                       bt_out_row_stride, free_pages_out, src_pages, dst_pages, max_moves, num_moves,
                                       status},
                           static_cast<cudaStream_t>(stream));
}

int paged_kv_copy(void* const* pools, const int64_t* page_strides, const int64_t* page_bytes, int32_t num_pools,
                  int64_t num_pages, const int32_t* src_pages, const int32_t* dst_pages, int32_t num_entries,
                  const int32_t* count, int32_t* status, void* stream) {
  NvtxRange nvtx_range("pka::paged_kv_copy");
  clear_error();
  PKA_CHECK_ARG(num_pools >= 0 && (num_pools == 0 || (pools && page_strides && page_bytes)),
                "num_pools must be >= 0 and the pool arrays not NULL");
  PKA_CHECK_ARG(num_pages >= 1 && num_pages <= INT32_MAX, "num_pages must be in [1, 2^31 - 1] (got %lld)",
                (long long)num_pages);
  PKA_CHECK_ARG(num_entries >= 0 && (num_entries == 0 || (src_pages && dst_pages)),
                "num_entries must be >= 0 and its arrays not NULL");
  PKA_CHECK_ARG(aligned4({src_pages, dst_pages, count, status}), "int32 arrays must be 4-byte aligned");
  for (int32_t i = 0; i < num_pools; ++i) {
    PKA_CHECK_ARG(pools[i] != nullptr && aligned(pools[i], 16), "pool %d is NULL or not 16-byte aligned", i);
    PKA_CHECK_ARG(page_bytes[i] >= 0 && page_bytes[i] % 16 == 0 && page_strides[i] % 16 == 0 &&
                      page_strides[i] >= page_bytes[i],
                  "pool %d: pages of %lld bytes every %lld; both must be multiples of 16", i, (long long)page_bytes[i],
                  (long long)page_strides[i]);
    PKA_CHECK_ARG(page_strides[i] <= INT64_MAX / num_pages, "pool %d is too large", i);
  }
  if (num_entries == 0) return PKA_OK;
  for (int32_t first = 0; first < num_pools; first += kPoolsPerLaunch) {
    CopyArgs a{};
    a.num_pools = num_pools - first < kPoolsPerLaunch ? num_pools - first : kPoolsPerLaunch;
    for (int32_t i = 0; i < a.num_pools; ++i)
      a.pools[i] = PagePool{static_cast<uint8_t*>(pools[first + i]), page_strides[first + i], page_bytes[first + i]};
    a.src_pages = src_pages;
    a.dst_pages = dst_pages;
    a.count = count;
    a.num_entries = num_entries;
    a.num_pages = (int32_t)num_pages;
    a.status = status;
    const int rc = launch_kv_copy(a, static_cast<cudaStream_t>(stream));
    if (rc != PKA_OK) return rc;
  }
  return PKA_OK;
}

}  // extern "C"
