// extern "C" entry points of page tables and latent attention: argument
// checks, plan ownership, launch dispatch.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <exception>
#include <new>
#include <utility>

#include "host_common.h"
#include "latent.h"
#include "tmap.h"

using namespace pka;

namespace {

// Runs `f`, turning a C++ exception (a host allocation that failed) into an error code.
template <typename F>
int guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    return fail(PKA_ERR_INVALID_ARG, "host error: %s", e.what());
  }
}

// Whether two byte ranges share a byte.
bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return n > 0 && m > 0 && a < b + m && b < a + n;
}

// Makes `next`, whose host arrays are built, the plan *p on the device: in p's buffers, or
// in larger ones.  Where anything fails p stays the plan that it was.
// One asynchronous copy of the arrays from a pinned image, which is rewritten only after
// the copy that last read it has completed.
int install_latent_plan(pka_latent_plan& p, pka_latent_plan&& next, cudaStream_t stream) {
  const size_t n_pieces = next.items.size() * sizeof(LatentPiece);
  const size_t n_more = next.segments.size() * sizeof(int32_t);
  const size_t n_splits = next.splits.size() * sizeof(LatentReq);
  const size_t off_more = up256(n_pieces), off_splits = off_more + up256(n_more);
  const size_t off_status = off_splits + up256(n_splits);
  const size_t total = off_status + 256;
  if (p.stage_done == nullptr)
    PKA_CUDA_TRY(cudaEventCreateWithFlags(&p.stage_done, cudaEventDisableTiming),
                 "cudaEventCreate(plan upload)");
  else
    PKA_CUDA_TRY(cudaEventSynchronize(p.stage_done), "cudaEventSynchronize(plan upload)");
  next.dev_buf = p.dev_buf;
  next.host_stage = p.host_stage;
  next.capacity = p.capacity;
  next.device = p.device;
  next.stage_done = p.stage_done;
  const bool grow = total > p.capacity;
  if (grow) {
    next.capacity = std::max<size_t>(4096, total + total / 2);
    PKA_CUDA_TRY(cudaGetDevice(&next.device), "cudaGetDevice");
    PKA_CUDA_TRY(cudaMalloc(&next.dev_buf, next.capacity), "cudaMalloc(latent plan)");
    const cudaError_t e = cudaMallocHost(&next.host_stage, next.capacity);
    if (e != cudaSuccess) {
      cudaFree(next.dev_buf);
      return cuda_fail(e, "cudaMallocHost(plan image)");
    }
  }
  uint8_t* base = static_cast<uint8_t*>(next.dev_buf);
  next.d_pieces = reinterpret_cast<const LatentPiece*>(base);
  next.d_more = reinterpret_cast<const int32_t*>(base + off_more);
  next.d_splits = reinterpret_cast<const LatentReq*>(base + off_splits);
  next.d_status = reinterpret_cast<int32_t*>(base + off_status);
  uint8_t* img = static_cast<uint8_t*>(next.host_stage);
  LatentPiece* pieces = reinterpret_cast<LatentPiece*>(img);
  int32_t* more = reinterpret_cast<int32_t*>(img + off_more);
  auto piece = [&](int32_t i) {
    const LatentItem& it = next.items[(size_t)i];
    const LatentReq& r = next.reqs[(size_t)it.request];
    return LatentPiece{it.request, it.tile_lo, it.tile_hi, it.part, r.q_start, r.q_len, r.kv_len, r.part_base};
  };
  const int32_t segs = (int32_t)next.segments.size() - 1;
  int32_t at = segs;
  for (int32_t s = 0; s < segs; ++s) {   // no segment is empty
    const size_t first = (size_t)next.segments[(size_t)s];
    more[s] = at;
    pieces[s] = piece((int32_t)first);
    for (int32_t i = (int32_t)first + 1; i < next.segments[(size_t)s + 1]; ++i) pieces[at++] = piece(i);
  }
  more[segs] = at;
  if (n_splits) std::memcpy(img + off_splits, next.splits.data(), n_splits);
  std::memset(img + off_status, 0, 256);
  cudaError_t e = cudaMemcpyAsync(base, img, total, cudaMemcpyHostToDevice, stream);
  if (e != cudaSuccess) {
    if (grow) {
      cudaFree(next.dev_buf);
      cudaFreeHost(next.host_stage);
    }
    return cuda_fail(e, "cudaMemcpyAsync(latent plan)");
  }
  // from here on the device has the new plan; a copy that no event follows is waited for
  e = cudaEventRecord(next.stage_done, stream);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    e = cudaStreamSynchronize(stream);
  }
  if (grow) {
    cudaFree(p.dev_buf);
    cudaFreeHost(p.host_stage);
  }
  p = std::move(next);
  return e == cudaSuccess ? PKA_OK : cuda_fail(e, "cudaEventRecord(plan upload)");
}

// Builds a plan and makes it *p; p stays the plan that it was where that fails.
int make_latent_plan(pka_latent_plan& p, const pka_latent_desc& desc, const int32_t* seq_lens_kv,
                     const int32_t* qo_indptr, cudaStream_t stream) {
  pka_latent_plan next;
  const int rc = build_latent_plan(next, desc, seq_lens_kv, qo_indptr);
  if (rc != PKA_OK) return rc;
  if (!(desc.flags & PKA_PLAN_HOST_ONLY)) return install_latent_plan(p, std::move(next), stream);
  p = std::move(next);
  return PKA_OK;
}

}  // namespace

// Partial outputs and LSEs of a latent prefill's pieces, 256 rows each.
static size_t prefill_workspace(const pka_prefill_plan& p) { return (size_t)p.num_parts * 256 * 129 * sizeof(float); }

extern "C" {

// ---------------------------------------------------------------------------
// page tables
// ---------------------------------------------------------------------------

int paged_kv_tables(const int32_t* kv_lens, const int32_t* new_lens, int32_t batch_size,
                    const int32_t* free_pages, int32_t num_free, const int32_t* free_head,
                    int32_t page_size, int32_t* block_tables, int64_t bt_row_stride,
                    int32_t max_pages_per_seq, int32_t* seq_lens, int32_t* qo_indptr,
                    int64_t* slot_map, int64_t num_slots, int32_t* free_head_out, int32_t* status,
                    void* stream) {
  NvtxRange nvtx_range("pka::paged_kv_tables");
  clear_error();
  PKA_CHECK_ARG(kv_lens && new_lens && free_head && block_tables && seq_lens && qo_indptr &&
                    slot_map && free_head_out,
                "only free_pages (with num_free 0) and status may be NULL");
  PKA_CHECK_ARG(batch_size >= 1, "batch_size must be >= 1 (got %d)", batch_size);
  PKA_CHECK_ARG(num_free >= 0 && (free_pages != nullptr || num_free == 0),
                "num_free must be >= 0 and free_pages not NULL");
  PKA_CHECK_ARG(page_size >= 1 && page_size <= 65536, "page_size must be in [1, 65536] (got %d)",
                page_size);
  PKA_CHECK_ARG(max_pages_per_seq >= 1 && bt_row_stride >= max_pages_per_seq,
                "block_tables rows of %d entries, row stride %lld", max_pages_per_seq,
                (long long)bt_row_stride);
  PKA_CHECK_ARG(num_slots >= 1, "num_slots must be >= 1 (got %lld)", (long long)num_slots);
  for (const void* p : {(const void*)kv_lens, (const void*)new_lens, (const void*)free_pages,
                        (const void*)free_head, (const void*)block_tables, (const void*)seq_lens,
                        (const void*)qo_indptr, (const void*)free_head_out, (const void*)status})
    PKA_CHECK_ARG(aligned(p, 4), "int32 arrays must be 4-byte aligned");
  PKA_CHECK_ARG(aligned(slot_map, 8), "slot_map must be 8-byte aligned");
  struct Range {
    const void* p;
    size_t n;
  };
  const size_t B = (size_t)batch_size;
  const Range ins[] = {{kv_lens, B * 4}, {new_lens, B * 4}, {free_pages, (size_t)num_free * 4},
                       {free_head, 4}};
  const Range outs[] = {{block_tables, ((B - 1) * (size_t)bt_row_stride + max_pages_per_seq) * 4},
                        {seq_lens, B * 4}, {qo_indptr, (B + 1) * 4},
                        {slot_map, (size_t)num_slots * 8}, {free_head_out, 4},
                        {status, status != nullptr ? size_t(4) : 0}};
  for (const Range& o : outs) {
    for (const Range& i : ins)
      PKA_CHECK_ARG(!overlap(o.p, o.n, i.p, i.n), "an output overlaps an input");
    for (const Range& u : outs)
      PKA_CHECK_ARG(&u == &o || !overlap(o.p, o.n, u.p, u.n), "two outputs overlap");
  }
  return launch_kv_tables(kv_lens, new_lens, batch_size, free_pages, num_free, free_head,
                          page_size, block_tables, bt_row_stride, max_pages_per_seq, seq_lens,
                          qo_indptr, slot_map, num_slots, free_head_out, status,
                          static_cast<cudaStream_t>(stream));
}

// ---------------------------------------------------------------------------
// latent cache
// ---------------------------------------------------------------------------

int paged_latent_append(const void* latent, int64_t latent_stride, const void* rope,
                        int64_t rope_stride, int32_t latent_dim, int32_t rope_dim,
                        const int64_t* slot_map, int64_t num_tokens, void* pages,
                        int64_t num_pages, int32_t page_size, int64_t stride_page, int32_t dtype,
                        int32_t* status, void* stream) {
  NvtxRange nvtx_range("pka::paged_latent_append");
  clear_error();
  PKA_CHECK_ARG(latent && slot_map && pages, "latent, slot_map and pages must not be NULL");
  if (dtype != PKA_DTYPE_BF16 && dtype != PKA_DTYPE_F16)
    return fail(PKA_ERR_UNSUPPORTED, "the pool must be bf16 or f16 (dtype %d)", dtype);
  PKA_CHECK_ARG(latent_dim >= 8 && latent_dim % 8 == 0 && latent_dim <= 65536,
                "latent_dim must be a multiple of 8 in [8, 65536] (got %d)", latent_dim);
  PKA_CHECK_ARG(rope_dim >= 0 && rope_dim % 8 == 0 && rope_dim <= 65536 &&
                    (rope_dim == 0) == (rope == nullptr),
                "rope_dim must be a multiple of 8 in [0, 65536], rope NULL only with 0 (got %d)",
                rope_dim);
  PKA_CHECK_ARG(num_tokens >= 0 && num_pages >= 1 && page_size >= 1,
                "num_tokens must be >= 0, num_pages and page_size >= 1");
  PKA_CHECK_ARG(num_pages <= INT64_MAX / page_size / 65536, "the pool is too large");
  PKA_CHECK_ARG(latent_stride >= 0 && rope_stride >= 0 && latent_stride % 8 == 0 &&
                    rope_stride % 8 == 0 && stride_page % 8 == 0,
                "strides must be non-negative multiples of 8 elements");
  PKA_CHECK_ARG(stride_page >= (int64_t)page_size * (latent_dim + rope_dim),
                "stride_page (%lld) is smaller than a page", (long long)stride_page);
  PKA_CHECK_ARG(aligned(latent, 16) && aligned(rope, 16) && aligned(pages, 16) &&
                    aligned(slot_map, 8) && aligned(status, 4),
                "latent, rope and pages must be 16-byte aligned, slot_map 8-byte aligned");
  PKA_CHECK_ARG(num_tokens <= (INT64_MAX / 2) / ((latent_dim + rope_dim) / 8), "too many tokens");
  return launch_latent_append(latent, latent_stride, rope, rope_stride, latent_dim, rope_dim,
                              slot_map, num_tokens, pages, num_pages, page_size, stride_page,
                              status, static_cast<cudaStream_t>(stream));
}

// ---------------------------------------------------------------------------
// latent decode
// ---------------------------------------------------------------------------

int paged_latent_decode_plan(pka_latent_plan** plan_out, const pka_latent_desc* desc,
                             const int32_t* seq_lens_kv_host, const int32_t* qo_indptr_host,
                             size_t* workspace_bytes_out, void* stream) {
  NvtxRange nvtx_range("pka::paged_latent_decode_plan");
  clear_error();
  PKA_CHECK_ARG(plan_out != nullptr && desc != nullptr, "plan_out and desc must not be NULL");
  *plan_out = nullptr;
  pka_latent_plan* p = new (std::nothrow) pka_latent_plan();
  if (p == nullptr) return fail(PKA_ERR_INVALID_ARG, "out of host memory");
  const int rc = guarded([&] {
    return make_latent_plan(*p, *desc, seq_lens_kv_host, qo_indptr_host, static_cast<cudaStream_t>(stream));
  });
  if (rc != PKA_OK) {
    paged_latent_decode_plan_destroy(p);
    return rc;
  }
  if (workspace_bytes_out) *workspace_bytes_out = (size_t)p->workspace_bytes;
  *plan_out = p;
  return PKA_OK;
}

int paged_latent_decode_plan_update(pka_latent_plan* p, int32_t batch_size,
                                    const int32_t* seq_lens_kv_host,
                                    const int32_t* qo_indptr_host, size_t* workspace_bytes_out,
                                    void* stream) {
  NvtxRange nvtx_range("pka::paged_latent_decode_plan_update");
  clear_error();
  PKA_CHECK_ARG(p != nullptr, "plan must not be NULL");
  const bool host_only = p->desc.flags & PKA_PLAN_HOST_ONLY;
  if (!host_only) {
    const int rc = check_device(p->device);
    if (rc != PKA_OK) return rc;
  }
  const int rc = guarded([&] {
    pka_latent_desc d = p->desc;
    d.batch_size = batch_size;
    return make_latent_plan(*p, d, seq_lens_kv_host, qo_indptr_host, static_cast<cudaStream_t>(stream));
  });
  if (rc != PKA_OK) return rc;
  if (workspace_bytes_out) *workspace_bytes_out = (size_t)p->workspace_bytes;
  return PKA_OK;
}

void paged_latent_decode_plan_destroy(pka_latent_plan* plan) {
  if (plan == nullptr) return;
  if (plan->stage_done != nullptr) {
    cudaEventSynchronize(plan->stage_done);   // the image is not freed under a pending copy
    cudaEventDestroy(plan->stage_done);
  }
  if (plan->host_stage != nullptr) cudaFreeHost(plan->host_stage);
  if (plan->dev_buf != nullptr) cudaFree(plan->dev_buf);
  delete plan;
}

int paged_latent_decode_plan_info(const pka_latent_plan* p, pka_latent_plan_info* info) {
  clear_error();
  PKA_CHECK_ARG(p != nullptr && info != nullptr, "plan and info must not be NULL");
  info->num_segments = (int32_t)p->segments.size() - 1;
  info->num_items = (int32_t)p->items.size();
  info->num_split = (int32_t)p->splits.size();
  info->row_tile = p->row_tile;
  info->row_blocks = p->row_blocks;
  info->partial_rows = p->partial_rows;
  info->workspace_bytes = p->workspace_bytes;
  info->total_q = p->total_q;
  info->num_sms = p->desc.num_sms;
  return PKA_OK;
}

int paged_latent_decode_plan_export(const pka_latent_plan* p, int32_t* items, int32_t* segments) {
  clear_error();
  PKA_CHECK_ARG(p != nullptr, "plan must not be NULL");
  if (items != nullptr && !p->items.empty())
    std::memcpy(items, p->items.data(), p->items.size() * sizeof(LatentItem));
  if (segments != nullptr)
    std::memcpy(segments, p->segments.data(), p->segments.size() * sizeof(int32_t));
  return PKA_OK;
}

int paged_latent_decode_plan_check(const pka_latent_plan* p, void* stream) {
  clear_error();
  PKA_CHECK_ARG(p != nullptr && p->d_status != nullptr, "plan has no device state");
  return read_status(p->d_status, static_cast<cudaStream_t>(stream));
}

int paged_latent_decode_run(const pka_latent_plan* p, const void* q, int64_t q_stride_tok,
                            int64_t q_stride_head, const void* pages, int64_t stride_page,
                            const int32_t* block_tables, int64_t bt_row_stride,
                            const int32_t* seq_lens_kv_dev, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("pka::paged_latent_decode_run");
  clear_error();
  PKA_CHECK_ARG(p != nullptr, "plan must not be NULL");
  PKA_CHECK_ARG(p->dev_buf != nullptr, "plan was built with PKA_PLAN_HOST_ONLY and cannot run");
  if (p->items.empty()) return PKA_OK;   // no query rows: q and out may be empty, of address NULL
  const pka_latent_desc& d = p->desc;
  PKA_CHECK_ARG(q && pages && block_tables && out,
                "q, pages, block_tables and out must not be NULL");
  PKA_CHECK_ARG(d.freeze_seq_lens || seq_lens_kv_dev != nullptr,
                "seq_lens_kv_dev is required when the plan does not freeze the lengths");
  PKA_CHECK_ARG(!d.return_lse || lse != nullptr, "the plan returns the LSE: lse is NULL");
  PKA_CHECK_ARG(aligned(q, 16) && q_stride_tok % 8 == 0 && q_stride_head % 8 == 0 &&
                    q_stride_tok >= 0 && q_stride_head >= 0,
                "q must be 16-byte aligned with non-negative strides that are multiples of 8");
  PKA_CHECK_ARG(aligned(pages, 16) && stride_page % 8 == 0, "pages must be 16-byte aligned with "
                "a stride_page that is a multiple of 8");
  PKA_CHECK_ARG(stride_page >= (int64_t)d.page_size * (d.latent_dim + d.rope_dim),
                "stride_page (%lld) is smaller than a page", (long long)stride_page);
  PKA_CHECK_ARG(aligned(out, 16) && aligned(lse, 4) && aligned(block_tables, 4) &&
                    aligned(seq_lens_kv_dev, 4),
                "out must be 16-byte aligned, lse, block_tables and lengths 4-byte aligned");
  PKA_CHECK_ARG(bt_row_stride >= d.max_pages_per_seq,
                "bt_row_stride (%lld) is smaller than the table width %d",
                (long long)bt_row_stride, d.max_pages_per_seq);
  if (p->workspace_bytes > 0) {
    if (workspace == nullptr || workspace_bytes < (size_t)p->workspace_bytes)
      return fail(PKA_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, the plan needs %lld",
                  workspace_bytes, (long long)p->workspace_bytes);
    PKA_CHECK_ARG(aligned(workspace, 256), "workspace must be 256-byte aligned");
  }
  const int rc = check_device(p->device);
  if (rc != PKA_OK) return rc;
  LatentArgs a{};
  a.q = q;
  a.q_stride_tok = q_stride_tok;
  a.q_stride_head = q_stride_head;
  a.block_tables = block_tables;
  a.bt_row_stride = bt_row_stride;
  a.seq_lens_live = d.freeze_seq_lens ? nullptr : seq_lens_kv_dev;
  a.out = out;
  a.lse = d.return_lse ? lse : nullptr;
  a.ws_o = static_cast<float*>(workspace);
  a.ws_lse = workspace ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                                  p->ws_lse_offset)
                       : nullptr;
  a.pieces = p->d_pieces;
  a.more = p->d_more;
  a.splits = p->d_splits;
  a.status = p->d_status;
  a.num_segments = (int32_t)p->segments.size() - 1;
  a.num_splits = (int32_t)p->splits.size();
  a.num_many = p->num_many;
  a.row_blocks = p->row_blocks;
  a.max_rows = p->max_rows;
  a.num_heads = d.num_heads;
  a.page_size = d.page_size;
  a.box_rows = 8;
  while (a.box_rows < kLatentTile && d.page_size % (2 * a.box_rows) == 0) a.box_rows *= 2;
  a.num_pages = (int32_t)d.num_pages;
  a.causal = d.mask == PKA_MASK_CAUSAL;
  a.scale_log2 = d.scale * 1.4426950408889634f;
  a.output_scale = d.output_scale;
  a.out_dtype = d.out_dtype;
  return launch_latent_decode(*p, a, pages, stride_page, static_cast<cudaStream_t>(stream));
}

// ---------------------------------------------------------------------------
// latent prefill
// ---------------------------------------------------------------------------

int batch_latent_prefill_plan(pka_prefill_plan** plan_out, const pka_latent_prefill_desc* desc,
                              const int32_t* qo_indptr_host, const int32_t* kv_indptr_host,
                              size_t* workspace_bytes_out, int32_t* num_tiles_out, void* stream) {
  clear_error();
  PKA_CHECK_ARG(plan_out != nullptr && desc != nullptr, "plan_out and desc must not be NULL");
  *plan_out = nullptr;
  if (desc->nope_dim != 128 || desc->rope_dim != kLatentRopeDim || desc->value_dim != 128)
    return fail(PKA_ERR_UNSUPPORTED, "latent prefill takes heads of 128 + %d key and 128 value "
                "dimensions (got %d + %d, %d)", kLatentRopeDim, desc->nope_dim, desc->rope_dim,
                desc->value_dim);
  PKA_CHECK_ARG(desc->mask == PKA_MASK_DENSE || desc->mask == PKA_MASK_CAUSAL, "unknown mask %d",
                desc->mask);
  pka_prefill_desc d{};
  d.batch_size = desc->batch_size;
  d.num_qo_heads = desc->num_heads;
  d.num_kv_heads = desc->num_heads;
  d.head_dim = 128;
  d.dtype = desc->dtype;
  d.mask = desc->mask;
  d.window_left = -1;
  d.sm_scale = std::isnan(desc->sm_scale) ? 1.0f / std::sqrt(128.0f + kLatentRopeDim) : desc->sm_scale;
  d.output_scale = desc->output_scale;
  d.return_lse = desc->return_lse;
  d.num_sms = desc->num_sms;
  d.flags = desc->flags;
  d.out_dtype = desc->out_dtype;
  pka_prefill_plan* p = nullptr;
  const int rc = guarded([&] {
    return make_prefill_plan(&p, d, qo_indptr_host, kv_indptr_host, true, num_tiles_out,
                             static_cast<cudaStream_t>(stream));
  });
  if (rc != PKA_OK) return rc;
  if (workspace_bytes_out) *workspace_bytes_out = prefill_workspace(*p);
  *plan_out = p;
  return PKA_OK;
}

int batch_latent_prefill_run(const pka_prefill_plan* p, const void* q, int64_t q_stride_tok,
                             int64_t q_stride_head, const void* k_nope, const void* k_rope,
                             int64_t rope_stride, const void* v, int64_t kv_stride_tok,
                             int64_t kv_stride_head, void* out, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("pka::batch_latent_prefill_run");
  clear_error();
  PKA_CHECK_ARG(p != nullptr, "plan must not be NULL");
  PKA_CHECK_ARG(p->latent, "the plan was made by batch_prefill_plan");
  PKA_CHECK_ARG(p->dev_buf != nullptr, "plan was built with PKA_PLAN_HOST_ONLY and cannot run");
  if (p->tiles.empty()) return PKA_OK;   // no query rows: tensors may be empty, of address NULL
  PKA_CHECK_ARG(q && k_nope && k_rope && v && out,
                "q, k_nope, k_rope, v and out must not be NULL");
  PKA_CHECK_ARG(!p->desc.return_lse || lse != nullptr, "the plan returns the LSE: lse is NULL");
  PKA_CHECK_ARG(aligned(out, 16) && aligned(lse, 4), "out must be 16-byte aligned, lse 4-byte");
  for (int64_t s : {q_stride_tok, q_stride_head, rope_stride, kv_stride_tok, kv_stride_head})
    PKA_CHECK_ARG(s > 0 && s % 8 == 0, "strides must be positive multiples of 8 elements");
  int rc = check_device(p->device);
  if (rc != PKA_OK) return rc;
  if (p->num_parts > 0) {
    PKA_CHECK_ARG(workspace != nullptr && aligned(workspace, 256), "workspace must be 256-byte aligned");
    if (workspace_bytes < prefill_workspace(*p))
      return fail(PKA_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, the plan needs %zu", workspace_bytes,
                  prefill_workspace(*p));
  }
  CUtensorMap qmap, kmap, rmap, vmap;
  const uint64_t H = (uint64_t)p->Hq, nk = (uint64_t)p->total_kv;
  const uint32_t qbox[3] = {64, 1, 128}, kbox[3] = {64, 1, 32}, vbox[3] = {64, 1, 64};
  {
    const uint64_t dims[3] = {192, H, (uint64_t)p->total_q};
    const uint64_t strides[2] = {(uint64_t)q_stride_head * 2, (uint64_t)q_stride_tok * 2};
    rc = encode_bf16_map(&qmap, q, 3, dims, strides, qbox);
    if (rc != PKA_OK) return rc;
  }
  {
    const uint64_t dims[3] = {128, H, nk};
    const uint64_t strides[2] = {(uint64_t)kv_stride_head * 2, (uint64_t)kv_stride_tok * 2};
    rc = encode_bf16_map(&kmap, k_nope, 3, dims, strides, kbox);
    if (rc != PKA_OK) return rc;
    rc = encode_bf16_map(&vmap, v, 3, dims, strides, vbox);
    if (rc != PKA_OK) return rc;
  }
  {
    const uint64_t dims[3] = {64, 1, nk};
    const uint64_t strides[2] = {128, (uint64_t)rope_stride * 2};
    rc = encode_bf16_map(&rmap, k_rope, 3, dims, strides, kbox);
    if (rc != PKA_OK) return rc;
  }
  PrefillArgs a{};
  a.q = q;
  a.q_stride_tok = q_stride_tok;
  a.q_stride_head = q_stride_head;
  a.out = out;
  a.lse = p->desc.return_lse ? lse : nullptr;
  a.tiles = p->d_tiles;
  a.status = p->d_status;
  a.num_qo_heads = p->Hq;
  a.num_kv_heads = p->Hkv;
  a.group = 1;
  a.causal = p->desc.mask == PKA_MASK_CAUSAL;
  a.window_left = -1;
  a.scale_log2 = p->scale * 1.4426950408889634f;
  a.output_scale = p->desc.output_scale;
  a.out_dtype = p->desc.out_dtype;
  LatentPrefillParts parts{};
  parts.segments = p->d_segments;
  parts.part = p->d_part;
  parts.cuts = reinterpret_cast<const LatentPrefillCut*>(p->d_cuts);
  parts.ws_o = static_cast<float*>(workspace);
  parts.ws_lse = parts.ws_o + (size_t)p->num_parts * 256 * 128;
  parts.num_segments = (int32_t)p->segments.size() - 1;
  parts.num_cuts = (int32_t)(p->cuts.size() * 4 / sizeof(LatentPrefillCut));
  return launch_latent_prefill(*p, a, parts, qmap, kmap, rmap, vmap, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
