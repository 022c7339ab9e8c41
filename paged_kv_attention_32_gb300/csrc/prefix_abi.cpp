// extern "C" entry points of decode behind shared prefixes: argument checks, plan
// ownership, launch dispatch.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <utility>

#include "host_common.h"
#include "kernels.h"
#include "prefix.h"
#include "tmap.h"

using namespace pka;

namespace {

// Makes `next`, whose host arrays are built, the plan *p on the device: in p's buffers, or
// in larger ones.  Where anything fails p stays the plan that it was.
int install_prefix_plan(pka_prefix_plan& p, pka_prefix_plan&& next, cudaStream_t stream) {
  const size_t size[] = {next.items.size() * sizeof(PrefixItem),
                         next.pieces.size() * sizeof(OwnPiece),
                         next.runs.size() * sizeof(StateRun),
                         next.tokens.size() * sizeof(TokenStates),
                         next.more.size() * sizeof(int32_t),
                         next.rows.size() * sizeof(RowPages),
                         256};
  const void* from[] = {next.items.data(), next.pieces.data(), next.runs.data(), next.tokens.data(),
                        next.more.data(), next.rows.data()};
  constexpr int kArrays = 6;
  size_t off[kArrays + 1], total = 0;
  for (int i = 0; i <= kArrays; ++i) {
    off[i] = total;
    total += up256(size[i]);
  }
  if (p.stage_done == nullptr)
    PKA_CUDA_TRY(cudaEventCreateWithFlags(&p.stage_done, cudaEventDisableTiming), "cudaEventCreate(plan upload)");
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
    PKA_CUDA_TRY(cudaMalloc(&next.dev_buf, next.capacity), "cudaMalloc(prefix plan)");
    const cudaError_t e = cudaMallocHost(&next.host_stage, next.capacity);
    if (e != cudaSuccess) {
      const int rc = cuda_fail(e, "cudaMallocHost(plan image)");
      ignored(cudaFree(next.dev_buf));
      return rc;
    }
  }
  uint8_t* base = static_cast<uint8_t*>(next.dev_buf);
  next.d_items = reinterpret_cast<const PrefixItem*>(base + off[0]);
  next.d_pieces = reinterpret_cast<const OwnPiece*>(base + off[1]);
  next.d_runs = reinterpret_cast<const StateRun*>(base + off[2]);
  next.d_tokens = reinterpret_cast<const TokenStates*>(base + off[3]);
  next.d_more = reinterpret_cast<const int32_t*>(base + off[4]);
  next.d_rows = reinterpret_cast<const RowPages*>(base + off[5]);
  next.d_status = reinterpret_cast<int32_t*>(base + off[kArrays]);
  uint8_t* img = static_cast<uint8_t*>(next.host_stage);
  for (int i = 0; i < kArrays; ++i)
    if (size[i] > 0) std::memcpy(img + off[i], from[i], size[i]);
  std::memset(img + off[kArrays], 0, 256);
  cudaError_t e = cudaMemcpyAsync(base, img, total, cudaMemcpyHostToDevice, stream);
  if (e != cudaSuccess) {
    if (grow) {
      ignored(cudaFree(next.dev_buf));
      ignored(cudaFreeHost(next.host_stage));
    }
    return cuda_fail(e, "cudaMemcpyAsync(prefix plan)");
  }
  // from here on the device has the new plan; a copy that no event follows is waited for
  e = cudaEventRecord(next.stage_done, stream);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    e = cudaStreamSynchronize(stream);
  }
  if (grow) {
    ignored(cudaFree(p.dev_buf));
    ignored(cudaFreeHost(p.host_stage));
  }
  keep_decode_buffers(next.base, p.base);   // for a batch that shares nothing
  p = std::move(next);
  return e == cudaSuccess ? PKA_OK : cuda_fail(e, "cudaEventRecord(plan upload)");
}

// Builds a plan and makes it *p; p stays the plan that it was where that fails.
int make_prefix_plan(pka_prefix_plan& p, const pka_decode_desc& desc, const int32_t* seq_lens_kv,
                     const int32_t* qo_indptr, const int32_t* group_indptr, int32_t num_groups,
                     const int32_t* prefix_pages, int64_t min_shared_bytes, cudaStream_t stream) {
  pka_prefix_plan next;
  int rc = build_prefix_plan(next, desc, seq_lens_kv, qo_indptr, group_indptr, num_groups, prefix_pages,
                             min_shared_bytes);
  if (rc != PKA_OK) return rc;
  if (desc.flags & PKA_PLAN_HOST_ONLY) {
    p = std::move(next);
    return PKA_OK;
  }
  if (next.shared) return install_prefix_plan(p, std::move(next), stream);
  if (p.base.dev_buf == nullptr) {
    PKA_CUDA_TRY(cudaGetDevice(&next.base.device), "cudaGetDevice");
    rc = upload_decode_plan(next.base, stream);
    if (rc != PKA_OK) {
      release_decode_plan(next.base);
      return rc;
    }
    p.base = std::move(next.base);
  } else {
    rc = check_device(p.base.device);
    if (rc == PKA_OK) rc = replace_decode_plan(p.base, std::move(next.base), stream);
    if (rc != PKA_OK) return rc;
  }
  p.shared = false;   // only now: what fails leaves the plan as it was
  p.min_shared_bytes = next.min_shared_bytes;
  p.items.clear();
  p.pieces.clear();
  p.partial_rows = next.partial_rows;
  p.most_states = next.most_states;
  p.workspace_bytes = next.workspace_bytes;
  return PKA_OK;
}

}  // namespace

extern "C" {

int paged_prefix_decode_plan(pka_prefix_plan** plan_out, const pka_decode_desc* desc,
                             const int32_t* seq_lens_kv_host, const int32_t* qo_indptr_host,
                             const int32_t* group_indptr_host, int32_t num_groups,
                             const int32_t* prefix_pages_host, int64_t min_shared_bytes,
                             size_t* workspace_bytes_out, void* stream) {
  NvtxRange nvtx_range("pka::paged_prefix_decode_plan");
  clear_error();
  PKA_CHECK_ARG(plan_out != nullptr && desc != nullptr, "plan_out and desc must not be NULL");
  *plan_out = nullptr;
  pka_prefix_plan* p = new (std::nothrow) pka_prefix_plan();
  if (p == nullptr) return fail(PKA_ERR_INVALID_ARG, "out of host memory");
  const int rc = guarded([&] {
    return make_prefix_plan(*p, *desc, seq_lens_kv_host, qo_indptr_host, group_indptr_host, num_groups,
                            prefix_pages_host, min_shared_bytes, static_cast<cudaStream_t>(stream));
  });
  if (rc != PKA_OK) {
    paged_prefix_decode_plan_destroy(p);
    return rc;
  }
  if (workspace_bytes_out) *workspace_bytes_out = (size_t)p->workspace_bytes;
  *plan_out = p;
  return PKA_OK;
}

int paged_prefix_decode_plan_update(pka_prefix_plan* p, int32_t batch_size, const int32_t* seq_lens_kv_host,
                                    const int32_t* qo_indptr_host, const int32_t* group_indptr_host,
                                    int32_t num_groups, const int32_t* prefix_pages_host,
                                    size_t* workspace_bytes_out, void* stream) {
  NvtxRange nvtx_range("pka::paged_prefix_decode_plan_update");
  clear_error();
  PKA_CHECK_ARG(p != nullptr, "plan must not be NULL");
  if (!(p->base.desc.flags & PKA_PLAN_HOST_ONLY)) {
    const int rc = check_device(p->shared ? p->device : p->base.device);
    if (rc != PKA_OK) return rc;
  }
  const int rc = guarded([&] {
    pka_decode_desc d = p->base.desc;
    d.batch_size = batch_size;
    return make_prefix_plan(*p, d, seq_lens_kv_host, qo_indptr_host, group_indptr_host, num_groups,
                            prefix_pages_host, p->min_shared_bytes, static_cast<cudaStream_t>(stream));
  });
  if (rc != PKA_OK) return rc;
  if (workspace_bytes_out) *workspace_bytes_out = (size_t)p->workspace_bytes;
  return PKA_OK;
}

void paged_prefix_decode_plan_destroy(pka_prefix_plan* p) {
  if (p == nullptr) return;
  if (p->stage_done != nullptr) {
    ignored(cudaEventSynchronize(p->stage_done));   // the image is not freed under a pending copy
    ignored(cudaEventDestroy(p->stage_done));
  }
  if (p->host_stage != nullptr) ignored(cudaFreeHost(p->host_stage));
  if (p->dev_buf != nullptr) ignored(cudaFree(p->dev_buf));
  release_decode_plan(p->base);
  delete p;
}

int paged_prefix_decode_plan_info(const pka_prefix_plan* p, pka_prefix_plan_info* info) {
  clear_error();
  PKA_CHECK_ARG(p != nullptr && info != nullptr, "plan and info must not be NULL");
  *info = pka_prefix_plan_info{};
  info->shared = p->shared;
  info->num_prefix_pieces = (int32_t)p->items.size();
  info->num_own_pieces = (int32_t)p->pieces.size();
  info->num_pairs = p->shared ? (int32_t)p->more.size() - 1 : 0;
  info->num_warps = p->shared ? p->own_ctas * kOwnWarps : 0;
  info->dense = p->shared && p->dense;
  info->partial_rows = p->partial_rows;
  info->total_q = p->base.total_q;
  info->num_sms = p->base.desc.num_sms;
  info->workspace_bytes = p->workspace_bytes;
  return PKA_OK;
}

int paged_prefix_decode_plan_export(const pka_prefix_plan* p, int32_t* prefix_pieces, int32_t* own_pieces) {
  clear_error();
  PKA_CHECK_ARG(p != nullptr, "plan must not be NULL");
  for (size_t i = 0; prefix_pieces != nullptr && i < p->items.size(); ++i) {
    const PrefixItem& x = p->items[i];
    const int32_t v[6] = {x.row, x.kv_head, x.row0, x.tile_lo, x.tile_hi, x.state};
    std::memcpy(prefix_pieces + 6 * i, v, sizeof(v));
  }
  for (size_t i = 0; own_pieces != nullptr && i < p->pieces.size(); ++i) {
    const OwnPiece& x = p->pieces[i];
    const int32_t v[6] = {x.request, x.head_tile & 0xffff, (x.head_tile >> 16) * kOwnRows, x.unit_lo, x.unit_hi, x.state};
    std::memcpy(own_pieces + 6 * i, v, sizeof(v));
  }
  return PKA_OK;
}

int paged_prefix_decode_plan_check(const pka_prefix_plan* p, void* stream) {
  PKA_CHECK_ARG(p != nullptr, "plan must not be NULL");
  if (!p->shared || p->d_status == nullptr) return paged_decode_plan_check(&p->base, stream);
  clear_error();
  const int rc = check_device(p->device);
  if (rc != PKA_OK) return rc;
  return read_status(p->d_status, static_cast<cudaStream_t>(stream));
}

int paged_prefix_decode_check_tables(const pka_prefix_plan* p, const int32_t* block_tables, int64_t bt_row_stride,
                                     const int32_t* seq_lens_kv_dev, void* stream) {
  NvtxRange nvtx_range("pka::paged_prefix_decode_check_tables");
  clear_error();
  PKA_CHECK_ARG(p != nullptr, "plan must not be NULL");
  if (!p->shared) return paged_decode_check_tables(&p->base, block_tables, bt_row_stride, seq_lens_kv_dev, stream);
  PKA_CHECK_ARG(p->dev_buf != nullptr, "plan has no device state");
  PKA_CHECK_ARG(block_tables != nullptr, "block_tables must not be NULL");
  PKA_CHECK_ARG(bt_row_stride >= p->base.C, "bt_row_stride (%lld) is smaller than the table width %d",
                (long long)bt_row_stride, p->base.C);
  const int rc = check_device(p->device);
  if (rc != PKA_OK) return rc;
  return launch_prefix_check(p->d_rows, (int32_t)p->rows.size(), block_tables, bt_row_stride,
                             p->base.desc.freeze_seq_lens ? nullptr : seq_lens_kv_dev, p->base.ps,
                             (int32_t)p->base.desc.num_pages, p->d_status, static_cast<cudaStream_t>(stream));
}

int paged_prefix_decode_run(const pka_prefix_plan* p, const void* q, int64_t q_stride_tok, int64_t q_stride_head,
                            const void* k_pages, const void* v_pages, int64_t kv_stride_page, int64_t kv_stride_head,
                            const int32_t* block_tables, int64_t bt_row_stride, const int32_t* seq_lens_kv_dev,
                            const float* sinks, void* out, float* lse, void* workspace, size_t workspace_bytes,
                            void* stream_ptr) {
  NvtxRange nvtx_range("pka::paged_prefix_decode_run");
  clear_error();
  PKA_CHECK_ARG(p != nullptr, "plan must not be NULL");
  if (!p->shared)
    return run_decode_plan(p->base, q, q_stride_tok, q_stride_head, k_pages, v_pages, kv_stride_page, kv_stride_head,
                           block_tables, bt_row_stride, seq_lens_kv_dev, sinks, out, lse, workspace, workspace_bytes,
                           stream_ptr);
  PKA_CHECK_ARG(p->dev_buf != nullptr, "plan was built with PKA_PLAN_HOST_ONLY and cannot run");
  const pka_plan& base = p->base;
  OwnArgs own{};
  CUtensorMap kmap, vmap, kbox, vbox;
  int rc = prepare_decode_run(&base, q, q_stride_tok, q_stride_head, k_pages, v_pages, kv_stride_page, kv_stride_head,
                              block_tables, bt_row_stride, seq_lens_kv_dev, sinks, out, lse, &own.decode, &kmap, &vmap);
  if (rc != PKA_OK) return rc;
  if (workspace == nullptr || workspace_bytes < (size_t)p->workspace_bytes)
    return fail(PKA_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, the plan needs %lld", workspace_bytes,
                (long long)p->workspace_bytes);
  PKA_CHECK_ARG(aligned(workspace, 256), "workspace must be 256-byte aligned");
  rc = check_device(p->device);
  if (rc != PKA_OK) return rc;
  const int64_t num_pages = base.desc.num_pages;
  const int32_t v_rows = base.ps % 64 == 0 ? 64 : base.ps % 32 == 0 ? 32 : 16, k_rows = v_rows < 32 ? 16 : 32;
  rc = encode_kv_box_map(&kbox, k_pages, num_pages, base.Hkv, base.ps, kv_stride_page, kv_stride_head, k_rows,
                         k_rows == 32 ? 2 : 1);
  if (rc != PKA_OK) return rc;
  rc = encode_kv_box_map(&vbox, v_pages, num_pages, base.Hkv, base.ps, kv_stride_page, kv_stride_head, v_rows, 1);
  if (rc != PKA_OK) return rc;

  const cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  float* ws_o = static_cast<float*>(workspace);
  float* ws_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p->ws_lse_offset);
  own.decode.ws_o = ws_o;
  own.decode.ws_lse = ws_lse;
  own.decode.status = p->d_status;
  own.pieces = p->d_pieces;
  own.next = p->d_status + 1;
  own.num_pieces = (int32_t)p->pieces.size();
  own.num_static = p->own_static;
  own.num_ctas = p->own_ctas;
  own.static_ctas = std::min(p->own_ctas, base.desc.num_sms);
  PrefixArgs x{};
  x.q = q;
  x.q_stride_tok = q_stride_tok;
  x.q_stride_head = q_stride_head;
  x.block_tables = block_tables;
  x.bt_row_stride = bt_row_stride;
  x.items = p->d_items;
  x.more = p->d_more;
  x.ws_o = ws_o;
  x.ws_lse = ws_lse;
  x.status = p->d_status;
  x.num_pairs = (int32_t)p->more.size() - 1;
  x.group = base.G;
  x.page_units = base.ps / 16;
  x.k_rows = k_rows;
  x.v_rows = v_rows;
  x.num_pages = (int32_t)num_pages;
  x.negate = own.decode.scale_log2 < 0.f ? 0x80008000u : 0u;
  x.scale_log2 = std::fabs(own.decode.scale_log2);
  PrefixMergeArgs m{};
  m.ws_o = ws_o;
  m.ws_lse = ws_lse;
  m.tokens = p->d_tokens;
  m.runs = p->d_runs;
  m.next = p->d_status + 1;
  m.sinks = sinks;
  m.out = out;
  m.lse = own.decode.lse;
  m.total_q = base.total_q;
  m.num_qo_heads = base.Hq;
  m.group = base.G;
  m.most_states = p->most_states;
  m.bmm2_scale = base.desc.bmm2_scale;
  m.out_dtype = base.desc.out_dtype;
  rc = launch_prefix(x, own.decode.in_f16 != 0, p->dense, kbox, vbox, stream);
  if (rc == PKA_OK) rc = launch_prefix_own(own, kmap, vmap, stream);
  if (rc == PKA_OK) rc = launch_prefix_merge(m, stream);
  if (rc != PKA_OK) (void)cudaMemsetAsync(p->d_status + 1, 0, sizeof(int32_t), stream);   // as the merge leaves it
  return rc;
}

}  // extern "C"
