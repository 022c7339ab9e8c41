// extern "C" entry points of decode behind shared prefixes: argument checks, plan
// ownership, launch dispatch.
#include <cmath>
#include <new>

#include "host_common.h"
#include "kernels.h"
#include "prefix.h"
#include "tmap.h"

using namespace pka;

struct pka_prefix_plan {
  pka_plan decode;   // the requests' own keys, and the prefixes' pieces
};

extern "C" {

int paged_prefix_decode_plan(pka_prefix_plan** plan_out, const pka_decode_desc* desc,
                             const int32_t* seq_lens_kv_host, const int32_t* qo_indptr_host,
                             const int32_t* group_indptr_host, int32_t num_groups,
                             const int32_t* prefix_pages_host, size_t* workspace_bytes_out, void* stream) {
  NvtxRange nvtx_range("pka::paged_prefix_decode_plan");
  clear_error();
  PKA_CHECK_ARG(plan_out != nullptr && desc != nullptr, "plan_out and desc must not be NULL");
  *plan_out = nullptr;
  pka_prefix_plan* p = new (std::nothrow) pka_prefix_plan();
  if (p == nullptr) return fail(PKA_ERR_INVALID_ARG, "out of host memory");
  const int rc = guarded([&] {
    const int built = build_prefix_plan(p->decode, *desc, seq_lens_kv_host, qo_indptr_host, group_indptr_host,
                                        num_groups, prefix_pages_host);
    if (built != PKA_OK || (desc->flags & PKA_PLAN_HOST_ONLY)) return built;
    return upload_decode_plan(p->decode, static_cast<cudaStream_t>(stream));
  });
  if (rc != PKA_OK) {
    paged_prefix_decode_plan_destroy(p);
    return rc;
  }
  if (workspace_bytes_out) *workspace_bytes_out = (size_t)p->decode.workspace_bytes;
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
  const int rc = guarded([&] {
    pka_decode_desc d = p->decode.desc;
    d.batch_size = batch_size;
    pka_plan fresh;
    const int built = build_prefix_plan(fresh, d, seq_lens_kv_host, qo_indptr_host, group_indptr_host, num_groups,
                                        prefix_pages_host);
    if (built != PKA_OK) return built;   // the old plan stays as it was
    return replace_decode_plan(p->decode, std::move(fresh), static_cast<cudaStream_t>(stream));
  });
  if (rc != PKA_OK) return rc;
  if (workspace_bytes_out) *workspace_bytes_out = (size_t)p->decode.workspace_bytes;
  return PKA_OK;
}

void paged_prefix_decode_plan_destroy(pka_prefix_plan* p) {
  if (p == nullptr) return;
  release_decode_plan(p->decode);
  delete p;
}

int paged_prefix_decode_plan_info(const pka_prefix_plan* p, pka_plan_info* info, int32_t* num_pieces_out,
                                  int32_t* prefix_chunks_out) {
  PKA_CHECK_ARG(p != nullptr, "plan must not be NULL");
  const int rc = paged_decode_plan_info(&p->decode, info);
  if (rc != PKA_OK) return rc;
  if (num_pieces_out) *num_pieces_out = (int32_t)p->decode.prefix_items.size();
  if (prefix_chunks_out)
    for (int32_t b = 0; b < p->decode.B; ++b)
      prefix_chunks_out[b] = p->decode.reqs[b].n_chunks - p->decode.reqs[b].n_items;
  return PKA_OK;
}

int paged_prefix_decode_plan_check(const pka_prefix_plan* p, void* stream) {
  PKA_CHECK_ARG(p != nullptr, "plan must not be NULL");
  return paged_decode_plan_check(&p->decode, stream);
}

int paged_prefix_decode_run(const pka_prefix_plan* plan, const void* q, int64_t q_stride_tok, int64_t q_stride_head,
                            const void* k_pages, const void* v_pages, int64_t kv_stride_page, int64_t kv_stride_head,
                            const int32_t* block_tables, int64_t bt_row_stride, const int32_t* seq_lens_kv_dev,
                            const float* sinks, void* out, float* lse, void* workspace, size_t workspace_bytes,
                            void* stream) {
  NvtxRange nvtx_range("pka::paged_prefix_decode_run");
  clear_error();
  PKA_CHECK_ARG(plan != nullptr, "plan must not be NULL");
  const pka_plan* p = &plan->decode;
  DecodeArgs a{};
  CUtensorMap kmap, vmap;
  int rc = prepare_decode_run(p, q, q_stride_tok, q_stride_head, k_pages, v_pages, kv_stride_page, kv_stride_head,
                              block_tables, bt_row_stride, seq_lens_kv_dev, sinks, out, lse, workspace,
                              workspace_bytes, &a, &kmap, &vmap);
  if (rc != PKA_OK) return rc;
  if (!p->prefix_items.empty()) {
    PrefixArgs x{};
    x.q = q;
    x.q_stride_tok = q_stride_tok;
    x.q_stride_head = q_stride_head;
    x.block_tables = block_tables;
    x.bt_row_stride = bt_row_stride;
    x.items = p->d_prefix_items;
    x.tokens = p->d_prefix_tokens;
    x.ws_o = a.ws_o;
    x.ws_lse = a.ws_lse;
    x.status = p->d_status;
    x.num_items = (int32_t)p->prefix_items.size();
    x.group = p->G;
    x.page_units = p->ps / 16;
    x.v_rows = p->ps % 64 == 0 ? 64 : p->ps % 32 == 0 ? 32 : 16;
    x.k_rows = x.v_rows < 32 ? 16 : 32;
    x.num_pages = (int32_t)p->desc.num_pages;
    x.negate = a.scale_log2 < 0.f ? 0x80008000u : 0u;
    x.scale_log2 = std::fabs(a.scale_log2);
    CUtensorMap kbox, vbox;
    rc = encode_kv_box_map(&kbox, k_pages, p->desc.num_pages, p->Hkv, p->ps, kv_stride_page, kv_stride_head,
                           x.k_rows, x.k_rows == 32 ? 2 : 1);
    if (rc != PKA_OK) return rc;
    rc = encode_kv_box_map(&vbox, v_pages, p->desc.num_pages, p->Hkv, p->ps, kv_stride_page, kv_stride_head,
                           x.v_rows, 1);
    if (rc != PKA_OK) return rc;
    rc = launch_prefix(x, a.in_f16 != 0, kbox, vbox, static_cast<cudaStream_t>(stream));
    if (rc != PKA_OK) return rc;
    a.behind_prefix = 1;
  }
  return launch_decode(*p, a, kmap, vmap, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
