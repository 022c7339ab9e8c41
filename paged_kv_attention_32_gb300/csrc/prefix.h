// Decode behind shared prefixes: the plan, the argument block of the prefix kernel and its
// launcher.  The requests' own keys go through the decode kernels.
#pragma once

#include <cstdint>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

#include "pka.h"
#include "plan.h"

namespace pka {

constexpr int kPrefixTile = 64;        // keys per tile
constexpr int kPrefixRows = 256;       // query rows (token, head of the KV head's group) of a pair of CTAs

struct PrefixArgs {
  const void* q;
  int64_t q_stride_tok, q_stride_head;
  const int32_t* block_tables;
  int64_t bt_row_stride;
  const PrefixItem* items;
  const PrefixToken* tokens;
  float* ws_o;                   // fp32 partial outputs [partial_rows, 128]
  float* ws_lse;                 // fp32 partial base-2 LSEs [partial_rows]
  int32_t* status;
  int32_t num_items;
  int32_t group;                 // Hq / Hkv
  int32_t page_units;            // page_size / 16
  int32_t k_rows, v_rows;        // cache rows of one copy
  int32_t num_pages;
  uint32_t negate;               // sign bits of a q word, flipped where the scale is negative
  float scale_log2;              // |scale| * log2(e)
};

// Fills a decode plan whose requests, in groups, begin with the same pages.  group_indptr
// [num_groups + 1] deals out the requests, prefix_pages [num_groups] are the shared ones.
int build_prefix_plan(pka_plan& plan, const pka_decode_desc& desc, const int32_t* seq_lens_kv,
                      const int32_t* qo_indptr, const int32_t* group_indptr, int32_t num_groups,
                      const int32_t* prefix_pages);

int launch_prefix(const PrefixArgs& args, bool f16, const CUtensorMap& kmap, const CUtensorMap& vmap,
                  cudaStream_t stream);

}  // namespace pka
