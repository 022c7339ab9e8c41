// Latent attention and the page bookkeeping around it: plan object, argument
// blocks and kernel launchers.
#pragma once

#include <cstdint>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

#include "pka.h"
#include "prefill.h"

namespace pka {

constexpr int kLatentTile = 64;        // keys per tile of the latent decode
constexpr int kLatentRopeDim = 64;
constexpr int kLatentFewPieces = 8;    // pieces that one CTA merges for a whole row

// A weight is held as 2^(score - reference + shift) on its way into P V.  A reference is at
// most 2^8 below the row's largest weight, so in f16, which ends at 2^16, there is room for
// 2^7 more: weights then keep f16's full precision down to 2^-21 of the largest and come in
// steps of 2^-31 of it below (without it 2^-14 and 2^-24: 20000 keys of 2^-25 each were lost
// from the output, not from the sum).  bf16 has the exponents of 32 bits.
template <bool F16>
constexpr float kLatentWeightShift = F16 ? 7.f : 0.f;

// A run of key tiles of one request (16 bytes, one aligned load).
struct LatentItem {
  int32_t request;
  int32_t tile_lo;
  int32_t tile_hi;
  int32_t part;      // which of the request's partial states, -1 when it is whole
};

// The same on the device, with what a CTA needs of the request (32 bytes): one load
// and not a chain of three behind the launch.
struct alignas(16) LatentPiece {
  int32_t request;
  int32_t tile_lo;
  int32_t tile_hi;
  int32_t part;
  int32_t q_start, q_len, kv_len, part_base;   // of LatentReq
};

// Per-request data (32 bytes).
struct LatentReq {
  int32_t q_start;    // first packed query row
  int32_t q_len;
  int32_t kv_len;     // planned key count (an upper bound when lengths are live)
  int32_t part_base;  // first fp32 partial row, -1 when the request is not split
  int32_t n_parts;
  int32_t pad0, pad1, pad2;
};

struct LatentArgs {
  const void* q;
  int64_t q_stride_tok;
  int64_t q_stride_head;
  const int32_t* block_tables;
  int64_t bt_row_stride;
  const int32_t* seq_lens_live;  // nullptr for a frozen plan
  void* out;
  float* lse;                    // nullptr: no LSE output
  float* ws_o;                   // fp32 partial outputs [partial_rows, latent_dim]
  float* ws_lse;                 // fp32 partial base-2 LSEs [partial_rows]
  const LatentPiece* pieces;     // the first of each segment, then its further ones by segment
  const int32_t* more;           // where each segment's further pieces begin, then their end
  const LatentReq* splits;       // the requests cut into pieces, those of many first
  int32_t* status;
  int32_t num_segments;
  int32_t num_splits;
  int32_t num_many;              // of them with more than kLatentFewPieces
  int32_t row_blocks;            // CTAs side by side over a request's rows
  int32_t max_rows;              // the most rows (token, head) of a request
  int32_t num_heads;
  int32_t page_size;
  int32_t box_rows;              // cache rows of one copy (divides page_size and 64)
  int32_t q_box;                 // query heads of one copy, 0: queries by plain loads
  int32_t num_pages;
  int32_t causal;
  float scale_log2;              // scale * log2(e)
  float output_scale;
  int32_t out_dtype;
};

// The pieces of one tile of a latent prefill that was cut along its keys (32 bytes).
struct LatentPrefillCut {
  int32_t head;
  int32_t q_tile;    // 256-row tile index inside the request
  int32_t q0;        // the request's first packed query row
  int32_t lq;        // its query rows
  int32_t part0;     // first of its partial states (256 rows each)
  int32_t n_parts;
  int32_t pad0, pad1;
};

struct LatentPrefillParts {
  const int32_t* segments;       // where each pair's tiles but its first begin, then the tile count
  const int32_t* part;           // per tile its partial state, -1 when it is whole
  const LatentPrefillCut* cuts;
  float* ws_o;                   // fp32 partial outputs [parts, 128 / 8, 256, 8]
  float* ws_lse;                 // fp32 partial base-2 LSEs [parts, 256]
  int32_t num_segments;
  int32_t num_cuts;
};

}  // namespace pka

struct pka_latent_plan {
  pka_latent_desc desc;       // normalised copy
  int32_t total_q = 0, max_rows = 0, row_tile = 0, row_blocks = 0;
  int32_t partial_rows = 0, num_many = 0;
  int64_t workspace_bytes = 0;
  int64_t ws_lse_offset = 0;
  std::vector<pka::LatentItem> items;
  std::vector<int32_t> segments;
  std::vector<pka::LatentReq> reqs, splits;
  // one device allocation: pieces | further pieces' offsets | splits | status word
  void* dev_buf = nullptr;
  size_t capacity = 0;          // of dev_buf and of host_stage
  const pka::LatentPiece* d_pieces = nullptr;
  const int32_t* d_more = nullptr;
  const pka::LatentReq* d_splits = nullptr;
  int32_t* d_status = nullptr;
  int device = -1;
  // pinned host image of dev_buf; stage_done marks when its last upload has read it
  void* host_stage = nullptr;
  cudaEvent_t stage_done = nullptr;
};

namespace pka {

// Fills the host arrays of a latent decode plan.
int build_latent_plan(pka_latent_plan& plan, const pka_latent_desc& desc,
                      const int32_t* seq_lens_kv, const int32_t* qo_indptr);

// The latent decode and, when requests are split, the merge of their pieces.
int launch_latent_decode(const pka_latent_plan& plan, const LatentArgs& args, const void* pages,
                         int64_t stride_page, cudaStream_t stream);

// The decode of plans whose row tile is 128, without the merge.
int launch_latent_decode_pair(const pka_latent_plan& plan, const LatentArgs& args, const void* pages,
                              int64_t stride_page, cudaStream_t stream);

int launch_kv_tables(const int32_t* kv_lens, const int32_t* new_lens, int32_t batch,
                     const int32_t* free_pages, int32_t num_free, const int32_t* free_head,
                     int32_t page_size, int32_t* tables, int64_t row_stride, int32_t width,
                     int32_t* seq_lens, int32_t* qo_indptr, int64_t* slot_map, int64_t num_slots,
                     int32_t* free_head_out, int32_t* status, cudaStream_t stream);

int launch_latent_append(const void* latent, int64_t latent_stride, const void* rope,
                         int64_t rope_stride, int32_t latent_dim, int32_t rope_dim,
                         const int64_t* slot_map, int64_t num_tokens, void* pages,
                         int64_t num_pages, int32_t page_size, int64_t stride_page,
                         int32_t* status, cudaStream_t stream);

// Expanded prefill over a prefill plan's tiles (heads of 128 + 64 key and 128
// value dimensions) and the merge of those that were cut.
int launch_latent_prefill(const pka_prefill_plan& plan, const PrefillArgs& args, const LatentPrefillParts& parts,
                          const CUtensorMap& qmap, const CUtensorMap& kmap,
                          const CUtensorMap& rmap, const CUtensorMap& vmap, cudaStream_t stream);

}  // namespace pka
