// Decode behind shared prefixes: plan object, argument blocks and kernel launchers.
#pragma once

#include <cstdint>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

#include "pka.h"
#include "plan.h"

namespace pka {

constexpr int kPrefixTile = 64;      // keys per tile of a shared prefix
constexpr int kPrefixRows = 256;     // query rows of a pair of CTAs
constexpr int kOwnRows = 16;         // query rows of a piece of a request's own keys
constexpr int kOwnWarps = 4;         // warps of a CTA over the requests' own keys
constexpr int kOwnCtas = 3;          // of them per SM

// A piece of a shared prefix for one KV head and up to 256 of its group's query rows (48 bytes, three aligned loads).  A query row is (token, head of the KV head's group).
struct alignas(16) PrefixItem {
  int32_t row;        // the table row that lists the prefix's pages
  int32_t kv_head;
  int32_t tile_lo;    // 64-key tiles [tile_lo, tile_hi)
  int32_t tile_hi;
  int32_t keys;       // of the whole prefix
  int32_t q_start;    // the group's first packed query row
  int32_t rows;       // its query rows times the heads of the KV head's group
  int32_t row0;       // the first of them here
  int32_t state;      // where the first row's partial state goes
  int32_t pad0, pad1, pad2;
};

// A run of 16-key units of one request's own keys, for one KV head and up to 16 of the
// request's query rows (32 bytes, two aligned loads).
struct alignas(16) OwnPiece {
  int32_t request;
  int32_t head_tile;  // KV head | 16-row tile << 16
  int32_t unit_lo;
  int32_t unit_hi;
  int32_t state;      // where the first row's partial state goes
  int32_t q_start, q_len, kv_len;   // of the request
};

// The partial states of a tile of rows: row r's are at base + k * rows + r, k < count.
struct StateRun {
  int32_t base, count, rows, pad;
};

// Where a packed query row's states are (32 bytes): of its request's own keys, row own_row + g
// (g: head of the KV head's group) in the runs own_run + kv_head * own_tiles + tile, and of the
// shared prefix, row pre_row + g alike; pre_row is -1 where nothing is shared.
struct alignas(16) TokenStates {
  int32_t own_row, own_run, own_tiles;
  int32_t pre_row, pre_run, pre_tiles;
  int32_t pad0, pad1;
};

// What the table row of a request is to hold: its pages, of which the first `shared` are those of
// row `first`.
struct alignas(16) RowPages {
  int32_t first, shared, pages, pad;
};

struct PrefixArgs {
  const void* q;
  int64_t q_stride_tok, q_stride_head;
  const int32_t* block_tables;
  int64_t bt_row_stride;
  const PrefixItem* items;       // the first of each pair, then the further ones by pair
  const int32_t* more;           // [pairs + 1]: where each pair's further items begin, then their end
  float* ws_o;                   // fp32 partial outputs [partial_rows, 128]
  float* ws_lse;                 // fp32 partial base-2 LSEs [partial_rows]
  int32_t* status;
  int32_t num_pairs;
  int32_t group;                 // Hq / Hkv
  int32_t page_units;            // page_size / 16
  int32_t k_rows, v_rows;        // cache rows of one copy
  int32_t num_pages;
  uint32_t negate;               // sign bits of a q word, flipped where the scale is negative
  float scale_log2;              // |scale| * log2(e)
};

struct OwnArgs {
  DecodeArgs decode;             // ws_o, ws_lse and status among it; no items
  const OwnPiece* pieces;
  int32_t* next;                 // pieces taken beyond the first num_static; 0 between runs
  int32_t num_pieces;
  int32_t num_static;            // the first pieces: those that warps of
  int32_t static_ctas;           // these CTAs begin with
  int32_t num_ctas;
};

struct PrefixMergeArgs {
  const float* ws_o;
  const float* ws_lse;
  const TokenStates* tokens;
  const StateRun* runs;
  int32_t* next;                 // set back for the next run
  const float* sinks;
  void* out;
  float* lse;
  int32_t total_q, num_qo_heads, group;
  int32_t most_states;           // that a row has
  float bmm2_scale;
  int32_t out_dtype;
};

// The prefix kernel over the plan's items, in the shape for products or for memory.
int launch_prefix(const PrefixArgs& args, bool f16, bool dense, const CUtensorMap& kmap,
                  const CUtensorMap& vmap, cudaStream_t stream);
// The requests' own keys, and the merge of all states; each starts while the kernel before
// it ends.
int launch_prefix_own(const OwnArgs& args, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream);
int launch_prefix_merge(const PrefixMergeArgs& args, cudaStream_t stream);

// Sets STATUS_PAGE_BOUNDS for an entry outside the pool, STATUS_PREFIX for one that a group's rows
// are to share and do not.
int launch_prefix_check(const RowPages* rows, int32_t batch, const int32_t* tables, int64_t row_stride,
                        const int32_t* seq_lens_live, int32_t page_size, int32_t num_pages, int32_t* status,
                        cudaStream_t stream);

}  // namespace pka

struct pka_prefix_plan {
  pka_plan base;               // the same batch without sharing: normalised, with its query
                               // rows, and what runs where nothing is worth sharing
  bool shared = false;
  int64_t min_shared_bytes = -1;   // as given
  bool dense = false;          // the prefixes' products take longer than all reads
  int32_t partial_rows = 0, most_states = 0;   // states in all, and at most of one row
  int64_t workspace_bytes = 0, ws_lse_offset = 0;
  std::vector<pka::PrefixItem> items;
  std::vector<int32_t> more;
  int32_t own_ctas = 0, own_static = 0;
  std::vector<pka::OwnPiece> pieces;
  std::vector<pka::StateRun> runs;
  std::vector<pka::TokenStates> tokens;
  std::vector<pka::RowPages> rows;
  // one device allocation: items | pieces | runs | tokens | more | rows | status word, count
  void* dev_buf = nullptr;
  size_t capacity = 0;         // of dev_buf and of host_stage
  const pka::PrefixItem* d_items = nullptr;
  const pka::OwnPiece* d_pieces = nullptr;
  const pka::StateRun* d_runs = nullptr;
  const pka::TokenStates* d_tokens = nullptr;
  const int32_t* d_more = nullptr;
  const pka::RowPages* d_rows = nullptr;
  int32_t* d_status = nullptr;   // with the count of pieces taken behind it
  int device = -1;
  // pinned host image of dev_buf; stage_done marks when its last upload has read it
  void* host_stage = nullptr;
  cudaEvent_t stage_done = nullptr;
};

namespace pka {

// Fills the host arrays of a plan.  group_indptr [num_groups + 1] deals out the requests,
// prefix_pages [num_groups] are the leading pages that a group's requests share.
int build_prefix_plan(pka_prefix_plan& plan, const pka_decode_desc& desc, const int32_t* seq_lens_kv,
                      const int32_t* qo_indptr, const int32_t* group_indptr, int32_t num_groups,
                      const int32_t* prefix_pages, int64_t min_shared_bytes);

}  // namespace pka
