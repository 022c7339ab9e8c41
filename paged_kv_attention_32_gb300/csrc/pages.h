// A K/V page pool at work: rows rotated and written to it, its pages forked, released,
// compacted and copied.  Argument blocks and kernel launchers.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "pka.h"

namespace pka {

constexpr int kRopeAxes = 4;            // position axes of a rotation
constexpr int kPoolsPerLaunch = 32;     // pools that one copy kernel serves
constexpr int kPageOpRows = 16384;      // table rows of a fork, release or compaction
constexpr int64_t kPageOpPages = 1 << 22;   // pages whose bits one cluster holds

struct RopeArgs {
  const void* q;                 // nullptr: no queries
  int64_t q_stride_tok, q_stride_head;
  void* q_out;
  int64_t qo_stride_tok, qo_stride_head;
  const void* k;
  const void* v;
  int64_t kv_stride_tok, kv_stride_head;
  const int32_t* positions;      // [axes, tokens], rows pos_stride apart
  int64_t pos_stride;
  const double* inv_freq;        // [rotary / 2]
  const int64_t* slot_map;
  void* k_pages;
  void* v_pages;
  int64_t stride_page, stride_head;
  int64_t num_slots;             // of the pool: pages * page_size
  int32_t* status;
  int32_t num_tokens;
  int32_t num_qo_heads, num_kv_heads;
  int32_t page_size;
  int32_t rotary;                // values of a row that are rotated
  int32_t axis_end[kRopeAxes];   // frequencies below axis_end[a] that no earlier axis has: axis a
};

int launch_rope_append(const RopeArgs& args, bool f16, bool halves, cudaStream_t stream);

struct ForkArgs {
  const int32_t* parents;
  const int32_t* children;
  int32_t num_forks;
  const int32_t* kv_lens;
  int32_t batch;
  const int32_t* free_pages;
  int32_t num_free;
  const int32_t* free_head;
  int32_t page_size;
  int32_t* tables;
  int64_t row_stride;
  int32_t width;
  int32_t* seq_lens;
  int32_t* src_pages;
  int32_t* dst_pages;
  int32_t* free_head_out;
  int32_t* status;
};

int launch_kv_fork(const ForkArgs& args, cudaStream_t stream);

struct ReleaseArgs {
  const int32_t* rows;
  int32_t num_rows;
  const int32_t* kv_lens;
  int32_t batch;
  int32_t* free_pages;
  int32_t num_free;
  const int32_t* free_head;
  int32_t page_size;
  const int32_t* tables;
  int64_t row_stride;
  int32_t width;
  int32_t num_pages;
  int32_t* seq_lens;
  int32_t* free_head_out;
  int32_t* status;
};

int launch_kv_free(const ReleaseArgs& args, cudaStream_t stream);

struct CompactArgs {
  const int32_t* kv_lens;
  int32_t batch;
  const int32_t* free_pages;
  int32_t num_free;
  const int32_t* free_head;
  int32_t page_size;
  const int32_t* tables;
  int64_t row_stride;
  int32_t width;
  int32_t num_pages;
  int32_t* tables_out;
  int64_t out_row_stride;
  int32_t* free_pages_out;
  int32_t* src_pages;
  int32_t* dst_pages;
  int32_t max_moves;
  int32_t* num_moves;
  int32_t* status;
};

int launch_kv_compact(const CompactArgs& args, cudaStream_t stream);

struct PagePool {
  uint8_t* base;
  int64_t stride;    // bytes from page to page
  int64_t bytes;     // of a page, a multiple of 16
};

struct CopyArgs {
  PagePool pools[kPoolsPerLaunch];
  const int32_t* src_pages;
  const int32_t* dst_pages;
  const int32_t* count;    // nullptr: num_entries
  int32_t num_entries;
  int32_t num_pools;
  int32_t num_pages;
  int32_t* status;
};

int launch_kv_copy(const CopyArgs& args, cudaStream_t stream);

}  // namespace pka
