// What the latent decode kernels share.
#pragma once

#include "device_common.cuh"
#include "latent.h"

namespace pka {
namespace dev {

constexpr float kRescaleThreshold = 8.0f;
constexpr uint32_t kSmemLimit = 232448;   // dynamic shared memory of one CTA

// A position in a ring of N slots and the parity of its round.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// Barrier of the four warps of softmax group g.
__device__ __forceinline__ void bar_sync_group(int g) {
  asm volatile("bar.sync %0, 128;" ::"r"(g + 1) : "memory");
}

// The same, true where `mine` is true in any thread of the group.
__device__ __forceinline__ bool bar_any_group(int g, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(g + 1), "r"((uint32_t)mine)
      : "memory");
  return any != 0;
}

// The pieces of a segment.  The first lies at the segment's own index, so that its
// load does not wait for the list's.
struct Pieces {
  int seg, more, count;
  __device__ __forceinline__ Pieces(const LatentArgs& a, int segment)
      : seg(segment), more(__ldg(a.more + segment)), count(1 + __ldg(a.more + segment + 1) - more) {}
  __device__ __forceinline__ int operator[](int i) const { return i == 0 ? seg : more + i - 1; }
  __device__ __forceinline__ bool has(int i) const { return i == 0 || i < count; }
};

// What a CTA needs to know of its piece.
struct Piece {
  LatentPiece rq;
  int request, kv, tile0, n, part, row0, rows;   // rows: live rows of the CTA's row block
  __device__ __forceinline__ Piece(const LatentArgs& a, int item, int row_block, int row_tile) {
    rq = a.pieces[item];
    request = rq.request;
    part = rq.part;
    kv = rq.kv_len;
    if (a.seq_lens_live != nullptr) kv = min(max(__ldg(a.seq_lens_live + request), 0), kv);
    row0 = row_block * row_tile;
    rows = min(row_tile, rq.q_len * a.num_heads - row0);
    tile0 = rq.tile_lo;
    n = rows > 0 ? max(0, min(rq.tile_hi, (kv + kLatentTile - 1) / kLatentTile) - tile0) : 0;
  }
};

// The page and slot of one token of every tile of a piece, 64 tokens apart: no
// division per tile, and the next tile's table entry is asked for a tile ahead.
// A token past the request's last is in page num_pages, outside the pool: a copy
// from there brings zeros.
struct PageWalk {
  const int32_t* table;
  int raw, slot;                        // table entry and slot of the current tile's token
  int tok, idx, kv, planned, ps, step_pages, step_slots, none;
  bool in;
  __device__ __forceinline__ PageWalk(const LatentArgs& a, const Piece& pc, int offset, bool active)
      : table(a.block_tables + (int64_t)pc.request * a.bt_row_stride), tok(pc.tile0 * kLatentTile + offset),
        kv(pc.kv), planned(pc.rq.kv_len), ps(a.page_size), none(a.num_pages), in(active) {
    idx = tok / ps;
    slot = tok - idx * ps;
    step_pages = kLatentTile / ps;
    step_slots = kLatentTile - step_pages * ps;
    raw = entry();
  }
  // Asked for by the planned length, which the table covers, so as not to wait for the
  // live one, and looked at no sooner than it is used.
  __device__ __forceinline__ int entry() const { return in && tok < planned ? __ldg(table + idx) : none; }
  __device__ __forceinline__ int page() const { return tok < kv ? raw : none; }
  __device__ __forceinline__ void next_tile() {
    tok += kLatentTile;
    idx += step_pages;
    slot += step_slots;
    if (slot >= ps) {
      slot -= ps;
      ++idx;
    }
    raw = entry();
  }
};

}  // namespace dev
}  // namespace pka
