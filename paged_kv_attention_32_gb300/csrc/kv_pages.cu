// Requests forked over a page pool's tables, released from them, and the pool compacted.
//
// No page carries a count of its holders: the tables say who holds what.
//   fork     a child's row takes its parent's full pages as they are and, where the parent's
//            last page is not full, a fresh page, whose contents the caller copies;
//   release  a page goes back to the free list when a released row holds it and no other
//            row does, found by one bit per page and kind of row;
//   compact  with U the pages in the tables and F those in the free list, the lowest |U|
//            pages of U + F take the pages in use: the i-th page of U above them goes to
//            the i-th page of F among them.
//
// A fork needs no wait between CTAs: each checks all forks and counts the fresh pages
// before its own itself, as they read only what none of them writes.  Release and
// compaction are one CTA, or for large tables a cluster of 16, that mark pages each in a copy
// of its own of the pool's bits, join the copies by slices over their shared memories, and rank pages by
// scans of bit counts: one launch does it all.  Latency bounds them: a launch, two waits for
// memory in turn (lengths, then entries) and the cluster barriers between the steps; for
// large tables the entries that 16 SMs' registers hold on their way.  Fork of 448 rows 7 us;
// release from 64 rows 6.4 us from start to end, from 2048 rows, 530000 entries, 20 us, of which
// 5 go to the marks, 5 to joining them; compaction of 256 rows 20 us.  Beyond that time goes with
// the entries on 16 SMs, and with the ranges of the pool, each of which reads the tables again:
// release from 16384 rows of 512 entries 74 us in a pool of 2^19 pages, 603 in one of 2^22 (seven
// ranges), compaction 164 and 1625; from 2048 rows in a pool of 2^22 pages 224 and 883.
#include <algorithm>

#include "device_common.cuh"
#include "host_common.h"
#include "pages.h"

namespace pka {

using namespace dev;

namespace {

constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ uint64_t warp_scan(uint64_t x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(FULL, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// Exclusive prefix of `x` over the block's WARPS * 32 threads, and the sum of all.
// sums: [WARPS + 1] in shared memory.
template <int WARPS>
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* sums, uint64_t& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t inc = warp_scan(x, lane);
  __syncthreads();   // an earlier scan's sums have been read
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const uint64_t s = lane < WARPS ? sums[lane] : 0, t = warp_scan(s, lane);
    if (lane < WARPS) sums[lane] = t - s;
    if (lane == 31) sums[WARPS] = t;
  }
  __syncthreads();
  all = sums[WARPS];
  return sums[warp] + inc - x;
}

__device__ __forceinline__ int pages_of(int len, int ps) {
  return (int)(((uint32_t)len + (uint32_t)ps - 1u) / (uint32_t)ps);
}

// ---- fork -------------------------------------------------------------------

constexpr int kForkThreads = 512;
constexpr int kForkPiece = 256;   // table entries a warp copies at a time

__global__ void __launch_bounds__(kForkThreads) kv_fork_kernel(const __grid_constant__ ForkArgs a) {
  extern __shared__ uint32_t smem[];
  const int n = a.num_forks, words = (a.batch + 31) / 32;
  uint32_t* pair = smem;                                       // [n] parent | child << 16
  int32_t* len = reinterpret_cast<int32_t*>(smem + n);         // [n] the parent's length
  uint32_t* fresh = smem + 2 * n;                              // [n] fresh pages taken before
  uint32_t* is_parent = smem + 3 * n;                          // a bit per row
  uint32_t* is_child = is_parent + words;
  __shared__ uint64_t warp_sums[kForkThreads / 32 + 1];
  __shared__ int s_bad, s_full;
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t head = __ldg(a.free_head);
  if (tid == 0) s_bad = s_full = 0;
  for (int w = tid; w < 2 * words; w += kForkThreads) is_parent[w] = 0u;
  __syncthreads();

  uint64_t taken = 0;   // by the forks of earlier rounds
  for (int i0 = 0; i0 < n; i0 += kForkThreads) {
    const int i = i0 + tid;
    uint64_t need = 0;
    if (i < n) {
      const int p = __ldg(a.parents + i), c = __ldg(a.children + i);
      int l = 0;
      if (p < 0 || p >= a.batch || c < 0 || c >= a.batch) {
        s_bad = 1;
        pair[i] = 0u;
      } else {
        pair[i] = (uint32_t)p | (uint32_t)c << 16;
        atomicOr(is_parent + (p >> 5), 1u << (p & 31));
        if (atomicOr(is_child + (c >> 5), 1u << (c & 31)) >> (c & 31) & 1u) s_bad = 1;
        l = __ldg(a.kv_lens + p);
        if (l < 0 || l > (int64_t)a.width * a.page_size) {
          s_full = 1;
          l = 0;
        }
        need = l % a.page_size != 0;
      }
      len[i] = l;
    }
    uint64_t all;
    const uint64_t before = block_scan<kForkThreads / 32>(need, warp_sums, all);
    if (i < n) fresh[i] = (uint32_t)(taken + before);
    taken += all;
  }
  __syncthreads();
  for (int w = tid; w < words; w += kForkThreads)
    if (is_parent[w] & is_child[w]) s_bad = 1;
  if (tid == 0 && (head < 0 || head + (int64_t)taken > a.num_free)) s_full = 1;
  __syncthreads();
  const bool bad = s_bad || s_full;

  const int64_t me = (int64_t)blockIdx.x * kForkThreads + tid, all = (int64_t)gridDim.x * kForkThreads;
  if (me == 0) {
    *a.free_head_out = (int32_t)(bad ? head : head + (int64_t)taken);
    if (bad && a.status != nullptr)
      atomicOr(a.status, (s_bad ? STATUS_ROWS : 0) | (s_full ? STATUS_CAPACITY : 0));
  }
  for (int64_t b = me; b < a.batch; b += all)
    if (bad || !(is_child[b >> 5] >> (b & 31) & 1u)) a.seq_lens[b] = __ldg(a.kv_lens + b);
  for (int64_t i = me; i < n; i += all) {
    int src = -1, dst = -1;
    if (!bad) {
      const int p = (int)(pair[i] & 0xffffu), c = (int)(pair[i] >> 16), l = len[i];
      a.seq_lens[c] = l;
      if (l % a.page_size != 0) {
        const int full = l / a.page_size;
        src = a.tables[p * a.row_stride + full];
        dst = __ldg(a.free_pages + head + fresh[i]);
        a.tables[c * a.row_stride + full] = dst;
      }
    }
    a.src_pages[i] = src;
    a.dst_pages[i] = dst;
  }
  if (bad) return;
  const int pieces = (a.width + kForkPiece - 1) / kForkPiece;
  const int64_t items = (int64_t)n * pieces;
  for (int64_t item = me >> 5; item < items; item += all >> 5) {
    const int i = (int)(item / pieces), j0 = (int)(item % pieces) * kForkPiece;
    const int full = len[i] / a.page_size;
    const int32_t* from = a.tables + (int64_t)(pair[i] & 0xffffu) * a.row_stride;
    int32_t* to = a.tables + (int64_t)(pair[i] >> 16) * a.row_stride;
    int32_t x[kForkPiece / 32];
#pragma unroll
    for (int k = 0; k < kForkPiece / 32; ++k)
      if (j0 + 32 * k + lane < full) x[k] = from[j0 + 32 * k + lane];
#pragma unroll
    for (int k = 0; k < kForkPiece / 32; ++k)
      if (j0 + 32 * k + lane < full) to[j0 + 32 * k + lane] = x[k];
  }
}

// ---- bits of a pool over the shared memories of a cluster ----------------------

constexpr int kMaxCluster = 16, kThreads = 1024, kWarps = kThreads / 32;
// Table entries up to which one CTA does without the others, whose barriers and joined bits
// then cost more than its share of the reads.  One CTA and 16: release from 16384 entries 10.3
// and 12.4 us, from 24576 11.9 and 12.4, from 32768 14.0 and 12.4; compaction, with the copies, of
// 2016 15.8 and 21.9, of 8032 24.7 and 26.7, of 12048 36.8 and 32.0.
constexpr int64_t kFewToFree = 24576, kFewToCompact = 8192;
constexpr int kDynamicSmem = 222 * 1024;

__device__ __forceinline__ void flag_set(uint32_t addr, uint32_t bits) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(bits) : "memory");
}
__device__ __forceinline__ uint4 load_remote4(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(addr)
               : "memory");
  return x;
}

// Every thread of the NC CTAs, whole warps again after branches that lanes took apart.
template <int NC>
__device__ __forceinline__ void sync_all() {
  __syncwarp();
  if constexpr (NC > 1) cluster_sync();
  else __syncthreads();
}

// The lowest `n` set bits of `x`.
__device__ __forceinline__ uint32_t lowest(uint32_t x, int64_t n) {
  if (n <= 0) return 0u;
  if (n >= __popc(x)) return x;
  uint32_t left = x;
  for (; n > 0 && left != 0u; --n) left &= left - 1u;
  return x & ~left;
}

// What the CTAs of the cluster tell each other: a flag anybody may set, and their counts.
struct ClusterBoard {
  uint64_t counts[2][kMaxCluster];
  int32_t flags;
  uint64_t warp_sums[kWarps + 1];
};

// Each CTA's `mine` into slot `which` of everybody's board; to be read behind a cluster barrier.
template <int NC>
__device__ __forceinline__ void publish(ClusterBoard& board, int which, uint32_t rank, uint64_t mine) {
  if (threadIdx.x < NC) {
    const uint32_t to = map_to_rank(smem_u32(&board.counts[which][rank]), threadIdx.x);
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(mine) : "memory");
  }
}
template <int NC>
__device__ __forceinline__ void raise_flag(ClusterBoard& board, int32_t bits) {
#pragma unroll 1
  for (uint32_t r = 0; r < NC; ++r) flag_set(map_to_rank(smem_u32(&board.flags), r), (uint32_t)bits);
}

// Calls `f(row, tag, column, entry)` for the first n table entries of every row, (n, tag) =
// `row_of(row)`, and returns what any of a thread's calls did: pieces of a row to the warps of
// the NC CTAs in turn, AT_ONCE of them in 16 loads a lane.  A warp asks for the lengths of its
// next 32 pieces at once and passes over those that are empty (each length asked for while the
// piece before is under way: a release from 2048 rows 33.8 us instead of 32.8).  Two pieces of
// 256 entries at once keep more loads on their way where rows end anywhere (the same release 24.8
// us, one piece of 512 29.1, four of 128 25.9); one of 512 is faster where whole rows fit (a
// release from 64 rows of 257 9.7 and 10.4, compaction of 256 rows by 2 us).
struct RowPart {
  int n, tag;
};
template <int NC, int AT_ONCE, typename Rows, typename F>
__device__ __forceinline__ int for_entries(const int32_t* tables, int64_t row_stride, int batch, int width,
                                            uint32_t rank, Rows&& row_of, F&& f) {
  constexpr int kWarpsAll = NC * kWarps, kPiece = 512 / AT_ONCE;
  const int lane = threadIdx.x & 31;
  const int pieces = (width + kPiece - 1) / kPiece;
  const int64_t items = (int64_t)batch * pieces;
  int flags = 0;
  for (int64_t item = (int64_t)(threadIdx.x >> 5) * NC + rank; item < items; item += 32 * kWarpsAll) {
    const int64_t mine = item + (int64_t)lane * kWarpsAll;   // this lane's piece
    int b_of = 0, j_of = 0;
    RowPart row{0, 0};
    if (mine < items) {
      b_of = (int)(mine / pieces);
      j_of = (int)(mine % pieces) * kPiece;
      row = row_of(b_of);
    }
    for (uint32_t todo = __ballot_sync(FULL, j_of < row.n); todo != 0u;) {
      int b[AT_ONCE], n[AT_ONCE], tag[AT_ONCE], j0[AT_ONCE], x[AT_ONCE][kPiece / 32];
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {   // none left: no entries
        const int from_lane = todo != 0u ? __ffs(todo) - 1 : 0;
        b[i] = __shfl_sync(FULL, b_of, from_lane);
        n[i] = todo != 0u ? __shfl_sync(FULL, row.n, from_lane) : 0;
        tag[i] = __shfl_sync(FULL, row.tag, from_lane);
        j0[i] = __shfl_sync(FULL, j_of, from_lane) + lane;
        todo &= todo - 1u;
        const int32_t* from = tables + b[i] * row_stride;
#pragma unroll
        for (int k = 0; k < kPiece / 32; ++k)
          if (j0[i] + 32 * k < n[i]) x[i][k] = from[j0[i] + 32 * k];
      }
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
        for (int k = 0; k < kPiece / 32; ++k)
          if (j0[i] + 32 * k < n[i]) flags |= f(b[i], tag[i], j0[i] + 32 * k, x[i][k]);
    }
  }
  return flags;
}

// Two bits per page, held twice: marks of a CTA's own over a range of the pool, set by ordinary
// shared-memory atomics (one to another CTA's shared memory takes some 4 cycles a lane: 2048
// rows of 270000 pages 181 us), and slices, a contiguous part of the pool per CTA, into which
// the marks of all CTAs are joined.  A pool of more pages than the marks hold takes several
// ranges, with the tables read once for each.  One CTA alone marks in its slice.
struct PageBits {
  uint32_t* slice[2];   // [per] words of this CTA's, one behind the other
  uint32_t* mark[2];    // [range] words, one behind the other
  uint32_t* spare[2];   // [per] words, or more; the marks are lost
  int per, words, range;   // per and range are whole vectors of four
};
template <int NC>
__device__ __forceinline__ PageBits page_bits(uint32_t* smem, int num_pages) {
  PageBits p;
  p.words = (num_pages + 31) / 32;
  p.per = ((p.words + NC - 1) / NC + 3) & ~3;
  p.slice[0] = smem;
  p.slice[1] = smem + p.per;
  p.range = NC == 1 ? p.per : min((kDynamicSmem / 4 - 2 * p.per) / 2 & ~3, (p.words + 3) & ~3);
  p.spare[0] = smem + 2 * p.per;
  p.spare[1] = p.spare[0] + p.range;
  p.mark[0] = NC == 1 ? p.slice[0] : p.spare[0];
  p.mark[1] = p.mark[0] + p.range;
  return p;
}
// Clears the marks; the CTA's threads are to meet before any is set.
__device__ __forceinline__ void clear_marks(const PageBits& p) {
  uint4* m = reinterpret_cast<uint4*>(p.mark[0]);
  for (int i = threadIdx.x; i < p.range / 2; i += kThreads) m[i] = make_uint4(0u, 0u, 0u, 0u);
}
// Joins everybody's marks of the words from `first` on into the slices, the CTAs beginning at
// different ones (all at the first: a release from 2048 rows 32.8 us instead of 30.7).  TWICE:
// bits of the second kind that two CTAs have are reported.
template <int NC, bool TWICE>
__device__ __forceinline__ bool join_marks(const PageBits& p, int first, uint32_t rank) {
  const int mine = (int)rank * p.per, w0 = max(mine, first), w1 = min(min(mine + p.per, first + p.range), p.words);
  bool twice = false;
  for (int i = threadIdx.x; i < (w1 - w0 + 3) / 4 * 2; i += kThreads) {
    const int kind = i & 1, w = w0 + (i >> 1) * 4;
    const uint32_t at = smem_u32(p.mark[0] + kind * p.range + (w - first));
    uint4 x[NC];
#pragma unroll
    for (int r = 0; r < NC; ++r) x[r] = load_remote4(map_to_rank(at, (rank + (uint32_t)r) % NC));
    uint4 any = make_uint4(0u, 0u, 0u, 0u);
    uint32_t again = 0u;
#pragma unroll
    for (int r = 0; r < NC; ++r) {
      if (TWICE) again |= (any.x & x[r].x) | (any.y & x[r].y) | (any.z & x[r].z) | (any.w & x[r].w);
      any.x |= x[r].x;
      any.y |= x[r].y;
      any.z |= x[r].z;
      any.w |= x[r].w;
    }
    if (TWICE && kind == 1 && again != 0u) twice = true;
    *reinterpret_cast<uint4*>(p.slice[0] + kind * p.per + (w - mine)) = any;
  }
  return twice;
}

// Writes the ids of the pages in `bits` to list[before of the word ..): a word a warp, a bit a
// lane.  bits and before [words] in shared memory, word w's bit 0 is page 32 (word0 + w).
__device__ __forceinline__ void write_pages(int32_t* list, const uint32_t* bits, const uint32_t* before, int words,
                                            int word0) {
  const int lane = threadIdx.x & 31;
  for (int w = threadIdx.x >> 5; w < words; w += kWarps) {
    const uint32_t x = bits[w];
    if (x >> lane & 1u) list[before[w] + __popc(x & ((1u << lane) - 1u))] = (word0 + w) * 32 + lane;
  }
}

// ---- release ------------------------------------------------------------------

template <int NC>
__global__ void __launch_bounds__(kThreads, 1) kv_free_kernel(const __grid_constant__ ReleaseArgs a) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ ClusterBoard board;
  __shared__ uint32_t released[kPageOpRows / 32];   // a bit per row, every CTA for itself
  const int tid = threadIdx.x;
  const uint32_t rank = NC > 1 ? cluster_rank() : 0u;
  const PageBits bits = page_bits<NC>(smem, a.num_pages);
  const int word0 = (int)rank * bits.per;   // the slice's first word
  const int head = __ldg(a.free_head);
  for (int w = tid; w < (a.batch + 31) / 32; w += kThreads) released[w] = 0u;
  if (NC > 1)
    for (int w = tid; w < 2 * bits.per; w += kThreads) smem[w] = 0u;
  clear_marks(bits);
  if (tid == 0) board.flags = 0;
  __syncthreads();
  int flags = 0;
  for (int i = tid; i < a.num_rows; i += kThreads) {
    const int b = __ldg(a.rows + i);
    if (b < 0 || b >= a.batch || (atomicOr(released + (b >> 5), 1u << (b & 31)) >> (b & 31) & 1u)) flags |= STATUS_ROWS;
  }
  for (int b = tid; b < a.batch; b += kThreads) {
    const int l = __ldg(a.kv_lens + b);
    if (l < 0 || l > (int64_t)a.width * a.page_size) flags |= STATUS_CAPACITY;
  }
  if (head < 0 || head > a.num_free) flags |= STATUS_CAPACITY;
  if (flags != 0) atomicOr(&board.flags, flags);   // each CTA finds the same
  __syncthreads();
  const bool fits = board.flags == 0;
  sync_all<NC>();   // the check is over: flags may come from other CTAs
  for (int first = 0; fits && first < bits.words; first += bits.range) {
    if (first > 0) {
      clear_marks(bits);
      __syncthreads();
    }
    const int found = for_entries<NC, NC == 1 ? 1 : 2>(
        a.tables, a.row_stride, a.batch, a.width, rank,
        [&](int b) {
          return RowPart{pages_of(__ldg(a.kv_lens + b), a.page_size),
                         (released[b >> 5] >> (b & 31) & 1u) ? bits.range : 0};   // which marks
        },
        [&](int, int tag, int, int page) -> int {
          const int w = (page >> 5) - first;
          if ((uint32_t)page >= (uint32_t)a.num_pages) return STATUS_PAGE_BOUNDS;
          if ((uint32_t)w < (uint32_t)bits.range) atomicOr(bits.mark[0] + tag + w, 1u << (page & 31));
          return 0;
        });
    if (found != 0) raise_flag<NC>(board, found);
    sync_all<NC>();
    if constexpr (NC > 1) {
      join_marks<NC, false>(bits, first, rank);
      sync_all<NC>();
    }
  }

  // the freed pages, in ascending order
  const int words = bits.per, per_thread = (words + kThreads - 1) / kThreads, w0 = tid * per_thread;
  uint32_t *kept = bits.slice[0], *gone = bits.slice[1];
  uint64_t mine = 0, all;
  for (int w = w0; w < min(w0 + per_thread, words); ++w) mine += __popc(gone[w] & ~kept[w]);
  const uint64_t before = block_scan<kWarps>(mine, board.warp_sums, all);
  publish<NC>(board, 0, rank, all);
  sync_all<NC>();
  int64_t freed = 0, at = 0;
  for (uint32_t r = 0; r < NC; ++r) {
    if (r < rank) at += (int64_t)board.counts[0][r];
    freed += (int64_t)board.counts[0][r];
  }
  flags = board.flags;
  if (flags == 0 && freed > head) flags = STATUS_CAPACITY;
  if (flags == 0) {
    uint32_t n = (uint32_t)before;
    for (int w = w0; w < min(w0 + per_thread, words); ++w) {
      const uint32_t m = gone[w] & ~kept[w];
      gone[w] = m;
      kept[w] = n;
      n += __popc(m);
    }
    __syncthreads();
    write_pages(a.free_pages + (head - freed + at), gone, kept, words, word0);
  }
  if (rank == 0 && tid == 0) {
    *a.free_head_out = flags == 0 ? (int32_t)(head - freed) : head;
    if (flags != 0 && a.status != nullptr) atomicOr(a.status, flags);
  }
  for (int b = (int)rank * kThreads + tid; b < a.batch; b += NC * kThreads)
    a.seq_lens[b] = flags == 0 && (released[b >> 5] >> (b & 31) & 1u) ? 0 : __ldg(a.kv_lens + b);
}

// ---- compaction -----------------------------------------------------------------

constexpr uint32_t kAbove = 0x80000000u;

template <int NC>
__global__ void __launch_bounds__(kThreads, 1) kv_compact_kernel(const __grid_constant__ CompactArgs a) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ ClusterBoard board;
  const int tid = threadIdx.x;
  const uint32_t rank = NC > 1 ? cluster_rank() : 0u;
  const PageBits bits = page_bits<NC>(smem, a.num_pages);
  const int word0 = (int)rank * bits.per;   // the slice's first word
  uint32_t* used = bits.slice[0];    // pages in the tables, then those of them that move
  uint32_t* open = bits.slice[1];    // pages in the free list, then the moving pages before each word
  const int head = __ldg(a.free_head);
  if (NC > 1)
    for (int w = tid; w < 2 * bits.per; w += kThreads) smem[w] = 0u;
  clear_marks(bits);
  if (tid == 0) board.flags = 0;
  __syncthreads();
  int flags = 0;
  for (int b = tid; b < a.batch; b += kThreads) {
    const int l = __ldg(a.kv_lens + b);
    if (l < 0 || l > (int64_t)a.width * a.page_size) flags |= STATUS_CAPACITY;
  }
  if (head < 0 || head > a.num_free) flags |= STATUS_CAPACITY;
  if (flags != 0) atomicOr(&board.flags, flags);   // each CTA finds the same
  __syncthreads();
  const bool fits = board.flags == 0;
  sync_all<NC>();   // the check is over: flags may come from other CTAs
  auto entries_of = [&](int b) { return RowPart{pages_of(__ldg(a.kv_lens + b), a.page_size), 0}; };
  // what lies before the list's head stays: each thread's first entry is asked for early
  const int me = (int)rank * kThreads + tid;
  const bool other_list = a.free_pages_out != a.free_pages;
  const int32_t before_head = other_list && fits && me < head ? a.free_pages[me] : 0;
  for (int first = 0; fits && first < bits.words; first += bits.range) {
    if (first > 0) {
      clear_marks(bits);
      __syncthreads();
    }
    int found = for_entries<NC, 1>(a.tables, a.row_stride, a.batch, a.width, rank, entries_of, [&](int, int, int, int page) -> int {
      const int w = (page >> 5) - first;
      if ((uint32_t)page >= (uint32_t)a.num_pages) return STATUS_PAGE_BOUNDS;
      if ((uint32_t)w < (uint32_t)bits.range) atomicOr(bits.mark[0] + w, 1u << (page & 31));
      return 0;
    });
    for (int64_t i = head + (int64_t)rank * kThreads + tid; i < a.num_free; i += NC * kThreads) {
      const int page = a.free_pages[i], w = (page >> 5) - first;
      if (page < 0 || page >= a.num_pages) found |= STATUS_PAGE_BOUNDS;
      else if (w >= 0 && w < bits.range && (atomicOr(bits.mark[1] + w, 1u << (page & 31)) >> (page & 31) & 1u))
        found |= STATUS_FREE_LIST;
    }
    if (found != 0) raise_flag<NC>(board, found);
    sync_all<NC>();
    if constexpr (NC > 1) {
      if (join_marks<NC, true>(bits, first, rank)) raise_flag<NC>(board, STATUS_FREE_LIST);
      sync_all<NC>();
    }
  }

  // U and U + F before each word
  const int words = bits.per, per_thread = (words + kThreads - 1) / kThreads, w0 = tid * per_thread;
  const int w1 = min(w0 + per_thread, words);
  uint64_t mine = 0, all;
  for (int w = w0; w < w1; ++w) {
    if (used[w] & open[w]) raise_flag<NC>(board, STATUS_FREE_LIST);   // in use and free
    mine += (uint64_t)__popc(used[w]) << 32 | (uint64_t)__popc(used[w] | open[w]);
  }
  uint64_t before = block_scan<kWarps>(mine, board.warp_sums, all);
  publish<NC>(board, 0, rank, all);
  sync_all<NC>();
  uint64_t base = 0, sum = 0;
  for (uint32_t r = 0; r < NC; ++r) {
    if (r < rank) base += board.counts[0][r];
    sum += board.counts[0][r];
  }
  const int64_t in_use = (int64_t)(sum >> 32);
  const int64_t z0 = (int64_t)((base + before) & 0xffffffffull);   // pages of U + F before this thread's

  // pages that move and where they may go
  mine = 0;
  int64_t z = z0;
  for (int w = w0; w < w1; ++w) {
    const uint32_t both = used[w] | open[w], low = lowest(both, in_use - z);
    z += __popc(both);
    mine += (uint64_t)__popc(used[w] & ~low) << 32 | (uint64_t)__popc(open[w] & low);
  }
  before = block_scan<kWarps>(mine, board.warp_sums, all);
  publish<NC>(board, 1, rank, all);
  sync_all<NC>();
  base = sum = 0;
  for (uint32_t r = 0; r < NC; ++r) {
    if (r < rank) base += board.counts[1][r];
    sum += board.counts[1][r];
  }
  const int64_t moves = (int64_t)(sum >> 32);   // as many holes
  flags = board.flags;
  if (flags == 0 && moves > a.max_moves) flags = STATUS_CAPACITY;
  if (flags == 0) {
    // Below the word where the pages in use end every free page is a hole and none moves, above
    // it all in use move and all pages are free afterwards: one list for holes and free pages.
    uint32_t m = (uint32_t)((base + before) >> 32), h = (uint32_t)(base + before);
    uint32_t *list = bits.spare[0], *at = bits.spare[1];
    z = z0;
    for (int w = w0; w < w1; ++w) {
      const uint32_t both = used[w] | open[w], low = lowest(both, in_use - z);
      const uint32_t hole = open[w] & low, move = used[w] & ~low;
      const bool above = z >= in_use;
      list[w] = above ? both : hole;
      at[w] = above ? (uint32_t)(z - in_use) | kAbove : h;
      if (!above)   // the rest of the one word that holds the end
        for (uint32_t x = both & ~low, i = 0; x != 0u; x &= x - 1u, ++i)
          a.free_pages_out[head + i] = (word0 + w) * 32 + __ffs(x) - 1;
      open[w] = m;
      used[w] = move;
      h += __popc(hole);
      m += __popc(move);
      z += __popc(both);
    }
    __syncthreads();
    write_pages(a.src_pages, used, open, words, word0);
    for (int w = tid >> 5, lane = tid & 31; w < words; w += kWarps) {
      const uint32_t x = list[w], n = at[w];
      if (x >> lane & 1u)
        (n & kAbove ? a.free_pages_out + head : a.dst_pages)[(n & ~kAbove) + __popc(x & ((1u << lane) - 1u))] =
            (word0 + w) * 32 + lane;
    }
  }
  if (me == 0) {
    *a.num_moves = flags == 0 ? (int32_t)moves : 0;
    if (flags != 0 && a.status != nullptr) atomicOr(a.status, flags);
  }
  for (int64_t i = (flags == 0 ? moves : 0) + me; i < a.max_moves; i += NC * kThreads)
    a.src_pages[i] = a.dst_pages[i] = -1;
  if (other_list) {   // before the head, or where the call is refused all of it
    if (fits && me < head) a.free_pages_out[me] = before_head;
    for (int64_t i = fits && me < head ? me + NC * kThreads : me; i < (flags == 0 ? head : a.num_free); i += NC * kThreads)
      a.free_pages_out[i] = a.free_pages[i];
  }
  sync_all<NC>();   // the moves are written, in global memory and in everybody's slices

  // the tables, each CTA with its own copy of a range of the slices
  const bool in_place = a.tables_out == a.tables;
  if (flags == 0 || !in_place) {
    for (int first = 0; first < bits.words; first += bits.range) {
      if (NC > 1 && first > 0) __syncthreads();   // the range before is done with
      const int vectors = bits.range / 2, start = (int)((int64_t)vectors * rank / NC);   // as in join_marks
      for (int n = tid; NC > 1 && flags == 0 && n < vectors; n += kThreads) {
        const int i = n + start < vectors ? n + start : n + start - vectors;
        const int kind = i & 1, w = first + (i >> 1) * 4;
        if (w < bits.words) {
          const int owner = w / words;
          *reinterpret_cast<uint4*>(bits.mark[0] + kind * bits.range + (w - first)) =
              load_remote4(map_to_rank(smem_u32(bits.slice[0] + kind * bits.per + (w - owner * words)), (uint32_t)owner));
        }
      }
      if (NC > 1) __syncthreads();
      for_entries<NC, 1>(a.tables, a.row_stride, a.batch, a.width, rank, [&](int b) { return RowPart{a.width, flags == 0 ? entries_of(b).n : 0}; },
                  [&](int b, int tag, int j, int page) -> int {
                    const bool live = j < tag;
                    const int w = live ? (page >> 5) - first : 0;
                    if (live ? w < 0 || w >= bits.range : first > 0) return 0;   // another range's
                    int to = page;
                    if (live) {
                      const uint32_t word = bits.mark[0][w], bit = 1u << (page & 31);
                      if (word & bit) to = __ldcg(a.dst_pages + bits.mark[1][w] + __popc(word & (bit - 1u)));
                    }
                    if (!in_place || to != page) a.tables_out[b * a.out_row_stride + j] = to;
                    return 0;
                  });
    }
  }
  sync_all<NC>();   // nobody's slices go while others read them
}

static_assert(kPageOpPages / 32 / kMaxCluster * 8 <= kDynamicSmem / 2, "slices of the largest pool leave room for marks");
// One CTA holds a pool's bits twice over up to here.
constexpr int64_t kFewPages = (int64_t)kDynamicSmem / 16 * 32 - 4096;

}  // namespace

int launch_kv_fork(const ForkArgs& a, cudaStream_t stream) {
  const int words = (a.batch + 31) / 32;
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = set_smem_once(kv_fork_kernel, kPageOpRows * 12 + kPageOpRows / 32 * 8, smem_set);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(kv_fork)");
  const int64_t warps = (int64_t)a.num_forks * ceil_div(a.width, kForkPiece);
  const int64_t work = std::max<int64_t>(warps * 32, a.batch);
  const int grid = (int)std::min<int64_t>(ceil_div(work, kForkThreads), 152);
  kv_fork_kernel<<<grid, kForkThreads, (size_t)a.num_forks * 12 + (size_t)words * 8, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv_fork_kernel launch");
  return PKA_OK;
}

// Launches NC CTAs, as a cluster where they are several (16 are more than is portable: asked
// for once per kernel and device).
template <int NC, typename Kernel, typename Args>
static int launch_cluster(Kernel kern, const Args& a, std::atomic<uint64_t>& done, const char* what,
                          cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (e == cudaSuccess && !(bit != 0 && (done.load(std::memory_order_acquire) & bit))) {
    if (NC > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynamicSmem);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  }
  if (e != cudaSuccess) return cuda_fail(e, what);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(NC);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kDynamicSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = NC;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = NC > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess) return cuda_fail(e, what);
  return PKA_OK;
}

static bool few(int32_t batch, int32_t width, int64_t entries, int32_t num_pages) {
  return (int64_t)batch * width <= entries && num_pages <= kFewPages;
}

int launch_kv_free(const ReleaseArgs& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done[2];
  if (few(a.batch, a.width, kFewToFree, a.num_pages))
    return launch_cluster<1>(kv_free_kernel<1>, a, done[0], "kv_free_kernel launch", stream);
  return launch_cluster<kMaxCluster>(kv_free_kernel<kMaxCluster>, a, done[1], "kv_free_kernel launch", stream);
}

int launch_kv_compact(const CompactArgs& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done[2];
  if (few(a.batch, a.width, kFewToCompact, a.num_pages))
    return launch_cluster<1>(kv_compact_kernel<1>, a, done[0], "kv_compact_kernel launch", stream);
  return launch_cluster<kMaxCluster>(kv_compact_kernel<kMaxCluster>, a, done[1], "kv_compact_kernel launch", stream);
}

}  // namespace pka
