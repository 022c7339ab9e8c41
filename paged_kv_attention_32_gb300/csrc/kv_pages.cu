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
// compaction are one cluster of 8 CTAs whose shared memories hold the pool's bits
// between them, a contiguous range of pages each, so that setting a bit is one write to
// another CTA's shared memory, ranks are scans of bit counts, and one launch does it all.
// Launch, table reads and the cluster barriers between the steps bound them.
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
template <int WARPS>
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* warp_sums, uint64_t& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t inc = warp_scan(x, lane);
  __syncthreads();   // an earlier scan's sums have been read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  uint64_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const uint64_t s = warp_sums[w];
    if (w < warp) before += s;
    all += s;
  }
  return before + inc - x;
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
  __shared__ uint64_t warp_sums[kForkThreads / 32];
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

constexpr int kCluster = 8, kThreads = 1024, kWarps = kThreads / 32;
constexpr int kPiece = 256;   // table entries a warp takes at a time

__device__ __forceinline__ void bit_set(uint32_t addr, uint32_t bit) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(bit) : "memory");
}
__device__ __forceinline__ uint32_t bit_test_set(uint32_t addr, uint32_t bit) {
  uint32_t old;
  asm volatile("atom.relaxed.cluster.shared::cluster.or.b32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(bit) : "memory");
  return old & bit;
}
__device__ __forceinline__ uint32_t load_remote(uint32_t addr) {
  uint32_t x;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
  return x;
}

// Every thread of the cluster, whole warps again after branches that lanes took apart.
__device__ __forceinline__ void sync_all() {
  __syncwarp();
  cluster_sync();
}

// The words of one bit per page: word w lies in CTA w >> shift of the cluster.
struct PageBits {
  int shift;
  __device__ __forceinline__ uint32_t addr(const uint32_t* mine, int page) const {
    const uint32_t w = (uint32_t)page >> 5;
    return map_to_rank(smem_u32(mine + (w & ((1u << shift) - 1u))), w >> shift);
  }
};

// The lowest `n` set bits of `x`.
__device__ __forceinline__ uint32_t lowest(uint32_t x, int64_t n) {
  if (n <= 0) return 0u;
  uint32_t left = x;
  for (; n > 0 && left != 0u; --n) left &= left - 1u;
  return x & ~left;
}

// What the CTAs of the cluster tell each other: a flag anybody may set, and their counts.
struct ClusterBoard {
  uint64_t counts[2][kCluster];
  int32_t flags;
  uint64_t warp_sums[kWarps];
};

// Each CTA's `mine` into slot `which` of everybody's board; to be read behind a cluster barrier.
__device__ __forceinline__ void publish(ClusterBoard& board, int which, uint32_t rank, uint64_t mine) {
  if (threadIdx.x < kCluster) {
    const uint32_t to = map_to_rank(smem_u32(&board.counts[which][rank]), threadIdx.x);
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(mine) : "memory");
  }
}
__device__ __forceinline__ void raise_flag(ClusterBoard& board, int32_t bits) {
#pragma unroll 1
  for (uint32_t r = 0; r < kCluster; ++r) bit_set(map_to_rank(smem_u32(&board.flags), r), (uint32_t)bits);
}

// Calls `f(row, column, entry)` for the first `entries_of(row)` table entries of every row, 8
// loads a lane at a time, spread over the cluster's warps.
template <typename Rows, typename F>
__device__ __forceinline__ void for_entries(const int32_t* tables, int64_t row_stride, int batch, int width,
                                            uint32_t rank, Rows&& entries_of, F&& f) {
  const int lane = threadIdx.x & 31, warp = (int)rank * kWarps + (threadIdx.x >> 5);
  const int pieces = (width + kPiece - 1) / kPiece;
  const int64_t items = (int64_t)batch * pieces;
  for (int64_t item = warp; item < items; item += kCluster * kWarps) {
    const int b = (int)(item / pieces), j0 = (int)(item % pieces) * kPiece;
    const int n = entries_of(b);
    if (j0 >= n) continue;
    int32_t x[kPiece / 32];
#pragma unroll
    for (int k = 0; k < kPiece / 32; ++k)
      if (j0 + 32 * k + lane < n) x[k] = tables[b * row_stride + j0 + 32 * k + lane];
#pragma unroll
    for (int k = 0; k < kPiece / 32; ++k)
      if (j0 + 32 * k + lane < n) f(b, j0 + 32 * k + lane, x[k]);
  }
}

// ---- release ------------------------------------------------------------------

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
kv_free_kernel(const __grid_constant__ ReleaseArgs a, int shift) {
  extern __shared__ uint32_t smem[];
  __shared__ ClusterBoard board;
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank();
  const int words = 1 << shift;
  uint32_t* gone = smem;            // pages of released rows
  uint32_t* kept = smem + words;    // of the others
  uint32_t* released = smem + 2 * words;   // a bit per row, every CTA for itself
  const int row_words = (a.batch + 31) / 32;
  const int head = __ldg(a.free_head);
  for (int w = tid; w < 2 * words + row_words; w += kThreads) smem[w] = 0u;
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
  sync_all();   // everybody's bits are zero, and the check is over
  const PageBits bits{shift};
  if (fits) {
    for_entries(a.tables, a.row_stride, a.batch, a.width, rank,
                [&](int b) { return pages_of(__ldg(a.kv_lens + b), a.page_size); },
                [&](int b, int, int page) {
                  if (page < 0 || page >= a.num_pages) raise_flag(board, STATUS_PAGE_BOUNDS);
                  else bit_set(bits.addr(released[b >> 5] >> (b & 31) & 1u ? gone : kept, page), 1u << (page & 31));
                });
  }
  sync_all();

  // the freed pages, in ascending order
  const int per_thread = (words + kThreads - 1) / kThreads, w0 = tid * per_thread;
  uint64_t mine = 0, all;
  for (int w = w0; w < min(w0 + per_thread, words); ++w) mine += __popc(gone[w] & ~kept[w]);
  const uint64_t before = block_scan<kWarps>(mine, board.warp_sums, all);
  publish(board, 0, rank, all);
  sync_all();
  int64_t freed = 0, at = 0;
  for (uint32_t r = 0; r < kCluster; ++r) {
    if (r < rank) at += (int64_t)board.counts[0][r];
    freed += (int64_t)board.counts[0][r];
  }
  flags = board.flags;
  if (flags == 0 && freed > head) flags = STATUS_CAPACITY;
  if (flags == 0) {
    int64_t to = head - freed + at + (int64_t)before;
    for (int w = w0; w < min(w0 + per_thread, words); ++w)
      for (uint32_t m = gone[w] & ~kept[w]; m != 0u; m &= m - 1u)
        a.free_pages[to++] = (((int)rank << shift) + w) * 32 + __ffs(m) - 1;
  }
  if (rank == 0 && tid == 0) {
    *a.free_head_out = flags == 0 ? (int32_t)(head - freed) : head;
    if (flags != 0 && a.status != nullptr) atomicOr(a.status, flags);
  }
  for (int b = (int)rank * kThreads + tid; b < a.batch; b += kCluster * kThreads)
    a.seq_lens[b] = flags == 0 && (released[b >> 5] >> (b & 31) & 1u) ? 0 : __ldg(a.kv_lens + b);
}

// ---- compaction -----------------------------------------------------------------

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
kv_compact_kernel(const __grid_constant__ CompactArgs a, int shift) {
  extern __shared__ uint32_t smem[];
  __shared__ ClusterBoard board;
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank();
  const int words = 1 << shift;
  uint32_t* used = smem;               // pages in the tables, then those of them that move
  uint32_t* open = smem + words;       // pages in the free list
  uint32_t* moved = smem + 2 * words;  // moving pages before each word
  const int head = __ldg(a.free_head);
  for (int w = tid; w < 2 * words; w += kThreads) smem[w] = 0u;
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
  sync_all();   // everybody's bits are zero, and the check is over
  const PageBits bits{shift};
  auto entries_of = [&](int b) { return pages_of(__ldg(a.kv_lens + b), a.page_size); };
  if (fits) {
    for_entries(a.tables, a.row_stride, a.batch, a.width, rank, entries_of, [&](int, int, int page) {
      if (page < 0 || page >= a.num_pages) raise_flag(board, STATUS_PAGE_BOUNDS);
      else bit_set(bits.addr(used, page), 1u << (page & 31));
    });
    for (int64_t i = head + (int64_t)rank * kThreads + tid; i < a.num_free; i += kCluster * kThreads) {
      const int page = a.free_pages[i];
      if (page < 0 || page >= a.num_pages) raise_flag(board, STATUS_PAGE_BOUNDS);
      else if (bit_test_set(bits.addr(open, page), 1u << (page & 31))) raise_flag(board, STATUS_FREE_LIST);
    }
  }
  sync_all();

  // U and U + F before each word
  const int per_thread = (words + kThreads - 1) / kThreads, w0 = tid * per_thread;
  const int w1 = min(w0 + per_thread, words);
  uint64_t mine = 0, all;
  for (int w = w0; w < w1; ++w) {
    if (used[w] & open[w]) raise_flag(board, STATUS_FREE_LIST);   // in use and free
    mine += (uint64_t)__popc(used[w]) << 32 | (uint64_t)__popc(used[w] | open[w]);
  }
  uint64_t before = block_scan<kWarps>(mine, board.warp_sums, all);
  publish(board, 0, rank, all);
  sync_all();
  uint64_t base = 0, sum = 0;
  for (uint32_t r = 0; r < kCluster; ++r) {
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
  publish(board, 1, rank, all);
  sync_all();
  base = sum = 0;
  for (uint32_t r = 0; r < kCluster; ++r) {
    if (r < rank) base += board.counts[1][r];
    sum += board.counts[1][r];
  }
  const int64_t moves = (int64_t)(sum >> 32);   // as many holes
  flags = board.flags;
  if (flags == 0 && moves > a.max_moves) flags = STATUS_CAPACITY;
  if (flags == 0) {
    int64_t m = (int64_t)((base + before) >> 32), h = (int64_t)((base + before) & 0xffffffffull);
    z = z0;
    for (int w = w0; w < w1; ++w) {
      const uint32_t both = used[w] | open[w], low = lowest(both, in_use - z);
      const int page0 = (((int)rank << shift) + w) * 32;
      uint32_t x = both & ~low;   // free afterwards
      for (int64_t to = head + z + __popc(low) - in_use; x != 0u; x &= x - 1u) a.free_pages_out[to++] = page0 + __ffs(x) - 1;
      for (x = open[w] & low; x != 0u; x &= x - 1u) a.dst_pages[h++] = page0 + __ffs(x) - 1;
      moved[w] = (uint32_t)m;
      x = used[w] & ~low;
      used[w] = x;
      for (; x != 0u; x &= x - 1u) a.src_pages[m++] = page0 + __ffs(x) - 1;
      z += __popc(both);
    }
  }
  const int me = (int)rank * kThreads + tid;
  if (me == 0) {
    *a.num_moves = flags == 0 ? (int32_t)moves : 0;
    if (flags != 0 && a.status != nullptr) atomicOr(a.status, flags);
  }
  for (int64_t i = (flags == 0 ? moves : 0) + me; i < a.max_moves; i += kCluster * kThreads)
    a.src_pages[i] = a.dst_pages[i] = -1;
  if (a.free_pages_out != a.free_pages)   // what lies before the list's head, or all of it
    for (int64_t i = me; i < (flags == 0 ? head : a.num_free); i += kCluster * kThreads)
      a.free_pages_out[i] = a.free_pages[i];
  sync_all();   // the moves are written, in global memory and in everybody's bits

  const bool in_place = a.tables_out == a.tables;
  if (flags != 0 && in_place) return;
  for_entries(a.tables, a.row_stride, a.batch, a.width, rank, [&](int) { return a.width; },
              [&](int b, int j, int page) {
                int to = page;
                if (flags == 0 && j < entries_of(b)) {
                  const uint32_t word = load_remote(bits.addr(used, page)), bit = 1u << (page & 31);
                  if (word & bit) to = __ldcg(a.dst_pages + load_remote(bits.addr(moved, page)) + __popc(word & (bit - 1u)));
                }
                if (!in_place || to != page) a.tables_out[b * a.out_row_stride + j] = to;
              });
  sync_all();   // nobody's bits go while others read them
}

// log2 of the words a CTA holds of `num_pages` bits.
int word_shift(int32_t num_pages) {
  const int64_t words = ceil_div(ceil_div(num_pages, 32), kCluster);
  int shift = 0;
  while ((int64_t(1) << shift) < words) ++shift;
  return shift;
}

constexpr int kMaxWords = (int)(kPageOpPages / 32 / kCluster);

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

int launch_kv_free(const ReleaseArgs& a, cudaStream_t stream) {
  const int shift = word_shift(a.num_pages);
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = set_smem_once(kv_free_kernel, kMaxWords * 8 + kPageOpRows / 8, smem_set);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(kv_free)");
  const size_t smem = ((size_t)2 << shift) * 4 + (size_t)((a.batch + 31) / 32) * 4;
  kv_free_kernel<<<kCluster, kThreads, smem, stream>>>(a, shift);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv_free_kernel launch");
  return PKA_OK;
}

int launch_kv_compact(const CompactArgs& a, cudaStream_t stream) {
  const int shift = word_shift(a.num_pages);
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = set_smem_once(kv_compact_kernel, kMaxWords * 12, smem_set);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(kv_compact)");
  kv_compact_kernel<<<kCluster, kThreads, ((size_t)3 << shift) * 4, stream>>>(a, shift);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv_compact_kernel launch");
  return PKA_OK;
}

}  // namespace pka
