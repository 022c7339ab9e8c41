// Block tables and slot maps of a step, built from request lengths.
//
// With have_b = ceil(kv_b / ps), need_b = ceil((kv_b + new_b) / ps) and
// exclusive prefix sums start (of new) and base (of need - have):
//   table[b, j]  = free[head + base_b + j - have_b],  have_b <= j < need_b
//   slot_map[t]  = table[b, pos / ps] * ps + pos % ps, pos = kv_b + t - start_b
// Every CTA scans the lengths itself (8 bytes a request, from L2 after the
// first CTA) and keeps them and both prefix sums in shared memory, so one launch
// without any wait between CTAs does the whole step, with one dependent load
// (a table entry or a free page) behind the first ones; tokens and pages are
// then spread over all threads, each finding its request by binary search, so
// one long request costs no more than many short ones.  A launch and those dependent
// loads bound it: 64 requests 4.0 us, 1024 requests and 65536 slots 6.1 us (0.08 us of
// bytes).
#include <algorithm>

#include "device_common.cuh"
#include "host_common.h"
#include "latent.h"

namespace pka {

namespace {

constexpr int kThreads = 512;
constexpr int kMaxBatch = 16384;   // three 32-bit values each in 192 KB of shared memory

// The last index b in [0, n) with start[b] <= x (start[0] = 0): requests that
// add nothing share their start with their successor and are passed over.
__device__ __forceinline__ int find_request(const uint32_t* start, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

__global__ void __launch_bounds__(kThreads)
kv_tables_kernel(const int32_t* __restrict__ kv_lens, const int32_t* __restrict__ new_lens, int batch,
                 const int32_t* __restrict__ free_pages, int num_free,
                 const int32_t* __restrict__ free_head, int ps, int32_t* tables,
                 int64_t row_stride, int width, int32_t* __restrict__ seq_lens,
                 int32_t* __restrict__ qo_indptr, int64_t* __restrict__ slot_map, int64_t num_slots,
                 int32_t* __restrict__ free_head_out, int32_t* status) {
  extern __shared__ uint32_t smem[];
  uint32_t* start = smem;           // [batch] tokens before the request
  uint32_t* base = smem + batch;    // [batch] fresh pages before it
  int32_t* lens = reinterpret_cast<int32_t*>(smem) + 2 * batch;   // [batch] kv_lens
  __shared__ int64_t warp_tok[kThreads / 32], warp_pg[kThreads / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t head = __ldg(free_head);
  if (tid == 0) s_bad = 0;
  __syncthreads();

  int64_t tok_sum = 0, pg_sum = 0;   // over the requests of earlier rounds
  for (int b0 = 0; b0 < batch; b0 += kThreads) {
    const int b = b0 + tid;
    int64_t nt = 0, np = 0;
    if (b < batch) {
      const int64_t kv = __ldg(kv_lens + b), nw = __ldg(new_lens + b);
      lens[b] = (int32_t)kv;
      if (kv < 0 || nw < 0 || kv + nw > (int64_t)width * ps || kv + nw > 0x7fffffff) {
        s_bad = 1;
      } else {
        nt = nw;
        np = (kv + nw + ps - 1) / ps - (kv + ps - 1) / ps;
      }
    }
    const int64_t it = warp_scan(nt, lane), ip = warp_scan(np, lane);
    if (lane == 31) {
      warp_tok[warp] = it;
      warp_pg[warp] = ip;
    }
    __syncthreads();
    int64_t bt = 0, bp = 0, at = 0, ap = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) {
        bt += warp_tok[w];
        bp += warp_pg[w];
      }
      at += warp_tok[w];
      ap += warp_pg[w];
    }
    if (b < batch) {
      start[b] = (uint32_t)(tok_sum + bt + it - nt);
      base[b] = (uint32_t)(pg_sum + bp + ip - np);
    }
    tok_sum += at;
    pg_sum += ap;
    __syncthreads();
  }
  const bool bad = s_bad || tok_sum > num_slots || tok_sum > 0x7fffffff || head < 0 ||
                   head + pg_sum > num_free;
  const int64_t me = (int64_t)blockIdx.x * kThreads + tid, all = (int64_t)gridDim.x * kThreads;
  if (me == 0) {
    *free_head_out = (int32_t)(bad ? head : head + pg_sum);
    qo_indptr[batch] = bad ? 0 : (int32_t)tok_sum;
    if (bad && status != nullptr) atomicOr(status, STATUS_CAPACITY);
  }
  for (int64_t b = me; b < batch; b += all) {
    qo_indptr[b] = bad ? 0 : (int32_t)start[b];
    seq_lens[b] = lens[b] + (bad ? 0 : __ldg(new_lens + b));
  }
  if (!bad) {
    for (int64_t p = me; p < pg_sum; p += all) {
      const int b = find_request(base, batch, (uint32_t)p);
      const int have = (int)(((uint32_t)lens[b] + (uint32_t)ps - 1u) / (uint32_t)ps);
      tables[b * row_stride + have + (p - base[b])] = __ldg(free_pages + head + p);
    }
  }
  for (int64_t t = me; t < num_slots; t += all) {
    int64_t slot = -1;
    if (!bad && t < tok_sum) {
      const int b = find_request(start, batch, (uint32_t)t);
      // a request has at most 2^31 - 1 tokens: 32-bit unsigned positions
      const uint32_t kv = (uint32_t)lens[b], pos = kv + ((uint32_t)t - start[b]);
      const int page = (int)(pos / (uint32_t)ps), have = (int)((kv + (uint32_t)ps - 1u) / (uint32_t)ps);
      // entries below `have` are inputs of this call, the others come from the list
      const int32_t id = page < have ? tables[b * row_stride + page]
                                     : __ldg(free_pages + head + base[b] + (page - have));
      slot = (int64_t)id * ps + pos % (uint32_t)ps;
    }
    slot_map[t] = slot;
  }
}

}  // namespace

int launch_kv_tables(const int32_t* kv_lens, const int32_t* new_lens, int32_t batch,
                     const int32_t* free_pages, int32_t num_free, const int32_t* free_head,
                     int32_t page_size, int32_t* tables, int64_t row_stride, int32_t width,
                     int32_t* seq_lens, int32_t* qo_indptr, int64_t* slot_map, int64_t num_slots,
                     int32_t* free_head_out, int32_t* status, cudaStream_t stream) {
  if (batch > kMaxBatch)
    return fail(PKA_ERR_UNSUPPORTED, "batch_size %d is above %d", batch, kMaxBatch);
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = set_smem_once(kv_tables_kernel, kMaxBatch * 12, smem_set);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(kv_tables)");
  const int64_t work = std::max<int64_t>(num_slots, batch);
  const int grid = (int)std::min<int64_t>(ceil_div(work, kThreads), 152);
  kv_tables_kernel<<<grid, kThreads, (size_t)batch * 12, stream>>>(
      kv_lens, new_lens, batch, free_pages, num_free, free_head, page_size, tables, row_stride,
      width, seq_lens, qo_indptr, slot_map, num_slots, free_head_out, status);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv_tables_kernel launch");
  return PKA_OK;
}

}  // namespace pka
