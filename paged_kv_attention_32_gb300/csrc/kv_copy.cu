// Pages copied inside their pools: entry i takes page src[i] to dst[i] of every pool.
//
// One read and one write of each page bound it (pages of 32 KB, 1.81 GB in all: 271 us, 6.7
// TB/s).  CTAs walk over pieces of 16 KB; the entries that count come first and their number
// may lie on the device, so that a list made there needs no look from the host and its empty
// tail costs little.
#include <algorithm>

#include "device_common.cuh"
#include "host_common.h"
#include "pages.h"

namespace pka {

using namespace dev;

namespace {

constexpr int kThreads = 256, kVecs = 4;
constexpr int64_t kPiece = kThreads * kVecs * 16;
// Four waves of CTAs: the later ones even out what the SMs differ in (one wave 290 us for the 1.81 GB,
// eight 267), and cost little where a long list is empty (3.5 us; one wave 1.7, eight 5.8).
constexpr int64_t kCtas = 152 * 32;

__global__ void __launch_bounds__(kThreads) kv_copy_kernel(const __grid_constant__ CopyArgs a, int pieces) {
  int64_t n = a.num_entries;
  if (a.count != nullptr) n = max(0, min(a.num_entries, __ldg(a.count)));
  const int64_t per_entry = (int64_t)a.num_pools * pieces;
  const int64_t items = n * per_entry;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t entry = item / per_entry;
    const int rest = (int)(item - entry * per_entry);
    const int src = __ldg(a.src_pages + entry), dst = __ldg(a.dst_pages + entry);
    if (src < 0 || dst < 0) continue;
    if (src >= a.num_pages || dst >= a.num_pages) {
      if (threadIdx.x == 0 && rest == 0 && a.status != nullptr) atomicOr(a.status, STATUS_PAGE_BOUNDS);
      continue;
    }
    const PagePool& pool = a.pools[rest / pieces];
    const int64_t at = (int64_t)(rest % pieces) * kPiece;
    const uint4* from = reinterpret_cast<const uint4*>(pool.base + src * pool.stride + at);
    uint4* to = reinterpret_cast<uint4*>(pool.base + dst * pool.stride + at);
    const int vecs = (int)(max((int64_t)0, min(kPiece, pool.bytes - at)) / 16);
    uint4 x[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      if (k * kThreads + (int)threadIdx.x < vecs) x[k] = from[k * kThreads + threadIdx.x];
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      if (k * kThreads + (int)threadIdx.x < vecs) to[k * kThreads + threadIdx.x] = x[k];
  }
}

}  // namespace

int launch_kv_copy(const CopyArgs& a, cudaStream_t stream) {
  int64_t most = 0;
  for (int i = 0; i < a.num_pools; ++i) most = std::max(most, a.pools[i].bytes);
  const int64_t pieces = ceil_div(most, kPiece);
  const int64_t items = (int64_t)a.num_entries * a.num_pools * pieces;
  if (items == 0) return PKA_OK;
  if (a.num_pools * pieces > 0x7fffffff) return fail(PKA_ERR_UNSUPPORTED, "pages of %lld bytes", (long long)most);
  kv_copy_kernel<<<(unsigned)std::min<int64_t>(items, kCtas), kThreads, 0, stream>>>(a, (int)pieces);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv_copy_kernel launch");
  return PKA_OK;
}

}  // namespace pka
