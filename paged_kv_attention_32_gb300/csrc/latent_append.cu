// New latent rows into the paged pool: row t, [latent[t] | rope[t]], to slot
// slot_map[t].  A copy: one read and one write of each row bound it.  One
// thread per 16 bytes of a row.
#include <algorithm>

#include "device_common.cuh"
#include "host_common.h"
#include "latent.h"

namespace pka {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
latent_append_kernel(const uint4* __restrict__ latent, int64_t latent_vecs,
                     const uint4* __restrict__ rope, int64_t rope_vecs, int nl, int nr,
                     const int64_t* __restrict__ slot_map, int64_t num_tokens,
                     uint4* __restrict__ pages, int64_t num_slots, int page_size,
                     int64_t page_vecs, int32_t* status) {
  const int row = nl + nr;
  const int64_t total = num_tokens * row, step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += step) {
    const int64_t t = i / row;
    const int v = (int)(i - t * row);
    const int64_t slot = __ldg(slot_map + t);
    if (slot < 0) continue;
    if (slot >= num_slots) {
      if (v == 0 && status != nullptr) atomicOr(status, STATUS_SLOT_BOUNDS);
      continue;
    }
    const uint4 x = v < nl ? __ldg(latent + t * latent_vecs + v) : __ldg(rope + t * rope_vecs + v - nl);
    const int64_t page = slot / page_size;
    pages[page * page_vecs + (slot - page * page_size) * row + v] = x;
  }
}

}  // namespace

int launch_latent_append(const void* latent, int64_t latent_stride, const void* rope,
                         int64_t rope_stride, int32_t latent_dim, int32_t rope_dim,
                         const int64_t* slot_map, int64_t num_tokens, void* pages,
                         int64_t num_pages, int32_t page_size, int64_t stride_page,
                         int32_t* status, cudaStream_t stream) {
  if (num_tokens == 0) return PKA_OK;
  const int64_t total = num_tokens * ((latent_dim + rope_dim) / 8);
  const int grid = (int)std::min<int64_t>(ceil_div(total, kThreads), 152 * 8);
  latent_append_kernel<<<grid, kThreads, 0, stream>>>(
      static_cast<const uint4*>(latent), latent_stride / 8, static_cast<const uint4*>(rope),
      rope_stride / 8, latent_dim / 8, rope_dim / 8, slot_map, num_tokens,
      static_cast<uint4*>(pages), num_pages * page_size, page_size, stride_page / 8, status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "latent_append_kernel launch");
  return PKA_OK;
}

}  // namespace pka
