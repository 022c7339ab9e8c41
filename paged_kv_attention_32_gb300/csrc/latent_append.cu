// New latent rows into the paged pool: row t, [latent[t] | rope[t]], to slot
// slot_map[t].  A copy: one read and one write of each row bound it.  A warp
// takes ROWS rows at a time, 16 bytes a lane, and asks for all of them and their
// slots before it looks at any: the loads of a row do not wait for its slot.
// Many tokens take 4 rows a warp (32768 rows of 576: 20.0 us with one vector per
// thread, its row found by division and its load behind the slot's); few take
// one, for the shortest chain.
#include <algorithm>

#include "device_common.cuh"
#include "host_common.h"
#include "latent.h"

namespace pka {

namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 3;   // 16-byte pieces of a row per lane and pass: 576 values in one pass

template <int ROWS>
__global__ void __launch_bounds__(kThreads)
latent_append_kernel(const uint4* __restrict__ latent, int64_t latent_vecs,
                     const uint4* __restrict__ rope, int64_t rope_vecs, int nl, int nr,
                     const int64_t* __restrict__ slot_map, int64_t num_tokens,
                     uint4* __restrict__ pages, int64_t num_slots, int page_size,
                     int64_t page_vecs, int32_t* status) {
  const int row = nl + nr, lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  const int64_t warp = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  for (int64_t t0 = warp * ROWS; t0 < num_tokens; t0 += warps * ROWS) {
    int64_t slot[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) slot[r] = t0 + r < num_tokens ? __ldg(slot_map + t0 + r) : -1;
    for (int v0 = lane; v0 < row; v0 += 32 * kVecs) {
      uint4 x[ROWS][kVecs];
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          const int v = v0 + 32 * k;
          const int64_t t = min(t0 + r, num_tokens - 1);
          if (v < row)
            x[r][k] = v < nl ? __ldg(latent + t * latent_vecs + v) : __ldg(rope + t * rope_vecs + (v - nl));
        }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (slot[r] < 0) continue;
        if (slot[r] >= num_slots) {
          if (v0 == 0 && status != nullptr) atomicOr(status, STATUS_SLOT_BOUNDS);
          continue;
        }
        // 64-bit division only where the pool needs it
        const int64_t page = slot[r] <= 0xffffffffll ? (int64_t)((uint32_t)slot[r] / (uint32_t)page_size)
                                                     : slot[r] / page_size;
        uint4* dst = pages + page * page_vecs + (slot[r] - page * page_size) * row;
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
          if (v0 + 32 * k < row) dst[v0 + 32 * k] = x[r][k];
      }
    }
  }
}

}  // namespace

int launch_latent_append(const void* latent, int64_t latent_stride, const void* rope,
                         int64_t rope_stride, int32_t latent_dim, int32_t rope_dim,
                         const int64_t* slot_map, int64_t num_tokens, void* pages,
                         int64_t num_pages, int32_t page_size, int64_t stride_page,
                         int32_t* status, cudaStream_t stream) {
  if (num_tokens == 0) return PKA_OK;
  const bool many = num_tokens >= 8192;
  const int64_t warps = ceil_div(num_tokens, many ? 4 : 1);
  const int grid = (int)std::min<int64_t>(ceil_div(warps, kThreads / 32), 152 * 64);
  auto kern = many ? latent_append_kernel<4> : latent_append_kernel<1>;
  kern<<<grid, kThreads, 0, stream>>>(
      static_cast<const uint4*>(latent), latent_stride / 8, static_cast<const uint4*>(rope),
      rope_stride / 8, latent_dim / 8, rope_dim / 8, slot_map, num_tokens,
      static_cast<uint4*>(pages), num_pages * page_size, page_size, stride_page / 8, status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "latent_append_kernel launch");
  return PKA_OK;
}

}  // namespace pka
