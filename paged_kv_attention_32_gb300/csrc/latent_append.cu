// New latent rows into the paged pool: row t, [latent[t] | rope[t]], to slot
// slot_map[t].  A copy: one read and one write of each row bound it.  A warp
// takes a row, 16 bytes a lane, and asks for all of it and then for its slot
// before it looks at either, so that no load waits for another.  Measured, rows
// of 576: one row 1.6 us, 64 rows 1.7, 32768 rows 13.4 us (5.6 TB/s of the 6.8
// that a plain copy reaches), 131072 rows 46.5 us (6.5 TB/s).  Measured and not
// kept, 32768 rows: the slot asked for first (14.7 us), four rows a warp (15.2),
// one vector per thread, its row found by division and its load behind the
// slot's (20.0); CTAs of 512 threads (15.4).
#include <algorithm>

#include "device_common.cuh"
#include "host_common.h"
#include "latent.h"

namespace pka {

namespace {

constexpr int kThreads = 128;
constexpr int kVecs = 3;   // 16-byte pieces of a row per lane and pass: 576 values in one pass

__global__ void __launch_bounds__(kThreads)
latent_append_kernel(const uint4* __restrict__ latent, int64_t latent_vecs,
                     const uint4* __restrict__ rope, int64_t rope_vecs, int nl, int nr,
                     const int64_t* __restrict__ slot_map, int64_t num_tokens,
                     uint4* __restrict__ pages, int64_t num_slots, int page_size,
                     int64_t page_vecs, int32_t* status) {
  const int row = nl + nr, lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  const int64_t warp = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  for (int64_t t = warp; t < num_tokens; t += warps) {
    for (int v0 = lane; v0 < row; v0 += 32 * kVecs) {
      uint4 x[kVecs];
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const int v = v0 + 32 * k;
        if (v < row)
          x[k] = v < nl ? __ldg(latent + t * latent_vecs + v) : __ldg(rope + t * rope_vecs + (v - nl));
      }
      const int64_t slot = __ldg(slot_map + t);
      if (slot < 0) continue;
      if (slot >= num_slots) {
        if (v0 == 0 && status != nullptr) atomicOr(status, STATUS_SLOT_BOUNDS);
        continue;
      }
      // 64-bit division only where the pool needs it
      const int64_t page = slot <= 0xffffffffll ? (int64_t)((uint32_t)slot / (uint32_t)page_size)
                                                : slot / page_size;
      uint4* dst = pages + page * page_vecs + (slot - page * page_size) * row;
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
        if (v0 + 32 * k < row) dst[v0 + 32 * k] = x[k];
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
  // a few waves at most, then a warp walks on
  const int grid = (int)std::min<int64_t>(ceil_div(num_tokens, kThreads / 32), 152 * 64);
  latent_append_kernel<<<grid, kThreads, 0, stream>>>(
      static_cast<const uint4*>(latent), latent_stride / 8, static_cast<const uint4*>(rope),
      rope_stride / 8, latent_dim / 8, rope_dim / 8, slot_map, num_tokens,
      static_cast<uint4*>(pages), num_pages * page_size, page_size, stride_page / 8, status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "latent_append_kernel launch");
  return PKA_OK;
}

}  // namespace pka
