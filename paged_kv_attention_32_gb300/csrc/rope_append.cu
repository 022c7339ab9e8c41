// New K/V rows into the paged pools, keys and queries rotated by their positions.
//
// Frequency j of a row turns the pair (x0, x1) by angle pos * inv_freq[j], pos being the
// token's position on the axis that the frequency belongs to (time, height, width, ...):
//   (x0, x1) -> (x0 cos - x1 sin, x1 cos + x0 sin).
// The angle is reduced to a fraction of a turn in 64 bits (a position of 10^6 times a
// frequency of 1 rounded to 32 bits is off by 0.03 radians) and only that fraction, at most
// half a turn, goes through sincospi in 32 bits.  The rotation is 32 bits, rounded once.
//
// Bytes bound it: every row read once and written once.  A warp takes a token, or where
// there are few a share of its heads: four rows at a time, eight lanes a row, 32 bytes a
// lane, six such passes asked for at once (16200 tokens of 32 and 8 heads, 401 MB: 66.5 us,
// 6.0 TB/s; 64 tokens, a kernel's start and one wait for memory: 6.2 us).  It computes the token's angles, two a lane, while
// they are on their way, and keeps in registers the eight that its lanes' values need.
#include <algorithm>

#include "device_common.cuh"
#include "host_common.h"
#include "pages.h"

namespace pka {

using namespace dev;

namespace {

constexpr int kDim = 128, kHalf = kDim / 2;
constexpr int kWarps = 4, kPasses = 6;
constexpr int kFill = 152 * 24;   // warps from which each takes a whole token

template <bool F16, bool HALVES>
__global__ void __launch_bounds__(kWarps * 32) rope_append_kernel(const __grid_constant__ RopeArgs a, int shares) {
  __shared__ __align__(16) float cosv[kWarps][kHalf], sinv[kWarps][kHalf];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t g = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t = g / shares;
  if (t >= a.num_tokens) return;
  const int share = (int)(g - t * shares);
  const int Hq = a.num_qo_heads, Hk = Hq + a.num_kv_heads, rows = Hk + a.num_kv_heads;
  const int passes = (rows + 3) / 4, r0 = lane >> 3, u = lane & 7;   // u: 16 values of a row
  const bool turned = u < a.rotary / 16;
  // where the lane's two pieces of 8 values begin in a row that is rotated, and in any other
  const int c0 = HALVES && turned ? 8 * u : 16 * u, c1 = HALVES && turned ? a.rotary / 2 + 8 * u : 16 * u + 8;
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + t * a.q_stride_tok;
  const uint16_t* k = static_cast<const uint16_t*>(a.k) + t * a.kv_stride_tok;
  const uint16_t* v = static_cast<const uint16_t*>(a.v) + t * a.kv_stride_tok;

  uint4 lo[kPasses], hi[kPasses];
  auto load = [&](int p0) {
#pragma unroll
    for (int n = 0; n < kPasses; ++n) {
      const int row = (p0 + n * shares) * 4 + r0;
      if (row < rows) {
        const uint16_t* src = row < Hq ? q + row * a.q_stride_head
                                       : (row < Hk ? k + (row - Hq) * a.kv_stride_head : v + (row - Hk) * a.kv_stride_head);
        lo[n] = *reinterpret_cast<const uint4*>(src + (row < Hk ? c0 : 16 * u));
        hi[n] = *reinterpret_cast<const uint4*>(src + (row < Hk ? c1 : 16 * u + 8));
      }
    }
  };
  load(share);
  const int64_t slot = __ldg(a.slot_map + t);

  float c[8], s[8];
  if (a.rotary > 0) {
#pragma unroll
    for (int j = lane; j < kHalf; j += 32)
      if (j < a.rotary / 2) {
        int axis = 0;
#pragma unroll
        for (int x = 0; x + 1 < kRopeAxes; ++x)
          if (j >= a.axis_end[x]) axis = x + 1;
        const double pos = (double)__ldg(a.positions + axis * a.pos_stride + t);
        const double turns = pos * (__ldg(a.inv_freq + j) * 0.15915494309189535);   // 1 / 2 pi
        const float part = (float)(turns - rint(turns));
        sincospif(2.f * part, &sinv[warp][j], &cosv[warp][j]);
      }
    __syncwarp();
    if (turned) {
#pragma unroll
      for (int x = 0; x < 8; x += 4) {
        *reinterpret_cast<float4*>(c + x) = *reinterpret_cast<const float4*>(&cosv[warp][8 * u + x]);
        *reinterpret_cast<float4*>(s + x) = *reinterpret_cast<const float4*>(&sinv[warp][8 * u + x]);
      }
    }
  }

  // where the token's keys and values go, nowhere for a slot that is negative or past the pool
  const bool write = slot >= 0 && slot < a.num_slots;
  if (slot >= a.num_slots && share == 0 && lane == 0 && a.status != nullptr) atomicOr(a.status, STATUS_SLOT_BOUNDS);
  int64_t at = 0;
  if (write) {
    // 64-bit division only where the pool needs it
    const int64_t page = slot <= 0xffffffffll ? (int64_t)((uint32_t)slot / (uint32_t)a.page_size) : slot / a.page_size;
    at = page * a.stride_page + (slot - page * a.page_size) * kDim;
  }
  uint16_t* q_out = static_cast<uint16_t*>(a.q_out) + t * a.qo_stride_tok;
  uint16_t* k_out = static_cast<uint16_t*>(a.k_pages) + at;
  uint16_t* v_out = static_cast<uint16_t*>(a.v_pages) + at;
  for (int p0 = share; p0 < passes; p0 += kPasses * shares) {
    if (p0 != share) load(p0);
#pragma unroll
    for (int n = 0; n < kPasses; ++n) {
      const int row = (p0 + n * shares) * 4 + r0;
      if (row >= rows || (row >= Hq && !write)) continue;
      if (row < Hk && turned) {
        uint32_t* x = reinterpret_cast<uint32_t*>(lo + n);
        uint32_t* y = reinterpret_cast<uint32_t*>(hi + n);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 e = unpack2<F16>(x[w]), f = unpack2<F16>(y[w]);
          if (HALVES) {   // pairs (lo, hi): frequencies 8 u + 2 w and the one behind
            x[w] = pack2<F16>(e.x * c[2 * w] - f.x * s[2 * w], e.y * c[2 * w + 1] - f.y * s[2 * w + 1]);
            y[w] = pack2<F16>(f.x * c[2 * w] + e.x * s[2 * w], f.y * c[2 * w + 1] + e.y * s[2 * w + 1]);
          } else {        // neighbours: word w of lo is pair 8 u + w, of hi pair 8 u + 4 + w
            x[w] = pack2<F16>(e.x * c[w] - e.y * s[w], e.y * c[w] + e.x * s[w]);
            y[w] = pack2<F16>(f.x * c[4 + w] - f.y * s[4 + w], f.y * c[4 + w] + f.x * s[4 + w]);
          }
        }
      }
      uint16_t* dst = row < Hq ? q_out + row * a.qo_stride_head
                               : (row < Hk ? k_out + (row - Hq) * a.stride_head : v_out + (row - Hk) * a.stride_head);
      *reinterpret_cast<uint4*>(dst + (row < Hk ? c0 : 16 * u)) = lo[n];
      *reinterpret_cast<uint4*>(dst + (row < Hk ? c1 : 16 * u + 8)) = hi[n];
    }
  }
}

template <bool F16, bool HALVES>
void launch(const RopeArgs& a, cudaStream_t stream) {
  // shares of a token: as many as fill the GPU, none without rows
  const int passes = (a.num_qo_heads + 2 * a.num_kv_heads + 3) / 4;
  const int shares = (int)std::max<int64_t>(1, std::min<int64_t>(passes, kFill / a.num_tokens));
  rope_append_kernel<F16, HALVES>
      <<<(unsigned)ceil_div((int64_t)a.num_tokens * shares, kWarps), kWarps * 32, 0, stream>>>(a, shares);
}

}  // namespace

int launch_rope_append(const RopeArgs& a, bool f16, bool halves, cudaStream_t stream) {
  if (a.num_tokens == 0) return PKA_OK;
  if (f16) halves ? launch<true, true>(a, stream) : launch<true, false>(a, stream);
  else halves ? launch<false, true>(a, stream) : launch<false, false>(a, stream);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "rope_append_kernel launch");
  return PKA_OK;
}

}  // namespace pka
