// New K/V rows into the paged pools, keys and queries rotated by their positions.
//
// Frequency j of a row turns the pair (x0, x1) by angle pos * inv_freq[j], pos being the
// token's position on the axis that the frequency belongs to (time, height, width, ...):
//   (x0, x1) -> (x0 cos - x1 sin, x1 cos + x0 sin).
// The angle is reduced to a fraction of a turn in 64 bits (a position of 10^6 times a
// frequency of 1 rounded to 32 bits is off by 0.03 radians) and only that fraction, at most
// half a turn, goes through sincospi in 32 bits.  The rotation is 32 bits, rounded once.
//
// Bytes bound it: every row read once and written once.  A CTA takes 1 or 4 tokens; a
// thread asks for all of its 16-byte pieces first, then computes one or two of the
// tokens' angles for everybody while they are on their way.
#include <algorithm>

#include "device_common.cuh"
#include "host_common.h"
#include "pages.h"

namespace pka {

using namespace dev;

namespace {

constexpr int kThreads = 256;
constexpr int kDim = 128, kUnits = kDim / 16;   // a unit is two pieces of 8 values
constexpr int kHalf = kDim / 2;
// At least this many tokens: four to a CTA, so that a thread has six units in flight.
constexpr int kManyTokens = 608;

// TB tokens a CTA, N units a thread and round.
template <bool F16, bool HALVES, int TB, int N>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float cosv[TB][kHalf], sinv[TB][kHalf];
  const int tid = threadIdx.x;
  const int t0 = (int)blockIdx.x * TB;
  const int tokens = min(TB, a.num_tokens - t0);
  const int Hq = a.num_qo_heads, Hk = Hq + a.num_kv_heads, rows = Hk + a.num_kv_heads;
  const int per_token = rows * kUnits, total = per_token * tokens;
  const int turned = a.rotary / 16;   // a row's first units, which are rotated

  uint4 lo[N], hi[N];
  // unit `i`'s token, row and unit of the row
  auto place = [&](int i, int& t, int& row, int& u) {
    t = 0;
#pragma unroll
    for (int k = 1; k < TB; ++k)
      if (i >= k * per_token) t = k;
    i -= t * per_token;
    row = i / kUnits;
    u = i % kUnits;
  };
  // where its two pieces begin in the row
  auto pieces = [&](int row, int u, int& c0, int& c1) {
    const bool split = HALVES && row < Hk && u < turned;
    c0 = split ? 8 * u : 16 * u;
    c1 = split ? a.rotary / 2 + 8 * u : 16 * u + 8;
  };
  auto load = [&](int first) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = first + n * kThreads + tid;
      if (i < total) {
        int t, row, u, c0, c1;
        place(i, t, row, u);
        pieces(row, u, c0, c1);
        const uint16_t* src;
        if (row < Hq)
          src = static_cast<const uint16_t*>(a.q) + (int64_t)(t0 + t) * a.q_stride_tok + row * a.q_stride_head;
        else
          src = static_cast<const uint16_t*>(row < Hk ? a.k : a.v) + (int64_t)(t0 + t) * a.kv_stride_tok +
                (row < Hk ? row - Hq : row - Hk) * a.kv_stride_head;
        lo[n] = *reinterpret_cast<const uint4*>(src + c0);
        hi[n] = *reinterpret_cast<const uint4*>(src + c1);
      }
    }
  };
  load(0);

  if (a.rotary > 0) {
    const int half = a.rotary / 2;
    for (int i = tid; i < TB * kHalf; i += kThreads) {
      const int t = i / kHalf, j = i % kHalf;
      if (t < tokens && j < half) {
        int axis = 0;
#pragma unroll
        for (int x = 0; x + 1 < kRopeAxes; ++x)
          if (j >= a.axis_end[x]) axis = x + 1;
        const double pos = (double)__ldg(a.positions + axis * a.pos_stride + t0 + t);
        const double turns = pos * (__ldg(a.inv_freq + j) * 0.15915494309189535);   // 1 / 2 pi
        const float part = (float)(turns - rint(turns));
        sincospif(2.f * part, &sinv[t][j], &cosv[t][j]);
      }
    }
    __syncthreads();
  }

  for (int first = 0; first < total; first += N * kThreads) {
    if (first > 0) load(first);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = first + n * kThreads + tid;
      if (i >= total) continue;
      int t, row, u, c0, c1;
      place(i, t, row, u);
      pieces(row, u, c0, c1);
      if (row < Hk && u < turned) {
        float c[8], s[8];
#pragma unroll
        for (int x = 0; x < 8; x += 4) {
          *reinterpret_cast<float4*>(c + x) = *reinterpret_cast<const float4*>(&cosv[t][8 * u + x]);
          *reinterpret_cast<float4*>(s + x) = *reinterpret_cast<const float4*>(&sinv[t][8 * u + x]);
        }
        uint32_t* x = reinterpret_cast<uint32_t*>(lo + n);
        uint32_t* y = reinterpret_cast<uint32_t*>(hi + n);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 p = unpack2<F16>(x[w]), r = unpack2<F16>(y[w]);
          if (HALVES) {   // pairs (lo, hi): frequencies 8 u + 2 w and the one behind
            x[w] = pack2<F16>(p.x * c[2 * w] - r.x * s[2 * w], p.y * c[2 * w + 1] - r.y * s[2 * w + 1]);
            y[w] = pack2<F16>(r.x * c[2 * w] + p.x * s[2 * w], r.y * c[2 * w + 1] + p.y * s[2 * w + 1]);
          } else {        // neighbours: word w of lo is pair 8 u + w, of hi pair 8 u + 4 + w
            x[w] = pack2<F16>(p.x * c[w] - p.y * s[w], p.y * c[w] + p.x * s[w]);
            y[w] = pack2<F16>(r.x * c[4 + w] - r.y * s[4 + w], r.y * c[4 + w] + r.x * s[4 + w]);
          }
        }
      }
      uint16_t* dst;
      if (row < Hq) {
        dst = static_cast<uint16_t*>(a.q_out) + (int64_t)(t0 + t) * a.qo_stride_tok + row * a.qo_stride_head;
      } else {
        const int64_t slot = __ldg(a.slot_map + t0 + t);
        if (slot < 0) continue;
        if (slot >= a.num_slots) {
          if (row == Hq && u == 0 && a.status != nullptr) atomicOr(a.status, STATUS_SLOT_BOUNDS);
          continue;
        }
        // 64-bit division only where the pool needs it
        const int64_t page = slot <= 0xffffffffll ? (int64_t)((uint32_t)slot / (uint32_t)a.page_size)
                                                  : slot / a.page_size;
        dst = static_cast<uint16_t*>(row < Hk ? a.k_pages : a.v_pages) + page * a.stride_page +
              (row < Hk ? row - Hq : row - Hk) * a.stride_head + (slot - page * a.page_size) * kDim;
      }
      *reinterpret_cast<uint4*>(dst + c0) = lo[n];
      *reinterpret_cast<uint4*>(dst + c1) = hi[n];
    }
  }
}

template <bool F16, bool HALVES>
void launch(const RopeArgs& a, cudaStream_t stream) {
  if (a.num_tokens >= kManyTokens)
    rope_append_kernel<F16, HALVES, 4, 6><<<(unsigned)ceil_div(a.num_tokens, 4), kThreads, 0, stream>>>(a);
  else
    rope_append_kernel<F16, HALVES, 1, 2><<<(unsigned)a.num_tokens, kThreads, 0, stream>>>(a);
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
