// Absorbed latent decode: s_j = scale * q . row_j over latent_dim + rope_dim
// values, p = softmax(s), o = sum_j p_j row_j[0 .. latent_dim), all heads over
// the same cached rows.
#include <algorithm>

#include <cuda_bf16.h>

#include "device_common.cuh"
#include "host_common.h"
#include "latent.h"

namespace pka {

using namespace dev;

namespace {

// One CTA per (piece, query row): each warp takes every fourth key with the
// row's values spread over its lanes, and keeps a running maximum and sum.
template <int DL, bool F16>
__global__ void __launch_bounds__(128)
latent_decode_rows_kernel(const __grid_constant__ LatentArgs a, const uint16_t* pages,
                          int64_t stride_page) {
  constexpr int D = DL + kLatentRopeDim, V = D / 64;   // 32-bit words of a row per lane
  __shared__ float s_o[4][DL];
  __shared__ float s_m[4], s_l[4];
  const LatentItem it = a.items[blockIdx.x];
  const LatentReq rq = a.reqs[it.request];
  const int r = blockIdx.y;
  if (r >= rq.q_len * a.num_heads) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i = r / a.num_heads, h = r % a.num_heads;
  int kv = rq.kv_len;
  if (a.seq_lens_live != nullptr) kv = min(max(__ldg(a.seq_lens_live + it.request), 0), kv);
  const int seen = a.causal ? min(kv, kv - rq.q_len + i + 1) : kv;
  const int k0 = it.tile_lo * kLatentTile, k1 = min(it.tile_hi * kLatentTile, seen);
  const int64_t t = rq.q_start + i;
  const uint32_t* q = reinterpret_cast<const uint32_t*>(
      static_cast<const uint16_t*>(a.q) + t * a.q_stride_tok + h * a.q_stride_head);
  float2 qv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) qv[v] = unpack2<F16>(__ldg(q + v * 32 + lane));
  float m = neg_inf(), l = 0.f;
  float2 o[V - 1];
#pragma unroll
  for (int v = 0; v < V - 1; ++v) o[v] = make_float2(0.f, 0.f);
  const int32_t* table = a.block_tables + (int64_t)it.request * a.bt_row_stride;
  for (int k = k0 + warp; k < k1; k += 4) {
    const int page = __ldg(table + k / a.page_size);
    float2 x[V];
    if (page >= 0 && page < a.num_pages) {
      const uint32_t* row = reinterpret_cast<const uint32_t*>(
          pages + page * stride_page + (int64_t)(k % a.page_size) * D);
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = unpack2<F16>(__ldg(row + v * 32 + lane));
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = make_float2(0.f, 0.f);
    }
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) s += qv[v].x * x[v].x + qv[v].y * x[v].y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s), sc = ex2(m - mn), p = ex2(s - mn);
    m = mn;
    l = l * sc + p;
#pragma unroll
    for (int v = 0; v < V - 1; ++v) {
      o[v].x = o[v].x * sc + p * x[v].x;
      o[v].y = o[v].y * sc + p * x[v].y;
    }
  }
#pragma unroll
  for (int v = 0; v < V - 1; ++v) {
    s_o[warp][v * 64 + lane * 2] = o[v].x;
    s_o[warp][v * 64 + lane * 2 + 1] = o[v].y;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  const float mm = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float w[4], ll = 0.f;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    w[x] = s_m[x] == neg_inf() ? 0.f : ex2(s_m[x] - mm);
    ll += w[x] * s_l[x];
  }
  const bool whole = it.part < 0;
  const int64_t prow = rq.part_base + (int64_t)max(it.part, 0) * rq.q_len * a.num_heads + r;
  const float inv = ll > 0.f ? (whole ? a.output_scale : 1.f) / ll : 0.f;
  for (int dd = tid; dd < DL; dd += 128) {
    const float v = (w[0] * s_o[0][dd] + w[1] * s_o[1][dd] + w[2] * s_o[2][dd] + w[3] * s_o[3][dd]) * inv;
    if (whole) store_out1(a.out, (t * a.num_heads + h) * DL + dd, v, a.out_dtype);
    else a.ws_o[prow * DL + dd] = v;
  }
  if (tid == 0) {
    const float lse = ll > 0.f ? mm + log2f(ll) : neg_inf();
    if (!whole) a.ws_lse[prow] = lse;
    else if (a.lse != nullptr) a.lse[t * a.num_heads + h] = lse;
  }
}

// The pieces of a cut request: out = sum_c w_c o_c / sum_c w_c with
// w_c = 2^(lse_c - max), one CTA per row.  Four thread groups take every
// fourth piece, so the loads of many pieces are in flight at once.
template <int DL>
__global__ void __launch_bounds__(DL)
latent_merge_kernel(const __grid_constant__ LatentArgs a) {
  constexpr int T = DL / 4;   // threads of a group: four values each
  __shared__ float4 s_o[3][T];
  const int b = a.splits[blockIdx.x / a.max_rows], r = blockIdx.x % a.max_rows;
  const LatentReq rq = a.reqs[b];
  const int rows = rq.q_len * a.num_heads;
  if (r >= rows) return;
  const int g = threadIdx.x / T, x = threadIdx.x % T;
  float m = neg_inf();
  for (int c = 0; c < rq.n_parts; ++c)
    m = fmaxf(m, __ldg(a.ws_lse + rq.part_base + (int64_t)c * rows + r));
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  if (m != neg_inf()) {
    for (int c = 0; c < rq.n_parts; ++c)
      sum += ex2(__ldg(a.ws_lse + rq.part_base + (int64_t)c * rows + r) - m);
#pragma unroll 4
    for (int c = g; c < rq.n_parts; c += 4) {
      const int64_t prow = rq.part_base + (int64_t)c * rows + r;
      const float lse = __ldg(a.ws_lse + prow);
      if (lse == neg_inf()) continue;   // a piece without keys has no output rows
      const float w = ex2(lse - m);
      const float4 v = __ldg(reinterpret_cast<const float4*>(a.ws_o + prow * DL) + x);
      o.x += w * v.x;
      o.y += w * v.y;
      o.z += w * v.z;
      o.w += w * v.w;
    }
  }
  if (g > 0) s_o[g - 1][x] = o;
  __syncthreads();
  if (g > 0) return;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    o.x += s_o[k][x].x;
    o.y += s_o[k][x].y;
    o.z += s_o[k][x].z;
    o.w += s_o[k][x].w;
  }
  const int64_t row = ((int64_t)rq.q_start + r / a.num_heads) * a.num_heads + r % a.num_heads;
  const float v[4] = {o.x, o.y, o.z, o.w};
  store_out<4>(a.out, row * DL + x * 4, v, sum > 0.f ? a.output_scale / sum : 0.f, a.out_dtype);
  if (x == 0 && a.lse != nullptr) a.lse[row] = sum > 0.f ? m + log2f(sum) : neg_inf();
}

template <int DL>
int launch(const pka_latent_plan& plan, const LatentArgs& a, const void* pages, int64_t stride_page,
           cudaStream_t stream) {
  const dim3 grid((unsigned)a.num_items, (unsigned)a.max_rows);
  auto kern = plan.desc.dtype == PKA_DTYPE_F16 ? latent_decode_rows_kernel<DL, true>
                                               : latent_decode_rows_kernel<DL, false>;
  kern<<<grid, 128, 0, stream>>>(a, static_cast<const uint16_t*>(pages), stride_page);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "latent decode kernel launch");
  if (a.num_splits > 0) {
    latent_merge_kernel<DL><<<(unsigned)(a.num_splits * a.max_rows), DL, 0, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "latent_merge_kernel launch");
  }
  return PKA_OK;
}

}  // namespace

int launch_latent_decode(const pka_latent_plan& plan, const LatentArgs& a, const void* pages,
                         int64_t stride_page, cudaStream_t stream) {
  if (a.num_items == 0) return PKA_OK;
  return plan.desc.latent_dim == 512 ? launch<512>(plan, a, pages, stride_page, stream)
                                     : launch<256>(plan, a, pages, stride_page, stream);
}

}  // namespace pka
