// The rest of a decode behind shared prefixes: the requests' own keys, and the merge of all
// partial states.
//
// Own keys: every warp streams pieces of up to 16 units of 16 keys (one request, KV head and
// 16-row tile), which it takes as they come, through the tensor-core step of the paged decode
// (mma.sync m16n8k16; a tile of up to 8 rows with the keys on the 16-row side).  Its copies
// run ahead over the borders of the pieces, the next of which is taken a piece early, and
// nothing waits for another warp: a piece ends with a 32-bit partial state of its rows.  p is
// rounded to the input type for the product with V, as the tensor core takes it, after its 32-bit sum.
// HBM bounds it; what an ordinary decode of many short requests loses to CTAs that start
// and end is the reason for the pieces (64 requests of 64 to 1024 keys: 35 us for 21 us of
// bytes; in pieces 28 us alone, 4.9 TB/s).  A CTA of 4 warps fits beside a CTA of the prefix
// kernel, whose memory time it shares; the others follow where that one ends (with 8192
// shared keys both, 171 MB, end after 33 us: 5.2 TB/s).
//
// Merge: a warp a row, every state's LSE and eight of the states at once, 16 bytes a lane.
// L2 bounds it: 2048 rows of 14 states, 14.6 MB, in 4 us.
#include <algorithm>

#include "decode_mma_tile.cuh"
#include "device_common.cuh"
#include "host_common.h"
#include "prefix.h"

namespace pka {

using namespace dev;

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kStages = 2;
constexpr int kUnit = kMmaUnitTok;
constexpr int kThreads = kOwnWarps * 32;
constexpr int kOwnRegs = 168;   // three CTAs an SM, or one beside the prefix kernel's 11 warps of 112

// As tma_load_kv_pair_elect; what it brings is the first to leave L2 again: it is read once,
// and the partial states that the merge reads are to stay.
__device__ __forceinline__ void load_kv_once(uint32_t dst_k, uint32_t dst_v, const CUtensorMap* map_k,
                                             const CUtensorMap* map_v, uint32_t bar, uint32_t bytes, int32_t slot,
                                             int32_t head, int32_t page, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%4], %5;\n\t"
      "@e cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%2, {%6, %7, %6, %8, %9}], [%4], %10;\n\t"
      "@e cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%1], [%3, {%6, %7, %6, %8, %9}], [%4], %10;\n\t}" ::"r"(dst_k),
      "r"(dst_v), "l"(reinterpret_cast<uint64_t>(map_k)), "l"(reinterpret_cast<uint64_t>(map_v)),
      "r"(bar), "r"(bytes), "r"(0), "r"(slot), "r"(head), "r"(page), "l"(policy)
      : "memory");
}

// Writes a tile's state: rows of O / l, and the base-2 LSE m + log2 l.
template <bool F16>
__device__ __forceinline__ void store_state(const MmaTileWarp<F16>& tw, float* o, float* lse, int rows, int lane) {
  const int g4 = lane >> 2, t4 = lane & 3;
  const float iA = tw.lA != 0.f ? 1.f / tw.lA : 0.f, iB = tw.lB != 0.f ? 1.f / tw.lB : 0.f;
#pragma unroll
  for (int n = 0; n < 16; ++n) {
    if (g4 < rows)
      *reinterpret_cast<float2*>(o + g4 * 128 + n * 8 + t4 * 2) = make_float2(tw.acc[n][0] * iA, tw.acc[n][1] * iA);
    if (g4 + 8 < rows)
      *reinterpret_cast<float2*>(o + (g4 + 8) * 128 + n * 8 + t4 * 2) =
          make_float2(tw.acc[n][2] * iB, tw.acc[n][3] * iB);
  }
  if (t4 == 0) {
    if (g4 < rows) lse[g4] = tw.lA != 0.f ? tw.mA + log2f(tw.lA) : neg_inf();
    if (g4 + 8 < rows) lse[g4 + 8] = tw.lB != 0.f ? tw.mB + log2f(tw.lB) : neg_inf();
  }
}
template <bool F16>
__device__ __forceinline__ void store_state(const MmaTileWarpT<F16>& tw, float* o, float* lse, int rows, int lane) {
  const int g4 = lane >> 2, rA = 2 * (lane & 3), rB = rA + 1;
  const float iA = tw.lA != 0.f ? 1.f / tw.lA : 0.f, iB = tw.lB != 0.f ? 1.f / tw.lB : 0.f;
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    if (rA < rows) {
      o[rA * 128 + m * 16 + g4] = tw.acc[m][0] * iA;
      o[rA * 128 + m * 16 + g4 + 8] = tw.acc[m][2] * iA;
    }
    if (rB < rows) {
      o[rB * 128 + m * 16 + g4] = tw.acc[m][1] * iB;
      o[rB * 128 + m * 16 + g4 + 8] = tw.acc[m][3] * iB;
    }
  }
  if (g4 == 0) {
    if (rA < rows) lse[rA] = tw.lA != 0.f ? tw.mA + log2f(tw.lA) : neg_inf();
    if (rB < rows) lse[rB] = tw.lB != 0.f ? tw.mB + log2f(tw.lB) : neg_inf();
  }
}

// NARROW: every tile has at most 8 rows.
template <bool F16, bool NARROW>
__global__ void __maxnreg__(kOwnRegs) prefix_own_kernel(const __grid_constant__ OwnArgs x, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv) {
  const DecodeArgs& a = x.decode;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* stages = smem + warp * kStages * kMmaUnitBytes;
  const uint32_t stage_u32 = smem_u32(stages);
  const uint32_t bar_u32 = smem_u32(smem) + kOwnWarps * kStages * kMmaUnitBytes + (uint32_t)warp * kStages * 8u;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bar_u32 + 8u * s, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  __syncwarp();

  const int upp = a.page_size / kUnit;
  const float sl2 = a.scale_log2;
  auto length = [&](const OwnPiece& p) -> int {
    int n = p.kv_len;
    if (a.seq_lens_live != nullptr) n = max(min(__ldg(a.seq_lens_live + p.request), n), p.q_len);
    return n;
  };
  auto units_of = [&](const OwnPiece& p, int kv_len) -> int {
    return max(0, min(p.unit_hi, (kv_len + kUnit - 1) / kUnit) - p.unit_lo);
  };
  // page of the lane's unit of a piece (of at most 32)
  auto pages_of = [&](const OwnPiece& p) -> int {
    const int u = p.unit_lo + lane;
    return u < p.unit_hi ? __ldg(a.block_tables + (int64_t)p.request * a.bt_row_stride + u / upp) : 0;
  };
  // The number of a piece to take is asked for a while before it is needed.
  int ticket = 0;
  auto ask = [&]() {
    if (lane == 0) ticket = x.num_static + atomicAdd(x.next, 1);
  };
  auto told = [&]() -> int { return __shfl_sync(FULL, ticket, 0); };

  // p: the piece whose rows are computed, of n units, pk of them copied; q: the one behind it
  OwnPiece p{}, q{};
  int len = 0, n = 0, pk = 0, p_pages = 0, q_len = 0, qn = 0, qk = 0, q_pages = 0;
  const int own = warp * x.static_ctas + (int)blockIdx.x;
  int at = own;
  if ((int)blockIdx.x >= x.static_ctas || own >= x.num_static) {
    ask();
    at = told();
  }
  bool p_any = at < x.num_pieces, q_any = false;
  if (p_any) {
    ask();
    p = x.pieces[at];
    len = length(p);
    n = units_of(p, len);
    p_pages = pages_of(p);
  }
  uint64_t once;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
  int issued = 0, used = 0;
  auto issue = [&]() -> bool {   // a unit of p, or behind it of q; false where neither has one
    const bool ahead = pk >= n;
    if (ahead && qk >= qn) return false;
    const int k = ahead ? qk : pk;
    const int page = __shfl_sync(FULL, ahead ? q_pages : p_pages, k);
    const int st = issued % kStages;
    const uint32_t dst = stage_u32 + (uint32_t)st * kMmaUnitBytes;
    load_kv_once(dst, dst + 2 * kMmaBoxBytes, &tmk, &tmv, bar_u32 + 8u * (uint32_t)st, kMmaUnitBytes,
                 ((ahead ? q.unit_lo : p.unit_lo) + k) % upp * kUnit, (ahead ? q : p).head_tile & 0xffff, page, once);
    if (ahead) ++qk;
    else ++pk;
    ++issued;
    return true;
  };
  auto look = [&]() {            // q's units and pages
    q_len = length(q);
    qn = units_of(q, q_len);
    q_pages = pages_of(q);
  };
  while (issued < kStages && issue()) {
  }

  bool ok = true;
  auto run = [&](auto& tw) {
    const int tile = p.head_tile >> 16;
    ReqInfo rq{};
    rq.q_start = p.q_start;
    rq.q_len = p.q_len;
    tw.init(a, rq, len, p.head_tile & 0xffff, tile, lane);
    const int all_hi = a.causal ? len - p.q_len + 1 : len;
    for (int k = 0; k < n; ++k) {
      const int st = used % kStages;
      if (!(ok = __all_sync(FULL, mbar_wait(bar_u32 + 8u * (uint32_t)st, (uint32_t)((used / kStages) & 1), a.status))))
        return;
      const int tok0 = (p.unit_lo + k) * kUnit;
      if (tok0 + kUnit > len) {   // slots past the last key may hold anything: 0 * inf is not 0
        uint8_t* v = stages + st * kMmaUnitBytes + 2 * kMmaBoxBytes + (lane >> 3) * kMmaBoxBytes + (lane & 7) * 16;
        if (lane < 16)
          for (int j = len - tok0; j < kUnit; ++j) *reinterpret_cast<uint4*>(v + j * 128) = make_uint4(0u, 0u, 0u, 0u);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // a copy comes into this stage again
        __syncwarp();
      }
      tw.step(stage_u32 + (uint32_t)st * kMmaUnitBytes, tok0, tok0 + kUnit <= all_hi, sl2, lane);
      __syncwarp();
      ++used;
      if (k == 0 && q_any) look();
      if (k == max(0, n - 2) && q_any) ask();
      issue();
    }
    tw.reduce_l();
    store_state(tw, a.ws_o + (int64_t)p.state * 128, a.ws_lse + p.state, min(kOwnRows, a.group * p.q_len - tile * kOwnRows),
                lane);
  };
  while (p_any) {
    const int next = told();
    q_any = next < x.num_pieces;
    qn = qk = 0;
    if (q_any) q = x.pieces[next];
    if (NARROW || a.group * p.q_len - (p.head_tile >> 16) * kOwnRows <= 8) {
      MmaTileWarpT<F16> tw;
      run(tw);
    } else {
      if constexpr (!NARROW) {
        MmaTileWarp<F16> tw;
        run(tw);
      }
    }
    if (!ok) break;
    if (n == 0 && q_any) {   // a request that ends before the piece: nothing was asked on the way
      look();
      ask();
    }
    p = q;
    len = q_len;
    n = qn;
    pk = qk;
    p_pages = q_pages;
    p_any = q_any;
    qn = qk = 0;
    while (p_any && issued < used + kStages && issue()) {
    }
  }
  // a wait gave up: let the copies still in flight land (bounded) before the CTA exits
  for (; used < issued; ++used)
    (void)mbar_wait(bar_u32 + 8u * (uint32_t)(used % kStages), (uint32_t)((used / kStages) & 1), nullptr);
  // The merge waits for this grid, and through one CTA of it for the prefix kernel before it;
  // the others make room for those that still wait for an SM.
  if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---- merge ----------------------------------------------------------------------

constexpr int kMergeWarps = 4, kMergeLoads = 8;
constexpr int kMergeCtas = 152 * 7;   // one wave
// Eight warps a row where few rows have many states (38 states of 16 rows of 8 heads: 10 us with a
// warp a row, 3 with eight; 4 requests of 8 heads on 2 behind 16384 keys 30.1 to 17.8 us in all).
constexpr int kSplitWarps = 8, kSplitRows = 152 * 3;

// A warp takes a row (W = 1), or W warps do, eight states each in turn.
template <int W>
__global__ void __launch_bounds__(W == 1 ? kMergeWarps * 32 : W * 32, W == 1 ? 7 : 3)
    prefix_merge_kernel(const __grid_constant__ PrefixMergeArgs a) {
  struct Part {
    alignas(16) float o[128];
    float m, sum;
  };
  __shared__ Part part[W == 1 ? 1 : W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = W == 1 ? 0 : warp;
  const int64_t rows = (int64_t)a.total_q * a.num_qo_heads, step = (int64_t)gridDim.x * (W == 1 ? kMergeWarps : 1);
  int64_t row = W == 1 ? (int64_t)blockIdx.x * kMergeWarps + warp : (int64_t)blockIdx.x;
  // where a row's states are: the request's own first
  struct Place {
    int own, pre;        // row in the runs' tiles
    StateRun r0, r1;
  };
  auto place = [&](int64_t r) -> Place {
    Place p{0, 0, {0, 0, 0, 0}, {0, 0, 0, 0}};
    if (r < rows) {
      const int t = (int)(r / a.num_qo_heads), h = (int)(r % a.num_qo_heads), hk = h / a.group, g = h % a.group;
      const TokenStates ts = a.tokens[t];
      const int own = ts.own_row + g, pre = ts.pre_row + g;
      p.own = own % kOwnRows;
      p.r0 = a.runs[ts.own_run + hk * ts.own_tiles + own / kOwnRows];
      if (ts.pre_row >= 0) {
        p.pre = pre % kPrefixRows;
        p.r1 = a.runs[ts.pre_run + hk * ts.pre_tiles + pre / kPrefixRows];
      }
    }
    return p;
  };
  Place now = place(row);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row == 0 && w == 0 && lane == 0) *a.next = 0;   // every piece has been taken
  for (; row < rows; row += step) {
    const int all = now.r0.count + now.r1.count, left = all % (W * kMergeLoads) - w * kMergeLoads;
    const int n = W == 1 ? all : all / (W * kMergeLoads) * kMergeLoads + min(max(left, 0), kMergeLoads);   // this warp's
    auto at = [&](int i) -> int64_t {
      const int k = W == 1 ? i : (i / kMergeLoads * W + w) * kMergeLoads + i % kMergeLoads;
      return k < now.r0.count ? now.r0.base + (int64_t)k * now.r0.rows + now.own
                              : now.r1.base + (int64_t)(k - now.r0.count) * now.r1.rows + now.pre;
    };
    float m = neg_inf(), sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    Place next;
    for (int k0 = 0; k0 < n; k0 += 32) {
      const int end = min(k0 + 32, n);
      // eight states are asked for at once, the first ones together with the LSEs
      float4 v[kMergeLoads];
      auto load = [&](int k) {
#pragma unroll
        for (int i = 0; i < kMergeLoads; ++i)
          if (k + i < end) v[i] = __ldcg(reinterpret_cast<const float4*>(a.ws_o + at(k + i) * 128) + lane);
      };
      load(k0);
      const float l = k0 + lane < n ? __ldcg(a.ws_lse + at(k0 + lane)) : neg_inf();
      float top = l;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, d));
      const float m_new = fmaxf(m, top);
      if (m_new == neg_inf() && !__any_sync(FULL, l != l)) continue;   // no keys so far
      const float keep = m == neg_inf() ? 0.f : ex2(m - m_new);
      m = m_new;
      sum *= keep;
      o.x *= keep;
      o.y *= keep;
      o.z *= keep;
      o.w *= keep;
      const float w = l == neg_inf() ? 0.f : ex2(l - m);
#pragma unroll 1
      for (int k = k0; k < end; k += kMergeLoads) {
        if (k > k0) load(k);
#pragma unroll
        for (int i = 0; i < kMergeLoads; ++i) {
          const float wi = __shfl_sync(FULL, w, (k - k0 + i) & 31);
          if (k + i < end && wi != 0.f) {   // else the state weighs nothing
            sum += wi;
            o.x += wi * v[i].x;
            o.y += wi * v[i].y;
            o.z += wi * v[i].z;
            o.w += wi * v[i].w;
          }
        }
      }
    }
    next = place(row + step);
    if (W > 1) {
      *reinterpret_cast<float4*>(part[w].o + lane * 4) = o;
      if (lane == 0) {
        part[w].m = m;
        part[w].sum = sum;
      }
      __syncthreads();
      if (w == 0) {
#pragma unroll
        for (int i = 1; i < W; ++i) m = fmaxf(m, part[i].m);
        sum = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          // without a maximum a part holds zeros, or NaN that are kept
          const float f = part[i].m != neg_inf() ? ex2(part[i].m - m) : part[i].sum == 0.f ? 0.f : 1.f;
          const float4 v = *reinterpret_cast<const float4*>(part[i].o + lane * 4);
          if (f != 0.f) {
            sum += f * part[i].sum;
            o.x += f * v.x;
            o.y += f * v.y;
            o.z += f * v.z;
            o.w += f * v.w;
          }
        }
      }
      __syncthreads();
      if (w != 0) {
        now = next;
        continue;
      }
    }
    const int h = (int)(row % a.num_qo_heads);
    float denom = sum;
    if (a.sinks != nullptr && m != neg_inf()) denom += ex2(__ldg(a.sinks + h) * kLog2e - m);
    const float f = denom != 0.f ? a.bmm2_scale / denom : 0.f;
    const float r[4] = {o.x, o.y, o.z, o.w};
    store_out<4>(a.out, row * 128 + lane * 4, r, f, a.out_dtype);
    if (a.lse != nullptr && lane == 0) a.lse[row] = sum != 0.f ? m + log2f(sum) : neg_inf();
    now = next;
  }
}

// ---- what the tables hold -----------------------------------------------------------

// A CTA a request.
__global__ void __launch_bounds__(128) prefix_check_kernel(const RowPages* rows, const int32_t* tables,
                                                           int64_t row_stride, const int32_t* seq_lens_live,
                                                           int32_t page_size, int32_t num_pages, int32_t* status) {
  const RowPages r = rows[blockIdx.x];
  int n = r.pages;
  if (seq_lens_live != nullptr) {   // the shared pages are read all the same
    const int live = max(__ldg(seq_lens_live + blockIdx.x), 0);
    n = max(r.shared, min(n, (int)((live + (int64_t)page_size - 1) / page_size)));
  }
  const int32_t* row = tables + (int64_t)blockIdx.x * row_stride;
  const int32_t* first = tables + (int64_t)r.first * row_stride;
  int bad = 0;
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int32_t page = __ldg(row + j);
    if ((uint32_t)page >= (uint32_t)num_pages) bad |= STATUS_PAGE_BOUNDS;
    if (j < r.shared && page != __ldg(first + j)) bad |= STATUS_PREFIX;
  }
  if (bad != 0) atomicOr(status, bad);
}

cudaLaunchConfig_t behind(int64_t grid, int threads, size_t smem, cudaStream_t stream, cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <bool F16, bool NARROW>
int launch_own(const OwnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
  constexpr size_t smem = (size_t)kOwnWarps * kStages * (kMmaUnitBytes + 8);
  auto kern = prefix_own_kernel<F16, NARROW>;
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = set_smem_once(kern, (int)smem, smem_set, true);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(prefix_own)");
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = behind(a.num_ctas, kThreads, smem, stream, &attr);
  e = cudaLaunchKernelEx(&cfg, kern, a, kmap, vmap);
  if (e != cudaSuccess) return cuda_fail(e, "prefix_own_kernel launch");
  return PKA_OK;
}

}  // namespace

int launch_prefix_own(const OwnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
  const bool f16 = a.decode.in_f16 != 0;
  if (a.decode.rows_per_cta <= 8)
    return f16 ? launch_own<true, true>(a, kmap, vmap, stream) : launch_own<false, true>(a, kmap, vmap, stream);
  return f16 ? launch_own<true, false>(a, kmap, vmap, stream) : launch_own<false, false>(a, kmap, vmap, stream);
}

int launch_prefix_merge(const PrefixMergeArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.total_q * a.num_qo_heads;
  cudaLaunchAttribute attr;
  // Few rows of many states get eight warps each: a warp alone reads them eight at a time.
  const bool split = rows <= kSplitRows && a.most_states > kMergeLoads;
  const cudaLaunchConfig_t cfg = split ? behind(rows, kSplitWarps * 32, 0, stream, &attr)
                                       : behind(std::min<int64_t>(ceil_div(rows, kMergeWarps), kMergeCtas),
                                                kMergeWarps * 32, 0, stream, &attr);
  const cudaError_t e = split ? cudaLaunchKernelEx(&cfg, prefix_merge_kernel<kSplitWarps>, a)
                              : cudaLaunchKernelEx(&cfg, prefix_merge_kernel<1>, a);
  if (e != cudaSuccess) return cuda_fail(e, "prefix_merge_kernel launch");
  return PKA_OK;
}

int launch_prefix_check(const RowPages* rows, int32_t batch, const int32_t* tables, int64_t row_stride,
                        const int32_t* seq_lens_live, int32_t page_size, int32_t num_pages, int32_t* status,
                        cudaStream_t stream) {
  prefix_check_kernel<<<batch, 128, 0, stream>>>(rows, tables, row_stride, seq_lens_live, page_size, num_pages, status);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "prefix_check_kernel launch");
  return PKA_OK;
}

}  // namespace pka
