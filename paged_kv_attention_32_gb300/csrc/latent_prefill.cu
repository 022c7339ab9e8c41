// Expanded latent prefill on the 5th-generation tensor cores (tcgen05 + TMEM):
// heads whose key is 128 values of their own and 64 rotary values shared by
// all heads, and whose value is 128 wide.
//
//   s = sm_scale * (q[0..128) . k_nope + q[128..192) . k_rope),  o = softmax(s) v
//
// One CTA = one 128-row query tile of one request and head, keys in tiles of
// 64, so that two CTAs share an SM and hide each other's softmax latency (two
// heads or two row tiles in one CTA measured slower on the 128-wide prefill).
// The shared rotary keys come in by their own tensor map as the third 64-column
// block of a K tile: the concatenated key is never written anywhere.
// Shared memory for two CTAs per SM is 114 KB each: Q 48 KB, a ring of kKBlocks
// 8 KB key blocks freed one by one as their products finish, and kVStages
// value stages of 16 KB.
//   warp 4      TMA producer;
//   warp 5      issues every tcgen05.mma: S_b = Q K^T (M=128, N=64, 12 k-steps)
//               into one of two S buffers, two key tiles ahead of the softmax,
//               and O += P V (M=128, N=128, 4 k-steps of 16 keys, P from TMEM);
//   warps 0-3   softmax, one thread per query row: lazy rescaling of O only when
//               the row maximum grew by more than 2^8, P in 16 bits over the S
//               buffer (its rounding enters O like the inputs' own; the sum of
//               p is taken in 32 bits before it), final O / l and LSE.
// TMEM columns: S0 [0,64) S1 [64,128) O [128,256).
#include <cuda_bf16.h>

#include "device_common.cuh"
#include "host_common.h"
#include "latent.h"
#include "prefill_softmax.cuh"
#include "tcgen05.cuh"

namespace pka {

using namespace dev;

namespace {

constexpr int kTileQ = 128, kTileK = 64, kDV = 128;
constexpr int kQBlocks = 3, kVBlocks = 2;   // 64-column blocks of a query or key row, of a value
constexpr uint32_t kQBox = 16384;           // 128 rows x 128 bytes
constexpr uint32_t kKBox = 8192;            // 64 rows x 128 bytes
constexpr int kKBlocks = 4, kVStages = 2;
constexpr int kThreads = 192;
constexpr float kRescaleThreshold = 8.0f;
constexpr uint32_t kColO = 128, kTmemCols = 256;

constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kQBlocks * kQBox;
constexpr uint32_t kOffV = kOffK + kKBlocks * kKBox;
constexpr uint32_t kOffBar = kOffV + kVStages * kVBlocks * kKBox;
constexpr size_t kSmemBytes = kOffBar + 256;
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs share an SM");

// mbarriers.  Parity waits stay correct because every barrier has one waiting
// role that waits for its phases in order; the O-done waits for P V of tile
// j - 1 come after S of tile j, issued after P V of tile j - 2.
enum {
  B_Q = 0, B_KFULL = 1, B_KEMPTY = B_KFULL + kKBlocks, B_VFULL = B_KEMPTY + kKBlocks,
  B_VEMPTY = B_VFULL + kVStages, B_SFULL = B_VEMPTY + kVStages, B_PFULL = B_SFULL + 2,
  B_ODONE = B_PFULL + 2, B_MMADONE = B_ODONE + 2, B_COUNT = B_MMADONE + 1
};
static_assert(B_COUNT * 8 + 4 <= 256, "barriers and the TMEM address slot");

template <bool F16> constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 64, 0, 0, F16);
template <bool F16> constexpr uint32_t kIdescPV = idesc_bf16_f32(128, kDV, 0, 1, F16);

// A position in a ring of N slots and the parity of its current round.
template <int N>
struct RingPos {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

template <bool F16>
__global__ void __launch_bounds__(kThreads, 2)
latent_prefill_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ CUtensorMap tmq,
                      const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmr,
                      const __grid_constant__ CUtensorMap tmv) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + B_COUNT * 8);
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * (uint32_t)i; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PrefillTile tile = a.tiles[blockIdx.x];
  const int h = tile.head, n_kv = tile.n_kv, kv0 = tile.kv0;
  const int q0 = tile.q0, Lq = tile.lq, k0 = tile.k0, Lk = tile.lk;

  if (tid == 0) {
    mbar_init(bar(B_Q), 1);
    for (int s = 0; s < kKBlocks; ++s) {
      mbar_init(bar(B_KFULL + s), 1);
      mbar_init(bar(B_KEMPTY + s), 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(bar(B_VFULL + s), 1);
      mbar_init(bar(B_VEMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_SFULL + s), 1);
      mbar_init(bar(B_PFULL + s), 128);
      mbar_init(bar(B_ODONE + s), 1);
    }
    mbar_init(bar(B_MMADONE), 1);
    fence_barrier_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      tma_prefetch_desc(&tmq);
      tma_prefetch_desc(&tmk);
      tma_prefetch_desc(&tmr);
      tma_prefetch_desc(&tmv);
      mbar_arrive_expect_tx(bar(B_Q), kQBlocks * kQBox);
      for (int blk = 0; blk < kQBlocks; ++blk)
        tma_load_3d(sbase + kOffQ + (uint32_t)blk * kQBox, &tmq, bar(B_Q), blk * 64, h,
                    q0 + tile.q_tile * kTileQ);
      RingPos<kKBlocks> kp;
      RingPos<kVStages> vp;
      int kb = 0, vd = 0;   // key blocks and value stages issued
      // an empty barrier's first round is free: wait for the previous round's parity
      auto load_k = [&](int j) -> bool {
        for (int blk = 0; blk < kQBlocks; ++blk) {
          if (kb >= kKBlocks && !mbar_wait(bar(B_KEMPTY + kp.slot), kp.parity ^ 1u, a.status))
            return false;
          const uint32_t dst = sbase + kOffK + (uint32_t)kp.slot * kKBox, full = bar(B_KFULL + kp.slot);
          mbar_arrive_expect_tx(full, kKBox);
          const int row = k0 + (kv0 + j) * kTileK;
          if (blk < 2) tma_load_3d(dst, &tmk, full, blk * 64, h, row);
          else tma_load_3d(dst, &tmr, full, 0, 0, row);
          kp.next();
          ++kb;
        }
        return true;
      };
      auto load_v = [&](int j) -> bool {
        if (vd >= kVStages && !mbar_wait(bar(B_VEMPTY + vp.slot), vp.parity ^ 1u, a.status))
          return false;
        const uint32_t dst = sbase + kOffV + (uint32_t)vp.slot * kVBlocks * kKBox;
        mbar_arrive_expect_tx(bar(B_VFULL + vp.slot), kVBlocks * kKBox);
        for (int blk = 0; blk < kVBlocks; ++blk)
          tma_load_3d(dst + (uint32_t)blk * kKBox, &tmv, bar(B_VFULL + vp.slot), blk * 64, h,
                      k0 + (kv0 + j) * kTileK);
        vp.next();
        ++vd;
        return true;
      };
      // order K0 K1 V0 K2 V1 ...: S of tile j + 2 is issued after P V of tile j
      bool ok = true;
      for (int j = 0; ok && j < n_kv + 1; ++j) {
        if (j < n_kv) ok = load_k(j);
        if (ok && j > 0) ok = load_v(j - 1);
      }
      if (!ok) {   // give the copies already issued a bounded chance to land
        mbar_wait(bar(B_Q), 0, nullptr);
        for (int i = max(0, kb - kKBlocks); i < kb; ++i)
          mbar_wait(bar(B_KFULL + i % kKBlocks), (uint32_t)((i / kKBlocks) & 1), nullptr);
        for (int i = max(0, vd - kVStages); i < vd; ++i)
          mbar_wait(bar(B_VFULL + i % kVStages), (uint32_t)((i / kVStages) & 1), nullptr);
      }
    }
  } else if (warp == 5) {
    // ---------------- MMA issuer: the warp waits, one elected lane issues ----------------
    RingPos<kKBlocks> kp;
    RingPos<kVStages> vp;
    auto issue_qk = [&](int j) -> bool {   // S of tile j into buffer j & 1
      const uint32_t d = tmem + (uint32_t)(j & 1) * 64u;
#pragma unroll
      for (int blk = 0; blk < kQBlocks; ++blk) {
        if (!warp_wait(bar(B_KFULL + kp.slot), kp.parity, a.status)) return false;
        tc_fence_after();
        umma_ss_k4(d, smem_desc_sw128(sbase + kOffQ + (uint32_t)blk * kQBox, 16u, 1024u),
                   smem_desc_sw128(sbase + kOffK + (uint32_t)kp.slot * kKBox, 16u, 1024u),
                   kIdescQK<F16>, blk > 0 ? 1u : 0u);
        umma_commit_elect(bar(B_KEMPTY + kp.slot));
        kp.next();
      }
      umma_commit_elect(bar(B_SFULL + (j & 1)));
      return true;
    };
    bool ok = warp_wait(bar(B_Q), 0, a.status);
    for (int j = 0; ok && j < n_kv && j < 2; ++j) ok = issue_qk(j);
    for (int j = 0; ok && j < n_kv; ++j) {
      const int st = j & 1;
      ok = warp_wait(bar(B_VFULL + vp.slot), vp.parity, a.status) &&
           warp_wait(bar(B_PFULL + st), (uint32_t)((j >> 1) & 1), a.status);
      if (!ok) break;
      const int past = (kv0 + j + 1) * kTileK - Lk;   // rows of the tile past the last key
      if (past > 0) {   // another request's values: p = 0 there, but 0 * inf is not
        uint8_t* v0 = smem + kOffV + (uint32_t)vp.slot * kVBlocks * kKBox;
        for (int c = lane; c < past * 16; c += 32) {
          const int row = kTileK - past + (c >> 4);
          *reinterpret_cast<uint4*>(v0 + (uint32_t)((c >> 3) & 1) * kKBox + row * 128 + (c & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      tc_fence_after();
      const uint32_t vb = sbase + kOffV + (uint32_t)vp.slot * kVBlocks * kKBox;
      // 4 k-steps of 16 keys: P columns +8, V rows +16 (2048 bytes)
      umma_ts_k4<2048 / 16>(tmem + kColO, tmem + (uint32_t)st * 64u,
                            smem_desc_sw128(vb, kKBox, 1024u), kIdescPV<F16>, j > 0 ? 1u : 0u);
      umma_commit_elect(bar(B_ODONE + st));
      umma_commit_elect(bar(B_VEMPTY + vp.slot));
      vp.next();
      // S buffer st is free again once this P V has read P (issue order)
      if (j + 2 < n_kv) ok = issue_qk(j + 2);
    }
    umma_commit_elect(bar(B_MMADONE));
    warp_wait(bar(B_MMADONE), 0, a.status);   // nothing of ours still runs on the tensor core
  } else {
    // ---------------- softmax: one thread per query row ----------------
    const int t = tile.q_tile * kTileQ + tid;   // row of the request
    const bool row_valid = t < Lq;
    const int hi = a.causal ? min(Lk, Lk - Lq + t + 1) : Lk;   // keys [0, hi) visible
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t o_tm = tmem + lane_off + kColO;
    const float sl2 = a.scale_log2;
    float m_ref = neg_inf(), l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_kv; ++j) {
      const int st = j & 1;
      if (!(ok = warp_wait(bar(B_SFULL + st), (uint32_t)((j >> 1) & 1), a.status))) break;
      tc_fence_after();
      const uint32_t s_tm = tmem + lane_off + (uint32_t)st * 64u;
      const int key0 = (kv0 + j) * kTileK;
      const bool masked = __any_sync(0xffffffffu, key0 + kTileK > hi);   // warp-uniform
      uint32_t ra[32], rb[32];
      tmem_ld32(s_tm, ra);
      tmem_ld32(s_tm + 32u, rb);
      tmem_wait_ld();
      reg_fence32(ra);
      reg_fence32(rb);
      uint32_t w0 = 0xffffffffu, w1 = 0xffffffffu;
      if (masked) {
        visible_bits(key0, 0, (unsigned)hi, w0, w1);
        mask_scores64(ra, rb, w0, w1);
      }
      const float mraw = row_max64(ra, rb);
      const float mx = mraw == neg_inf() ? neg_inf() : mraw * sl2;
      const bool grow = mx > m_ref + kRescaleThreshold;
      const float m_new = grow ? mx : m_ref;
      const bool rescale = grow && m_ref != neg_inf();   // else O and l are still zero
      const float alpha = rescale ? ex2(m_ref - m_new) : 1.f;
      if (j > 0 && __any_sync(0xffffffffu, rescale)) {
        // O holds tiles before j: wait for P V of tile j - 1 before rescaling
        if (!(ok = warp_wait(bar(B_ODONE + ((j - 1) & 1)), (uint32_t)(((j - 1) >> 1) & 1),
                             a.status)))
          break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < kDV / 32; ++c) {
          uint32_t r[32];
          tmem_ld32_sync(o_tm + (uint32_t)c * 32u, r);
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
          tmem_st32(o_tm + (uint32_t)c * 32u, r);
        }
        tmem_wait_st();
      }
      m_ref = m_new;
      // A row with no visible key so far keeps m_ref = -inf: exp2(-inf) = 0.
      // Masked scores give 0 through their -inf unless the scale is 0.
      const float neg_m = m_ref == neg_inf() ? 0.f : -m_ref;
      const bool zero_again = masked && !(sl2 > 0.f);
      const float2 sum = zero_again ? exp_tile<true, F16>(ra, rb, sl2, neg_m, w0, w1, s_tm)
                                    : exp_tile<false, F16>(ra, rb, sl2, neg_m, w0, w1, s_tm);
      tmem_wait_st();
      l = l * alpha + (sum.x + sum.y);
      tc_fence_before();
      mbar_arrive(bar(B_PFULL + st));
    }
    if (ok && n_kv > 0 &&
        warp_wait(bar(B_ODONE + ((n_kv - 1) & 1)), (uint32_t)(((n_kv - 1) >> 1) & 1), a.status)) {
      tc_fence_after();
      const float inv = l > 0.f ? a.output_scale / l : 0.f;
      if (a.out_dtype == PKA_DTYPE_F32) {
        const int64_t dst = ((int64_t)(q0 + t) * a.num_qo_heads + h) * kDV;
#pragma unroll 1
        for (int c = 0; c < kDV / 32; ++c) {
          uint32_t r[32];
          tmem_ld32_sync(o_tm + (uint32_t)c * 32u, r);
          if (row_valid) {
#pragma unroll
            for (int qd = 0; qd < 2; ++qd) {
              float f[16];
#pragma unroll
              for (int x = 0; x < 16; ++x) f[x] = __uint_as_float(r[16 * qd + x]);
              store_out<16>(a.out, dst + c * 32 + qd * 16, f, inv, a.out_dtype);
            }
          }
        }
      } else {
        // each warp stages its 32 rows in the Q buffer (every QK has completed),
        // 16-byte chunks XOR-swizzled by row, then writes whole 256-byte rows
        constexpr int kRowBytes = kDV * 2;
        uint8_t* wbuf = smem + kOffQ + (uint32_t)warp * 32u * kRowBytes;
        const bool f16o = a.out_dtype == PKA_DTYPE_F16;
#pragma unroll 1
        for (int c = 0; c < kDV / 32; ++c) {
          uint32_t r[32];
          tmem_ld32_sync(o_tm + (uint32_t)c * 32u, r);
#pragma unroll
          for (int k = 0; k < 4; ++k) {   // 8 values = one 16-byte chunk
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float lo = __uint_as_float(r[8 * k + 2 * x]) * inv;
              const float hi2 = __uint_as_float(r[8 * k + 2 * x + 1]) * inv;
              w[x] = f16o ? pack2<true>(lo, hi2) : pack2<false>(lo, hi2);
            }
            *reinterpret_cast<uint4*>(wbuf + lane * kRowBytes + (((c * 4 + k) ^ (lane & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
        const int q = lane % 16;
#pragma unroll 4
        for (int r0 = 0; r0 < 32; r0 += 2) {
          const int rr = r0 + lane / 16, tr = tile.q_tile * kTileQ + warp * 32 + rr;
          const uint4 val =
              *reinterpret_cast<const uint4*>(wbuf + rr * kRowBytes + ((q ^ (rr & 7)) << 4));
          if (tr < Lq)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) +
                                      ((int64_t)(q0 + tr) * a.num_qo_heads + h) * kRowBytes +
                                      q * 16) = val;
        }
      }
      if (row_valid && a.lse != nullptr)
        a.lse[(int64_t)(q0 + t) * a.num_qo_heads + h] = l > 0.f ? m_ref + log2f(l) : neg_inf();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

int launch_latent_prefill(const pka_prefill_plan& plan, const PrefillArgs& args,
                          const CUtensorMap& qmap, const CUtensorMap& kmap,
                          const CUtensorMap& rmap, const CUtensorMap& vmap, cudaStream_t stream) {
  if (args.num_tiles == 0) return PKA_OK;
  const bool f16 = plan.desc.dtype == PKA_DTYPE_F16;
  auto kern = f16 ? latent_prefill_kernel<true> : latent_prefill_kernel<false>;
  static std::atomic<uint64_t> smem_set[2];   // per input type: devices whose limit was raised
  cudaError_t e = set_smem_once(kern, (int)kSmemBytes, smem_set[f16]);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(latent_prefill)");
  kern<<<args.num_tiles, kThreads, kSmemBytes, stream>>>(args, qmap, kmap, rmap, vmap);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "latent_prefill_kernel launch");
  return PKA_OK;
}

}  // namespace pka
