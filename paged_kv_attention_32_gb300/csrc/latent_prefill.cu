// Expanded latent prefill on the 5th-generation tensor cores (tcgen05 + TMEM):
// heads whose key is 128 values of their own and 64 rotary values shared by
// all heads, and whose value is 128 wide.
//
//   s = sm_scale * (q[0..128) . k_nope + q[128..192) . k_rope),  o = softmax(s) v
//
// A pair of CTAs (cta_group::2, one cluster, two SMs) takes 256 query rows of one
// request and head, 128 each, and walks the keys in tiles of 64.  Each CTA holds
// its own queries and only half of every tile: 32 of the keys (half of B's N in
// S = Q K^T) and 64 of the value dimensions (half of N in O += P V).  What bounds
// a single CTA's kernel is the shared-memory port, which the tensor core's
// operands and the incoming copies share: per tile and CTA 48 KB of Q, 24 of K,
// 16 of V and 40 of copies; in a pair 48 + 12 + 8 + 20.  Measured, 2 x 1024 rows
// behind 7168 keys, 32 heads: 261 us with single CTAs, 229 in pairs (1397 TFLOP/s);
// 8 ragged prompts of 512 to 4096: 445 and 441 (256-row tiles compute more beyond the
// diagonal).  A pair's tile takes ~760 cycles an SM, the tensor core's own time at
// N = 64 (12 products of 48 cycles and 4 of 64).
// The shared rotary keys come in by their own tensor map as the third 64-column
// block of a K tile: the concatenated key is never written anywhere.
// Two CTAs of different pairs share an SM (113 KB, 256 TMEM columns each) and hide
// each other's softmax latency.
//   warp 4      TMA producer of this CTA's halves; the tile that holds the last
//               key it clears past it (0 * inf is not 0) before handing it over;
//   warp 5      in the leader, issues every tcgen05.mma for both CTAs:
//               S_b = Q K^T (M=256, N=64, 12 k-steps) into one of two S buffers,
//               two key tiles ahead of the softmax, and O += P V (M=256, N=128,
//               4 k-steps of 16 keys, P from TMEM);
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
constexpr int kQBlocks = 3;                 // 64-column blocks of a query or key row
constexpr uint32_t kQBox = 16384;           // 128 rows x 128 bytes
constexpr uint32_t kKBox = 4096;            // 32 keys x 128 bytes
constexpr uint32_t kKBytes = kQBlocks * kKBox, kVBytes = 8192;   // a CTA's half of a tile
constexpr int kKStages = 3, kVStages = 3;
constexpr int kThreads = 192;
constexpr float kRescaleThreshold = 8.0f;
constexpr uint32_t kColO = 128, kTmemCols = 256;

constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kQBlocks * kQBox;
constexpr uint32_t kOffV = kOffK + kKStages * kKBytes;
constexpr uint32_t kOffBar = kOffV + kVStages * kVBytes;
constexpr size_t kSmemBytes = kOffBar + 256;
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs share an SM");

// mbarriers.  Q, K, V and P are waited for by the leader's MMA warp, on the leader's
// barriers, where both CTAs arrive; the others are signalled in both CTAs by the
// commits.  Parity waits stay correct because every barrier has one waiting role
// that waits for its phases in order; the O-done waits for P V of tile j - 1
// come after S of tile j, issued after P V of tile j - 2.
enum {
  B_Q = 0, B_KFULL = 1, B_KEMPTY = B_KFULL + kKStages, B_VFULL = B_KEMPTY + kKStages,
  B_VEMPTY = B_VFULL + kVStages, B_SFULL = B_VEMPTY + kVStages, B_PFULL = B_SFULL + 2,
  B_ODONE = B_PFULL + 2, B_MMADONE = B_ODONE + 2, B_TAIL = B_MMADONE + 1, B_COUNT = B_TAIL + 1
};
static_assert(B_COUNT * 8 + 4 <= 256, "barriers and the TMEM address slot");

template <bool F16> constexpr uint32_t kIdescQK = idesc_bf16_f32(256, 64, 0, 0, F16);
template <bool F16> constexpr uint32_t kIdescPV = idesc_bf16_f32(256, kDV, 0, 1, F16);

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
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 2)
latent_prefill_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ CUtensorMap tmq,
                      const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmr,
                      const __grid_constant__ CUtensorMap tmv) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + B_COUNT * 8);
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * (uint32_t)i; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();   // 0: the leader
  const PrefillTile tile = a.tiles[blockIdx.x >> 1];
  const int h = tile.head, n_kv = tile.n_kv, kv0 = tile.kv0;
  const int q0 = tile.q0, Lq = tile.lq, k0 = tile.k0, Lk = tile.lk;
  const int row0 = tile.q_tile * 2 * kTileQ + (int)rank * kTileQ;   // this CTA's first query row

  if (tid == 0) {
    mbar_init(bar(B_Q), 2);
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(bar(B_KFULL + s), 2);
      mbar_init(bar(B_KEMPTY + s), 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(bar(B_VFULL + s), 2);
      mbar_init(bar(B_VEMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_SFULL + s), 1);
      mbar_init(bar(B_PFULL + s), 8);   // one arrival per softmax warp of the pair
      mbar_init(bar(B_ODONE + s), 1);
    }
    mbar_init(bar(B_MMADONE), 1);
    mbar_init(bar(B_TAIL), 1);
    fence_barrier_init();
  }
  __syncwarp();
  cluster_arrive();
  if (warp == 5) tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_wait();   // both CTAs' barriers stand before anyone arrives on them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      tma_prefetch_desc(&tmq);
      tma_prefetch_desc(&tmk);
      tma_prefetch_desc(&tmr);
      tma_prefetch_desc(&tmv);
      const uint32_t full = map_to_rank(bar(B_Q), 0);
      mbar_arrive_expect_tx_cluster(full, kQBlocks * kQBox);
      for (int blk = 0; blk < kQBlocks; ++blk)
        tma_load_3d_pair(sbase + kOffQ + (uint32_t)blk * kQBox, &tmq, full, blk * 64, h, q0 + row0);
    }
    __syncwarp();
    RingPos<kKStages> kp;
    RingPos<kVStages> vp;
    auto load_k = [&](int j) -> bool {   // keys 32 rank .. 32 rank + 31 of tile j
      if (j >= kKStages && !warp_wait(bar(B_KEMPTY + kp.slot), kp.parity ^ 1u, a.status)) return false;
      if (lane == 0) {
        const uint32_t dst = sbase + kOffK + (uint32_t)kp.slot * kKBytes;
        const uint32_t full = map_to_rank(bar(B_KFULL + kp.slot), 0);
        const int row = k0 + (kv0 + j) * kTileK + (int)rank * 32;
        mbar_arrive_expect_tx_cluster(full, kKBytes);
        tma_load_3d_pair(dst, &tmk, full, 0, h, row);
        tma_load_3d_pair(dst + kKBox, &tmk, full, 64, h, row);
        tma_load_3d_pair(dst + 2 * kKBox, &tmr, full, 0, 0, row);
      }
      __syncwarp();
      kp.next();
      return true;
    };
    auto load_v = [&](int j) -> bool {   // dimensions 64 rank .. 64 rank + 63 of tile j
      if (j >= kVStages && !warp_wait(bar(B_VEMPTY + vp.slot), vp.parity ^ 1u, a.status)) return false;
      const uint32_t off = kOffV + (uint32_t)vp.slot * kVBytes;
      const uint32_t full = map_to_rank(bar(B_VFULL + vp.slot), 0);
      const int past = (kv0 + j + 1) * kTileK - Lk;   // rows of the tile past the last key
      if (lane == 0) {
        if (past > 0) mbar_arrive_expect_tx(bar(B_TAIL), kVBytes);
        else mbar_arrive_expect_tx_cluster(full, kVBytes);
        tma_load_3d_pair(sbase + off, &tmv, past > 0 ? map_to_rank(bar(B_TAIL), rank) : full,
                         (int)rank * 64, h, k0 + (kv0 + j) * kTileK);
      }
      __syncwarp();
      if (past > 0) {   // the last tile: another request's values, p = 0 there, but 0 * inf is not 0
        if (!warp_wait(bar(B_TAIL), 0, a.status)) return false;
        for (int c = lane; c < past * 8; c += 32)
          *reinterpret_cast<uint4*>(smem + off + (uint32_t)(kTileK - past + (c >> 3)) * 128u +
                                    (uint32_t)(c & 7) * 16u) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(full);
      }
      vp.next();
      return true;
    };
    // order K0 K1 V0 K2 V1 ...: S of tile j + 2 is issued after P V of tile j
    bool ok = true;
    for (int j = 0; ok && j < n_kv + 1; ++j) {
      if (j < n_kv) ok = load_k(j);
      if (ok && j > 0) ok = load_v(j - 1);
    }
    // When a wait gave up, copies still in flight land before the cluster leaves:
    // their barriers may be the other CTA's, so there is only time to go by.
    if (!ok) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 1000000ull) {
      }
    }
  } else if (warp == 5) {
    // ---------------- MMA issuer, the leader's: one elected lane issues for the pair ----
    if (rank == 0) {
      RingPos<kKStages> kp;
      RingPos<kVStages> vp;
      auto issue_qk = [&](int j) -> bool {   // S of tile j into buffer j & 1
        const uint32_t d = tmem + (uint32_t)(j & 1) * 64u;
        if (!warp_wait(bar(B_KFULL + kp.slot), kp.parity, a.status)) return false;
        tc_fence_after();
#pragma unroll
        for (int blk = 0; blk < kQBlocks; ++blk)
          umma_pair_ss_k4(d, smem_desc_sw128(sbase + kOffQ + (uint32_t)blk * kQBox, 16u, 1024u),
                          smem_desc_sw128(sbase + kOffK + (uint32_t)kp.slot * kKBytes + (uint32_t)blk * kKBox,
                                          16u, 1024u),
                          kIdescQK<F16>, blk > 0 ? 1u : 0u);
        umma_pair_commit_elect(bar(B_SFULL + (j & 1)));
        umma_pair_commit_elect(bar(B_KEMPTY + kp.slot));
        kp.next();
        return true;
      };
      bool ok = warp_wait(bar(B_Q), 0, a.status);
      for (int j = 0; ok && j < n_kv && j < 2; ++j) ok = issue_qk(j);
      for (int j = 0; ok && j < n_kv; ++j) {
        const int st = j & 1;
        ok = warp_wait(bar(B_VFULL + vp.slot), vp.parity, a.status) &&
             warp_wait(bar(B_PFULL + st), (uint32_t)((j >> 1) & 1), a.status);
        if (!ok) break;
        tc_fence_after();
        // 4 k-steps of 16 keys: P columns +8, V rows +16 (2048 bytes)
        umma_pair_ts_k4<2048 / 16>(tmem + kColO, tmem + (uint32_t)st * 64u,
                                   smem_desc_sw128(sbase + kOffV + (uint32_t)vp.slot * kVBytes, kVBytes, 1024u),
                                   kIdescPV<F16>, j > 0 ? 1u : 0u);
        umma_pair_commit_elect(bar(B_ODONE + st));
        umma_pair_commit_elect(bar(B_VEMPTY + vp.slot));
        vp.next();
        // S buffer st is free again once this P V has read P (issue order)
        if (j + 2 < n_kv) ok = issue_qk(j + 2);
      }
      umma_pair_commit_elect(bar(B_MMADONE));
    }
    // nothing of the pair's still runs on the tensor cores, and every commit has landed here
    warp_wait(bar(B_MMADONE), 0, a.status);
  } else {
    // ---------------- softmax: one thread per query row ----------------
    const int t = row0 + tid;   // row of the request
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
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(map_to_rank(bar(B_PFULL + st), 0));
    }
    if (ok && n_kv > 0 &&
        warp_wait(bar(B_ODONE + ((n_kv - 1) & 1)), (uint32_t)(((n_kv - 1) >> 1) & 1), a.status)) {
      tc_fence_after();
      // != and not >: a sum that is NaN stays one, in the LSE as in the output
      const float inv = l != 0.f ? a.output_scale / l : 0.f;
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
          const int rr = r0 + lane / 16, tr = row0 + warp * 32 + rr;
          const uint4 val =
              *reinterpret_cast<const uint4*>(wbuf + rr * kRowBytes + ((q ^ (rr & 7)) << 4));
          if (tr < Lq)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) +
                                      ((int64_t)(q0 + tr) * a.num_qo_heads + h) * kRowBytes +
                                      q * 16) = val;
        }
      }
      if (row_valid && a.lse != nullptr)
        a.lse[(int64_t)(q0 + t) * a.num_qo_heads + h] = l != 0.f ? m_ref + log2f(l) : neg_inf();
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA's shared memory nor TMEM goes while the pair still uses it
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
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
  kern<<<2 * args.num_tiles, kThreads, kSmemBytes, stream>>>(args, qmap, kmap, rmap, vmap);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "latent_prefill_kernel launch");
  return PKA_OK;
}

}  // namespace pka
