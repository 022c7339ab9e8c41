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
// 16 of V and 40 of copies; in a pair 48 + 12 + 8 + 20.  The shared rotary keys come
// in by their own tensor map as the third 64-column block of a K tile: the
// concatenated key is never written anywhere.  Two CTAs of different pairs share an
// SM (113 KB, 256 TMEM columns each) and hide each other's softmax latency.
// The host deals the tiles of 256 rows out to one wave of pairs, which take theirs in
// turn, the next one's queries and keys copied while the last one ends; a tile that
// fills a pair's share is cut there, along its keys, and its pieces are merged.
//
// Measured: 152 tiles of 2048 x 8192 keys 0.84 us a key tile and two pairs of an SM, as
// many products a second as the library's bf16 product reaches (1890 TFLOP/s): the
// tensor core bounds it.  2 x 1024 rows behind 7168 keys, 32 heads: 261 us with single
// CTAs, 225 in pairs that took one tile each, 212 dealt out; 8 ragged prompts of 512 to
// 4096: 445, 437, 400 (15 % of whose products lie beyond the diagonal); 4 prompts of
// 512, 128 heads: 66 us, where the ends of the tiles count (74 with 16-byte stores).
// Not kept: tiles of 128 keys, whose scores take a sixth less of the tensor core's
// time but leave one S buffer: 232 and 475 us where tiles of 64 then took 225 and 437.
//   warp 4      TMA producer of this CTA's halves; the tile that holds the last
//               key it clears past it (0 * inf is not 0) before handing it over;
//   warp 5      in the leader, issues every tcgen05.mma for both CTAs:
//               S_b = Q K^T (M=256, N=64, 12 k-steps) into one of two S buffers,
//               two key tiles ahead of the softmax, and O += P V (M=256, N=128,
//               4 k-steps of 16 keys, P from TMEM);
//   warps 0-3   softmax, one thread per query row: lazy rescaling of O only when
//               the row maximum grew by more than 2^8, P in 16 bits over the S
//               buffer (its rounding enters O like the inputs' own; the sum of p is
//               taken in 32 bits before it), final O / l and LSE.
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

// mbarriers.  Q, K, V, P and O-free are waited for by the leader's MMA warp, on the
// leader's barriers, where both CTAs arrive; the others are signalled in both CTAs by
// the commits.  T counts a pair's key tiles over all its items: S, P and O barriers
// T & 1.  No barrier runs a phase past one that somebody still has to see: S(T) is
// issued behind P V(T - 2), P(T) written once S(T) is complete, the next item's Q
// copied once this one's last S is complete and its first P V issued once O is free.
enum {
  B_QFULL = 0, B_QFREE, B_OFREE, B_KFULL, B_KEMPTY = B_KFULL + kKStages, B_VFULL = B_KEMPTY + kKStages,
  B_VEMPTY = B_VFULL + kVStages, B_SFULL = B_VEMPTY + kVStages, B_PFULL = B_SFULL + 2,
  B_ODONE = B_PFULL + 2, B_MMADONE = B_ODONE + 2, B_TAIL, B_COUNT
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

// 32 bytes by one store, or by two where the address is 16-byte aligned only.
__device__ __forceinline__ void store_sector(void* dst, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <bool F16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 2)
latent_prefill_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ LatentPrefillParts parts,
                      const __grid_constant__ CUtensorMap tmq,
                      const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmr,
                      const __grid_constant__ CUtensorMap tmv) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + B_COUNT * 8);
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * (uint32_t)i; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();   // 0: the leader
  const int pair = blockIdx.x >> 1;

  if (tid == 0) {   // the first tile comes in while the pair sets up
    ask_line(a.tiles + pair);
    ask_line(parts.segments + pair);
    mbar_init(bar(B_QFULL), 2);
    mbar_init(bar(B_QFREE), 1);
    mbar_init(bar(B_OFREE), 8);
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

  // the merge's CTAs may start taking free SMs; they wait for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // The pair's first tile lies at its own index, so that its loads need not wait for
  // the list's; the others one behind the other from more0 on.
  const int more0 = __ldg(parts.segments + pair);
  const int n_items = 1 + __ldg(parts.segments + pair + 1) - more0;
  auto index = [&](int k) -> int { return k == 0 ? pair : more0 + k - 1; };

  if (warp == 4) {
    // ---------------- TMA producer ----------------
    if (lane < 4) tma_prefetch_desc(lane == 0 ? &tmq : lane == 1 ? &tmk : lane == 2 ? &tmr : &tmv);
    RingPos<kKStages> kp;
    RingPos<kVStages> vp;
    int nk = 0, nv = 0, tails = 0;   // stages filled so far, cleared tiles
    bool ok = true;
    PrefillTile tile = a.tiles[pair];
    for (int i = 0; ok && i < n_items; ++i) {
      const PrefillTile next = a.tiles[i + 1 < n_items ? index(i + 1) : pair];
      const int h = tile.head, n_kv = tile.n_kv, key_tile0 = tile.kv0, Lk = tile.lk;
      const int row0 = tile.q0 + (tile.q_tile * 2 + (int)rank) * kTileQ;   // this CTA's first query row
      auto load_q = [&]() -> bool {
        if (i > 0 && !warp_wait(bar(B_QFREE), (uint32_t)((i - 1) & 1), a.status)) return false;
        if (lane == 0) {
          const uint32_t full = map_to_rank(bar(B_QFULL), 0);
          mbar_arrive_expect_tx_cluster(full, kQBlocks * kQBox);
          for (int blk = 0; blk < kQBlocks; ++blk)
            tma_load_3d_pair(sbase + kOffQ + (uint32_t)blk * kQBox, &tmq, full, blk * 64, h, row0);
        }
        __syncwarp();
        return true;
      };
      auto load_k = [&](int j) -> bool {   // keys 32 rank .. 32 rank + 31 of tile j
        if (nk >= kKStages && !warp_wait(bar(B_KEMPTY + kp.slot), kp.parity ^ 1u, a.status)) return false;
        if (lane == 0) {
          const uint32_t dst = sbase + kOffK + (uint32_t)kp.slot * kKBytes;
          const uint32_t full = map_to_rank(bar(B_KFULL + kp.slot), 0);
          const int row = tile.k0 + (key_tile0 + j) * kTileK + (int)rank * 32;
          mbar_arrive_expect_tx_cluster(full, kKBytes);
          tma_load_3d_pair(dst, &tmk, full, 0, h, row);
          tma_load_3d_pair(dst + kKBox, &tmk, full, 64, h, row);
          tma_load_3d_pair(dst + 2 * kKBox, &tmr, full, 0, 0, row);
        }
        __syncwarp();
        kp.next();
        ++nk;
        return true;
      };
      auto load_v = [&](int j) -> bool {   // dimensions 64 rank .. 64 rank + 63 of tile j
        if (nv >= kVStages && !warp_wait(bar(B_VEMPTY + vp.slot), vp.parity ^ 1u, a.status)) return false;
        const uint32_t off = kOffV + (uint32_t)vp.slot * kVBytes;
        const uint32_t full = map_to_rank(bar(B_VFULL + vp.slot), 0);
        const int past = (key_tile0 + j + 1) * kTileK - Lk;   // rows of the tile past the last key
        if (lane == 0) {
          if (past > 0) mbar_arrive_expect_tx(bar(B_TAIL), kVBytes);
          else mbar_arrive_expect_tx_cluster(full, kVBytes);
          tma_load_3d_pair(sbase + off, &tmv, past > 0 ? map_to_rank(bar(B_TAIL), rank) : full,
                           (int)rank * 64, h, tile.k0 + (key_tile0 + j) * kTileK);
        }
        __syncwarp();
        if (past > 0) {   // a last tile: another request's values, p = 0 there, but 0 * inf is not 0
          if (!warp_wait(bar(B_TAIL), (uint32_t)(tails++ & 1), a.status)) return false;
          for (int c = lane; c < past * 8; c += 32)
            *reinterpret_cast<uint4*>(smem + off + (uint32_t)(kTileK - past + (c >> 3)) * 128u +
                                      (uint32_t)(c & 7) * 16u) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(full);
        }
        vp.next();
        ++nv;
        return true;
      };
      // order K0 Q K1 V0 K2 V1 ...: S of tile j + 2 is issued after P V of tile j
      for (int j = 0; ok && j < n_kv + 1; ++j) {
        if (j < n_kv) ok = load_k(j);
        if (ok && j == 0) ok = load_q();
        if (ok && j > 0) ok = load_v(j - 1);
      }
      tile = next;
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
      int T = 0;   // key tiles before this one
      bool ok = true;
      int n_kv = __ldg(&a.tiles[pair].n_kv);
      for (int i = 0; ok && i < n_items; ++i) {
        const int next_n = __ldg(&a.tiles[i + 1 < n_items ? index(i + 1) : pair].n_kv);
        auto issue_qk = [&](int j) -> bool {   // S of tile j into buffer (T + j) & 1
          if (!warp_wait(bar(B_KFULL + kp.slot), kp.parity, a.status)) return false;
          tc_fence_after();
          const int st = (T + j) & 1;
#pragma unroll
          for (int blk = 0; blk < kQBlocks; ++blk)
            umma_pair_ss_k4(tmem + (uint32_t)st * 64u,
                            smem_desc_sw128(sbase + kOffQ + (uint32_t)blk * kQBox, 16u, 1024u),
                            smem_desc_sw128(sbase + kOffK + (uint32_t)kp.slot * kKBytes + (uint32_t)blk * kKBox,
                                            16u, 1024u),
                            kIdescQK<F16>, blk > 0 ? 1u : 0u);
          umma_pair_commit_elect(bar(B_SFULL + st));
          umma_pair_commit_elect(bar(B_KEMPTY + kp.slot));
          if (j == n_kv - 1) umma_pair_commit_elect(bar(B_QFREE));
          kp.next();
          return true;
        };
        ok = warp_wait(bar(B_QFULL), (uint32_t)(i & 1), a.status);
        for (int j = 0; ok && j < n_kv && j < 2; ++j) ok = issue_qk(j);
        for (int j = 0; ok && j < n_kv; ++j) {
          const int st = (T + j) & 1;
          // cleared values: ordinary writes, of the other CTA too; P is in tensor memory
          ok = warp_wait<true>(bar(B_VFULL + vp.slot), vp.parity, a.status) &&
               warp_wait(bar(B_PFULL + st), (uint32_t)(((T + j) >> 1) & 1), a.status);
          if (ok && j == 0 && i > 0) ok = warp_wait(bar(B_OFREE), (uint32_t)((i - 1) & 1), a.status);
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
        T += n_kv;
        n_kv = next_n;
      }
      umma_pair_commit_elect(bar(B_MMADONE));
    }
  } else {
    // ---------------- softmax: one thread per query row ----------------
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t o_tm = tmem + lane_off + kColO;
    const float sl2 = a.scale_log2;
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    int T = 0;   // key tiles before this one
    bool ok = true;
    PrefillTile tile = a.tiles[pair];
    int part = __ldg(parts.part + pair);
    for (int i = 0; ok && i < n_items; ++i) {
      const int after = i + 1 < n_items ? index(i + 1) : pair;
      const PrefillTile next = a.tiles[after];
      const int next_part = __ldg(parts.part + after), n_kv = tile.n_kv;
      const int r = (int)rank * kTileQ + tid;                // row of the tile
      const int t = tile.q_tile * 2 * kTileQ + r;            // row of the request
      const int hi = a.causal ? min(tile.lk, tile.lk - tile.lq + t + 1) : tile.lk;   // keys [0, hi) visible
      float m_ref = neg_inf(), l = 0.f;
      for (int j = 0; j < n_kv; ++j, ++T) {
        const int st = T & 1;
        if (!(ok = warp_wait(bar(B_SFULL + st), (uint32_t)((T >> 1) & 1), a.status))) break;
        tc_fence_after();
        const uint32_t s_tm = tmem + lane_off + (uint32_t)st * 64u;
        const int key0 = (tile.kv0 + j) * kTileK;
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
          // O holds the tiles before: wait for P V of the last of them before rescaling
          if (!(ok = warp_wait(bar(B_ODONE + (st ^ 1)), (uint32_t)(((T - 1) >> 1) & 1), a.status))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kDV / 32; ++c) {
            uint32_t o[32];
            tmem_ld32_sync(o_tm + (uint32_t)c * 32u, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(o_tm + (uint32_t)c * 32u, o);
          }
          tmem_wait_st();
        }
        m_ref = m_new;
        // A row with no visible key so far keeps m_ref = -inf: exp2(-inf) = 0.
        // Masked scores give 0 through their -inf unless the scale is 0.
        const float neg_m = m_ref == neg_inf() ? 0.f : kLatentWeightShift<F16> - m_ref;
        const bool zero_again = masked && !(sl2 > 0.f);
        const float2 sum = zero_again ? exp_tile<true, F16>(ra, rb, sl2, neg_m, w0, w1, s_tm)
                                      : exp_tile<false, F16>(ra, rb, sl2, neg_m, w0, w1, s_tm);
        tmem_wait_st();
        l = l * alpha + (sum.x + sum.y);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(map_to_rank(bar(B_PFULL + st), 0));
      }
      if (!ok || !(ok = warp_wait(bar(B_ODONE + ((T - 1) & 1)), (uint32_t)(((T - 1) >> 1) & 1), a.status))) break;
      tc_fence_after();
      // != and not >: a sum that is NaN stays one, in the LSE as in the output
      const float inv = l != 0.f ? (part < 0 ? a.output_scale : 1.f) / l : 0.f;
      const float lse = l != 0.f ? m_ref - kLatentWeightShift<F16> + log2f(l) : neg_inf();
      const bool row_valid = t < tile.lq;
      const int64_t orow = (int64_t)(tile.q0 + t) * a.num_qo_heads + tile.head;
      // Whole 32-byte sectors, one a store and lane.  A partial state is kept as blocks of
      // 8 dimensions of all its rows, so that a warp's sectors are one run of 1 KB.
#pragma unroll 1
      for (int c = 0; c < kDV; c += 32) {
        uint32_t o[32];
        __syncwarp();   // the lanes whose rows are stored and the others load together
        tmem_ld32_sync(o_tm + (uint32_t)c, o);
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * inv);
        if (row_valid && part >= 0) {
          float* dst = parts.ws_o + ((int64_t)part * kDV + c) * (2 * kTileQ) + r * 8;
#pragma unroll
          for (int k = 0; k < 4; ++k) store_sector(dst + k * 8 * (2 * kTileQ), o + 8 * k, true);
        } else if (row_valid && a.out_dtype == PKA_DTYPE_F32) {
          float* dst = static_cast<float*>(a.out) + orow * kDV + c;
#pragma unroll
          for (int k = 0; k < 4; ++k) store_sector(dst + 8 * k, o + 8 * k, wide);
        } else if (row_valid) {
          uint16_t* dst = static_cast<uint16_t*>(a.out) + orow * kDV + c;
          uint32_t w[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float lo = __uint_as_float(o[2 * x]), up = __uint_as_float(o[2 * x + 1]);
            w[x] = a.out_dtype == PKA_DTYPE_F16 ? pack2<true>(lo, up) : pack2<false>(lo, up);
          }
          store_sector(dst, w, wide);
          store_sector(dst + 16, w + 8, wide);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(map_to_rank(bar(B_OFREE), 0));
      if (row_valid) {
        if (part >= 0) parts.ws_lse[(int64_t)part * (2 * kTileQ) + r] = lse;
        else if (a.lse != nullptr) a.lse[orow] = lse;
      }
      tile = next;
      part = next_part;
    }
  }

  tc_fence_before();
  __syncthreads();
  // Nothing of the pair's still runs on the tensor cores, and every commit has landed here.
  // Waited for only now: all of a pair's tiles may take longer than any one wait may.
  if (warp == 5) warp_wait(bar(B_MMADONE), 0, a.status);
  cluster_sync();   // neither CTA's shared memory nor TMEM goes while the pair still uses it
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// The pieces of the tiles that were cut: out = sum_c w_c o_c / sum_c w_c with
// w_c = 2^(lse_c - max).  A warp takes four rows: eight lanes read 128 bytes, 8
// dimensions of all four, and a row belongs to the eight lanes with its (lane / 2) % 4,
// 16 dimensions each.  Launched while the prefill still runs, it waits for that grid's
// end.
constexpr int kMergeWarps = 4, kMergeRows = 4 * kMergeWarps;
__global__ void __launch_bounds__(kMergeWarps * 32)
latent_prefill_merge_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ LatentPrefillParts parts) {
  constexpr int kCtas = 2 * kTileQ / kMergeRows;
  const int lane = threadIdx.x & 31, half = lane & 1, quarter = lane >> 3;
  const int r = (int)(blockIdx.x % kCtas) * kMergeRows + (threadIdx.x >> 5) * 4 + ((lane >> 1) & 3);
  const LatentPrefillCut cut = parts.cuts[blockIdx.x / kCtas];
  const int t = cut.q_tile * 2 * kTileQ + r;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (t - ((lane >> 1) & 3) >= cut.lq) return;   // none of the warp's rows
  const float* lse = parts.ws_lse + (int64_t)cut.part0 * (2 * kTileQ) + r;
  const float* src = parts.ws_o + ((int64_t)cut.part0 * kDV + quarter * 8) * (2 * kTileQ) + r * 8 + half * 4;
  const bool live = t < cut.lq;   // rows past the request's last were never written
  float m = neg_inf(), sum = 0.f;
  if (live)
    for (int c = quarter * 2 + half; c < cut.n_parts; c += 8) m = fmaxf(m, __ldcg(lse + (int64_t)c * (2 * kTileQ)));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
  if (!live) return;
  float o[4][4] = {};   // dimensions 32 i + 8 quarter + 4 half on
  // two pieces are asked for at once
  for (int c0 = 0; c0 < cut.n_parts; c0 += 2) {
    float x[2];
    float4 v[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x[k] = neg_inf();
      if (c0 + k < cut.n_parts) {
        x[k] = __ldcg(lse + (int64_t)(c0 + k) * (2 * kTileQ));
        const float* p = src + (int64_t)(c0 + k) * kDV * (2 * kTileQ);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k][i] = __ldcg(reinterpret_cast<const float4*>(p + i * 32 * (2 * kTileQ)));
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (x[k] != neg_inf()) {   // else the piece weighs nothing
        const float w = ex2(x[k] - m);
        sum += w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[i][0] += w * v[k][i].x;
          o[i][1] += w * v[k][i].y;
          o[i][2] += w * v[k][i].z;
          o[i][3] += w * v[k][i].w;
        }
      }
  }
  const int64_t row = (int64_t)(cut.q0 + t) * a.num_qo_heads + cut.head;
  const float f = sum != 0.f ? a.output_scale / sum : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    store_out<4>(a.out, row * kDV + i * 32 + quarter * 8 + half * 4, o[i], f, a.out_dtype);
  if (quarter * 2 + half == 0 && a.lse != nullptr) a.lse[row] = sum != 0.f ? m + log2f(sum) : neg_inf();
}

}  // namespace

int launch_latent_prefill(const pka_prefill_plan& plan, const PrefillArgs& args, const LatentPrefillParts& parts,
                          const CUtensorMap& qmap, const CUtensorMap& kmap,
                          const CUtensorMap& rmap, const CUtensorMap& vmap, cudaStream_t stream) {
  const bool f16 = plan.desc.dtype == PKA_DTYPE_F16;
  auto kern = f16 ? latent_prefill_kernel<true> : latent_prefill_kernel<false>;
  static std::atomic<uint64_t> smem_set[2];   // per input type: devices whose limit was raised
  cudaError_t e = set_smem_once(kern, (int)kSmemBytes, smem_set[f16]);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(latent_prefill)");
  kern<<<2 * parts.num_segments, kThreads, kSmemBytes, stream>>>(args, parts, qmap, kmap, rmap, vmap);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "latent_prefill_kernel launch");
  if (parts.num_cuts > 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)parts.num_cuts * (2 * kTileQ / kMergeRows));
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, latent_prefill_merge_kernel, args, parts);
    if (e != cudaSuccess) return cuda_fail(e, "latent_prefill_merge_kernel launch");
  }
  return PKA_OK;
}

}  // namespace pka
