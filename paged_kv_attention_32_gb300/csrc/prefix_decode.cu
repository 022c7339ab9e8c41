// Attention of many query rows over one shared, paged prefix, on the 5th-generation
// tensor cores (tcgen05 + TMEM): the part of a decode that its requests have in common.
//
// For the rows r = (token, head of the KV head's group) of a group of requests and the
// prefix's keys j of one piece
//   s_j = scale * q_r . k_j,  m = max s, l = sum exp(s - m),  o = sum exp(s - m) v / l,
// stored as a 32-bit partial state (o and the base-2 LSE) that the merge kernel joins with
// the states of the requests' own keys.  Every row sees the whole prefix, so the only
// mask is the piece's end.
//
// A pair of CTAs (cta_group::2, one cluster, two SMs) takes 256 rows, 128 each, and walks the
// keys in tiles of 64.  Each CTA holds its own queries and only half of every tile: 32 of the
// keys (half of B's N in S = Q K^T) and 64 of the value dimensions (half of N in O += P V),
// which halves what the shared-memory port moves for K and V and the copies.  The host deals
// the work out evenly to one wave of pairs, which take their pieces in turn, the next one's
// queries and keys copied while the last one ends.
//   softmax     groups of four warps: gather the query rows (any token and head strides, any
//               group size), then one thread per row: O rescaled only when the row maximum grew
//               by more than 2^8, P in 16 bits over the S buffer (its rounding enters O like
//               the inputs' own; the sum of p is taken in 32 bits before it);
//   one warp    copies this CTA's half of the keys, page by page (TMA);
//   one warp    the leader's issues every tcgen05.mma for both CTAs: S_b (M=256, N=64, 8
//               k-steps) into a ring of S buffers, and O += P V (M=256, N=128, 4 k-steps of
//               16 keys, P from TMEM);
//   one warp    copies this CTA's half of the values.
// Two shapes.  DENSE, where the products bound the whole: two CTAs of different pairs share an
// SM and hide each other's softmax, with two S buffers each.  Else, where memory does: one
// CTA an SM with four S buffers, beside a CTA of the kernel over the requests' own keys, so
// that both read at once; two softmax groups take the tiles in turn, each with its own maximum,
// sum and O, joined at a piece's end (with one group 4 requests of 32 heads on 8 behind 16384
// keys 34.8 us in all, 64 behind 4096 32.3; with two 32.8 and 29.8).
// Measured: DENSE, 65536 keys and 1024 rows of 8 heads, 275 GFLOP: 177 to 200 us from the first
// CTA to the last, 1380 to 1550 TFLOP/s.  Softmax and tensor core bound it together: of the 8
// softmax warps of an SM each waits for its S while the others' exponentials run, and the
// tensor pipe is busy half the time at a quarter of the keys.  Else, 8192 keys and 256 rows of
// 8 heads, 34 MB, beside the other kernel's 137: 20 to 24 us (24 to 28 with one softmax group),
// both 33, 5.2 TB/s.
// Not kept, the first case: one CTA an SM with two row tiles and one issuing warp 212 us, the
// same with two threads a row 240.
#include <cuda_bf16.h>

#include "device_common.cuh"
#include "host_common.h"
#include "latent.h"
#include "prefill_softmax.cuh"
#include "prefix.h"
#include "tcgen05.cuh"

namespace pka {

using namespace dev;

namespace {

constexpr int kTileQ = 128, kTileK = kPrefixTile, kD = 128;
constexpr uint32_t kQBox = 16384;           // 128 rows x 128 bytes
constexpr uint32_t kKBox = 4096;            // 32 keys x 128 bytes
constexpr uint32_t kKBytes = 2 * kKBox, kVBytes = 8192;   // a CTA's half of a tile
constexpr float kRescaleThreshold = 8.0f;

template <bool DENSE>
struct Geo {
  static constexpr int kStages = DENSE ? 5 : 7, kScores = DENSE ? 2 : 4;
  // groups of four softmax warps that take the tiles of a piece in turn, each with its own O
  static constexpr int kGroups = DENSE ? 1 : 2, kSoft = 4 * kGroups, kThreads = (kSoft + 3) * 32;
  static constexpr int kRegs = DENSE ? 128 : 112;   // 112: a CTA of the own keys' kernel fits beside
  static constexpr uint32_t kOffK = 2 * kQBox, kOffV = kOffK + kStages * kKBytes;
  static constexpr uint32_t kOffBar = kOffV + kStages * kVBytes;
  static constexpr uint32_t kOffSums = kOffBar + 512;   // each group's maximum and sum of every row
  static constexpr size_t kSmemBytes = kOffSums + (kGroups > 1 ? kGroups * kTileQ * 8 : 0);
  static constexpr uint32_t kColO = kScores * 64, kTmemCols = kColO + kGroups * kD <= 256 ? 256 : 512;
  // Q, K, V, P and O-free are waited for by the leader's MMA warp, on the leader's barriers,
  // where both CTAs arrive; the others are signalled in both CTAs by the commits.  T counts a
  // pair's key tiles over all its pieces: S, P and O barriers T % kScores.  No barrier runs a
  // phase past one that somebody still has to see: S(T) is issued behind P V(T - kScores), P(T)
  // written once S(T) is complete, the next piece's Q written once this one's last S is
  // complete and its first P V issued once O is free.
  static constexpr int kQFull = 0, kOFree = 1, kMmaDone = 2, kKFull = 3, kKEmpty = kKFull + kStages,
                       kVFull = kKEmpty + kStages, kVEmpty = kVFull + kStages, kSFull = kVEmpty + kStages,
                       kPFull = kSFull + kScores, kODone = kPFull + kScores, kCount = kODone + kScores;
  static_assert(kCount * 8 + 4 <= 512, "barriers and the TMEM address slot");
};
static_assert(2 * (Geo<true>::kSmemBytes + 1024) <= 228 * 1024, "two CTAs share an SM");
// All of an SM's tensor memory: no CTA of another pair may wait for it beside one that waits for
// its own other half elsewhere.
static_assert(Geo<false>::kTmemCols == 512 && Geo<false>::kSmemBytes + Geo<true>::kSmemBytes > 228 * 1024,
              "no pair's CTA beside this one");

template <bool F16> constexpr uint32_t kIdescQK = idesc_bf16_f32(256, 64, 0, 0, F16);
template <bool F16> constexpr uint32_t kIdescPV = idesc_bf16_f32(256, kD, 0, 1, F16);

// A position in a ring of N and the parity of its current round.
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

__device__ __forceinline__ void store_sector(float* dst, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Waits at named barrier ID for its N threads; whether all of them are well.
template <int ID, int N>
__device__ __forceinline__ bool all_meet(bool well) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.and.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)well), "n"(ID), "n"(N)
      : "memory");
  return all != 0u;
}

template <bool F16, bool DENSE>
__global__ void __cluster_dims__(2, 1, 1) __maxnreg__(Geo<DENSE>::kRegs)
prefix_kernel(const __grid_constant__ PrefixArgs a, const __grid_constant__ CUtensorMap tmk,
              const __grid_constant__ CUtensorMap tmv) {
  using Gm = Geo<DENSE>;
  constexpr int kStages = Gm::kStages, kScores = Gm::kScores, kGroups = Gm::kGroups, kSoft = Gm::kSoft;
  constexpr uint32_t kOffK = Gm::kOffK, kOffV = Gm::kOffV;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Gm::kOffBar + Gm::kCount * 8);
  auto bar = [&](int i) -> uint32_t { return sbase + Gm::kOffBar + 8u * (uint32_t)i; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();   // 0: the leader
  const int pair = blockIdx.x >> 1;
  // the other kernel's CTAs may start; the merge behind it waits for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // A pair's first piece lies at its own index, so that its loads need not wait for the
  // list's; the others one behind the other from more0 on.
  const int mine = (int)rank * kTileQ + (tid & (kTileQ - 1));   // softmax: the thread's row of a piece
  const int group = kGroups > 1 ? warp >> 2 : 0, rows4 = (warp & 3) * 32;   // softmax: its group, its first row of the CTA's
  constexpr int kAsk = 16 / kGroups;   // rows that a lane brings 16 bytes of
  uint4 rows[kAsk];
  // asks for the query rows of a piece, the groups' warps for a part each, two rows at a time, 16 lanes
  // a row; zeros where there is none
  auto ask_rows = [&](int i) {
    const PrefixItem it = a.items[i];
    const int r = it.row0 + mine;
    const int64_t src = r < it.rows ? (int64_t)(it.q_start + r / a.group) * a.q_stride_tok +
                                          (int64_t)(it.kv_head * a.group + r % a.group) * a.q_stride_head
                                    : -1;
#pragma unroll
    for (int k = 0; k < kAsk; ++k) {
      const int64_t at = __shfl_sync(0xffffffffu, src, 2 * (group * kAsk + k) + (lane >> 4));
      rows[k] = make_uint4(0u, 0u, 0u, 0u);
      if (at >= 0) rows[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at) + (lane & 15));
    }
  };
  // The first ones before anything else: behind the first keys and values of all CTAs they
  // would wait 5 us for memory.
  if (warp < kSoft) ask_rows(pair);
  if (tid == 0) {   // the list comes in while the pair sets up
    ask_line(a.more + pair);
    mbar_init(bar(Gm::kQFull), 2 * kSoft);   // the pair's softmax warps
    mbar_init(bar(Gm::kOFree), 2 * kSoft);
    mbar_init(bar(Gm::kMmaDone), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(Gm::kKFull + s), 2);
      mbar_init(bar(Gm::kKEmpty + s), 1);
      mbar_init(bar(Gm::kVFull + s), 2);
      mbar_init(bar(Gm::kVEmpty + s), 1);
    }
    for (int s = 0; s < kScores; ++s) {
      mbar_init(bar(Gm::kSFull + s), 1);
      mbar_init(bar(Gm::kPFull + s), 8);   // of one group
      mbar_init(bar(Gm::kODone + s), 1);
    }
    fence_barrier_init();
  }
  __syncwarp();
  cluster_arrive();
  if (warp == kSoft + 1) tmem_alloc_pair(smem_u32(tmem_slot), Gm::kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_wait();   // both CTAs' barriers stand before anyone arrives on them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int more0 = __ldg(a.more + pair);
  const int n_items = 1 + __ldg(a.more + pair + 1) - more0;
  auto index = [&](int i) -> int { return i == 0 ? pair : more0 + i - 1; };
  if (warp == kSoft || warp == kSoft + 2) {
    // ---------------- producers: one lane per copy of a tile ----------------
    const bool is_v = warp == kSoft + 2;
    const CUtensorMap* map = is_v ? &tmv : &tmk;
    if (lane == 0) tma_prefetch_desc(map);
    const int full0 = is_v ? Gm::kVFull : Gm::kKFull, empty0 = is_v ? Gm::kVEmpty : Gm::kKEmpty;
    // K: 32 keys of both halves, V: 64 keys of one half; a lane's 16-key unit in the tile,
    // half and place in the stage
    const int copies = is_v ? kTileK / a.v_rows : a.k_rows == 32 ? 1 : 4;
    const int unit = is_v ? lane * (a.v_rows / 16) : (int)rank * 2 + (lane & 1);
    const int half = is_v ? (int)rank : lane >> 1;
    const uint32_t off = is_v ? kOffV + (uint32_t)unit * 2048u : kOffK + (uint32_t)(lane >> 1) * kKBox + (uint32_t)(lane & 1) * 2048u;
    RingPos<kStages> pos;
    int filled = 0;
    bool ok = true;
    PrefixItem it = a.items[pair];
    for (int i = 0; ok && i < n_items; ++i) {
      const PrefixItem behind = a.items[i + 1 < n_items ? index(i + 1) : pair];
      const int32_t* row = a.block_tables + (int64_t)it.row * a.bt_row_stride;
      const int units = it.keys / 16, n_kv = it.tile_hi - it.tile_lo;
      // page of this lane's unit of tile j: past the prefix one past the pool, which reads as zeros
      auto page_of = [&](int j) -> int {
        const int u = (it.tile_lo + j) * (kTileK / 16) + unit;
        return lane < copies && j < n_kv && u < units ? __ldg(row + u / a.page_units) : a.num_pages;
      };
      int page = page_of(0);
      for (int j = 0; j < n_kv; ++j) {
        const int next = page_of(j + 1);
        if (filled >= kStages && !(ok = warp_wait(bar(empty0 + pos.slot), pos.parity ^ 1u, a.status))) break;
        const uint32_t full = map_to_rank(bar(full0 + pos.slot), 0);
        if (lane == 0) mbar_arrive_expect_tx_cluster(full, kKBytes);
        __syncwarp();
        if (lane < copies) {
          const int u = (it.tile_lo + j) * (kTileK / 16) + unit;
          tma_load_5d_pair(sbase + off + (uint32_t)pos.slot * kKBytes, map, full, 0, (u % a.page_units) * 16, half,
                           it.kv_head, page);
        }
        __syncwarp();
        page = next;
        pos.next();
        ++filled;
      }
      it = behind;
    }
    // When a wait gave up, copies still in flight land before the cluster leaves:
    // their barriers may be the other CTA's, so there is only time to go by.
    if (!ok) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 1000000ull) {
      }
    }
  } else if (warp == kSoft + 1) {
    // ---------------- MMA issuer, the leader's: one elected lane issues for the pair ----
    if (rank == 0) {
      RingPos<kStages> kp, vp;
      RingPos<kScores> sp, pp;   // the next S to issue and the next P to wait for
      bool ok = true;
      for (int i = 0; ok && i < n_items; ++i) {
        const int n_kv = __ldg(&a.items[index(i)].tile_hi) - __ldg(&a.items[index(i)].tile_lo);
        auto issue_qk = [&]() -> bool {   // S of the next key tile into the next buffer
          if (!warp_wait(bar(Gm::kKFull + kp.slot), kp.parity, a.status)) return false;
          tc_fence_after();
#pragma unroll
          for (int blk = 0; blk < 2; ++blk)
            umma_pair_ss_k4(tmem + (uint32_t)sp.slot * 64u,
                            smem_desc_sw128(sbase + (uint32_t)blk * kQBox, 16u, 1024u),
                            smem_desc_sw128(sbase + kOffK + (uint32_t)kp.slot * kKBytes + (uint32_t)blk * kKBox, 16u,
                                            1024u),
                            kIdescQK<F16>, blk > 0 ? 1u : 0u);
          umma_pair_commit_elect(bar(Gm::kSFull + sp.slot));
          umma_pair_commit_elect(bar(Gm::kKEmpty + kp.slot));
          kp.next();
          sp.next();
          return true;
        };
        // queries: ordinary writes, of the other CTA too
        ok = warp_wait<true>(bar(Gm::kQFull), (uint32_t)(i & 1), a.status);
        for (int j = 0; ok && j < n_kv && j < kScores; ++j) ok = issue_qk();
        for (int j = 0; ok && j < n_kv; ++j) {
          ok = warp_wait(bar(Gm::kVFull + vp.slot), vp.parity, a.status) &&
               warp_wait(bar(Gm::kPFull + pp.slot), pp.parity, a.status);
          if (ok && j == 0 && i > 0) ok = warp_wait(bar(Gm::kOFree), (uint32_t)((i - 1) & 1), a.status);
          if (!ok) break;
          tc_fence_after();
          // 4 k-steps of 16 keys: P columns +8, V rows +16 (2048 bytes)
          umma_pair_ts_k4<2048 / 16>(tmem + Gm::kColO + (uint32_t)(j % kGroups * kD), tmem + (uint32_t)pp.slot * 64u,
                                     smem_desc_sw128(sbase + kOffV + (uint32_t)vp.slot * kVBytes, kVBytes, 1024u),
                                     kIdescPV<F16>, j >= kGroups ? 1u : 0u);
          umma_pair_commit_elect(bar(Gm::kODone + pp.slot));
          umma_pair_commit_elect(bar(Gm::kVEmpty + vp.slot));
          vp.next();
          pp.next();
          // the S buffer is free again once this P V has read P (issue order)
          if (j + kScores < n_kv) ok = issue_qk();
        }
      }
      umma_pair_commit_elect(bar(Gm::kMmaDone));
    }
  } else {
    // ---------------- softmax: one thread per query row ----------------
    // the query rows asked for into shared memory
    auto give_rows = [&]() {
#pragma unroll
      for (int k = 0; k < kAsk; ++k) {
        const int rr = 2 * (group * kAsk + k) + (lane >> 4), c = lane & 15;
        rows[k].x ^= a.negate;
        rows[k].y ^= a.negate;
        rows[k].z ^= a.negate;
        rows[k].w ^= a.negate;
        *reinterpret_cast<uint4*>(smem + (uint32_t)(c >> 3) * kQBox + swz128((uint32_t)(rows4 + rr), (uint32_t)(c & 7))) = rows[k];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_rank(bar(Gm::kQFull), 0));
    };
    const uint32_t lane_off = (uint32_t)rows4 << 16;
    const uint32_t o_tm = tmem + lane_off + Gm::kColO + (uint32_t)(group * kD);   // the group's O
    const float sl2 = a.scale_log2;   // >= 0
    RingPos<kScores> sp;
    uint32_t last_o = 0, last_parity = 0;   // O barrier of the group's tile before and its parity
    float2* sums = reinterpret_cast<float2*>(smem + Gm::kOffSums) + (tid & (kTileQ - 1));
    // The groups' warps with the same rows meet, also when a wait of one gave up: none is left
    // waiting for the others.  Whether all are well.
    auto meet = [&](bool well) -> bool {
      if (kGroups == 1) return well;
      __syncwarp();
      switch (warp & 3) {
        case 0: return all_meet<1, kGroups * 32>(well);
        case 1: return all_meet<2, kGroups * 32>(well);
        case 2: return all_meet<3, kGroups * 32>(well);
        default: return all_meet<4, kGroups * 32>(well);
      }
    };
    bool ok = true;
    give_rows();
    for (int i = 0; ok && i < n_items; ++i) {
      const PrefixItem it = a.items[index(i)];
      const int n_kv = it.tile_hi - it.tile_lo;
      const bool live = it.row0 + mine < it.rows, any_live = __any_sync(0xffffffffu, live);
      float m_ref = neg_inf(), l = 0.f;
      for (int j = 0; j < n_kv; ++j) {
        if (kGroups > 1 && j % kGroups != group) {   // another's
          sp.next();
          continue;
        }
        if (!(ok = warp_wait(bar(Gm::kSFull + sp.slot), sp.parity, a.status))) break;
        if (any_live) {   // else P may be anything: rows stay apart
          tc_fence_after();
          const uint32_t s_tm = tmem + lane_off + (uint32_t)sp.slot * 64u;
          const int key0 = (it.tile_lo + j) * kTileK;
          const bool masked = key0 + kTileK > it.keys;
          uint32_t ra[32], rb[32];
          tmem_ld32(s_tm, ra);
          tmem_ld32(s_tm + 32u, rb);
          tmem_wait_ld();
          reg_fence32(ra);
          reg_fence32(rb);
          uint32_t w0 = 0xffffffffu, w1 = 0xffffffffu;
          if (masked) {
            visible_bits(key0, 0, (unsigned)it.keys, w0, w1);
            mask_scores64(ra, rb, w0, w1);
          }
          const float mraw = row_max64(ra, rb);
          const float mx = mraw == neg_inf() ? neg_inf() : mraw * sl2;
          const bool grow = mx > m_ref + kRescaleThreshold;
          const float m_new = grow ? mx : m_ref;
          const bool rescale = grow && m_ref != neg_inf();   // else O and l are still zero
          const float alpha = rescale ? ex2(m_ref - m_new) : 1.f;
          if (j >= kGroups && __any_sync(0xffffffffu, rescale)) {
            // O holds the group's tiles before: wait for P V of the last of them before rescaling
            if (!(ok = warp_wait(last_o, last_parity, a.status))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kD; c += 16) {   // 16 at a time: the scores stay in registers
              uint32_t o[16];
              tmem_ld16(o_tm + (uint32_t)c, o);
              tmem_wait_ld();
              reg_fence<16>(o);
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
              tmem_st16(o_tm + (uint32_t)c, o);
            }
            tmem_wait_st();
          }
          m_ref = m_new;
          // A row whose scores are all -inf keeps m_ref = -inf: exp2(-inf) = 0.  Masked scores
          // give 0 through their -inf unless the scale is 0.
          const float neg_m = m_ref == neg_inf() ? 0.f : kLatentWeightShift<F16> - m_ref;
          const bool zero_again = masked && !(sl2 > 0.f);
          const float2 sum = zero_again ? exp_tile<true, F16>(ra, rb, sl2, neg_m, w0, w1, s_tm)
                                        : exp_tile<false, F16>(ra, rb, sl2, neg_m, w0, w1, s_tm);
          tmem_wait_st();
          l = l * alpha + (sum.x + sum.y);
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(map_to_rank(bar(Gm::kPFull + sp.slot), 0));
        last_o = bar(Gm::kODone + sp.slot);
        last_parity = sp.parity;
        sp.next();
      }
      // every S of this piece is complete: its queries make room for the next one's
      if constexpr (kGroups > 1) ok = meet(ok);
      if (!ok) break;
      if (i + 1 < n_items) {
        ask_rows(index(i + 1));
        give_rows();
      }
      if constexpr (kGroups > 1) {
        sums[group * kTileQ] = make_float2(m_ref, l);
        ok = meet(group >= n_kv || warp_wait(last_o, last_parity, a.status));   // without a tile there is no O
      } else {
        ok = warp_wait(last_o, last_parity, a.status);
      }
      if (!ok) break;
      tc_fence_after();
      if (any_live) {
        float scale[kGroups] = {};   // of each group's O
        if constexpr (kGroups == 1) {
          // != and not >: a sum that is NaN stays one, in the LSE as in the output
          scale[0] = l != 0.f ? 1.f / l : 0.f;
        } else {
          const float2 x = sums[0], y = sums[kTileQ];
          m_ref = fmaxf(x.x, y.x);
          scale[0] = x.x == neg_inf() ? 0.f : ex2(x.x - m_ref);
          scale[1] = y.x == neg_inf() ? 0.f : ex2(y.x - m_ref);
          l = x.y * scale[0] + y.y * scale[1];
          const float inv = l != 0.f ? 1.f / l : 0.f;
          scale[0] *= inv;
          scale[1] *= inv;
        }
        const int64_t state = (int64_t)it.state + mine;
        const int c0 = group * (kD / kGroups);   // the dimensions that this warp stores
        const uint32_t o0 = tmem + lane_off + Gm::kColO;
#pragma unroll 1
        for (int c = c0; c < c0 + kD / kGroups; c += 32) {
          uint32_t o[32];
          __syncwarp();   // the lanes whose rows are stored and the others load together
          tmem_ld32_sync(o0 + (uint32_t)c, o);
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * scale[0]);
          if (kGroups > 1 && n_kv > 1) {
            uint32_t o1[32];
            tmem_ld32_sync(o0 + (uint32_t)(kD + c), o1);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              o[x] = __float_as_uint(__uint_as_float(o[x]) + __uint_as_float(o1[x]) * scale[kGroups - 1]);
          }
          if (live) {
#pragma unroll
            for (int x = 0; x < 4; ++x) store_sector(a.ws_o + state * kD + c + 8 * x, o + 8 * x);
          }
        }
        if (live && group == 0) a.ws_lse[state] = l != 0.f ? m_ref - kLatentWeightShift<F16> + log2f(l) : neg_inf();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(map_to_rank(bar(Gm::kOFree), 0));
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // Nothing of the pair's still runs on the tensor cores, and every commit has landed here.
  // Waited for only now: all of a pair's tiles may take longer than any one wait may.
  if (warp == kSoft + 1) warp_wait(bar(Gm::kMmaDone), 0, a.status);
  cluster_sync();   // neither CTA's shared memory nor TMEM goes while the pair still uses it
  if (warp == kSoft + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, Gm::kTmemCols);
  }
}

template <bool F16, bool DENSE>
int launch(const PrefixArgs& args, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
  auto kern = prefix_kernel<F16, DENSE>;
  static std::atomic<uint64_t> smem_set{0};   // devices whose limit was raised
  cudaError_t e = set_smem_once(kern, (int)Geo<DENSE>::kSmemBytes, smem_set, true);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(prefix)");
  kern<<<2 * args.num_pairs, Geo<DENSE>::kThreads, Geo<DENSE>::kSmemBytes, stream>>>(args, kmap, vmap);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "prefix_kernel launch");
  return PKA_OK;
}

}  // namespace

int launch_prefix(const PrefixArgs& args, bool f16, bool dense, const CUtensorMap& kmap, const CUtensorMap& vmap,
                  cudaStream_t stream) {
  if (dense) return f16 ? launch<true, true>(args, kmap, vmap, stream) : launch<false, true>(args, kmap, vmap, stream);
  return f16 ? launch<true, false>(args, kmap, vmap, stream) : launch<false, false>(args, kmap, vmap, stream);
}

}  // namespace pka
