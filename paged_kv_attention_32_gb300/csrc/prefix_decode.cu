// Attention of many query rows over one shared, paged prefix, on the 5th-generation
// tensor cores (tcgen05 + TMEM): the part of a decode that its requests have in common.
//
// For the rows r = (token, head of the KV head's group) of a group of requests and the
// prefix's keys j of one piece
//   s_j = scale * q_r . k_j,  m = max s, l = sum exp(s - m),  o = sum exp(s - m) v / l,
// stored as a 32-bit partial state (o and the base-2 LSE) that the decode kernel merges
// with the states of the request's own keys.  Every row sees the whole prefix, so the only
// mask is the piece's end.
//
// A pair of CTAs (cta_group::2, one cluster, two SMs) takes 256 rows, 128 each, and walks
// the keys in tiles of 64.  Each CTA holds its own queries and only half of every tile: 32
// of the keys (half of B's N in S = Q K^T) and 64 of the value dimensions (half of N in
// O += P V), which halves what the shared-memory port moves for K and V and the copies.
// Two CTAs of different pairs share an SM and hide each other's softmax and start.
//   warp 4      copies this CTA's half of the keys, page by page (TMA);
//   warp 6      its half of the values;
//   warp 5      in the leader, issues every tcgen05.mma for both CTAs: S_b (M=256, N=64,
//               8 k-steps) into one of two S buffers, two tiles ahead of the softmax, and
//               O += P V (M=256, N=128, 4 k-steps of 16 keys, P from TMEM);
//   warps 0-3   gather the query rows (any token and head strides, any group size), then
//               softmax, one thread per row: O rescaled only when the row maximum grew by
//               more than 2^8, P in 16 bits over the S buffer (its rounding enters O like
//               the inputs' own; the sum of p is taken in 32 bits before it).
// TMEM columns: S0 [0,64) S1 [64,128) O [128,256).
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
constexpr int kStages = 5;
constexpr int kThreads = 224;
constexpr float kRescaleThreshold = 8.0f;
constexpr uint32_t kColO = 128, kTmemCols = 256;

constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = 2 * kQBox;
constexpr uint32_t kOffV = kOffK + kStages * kKBytes;
constexpr uint32_t kOffBar = kOffV + kStages * kVBytes;
constexpr size_t kSmemBytes = kOffBar + 256;
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs share an SM");

// Q, K, V and P are waited for by the leader's MMA warp, on the leader's barriers, where
// both CTAs arrive; the others are signalled in both CTAs by the commits.  Tile j uses S, P
// and O barriers j & 1.  No barrier runs a phase past one that somebody still has to see:
// S(j) is issued behind P V(j - 2), and P(j) is written once S(j) is complete.
enum {
  B_QFULL = 0, B_KFULL, B_KEMPTY = B_KFULL + kStages, B_VFULL = B_KEMPTY + kStages, B_VEMPTY = B_VFULL + kStages,
  B_SFULL = B_VEMPTY + kStages, B_PFULL = B_SFULL + 2, B_ODONE = B_PFULL + 2, B_MMADONE = B_ODONE + 2, B_COUNT
};
static_assert(B_COUNT * 8 + 4 <= 256, "barriers and the TMEM address slot");

template <bool F16> constexpr uint32_t kIdescQK = idesc_bf16_f32(256, 64, 0, 0, F16);
template <bool F16> constexpr uint32_t kIdescPV = idesc_bf16_f32(256, kD, 0, 1, F16);

__device__ __forceinline__ void store_sector(float* dst, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

template <bool F16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 2)
prefix_kernel(const __grid_constant__ PrefixArgs a, const __grid_constant__ CUtensorMap tmk,
              const __grid_constant__ CUtensorMap tmv) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + B_COUNT * 8);
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * (uint32_t)i; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();   // 0: the leader
  const PrefixItem it = a.items[blockIdx.x >> 1];

  if (tid == 0) {
    mbar_init(bar(B_QFULL), 8);             // the pair's softmax warps
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(B_KFULL + s), 2);
      mbar_init(bar(B_KEMPTY + s), 1);
      mbar_init(bar(B_VFULL + s), 2);
      mbar_init(bar(B_VEMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_SFULL + s), 1);
      mbar_init(bar(B_PFULL + s), 8);
      mbar_init(bar(B_ODONE + s), 1);
    }
    mbar_init(bar(B_MMADONE), 1);
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
  // the decode's CTAs may start taking free SMs; their merges wait for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int n_kv = it.tile_hi - it.tile_lo;
  if (warp == 4 || warp == 6) {
    // ---------------- producers: one lane per copy of a tile ----------------
    const bool is_v = warp == 6;
    const CUtensorMap* map = is_v ? &tmv : &tmk;
    if (lane == 0) tma_prefetch_desc(map);
    const int full0 = is_v ? B_VFULL : B_KFULL, empty0 = is_v ? B_VEMPTY : B_KEMPTY;
    // K: 32 keys of both halves, V: 64 keys of one half; a lane's 16-key unit in the tile,
    // half and place in the stage
    const int copies = is_v ? kTileK / a.v_rows : a.k_rows == 32 ? 1 : 4;
    const int unit = is_v ? lane * (a.v_rows / 16) : (int)rank * 2 + (lane & 1);
    const int half = is_v ? (int)rank : lane >> 1;
    const uint32_t off = is_v ? kOffV + (uint32_t)unit * 2048u : kOffK + (uint32_t)(lane >> 1) * kKBox + (uint32_t)(lane & 1) * 2048u;
    const int32_t* row = a.block_tables + (int64_t)it.row * a.bt_row_stride;
    const int units = it.keys / 16;
    // page of this lane's unit of tile j: past the prefix one past the pool, which reads as zeros
    auto page_of = [&](int j) -> int {
      const int u = (it.tile_lo + j) * (kTileK / 16) + unit;
      return lane < copies && j < n_kv && u < units ? __ldg(row + u / a.page_units) : a.num_pages;
    };
    int page = page_of(0), stage = 0;
    uint32_t parity = 0;
    bool ok = true;
    for (int j = 0; j < n_kv; ++j) {
      const int next = page_of(j + 1);
      if (j >= kStages && !(ok = warp_wait(bar(empty0 + stage), parity ^ 1u, a.status))) break;
      const uint32_t full = map_to_rank(bar(full0 + stage), 0);
      if (lane == 0) mbar_arrive_expect_tx_cluster(full, kKBytes);
      __syncwarp();
      if (lane < copies) {
        const int u = (it.tile_lo + j) * (kTileK / 16) + unit;
        tma_load_5d_pair(sbase + off + (uint32_t)stage * kKBytes, map, full, 0, (u % a.page_units) * 16, half,
                         it.kv_head, page);
      }
      __syncwarp();
      page = next;
      if (++stage == kStages) {
        stage = 0;
        parity ^= 1u;
      }
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
      int ks = 0, vs = 0;
      uint32_t kpar = 0, vpar = 0;
      auto issue_qk = [&](int j) -> bool {   // S of tile j into buffer j & 1
        if (!warp_wait(bar(B_KFULL + ks), kpar, a.status)) return false;
        tc_fence_after();
        const int st = j & 1;
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
          umma_pair_ss_k4(tmem + (uint32_t)st * 64u,
                          smem_desc_sw128(sbase + kOffQ + (uint32_t)blk * kQBox, 16u, 1024u),
                          smem_desc_sw128(sbase + kOffK + (uint32_t)ks * kKBytes + (uint32_t)blk * kKBox, 16u, 1024u),
                          kIdescQK<F16>, blk > 0 ? 1u : 0u);
        umma_pair_commit_elect(bar(B_SFULL + st));
        umma_pair_commit_elect(bar(B_KEMPTY + ks));
        if (++ks == kStages) {
          ks = 0;
          kpar ^= 1u;
        }
        return true;
      };
      // queries: ordinary writes, of the other CTA too
      bool ok = warp_wait<true>(bar(B_QFULL), 0, a.status);
      for (int j = 0; ok && j < n_kv && j < 2; ++j) ok = issue_qk(j);
      for (int j = 0; ok && j < n_kv; ++j) {
        const int st = j & 1;
        ok = warp_wait(bar(B_VFULL + vs), vpar, a.status) &&
             warp_wait(bar(B_PFULL + st), (uint32_t)((j >> 1) & 1), a.status);
        if (!ok) break;
        tc_fence_after();
        // 4 k-steps of 16 keys: P columns +8, V rows +16 (2048 bytes)
        umma_pair_ts_k4<2048 / 16>(tmem + kColO, tmem + (uint32_t)st * 64u,
                                   smem_desc_sw128(sbase + kOffV + (uint32_t)vs * kVBytes, kVBytes, 1024u),
                                   kIdescPV<F16>, j > 0 ? 1u : 0u);
        umma_pair_commit_elect(bar(B_ODONE + st));
        umma_pair_commit_elect(bar(B_VEMPTY + vs));
        if (++vs == kStages) {
          vs = 0;
          vpar ^= 1u;
        }
        // S buffer st is free again once this P V has read P (issue order)
        if (j + 2 < n_kv) ok = issue_qk(j + 2);
      }
      umma_pair_commit_elect(bar(B_MMADONE));
    }
  } else {
    // ---------------- softmax: one thread per query row ----------------
    const int r = it.row0 + (int)rank * kTileQ + tid;
    const bool live = r < it.rows;
    const int token = it.q_start + r / a.group, head = it.kv_head * a.group + r % a.group;
    // a warp's rows, two at a time, 16 lanes a row; zeros where there is none
    const int64_t src = live ? (int64_t)token * a.q_stride_tok + (int64_t)head * a.q_stride_head : -1;
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const int rr = 2 * i + (lane >> 4), c = lane & 15;
      const int64_t at = __shfl_sync(0xffffffffu, src, rr);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (at >= 0) v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at) + c);
      v.x ^= a.negate;
      v.y ^= a.negate;
      v.z ^= a.negate;
      v.w ^= a.negate;
      *reinterpret_cast<uint4*>(smem + kOffQ + (uint32_t)(c >> 3) * kQBox +
                                swz128((uint32_t)(warp * 32 + rr), (uint32_t)(c & 7))) = v;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(map_to_rank(bar(B_QFULL), 0));

    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t o_tm = tmem + lane_off + kColO;
    const float sl2 = a.scale_log2;   // >= 0
    const bool any_live = __any_sync(0xffffffffu, live);
    float m_ref = neg_inf(), l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_kv; ++j) {
      const int st = j & 1;
      if (!(ok = warp_wait(bar(B_SFULL + st), (uint32_t)((j >> 1) & 1), a.status))) break;
      if (any_live) {   // else P may be anything: rows stay apart
        tc_fence_after();
        const uint32_t s_tm = tmem + lane_off + (uint32_t)st * 64u;
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
        if (j > 0 && __any_sync(0xffffffffu, rescale)) {
          // O holds the tiles before: wait for P V of the last of them before rescaling
          if (!(ok = warp_wait(bar(B_ODONE + (st ^ 1)), (uint32_t)(((j - 1) >> 1) & 1), a.status))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kD / 32; ++c) {
            uint32_t o[32];
            tmem_ld32_sync(o_tm + (uint32_t)c * 32u, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(o_tm + (uint32_t)c * 32u, o);
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
      if (lane == 0) mbar_arrive_remote(map_to_rank(bar(B_PFULL + st), 0));
    }
    if (ok && any_live && warp_wait(bar(B_ODONE + ((n_kv - 1) & 1)), (uint32_t)(((n_kv - 1) >> 1) & 1), a.status)) {
      tc_fence_after();
      // != and not >: a sum that is NaN stays one, in the LSE as in the output
      const float inv = l != 0.f ? 1.f / l : 0.f;
      int64_t part = 0;
      if (live) {
        const PrefixToken t = a.tokens[token];
        part = (int64_t)t.part0 + (int64_t)it.chunk * t.stride + head;
      }
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        uint32_t o[32];
        __syncwarp();   // the lanes whose rows are stored and the others load together
        tmem_ld32_sync(o_tm + (uint32_t)c, o);
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * inv);
        if (live) {
#pragma unroll
          for (int k = 0; k < 4; ++k) store_sector(a.ws_o + part * kD + c + 8 * k, o + 8 * k);
        }
      }
      if (live) a.ws_lse[part] = l != 0.f ? m_ref - kLatentWeightShift<F16> + log2f(l) : neg_inf();
    }
  }

  __syncwarp();
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

}  // namespace

int launch_prefix(const PrefixArgs& args, bool f16, const CUtensorMap& kmap, const CUtensorMap& vmap,
                  cudaStream_t stream) {
  auto kern = f16 ? prefix_kernel<true> : prefix_kernel<false>;
  static std::atomic<uint64_t> smem_set[2];   // per input type: devices whose limit was raised
  cudaError_t e = set_smem_once(kern, (int)kSmemBytes, smem_set[f16]);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(prefix)");
  kern<<<2 * args.num_items, kThreads, kSmemBytes, stream>>>(args, kmap, vmap);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "prefix_kernel launch");
  return PKA_OK;
}

}  // namespace pka
