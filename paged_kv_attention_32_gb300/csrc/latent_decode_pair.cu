// Absorbed latent decode for more than 64 query rows (token, head) a request, by
// pairs of CTAs (cta_group::2): 128 rows, 64 in each CTA, over tiles of 64 keys.
//
//   S = Q K^T    M=128 (rows), N=64 (keys), 576 or 320 columns deep
//   O += P V     M=128 (rows), N=256 (latent dimensions), 64 keys deep
//
// With many rows the work is bound by the shared-memory port.  The transposed kernel (latent_decode.cu) holds a tile once for 64
// rows and reads 2 + 2 KB for each 64 x 64 x 16 step of S; here a CTA holds its
// own 64 queries, half of the tile's keys (32) for S and half of the latent
// dimensions (of all 64 keys) for P V, and the pair reads 3 KB a CTA for twice the
// rows.  Measured per instruction: M=64 N=64 single 32 cycles; M=128 N=64 in a
// pair 25, N=256 64.  The two halves overlap in a quarter of the tile, which
// comes twice (from L2).  A tile's bytes through the port of a CTA: 108 KB of operands
// of S, 48 of P V, 70 of copies and 8 of P, 1860 cycles at 128 B; the tensor core's own
// time is 1430.  Measured: 64 ragged requests of 128 heads, 512 + 64 columns, 77 us (floor
// 49.3, its 335 MB at the copy rate); 32 requests of 4 causal rows of 64 heads 125 us
// (floor 83.5, its products at the library's rate).  256 + 64 columns, 76 requests of
// 4096 keys, 128 heads: 54 us, of which 199 MB are 29.
// Each CTA's warps:
//   0  copies queries and its half of the keys;   3  its half of the values, which
//      in the tile that holds the last key it clears past it (0 * inf is not 0)
//      before handing it over (one warp for both was what bounded the pair);
//   1  in the leader: issues S for both CTAs;   2  in the leader: issues P V;
//   4-7  softmax and output: TMEM lane i of a CTA is row i % 64, and lanes of
//      64 on hold the second half of a tile's keys, of each 256 dimensions.
// TMEM columns: O blocks of 256 dimensions (128 each), then two S buffers (32).
#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>

#include "device_common.cuh"
#include "host_common.h"
#include "latent.h"
#include "latent_decode.cuh"
#include "prefill_softmax.cuh"
#include "tcgen05.cuh"
#include "tmap.h"

namespace pka {

using namespace dev;

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;   // query rows of a CTA

template <int DL>
struct Pair {
  static constexpr int NC = DL / 64 + 1;                // 64-column chunks of a row
  static constexpr int ND = DL / 256;                   // 256-wide blocks of P V
  static constexpr uint32_t kGroup = NC * 1024;         // 8 whole rows: NC atoms of 8 x 128 bytes
  static constexpr uint32_t kQ = 8 * kGroup;
  static constexpr uint32_t kK = 4 * kGroup;            // 32 keys
  static constexpr uint32_t kV = ND * 16384;            // 64 keys x 128 dims, ND times
  static constexpr uint32_t kP = 8192;                  // 64 rows x 64 keys
  static constexpr uint32_t kMisc = 2048;
  static constexpr int kFit = (kSmemLimit - kMisc - kQ - 2 * kP) / (kK + kV);
  static constexpr int NS = kFit < 4 ? kFit : 4;        // stages of keys, and of values
  static constexpr uint32_t kOffK = kQ;
  static constexpr uint32_t kOffV = kOffK + NS * kK;
  static constexpr uint32_t kOffP = kOffV + NS * kV;
  static constexpr uint32_t kOffMisc = kOffP + 2 * kP;
  static constexpr uint32_t kSmem = kOffMisc + kMisc;
  static constexpr uint32_t kColS = ND * 128;
  static_assert(NS >= 2 && kSmem <= kSmemLimit, "two stages");
};

struct PairMaps {
  CUtensorMap keys, values, q;   // whole rows, two chunks, whole rows of queries
};

// mbarriers.  Q, K, V, P and O-free are waited for in the leader, on its
// barriers, where both CTAs arrive; the others are signalled in both CTAs by the
// commits.  T counts tiles over all pieces.  No barrier runs a phase past one
// that somebody still has to see: S(T) is issued once P(T - 2) is written, P(T)
// written once P V(T - 2) is complete.
enum {
  R_KFULL = 0, R_KEMPTY = 4, R_VFULL = 8, R_VEMPTY = 12, R_SFULL = 16, R_PFULL = 18, R_PV = 20,
  R_QFULL = 22, R_QFREE = 23, R_OFREE = 24, R_SDONE = 25, R_ODONE = 26, R_TAIL = 27, R_COUNT = 28
};
static_assert(R_COUNT * 8 + 4 + 12 <= 256, "barriers, TMEM address, failure flags");

// When a wait gave up, copies still in flight land before the cluster leaves:
// their barriers may be the other CTA's, so there is only time to go by.
__device__ __forceinline__ void let_copies_land() {
  const uint64_t t0 = global_timer_ns();
  while (global_timer_ns() - t0 < 1000000ull) {
  }
}

template <int DL, bool F16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
latent_decode_pair_kernel(const __grid_constant__ LatentArgs a, const __grid_constant__ PairMaps maps) {
  using G = Pair<DL>;
  constexpr int NC = G::NC, ND = G::ND, NS = G::NS;
  constexpr uint32_t kIdescS = idesc_bf16_f32(128, 64, 0, 0, F16);
  constexpr uint32_t kIdescO = idesc_bf16_f32(128, 256, 0, 1, F16);
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  uint8_t* misc = smem + G::kOffMisc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + R_COUNT * 8);
  volatile int* s_fail = reinterpret_cast<volatile int*>(tmem_slot + 1);   // [3]
  float* s_max = reinterpret_cast<float*>(misc + 256);    // [2 halves][64 rows]
  float* s_sum = s_max + 2 * kRows;                       // [2 halves][64 rows]
  auto bar = [&](int i) -> uint32_t { return sbase + G::kOffMisc + 8u * (uint32_t)i; };
  auto lead = [&](int i) -> uint32_t { return map_to_rank(bar(i), 0); };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();   // 0: the leader
  const int pair = blockIdx.x >> 1, seg = pair / a.row_blocks, rb = pair % a.row_blocks;

  if (tid == 0) {   // the first piece comes in while the CTA sets up
    ask_line(a.pieces + seg);
    ask_line(a.more + seg);
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(R_KFULL + s), 1);   // the leader expects both CTAs' bytes
      mbar_init(bar(R_KEMPTY + s), 1);
      mbar_init(bar(R_VFULL + s), 2);
      mbar_init(bar(R_VEMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(R_SFULL + s), 1);
      mbar_init(bar(R_PFULL + s), 8);   // one arrival per softmax warp of the pair
      mbar_init(bar(R_PV + s), 1);
    }
    mbar_init(bar(R_QFULL), a.q_box > 0 ? 1 : 8);
    mbar_init(bar(R_QFREE), 1);
    mbar_init(bar(R_OFREE), 8);
    mbar_init(bar(R_SDONE), 1);
    mbar_init(bar(R_ODONE), 1);
    mbar_init(bar(R_TAIL), 1);
    for (int i = 0; i < 3; ++i) tmem_slot[1 + i] = 0;   // failure flags
    fence_barrier_init();
  }
  __syncwarp();
  cluster_arrive();
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  cluster_wait();   // both CTAs' barriers stand before anyone arrives on them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the merge's CTAs may start taking free SMs; they wait for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Pieces pieces(a, seg);

  if (warp == 0) {
    // ---------------- queries and keys: lane i copies box i ----------------
    if (lane < 2) tma_prefetch_desc(lane == 0 ? &maps.keys : &maps.q);
    const int krows = min(a.box_rows, 32), boxes = 32 / krows;   // cache rows of a key box
    Ring<NS> kp;
    int nk = 0, I = 0;   // stages filled so far, pieces
    bool ok = true;
    for (int item = 0; ok && pieces.has(item); ++item) {
      const Piece pc(a, pieces[item], rb, 2 * kRows);
      if (pc.n == 0) continue;
      if (a.q_box > 0) {   // whole groups of 8 heads: the queries come by TMA too
        if (I > 0 && !(ok = warp_wait(bar(R_QFREE), (uint32_t)((I - 1) & 1), a.status))) break;
        if (lane == 0 && rank == 0) mbar_arrive_expect_tx(bar(R_QFULL), 2 * G::kQ);
        __syncwarp();
        if (lane < kRows / a.q_box) {   // rows past the request's last are copied, and never stored
          const int r = pc.row0 + (int)rank * kRows + lane * a.q_box;
          tma_load_5d_pair(sbase + (uint32_t)(lane * a.q_box / 8) * G::kGroup, &maps.q, lead(R_QFULL), 0, 0, 0,
                           r % a.num_heads / 8, pc.rq.q_start + r / a.num_heads);
        }
        __syncwarp();
      }
      ++I;
      PageWalk walk(a, pc, (int)rank * 32 + lane * krows, lane < boxes);
      // With two stages the tile behind them is asked for in L2 (both CTAs' keys are its
      // values too): 76 requests of 4096 keys, 128 heads, 512 + 64 columns 75.9 -> 68.3 us;
      // a tile further 68.3, two 70.1.  With four stages it costs more than it gives (256 +
      // 64: 47.4 -> 48.4).  The other row blocks read the same keys at about the same time.
      const bool ask_ahead = NS == 2 && rb == 0;
      PageWalk ahead = walk;
      if (ask_ahead)
        for (int j = 0; j < NS; ++j) ahead.next_tile();
      for (int j = 0; j < pc.n; ++j) {
        const int page = walk.page(), slot8 = walk.slot / 8;
        walk.next_tile();
        if (nk >= NS && !(ok = warp_wait(bar(R_KEMPTY + kp.slot), kp.parity ^ 1u, a.status))) break;
        if (lane == 0 && rank == 0) mbar_arrive_expect_tx(bar(R_KFULL + kp.slot), 2 * G::kK);
        __syncwarp();
        if (lane < boxes)
          tma_load_5d_pair(sbase + G::kOffK + (uint32_t)kp.slot * G::kK + (uint32_t)(lane * krows / 8) * G::kGroup,
                           &maps.keys, lead(R_KFULL + kp.slot), 0, 0, 0, slot8, page);
        __syncwarp();
        if (ask_ahead && j + NS < pc.n) {
          if (lane < boxes) tma_prefetch_5d(&maps.keys, 0, 0, 0, ahead.slot / 8, ahead.page());
          ahead.next_tile();
        }
        kp.next();
        ++nk;
      }
    }
    if (!ok) let_copies_land();
  } else if (warp == 3) {
    // ---------------- values: lane i copies box i ----------------
    if (lane == 0) tma_prefetch_desc(&maps.values);
    const int boxes = kLatentTile / a.box_rows;
    Ring<NS> vp;
    int nv = 0, tails = 0;   // stages filled so far, cleared tiles
    bool ok = true;
    for (int item = 0; ok && pieces.has(item); ++item) {
      const Piece pc(a, pieces[item], rb, 2 * kRows);
      if (pc.n == 0) continue;
      PageWalk walk(a, pc, lane * a.box_rows, lane < boxes);
      for (int j = 0; j < pc.n; ++j) {
        const int page = walk.page(), slot8 = walk.slot / 8;
        walk.next_tile();
        if (nv >= NS && !(ok = warp_wait(bar(R_VEMPTY + vp.slot), vp.parity ^ 1u, a.status))) break;
        const uint32_t off = G::kOffV + (uint32_t)vp.slot * G::kV, full = lead(R_VFULL + vp.slot);
        const int live = pc.kv - (pc.tile0 + j) * kLatentTile;
        const bool tail = live < kLatentTile;
        const uint32_t landed = tail ? map_to_rank(bar(R_TAIL), rank) : full;
        if (lane == 0) mbar_arrive_expect_tx_cluster(landed, G::kV);
        __syncwarp();
        if (lane < boxes)
          for (int d = 0; d < ND; ++d)
            tma_load_5d_pair(sbase + off + (uint32_t)d * 16384u + (uint32_t)(lane * a.box_rows / 8) * 2048u,
                             &maps.values, landed, 0, 0, 4 * d + 2 * (int)rank, slot8, page);
        __syncwarp();
        if (tail) {
          // rows past the last token may hold anything, and 0 * inf is not 0: clear
          // them to the end of their box (boxes past it brought zeros)
          if (!(ok = warp_wait(bar(R_TAIL), (uint32_t)(tails & 1), a.status))) break;
          ++tails;
          const int end = (live + a.box_rows - 1) / a.box_rows * a.box_rows;
          for (int i = lane; i < (end - live) * ND * 16; i += 32) {
            const int r = live + i / (ND * 16), c = i % (ND * 16);
            *reinterpret_cast<uint4*>(smem + off + (uint32_t)(c >> 4) * 16384u + (uint32_t)(r >> 3) * 2048u +
                                      (uint32_t)((c >> 3) & 1) * 1024u + (uint32_t)(r & 7) * 128u +
                                      (uint32_t)(c & 7) * 16u) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(full);
        }
        vp.next();
        ++nv;
      }
    }
    if (!ok) let_copies_land();
  } else if (warp == 1) {
    // ---------------- the leader's: issues S = Q K^T ----------------
    if (rank == 0) {
      const uint64_t dq = smem_desc_sw128(sbase, 16u, G::kGroup);
      const uint64_t dk = smem_desc_sw128(sbase + G::kOffK, 16u, G::kGroup);
      Ring<NS> kp;
      int T = 0, I = 0;   // tiles and non-empty pieces before this one
      bool ok = true;
      for (int item = 0; ok && pieces.has(item); ++item) {
        const Piece pc(a, pieces[item], rb, 2 * kRows);
        if (pc.n == 0) continue;
        // queries by plain loads: ordinary writes, of the other CTA too
        ok = warp_wait<true>(bar(R_QFULL), (uint32_t)(I & 1), a.status);
        ++I;
        for (int j = 0; ok && j < pc.n; ++j, ++T) {
          // P(T - 2) written means S(T - 2) read: this S buffer is free
          ok = (T < 2 || warp_wait(bar(R_PFULL + (T & 1)), (uint32_t)(((T >> 1) - 1) & 1), a.status)) &&
               warp_wait(bar(R_KFULL + kp.slot), kp.parity, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + G::kColS + (uint32_t)(T & 1) * 32u;
          const uint64_t x = dk + (uint32_t)kp.slot * (G::kK / 16);
#pragma unroll
          for (int c = 0; c < NC; ++c) umma_pair_ss_k4(d, dq + c * 64, x + c * 64, kIdescS, c > 0 ? 1u : 0u);
          umma_pair_commit_elect(bar(R_SFULL + (T & 1)));
          umma_pair_commit_elect(bar(R_KEMPTY + kp.slot));
          kp.next();
        }
        if (ok) umma_pair_commit_elect(bar(R_QFREE));
      }
      umma_pair_commit_elect(bar(R_SDONE));
    }
  } else if (warp == 2) {
    // ---------------- the leader's: issues O += P V ----------------
    if (rank == 0) {
      const uint64_t dp = smem_desc_sw128(sbase + G::kOffP, 16u, 1024u);
      const uint64_t dv = smem_desc_sw128(sbase + G::kOffV, 1024u, 2048u);
      Ring<NS> vp;
      int T = 0, I = 0;
      bool ok = true;
      for (int item = 0; ok && pieces.has(item); ++item) {
        const Piece pc(a, pieces[item], rb, 2 * kRows);
        if (pc.n == 0) continue;
        for (int j = 0; j < pc.n; ++j, ++T) {
          // cleared values and weights: ordinary writes, of the other CTA too
          ok = warp_wait<true>(bar(R_VFULL + vp.slot), vp.parity, a.status) &&
               warp_wait<true>(bar(R_PFULL + (T & 1)), (uint32_t)((T >> 1) & 1), a.status);
          if (ok && j == 0 && I > 0) ok = warp_wait(bar(R_OFREE), (uint32_t)((I - 1) & 1), a.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t p = dp + (uint32_t)(T & 1) * (G::kP / 16);
          const uint64_t v = dv + (uint32_t)vp.slot * (G::kV / 16);
#pragma unroll
          for (int d = 0; d < ND; ++d)   // 128 rows x 256 dims += 64 keys
            umma_pair_ss_k4_steps<2, 4096 / 16>(tmem + (uint32_t)d * 128u, p, v + d * 1024, kIdescO,
                                                j > 0 ? 1u : 0u);
          umma_pair_commit_elect(bar(R_VEMPTY + vp.slot));
          umma_pair_commit_elect(bar(R_PV + (T & 1)));
          vp.next();
        }
        ++I;
      }
      umma_pair_commit_elect(bar(R_ODONE));
    }
  } else {
    // ---------------- softmax and output ----------------
    const int quad = warp & 3;                      // TMEM lanes 32 quad .. + 31
    const int row = (quad & 1) * 32 + lane, half = quad >> 1;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int gt = tid - 128;                       // thread of the four warps
    const float sl2 = a.scale_log2;

    // queries by plain loads (heads not a multiple of 8), laid out like keys
    auto load_q = [&](const Piece& pc) {
      constexpr int V = (DL + kLatentRopeDim) / 8;   // 16-byte pieces of a row
#pragma unroll 4
      for (int i = gt; i < kRows * V; i += 128) {
        const int r = i / V, c = i % V, at = pc.row0 + (int)rank * kRows + r;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if ((int)rank * kRows + r < pc.rows)
          x = __ldg(reinterpret_cast<const uint4*>(
                        static_cast<const uint16_t*>(a.q) +
                        (int64_t)(pc.rq.q_start + at / a.num_heads) * a.q_stride_tok +
                        (int64_t)(at % a.num_heads) * a.q_stride_head) + c);
        *reinterpret_cast<uint4*>(smem + (uint32_t)(r >> 3) * G::kGroup + (uint32_t)(c >> 3) * 1024u +
                                  swz128((uint32_t)(r & 7), (uint32_t)(c & 7))) = x;
      }
      fence_proxy_async_smem();   // generic writes -> the tensor core's operand reads
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(lead(R_QFULL));
    };
    int I = 0;
    bool ok = true;
    auto next_q = [&](int item) {   // the next piece that has tiles, from `item` on
      if (a.q_box > 0) return;
      for (; pieces.has(item); ++item) {
        const Piece pc(a, pieces[item], rb, 2 * kRows);
        if (pc.n > 0) {
          if (I > 0 && !warp_wait(bar(R_QFREE), (uint32_t)((I - 1) & 1), a.status)) s_fail[2] = 1;
          load_q(pc);
          return;
        }
      }
    };
    next_q(0);

    int T = 0;
    for (int item = 0; ok && pieces.has(item); ++item) {
      const Piece pc(a, pieces[item], rb, 2 * kRows);
      if (pc.rows <= 0) continue;
      const bool whole = pc.part < 0;
      const int live = min(kRows, pc.rows - (int)rank * kRows);   // this CTA's rows, may be < 1
      const int64_t orow = (int64_t)pc.rq.q_start * a.num_heads + pc.row0 + (int)rank * kRows;
      const int64_t prow = (int64_t)pc.rq.part_base +
                           (int64_t)max(pc.part, 0) * pc.rq.q_len * a.num_heads + pc.row0 + (int)rank * kRows;
      if (pc.n == 0) {   // no keys here: zero rows, or a piece that weighs nothing
        for (int i = gt; i < live; i += 128) {
          if (!whole) a.ws_lse[prow + i] = neg_inf();
          else if (a.lse != nullptr) a.lse[orow + i] = neg_inf();
        }
        if (whole)
          for (int i = gt; i < live * DL; i += 128) store_out1(a.out, orow * DL + i, 0.f, a.out_dtype);
        continue;
      }
      const int tok = (pc.row0 + (int)rank * kRows + row) / a.num_heads;
      const int seen = a.causal ? min(pc.kv, pc.kv - pc.rq.q_len + tok + 1) : pc.kv;
      float m = neg_inf(), l = 0.f;
      bool gave_up = false;
      for (int j = 0; j < pc.n; ++j, ++T) {
        const int key0 = (pc.tile0 + j) * kLatentTile + half * 32;   // this thread's 32 keys
        if (!warp_wait(bar(R_SFULL + (T & 1)), (uint32_t)((T >> 1) & 1), a.status)) {
          s_fail[T & 1] = 1;
          gave_up = true;
        }
        tc_fence_after();
        uint32_t s[32];
        tmem_ld32_sync(tmem + lane_off + G::kColS + (uint32_t)(T & 1) * 32u, s);
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(s[i]) * sl2;
        if (__any_sync(0xffffffffu, key0 + 32 > seen)) {
          const int n = min(max(seen - key0, 0), 32);
          const uint32_t bits = n >= 32 ? 0xffffffffu : (1u << n) - 1u;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(bits & (1u << i))) x[i] = neg_inf();
        }
        float top4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int i = 4; i < 32; i += 4)
#pragma unroll
          for (int k = 0; k < 4; ++k) top4[k] = fmaxf(top4[k], x[i + k]);
        const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
        // Lazy rescale: the reference of a row moves only when a score is more than
        // 2^8 above it; only then do the two threads of a row trade their maxima.
        if (bar_any_group(0, gave_up || top > m + kRescaleThreshold)) {
          if (s_fail[T & 1]) {
            ok = false;
            break;
          }
          s_max[half * kRows + row] = top;
          bar_sync_group(0);
          const float mx = fmaxf(s_max[row], s_max[kRows + row]);
          const bool up = mx > m + kRescaleThreshold, had = m != neg_inf();
          // a row without visible keys so far still has O = 0 and l = 0
          const float al = up && had ? ex2(m - mx) : 1.f;
          if (up) m = mx;
          l *= al;
          if (__any_sync(0xffffffffu, up && had)) {
            if (!warp_wait(bar(R_PV + ((T - 1) & 1)), (uint32_t)(((T - 1) >> 1) & 1), a.status))
              s_fail[2] = 1;   // seen at the end of the piece
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < ND * 4; ++c) {
              uint32_t r[32];
              const uint32_t o_tm = tmem + lane_off + (uint32_t)c * 32u;
              tmem_ld32_sync(o_tm, r);
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * al);
              tmem_st32(o_tm, r);
            }
            tmem_wait_st();
          }
          bar_sync_group(0);   // s_max is free again
        }
        // p = exp2(x - m), summed in 32 bits, rounded to the inputs' format for P V
        const float neg = m == neg_inf() ? 0.f : kLatentWeightShift<F16> - m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          x[i] = ex2(x[i] + neg);
          sum[i & 3] += x[i];
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        // P(T) only once P V(T - 2) is complete
        if (T >= 2 && !warp_wait(bar(R_PV + (T & 1)), (uint32_t)(((T >> 1) - 1) & 1), a.status)) {
          s_fail[(T + 1) & 1] = 1;   // seen behind the next tile's barrier
          gave_up = true;
        }
        uint8_t* pb = smem + G::kOffP + (uint32_t)(T & 1) * G::kP + (uint32_t)(row >> 3) * 1024u;
#pragma unroll
        for (int c = 0; c < 4; ++c)   // 8 keys = one 16-byte chunk
          *reinterpret_cast<uint4*>(pb + swz128((uint32_t)(row & 7), (uint32_t)(half * 4 + c))) =
              make_uint4(pack2<F16>(x[8 * c], x[8 * c + 1]), pack2<F16>(x[8 * c + 2], x[8 * c + 3]),
                         pack2<F16>(x[8 * c + 4], x[8 * c + 5]), pack2<F16>(x[8 * c + 6], x[8 * c + 7]));
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive(bar(R_PFULL + (T & 1)));
          else mbar_arrive_cluster(lead(R_PFULL + (T & 1)));
        }
      }
      if (!ok) break;
      ++I;
      next_q(item + 1);

      // ---- output: O / l; each warp turns 32 rows x 128 bytes at a time in the P buffers ----
      s_sum[half * kRows + row] = l;
      if (!warp_wait(bar(R_PV + ((T - 1) & 1)), (uint32_t)(((T - 1) >> 1) & 1), a.status)) s_fail[2] = 1;
      bar_sync_group(0);
      if (s_fail[2]) {
        ok = false;
        break;
      }
      const float total = s_sum[row] + s_sum[kRows + row];
      // != and not >: a sum that is NaN stays one, in the LSE as in the output
      const float inv = total != 0.f ? (whole ? a.output_scale : 1.f) / total : 0.f;
      if (half == 0 && row < live) {
        const float lse = total != 0.f ? m - kLatentWeightShift<F16> + log2f(total) : neg_inf();
        if (!whole) a.ws_lse[prow + row] = lse;
        else if (a.lse != nullptr) a.lse[orow + row] = lse;
      }
      __syncwarp();   // the whole warp loads what follows
      tc_fence_after();
      // the P buffer that the last tile did not use is free, the other one as well:
      // its P V is complete, and the next piece's P(T) waits for both groups' output
      uint8_t* wbuf = smem + G::kOffP + (uint32_t)quad * 4096u;
      auto write = [&](auto* out, int64_t first) {
        using T_ = typename std::remove_pointer<decltype(out)>::type;
        constexpr int W = 128 / (int)sizeof(T_);          // values of a 128-byte piece of a row
        const int r0 = (quad & 1) * 32;                    // the warp's first row
#pragma unroll 1
        for (int c = 0; c < ND * 128; c += W) {
          const int dim = c / 128 * 256 + half * 128 + c % 128;
#pragma unroll
          for (int h = 0; h < W; h += 32) {
            uint32_t r[32];
            tmem_ld32_sync(tmem + lane_off + (uint32_t)(c + h), r);
            constexpr int E = 16 / (int)sizeof(T_);        // values of a 16-byte chunk
#pragma unroll
            for (int k = 0; k < 32 / E; ++k) {
              uint32_t w[4];
              if constexpr (sizeof(T_) == 4) {
#pragma unroll
                for (int x = 0; x < 4; ++x) w[x] = __float_as_uint(__uint_as_float(r[4 * k + x]) * inv);
              } else {
                constexpr bool F = std::is_same<T_, __half>::value;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  w[x] = pack2<F>(__uint_as_float(r[8 * k + 2 * x]) * inv, __uint_as_float(r[8 * k + 2 * x + 1]) * inv);
              }
              *reinterpret_cast<uint4*>(wbuf + swz128((uint32_t)lane, (uint32_t)(h / E + k))) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {   // four rows of 128 bytes at a time
            const int rr = k * 4 + (lane >> 3);
            const uint4 v = *reinterpret_cast<const uint4*>(wbuf + swz128((uint32_t)rr, (uint32_t)(lane & 7)));
            if (r0 + rr < live)
              *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(out + (first + r0 + rr) * DL + dim) +
                                        (lane & 7) * 16) = v;
          }
          __syncwarp();
        }
      };
      if (!whole) write(a.ws_o, prow);
      else if (a.out_dtype == PKA_DTYPE_F32) write(static_cast<float*>(a.out), orow);
      else if (a.out_dtype == PKA_DTYPE_F16) write(static_cast<__half*>(a.out), orow);
      else write(static_cast<__nv_bfloat16*>(a.out), orow);
      tc_fence_before();
      bar_sync_group(0);   // the P buffers are everybody's again
      if (lane == 0) mbar_arrive_remote(lead(R_OFREE));
    }
  }

  tc_fence_before();
  __syncthreads();
  // Nothing of the pair's still runs on the tensor cores, and every commit has landed here.
  // Waited for only now: all of a pair's tiles may take longer than any one wait may.
  if (warp == 1) {
    warp_wait(bar(R_SDONE), 0, a.status);
    warp_wait(bar(R_ODONE), 0, a.status);
  }
  cluster_sync();   // neither CTA's shared memory nor TMEM goes while the pair still uses it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int DL, bool F16>
int launch(const LatentArgs& a, const PairMaps& maps, cudaStream_t stream) {
  auto kern = latent_decode_pair_kernel<DL, F16>;
  static std::atomic<uint64_t> smem_set{0};   // devices whose limit was raised
  cudaError_t e = set_smem_once(kern, (int)Pair<DL>::kSmem, smem_set);
  if (e == cudaSuccess) {
    kern<<<(unsigned)(2 * a.num_segments * a.row_blocks), kThreads, Pair<DL>::kSmem, stream>>>(a, maps);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return cuda_fail(e, "latent_decode_pair_kernel launch");
  return PKA_OK;
}

}  // namespace

int launch_latent_decode_pair(const pka_latent_plan& plan, const LatentArgs& args, const void* pages,
                              int64_t stride_page, cudaStream_t stream) {
  LatentArgs a = args;
  const uint64_t row = (uint64_t)(plan.desc.latent_dim + plan.desc.rope_dim) * 2;
  const uint32_t nc = (uint32_t)plan.desc.latent_dim / 64 + 1;
  PairMaps maps;
  {
    const uint64_t dims[5] = {64, 8, nc, (uint64_t)plan.desc.page_size / 8, (uint64_t)plan.desc.num_pages};
    const uint64_t strides[4] = {row, 128, 8 * row, (uint64_t)stride_page * 2};
    const uint32_t kbox[5] = {64, 8, nc, (uint32_t)std::min(a.box_rows, 32) / 8, 1};
    const uint32_t vbox[5] = {64, 8, 2, (uint32_t)a.box_rows / 8, 1};
    int rc = encode_bf16_map(&maps.keys, pages, 5, dims, strides, kbox);
    if (rc == PKA_OK) rc = encode_bf16_map(&maps.values, pages, 5, dims, strides, vbox);
    if (rc != PKA_OK) return rc;
  }
  a.q_box = 0;
  maps.q = maps.keys;
  if (a.num_heads % 8 == 0 && a.q_stride_head > 0 && (a.q_stride_tok > 0 || plan.total_q == 1)) {
    a.q_box = kRows;
    while (a.num_heads % a.q_box != 0) a.q_box /= 2;
    const uint64_t hs = (uint64_t)a.q_stride_head * 2;
    const uint64_t dims[5] = {64, 8, nc, (uint64_t)a.num_heads / 8, (uint64_t)plan.total_q};
    const uint64_t strides[4] = {hs, 128, 8 * hs, std::max((uint64_t)a.q_stride_tok * 2, (uint64_t)16)};
    const uint32_t box[5] = {64, 8, nc, (uint32_t)a.q_box / 8, 1};
    const int rc = encode_bf16_map(&maps.q, a.q, 5, dims, strides, box);
    if (rc != PKA_OK) return rc;
  }
  const bool f16 = plan.desc.dtype == PKA_DTYPE_F16;
  if (plan.desc.latent_dim == 512)
    return f16 ? launch<512, true>(a, maps, stream) : launch<512, false>(a, maps, stream);
  return f16 ? launch<256, true>(a, maps, stream) : launch<256, false>(a, maps, stream);
}

}  // namespace pka
