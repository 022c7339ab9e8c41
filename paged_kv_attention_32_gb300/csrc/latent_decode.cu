// Absorbed latent decode: s_j = scale * q . row_j over latent_dim + rope_dim
// values, p = softmax(s), o = sum_j p_j row_j[0 .. latent_dim), all heads over
// the same cached rows.  A CTA takes up to 64 query rows (token, head) of a request
// and streams tiles of 64 keys past them, in the transposed form
//   S^T = K Q^T      M=64 (keys), N rows, 576 or 320 columns deep
//   O^T += V^T P^T   M=128 (latent dimensions), N rows, 64 keys deep
// in which few rows are few columns.  A tile is copied once and is both operands.
// The softmax keeps a running reference and sum per row in 32 bits; P is rounded to
// the inputs' type, as they are.  What bounds it is HBM: 2 (latent_dim + 64) bytes a
// key, however many rows share it.  Measured, 152 requests of 4096 keys in pages of 64:
// 256 + 64 columns, 8 / 32 / 64 heads 64 / 65 / 68 us (6.2, 6.2, 6.0 TB/s; a copy
// reaches 6.8); 512 + 64 columns 116 / 117 / 116 us (6.2, 6.2, 6.3 TB/s).  64 ragged
// requests of 32 heads, 512 + 64: 64.5 us against a floor of 47.4: launch, first tile,
// output and merge are the difference.
// Warps: 0 copies, 1 issues S, 2 issues P V, then a group of four per 16 rows for the
// softmax and the output.  TMEM columns: O^T (latent_dim / 128 blocks of N), two S.
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

// ---- the decode kernel -----------------------------------------------------------


// Shared memory and TMEM of latent_dim DL with N query rows.  A stage is a tile
// of 64 keys as blocks of 256 latent dimensions and one of the 64 rotary ones;
// a block is groups of 8 keys, each 4 (rotary: 1) swizzled atoms of 8 x 128
// bytes.  Every block has barriers of its own: scores start with the first that
// lands, and a block is asked for again as soon as its own products are done.
// The rotary block is dead once S is complete, and the weights of the tile (N
// rows of 64, the same layout) are written over it.
template <int DL, int N>
struct Geo {
  static constexpr int NB = DL / 128;                   // 128-wide latent blocks of P V
  static constexpr int NH = DL / 256;                   // 256-wide blocks of a stage
  static constexpr int SG = N / 16;                     // softmax groups: four warps, 16 rows
  static constexpr int kThreads = 96 + 128 * SG;
  static constexpr uint32_t kBlock = 32768, kRope = 8192;
  static constexpr uint32_t kTile = NH * kBlock + kRope;
  static constexpr uint32_t kQBlock = N * 512;          // the queries, laid out like keys
  static constexpr uint32_t kQ = NH * kQBlock + N * 128;
  static constexpr uint32_t kMisc = 512 + (8 + 2) * N * 4;
  static constexpr int kFit = (kSmemLimit - kMisc - kQ) / kTile;
  static constexpr int NS = kFit < 4 ? kFit : 4;        // stages
  static constexpr uint32_t kOffQ = NS * kTile;
  static constexpr uint32_t kOffMisc = kOffQ + kQ;
  static constexpr uint32_t kSmem = kOffMisc + kMisc;
  static constexpr uint32_t kOffR = NH * kBlock;        // inside a stage
  static constexpr uint32_t kColS = NB * N;             // O blocks, then the two S buffers
  static constexpr uint32_t kCols = kColS + 2 * N;
  static constexpr uint32_t kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(NS >= 2 && kSmem <= kSmemLimit, "two stages");
};

// mbarriers.  T counts a CTA's tiles over all its pieces: S, P and P V barriers
// T & 1.  No barrier runs a phase past one that somebody still has to see: S(T)
// is issued once P(T - 2) is written, P(T) written once P V(T - 2) is complete.
enum {
  L_KFULL = 0, L_KEMPTY = 12, L_SFULL = 24, L_PFULL = 26, L_PV = 28, L_QFULL = 30, L_QFREE = 31,
  L_OFREE = 32, L_SDONE = 33, L_ODONE = 34, L_COUNT = 35   // K: three blocks a stage at most
};
static_assert(L_COUNT * 8 + 4 + 48 <= 512, "barriers, TMEM address, failure flags");

// Max or sum of four values each over the eight lanes that share lane % 4.  The
// lanes trade halves, so that each ends with one total: value first_value(lane).
template <typename Op>
__device__ __forceinline__ float reduce_rows(const float* x, int lane, Op op) {
  const bool b4 = lane & 16, b3 = lane & 8;
  float y[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    y[i] = op(b4 ? x[i + 2] : x[i], __shfl_xor_sync(0xffffffffu, b4 ? x[i] : x[i + 2], 16));
  const float z = op(b3 ? y[1] : y[0], __shfl_xor_sync(0xffffffffu, b3 ? y[0] : y[1], 8));
  return op(z, __shfl_xor_sync(0xffffffffu, z, 4));
}
__device__ __forceinline__ int first_value(int lane) { return 2 * ((lane >> 4) & 1) + ((lane >> 3) & 1); }

struct LatentMaps {
  CUtensorMap pool, pool_rope, q, q_rope;
};

// Four values of each of 16 columns: r[i] of lane d holds column i of dimension
// d; afterwards v[k] holds column 4k + lane % 4 of dimensions 4 (lane / 4) on.
__device__ __forceinline__ void transpose_quads(const float* r, float4* v, int lane) {
  const bool odd = lane & 1, high = lane & 2;
  float2 u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? r[2 * i] : r[2 * i + 1], 1);
    u[i] = odd ? make_float2(got, r[2 * i + 1]) : make_float2(r[2 * i], got);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 keep = high ? u[2 * k + 1] : u[2 * k], send = high ? u[2 * k] : u[2 * k + 1];
    const float2 got = make_float2(__shfl_xor_sync(0xffffffffu, send.x, 2),
                                   __shfl_xor_sync(0xffffffffu, send.y, 2));
    v[k] = high ? make_float4(got.x, got.y, keep.x, keep.y) : make_float4(keep.x, keep.y, got.x, got.y);
  }
}

// 16 consecutive columns of TMEM (one dimension per lane) times their factors, as
// rows of the output: column i to row i, `base` being row 0's first dimension of
// this warp.  32-bit values go out as they lie, 128 bytes of a row a store; 16-bit
// ones are turned first, so that a lane has four dimensions of a row.
template <typename T, int DL>
__device__ __forceinline__ void store_columns(uint32_t taddr, const float* factor, int live, T* base,
                                              int lane) {
  uint32_t r[16];
  __syncwarp();   // lanes that stored the last columns and lanes that did not
  tmem_ld16(taddr, r);
  tmem_wait_ld();
  reg_fence<16>(r);
  float f[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 x = reinterpret_cast<const float4*>(factor)[i];
    f[4 * i] = x.x * __uint_as_float(r[4 * i]);
    f[4 * i + 1] = x.y * __uint_as_float(r[4 * i + 1]);
    f[4 * i + 2] = x.z * __uint_as_float(r[4 * i + 2]);
    f[4 * i + 3] = x.w * __uint_as_float(r[4 * i + 3]);
  }
  if constexpr (sizeof(T) == 4) {
    T* dst = base + lane;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < live) dst[i * DL] = f[i];
  } else {
    float4 v[4];
    transpose_quads(f, v, lane);
    T* dst = base + (lane & 3) * DL + (lane >> 2) * 4;
    constexpr bool F = std::is_same<T, __half>::value;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (4 * k + (lane & 3) < live)
        *reinterpret_cast<uint2*>(dst + 4 * k * DL) = make_uint2(pack2<F>(v[k].x, v[k].y), pack2<F>(v[k].z, v[k].w));
  }
}

template <int DL, int N, bool F16>
__global__ void __launch_bounds__(Geo<DL, N>::kThreads, 1)
latent_decode_kernel(const __grid_constant__ LatentArgs a, const __grid_constant__ LatentMaps maps) {
  using G = Geo<DL, N>;
  constexpr int NB = G::NB, NH = G::NH, NS = G::NS, SG = G::SG, NG = 16, C = NG / 4;
  constexpr uint32_t kIdescQK = idesc_bf16_f32(64, N, 0, 0, F16);
  constexpr uint32_t kIdescPV = idesc_bf16_f32(128, N, 1, 0, F16);
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  uint8_t* misc = smem + G::kOffMisc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + L_COUNT * 8);
  float* s_max = reinterpret_cast<float*>(misc + 512);   // [SG][2][4 warps][16]
  float* s_col = s_max + 8 * N;                          // [N] rescale factors, then 1 / l
  int* s_seen = reinterpret_cast<int*>(s_col + N);       // [N] keys each row sees
  float* s_ref = s_col + N;                              // then the rows' reference maxima
  auto bar = [&](int i) -> uint32_t { return sbase + G::kOffMisc + 8u * (uint32_t)i; };

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = tid >> 5;   // 0: copies, 1: S, 2: P V, then the softmax groups
  const int seg = blockIdx.x / a.row_blocks, rb = blockIdx.x % a.row_blocks;

  if (tid == 0) {   // the first piece comes in while the CTA sets up
    ask_line(a.pieces + seg);
    ask_line(a.more + seg);
    for (int s = 0; s < 12; ++s) {
      mbar_init(bar(L_KFULL + s), 1);
      mbar_init(bar(L_KEMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(L_SFULL + s), 1);
      mbar_init(bar(L_PFULL + s), 4 * SG);   // one arrival per softmax warp
      mbar_init(bar(L_PV + s), 1);
    }
    mbar_init(bar(L_QFULL), a.q_box > 0 ? 1 : 4 * SG);
    mbar_init(bar(L_QFREE), 1);
    mbar_init(bar(L_OFREE), 4 * SG);
    mbar_init(bar(L_SDONE), 1);
    mbar_init(bar(L_ODONE), 1);
    for (int i = 0; i < 3 * SG; ++i) tmem_slot[1 + i] = 0;   // failure flags
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), G::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the merge's CTAs may start taking free SMs; they wait for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Pieces pieces(a, seg);

  if (warp == 0) {
    // ---------------- TMA producer: lane i copies box i of a tile ----------------
    if (lane < 4) tma_prefetch_desc(lane == 0 ? &maps.pool : lane == 1 ? &maps.pool_rope
                                    : lane == 2 ? &maps.q : &maps.q_rope);
    const int boxes = kLatentTile / a.box_rows, groups = a.box_rows / 8;
    Ring<NS> kp;
    int nk = 0, blocks = 0, I = 0;   // stages and blocks asked for so far, pieces
    bool ok = true;
    for (int item = 0; ok && pieces.has(item); ++item) {
      const Piece pc(a, pieces[item], rb, N);
      if (pc.n == 0) continue;
      if (a.q_box > 0) {   // whole groups of 8 heads: the queries come by TMA too
        if (I > 0 && !(ok = warp_wait(bar(L_QFREE), (uint32_t)((I - 1) & 1), a.status))) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(L_QFULL), G::kQ);
        __syncwarp();
        if (lane < N / a.q_box) {   // rows past the request's last are copied, and never stored
          const int r = pc.row0 + lane * a.q_box;
          const int h8 = r % a.num_heads / 8, t = pc.rq.q_start + r / a.num_heads;
          const uint32_t g8 = (uint32_t)(lane * a.q_box / 8), dst = sbase + G::kOffQ;
          for (int h = 0; h < NH; ++h)
            tma_load_5d(dst + (uint32_t)h * G::kQBlock + g8 * 4096u, &maps.q, bar(L_QFULL), 0, 0, 4 * h, h8, t);
          tma_load_5d(dst + NH * G::kQBlock + g8 * 1024u, &maps.q_rope, bar(L_QFULL), 0, 0, 4 * NH, h8, t);
        }
        __syncwarp();
      }
      ++I;
      PageWalk walk(a, pc, lane * a.box_rows, lane < boxes);
      // With two stages the tile behind them is asked for in L2: one box at a time in
      // flight a stage is too little for HBM (152 requests of 4096 keys, 64 heads, 512 +
      // 64: 123 -> 116 us; a request of 131072 among 15 57.2 -> 58.4).  With three and more
      // stages it costs more than it gives (512 + 64, 8 heads 116 -> 114; 256 + 64 64 -> 68).
      // The other row blocks read the same keys at about the same time.
      const bool ask_ahead = NS == 2 && rb == 0;
      PageWalk ahead = walk;
      if (ask_ahead)
        for (int j = 0; j < NS; ++j) ahead.next_tile();
      for (int j = 0; j < pc.n; ++j) {
        const int page = walk.page(), slot8 = walk.slot / 8;
        walk.next_tile();
        const uint32_t dst = sbase + (uint32_t)kp.slot * G::kTile;
        for (int h = 0; h <= NH; ++h) {   // blocks in the order P V lets go of them
          const int i = 3 * kp.slot + h;
          if (nk >= NS && !(ok = warp_wait(bar(L_KEMPTY + i), kp.parity ^ 1u, a.status))) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(L_KFULL + i), h < NH ? G::kBlock : G::kRope);
          __syncwarp();
          if (lane < boxes)
            tma_load_5d(dst + (uint32_t)h * G::kBlock + (uint32_t)(lane * groups) * (h < NH ? 4096u : 1024u),
                        h < NH ? &maps.pool : &maps.pool_rope, bar(L_KFULL + i), 0, 0, 4 * h, slot8, page);
          __syncwarp();
          ++blocks;
        }
        if (!ok) break;
        if (ask_ahead && j + NS < pc.n) {
          if (lane < boxes) {
            for (int h = 0; h < NH; ++h) tma_prefetch_5d(&maps.pool, 0, 0, 4 * h, ahead.slot / 8, ahead.page());
            tma_prefetch_5d(&maps.pool_rope, 0, 0, 4 * NH, ahead.slot / 8, ahead.page());
          }
          ahead.next_tile();
        }
        kp.next();
        ++nk;
      }
    }
    if (!ok) {   // give the copies already issued a bounded chance to land
      for (int i = max(0, blocks - NS * (NH + 1)); i < blocks; ++i)
        mbar_wait(bar(L_KFULL + 3 * (i / (NH + 1) % NS) + i % (NH + 1)),
                  (uint32_t)((i / (NH + 1) / NS) & 1), nullptr);
      if (a.q_box > 0 && I > 0) mbar_wait(bar(L_QFULL), (uint32_t)((I - 1) & 1), nullptr);
    }
  } else if (warp == 1) {
    // ---------------- issues S^T = K Q^T ----------------
    // Its own warp, so that neither products of keys that are still on their way
    // hold up a ready P V nor the other way round.
    const uint64_t dk = smem_desc_sw128(sbase, 16u, 4096u);
    const uint64_t dq = smem_desc_sw128(sbase + G::kOffQ, 16u, 4096u);
    const uint64_t dkr = smem_desc_sw128(sbase + G::kOffR, 16u, 1024u);
    const uint64_t dqr = smem_desc_sw128(sbase + G::kOffQ + NH * G::kQBlock, 16u, 1024u);
    // rows past the last token may hold anything, and 0 * inf is not 0: clear them
    // to the end of their box (boxes past it brought zeros)
    auto clear_rows = [&](uint32_t off, int atoms, int live) {
      const int end = (live + a.box_rows - 1) / a.box_rows * a.box_rows;
      for (int i = lane; i < (end - live) * atoms * 8; i += 32) {
        const int r = live + i / (atoms * 8), c = i % (atoms * 8);
        *reinterpret_cast<uint4*>(smem + off + (uint32_t)((r >> 3) * atoms + (c >> 3)) * 1024u +
                                  (uint32_t)(r & 7) * 128u + (uint32_t)(c & 7) * 16u) =
            make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    Ring<NS> kp;
    int T = 0, I = 0;   // tiles and non-empty pieces before this one
    bool ok = true;
    for (int item = 0; ok && pieces.has(item); ++item) {
      const Piece pc(a, pieces[item], rb, N);
      if (pc.n == 0) continue;
      ok = warp_wait(bar(L_QFULL), (uint32_t)(I & 1), a.status);
      ++I;
      for (int j = 0; ok && j < pc.n; ++j, ++T) {
        // P(T - 2) written means S(T - 2) read: this S buffer is free
        ok = T < 2 || warp_wait(bar(L_PFULL + (T & 1)), (uint32_t)(((T >> 1) - 1) & 1), a.status);
        const int live = pc.kv - (pc.tile0 + j) * kLatentTile;
        const uint32_t d = tmem + G::kColS + (uint32_t)(T & 1) * N, off = (uint32_t)kp.slot * G::kTile;
#pragma unroll
        for (int h = 0; h <= NH; ++h) {   // 64 keys x N rows += 256 columns of each, then 64
          ok = ok && warp_wait(bar(L_KFULL + 3 * kp.slot + h), kp.parity, a.status);
          if (!ok) break;
          if (live < kLatentTile) clear_rows(off + (uint32_t)h * G::kBlock, h < NH ? 4 : 1, live);
          tc_fence_after();
          if (h < NH) {
            const uint64_t x = dk + (off + (uint32_t)h * G::kBlock) / 16, y = dq + h * (G::kQBlock / 16);
#pragma unroll
            for (int c = 0; c < 4; ++c) umma_ss_k4(d, x + c * 64, y + c * 64, kIdescQK, h + c > 0 ? 1u : 0u);
          } else {
            umma_ss_k4(d, dkr + off / 16, dqr, kIdescQK, 1u);
          }
        }
        if (!ok) break;
        umma_commit_elect(bar(L_SFULL + (T & 1)));
        kp.next();
      }
      if (ok) umma_commit_elect(bar(L_QFREE));
    }
    umma_commit_elect(bar(L_SDONE));
    warp_wait(bar(L_SDONE), 0, a.status);   // nothing of this warp's still runs on the tensor core
  } else if (warp == 2) {
    // ---------------- issues O^T += V^T P^T ----------------
    const uint64_t dv = smem_desc_sw128(sbase, 1024u, 4096u);
    const uint64_t dp = smem_desc_sw128(sbase + G::kOffR, 16u, 1024u);
    Ring<NS> kp;
    int T = 0, I = 0;
    bool ok = true;
    for (int item = 0; ok && pieces.has(item); ++item) {
      const Piece pc(a, pieces[item], rb, N);
      if (pc.n == 0) continue;
      for (int j = 0; j < pc.n; ++j, ++T) {
        ok = warp_wait(bar(L_PFULL + (T & 1)), (uint32_t)((T >> 1) & 1), a.status);
        if (ok && j == 0 && I > 0) ok = warp_wait(bar(L_OFREE), (uint32_t)((I - 1) & 1), a.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t off = (uint32_t)kp.slot * G::kTile;
#pragma unroll
        for (int b = 0; b < NB; ++b) {   // 128 dims x N rows += 64 keys
          umma_ss_k4_steps<2 * 4096 / 16, 2>(tmem + (uint32_t)b * N,
                                             dv + (off + (uint32_t)(b >> 1) * G::kBlock + (b & 1) * 2048u) / 16,
                                             dp + off / 16, kIdescPV, j > 0 ? 1u : 0u);
          if (b & 1) umma_commit_elect(bar(L_KEMPTY + 3 * kp.slot + (b >> 1)));
        }
        umma_commit_elect(bar(L_KEMPTY + 3 * kp.slot + NH));
        umma_commit_elect(bar(L_PV + (T & 1)));
        kp.next();
      }
      ++I;
    }
    umma_commit_elect(bar(L_ODONE));
    warp_wait(bar(L_ODONE), 0, a.status);
  } else {
    // ---------------- softmax and output: group g takes rows g NG .. ----------------
    const int g = (warp - 3) >> 2, quad = warp & 3;     // TMEM lanes 32 quad .. + 31
    const int gt = ((warp - 3) & 3) * 32 + lane;        // thread of the group
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int col0 = 2 * (lane & 3);   // this thread's columns: g NG + 8j + col0 + {0, 1}
    const int gc = g * NG;
    const float sl2 = a.scale_log2;
    volatile int* s_fail = reinterpret_cast<volatile int*>(tmem_slot + 1 + 3 * g);
    float* g_max = s_max + g * 8 * NG;

    // queries by plain loads (heads not a multiple of 8), laid out like keys
    auto load_q = [&](const Piece& pc) {
      constexpr int V = (DL + kLatentRopeDim) / 8;   // 16-byte pieces of a row
#pragma unroll 4
      for (int i = g * 128 + gt; i < N * V; i += 128 * SG) {
        const int r = i / V, c = i % V;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < pc.rows) {
          const int tok = (pc.row0 + r) / a.num_heads, h = (pc.row0 + r) % a.num_heads;
          x = __ldg(reinterpret_cast<const uint4*>(
                        static_cast<const uint16_t*>(a.q) + (int64_t)(pc.rq.q_start + tok) * a.q_stride_tok +
                        (int64_t)h * a.q_stride_head) + c);
        }
        const uint32_t at = c < DL / 8 ? (uint32_t)(c >> 5) * G::kQBlock + (uint32_t)(r >> 3) * 4096u +
                                             (uint32_t)((c >> 3) & 3) * 1024u
                                       : NH * G::kQBlock + (uint32_t)(r >> 3) * 1024u;
        *reinterpret_cast<uint4*>(smem + G::kOffQ + at + swz128((uint32_t)(r & 7), (uint32_t)(c & 7))) = x;
      }
      fence_proxy_async_smem();   // generic writes -> the tensor core's operand reads
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L_QFULL));
    };
    // the next piece that has tiles, from `item` on; the last S of the one before
    // is complete for this thread's group, and QFREE says so for both
    int I = 0;
    bool ok = true;
    auto next_q = [&](int item) {
      if (a.q_box > 0) return;
      for (; pieces.has(item); ++item) {
        const Piece pc(a, pieces[item], rb, N);
        if (pc.n > 0) {
          if (I > 0 && !warp_wait(bar(L_QFREE), (uint32_t)((I - 1) & 1), a.status)) s_fail[2] = 1;
          load_q(pc);
          return;
        }
      }
    };
    next_q(0);

    Ring<NS> kp;
    int T = 0;
    for (int item = 0; ok && pieces.has(item); ++item) {
      const Piece pc(a, pieces[item], rb, N);
      if (pc.rows <= 0) continue;
      const bool whole = pc.part < 0;
      const int64_t orow = (int64_t)pc.rq.q_start * a.num_heads + pc.row0;   // first output row
      const int64_t prow = (int64_t)pc.rq.part_base +
                           (int64_t)max(pc.part, 0) * pc.rq.q_len * a.num_heads + pc.row0;
      if (pc.n == 0) {   // no keys here: zero rows, or a piece that weighs nothing
        for (int i = g * 128 + gt; i < pc.rows; i += 128 * SG) {
          if (!whole) a.ws_lse[prow + i] = neg_inf();
          else if (a.lse != nullptr) a.lse[orow + i] = neg_inf();
        }
        if (whole)
          for (int i = g * 128 + gt; i < pc.rows * DL; i += 128 * SG)
            store_out1(a.out, orow * DL + i, 0.f, a.out_dtype);
        continue;
      }
      if (gt < NG) {
        const int tok = (pc.row0 + gc + gt) / a.num_heads;
        s_seen[gc + gt] = a.causal ? min(pc.kv, pc.kv - pc.rq.q_len + tok + 1) : pc.kv;
      }
      // the first row of the block sees the fewest keys
      const int seen_min =
          a.causal ? min(pc.kv, pc.kv - pc.rq.q_len + pc.row0 / a.num_heads + 1) : pc.kv;
      float m[C], l[C];
#pragma unroll
      for (int q = 0; q < C; ++q) {
        m[q] = neg_inf();
        l[q] = 0.f;
      }
      bool gave_up = false;
      bar_sync_group(g);
      for (int j = 0; j < pc.n; ++j, ++T) {
        const int key0 = (pc.tile0 + j) * kLatentTile;
        if (!warp_wait(bar(L_SFULL + (T & 1)), (uint32_t)((T >> 1) & 1), a.status)) {
          s_fail[T & 1] = 1;
          gave_up = true;
        }
        tc_fence_after();
        uint32_t s[NG / 2];
        const uint32_t s_tm = tmem + lane_off + G::kColS + (uint32_t)(T & 1) * N + (uint32_t)gc;
        tmem_ld_frag2(s_tm, s);
        tmem_wait_ld();
        reg_fence<NG / 2>(s);
        float x[NG / 2];
#pragma unroll
        for (int i = 0; i < NG / 2; ++i) x[i] = __uint_as_float(s[i]) * sl2;
        if (key0 + kLatentTile > seen_min) {
          const int k = key0 + quad * 16 + (lane >> 2);
#pragma unroll
          for (int jj = 0; jj < NG / 8; ++jj)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int seen = s_seen[gc + 8 * jj + col0 + e];
              if (k >= seen) x[4 * jj + e] = neg_inf();
              if (k + 8 >= seen) x[4 * jj + 2 + e] = neg_inf();
            }
        }
        // Lazy rescale: the reference of a row moves only when a score is more than
        // 2^8 above it, so most tiles need no maximum at all, just the word of every
        // thread of the group that none of its scores is.
        bool grow = gave_up;
#pragma unroll
        for (int q = 0; q < C; ++q) {
          const float top = fmaxf(x[4 * (q >> 1) + (q & 1)], x[4 * (q >> 1) + 2 + (q & 1)]);
          grow = grow || top > m[q] + kRescaleThreshold;
        }
        if (bar_any_group(g, grow)) {
          if (s_fail[T & 1]) {
            ok = false;
            break;
          }
          // row maxima over the tile's 64 keys: lanes, then warps
          float mx[C];
#pragma unroll
          for (int q = 0; q < C; ++q)
            mx[q] = fmaxf(x[4 * (q >> 1) + (q & 1)], x[4 * (q >> 1) + 2 + (q & 1)]);
          float* wm = g_max + (T & 1) * 4 * NG;
          wm[quad * NG + (lane & 3) * C + first_value(lane)] =
              reduce_rows(mx, lane, [](float u, float v) { return fmaxf(u, v); });
          bar_sync_group(g);
          float4 u = *reinterpret_cast<const float4*>(wm + (lane & 3) * C);
#pragma unroll
          for (int w = 1; w < 4; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(wm + w * NG + (lane & 3) * C);
            u = make_float4(fmaxf(u.x, v.x), fmaxf(u.y, v.y), fmaxf(u.z, v.z), fmaxf(u.w, v.w));
          }
          mx[0] = u.x;
          mx[1] = u.y;
          mx[2] = u.z;
          mx[3] = u.w;
          // Every warp of the group holds the same maxima, so all decide alike.  A row
          // without visible keys so far still has O = 0 and l = 0 and takes its first
          // reference without a rescale.
          float al[C];
          bool rescale = false;
#pragma unroll
          for (int q = 0; q < C; ++q) {
            const bool up = mx[q] > m[q] + kRescaleThreshold, had = m[q] != neg_inf();
            al[q] = up && had ? ex2(m[q] - mx[q]) : 1.f;
            rescale = rescale || (up && had);
            if (up) m[q] = mx[q];
          }
          if (__any_sync(0xffffffffu, rescale)) {
            if (!warp_wait(bar(L_PV + ((T - 1) & 1)), (uint32_t)(((T - 1) >> 1) & 1), a.status))
              s_fail[2] = 1;
            tc_fence_after();
            if (gt < 4)
#pragma unroll
              for (int q = 0; q < C; ++q) s_col[gc + 8 * (q >> 1) + col0 + (q & 1)] = al[q];
            bar_sync_group(g);
            if (s_fail[2]) {
              ok = false;
              break;
            }
#pragma unroll
            for (int q = 0; q < C; ++q) l[q] *= al[q];
#pragma unroll 1
            for (int c = 0; c < NB; ++c) {
              uint32_t r[NG];
              const uint32_t o_tm = tmem + lane_off + (uint32_t)(c * N + gc);
              tmem_ld16(o_tm, r);
              tmem_wait_ld();
              reg_fence<NG>(r);
#pragma unroll
              for (int i = 0; i < NG; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * s_col[gc + i]);
              tmem_st16(o_tm, r);
            }
            tmem_wait_st();
            bar_sync_group(g);   // s_col is free again
          }
        }
        // p = exp2(x - m), summed in 32 bits, rounded to the inputs' format for P V
#pragma unroll
        for (int q = 0; q < C; ++q) {
          const float neg = m[q] == neg_inf() ? 0.f : kLatentWeightShift<F16> - m[q];
          const int i = 4 * (q >> 1) + (q & 1);
          x[i] = ex2(x[i] + neg);
          x[i + 2] = ex2(x[i + 2] + neg);
          l[q] += x[i] + x[i + 2];
        }
        // P(T) only once P V(T - 2) is complete (nearly always it is): nobody then
        // waits for a phase of the P and P V barriers that is not the next one
        if (T >= 2 && !warp_wait(bar(L_PV + (T & 1)), (uint32_t)(((T >> 1) - 1) & 1), a.status)) {
          s_fail[(T + 1) & 1] = 1;   // seen behind the next tile's barrier
          gave_up = true;
        }
        // it takes the place of the tile's rotary columns
        const uint32_t pb = sbase + (uint32_t)kp.slot * G::kTile + G::kOffR;
        kp.next();
#pragma unroll
        for (int jj = 0; jj < NG / 8; jj += 2) {
          // matrices: rows 8jj.. keys 0-7 and 8-15 of the warp, rows 8(jj + 1).. alike
          const int mt = lane >> 3;
          const uint32_t row = (uint32_t)(gc + 8 * (jj + (mt >> 1)) + (lane & 7));
          stmatrix_x4_trans(pb + swz128(row, (uint32_t)(2 * quad + (mt & 1))),
                            pack2<F16>(x[4 * jj], x[4 * jj + 1]),
                            pack2<F16>(x[4 * jj + 2], x[4 * jj + 3]),
                            pack2<F16>(x[4 * jj + 4], x[4 * jj + 5]),
                            pack2<F16>(x[4 * jj + 6], x[4 * jj + 7]));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L_PFULL + (T & 1)));
      }
      if (!ok) break;
      ++I;
      next_q(item + 1);

      // ---- output: O^T / l, one latent dimension per lane of a 128-wide block ----
      float* s_sum = g_max + (T & 1) * 4 * NG;   // the half the last tile did not use
      s_sum[quad * NG + (lane & 3) * C + first_value(lane)] =
          reduce_rows(l, lane, [](float u, float v) { return u + v; });
      if (gt < 4)
#pragma unroll
        for (int q = 0; q < C; ++q) s_ref[gc + 8 * (q >> 1) + col0 + (q & 1)] = m[q] - kLatentWeightShift<F16>;
      if (!warp_wait(bar(L_PV + ((T - 1) & 1)), (uint32_t)(((T - 1) >> 1) & 1), a.status)) s_fail[2] = 1;
      bar_sync_group(g);
      if (s_fail[2]) {
        ok = false;
        break;
      }
      if (gt < NG) {
        const int q = ((gt & 7) >> 1) * C + 2 * (gt >> 3) + (gt & 1);   // column gt in s_sum
        const float sum = (s_sum[q] + s_sum[NG + q]) + (s_sum[2 * NG + q] + s_sum[3 * NG + q]);
        const int n = gc + gt;
        // != and not >: a sum that is NaN stays one, in the LSE as in the output
        s_col[n] = sum != 0.f ? (whole ? a.output_scale : 1.f) / sum : 0.f;
        if (n < pc.rows) {
          const float lse = sum != 0.f ? s_ref[n] + log2f(sum) : neg_inf();
          if (!whole) a.ws_lse[prow + n] = lse;
          else if (a.lse != nullptr) a.lse[orow + n] = lse;
        }
      }
      bar_sync_group(g);
      tc_fence_after();
      auto write = [&](auto* out, int64_t row) {
        out += (row + gc) * DL + quad * 32;
#pragma unroll 1
        for (int blk = 0; blk < DL / 128; ++blk)
          store_columns<typename std::remove_pointer<decltype(out)>::type, DL>(
              tmem + lane_off + (uint32_t)(blk * N + gc), s_col + gc, pc.rows - gc, out + blk * 128, lane);
      };
      if (!whole) write(a.ws_o, prow);
      else if (a.out_dtype == PKA_DTYPE_F32) write(static_cast<float*>(a.out), orow);
      else if (a.out_dtype == PKA_DTYPE_F16) write(static_cast<__half*>(a.out), orow);
      else write(static_cast<__nv_bfloat16*>(a.out), orow);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L_OFREE));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kTmemCols);
  }
}

// The pieces of a cut request: out = sum_c w_c o_c / sum_c w_c with
// w_c = 2^(lse_c - max).  A short chain of dependent loads per row, and few
// instructions: with four values a thread (each making every weight for itself)
// the issue slots bounded it (5760 rows of 2-3 pieces of 512 values 9.5 us; with eight 7.0).  A
// row of up to kLatentFewPieces (nearly all) is one CTA's, every LSE and four
// pieces at a time asked for at once.  A row of more is shared out to 8 CTAs of 64 (32)
// dimensions, whose four groups of threads deal the pieces out; the planner lists
// such requests first.  Measured with 16 / 64 / 128 dimensions a CTA, 64 heads, the whole
// decode: 16 requests in 9 pieces each 49 / 27 / 25 us, 4 in 38 43 / 31 / 32, one in 152
// 53 / 53 / 59.  Launched while the decode still runs, it
// waits for that grid's end.
template <int DL>
__global__ void __launch_bounds__(DL / 8, 1024 / (DL / 8))
latent_merge_kernel(const __grid_constant__ LatentArgs a) {
  constexpr int T = DL / 8, GROUPS = 4, QUADS = T / GROUPS, SLABS = 8;
  static_assert(SLABS * QUADS * 4 == DL, "every dimension once");
  __shared__ float4 s_o[GROUPS - 1][QUADS];
  const int tid = threadIdx.x, lane = tid & 31;
  const int many_ctas = a.num_many * a.max_rows * SLABS;
  const bool few = (int)blockIdx.x >= many_ctas;
  const int at = few ? a.num_many * a.max_rows + (int)blockIdx.x - many_ctas : blockIdx.x / SLABS;
  const int which = at / a.max_rows, r = at - which * a.max_rows;
  const LatentReq rq = a.splits[which];
  const int rows = rq.q_len * a.num_heads, n = rq.n_parts;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (r >= rows) return;
  const int64_t row = (int64_t)rq.q_start * a.num_heads + r, p0 = (int64_t)rq.part_base + r;
  const float* lse = a.ws_lse + p0;
  const float4* part = reinterpret_cast<const float4*>(a.ws_o + p0 * DL);
  const int64_t step = (int64_t)rows * (DL / 4);   // from piece to piece
  // A piece without keys (LSE -inf) has no output rows, what lies there is not used.
  auto lse_of = [&](int c) { return c < n ? __ldcg(lse + (int64_t)c * rows) : neg_inf(); };
  float m = neg_inf(), sum = 0.f;
  auto add = [](float4& o, float w, float4 v) {
    o.x += w * v.x;
    o.y += w * v.y;
    o.z += w * v.z;
    o.w += w * v.w;
  };
  auto store = [&](int x, float4 o) {
    const float f[4] = {o.x, o.y, o.z, o.w};
    store_out<4>(a.out, row * DL + x * 4, f, sum != 0.f ? a.output_scale / sum : 0.f, a.out_dtype);
  };
  if (few) {
    float4 o0 = make_float4(0.f, 0.f, 0.f, 0.f), o1 = o0, v0[4], v1[4];
    float s[4], more[kLatentFewPieces - 4];
    auto ask = [&](int c0) {
      const float4* src = part + c0 * step + tid;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (c0 + i < n) {
          v0[i] = __ldcg(src);
          v1[i] = __ldcg(src + T);
        }
        src += step;
      }
    };
    auto take = [&](const float* l, int c0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + i < n && l[i] != neg_inf()) {
          const float w = ex2(l[i] - m);
          sum += w;
          add(o0, w, v0[i]);
          add(o1, w, v1[i]);
        }
    };
    ask(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = lse_of(i);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, s[i]);
    if (n > 4) {
#pragma unroll
      for (int i = 0; i < kLatentFewPieces - 4; ++i) {
        more[i] = lse_of(4 + i);
        m = fmaxf(m, more[i]);
      }
    }
    take(s, 0);
    if (n > 4) {
      ask(4);
      take(more, 4);
    }
    store(tid, o0);
    store(tid + T, o1);
    if (tid == 0 && a.lse != nullptr) a.lse[row] = sum != 0.f ? m + log2f(sum) : neg_inf();
    return;
  }
  const int g = tid / QUADS, x = blockIdx.x % SLABS * QUADS + tid % QUADS;
  constexpr int W = 8;   // pieces a thread has in flight
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f), v[W];
  auto ask = [&](int c0) {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (c0 + i * GROUPS < n) v[i] = __ldcg(part + (int64_t)(c0 + i * GROUPS) * step + x);
  };
  ask(g);
  // each warp for itself: four pieces a lane and round, a running maximum and sum
  for (int c0 = 0; c0 < n; c0 += 128) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = lse_of(c0 + 32 * i + lane);
    float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (top > m) {
      sum *= m == neg_inf() ? 0.f : ex2(m - top);
      m = top;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += y[i] == neg_inf() ? 0.f : ex2(y[i] - m);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  for (int c0 = g; c0 < n; c0 += GROUPS * W) {
    if (c0 > g) ask(c0);
    float s[W];
#pragma unroll
    for (int i = 0; i < W; ++i) s[i] = lse_of(c0 + i * GROUPS);
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (s[i] != neg_inf()) add(o, ex2(s[i] - m), v[i]);
  }
  if (g > 0) s_o[g - 1][tid % QUADS] = o;
  __syncthreads();
  if (g > 0) return;
#pragma unroll
  for (int i = 0; i < GROUPS - 1; ++i) add(o, 1.f, s_o[i][tid]);
  store(x, o);
  if (x == 0 && a.lse != nullptr) a.lse[row] = sum != 0.f ? m + log2f(sum) : neg_inf();
}

template <int DL, int N, bool F16>
cudaError_t launch_tiles(const LatentArgs& a, const LatentMaps& maps, cudaStream_t stream) {
  auto kern = latent_decode_kernel<DL, N, F16>;
  static std::atomic<uint64_t> smem_set{0};   // devices whose limit was raised
  const cudaError_t e = set_smem_once(kern, (int)Geo<DL, N>::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(a.num_segments * a.row_blocks), Geo<DL, N>::kThreads, Geo<DL, N>::kSmem, stream>>>(
      a, maps);
  return cudaGetLastError();
}

template <int DL, bool F16>
int launch(const pka_latent_plan& plan, const LatentArgs& a, const LatentMaps& maps,
           cudaStream_t stream) {
  cudaError_t e = plan.row_tile == 16   ? launch_tiles<DL, 16, F16>(a, maps, stream)
                  : plan.row_tile == 32 ? launch_tiles<DL, 32, F16>(a, maps, stream)
                                        : launch_tiles<DL, 64, F16>(a, maps, stream);
  if (e != cudaSuccess) return cuda_fail(e, "latent_decode_kernel launch");
  return PKA_OK;
}

template <int DL>
int launch_merge(const LatentArgs& a, cudaStream_t stream) {
  if (a.num_splits > 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.num_splits + a.num_many * 7) * (unsigned)a.max_rows);   // 8 CTAs a row of many
    cfg.blockDim = dim3(DL / 8);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, latent_merge_kernel<DL>, a);
    if (e != cudaSuccess) return cuda_fail(e, "latent_merge_kernel launch");
  }
  return PKA_OK;
}

}  // namespace

namespace {

int launch_single(const pka_latent_plan& plan, const LatentArgs& args, const void* pages,
                  int64_t stride_page, cudaStream_t stream) {
  LatentArgs a = args;
  // The pool as (64 columns, slot in 8, column chunk, slot / 8, page): one box of
  // box_rows rows and four chunks (one for the rotary columns) lands as groups of
  // 8 keys, each a swizzled 8 x 128 byte atom per chunk.  Groups are evenly spaced
  // whatever the page size, so 64 keys from any number of pages are one operand,
  // as keys (K-major) and as values (MN-major).
  const uint64_t row = (uint64_t)(plan.desc.latent_dim + plan.desc.rope_dim) * 2;
  const uint64_t nc = (uint64_t)plan.desc.latent_dim / 64 + 1;
  auto encode = [](CUtensorMap* four, CUtensorMap* one, const void* base, const uint64_t* dims,
                   const uint64_t* strides, uint32_t groups) {
    const uint32_t box4[5] = {64, 8, 4, groups, 1}, box1[5] = {64, 8, 1, groups, 1};
    const int rc = encode_bf16_map(four, base, 5, dims, strides, box4);
    return rc != PKA_OK ? rc : encode_bf16_map(one, base, 5, dims, strides, box1);
  };
  LatentMaps maps;
  {
    const uint64_t dims[5] = {64, 8, nc, (uint64_t)plan.desc.page_size / 8, (uint64_t)plan.desc.num_pages};
    const uint64_t strides[4] = {row, 128, 8 * row, (uint64_t)stride_page * 2};
    const int rc = encode(&maps.pool, &maps.pool_rope, pages, dims, strides, (uint32_t)a.box_rows / 8);
    if (rc != PKA_OK) return rc;
  }
  // The queries alike, where heads come in groups of 8: (64 columns, head in 8,
  // chunk, head / 8, token), boxes of q_box heads that stay inside a token.
  a.q_box = 0;
  maps.q = maps.pool;
  maps.q_rope = maps.pool;
  if (a.num_heads % 8 == 0 && a.q_stride_head > 0 && (a.q_stride_tok > 0 || plan.total_q == 1)) {
    a.q_box = plan.row_tile;
    while (a.num_heads % a.q_box != 0) a.q_box /= 2;
    const uint64_t hs = (uint64_t)a.q_stride_head * 2;
    const uint64_t dims[5] = {64, 8, nc, (uint64_t)a.num_heads / 8, (uint64_t)plan.total_q};
    const uint64_t strides[4] = {hs, 128, 8 * hs, std::max((uint64_t)a.q_stride_tok * 2, (uint64_t)16)};
    const int rc = encode(&maps.q, &maps.q_rope, a.q, dims, strides, (uint32_t)a.q_box / 8);
    if (rc != PKA_OK) return rc;
  }
  const bool f16 = plan.desc.dtype == PKA_DTYPE_F16;
  if (plan.desc.latent_dim == 512)
    return f16 ? launch<512, true>(plan, a, maps, stream) : launch<512, false>(plan, a, maps, stream);
  return f16 ? launch<256, true>(plan, a, maps, stream) : launch<256, false>(plan, a, maps, stream);
}

}  // namespace

int launch_latent_decode(const pka_latent_plan& plan, const LatentArgs& a, const void* pages,
                         int64_t stride_page, cudaStream_t stream) {
  const int rc = plan.row_tile == 128 ? launch_latent_decode_pair(plan, a, pages, stride_page, stream)
                                      : launch_single(plan, a, pages, stride_page, stream);
  if (rc != PKA_OK) return rc;
  return plan.desc.latent_dim == 512 ? launch_merge<512>(a, stream) : launch_merge<256>(a, stream);
}

}  // namespace pka
