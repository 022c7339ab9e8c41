// Host planners of the latent decode and prefill.  The decode's:
//
// All heads of a request read the same cached row, so a CTA takes a block of
// up to 64 query rows (token, head), a pair of CTAs one of 128, and streams keys
// past them.  Key tiles of 64 are dealt to as many segments of equal cost as there
// are CTAs (pairs) per row block, each one of them for the whole run: requests are
// laid end to end and cut where a segment is full, so at most two pieces of a segment
// belong to requests that are cut, whatever the lengths.  A piece costs its tiles plus
// a fixed part (its queries in, its output out).  The pieces of a cut request meet in a
// merge over their base-2 LSEs.
#include <algorithm>
#include <cmath>
#include <climits>
#include <queue>

#include "host_common.h"
#include "latent.h"

namespace pka {

namespace {
// A piece's fixed cost, in tiles.  Measured with 0 / 1 / 2 / 4: 64 ragged requests of 32
// heads 67.7 / 66.9 / 66.7 / 67.0 us, of 128 heads 87.6 / 84.7 / 84.0 / 83.7, one of
// 131072 keys among 15 59.3 / 57.7 / 57.5 / 58.2.
constexpr int64_t kItemCost = 2;
// Tiles below which a request is not cut further.  With 2 / 4 / 8: 4 short requests
// 7.8 / 8.3 / 10.4 us, 64 ragged ones 65.2 / 66.7 / 68.0.
constexpr int64_t kMinPiece = 2;
constexpr int32_t kMaxRows = 65536;
constexpr int32_t kMaxSms = 1024;
// the prefill's, in tiles of 64 keys for 256 rows (0.4 us each where pairs share SMs)
constexpr int64_t kPrefillItemCost = 3;   // a piece's queries in and output out: 1 and 6 measure alike
constexpr int64_t kPrefillMinPiece = 8;   // below which a tile is not cut further
constexpr int64_t kPrefillCutCost = 12;   // the merge of pieces: 4 to 8 us, whatever their number
}  // namespace

int build_latent_plan(pka_latent_plan& p, const pka_latent_desc& d_in, const int32_t* seq,
                      const int32_t* indptr) {
  pka_latent_desc d = d_in;
  PKA_CHECK_ARG(d.batch_size >= 1, "batch_size must be >= 1 (got %d)", d.batch_size);
  PKA_CHECK_ARG(seq != nullptr, "seq_lens_kv_host is NULL");
  PKA_CHECK_ARG(d.num_heads >= 1, "num_heads must be >= 1 (got %d)", d.num_heads);
  if (d.num_heads > 1024)
    return fail(PKA_ERR_UNSUPPORTED, "num_heads must be <= 1024 (got %d)", d.num_heads);
  if (d.latent_dim != 256 && d.latent_dim != 512)
    return fail(PKA_ERR_UNSUPPORTED, "latent_dim must be 256 or 512 (got %d)", d.latent_dim);
  if (d.rope_dim != kLatentRopeDim)
    return fail(PKA_ERR_UNSUPPORTED, "rope_dim must be %d (got %d)", kLatentRopeDim, d.rope_dim);
  if (d.page_size < 8 || d.page_size > 256 || d.page_size % 8 != 0)
    return fail(PKA_ERR_UNSUPPORTED, "page_size must be a multiple of 8 in [8, 256] (got %d)",
                d.page_size);
  if (d.dtype != PKA_DTYPE_BF16 && d.dtype != PKA_DTYPE_F16)
    return fail(PKA_ERR_UNSUPPORTED, "q and the pool must be bf16 or f16 (dtype %d)", d.dtype);
  PKA_CHECK_ARG(d.out_dtype == PKA_DTYPE_BF16 || d.out_dtype == PKA_DTYPE_F16 ||
                    d.out_dtype == PKA_DTYPE_F32,
                "out_dtype must be bf16, f16 or f32 (got %d)", d.out_dtype);
  PKA_CHECK_ARG(d.mask == PKA_MASK_DENSE || d.mask == PKA_MASK_CAUSAL, "unknown mask %d", d.mask);
  PKA_CHECK_ARG(std::isfinite(d.scale) && std::isfinite(d.output_scale),
                "scale and output_scale must be finite");
  PKA_CHECK_ARG(d.max_pages_per_seq >= 1, "max_pages_per_seq must be >= 1");
  PKA_CHECK_ARG(d.num_pages >= 1 && d.num_pages < (int64_t)INT32_MAX,
                "num_pages must be in [1, 2^31-2]");
  PKA_CHECK_ARG(d.num_sms >= 0 && d.num_sms <= kMaxSms, "num_sms must be in [0, %d]", kMaxSms);
  if (d.num_sms == 0) {
    int dev = 0, sms = 0;
    PKA_CUDA_TRY(cudaGetDevice(&dev), "cudaGetDevice");
    PKA_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev),
                 "cudaDeviceGetAttribute(SM count)");
    d.num_sms = std::min(sms, kMaxSms);
  }
  const int32_t B = d.batch_size, H = d.num_heads;
  if (indptr == nullptr) {
    PKA_CHECK_ARG(d.q_len >= 1, "q_len must be >= 1 in fixed-query mode (got %d)", d.q_len);
    PKA_CHECK_ARG((int64_t)B * d.q_len <= INT32_MAX, "batch_size * q_len exceeds 2^31 - 1");
  } else {
    PKA_CHECK_ARG(indptr[0] == 0, "qo_indptr[0] must be 0 (got %d)", indptr[0]);
  }

  // ---- requests ----
  p.desc = d;
  p.reqs.assign(B, LatentReq{});
  std::vector<int64_t> tiles(B);
  int64_t max_rows = 0, cost = 0;
  for (int32_t b = 0; b < B; ++b) {
    const int64_t n = seq[b];
    PKA_CHECK_ARG(n >= 0 && n <= (int64_t)d.max_pages_per_seq * d.page_size,
                  "request %d: kv_len %lld outside [0, %d pages x %d]", b, (long long)n,
                  d.max_pages_per_seq, d.page_size);
    PKA_CHECK_ARG(n <= INT32_MAX - 4 * kLatentTile,   // positions a tile or two past it
                  "request %d: kv_len %lld is too long", b, (long long)n);
    const int64_t l = indptr == nullptr ? d.q_len : (int64_t)indptr[b + 1] - indptr[b];
    PKA_CHECK_ARG(l >= 0, "qo_indptr must be non-decreasing (request %d)", b);
    LatentReq& r = p.reqs[b];
    r.q_start = indptr == nullptr ? b * d.q_len : indptr[b];
    r.q_len = (int32_t)l;
    r.kv_len = (int32_t)n;
    r.part_base = -1;
    // a request without keys still writes its zero rows: one empty tile
    tiles[b] = l == 0 ? 0 : std::max<int64_t>(1, ceil_div(n, kLatentTile));
    if (l > 0) cost += tiles[b] + kItemCost;
    max_rows = std::max(max_rows, l * H);
  }
  if (max_rows > kMaxRows)
    return fail(PKA_ERR_UNSUPPORTED, "%lld query rows (token, head) of a request exceed %d",
                (long long)max_rows, kMaxRows);
  p.total_q = indptr == nullptr ? B * d.q_len : indptr[B];
  p.max_rows = (int32_t)max_rows;
  // The smallest block that holds a request's rows: fewer rows leave shared memory for
  // more key stages (152 requests of 4096 keys, 512 + 64 columns: 116 us with 16 or 32
  // rows, 124 with 64; a few short requests 7.8 us with 16 rows, 8.4 with 32).  More than
  // 64 rows go to pairs of CTAs with 64 each (76 requests, 128 heads: 48.7 us against
  // 57.9 for two blocks of 64 with 256 + 64 columns, 77 against 116 with 512 + 64); up to
  // 64 leave half of a pair idle (152 requests, 48 heads: 87 us against 68, 143 against 125).
  p.row_tile = max_rows <= 16 ? 16 : max_rows <= 32 ? 32 : max_rows <= 64 ? 64 : 128;
  p.row_blocks = (int32_t)std::max<int64_t>(1, ceil_div(max_rows, p.row_tile));

  // ---- segments: the smallest equal cost that fits the CTAs at hand ----
  const int64_t max_segments = std::max(1, d.num_sms / (p.row_blocks * (p.row_tile == 128 ? 2 : 1)));
  int64_t target = std::max(ceil_div(cost, max_segments), kMinPiece + kItemCost);
  while (true) {
    p.items.clear();
    p.segments.assign(1, 0);
    int64_t load = 0;
    bool fits = true;
    auto close = [&] {
      if ((int32_t)p.items.size() > p.segments.back()) p.segments.push_back((int32_t)p.items.size());
      load = 0;
      fits = (int64_t)p.segments.size() - 1 <= max_segments;
    };
    for (int32_t b = 0; b < B && fits; ++b) {
      int64_t lo = 0;
      while (lo < tiles[b] && fits) {
        const int64_t left = tiles[b] - lo, room = target - load - kItemCost;
        if (load > 0 && room < std::min(left, kMinPiece)) {
          close();
          continue;
        }
        int64_t take = std::min(left, std::max(room, kMinPiece));
        if (left - take < kMinPiece && left - take <= target / 8) take = left;   // no sliver
        p.items.push_back(LatentItem{b, (int32_t)lo, (int32_t)(lo + take), -1});
        lo += take;
        load += take + kItemCost;
        if (load >= target) close();
      }
    }
    if (fits) close();
    if (fits) break;
    target += std::max<int64_t>(1, target / 64);
  }

  // ---- cut requests: partial rows, workspace ----
  std::vector<int32_t> count(B, 0);
  for (const LatentItem& it : p.items) ++count[it.request];
  for (LatentItem& it : p.items)
    if (count[it.request] > 1) it.part = p.reqs[it.request].n_parts++;
  p.splits.clear();
  int64_t prow = 0;
  for (int32_t b = 0; b < B; ++b) {
    LatentReq& r = p.reqs[b];
    if (r.n_parts > 1) {
      r.part_base = (int32_t)prow;
      prow += (int64_t)r.n_parts * r.q_len * H;
      PKA_CHECK_ARG(prow <= (int64_t)INT32_MAX, "too many partial rows");
      p.splits.push_back(r);
    }
  }
  p.num_many = (int32_t)(std::stable_partition(p.splits.begin(), p.splits.end(),
                                               [](const LatentReq& r) {
                                                 return r.n_parts > kLatentFewPieces;
                                               }) -
                         p.splits.begin());
  PKA_CHECK_ARG((int64_t)p.splits.size() * max_rows * (d.latent_dim / 16) <= INT32_MAX,
                "too many rows of cut requests");
  p.partial_rows = (int32_t)prow;
  p.ws_lse_offset = ceil_div(prow * d.latent_dim * 4, 256) * 256;
  p.workspace_bytes = prow ? p.ws_lse_offset + prow * 4 : 0;
  return PKA_OK;
}

// Tiles in their order (by head, so that the tiles of a head run together), each to
// the pair of CTAs that is free first.  Where that ends unevenly every pair gets the
// same share instead, and the tile that fills one is cut there: what is left of it
// goes to the next.
int deal_prefill_tiles(pka_prefill_plan& p) {
  PKA_CHECK_ARG(p.desc.num_sms >= 0 && p.desc.num_sms <= kMaxSms, "num_sms must be in [0, %d]", kMaxSms);
  int sms = p.desc.num_sms;
  if (sms == 0 && (p.desc.flags & PKA_PLAN_HOST_ONLY)) sms = 152;
  if (sms == 0) {
    int dev = 0;
    PKA_CUDA_TRY(cudaGetDevice(&dev), "cudaGetDevice");
    PKA_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev),
                 "cudaDeviceGetAttribute(SM count)");
    sms = std::min(sms, kMaxSms);
  }
  if (p.tiles.empty()) {
    p.segments.assign(1, 0);
    return PKA_OK;
  }
  struct Piece {
    int32_t tile, kv0, n;
  };
  using Slot = std::pair<int64_t, int32_t>;   // load, index: the least loaded first, then the first
  std::vector<std::vector<Piece>> slots((size_t)sms);   // pairs of CTAs: two CTAs share an SM
  const int32_t n_tiles = (int32_t)p.tiles.size();
  int64_t cost = 0;
  for (const PrefillTile& t : p.tiles) cost += t.n_kv + kPrefillItemCost;
  // what every slot may take, INT64_MAX: nothing is cut; the longest load, or -1 if it does not fit
  auto deal = [&](int64_t target) -> int64_t {
    for (auto& s : slots) s.clear();
    std::priority_queue<Slot, std::vector<Slot>, std::greater<Slot>> free;
    for (int32_t i = 0; i < sms; ++i) free.push({0, i});
    int64_t longest = 0;
    for (int32_t i = 0; i < n_tiles; ++i) {
      int64_t lo = 0;
      const int64_t n = p.tiles[i].n_kv;
      while (lo < n) {
        if (free.empty()) return -1;
        const Slot s = free.top();
        free.pop();
        const int64_t left = n - lo, room = target == INT64_MAX ? left : target - s.first - kPrefillItemCost;
        if (room < std::min(left, kPrefillMinPiece)) continue;   // full
        const int64_t take = left - room < kPrefillMinPiece ? left : room;
        slots[(size_t)s.second].push_back(Piece{i, (int32_t)lo, (int32_t)take});
        lo += take;
        const int64_t load = s.first + take + kPrefillItemCost;
        longest = std::max(longest, load);
        if (load < target) free.push({load, s.second});
      }
    }
    return longest;
  };
  const int64_t whole = deal(INT64_MAX);
  int64_t target = std::max(ceil_div(cost, sms), kPrefillMinPiece + kPrefillItemCost);
  if (whole > target + kPrefillCutCost) {
    int64_t even;
    while ((even = deal(target)) < 0) target += std::max<int64_t>(1, target / 64);
    if (even + kPrefillCutCost >= whole) deal(INT64_MAX);   // not worth a merge
  }
  std::vector<int32_t> pieces((size_t)n_tiles, 0), first((size_t)n_tiles, -1), next((size_t)n_tiles, 0);
  for (const auto& s : slots)
    for (const Piece& c : s) ++pieces[(size_t)c.tile];
  for (int32_t i = 0; i < n_tiles; ++i)
    if (pieces[(size_t)i] > 1) {
      const PrefillTile& t = p.tiles[(size_t)i];
      first[(size_t)i] = p.num_parts;
      for (int32_t word : {t.head, t.q_tile, t.q0, t.lq, p.num_parts, pieces[(size_t)i], 0, 0}) p.cuts.push_back(word);
      p.num_parts += pieces[(size_t)i];
    }
  // every pair's first piece, then the others of the first pair, of the second, ...
  std::vector<PrefillTile> dealt;
  auto lay = [&](const Piece& c) {
    dealt.push_back(p.tiles[(size_t)c.tile]);
    dealt.back().kv0 += c.kv0;
    dealt.back().n_kv = c.n;
    p.part.push_back(first[(size_t)c.tile] < 0 ? -1 : first[(size_t)c.tile] + next[(size_t)c.tile]++);
  };
  for (const auto& s : slots)
    if (!s.empty()) lay(s[0]);
  p.segments.assign(1, (int32_t)dealt.size());
  for (const auto& s : slots) {
    if (s.empty()) continue;
    for (size_t i = 1; i < s.size(); ++i) lay(s[i]);
    p.segments.push_back((int32_t)dealt.size());
  }
  p.tiles = std::move(dealt);
  return PKA_OK;
}

}  // namespace pka
