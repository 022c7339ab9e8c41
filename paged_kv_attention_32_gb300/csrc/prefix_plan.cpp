// Host planner of decode behind shared prefixes.
//
// A group of requests that begin with the same pages attends to them once: the query
// rows of all its requests, times the heads of a KV head's group, are the rows of one
// product with the prefix's keys, in tiles of 256 rows and 64 keys.  A prefix is cut along
// its keys into chunks alike for every group, KV head and row tile, c tiles each, where
// (waves of pairs of CTAs) * (c + what a piece costs besides its tiles) is least; each
// chunk is one partial state of the group's rows.  What the requests have behind the
// prefix is planned as decode work, whose states come behind those.
#include <algorithm>
#include <cmath>
#include <vector>

#include "host_common.h"
#include "prefix.h"

namespace pka {

namespace {

// What a piece costs besides its tiles (start, query rows, partial states), in tiles.
constexpr int64_t kPieceTiles = 8;

}  // namespace

int build_prefix_plan(pka_plan& p, const pka_decode_desc& d_in, const int32_t* seq, const int32_t* indptr,
                      const int32_t* group_indptr, int32_t num_groups, const int32_t* prefix_pages) {
  PKA_CHECK_ARG(num_groups >= 1 && group_indptr != nullptr && prefix_pages != nullptr,
                "num_groups must be >= 1, group_indptr and prefix_pages not NULL");
  const int32_t B = d_in.batch_size;
  PKA_CHECK_ARG(group_indptr[0] == 0, "group_indptr[0] must be 0 (got %d)", group_indptr[0]);
  for (int32_t g = 0; g < num_groups; ++g) {
    PKA_CHECK_ARG(group_indptr[g + 1] >= group_indptr[g], "group_indptr must not decrease (group %d)", g);
    PKA_CHECK_ARG(prefix_pages[g] >= 0, "prefix_pages[%d] is negative", g);
  }
  PKA_CHECK_ARG(group_indptr[num_groups] == B, "group_indptr must end at batch_size %d (got %d)", B,
                group_indptr[num_groups]);
  if (d_in.window_left != -1)
    return fail(PKA_ERR_UNSUPPORTED, "a window over a shared prefix is not built (window_left %d)", d_in.window_left);
  pka_decode_desc d = d_in;
  d.mma_min_rows = 1;   // the tensor-core decode, which may start before the prefix kernel ends

  // a plan without sharing first: it checks the arguments, and gives the query rows
  int rc = build_decode_plan(p, d, seq, indptr);
  if (rc != PKA_OK) return rc;
  const int32_t G = p.G, Hkv = p.Hkv, Hq = p.Hq, ps = p.ps;
  for (int32_t g = 0; g < num_groups; ++g)
    for (int32_t b = group_indptr[g]; b < group_indptr[g + 1]; ++b) {
      const int64_t first_row = (int64_t)seq[b] - (d.mask == PKA_MASK_CAUSAL ? p.reqs[b].q_len - 1 : 0);
      PKA_CHECK_ARG((int64_t)prefix_pages[g] * ps <= first_row,
                    "request %d: its first row sees %lld keys, the shared prefix has %lld", b, (long long)first_row,
                    (long long)prefix_pages[g] * ps);
    }

  // ---- which groups share, and in how many pieces ----
  struct Shared {
    int32_t group;
    int64_t tiles, row_tiles, rows;
  };
  std::vector<Shared> shared;
  int64_t most_tiles = 0;
  for (int32_t g = 0; g < num_groups; ++g) {
    const int32_t b0 = group_indptr[g], b1 = group_indptr[g + 1];
    if (b1 - b0 < 2 || prefix_pages[g] == 0) continue;   // nothing to read once instead of twice
    const ReqInfo& last = p.reqs[b1 - 1];
    const int64_t rows = (int64_t)(last.q_start + last.q_len - p.reqs[b0].q_start) * G;
    PKA_CHECK_ARG(rows <= INT32_MAX, "group %d has too many query rows", g);
    const int64_t tiles = ceil_div((int64_t)prefix_pages[g] * ps, kPrefixTile);
    shared.push_back(Shared{g, tiles, ceil_div(rows, kPrefixRows), rows});
    most_tiles = std::max(most_tiles, tiles);
  }
  if (shared.empty()) return PKA_OK;
  const int64_t pairs = p.desc.num_sms;   // two CTAs an SM, two CTAs a pair
  int64_t best = 0, chunk = 1;
  for (int64_t c = 1; c <= most_tiles; c = std::max(c + 1, c * 65 / 64)) {
    int64_t n = 0;
    for (const Shared& s : shared) n += Hkv * s.row_tiles * ceil_div(s.tiles, c);
    const int64_t cost = ceil_div(n, pairs) * (c + kPieceTiles);
    if (best == 0 || cost < best) {
      best = cost;
      chunk = c;
    }
  }
  std::vector<int32_t> pages(B, 0), chunks(B, 0);
  for (const Shared& s : shared)
    for (int32_t b = group_indptr[s.group]; b < group_indptr[s.group + 1]; ++b) {
      pages[b] = prefix_pages[s.group];
      chunks[b] = (int32_t)std::min<int64_t>(ceil_div(s.tiles, chunk), INT32_MAX);
    }

  // ---- the requests' own keys, and where every state goes ----
  const SharedPrefix behind{pages.data(), chunks.data()};
  rc = build_decode_plan(p, d, seq, indptr, &behind);
  if (rc != PKA_OK) return rc;
  p.prefix_tokens.assign((size_t)p.total_q, PrefixToken{0, 0});
  for (int32_t b = 0; b < B; ++b) {
    const ReqInfo& r = p.reqs[b];
    if (chunks[b] == 0) continue;
    for (int32_t i = 0; i < r.q_len; ++i) p.prefix_tokens[r.q_start + i] = PrefixToken{r.part_base + i * Hq, r.q_len * Hq};
  }
  for (const Shared& s : shared) {
    const int32_t b0 = group_indptr[s.group];
    const int64_t n = ceil_div(s.tiles, chunk);
    for (int64_t ci = 0; ci < n; ++ci)
      for (int32_t hk = 0; hk < Hkv; ++hk)
        for (int64_t rt = 0; rt < s.row_tiles; ++rt)
          p.prefix_items.push_back(PrefixItem{b0, hk, (int32_t)(s.tiles * ci / n), (int32_t)(s.tiles * (ci + 1) / n),
                                              prefix_pages[s.group] * ps, (int32_t)ci, p.reqs[b0].q_start,
                                              (int32_t)s.rows, (int32_t)(rt * kPrefixRows), 0, 0, 0});
  }
  PKA_CHECK_ARG(p.prefix_items.size() <= (size_t)INT32_MAX / 2, "too many pieces of prefixes");
  return PKA_OK;
}

}  // namespace pka
