// Host planner of decode behind shared prefixes.
//
// A group of requests that begin with the same pages attends to them once: the query
// rows of all its requests, times the heads of a KV head's group, are the rows of one
// product with the prefix's keys.  The products (group, KV head, row tile) are laid end to
// end and dealt out evenly, in tiles of 64 keys, to one wave of pairs of CTAs; what the
// requests have behind the prefix (request, KV head, 16 rows) is cut into pieces of up to 16
// units of 16 keys, which the warps of one wave of CTAs take as they come.  Every piece
// writes a partial state of its rows, and a merge takes all of a row's.
#include <algorithm>
#include <cmath>
#include <vector>

#include "host_common.h"
#include "prefix.h"

namespace pka {

namespace {

// Sharing saves what reading a prefix for every request costs, at 14 TB/s for the most part from
// L2, and costs its tiles (a pair takes 16 heads or rows of a head for the time of 256) and two
// launches with the join of the states: 5 us.  32 heads on 8, shared and not: 4 requests behind
// 16384 keys 32.7 and 28.3 us, behind 65536 63.5 and 76.0; 16 behind 1024 16.4 and 14.4, behind
// 4096 19.8 and 28.7; 64 behind 256 23.8 and 29.1.
constexpr double kReadAgain = 14e12, kTileCost = 5.5e-9, kShareCost = 5e-6;
// Without DENSE a piece has no fewer tiles than this; with it so many fall on each pair, or the
// states cost what two CTAs an SM gain (32 heads on 8, with and without: 16 requests behind 4096
// keys, 3 tiles a pair, 27.4 and 20.1 us; 4 behind 16384, 13, 32.9 and 32.8; behind 32768, 27,
// 43.3 and 51.3; behind 65536, 54, 63.1 and 87.9; 16 heads on 1, 64 behind 65536, 27, 61.0 and
// 55.3).
constexpr int64_t kMinDenseTiles = 32;
constexpr int64_t kMinPrefixTiles = 3;   // a piece is no shorter, its row tile's keys allowing
constexpr int64_t kMinOwnUnits = 6, kMaxOwnUnits = 16;   // of 16 keys, in a piece of a request

// Cuts runs of work laid end to end into `parts` shares: even ones, or, with `skewed`, 17 to 15
// between the first half of the parts and the second.  Of two CTAs of the prefix kernel that
// share an SM the one that started first gets the tensor core more often (65536 keys, 1024 rows
// of 8 heads: even shares end after 180 and 213 us).
class Dealer {
 public:
  Dealer(int64_t total, int64_t parts, int64_t least, bool skewed)
      : total_(total), parts_(parts), least_(least), half_(skewed ? parts / 2 : 0) {}
  // The share that takes the next piece of a run of `left` units, and how many of them.
  int64_t take(int64_t left, int64_t* units) {
    auto room = [&] { return total_ * upto(part_ + 1) / upto(parts_) - done_; };
    while (room() < std::min(least_, left) && part_ + 1 < parts_) ++part_;
    int64_t n = part_ + 1 == parts_ ? left : std::min(left, std::max(room(), std::min(least_, left)));
    if (left - n < least_) n = left;
    done_ += n;
    *units = n;
    return part_;
  }

 private:
  int64_t upto(int64_t part) const { return part <= half_ ? 17 * part : 15 * part + 2 * half_; }
  int64_t total_, parts_, least_, half_, part_ = 0, done_ = 0;
};

}  // namespace

int build_prefix_plan(pka_prefix_plan& p, const pka_decode_desc& d_in, const int32_t* seq, const int32_t* indptr,
                      const int32_t* group_indptr, int32_t num_groups, const int32_t* prefix_pages,
                      int64_t min_shared_bytes) {
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
  const int rc = build_decode_plan(p.base, d_in, seq, indptr);
  if (rc != PKA_OK) return rc;
  const pka_decode_desc& d = p.base.desc;
  const int32_t G = p.base.G, Hkv = p.base.Hkv, ps = p.base.ps;
  const std::vector<ReqInfo>& reqs = p.base.reqs;
  double saved = 0, again = 0, all_tiles = 0;   // bytes, and tiles
  int64_t most_rows = 0;
  for (int32_t g = 0; g < num_groups; ++g) {
    const int32_t b0 = group_indptr[g], b1 = group_indptr[g + 1];
    const int64_t keys = (int64_t)prefix_pages[g] * ps;
    for (int32_t b = b0; b < b1; ++b) {
      const int64_t first_row = (int64_t)seq[b] - (d.mask == PKA_MASK_CAUSAL ? reqs[b].q_len - 1 : 0);
      PKA_CHECK_ARG(keys <= first_row, "request %d: its first row sees %lld keys, the shared prefix has %lld", b,
                    (long long)first_row, (long long)keys);
    }
    if (b1 - b0 >= 2 && keys > 0) {
      const int64_t rows = (int64_t)(reqs[b1 - 1].q_start + reqs[b1 - 1].q_len - reqs[b0].q_start) * G;
      int64_t passes = 0;   // of the decode without sharing over the prefix
      for (int32_t b = b0; b < b1; ++b) passes += ceil_div((int64_t)reqs[b].q_len * G, p.base.rows_per_cta);
      const double bytes = (double)keys * Hkv * 512;
      saved += (b1 - b0 - 1) * bytes;
      again += (double)(passes - 1) * bytes;
      all_tiles += (double)Hkv * ceil_div(keys, kPrefixTile) * ceil_div(rows, kPrefixRows);
      most_rows = std::max(most_rows, rows);
    }
  }
  p.min_shared_bytes = min_shared_bytes;
  p.shared = saved > 0 && (min_shared_bytes >= 0 ? saved >= (double)min_shared_bytes
                                                 : again / kReadAgain > all_tiles * kTileCost + kShareCost);
  if (!p.shared) {
    p.workspace_bytes = p.base.workspace_bytes;
    p.partial_rows = p.base.partial_rows;
    return PKA_OK;
  }
  PKA_CHECK_ARG(most_rows <= INT32_MAX - kPrefixRows, "a group has too many query rows");
  p.tokens.assign((size_t)p.base.total_q, TokenStates{0, 0, 0, -1, 0, 0, 0, 0});
  std::vector<int32_t> own_page(B, 0);
  int64_t states = 0;

  // ---- the shared prefixes ----
  int64_t total = 0, bytes = 0;
  int32_t most_pre = 0, most_own = 0;
  std::vector<PrefixItem> in_turn;
  std::vector<int32_t> by_pair;
  for (int pass = 0; pass < 2; ++pass) {   // the work, then its pieces
    if (pass == 1) {
      // A tile of 256 rows and 64 keys (8.4 MFLOP) takes 8.8 ns of the GPU without DENSE, in which one
      // CTA an SM waits for itself; where many of them take longer than the bytes, at 6.7 TB/s, the
      // products bound the whole.
      for (int32_t b = 0; b < B; ++b) bytes += (seq[b] - (int64_t)own_page[b] * ps) * Hkv * 512;
      p.dense = total >= kMinDenseTiles * d.num_sms && (double)total * 8.8e-9 > (double)bytes / 6.7e12;
    }
    // where memory bounds the whole, a sixth of the SMs is left to the requests' own keys from the
    // start (76 pairs of 152 SMs: 64 requests behind 8192 keys 48.0 us, 64 pairs 45.5; with two softmax
    // groups 75 pairs 38.4 us, 64 34.8 where their own keys are few)
    Dealer deal(total, std::max(1, p.dense ? d.num_sms : d.num_sms * 27 / 64), kMinPrefixTiles, p.dense);
    for (int32_t g = 0; g < num_groups; ++g) {
      const int32_t b0 = group_indptr[g], b1 = group_indptr[g + 1];
      if (b1 - b0 < 2 || prefix_pages[g] == 0) continue;
      const int32_t q0 = reqs[b0].q_start;
      const int64_t rows = (int64_t)(reqs[b1 - 1].q_start + reqs[b1 - 1].q_len - q0) * G;
      const int64_t keys = (int64_t)prefix_pages[g] * ps, tiles = ceil_div(keys, kPrefixTile);
      const int64_t row_tiles = ceil_div(rows, kPrefixRows);
      if (pass == 0) {
        total += Hkv * tiles * row_tiles;
        bytes += keys * Hkv * 512;
        for (int32_t b = b0; b < b1; ++b) own_page[b] = prefix_pages[g];
        continue;
      }
      for (int32_t b = b0; b < b1; ++b)
        for (int32_t i = 0; i < reqs[b].q_len; ++i) {
          TokenStates& t = p.tokens[reqs[b].q_start + i];
          t.pre_row = (reqs[b].q_start + i - q0) * G;
          t.pre_run = (int32_t)p.runs.size();
          t.pre_tiles = (int32_t)row_tiles;
        }
      for (int32_t hk = 0; hk < Hkv; ++hk)
        for (int64_t rt = 0; rt < row_tiles; ++rt) {
          const int64_t here = std::min<int64_t>(kPrefixRows, rows - rt * kPrefixRows);
          StateRun run{(int32_t)states, 0, (int32_t)here, 0};
          for (int64_t t = 0; t < tiles; ++run.count) {
            int64_t n = 0;
            const int64_t pair = deal.take(tiles - t, &n);
            PKA_CHECK_ARG(states + here <= INT32_MAX, "too many partial rows");
            by_pair.push_back((int32_t)pair);
            in_turn.push_back(PrefixItem{b0, hk, (int32_t)t, (int32_t)(t + n), (int32_t)keys, q0, (int32_t)rows,
                                         (int32_t)(rt * kPrefixRows), (int32_t)states, 0, 0, 0});
            states += here;
            t += n;
          }
          most_pre = std::max(most_pre, run.count);
          p.runs.push_back(run);
        }
    }
  }
  // each pair's first piece at the pair's own index, those behind it in turn (no pair is idle)
  std::vector<PrefixItem> further;
  for (size_t i = 0; i < in_turn.size(); ++i) {
    const bool first = i == 0 || by_pair[i] != by_pair[i - 1];
    if (first) p.more.push_back((int32_t)further.size());
    (first ? p.items : further).push_back(in_turn[i]);
  }
  p.more.push_back((int32_t)further.size());
  for (int32_t& m : p.more) m += (int32_t)p.items.size();
  p.items.insert(p.items.end(), further.begin(), further.end());

  // ---- the requests' own keys ----
  const int64_t upp = ps / 16;
  int64_t units = 0;
  for (int32_t b = 0; b < B; ++b)
    units += std::max<int64_t>(0, ceil_div(seq[b], 16) - own_page[b] * upp) * Hkv *
             ceil_div((int64_t)G * reqs[b].q_len, kOwnRows);
  const int64_t warps = (int64_t)d.num_sms * kOwnCtas * kOwnWarps;
  const int64_t most = std::min(std::max(units * 2 / (3 * warps), kMinOwnUnits), kMaxOwnUnits);
  for (int32_t b = 0; b < B; ++b) {
    const int64_t u0 = own_page[b] * upp, u1 = ceil_div(seq[b], 16), rows = (int64_t)G * reqs[b].q_len;
    const int64_t row_tiles = ceil_div(rows, kOwnRows), n = ceil_div(std::max<int64_t>(0, u1 - u0), most);
    PKA_CHECK_ARG((int64_t)p.runs.size() + Hkv * row_tiles <= INT32_MAX, "too many row tiles");
    if (row_tiles > 0x7fff || Hkv > 0xffff)
      return fail(PKA_ERR_UNSUPPORTED, "request %d has %lld query rows of %d KV heads", b, (long long)rows, Hkv);
    for (int32_t i = 0; i < reqs[b].q_len; ++i) {
      TokenStates& t = p.tokens[reqs[b].q_start + i];
      t.own_row = i * G;
      t.own_run = (int32_t)p.runs.size();
      t.own_tiles = (int32_t)row_tiles;
    }
    most_own = std::max(most_own, (int32_t)n);
    for (int32_t hk = 0; hk < Hkv; ++hk)
      for (int64_t rt = 0; rt < row_tiles; ++rt) {
        const int64_t here = std::min<int64_t>(kOwnRows, rows - rt * kOwnRows);
        p.runs.push_back(StateRun{(int32_t)states, (int32_t)n, (int32_t)here, 0});
        PKA_CHECK_ARG(states + n * here <= INT32_MAX, "too many partial rows");
        for (int64_t k = 0; k < n; ++k, states += here)
          p.pieces.push_back(OwnPiece{b, hk | (int32_t)rt << 16, (int32_t)(u0 + (u1 - u0) * k / n),
                                      (int32_t)(u0 + (u1 - u0) * (k + 1) / n), (int32_t)states, reqs[b].q_start,
                                      reqs[b].q_len, reqs[b].kv_len});
      }
  }
  for (int32_t g = 0; g < num_groups; ++g)
    for (int32_t b = group_indptr[g]; b < group_indptr[g + 1]; ++b)
      p.rows.push_back(RowPages{group_indptr[g], own_page[b], (int32_t)ceil_div(seq[b], ps), 0});
  // the longest first, equal ones in the order of the requests
  std::stable_sort(p.pieces.begin(), p.pieces.end(), [](const OwnPiece& x, const OwnPiece& y) {
    return x.unit_hi - x.unit_lo > y.unit_hi - y.unit_lo;
  });
  const int64_t n_pieces = (int64_t)p.pieces.size();
  p.own_ctas = (int32_t)std::max<int64_t>(1, std::min<int64_t>((int64_t)d.num_sms * kOwnCtas, ceil_div(n_pieces, kOwnWarps)));
  // CTAs that find no place beside the prefix kernel start late: they begin with what is left
  p.own_static = (int32_t)std::min<int64_t>(n_pieces, std::min<int64_t>(p.own_ctas, d.num_sms) * kOwnWarps);
  PKA_CHECK_ARG(p.items.size() < (size_t)INT32_MAX / 2 && p.pieces.size() < (size_t)INT32_MAX / 2, "too many pieces");
  p.partial_rows = (int32_t)states;
  p.most_states = most_pre + most_own;
  p.ws_lse_offset = (int64_t)up256((size_t)states * 512);
  p.workspace_bytes = p.ws_lse_offset + states * 4;
  return PKA_OK;
}

}  // namespace pka
