// Decode plans, ordinary ones and those behind shared prefixes, whose CUDA calls fail, on the host: the
// entry points of abi.cpp and prefix_abi.cpp with their planners over a fake runtime that refuses
// the calls it is told to.  A plan made in vain leaks nothing.  An update, to a batch that shares or
// one that does not, succeeds or leaves the plan as it was: either way what a run launches with is
// one batch's, whole, and no error is left for the next launch to find.  So too where host memory
// runs out, which no entry point lets out as an exception.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <new>
#include <string>
#include <vector>

#include "host_common.h"
#include "kernels.h"
#include "prefill.h"
#include "prefix.h"
#include "tmap.h"

namespace {

std::map<const void*, size_t> g_device, g_pinned;   // live allocations
size_t g_kept = 0;        // of them those whose release was refused
int g_events = 0;
std::string g_refuse;     // the call that fails
int g_refused = 0;
int64_t g_news = -1;      // host allocations until all fail, -1: none does
bool g_last = false;      // a refusal that cudaGetLastError would still tell of
// what the last run launched
const pka_plan* g_plan = nullptr;
pka::DecodeArgs g_decode;
pka::PrefixArgs g_prefix;
pka::OwnArgs g_own;
pka::PrefixMergeArgs g_merge;
int g_plain = 0, g_merges = 0;

#define REQUIRE(cond)                                                                    \
  do {                                                                                   \
    if (!(cond)) {                                                                       \
      std::printf("line %d: %s, %s refused (%s)\n", __LINE__, #cond, g_refuse.c_str(),   \
                  pka_last_error());                                                     \
      std::exit(1);                                                                      \
    }                                                                                    \
  } while (0)

// "capture": what a thread may not call while a stream of it captures.
bool refused(const char* name) {
  const bool unsafe = std::strcmp(name, "cudaMalloc") == 0 || std::strcmp(name, "cudaMallocHost") == 0 ||
                      std::strcmp(name, "cudaFree") == 0 || std::strcmp(name, "cudaEventSynchronize") == 0;
  if (g_refuse != name && !(g_refuse == "capture" && unsafe)) return false;
  ++g_refused;
  return g_last = true;
}

bool inside(const void* p, size_t n) {
  for (const auto& [base, size] : g_device) {
    const char *b = static_cast<const char*>(base), *q = static_cast<const char*>(p);
    if (q >= b && q + n <= b + size) return true;
  }
  return false;
}

cudaError_t allocate(std::map<const void*, size_t>& all, void** p, size_t n) {
  *p = std::aligned_alloc(256, (n + 255) / 256 * 256);
  std::memset(*p, 0xee, n);
  const int64_t news = g_news;   // not the runtime's own
  g_news = -1;
  all[*p] = n;
  g_news = news;
  return cudaSuccess;
}

void release(std::map<const void*, size_t>& all, void* p) {
  if (p == nullptr) return;
  REQUIRE(all.erase(p) == 1);
  std::free(p);
}

}  // namespace

void* operator new(size_t n) {
  if (g_news == 0) throw std::bad_alloc();
  if (g_news > 0) --g_news;
  void* p = std::malloc(n > 0 ? n : 1);
  if (p == nullptr) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }

extern "C" {
cudaError_t cudaMalloc(void** p, size_t n) {
  return refused("cudaMalloc") ? cudaErrorMemoryAllocation : allocate(g_device, p, n);
}
cudaError_t cudaMallocHost(void** p, size_t n) {
  return refused("cudaMallocHost") ? cudaErrorMemoryAllocation : allocate(g_pinned, p, n);
}
cudaError_t cudaFree(void* p) {
  if (p != nullptr && refused("cudaFree")) {
    ++g_kept;
    return cudaErrorStreamCaptureUnsupported;
  }
  release(g_device, p);
  return cudaSuccess;
}
cudaError_t cudaFreeHost(void* p) {
  release(g_pinned, p);
  return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void* dst, const void* src, size_t n, cudaMemcpyKind, cudaStream_t) {
  if (refused("cudaMemcpyAsync")) return cudaErrorInvalidValue;
  REQUIRE(inside(dst, n));
  std::memcpy(dst, src, n);
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t) {
  if (refused("cudaMemsetAsync")) return cudaErrorInvalidValue;
  REQUIRE(inside(p, n));
  std::memset(p, v, n);
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) {
  if (refused("cudaGetDevice")) return cudaErrorInvalidDevice;
  *d = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;
  return cudaSuccess;
}
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) {
  if (refused("cudaEventCreate")) return cudaErrorMemoryAllocation;
  *e = reinterpret_cast<cudaEvent_t>(std::malloc(1));
  ++g_events;
  return cudaSuccess;
}
cudaError_t cudaEventRecord(cudaEvent_t e, cudaStream_t) {
  REQUIRE(e != nullptr);
  return refused("cudaEventRecord") ? cudaErrorInvalidValue : cudaSuccess;
}
cudaError_t cudaEventSynchronize(cudaEvent_t e) {
  REQUIRE(e != nullptr);
  return refused("cudaEventSynchronize") ? cudaErrorInvalidValue : cudaSuccess;
}
cudaError_t cudaEventDestroy(cudaEvent_t e) {
  std::free(e);
  --g_events;
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError() {
  g_last = false;
  return cudaSuccess;
}
const char* cudaGetErrorString(cudaError_t) { return "refused"; }
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes*, const void*) { return cudaErrorInvalidValue; }
}

namespace pka {
int encode_bf16_map(CUtensorMap*, const void*, int, const uint64_t*, const uint64_t*, const uint32_t*) { return PKA_OK; }
int encode_kv_pool_map(CUtensorMap*, const void*, int64_t, int32_t, int32_t, int32_t, int64_t, int64_t) {
  return PKA_OK;
}
int encode_kv_box_map(CUtensorMap*, const void*, int64_t, int32_t, int32_t, int64_t, int64_t, int32_t, int32_t) {
  return PKA_OK;
}
int launch_decode(const pka_plan& plan, const DecodeArgs& a, const CUtensorMap&, const CUtensorMap&, cudaStream_t) {
  g_plan = &plan;
  g_decode = a;
  ++g_plain;
  return PKA_OK;
}
int launch_check_tables(const WorkItem*, int32_t, const ReqInfo*, const int32_t*, int64_t, const int32_t*, int32_t,
                        int64_t, int32_t*, cudaStream_t) {
  return PKA_OK;
}
int launch_prefix(const PrefixArgs& a, bool, bool, const CUtensorMap&, const CUtensorMap&, cudaStream_t) {
  g_prefix = a;
  return PKA_OK;
}
int launch_prefix_own(const OwnArgs& a, const CUtensorMap&, const CUtensorMap&, cudaStream_t) {
  g_own = a;
  return PKA_OK;
}
int launch_prefix_merge(const PrefixMergeArgs& a, cudaStream_t) {
  g_merge = a;
  ++g_merges;
  return PKA_OK;
}
// not reached by what is called here
int launch_prefix_check(const RowPages*, int32_t, const int32_t*, int64_t, const int32_t*, int32_t, int32_t, int32_t*,
                        cudaStream_t) {
  std::abort();
}
int launch_prefill_1h(const pka_prefill_plan&, const PrefillArgs&, const CUtensorMap&, const CUtensorMap&,
                      const CUtensorMap&, cudaStream_t) {
  std::abort();
}
int launch_wait_probe(uint64_t, int32_t*, cudaStream_t) { std::abort(); }
int launch_merge_states(const float*, const float*, int32_t, int32_t, int32_t, int32_t, void*, int32_t, float*,
                        cudaStream_t) {
  std::abort();
}
int launch_paged_gather(const CUtensorMap&, const int32_t*, int64_t, int32_t, int32_t, int32_t, int32_t, int32_t, void*,
                        cudaStream_t) {
  std::abort();
}
int noalloc_status_word(cudaStream_t, int32_t**) { std::abort(); }
int deal_prefill_tiles(pka_prefill_plan&) { std::abort(); }
}  // namespace pka

namespace {

constexpr int kHeads = 8, kKvHeads = 2;

struct Batch {
  std::vector<int32_t> lens, groups, pages;
  bool shared;
};

alignas(256) char g_any[64];   // an address for the run's tensors
std::vector<char> g_space(1 << 28);
char* g_ws = g_space.data() + (256 - reinterpret_cast<uintptr_t>(g_space.data()) % 256) % 256;
const size_t kWsBytes = g_space.size() - 256;

// A plain run of batch `b`: its items and requests lie on the device, its counters at 0.
void launched_plain(const Batch& b) {
  const pka_plan& p = *g_plan;
  const pka::DecodeArgs& a = g_decode;
  REQUIRE(p.B == (int)b.lens.size() && p.total_q == p.B && a.num_items == (int)p.items.size() && a.num_items > 0);
  REQUIRE(inside(a.items, p.items.size() * sizeof(pka::WorkItem)));
  REQUIRE(inside(a.reqs, b.lens.size() * sizeof(pka::ReqInfo)) && inside(a.status, 4));
  REQUIRE(std::memcmp(a.items, p.items.data(), p.items.size() * sizeof(pka::WorkItem)) == 0);
  REQUIRE(std::memcmp(a.reqs, p.reqs.data(), p.reqs.size() * sizeof(pka::ReqInfo)) == 0);
  for (size_t i = 0; i < b.lens.size(); ++i) REQUIRE(a.reqs[i].kv_len == b.lens[i]);
  REQUIRE(*a.status == 0 && inside(a.merge_cnt, 4 * (size_t)p.num_merge_counters));
  for (int i = 0; i < p.num_merge_counters; ++i) REQUIRE(a.merge_cnt[i] == 0);
}

void runs_as(const pka_plan* p, const Batch& b) {
  REQUIRE(!g_last);
  const int plain = g_plain;
  REQUIRE(paged_decode_run(p, g_any, 1024, 128, g_any, g_any, 4096, 2048, reinterpret_cast<int32_t*>(g_any), 1 << 16,
                           nullptr, nullptr, g_any, nullptr, g_ws, kWsBytes, nullptr) == PKA_OK);
  REQUIRE(g_plain == plain + 1);
  launched_plain(b);
  pka_plan_info info;
  REQUIRE(paged_decode_plan_info(p, &info) == PKA_OK && info.total_q == (int)b.lens.size());
}

void runs_as(const pka_prefix_plan* p, const Batch& b) {
  REQUIRE(!g_last);
  const int plain = g_plain, merges = g_merges;
  pka_prefix_plan_info info;
  REQUIRE(paged_prefix_decode_plan_info(p, &info) == PKA_OK);
  REQUIRE(info.shared == (int)b.shared && info.total_q == (int)b.lens.size());
  REQUIRE(paged_prefix_decode_run(p, g_any, 1024, 128, g_any, g_any, 4096, 2048, reinterpret_cast<int32_t*>(g_any),
                                  1 << 16, nullptr, nullptr, g_any, nullptr, g_ws, kWsBytes, nullptr) == PKA_OK);
  if (!b.shared) {
    REQUIRE(g_plain == plain + 1 && g_merges == merges && info.num_prefix_pieces == 0 && info.num_own_pieces == 0);
    launched_plain(b);
    REQUIRE(info.workspace_bytes == g_plan->workspace_bytes && info.partial_rows == g_plan->partial_rows);
    return;
  }
  REQUIRE(g_merges == merges + 1 && g_plain == plain && g_merge.total_q == (int)b.lens.size());
  REQUIRE(inside(g_prefix.items, info.num_prefix_pieces * sizeof(pka::PrefixItem)));
  REQUIRE(inside(g_prefix.more, (g_prefix.num_pairs + 1) * sizeof(int32_t)));
  REQUIRE(inside(g_own.pieces, g_own.num_pieces * sizeof(pka::OwnPiece)) && g_own.num_pieces == info.num_own_pieces);
  REQUIRE(inside(g_merge.tokens, b.lens.size() * sizeof(pka::TokenStates)));
  REQUIRE(inside(g_prefix.status, 8) && *g_own.next == 0);
  int64_t tiles = 0, want = 0, units = 0, want_units = 0;
  for (int i = 0; i < info.num_prefix_pieces; ++i) tiles += g_prefix.items[i].tile_hi - g_prefix.items[i].tile_lo;
  for (int i = 0; i < g_own.num_pieces; ++i) {
    units += g_own.pieces[i].unit_hi - g_own.pieces[i].unit_lo;
    REQUIRE(g_own.pieces[i].kv_len == b.lens[g_own.pieces[i].request]);
  }
  for (size_t g = 0; g < b.pages.size(); ++g) {
    const int n = b.groups[g + 1] - b.groups[g];
    const bool shares = n > 1 && b.pages[g] > 0;
    if (shares) want += kKvHeads * ((b.pages[g] + 3) / 4) * ((n * (kHeads / kKvHeads) + 255) / 256);
    for (int r = b.groups[g]; r < b.groups[g + 1]; ++r)
      want_units += kKvHeads * ((b.lens[r] + 15) / 16 - (shares ? b.pages[g] : 0));
  }
  REQUIRE(tiles == want && units == want_units);
}

void nothing_left() { REQUIRE(g_device.size() == g_kept && g_pinned.empty() && g_events == 0); }

void forget_kept() {
  nothing_left();
  for (const auto& [q, n] : g_device) std::free(const_cast<void*>(q));
  g_device.clear();
  g_kept = 0;
}

pka_decode_desc g_desc;

int make(const Batch& b, pka_plan** p) {
  size_t bytes;
  g_desc.batch_size = (int32_t)b.lens.size();
  return paged_decode_plan(p, &g_desc, b.lens.data(), nullptr, &bytes, nullptr);
}
int make(const Batch& b, pka_prefix_plan** p) {
  size_t bytes;
  g_desc.batch_size = (int32_t)b.lens.size();
  return paged_prefix_decode_plan(p, &g_desc, b.lens.data(), nullptr, b.groups.data(), (int32_t)b.pages.size(),
                                  b.pages.data(), 0, &bytes, nullptr);
}
int update(pka_plan* p, const Batch& b) {
  size_t bytes;
  return paged_decode_plan_update(p, (int32_t)b.lens.size(), b.lens.data(), nullptr, &bytes, nullptr);
}
int update(pka_prefix_plan* p, const Batch& b) {
  size_t bytes;
  return paged_prefix_decode_plan_update(p, (int32_t)b.lens.size(), b.lens.data(), nullptr, b.groups.data(),
                                         (int32_t)b.pages.size(), b.pages.data(), &bytes, nullptr);
}
void destroy(pka_plan* p) { paged_decode_plan_destroy(p); }
void destroy(pka_prefix_plan* p) { paged_prefix_decode_plan_destroy(p); }

const char* const kCalls[] = {"cudaMalloc",      "cudaMallocHost",  "cudaMemcpyAsync",      "cudaMemsetAsync", "cudaGetDevice",
                              "cudaEventCreate", "cudaEventRecord", "cudaEventSynchronize", "cudaFree",        "capture"};

// Plans of Plan's kind made, and updated from each batch to each, while each call is refused.
template <typename Plan>
void refuse_all(const std::vector<Batch>& batches) {
  for (const Batch& b : batches)
    for (const char* call : kCalls) {
      Plan* p = nullptr;
      g_refuse = call;
      g_refused = 0;
      const int rc = make(b, &p);
      g_refuse.clear();
      REQUIRE(!g_last);   // told of by the code
      REQUIRE(rc == PKA_OK || (rc == PKA_ERR_CUDA && p == nullptr && g_refused > 0));
      if (rc == PKA_OK) {
        runs_as(p, b);
        destroy(p);
      }
      nothing_left();
      // a plan destroyed then: its memory may stay, an error that the next launch would find may not
      REQUIRE(make(b, &p) == PKA_OK);
      g_refuse = call;
      destroy(p);
      g_refuse.clear();
      REQUIRE(!g_last && g_pinned.empty() && g_events == 0);
      forget_kept();
    }

  // from a new plan, and from one that has been every other batch and so has the largest buffers
  for (const Batch& from : batches)
    for (const Batch& to : batches)
      for (const bool been : {false, true})
        for (const char* call : kCalls) {
          Plan* p = nullptr;
          REQUIRE(make(from, &p) == PKA_OK);
          if (been)
            for (const Batch& b : {batches[0], batches.back(), batches[1], batches[0], from}) REQUIRE(update(p, b) == PKA_OK);
          runs_as(p, from);
          const Batch* now = &from;
          for (int again = 0; again < 2; ++again) {
            g_refuse = call;
            g_refused = 0;
            const int rc = update(p, to);
            g_refuse.clear();
            REQUIRE(rc == PKA_OK || (rc == PKA_ERR_CUDA && g_refused > 0));
            if (rc == PKA_OK) now = &to;
            runs_as(p, *now);
          }
          for (const Batch& next : batches) {
            REQUIRE(update(p, next) == PKA_OK);
            runs_as(p, next);
          }
          destroy(p);
          nothing_left();
          forget_kept();
        }
}

// Host memory that runs out at every allocation of a plan in turn.
template <typename Plan>
void run_out_all(const Batch& from, const Batch& to) {
  for (int64_t at = 0, done = 0; !done; ++at) {
    Plan* p = nullptr;
    g_news = at;
    const int rc = make(from, &p);
    done = g_news > 0;
    g_news = -1;
    REQUIRE(rc == PKA_OK ? p != nullptr : rc == PKA_ERR_INVALID_ARG && p == nullptr && !done);
    if (rc == PKA_OK) {
      runs_as(p, from);
      destroy(p);
    }
    nothing_left();
  }
  Plan* p = nullptr;
  REQUIRE(make(from, &p) == PKA_OK);
  for (int64_t at = 0, done = 0; !done; ++at) {
    g_news = at;
    const int rc = update(p, to);
    done = g_news > 0;
    g_news = -1;
    REQUIRE(rc == PKA_OK || (rc == PKA_ERR_INVALID_ARG && !done));
    runs_as(p, rc == PKA_OK ? to : from);
    if (rc == PKA_OK) REQUIRE(update(p, from) == PKA_OK);
  }
  destroy(p);
  nothing_left();
}

// The same of the prefill's plans.
template <typename Make>
void run_out_prefill(Make make_plan) {
  for (int64_t at = 0, done = 0; !done; ++at) {
    pka_prefill_plan* p = nullptr;
    g_news = at;
    const int rc = make_plan(&p);
    done = g_news > 0;
    g_news = -1;
    REQUIRE(rc == PKA_OK ? p != nullptr : rc == PKA_ERR_INVALID_ARG && p == nullptr && !done);
    batch_prefill_plan_destroy(p);
    nothing_left();
  }
}

}  // namespace

int main() {
  g_desc = pka_decode_desc{};
  g_desc.num_qo_heads = kHeads;
  g_desc.num_kv_heads = kKvHeads;
  g_desc.head_dim = 128;
  g_desc.page_size = 16;
  g_desc.max_pages_per_seq = 64;
  g_desc.num_pages = 6000;
  g_desc.q_len = 1;
  g_desc.window_left = -1;
  g_desc.scale = 0.1f;
  g_desc.bmm2_scale = 1.f;
  g_desc.freeze_seq_lens = 1;
  const Batch few{{300, 400}, {0, 2}, {10}, true}, other{{500, 90, 700}, {0, 1, 3}, {9, 4}, true},
      none{{300, 400, 20}, {0, 3}, {0}, false}, alone{{1000, 900}, {0, 1, 2}, {30, 20}, false};
  Batch many{std::vector<int32_t>(2000, 500), {0, 2000}, {20}, true},
      none_many{std::vector<int32_t>(2100, 300), {0, 2100}, {0}, false};
  for (size_t i = 0; i < none_many.lens.size(); ++i) none_many.lens[i] += (int32_t)(i % 600);
  refuse_all<pka_plan>({few, none, alone, many, none_many});
  refuse_all<pka_prefix_plan>({few, none, other, alone, many, none_many});
  for (const Batch& from : {few, alone, many})
    for (const Batch& to : {few, none, other}) {
      run_out_all<pka_plan>(from, to);
      run_out_all<pka_prefix_plan>(from, to);
    }
  pka_prefill_desc f{};
  f.batch_size = 3;
  f.num_qo_heads = kHeads;
  f.num_kv_heads = kKvHeads;
  f.head_dim = 128;
  f.sm_scale = 0.1f;
  f.output_scale = 1.f;
  f.window_left = -1;
  f.mask = PKA_MASK_CAUSAL;
  const int32_t rows[] = {0, 200, 200, 1000};
  size_t bytes = 0;
  int32_t tiles = 0;
  run_out_prefill([&](pka_prefill_plan** p) { return batch_prefill_plan(p, &f, rows, rows, &bytes, &tiles, nullptr); });
  run_out_prefill([&](pka_prefill_plan** p) {
    return batch_prefill_plan_fixed(p, &f, 100, 150, nullptr, nullptr, &bytes, &tiles, nullptr);
  });
  std::puts("ok");
  return 0;
}
