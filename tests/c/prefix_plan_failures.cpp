// Plans of a decode behind shared prefixes whose CUDA calls fail, on the host: the entry points of
// prefix_abi.cpp and the planner over a fake runtime that refuses the calls it is told to.  A
// plan made in vain leaks nothing; an update that fails leaves the plan as it was, sharing or
// not, and it still runs and still updates to either.
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <utility>
#include <vector>

#include "host_common.h"
#include "kernels.h"
#include "prefix.h"
#include "tmap.h"

namespace {

std::map<const void*, size_t> g_device, g_pinned;   // live allocations
int g_events = 0;
std::string g_refuse;     // the call that fails
int g_refused = 0;
std::string g_error;
// what the last run launched
pka::PrefixArgs g_prefix;
pka::OwnArgs g_own;
pka::PrefixMergeArgs g_merge;
int g_merges = 0, g_plain = 0, g_checks = 0;

#define REQUIRE(cond)                                                          \
  do {                                                                         \
    if (!(cond)) {                                                             \
      std::printf("line %d: %s (%s)\n", __LINE__, #cond, g_error.c_str());     \
      std::exit(1);                                                            \
    }                                                                          \
  } while (0)

bool refused(const char* name) {
  if (g_refuse != name) return false;
  ++g_refused;
  return true;
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
  all[*p] = n;
  return cudaSuccess;
}

void release(std::map<const void*, size_t>& all, void* p) {
  if (p == nullptr) return;
  REQUIRE(all.erase(p) == 1);
  std::free(p);
}

}  // namespace

extern "C" {
cudaError_t cudaMalloc(void** p, size_t n) {
  return refused("cudaMalloc") ? cudaErrorMemoryAllocation : allocate(g_device, p, n);
}
cudaError_t cudaMallocHost(void** p, size_t n) {
  return refused("cudaMallocHost") ? cudaErrorMemoryAllocation : allocate(g_pinned, p, n);
}
cudaError_t cudaFree(void* p) {
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
  REQUIRE(inside(p, n));
  std::memset(p, v, n);
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) {
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
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "refused"; }
int paged_decode_plan_check(const pka_plan*, void*) { return PKA_OK; }
int paged_decode_check_tables(const pka_plan* p, const int32_t*, int64_t, const int32_t*, void*) {
  REQUIRE(p->dev_buf != nullptr);
  return PKA_OK;
}
}

namespace pka {
int fail(int code, const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(text, sizeof text, fmt, ap);
  va_end(ap);
  g_error = text;
  return code;
}
void clear_error() { g_error.clear(); }
int check_device(int d) { return d == 0 ? PKA_OK : PKA_ERR_INVALID_ARG; }
int read_status(int32_t*, cudaStream_t) { return PKA_OK; }
int encode_kv_box_map(CUtensorMap*, const void*, int64_t, int32_t, int32_t, int64_t, int64_t, int32_t, int32_t) {
  return PKA_OK;
}

// The decode's own plan: a device buffer, its upload.
int upload_decode_plan(pka_plan& p, cudaStream_t) {
  if (p.dev_buf == nullptr) PKA_CUDA_TRY(cudaMalloc(&p.dev_buf, 64), "cudaMalloc(plan)");
  PKA_CUDA_TRY(cudaMemcpyAsync(p.dev_buf, &p.total_q, 4, cudaMemcpyHostToDevice, nullptr), "cudaMemcpyAsync(plan)");
  return PKA_OK;
}
void keep_decode_buffers(pka_plan& plan, pka_plan& from) {
  plan.dev_buf = from.dev_buf;
  plan.device = from.device;
  from.dev_buf = nullptr;
}
int replace_decode_plan(pka_plan& p, pka_plan&& fresh, cudaStream_t stream) {
  keep_decode_buffers(fresh, p);
  p = std::move(fresh);
  return upload_decode_plan(p, stream);
}
void release_decode_plan(pka_plan& p) {
  if (p.dev_buf != nullptr) cudaFree(p.dev_buf);
}
int prepare_decode_run(const pka_plan*, const void*, int64_t, int64_t, const void*, const void*, int64_t, int64_t,
                       const int32_t*, int64_t, const int32_t*, const float*, void*, float*, DecodeArgs*, CUtensorMap*,
                       CUtensorMap*) {
  return PKA_OK;
}
int run_decode_plan(const pka_plan& p, const void*, int64_t, int64_t, const void*, const void*, int64_t, int64_t,
                    const int32_t*, int64_t, const int32_t*, const float*, void*, float*, void*, size_t, void*) {
  REQUIRE(p.dev_buf != nullptr && inside(p.dev_buf, 64));
  REQUIRE(*static_cast<int32_t*>(p.dev_buf) == p.total_q);
  ++g_plain;
  return PKA_OK;
}
int launch_prefix(const PrefixArgs& a, bool, bool, const CUtensorMap&, const CUtensorMap&, cudaStream_t) {
  if (refused("launch_prefix")) return PKA_ERR_CUDA;
  g_prefix = a;
  return PKA_OK;
}
int launch_prefix_own(const OwnArgs& a, const CUtensorMap&, const CUtensorMap&, cudaStream_t) {
  *a.next += 3;   // pieces taken, put back by the merge
  g_own = a;
  return PKA_OK;
}
int launch_prefix_merge(const PrefixMergeArgs& a, cudaStream_t) {
  if (refused("launch_merge")) return PKA_ERR_CUDA;
  *a.next = 0;
  g_merge = a;
  ++g_merges;
  return PKA_OK;
}
int launch_prefix_check(const RowPages* rows, int32_t batch, const int32_t*, int64_t, const int32_t*, int32_t, int32_t,
                        int32_t* status, cudaStream_t) {
  REQUIRE(inside(rows, batch * sizeof(RowPages)) && status == g_prefix.status);
  for (int32_t b = 0; b < batch; ++b) REQUIRE(rows[b].first <= b && rows[b].shared <= rows[b].pages);
  ++g_checks;
  return PKA_OK;
}
}  // namespace pka

namespace {

struct Batch {
  std::vector<int32_t> lens, groups, pages;
  bool shared;
};

alignas(256) char g_any[64];   // an address for the run's tensors
std::vector<char> g_ws(1 << 28);

int run(const pka_prefix_plan* p) {
  void* ws = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(g_ws.data()) + 255) & ~uintptr_t(255));
  return paged_prefix_decode_run(p, g_any, 1024, 128, g_any, g_any, 4096, 2048, reinterpret_cast<int32_t*>(g_any),
                                 1 << 16, nullptr, nullptr, g_any, nullptr, ws, g_ws.size() - 256, nullptr);
}

// The plan runs as one of `b`: every key and row of it in what the kernels get.
void runs_as(const pka_prefix_plan* p, const Batch& b) {
  const int merges = g_merges, plain = g_plain;
  pka_prefix_plan_info info;
  REQUIRE(run(p) == PKA_OK && paged_prefix_decode_plan_info(p, &info) == PKA_OK);
  REQUIRE(info.shared == (int)b.shared && info.total_q == (int)b.lens.size());
  const int checks = g_checks;
  REQUIRE(paged_prefix_decode_check_tables(p, reinterpret_cast<int32_t*>(g_any), 64, nullptr, nullptr) == PKA_OK);
  REQUIRE(g_checks == checks + (b.shared ? 1 : 0));
  if (!b.shared) {
    REQUIRE(g_plain == plain + 1 && g_merges == merges);
    return;
  }
  REQUIRE(g_merges == merges + 1 && g_plain == plain && g_merge.total_q == (int)b.lens.size());
  REQUIRE(*g_merge.next == 0 && g_merge.next == g_own.next && g_own.next == g_prefix.status + 1);
  REQUIRE(inside(g_prefix.items, info.num_prefix_pieces * sizeof(pka::PrefixItem)));
  REQUIRE(inside(g_prefix.more, (g_prefix.num_pairs + 1) * sizeof(int32_t)));
  REQUIRE(inside(g_own.pieces, g_own.num_pieces * sizeof(pka::OwnPiece)));
  REQUIRE(inside(g_merge.tokens, b.lens.size() * sizeof(pka::TokenStates)) && inside(g_prefix.status, 8));
  int64_t tiles = 0, want = 0, units = 0, want_units = 0;
  for (int i = 0; i < info.num_prefix_pieces; ++i) tiles += g_prefix.items[i].tile_hi - g_prefix.items[i].tile_lo;
  for (int i = 0; i < g_own.num_pieces; ++i) units += g_own.pieces[i].unit_hi - g_own.pieces[i].unit_lo;
  for (size_t g = 0; g < b.pages.size(); ++g) {
    const int n = b.groups[g + 1] - b.groups[g];
    const bool shares = n > 1 && b.pages[g] > 0;
    if (shares) want += 2 * ((b.pages[g] + 3) / 4) * ((n * 4 + 255) / 256);   // 2 KV heads, 4 rows a request
    for (int r = b.groups[g]; r < b.groups[g + 1]; ++r) want_units += 2 * ((b.lens[r] + 15) / 16 - (shares ? b.pages[g] : 0));
  }
  REQUIRE(tiles == want && units == want_units);
}

void nothing_left() { REQUIRE(g_device.empty() && g_pinned.empty() && g_events == 0); }

}  // namespace

int main() {
  const Batch few{{300, 400}, {0, 2}, {10}, true}, other{{500, 90, 700}, {0, 1, 3}, {9, 4}, true},
      many{std::vector<int32_t>(3000, 500), {0, 3000}, {20}, true}, none{{300, 400, 20}, {0, 3}, {0}, false};
  pka_decode_desc d{};
  d.num_qo_heads = 8;
  d.num_kv_heads = 2;
  d.head_dim = 128;
  d.page_size = 16;
  d.max_pages_per_seq = 64;
  d.num_pages = 6000;
  d.q_len = 1;
  d.window_left = -1;
  d.scale = 0.1f;
  d.bmm2_scale = 1.f;
  d.freeze_seq_lens = 1;
  size_t bytes = 0;
  auto make = [&](const Batch& b, pka_prefix_plan** p) {
    d.batch_size = (int32_t)b.lens.size();
    return paged_prefix_decode_plan(p, &d, b.lens.data(), nullptr, b.groups.data(), (int32_t)b.pages.size(),
                                    b.pages.data(), 0, &bytes, nullptr);
  };
  auto update = [&](pka_prefix_plan* p, const Batch& b) {
    return paged_prefix_decode_plan_update(p, (int32_t)b.lens.size(), b.lens.data(), nullptr, b.groups.data(),
                                           (int32_t)b.pages.size(), b.pages.data(), &bytes, nullptr);
  };

  // plans that cannot be made
  for (const Batch& b : {few, none})
    for (const char* call : {"cudaMalloc", "cudaMallocHost", "cudaMemcpyAsync", "cudaEventCreate"}) {
      if (!b.shared && (std::strcmp(call, "cudaMallocHost") == 0 || std::strcmp(call, "cudaEventCreate") == 0)) continue;
      pka_prefix_plan* p = nullptr;
      g_refuse = call;
      g_refused = 0;
      REQUIRE(make(b, &p) == PKA_ERR_CUDA && p == nullptr && g_refused > 0);
      g_refuse.clear();
      nothing_left();
    }

  // updates that fail, from a plan that shares, one that does not, and one that has done both
  for (const Batch& first : {few, none})
    for (const bool both : {false, true})
      for (const Batch& to : {many, other})
        for (const char* call : {"cudaMalloc", "cudaMallocHost", "cudaMemcpyAsync", "cudaEventSynchronize"}) {
          pka_prefix_plan* p = nullptr;
          REQUIRE(make(first, &p) == PKA_OK);
          if (both) {
            REQUIRE(update(p, first.shared ? none : few) == PKA_OK);
            runs_as(p, first.shared ? none : few);
            REQUIRE(update(p, first) == PKA_OK);
          }
          runs_as(p, first);
          const Batch* now = &first;
          for (int again = 0; again < 2; ++again) {
            g_refuse = call;
            g_refused = 0;
            const int rc = update(p, to);
            g_refuse.clear();
            REQUIRE(rc == (g_refused > 0 ? PKA_ERR_CUDA : PKA_OK));
            if (rc == PKA_OK) now = &to;   // the call was not made, as nothing had to be waited for or grow
            runs_as(p, *now);
          }
          for (const Batch& next : {other, none, many, few, none, other}) {
            REQUIRE(update(p, next) == PKA_OK);
            runs_as(p, next);
          }
          REQUIRE(g_device.size() == 2 && g_pinned.size() == 1 && g_events == 1);
          paged_prefix_decode_plan_destroy(p);
          nothing_left();
        }

  // a copy that cannot be followed by an event is waited for
  {
    pka_prefix_plan* p = nullptr;
    g_refuse = "cudaEventRecord";
    REQUIRE(make(few, &p) == PKA_OK);
    runs_as(p, few);
    REQUIRE(update(p, many) == PKA_OK);
    g_refuse.clear();
    runs_as(p, many);
    paged_prefix_decode_plan_destroy(p);
    nothing_left();
  }

  // refused arguments change nothing, nor does a run whose launches fail; the count of pieces taken is put back
  {
    pka_prefix_plan* p = nullptr;
    REQUIRE(make(few, &p) == PKA_OK);
    REQUIRE(update(p, Batch{{300, 100}, {0, 2}, {10}, true}) == PKA_ERR_INVALID_ARG);
    runs_as(p, few);
    for (const char* call : {"launch_prefix", "launch_merge"}) {
      g_refuse = call;
      REQUIRE(run(p) == PKA_ERR_CUDA);
      g_refuse.clear();
      REQUIRE(*g_own.next == 0);
      runs_as(p, few);
    }
    paged_prefix_decode_plan_destroy(p);
    nothing_left();
  }
  std::puts("ok");
  return 0;
}
