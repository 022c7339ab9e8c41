// Latent decode plans whose CUDA calls fail, on the host: the entry points of
// latent_abi.cpp and the planner over a fake runtime that refuses the calls it is told
// to.  A plan made or updated in vain leaks nothing, and an update that fails leaves the
// plan as it was, which still runs and still updates.
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <memory>
#include <string>
#include <vector>

#include "host_common.h"
#include "latent.h"
#include "tmap.h"

namespace {

std::map<const void*, size_t> g_device, g_pinned;   // live allocations
int g_events = 0;
std::string g_refuse;     // the call that fails
int g_refused = 0;        // how often it did
bool g_last = false;      // a refusal that cudaGetLastError would still tell of
pka::LatentArgs g_run;    // what the last run was launched with
int g_runs = 0;
std::string g_error;

bool refused(const char* name) {
  if (g_refuse != name) return false;
  ++g_refused;
  return g_last = true;
}

#define REQUIRE(cond)                                                          \
  do {                                                                         \
    if (!(cond)) {                                                             \
      std::printf("line %d: %s (%s)\n", __LINE__, #cond, g_error.c_str());     \
      std::exit(1);                                                            \
    }                                                                          \
  } while (0)

bool inside(const std::map<const void*, size_t>& all, const void* p, size_t n) {
  for (const auto& [base, size] : all) {
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
  REQUIRE(inside(g_device, dst, n) && inside(g_pinned, src, n));
  std::memcpy(dst, src, n);
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
  const bool last = g_last;
  g_last = false;
  return last ? cudaErrorUnknown : cudaSuccess;
}
const char* cudaGetErrorString(cudaError_t) { return "refused"; }
void batch_prefill_plan_destroy(pka_prefill_plan*) {}
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
int encode_bf16_map(CUtensorMap*, const void*, int, const uint64_t*, const uint64_t*, const uint32_t*) {
  return PKA_OK;
}
int make_prefill_plan(pka_prefill_plan**, const pka_prefill_desc&, const int32_t*, const int32_t*, bool,
                      int32_t*, cudaStream_t) {
  return PKA_ERR_UNSUPPORTED;
}
int launch_latent_decode(const pka_latent_plan&, const LatentArgs& a, const void*, int64_t, cudaStream_t) {
  if (cudaGetLastError() != cudaSuccess) return fail(PKA_ERR_CUDA, "an earlier call's error at a launch");
  g_run = a;
  ++g_runs;
  return PKA_OK;
}
int launch_latent_prefill(const pka_prefill_plan&, const PrefillArgs&, const LatentPrefillParts&,
                          const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                          cudaStream_t) {
  return PKA_OK;
}
int launch_kv_tables(const int32_t*, const int32_t*, int32_t, const int32_t*, int32_t, const int32_t*, int32_t,
                     int32_t*, int64_t, int32_t, int32_t*, int32_t*, int64_t*, int64_t, int32_t*, int32_t*,
                     cudaStream_t) {
  return PKA_OK;
}
int launch_latent_append(const void*, int64_t, const void*, int64_t, int32_t, int32_t, const int64_t*, int64_t,
                         void*, int64_t, int32_t, int64_t, int32_t*, cudaStream_t) {
  return PKA_OK;
}
}  // namespace pka

namespace {

alignas(256) char g_any[64];   // an address for the run's tensors
std::vector<char> g_ws(1 << 28);

// The plan runs, over pieces that lie on the device and are those of `lens`.
void runs_over(const pka_latent_plan* p, const std::vector<int32_t>& lens) {
  const int before = g_runs;
  void* ws = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(g_ws.data()) + 255) & ~uintptr_t(255));
  const int rc = paged_latent_decode_run(p, g_any, 320 * 16, 320, g_any, 16 * 320,
                                         reinterpret_cast<int32_t*>(g_any), 1 << 16, nullptr, g_any, nullptr, ws,
                                         g_ws.size() - 256, nullptr);
  REQUIRE(rc == PKA_OK && g_runs == before + 1);
  pka_latent_plan_info info;
  REQUIRE(paged_latent_decode_plan_info(p, &info) == PKA_OK);
  REQUIRE(info.total_q == (int)lens.size() && g_run.num_segments == info.num_segments);
  REQUIRE(inside(g_device, g_run.pieces, info.num_items * sizeof(pka::LatentPiece)));
  REQUIRE(inside(g_device, g_run.more, (info.num_segments + 1) * sizeof(int32_t)));
  REQUIRE(inside(g_device, g_run.status, 4));
  std::vector<int64_t> tiles(lens.size(), 0);
  for (int i = 0; i < info.num_items; ++i) {
    const pka::LatentPiece& c = g_run.pieces[i];
    REQUIRE(c.request >= 0 && c.request < (int)lens.size() && c.kv_len == lens[c.request]);
    tiles[c.request] += c.tile_hi - c.tile_lo;
  }
  for (size_t b = 0; b < lens.size(); ++b) REQUIRE(tiles[b] == (lens[b] + 63) / 64);
}

void nothing_left() { REQUIRE(g_device.empty() && g_pinned.empty() && g_events == 0); }

}  // namespace

int main() {
  const std::vector<int32_t> small = {300, 40}, large(4000, 500), other = {64, 129, 7};
  pka_latent_desc d{};
  d.batch_size = 2;
  d.num_heads = 16;
  d.latent_dim = 256;
  d.rope_dim = 64;
  d.page_size = 16;
  d.max_pages_per_seq = 64;
  d.num_pages = 64;
  d.dtype = PKA_DTYPE_BF16;
  d.out_dtype = PKA_DTYPE_BF16;
  d.q_len = 1;
  d.scale = 0.1f;
  d.output_scale = 1.f;
  d.freeze_seq_lens = 1;
  size_t bytes = 0;
  auto update = [&](pka_latent_plan* p, const std::vector<int32_t>& lens) {
    return paged_latent_decode_plan_update(p, (int32_t)lens.size(), lens.data(), nullptr, &bytes, nullptr);
  };

  // plans that cannot be made
  for (const char* call : {"cudaMalloc", "cudaMallocHost", "cudaMemcpyAsync", "cudaEventCreate", "cudaGetDevice"}) {
    pka_latent_plan* p = nullptr;
    g_refuse = call;
    g_refused = 0;
    REQUIRE(paged_latent_decode_plan(&p, &d, small.data(), nullptr, &bytes, nullptr) == PKA_ERR_CUDA);
    REQUIRE(p == nullptr && g_refused > 0);
    g_refuse.clear();
    nothing_left();
  }

  // updates that fail, where the buffers have to grow and where they do not
  for (const auto& lens : {large, other})
    for (const char* call : {"cudaMalloc", "cudaMallocHost", "cudaMemcpyAsync", "cudaEventSynchronize"}) {
      const bool grows = lens.size() > 100;
      if (!grows && std::strncmp(call, "cudaMalloc", 10) == 0) continue;
      pka_latent_plan* p = nullptr;
      REQUIRE(paged_latent_decode_plan(&p, &d, small.data(), nullptr, &bytes, nullptr) == PKA_OK);
      runs_over(p, small);
      for (int again = 0; again < 2; ++again) {
        g_refuse = call;
        g_refused = 0;
        REQUIRE(update(p, lens) == PKA_ERR_CUDA && g_refused > 0);
        g_refuse.clear();
        runs_over(p, small);          // as it was
      }
      REQUIRE(update(p, other) == PKA_OK);
      runs_over(p, other);
      REQUIRE(update(p, large) == PKA_OK);
      runs_over(p, large);
      REQUIRE(update(p, small) == PKA_OK);
      runs_over(p, small);
      REQUIRE(g_device.size() == 1 && g_pinned.size() == 1 && g_events == 1);
      paged_latent_decode_plan_destroy(p);
      nothing_left();
    }

  // a copy that cannot be followed by an event is waited for
  {
    pka_latent_plan* p = nullptr;
    g_refuse = "cudaEventRecord";
    REQUIRE(paged_latent_decode_plan(&p, &d, small.data(), nullptr, &bytes, nullptr) == PKA_OK);
    runs_over(p, small);
    REQUIRE(update(p, large) == PKA_OK);
    g_refuse.clear();
    runs_over(p, large);
    paged_latent_decode_plan_destroy(p);
    nothing_left();
  }

  // refused arguments change nothing either
  {
    pka_latent_plan* p = nullptr;
    const std::vector<int32_t> wrong = {300, -1};
    REQUIRE(paged_latent_decode_plan(&p, &d, small.data(), nullptr, &bytes, nullptr) == PKA_OK);
    REQUIRE(update(p, wrong) == PKA_ERR_INVALID_ARG);
    runs_over(p, small);
    paged_latent_decode_plan_destroy(p);
    nothing_left();
  }
  std::puts("ok");
  return 0;
}
