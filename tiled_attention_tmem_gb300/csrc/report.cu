// What the library says of itself: status texts, kernel names and the profile.  Nothing
// here changes what a kernel does, so this file is not among those that the benchmark's
// recorded memory traffic depends on.
#include <mutex>
#include <vector>

#include "fa.h"
#include "fa_paged.h"
#include "host.h"

namespace fa {
namespace {
struct ProfRecord {
  int kind;
  cudaEvent_t a, b;
};
std::mutex g_prof_mutex;
bool g_prof_on = false;
std::vector<ProfRecord> g_prof;       // records of the current session
std::vector<cudaEvent_t> g_evt_pool;  // events reused across sessions
size_t g_prof_used_events = 0;
thread_local cudaEvent_t g_pending = nullptr;

cudaEvent_t pool_event() {
  if (g_prof_used_events < g_evt_pool.size()) return g_evt_pool[g_prof_used_events++];
  cudaEvent_t e = nullptr;
  if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
  g_evt_pool.push_back(e);
  ++g_prof_used_events;
  return e;
}
}  // namespace

void prof_before(int kind, cudaStream_t st) {
  (void)kind;
  std::lock_guard<std::mutex> lock(g_prof_mutex);
  if (!g_prof_on) return;
  g_pending = pool_event();
  if (g_pending) cudaEventRecord(g_pending, st);
}

void prof_after(int kind, cudaStream_t st) {
  std::lock_guard<std::mutex> lock(g_prof_mutex);
  if (!g_prof_on || !g_pending) return;
  cudaEvent_t b = pool_event();
  if (!b) return;
  cudaEventRecord(b, st);
  g_prof.push_back({kind, g_pending, b});
  g_pending = nullptr;
}

}  // namespace fa

using namespace fa;

extern "C" {

const char* fa_strerror(fa_status s) {
  switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported head dimension or variant";
    case FA_ERR_MISALIGNED: return "pointer not aligned as the call requires";
    case FA_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
    case FA_ERR_LAUNCH: return "CUDA launch failed";
    case FA_ERR_DEVICE_TIMEOUT: return "in-kernel wait timed out";
  }
  return "unknown status";
}

int fa_profile_start(void) {
  std::lock_guard<std::mutex> lock(g_prof_mutex);
  g_prof.clear();
  g_prof_used_events = 0;
  g_prof_on = true;
  return FA_OK;
}

int fa_profile_stop_kinds(int kinds, int* launches, double* ms) {
  if (kinds < 0) return FA_ERR_INVALID_ARG;
  std::lock_guard<std::mutex> lock(g_prof_mutex);
  g_prof_on = false;
  for (int k = 0; k < kinds; ++k) {
    if (launches) launches[k] = 0;
    if (ms) ms[k] = 0.0;
  }
  int status = FA_OK;
  for (const ProfRecord& r : g_prof) {
    float t = 0.f;
    if (cudaEventSynchronize(r.b) != cudaSuccess || cudaEventElapsedTime(&t, r.a, r.b) != cudaSuccess) {
      status = FA_ERR_LAUNCH;
      continue;
    }
    if (r.kind < 0 || r.kind >= kinds) continue;
    if (launches) launches[r.kind] += 1;
    if (ms) ms[r.kind] += t;
  }
  g_prof.clear();
  g_prof_used_events = 0;
  return status;
}

int fa_profile_stop(fa_profile* out) {
  return fa_profile_stop_kinds(FA_KERNEL_KINDS, out ? out->launches : nullptr, out ? out->ms : nullptr);
}

const char* fa_kernel_name(int kind) {
  switch (kind) {
    case FA_KERNEL_FWD: return "fwd";
    case FA_KERNEL_BWD_PRE: return "bwd_pre";
    case FA_KERNEL_BWD_KV5: return "bwd_kv5";
    case FA_KERNEL_BWD_CONV: return "bwd_conv";
    case FA_KERNEL_BWD_KV7: return "bwd_kv7";
    case FA_KERNEL_BWD_Q7: return "bwd_q7";
    case FA_KERNEL_FWD_MERGE: return "fwd_merge";
    case FA_KERNEL_BWD_KVSUM: return "bwd_kvsum";
    case FA_KERNEL_BWD_QSUM: return "bwd_qsum";
    case FA_KERNEL_PAGE: return "page";
    case FA_KERNEL_KV4_STORE: return "kv4_store";
    case FA_KERNEL_KV4_LOAD: return "kv4_load";
    case FA_KERNEL_KV4_ATTN: return "kv4_attn";
    case FA_KERNEL_KV4_MERGE: return "kv4_merge";
  }
  return "unknown";
}

}  // extern "C"
