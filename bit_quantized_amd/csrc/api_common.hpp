// Shared by the C ABI's translation units (api.cpp, api_block.cpp): device
// check, alignment, and the optional timing of every launch.
#pragma once

#include "../../include/fourtune.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <mutex>
#include <vector>

namespace ft {
namespace api {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr int64_t kMaxDim = int64_t(1) << 30;

// FT_OK if the current device is gfx950 (cached per device).
ft_status device_check();

inline ft_status launched(hipError_t e) { return e == hipSuccess ? FT_OK : FT_EDEVICE; }

// ---- optional per-kernel timing (benchmarks): hipEvents around each launch
// Kernel names are string literals (static storage), so the pointers handed
// out by fourtune_timing_read stay valid for the life of the process.
struct TimingState {
  std::mutex mu;
  std::atomic<bool> on{false};
  std::vector<hipEvent_t> pool;
  struct Pending { int slot; hipEvent_t a, b; };
  std::vector<Pending> pending;
  std::vector<const char*> names;
  std::vector<double> total_ms;
  std::vector<int64_t> counts;
  int slot(const char* n);
  hipEvent_t take() {
    if (pool.empty()) {
      hipEvent_t e = nullptr;
      if (hipEventCreate(&e) != hipSuccess) return nullptr;
      return e;
    }
    hipEvent_t e = pool.back();
    pool.pop_back();
    return e;
  }
  void drain() {  // caller holds mu
    for (auto& p : pending) {
      float ms = 0.f;
      if (hipEventSynchronize(p.b) == hipSuccess && hipEventElapsedTime(&ms, p.a, p.b) == hipSuccess) {
        total_ms[p.slot] += ms;
        counts[p.slot] += 1;
      }
      pool.push_back(p.a);
      pool.push_back(p.b);
    }
    pending.clear();
  }
};
extern TimingState g_tm;
// Set by the entry point that allocates nothing while it runs: no timing
// events are created for its launches (creating one allocates).
extern thread_local bool t_no_timing;

// Brackets one launch with events when timing is on.
struct Timed {
  hipEvent_t a = nullptr, b = nullptr;
  int slot = -1;
  hipStream_t st;
  Timed(const char* name, hipStream_t s) : st(s) {
    if (t_no_timing || !g_tm.on.load(std::memory_order_relaxed)) return;
    std::lock_guard<std::mutex> lk(g_tm.mu);
    slot = g_tm.slot(name);
    a = g_tm.take();
    b = g_tm.take();
    if (a && b) hipEventRecord(a, st);
  }
  hipError_t done(hipError_t e) {
    if (a && b) {
      hipEventRecord(b, st);
      std::lock_guard<std::mutex> lk(g_tm.mu);
      g_tm.pending.push_back({slot, a, b});
    }
    return e;
  }
};

}  // namespace api
}  // namespace ft
