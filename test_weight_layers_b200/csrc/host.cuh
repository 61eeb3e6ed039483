// Host-side helpers shared by the library's translation units: launch
// accounting, per-kernel event timing, status macros and launch wrappers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cstdlib>
#include <mutex>
#include <vector>

#include "ttt.h"

namespace ttt {

inline std::atomic<uint64_t> g_launches{0};

// ---- per-kernel event timing (ttt_profile_*)
struct ProfPair {
  cudaEvent_t a, b;
  int kind;
};
inline std::mutex g_prof_mu;
inline std::atomic<bool> g_prof_on{false};
inline std::vector<ProfPair> g_prof_pending;
inline std::vector<cudaEvent_t> g_prof_pool;
inline double g_prof_ms[TTT_PROF_KINDS] = {0};
inline uint64_t g_prof_n[TTT_PROF_KINDS] = {0};

inline cudaEvent_t prof_event() {
  if (!g_prof_pool.empty()) {
    cudaEvent_t e = g_prof_pool.back();
    g_prof_pool.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
  return e;
}

// Records an event pair around the launches issued during its lifetime.
struct ProfScope {
  cudaEvent_t a = nullptr, b = nullptr;
  cudaStream_t s;
  int kind;
  ProfScope(int k, cudaStream_t st) : s(st), kind(k) {
    if (!g_prof_on.load(std::memory_order_relaxed)) return;
    std::lock_guard<std::mutex> lk(g_prof_mu);
    a = prof_event();
    b = prof_event();
    if (a && b) cudaEventRecord(a, s);
  }
  ~ProfScope() {
    if (!a || !b) return;
    cudaEventRecord(b, s);
    std::lock_guard<std::mutex> lk(g_prof_mu);
    g_prof_pending.push_back({a, b, kind});
  }
};
constexpr unsigned long long kDefaultTimeoutNs = 2000000000ull;  // 2 s per device-side wait

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int sm_count() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 0 || dev >= 64) return 148;
  if (!cache[dev]) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) v = 148;
    cache[dev] = v;
  }
  return cache[dev];
}

inline unsigned long long wait_timeout_ns() {
  static unsigned long long v = [] {
    const char* e = std::getenv("TTT_WAIT_TIMEOUT_MS");
    if (e && *e) {
      long long ms = std::atoll(e);
      if (ms > 0) return (unsigned long long)ms * 1000000ull;
    }
    return kDefaultTimeoutNs;
  }();
  return v;
}

#define TTT_LAUNCHED()                                         \
  do {                                                         \
    g_launches.fetch_add(1, std::memory_order_relaxed);        \
    if (cudaPeekAtLastError() != cudaSuccess) {                \
      (void)cudaGetLastError();                                \
      return TTT_ERR_CUDA;                                     \
    }                                                          \
  } while (0)

#define TTT_CHECK(expr)                        \
  do {                                         \
    if ((expr) != cudaSuccess) {               \
      (void)cudaGetLastError();                \
      return TTT_ERR_CUDA;                     \
    }                                          \
  } while (0)

#define TTT_TRY(expr)           \
  do {                          \
    int rc_ = (expr);           \
    if (rc_ != TTT_OK) return rc_; \
  } while (0)

inline int grid1d(int64_t n, int threads) {
  int64_t b = (n + threads - 1) / threads;
  return (int)std::max<int64_t>(1, std::min<int64_t>(b, (int64_t)sm_count() * 32));
}

inline size_t esize(ttt_dtype dt) { return dt == TTT_BF16 ? 2 : 4; }


// Launch with programmatic stream serialisation: the kernel may begin while the
// previous kernel on the stream finishes, and must call pdl_wait() before it
// touches memory that kernel writes.  Used for the short dependent kernels of
// the Muon step, whose launch latency is otherwise a large share of their time.
template <typename... KArgs, typename... Args>
int launch_pdl(void (*k)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  TTT_CHECK(cudaLaunchKernelEx(&cfg, k, static_cast<KArgs>(args)...));
  return TTT_OK;
}

}  // namespace ttt
