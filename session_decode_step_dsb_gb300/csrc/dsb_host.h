// Host-side state shared by the C ABI's translation units: the calling
// thread's error message, the workspace and its ring of metadata slots, device
// queries and the argument checks that more than one of them makes.
#pragma once
#include <cuda_runtime.h>

#include <chrono>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <thread>
#include <vector>

#include "dsb.h"

namespace dsbh {

inline thread_local std::string g_last_error;

inline dsb_status fail(dsb_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  try {
    g_last_error = buf;
  } catch (...) {  // no memory for the message: it is called while an entry point reports just that
    g_last_error.clear();
  }
  return st;
}

inline dsb_status cuda_fail(cudaError_t e, const char* where) {
  return fail(DSB_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorString(e), cudaGetErrorName(e));
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kSlots = 16;
constexpr size_t kMetaHeader = 16;
constexpr size_t kMetaWords = kMetaHeader + 3 * (size_t)DSB_MAX_SEQS + 1 + (size_t)DSB_MAX_TOKENS;
constexpr size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
constexpr size_t kMetaSlotBytes = round_up(kMetaWords * sizeof(int32_t), 256);
constexpr size_t kMetaBytes = kSlots * kMetaSlotBytes;
constexpr double kHostWaitSeconds = 30.0;

struct DeviceInfo {
  int sms = 0;
  int max_smem_optin = 0;
};

inline dsb_status device_info(DeviceInfo* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  static std::mutex mu;
  static DeviceInfo cache[64];
  if (dev >= 0 && dev < 64) {
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev].sms > 0) {
      *out = cache[dev];
      return DSB_OK;
    }
  }
  DeviceInfo d;
  e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(SM count)");
  e = cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(shared memory)");
  if (dev >= 0 && dev < 64) {
    std::lock_guard<std::mutex> lock(mu);
    cache[dev] = d;
  }
  *out = d;
  return DSB_OK;
}

}  // namespace dsbh

struct dsb_workspace {
  int device = -1;
  char* dev = nullptr;
  size_t dev_bytes = 0;
  char* host = nullptr;  // pinned, kSlots * kMetaSlotBytes
  cudaEvent_t ev[dsbh::kSlots] = {};
  bool pending[dsbh::kSlots] = {};
  int next = 0;
};

namespace dsbh {

// Copy `n` int32 words of metadata into the next staging slot and enqueue
// the host -> device copy.  Returns the device address of the slot.
inline dsb_status stage(dsb_workspace* ws, const std::vector<int32_t>& words, cudaStream_t st, const int32_t** dev_out) {
  if (words.size() > kMetaWords) return fail(DSB_ERR_INVALID_ARG, "metadata exceeds the staging slot");
  const int slot = ws->next;
  ws->next = (slot + 1) % kSlots;
  if (ws->pending[slot]) {
    const auto t0 = std::chrono::steady_clock::now();
    for (;;) {
      cudaError_t q = cudaEventQuery(ws->ev[slot]);
      if (q == cudaSuccess) break;
      if (q != cudaErrorNotReady) return cuda_fail(q, "cudaEventQuery(staging slot)");
      if (std::chrono::duration<double>(std::chrono::steady_clock::now() - t0).count() > kHostWaitSeconds)
        return fail(DSB_ERR_TIMEOUT, "staging slot still in use after %.0f s", kHostWaitSeconds);
      std::this_thread::yield();
    }
    ws->pending[slot] = false;
  }
  char* h = ws->host + (size_t)slot * kMetaSlotBytes;
  char* d = ws->dev + (size_t)slot * kMetaSlotBytes;
  std::memcpy(h, words.data(), words.size() * sizeof(int32_t));
  cudaError_t e = cudaMemcpyAsync(d, h, words.size() * sizeof(int32_t), cudaMemcpyHostToDevice, st);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyAsync(metadata)");
  e = cudaEventRecord(ws->ev[slot], st);
  if (e != cudaSuccess) return cuda_fail(e, "cudaEventRecord(metadata)");
  ws->pending[slot] = true;
  *dev_out = reinterpret_cast<const int32_t*>(d);
  return DSB_OK;
}

inline char* partial_base(dsb_workspace* ws) { return ws->dev + kMetaBytes; }
inline size_t partial_capacity(const dsb_workspace* ws) { return ws->dev_bytes > kMetaBytes ? ws->dev_bytes - kMetaBytes : 0; }

inline dsb_status check_rope(const dsb_rope* r) {
  if (!r) return fail(DSB_ERR_INVALID_ARG, "rope is NULL");
  if (!(r->theta > 0.0f) || !std::isfinite(r->theta)) return fail(DSB_ERR_INVALID_ARG, "theta must be finite and > 0");
  if (std::isnan(r->yarn_factor) || std::isinf(r->yarn_factor))
    return fail(DSB_ERR_INVALID_ARG, "yarn_factor must be finite");
  if (r->yarn_factor > 1.0f) {
    if (r->yarn_orig_ctx < 1) return fail(DSB_ERR_INVALID_ARG, "yarn_orig_ctx=%d < 1", r->yarn_orig_ctx);
    if (!(r->yarn_beta_slow > 0.0f) || !(r->yarn_beta_fast > r->yarn_beta_slow) || !std::isfinite(r->yarn_beta_fast))
      return fail(DSB_ERR_INVALID_ARG, "yarn betas must satisfy 0 < beta_slow < beta_fast, finite");
  }
  return DSB_OK;
}

}  // namespace dsbh
