// Host-side checks shared by the C entry points: devices, streams, pointers,
// graph capture (internal to the library).
#pragma once

#include "mqa_fp4_topk.h"

#include <hip/hip_runtime.h>

#include <cstring>
#include <mutex>

namespace mqa {
namespace host {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  bool probed = false;
  bool gfx950 = false;
  int cus = 0;
  bool pool_ready = false;
};

inline std::mutex g_mu;
inline DeviceInfo g_dev[kMaxDevices];

// Probes (once) whether `dev` is a gfx950 and how many CUs it has.
inline int32_t device_info(int dev, DeviceInfo* out) {
  if (dev < 0 || dev >= kMaxDevices) return MQA_ERR_DEVICE;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.probed) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
      (void)hipGetLastError();
      return MQA_ERR_HIP;
    }
    d.gfx950 = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    d.cus = prop.multiProcessorCount;
    d.probed = true;
  }
  if (!d.pool_ready && d.gfx950) {
    // keep freed scratch in the device's default pool instead of returning it
    hipMemPool_t pool;
    if (hipDeviceGetDefaultMemPool(&pool, dev) == hipSuccess) {
      uint64_t thr = ~0ull;
      (void)hipMemPoolSetAttribute(pool, hipMemPoolAttrReleaseThreshold, &thr);
    }
    (void)hipGetLastError();
    d.pool_ready = true;
  }
  *out = d;
  return d.gfx950 ? MQA_OK : MQA_ERR_DEVICE;
}

// Restores the caller's current device on scope exit.
struct DeviceGuard {
  int saved = -1;
  bool changed = false;
  int32_t enter(int dev) {
    if (hipGetDevice(&saved) != hipSuccess) {
      (void)hipGetLastError();
      return MQA_ERR_HIP;
    }
    if (saved != dev) {
      if (hipSetDevice(dev) != hipSuccess) {
        (void)hipGetLastError();
        return MQA_ERR_HIP;
      }
      changed = true;
    }
    return MQA_OK;
  }
  ~DeviceGuard() {
    if (changed) (void)hipSetDevice(saved);
  }
};

inline int32_t stream_device(hipStream_t st, int* dev) {
  const bool ok = (st == nullptr ? hipGetDevice(dev) : hipStreamGetDevice(st, dev)) == hipSuccess;
  if (!ok) (void)hipGetLastError();   // reported through the return code only
  return ok ? MQA_OK : st == nullptr ? MQA_ERR_HIP : MQA_ERR_DEVICE;
}

// A non-null pointer must be device (or managed) memory of device `dev`.
inline int32_t check_ptr_device(const void* p, int dev) {
  if (p == nullptr) return MQA_OK;
  hipPointerAttribute_t attr;
  std::memset(&attr, 0, sizeof(attr));
  if (hipPointerGetAttributes(&attr, p) != hipSuccess) {
    (void)hipGetLastError();
    return MQA_ERR_DEVICE;
  }
  if (attr.type != hipMemoryTypeDevice && attr.type != hipMemoryTypeManaged) return MQA_ERR_DEVICE;
  if (attr.device != dev) return MQA_ERR_DEVICE;
  return MQA_OK;
}

struct PtrSpec {
  const void* p;
  bool required;
  uintptr_t align;
};

// Host-only pointer checks (no HIP call): presence and alignment.
inline int32_t check_ptrs_host(const PtrSpec* specs, int n) {
  for (int i = 0; i < n; ++i)
    if (specs[i].required && specs[i].p == nullptr) return MQA_ERR_NULL_POINTER;
  for (int i = 0; i < n; ++i)
    if (specs[i].p && reinterpret_cast<uintptr_t>(specs[i].p) % specs[i].align) return MQA_ERR_MISALIGNED;
  return MQA_OK;
}

inline int32_t check_ptrs_device(const PtrSpec* specs, int n, int dev) {
  for (int i = 0; i < n; ++i) {
    const int32_t rc = check_ptr_device(specs[i].p, dev);
    if (rc != MQA_OK) return rc;
  }
  return MQA_OK;
}

// Memory that a call reads or writes: `rows` pieces of `bytes` bytes at a byte stride.
struct Span {
  const void* p;
  int64_t rows, stride, bytes;

  Span(const void* p_, int64_t rows_, int64_t stride_, int64_t bytes_) : p(p_), rows(rows_), stride(stride_), bytes(bytes_) {
    if (rows > 1 && stride <= bytes) {   // one piece
      bytes += (rows - 1) * stride;
      rows = 1;
    }
  }
};

// Whether two spans share a byte. Two of several rows each and different strides count as apart.
inline bool overlap(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr || a.rows < 1 || b.rows < 1 || a.bytes < 1 || b.bytes < 1) return false;
  if (a.rows > 1 && b.rows > 1 && a.stride != b.stride) return false;
  const __int128 d = static_cast<__int128>(reinterpret_cast<uintptr_t>(b.p)) - reinterpret_cast<uintptr_t>(a.p);
  const __int128 s = a.rows > 1 ? a.stride : b.rows > 1 ? b.stride : 0;
  // row j of b begins k = j - i strides and d bytes behind row i of a: is -b.bytes < d + k s < a.bytes for any k?
  __int128 k = 1 - static_cast<__int128>(a.rows);
  if (s > 0 && d + k * s <= -static_cast<__int128>(b.bytes)) k += (-b.bytes - (d + k * s)) / s + 1;   // the first above -b.bytes
  return k < b.rows && d + k * s > -static_cast<__int128>(b.bytes) && d + k * s < a.bytes;
}

// No output may overlap an input or an output behind it.
inline int32_t check_apart(const Span* outs, int n_outs, const Span* ins, int n_ins) {
  for (int i = 0; i < n_outs; ++i) {
    for (int j = i + 1; j < n_outs; ++j)
      if (overlap(outs[i], outs[j])) return MQA_ERR_OVERLAP;
    for (int j = 0; j < n_ins; ++j)
      if (overlap(outs[i], ins[j])) return MQA_ERR_OVERLAP;
  }
  return MQA_OK;
}

inline int32_t check_capture(hipStream_t st) {
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(st, &cs) != hipSuccess) {
    (void)hipGetLastError();
    return MQA_ERR_HIP;
  }
  return cs == hipStreamCaptureStatusNone ? MQA_OK : MQA_ERR_CAPTURING;
}

// Common entry checks; on success the guard holds the tensors' device.
// Order: host-only checks first (testable without a GPU), then device checks.
inline int32_t enter(hipStream_t st, const PtrSpec* specs, int nspecs, DeviceGuard& guard, DeviceInfo* info,
              bool allow_capture = false) {
  int32_t rc = check_ptrs_host(specs, nspecs);
  if (rc != MQA_OK) return rc;
  int dev = -1;
  rc = stream_device(st, &dev);
  if (rc != MQA_OK) return rc;
  if (!allow_capture) {
    rc = check_capture(st);
    if (rc != MQA_OK) return rc;
  }
  rc = device_info(dev, info);
  if (rc != MQA_OK) return rc;
  rc = check_ptrs_device(specs, nspecs, dev);
  if (rc != MQA_OK) return rc;
  return guard.enter(dev);
}

inline int32_t hip_rc(hipError_t e) {
  if (e == hipSuccess) return MQA_OK;
  (void)hipGetLastError();
  return MQA_ERR_HIP;
}

}  // namespace host
}  // namespace mqa
