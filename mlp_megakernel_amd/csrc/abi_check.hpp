// What every file of the C ABI uses: the last error, the device's compute
// units, and the checks of operands.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "../../include/coalesce.h"
#include "launch.hpp"

namespace coalesce {

inline thread_local char g_last_error[512] = "";

inline coalesce_status fail(coalesce_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return s;
}

inline coalesce_status ok() {
  g_last_error[0] = '\0';
  return COALESCE_OK;
}

inline coalesce_status device_fail(hipError_t e, const char* what) {
  return fail(COALESCE_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
}

constexpr int kMaxDevices = 64;
inline std::mutex g_props_mutex;
inline int g_cu_count[kMaxDevices] = {0};

// CU count of the current device, queried once per device.
inline coalesce_status current_cus(int* out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return device_fail(e, "hipGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(COALESCE_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_props_mutex);
  if (g_cu_count[dev] == 0) {
    int cus = 0;
    e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return device_fail(e, "hipDeviceGetAttribute");
    if (cus <= 0) return fail(COALESCE_ERR_DEVICE, "device reports %d compute units", cus);
    g_cu_count[dev] = cus;
  }
  *out = g_cu_count[dev];
  return COALESCE_OK;
}

inline bool valid_dtype(int d) { return d == COALESCE_F32 || d == COALESCE_F16 || d == COALESCE_BF16; }
inline bool valid_act(int a) {
  return a == COALESCE_ACT_NONE || a == COALESCE_ACT_GELU_ERF || a == COALESCE_ACT_SOFTPLUS || a == COALESCE_ACT_RELU;
}
inline int64_t dsize(int d) { return d == COALESCE_F32 ? 4 : 2; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr int64_t kMaxExtent = (int64_t)INT32_MAX;

// Byte range [lo, hi) covered by a rows x cols matrix with leading dimension ld.
struct Range {
  uintptr_t lo, hi;
};
inline Range span(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t es) {
  uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (!p || rows <= 0 || cols <= 0) return {lo, lo};
  return {lo, lo + (uintptr_t)(((rows - 1) * ld + cols) * es)};
}
inline bool overlap(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

inline int act_code(coalesce_act a) {
  return a == COALESCE_ACT_GELU_ERF ? ACT_GELU
         : a == COALESCE_ACT_SOFTPLUS ? ACT_SOFTPLUS
         : a == COALESCE_ACT_RELU     ? ACT_RELU
                                      : ACT_NONE;
}

// Activations of the feed-forward operators: those of the GEMM and SiLU.
inline bool valid_ffn_act(int a) { return valid_act((coalesce_act)a) || a == COALESCE_ACT_SILU; }
inline int ffn_act_code(coalesce_act a) { return a == COALESCE_ACT_SILU ? (int)ACT_SILU : act_code(a); }
inline DType dt_code(coalesce_dtype d) { return d == COALESCE_F32 ? DT_F32 : d == COALESCE_F16 ? DT_F16 : DT_BF16; }

// A rows x cols matrix operand that has elements: present, pitch at least the
// row and at most 2^23 (256 rows are addressed with 32-bit byte offsets),
// 16-byte aligned rows.
inline coalesce_status check_mat(const void* t, int64_t ld, int64_t cols, int64_t es, const char* name) {
  if (!t) return fail(COALESCE_ERR_INVALID_ARGUMENT, "%s is NULL", name);
  if (ld < cols) return fail(COALESCE_ERR_INVALID_ARGUMENT, "the pitch of %s is shorter than the row", name);
  if (ld >= (int64_t(1) << 23)) return fail(COALESCE_ERR_UNSUPPORTED, "the pitch of %s must be below 2^23", name);
  if (!aligned16(t) || (ld * es) % 16)
    return fail(COALESCE_ERR_UNSUPPORTED, "%s must be 16-byte aligned with a 16-byte row pitch", name);
  return COALESCE_OK;
}
inline coalesce_status check_vec(const void* t, const char* name) {
  if (t && !aligned16(t)) return fail(COALESCE_ERR_UNSUPPORTED, "%s must be 16-byte aligned", name);
  return COALESCE_OK;
}

// Operands of a call, to refuse outputs that overlap anything else.  Matrices
// of one pitch may interleave (the halves of a wider matrix): their rows are
// disjoint where the distance between the bases, modulo the pitch, leaves room
// for both rows.
struct Operand {
  Range r;
  const char* name;
  bool out;
  uint64_t row = 0, pitch = 0;  // bytes; pitch 0: one run of memory
};
inline bool interleaved(const Operand& a, const Operand& b) {
  if (!a.pitch || a.pitch != b.pitch) return false;
  const uint64_t dist = b.r.lo >= a.r.lo ? (uint64_t)(b.r.lo - a.r.lo) % a.pitch
                                         : (a.pitch - (uint64_t)(a.r.lo - b.r.lo) % a.pitch) % a.pitch;
  return dist >= a.row && dist + b.row <= a.pitch;
}
struct Operands {
  Operand v[16];
  int n = 0;
  void mat(bool out, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t es, const char* name) {
    v[n++] = {span(p, rows, cols, ld, es), name, out, (uint64_t)(cols * es), (uint64_t)(ld * es)};
  }
  void run(bool out, const Range& r, const char* name) { v[n++] = {r, name, out}; }
  coalesce_status check() const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j)
        if ((v[i].out || v[j].out) && overlap(v[i].r, v[j].r) && !interleaved(v[i], v[j]))
          return fail(COALESCE_ERR_INVALID_ARGUMENT, "%s overlaps %s", v[v[i].out ? i : j].name,
                      v[v[i].out ? j : i].name);
    return COALESCE_OK;
  }
};

inline coalesce_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return COALESCE_OK;
  if (!ws) return fail(COALESCE_ERR_INVALID_ARGUMENT, "workspace is NULL (%zu bytes are needed)", need);
  if (!aligned16(ws)) return fail(COALESCE_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
  if (have < need)
    return fail(COALESCE_ERR_INVALID_ARGUMENT, "workspace of %zu bytes is smaller than the %zu needed", have, need);
  return COALESCE_OK;
}

}  // namespace coalesce
