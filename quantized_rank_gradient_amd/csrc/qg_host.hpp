// What the host sides of the entry points share: argument checks and errors.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <string>

#include "qg_kernels.hpp"
#include "qgalore.h"

namespace qg_host {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

// Text of this thread's last QG_ERR_HIP.
extern thread_local std::string g_last_error;
qg_status hip_fail(hipError_t e, const char* what);
qg_status device_present();

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
inline bool finite(float x) { return std::isfinite(x); }
// Whether p's np bytes and q's nq bytes share any (never with a null pointer).
inline bool overlap(const void* p, int64_t np, const void* q, int64_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && (a <= b ? b - a < (uintptr_t)np : a - b < (uintptr_t)nq);
}
struct Span {
  const void* p;
  int64_t bytes;
};
inline bool clash(const Span& out, std::initializer_list<Span> others) {
  for (const Span& s : others)
    if (overlap(out.p, out.bytes, s.p, s.bytes)) return true;
  return false;
}
inline qg_status check_scratch(const void* p, size_t have, int64_t need) {
  if (need == 0) return QG_OK;
  if (!p) return QG_ERR_NULL;
  if (!aligned(p, 16)) return QG_ERR_ALIGN;
  return have >= (size_t)need ? QG_OK : QG_ERR_WORKSPACE;
}

}  // namespace qg_host
