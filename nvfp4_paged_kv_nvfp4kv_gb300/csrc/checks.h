// checks.h -- argument checks shared by the host files of the serving-step entry
// points (api_step.cpp, api_tree.cpp).
#pragma once

#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include <cuda_runtime_api.h>

#include "internal.h"
#include "nvfp4kv.h"

namespace nvfp4kv {

inline int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_error_detail(status, buf);
}
inline int ok() { return set_error_detail(NVFP4KV_OK, ""); }
inline int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ok();
  return fail(NVFP4KV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}
inline bool aligned(const void* p, uint64_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool bad_row_strides(const void* p, int64_t st, int64_t sh) {
  return !aligned(p, 16) || st % 8 || sh % 8 || st < 0 || sh < 0;
}

// Whether runs of `run` units at all multiples 0 .. count - 1 of the strides lie
// apart: in order of their strides, each step passes all that lies below it.
struct Span {
  int64_t count, stride;
};
inline bool lie_apart(int64_t run, std::initializer_list<Span> spans) {
  Span by[3];
  int n = 0;
  for (const Span& s : spans)
    if (s.count > 1) by[n++] = s;
  std::sort(by, by + n, [](const Span& a, const Span& b) { return a.stride < b.stride; });
  __int128 extent = run;
  for (int i = 0; i < n; ++i) {
    if (by[i].stride < extent) return false;
    extent += static_cast<__int128>(by[i].count - 1) * by[i].stride;
  }
  return true;
}

// The checks of a cache's arguments (api.cpp, api_step.cpp).
int check_paged_cache(const nvfp4kv_paged_cache* cache, bool for_attention);
int check_e4m3_cache(const nvfp4kv_e4m3_cache* cache);

}  // namespace nvfp4kv
