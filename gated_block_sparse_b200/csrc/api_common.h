// Argument checks and error reporting shared by the C ABI's source files.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/sas.h"

namespace sas {

void clear_error();
// Records the message of the calling thread's last error; returns s.
sas_status fail(sas_status s, const char* fmt, ...);
sas_status cuda_status(cudaError_t e, const char* where);
sas_status check_common(sas_dtype dt, int B, int Hq, int Hkv, int N, int d, int topk);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline float resolve_scale(float scale, int d) {
  return scale > 0.f ? scale : 1.0f / sqrtf((float)d);
}
inline size_t a16(size_t x) { return (x + 15) & ~(size_t)15; }

}  // namespace sas

#define REQUIRE(cond, st, ...) \
  do {                         \
    if (!(cond)) return sas::fail(st, __VA_ARGS__); \
  } while (0)

#define REQUIRE_PTR(p)                                                                     \
  do {                                                                                     \
    if ((p) == nullptr) return sas::fail(SAS_ERR_INVALID_ARG, "%s must not be NULL", #p);  \
    if (!sas::aligned16(p))                                                                \
      return sas::fail(SAS_ERR_INVALID_ARG, "%s must be 16-byte aligned", #p);             \
  } while (0)
