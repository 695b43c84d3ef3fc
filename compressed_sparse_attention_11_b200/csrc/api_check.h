// Argument checks of the C ABI layer: each macro returns from the entry point
// with a status and a one-line reason (csa_last_error) before anything is
// launched.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace csa {

inline csa_status api_ok() { return set_last_error(CSA_OK, "%s", ""); }
inline csa_status api_cuda(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return api_ok();
  return set_last_error(CSA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}
inline bool api_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool api_valid_dt(csa_dtype dt) { return dt == CSA_F32 || dt == CSA_BF16; }
inline size_t api_elt(csa_dtype dt) { return dt == CSA_F32 ? 4 : 2; }
// Whether [a, a + na) and [b, b + nb) share a byte.
inline bool api_overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

}  // namespace csa

#define API_REQUIRE(cond, ...) \
  do { if (!(cond)) return csa::set_last_error(CSA_ERR_INVALID_ARG, __VA_ARGS__); } while (0)
#define API_REQUIRE_PTR(p) \
  do { \
    API_REQUIRE((p) != nullptr, "%s is NULL", #p); \
    API_REQUIRE(csa::api_aligned16(p), "%s is not 16-byte aligned", #p); \
  } while (0)
#define API_REQUIRE_OPT_PTR(p) \
  API_REQUIRE((p) == nullptr || csa::api_aligned16(p), "%s is not 16-byte aligned", #p)
// Lists and scalars that the kernels read one element at a time.
#define API_REQUIRE_LIST(p) \
  do { \
    API_REQUIRE((p) != nullptr, "%s is NULL", #p); \
    API_REQUIRE(reinterpret_cast<uintptr_t>(p) % sizeof(*(p)) == 0, "%s is misaligned", #p); \
  } while (0)
#define API_REQUIRE_OPT_LIST(p) \
  API_REQUIRE((p) == nullptr || reinterpret_cast<uintptr_t>(p) % sizeof(*(p)) == 0, \
              "%s is misaligned", #p)
#define API_SUPPORTED(cond, ...) \
  do { if (!(cond)) return csa::set_last_error(CSA_ERR_UNSUPPORTED, __VA_ARGS__); } while (0)
