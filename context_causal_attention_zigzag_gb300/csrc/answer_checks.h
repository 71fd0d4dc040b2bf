// Argument checks that the answering and cache calls share.  Host only.
#pragma once

#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "cpattn.h"
#include "cpattn_internal.h"

namespace cpattn {
namespace checks {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// CPATTN_OK, or why these heads and types are not taken.
inline int check_heads(int H, int Hkv, int D, int dtype) {
  if (dtype == CPATTN_F32) return CPATTN_ERR_UNSUPPORTED;
  if (dtype != CPATTN_BF16 && dtype != CPATTN_F16) return CPATTN_ERR_INVALID_ARG;
  if (H < 1 || Hkv < 1 || H % Hkv != 0 || H / Hkv > 128 || H > 65535)
    return CPATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return CPATTN_ERR_INVALID_ARG;
  return CPATTN_OK;
}

// Rows of [heads, D] elements, `stride` apart: 16-byte steps, no overlap.
inline bool check_rows(const void* p, int64_t stride, int heads, int D) {
  return p != nullptr && aligned(p, 16) && stride % 8 == 0 && stride >= (int64_t)heads * D &&
         stride < ((int64_t)1 << 38);
}

inline bool page_size_ok(int P) {
  return P == 16 || P == 32 || P == 64 || (P >= 128 && P <= 1024 && P % 128 == 0);
}

inline bool check_cache(const void* k, const void* v, const CacheShape& c, int D) {
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return false;
  if (!page_size_ok(c.page_size) || c.num_pages < 1 || c.num_pages > INT32_MAX / c.page_size)
    return false;
  for (int64_t s : {c.page_stride, c.token_stride, c.head_stride})
    if (s < D || s % 8 != 0 || s >= ((int64_t)1 << 38)) return false;
  return true;
}

// Rows of a packed tensor, positions of a request in the cache and requests (the
// empty ones are passed one by one): within these an item, and the way to it, take
// less than the kernels' bounded waits allow (2 s), some of which last a whole item.
// A key tile of packed keys takes 1.6 us at 1.9 GHz and 2.1 us at 1.5, where a GPU at
// its power limit was seen: 2^19 of them 1.1 s.  In pages of 16 it takes 2.0 us (items
// of 128 rows behind 131072 positions), 2.5 us at 1.5 GHz: 1.3 s.
constexpr int kMostRows = 1 << 26;
constexpr int kMostPositions = 1 << 26;
constexpr int kMostRequests = 1 << 20;

inline bool scale_ok(float s) { return s <= 0.f || isfinite(s); }

inline int status(cudaError_t e) { return e == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA; }

}  // namespace checks
}  // namespace cpattn
