// Argument checks that the C-ABI files of the operators share.
#pragma once

#include <math.h>

#include "layer_internal.h"

namespace dion3 {
namespace {

#define HIP_TRY(expr)                                    \
  do {                                                   \
    const hipError_t _e = (expr);                        \
    if (_e != hipSuccess) return note_hip_error(_e);     \
  } while (0)

// Row strides up to this keep every tile's 32-bit byte offsets below 2^31
// (256 rows of 2^21 16-bit elements).
constexpr long long kMaxLd = 1LL << 21;

bool type16(int t) { return t == DION3_BF16 || t == DION3_F16; }

// Sizes: a negative token count or a side below 1 is an argument error, a
// valid size past the limits unsupported.
dion3_status check_sizes(long long T, long long a, long long b) {
  if (T < 0 || a < 1 || b < 1) return DION3_ERR_ARG;
  if (T > DION3_MAX_TOKENS || a > DION3_MAX_DIM || b > DION3_MAX_DIM) return DION3_ERR_UNSUPPORTED;
  // a launch's side holds fewer than 2^32 threads, which 2^22 of the tiles that
  // outputs of this size take (256 x 256) stay below
  constexpr long long most = 1LL << 38;
  if (T * a > most || T * b > most || a * b > most) return DION3_ERR_UNSUPPORTED;
  return DION3_OK;
}

dion3_status check_ld(long long ld, long long cols) {
  if (ld < cols) return DION3_ERR_ARG;
  return ld > kMaxLd ? DION3_ERR_UNSUPPORTED : DION3_OK;
}

// Rows that are addressed in 64 bits.
dion3_status check_far_ld(long long ld, long long cols) {
  if (ld < cols) return DION3_ERR_ARG;
  return ld > 1LL << 38 ? DION3_ERR_UNSUPPORTED : DION3_OK;
}

// 16-bit (and fp32) elements must be aligned to their own size.
bool elem_aligned(const void* p, int size) { return ((uintptr_t)p & (size - 1)) == 0; }

dion3_status check_scratch(const void* ws, size_t have, size_t need) {
  if (need == 0) return DION3_OK;
  if (!ws || ((uintptr_t)ws & 255) != 0 || have < need) return DION3_ERR_WORKSPACE;
  return DION3_OK;
}

#define TRY(expr)                                \
  do {                                           \
    const dion3_status _s = (expr);              \
    if (_s != DION3_OK) return _s;               \
  } while (0)

}  // namespace
}  // namespace dion3
