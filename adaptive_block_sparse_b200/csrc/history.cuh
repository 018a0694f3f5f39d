// Shared pieces of the operators on a paged history (rotary positions, cache append,
// prefix attention): device status codes, host checks and the 16-bit element types.
#pragma once

#include "common.cuh"
#include "device_status.h"

namespace nabla {

// Device status codes of these operators.  Append: first error wins, as for every other call;
// prefix attention: the largest rank of device_status.h is reported.
enum : uint32_t {
  kDevBadPage = 0x301,     // a page number outside the cache: that page was not touched
  kDevBadLength = 0x302,   // a negative length, or one beyond the page table or the call's tokens
};

// Host checks shared by the entry points.
inline bool is_16bit(int32_t dtype) { return dtype == NABLA_BF16 || dtype == NABLA_F16; }
inline bool known_dtype(int32_t dtype) { return is_16bit(dtype) || dtype == NABLA_F32; }
inline int element_bytes(int32_t dtype) { return dtype == NABLA_F32 ? 4 : 2; }

// Geometry of a paged cache [n_pages, H, page, D].
inline nabla_status check_cache(const nabla_cache& c) {
  if (c.n_pages < 1 || c.H < 1 || c.page < 1 || c.D < 1) return NABLA_ERR_INVALID_ARG;
  if (c.D != 64 && c.D != 128) return NABLA_ERR_UNSUPPORTED;
  if (c.page < 16 || c.page > 4096 || (c.page & (c.page - 1))) return NABLA_ERR_UNSUPPORTED;
  if (!is_16bit(c.dtype)) return NABLA_ERR_INVALID_ARG;
  if (!c.k || !c.v || !aligned16(c.k) || !aligned16(c.v)) return NABLA_ERR_INVALID_ARG;
  return NABLA_OK;
}

// A strided [B, H, S, D] view: 16-byte aligned rows, no negative stride.  `out`: every
// element has an address of its own as far as single strides tell.
inline nabla_status check_heads(const nabla_heads& x, int32_t B, int64_t S, bool out) {
  if (!x.ptr || !aligned16(x.ptr) || x.H < 1 || !known_dtype(x.dtype)) return NABLA_ERR_INVALID_ARG;
  const int64_t st[3] = {x.stride_b, x.stride_h, x.stride_s};
  const int64_t n[3] = {B, x.H, S};
  const int64_t unit = 16 / element_bytes(x.dtype);
  for (int i = 0; i < 3; ++i) {
    if (st[i] < 0 || (n[i] > 1 && st[i] % unit)) return NABLA_ERR_INVALID_ARG;
    if (out && n[i] > 1 && st[i] == 0) return NABLA_ERR_INVALID_ARG;
  }
  return NABLA_OK;
}

// One past the last byte of the view.
inline const char* heads_end(const nabla_heads& x, int32_t B, int64_t S, int D) {
  const int64_t last = (B - 1) * x.stride_b + (x.H - 1) * x.stride_h + (S - 1) * x.stride_s + D;
  return static_cast<const char*>(x.ptr) + last * element_bytes(x.dtype);
}
inline bool heads_overlap(const nabla_heads& a, const nabla_heads& b, int32_t B, int64_t S, int D) {
  return static_cast<const char*>(a.ptr) < heads_end(b, B, S, D) &&
         static_cast<const char*>(b.ptr) < heads_end(a, B, S, D);
}

}  // namespace nabla
