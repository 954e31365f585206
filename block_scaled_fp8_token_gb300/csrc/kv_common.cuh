// kv_common.cuh -- what the steps around the paged 8-bit KV cache share: the
// page sizes, the checks of a cache description, and the scales' bytes.
//
// A page's keys (or values) of one head hold E4M3 codes with one scale 2^e,
// stored as the byte e + 127. A power of two costs at most one binade of
// E4M3's range and none of its precision, and makes every use of the scale
// exact: quantizing multiplies by 2^-e, a page whose scale grows has its codes
// moved without a second rounding (above E4M3's subnormals), and attention
// folds it into exponents.
#pragma once

#include "attention_layer.h"

namespace bfp8 {

constexpr int kHeadDim = 128;
// Exponents a page's scale takes: values up to 448 * 2^40 are kept, larger ones
// saturate, and a page of zeros has 2^-40.
constexpr int kMinExp = -40, kMaxExp = 40;

inline bool kv_page_size_ok(int32_t page) {
  return page == 16 || page == 32 || page == 64 || page == 128;
}
inline int kv_page_shift(int32_t page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

// Geometry of a cache description (its pointers are checked where they are used).
inline int check_kv_cache(const bfp8_kv_cache& c) {
  if (c.n_pages < 0 || c.n_kv_heads < 1) return BFP8_ERR_INVALID_ARG;
  if (c.n_pages == 0 || !c.k_e4m3 || !c.v_e4m3 || !c.k_exp || !c.v_exp) return BFP8_ERR_INVALID_ARG;
  if (!kv_page_size_ok(c.page_size) || c.head_dim != kHeadDim || c.n_pages > 0x7FFFFFFF ||
      c.n_kv_heads > 65535)
    return BFP8_ERR_UNSUPPORTED;
  const int64_t strides[6] = {c.k_stride_page, c.k_stride_head, c.k_stride_token,
                              c.v_stride_page, c.v_stride_head, c.v_stride_token};
  for (int64_t s : strides) {
    if (s < kHeadDim) return BFP8_ERR_INVALID_ARG;
    if (s % 16) return BFP8_ERR_UNSUPPORTED;
  }
  if (c.exp_stride_page < 1 || c.exp_stride_head < 1) return BFP8_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(c.k_e4m3) % 16 || reinterpret_cast<uintptr_t>(c.v_e4m3) % 16)
    return BFP8_ERR_UNSUPPORTED;
  return BFP8_OK;
}

namespace dev {

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The least e with amax <= 448 * 2^e, in [kMinExp, kMaxExp]: 448 = 1.75 * 2^8,
// so it is amax's own exponent less 8, and one more where its significand is
// above 1.75. amax is a non-negative BF16 value or infinity.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kMinExp), kMaxExp);
}

}  // namespace dev
}  // namespace bfp8
