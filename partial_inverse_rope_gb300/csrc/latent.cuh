// Row layout of the latent cache (include/latent_attn.h) and the conversion of
// e4m3 codes with power-of-two scales to bf16, shared by the cache's and the
// attention's kernels.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>

#include "latent_attn.h"

// Debug-bounds builds (build.py --debug-bounds) check on the device that indices
// stay in bounds, and record 0xDB40 | id in the translation unit's fault word
// where one does not, without trapping.
#ifdef INVROPE_DEBUG_BOUNDS
#define LATENT_DBG_CHECK(word, cond, id)                      \
  do {                                                        \
    if (!(cond)) atomicCAS(&(word), 0u, 0xDB40u | (id));      \
  } while (0)
#else
#define LATENT_DBG_CHECK(word, cond, id) \
  do {                                   \
  } while (0)
#endif

namespace invrope {
namespace latent {

constexpr int kGroup = 64;   // channels that share a scale
constexpr int kMaxD = 512;
constexpr int kEMin = -120;  // smallest scale: 2^-120 * 2^-9 (least e4m3 step) is still exact in bf16
constexpr int kEMax = 119;   // largest: 448 * 2^119 is bf16's range, 448 * 2^120 is not

struct RowLayout {
  int nope, pe, d;
  int row_bytes;
  int scale_off;  // byte offset of the scales (e4m3 rows)
};

// Returns INVROPE_OK and fills *l, or an error status.
inline int row_layout(int nope, int pe, int fmt, RowLayout* l) {
  if (fmt != KV_LATENT_BF16 && fmt != KV_LATENT_E4M3) return INVROPE_ERR_INVALID_ARG;
  if (nope < 0 || pe < 0 || nope > (1 << 20) || pe > (1 << 20)) return INVROPE_ERR_INVALID_ARG;
  const int d = nope + pe;
  if (d < 8 || d % 8) return INVROPE_ERR_INVALID_ARG;
  if (fmt == KV_LATENT_E4M3 && (nope < 16 || nope % 16 || pe % 8)) return INVROPE_ERR_INVALID_ARG;
  if (d > kMaxD) return INVROPE_ERR_UNSUPPORTED;
  l->nope = nope;
  l->pe = pe;
  l->d = d;
  l->scale_off = nope + 2 * pe;
  l->row_bytes = fmt == KV_LATENT_BF16 ? 2 * d : (l->scale_off + (nope + kGroup - 1) / kGroup + 15) / 16 * 16;
  return INVROPE_OK;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A scale byte as two equal bf16 values 2^(byte-127); 255 gives NaN. The byte is
// bf16's exponent field, but for 0: 2^-127 is a subnormal. (The writer keeps it
// within 7..246, or 255; rows from elsewhere may hold any.)
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t byte) {
  const uint32_t h = byte == 255u ? 0x7FC0u : byte == 0u ? 0x0040u : byte << 7;
  return h | (h << 16);
}

// Four e4m3 codes -> four bf16 values. A code's exponent and mantissa bits,
// moved into bf16's fields, read as value * 2^-120 (e4m3's bias is 7, bf16's
// 127; e4m3 subnormals become bf16 subnormals); the product with `factor`, a
// power of two twice, is exact. Two codes are put in bytes 1 and 3, with byte 2
// the copies of the first one's sign: one arithmetic shift by 4 then brings
// both signs and fields to where bf16 has them, and one mask leaves just those.
// The codes 0x7F and 0xFF come out as 480 and -480, as the format says: a test for
// them, 10 instructions for 16 codes, takes 5% of the attention's time (96 rows of
// 4000 to 20000 tokens: 287 us against 274).
__device__ __forceinline__ uint32_t prmt_signs(uint32_t w, uint32_t selector) {  // 8 + n: byte n's sign, 8 times
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "r"(selector));
  return r;
}
__device__ __forceinline__ void e4m3x4_times(uint32_t w, uint32_t factor, uint32_t& lo, uint32_t& hi) {
  const int a = static_cast<int>(prmt_signs(w, 0x1800u)), b = static_cast<int>(prmt_signs(w, 0x3A22u));
  lo = mul_bf16x2(static_cast<uint32_t>(a >> 4) & 0x87F087F0u, factor);
  hi = mul_bf16x2(static_cast<uint32_t>(b >> 4) & 0x87F087F0u, factor);
}

// The same times the group's scale: 2^120 and the scale, which together may
// have no bf16 value, one after the other.
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t w, uint32_t scale2, uint32_t& lo, uint32_t& hi) {
  e4m3x4_times(w, 0x7B807B80u, lo, hi);
  lo = mul_bf16x2(lo, scale2);
  hi = mul_bf16x2(hi, scale2);
}

}  // namespace latent
}  // namespace invrope
