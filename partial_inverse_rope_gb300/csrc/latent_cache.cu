// Writing the paged latent cache and reading it back (include/latent_attn.h).
//
// Both are one pass: a thread holds 8 channels of one token (16 bytes of bf16),
// so the 8 threads of a 64-channel group sit in one warp and find the group's
// largest magnitude with three shuffles; codes, scales and pe channels leave
// in the same pass.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.h"
#include "latent.cuh"
#include "ptx.cuh"

namespace invrope {
namespace {

using latent::RowLayout;

constexpr int kThreads = 256;

// The scale's exponent: the least e with amax <= 448 * 2^e, kept to [kEMin, kEMax].
// amax = m * 2^k with 1 <= m < 2 and 448 = 1.75 * 2^8, so e = k - 8, or k - 7
// where m > 1.75; from the bits of amax. amax below 2^-126 (bf16 subnormals)
// has a zero exponent field and ends at kEMin either way.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, latent::kEMin), latent::kEMax);
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads)
    latent_write_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ slots, char* __restrict__ cache,
                        int64_t n, int64_t num_slots, RowLayout l) {
  const int units = l.d / 8;                 // 16-byte units of a token
  const int padded = (units + 7) / 8 * 8;    // whole groups of 8 threads
  const int64_t total = n * padded;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads; base < total; base += step) {
    const int64_t g = base + threadIdx.x;
    const int64_t i = g / padded;
    const int u = static_cast<int>(g - i * padded);
    const bool live = g < total && u < units;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    int64_t slot = -1;
    if (live) {
      v = __ldcs(x + i * units + u);
      slot = slots[i];
    }
    const bool ok = live && slot >= 0 && slot < num_slots;
    char* row = cache + (ok ? slot : 0) * static_cast<int64_t>(l.row_bytes);
    if (!E4M3) {
      if (ok) *reinterpret_cast<uint4*>(row + u * 16) = v;
      continue;
    }
    const int c = u * 8;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8], amax = 0.f;
    bool finite = true;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = ptx::bf16_lo_f32(w[k]);
      f[2 * k + 1] = ptx::bf16_hi_f32(w[k]);
      finite = finite && (w[k] & 0x7F80u) != 0x7F80u && (w[k] & 0x7F800000u) != 0x7F800000u;
      amax = fmaxf(amax, fmaxf(fabsf(f[2 * k]), fabsf(f[2 * k + 1])));
    }
    if (!live || c >= l.nope) {  // a pe unit beside the last group's codes
      amax = 0.f;
      finite = true;
    }
    if (!finite) amax = __uint_as_float(0x7F800000u);
#pragma unroll
    for (int s = 1; s < 8; s *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, s));
    if (!ok) continue;
    if (c >= l.nope) {
      *reinterpret_cast<uint4*>(row + l.nope + 2 * (c - l.nope)) = v;
      continue;
    }
    const bool bad = __float_as_uint(amax) == 0x7F800000u;
    const int e = bad ? 0 : scale_exponent(amax);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e
    uint32_t code[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      code[k] = bad ? 0u
                    : __nv_cvt_float2_to_fp8x2(make_float2(f[2 * k] * inv, f[2 * k + 1] * inv), __NV_SATFINITE,
                                               __NV_E4M3);
    *reinterpret_cast<uint2*>(row + c) = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
    if (c % latent::kGroup == 0)
      reinterpret_cast<unsigned char*>(row)[l.scale_off + c / latent::kGroup] =
          static_cast<unsigned char>(bad ? 255 : e + 127);
  }
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads)
    latent_read_kernel(const char* __restrict__ cache, const int32_t* __restrict__ slots, uint4* __restrict__ out,
                       int64_t n, int64_t num_slots, RowLayout l) {
  const int units = l.d / 8;
  const int64_t total = n * units;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; g < total; g += step) {
    const int64_t i = g / units;
    const int u = static_cast<int>(g - i * units);
    const int64_t slot = slots[i];
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= 0 && slot < num_slots) {
      const char* row = cache + slot * static_cast<int64_t>(l.row_bytes);
      const int c = u * 8;
      if (!E4M3) {
        v = __ldg(reinterpret_cast<const uint4*>(row + u * 16));
      } else if (c >= l.nope) {
        v = __ldg(reinterpret_cast<const uint4*>(row + l.nope + 2 * (c - l.nope)));
      } else {
        const uint2 codes = __ldg(reinterpret_cast<const uint2*>(row + c));
        const uint32_t s =
            latent::scale_bf16x2(__ldg(reinterpret_cast<const unsigned char*>(row) + l.scale_off + c / latent::kGroup));
        latent::e4m3x4_to_bf16(codes.x, s, v.x, v.y);
        latent::e4m3x4_to_bf16(codes.y, s, v.z, v.w);
      }
    }
    __stcs(out + g, v);
  }
}

// Checks common to both calls; *skip is set when there is nothing to do.
int check_rows(const void* vectors, const int32_t* slots, const void* cache, int64_t n, int64_t num_slots, int nope,
               int pe, int fmt, RowLayout* l, bool* skip) {
  const int st = latent::row_layout(nope, pe, fmt, l);
  if (st != INVROPE_OK) return st;
  if (n < 0 || num_slots < 1) return INVROPE_ERR_INVALID_ARG;
  if (num_slots > 0x7FFFFFFF || n > 0x7FFFFFFF) return INVROPE_ERR_UNSUPPORTED;
  *skip = n == 0;
  if (*skip) return INVROPE_OK;
  if (!vectors || !slots || !cache || !aligned(vectors, 16) || !aligned(cache, 16) || !aligned(slots, 4))
    return INVROPE_ERR_INVALID_ARG;
  return INVROPE_OK;
}

unsigned grid_for(int64_t threads, const DeviceInfo& dev) {
  const int64_t blocks = (threads + kThreads - 1) / kThreads, most = static_cast<int64_t>(dev.sms) * 8;
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

}  // namespace
}  // namespace invrope

using namespace invrope;

extern "C" size_t kv_latent_row_bytes(int nope, int pe, int fmt) {
  RowLayout l;
  return latent::row_layout(nope, pe, fmt, &l) == INVROPE_OK ? static_cast<size_t>(l.row_bytes) : 0;
}

extern "C" int kv_latent_write(const void* x, const int32_t* slots, void* cache, int64_t n, int64_t num_slots,
                               int nope, int pe, int fmt, struct CUstream_st* stream) {
  RowLayout l;
  bool skip = false;
  int st = check_rows(x, slots, cache, n, num_slots, nope, pe, fmt, &l, &skip);
  if (st != INVROPE_OK || skip) return st;
  const size_t cache_bytes = static_cast<size_t>(num_slots) * l.row_bytes;
  if (overlaps(cache, cache_bytes, x, static_cast<size_t>(n) * l.d * 2) ||
      overlaps(cache, cache_bytes, slots, static_cast<size_t>(n) * 4))
    return INVROPE_ERR_INVALID_ARG;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != INVROPE_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = grid_for(n * ((l.d / 8 + 7) / 8 * 8), dev);
  if (fmt == KV_LATENT_E4M3)
    latent_write_kernel<true><<<grid, kThreads, 0, s>>>(static_cast<const uint4*>(x), slots, static_cast<char*>(cache),
                                                        n, num_slots, l);
  else
    latent_write_kernel<false><<<grid, kThreads, 0, s>>>(static_cast<const uint4*>(x), slots,
                                                         static_cast<char*>(cache), n, num_slots, l);
  return check_launch();
}

extern "C" int kv_latent_read(const void* cache, const int32_t* slots, void* out, int64_t n, int64_t num_slots,
                              int nope, int pe, int fmt, struct CUstream_st* stream) {
  RowLayout l;
  bool skip = false;
  int st = check_rows(out, slots, cache, n, num_slots, nope, pe, fmt, &l, &skip);
  if (st != INVROPE_OK || skip) return st;
  const size_t out_bytes = static_cast<size_t>(n) * l.d * 2;
  if (overlaps(out, out_bytes, cache, static_cast<size_t>(num_slots) * l.row_bytes) ||
      overlaps(out, out_bytes, slots, static_cast<size_t>(n) * 4))
    return INVROPE_ERR_INVALID_ARG;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != INVROPE_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = grid_for(n * (l.d / 8), dev);
  if (fmt == KV_LATENT_E4M3)
    latent_read_kernel<true><<<grid, kThreads, 0, s>>>(static_cast<const char*>(cache), slots,
                                                       static_cast<uint4*>(out), n, num_slots, l);
  else
    latent_read_kernel<false><<<grid, kThreads, 0, s>>>(static_cast<const char*>(cache), slots,
                                                        static_cast<uint4*>(out), n, num_slots, l);
  return check_launch();
}
