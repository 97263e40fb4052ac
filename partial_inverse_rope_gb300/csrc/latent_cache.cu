// Writing the paged latent cache and reading it back (include/latent_attn.h).
//
// Both are one pass, bound by memory: a thread holds 16 channels of a token, a
// warp one token of 512 channels, and each thread kRows tokens at a time, whose
// loads are all in flight before the first is used. The 4 threads of a 64-channel
// group find its largest magnitude with two shuffles; codes, scales and pe
// channels leave in the same pass. Vectors go past the cache's lines (streaming
// loads and stores): they are used once.
//
// Measured for rows of 448 + 64 channels: 65536 e4m3 rows are read back in 24.4 us
// (106 MB, 4.35 TB/s; with 8 channels and one token a thread at a time 28.8), of
// which launch and tail are 5; 16384 are written in 8.8 us and read in 9.3 on the
// GPU alone, with the vectors out of DRAM. A few rows take 4-5 us, one round of
// dependent reads (slot, row) and a launch.
//
// Rounding: a code is rounded once, to nearest even, from x * 2^-e, which is exact
// in fp32; what is read back, code * 2^e, is exact in bf16.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.h"
#include "latent.cuh"
#include "ptx.cuh"

namespace invrope {

#ifdef INVROPE_DEBUG_BOUNDS
// The debug-bounds build's fault word of this translation unit (nothing here
// waits); take_latent_fault() reads and clears it with its own.
__device__ unsigned int g_cache_fault = 0;

int take_cache_fault(unsigned int* code) {
  cudaError_t err = cudaMemcpyFromSymbol(code, g_cache_fault, sizeof(*code));
  if (err != cudaSuccess) return cuda_fail(err);
  const unsigned int zero = 0;
  if ((err = cudaMemcpyToSymbol(g_cache_fault, &zero, sizeof(zero))) != cudaSuccess) return cuda_fail(err);
  return INVROPE_OK;
}
#endif

namespace {

using latent::RowLayout;

constexpr int kThreads = 256;
constexpr int kRows = 4;

// The scale's exponent: the least e with amax <= 448 * 2^e, kept to [kEMin, kEMax].
// amax = m * 2^k with 1 <= m < 2 and 448 = 1.75 * 2^8, so e = k - 8, or k - 7
// where m > 1.75; from the bits of amax. amax below 2^-126 (bf16 subnormals)
// has a zero exponent field and ends at kEMin either way.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, latent::kEMin), latent::kEMax);
}

// `shift`: log2 of the threads a token has, a power of two >= ceil(d / 16), at
// least the 4 of a group.
template <bool E4M3>
__global__ void __launch_bounds__(kThreads)
    latent_write_kernel(const char* __restrict__ x, const int32_t* __restrict__ slots, char* __restrict__ cache,
                        int64_t n, int64_t num_slots, RowLayout l, int shift) {
  const int c = 16 * (threadIdx.x & ((1 << shift) - 1));
  const int per = kThreads >> shift;  // tokens a block takes side by side
  const bool one = c < l.d, two = c + 8 < l.d;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * per * kRows + (threadIdx.x >> shift);
       i0 - (threadIdx.x >> shift) < n; i0 += static_cast<int64_t>(gridDim.x) * per * kRows) {
    uint4 v[kRows][2];
    int slot[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t i = i0 + r * per;
      const bool live = i < n;
      const char* row = x + i * (2 * l.d) + 2 * c;
      v[r][0] = live && one ? __ldcs(reinterpret_cast<const uint4*>(row)) : make_uint4(0u, 0u, 0u, 0u);
      v[r][1] = live && two ? __ldcs(reinterpret_cast<const uint4*>(row) + 1) : make_uint4(0u, 0u, 0u, 0u);
      slot[r] = live ? __ldg(slots + i) : -1;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const bool ok = one && slot[r] >= 0 && slot[r] < num_slots;
      char* row = cache + static_cast<int64_t>(ok ? slot[r] : 0) * l.row_bytes;
      LATENT_DBG_CHECK(g_cache_fault, !ok || (slot[r] >= 0 && slot[r] < num_slots && c < l.d), 1);
      if (!E4M3 || c >= l.nope) {
        if (ok) {
          LATENT_DBG_CHECK(g_cache_fault,
                           (E4M3 ? l.nope + 2 * (c - l.nope) : 2 * c) + (two ? 32 : 16) <=
                               (E4M3 ? l.scale_off : l.row_bytes),
                           2);
          uint4* to = reinterpret_cast<uint4*>(E4M3 ? row + l.nope + 2 * (c - l.nope) : row + 2 * c);
          to[0] = v[r][0];
          if (two) to[1] = v[r][1];
        }
      }
      if (!E4M3) continue;
      const uint32_t w[8] = {v[r][0].x, v[r][0].y, v[r][0].z, v[r][0].w, v[r][1].x, v[r][1].y, v[r][1].z, v[r][1].w};
      float amax = 0.f;
      bool finite = true;
      if (c < l.nope) {  // nope is a multiple of 16: all codes or none
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          finite = finite && (w[k] & 0x7F80u) != 0x7F80u && (w[k] & 0x7F800000u) != 0x7F800000u;
          amax = fmaxf(amax, fmaxf(fabsf(ptx::bf16_lo_f32(w[k])), fabsf(ptx::bf16_hi_f32(w[k]))));
        }
        if (!finite) amax = __uint_as_float(0x7F800000u);
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      if (!ok || c >= l.nope) continue;
      LATENT_DBG_CHECK(g_cache_fault, c + 16 <= l.nope && l.scale_off + c / latent::kGroup < l.row_bytes, 3);
      const bool bad = __float_as_uint(amax) == 0x7F800000u;
      const int e = bad ? 0 : scale_exponent(amax);
      const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e
      uint32_t code[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        code[k] = bad ? 0u
                      : __nv_cvt_float2_to_fp8x2(
                            make_float2(ptx::bf16_lo_f32(w[k]) * inv, ptx::bf16_hi_f32(w[k]) * inv), __NV_SATFINITE,
                            __NV_E4M3);
      *reinterpret_cast<uint4*>(row + c) = make_uint4(code[0] | code[1] << 16, code[2] | code[3] << 16,
                                                      code[4] | code[5] << 16, code[6] | code[7] << 16);
      if (c % latent::kGroup == 0)
        reinterpret_cast<unsigned char*>(row)[l.scale_off + c / latent::kGroup] =
            static_cast<unsigned char>(bad ? 255 : e + 127);
    }
  }
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads)
    latent_read_kernel(const char* __restrict__ cache, const int32_t* __restrict__ slots, char* __restrict__ out,
                       int64_t n, int64_t num_slots, RowLayout l, int shift) {
  const int c = 16 * (threadIdx.x & ((1 << shift) - 1));
  const int per = kThreads >> shift;
  const bool one = c < l.d, two = c + 8 < l.d, codes = E4M3 && c < l.nope;
  const int at = !E4M3 ? 2 * c : codes ? c : l.nope + 2 * (c - l.nope);
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * per * kRows + (threadIdx.x >> shift); i0 < n;
       i0 += static_cast<int64_t>(gridDim.x) * per * kRows) {
    int slot[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) slot[r] = i0 + r * per < n ? __ldg(slots + i0 + r * per) : -1;
    uint4 v[kRows][2];
    uint32_t byte[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const bool ok = one && slot[r] >= 0 && slot[r] < num_slots;
      const char* row = cache + static_cast<int64_t>(ok ? slot[r] : 0) * l.row_bytes;
      LATENT_DBG_CHECK(g_cache_fault,
                       !ok || (slot[r] < num_slots && at + (codes || !two ? 16 : 32) <= l.row_bytes), 4);
      v[r][0] = ok ? __ldg(reinterpret_cast<const uint4*>(row + at)) : make_uint4(0u, 0u, 0u, 0u);
      v[r][1] = ok && two && !codes ? __ldg(reinterpret_cast<const uint4*>(row + at) + 1) : make_uint4(0u, 0u, 0u, 0u);
      byte[r] = ok && codes
                    ? __ldg(reinterpret_cast<const unsigned char*>(row) + l.scale_off + c / latent::kGroup)
                    : 127u;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t i = i0 + r * per;
      if (codes) {
        const uint32_t s = latent::scale_bf16x2(byte[r]);
        const uint4 w = v[r][0];
        latent::e4m3x4_to_bf16(w.x, s, v[r][0].x, v[r][0].y);
        latent::e4m3x4_to_bf16(w.y, s, v[r][0].z, v[r][0].w);
        latent::e4m3x4_to_bf16(w.z, s, v[r][1].x, v[r][1].y);
        latent::e4m3x4_to_bf16(w.w, s, v[r][1].z, v[r][1].w);
      }
      uint4* to = reinterpret_cast<uint4*>(out + i * (2 * l.d) + 2 * c);
      if (one && i < n) __stcs(to, v[r][0]);
      if (two && i < n) __stcs(to + 1, v[r][1]);
    }
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

// log2 of the threads a token has.
int threads_shift(const RowLayout& l) {
  int shift = 2;
  while ((16 << shift) < l.d) ++shift;
  return shift;
}

unsigned grid_for(int64_t n, int shift, const DeviceInfo& dev) {
  const int64_t each = static_cast<int64_t>(kThreads >> shift) * kRows;
  const int64_t blocks = (n + each - 1) / each, most = static_cast<int64_t>(dev.sms) * 8;
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
  const int shift = threads_shift(l);
  const unsigned grid = grid_for(n, shift, dev);
  if (fmt == KV_LATENT_E4M3)
    latent_write_kernel<true><<<grid, kThreads, 0, s>>>(static_cast<const char*>(x), slots, static_cast<char*>(cache),
                                                        n, num_slots, l, shift);
  else
    latent_write_kernel<false><<<grid, kThreads, 0, s>>>(static_cast<const char*>(x), slots,
                                                         static_cast<char*>(cache), n, num_slots, l, shift);
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
  const int shift = threads_shift(l);
  const unsigned grid = grid_for(n, shift, dev);
  if (fmt == KV_LATENT_E4M3)
    latent_read_kernel<true><<<grid, kThreads, 0, s>>>(static_cast<const char*>(cache), slots,
                                                       static_cast<char*>(out), n, num_slots, l, shift);
  else
    latent_read_kernel<false><<<grid, kThreads, 0, s>>>(static_cast<const char*>(cache), slots,
                                                        static_cast<char*>(out), n, num_slots, l, shift);
  return check_launch();
}
