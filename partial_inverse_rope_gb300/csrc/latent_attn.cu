// Attention over the latent cache (include/latent_attn.h): keys and values are
// the same rows, addressed through pages or through an index table.
//
// One thread block per (row, head): 128 tokens at a time, a thread scores one
// token, then owns channels tid, tid + 128, ... of the output. Running maximum
// and sum in fp32. No reuse of a row between heads: bound by L2 reads.
#include <cuda_runtime.h>

#include <cmath>

#include "common.h"
#include "latent.cuh"
#include "ptx.cuh"

namespace invrope {
namespace {

using latent::RowLayout;

struct AttnParams {
  const __nv_bfloat16* q;
  const char* cache;
  const int32_t* table;  // page table [rows, width] or index table [rows, width]
  const int32_t* lens;   // NULL: an index table
  __nv_bfloat16* O;
  float* lse;
  int64_t rows, width, num_slots, num_pages;
  int nh, page_size;
  float scale_log2;  // scale * log2(e)
  RowLayout l;
};

__device__ __forceinline__ int64_t tokens_of(const AttnParams& p, int64_t r) {
  if (!p.lens) return p.width;
  const int64_t n = p.lens[r], most = p.width * p.page_size;
  return n < 0 ? 0 : n < most ? n : most;
}

// The cache slot of token t of row r, or -1 when it is left out.
__device__ __forceinline__ int slot_of(const AttnParams& p, int64_t r, int64_t t) {
  if (!p.lens) {
    const int s = p.table[r * p.width + t];
    return s >= 0 && s < p.num_slots ? s : -1;
  }
  const int64_t pg = t / p.page_size;
  const int g = p.table[r * p.width + pg];
  return g >= 0 && g < p.num_pages ? g * p.page_size + static_cast<int>(t - pg * p.page_size) : -1;
}

// 8 channels from c on of a cache row, as bf16.
template <bool E4M3>
__device__ __forceinline__ uint4 load_unit(const char* row, int c, const RowLayout& l) {
  if (!E4M3) return __ldg(reinterpret_cast<const uint4*>(row + 2 * c));
  if (c >= l.nope) return __ldg(reinterpret_cast<const uint4*>(row + l.nope + 2 * (c - l.nope)));
  const uint2 codes = __ldg(reinterpret_cast<const uint2*>(row + c));
  const uint32_t s =
      latent::scale_bf16x2(__ldg(reinterpret_cast<const unsigned char*>(row) + l.scale_off + c / latent::kGroup));
  uint4 v;
  latent::e4m3x4_to_bf16(codes.x, s, v.x, v.y);
  latent::e4m3x4_to_bf16(codes.y, s, v.z, v.w);
  return v;
}

constexpr int kThreads = 128;

template <bool E4M3>
__global__ void __launch_bounds__(kThreads) latent_attn_kernel(AttnParams p) {
  __shared__ float sq[latent::kMaxD];
  __shared__ float sp[kThreads];
  __shared__ int ss[kThreads];
  __shared__ float red[4];
  __shared__ uint4 tile[kThreads];
  const int64_t r = blockIdx.x / p.nh;
  const int h = static_cast<int>(blockIdx.x - r * p.nh);
  const int d = p.l.d, tid = threadIdx.x;
  const __nv_bfloat16* q = p.q + (r * p.nh + h) * d;
  for (int c = tid; c < d; c += kThreads) sq[c] = __bfloat162float(q[c]);
  const int64_t n = tokens_of(p, r);
  float m = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  for (int64_t t0 = 0; t0 < n; t0 += kThreads) {
    const int slot = t0 + tid < n ? slot_of(p, r, t0 + tid) : -1;
    float s = -INFINITY;
    if (slot >= 0) {
      const char* row = p.cache + slot * static_cast<int64_t>(p.l.row_bytes);
      float dot = 0.f;
      for (int c = 0; c < d; c += 8) {
        const uint4 v = load_unit<E4M3>(row, c, p.l);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          dot += sq[c + 2 * k] * ptx::bf16_lo_f32(w[k]) + sq[c + 2 * k + 1] * ptx::bf16_hi_f32(w[k]);
      }
      s = dot * p.scale_log2;
    }
    float top = s;
    for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if ((tid & 31) == 0) red[tid / 32] = top;
    __syncthreads();
    top = fmaxf(fmaxf(m, fmaxf(red[0], red[1])), fmaxf(red[2], red[3]));
    const float ref = top == -INFINITY ? 0.f : top;  // nothing so far: every weight is 0
    const float keep = exp2f(m - ref);
    sp[tid] = exp2f(s - ref);
    ss[tid] = slot;
    m = top;
    sum *= keep;
    for (int k = 0; k < 4; ++k) acc[k] *= keep;
    __syncthreads();
    const int here = static_cast<int>(n - t0 < kThreads ? n - t0 : kThreads);
    for (int t = 0; t < here; ++t) {
      if (ss[t] < 0) continue;
      const char* row = p.cache + ss[t] * static_cast<int64_t>(p.l.row_bytes);
      if (tid < d / 8) tile[tid] = load_unit<E4M3>(row, tid * 8, p.l);
      __syncthreads();
      sum += sp[t];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (tid + k * kThreads < d)
          acc[k] += sp[t] * __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(tile)[tid + k * kThreads]);
      __syncthreads();
    }
  }
  __nv_bfloat16* o = p.O + (r * p.nh + h) * d;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (tid + k * kThreads < d) o[tid + k * kThreads] = __float2bfloat16_rn(sum == 0.f ? 0.f : acc[k] / sum);
  if (p.lse && tid == 0) p.lse[r * p.nh + h] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
}

// Checks common to both calls; *skip is set when there is nothing to do.
int check_attn(const AttnParams& p, const void* workspace, size_t workspace_bytes, size_t need, int fmt, double scale,
               bool* skip) {
  *skip = p.rows == 0;
  if (*skip) return INVROPE_OK;
  if (!p.q || !p.cache || !p.O || !aligned(p.q, 16) || !aligned(p.cache, 16) || !aligned(p.O, 16))
    return INVROPE_ERR_INVALID_ARG;
  if ((p.width > 0 && !p.table) || !aligned(p.table, 4) || !aligned(p.lens, 4) || !aligned(p.lse, 4))
    return INVROPE_ERR_INVALID_ARG;
  const size_t heads = static_cast<size_t>(p.rows) * p.nh, vec = heads * p.l.d * 2;
  const struct {
    const void* at;
    size_t bytes;
  } in[] = {{p.q, vec},
            {p.cache, static_cast<size_t>(p.num_slots) * p.l.row_bytes},
            {p.table, static_cast<size_t>(p.rows) * p.width * 4},
            {p.lens, p.lens ? static_cast<size_t>(p.rows) * 4 : 0}},
    out[] = {{p.O, vec}, {p.lse, p.lse ? heads * 4 : 0}, {workspace, workspace ? need : 0}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& x : in)
      if (overlaps(out[i].at, out[i].bytes, x.at, x.bytes)) return INVROPE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i].at, out[i].bytes, out[j].at, out[j].bytes)) return INVROPE_ERR_INVALID_ARG;
  }
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return INVROPE_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return INVROPE_ERR_INVALID_ARG;
  }
  (void)fmt;
  (void)scale;
  return INVROPE_OK;
}

int shape_status(int64_t rows, int nh, double scale) {
  if (rows < 0 || nh < 1 || !std::isfinite(scale)) return INVROPE_ERR_INVALID_ARG;
  if (nh > 128 || rows > 0x7FFFFFFF / nh) return INVROPE_ERR_UNSUPPORTED;
  return INVROPE_OK;
}

int launch(const AttnParams& p, int fmt, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(p.rows * p.nh);
  if (fmt == KV_LATENT_E4M3)
    latent_attn_kernel<true><<<grid, kThreads, 0, s>>>(p);
  else
    latent_attn_kernel<false><<<grid, kThreads, 0, s>>>(p);
  return check_launch();
}

}  // namespace
}  // namespace invrope

using namespace invrope;

extern "C" size_t latent_attn_workspace_bytes(int64_t rows, int nh, int64_t max_tokens, int nope, int pe) {
  (void)rows, (void)nh, (void)max_tokens, (void)nope, (void)pe;
  return 0;
}

extern "C" int latent_attn_decode(const void* q, const void* cache, const int32_t* page_table, const int32_t* lens,
                                  void* O, float* lse, void* workspace, size_t workspace_bytes, int64_t rows, int nh,
                                  int nope, int pe, int fmt, int64_t num_pages, int page_size, int64_t max_pages,
                                  double scale, struct CUstream_st* stream) {
  AttnParams p = {};
  int st = latent::row_layout(nope, pe, fmt, &p.l);
  if (st != INVROPE_OK) return st;
  if ((st = shape_status(rows, nh, scale)) != INVROPE_OK) return st;
  if (num_pages < 1 || page_size < 1 || max_pages < 0) return INVROPE_ERR_INVALID_ARG;
  if (num_pages > 0x7FFFFFFF / page_size || max_pages > 0x7FFFFFFF / page_size) return INVROPE_ERR_UNSUPPORTED;
  if (rows > 0 && !lens) return INVROPE_ERR_INVALID_ARG;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cache = static_cast<const char*>(cache);
  p.table = page_table;
  p.lens = lens;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  p.rows = rows;
  p.width = max_pages;
  p.num_slots = num_pages * page_size;
  p.num_pages = num_pages;
  p.nh = nh;
  p.page_size = page_size;
  p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  bool skip = false;
  const size_t need = latent_attn_workspace_bytes(rows, nh, max_pages * page_size, nope, pe);
  if ((st = check_attn(p, workspace, workspace_bytes, need, fmt, scale, &skip)) != INVROPE_OK || skip) return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != INVROPE_OK) return st;
  return launch(p, fmt, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int latent_attn_sparse(const void* q, const void* cache, const int32_t* idx, void* O, float* lse,
                                  void* workspace, size_t workspace_bytes, int64_t rows, int nh, int nope, int pe,
                                  int fmt, int64_t num_slots, int64_t topk, double scale, struct CUstream_st* stream) {
  AttnParams p = {};
  int st = latent::row_layout(nope, pe, fmt, &p.l);
  if (st != INVROPE_OK) return st;
  if ((st = shape_status(rows, nh, scale)) != INVROPE_OK) return st;
  if (num_slots < 1 || topk < 0) return INVROPE_ERR_INVALID_ARG;
  if (num_slots > 0x7FFFFFFF || topk > 0x7FFFFFFF) return INVROPE_ERR_UNSUPPORTED;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cache = static_cast<const char*>(cache);
  p.table = idx;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  p.rows = rows;
  p.width = topk;
  p.num_slots = num_slots;
  p.num_pages = num_slots;
  p.nh = nh;
  p.page_size = 1;
  p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  bool skip = false;
  const size_t need = latent_attn_workspace_bytes(rows, nh, topk, nope, pe);
  if ((st = check_attn(p, workspace, workspace_bytes, need, fmt, scale, &skip)) != INVROPE_OK || skip) return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != INVROPE_OK) return st;
  return launch(p, fmt, reinterpret_cast<cudaStream_t>(stream));
}
