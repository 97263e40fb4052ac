// Rotary positions (include/rope.h).
//
// One pass, bound by memory: a thread holds the same channels of up to kHeads heads
// of a row, whose loads are all in flight before the first is used, and forms its
// pairs' sines and cosines once for all of them. (Of tensors with one or two heads, it
// holds those of as many rows.) In the half layout a thread takes a
// vector of first halves and that of their partners, so that a call in place reads
// both before it writes either; interleaved pairs lie within a vector. Channels that
// are not rotated are further vectors of the row, in calls that are not in place.
//
// Measured (one GB300): 16384 rows of 64 heads of 448 + 64 channels, bf16: 327 us, 6.57
// TB/s of the 6.80 of a copy (warps with both kinds of vectors: 367; counters of 4096 rows:
// DRAM bytes as they should be, issue slots 35% busy); in place, 64 channels of each, 46 us;
// 10007 rows of 48 heads of 128 fp32 channels 72 us, 6.83 TB/s. 64 rows: 3.1 us, a launch
// and one round of loads. What is further from a copy:
//   - one or two heads in the half layout: 131072 rows of 448 + 64 bf16 channels 56 us, 4.8
//     TB/s (interleaved 41, 6.5): 90 registers leave 21% of the warps, which wait for their
//     loads, and DRAM 52% busy (interleaved 51 registers, 42%, 71%).
//   - vectors of rows whose rotated channels are none: 16384 x 64 heads of 86 + 10 channels 82
//     us, 4.9 TB/s: issue slots 78% busy, nine loads for each store (partners one by one).
//   - single channels: 2.3 to 2.6 TB/s: issue slots 84% busy.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "common.h"
#include "latent.cuh"
#include "ptx.cuh"
#include "rope.h"

namespace invrope {

#ifdef INVROPE_DEBUG_BOUNDS
// The debug-bounds build's fault word of this translation unit, which waits for nothing
// on the device; take_latent_fault() reads and clears it with its own.
__device__ unsigned int g_rope_fault = 0;

int take_rope_fault(unsigned int* code) {
  cudaError_t err = cudaMemcpyFromSymbol(code, g_rope_fault, sizeof(*code));
  if (err != cudaSuccess) return cuda_fail(err);
  const unsigned int zero = 0;
  if ((err = cudaMemcpyToSymbol(g_rope_fault, &zero, sizeof(zero))) != cudaSuccess) return cuda_fail(err);
  return INVROPE_OK;
}
#endif

namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;
constexpr int kMaxPairs = 256;
constexpr int64_t kManyRows = 4096;
constexpr int64_t kMaxRowChannels = 65536;  // a band's work items' numbers have 32 bits
constexpr int kBand = 32;

struct Span {
  const char* x;
  char* out;
  int64_t x_row, x_head, out_row, out_head;  // bytes
  int heads, groups;      // heads, and groups of kHeads of them (kRows: heads)
  int pair_units, copy_units;  // vectors (or pairs of vectors) of a head: rotated, copied
  int offset, below;      // first rotated channel, copied vectors below it
  int64_t first;          // the tensor's first thread block
  int narrow;             // its work items' numbers have 32 bits
};

// Pairs: the most that a call's parameters hold (a launch takes longer with 2 KB of them).
template <int kPairs>
struct RopeParams {
  Span span[ROPE_MAX_TENSORS];
  int count;
  int half;  // pairs
  float amplitude;
  int inverse;
  int64_t n, pos0;
  const int32_t* positions;
  uint64_t turns[kPairs];  // turns a position, 0.64 fixed point
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }

// V elements: one 16-byte access, or one each.
template <typename T, int V>
struct alignas(V * sizeof(T) == 16 ? 16 : sizeof(T)) Vec {
  T v[V];
};
template <typename T, int V>
__device__ __forceinline__ void load(Vec<T, V>& to, const char* at) {
  if constexpr (V * sizeof(T) == 16) {
    *reinterpret_cast<uint4*>(&to) = *reinterpret_cast<const uint4*>(at);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) to.v[k] = reinterpret_cast<const T*>(at)[k];
  }
}
template <typename T, int V>
__device__ __forceinline__ void store(char* at, const Vec<T, V>& from) {
  if constexpr (V * sizeof(T) == 16) {
    *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(&from);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) reinterpret_cast<T*>(at)[k] = from.v[k];
  }
}

// Cosine and sine of `turns` (0.64 fixed point, whole turns dropped). 16-bit types: the
// hardware's, within 2^-21.2 on [-pi, pi), of an angle that is rounded twice (2^-22.3
// each), 2^-20 in all. fp32: the nearest quarter turn is taken off exactly, the rest, at
// most an eighth, is rounded to fp32 (by 2^-25.3), and its sine and cosine are within 1
// ulp: 2^-23 in all.
template <bool kExact>
__device__ __forceinline__ void cos_sin(uint64_t turns, float& c, float& s) {
  const int32_t t = static_cast<int32_t>(turns >> 32);
  if constexpr (!kExact) {
    __sincosf(6.28318530717958648f * (static_cast<float>(t) * 2.3283064365386963e-10f), &s, &c);
  } else {
    const uint32_t quarter = (static_cast<uint32_t>(t) + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>(t) - (quarter << 30));
    float a, b;
    sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &a, &b);  // half turns
    const float x = quarter & 1 ? a : b, y = quarter & 1 ? b : a;
    c = (quarter + 1) & 2 ? -x : x;
    s = quarter & 2 ? -y : y;
  }
}

// What a call takes of the memory's layout: kVector 16-byte vectors of pairs (and of copied
// channels); kMixed rows that are vectors, but whose rotated channels do not begin or end
// with them: a thread takes a vector of the row, whatever is in it, and reads its rotated
// channels' partners one by one, which a call in place must not; kSingle single channels.
enum Layout { kVector, kMixed, kSingle };

template <typename T, int V, bool kInter, int kPairs, Layout kLayout, bool kRows>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams<kPairs> p) {
  constexpr int kPer = kInter ? V / 2 : V;  // pairs of a thread
  constexpr int kCopy = kLayout == kSingle ? 1 : V;  // channels of a copied vector
  __shared__ uint64_t turns[kPairs];
  for (int i = threadIdx.x; i < p.half; i += kThreads) turns[i] = p.turns[i];
  int which = 0;
#pragma unroll
  for (int k = 1; k < ROPE_MAX_TENSORS; ++k)
    if (k < p.count && static_cast<int64_t>(blockIdx.x) >= p.span[k].first) which = k;
  const Span& sp = p.span[which];
  // the block's first row, and this thread's row, heads and vector
  const int64_t item0 = (static_cast<int64_t>(blockIdx.x) - sp.first) * kThreads;
  // (kRows: for kBand bundles of kHeads rows what is a row's else)
  constexpr uint32_t kBundles = kRows ? kBand : 1;
  const uint32_t lists = sp.groups * kBundles;
  const uint32_t per_row = lists * (sp.pair_units + sp.copy_units);
  const int64_t row0 = sp.narrow ? static_cast<uint32_t>(item0) / per_row : item0 / per_row;
  uint32_t at = static_cast<uint32_t>(item0 - row0 * per_row) + threadIdx.x;
  const uint32_t past = at / per_row;
  at -= past * per_row;
  const int64_t band = row0 + past;
  // a row's rotated vectors come before its others: warps do one or the other (with both
  // in a head's order, 4 lanes of every other warp of 448 + 64 channels formed sines)
  const uint32_t pairs = lists * sp.pair_units;
  const bool pair = kLayout != kMixed && at < pairs;
  const uint32_t each = pair ? sp.pair_units : sp.copy_units, in = pair ? at : at - pairs;
  const int list = static_cast<int>(in / each);
  const int u = static_cast<int>(in) - list * static_cast<int>(each);
  const int bundle = kRows ? list / sp.groups : 0, g = kRows ? list - bundle * sp.groups : list;
  const int64_t r = kRows ? (band * kBand + bundle) * kHeads : band;
  const bool live = r < p.n;
  const int ch = pair           ? sp.offset + u * V
                 : u < sp.below ? u * kCopy
                                : sp.offset + 2 * p.half + (u - sp.below) * kCopy;
  const int h0 = kRows ? g : g * kHeads;
  // instances of the thread's channels: heads of a row, or rows of a head
  const int64_t x_step = kRows ? sp.x_row : sp.x_head, out_step = kRows ? sp.out_row : sp.out_head;
  const int64_t left = kRows ? p.n - r : sp.heads - h0;
  const char* x = sp.x + r * sp.x_row + h0 * sp.x_head + static_cast<int64_t>(ch) * sizeof(T);
  char* out = sp.out + r * sp.out_row + h0 * sp.out_head + static_cast<int64_t>(ch) * sizeof(T);
  LATENT_DBG_CHECK(g_rope_fault,
                   !live || (r >= 0 && h0 < sp.heads && ch >= 0 && list >= 0 && u >= 0 && u < static_cast<int>(each) &&
                             (kLayout == kMixed ? u < sp.copy_units
                              : pair            ? ch + (kInter ? V : p.half + V) <= sp.offset + 2 * p.half &&
                                                      (u + 1) * kPer <= p.half
                                                : ch + kCopy <= sp.offset || ch >= sp.offset + 2 * p.half)),
                   29);
  const int partner = kInter ? 0 : p.half * static_cast<int>(sizeof(T));
  Vec<T, V> a[kHeads], b[kHeads];
#pragma unroll
  for (int k = 0; k < kHeads; ++k)
    if (live && k < left) {
      if (kCopy < V && !pair)
        a[k].v[0] = *reinterpret_cast<const T*>(x + k * x_step);
      else
        load(a[k], x + k * x_step);
      if (!kInter && pair) load(b[k], x + k * x_step + partner);
    }
  __syncthreads();  // turns
  if (!live) return;
  if (kLayout == kMixed) {
    if (ch + V > sp.offset && ch < sp.offset + 2 * p.half) {
      const uint64_t pos = static_cast<uint64_t>(p.pos0) + static_cast<uint64_t>(p.positions ? static_cast<int64_t>(__ldg(p.positions + r)) : r);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int rel = ch + e - sp.offset;
        if (rel < 0 || rel >= 2 * p.half) continue;
        const bool second = kInter ? rel & 1 : rel >= p.half;
        const int away = (kInter ? 1 : p.half) * (second ? -1 : 1);
        float c, s;
        cos_sin<sizeof(T) == 4>(pos * turns[kInter ? rel / 2 : second ? rel - p.half : rel], c, s);
        c *= p.amplitude;
        s *= p.inverse ? -p.amplitude : p.amplitude;
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
          if (k < left) {
            const float own = to_f32<T>(a[k].v[e]);
            const float other = to_f32<T>(reinterpret_cast<const T*>(x + k * x_step)[e + away]);
            const float turned = __fmul_rn(other, s);
            a[k].v[e] = from_f32<T>(fmaf(own, c, second ? turned : -turned));
          }
      }
    }
  }
  if (pair) {
    float c[kPer], s[kPer];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      if (kRows && k >= left) break;
      if (k == 0 || kRows) {
        const int64_t at_row = kRows ? r + k : r;
        const uint64_t pos = static_cast<uint64_t>(p.pos0) +
                             static_cast<uint64_t>(p.positions ? static_cast<int64_t>(__ldg(p.positions + at_row)) : at_row);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          cos_sin<sizeof(T) == 4>(pos * turns[u * kPer + i], c[i], s[i]);
          c[i] *= p.amplitude;
          s[i] *= p.inverse ? -p.amplitude : p.amplitude;
        }
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        T& first = kInter ? a[k].v[2 * i] : a[k].v[i];
        T& second = kInter ? a[k].v[2 * i + 1] : b[k].v[i];
        const float x1 = to_f32<T>(first), x2 = to_f32<T>(second);
        // (which product is rounded is said here: the same bits in every variant)
        first = from_f32<T>(fmaf(x1, c[i], -__fmul_rn(x2, s[i])));
        second = from_f32<T>(fmaf(x2, c[i], __fmul_rn(x1, s[i])));
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kHeads; ++k)
    if (k < left) {
      if (kCopy < V && !pair)
        *reinterpret_cast<T*>(out + k * out_step) = a[k].v[0];
      else
        store(out + k * out_step, a[k]);
      if (!kInter && pair) store(out + k * out_step + partner, b[k]);
    }
}

// ---------------------------------------------------------------- host side

// f / (2 pi) without its whole turns, in 0.64 fixed point: positions are whole, so
// whole turns a position do not show. The product is formed with its rounding error,
// and 1 / (2 pi) to 107 bits.
uint64_t fixed_turns(double f) {
  constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double q = f * hi, rest = std::fma(f, hi, -q) + f * lo;
  const double part = std::fabs(q - std::trunc(q));  // exact, below 1
  uint64_t a = static_cast<uint64_t>(std::nearbyint(std::ldexp(part, 64)));
  if (q < 0.0) a = 0 - a;
  // at most 2^-53 of q, of either sign
  const double more = std::ldexp(rest - std::nearbyint(rest), 64);
  const uint64_t b = more < 0x1p63 ? static_cast<uint64_t>(static_cast<int64_t>(std::nearbyint(more))) : uint64_t(1) << 63;
  return a + b;
}

struct Extent {
  uintptr_t at;
  size_t bytes;    // from the first element to behind the last
  int64_t row;     // bytes from a row to the next; 0: one row
  size_t in_row;   // from a row's first element to behind its last
};

Extent extent_of(const void* p, int64_t n, const RopeTensor& t, int64_t row, int64_t head, int size) {
  Extent e;
  e.at = reinterpret_cast<uintptr_t>(p);
  e.in_row = static_cast<size_t>((t.heads - 1) * head + t.d) * size;
  e.row = n > 1 ? row * size : 0;
  e.bytes = static_cast<size_t>(n - 1) * row * size + e.in_row;
  return e;
}

bool apart(const Extent& a, const Extent& b) {
  if (!(a.at < b.at + b.bytes && b.at < a.at + a.bytes)) return true;
  // beside each other in rows of one stride
  if (a.row != b.row || a.row <= 0) return false;
  const int64_t row = a.row;
  const uintptr_t step = b.at >= a.at ? (b.at - a.at) % row : (row - (a.at - b.at) % row) % row;
  return step >= a.in_row && step + b.in_row <= static_cast<uintptr_t>(row);
}

bool strides_apart(int64_t n, const RopeTensor& t) {  // an output's elements do not share memory
  if (t.out_row < 0 || t.out_head < 0) return false;
  const bool rows_outside = (t.heads == 1 || t.out_head >= t.d) && (n == 1 || t.out_row >= (t.heads - 1) * t.out_head + t.d);
  const bool heads_outside = (n == 1 || t.out_row >= t.d) && (t.heads == 1 || t.out_head >= (n - 1) * t.out_row + t.d);
  return rows_outside || heads_outside;
}

template <typename T, int V, bool kInter, Layout kLayout, bool kRows>
int launch(const RopeTensor* tensors, int count, const uint64_t* turns, const int32_t* positions, int64_t pos0, int64_t n,
           int pe, double amplitude, int inverse, cudaStream_t s) {
  const auto fill = [&](auto& p) -> int64_t {
    int64_t blocks = 0;
    p.count = 0;
    for (int k = 0; k < count; ++k) {
      const RopeTensor& t = tensors[k];
      const int size = sizeof(T);
      Span& sp = p.span[p.count++];
      sp.x = static_cast<const char*>(t.x);
      sp.out = static_cast<char*>(t.out);
      sp.x_row = t.x_row * size, sp.x_head = t.x_head * size;
      sp.out_row = t.out_row * size, sp.out_head = t.out_head * size;
      sp.heads = static_cast<int>(t.heads);
      sp.groups = kRows ? sp.heads : (sp.heads + kHeads - 1) / kHeads;
      sp.offset = static_cast<int>(t.offset);
      constexpr int kCopy = kLayout == kSingle ? 1 : V;
      if (kLayout == kMixed) {  // vectors of the whole row
        sp.pair_units = 0;
        sp.copy_units = static_cast<int>(t.d / V);
        sp.below = sp.copy_units;
      } else {
        sp.pair_units = (kInter ? pe : pe / 2) / V;
        sp.copy_units = t.x == t.out ? 0 : static_cast<int>((t.d - pe) / kCopy);
        sp.below = sp.offset / kCopy;
      }
      sp.first = blocks;
      const int64_t per_row = static_cast<int64_t>(sp.groups) * (kRows ? kBand : 1) * (sp.pair_units + sp.copy_units);
      const int64_t items = (kRows ? (n + kHeads * kBand - 1) / (kHeads * kBand) : n) * per_row;
      sp.narrow = items < int64_t(1) << 32;
      blocks += (items + kThreads - 1) / kThreads;
    }
    p.half = pe / 2;
    p.amplitude = static_cast<float>(amplitude);
    p.inverse = inverse;
    p.n = n;
    p.pos0 = pos0;
    p.positions = positions;
    for (int i = 0; i < pe / 2; ++i) p.turns[i] = turns[i];
    return blocks;
  };
  if (pe <= 128) {
    RopeParams<64> p = {};
    const int64_t blocks = fill(p);
    if (blocks == 0) return INVROPE_OK;
    if (blocks > 0x7FFFFFFF) return INVROPE_ERR_UNSUPPORTED;
    rope_kernel<T, V, kInter, 64, kLayout, kRows><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
  } else {
    RopeParams<kMaxPairs> p = {};
    const int64_t blocks = fill(p);
    if (blocks == 0) return INVROPE_OK;
    if (blocks > 0x7FFFFFFF) return INVROPE_ERR_UNSUPPORTED;
    rope_kernel<T, V, kInter, kMaxPairs, kLayout, kRows><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
  }
  return check_launch();
}

template <typename T>
int launch_any(const RopeTensor* tensors, int count, const uint64_t* turns, const int32_t* positions, int64_t pos0,
               int64_t n, int pe, double amplitude, int interleaved, int inverse, cudaStream_t s) {
  // By tensor; those of one layout share a launch.
  constexpr int kVec = 16 / sizeof(T);
  RopeTensor list[4][ROPE_MAX_TENSORS];  // by layout, and kVector's of few heads
  int n_of[4] = {0, 0, 0, 0};
  for (int k = 0; k < count; ++k) {
    const RopeTensor& t = tensors[k];
    if (t.heads == 0) continue;
    const bool rows = aligned(t.x, 16) && aligned(t.out, 16) &&
                      (n == 1 || (t.x_row % kVec == 0 && t.out_row % kVec == 0)) &&
                      (t.heads == 1 || (t.x_head % kVec == 0 && t.out_head % kVec == 0));
    const bool pairs = (interleaved ? pe : pe / 2) % kVec == 0 && t.offset % kVec == 0;
    const bool copied = t.x != t.out && t.d % kVec == 0;
    const Layout layout = rows && pairs && (copied || t.x == t.out) ? kVector : rows && copied ? kMixed : kSingle;
    // 131072 rows of one head of 448 + 64 channels: 157 us by heads, 56 by rows; in a
    // short call both launches' time counts more
    const bool rows_of = layout == kVector && t.heads <= 2 && t.d <= kMaxRowChannels && n >= kManyRows;
    const int which = rows_of ? 3 : layout;
    list[which][n_of[which]++] = t;
  }
  const auto go = [&](auto kernel, int which) {
    return n_of[which] == 0 ? INVROPE_OK
                            : kernel(list[which], n_of[which], turns, positions, pos0, n, pe, amplitude, inverse, s);
  };
  int st = interleaved ? go(launch<T, kVec, true, kVector, false>, kVector) : go(launch<T, kVec, false, kVector, false>, kVector);
  if (st != INVROPE_OK) return st;
  st = interleaved ? go(launch<T, kVec, true, kVector, true>, 3) : go(launch<T, kVec, false, kVector, true>, 3);
  if (st != INVROPE_OK) return st;
  st = interleaved ? go(launch<T, kVec, true, kMixed, false>, kMixed) : go(launch<T, kVec, false, kMixed, false>, kMixed);
  if (st != INVROPE_OK) return st;
  return interleaved ? go(launch<T, 2, true, kSingle, false>, kSingle) : go(launch<T, 1, false, kSingle, false>, kSingle);
}

}  // namespace
}  // namespace invrope

using namespace invrope;

extern "C" int rope_freqs(int pe, double theta, int scaling, double factor, double original, double beta_fast,
                          double beta_slow, double* freqs, double* amplitude) {
  if (pe < 2 || pe % 2 || !amplitude || !std::isfinite(theta) || theta <= 0.0) return INVROPE_ERR_INVALID_ARG;
  if (pe > 2 * kMaxPairs) return INVROPE_ERR_UNSUPPORTED;
  if (!freqs) return INVROPE_ERR_INVALID_ARG;
  if (scaling < ROPE_SCALE_NONE || scaling > ROPE_SCALE_YARN) return INVROPE_ERR_INVALID_ARG;
  if (scaling != ROPE_SCALE_NONE && !(std::isfinite(factor) && factor >= 1.0)) return INVROPE_ERR_INVALID_ARG;
  if (scaling >= ROPE_SCALE_NTK && theta <= 1.0) return INVROPE_ERR_INVALID_ARG;
  double low = 0.0, high = 1.0, base = theta;
  if (scaling == ROPE_SCALE_NTK) {
    if (pe < 4) return INVROPE_ERR_INVALID_ARG;
    base = theta * std::pow(factor, static_cast<double>(pe) / (pe - 2));
    if (!std::isfinite(base)) return INVROPE_ERR_INVALID_ARG;
  }
  if (scaling == ROPE_SCALE_YARN) {
    if (!(std::isfinite(original) && original > 0.0 && std::isfinite(beta_fast) && beta_fast > beta_slow && beta_slow > 0.0))
      return INVROPE_ERR_INVALID_ARG;
    const auto pair = [&](double turns) {
      return pe * std::log(original / (6.283185307179586 * turns)) / (2.0 * std::log(theta));
    };
    low = std::fmax(0.0, std::floor(pair(beta_fast)));
    high = std::fmin(pe - 1.0, std::ceil(pair(beta_slow)));
  }
  for (int i = 0; i < pe / 2; ++i) {
    double f = std::pow(base, -2.0 * i / pe);
    if (scaling == ROPE_SCALE_LINEAR) f /= factor;
    if (scaling == ROPE_SCALE_YARN) {
      const double r = std::fmin(1.0, std::fmax(0.0, (i - low) / std::fmax(high - low, 1e-3)));
      f *= r / factor + 1.0 - r;
    }
    freqs[i] = f;
  }
  *amplitude = scaling == ROPE_SCALE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return INVROPE_OK;
}

extern "C" int rope_apply(const RopeTensor* tensors, int count, const double* freqs, const int32_t* positions, int64_t pos0,
                          int64_t n, int pe, double amplitude, int dtype, int interleaved, int inverse,
                          struct CUstream_st* stream) {
  if (!tensors || count < 1 || count > ROPE_MAX_TENSORS || !freqs || n < 0 || pe < 2 || pe % 2 || dtype < ROPE_BF16 ||
      dtype > ROPE_FP32 || !(std::fabs(amplitude) <= 3.4028234663852886e38) || !aligned(positions, 4))
    return INVROPE_ERR_INVALID_ARG;
  if (pe > 2 * kMaxPairs || n > 0x7FFFFFFF) return INVROPE_ERR_UNSUPPORTED;
  uint64_t turns[kMaxPairs];
  for (int i = 0; i < pe / 2; ++i) {
    if (!std::isfinite(freqs[i])) return INVROPE_ERR_INVALID_ARG;
    turns[i] = fixed_turns(freqs[i]);
  }
  const int size = dtype == ROPE_FP32 ? 4 : 2;
  constexpr int64_t kMost = int64_t(1) << 30;
  constexpr int64_t kFar = int64_t(1) << 56;  // elements from a tensor's first to its last row, or head
  for (int k = 0; k < count; ++k) {
    const RopeTensor& t = tensors[k];
    if (t.heads < 0 || t.d < 1 || t.offset < 0 || t.offset > t.d - pe || t.x_row < 0 || t.x_head < 0)
      return INVROPE_ERR_INVALID_ARG;
    if (t.d >= kMost || t.heads >= kMost || t.heads * t.d >= kMost ||
        (n > 1 && (t.x_row > kFar / n || t.out_row > kFar / n)) ||
        (t.heads > 1 && (t.x_head > kFar / t.heads || t.out_head > kFar / t.heads)))
      return INVROPE_ERR_UNSUPPORTED;
    if (n == 0 || t.heads == 0) continue;
    if (!t.x || !t.out || !aligned(t.x, size) || !aligned(t.out, size) || !strides_apart(n, t)) return INVROPE_ERR_INVALID_ARG;
    if (t.x == t.out && ((n > 1 && t.x_row != t.out_row) || (t.heads > 1 && t.x_head != t.out_head)))
      return INVROPE_ERR_INVALID_ARG;
  }
  if (n == 0) return INVROPE_OK;
  for (int k = 0; k < count; ++k) {
    if (tensors[k].heads == 0) continue;
    const Extent out = extent_of(tensors[k].out, n, tensors[k], tensors[k].out_row, tensors[k].out_head, size);
    const Extent pos = {reinterpret_cast<uintptr_t>(positions), positions ? static_cast<size_t>(n) * 4 : 0, 0, 0};
    if (pos.bytes > 0 && !apart(out, pos)) return INVROPE_ERR_INVALID_ARG;
    for (int j = 0; j < count; ++j) {
      const RopeTensor& t = tensors[j];
      if (t.heads == 0) continue;
      const Extent in = extent_of(t.x, n, t, t.x_row, t.x_head, size);
      const bool own = j == k && t.x == t.out;
      if (!own && !apart(out, in)) return INVROPE_ERR_INVALID_ARG;
      if (j != k && !apart(out, extent_of(t.out, n, t, t.out_row, t.out_head, size))) return INVROPE_ERR_INVALID_ARG;
    }
  }
  DeviceInfo dev;
  const int st = current_device(&dev);
  if (st != INVROPE_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == ROPE_BF16)
    return launch_any<__nv_bfloat16>(tensors, count, turns, positions, pos0, n, pe, amplitude, interleaved, inverse, s);
  if (dtype == ROPE_FP16)
    return launch_any<__half>(tensors, count, turns, positions, pos0, n, pe, amplitude, interleaved, inverse, s);
  return launch_any<float>(tensors, count, turns, positions, pos0, n, pe, amplitude, interleaved, inverse, s);
}
