// Page tables, slots and positions of a paged cache (include/kv_pages.h).
//
// kv_pages_advance: every thread block reads the sequences and adds them up alike, so that
// no sum goes from one block to another, and then fills a part of the tokens. The state,
// which may be advanced in place, is written when all have read it: by the one block that
// a small step is, or by a second launch of one block, which adds up for itself too: it is
// prepared while the first launch runs and begins when that one's blocks have left. The
// sums saturate at 2^32 - 1: all they are compared with is below 2^31.
//
// A step is bound by its latency: a launch, the sequences, the table or queue entries
// that depend on them, the tokens' stores. 64 sequences of one token each take 4.8 us;
// 1000 sequences with 40 prompts, 84000 tokens, 10.9 in two launches (by a cluster of 8
// blocks 22).
//
// kv_idx_local_to_slots is one pass over the index table, bound by memory: 65536 x 2048
// entries 166 us, 6.5 TB/s of the 6.8 of a copy.
#include <cuda_runtime.h>

#include "common.h"
#include "kv_pages.h"
#include "latent.cuh"
#include "ptx.cuh"

namespace invrope {

#ifdef INVROPE_DEBUG_BOUNDS
// The debug-bounds build's fault word of this translation unit, which waits for nothing
// on the device; take_latent_fault() reads and clears it with its own.
__device__ unsigned int g_pages_fault = 0;

int take_pages_fault(unsigned int* code) {
  cudaError_t err = cudaMemcpyFromSymbol(code, g_pages_fault, sizeof(*code));
  if (err != cudaSuccess) return cuda_fail(err);
  const unsigned int zero = 0;
  if ((err = cudaMemcpyToSymbol(g_pages_fault, &zero, sizeof(zero))) != cudaSuccess) return cuda_fail(err);
  return INVROPE_OK;
}
#endif

namespace {

constexpr int kThreads = 512;
constexpr int kEach = 4;                    // sequences of a thread
constexpr int kChunk = kThreads * kEach;    // sequences at a time
constexpr int kAlone = 2048;                // tokens and sequences of a step that one block takes
constexpr int64_t kMostEntries = int64_t(1) << 56;  // of a table: its bytes are a 64-bit number
enum Mode { kWhole, kFill, kCommit };
constexpr int kBack = 8;                    // pages of a lane on their way back at a time

// n / d for n < 2^31 as a product: m = ceil(2^(31 + l) / d) with 2^l >= d is below 2^32,
// and n (m d - 2^(31 + l)) < 2^31 2^l, so that the quotient is right for every n.
struct Divisor {
  uint32_t d, m, shift;
};
Divisor divisor(uint32_t d) {
  uint32_t l = 0;
  while (l < 31 && (1u << l) < d) ++l;
  return Divisor{d, static_cast<uint32_t>(((uint64_t(1) << (31 + l)) + d - 1) / d), 31 + l};
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, const Divisor& x) {
  return static_cast<uint32_t>(static_cast<uint64_t>(n) * x.m >> x.shift);
}
__device__ __forceinline__ uint32_t pages_of(uint32_t tokens, const Divisor& page) {
  const uint32_t q = quotient(tokens, page);
  return q + (q * page.d != tokens ? 1u : 0u);
}

__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;
  return s < a ? 0xFFFFFFFFu : s;
}

struct Sums {
  uint32_t tokens, pages, back;  // asked for, needed, given back
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return Sums{add_sat(a.tokens, b.tokens), add_sat(a.pages, b.pages), add_sat(a.back, b.back)};
}

struct AdvanceParams {
  const int32_t* state;
  int32_t* state_out;
  int32_t* table;
  int32_t* queue;
  const int32_t* asked;
  int32_t *slots, *positions, *rows, *starts, *granted;
  int b, max_pages, num_pages, room, capacity;
  Divisor page;
};

__device__ __forceinline__ int wrap(uint32_t at, int n) {  // at < 2 n
  return static_cast<int>(at >= static_cast<uint32_t>(n) ? at - n : at);
}

template <Mode kMode>
__global__ void __launch_bounds__(kThreads) advance_kernel(const AdvanceParams p) {
  __shared__ uint32_t first[kChunk];  // a sequence's first token (kept to room)
  __shared__ uint32_t base[kChunk];   // pages needed, or given back, before it
  __shared__ int info[kChunk];        // >= 0: its length, and it gets its tokens; -1: nothing; -1 - k: gives k pages back
  __shared__ Sums part[kThreads / 32];
  __shared__ uint32_t handed;
  const uint32_t rank = blockIdx.x, ranks = gridDim.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  // (plain loads: the state may be written below)
  int head = *reinterpret_cast<const volatile int32_t*>(p.state + p.b);
  int count = *reinterpret_cast<const volatile int32_t*>(p.state + p.b + 1);
  head = head < 0 || head >= p.num_pages ? 0 : head;
  count = min(max(count, 0), p.num_pages);
  const uint32_t room = p.room;
  if (tid == 0) handed = 0;
  Sums carry = {0, 0, 0};
  uint32_t done = 0;  // tokens of the chunks before
  for (int64_t c0 = 0; c0 < p.b; c0 += kChunk) {
    const int n = static_cast<int>(min(static_cast<int64_t>(kChunk), p.b - c0));
    int len[kEach], want[kEach];
    Sums own[kEach], sum = {0, 0, 0};
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = kEach * tid + k;
      len[k] = i < n ? *reinterpret_cast<const volatile int32_t*>(p.state + c0 + i) : 0;
      want[k] = i < n ? __ldg(p.asked + c0 + i) : 0;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      len[k] = min(max(len[k], 0), p.capacity);
      const uint32_t used = pages_of(len[k], p.page);
      const bool fits = want[k] > 0 && want[k] <= p.capacity - len[k];
      own[k].tokens = max(want[k], 0);
      own[k].pages = fits ? pages_of(len[k] + want[k], p.page) - used : 0;
      own[k].back = want[k] < 0 ? used : 0;
      sum = sum + own[k];
    }
    Sums upto = sum;  // over the warp, then over the block
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const Sums v = {__shfl_up_sync(0xFFFFFFFFu, upto.tokens, o), __shfl_up_sync(0xFFFFFFFFu, upto.pages, o),
                      __shfl_up_sync(0xFFFFFFFFu, upto.back, o)};
      if (lane >= o) upto = upto + v;
    }
    Sums before = {__shfl_up_sync(0xFFFFFFFFu, upto.tokens, 1), __shfl_up_sync(0xFFFFFFFFu, upto.pages, 1),
                   __shfl_up_sync(0xFFFFFFFFu, upto.back, 1)};
    if (lane == 0) before = Sums{0, 0, 0};
    if (lane == 31) part[warp] = upto;
    __syncthreads();
    Sums all = carry, at = carry;
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k == warp) at = all;
      all = all + part[k];
    }
    at = at + before;
    carry = all;
    int next[kEach], gets[kEach], start[kEach];
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = kEach * tid + k;
      const Sums to = at + own[k];
      const bool fits = want[k] > 0 && want[k] <= p.capacity - len[k];
      const bool given = fits && (own[k].pages == 0 || to.pages <= static_cast<uint32_t>(count)) && to.tokens <= room;
      if (given && own[k].pages > 0) most = to.pages;
      first[i] = min(at.tokens, room);
      base[i] = own[k].back > 0 ? at.back : at.pages;
      info[i] = given ? len[k] : -1 - static_cast<int>(own[k].back);
      start[k] = static_cast<int>(min(to.tokens, room));
      gets[k] = given ? want[k] : 0;
      next[k] = want[k] < 0 ? 0 : len[k] + gets[k];
      at = to;
    }
    if (most > 0) atomicMax(&handed, most);
    __syncthreads();
    const uint32_t end = min(all.tokens, room);
    for (uint32_t t = done + rank * kThreads + tid; kMode != kCommit && t < end; t += ranks * kThreads) {
      int i = 0;  // the last sequence that begins at t or before
      for (int step = kChunk / 2; step > 0; step /= 2)
        if (i + step < n && first[i + step] <= t) i += step;
      const int length = info[i];
      int slot = -1, pos = 0;
      if (length >= 0) {
        pos = length + static_cast<int>(t - first[i]);
        const uint32_t e = quotient(pos, p.page), used = pages_of(length, p.page);
        const int place = pos - static_cast<int>(e * p.page.d);
        int32_t* entry = p.table + (c0 + i) * p.max_pages + e;
        const int32_t* from =
            e < used ? entry : p.queue + wrap(static_cast<uint32_t>(head) + base[i] + (e - used), p.num_pages);
        LATENT_DBG_CHECK(g_pages_fault,
                         e < static_cast<uint32_t>(p.max_pages) && c0 + i < p.b && place >= 0 && place < static_cast<int>(p.page.d) &&
                             (e < used || (from >= p.queue && from < p.queue + p.num_pages &&
                                           base[i] + (e - used) < static_cast<uint32_t>(count))),
                         25);
        const int page = *from;
        if (e >= used && place == 0) *entry = page;
        if (page >= 0 && page < p.num_pages) slot = page * static_cast<int>(p.page.d) + place;
      }
      LATENT_DBG_CHECK(g_pages_fault, t < room && i < n && pos >= 0 && pos < max(p.capacity, 1), 26);
      p.slots[t] = slot;
      p.positions[t] = pos;
      p.rows[t] = static_cast<int>(c0) + i;
    }
    done = end;
    // pages of sequences that ended, a warp to a sequence; the queue's entries that they
    // go to lie behind those that are handed out
    for (int i = rank * (kThreads / 32) + warp; kMode != kCommit && i < n; i += ranks * (kThreads / 32)) {
      if (info[i] >= -1) continue;
      const uint32_t free = static_cast<uint32_t>(p.num_pages - count), before = base[i];
      if (before >= free) continue;
      const uint32_t pages = min(static_cast<uint32_t>(-1 - info[i]), free - before);
      const int32_t* from = p.table + (c0 + i) * p.max_pages;
      LATENT_DBG_CHECK(g_pages_fault, pages <= static_cast<uint32_t>(p.max_pages) && count + before + pages <= static_cast<uint32_t>(p.num_pages), 27);
      for (uint32_t k0 = lane; k0 < pages; k0 += 32 * kBack) {
        int32_t page[kBack];
#pragma unroll
        for (int k = 0; k < kBack; ++k)
          if (k0 + 32 * k < pages) page[k] = from[k0 + 32 * k];
#pragma unroll
        for (int k = 0; k < kBack; ++k)
          if (k0 + 32 * k < pages) p.queue[wrap(static_cast<uint32_t>(head) + count + before + k0 + 32 * k, p.num_pages)] = page[k];
      }
    }
    if (kMode == kCommit) ptx::griddep_wait();  // the other blocks have read the state
    if (kMode != kFill) {
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int i = kEach * tid + k;
        if (i < n) {
          p.state_out[c0 + i] = next[k];
          p.granted[c0 + i] = gets[k];
          p.starts[c0 + i + 1] = start[k];
        }
      }
    }
    __syncthreads();  // the next chunk's tables
  }
  for (uint32_t t = done + rank * kThreads + tid; kMode != kCommit && t < room; t += ranks * kThreads) {
    p.slots[t] = -1;
    p.positions[t] = 0;
    p.rows[t] = -1;
  }
  __syncthreads();
  if (kMode == kCommit) ptx::griddep_wait();
  if (kMode != kFill && tid == 0) {
    p.starts[0] = 0;
    p.state_out[p.b] = wrap(static_cast<uint32_t>(head) + handed, p.num_pages);
    p.state_out[p.b + 1] =
        count - static_cast<int>(handed) + static_cast<int>(min(carry.back, static_cast<uint32_t>(p.num_pages - count)));
  }
}

struct SlotParams {
  const int32_t *idx, *table, *lens, *seq;
  int32_t* out;
  int64_t vectors;       // of the whole table
  uint32_t per;          // of a row
  int sq, seqs, max_pages, num_pages, capacity;
  Divisor page;
};

__device__ __forceinline__ int slot_of(int token, int limit, const int32_t* table, const SlotParams& p) {
  if (token < 0 || token >= limit) return -1;
  const uint32_t k = quotient(token, p.page);
  LATENT_DBG_CHECK(g_pages_fault, k < static_cast<uint32_t>(p.max_pages) && token < p.capacity, 28);
  const int page = table[k];
  return page >= 0 && page < p.num_pages ? page * static_cast<int>(p.page.d) + token - static_cast<int>(k * p.page.d) : -1;
}

template <typename V>
struct Load;
template <>
struct Load<int4> {
  static __device__ __forceinline__ int4 slots(int4 v, int limit, const int32_t* table, const SlotParams& p) {
    return make_int4(slot_of(v.x, limit, table, p), slot_of(v.y, limit, table, p), slot_of(v.z, limit, table, p),
                     slot_of(v.w, limit, table, p));
  }
};
template <>
struct Load<int> {
  static __device__ __forceinline__ int slots(int v, int limit, const int32_t* table, const SlotParams& p) {
    return slot_of(v, limit, table, p);
  }
};

constexpr int kSlotThreads = 256;
constexpr int kSlotPer = 4;

// V: four entries, or one. A block takes kSlotThreads * kSlotPer of them in a row.
template <typename V>
__global__ void __launch_bounds__(kSlotThreads) slots_kernel(const SlotParams p) {
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * (kSlotThreads * kSlotPer);
  const int64_t row0 = v0 / p.per;
  const uint32_t rest = static_cast<uint32_t>(v0 - row0 * p.per);
  V x[kSlotPer];
#pragma unroll
  for (int k = 0; k < kSlotPer; ++k) {
    const int64_t v = v0 + k * kSlotThreads + threadIdx.x;
    if (v < p.vectors) x[k] = __ldcs(reinterpret_cast<const V*>(p.idx) + v);
  }
#pragma unroll
  for (int k = 0; k < kSlotPer; ++k) {
    const int64_t v = v0 + k * kSlotThreads + threadIdx.x;
    if (v >= p.vectors) break;
    const uint32_t row = static_cast<uint32_t>(row0) + (rest + k * kSlotThreads + threadIdx.x) / p.per;
    const int s = p.seq ? __ldg(p.seq + row) : static_cast<int>(row / static_cast<uint32_t>(p.sq));
    const bool known = s >= 0 && s < p.seqs;
    const int limit = known ? min(__ldg(p.lens + s), p.capacity) : 0;
    __stcs(reinterpret_cast<V*>(p.out) + v,
           Load<V>::slots(x[k], limit, p.table + static_cast<int64_t>(known ? s : 0) * p.max_pages, p));
  }
}

// The same with the sequence's page table in shared memory, for tables of many rows a
// sequence: blocks take chunks in turn and read a sequence's table when its first chunk
// comes. (A random page a lane takes up to 32 accesses of L1 a warp, and of shared memory,
// with 32 lanes over 32 banks, 3.5.) A chunk's vectors of another sequence than its
// first one's read their table where it is.
constexpr int kStagedPages = 8192;
constexpr int kStagedPer = 8;

template <typename V>
__global__ void __launch_bounds__(kSlotThreads) slots_staged_kernel(const SlotParams p) {
  extern __shared__ int32_t staged[];
  int cur = -1, limit = 0;
  const int64_t chunk = kSlotThreads * kStagedPer;
  for (int64_t v0 = blockIdx.x * chunk; v0 < p.vectors; v0 += gridDim.x * chunk) {
    V x[kStagedPer];
#pragma unroll
    for (int k = 0; k < kStagedPer; ++k) {
      const int64_t v = v0 + k * kSlotThreads + threadIdx.x;
      if (v < p.vectors) x[k] = __ldcs(reinterpret_cast<const V*>(p.idx) + v);
    }
    const int64_t row0 = v0 / p.per;
    const uint32_t rest = static_cast<uint32_t>(v0 - row0 * p.per);
    const int64_t last = row0 + (rest + chunk - 1) / p.per;
    const int s0 = static_cast<int>(row0 / p.sq), s1 = static_cast<int>(last / p.sq);
    if (s0 != cur) {
      __syncthreads();  // the table before is read
      cur = s0;
      limit = cur < p.seqs ? min(__ldg(p.lens + cur), p.capacity) : 0;
      const int32_t* table = p.table + static_cast<int64_t>(cur) * p.max_pages;
      const int pages = limit > 0 ? static_cast<int>(pages_of(limit, p.page)) : 0;
      for (int k = threadIdx.x; k < pages; k += kSlotThreads) staged[k] = __ldg(table + k);
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kStagedPer; ++k) {
      const int64_t v = v0 + k * kSlotThreads + threadIdx.x;
      if (v >= p.vectors) break;
      if (s1 == s0) {
        __stcs(reinterpret_cast<V*>(p.out) + v, Load<V>::slots(x[k], limit, staged, p));
      } else {
        const uint32_t row = static_cast<uint32_t>(row0) + (rest + k * kSlotThreads + threadIdx.x) / p.per;
        const int s = static_cast<int>(row / static_cast<uint32_t>(p.sq));
        const int to = s < p.seqs ? min(__ldg(p.lens + s), p.capacity) : 0;
        __stcs(reinterpret_cast<V*>(p.out) + v,
               Load<V>::slots(x[k], to, p.table + static_cast<int64_t>(s < p.seqs ? s : 0) * p.max_pages, p));
      }
    }
  }
}

}  // namespace
}  // namespace invrope

using namespace invrope;

extern "C" int kv_pages_advance(const int32_t* state, int32_t* state_out, int32_t* page_table, int32_t* queue,
                                const int32_t* new_tokens, int32_t* slots, int32_t* positions, int32_t* rows,
                                int32_t* starts, int32_t* granted, int64_t b, int64_t max_pages, int64_t num_pages,
                                int page_size, int64_t max_tokens, struct CUstream_st* stream) {
  if (b < 0 || max_pages < 0 || num_pages < 1 || page_size < 1 || max_tokens < 0) return INVROPE_ERR_INVALID_ARG;
  if (b > 0x7FFFFFFD || max_tokens > 0x7FFFFFFF || num_pages > 0x7FFFFFFF / page_size || max_pages > 0x7FFFFFFF / page_size ||
      (max_pages > 0 && b > kMostEntries / max_pages))
    return INVROPE_ERR_UNSUPPORTED;
  struct Range {
    const void* at;
    size_t bytes;
    bool written;
  };
  const size_t n = static_cast<size_t>(b) * 4, t = static_cast<size_t>(max_tokens) * 4;
  const Range all[] = {{state, n + 8, false},
                       {state_out, n + 8, true},
                       {page_table, n * max_pages, true},
                       {queue, static_cast<size_t>(num_pages) * 4, true},
                       {new_tokens, n, false},
                       {slots, t, true},
                       {positions, t, true},
                       {rows, t, true},
                       {starts, n + 4, true},
                       {granted, n, true}};
  for (const Range& x : all) {
    if ((x.bytes > 0 && !x.at) || !aligned(x.at, 4)) return INVROPE_ERR_INVALID_ARG;
    for (const Range& y : all) {
      if (&y <= &x || !(x.written || y.written)) continue;
      if (&x == all && &y == all + 1 && state == state_out) continue;
      if (overlaps(x.at, x.bytes, y.at, y.bytes)) return INVROPE_ERR_INVALID_ARG;
    }
  }
  DeviceInfo dev;
  const int st = current_device(&dev);
  if (st != INVROPE_OK) return st;
  AdvanceParams p;
  p.state = state, p.state_out = state_out, p.table = page_table, p.queue = queue, p.asked = new_tokens;
  p.slots = slots, p.positions = positions, p.rows = rows, p.starts = starts, p.granted = granted;
  p.b = static_cast<int>(b), p.max_pages = static_cast<int>(max_pages), p.num_pages = static_cast<int>(num_pages);
  p.room = static_cast<int>(max_tokens), p.capacity = static_cast<int>(max_pages) * page_size;
  p.page = divisor(static_cast<uint32_t>(page_size));
  const cudaStream_t at = reinterpret_cast<cudaStream_t>(stream);
  if (max_tokens + b <= kAlone) {
    advance_kernel<kWhole><<<1, kThreads, 0, at>>>(p);
    return check_launch();
  }
  const int64_t blocks = (max_tokens + kThreads - 1) / kThreads, most = 2 * static_cast<int64_t>(dev.sms);
  advance_kernel<kFill><<<static_cast<unsigned>(blocks < 8 ? 8 : blocks < most ? blocks : most), kThreads, 0, at>>>(p);
  const int launched = check_launch();
  if (launched != INVROPE_OK) return launched;
  // programmatic dependent launch: its block waits in-kernel for the first launch
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = at;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, advance_kernel<kCommit>, p);
  if (err != cudaSuccess) return cuda_fail(err);
  return check_launch();
}

extern "C" int kv_idx_local_to_slots(const int32_t* idx, const int32_t* page_table, const int32_t* lens, const int32_t* seq,
                                     int32_t* out, int64_t rows, int64_t topk, int64_t sq, int64_t seqs, int64_t max_pages,
                                     int64_t num_pages, int page_size, struct CUstream_st* stream) {
  if (rows < 0 || topk < 0 || seqs < 0 || max_pages < 0 || num_pages < 1 || page_size < 1 || (!seq && sq < 1))
    return INVROPE_ERR_INVALID_ARG;
  if (rows > 0x7FFFFFFF || topk > 0x7FFFFFFF || seqs > 0x7FFFFFFF || num_pages > 0x7FFFFFFF / page_size ||
      max_pages > 0x7FFFFFFF / page_size || (topk > 0 && rows > kMostEntries / topk) ||
      (max_pages > 0 && seqs > kMostEntries / max_pages))
    return INVROPE_ERR_UNSUPPORTED;
  const int64_t n = rows * topk;
  if (n == 0) return INVROPE_OK;
  const size_t bytes = static_cast<size_t>(n) * 4, table = static_cast<size_t>(seqs) * max_pages * 4;
  if (!idx || !out || (table > 0 && !page_table) || (seqs > 0 && !lens) || !aligned(idx, 4) || !aligned(out, 4) ||
      !aligned(page_table, 4) || !aligned(lens, 4) || !aligned(seq, 4) || (out != idx && overlaps(out, bytes, idx, bytes)) ||
      overlaps(out, bytes, page_table, table) || overlaps(out, bytes, lens, static_cast<size_t>(seqs) * 4) ||
      overlaps(out, bytes, seq, seq ? static_cast<size_t>(rows) * 4 : 0))
    return INVROPE_ERR_INVALID_ARG;
  DeviceInfo dev;
  const int st = current_device(&dev);
  if (st != INVROPE_OK) return st;
  SlotParams p;
  p.idx = idx, p.table = page_table, p.lens = lens, p.seq = seq, p.out = out;
  p.sq = static_cast<int>(sq > 0x7FFFFFFF ? 0x7FFFFFFF : sq < 1 ? 1 : sq);
  p.seqs = static_cast<int>(seqs), p.max_pages = static_cast<int>(max_pages), p.num_pages = static_cast<int>(num_pages);
  p.capacity = static_cast<int>(max_pages) * page_size;
  p.page = divisor(static_cast<uint32_t>(page_size));
  const bool four = topk % 4 == 0 && aligned(idx, 16) && aligned(out, 16);
  p.per = static_cast<uint32_t>(four ? topk / 4 : topk);
  p.vectors = rows * p.per;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // A sequence's table is read once a block, so there have to be several chunks of a
  // sequence for each block: 65536 x 2048 entries of 4 sequences, 5% of them padding,
  // take 166 us so and 176 without; rows of 641, which are no vectors, 77 and 122. (Blocks
  // that take chunks in a row, and so need a table less often, take 181: DRAM has fewer
  // pages open where all blocks are near each other.)
  const int64_t chunks = (p.vectors + kSlotThreads * kStagedPer - 1) / (kSlotThreads * kStagedPer);
  const int64_t grid = static_cast<int64_t>(dev.sms) * 4;
  const int64_t of_sequence = static_cast<int64_t>(p.sq) * p.per;  // (sq itself may be any 64-bit number)
  if (!seq && max_pages <= kStagedPages && chunks >= 2 * grid && of_sequence >= 2 * grid * kSlotThreads * kStagedPer) {
    const size_t smem = static_cast<size_t>(max_pages) * 4;
    if (four)
      slots_staged_kernel<int4><<<static_cast<unsigned>(grid), kSlotThreads, smem, s>>>(p);
    else
      slots_staged_kernel<int><<<static_cast<unsigned>(grid), kSlotThreads, smem, s>>>(p);
    return check_launch();
  }
  const int64_t blocks = (p.vectors + kSlotThreads * kSlotPer - 1) / (kSlotThreads * kSlotPer);
  if (blocks > 0x7FFFFFFF) return INVROPE_ERR_UNSUPPORTED;
  if (four)
    slots_kernel<int4><<<static_cast<unsigned>(blocks), kSlotThreads, 0, s>>>(p);
  else
    slots_kernel<int><<<static_cast<unsigned>(blocks), kSlotThreads, 0, s>>>(p);
  return check_launch();
}
