// Attention over the latent cache (include/latent_attn.h): keys and values are
// the same rows c_t, addressed through pages or through an index table.
//
// One row's head tile (up to 64 heads) over a run of 64-token tiles:
//
//   S[64 heads, 64 tokens] = Q C^T             (tcgen05, M = 64, K = d)
//   P = exp2(scale log2(e) S - m), m a running reference per head
//   O^T[d, heads] += C^T P^T                   (tcgen05, M = 128 per 128 channels)
//
// Both products read the same copy of the tile in shared memory: C is K-major
// for S and, transposed by its descriptor, M-major for O^T. So a cache row is
// fetched once and used 4 * 64 * d times.
//
// Thread blocks take equal runs of a line on which every (row, head tile) has
// kOverhead units and its tiles, whatever the rows' lengths; a row that runs
// over several blocks leaves one partial (accumulators, reference and sum in
// fp32) for each, which latent_join_kernel adds up in a fixed order.
//
// Warps: 0-3 softmax and output (TMEM lanes), 4 MMA issue, 5 queries (TMA),
// 6-13 cache rows: global loads one tile ahead in registers, e4m3 codes
// converted on the way to shared memory.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <mutex>

#include "common.h"
#include "latent.cuh"
#include "ptx.cuh"

namespace invrope {

// This translation unit's fault word: invrope_take_device_fault() reads and
// clears it with the others.
__device__ unsigned int g_latent_fault = 0;

namespace {

using latent::RowLayout;

constexpr int kTile = 64;        // tokens per tile
constexpr int kBlock = 128;      // channels per stage of the ring
constexpr int kMaxBlocks = latent::kMaxD / kBlock;
constexpr int kStages = 9;       // two tiles of 512 channels and one stage more
constexpr int kStageBytes = kTile * kBlock * 2;
constexpr int kHalf = kTile * 128;       // one 64-channel half of a stage
constexpr int kMaskRing = 16;    // tiles whose token masks are kept (the ring holds at most 9)
constexpr int kOverhead = 2;     // what a row costs beside its tiles, in tiles
constexpr int kMinUnits = 4;     // units of the line a thread block takes at least

constexpr int kSoftmaxThreads = 128;
constexpr int kMmaWarp = 4, kQueryWarp = 5, kLoadWarp = 6, kLoadWarps = 8;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);

// shared memory, from a 1024-byte boundary
constexpr int kOffQ = 0;                                    // 8 x [64 heads][64 channels]
constexpr int kOffRing = kOffQ + latent::kMaxD * 128;       // kStages x 2 x [64 tokens][64 channels]
constexpr int kOffP = kOffRing + kStages * kStageBytes;     // 2 x [64 heads][64 tokens]
constexpr int kOffCtl = kOffP + 2 * 64 * 128;
struct Ctl {
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full, q_empty, s_full[2], p_full[2], o_done[2], drained;
  uint32_t mask[kMaskRing][4];  // a byte for 4 tokens, bit k: token 4 * byte + k is attended to
  float factor[2][64];
  float inv[64];
  int64_t sums[kThreads / 32];
  int64_t total, base;
  int row;
  int abort;
  uint32_t tmem;
};
constexpr int kSmem = kOffCtl + static_cast<int>(sizeof(Ctl)) + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory of one thread block");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 256;  // two S tiles of 64 columns; O^T takes 64 columns a channel block from 0

// fault codes: role in bits 8-11, barrier kind in bits 0-7
enum : unsigned { kFaultLoad = 0xA01, kFaultMma = 0xB01, kFaultQuery = 0xC01, kFaultSoftmax = 0xD01 };
constexpr uint64_t kWaitLimitNs = 2000000000ull;

struct AttnParams {
  CUtensorMap tm_q;      // [rows][nh][d], boxes of [1][heads of a tile][64]
  const char* cache;
  const int32_t* table;  // page table [rows, width] or index table [rows, width]
  const int32_t* lens;   // NULL: an index table
  __nv_bfloat16* O;
  float* lse;
  // partials of rows that are split: slot 2c is thread block c's last row when
  // it goes on in block c + 1, slot 2c + 1 its first when it began before c
  float* part;           // [slots][heads of a tile][d]
  float2* part_ml;       // [slots][heads of a tile] (reference, sum)
  int4* split;           // [blocks] (pieces, row, head tile, 0); pieces = 0: none begins in the block
  int64_t rows, width, num_slots, num_pages;
  int nh, head_tiles, tile_heads, page_size;
  float scale_log2;      // scale * log2(e)
  RowLayout l;
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned code) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t n = 1;; ++n) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if ((n & 63u) == 0 && ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicCAS(&g_latent_fault, 0u, code);
      *abort_flag = 1;
      return false;
    }
  }
}

// Bounded wait that ignores the abort flag: for what must land before the
// thread block frees what it is written to.
__device__ __forceinline__ void wait_bar_noabort(uint32_t bar, uint32_t parity) {
  if (ptx::mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(bar, parity))
    if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) return;
}

__device__ __forceinline__ int tokens_of(const AttnParams& p, int64_t r) {
  if (!p.lens) return static_cast<int>(p.width);
  const int n = __ldg(p.lens + r), most = static_cast<int>(p.width) * p.page_size;
  return n < 0 ? 0 : n < most ? n : most;
}

__device__ __forceinline__ int tiles_of(const AttnParams& p, int64_t r) {
  return static_cast<int>((static_cast<unsigned>(tokens_of(p, r)) + kTile - 1) / kTile);
}

// The cache slot of token t of row r, or -1 when it is left out.
__device__ __forceinline__ int slot_of(const AttnParams& p, int64_t r, int t) {
  if (!p.lens) {
    const int s = __ldg(p.table + r * p.width + t);
    return s >= 0 && s < p.num_slots ? s : -1;
  }
  const int pg = static_cast<int>(static_cast<unsigned>(t) / static_cast<unsigned>(p.page_size));
  const int g = __ldg(p.table + r * p.width + pg);
  return g >= 0 && g < p.num_pages ? g * p.page_size + (t - pg * p.page_size) : -1;
}

// First unit of thread block c's run of a line of `total` units cut into n runs,
// and the run that unit x lies in.
__device__ __forceinline__ int64_t run_begin(int64_t c, int64_t total, int64_t n) { return c * total / n; }
__device__ __forceinline__ int64_t run_of(int64_t x, int64_t total, int64_t n) { return ((x + 1) * n - 1) / total; }

// This thread block's pieces of rows, in order. Every role walks them alike.
struct Piece {
  int64_t row;
  int head_tile;
  int j0, j1;   // tiles [j0, j1) of the row's nt
  int nt;
  int64_t at;   // the row's first unit on the line
};
struct Walk {
  int64_t row, at, lo, hi;
  int head_tile;
  __device__ __forceinline__ bool next(const AttnParams& p, Piece& x) {
    while (row < p.rows && at < hi) {
      const int nt = tiles_of(p, row);
      const int64_t first = at + kOverhead;
      // (hi may lie within the row's overhead, lo beyond its tiles)
      const int64_t a = min(static_cast<int64_t>(nt), max(lo - first, static_cast<int64_t>(0)));
      const int64_t b = max(a, min(hi - first, static_cast<int64_t>(nt)));
      const bool mine = b > a || (nt == 0 && at >= lo);
      x = Piece{row, head_tile, static_cast<int>(a), static_cast<int>(b), nt, at};
      at = first + nt;
      if (++head_tile == p.head_tiles) {
        head_tile = 0;
        ++row;
      }
      if (mine) return true;
    }
    return false;
  }
};

// Runs of the line: the whole line's units and this block's first row. All
// threads of the block call it.
__device__ void find_run(const AttnParams& p, Ctl* ctl, Walk* w, int64_t* total, int64_t* nrun) {
  const int tid = threadIdx.x;
  if (!p.lens) {  // every row is as long: no table of lengths to add up
    const int64_t unit = static_cast<int64_t>(p.head_tiles) * (kOverhead + tiles_of(p, 0));
    *total = p.rows * unit;
    const int64_t most = *total / kMinUnits;
    *nrun = most < 1 ? 1 : most < gridDim.x ? most : gridDim.x;
    w->lo = run_begin(blockIdx.x, *total, *nrun);
    w->row = w->lo / unit;
    w->at = w->row * unit;
  } else {
    const int64_t per = (p.rows + kThreads - 1) / kThreads;
    const int64_t r0 = per * tid < p.rows ? per * tid : p.rows;
    const int64_t r1 = r0 + per < p.rows ? r0 + per : p.rows;
    int64_t sum = 0;
    for (int64_t r = r0; r < r1; ++r) sum += static_cast<int64_t>(p.head_tiles) * (kOverhead + tiles_of(p, r));
    int64_t upto = sum;  // inclusive over the warp, then over the block
    for (int o = 1; o < 32; o *= 2) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if ((tid & 31) >= o) upto += v;
    }
    if ((tid & 31) == 31) ctl->sums[tid / 32] = upto;
    __syncthreads();
    int64_t all = 0;
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k < tid / 32) upto += ctl->sums[k];
      all += ctl->sums[k];
    }
    *total = all;
    const int64_t most = all / kMinUnits;
    *nrun = most < 1 ? 1 : most < gridDim.x ? most : gridDim.x;
    w->lo = run_begin(blockIdx.x, all, *nrun);
    int64_t at = upto - sum;
    if (w->lo >= at && w->lo < upto) {  // the run begins in this thread's rows
      int64_t r = r0;
      for (;; ++r) {
        const int64_t unit = static_cast<int64_t>(p.head_tiles) * (kOverhead + tiles_of(p, r));
        if (w->lo < at + unit) break;
        at += unit;
      }
      ctl->row = static_cast<int>(r);
      ctl->base = at;
    }
    __syncthreads();
    w->row = ctl->row;
    w->at = ctl->base;
  }
  w->hi = run_begin(blockIdx.x + 1, *total, *nrun);
  w->head_tile = 0;
  if (static_cast<int64_t>(blockIdx.x) >= *nrun) w->hi = w->at = 0;  // nothing to do
}

__device__ __forceinline__ uint4 load_16(const char* at) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(at));
  return v;
}

__device__ __forceinline__ void store_16(uint32_t at, const uint4& v) { ptx::st_shared_v4(at, v.x, v.y, v.z, v.w); }

// One loading thread's share of a tile: tokens tok and tok + 32, and of each
// 128-channel block the 16 channels that thread j of 8 takes: units j and j + 8
// of 8 channels (bf16 rows), or the 16 channels from 16 j on (e4m3 rows).
struct Raw {
  uint4 a[kMaxBlocks][2], b[kMaxBlocks][2];
};

// Loads block b of the tile whose slots are given; what is not there reads 0.
template <bool E4M3>
__device__ __forceinline__ void load_block(const AttnParams& p, Raw& raw, int b, int j, const int (&slot)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const char* row = p.cache + static_cast<int64_t>(slot[k]) * p.l.row_bytes;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    if (!E4M3) {
      const int c = b * kBlock + 8 * j;
      raw.a[b][k] = slot[k] >= 0 && c < p.l.d ? load_16(row + 2 * c) : zero;
      raw.b[b][k] = slot[k] >= 0 && c + 64 < p.l.d ? load_16(row + 2 * c + 128) : zero;
    } else {
      const int c = b * kBlock + 16 * j;
      const int pe = p.l.nope + 2 * (c - p.l.nope);
      raw.a[b][k] = slot[k] >= 0 && c < p.l.d ? load_16(row + (c < p.l.nope ? c : pe)) : zero;
      raw.b[b][k] = slot[k] >= 0 && c >= p.l.nope && c + 8 < p.l.d ? load_16(row + pe + 16) : zero;
    }
  }
}

__device__ __forceinline__ uint32_t unit_addr(uint32_t stage, int tok, int unit) {
  return stage + (unit >> 3) * kHalf + tok * 128 + (((unit & 7) ^ (tok & 7)) << 4);
}

// Writes block b of a tile into its stage, 128-byte swizzled.
template <bool E4M3>
__device__ __forceinline__ void store_block(const AttnParams& p, const Raw& raw, int b, int j, int tok,
                                            const uint2 (&scales)[2], uint32_t stage) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int t = tok + 32 * k;
    if (!E4M3) {
      store_16(unit_addr(stage, t, j), raw.a[b][k]);
      store_16(unit_addr(stage, t, j + 8), raw.b[b][k]);
    } else {
      uint4 lo = raw.a[b][k], hi = raw.b[b][k];
      const int c = b * kBlock + 16 * j;
      if (c < p.l.nope) {
        const int g = c / latent::kGroup;  // 2b or 2b + 1
        const uint32_t byte = ((g < 4 ? scales[k].x : scales[k].y) >> (8 * (g & 3))) & 255u;
        const uint32_t s = latent::scale_bf16x2(byte);
        const uint4 w = lo;
        latent::e4m3x4_to_bf16(w.x, s, lo.x, lo.y);
        latent::e4m3x4_to_bf16(w.y, s, lo.z, lo.w);
        latent::e4m3x4_to_bf16(w.z, s, hi.x, hi.y);
        latent::e4m3x4_to_bf16(w.w, s, hi.z, hi.w);
      }
      // threads of the two 64-channel halves write the even and the odd unit
      // first in turn: 8 threads of a token then cover all 32 banks
      const int odd = j >> 2;
      store_16(unit_addr(stage, t, 2 * j + odd), odd ? hi : lo);
      store_16(unit_addr(stage, t, 2 * j + 1 - odd), odd ? lo : hi);
    }
  }
}

__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 16 lanes x 64 columns of fp32: thread t holds rows t / 4 (r[4j], r[4j+1]) and
// t / 4 + 8 (r[4j+2], r[4j+3]) at columns 8 j + 2 (t % 4) and the next.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// 16 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// True on all 128 softmax threads when it is on any of them; a barrier.
__device__ __forceinline__ bool any_softmax(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) latent_attn_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ char smem_raw[];
  const uint32_t base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  char* smem = smem_raw + (base - ptx::smem_u32(smem_raw));
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + kOffCtl);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  volatile int* abort_flag = &ctl->abort;
  const auto bar = [](uint64_t& b) { return ptx::smem_u32(&b); };

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar(ctl->full[s]), kLoadWarps);
      ptx::mbar_init(bar(ctl->empty[s]), 1);
    }
    ptx::mbar_init(bar(ctl->q_full), 1);
    ptx::mbar_init(bar(ctl->q_empty), 1);
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(bar(ctl->s_full[k]), 1);
      ptx::mbar_init(bar(ctl->p_full[k]), kSoftmaxThreads);
      ptx::mbar_init(bar(ctl->o_done[k]), 1);
    }
    ptx::mbar_init(bar(ctl->drained), 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&ctl->tmem), kTmemCols);
    ptx::tmem_relinquish();
  }
  Walk w;
  int64_t total, nrun;
  find_run(p, ctl, &w, &total, &nrun);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  const int nblk = (p.l.d + kBlock - 1) / kBlock;
  Piece x;

  if (warp < kMmaWarp) {
    // ---------------------------------------------------------------- softmax and output
    const int hq = 16 * warp + lane / 4;  // this thread's heads: hq and hq + 8 of the tile
    const uint32_t lanes = static_cast<uint32_t>(warp) << 21;  // TMEM lane field, 32 * warp
    bool begun = false;  // a split row began in this block
    uint32_t g = 0;      // tiles so far
    while (w.next(p, x)) {
      const int h0 = x.head_tile * p.tile_heads;
      const int heads = min(p.tile_heads, p.nh - h0);
      float m[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
      for (int j = x.j0; j < x.j1; ++j, ++g) {
        wait_bar(bar(ctl->s_full[g & 1]), (g >> 1) & 1, abort_flag, kFaultSoftmax);
        // the tile's masks were written before its stages were filled; its
        // stages are still full (only this tile's weights let them go)
        const uint32_t n0 = g * nblk;
        wait_bar(bar(ctl->full[n0 % kStages]), (n0 / kStages) & 1, abort_flag, kFaultSoftmax);
        ptx::tc_fence_after();
        uint32_t r[32];
        tmem_ld_16x64(tmem + kColS + (g & 1) * 64 + lanes, r);
        const uint32_t* mk = ctl->mask[g % kMaskRing];
        const uint32_t mk0 = mk[0], mk1 = mk[1], mk2 = mk[2], mk3 = mk[3];
        ptx::tmem_ld_wait(r);
        float s[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) s[k] = __uint_as_float(r[k]) * p.scale_log2;
        if ((mk0 & mk1 & mk2 & mk3) != 0x0F0F0F0Fu) {
          const uint32_t word[4] = {mk0, mk1, mk2, mk3};
#pragma unroll
          for (int u = 0; u < 8; ++u) {  // columns 8 u + 2 (lane % 4) and the next
            const uint32_t bits = word[u >> 1] >> (16 * (u & 1) + 8 * ((lane & 3) >> 1) + 2 * (lane & 1));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (!(bits >> (k & 1) & 1u)) s[4 * u + k] = -INFINITY;
          }
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 32; ++k) top[(k >> 1) & 1] = fmaxf(top[(k >> 1) & 1], s[k]);
        bool move = false;
        float ref[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
          // The reference follows the maximum only when it falls behind by
          // more than 2^8: weights stay below 2^8, fp32 sums are as exact, and
          // the accumulators are rescaled in few tiles instead of most.
          float f = 1.f;
          if (top[i] > m[i] + 8.f) {
            if (m[i] != -INFINITY) {
              f = exp2_fast(m[i] - top[i]);
              sum[i] *= f;
              move = move || hq + 8 * i < heads;
            }
            m[i] = top[i];
          }
          if ((lane & 3) == 0) ctl->factor[g & 1][hq + 8 * i] = f;
          ref[i] = m[i] == -INFINITY ? 0.f : m[i];
        }
        const uint32_t pt = base + kOffP + (g & 1) * 8192u;
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float a = exp2_fast(s[4 * u + 2 * i] - ref[i]), b = exp2_fast(s[4 * u + 2 * i + 1] - ref[i]);
            sum[i] += a + b;
            const int h = hq + 8 * i;
            // the weights are rounded to bf16 here, as the second product's operand
            const uint32_t at = pt + h * 128 + ((u ^ (h & 7)) << 4) + 4 * (lane & 3);
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(ptx::pack_bf16x2(a, b)) : "memory");
          }
        ptx::fence_proxy_async_smem();
        if (any_softmax(move) && j > x.j0) {
          // O^T[:, h] *= factor[h], once the products of the tiles before are in
          wait_bar(bar(ctl->o_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, abort_flag, kFaultSoftmax);
          ptx::tc_fence_after();
          const float* f = ctl->factor[g & 1];
          for (int b = 0; b < nblk; ++b)
            for (int c = 0; c < p.tile_heads; c += 16) {
              uint32_t v[16];
              tmem_ld_x16(tmem + lanes + b * 64 + c, v);
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f[c + k]);
              tmem_st_x16(tmem + lanes + b * 64 + c, v);
            }
          ptx::tmem_st_wait();
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(ctl->p_full[g & 1]));
      }
      // the row's (or the piece's) sums, and what its heads are divided by
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 2);
      }
      const bool whole = x.j1 - x.j0 == x.nt;
      const int64_t out = x.row * p.nh + h0;
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (x.j0 > 0 ? 1 : 0);
      if ((lane & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = hq + 8 * i;
          if (whole) {
            ctl->inv[h] = sum[i] == 0.f ? 0.f : 1.f / sum[i];
            if (p.lse && h < heads)
              p.lse[out + h] = sum[i] == 0.f ? -INFINITY : (m[i] + log2f(sum[i])) * 0.6931471805599453f;
          } else if (h < heads) {
            ctl->inv[h] = 1.f;
            p.part_ml[slot * p.tile_heads + h] = make_float2(m[i], sum[i]);
          }
        }
      }
      if (!whole && x.j0 == 0) {
        begun = true;
        if (tid == 0) {
          const int64_t first = x.at + kOverhead;
          const int64_t pieces = run_of(first + x.nt - 1, total, nrun) - run_of(first, total, nrun) + 1;
          p.split[blockIdx.x] = make_int4(static_cast<int>(pieces), static_cast<int>(x.row), x.head_tile, 0);
        }
      }
      ptx::named_bar_sync(1, kSoftmaxThreads);  // inv is written
      if (x.j1 > x.j0) {
        // the last tile's product (s_full of that tile stood for the one two
        // before it, so the parity is of this phase or the one before)
        wait_bar(bar(ctl->o_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, abort_flag, kFaultSoftmax);
        ptx::tc_fence_after();
      }
      for (int b = 0; b < nblk; ++b) {
        const int c = b * kBlock + 32 * warp + lane;
        for (int h1 = 0; h1 < heads; h1 += 16) {
          uint32_t v[16] = {};
          if (x.j1 > x.j0) tmem_ld_x16(tmem + lanes + b * 64 + h1, v);
          if (c < p.l.d) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int h = h1 + k;
              if (h < heads) {
                const float o = __uint_as_float(v[k]);
                if (whole)
                  p.O[(out + h) * p.l.d + c] = __float2bfloat16_rn(o * ctl->inv[h]);
                else
                  p.part[(slot * p.tile_heads + h) * p.l.d + c] = o;
              }
            }
          }
          __syncwarp();
        }
      }
      ptx::tc_fence_before();  // the next row's products overwrite O^T after this thread's next weights
    }
    if (!begun && tid == 0 && p.split) p.split[blockIdx.x] = make_int4(0, 0, 0, 0);
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      const uint32_t id_s = ptx::idesc_bf16_f32(64, kTile, false, false);
      const uint32_t id_o = ptx::idesc_bf16_f32(128, p.tile_heads, true, false);
      uint32_t g = 0, item = 0, n = 0;  // tiles, pieces with tiles, stages filled so far
      bool ok = true;
      // O^T += C^T P^T of tile t, whose first stage is the n0-th
      const auto weigh = [&](uint32_t t, uint32_t n0, bool first) {
        if (!wait_bar(bar(ctl->p_full[t & 1]), (t >> 1) & 1, abort_flag, kFaultMma)) return false;
        ptx::tc_fence_after();
        const uint32_t pt = base + kOffP + (t & 1) * 8192u;
        for (int b = 0; b < nblk; ++b) {
          const uint32_t s = (n0 + b) % kStages, st = base + kOffRing + s * kStageBytes;
          for (int k = 0; k < kTile / 16; ++k)
            ptx::tc_mma_ss(tmem + b * 64, ptx::smem_desc_sw128(st + k * 2048, kHalf, 1024),
                           ptx::smem_desc_sw128(pt + k * 32, 16, 1024), id_o, !first || k > 0);
          ptx::tc_commit(bar(ctl->empty[s]));
        }
        ptx::tc_commit(bar(ctl->o_done[t & 1]));
        return true;
      };
      while (ok && w.next(p, x)) {
        if (x.j1 == x.j0) continue;
        if (!wait_bar(bar(ctl->q_full), item & 1, abort_flag, kFaultMma)) break;
        for (int j = x.j0; ok && j < x.j1; ++j) {
          const uint32_t n0 = n;
          for (int b = 0; ok && b < nblk; ++b, ++n) {
            const uint32_t s = n % kStages, st = base + kOffRing + s * kStageBytes;
            ok = wait_bar(bar(ctl->full[s]), (n / kStages) & 1, abort_flag, kFaultMma);
            if (!ok) break;
            ptx::tc_fence_after();
            const int steps = min(8, (p.l.d - b * kBlock + 15) / 16);
            for (int k = 0; k < steps; ++k) {
              const uint32_t at = (k >> 2) * 8192u + (k & 3) * 32u;
              ptx::tc_mma_ss(tmem + kColS + (g & 1) * 64,
                             ptx::smem_desc_sw128(base + kOffQ + b * 16384u + at, 16, 1024),
                             ptx::smem_desc_sw128(st + at, 16, 1024), id_s, b > 0 || k > 0);
            }
          }
          if (!ok) break;
          ptx::tc_commit(bar(ctl->s_full[g & 1]));
          if (j == x.j1 - 1) ptx::tc_commit(bar(ctl->q_empty));
          // a tile's second product goes out behind the next tile's first, so
          // that the softmax of one runs beside the products of the other
          if (j > x.j0) ok = weigh(g - 1, n0 - nblk, j - 1 == x.j0);
          if (ok && j == x.j1 - 1) ok = weigh(g, n0, j == x.j0);
          ++g;
        }
        ++item;
      }
      // nothing may be in flight when the thread block frees TMEM
      ptx::tc_commit(bar(ctl->drained));
      wait_bar_noabort(bar(ctl->drained), 0);
    }
    __syncwarp();
  } else if (warp == kQueryWarp) {
    // ---------------------------------------------------------------- queries
    if (lane == 0) {
      const int chunks = (p.l.d + 63) / 64;
      uint32_t item = 0;
      while (w.next(p, x)) {
        if (x.j1 == x.j0) continue;
        if (item > 0 && !wait_bar(bar(ctl->q_empty), (item - 1) & 1, abort_flag, kFaultQuery)) break;
        ptx::mbar_arrive_expect_tx(bar(ctl->q_full), chunks * p.tile_heads * 128);
        for (int c = 0; c < chunks; ++c)
          ptx::tma_load_3d(base + kOffQ + c * 8192u, &p.tm_q, c * 64, x.head_tile * p.tile_heads, static_cast<int>(x.row),
                      bar(ctl->q_full));
        ++item;
      }
      if (item > 0) wait_bar_noabort(bar(ctl->q_full), (item - 1) & 1);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- cache rows
    const int lt = tid - 32 * kLoadWarp;
    const int j = lt & 7, tok = lt >> 3;
    // the tiles in order: (row, first token, tokens)
    int64_t row = 0;
    int tile = 0, end = 0, ntok = 0;
    const auto next_slots = [&](int(&slot)[2]) {
      while (tile == end) {
        if (!w.next(p, x)) return false;
        row = x.row;
        tile = x.j0;
        end = x.j1;
        ntok = tokens_of(p, row);
      }
      for (int k = 0; k < 2; ++k) {
        const int t = tile * kTile + tok + 32 * k;
        slot[k] = t < ntok ? slot_of(p, row, t) : -1;
      }
      ++tile;
      return true;
    };
    const auto load_scales = [&](const int(&slot)[2], uint2(&sc)[2]) {
      for (int k = 0; k < 2; ++k)
        sc[k] = E4M3 && slot[k] >= 0
                    ? __ldg(reinterpret_cast<const uint2*>(p.cache + static_cast<int64_t>(slot[k]) * p.l.row_bytes +
                                                           p.l.scale_off))
                    : make_uint2(0u, 0u);
    };
    Raw raw;
    uint2 scales[2], scales1[2];
    int slot[2], slot1[2] = {-1, -1};
    bool live = next_slots(slot), live1 = false;
    if (live) {
      load_scales(slot, scales);
#pragma unroll
      for (int b = 0; b < kMaxBlocks; ++b)
        if (b < nblk) load_block<E4M3>(p, raw, b, j, slot);
      live1 = next_slots(slot1);
    }
    uint32_t n = 0, g = 0;
    bool ok = true;
    while (ok && live) {
      int slot2[2] = {-1, -1};
      const bool live2 = live1 && next_slots(slot2);
      load_scales(slot1, scales1);
      // masks: this warp's tokens are 4 * (warp - kLoadWarp) + 0..3, and those + 32
      const uint32_t b0 = __ballot_sync(0xFFFFFFFFu, slot[0] >= 0), b1 = __ballot_sync(0xFFFFFFFFu, slot[1] >= 0);
      if (lane == 0) {
        const auto nibble = [](uint32_t v) {
          return static_cast<unsigned char>((v & 1u) | (v >> 7 & 2u) | (v >> 14 & 4u) | (v >> 21 & 8u));
        };
        unsigned char* mk = reinterpret_cast<unsigned char*>(ctl->mask[g % kMaskRing]);
        mk[warp - kLoadWarp] = nibble(b0);
        mk[8 + warp - kLoadWarp] = nibble(b1);
      }
#pragma unroll
      for (int b = 0; b < kMaxBlocks; ++b) {
        if (b < nblk && ok) {
          const uint32_t s = n % kStages;
          if (lane == 0 && n >= kStages)
            ok = wait_bar(bar(ctl->empty[s]), (n / kStages - 1) & 1, abort_flag, kFaultLoad);
          ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
          if (ok) {
            store_block<E4M3>(p, raw, b, j, tok, scales, base + kOffRing + s * kStageBytes);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(ctl->full[s]));
            if (live1) load_block<E4M3>(p, raw, b, j, slot1);
            ++n;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        slot[k] = slot1[k];
        slot1[k] = slot2[k];
        scales[k] = scales1[k];
      }
      live = live1;
      live1 = live2;
      ++g;
    }
  }

  // ------------------------------------------------------------------ teardown
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// Adds up the partials of the rows that were split, in the order of their
// tiles: one thread block a (row, head) at a time, a thread 4 channels.
constexpr int kJoinThreads = latent::kMaxD / 4;
constexpr int kMaxRuns = 256;

struct JoinParams {
  const float* part;
  const float2* part_ml;
  const int4* split;
  __nv_bfloat16* O;
  float* lse;
  int runs, nh, tile_heads, d;
};

__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(JoinParams p) {
  __shared__ int4 todo[kMaxRuns];  // (pieces, row, head tile, first run) of the split rows
  __shared__ int count[kMaxRuns / 32];
  __shared__ float weight[kMaxRuns];
  __shared__ float red[kJoinThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  ptx::griddep_wait();  // launched early: wait for the partials
  int n = 0;
  for (int c0 = 0; c0 < p.runs; c0 += kJoinThreads) {
    const int c = c0 + tid;
    int4 e = make_int4(0, 0, 0, 0);
    if (c < p.runs) e = p.split[c];
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, e.x > 0);
    if (lane == 0) count[warp] = __popc(some);
    __syncthreads();
    int at = n;
    for (int k = 0; k < kJoinThreads / 32; ++k) {
      if (k < warp) at += count[k];
      n += count[k];
    }
    if (e.x > 0) {
      e.w = c;
      todo[at + __popc(some & ((1u << lane) - 1u))] = e;
    }
    __syncthreads();
  }
  const int units = n * p.tile_heads;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int4 e = todo[u / p.tile_heads];
    const int h = u % p.tile_heads, head = e.z * p.tile_heads + h;
    if (head >= p.nh) continue;
    const auto slot = [&](int k) { return static_cast<int64_t>(k == 0 ? 2 * e.w : 2 * (e.w + k) + 1) * p.tile_heads + h; };
    float top = -INFINITY;
    for (int k = tid; k < e.x; k += kJoinThreads) top = fmaxf(top, p.part_ml[slot(k)].x);
    for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (lane == 0) red[warp] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    __syncthreads();
    float sum = 0.f;
    for (int k = tid; k < e.x; k += kJoinThreads) {
      const float2 ml = p.part_ml[slot(k)];
      const float w = top == -INFINITY ? 0.f : exp2_fast(ml.x - top);
      weight[k] = w;
      sum += w * ml.y;
    }
    for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = (red[0] + red[1]) + (red[2] + red[3]);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t out = static_cast<int64_t>(e.y) * p.nh + head;
    if (tid * 4 < p.d) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int k = 0; k < e.x; ++k) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(p.part + slot(k) * p.d) + tid);
        const float w = weight[k];
        acc.x += w * v.x;
        acc.y += w * v.y;
        acc.z += w * v.z;
        acc.w += w * v.w;
      }
      uint2 o;
      o.x = ptx::pack_bf16x2(acc.x * inv, acc.y * inv);
      o.y = ptx::pack_bf16x2(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(p.O + out * p.d + tid * 4) = o;
    }
    if (p.lse && tid == 0) p.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    __syncthreads();  // weight and red are read
  }
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Queries [rows][nh][d]: heads past nh and channels past d read as zero.
bool query_map(CUtensorMap* m, const void* q, int64_t rows, int nh, int d, int tile_heads) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(nh), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(d) * nh * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(tile_heads), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a call is cut: head tiles, thread blocks, and the workspace's parts.
struct Plan {
  int head_tiles, tile_heads, grid;
  size_t ml_off, split_off, bytes;  // bytes 0: one thread block, nothing is split
};

Plan make_plan(int64_t rows, int nh, int64_t max_tokens, int d, int sms) {
  Plan n;
  n.head_tiles = nh > 64 ? 2 : 1;
  n.tile_heads = ((nh + n.head_tiles - 1) / n.head_tiles + 15) / 16 * 16;
  const int64_t units = rows * n.head_tiles * (kOverhead + (max_tokens + kTile - 1) / kTile) / kMinUnits;
  const int most = sms < kMaxRuns ? sms : kMaxRuns;
  n.grid = static_cast<int>(units < 1 ? 1 : units < most ? units : most);
  const size_t slots = 2 * static_cast<size_t>(n.grid) * n.tile_heads;
  n.ml_off = slots * d * sizeof(float);
  n.split_off = n.ml_off + slots * sizeof(float2);
  n.bytes = n.grid > 1 ? n.split_off + n.grid * sizeof(int4) : 0;
  return n;
}

// Sizes of a call that are checked before anything else.
int check_shape(int64_t rows, int nh, int64_t max_tokens, double scale) {
  if (rows < 0 || nh < 1 || max_tokens < 0 || !std::isfinite(scale)) return INVROPE_ERR_INVALID_ARG;
  if (nh > 128 || rows >= (int64_t(1) << 31) / nh || max_tokens > 0x7FFFFFFF) return INVROPE_ERR_UNSUPPORTED;
  // units of the line, times thread blocks, are 64-bit numbers
  if (rows > 0 && (max_tokens / kTile + 3) > (int64_t(1) << 52) / rows) return INVROPE_ERR_UNSUPPORTED;
  return INVROPE_OK;
}

bool opt_in_smem(int device) {
  static std::mutex mu;
  static bool done[64] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (!done[device])
    done[device] = cudaFuncSetAttribute(latent_attn_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        kSmem) == cudaSuccess &&
                   cudaFuncSetAttribute(latent_attn_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        kSmem) == cudaSuccess;
  return done[device];
}

// The common part of both calls, after their own shape checks; p holds all but
// the plan, the tensor map and the workspace.
int attend(AttnParams& p, const void* q, void* workspace, size_t workspace_bytes, int fmt, int64_t max_tokens,
           cudaStream_t s) {
  if (p.rows == 0) return INVROPE_OK;
  if (!q || !p.cache || !p.O || !aligned(q, 16) || !aligned(p.cache, 16) || !aligned(p.O, 16) ||
      (p.width > 0 && !p.table) || !aligned(p.table, 4) || !aligned(p.lens, 4) || !aligned(p.lse, 4))
    return INVROPE_ERR_INVALID_ARG;
  const size_t heads = static_cast<size_t>(p.rows) * p.nh, vec = heads * p.l.d * 2;
  struct Range {
    const void* at;
    size_t bytes;
  };
  const Range in[] = {{q, vec},
                      {p.cache, static_cast<size_t>(p.num_slots) * p.l.row_bytes},
                      {p.table, static_cast<size_t>(p.rows) * p.width * 4},
                      {p.lens, p.lens ? static_cast<size_t>(p.rows) * 4 : 0}};
  Range out[] = {{p.O, vec}, {p.lse, p.lse ? heads * 4 : 0}, {workspace, 0}};
  const auto clash = [&] {
    for (int i = 0; i < 3; ++i) {
      for (const Range& x : in)
        if (overlaps(out[i].at, out[i].bytes, x.at, x.bytes)) return true;
      for (int j = 0; j < i; ++j)
        if (overlaps(out[i].at, out[i].bytes, out[j].at, out[j].bytes)) return true;
    }
    return false;
  };
  if (clash()) return INVROPE_ERR_INVALID_ARG;
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != INVROPE_OK) return st;
  const Plan n = make_plan(p.rows, p.nh, max_tokens, p.l.d, dev.sms);
  if (n.bytes > 0) {
    if (!workspace || workspace_bytes < n.bytes) return INVROPE_ERR_WORKSPACE;
    out[2].bytes = n.bytes;
    if (!aligned(workspace, 16) || clash()) return INVROPE_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    p.part = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + n.ml_off);
    p.split = reinterpret_cast<int4*>(ws + n.split_off);
  }
  p.head_tiles = n.head_tiles;
  p.tile_heads = n.tile_heads;
  if (!opt_in_smem(dev.device) || !query_map(&p.tm_q, q, p.rows, p.nh, p.l.d, n.tile_heads)) return INVROPE_ERR_CUDA;
  if (fmt == KV_LATENT_E4M3)
    latent_attn_kernel<true><<<n.grid, kThreads, kSmem, s>>>(p);
  else
    latent_attn_kernel<false><<<n.grid, kThreads, kSmem, s>>>(p);
  if ((st = check_launch()) != INVROPE_OK || n.bytes == 0) return st;
  // programmatic dependent launch: the join's launch is processed while the
  // attention drains; its blocks wait in-kernel for the partials
  const JoinParams jp{p.part, p.part_ml, p.split, p.O, p.lse, n.grid, p.nh, n.tile_heads, p.l.d};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(dev.sms * 2));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, latent_join_kernel, jp);
  if (err != cudaSuccess) return cuda_fail(err);
  return check_launch();
}

AttnParams params(const RowLayout& l, const void* cache, const int32_t* table, const int32_t* lens, void* O, float* lse,
                  int64_t rows, int64_t width, int64_t num_pages, int page_size, int nh, double scale) {
  AttnParams p = {};
  p.cache = static_cast<const char*>(cache);
  p.table = table;
  p.lens = lens;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  p.rows = rows;
  p.width = width;
  p.num_slots = num_pages * page_size;
  p.num_pages = num_pages;
  p.nh = nh;
  p.page_size = page_size;
  p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  p.l = l;
  return p;
}

}  // namespace

int take_latent_fault(unsigned int* code) {
  cudaError_t err = cudaMemcpyFromSymbol(code, g_latent_fault, sizeof(*code));
  if (err != cudaSuccess) return cuda_fail(err);
  const unsigned int zero = 0;
  if ((err = cudaMemcpyToSymbol(g_latent_fault, &zero, sizeof(zero))) != cudaSuccess) return cuda_fail(err);
  return INVROPE_OK;
}

}  // namespace invrope

using namespace invrope;

extern "C" size_t latent_attn_workspace_bytes(int64_t rows, int nh, int64_t max_tokens, int nope, int pe) {
  RowLayout l;
  if (latent::row_layout(nope, pe, KV_LATENT_BF16, &l) != INVROPE_OK ||
      check_shape(rows, nh, max_tokens, 1.0) != INVROPE_OK || rows == 0)
    return 0;
  DeviceInfo dev;
  if (current_device(&dev) != INVROPE_OK) return 0;
  return make_plan(rows, nh, max_tokens, l.d, dev.sms).bytes;
}

extern "C" int latent_attn_decode(const void* q, const void* cache, const int32_t* page_table, const int32_t* lens,
                                  void* O, float* lse, void* workspace, size_t workspace_bytes, int64_t rows, int nh,
                                  int nope, int pe, int fmt, int64_t num_pages, int page_size, int64_t max_pages,
                                  double scale, struct CUstream_st* stream) {
  RowLayout l;
  int st = latent::row_layout(nope, pe, fmt, &l);
  if (st != INVROPE_OK) return st;
  if (num_pages < 1 || page_size < 1 || max_pages < 0) return INVROPE_ERR_INVALID_ARG;
  if (num_pages > 0x7FFFFFFF / page_size || max_pages > 0x7FFFFFFF / page_size) return INVROPE_ERR_UNSUPPORTED;
  if ((st = check_shape(rows, nh, max_pages * page_size, scale)) != INVROPE_OK) return st;
  if (rows > 0 && !lens) return INVROPE_ERR_INVALID_ARG;
  AttnParams p = params(l, cache, page_table, lens, O, lse, rows, max_pages, num_pages, page_size, nh, scale);
  return attend(p, q, workspace, workspace_bytes, fmt, max_pages * page_size, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int latent_attn_sparse(const void* q, const void* cache, const int32_t* idx, void* O, float* lse,
                                  void* workspace, size_t workspace_bytes, int64_t rows, int nh, int nope, int pe,
                                  int fmt, int64_t num_slots, int64_t topk, double scale, struct CUstream_st* stream) {
  RowLayout l;
  int st = latent::row_layout(nope, pe, fmt, &l);
  if (st != INVROPE_OK) return st;
  if (num_slots < 1 || topk < 0) return INVROPE_ERR_INVALID_ARG;
  if (num_slots > 0x7FFFFFFF) return INVROPE_ERR_UNSUPPORTED;
  if ((st = check_shape(rows, nh, topk, scale)) != INVROPE_OK) return st;
  AttnParams p = params(l, cache, idx, nullptr, O, lse, rows, topk, num_slots, 1, nh, scale);
  return attend(p, q, workspace, workspace_bytes, fmt, topk, reinterpret_cast<cudaStream_t>(stream));
}
