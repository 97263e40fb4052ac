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
// Rows reach shared memory by cp.async, 16 bytes a thread (6.6 TB/s on pages of
// 64 rows of 1 KB; boxes of 64 rows x 128 bytes through TMA went no faster than
// 4.4). e4m3 codes land in the stage that they are converted in (copy_codes). 256
// channels of the queries lie in TMEM, which leaves the ring nearly three tiles:
// with two, a tile's loads began when the one two before was done (5% slower).
//
// Warps: 0-3 softmax and output (TMEM lanes), 4 S of even tiles, 5 S of odd tiles
// (one issues while the other waits, so that the tensor core does not), 6 O^T
// (either product goes out as soon as what it needs is there: a late tile does not
// hold up the one that frees its stages), 7 the tokens' slots, then 8 that load
// bf16 rows after 4 that bring queries to TMEM, or 16 that load e4m3 rows (there
// the softmax warps bring the queries: 28 warps would have 72 registers each).
//
// Bound: a tile of 64 tokens x 512 channels takes the tensor core 1840 cycles (32
// MMAs of 33 cycles for S, M = 64 being half its rate, 16 of 49 for O^T, whose
// operands shared memory delivers in 48) and DRAM, at 6.8 TB/s over 152 SMs, 2800
// cycles with bf16 rows and 1650 with e4m3. Measured, alone on the GPU:
//   bf16, 2048 rows of 2048 tokens of 65536 (L2 hits): 641 us, 858 TFLOP/s, 2900
//     cycles a tile; 596 us where they are of 64, 618 with nothing to load, so it is
//     not the rows: shared memory delivers for 1540 cycles a tile to the MMAs and
//     takes in and gives out the rest for 680, most of it beside O^T's, which use all
//     that it delivers.
//   bf16, 32 rows of 1 to 16384 tokens: 67.3 us, 4.05 TB/s with start and join, 6.2
//     in between.
//   e4m3, 96 rows of 4000 to 20000 tokens: 273 us, 2.5 TB/s, 552 TFLOP/s; 4350
//     cycles a tile, of which shared memory is busy for 3570: 1536 for the MMAs'
//     operands and 2040 for loads and stores. Of these the codes' way (landing with
//     the pe channels 290, reading 224, bf16 values 450) and the weights (64) need
//     1030; the rest is the loading warps' own: a token's scales copied with every
//     block and read by bytes, reads by lanes that have no codes, barriers, and bank
//     conflicts (540 counted). Issue slots are 59% busy.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cfloat>
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
constexpr int kStageBytes = kTile * kBlock * 2;
constexpr int kHalf = kTile * 128;       // one 64-channel half of a stage
constexpr int kSlotRing = 4;     // tiles whose slots are looked up ahead of their loads
constexpr int kMaskRing = 32;    // tiles whose token masks are kept: those of both rings and in between, at most 17
constexpr int kOverhead = 2;     // what a row costs beside its tiles, in tiles
constexpr int kMinUnits = 4;     // units of the line a thread block takes at least

constexpr int kSoftmaxThreads = 128;
constexpr int kScoreWarp = 4, kValueWarp = 6, kTokenWarp = 7;
constexpr int kQueryChunk = 64 * 128;    // [64 heads][64 channels]
constexpr int kQueryBlocks = 2;  // 128-channel blocks of the queries in TMEM, two bf16 a column
constexpr int kStages = 11;      // a tile is up to 4
template <bool E4M3>
struct Cfg {
  static constexpr int kQueryWarp = 8;
  static constexpr int kLoadWarp = E4M3 ? 8 : 12;
  static constexpr int kLoadWarps = E4M3 ? 16 : 8;
  static constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);
};
constexpr int kMaxWarps = Cfg<true>::kThreads / 32;
// shared memory, from a 1024-byte boundary: the other blocks of the queries, the
// ring (stages of 2 x [64 tokens][64 channels]), weights, barriers and tables
constexpr int kOffRing = (kMaxBlocks - kQueryBlocks) * 2 * kQueryChunk;
constexpr int kOffP = kOffRing + kStages * kStageBytes;  // 2 x [64 heads][64 tokens]
constexpr int kOffCtl = kOffP + 2 * 64 * 128;
struct Ctl {
  uint64_t full[kStages], empty[kStages];
  uint64_t slots_full[kSlotRing], slots_empty[kSlotRing];
  uint64_t q_full, q_empty, s_full[2], s_empty[2], p_full[2], o_done[2], drained[3];
  uint64_t mask[kMaskRing];     // bit t: token t of the tile is attended to
  int slot[kSlotRing][kTile];   // -1: left out; kNoTile: no more tiles
  float factor[2][64];
  float inv[64];
  int64_t sums[kMaxWarps];
  int64_t base;
  int row;
  int abort;
  uint32_t tmem;
};
constexpr int kNoTile = -2;
constexpr int kSmem = kOffCtl + static_cast<int>(sizeof(Ctl));
static_assert(kSmem <= 227 * 1024, "shared memory of one thread block");

constexpr uint32_t kTmemCols = 512;
// O^T takes 64 columns a channel block from 0; two S tiles; two blocks of the
// queries, two bf16 a column
constexpr uint32_t kColS = 256, kColQ = 384;

// fault codes: role in bits 8-11, barrier kind in bits 0-7
enum : unsigned {
  kFaultLoad = 0xA01,
  kFaultScore = 0xB01,
  kFaultValue = 0xC01,
  kFaultSoftmax = 0xD01,
  kFaultToken = 0xE01,
  kFaultQuery = 0xE03,
  kFaultTmem = 0xF02,  // TMEM does not begin at column 0
  kFaultSmem = 0xF01  // shared memory does not begin on a 1024-byte boundary
};
constexpr uint64_t kWaitLimitNs = 2000000000ull;

struct AttnParams {
  const __nv_bfloat16* q;
  CUtensorMap tm_q;      // the queries [rows][nh][d], boxes of [1][heads of a tile][64]
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
  int64_t rows, width, num_slots;
  int num_pages;         // entries of an index table are pages of one slot
  int nh, head_tiles, tile_heads, page_size;
  float scale_log2;      // scale * log2(e)
  RowLayout l;
};

// Out of line, like every path that is not taken often: the roles' code together
// has to stay in the instruction cache.
__device__ __noinline__ bool wait_bar_on(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned code) {
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
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned code) {
  return ptx::mbar_try_wait(bar, parity) || wait_bar_on(bar, parity, abort_flag, code);
}

// The same without a call: uniform registers, where an MMA takes its operands
// from, do not outlive one.
__device__ __forceinline__ void wait_bar_here(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned code) {
  uint64_t t0 = 0;
  for (uint32_t n = 0; !ptx::mbar_try_wait(bar, parity); ++n) {
    if (*abort_flag) return;
    if ((n & 63u) != 0) continue;
    const uint64_t t = ptx::globaltimer_ns();
    if (n == 0) {
      t0 = t;
    } else if (t - t0 > kWaitLimitNs) {
      atomicCAS(&g_latent_fault, 0u, code);
      *abort_flag = 1;
      return;
    }
  }
}

// Bounded wait that ignores the abort flag: for what must land before the
// thread block frees what it is written to.
__device__ __noinline__ void wait_bar_noabort(uint32_t bar, uint32_t parity) {
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

// Token t of row r as its table entry (a page, or a slot as a page of one) and
// place in the page; slot_of turns them into a cache slot, or -1 when the token
// is left out. Apart, so that an entry's load is not waited for where it is issued.
struct Ref {
  int entry, place;
};
__device__ __forceinline__ int load_entry(const int32_t* at) {  // volatile: stays where it is issued
  int v;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(at));
  return v;
}
__device__ __forceinline__ Ref ref_of(const AttnParams& p, int64_t r, int t) {
  LATENT_DBG_CHECK(g_latent_fault, r >= 0 && r < p.rows && t >= 0, 8);
  if (!p.lens) {
    LATENT_DBG_CHECK(g_latent_fault, t < p.width, 9);
    return Ref{load_entry(p.table + r * p.width + t), 0};
  }
  const int pg = static_cast<int>(static_cast<unsigned>(t) / static_cast<unsigned>(p.page_size));
  LATENT_DBG_CHECK(g_latent_fault, pg >= 0 && pg < p.width, 9);
  return Ref{load_entry(p.table + r * p.width + pg), t - pg * p.page_size};
}
__device__ __forceinline__ int slot_of(const AttnParams& p, const Ref& x) {
  return x.entry >= 0 && x.entry < p.num_pages ? x.entry * p.page_size + x.place : -1;
}

// First unit of thread block c's run of a line of `total` units cut into n runs,
// and the run that unit x lies in.
__device__ __noinline__ int64_t run_begin(int64_t c, int64_t total, int64_t n) { return c * total / n; }
__device__ __noinline__ int64_t run_of(int64_t x, int64_t total, int64_t n) { return ((x + 1) * n - 1) / total; }

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
template <int kThreads>
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

__device__ __forceinline__ void store_16(uint32_t at, const uint4& v) { ptx::st_shared_v4(at, v.x, v.y, v.z, v.w); }

__device__ __forceinline__ uint32_t unit_addr(uint32_t stage, int tok, int unit) {  // 8 channels a unit
  return stage + (unit >> 3) * kHalf + tok * 128 + (((unit & 7) ^ (tok & 7)) << 4);
}

// 16 bytes global -> shared without a register; zeros where !there.
__device__ __forceinline__ void copy_16(uint32_t to, const char* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}

// This thread's arrival on `bar` when its copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// All loading warps (of e4m3 rows, every other one) take a few tokens of a block,
// so that a stage that comes free is full again after the work of those few: with
// a block to a warp its 32 copies, or 8 to 16 conversions, lay between any stage's
// release and its next use (1100 and 2800-3500 cycles of a 6500-cycle loop).

// bf16 rows: 8 tokens a warp, two an instruction (16 lanes a token's 256 bytes).
__device__ __forceinline__ void copy_block(const AttnParams& p, const int (&slot)[4], int b, int tok, int lane,
                                           uint32_t stage) {
  const int unit = lane & 15, c = b * kBlock + 8 * unit;
  const char* from = p.cache + (c < p.l.d ? 2 * c : 0);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool there = slot[k] >= 0 && c < p.l.d;
    LATENT_DBG_CHECK(g_latent_fault, slot[k] < p.num_slots && tok + 2 * k < kTile && (!there || c + 8 <= p.l.d), 10);
    copy_16(unit_addr(stage, tok + 2 * k, unit), from + static_cast<int64_t>(there ? slot[k] : 0) * p.l.row_bytes,
            there);
  }
}

// e4m3 rows: half of the warps take even blocks, half odd ones, 8 lanes a token,
// 16 codes a lane. The codes land in the stage itself, in the token's own units,
// and the token's scales behind them: in a block of codes alone in their order,
// else, where the pe channels lie already, each in the first of the two units that
// its lane will write the bf16 values to (everywhere so, 32 bytes of a row came
// apart in two: 281 against 272 us). (Loads to registers went through
// what L1 has left beside 227 KB of shared memory, and with it full every access
// of the SM waited: 96 ragged rows took 305 us whatever was in flight, and 220
// without their loads.) Two blocks in flight a warp: with 281 us for that, one took
// 325 and three, which hold stages for longer, 300; 8 warps of twice the tokens
// 299, and 16 that take 4 tokens of every block 377.
constexpr int kCodeTokens = 2;  // tokens a lane has codes of
constexpr int kCodeStep = kTile / kCodeTokens;
constexpr uint32_t kCodesAhead = 2;  // blocks of a warp in flight

__device__ __forceinline__ void copy_codes(const AttnParams& p, const int (&slot)[kCodeTokens], int b, int item,
                                           uint32_t to, uint32_t scales) {
  const int c = b * kBlock + 16 * item;
  if (c >= p.l.nope) return;
#pragma unroll
  for (int k = 0; k < kCodeTokens; ++k) {
    const bool there = slot[k] >= 0;
    LATENT_DBG_CHECK(g_latent_fault,
                     slot[k] < p.num_slots && c + 16 <= p.l.nope && p.l.scale_off + 16 <= p.l.row_bytes, 11);
    const char* row = p.cache + static_cast<int64_t>(there ? slot[k] : 0) * p.l.row_bytes;
    copy_16(to + k * kCodeStep * 128, row + c, there);
    if (item == 0) copy_16(scales + k * kCodeStep * 128, row + p.l.scale_off, there);  // rows end on 16 bytes
  }
}

__device__ __forceinline__ uint4 load_16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load_byte(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// 16 codes with the scale byte `byte` to the units at `to` and at to ^ 16.
__device__ __forceinline__ void store_codes(const uint4& w, uint32_t byte, uint32_t to) {
  // 2^(byte - 127) times the 2^120 of the conversion is one bf16 factor up to a
  // scale of 2^7; above, 2^127 is, and the rest of it (or NaN) another.
  const uint32_t f = min(byte + 120u, 254u) * 0x00800080u;
  uint4 lo, hi;
  latent::e4m3x4_times(w.x, f, lo.x, lo.y);
  latent::e4m3x4_times(w.y, f, lo.z, lo.w);
  latent::e4m3x4_times(w.z, f, hi.x, hi.y);
  latent::e4m3x4_times(w.w, f, hi.z, hi.w);
  if (byte > 134u) {
    const uint32_t r = latent::scale_bf16x2(byte == 255u ? byte : byte - 7u);
    lo.x = latent::mul_bf16x2(lo.x, r), lo.y = latent::mul_bf16x2(lo.y, r);
    lo.z = latent::mul_bf16x2(lo.z, r), lo.w = latent::mul_bf16x2(lo.w, r);
    hi.x = latent::mul_bf16x2(hi.x, r), hi.y = latent::mul_bf16x2(hi.y, r);
    hi.z = latent::mul_bf16x2(hi.z, r), hi.w = latent::mul_bf16x2(hi.w, r);
  }
  store_16(to, lo);
  store_16(to ^ 16u, hi);
}

// The pe channels of block b, and zeros behind the last channel, of tokens tok,
// tok + 2, tok + 32 and tok + 34: 16 lanes take a token's units of 8 channels.
__device__ __forceinline__ void copy_pe(const AttnParams& p, const int (&slot)[2 * kCodeTokens], int b, int tok,
                                        int lane, uint32_t stage) {
  const int unit = lane & 15, c = b * kBlock + 8 * unit;
  if (c < p.l.nope) return;
  const char* from = p.cache + (c < p.l.d ? p.l.nope + 2 * (c - p.l.nope) : 0);
#pragma unroll
  for (int k = 0; k < 2 * kCodeTokens; ++k) {
    const bool there = slot[k] >= 0 && c < p.l.d;
    LATENT_DBG_CHECK(g_latent_fault,
                     slot[k] < p.num_slots && tok + 2 + kCodeStep < kTile &&
                         (!there || p.l.nope + 2 * (c - p.l.nope) + 16 <= p.l.scale_off),
                     12);
    copy_16(unit_addr(stage, tok + 2 * (k & 1) + kCodeStep * (k >> 1), unit),
            from + static_cast<int64_t>(there ? slot[k] : 0) * p.l.row_bytes, there);
  }
}

__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// What a head's accumulators are multiplied by: 0 where nothing was attended to,
// NaN (0 / 0) where all scores were -inf.
__device__ __forceinline__ float inverse_of(float sum, float m) {
  if (sum != 0.f) return 1.f / sum;
  return m == -INFINITY ? 0.f : NAN;
}

// (These loads end with their own wait: a register moved or spilled between a
// load and a wait apart from it would be read too early.)
// 16 lanes x 64 columns of fp32: thread t holds rows t / 4 (r[4j], r[4j+1]) and
// t / 4 + 8 (r[4j+2], r[4j+3]) at columns 8 j + 2 (t % 4) and the next.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// 16 lanes x 32 columns, laid out over the warp alike.
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
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

// A condition that is the same on all lanes, as one the compiler knows to be.
__device__ __forceinline__ bool warp_any(bool x) { return __any_sync(0xFFFFFFFFu, x); }

// The first `channels` channels of a piece's queries into TMEM, by four warps:
// head h of the tile in lane 32 (h / 16) + h % 16, as S's row will be. `ready`
// waits for the products with the queries before, half of the loads in flight.
template <typename Ready>
__device__ __forceinline__ void put_queries(const AttnParams& p, const Piece& x, int channels, int quarter, int lane,
                                            uint32_t to, Ready ready) {
  const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;
  const int h = 16 * quarter + lane / 4;  // and h + 8
  const int chunks = (min(p.l.d, channels) + 63) / 64;
  const int h0 = x.head_tile * p.tile_heads, heads = min(p.tile_heads, p.nh - h0);
  LATENT_DBG_CHECK(g_latent_fault, x.row >= 0 && x.row < p.rows && heads > 0 && h0 + heads <= p.nh && p.l.d % 8 == 0, 13);
  const __nv_bfloat16* q = p.q + (x.row * p.nh + h0 + h) * p.l.d + 4 * (lane & 3);
  uint32_t r[2][16];
  const auto load = [&](int c0) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int u = 0; u < 8; ++u) {  // 16 channels (u / 2) of head h + 8 (u % 2)
        const int c = 64 * (c0 + i) + 16 * (u >> 1);
        uint2 v = make_uint2(0u, 0u);
        if (h + 8 * (u & 1) < heads && c + 4 * (lane & 3) < p.l.d && c0 + i < chunks)
          v = __ldg(reinterpret_cast<const uint2*>(q + 8 * (u & 1) * p.l.d + c));
        r[i][4 * (u >> 1) + 2 * (u & 1)] = v.x;
        r[i][4 * (u >> 1) + 2 * (u & 1) + 1] = v.y;
      }
  };
  const auto store = [&](int c0) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (c0 + i < chunks) tmem_st_16x32(to + 32 * (c0 + i) + lanes, r[i]);
  };
  load(0);
  ready();
  store(0);
  if (chunks > 2) {
    load(2);
    store(2);
  }
  ptx::tmem_st_wait();
  ptx::tc_fence_before();
  __syncwarp();
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
__global__ void __launch_bounds__(Cfg<E4M3>::kThreads, 1) latent_attn_kernel(const __grid_constant__ AttnParams p) {
  using C = Cfg<E4M3>;
  extern __shared__ __align__(1024) char smem[];
  const uint32_t base = ptx::smem_u32(smem);
  if (base & 1023u) {  // never: the declaration asks for it
    if (threadIdx.x == 0) {
      atomicCAS(&g_latent_fault, 0u, static_cast<unsigned>(kFaultSmem));
      if (p.split) p.split[blockIdx.x] = make_int4(0, 0, 0, 0);  // the join follows what stands there
    }
    return;
  }
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + kOffCtl);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  volatile int* abort_flag = &ctl->abort;
  const int nblk = (p.l.d + kBlock - 1) / kBlock;
  const auto bar = [](uint64_t& b) { return ptx::smem_u32(&b); };

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar(ctl->full[s]), E4M3 ? C::kLoadWarps / 2 : C::kLoadWarps * 32);
      ptx::mbar_init(bar(ctl->empty[s]), 1);
    }
    for (int i = 0; i < kSlotRing; ++i) {
      ptx::mbar_init(bar(ctl->slots_full[i]), 1);
      ptx::mbar_init(bar(ctl->slots_empty[i]), C::kLoadWarps);
    }
    ptx::mbar_init(bar(ctl->q_full), 4 + (nblk > kQueryBlocks ? 1 : 0));
    ptx::mbar_init(bar(ctl->q_empty), 2);
    ptx::mbar_init(bar(ctl->drained[2]), 1);
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(bar(ctl->s_full[k]), 1);
      ptx::mbar_init(bar(ctl->s_empty[k]), kSoftmaxThreads);
      ptx::mbar_init(bar(ctl->drained[k]), 1);
      ptx::mbar_init(bar(ctl->p_full[k]), kSoftmaxThreads);
      ptx::mbar_init(bar(ctl->o_done[k]), 1);
    }
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kScoreWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&ctl->tmem), kTmemCols);
    ptx::tmem_relinquish();
  }
  Walk w;
  int64_t total, nrun;
  find_run<C::kThreads>(p, ctl, &w, &total, &nrun);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  // All 512 columns are this block's, so the first is column 0: a constant to
  // the MMAs.
  constexpr uint32_t tmem = 0;
  if (ctl->tmem != tmem) {  // never
    if (tid == 0) atomicCAS(&g_latent_fault, 0u, static_cast<unsigned>(kFaultTmem));
    w.hi = w.at = 0;  // no tiles
  }
  Piece x;

  if (warp < kScoreWarp) {
    // ---------------------------------------------------------------- softmax and output
    const int hq = 16 * warp + lane / 4;  // this thread's heads: hq and hq + 8 of the tile
    const uint32_t lanes = static_cast<uint32_t>(warp) << 21;  // TMEM lane field, 32 * warp
    bool begun = false;  // a split row began in this block
    uint32_t g = 0;      // tiles so far
    uint32_t item = 0;   // rows with tiles whose queries this warp has brought
    while (w.next(p, x)) {
      const int h0 = x.head_tile * p.tile_heads;
      const int heads = min(p.tile_heads, p.nh - h0);
      float m[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
      if (E4M3 && x.j1 > x.j0) {
        // (the products with the queries before are in; but a warp of S that had no
        // tile of that row may not have looked at its phase of q_full yet)
        put_queries(p, x, kQueryBlocks * kBlock, warp, lane, tmem + kColQ, [&] {
          if (item > 0) wait_bar(bar(ctl->q_empty), (item - 1) & 1, abort_flag, kFaultQuery);
          ptx::tc_fence_after();
        });
        if (lane == 0) ptx::mbar_arrive(bar(ctl->q_full));
        ++item;
      }
      for (int j = x.j0; j < x.j1; ++j, ++g) {
        wait_bar(bar(ctl->s_full[g & 1]), (g >> 1) & 1, abort_flag, kFaultSoftmax);
        // the tile's mask was written before its stages were filled; they are
        // still full (only this tile's weights let them go)
        const uint32_t n0 = g * nblk;
        wait_bar(bar(ctl->full[n0 % kStages]), (n0 / kStages) & 1, abort_flag, kFaultSoftmax);
        ptx::tc_fence_after();
        uint32_t r[32];
        tmem_ld_16x64(tmem + kColS + (g & 1) * 64 + lanes, r);
        const uint64_t mask = ctl->mask[g % kMaskRing];
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(ctl->s_empty[g & 1]));
        float s[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) s[k] = __uint_as_float(r[k]) * p.scale_log2;
        if (~mask != 0) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {  // columns 8 u + 2 (lane % 4) and the next
            const uint32_t bits = static_cast<uint32_t>(mask >> (8 * u)) >> (2 * (lane & 3));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (!(bits >> (k & 1) & 1u)) s[4 * u + k] = -INFINITY;
          }
        }
        // A tile with a token that is attended to has a maximum above -inf even where
        // all its scores are -inf (their weights are 0 all the same): so m says
        // whether there was such a token, which a sum of 0 leaves open.
        const float least = mask != 0 ? -FLT_MAX : -INFINITY;
        float top[2] = {least, least};
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
        // the weights of two tiles before are read
        if (g >= 2) wait_bar(bar(ctl->o_done[g & 1]), ((g >> 1) - 1) & 1, abort_flag, kFaultSoftmax);
        const uint32_t pt = base + kOffP + (g & 1) * 8192u;
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float a = exp2_fast(s[4 * u + 2 * i] - ref[i]), b = exp2_fast(s[4 * u + 2 * i + 1] - ref[i]);
            sum[i] += a + b;
            const int h = hq + 8 * i;
            // the weights are rounded to bf16 here, as the second product's operand (of
            // the rows' type): O's relative error over a call is 0.0017 to 0.0021, of
            // which its own rounding is 0.0017; the sum, which lse needs, takes them as
            // they are
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
      LATENT_DBG_CHECK(g_latent_fault,
                       x.row >= 0 && x.row < p.rows && heads > 0 && x.j0 >= 0 && x.j1 <= x.nt &&
                           (whole || (p.part != nullptr && slot < 2 * static_cast<int64_t>(gridDim.x))),
                       14);
      if ((lane & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = hq + 8 * i;
          if (whole) {
            // not for a row without tiles: no barrier of a tile lies between this
            // and another warp's output of the row before, which reads inv
            if (x.j1 > x.j0) ctl->inv[h] = inverse_of(sum[i], m[i]);
            if (p.lse && h < heads)
              p.lse[out + h] = sum[i] == 0.f ? -INFINITY : (m[i] + log2f(sum[i])) * 0.6931471805599453f;
          } else if (h < heads) {
            p.part_ml[slot * p.tile_heads + h] = make_float2(m[i], sum[i]);
          }
        }
      }
      if (!whole && x.j0 == 0) {
        begun = true;
        if (tid == 0) {
          const int64_t first = x.at + kOverhead;
          const int64_t pieces = run_of(first + x.nt - 1, total, nrun) - run_of(first, total, nrun) + 1;
          LATENT_DBG_CHECK(g_latent_fault,
                           pieces > 1 && blockIdx.x + pieces <= gridDim.x &&
                               run_of(first, total, nrun) == static_cast<int64_t>(blockIdx.x),
                           15);
          p.split[blockIdx.x] = make_int4(static_cast<int>(pieces), static_cast<int>(x.row), x.head_tile, 0);
        }
      }
      ptx::named_bar_sync(1, kSoftmaxThreads);  // inv is written
      if (x.j1 > x.j0) {
        // the last tile's product (the one two before it is known to be in,
        // so the parity is of this phase or the one before)
        wait_bar(bar(ctl->o_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, abort_flag, kFaultSoftmax);
        ptx::tc_fence_after();
      }
      if (whole) {
        // two lanes swap a head each: a lane then stores two channels of one head
        const int odd = lane & 1;
        for (int b = 0; b < nblk; ++b) {
          const int c = b * kBlock + 32 * warp + lane - odd;
          __nv_bfloat16* to = p.O + (out + odd) * p.l.d + c;
          for (int h1 = 0; h1 < heads; h1 += 16, to += 16 * p.l.d) {
            uint32_t v[16] = {};
            if (x.j1 > x.j0) tmem_ld_x16(tmem + lanes + b * 64 + h1, v);
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float2 f = make_float2(0.f, 0.f);
              if (x.j1 > x.j0) f = *reinterpret_cast<const float2*>(ctl->inv + h1 + 2 * k);
              const float even_h = __uint_as_float(v[2 * k]) * f.x, odd_h = __uint_as_float(v[2 * k + 1]) * f.y;
              const float give = odd ? even_h : odd_h, keep = odd ? odd_h : even_h;
              const float got = __shfl_xor_sync(0xFFFFFFFFu, give, 1);
              o[k] = odd ? ptx::pack_bf16x2(got, keep) : ptx::pack_bf16x2(keep, got);
            }
            if (c < p.l.d) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (h1 + 2 * k + odd < heads) *reinterpret_cast<uint32_t*>(to + 2 * k * p.l.d) = o[k];
            }
            __syncwarp();
          }
        }
      } else {
        for (int b = 0; b < nblk; ++b) {
          const int c = b * kBlock + 32 * warp + lane;
          float* to = p.part + slot * p.tile_heads * p.l.d + c;
          for (int h1 = 0; h1 < p.tile_heads; h1 += 16, to += 16 * p.l.d) {
            uint32_t v[16];
            tmem_ld_x16(tmem + lanes + b * 64 + h1, v);
            if (c < p.l.d) {
#pragma unroll
              for (int k = 0; k < 16; ++k) to[k * p.l.d] = __uint_as_float(v[k]);
            }
            __syncwarp();
          }
        }
      }
      ptx::tc_fence_before();  // the next row's products overwrite O^T after this thread's next weights
    }
    if (!begun && tid == 0 && p.split) p.split[blockIdx.x] = make_int4(0, 0, 0, 0);
  } else if (warp < kValueWarp) {
    // ---------------------------------------------------------------- S
    // The whole warp walks, every branch around the products is on a vote, TMEM
    // columns are constants and no call comes between: so operands stay in
    // uniform registers, where an MMA takes them from (moving them there took
    // 60-130 cycles an MMA, against 33 and 49 of the tensor core for S and O^T).
    const uint32_t id_s = ptx::idesc_bf16_f32(64, kTile, false, false);
    // operands' descriptors, to which address steps (in 16-byte units) are added
    const uint64_t q_desc = ptx::smem_desc_sw128(base, 16, 1024);
    const uint64_t c_desc = ptx::smem_desc_sw128(base + kOffRing, 16, 1024);
    const int chunks = (p.l.d - kQueryBlocks * kBlock + 63) / 64;
    const bool even = (p.l.d + 63) / 64 % 2 == 0;  // the last block has both its 64-channel halves
    const uint32_t mine = warp - kScoreWarp;  // tiles g with g % 2 == mine
    uint32_t g = 0, item = 0;
    while (warp_any(w.next(p, x))) {
      if (!warp_any(x.j1 > x.j0)) continue;
      if (mine == 0) {
        if (item > 0) wait_bar_here(bar(ctl->q_empty), (item - 1) & 1, abort_flag, kFaultScore);
        // the channels that TMEM has no room for (after a wait that ran out nothing
        // is begun that could land when the block has left)
        if (nblk > kQueryBlocks && !warp_any(*abort_flag != 0) && ptx::elect_one()) {
          ptx::mbar_arrive_expect_tx(bar(ctl->q_full), chunks * p.tile_heads * 128);
          for (int c = 0; c < chunks; ++c)
            ptx::tma_load_3d(base + c * 8192u, &p.tm_q, kQueryBlocks * kBlock + c * 64,
                             x.head_tile * p.tile_heads, static_cast<int>(x.row), bar(ctl->q_full));
        }
      }
      __syncwarp();
      wait_bar_here(bar(ctl->q_full), item & 1, abort_flag, kFaultScore);
      for (int j = x.j0; warp_any(j < x.j1); ++j, ++g) {
        if ((g & 1) != mine) continue;
        if (g >= 2) wait_bar_here(bar(ctl->s_empty[g & 1]), ((g >> 1) - 1) & 1, abort_flag, kFaultScore);
        const uint32_t ds = kColS + mine * 64, n0 = g * nblk;
        uint32_t s = n0 % kStages, phase = n0 / kStages & 1;
#pragma unroll 1
        for (int b = 0; b < nblk; ++b) {
          wait_bar_here(bar(ctl->full[s]), phase, abort_flag, kFaultScore);
          ptx::fence_proxy_async_smem();
          ptx::tc_fence_after();
          LATENT_DBG_CHECK(g_latent_fault, s < kStages && b < kMaxBlocks, 16);
          const uint64_t cd = c_desc + s * (kStageBytes >> 4);
          const bool two = b < nblk - 1 || even;  // 64-channel halves
          if (ptx::elect_one()) {
            if (b < kQueryBlocks) {
              const uint32_t qt = kColQ + 64 * b;
#pragma unroll
              for (int i = 0; i < 4; ++i) ptx::tc_mma_ts(ds, qt + 8 * i, cd + 2 * i, id_s, i + b > 0);
              if (two) {
#pragma unroll
                for (int i = 0; i < 4; ++i) ptx::tc_mma_ts(ds, qt + 32 + 8 * i, cd + (kHalf >> 4) + 2 * i, id_s, 1);
              }
            } else {
              const uint64_t qd = q_desc + (b - kQueryBlocks) * (16384 >> 4);
#pragma unroll
              for (int i = 0; i < 4; ++i) ptx::tc_mma_ss(ds, qd + 2 * i, cd + 2 * i, id_s, i + b > 0);
              if (two) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  ptx::tc_mma_ss(ds, qd + (8192 >> 4) + 2 * i, cd + (kHalf >> 4) + 2 * i, id_s, 1);
              }
            }
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (ptx::elect_one()) ptx::tc_commit(bar(ctl->s_full[mine]));
        __syncwarp();
      }
      if (ptx::elect_one()) ptx::tc_commit(bar(ctl->q_empty));  // this warp's products with these queries
      __syncwarp();
      ++item;
    }
    // nothing may be in flight when the thread block leaves
    if (item > 0 && nblk > kQueryBlocks) wait_bar_noabort(bar(ctl->q_full), (item - 1) & 1);
    if (ptx::elect_one()) ptx::tc_commit(bar(ctl->drained[mine]));
    __syncwarp();
    wait_bar_noabort(bar(ctl->drained[mine]), 0);
    __syncwarp();
  } else if (warp == kValueWarp) {
    // ---------------------------------------------------------------- O^T += C^T P^T
    const uint32_t id_o = ptx::idesc_bf16_f32(128, p.tile_heads, true, false);
    const uint64_t c_desc = ptx::smem_desc_sw128(base + kOffRing, kHalf, 1024);
    const uint64_t p_desc = ptx::smem_desc_sw128(base + kOffP, 16, 1024);
    uint32_t g = 0, s = 0;
    while (warp_any(w.next(p, x))) {
      bool first = true;
      for (int j = x.j0; warp_any(j < x.j1); ++j, ++g, first = false) {
        wait_bar_here(bar(ctl->p_full[g & 1]), (g >> 1) & 1, abort_flag, kFaultValue);
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_after();
        const uint64_t pd = p_desc + (g & 1) * (8192u >> 4);
#pragma unroll 1
        for (int b = 0; b < nblk; ++b) {
          LATENT_DBG_CHECK(g_latent_fault, s < kStages && b < kMaxBlocks, 17);
          const uint64_t cd = c_desc + s * (kStageBytes >> 4);
          if (ptx::elect_one()) {
            ptx::tc_mma_ss(b * 64, cd, pd, id_o, !first);
#pragma unroll
            for (int k = 1; k < kTile / 16; ++k)
              ptx::tc_mma_ss(b * 64, cd + k * (2048 >> 4), pd + k * (32 >> 4), id_o, 1);
            ptx::tc_commit(bar(ctl->empty[s]));
            if (b == nblk - 1) ptx::tc_commit(bar(ctl->o_done[g & 1]));
          }
          __syncwarp();
          if (++s == kStages) s = 0;
        }
      }
    }
    if (ptx::elect_one()) ptx::tc_commit(bar(ctl->drained[2]));
    __syncwarp();
    wait_bar_noabort(bar(ctl->drained[2]), 0);
    __syncwarp();
  } else if (warp == kTokenWarp) {
    // ---------------------------------------------------------------- slots and masks
    // A lane takes tokens lane and lane + 32 of each tile; table entries are
    // loaded one tile ahead.
    uint32_t g = 0;
    int tile = 0, end = 0, ntok = 0;
    Ref ref[2];
    const auto look_up = [&]() {
      while (tile == end) {
        if (!w.next(p, x)) return false;
        tile = x.j0;
        end = x.j1;
        ntok = tokens_of(p, x.row);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = tile * kTile + lane + 32 * k;
        ref[k] = t < ntok ? ref_of(p, x.row, t) : Ref{-1, 0};
      }
      ++tile;
      return true;
    };
    bool live = look_up(), marked = false;
    for (bool ok = true; ok && !marked; ++g) {
      const int s0 = live ? slot_of(p, ref[0]) : kNoTile, s1 = live ? slot_of(p, ref[1]) : kNoTile;
      const bool more = live && look_up();
      const uint32_t i = g % kSlotRing;
      if (g >= kSlotRing) ok = wait_bar(bar(ctl->slots_empty[i]), (g / kSlotRing - 1) & 1, abort_flag, kFaultToken);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      ctl->slot[i][lane] = s0;
      ctl->slot[i][lane + 32] = s1;
      const uint32_t lo = __ballot_sync(0xFFFFFFFFu, s0 >= 0), hi = __ballot_sync(0xFFFFFFFFu, s1 >= 0);
      if (lane == 0 && live) ctl->mask[g % kMaskRing] = lo | static_cast<uint64_t>(hi) << 32;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(ctl->slots_full[i]));
      marked = !live;  // behind the last tile, the mark that there is none
      live = more;
    }
  } else if (!E4M3 && warp < C::kLoadWarp) {
    // ---------------------------------------------------------------- queries
    uint32_t item = 0;
    while (w.next(p, x)) {
      if (x.j1 == x.j0) continue;
      put_queries(p, x, kQueryBlocks * kBlock, warp - C::kQueryWarp, lane, tmem + kColQ, [&] {
        if (item > 0) wait_bar(bar(ctl->q_empty), (item - 1) & 1, abort_flag, kFaultQuery);
        ptx::tc_fence_after();
      });
      if (lane == 0) ptx::mbar_arrive(bar(ctl->q_full));
      ++item;
    }
  } else {
    // ---------------------------------------------------------------- cache rows
    const int v = warp - C::kLoadWarp;
    uint32_t g = 0, s = 0, phase = 1;  // tiles looked up; stage, and the phase of `empty` that lets it be filled
    bool ok = true;
    // The slots of the next tile, read with `take`; false behind the last.
    const auto next_slots = [&](auto take) {
      const uint32_t i = g % kSlotRing;
      ok = __all_sync(0xFFFFFFFFu, wait_bar(bar(ctl->slots_full[i]), (g / kSlotRing) & 1, abort_flag, kFaultLoad));
      const int* slots = ctl->slot[i];
      const bool some = slots[0] != kNoTile;
      take(slots);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(ctl->slots_empty[i]));
      ++g;
      return ok && some;
    };
    const auto next_stage = [&] {
      if (++s == kStages) {
        s = 0;
        phase ^= 1;
      }
    };
    const auto wait_stage = [&] {
      ok = __all_sync(0xFFFFFFFFu, wait_bar(bar(ctl->empty[s]), phase, abort_flag, kFaultLoad));
      return ok;
    };
    if (!E4M3) {
      const int tok = 8 * v + (lane >> 4);
      int slot[4];
      while (next_slots([&](const int* slots) {
        for (int k = 0; k < 4; ++k) slot[k] = slots[tok + 2 * k];
      })) {
        for (int b = 0; b < nblk; ++b) {
          if (!wait_stage()) break;
          LATENT_DBG_CHECK(g_latent_fault, s < kStages, 18);
          copy_block(p, slot, b, tok, lane, base + kOffRing + s * kStageBytes);
          copies_arrive(bar(ctl->full[s]));
          next_stage();
        }
        if (!ok) break;
      }
    } else {
      const int odd = v & 1, tok = 4 * (v >> 1) + 2 * (lane >> 4) + (lane >> 2 & 1);
      const int item = (lane >> 1 & 4) | (lane & 3);
      const uint32_t off = unit_addr(0, tok, 2 * item);
      // where codes and scales land: in a block of codes alone, in order
      const auto land = [&](int b) {
        return (b + 1) * kBlock > p.l.nope ? off : tok * 128 + ((item ^ (tok & 1) << 2) << 4);
      };
      const auto land_scales = [&](int b) {
        return (b + 1) * kBlock > p.l.nope ? unit_addr(0, tok, 1) : kHalf + tok * 128 + ((tok & 7) << 4);
      };
      const int mine = (nblk - odd + 1) / 2;  // blocks of a tile that are this warp's
      int slot[kCodeTokens];
      int next = mine, oldest = 0;      // of a tile's blocks: the next to be copied, the oldest in flight
      uint32_t tile = 0, s_out = 0, pending = 0;
      bool more = true;
      for (;;) {
        while (more && pending < kCodesAhead) {
          if (next == mine) {
            if (tile++ > 0) {
              s += nblk;
              if (s >= kStages) {
                s -= kStages;
                phase ^= 1;
              }
            }
            more = next_slots([&](const int* slots) {
#pragma unroll
              for (int k = 0; k < kCodeTokens; ++k) slot[k] = slots[tok + kCodeStep * k];
            });
            next = 0;
            continue;
          }
          const int b = 2 * next + odd;
          const bool wrap = s + b >= kStages;
          const uint32_t at = wrap ? s + b - kStages : s + b, ph = wrap ? phase ^ 1 : phase;
          if (pending > 0) {  // if it is not free yet, the blocks in flight come first
            if (!__all_sync(0xFFFFFFFFu, ptx::mbar_test_wait(bar(ctl->empty[at]), ph))) break;
          } else {
            ok = __all_sync(0xFFFFFFFFu, wait_bar(bar(ctl->empty[at]), ph, abort_flag, kFaultLoad));
            if (!ok) break;
          }
          LATENT_DBG_CHECK(g_latent_fault, at < kStages && b < nblk, 18);
          const uint32_t stage = base + kOffRing + at * kStageBytes;
          copy_codes(p, slot, b, item, stage + land(b), stage + land_scales(b));
          if ((b + 1) * kBlock > p.l.nope) {
            int pe_slot[2 * kCodeTokens];
#pragma unroll
            for (int k = 0; k < 2 * kCodeTokens; ++k)
              pe_slot[k] = __shfl_sync(0xFFFFFFFFu, slot[k >> 1], 16 * (k & 1) + 4 * (lane >> 4));
            copy_pe(p, pe_slot, b, 4 * (v >> 1) + (lane >> 4), lane, stage);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          ++next;
          ++pending;
        }
        if (!ok || pending == 0) break;
        if (pending == 1)
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        else
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();  // the scales are another lane's copy
        const int b = 2 * oldest + odd;
        const uint32_t at = s_out + b >= kStages ? s_out + b - kStages : s_out + b;
        LATENT_DBG_CHECK(g_latent_fault, at < kStages && b < nblk, 19);
        const uint32_t to = base + kOffRing + at * kStageBytes;
        if (b * kBlock < p.l.nope) {
          const bool codes = b * kBlock + 16 * item < p.l.nope;
          uint4 w[kCodeTokens];
          uint32_t byte[kCodeTokens];
#pragma unroll
          for (int k = 0; k < kCodeTokens; ++k) {
            w[k] = load_16(to + land(b) + k * kCodeStep * 128);
            byte[k] = load_byte(to + land_scales(b) + k * kCodeStep * 128 + 2 * b + (item >> 2));
          }
          __syncwarp();  // all have read them
          if (codes) {
#pragma unroll
            for (int k = 0; k < kCodeTokens; ++k) store_codes(w[k], byte[k], to + off + k * kCodeStep * 128);
          }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(ctl->full[at]));
        --pending;
        if (++oldest == mine) {
          oldest = 0;
          s_out += nblk;
          if (s_out >= kStages) s_out -= kStages;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // nothing lands after the block has left
  }

  // ------------------------------------------------------------------ teardown
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kScoreWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// Adds up the partials of the rows that were split, in the order of their
// tiles: O = sum_k w_k part_k / sum_k w_k sum_k, w_k = 2^(reference_k - the
// largest). A warp takes a (row, head), 4 x 128 channels; with few of them (a
// long row over many runs) a block takes 128 channels of one, a warp every
// eighth partial. All reads of a step are in flight at once: the time is a few
// L2 latencies, 8 us behind 32 ragged rows (one block a head with its loads in
// turn took 20-40 us; weights computed beside the partials' loads 1 us more).
constexpr int kJoinWarps = 8;
constexpr int kMaxRuns = 256;

struct JoinParams {
  const float* part;
  const float2* part_ml;
  const int4* split;
  __nv_bfloat16* O;
  float* lse;
  int runs, nh, tile_heads, d;
};

__global__ void __launch_bounds__(32 * kJoinWarps, 4) latent_join_kernel(JoinParams p) {
  __shared__ int4 todo[kMaxRuns];  // (pieces, row, head tile, first run) of the split rows
  __shared__ int count[kJoinWarps];
  __shared__ float4 sums[kJoinWarps][32];
  __shared__ float weight[kJoinWarps][kMaxRuns];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  // Launched early: wait for the partials. (They are read with plain loads: the
  // read-only path is for what does not change while this kernel runs.)
  ptx::griddep_wait();
  int n = 0;
  for (int c0 = 0; c0 < p.runs; c0 += 32 * kJoinWarps) {
    const int c = c0 + tid;
    int4 e = make_int4(0, 0, 0, 0);
    if (c < p.runs) e = p.split[c];
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, e.x > 0);
    if (lane == 0) count[warp] = __popc(some);
    __syncthreads();
    int at = n;
    for (int k = 0; k < kJoinWarps; ++k) {
      if (k < warp) at += count[k];
      n += count[k];
    }
    if (e.x > 0) {
      LATENT_DBG_CHECK(g_latent_fault, c + e.x <= p.runs && e.x <= kMaxRuns, 20);
      e.w = c;
      const int k = at + __popc(some & ((1u << lane) - 1u));
      LATENT_DBG_CHECK(g_latent_fault, k < kMaxRuns, 21);
      todo[k] = e;
    }
    __syncthreads();
  }
  const int heads = n * p.tile_heads, quarters = (p.d + 127) / 128;
  const bool wide = heads * quarters <= static_cast<int>(gridDim.x);  // a block to a quarter of a head
  const int units = wide ? heads * quarters : heads;
  const int per = wide ? 1 : kJoinWarps;
  for (int u0 = blockIdx.x * per; u0 < units; u0 += gridDim.x * per) {
    const int u = wide ? u0 : u0 + warp;
    const int unit = wide ? u / quarters : u, q0 = wide ? u - unit * quarters : 0, q1 = wide ? q0 + 1 : quarters;
    const int4 e = u < units ? todo[unit / p.tile_heads] : make_int4(0, 0, 0, 0);
    const int h = unit % p.tile_heads, head = e.z * p.tile_heads + h;
    const bool live = u < units && head < p.nh;
    const int pieces = live ? e.x : 0;
    LATENT_DBG_CHECK(g_latent_fault, !live || (pieces > 1 && unit / p.tile_heads < n && e.y >= 0), 22);
    const auto slot = [&](int k) {
      return static_cast<int64_t>(k == 0 ? 2 * e.w : 2 * (e.w + k) + 1) * p.tile_heads + h;
    };
    float2 ml[kMaxRuns / 32];
    float top = -INFINITY, sum = 0.f;
    if (pieces <= 32) {
      ml[0] = make_float2(-INFINITY, 0.f);
      if (lane < pieces) ml[0] = p.part_ml[slot(lane)];
      top = ml[0].x;
    } else {
#pragma unroll
      for (int i = 0; i < kMaxRuns / 32; ++i) {
        ml[i] = make_float2(-INFINITY, 0.f);
        if (lane + 32 * i < pieces) ml[i] = p.part_ml[slot(lane + 32 * i)];
      }
#pragma unroll
      for (int i = 0; i < kMaxRuns / 32; ++i) top = fmaxf(top, ml[i].x);
    }
    for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int i = 0; i < kMaxRuns / 32; ++i) {
      if (32 * i >= pieces) break;
      const float w = exp2_fast(ml[i].x - ref);
      sum += w * ml[i].y;
      weight[warp][lane + 32 * i] = w;
    }
    for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    __syncwarp();
    const float inv = inverse_of(sum, top);
    const int64_t out = static_cast<int64_t>(e.y) * p.nh + head;
    // partials k0, k0 + step, ... of channels 128 q + 4 lane and on
    const auto add = [&](float4& acc, int k0, int step, int q) {
      const int c = 128 * q + 4 * lane;
#pragma unroll 8
      for (int k = k0; k < pieces; k += step) {
        const float w = weight[warp][k];
        if (c < p.d) {
          const float4 v = *reinterpret_cast<const float4*>(p.part + slot(k) * p.d + c);
          acc.x += w * v.x;
          acc.y += w * v.y;
          acc.z += w * v.z;
          acc.w += w * v.w;
        }
      }
    };
    const auto store = [&](const float4& acc, int q) {
      const int c = 128 * q + 4 * lane;
      if (live && c < p.d) {
        uint2 o;
        o.x = ptx::pack_bf16x2(acc.x * inv, acc.y * inv);
        o.y = ptx::pack_bf16x2(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(p.O + out * p.d + c) = o;
      }
    };
    if (wide) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      add(acc, warp, kJoinWarps, q0);
      sums[warp][lane] = acc;
      __syncthreads();
      if (warp == 0) {
        for (int k = 1; k < kJoinWarps; ++k) {
          const float4 v = sums[k][lane];
          acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
        store(acc, q0);
      }
      __syncthreads();
    } else {
      float4 acc[kMaxBlocks] = {};
#pragma unroll 4
      for (int k = 0; k < pieces; ++k) {
        const float w = weight[warp][k];
#pragma unroll
        for (int q = 0; q < kMaxBlocks; ++q) {
          const int c = 128 * q + 4 * lane;
          if (c < p.d) {
            const float4 v = *reinterpret_cast<const float4*>(p.part + slot(k) * p.d + c);
            acc[q].x += w * v.x;
            acc[q].y += w * v.y;
            acc[q].z += w * v.z;
            acc[q].w += w * v.w;
          }
        }
      }
#pragma unroll
      for (int q = 0; q < kMaxBlocks; ++q)
        if (q < q1) store(acc[q], q);
    }
    __syncwarp();  // the weights are read
    if (live && p.lse && lane == 0 && q0 == 0 && (!wide || warp == 0))
      p.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
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

constexpr double kLog2e = 1.4426950408889634;

// Sizes of a call that are checked before anything else.
int check_shape(int64_t rows, int nh, int64_t max_tokens, double scale) {
  // (the kernel has scale * log2(e) in fp32; NaN fails the comparison too)
  if (rows < 0 || nh < 1 || max_tokens < 0 || !(std::fabs(scale) * kLog2e <= FLT_MAX)) return INVROPE_ERR_INVALID_ARG;
  if (nh > 128 || rows > 0x7FFFFFFF / nh || max_tokens > 0x7FFFFFFF) return INVROPE_ERR_UNSUPPORTED;
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
  // of the workspace, what any device with at least two thread blocks uses; below,
  // what this one does
  Range out[] = {{p.O, vec}, {p.lse, p.lse ? heads * 4 : 0},
                 {workspace, workspace ? make_plan(p.rows, p.nh, max_tokens, p.l.d, 2).bytes : 0}};
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
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.head_tiles = n.head_tiles;
  p.tile_heads = n.tile_heads;
  if (!opt_in_smem(dev.device) || !query_map(&p.tm_q, q, p.rows, p.nh, p.l.d, n.tile_heads)) return INVROPE_ERR_CUDA;
  if (fmt == KV_LATENT_E4M3)
    latent_attn_kernel<true><<<n.grid, Cfg<true>::kThreads, kSmem, s>>>(p);
  else
    latent_attn_kernel<false><<<n.grid, Cfg<false>::kThreads, kSmem, s>>>(p);
  if ((st = check_launch()) != INVROPE_OK || n.bytes == 0) return st;
  // programmatic dependent launch: the join's launch is processed while the
  // attention drains; its blocks wait in-kernel for the partials
  const JoinParams jp{p.part, p.part_ml, p.split, p.O, p.lse, n.grid, p.nh, n.tile_heads, p.l.d};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(dev.sms * 4));
  cfg.blockDim = dim3(32 * kJoinWarps);
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
                  int64_t rows, int64_t width, int num_pages, int page_size, int nh, double scale) {
  AttnParams p = {};
  p.cache = static_cast<const char*>(cache);
  p.table = table;
  p.lens = lens;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  p.rows = rows;
  p.width = width;
  p.num_slots = static_cast<int64_t>(num_pages) * page_size;
  p.num_pages = num_pages;
  p.nh = nh;
  p.page_size = page_size;
  p.scale_log2 = static_cast<float>(scale * kLog2e);
  p.l = l;
  return p;
}

}  // namespace

#ifdef INVROPE_DEBUG_BOUNDS
int take_cache_fault(unsigned int* code);  // latent_cache.cu

namespace {

// One thread waits in each of the ways of the roles for a barrier that nothing
// arrives on; a second one then finds the abort flag set and does not wait.
// done[0] counts the waits that came back, done[1] those that said so.
__global__ void wait_selftest_kernel(int which, int* done) {
  __shared__ __align__(8) uint64_t never;
  __shared__ int abort_flag;
  const uint32_t bar = ptx::smem_u32(&never);
  ptx::mbar_init(bar, 1);
  abort_flag = 0;
  ptx::fence_mbar_init();
  for (int k = 0; k < 2; ++k) {
    if (which == 0) {
      done[1] += wait_bar(bar, 0, &abort_flag, kFaultLoad) ? 0 : 1;
    } else if (which == 1) {
      wait_bar_here(bar, 0, &abort_flag, kFaultScore);
      done[1] += abort_flag;
    } else if (k == 0) {
      wait_bar_noabort(bar, 0);
    }
    done[0] += 1;
  }
}

}  // namespace
#endif

int take_latent_fault(unsigned int* code) {
  cudaError_t err = cudaMemcpyFromSymbol(code, g_latent_fault, sizeof(*code));
  if (err != cudaSuccess) return cuda_fail(err);
  const unsigned int zero = 0;
  if ((err = cudaMemcpyToSymbol(g_latent_fault, &zero, sizeof(zero))) != cudaSuccess) return cuda_fail(err);
#ifdef INVROPE_DEBUG_BOUNDS
  unsigned int cache = 0;
  const int st = take_cache_fault(&cache);
  if (st != INVROPE_OK) return st;
  if (*code == 0) *code = cache;
#endif
  return INVROPE_OK;
}

}  // namespace invrope

using namespace invrope;

#ifdef INVROPE_DEBUG_BOUNDS
// Test hook of the debug-bounds build: lets a wait of the attention's roles run
// out (`which`: 0 wait_bar, 1 wait_bar_here, 2 wait_bar_noabort; about 2 s);
// done[2] as above, in host memory. The fault word then holds the wait's code
// (none for 2).
extern "C" int latent_debug_wait(int which, int* done) {
  if (which < 0 || which > 2 || !done) return INVROPE_ERR_INVALID_ARG;
  int* d = nullptr;
  cudaError_t err = cudaMalloc(&d, 2 * sizeof(int));
  if (err != cudaSuccess) return cuda_fail(err);
  if ((err = cudaMemset(d, 0, 2 * sizeof(int))) == cudaSuccess) {
    wait_selftest_kernel<<<1, 1>>>(which, d);
    if ((err = cudaGetLastError()) == cudaSuccess)
      err = cudaMemcpy(done, d, 2 * sizeof(int), cudaMemcpyDeviceToHost);
  }
  cudaFree(d);
  return err == cudaSuccess ? INVROPE_OK : cuda_fail(err);
}
#endif

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
  AttnParams p = params(l, cache, page_table, lens, O, lse, rows, max_pages, static_cast<int>(num_pages), page_size, nh,
                        scale);
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
  AttnParams p = params(l, cache, idx, nullptr, O, lse, rows, topk, static_cast<int>(num_slots), 1, nh, scale);
  return attend(p, q, workspace, workspace_bytes, fmt, topk, reinterpret_cast<cudaStream_t>(stream));
}
