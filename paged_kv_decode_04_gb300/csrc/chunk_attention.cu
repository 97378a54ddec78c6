// chunk_attention.cu -- attention of a ragged batch of new tokens over the
// paged cache under a causal mask, a sliding window and sink tokens, on the
// fifth-generation tensor cores (tcgen05, accumulators in TMEM).
//
// A query at position p sees token t when t <= p and (t > p - window or
// t < sinks).  A tile is up to 64 consecutive new tokens of one sequence; for
// one kv head their 4 query heads each make 256 rows (row = 4 token + head),
// two MMA row tiles of 128, which share every K/V row that is loaded.  The
// cached tokens come in tiles of 128 (8 pages).  Per row tile and kv tile
//
//   S = Q K^T   (128 x 128, 4 MMAs of K = 16; Q and K rows in shared memory)
//   P = 2^(c S - m), the FP32 online softmax, one thread per row
//   O += P V    (128 x 64, 8 MMAs of K = 16; P in TMEM, V rows in shared)
//
// A tile of at most 32 tokens has one row tile only; the two softmax warp
// groups then take the even and the odd kv tiles of the same rows, and their
// states are joined at the end like two ranges.
//
// TMEM (512 columns): S of row tile / group w at 128 w, P at 256 + 64 w, O at
// 384 + 64 w.  P does not lie over S, so S of the next kv tile is computed
// while this one's exponentials are taken.
//
// Warps, one persistent CTA per SM, each role walking the CTA's items (tile,
// kv head, range of the kv tiles) and handing over through mbarriers, so the
// next item's loads and first products run under the last one's epilogue:
//   0-3, 4-7  softmax of S_0 and S_1, rescaling of O, epilogue
//   8, 11     issue QK and PV.  A unit is a (row tile, kv tile) pair; units
//             alternate between S_0 and S_1, across items too
//   9         loads: Q by one box per row tile, K and V by 2 KiB boxes of one
//             page and head; pages outside every row's sight (or with a bad
//             id) are read at a page index past the pool, i.e. as zeros
//   10        finds the CTA's next items from the offsets and lengths (items
//             without any kv tile it answers itself), and relays "V has
//             landed": in the tiles that some row sees in part only it first
//             replaces non-finite V values by zero (a masked weight is zero,
//             but 0 x NaN is not); rows that do see such a value get it added
//             in the epilogue
// Measured on 2 x 4096 tokens over 8192 (391 GFLOP): 354 us, 1.10 PFLOP/s, 0.59
// of the card's cuBLAS bf16 rate.  A unit takes 1060 cycles of an SM, of which
// its MMAs fill 440 and its exponentials 546 (30 a clock), the rest being the
// latencies of the chain scores -> registers -> P -> PV; the two groups' chains
// overlap, but two warps to a scheduler do not hide them all.  What moved it:
//  * the issue of QK and PV by two warps (680 -> 567 us): the issuing warps'
//    instruction streams are slow next to the softmax (they share the
//    schedulers' instruction caches), and one warp for both took 1400 cycles a
//    unit;
//  * no register spills in the softmax (567 -> 449 us): the epilogue runs in
//    16-column steps, and what the loop needs of an item it reads again;
//  * one elected lane for the copies of a kv tile, and no maximum per tile
//    (449 -> 413 us);
//  * the exponentials of a unit as one straight block, its weights stored in
//    two parts of 64 columns and the wait for the group's last PV before it
//    (412 -> 356 us; four parts of 32 with the wait after the first part left
//    the compiler short of registers, and all 64 words stored at the end cost
//    451 us);
//  * the relay of V scans only the pages that some row does not see (a prompt
//    of 8192 under a window of 1024: 109 -> 104 us then);
//  * not: 16 softmax warps of half a row each (558 us: twice the hand-over
//    instructions), four groups of 128 x 64 units with P over S (485 us: twice
//    the units for the issuing warps), the row in two rolled halves with S given
//    back at the end (484 us), four more warps for the epilogue (402 us: fewer
//    registers for every role), scalar instead of packed FP32 (493 us), skipping
//    32-column steps that no row sees (463 us: no overlap between steps).
// P enters the product with V as bf16 (8 significant bits, an error of at
// most 2^-8 of sum p |v|, averaged over the tokens, below the output's own
// bf16 rounding); the row sums take the unrounded FP32 values.  The reference
// maximum m is the first tile's and moves only when a tile's weights sum to
// 2^16, so the other tiles take one pass over their scores and no maximum.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kQTokens = kChunkTileTokens;    // 64 tokens a tile
constexpr int kHalfTokens = kQTokens / 2;     // 32 tokens: one MMA row tile
constexpr int kKvTokens = kChunkKvTokens;     // 128 cached tokens a kv tile
constexpr int kKvPages = kKvTokens / kPageSize;
constexpr int kRow = kHeadDim * 2;            // 128 B
constexpr int kRowTileBytes = 128 * kRow;     // 16 KiB: a row tile of Q, a kv tile of K or V
constexpr int kPageBytes = kPageSize * kRow;  // 2 KiB: one head's K (or V) rows of a page
constexpr int kStages = 4;                    // kv tiles in flight
constexpr int kItems = 8;                     // slots for published items
constexpr int kAhead = 3;                     // items published before the relay starts one
constexpr int kSoftmaxWarps = 8;
constexpr int kQkWarp = 8, kLoadWarp = 9, kSchedWarp = 10;  // and 11 issues PV
constexpr int kThreads = 32 * 12;
// Registers: 168 x 384 threads at launch = 64512 = 256 x 200 + 128 x 104.
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 200, kOtherRegs = 104;
static_assert(kSoftmaxRegs * 256 + kOtherRegs * 128 <= kLaunchRegs * kThreads,
              "the split stays within the registers the block starts with");
constexpr float kRescale = 65536.f;  // 2^16

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemP = 256, kTmemO = 384;
constexpr uint32_t kIdescQK = tc_idesc_bf16(128, kKvTokens, false);
constexpr uint32_t kIdescPV = tc_idesc_bf16(128, kHeadDim, true);

// Shared memory, from a 1024-byte aligned base.
constexpr int kOffQ = 0;                               // [2 items][2 row tiles]
constexpr int kOffK = kOffQ + 4 * kRowTileBytes;
constexpr int kOffV = kOffK + kStages * kRowTileBytes;
constexpr int kOffOut = kOffV + kStages * kRowTileBytes;  // [warp][32 rows] of 128 B
constexpr int kOutBytes = 32 * 128;
constexpr int kOffMl = kOffOut + kSoftmaxWarps * kOutBytes;  // [128] (m, l) handed between groups
constexpr int kOffItems = kOffMl + 128 * 8;
constexpr int kItemWords = 16;
constexpr int kOffBars = kOffItems + kItems * kItemWords * 4;
enum {
  kBarKFull = 0,
  kBarKEmpty = kBarKFull + kStages,
  kBarVFull = kBarKEmpty + kStages,
  kBarVReady = kBarVFull + kStages,
  kBarVEmpty = kBarVReady + kStages,
  kBarQFull = kBarVEmpty + kStages,
  kBarQEmpty = kBarQFull + 2,
  kBarSFull = kBarQEmpty + 2,
  kBarSFree = kBarSFull + 2,
  kBarPFull = kBarSFree + 2,
  kBarPvDone = kBarPFull + 2,
  kBarItemFull = kBarPvDone + 2,
  kBarItemEmpty = kBarItemFull + kItems,
  kBarXFull = kBarItemEmpty + kItems,
  kBarXFree,
  kBarQkFin,
  kBarPvFin,
  kNumBars
};
// The loader's notes on the last kv tiles (place in the sequence; bits of bad
// pages, and kPartial), then the TMEM address.  Twice the stages: while a
// softmax group reads kv tile j's, QK(j + 2) has not been issued, so the loads
// are at tile j + 1 + kStages at most.
constexpr int kMeta = 2 * kStages;
constexpr uint32_t kPartial = 0x100;  // some row does not see some token
constexpr int kOffMeta = kOffBars + 8 * kNumBars;
constexpr int kSmem = 1024 + kOffMeta + 4 * (2 * kMeta + 4);
static_assert(kSmem <= 227 * 1024, "fits one CTA");

// One item as the roles see it (also its words in shared memory).
struct Item {
  int b;        // sequence, -1: no more items
  int row0;     // row of q of the tile's first token
  int nt;       // its tokens
  int pos0;     // position of the first (negative: before the sequence)
  int g;        // kv head
  int split;    // range
  int ns;       // kv tiles of sinks in front of the window's
  int w0;       // first kv tile of the window
  int t0, t1;   // range [t0, t1) of the tile's list: sinks, then window
  int lo;       // first token of any row's window
  int first_w;  // softmax group of the first unit
  // in shared memory also: whether a live non-finite V value was replaced (the
  // relay's answer), units(), tiles() and halves() (what the MMA warp reads)

  __device__ __forceinline__ bool halves() const { return nt <= kHalfTokens; }
  __device__ __forceinline__ int tiles() const { return t1 - t0; }
  __device__ __forceinline__ int units() const { return halves() ? tiles() : 2 * tiles(); }
  __device__ __forceinline__ int units_of(int w) const {
    return halves() ? (tiles() + (w == first_w ? 1 : 0)) >> 1 : tiles();
  }
  __device__ __forceinline__ int tile(int k) const { return k < ns ? k : w0 + (k - ns); }
  __device__ __forceinline__ int end() const { return pos0 + nt; }  // tokens seen by the last row
  // Some row of the tile does not see some token of this kv tile.
  __device__ __forceinline__ bool partial(int tile, const MaskedArgs& a) const {
    const int base = tile * kKvTokens, last = base + kKvTokens - 1;
    if (last > pos0) return true;
    // the last token out of the last row's window
    const int64_t gone = static_cast<int64_t>(end()) - 1 - a.window;
    const int64_t from = base > a.sinks ? base : a.sinks;
    return from <= (gone < last ? gone : last);
  }
};
static_assert(sizeof(Item) + 16 == kItemWords * 4, "item words");

// (volatile loads: the softmax reads the item where it needs it, rather than
// hold its words in registers next to a row of scores)
__device__ __forceinline__ Item read_item(uint32_t addr) {
  Item it;
  const uint4 a = lds128(addr), b = lds128(addr + 16), c = lds128(addr + 32);
  it.b = a.x; it.row0 = a.y; it.nt = a.z; it.pos0 = a.w;
  it.g = b.x; it.split = b.y; it.ns = b.z; it.w0 = b.w;
  it.t0 = c.x; it.t1 = c.y; it.lo = c.z; it.first_w = c.w;
  return it;
}

// 3-D box of a tensor map, with the default L2 policy: K/V rows are read again
// by the other row tiles.
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                             int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 32 consecutive 32-bit columns of this thread's TMEM lane; the registers hold
// them after tmem_wait_ld and reg_after_wait32.
#define PKV_R16(r, i)                                                                       \
  "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
      "=r"(r[i + 6]), "=r"(r[i + 7]), "=r"(r[i + 8]), "=r"(r[i + 9]), "=r"(r[i + 10]),      \
      "=r"(r[i + 11]), "=r"(r[i + 12]), "=r"(r[i + 13]), "=r"(r[i + 14]), "=r"(r[i + 15])
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : PKV_R16(r, 0), PKV_R16(r, 16)
      : "r"(taddr)
      : "memory");
}
#define PKV_I16(r, i)                                                                       \
  "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
      "r"(r[i + 6]), "r"(r[i + 7]), "r"(r[i + 8]), "r"(r[i + 9]), "r"(r[i + 10]),      \
      "r"(r[i + 11]), "r"(r[i + 12]), "r"(r[i + 13]), "r"(r[i + 14]), "r"(r[i + 15])
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(taddr), PKV_I16(r, 0), PKV_I16(r, 16)
      : "memory");
}
#undef PKV_R16
__device__ __forceinline__ void reg_after_wait32(uint32_t (&r)[32]) {
  reg_after_wait(*reinterpret_cast<uint32_t(*)[16]>(&r[0]));
  reg_after_wait(*reinterpret_cast<uint32_t(*)[16]>(&r[16]));
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ int lds_int(uint32_t addr) {
  int v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// True in one lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// The MMAs with sw128_desc's descriptors given by their low words: the high
// word is the same for every tile, and a step inside a tile adds its offset
// in units of 16 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | ((1024u >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  unsigned long long ra, rb, rd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
  return d;
}

// Wait of a whole warp for phase `phase` (mod 2) of a barrier; false for all
// lanes when the limit ran out.
__device__ __forceinline__ bool warp_wait(uint32_t bar, int phase, unsigned long long limit_ns) {
  const uint32_t parity = static_cast<uint32_t>(phase) & 1u;
  if (__builtin_expect(__all_sync(kFull, mbar_test_wait(bar, parity)), 1)) return true;
  return __all_sync(kFull, mbar_wait_bounded(bar, parity, limit_ns)) != 0;
}

// Bits [lo, hi) of 32 (bounds outside are clamped).
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  lo = lo < 0 ? 0 : lo;
  hi = hi > 32 ? 32 : hi;
  if (lo >= hi) return 0u;
  return (0xFFFFFFFFu >> (32 - hi)) & (0xFFFFFFFFu << lo);
}

__device__ __forceinline__ int clamp_cols(int64_t v) {
  return v < -1 ? -1 : (v > kKvTokens ? kKvTokens : static_cast<int>(v));
}

// Add to dims [d0, d0 + 16) of a row at position pos the non-finite V values
// that the relay replaced by zero and the row sees (rare: plain loads).
__device__ __forceinline__ void add_nonfinite(const MaskedArgs& a, const Item& it, int pos, int d0,
                                              float (&o)[16]) {
#pragma unroll 1
  for (int k = it.t0; k < it.t1; ++k) {
    const int tile = it.tile(k);
    if (!it.partial(tile, a)) continue;
#pragma unroll 1
    for (int x = 0; x < kKvTokens; ++x) {
      const int t = tile * kKvTokens + x;
      if (t > pos || (static_cast<int64_t>(t) <= static_cast<int64_t>(pos) - a.window &&
                      t >= a.sinks))
        continue;
      const int pid = a.block_table[static_cast<int64_t>(it.b) * a.max_blocks + t / kPageSize];
      if (pid < 0 || pid >= a.num_pages) continue;
      const uint16_t* vr = a.pool + (((static_cast<int64_t>(pid) * 2 + 1) * kPageSize +
                                      t % kPageSize) * kNumKvHeads + it.g) * kHeadDim + d0;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float f = bf16_to_float(vr[e]);
        if (!(fabsf(f) < INFINITY)) o[e] += f;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1) paged_chunk_kernel(
    const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap page_map,
    const MaskedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_addr(smem);
  auto bar = [&](int i) { return sb + kOffBars + 8u * i; };
  auto wait = [&](int i, int phase) { return warp_wait(bar(i), phase, a.wait_ns); };
  int* s_items = reinterpret_cast<int*>(smem + kOffItems);
  auto item_addr = [&](int slot) { return sb + kOffItems + 4u * kItemWords * slot; };
  // [kMeta][2], then the TMEM address
  uint32_t* s_meta = reinterpret_cast<uint32_t*>(smem + kOffMeta);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // Barriers and TMEM before a dependent grid may start: its CTAs then never
  // take columns that this one still needs.
  if (tid == 0) {
    tma_prefetch_desc(&q_map);
    tma_prefetch_desc(&page_map);
    for (int i = 0; i < kNumBars; ++i) {
      int n = 1;
      if (i >= kBarSFree && i < kBarPvDone) n = 4;               // s_free, p_full
      if (i >= kBarItemEmpty && i < kBarXFull) n = kSoftmaxWarps + 4;
      if (i == kBarXFull || i == kBarXFree) n = 4;
      mbar_init(bar(i), n);
    }
    fence_barrier_init();
  }
  if (warp == kQkWarp) {
    __syncwarp();
    tmem_alloc(sb + kOffMeta + 8 * kMeta, kTmemCols);
    tmem_relinquish_alloc_permit();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_meta[2 * kMeta];
  wait_for_prior_grids();
  allow_dependent_grids();

  bool ok = true;
  if (warp >= kQkWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kSchedWarp) {
      // --------------------------------------------- scheduler, V's relay
      // Items in order (tile, range, head); the tiles of a sequence from its
      // last (under a causal mask the longest) to its first.  Every second
      // round runs through the CTAs backwards, so that long items pair with
      // short ones.
      const uint32_t per_tile = a.num_splits * kNumKvHeads;
      int b0 = -32, before = 0, sum = 0;      // 32 sequences from b0: tiles before them, theirs
      int cnt = 0, incl = 0, o0 = 0, o1 = 0, len = 0;  // this lane's sequence
      int parity = 0, out_i = 0;              // units so far mod 2, items published
      int round = 0, kt = 0;
      bool more = true;
      // publish the next item (or the end); false: a wait ran out
      auto publish = [&]() {
       for (;; ++round) {
        const int64_t idx = static_cast<int64_t>(round) * gridDim.x +
                            ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        // (a 64-bit division takes as long as the rest of this)
        const int64_t tile64 = idx >> 32 == 0 ? static_cast<uint32_t>(idx) / per_tile
                                              : idx / per_tile;
        const int rest = static_cast<int>(idx - tile64 * per_tile);
        while (b0 < a.batch && tile64 >= static_cast<int64_t>(before) + sum) {
          before += sum;
          b0 += 32;
          const int b = b0 + lane;
          cnt = 0;
          if (b < a.batch) {
            o0 = a.token_offsets[b];
            o1 = a.token_offsets[b + 1];
            len = a.seq_lens[b];
            if (o0 < 0 || o1 < o0 || o1 > a.num_tokens) {
              if (blockIdx.x == 0) record_error(a.dev_err, kErrOffsets);
            } else {
              // (shorter chunks are the other kernel's)
              cnt = o1 - o0 > kShortTokens ? (o1 - o0 + kQTokens - 1) / kQTokens : 0;
            }
          }
          incl = cnt;
#pragma unroll
          for (int x = 1; x < 32; x <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, x);
            if (lane >= x) incl += y;
          }
          sum = __shfl_sync(kFull, incl, 31);
        }
        Item it = {};
        it.b = -1;
        more = b0 < a.batch;
        if (more) {
          const int at = static_cast<int>(tile64 - before);
          const int src = __ffs(__ballot_sync(kFull, at < incl)) - 1;
          const int s_incl = __shfl_sync(kFull, incl, src);
          const int s_o0 = __shfl_sync(kFull, o0, src), s_o1 = __shfl_sync(kFull, o1, src);
          const int n = s_o1 - s_o0;
          const int qt = s_incl - 1 - at;  // the last tile of the sequence first
          it.b = b0 + src;
          it.row0 = s_o0 + qt * kQTokens;
          it.nt = min(kQTokens, n - qt * kQTokens);
          it.g = rest % kNumKvHeads;
          it.split = rest / kNumKvHeads;
          const int Lmax = a.max_blocks * kPageSize;
          int L = __shfl_sync(kFull, len, src);
          if (L < 0 || L > Lmax) {
            if (lane == 0) record_error(a.dev_err, kErrSeqLen);
            L = L < 0 ? 0 : Lmax;
          }
          it.pos0 = L - n + qt * kQTokens;
          if (it.pos0 < 0 && lane == 0) record_error(a.dev_err, kErrPosition);
          const int p0 = max(it.pos0, 0);
          it.lo = p0 >= a.window ? p0 - a.window + 1 : 0;
          it.w0 = it.lo / kKvTokens;
          auto kv_tiles = [](int n) {  // (n + 127 may pass 2^31)
            return static_cast<int>((static_cast<uint32_t>(n) + kKvTokens - 1) / kKvTokens);
          };
          it.ns = min(kv_tiles(min(a.sinks, it.lo)), it.w0);
          const int tiles = it.end() > 0 ? it.ns + kv_tiles(it.end()) - it.w0 : 0;
          it.t0 = static_cast<int>(static_cast<int64_t>(tiles) * it.split / a.num_splits);
          it.t1 = static_cast<int>(static_cast<int64_t>(tiles) * (it.split + 1) / a.num_splits);
          if (it.tiles() == 0) {
            // nothing to see in this range: zero rows, or empty partials
            for (int r = lane; r < it.nt * kGroup; r += 32) {
              const int64_t row = static_cast<int64_t>(it.row0 + r / kGroup) * kNumQHeads +
                                  it.g * kGroup + r % kGroup;
              if (a.num_splits == 1) {
                uint4* dst = reinterpret_cast<uint4*>(a.out + row * kHeadDim);
                for (int q = 0; q < 8; ++q) dst[q] = make_uint4(0u, 0u, 0u, 0u);
              } else {
                *reinterpret_cast<float2*>(a.part_ml + 2 * (row * a.num_splits + it.split)) =
                    make_float2(-INFINITY, 0.f);
              }
            }
            continue;
          }
          it.first_w = parity;
          parity = (parity + it.units()) & 1;
        }
        const int slot = out_i % kItems;
        if (out_i >= kItems && !wait(kBarItemEmpty + slot, out_i / kItems - 1)) return false;
        if (lane == 0) {
          int4* w = reinterpret_cast<int4*>(s_items + slot * kItemWords);
          w[0] = make_int4(it.b, it.row0, it.nt, it.pos0);
          w[1] = make_int4(it.g, it.split, it.ns, it.w0);
          w[2] = make_int4(it.t0, it.t1, it.lo, it.first_w);
          w[3] = make_int4(0, it.b < 0 ? 0 : it.units(), it.tiles(), it.halves() ? 1 : 0);
          mbar_arrive(bar(kBarItemFull + slot));
        }
        __syncwarp();
        ++out_i;
        ++round;
        return true;
       }
      };
      for (int i = 0; ok; ++i) {
        while (ok && more && out_i <= i + kAhead) ok = publish();
        const int slot = i % kItems;
        if (!ok || !wait(kBarItemFull + slot, i / kItems)) {
          ok = false;
          break;
        }
        const Item it = read_item(item_addr(slot));
        if (it.b < 0) break;
        bool live_bad = false;
        for (int k = it.t0; k < it.t1; ++k, ++kt) {
          const int st = kt % kStages, tile = it.tile(k);
          if (!wait(kBarVFull + st, kt / kStages)) {
            ok = false;
            break;
          }
          if (it.partial(tile, a)) {
            // 4 rows of 8 16-byte chunks at a time (the swizzle permutes
            // chunks within a row only)
            const uint32_t v0 = sb + kOffV + st * kRowTileBytes + lane * 16;
            const int base = tile * kKvTokens;
            const int row_end = it.end() - base;  // rows that some query sees
            const int64_t gone = static_cast<int64_t>(it.end()) - 1 - a.window;
            bool wrote = false;
#pragma unroll 1
            for (int r = 0; r < kKvTokens && r < row_end; r += kPageSize) {
              // pages that every query sees stand, those that none does are zeros
              const int t = base + r;
              if (t + kPageSize - 1 <= it.pos0 && (t > gone || t + kPageSize <= a.sinks)) continue;
              if (t + kPageSize <= it.lo && t >= a.sinks) continue;
              uint4 x[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = lds128(v0 + (r + 4 * e) * kRow);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t m0 = nonfinite_halves(x[e].x), m1 = nonfinite_halves(x[e].y),
                               m2 = nonfinite_halves(x[e].z), m3 = nonfinite_halves(x[e].w);
                if ((m0 | m1 | m2 | m3) != 0u) {
                  if (r + 4 * e + (lane >> 3) < row_end) live_bad = true;
                  wrote = true;
                  sts128(v0 + (r + 4 * e) * kRow, x[e].x & ~m0, x[e].y & ~m1, x[e].z & ~m2,
                         x[e].w & ~m3);
                }
              }
            }
            if (wrote) fence_proxy_async_smem();
          }
          const bool any = __any_sync(kFull, live_bad);
          if (lane == 0) {
            if (k == it.t1 - 1) s_items[slot * kItemWords + 12] = any ? 1 : 0;
            mbar_arrive(bar(kBarVReady + st));
          }
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(bar(kBarItemEmpty + slot));
      }
    } else if (warp == kLoadWarp) {
      // ----------------------------------------------------------- loads
      // One elected lane issues the copies (a lane apiece took 76 cycles a
      // copy, one lane for all 48).  Lane 8 j + p holds the id of page p of
      // the j-th of the next four kv tiles, fetched four tiles ahead, across
      // items too.
      const bool issuer = elect_one();
      int kt = 0, qn = 0;  // kv tiles and items loaded so far
      int k_issued = 0, v_issued = 0;
      auto fetch = [&](int i, Item& it) {
        if (!wait(kBarItemFull + i % kItems, i / kItems)) return false;
        it = read_item(item_addr(i % kItems));
        return true;
      };
      auto load_ids = [&](const Item& it, int k0) {
        int pid = -2;  // no row sees it
        const int k = k0 + (lane >> 3);
        if (k < it.t1) {
          const int page = it.tile(k) * kKvPages + (lane & 7), t = page * kPageSize;
          if (t < it.end() && (t + kPageSize > it.lo || t < a.sinks)) {
            pid = a.block_table[static_cast<int64_t>(it.b) * a.max_blocks + page];
            if (pid < 0 || pid >= a.num_pages) {
              record_error(a.dev_err, kErrPage);
              pid = -1;
            }
          }
        }
        return pid;
      };
      Item it, nx;
      ok = fetch(0, it);
      int ids = ok && it.b >= 0 ? load_ids(it, it.t0) : 0;
      for (int i = 0; ok && it.b >= 0; ++i) {
        const int qb = qn & 1;
        if (qn >= 2 && !(ok = wait(kBarQEmpty + qb, qn / 2 - 1))) break;
        if (issuer) {
          const uint32_t qbar = bar(kBarQFull + qb);
          const uint32_t dst = sb + kOffQ + qb * 2 * kRowTileBytes;
          mbar_arrive_expect_tx(qbar, (it.halves() ? 1 : 2) * kRowTileBytes);
          tma_load_box(dst, &q_map, qbar, 0, it.g * kGroup, it.row0);
          if (!it.halves())
            tma_load_box(dst + kRowTileBytes, &q_map, qbar, 0, it.g * kGroup,
                         it.row0 + kHalfTokens);
        }
        __syncwarp();
        ++qn;
        for (int k0 = it.t0; ok && k0 < it.t1; k0 += 4) {
          int ids_next = 0;
          if (k0 + 4 < it.t1) {
            ids_next = load_ids(it, k0 + 4);
          } else {
            if (!(ok = fetch(i + 1, nx))) break;
            if (nx.b >= 0) ids_next = load_ids(nx, nx.t0);
          }
          const unsigned bad = __ballot_sync(kFull, ids == -1);
          const int z = ids < 0 ? static_cast<int>(a.num_pages) : ids;  // past the pool: zeros
          for (int j = 0; j < 4 && k0 + j < it.t1; ++j, ++kt) {
            const int st = kt % kStages;
            if (kt >= kStages && !(ok = wait(kBarKEmpty + st, kt / kStages - 1))) break;
            const int tile = it.tile(k0 + j);
            const bool part = it.partial(tile, a);
            int zp[kKvPages];
#pragma unroll
            for (int p = 0; p < kKvPages; ++p) zp[p] = __shfl_sync(kFull, z, 8 * j + p);
            const int x = it.g * kHeadDim;
            if (issuer) {
              *reinterpret_cast<uint2*>(s_meta + 2 * (kt % kMeta)) =
                  make_uint2(tile, ((bad >> (8 * j)) & 0xFFu) | (part ? kPartial : 0u));
              const uint32_t full = bar(kBarKFull + st), dst = sb + kOffK + st * kRowTileBytes;
              mbar_arrive_expect_tx(full, kRowTileBytes);
#pragma unroll
              for (int p = 0; p < kKvPages; ++p)
                tma_load_box(dst + p * kPageBytes, &page_map, full, x, 0, zp[p]);
            }
            k_issued = kt + 1;
            if (kt >= kStages && !(ok = wait(kBarVEmpty + st, kt / kStages - 1))) break;
            if (issuer) {
              const uint32_t full = bar(kBarVFull + st), dst = sb + kOffV + st * kRowTileBytes;
              mbar_arrive_expect_tx(full, kRowTileBytes);
#pragma unroll
              for (int p = 0; p < kKvPages; ++p)
                tma_load_box(dst + p * kPageBytes, &page_map, full, x, kPageSize, zp[p]);
            }
            __syncwarp();
            v_issued = kt + 1;
          }
          ids = ids_next;
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(bar(kBarItemEmpty + i % kItems));
        it = nx;
      }
      // every copy issued has landed before the CTA ends (full limit)
      for (int j = max(0, k_issued - kStages); j < k_issued; ++j)
        if (!mbar_wait_bounded(bar(kBarKFull + j % kStages), (j / kStages) & 1) && lane == 0)
          record_error(a.dev_err, kErrTimeout);
      for (int j = max(0, v_issued - kStages); j < v_issued; ++j)
        if (!mbar_wait_bounded(bar(kBarVFull + j % kStages), (j / kStages) & 1) && lane == 0)
          record_error(a.dev_err, kErrTimeout);
      for (int j = max(0, qn - 2); j < qn; ++j)
        if (!mbar_wait_bounded(bar(kBarQFull + (j & 1)), (j >> 1) & 1) && lane == 0)
          record_error(a.dev_err, kErrTimeout);
    } else if (warp == kQkWarp) {
      // -------------------------------------------------------- S = Q K^T
      // (the whole warp walks the units, so that what the instructions take
      // is uniform over it; one elected lane issues them)
      const bool issuer = elect_one();
      int n = 0, kt = 0;  // units and kv tiles before; unit n is group (n & 1)'s n / 2th
      for (int i = 0; ok; ++i) {
        const int slot = i % kItems, qb = i & 1;
        if (!(ok = wait(kBarItemFull + slot, i / kItems))) break;
        const int4 x = *reinterpret_cast<const int4*>(s_items + slot * kItemWords + 12);
        const int U = x.y;
        const bool one = x.w != 0;
        if (U == 0) break;
        if (!(ok = wait(kBarQFull + qb, i >> 1))) break;
        const uint32_t q0 = desc_lo(sb + kOffQ + 2 * qb * kRowTileBytes);
        for (int u = 0; u < U; ++u, ++n) {
          const int w = n & 1, st = kt % kStages;
          const bool last = one || (u & 1);  // use of this kv tile
          if (!(ok = wait(kBarKFull + st, kt / kStages))) break;
          if (n >= 2 && !(ok = wait(kBarSFree + w, (n >> 1) - 1))) break;
          tc_fence_after_sync();
          const uint32_t q = q0 + (one ? 0 : w) * (kRowTileBytes >> 4);
          const uint32_t kr = desc_lo(sb + kOffK) + st * (kRowTileBytes >> 4);
          if (issuer) {
#pragma unroll
            for (int kk = 0; kk < kHeadDim / 16; ++kk)
              mma_ss(tmem + 128 * w, q + 2 * kk, kr + 2 * kk, kIdescQK, kk > 0);
            tc_commit(bar(kBarSFull + w));
            if (last) tc_commit(bar(kBarKEmpty + st));
            if (u == U - 1) tc_commit(bar(kBarQEmpty + qb));
          }
          if (last) ++kt;
        }
        if (issuer) mbar_arrive(bar(kBarItemEmpty + slot));
      }
      // no MMA in flight past here
      if (issuer) {
        tc_commit(bar(kBarQkFin));
        if (!mbar_wait_bounded(bar(kBarQkFin), 0)) record_error(a.dev_err, kErrTimeout);
      }
      __syncwarp();
    } else {
      // --------------------------------------------------------- O += P V
      const bool issuer = elect_one();
      int n = 0, kt = 0;
      for (int i = 0; ok; ++i) {
        const int slot = i % kItems;
        if (!(ok = wait(kBarItemFull + slot, i / kItems))) break;
        const int4 x = *reinterpret_cast<const int4*>(s_items + slot * kItemWords + 12);
        const int U = x.y;
        const bool one = x.w != 0;
        if (U == 0) break;
        for (int u = 0; u < U; ++u, ++n) {
          const int w = n & 1, st = kt % kStages;
          const bool last = one || (u & 1);
          if (!(ok = wait(kBarVReady + st, kt / kStages))) break;
          if (!(ok = wait(kBarPFull + w, n >> 1))) break;
          tc_fence_after_sync();
          const uint32_t vr = desc_lo(sb + kOffV) + st * (kRowTileBytes >> 4);
          if (issuer) {
            const uint32_t d = tmem + kTmemO + kHeadDim * w, pa = tmem + kTmemP + 64 * w;
            mma_ts(d, pa, vr, kIdescPV, u >= 2);  // a group's first unit of the item starts O
#pragma unroll
            for (int p = 1; p < kKvPages; ++p)
              mma_ts(d, pa + 8 * p, vr + p * (kPageBytes >> 4), kIdescPV, true);
            tc_commit(bar(kBarPvDone + w));
            if (last) tc_commit(bar(kBarVEmpty + st));
          }
          if (last) ++kt;
        }
        if (issuer) mbar_arrive(bar(kBarItemEmpty + slot));
      }
      if (issuer) {
        tc_commit(bar(kBarPvFin));
        if (!mbar_wait_bounded(bar(kBarPvFin), 0)) record_error(a.dev_err, kErrTimeout);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // --------------------------------------------------- softmax, epilogue
    const int w = warp >> 2;
    const int row = tid & 127;                 // MMA row = TMEM lane
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tS = t_lane + 128 * w, tP = t_lane + kTmemP + 64 * w,
                   tO = t_lane + kTmemO + kHeadDim * w;
    const float c = a.scale_log2;
    // this group's units, kv tiles of the items before, rows handed over
    int units = 0, kt0 = 0, xn = 0;
    bool held = false;  // the second group's O has not been read by the first yet
    for (int i = 0; ok; ++i) {
      const int slot = i % kItems;
      if (!(ok = wait(kBarItemFull + slot, i / kItems))) break;
      bool one, idle;  // one row tile; no row of this warp is a token's
      int nu, first;   // this group's units, its first place in the list of kv tiles
      {
        const Item it = read_item(item_addr(slot));
        if (it.b < 0) break;
        one = it.halves();
        idle = ((row & ~31) >> 2) + (one ? 0 : kHalfTokens * w) >= it.nt;
        nu = it.units_of(w);
        first = one && w != it.first_w ? 1 : 0;
      }
      float m_ref = -INFINITY, l_run = 0.f;
      for (int v = 0; v < nu; ++v, ++units) {
        if (!(ok = wait(kBarSFull + w, units))) break;
        tc_fence_after_sync();
        // PV of the group's last tile has read P and added to O; the item's
        // first may start O once the first group has read what it holds
        auto o_ready = [&]() {
          if (v > 0) return wait(kBarPvDone + w, units - 1);
          if (held) {
            held = false;
            return wait(kBarXFree, xn - 1);
          }
          return true;
        };
        // (written before the loads that QK waited for)
        const uint2 note = lds64(sb + kOffMeta + 8u * ((kt0 + first + (one ? 2 * v : v)) % kMeta));
        if (idle) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarSFree + w));
          if (!(ok = o_ready())) break;
        } else {
          // the whole row of scores, so that QK may overwrite S at once
          uint32_t x[4][32];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(tS + 32 * q, x[q]);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 4; ++q) reg_after_wait32(x[q]);
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarSFree + w));
          if (note.y != 0u) {  // columns that this row does not see
            const uint32_t bad = note.y;
            const int pos =
                lds_int(item_addr(slot) + 12) + (row >> 2) + (one ? 0 : kHalfTokens * w);
            const int64_t base = static_cast<int64_t>(note.x) * kKvTokens;
            const int ch = clamp_cols(pos - base) + 1;  // columns [0, ch): t <= pos
            // [cl, ..): t > pos - window; [0, cs): t < sinks
            const int cl = clamp_cols(static_cast<int64_t>(pos) - a.window - base) + 1;
            const int cs = clamp_cols(a.sinks - base);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t vis = bits_between(0, ch - 32 * q) &
                             (bits_between(cl - 32 * q, 32) | bits_between(0, cs - 32 * q));
              if ((bad >> (2 * q)) & 1u) vis &= 0xFFFF0000u;
              if ((bad >> (2 * q + 1)) & 1u) vis &= 0x0000FFFFu;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((vis >> e) & 1u)) x[q][e] = 0xFF800000u;  // -inf
            }
          }
          // The reference maximum is set by the first tile a row sees anything
          // of, and moves only when a tile's weights sum to 2^kRescale or more
          // (FP32 sums and bf16 weights keep their relative precision below).
          bool measure = __any_sync(kFull, m_ref == -INFINITY);
          if (!(ok = o_ready())) break;
          tc_fence_after_sync();
          for (;;) {
            float alpha = 1.f;
            if (measure) {
              float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                  mx[(e >> 1) & 1] = fmax3(mx[(e >> 1) & 1], __uint_as_float(x[q][e]),
                                           __uint_as_float(x[q][e + 1]));
              const float top = fmaxf(mx[0], mx[1]) * c;
              if (top > m_ref) {
                alpha = fast_exp2(m_ref - top);  // 0 on the first live tile
                m_ref = top;
              }
              if (v > 0 && __any_sync(kFull, alpha != 1.f)) {
                l_run *= alpha;
#pragma unroll 1
                for (int q = 0; q < kHeadDim / 16; ++q) {
                  uint32_t o[16];
                  tmem_ld16(tO + 16 * q, o);
                  tmem_wait_ld();
                  reg_after_wait(o);
#pragma unroll
                  for (int e = 0; e < 16; ++e)
                    o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                  tmem_st16(tO + 16 * q, o);
                }
              }
            }
            // (a row that has seen no token yet: every weight 2^(-inf) = 0)
            const float m = m_ref == -INFINITY ? 0.f : m_ref;
            const float2 c2 = make_float2(c, c), m2 = make_float2(-m, -m);
            float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t pw[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const uint32_t* s2 = &x[2 * q + (e >> 4)][2 * (e & 15)];
                float2 y = ffma2(make_float2(__uint_as_float(s2[0]), __uint_as_float(s2[1])),
                                 c2, m2);
                y.x = fast_exp2(y.x);
                y.y = fast_exp2(y.y);
                ls[e & 1] = fadd2(ls[e & 1], y);
                pw[e] = pack_bf16x2(y.x, y.y);
              }
              tmem_st32(tP + 32 * q, pw);
            }
            const float2 l2 = fadd2(ls[0], ls[1]);
            const float sum = l2.x + l2.y;
            // (NaN too; a tile that has just been measured stands as it is)
            const bool over = !(sum < kRescale);
            if (measure || !__any_sync(kFull, over)) {
              l_run += sum;
              break;
            }
            measure = true;
          }
          tmem_wait_st();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPFull + w));
      }
      if (!ok) break;
      const Item it = read_item(item_addr(slot));
      kt0 += it.tiles();
      const int tok = (row >> 2) + (one ? 0 : kHalfTokens * w);
      const int pos = it.pos0 + tok;

      // ---- epilogue
      if (nu > 0 && !(ok = wait(kBarPvDone + w, units - 1))) break;
      tc_fence_after_sync();
      bool writes = tok < it.nt;
      const bool other = one && it.units_of(1) > 0;  // both groups saw these rows
      float2* xml = reinterpret_cast<float2*>(smem + kOffMl) + row;
      if (one && w == 1) {
        // the first group takes this one's rows from TMEM (the same lanes)
        writes = false;
        if (other) {
          *xml = make_float2(m_ref, l_run);
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarXFull));
          held = true;
        }
      }
      float w0 = 1.f, w1 = 0.f;
      if (other && w == 0) {
        if (!(ok = wait(kBarXFull, xn))) break;
        tc_fence_after_sync();
        const float2 ml = *xml;
        const float M = fmaxf(m_ref, ml.x);
        // (a group whose tiles the row did not see: zeros)
        w0 = m_ref == -INFINITY ? 1.f : fast_exp2(m_ref - M);
        w1 = ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - M);
        l_run = l_run * w0 + ml.y * w1;
        m_ref = M;
      }
      // (written before the last kv tile's V was handed to its PV, which this
      // row's group, or the other one, has waited for)
      const int bad_v = *reinterpret_cast<volatile int*>(s_items + slot * kItemWords + 12);
      if (!(one && w == 1) && !idle) {
        const int tok0 = ((row & ~31) >> 2) + (one ? 0 : kHalfTokens * w);  // the warp's first
        const int64_t r0 = static_cast<int64_t>(it.row0 + tok0) * kNumQHeads + it.g * kGroup;
        const uint32_t stage = sb + kOffOut + warp * kOutBytes + lane * 128;
        // 128 B of each of the warp's rows, staged in shared memory (16-byte
        // pieces swizzled by the row), to base + row of the output x stride:
        // whole rows to a store instruction
        auto write_rows = [&](void* base, int64_t stride) {
          __syncwarp();
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const int y = 4 * t + (lane >> 3);
            const uint4 v = lds128(sb + kOffOut + warp * kOutBytes + y * 128 +
                                   (((lane ^ y) & 7) << 4));
            if (tok0 + t < it.nt)
              *reinterpret_cast<uint4*>(static_cast<char*>(base) +
                                        (t * kNumQHeads + (lane >> 3)) * stride +
                                        16 * (lane & 7)) = v;
          }
          __syncwarp();
        };
        const float inv = l_run > 0.f || l_run != l_run ? 1.f / l_run : 0.f;
        if (a.num_splits > 1 && writes)
          *reinterpret_cast<float2*>(
              a.part_ml +
              2 * ((r0 + (tok - tok0) * kNumQHeads + (row & 3)) * a.num_splits + it.split)) =
              make_float2(m_ref, l_run);
#pragma unroll 1
        for (int q = 0; q < kHeadDim / 16; ++q) {
          uint32_t x[16];
          float o[16];
          if (nu > 0) {
            tmem_ld16(tO + 16 * q, x);
            tmem_wait_ld();
            reg_after_wait(x);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(x[e]) * w0;
          if (other) {
            tmem_ld16(tO + kHeadDim + 16 * q, x);
            tmem_wait_ld();
            reg_after_wait(x);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = fmaf(__uint_as_float(x[e]), w1, o[e]);
          }
          if (bad_v != 0 && writes) add_nonfinite(a, it, pos, 16 * q, o);
          if (a.num_splits == 1) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              sts128(stage + (((2 * q + e) ^ (lane & 7)) << 4),
                     pack_bf16x2(o[8 * e] * inv, o[8 * e + 1] * inv),
                     pack_bf16x2(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                     pack_bf16x2(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                     pack_bf16x2(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
            if (q == 3) write_rows(a.out + r0 * kHeadDim, kHeadDim * 2);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sts128(stage + (((4 * (q & 1) + e) ^ (lane & 7)) << 4),
                     __float_as_uint(o[4 * e]), __float_as_uint(o[4 * e + 1]),
                     __float_as_uint(o[4 * e + 2]), __float_as_uint(o[4 * e + 3]));
            if (q & 1)
              write_rows(a.part_acc + (r0 * a.num_splits + it.split) * kHeadDim + 32 * (q >> 1),
                         static_cast<int64_t>(a.num_splits) * kHeadDim * 4);
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (other && w == 0) mbar_arrive(bar(kBarXFree));
        mbar_arrive(bar(kBarItemEmpty + slot));
      }
      if (other) ++xn;
    }
  }
  if (!ok && lane == 0) record_error(a.dev_err, kErrTimeout);

  // ---- every copy and MMA of this CTA has completed; the columns go back
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kQkWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Combine the ranges of each query row: one warp per row, lane l holding dims
// 2l and 2l + 1; the ranges are added in order.
constexpr int kMergeRows = 4;
__global__ void __launch_bounds__(32 * kMergeRows) merge_chunk_kernel(const MaskedArgs a) {
  allow_dependent_grids();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeRows + (threadIdx.x >> 5);
  const int tok = static_cast<int>(row / kNumQHeads);
  // rows of no sequence keep what they hold
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.token_offsets[mid] <= tok) lo = mid; else hi = mid;
  }
  const int o0 = a.token_offsets[lo], o1 = a.token_offsets[lo + 1];
  if (o0 < 0 || o1 > a.num_tokens || tok < o0 || tok >= o1) return;
  if (o1 - o0 <= kShortTokens) return;  // the other kernel's
  const int splits = a.num_splits;
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + row * a.num_splits;
  const float2* acc = reinterpret_cast<const float2*>(a.part_acc) +
                      row * a.num_splits * (kHeadDim / 2) + lane;
  reinterpret_cast<uint32_t*>(a.out + row * kHeadDim)[lane] = merge_ranges(ml, acc, splits, lane);
}

cudaError_t configure(int device) {
  static std::atomic<unsigned long long> done{0};
  const unsigned long long bit = 1ull << (device & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaFuncAttributes fa;
  cudaError_t err = cudaFuncGetAttributes(&fa, paged_chunk_kernel);
  if (err != cudaSuccess) return err;
  // the register split must stay within what the block starts with
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  err = cudaFuncSetAttribute(paged_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmem);
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return err;
}

}  // namespace

cudaError_t launch_chunk_attention(const CUtensorMap& q_map, const CUtensorMap& page_map,
                                   const MaskedArgs& args, int grid, cudaStream_t stream) {
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  if ((err = configure(device)) != cudaSuccess) return err;
  return launch_pdl(paged_chunk_kernel, dim3(grid), dim3(kThreads), kSmem, stream, q_map, page_map,
                    args);
}

cudaError_t launch_chunk_merge(const MaskedArgs& args, cudaStream_t stream) {
  static_assert(kNumQHeads % kMergeRows == 0, "whole CTAs of rows");
  return launch_pdl(merge_chunk_kernel, dim3(args.num_tokens * (kNumQHeads / kMergeRows)),
                    dim3(32 * kMergeRows), 0, stream, args);
}

}  // namespace pkv
