// kv_evict.cu -- eviction from the paged cache by accumulated attention
// weight: each (sequence, kv head) keeps its first `sinks` tokens, its last
// `recent` ones and, of the others, the heaviest that fit the budget, packed
// in token order into the pages of another block table.
//
// Selection: the weights map to 32-bit keys whose unsigned order is the
// weights' order (NaN above +inf, -0 as +0); a radix descent of four 8-bit
// digits over a shared-memory histogram finds the key of the last token kept
// and how many tokens of that key are kept, lowest index first.  Counts only:
// the result does not depend on the order of the atomics.  Then every warp
// takes a contiguous part of the tokens, counts its kept ones with ballots,
// and writes them at the sum of the counts before it.
//
// The copy is bound by memory (512 bytes a kept token and head, as 128-byte
// rows) and wants many CTAs, the selection reads 4 bytes a token and is short:
// so a (sequence, kv head) gets several CTAs, each of which repeats the
// selection and copies its own part of the kept rows -- one launch, and no
// CTA waits for another.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xFFFFFFFFu;
// Tables up to this many tokens keep the keys in shared memory; longer ones
// read the weights again (from L2) in every pass.
constexpr int kSmemTokens = 12288;
constexpr int kCopyRows = 4;  // tokens whose rows a group of 8 lanes has in flight

// Order-preserving key of a weight.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <bool kSmemKeys>
__global__ void __launch_bounds__(kThreads) kv_evict_kernel(const EvictArgs a) {
  extern __shared__ uint32_t s_keys[];
  __shared__ int s_hist[256];
  __shared__ int s_eq[kWarps], s_keep[kWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.x % kNumKvHeads, part = blockIdx.x / kNumKvHeads, b = blockIdx.y;
  const int parts = gridDim.x / kNumKvHeads;
  wait_for_prior_grids();
  allow_dependent_grids();
  const int Lmax = a.max_blocks * kPageSize;
  int L = a.seq_lens[b];
  if (L < 0 || L > Lmax) {
    if (tid == 0) record_error(a.dev_err, kErrSeqLen);
    L = L < 0 ? 0 : Lmax;
  }
  const int n = min(L, a.budget);
  const int64_t bg = static_cast<int64_t>(b) * kNumKvHeads + g;
  const float* mass = a.mass + bg * a.mass_stride;
  // this CTA's kept tokens [c0, c1)
  const int c0 = static_cast<int>(static_cast<int64_t>(n) * part / parts);
  const int c1 = static_cast<int>(static_cast<int64_t>(n) * (part + 1) / parts);
  float* new_mass = a.new_mass + bg * a.new_mass_stride;
  int32_t* kept = a.kept + bg * a.budget;
  if (part == 0 && tid == 0 && g == 0) a.new_lens[b] = n;
  for (int64_t i = n + part * kThreads + tid; i < a.new_mass_stride; i += parts * kThreads)
    new_mass[i] = 0.f;
  for (int64_t i = n + part * kThreads + tid; i < a.budget; i += parts * kThreads) kept[i] = -1;

  if (L <= a.budget) {  // everything stays
    for (int i = c0 + tid; i < c1; i += kThreads) {
      kept[i] = i;
      new_mass[i] = mass[i];
    }
  } else {
    // tokens [lo, hi) compete; the others stay
    const int lo = a.sinks, hi = L - a.recent;
    if (kSmemKeys) {
      for (int t = lo + tid; t < hi; t += kThreads) s_keys[t] = weight_key(mass[t]);
    }
    auto key = [&](int t) { return kSmemKeys ? s_keys[t] : weight_key(mass[t]); };
    uint32_t prefix = 0;
    int need = a.budget - a.sinks - a.recent;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) s_hist[tid] = 0;
      __syncthreads();
      const uint32_t high = shift == 24 ? 0u : ~0u << (shift + 8);
      for (int t = lo + tid; t < hi; t += kThreads) {
        const uint32_t k = key(t);
        if ((k & high) != prefix) continue;
        // one atomic per digit and warp: the first digit of weights of like
        // size is the same for nearly all
        const int d = (k >> shift) & 255;
        const unsigned same = __match_any_sync(__activemask(), d);
        if (lane == __ffs(same) - 1) atomicAdd(&s_hist[d], __popc(same));
      }
      __syncthreads();
      if (warp == 0) {
        // lane l holds digits 8 l .. 8 l + 7; from the highest digit down, the
        // first one whose running count reaches need
        int h[8], sum = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += h[e] = s_hist[8 * lane + e];
        int above = sum;  // tokens of this lane's digits and higher ones
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
          const int y = __shfl_down_sync(kFull, above, x);
          if (lane + x < 32) above += y;
        }
        const unsigned reach = __ballot_sync(kFull, above >= need);
        if (lane == 31 - __clz(reach)) {
          int left = need - (above - sum), d = 7;
#pragma unroll
          for (int e = 7; e > 0; --e)
            if (d == e && h[e] < left) {
              left -= h[e];
              d = e - 1;
            }
          s_prefix = prefix | (static_cast<uint32_t>(8 * lane + d) << shift);
          s_need = left;
        }
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
    // kept: keys above prefix, and the first `need` tokens of that key
    const int span = ((L + kWarps - 1) / kWarps + 31) & ~31;
    const int t0 = min(warp * span, L), t1 = min(t0 + span, L);
    int eq = 0;
    for (int t = t0 + lane; t < t1; t += 32) eq += t >= lo && t < hi && key(t) == prefix;
    eq = __reduce_add_sync(kFull, eq);
    if (lane == 0) s_eq[warp] = eq;
    __syncthreads();
    int eq_base = 0;
    for (int x = 0; x < warp; ++x) eq_base += s_eq[x];
    // at(t): how many are kept in [t & ~31, t) of the warp's 32 tokens
    auto step = [&](int tt, int& eqs, bool& keep) {
      const int t = tt + lane;
      const bool in = t < t1, contest = in && t >= lo && t < hi;
      const uint32_t k = contest ? key(t) : 0u;
      const bool e = contest && k == prefix;
      const unsigned eb = __ballot_sync(kFull, e);
      keep = in && (!contest || k > prefix ||
                    (e && eqs + __popc(eb & ((1u << lane) - 1u)) < need));
      eqs += __popc(eb);
      return __ballot_sync(kFull, keep);
    };
    int cnt = 0, eqs = eq_base;
    bool keep;
    for (int tt = t0; tt < t1; tt += 32) cnt += __popc(step(tt, eqs, keep));
    if (lane == 0) s_keep[warp] = cnt;
    __syncthreads();
    int at = 0;
    for (int x = 0; x < warp; ++x) at += s_keep[x];
    eqs = eq_base;
    if (at < c1 && at + cnt > c0) {
      for (int tt = t0; tt < t1; tt += 32) {
        const unsigned kb = step(tt, eqs, keep);
        const int i = at + __popc(kb & ((1u << lane) - 1u));
        if (keep && i >= c0 && i < c1) {
          kept[i] = tt + lane;
          new_mass[i] = mass[tt + lane];
        }
        at += __popc(kb);
      }
    }
  }
  __syncthreads();

  // ---- the rows: 8 lanes copy a token's K and V rows, 16 bytes a lane
  const int group = tid >> 3, chunk = tid & 7;
  constexpr int kGroups = kThreads / 8;
  const int64_t slot_row = kNumKvHeads * kHeadDim;  // elements between slots
  uint4 x[kCopyRows][2];
  uint16_t* dst[kCopyRows];
  for (int i0 = c0 + group; i0 < c1; i0 += kGroups * kCopyRows) {
#pragma unroll
    for (int e = 0; e < kCopyRows; ++e) {
      const int i = i0 + e * kGroups;
      dst[e] = nullptr;
      if (i >= c1) continue;
      const int t = __ldcg(kept + i);
      const int32_t sp = a.block_table[static_cast<int64_t>(b) * a.max_blocks + t / kPageSize];
      const int32_t dp =
          a.dst_block_table[static_cast<int64_t>(b) * a.dst_max_blocks + i / kPageSize];
      if (sp < 0 || sp >= a.num_pages || dp < 0 || dp >= a.num_pages) {
        if (chunk == 0) record_error(a.dev_err, kErrPage);
        continue;
      }
      const uint16_t* src = a.pool +
                            (static_cast<int64_t>(sp) * 2 * kPageSize + t % kPageSize) * slot_row +
                            g * kHeadDim + chunk * 8;
      dst[e] = a.pool + (static_cast<int64_t>(dp) * 2 * kPageSize + i % kPageSize) * slot_row +
               g * kHeadDim + chunk * 8;
      x[e][0] = *reinterpret_cast<const uint4*>(src);
      x[e][1] = *reinterpret_cast<const uint4*>(src + kPageSize * slot_row);
    }
#pragma unroll
    for (int e = 0; e < kCopyRows; ++e) {
      if (dst[e] == nullptr) continue;
      *reinterpret_cast<uint4*>(dst[e]) = x[e][0];
      *reinterpret_cast<uint4*>(dst[e] + kPageSize * slot_row) = x[e][1];
    }
  }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& args, int num_sms, cudaStream_t stream) {
  // CTAs for about two waves of two per SM, at least 64 kept rows each
  const long long units = static_cast<long long>(args.batch) * kNumKvHeads;
  const long long parts = std::max(
      1LL, std::min((4LL * num_sms + units - 1) / units, (args.budget + 63LL) / 64));
  const dim3 grid(static_cast<unsigned>(kNumKvHeads * parts), args.batch);
  const int64_t tokens = static_cast<int64_t>(args.max_blocks) * kPageSize;
  return tokens <= kSmemTokens
             ? launch_pdl(kv_evict_kernel<true>, grid, dim3(kThreads), tokens * sizeof(uint32_t),
                          stream, args)
             : launch_pdl(kv_evict_kernel<false>, grid, dim3(kThreads), 0, stream, args);
}

}  // namespace pkv
