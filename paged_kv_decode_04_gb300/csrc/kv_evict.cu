// kv_evict.cu -- eviction from the paged cache by accumulated attention
// weight: each (sequence, kv head) keeps its first `sinks` tokens, its last
// `recent` ones and, of the others, the heaviest that fit the budget, packed
// in token order into the pages of another block table.
//
// Selection: the weights map to 32-bit keys whose unsigned order is the
// weights' order (NaN above +inf, -0 as +0); a radix descent of three digits
// (11, 11 and 10 bits: the first one holds the exponent and two bits more, so
// that weights of like size spread over many counters) over a shared-memory
// histogram finds the key of the last token kept and how many tokens of that
// key are kept, lowest index first.  Counts only: the result does not depend
// on the order of the atomics.  Then every warp takes a contiguous part of the
// tokens, counts its kept ones with ballots, and writes them at the sum of the
// counts before it.
//
// The copy is bound by memory (512 bytes a kept token and head, as 128-byte
// rows) and wants many CTAs, the selection reads 4 bytes a token and is short:
// so a (sequence, kv head) gets several CTAs, each of which repeats the
// selection and copies its own part of the kept rows -- one launch, and no
// CTA waits for another.  64 sequences of 4096 tokens down to 1024 (279 MB)
// took 63 us, 4.4 TB/s, 57 us on the device; about 12 us of it are the
// selection, in which every CTA of the one wave is at once.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

// Tables of up to kSmallTokens tokens: CTAs of 256 threads, four to an SM.
// Longer ones: CTAs of 1024 threads (the selection is the longer part), one to
// an SM, or of 512, two to an SM, for tables of up to kPairTokens when there are
// more (sequence, kv head) pairs than SMs; up to kSmemTokens the keys stay in
// shared memory, beyond it every pass reads the weights again (from L2).  One
// sequence of 32768 tokens took 119 us with small CTAs, 29.5 us with large ones;
// 40 of 12000 43 us with large, 35 with pairs; 10 of 20000 37 and 45.
enum Kind { kSmall, kPair, kLarge };
constexpr int kSmallTokens = 8192, kPairTokens = 24576, kSmemTokens = 49152;
template <Kind kKind>
struct Shape {
  static constexpr int kThreads = kKind == kSmall ? 256 : kKind == kPair ? 512 : 1024;
  static constexpr int kCtas = kKind == kSmall ? 4 : kKind == kPair ? 2 : 1;
  static constexpr int kKeys =
      kKind == kSmall ? kSmallTokens : kKind == kPair ? kPairTokens : kSmemTokens;
};
constexpr int kBins = 2048;
constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kLoads = 8;  // weights a thread has in flight
// Tokens whose rows a group of 8 lanes has in flight (when chosen, two: 65.4 us on
// the batch above, three 65.0, four spill registers: 71.3; 512 threads and two
// CTAs 77.7).
constexpr int kCopyRows = 3;

// Order-preserving key of a weight.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <Kind kKind, bool kSmemKeys>
__global__ void __launch_bounds__(Shape<kKind>::kThreads, Shape<kKind>::kCtas)
    kv_evict_kernel(const EvictArgs a) {
  constexpr int kThreads = Shape<kKind>::kThreads, kWarps = kThreads / 32;
  extern __shared__ uint32_t s_keys[];
  __shared__ __align__(16) int s_hist[kBins];
  __shared__ int s_above[kWarps], s_eq[kWarps], s_gt[kWarps];
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
    // this thread's share of the competing tokens' keys
    auto each_key = [&](auto&& f) {
      for (int t0 = lo + tid; t0 < hi; t0 += kLoads * kThreads) {
        float v[kLoads];
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
          const int t = t0 + e * kThreads;
          v[e] = t < hi ? mass[t] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
          const int t = t0 + e * kThreads;
          if (t < hi) f(t, weight_key(v[e]));
        }
      }
    };
    auto key = [&](int t) { return kSmemKeys ? s_keys[t] : weight_key(mass[t]); };
    uint32_t prefix = 0;
    int need = a.budget - a.sinks - a.recent;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t digits = pass == 2 ? 1023u : 2047u;
      const uint32_t high = pass == 0 ? 0u : (pass == 1 ? ~0u << 21 : ~0u << 10);
      constexpr int kMine = kBins / kThreads;  // consecutive counters of one thread
      int2* mine = reinterpret_cast<int2*>(s_hist + tid * kMine);
#pragma unroll
      for (int e = 0; e < kMine / 2; ++e) mine[e] = make_int2(0, 0);
      __syncthreads();
      auto count = [&](int, uint32_t k) {
        if ((k & high) == prefix) atomicAdd(&s_hist[(k >> shift) & digits], 1);
      };
      if (kSmemKeys && pass == 0) {
        each_key([&](int t, uint32_t k) {
          s_keys[t] = k;
          count(t, k);
        });
      } else if (kSmemKeys) {
        for (int t = lo + tid; t < hi; t += kThreads) count(t, s_keys[t]);
      } else {
        each_key(count);
      }
      __syncthreads();
      // from the highest digit down, the first whose running count reaches need
      int h[kMine], sum = 0;
#pragma unroll
      for (int e = 0; e < kMine / 2; ++e) {
        const int2 v = mine[e];
        h[2 * e] = v.x;
        h[2 * e + 1] = v.y;
      }
#pragma unroll
      for (int e = 0; e < kMine; ++e) sum += h[e];
      int above = sum;  // tokens of this thread's digits and the warp's higher ones
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_down_sync(kFull, above, x);
        if (lane + x < 32) above += y;
      }
      if (lane == 0) s_above[warp] = above;
      __syncthreads();
      for (int x = warp + 1; x < kWarps; ++x) above += s_above[x];
      // one thread's digits hold the need-th token (need 0: the highest digit)
      if ((above >= need && above - sum < need) || (need == 0 && tid == kThreads - 1)) {
        int left = need - (above - sum), d = kMine - 1;
#pragma unroll
        for (int e = kMine - 1; e > 0; --e)
          if (d == e && h[e] < left) {
            left -= h[e];
            d = e - 1;
          }
        s_prefix = prefix | (static_cast<uint32_t>(tid * kMine + d) << shift);
        s_need = left;
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
    // kept: keys above prefix, and the first `need` tokens of that key
    const int span = ((L + kWarps - 1) / kWarps + 31) & ~31;
    const int t0 = min(warp * span, L), t1 = min(t0 + span, L);
    int eq = 0, gt = 0;
#pragma unroll 4
    for (int t = t0 + lane; t < t1; t += 32) {
      const bool contest = t >= lo && t < hi;
      const uint32_t k = contest ? key(t) : 0xFFFFFFFFu;
      eq += contest && k == prefix;
      gt += !contest || k > prefix;
    }
    eq = __reduce_add_sync(kFull, eq);
    gt = __reduce_add_sync(kFull, gt);
    if (lane == 0) {
      s_eq[warp] = eq;
      s_gt[warp] = gt;
    }
    __syncthreads();
    int at = 0, eqs = 0;  // kept, and of key prefix, before this warp's tokens
    for (int x = 0; x < warp; ++x) {
      at += s_gt[x] + min(max(need - eqs, 0), s_eq[x]);
      eqs += s_eq[x];
    }
    if (at < c1) {
      for (int tt = t0; tt < t1 && at < c1; tt += 32) {
        const int t = tt + lane;
        const bool in = t < t1, contest = in && t >= lo && t < hi;
        const uint32_t k = contest ? key(t) : 0u;
        const unsigned eb = __ballot_sync(kFull, contest && k == prefix);
        const int rank = eqs + __popc(eb & ((1u << lane) - 1u));
        const bool keep =
            in && (!contest || k > prefix || (k == prefix && rank < need));
        const unsigned kb = __ballot_sync(kFull, keep);
        const int i = at + __popc(kb & ((1u << lane) - 1u));
        if (keep && i >= c0 && i < c1) {
          kept[i] = t;
          new_mass[i] = mass[t];
        }
        eqs += __popc(eb);
        at += __popc(kb);
      }
    }
  }
  __syncthreads();

  // ---- the rows: 8 lanes copy a token's K and V rows, 16 bytes a lane
  const int group = tid >> 3, chunk = tid & 7;
  constexpr int kGroups = kThreads / 8;
  const int64_t slot_row = kNumKvHeads * kHeadDim;  // elements between slots
  const int32_t* src_table = a.block_table + static_cast<int64_t>(b) * a.max_blocks;
  const int32_t* dst_table = a.dst_block_table + static_cast<int64_t>(b) * a.dst_max_blocks;
  // addresses of the next kCopyRows tokens of this group, fetched while the
  // rows of the last ones are on their way
  const uint16_t* src[kCopyRows];
  uint16_t* dst[kCopyRows];
  auto addresses = [&](int i0) {
    int t[kCopyRows], sp[kCopyRows], dp[kCopyRows];
#pragma unroll
    for (int e = 0; e < kCopyRows; ++e) {
      const int i = i0 + e * kGroups;
      t[e] = i < c1 ? __ldcg(kept + i) : -1;
      dp[e] = i < c1 ? dst_table[i / kPageSize] : 0;
    }
#pragma unroll
    for (int e = 0; e < kCopyRows; ++e) sp[e] = t[e] >= 0 ? src_table[t[e] / kPageSize] : 0;
#pragma unroll
    for (int e = 0; e < kCopyRows; ++e) {
      const int i = i0 + e * kGroups;
      dst[e] = nullptr;
      if (t[e] < 0) continue;
      if (sp[e] < 0 || sp[e] >= a.num_pages || dp[e] < 0 || dp[e] >= a.num_pages) {
        if (chunk == 0) record_error(a.dev_err, kErrPage);
        continue;
      }
      src[e] = a.pool +
               (static_cast<int64_t>(sp[e]) * 2 * kPageSize + t[e] % kPageSize) * slot_row +
               g * kHeadDim + chunk * 8;
      dst[e] = a.pool + (static_cast<int64_t>(dp[e]) * 2 * kPageSize + i % kPageSize) * slot_row +
               g * kHeadDim + chunk * 8;
    }
  };
  addresses(c0 + group);
  for (int i0 = c0 + group; i0 < c1; i0 += kGroups * kCopyRows) {
    uint4 x[kCopyRows][2];
    uint16_t* to[kCopyRows];
#pragma unroll
    for (int e = 0; e < kCopyRows; ++e) {
      to[e] = dst[e];
      if (to[e] == nullptr) continue;
      x[e][0] = __ldcs(reinterpret_cast<const uint4*>(src[e]));
      x[e][1] = __ldcs(reinterpret_cast<const uint4*>(src[e] + kPageSize * slot_row));
    }
    addresses(i0 + kGroups * kCopyRows);
#pragma unroll
    for (int e = 0; e < kCopyRows; ++e) {
      if (to[e] == nullptr) continue;
      *reinterpret_cast<uint4*>(to[e]) = x[e][0];
      *reinterpret_cast<uint4*>(to[e] + kPageSize * slot_row) = x[e][1];
    }
  }
}

template <Kind kKind, bool kSmemKeys>
cudaError_t launch(const EvictArgs& args, int num_sms, cudaStream_t stream) {
  using Sh = Shape<kKind>;
  const int64_t tokens = static_cast<int64_t>(args.max_blocks) * kPageSize;
  const size_t smem = kSmemKeys ? tokens * sizeof(uint32_t) : 0;
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  static std::atomic<unsigned long long> done{0};
  const unsigned long long bit = 1ull << (device & 63);
  if (kSmemKeys && !(done.load(std::memory_order_acquire) & bit)) {
    err = cudaFuncSetAttribute(
        kv_evict_kernel<kKind, kSmemKeys>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        Sh::kKeys * static_cast<int>(sizeof(uint32_t)));
    if (err != cudaSuccess) return err;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  // one wave of CTAs, at least 64 kept rows each
  const long long units = static_cast<long long>(args.batch) * kNumKvHeads;
  const long long parts = std::max(1LL, std::min(static_cast<long long>(Sh::kCtas) * num_sms / units,
                                                 (args.budget + 63LL) / 64));
  return launch_pdl(kv_evict_kernel<kKind, kSmemKeys>,
                    dim3(static_cast<unsigned>(kNumKvHeads * parts), args.batch),
                    dim3(Sh::kThreads), smem, stream, args);
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& args, int num_sms, cudaStream_t stream) {
  const int64_t tokens = static_cast<int64_t>(args.max_blocks) * kPageSize;
  if (tokens <= kSmallTokens) return launch<kSmall, true>(args, num_sms, stream);
  if (tokens <= kPairTokens && static_cast<int64_t>(args.batch) * kNumKvHeads > num_sms)
    return launch<kPair, true>(args, num_sms, stream);
  return tokens <= kSmemTokens ? launch<kLarge, true>(args, num_sms, stream)
                               : launch<kLarge, false>(args, num_sms, stream);
}

}  // namespace pkv
