// kv_evict.cu -- eviction from the paged cache by accumulated attention
// weight: each (sequence, kv head) keeps its first `sinks` tokens, its last
// `recent` ones and, of the others, the heaviest that fit the budget, packed
// in token order into the pages of another block table.
//
// Selection: the weights map to 32-bit keys whose unsigned order is the
// weights' order (NaN above +inf, -0 as +0); a radix descent of four 8-bit
// digits over shared-memory histograms finds the key of the last one kept
// and how many tokens of that key are kept, lowest index first.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kEvThreads = 256;
constexpr int kEvWarps = kEvThreads / 32;

// Order-preserving key of a weight.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kEvThreads) kv_evict_kernel(const EvictArgs a) {
  __shared__ int s_hist[256];
  __shared__ int s_warp[2][kEvWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.x, b = blockIdx.y;
  wait_for_prior_grids();
  allow_dependent_grids();
  const int Lmax = a.max_blocks * kPageSize;
  int L = a.seq_lens[b];
  if (L < 0 || L > Lmax) {
    if (tid == 0 && g == 0) record_error(a.dev_err, kErrSeqLen);
    L = L < 0 ? 0 : Lmax;
  }
  const int n = min(L, a.budget);
  const int64_t bg = static_cast<int64_t>(b) * kNumKvHeads + g;
  const float* mass = a.mass + bg * a.mass_stride;
  // tokens [lo, hi) compete; the others stay
  const bool all = L <= a.budget;
  const int lo = all ? L : a.sinks, hi = all ? L : L - a.recent;
  uint32_t thr = 0;
  int ties = 0;  // how many tokens of key thr are kept
  if (!all) {
    if (tid == 0) {
      s_prefix = 0;
      s_need = a.budget - a.sinks - a.recent;
    }
    for (int shift = 24; shift >= 0; shift -= 8) {
      s_hist[tid] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix;
      const uint32_t high = shift == 24 ? 0u : ~0u << (shift + 8);
      for (int t = lo + tid; t < hi; t += kEvThreads) {
        const uint32_t k = weight_key(mass[t]);
        if ((k & high) == (prefix & high)) atomicAdd(&s_hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int need = s_need, d = 255;
        while (d > 0 && s_hist[d] < need) need -= s_hist[d--];
        s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
        s_need = need;
      }
      __syncthreads();
    }
    thr = s_prefix;
    ties = s_need;
  }
  if (tid == 0 && g == 0) a.new_lens[b] = n;
  float* new_mass = a.new_mass + bg * a.new_mass_stride;
  int32_t* kept = a.kept + bg * a.budget;
  for (int64_t i = n + tid; i < a.new_mass_stride; i += kEvThreads) new_mass[i] = 0.f;
  for (int i = n + tid; i < a.budget; i += kEvThreads) kept[i] = -1;
  // tokens in order: kept ones get consecutive places
  int base = 0, eq_base = 0;
  for (int t0 = 0; t0 < L; t0 += kEvThreads) {
    const int t = t0 + tid;
    const bool in = t < L, free_ = in && t >= lo && t < hi;
    const float w = in ? mass[t] : 0.f;
    const uint32_t k = weight_key(w);
    const bool eq = free_ && k == thr;
    const unsigned eqb = __ballot_sync(0xFFFFFFFFu, eq);
    if (lane == 0) s_warp[0][warp] = __popc(eqb);
    __syncthreads();
    int eq_before = eq_base;
    for (int x = 0; x < warp; ++x) eq_before += s_warp[0][x];
    const int rank = eq_before + __popc(eqb & ((1u << lane) - 1u));
    const bool keep = in && (!free_ || k > thr || (eq && rank < ties));
    const unsigned kb = __ballot_sync(0xFFFFFFFFu, keep);
    if (lane == 0) s_warp[1][warp] = __popc(kb);
    __syncthreads();
    int at = base;
    for (int x = 0; x < warp; ++x) at += s_warp[1][x];
    at += __popc(kb & ((1u << lane) - 1u));
    for (int x = 0; x < kEvWarps; ++x) {
      base += s_warp[1][x];
      eq_base += s_warp[0][x];
    }
    __syncthreads();
    if (!keep) continue;
    kept[at] = t;
    new_mass[at] = w;
    const int32_t sp = a.block_table[static_cast<int64_t>(b) * a.max_blocks + t / kPageSize];
    const int32_t dp =
        a.dst_block_table[static_cast<int64_t>(b) * a.dst_max_blocks + at / kPageSize];
    if (sp < 0 || sp >= a.num_pages || dp < 0 || dp >= a.num_pages) {
      record_error(a.dev_err, kErrPage);
      continue;
    }
    for (int kv = 0; kv < 2; ++kv) {
      const uint4* src = reinterpret_cast<const uint4*>(
          a.pool + (((static_cast<int64_t>(sp) * 2 + kv) * kPageSize + t % kPageSize) * kNumKvHeads +
                    g) * kHeadDim);
      uint4* dst = reinterpret_cast<uint4*>(
          a.pool + (((static_cast<int64_t>(dp) * 2 + kv) * kPageSize + at % kPageSize) *
                        kNumKvHeads + g) * kHeadDim);
      for (int c = 0; c < 8; ++c) dst[c] = src[c];
    }
  }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& args, cudaStream_t stream) {
  return launch_pdl(kv_evict_kernel, dim3(kNumKvHeads, args.batch), dim3(kEvThreads), 0, stream,
                    args);
}

}  // namespace pkv
