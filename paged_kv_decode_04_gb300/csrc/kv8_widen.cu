// kv8_widen.cu -- the pages of an 8-bit cache that long chunks see, as bf16 pages
// in a workspace, where the tcgen05 kernel of chunk_attention.cu reads them.
//
// Every cached value is a bf16 number, so nothing is lost, and a long chunk reads
// its pages many times (64 new tokens to a tile, 8 kv heads): one pass that reads
// 1 KiB a token and writes 2 is small beside that.  The other way, converting in
// the attention kernel, was built and measured: four more warps of each CTA turning
// codes into f16 for every kv tile took 617 us (int8; e4m3 581) for 2 x 4096 tokens
// over 8192, of which the bf16 kernel takes 361, as the conversions compete with
// the softmax for issue slots and shared memory; 64 x 16 tokens over 2048, bound by
// memory, took 106 us there.
//
// One CTA to a page, warp h of it for kv head h, lane 8 r + q the codes [8 q, 8 q + 8)
// of slots r, r + 4, r + 8 and r + 12.  The pages are counted on through the batch (a scan
// of the lengths in every CTA), so their places follow from the sizes alone.
// Bound by memory: 11 us for the 1024 pages of 2 x 8192 tokens (50 MB); 4 us where
// there is no long chunk.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv8.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kThreads = 32 * kNumKvHeads;
constexpr int kSeqs = 2 * kThreads;  // sequences scanned at a time
constexpr unsigned kFull = 0xFFFFFFFFu;

// The pages that a long chunk's rows see: sinks' first, then the windows'.
struct Seen {
  int ns, w0, n;
  __device__ __forceinline__ int page(int i) const { return i < ns ? i : w0 + (i - ns); }
};

__device__ __forceinline__ Seen seen_pages(const WidenArgs& a, int b) {
  Seen s = {0, 0, 0};
  const int o0 = a.token_offsets[b], o1 = a.token_offsets[b + 1];
  if (o0 < 0 || o1 < o0 || o1 > a.num_tokens || o1 - o0 <= kShortTokens) return s;
  const int L = min(max(a.seq_lens[b], 0), a.cache.max_blocks * kPageSize);
  const int first = max(L - (o1 - o0), 0);
  const int lo = first >= a.window ? first - a.window + 1 : 0;
  s.w0 = lo / kPageSize;
  s.ns = min((min(a.sinks, lo) + kPageSize - 1) / kPageSize, s.w0);
  s.n = s.ns + (L + kPageSize - 1) / kPageSize - s.w0;
  return s;
}

template <int kFmt>
__global__ void __launch_bounds__(kThreads) widen_kernel(const WidenArgs a) {
  __shared__ int64_t s_base[kSeqs + 1];  // pages before each of the sequences scanned
  __shared__ int64_t s_warp[kNumKvHeads];
  const int tid = threadIdx.x, lane = tid & 31, h = tid >> 5;
  wait_for_prior_grids();
  allow_dependent_grids();
  const Kv8& c = a.cache;
  int64_t before = 0;
  for (int b0 = 0; b0 < c.batch; b0 += kSeqs) {
    // thread t takes sequences b0 + 2 t and b0 + 2 t + 1
    const int b = b0 + 2 * tid;
    const int n0 = b < c.batch ? seen_pages(a, b).n : 0;
    const int n1 = b + 1 < c.batch ? seen_pages(a, b + 1).n : 0;
    int64_t incl = static_cast<int64_t>(n0) + n1;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int64_t y = __shfl_up_sync(kFull, incl, x);
      if (lane >= x) incl += y;
    }
    if (lane == 31) s_warp[h] = incl;
    __syncthreads();
    int64_t base = before + incl - n0 - n1;
    for (int w = 0; w < h; ++w) base += s_warp[w];
    s_base[2 * tid] = base;
    s_base[2 * tid + 1] = base + n0;
    if (tid == kThreads - 1) s_base[kSeqs] = base + n0 + n1;
    if (a.rounds != nullptr && blockIdx.x == 0) {
      if (b < c.batch) a.rounds[b] = static_cast<int32_t>(base / a.per_round);
      if (b + 1 < c.batch) a.rounds[b + 1] = static_cast<int32_t>((base + n0) / a.per_round);
    }
    __syncthreads();
    const int64_t total = s_base[kSeqs];
    for (int64_t u = before + blockIdx.x; u < total; u += gridDim.x) {
      // the sequence of page u, the same in every thread
      int lo = 0, n = kSeqs;
      while (n > 1) {  // 32 places at a time
        const int step = (n + 31) / 32, at = lane * step;
        const unsigned below = __ballot_sync(kFull, at < n && s_base[lo + min(at, n - 1)] <= u);
        const int cut = (__popc(below) - 1) * step;
        lo += cut;
        n = min(step, n - cut);
      }
      const int64_t first = s_base[lo];
      const int64_t round = first / a.per_round;
      const int64_t place = u - round * a.per_round;
      if (round >= a.num_rounds || place >= a.places) {
        // (ranges of token_offsets that overlap: more chunks than the tokens allow)
        if (tid == 0) record_error(a.dev_err, kErrOffsets);
        continue;
      }
      if (round != a.round) continue;
      const int seq = b0 + lo;
      const Seen s = seen_pages(a, seq);
      const int page = s.page(static_cast<int>(u - first));
      const int64_t at = static_cast<int64_t>(seq) * c.max_blocks + page;
      const int pid = c.block_table[at];
      const bool good = pid >= 0 && pid < c.num_pages;
      if (tid == 0) a.table[at] = good ? static_cast<int32_t>(place) : -1;
      if (!good) continue;  // (reported where it is read)
      const int r = lane >> 3, q = lane & 7;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint2* src = reinterpret_cast<const uint2*>(c.pool + block_at(pid, kv, h)) + lane;
        uint2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __ldcs(src + 32 * i);
        const float f = scale_value(stored_scale(c.scales[scale_at(pid, kv, h)]));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(
              a.pages +
              (((place * 2 + kv) * kPageSize + r + 4 * i) * kNumKvHeads + h) * kHeadDim + 8 * q) =
              widen8<kFmt>(w[i], f);
      }
    }
    before = total;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_widen(const WidenArgs& args, int num_sms, cudaStream_t stream) {
  return launch_pdl(args.cache.format == kKv8E4m3 ? widen_kernel<kKv8E4m3> : widen_kernel<kKv8Int8>,
                    dim3(static_cast<int>(std::min<int64_t>(num_sms * 8, args.places))),
                    dim3(kThreads), 0, stream, args);
}

}  // namespace pkv
