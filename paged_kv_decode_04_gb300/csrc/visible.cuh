// visible.cuh -- the pages that a one-token query under a sliding window with
// sink tokens sees.
#pragma once

#include <stdint.h>

#include "pkv_device.cuh"

namespace pkv {

// The list of pages a query at position L - 1 sees.
struct Visible {
  int L, lo, sinks;  // t < L and (t >= lo or t < sinks)
  int ns, w0, n;     // sink pages in front, first page of the window, pages
  __device__ __forceinline__ Visible(int len, int window, int sink_tokens) {
    L = len;
    sinks = sink_tokens;
    lo = L > window ? L - window : 0;
    w0 = lo / kPageSize;
    ns = min((min(sinks, lo) + kPageSize - 1) / kPageSize, w0);
    n = L > 0 ? ns + (L + kPageSize - 1) / kPageSize - w0 : 0;
  }
  __device__ __forceinline__ int page(int k) const { return k < ns ? k : w0 + (k - ns); }
  // Is every slot of the page seen?
  __device__ __forceinline__ bool whole(int page) const {
    const int base = page * kPageSize;
    return base + kPageSize <= L && (base >= lo || base + kPageSize <= sinks);
  }
  // Bits of the page's slots that are seen.
  __device__ __forceinline__ uint32_t mask(int page) const {
    auto below = [](int x) { return x <= 0 ? 0u : (x >= kPageSize ? 0xFFFFu : (1u << x) - 1u); };
    const int base = page * kPageSize;
    return below(L - base) & ((0xFFFFu & ~below(lo - base)) | below(sinks - base));
  }
};

__device__ __forceinline__ int clamped_len(const MaskedArgs& a, int b, bool report) {
  const int Lmax = a.max_blocks * kPageSize;
  int L = a.seq_lens[b];
  if (L < 0 || L > Lmax) {
    if (report) record_error(a.dev_err, kErrSeqLen);
    L = L < 0 ? 0 : Lmax;
  }
  return L;
}

}  // namespace pkv
