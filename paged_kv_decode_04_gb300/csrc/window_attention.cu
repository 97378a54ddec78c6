// window_attention.cu -- attention of new tokens over the paged cache under a
// causal mask, a sliding window and sink tokens, and the accumulation of the
// attention weights.
//
// One CTA per (query token, kv head), one warp per query head of the group:
// lane i of a warp scores key t0 + i (64 dims in registers of the query), the
// warp takes one FP32 online-softmax step per 32 keys, and lane i then adds
// the weighted values of dims 2i and 2i + 1.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

// Dot product of a query row (floats in shared memory) and a key row.
__device__ __forceinline__ float dot_row(const float* q, const uint16_t* k) {
  const uint4* kw = reinterpret_cast<const uint4*>(k);
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 w = kw[c];
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = bf16x2_to_float2(ws[e]);
      s = fmaf(f.x, q[8 * c + 2 * e], s);
      s = fmaf(f.y, q[8 * c + 2 * e + 1], s);
    }
  }
  return s;
}

__global__ void __launch_bounds__(128) masked_attention_kernel(const MaskedArgs a) {
  __shared__ float s_q[kGroup][kHeadDim];
  __shared__ float s_m[kGroup], s_l[kGroup];
  const int g = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;  // query token
  wait_for_prior_grids();
  allow_dependent_grids();
  int b = static_cast<int>(row), ahead = 0;  // tokens of the sequence after this one
  if (a.token_offsets != nullptr) {
    if (row == 0 && g == 0)
      for (int i = threadIdx.x; i <= a.batch; i += 128) {
        const int32_t o = a.token_offsets[i];
        if (o < 0 || o > a.num_tokens || (i > 0 && o < a.token_offsets[i - 1]))
          record_error(a.dev_err, kErrOffsets);
      }
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.token_offsets[mid] <= row) lo = mid; else hi = mid;
    }
    b = lo;
    if (row < a.token_offsets[b] || row >= a.token_offsets[b + 1]) return;  // no sequence's token
    ahead = static_cast<int>(a.token_offsets[b + 1] - 1 - row);
  }
  const int Lmax = a.max_blocks * kPageSize;
  int L = a.seq_lens[b];
  if (L < 0 || L > Lmax) {
    if (threadIdx.x == 0) record_error(a.dev_err, kErrSeqLen);
    L = L < 0 ? 0 : Lmax;
  }
  const int pos = L - 1 - ahead;
  if (pos < 0 && a.token_offsets != nullptr && threadIdx.x == 0) record_error(a.dev_err, kErrPosition);
  const int64_t qrow = row * kNumQHeads + g * kGroup + warp;
  s_q[warp][2 * lane] = bf16_to_float(a.q[qrow * kHeadDim + 2 * lane]);
  s_q[warp][2 * lane + 1] = bf16_to_float(a.q[qrow * kHeadDim + 2 * lane + 1]);
  __syncwarp();
  const int first = pos >= a.window ? pos - a.window + 1 : 0;  // of the window
  const int sink = min(a.sinks, first);
  // visible index i: sinks, then the window
  const int n = pos < 0 ? 0 : sink + (pos + 1 - first);
  auto token = [&](int i) { return i < sink ? i : first + (i - sink); };
  auto key_row = [&](int t) -> const uint16_t* {
    const int32_t pid = a.block_table[static_cast<int64_t>(b) * a.max_blocks + t / kPageSize];
    if (pid < 0 || pid >= a.num_pages) {
      record_error(a.dev_err, kErrPage);
      return nullptr;
    }
    return a.pool + ((static_cast<int64_t>(pid) * 2 * kPageSize + t % kPageSize) * kNumKvHeads + g) *
                        kHeadDim;
  };
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const uint16_t* kr = i0 + lane < n ? key_row(token(i0 + lane)) : nullptr;
    const float s = kr != nullptr ? dot_row(s_q[warp], kr) * a.scale_log2 : -INFINITY;
    float mx = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, x));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;  // no live key so far
    const float r = fast_exp2(m - mn);
    const float p = kr != nullptr ? fast_exp2(s - mn) : 0.f;
    m = mn;
    l = l * r + p;
    o0 *= r;
    o1 *= r;
    for (int k = 0; k < 32; ++k) {
      const float pk = __shfl_sync(kFull, p, k);
      const unsigned long long vp = __shfl_sync(kFull, reinterpret_cast<unsigned long long>(kr), k);
      if (vp == 0) continue;
      const uint32_t w = reinterpret_cast<const uint32_t*>(
          reinterpret_cast<const uint16_t*>(vp) + kPageSize * kNumKvHeads * kHeadDim)[lane];
      const float2 v = bf16x2_to_float2(w);
      o0 = fmaf(pk, v.x, o0);
      o1 = fmaf(pk, v.y, o1);
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(kFull, l, x);
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  reinterpret_cast<uint32_t*>(a.out + qrow * kHeadDim)[lane] = pack_bf16x2(o0 * inv, o1 * inv);
  if (a.mass == nullptr) return;
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = inv;
  }
  __syncthreads();
  float* mass = a.mass + (static_cast<int64_t>(b) * kNumKvHeads + g) * a.mass_stride;
  for (int i = threadIdx.x; i < n; i += 128) {
    const int t = token(i);
    const uint16_t* kr = key_row(t);
    if (kr == nullptr) continue;
    float w = 0.f;
    for (int r = 0; r < kGroup; ++r)
      if (s_l[r] != 0.f) w += fast_exp2(dot_row(s_q[r], kr) * a.scale_log2 - s_m[r]) * s_l[r];
    mass[t] += w;
  }
}

}  // namespace

cudaError_t launch_masked_attention(const MaskedArgs& args, cudaStream_t stream) {
  return launch_pdl(masked_attention_kernel, dim3(args.num_tokens, kNumKvHeads), dim3(128), 0,
                    stream, args);
}

}  // namespace pkv
