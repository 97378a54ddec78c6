// kv8_write.cu -- writing the 8-bit cache (one token a sequence, or ragged
// prompts) with rotate-half RoPE on the way, and reading it back as bf16.
//
// The key that is rounded to a block's scale is the one a bf16 cache would hold
// (rotate_pair's bits).  A block's scale is the smallest power of two that takes
// the largest magnitude it was given to at most the largest code; tokens that
// come to a block holding earlier ones keep at least its scale, and round the
// earlier codes again where they need a larger one.  Values that are not finite
// are stored as zero and reported (kErrValue).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "kv8.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kHalf = kHeadDim / 2;
constexpr int kThreads = 32 * kNumKvHeads;  // a warp to a kv head
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

__device__ __forceinline__ bool finite_bf16(uint32_t h) { return (h & 0x7F80u) != 0x7F80u; }

// (cos, sin) of a rotation, as floats and what they leave.
struct Angle {
  float c, s, c_lo, s_lo;
};
__device__ __forceinline__ Angle make_angle(double c, double s) {
  Angle t;
  t.c = static_cast<float>(c);
  t.s = static_cast<float>(s);
  t.c_lo = static_cast<float>(__dsub_rn(c, static_cast<double>(t.c)));
  t.s_lo = static_cast<float>(__dsub_rn(s, static_cast<double>(t.s)));
  return t;
}

// x + y and what rounding it left.
__device__ __forceinline__ float two_sum(float x, float y, float& e) {
  const float h = __fadd_rn(x, y), z = __fsub_rn(h, x);
  e = __fadd_rn(__fsub_rn(x, __fsub_rn(h, z)), __fsub_rn(y, z));
  return h;
}

// a c + b s rounded once to bf16, where FP32 with the rounding errors carried along
// decides it: off by at most 2^-43 (|a| + |b|) (2^-24 of terms of 2^-23 of that, and
// what is left of cos and sin), it rounds as the exact value, and as FP64, unless it
// is that close to a midpoint or so small that half its FP32 spacing is below that.
// a, b: bf16 values, not too far from 1.
__device__ __forceinline__ bool turn_exactly(float a, float b, const Angle& t, uint16_t* out) {
  const float p = a * t.c, q = b * t.s;
  const float pe = fmaf(a, t.c, -p), qe = fmaf(b, t.s, -q);  // exactly what they left
  float e, lo;
  const float h = two_sum(p, q, e);
  const float hi = two_sum(h, __fadd_rn(e, __fadd_rn(__fadd_rn(pe, qe),
                                                     fmaf(a, t.c_lo, b * t.s_lo))), lo);
  // hi + lo is on hi's side of a bf16 midpoint, half a spacing from it, unless hi is
  // one
  const uint32_t bits = __float_as_uint(hi);
  const float s0 = fabsf(a) + fabsf(b);
  const bool large = fabsf(hi) > 0x1p-18f * s0;
  if ((bits & 0xFFFFu) != 0x8000u) {
    *out = float_to_bf16_rne(hi);
    return large;
  }
  const float away = hi < 0.f ? -lo : lo;  // beyond the midpoint, as a magnitude
  *out = static_cast<uint16_t>((bits >> 16) + (away > 0.f ? 1u : 0u));
  return large && fabsf(lo) > 0x1p-43f * s0;
}

// Both values of a rotated pair, rotate_pair's bits.
__device__ __noinline__ uint2 rotate_in_fp64(uint32_t h1, uint32_t h2, int pos, double freq) {
  double c, s;
  sincos(__dmul_rn(static_cast<double>(pos), freq), &s, &c);
  uint16_t y1, y2;
  rotate_pair(static_cast<uint16_t>(h1), static_cast<uint16_t>(h2), c, s, &y1, &y2);
  return make_uint2(y1, y2);
}
__device__ __forceinline__ void rotate_carefully(uint32_t h1, uint32_t h2, const Angle& t,
                                                 int pos, const double* freq, uint16_t* y1,
                                                 uint16_t* y2) {
  const float u = __uint_as_float(h1 << 16), v = __uint_as_float(h2 << 16);
  const float s0 = fabsf(u) + fabsf(v);
  // (tiny, huge, not finite: FP32 would lose them)
  const bool fine = s0 >= 0x1p-70f && s0 <= 0x1p+100f;
  Angle n = t;
  n.s = -t.s;
  n.s_lo = -t.s_lo;
  const bool ok1 = turn_exactly(u, v, n, y1), ok2 = turn_exactly(v, u, t, y2);
  if (!(fine && ok1 && ok2)) {
    const uint2 y = rotate_in_fp64(h1 & 0xFFFFu, h2 & 0xFFFFu, pos, *freq);
    *y1 = static_cast<uint16_t>(y.x);
    *y2 = static_cast<uint16_t>(y.y);
  }
}

// FP32 rotation (a c + b s) with a bound on its error: values at and below, and at
// and above, the FP64 one.  y is off by at most 3 x 2^-24 (|a| + |b|): 2^-24 of both
// factors for cos and sin, of one product, and of y, |y| <= |a| + |b|; y - A and y + A,
// A = 1.125 x 2^-22 (|a| + |b|), are off by another 2^-24 of that.  For |a| + |b| in
// [2^-70, 2^100].
constexpr float kTurnBound = 0x1.2p-22f;
constexpr uint32_t kTiny = (127u - 60u) << 7, kHuge = (127u + 99u) << 7;  // bf16 2^-60, 2^99

// A warp stores the largest magnitude's scale of a block that holds `earlier`
// tokens already, whose codes follow it, and returns the scale.
template <int kFmt>
__device__ __forceinline__ uint32_t settle_scale(const Kv8& c, int64_t page, int kv, int g,
                                                 uint32_t top, int earlier, uint32_t old,
                                                 int lane) {
  uint32_t e = needed_scale<kFmt>(top);
  if (earlier > 0) {
    if (e > old) {
      rescale_rows<kFmt>(c.pool + block_at(page, kv, g), earlier, e - old, lane);
    } else {
      e = old;
    }
  }
  if (lane == 0) c.scales[scale_at(page, kv, g)] = static_cast<uint8_t>(e);
  return e;
}

// One CTA per sequence, warp h of it for kv head h: lane i rotates pair i of K
// (and of query heads h, h + 8, h + 16, h + 24 when asked) and takes dims 2i and
// 2i + 1 of V.  Bound by its chain of loads (position, page, scale, codes to round
// again): 13 us for 2048 sequences, three waves of five CTAs an SM, 6 for one wave.
template <int kFmt>
__global__ void __launch_bounds__(kThreads)
    kv8_append_kernel(const uint16_t* __restrict__ k_new, const uint16_t* __restrict__ v_new,
                      const Kv8 c, const int32_t* __restrict__ positions,
                      const int32_t* __restrict__ slots,
                      const __grid_constant__ RopeFreqs freqs,
                      const uint16_t* __restrict__ q_in, uint16_t* __restrict__ q_out,
                      int32_t* dev_err) {
  const int b = blockIdx.x;
  const int tid = threadIdx.x;
  const int h = tid / kHalf, i = tid % kHalf;
  wait_for_prior_grids();
  allow_dependent_grids();

  const int64_t src = (static_cast<int64_t>(b) * kNumKvHeads + h) * kHeadDim;
  const uint16_t k1 = k_new[src + i];
  const uint16_t k2 = k_new[src + i + kHalf];
  const uint32_t vw = reinterpret_cast<const uint32_t*>(v_new + src)[i];
  const bool table_ok = rope_table_ready(freqs);
  const int32_t pos = positions[b];
  const int32_t at = slots != nullptr ? slots[b] : pos;
  const bool pos_ok = pos >= 0 && at >= 0 && at < c.max_blocks * kPageSize;
  const int32_t page =
      pos_ok ? c.block_table[static_cast<int64_t>(b) * c.max_blocks + at / kPageSize] : -1;
  const bool page_ok = page >= 0 && page < c.num_pages;
  const int slot = at % kPageSize;
  // (scales of a fresh block are not read)
  uint32_t old_k = 0, old_v = 0;
  if (page_ok && slot > 0) {
    old_k = stored_scale(c.scales[scale_at(page, 0, h)]);
    old_v = stored_scale(c.scales[scale_at(page, 1, h)]);
  }
  // Past the table a pair's FP64 sincos is taken once and shared by the 8 heads'
  // threads (as in kv_append_kernel); a table that is still being built is left to
  // each thread.
  __shared__ Angle s_angle[kHalf];
  Angle t;
  auto angle = [&]() { return __dmul_rn(static_cast<double>(pos), freqs.inv_freq[i]); };
  if (freqs.table_theta == nullptr || pos < 0 || pos >= kRopeTablePositions) {
    if (h == 0) {
      double s64, c64;
      sincos(angle(), &s64, &c64);
      s_angle[i] = make_angle(c64, s64);
    }
    __syncthreads();
    t = s_angle[i];
  } else if (table_ok) {
    const float2 hi = freqs.table32[pos * kHalf + i], lo = freqs.table_lo[pos * kHalf + i];
    t = {hi.x, hi.y, lo.x, lo.y};
  } else {
    double s64, c64;
    sincos(angle(), &s64, &c64);
    t = make_angle(c64, s64);
  }
  auto rotate = [&](uint16_t x1, uint16_t x2, uint16_t* y1, uint16_t* y2) {
    const float u = bf16_to_float(x1), v = bf16_to_float(x2), s0 = fabsf(u) + fabsf(v);
    const float a = fmaf(u, t.c, -(v * t.s)), b = fmaf(v, t.c, u * t.s), A = s0 * kTurnBound;
    const uint32_t lo = cvt_bf16x2_rn(a - A, b - A);
    *y1 = static_cast<uint16_t>(lo);
    *y2 = static_cast<uint16_t>(lo >> 16);
    // (zeros keep their signs in FP32)
    if (s0 != 0.f &&
        (lo != cvt_bf16x2_rn(a + A, b + A) || !(s0 >= 0x1p-70f && s0 <= 0x1p+100f)))
      rotate_carefully(x1, x2, t, pos, freqs.inv_freq + i, y1, y2);
  };

  if (q_in != nullptr) {
    const int64_t qbase = static_cast<int64_t>(b) * kNumQHeads * kHeadDim;
    uint16_t x1[4], x2[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t o = qbase + (h + 8 * k) * kHeadDim + i;
      x1[k] = q_in[o];
      x2[k] = q_in[o + kHalf];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t o = qbase + (h + 8 * k) * kHeadDim + i;
      uint16_t y1, y2;
      rotate(x1[k], x2[k], &y1, &y2);
      q_out[o] = y1;
      q_out[o + kHalf] = y2;
    }
  }
  if (!page_ok) {
    if (tid == 0) record_error(dev_err, pos_ok ? kErrPage : kErrPosition);
    return;
  }

  uint16_t y1, y2;
  rotate(k1, k2, &y1, &y2);
  uint32_t v1 = vw & 0xFFFFu, v2 = vw >> 16;
  if (!finite_bf16(y1) || !finite_bf16(y2) || !finite_bf16(v1) || !finite_bf16(v2)) {
    record_error(dev_err, kErrValue);
    if (!finite_bf16(y1)) y1 = 0;
    if (!finite_bf16(y2)) y2 = 0;
    if (!finite_bf16(v1)) v1 = 0;
    if (!finite_bf16(v2)) v2 = 0;
  }
  const uint32_t top_k = __reduce_max_sync(kFull, max(y1 & 0x7FFFu, y2 & 0x7FFFu));
  const uint32_t top_v = __reduce_max_sync(kFull, max(v1 & 0x7FFFu, v2 & 0x7FFFu));
  const uint32_t ek = settle_scale<kFmt>(c, page, 0, h, top_k, slot, old_k, i);
  const uint32_t ev = settle_scale<kFmt>(c, page, 1, h, top_v, slot, old_v, i);
  const float fk = scale_inverse(ek), fv = scale_inverse(ev);
  const uint32_t wk = encode4<kFmt, true>(bf16_to_float(y1), bf16_to_float(y2), 0.f, 0.f, fk);
  const uint32_t wv =
      encode4<kFmt, true>(__uint_as_float(v1 << 16), __uint_as_float(v2 << 16), 0.f, 0.f, fv);
  uint8_t* kd = c.pool + block_at(page, 0, h) + slot * kHeadDim;
  uint8_t* vd = c.pool + block_at(page, 1, h) + slot * kHeadDim;
  kd[i] = static_cast<uint8_t>(wk);
  kd[i + kHalf] = static_cast<uint8_t>(wk >> 8);
  reinterpret_cast<uint16_t*>(vd)[i] = static_cast<uint16_t>(wv);
}

// A unit is one page of one sequence.  Units are numbered so that a sequence's
// first is off[b] / 16 + 2 b: n tokens touch at most n / 16 + 2 pages, so the
// ranges of numbers do not meet (some numbers name no page), and the sequence of
// a unit is found by search, without a prefix sum.  A CTA takes consecutive
// numbers, 32 at a time: each lane finds one unit, so the searches and the loads
// behind them (lengths, places, table entries) cost their latency once for 32.
struct Unit {
  int64_t row0;         // row of k and v of the token in slot 0 of the page
  int pool_page;        // -1: no unit
  int page;             // page of the sequence
  int s0, s1;           // slots [s0, s1) are the call's
};

__host__ __device__ inline int64_t unit_count(int num_tokens, int batch) {
  return num_tokens / kPageSize + 2 * static_cast<int64_t>(batch);
}

__device__ __forceinline__ bool bad_offsets(int o0, int o1, int num_tokens) {
  return o0 < 0 || o1 < o0 || o1 > num_tokens;
}

// The unit of number u, by each lane for itself (found where offsets do not fall);
// `report`: one warp of a CTA reports what is wrong with it.
__device__ __forceinline__ Unit find_unit(int64_t u, int64_t end, const Kv8& c,
                                          const int32_t* __restrict__ off,
                                          const int32_t* __restrict__ starts, int num_tokens,
                                          int32_t* dev_err, bool report) {
  Unit r = {0, -1, 0, 0, 0};
  if (u >= end) return r;
  auto first = [&](int b) { return static_cast<int64_t>(off[b] / kPageSize) + 2ll * b; };
  int lo = 0, hi = c.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first(mid) <= u) lo = mid; else hi = mid;
  }
  const int o0 = off[lo], o1 = off[lo + 1];
  if (bad_offsets(o0, o1, num_tokens)) return r;  // (reported by check_offsets)
  const int64_t start = starts[lo], past = start + (o1 - o0);
  const int64_t limit = static_cast<int64_t>(c.max_blocks) * kPageSize;
  const int64_t p0 = start > 0 ? start : 0, p1 = past < limit ? past : limit;
  if (o1 > o0 && (p0 != start || p1 != past) && report) record_error(dev_err, kErrPosition);
  const int64_t page = p0 / kPageSize + (u - first(lo));
  if (u < first(lo) || p1 <= p0 || page * kPageSize >= p1) return r;
  const int pid = c.block_table[static_cast<int64_t>(lo) * c.max_blocks + page];
  if (pid < 0 || pid >= c.num_pages) {
    if (report) record_error(dev_err, kErrPage);
    return r;
  }
  r.pool_page = pid;
  r.page = static_cast<int>(page);
  r.s0 = max(static_cast<int>(p0 - page * kPageSize), 0);
  r.s1 = p1 - page * kPageSize < kPageSize ? static_cast<int>(p1 - page * kPageSize) : kPageSize;
  r.row0 = o0 + page * kPageSize - start;
  return r;
}

// Lane `src`'s unit.
__device__ __forceinline__ Unit unit_of(const Unit& t, int src) {
  Unit r;
  r.row0 = __shfl_sync(kFull, t.row0, src);
  r.pool_page = __shfl_sync(kFull, t.pool_page, src);
  r.page = __shfl_sync(kFull, t.page, src);
  const int s = __shfl_sync(kFull, t.s0 | (t.s1 << 8), src);
  r.s0 = s & 0xFF;
  r.s1 = s >> 8;
  return r;
}

// The numbers [u0, u1) of a CTA.
struct Share {
  int64_t u0, u1;
  __device__ __forceinline__ explicit Share(int64_t units) {
    u0 = units * blockIdx.x / gridDim.x;
    u1 = units * (blockIdx.x + 1) / gridDim.x;
  }
};

// Offsets that do not begin at 0 and end at the number of tokens, or are bad between;
// by the first CTA, as units of sequences with bad ones may not be found.
__device__ __forceinline__ void check_offsets(const Kv8& c, const int32_t* off, int num_tokens,
                                              int32_t* dev_err) {
  if (blockIdx.x != 0) return;
  bool bad = threadIdx.x == 0 && (off[0] != 0 || off[c.batch] != num_tokens);
  for (int b = threadIdx.x; b < c.batch; b += kThreads)
    bad |= bad_offsets(off[b], off[b + 1], num_tokens);
  if (bad) record_error(dev_err, kErrOffsets);
}

// RoPE of the 8 pairs (x1, x2) = dims (8 q + p, 32 + 8 q + p) of a row: x1, x2 become
// bf16 values at or below the rotated ones, y1, y2 at or above them (mostly the same:
// one pair in 500 differs, where its values cancel or one is much larger).  turn: the
// pairs' (cos, sin) in shared memory.
__device__ __forceinline__ void rotate8(uint32_t turn, uint4& x1, uint4& x2, uint4& y1,
                                        uint4& y2) {
  const uint32_t a[4] = {x1.x, x1.y, x1.z, x1.w}, b[4] = {x2.x, x2.y, x2.z, x2.w};
  uint32_t l1[4], l2[4], h1[4], h2[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint4 w = lds128(turn + 16 * e);
    const float2 u = bf16x2_to_float2(a[e]), v = bf16x2_to_float2(b[e]);
    const float c0 = __uint_as_float(w.x), s0 = __uint_as_float(w.y);
    const float c1 = __uint_as_float(w.z), s1 = __uint_as_float(w.w);
    const float p0 = fmaf(u.x, c0, -(v.x * s0)), q0 = fmaf(v.x, c0, u.x * s0);
    const float p1 = fmaf(u.y, c1, -(v.y * s1)), q1 = fmaf(v.y, c1, u.y * s1);
    const float A0 = (fabsf(u.x) + fabsf(v.x)) * kTurnBound;
    const float A1 = (fabsf(u.y) + fabsf(v.y)) * kTurnBound;
    l1[e] = cvt_bf16x2_rn(p0 - A0, p1 - A1);
    l2[e] = cvt_bf16x2_rn(q0 - A0, q1 - A1);
    h1[e] = cvt_bf16x2_rn(p0 + A0, p1 + A1);
    h2[e] = cvt_bf16x2_rn(q0 + A0, q1 + A1);
  }
  x1 = make_uint4(l1[0], l1[1], l1[2], l1[3]);
  x2 = make_uint4(l2[0], l2[1], l2[2], l2[3]);
  y1 = make_uint4(h1[0], h1[1], h1[2], h1[3]);
  y2 = make_uint4(h2[0], h2[1], h2[2], h2[3]);
}

// a x + b y of factors given as float pairs, rounded to float: off by 2^-25 where it is
// at most 1.
__device__ __forceinline__ float dot2(float a, float a_lo, float x, float x_lo, float b,
                                      float b_lo, float y, float y_lo) {
  const float p = __fmul_rn(a, x), pe = fmaf(a, x, -p), q = __fmul_rn(b, y), qe = fmaf(b, y, -q);
  float e;
  const float h = two_sum(p, q, e);
  return h + (e + (pe + qe) + fmaf(a, x_lo, b * y_lo) + fmaf(a_lo, x, b_lo * y));
}

// Bits of the pairs whose bounds differ.
__device__ __forceinline__ uint32_t pairs_apart(const uint4& x1, const uint4& x2, const uint4& y1,
                                                const uint4& y2) {
  const uint32_t d[4] = {(x1.x ^ y1.x) | (x2.x ^ y2.x), (x1.y ^ y1.y) | (x2.y ^ y2.y),
                         (x1.z ^ y1.z) | (x2.z ^ y2.z), (x1.w ^ y1.w) | (x2.w ^ y2.w)};
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((d[e] & 0xFFFFu) != 0u) m |= 1u << (2 * e);
    if ((d[e] >> 16) != 0u) m |= 2u << (2 * e);
  }
  return m;
}

// The pairs `bad` of a row again, exactly, from shared memory (the row's x1 at `row`,
// x2 64 bytes on; `left`: what the angles' floats leave, if it is known) and through it,
// by an index that is each lane's own: words picked so would go to memory.
__device__ __forceinline__ void rotate_again(uint32_t bad, const double* inv_freq, uint32_t row,
                                             uint32_t turn, const float2* left, int pos,
                                             uint4& x1, uint4& x2) {
  for (uint32_t rest = bad; rest != 0; rest &= rest - 1) {
    const int p = __ffs(rest) - 1;
    uint16_t y1, y2;
    if (left == nullptr) {
      const uint2 y = rotate_in_fp64(lds16(row + 2 * p), lds16(row + 64 + 2 * p), pos,
                                      inv_freq[p]);
      y1 = static_cast<uint16_t>(y.x);
      y2 = static_cast<uint16_t>(y.y);
    } else {
      const uint2 hi = lds64(turn + 8 * p);
      const float2 lo = left[p];
      const Angle t = {__uint_as_float(hi.x), __uint_as_float(hi.y), lo.x, lo.y};
      rotate_carefully(lds16(row + 2 * p), lds16(row + 64 + 2 * p), t, pos, inv_freq + p, &y1,
                       &y2);
    }
    sts16(row + 2 * p, y1);
    sts16(row + 64 + 2 * p, y2);
  }
  const uint4 c1 = lds128(row), c2 = lds128(row + 64);
  const uint32_t w1[4] = {c1.x, c1.y, c1.z, c1.w}, w2[4] = {c2.x, c2.y, c2.z, c2.w};
  uint32_t o1[4] = {x1.x, x1.y, x1.z, x1.w}, o2[4] = {x2.x, x2.y, x2.z, x2.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t m = ((bad >> (2 * e)) & 1u ? 0xFFFFu : 0u) |
                       ((bad >> (2 * e)) & 2u ? 0xFFFF0000u : 0u);
    o1[e] = (o1[e] & ~m) | (w1[e] & m);
    o2[e] = (o2[e] & ~m) | (w2[e] & m);
  }
  x1 = make_uint4(o1[0], o1[1], o1[2], o1[3]);
  x2 = make_uint4(o2[0], o2[1], o2[2], o2[3]);
}

// Zero the values of 8 that are not finite.
__device__ __forceinline__ void drop_nonfinite(uint4& x) {
  x = make_uint4(x.x & ~nonfinite_halves(x.x), x.y & ~nonfinite_halves(x.y),
                 x.z & ~nonfinite_halves(x.z), x.w & ~nonfinite_halves(x.w));
}

// The larger magnitude of each half (NaN where there is one), under a sign of no
// meaning.
__device__ __forceinline__ uint32_t top2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t top8(const uint4& x) {
  return top2(top2(x.x, x.y), top2(x.z, x.w));
}

// Magnitudes past 127 x 2^113, the largest that scales reach, become that.
__device__ __forceinline__ void saturate8(uint4& x) {
  uint32_t* w = &x.x;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (w[i] & 0x80008000u) | __vminu2(w[i] & 0x7FFF7FFFu, 0x7B7E7B7Eu);
}

template <int kFmt>
__device__ __forceinline__ uint2 encode8(const uint4& x, float f) {
  const float2 a = bf16x2_to_float2(x.x), b = bf16x2_to_float2(x.y), c = bf16x2_to_float2(x.z),
               d = bf16x2_to_float2(x.w);
  return make_uint2(encode4<kFmt, false>(a.x, a.y, b.x, b.y, f),
                    encode4<kFmt, false>(c.x, c.y, d.x, d.y, f));
}

// Ragged prompts: a CTA brings its units' rows of k and v (16 KiB each, in a row)
// into a ring of two stages in shared memory, so the next unit's are on their way
// while one is rotated and rounded, with the angles of its 16 positions, 4 KiB of the
// table; past the table they are worked out once for all heads.  Warp h takes the K and
// the V block of kv head h: lane 4 r + q holds dims [8 q, 8 q + 8) and [32 + 8 q, 32 +
// 8 q + 8) of slots r and r + 8 (odd r their other half first: a phase of 8 lanes then
// covers all banks).  Warp 0 fills the ring; the warps run apart by up to two units
// (barriers of the whole CTA instead: 79 us).
//
// Bound by its instructions, 960 a warp and unit at 61% of the issue slots: 64 prompts of
// 1024 to 2047 tokens (306 MB) 70 us, 4.4 TB/s.
constexpr int kWriteStages = 2, kWriteCtas = 3;
constexpr int kTokenBytes = kNumKvHeads * kHeadDim * 2;        // a row of k or v
constexpr int kHalfStage = kPageSize * kTokenBytes;            // 16 KiB
constexpr int kTurnRow = kHalf + 4;  // (cos, sin) of a position, and padding: two positions a phase
constexpr int kTurnBytes = kPageSize * kTurnRow * 8;
constexpr int kOffTurn = kWriteStages * 2 * kHalfStage;       // a stage's (cos, sin)
constexpr int kOffFirst = kOffTurn + kWriteStages * kTurnBytes;  // its first position's Angles
constexpr int kOffWriteBars = kOffFirst + kWriteStages * kHalf * 16;  // full, empty
constexpr size_t kWriteSmem = kOffWriteBars + 2 * 8 * kWriteStages;
static_assert(kWriteCtas * (kWriteSmem + 1024) <= 228 * 1024, "the CTAs of an SM fit");

template <int kFmt>
__global__ void __launch_bounds__(kThreads, kWriteCtas)
    kv8_write_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                     int num_tokens, const int32_t* __restrict__ off,
                     const int32_t* __restrict__ starts, const Kv8 c,
                     const __grid_constant__ RopeFreqs freqs, int32_t* dev_err,
                     unsigned long long wait_ns) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, h = tid >> 5;
  const int r = lane >> 2, q = lane & 3;
  const uint32_t sb = smem_addr(smem);
  auto full = [&](int st) { return sb + kOffWriteBars + 8 * st; };
  auto empty = [&](int st) { return sb + kOffWriteBars + 8 * (kWriteStages + st); };
  if (tid == 0) {
    for (int s = 0; s < kWriteStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kNumKvHeads);
    }
    fence_barrier_init();
  }
  __syncthreads();
  wait_for_prior_grids();
  allow_dependent_grids();
  check_offsets(c, off, num_tokens, dev_err);
  // The tag may be set meanwhile, by the call that builds the table on another stream,
  // and the warps' barriers, the copies and who works out the angles follow it: one
  // answer for the CTA.
  const bool tag_ok = __syncthreads_and(rope_table_ready(freqs));
  const Share share(unit_count(num_tokens, c.batch));
  const uint64_t policy = l2_policy_evict_first();
  int issued = 0, done = 0;  // units whose rows were asked for, units written
  auto is_near = [&](const Unit& t) {
    return tag_ok && (t.page + 1) * kPageSize <= kRopeTablePositions;
  };
  // Past the tables a page's angles are those of its first position turned by those of
  // positions 0 to 15: one FP64 sincos for a pair and page, not 16 (64 x 1536 tokens
  // from 4096 on took 240 us with those, 94 with this).  The angle itself, position x
  // frequency rounded to FP64, is then off by 2^-52 of it: below 2^24 by 2^-28, which
  // rotate8's bounds hold.
  const float top_freq = static_cast<float>(fmax(freqs.inv_freq[0], freqs.inv_freq[kHalf - 1]));
  auto is_far = [&](const Unit& t) {
    return tag_ok && static_cast<float>(t.page + 1) * kPageSize * top_freq <= 0x1p24f;
  };
  bool ok = true;
  for (int64_t u0 = share.u0; ok && u0 < share.u1; u0 += 32) {
    const Unit mine =
        find_unit(u0 + lane, share.u1, c, off, starts, num_tokens, dev_err, h == 0);
    // the units there are, in order; the same in every warp
    unsigned todo = __ballot_sync(kFull, mine.pool_page >= 0), ahead = todo;
    auto ask = [&]() {  // warp 0: the next unit's rows and angles into the next stage
      if (ahead == 0) return;
      const Unit t = unit_of(mine, __ffs(ahead) - 1);
      ahead &= ahead - 1;
      const int st = issued % kWriteStages;
      if (issued >= kWriteStages &&
          !__all_sync(kFull, mbar_wait_bounded(empty(st), (issued / kWriteStages - 1) & 1,
                                               wait_ns))) {
        ok = false;
        return;
      }
      const bool near = is_near(t);
      if (lane == 0) {
        const uint32_t dst = sb + st * 2 * kHalfStage;
        const uint32_t bytes = (t.s1 - t.s0) * kTokenBytes;
        const int64_t at = (t.row0 + t.s0) * (kTokenBytes / 2);
        mbar_arrive_expect_tx(full(st), 2 * bytes + (near ? kPageSize * kHalf * 8 : 0));
        bulk_load(dst + t.s0 * kTokenBytes, k + at, bytes, full(st), policy);
        bulk_load(dst + kHalfStage + t.s0 * kTokenBytes, v + at, bytes, full(st), policy);
      }
      __syncwarp();
      if (near && lane < kPageSize)
        bulk_load(sb + kOffTurn + st * kTurnBytes + lane * kTurnRow * 8,
                  freqs.table32 + (static_cast<int64_t>(t.page) * kPageSize + lane) * kHalf,
                  kHalf * 8, full(st), policy);
      ++issued;
    };
    if (h == 0)
      for (int s = 0; s < kWriteStages && ok; ++s) ask();
    while (ok && todo != 0) {
      const Unit t = unit_of(mine, __ffs(todo) - 1);
      todo &= todo - 1;
      const int st = done % kWriteStages;
      const int pos0 = t.page * kPageSize;
      const uint32_t old_k = t.s0 > 0 ? c.scales[scale_at(t.pool_page, 0, h)] : 0u;
      const uint32_t old_v = t.s0 > 0 ? c.scales[scale_at(t.pool_page, 1, h)] : 0u;
      ok = __all_sync(kFull, mbar_wait_bounded(full(st), (done / kWriteStages) & 1, wait_ns));
      if (!ok) break;
      const bool near = is_near(t), far = !near && is_far(t);
      float2* turn = reinterpret_cast<float2*>(smem + kOffTurn + st * kTurnBytes);
      float4* first = reinterpret_cast<float4*>(smem + kOffFirst) + st * kHalf;
      if (far) {  // (a warp in turn: the others wait for its sincos)
        if (h == done % kNumKvHeads) {
          double s64, c64;
          sincos(__dmul_rn(static_cast<double>(pos0), freqs.inv_freq[lane]), &s64, &c64);
          const Angle f = make_angle(c64, s64);
          first[lane] = make_float4(f.c, f.s, f.c_lo, f.s_lo);
        }
      } else if (!near) {
        for (int i = tid; i < kPageSize * kHalf; i += kThreads) {
          double s64, c64;
          sincos(__dmul_rn(static_cast<double>(pos0 + i / kHalf), freqs.inv_freq[i % kHalf]), &s64,
                 &c64);
          turn[i / kHalf * kTurnRow + i % kHalf] =
              make_float2(static_cast<float>(c64), static_cast<float>(s64));
        }
      }
      ++done;
      const uint32_t rows = sb + st * 2 * kHalfStage + h * (kHeadDim * 2) + 16 * q;
      uint4 x[2][2];  // [slot r, r + 8][dims 8 q, 32 + 8 q]
      auto load = [&](uint32_t at) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bool in = r + 8 * s >= t.s0 && r + 8 * s < t.s1;
          const uint32_t row = at + (r + 8 * s) * kTokenBytes;
          const uint4 y = lds128(row + 64 * (r & 1)), z = lds128(row + 64 * (~r & 1));
          const uint4 none = make_uint4(0u, 0u, 0u, 0u);
          x[s][0] = !in ? none : r & 1 ? z : y;
          x[s][1] = !in ? none : r & 1 ? y : z;
        }
      };
      auto top_of = [&](const uint4 (&y)[2][2]) {
        const uint32_t m =
            top2(top2(top8(y[0][0]), top8(y[0][1])), top2(top8(y[1][0]), top8(y[1][1])));
        return __reduce_max_sync(kFull, max(m & 0x7FFFu, (m >> 16) & 0x7FFFu));
      };
      // the largest magnitude, values that are not finite left out
      auto largest = [&](uint4 (&y)[2][2]) {
        const uint32_t top = top_of(y);
        if (top < 0x7F80u) return top;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          drop_nonfinite(y[s][0]);
          drop_nonfinite(y[s][1]);
        }
        if (lane == 0) record_error(dev_err, kErrValue);
        return top_of(y);
      };
      auto put = [&](int kv, uint32_t top, uint32_t old, const uint2 (&codes)[2][2]) {
        settle_scale<kFmt>(c, t.pool_page, kv, h, top, t.s0, old, lane);
        uint8_t* block = c.pool + block_at(t.pool_page, kv, h) + 8 * q;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int slot = r + 8 * s;
          if (slot < t.s0 || slot >= t.s1) continue;
#pragma unroll
          for (int d = 0; d < 2; ++d)
            *reinterpret_cast<uint2*>(block + slot * kHeadDim + kHalf * d) = codes[s][d];
        }
      };
      // codes of values whose largest is `top`
      auto encode = [&](uint4 (&y)[2][2], uint32_t top, uint32_t old, uint2 (&codes)[2][2]) {
        uint32_t e = needed_scale<kFmt>(top);
        if (t.s0 > 0) e = max(e, old);
        const float f = scale_inverse(e);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            if (kFmt == kKv8Int8 && e == kMostScale) saturate8(y[s][d]);
            codes[s][d] = encode8<kFmt>(y[s][d], f);
          }
      };
      uint2 codes[2][2];
      {
        load(rows + kHalfStage);
        const uint32_t top = largest(x), old = stored_scale(old_v);
        encode(x, top, old, codes);
        put(1, top, old, codes);
      }
      if (far) {
        __syncthreads();
#pragma unroll
        for (int j = h; j < kPageSize; j += kNumKvHeads) {
          const float4 f = first[lane];
          const float2 x = freqs.table32[j * kHalf + lane], x_lo = freqs.table_lo[j * kHalf + lane];
          turn[j * kTurnRow + lane] =
              make_float2(dot2(f.x, f.z, x.x, x_lo.x, -f.y, -f.w, x.y, x_lo.y),
                          dot2(f.y, f.w, x.x, x_lo.x, f.x, f.z, x.y, x_lo.y));
        }
      }
      if (!near) __syncthreads();  // (warps that gave up have left)
      load(rows);
      // Bounds x, y of the rotated keys, which give the same codes but for a key in a
      // few ten thousand.  (With barriers of the whole CTA, where this took 79 us,
      // deciding each of them exactly took 84; with FP64, whose rate here is a small
      // fraction of FP32's, 119; not at all 64.)
      uint4 y[2][2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        rotate8(smem_addr(turn) + ((r + 8 * s) * kTurnRow + 8 * q) * 8, x[s][0], x[s][1], y[s][0],
                y[s][1]);
        if (r + 8 * s < t.s0 || r + 8 * s >= t.s1)  // (zeros: their signs do not matter)
          y[s][0] = y[s][1] = x[s][0] = x[s][1] = make_uint4(0u, 0u, 0u, 0u);
      }
      auto again = [&](int s, uint32_t bad) {
        const int slot = r + 8 * s;
        rotate_again(bad, freqs.inv_freq + 8 * q, rows + slot * kTokenBytes,
                     smem_addr(turn) + (slot * kTurnRow + 8 * q) * 8,
                     near ? freqs.table_lo + static_cast<int64_t>(pos0 + slot) * kHalf + 8 * q
                          : nullptr,
                     pos0 + slot,
                     x[s][0], x[s][1]);
      };
      uint32_t top = top_of(x);
      const uint32_t old = stored_scale(old_k);
      // Pairs of less than 2^-70 matter only where the block's largest is tiny; where the
      // bounds of a pair overflow (|u| + |v| may, though the pair's length fits), or a key
      // is not finite, so is the largest.
      const bool odd = (top > 0 && top < kTiny) || top >= kHuge;
      encode(x, top, old, codes);
      uint32_t apart = 0;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int d = 0; d < 2; ++d)
          apart |= (x[s][d].x ^ y[s][d].x) | (x[s][d].y ^ y[s][d].y) | (x[s][d].z ^ y[s][d].z) |
                   (x[s][d].w ^ y[s][d].w);
      if (odd || __any_sync(kFull, apart != 0)) {
        bool differ = odd || needed_scale<kFmt>(top_of(y)) != needed_scale<kFmt>(top);
        if (!differ) {  // (the same in all lanes so far)
          uint2 z[2][2];
          encode(y, top, old, z);
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int d = 0; d < 2; ++d)
              differ |= ((codes[s][d].x ^ z[s][d].x) | (codes[s][d].y ^ z[s][d].y)) != 0u;
        }
        if (__any_sync(kFull, differ)) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const bool in = r + 8 * s >= t.s0 && r + 8 * s < t.s1;
            const uint32_t bad =
                !in ? 0u : odd ? 0xFFu : pairs_apart(x[s][0], x[s][1], y[s][0], y[s][1]);
            if (differ && bad != 0) again(s, bad);
          }
          __syncwarp();
          top = largest(x);
          encode(x, top, old, codes);
        }
      }
      put(0, top, old, codes);
      fence_proxy_async_smem();  // the stage's next copies come after what was written here
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(st));
      if (h == 0) ask();
    }
  }
  if (!ok && lane == 0) record_error(dev_err, kErrTimeout);
  // every copy asked for has landed before the CTA ends (full limit)
  if (tid == 0)
    for (int j = issued > kWriteStages ? issued - kWriteStages : 0; j < issued; ++j)
      mbar_wait_bounded(full(j % kWriteStages), (j / kWriteStages) & 1);
}

// Warp h of a CTA reads the K and the V block of kv head h of its units, the next
// one's codes on their way: lane 8 r + q holds dims [8 q, 8 q + 8) of slots r, r + 4, r +
// 8 and r + 12, so that a store fills whole lines.  (Lanes of 16 dims each, whose stores
// leave every other 16 bytes to the next, took 59 us for 32 x 4096
// tokens, int8; this takes 50: 6.0 TB/s of what it reads and writes.)
constexpr int kReadCtas = 4;
template <int kFmt>
__global__ void __launch_bounds__(kThreads, kReadCtas)
    kv8_read_kernel(uint16_t* __restrict__ k, uint16_t* __restrict__ v, int num_tokens,
                    const int32_t* __restrict__ off, const int32_t* __restrict__ starts,
                    const Kv8 c, int32_t* dev_err) {
  const int lane = threadIdx.x & 31, h = threadIdx.x >> 5;
  const int r = lane >> 3, q = lane & 7;
  wait_for_prior_grids();
  allow_dependent_grids();
  check_offsets(c, off, num_tokens, dev_err);
  const Share share(unit_count(num_tokens, c.batch));
  for (int64_t u0 = share.u0; u0 < share.u1; u0 += 32) {
    const Unit mine =
        find_unit(u0 + lane, share.u1, c, off, starts, num_tokens, dev_err, h == 0);
    unsigned todo = __ballot_sync(kFull, mine.pool_page >= 0);
    uint2 w[2][4];  // [K|V][slot r + 4 i]
    uint32_t e[2];
    auto load = [&](int src) {
      const int64_t page = __shfl_sync(kFull, mine.pool_page, src);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint2* at = reinterpret_cast<const uint2*>(c.pool + block_at(page, kv, h)) + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[kv][i] = __ldcs(at + 32 * i);
        e[kv] = c.scales[scale_at(page, kv, h)];
      }
    };
    if (todo != 0) load(__ffs(todo) - 1);
    while (todo != 0) {
      const Unit t = unit_of(mine, __ffs(todo) - 1);
      todo &= todo - 1;
      uint2 x[2][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i >> 2][i & 3] = w[i >> 2][i & 3];
      const float f[2] = {scale_value(stored_scale(e[0])), scale_value(stored_scale(e[1]))};
      if (todo != 0) load(__ffs(todo) - 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int slot = r + 4 * i;
        if (slot < t.s0 || slot >= t.s1) continue;
        const int64_t at = (t.row0 + slot) * (kNumKvHeads * kHeadDim) + h * kHeadDim + 8 * q;
        *reinterpret_cast<uint4*>(k + at) = widen8<kFmt>(x[0][i], f[0]);
        *reinterpret_cast<uint4*>(v + at) = widen8<kFmt>(x[1][i], f[1]);
      }
    }
  }
}

int unit_grid(int num_tokens, int batch, int num_sms, int per_sm) {
  return static_cast<int>(std::min<int64_t>(unit_count(num_tokens, batch),
                                            static_cast<int64_t>(num_sms) * per_sm));
}

template <int kFmt>
cudaError_t launch_write(const uint16_t* k, const uint16_t* v, int num_tokens,
                         const int32_t* token_offsets, const int32_t* start_positions,
                         const Kv8& cache, const RopeFreqs& freqs, int num_sms, int32_t* dev_err,
                         cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  const unsigned long long bit = 1ull << (device & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    err = cudaFuncSetAttribute(kv8_write_kernel<kFmt>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(kWriteSmem));
    if (err != cudaSuccess) return err;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  return launch_pdl(kv8_write_kernel<kFmt>,
                    dim3(unit_grid(num_tokens, cache.batch, num_sms, kWriteCtas)), dim3(kThreads),
                    kWriteSmem, stream, k, v, num_tokens, token_offsets, start_positions, cache,
                    freqs, dev_err, wait_limit_ns());
}

}  // namespace

cudaError_t launch_kv8_append(const uint16_t* k_new, const uint16_t* v_new, const Kv8& cache,
                              const int32_t* positions, const int32_t* slots,
                              const RopeFreqs& freqs, const uint16_t* q_in, uint16_t* q_out,
                              int32_t* dev_err, cudaStream_t stream) {
  return launch_pdl(cache.format == kKv8E4m3 ? kv8_append_kernel<kKv8E4m3>
                                             : kv8_append_kernel<kKv8Int8>,
                    dim3(cache.batch), dim3(kThreads), 0, stream, k_new, v_new, cache, positions,
                    slots, freqs, q_in, q_out, dev_err);
}

cudaError_t launch_kv8_write(const uint16_t* k, const uint16_t* v, int num_tokens,
                             const int32_t* token_offsets, const int32_t* start_positions,
                             const Kv8& cache, const RopeFreqs& freqs, int num_sms,
                             int32_t* dev_err, cudaStream_t stream) {
  return cache.format == kKv8E4m3
             ? launch_write<kKv8E4m3>(k, v, num_tokens, token_offsets, start_positions, cache,
                                      freqs, num_sms, dev_err, stream)
             : launch_write<kKv8Int8>(k, v, num_tokens, token_offsets, start_positions, cache,
                                      freqs, num_sms, dev_err, stream);
}

cudaError_t launch_kv8_read(uint16_t* k, uint16_t* v, int num_tokens,
                            const int32_t* token_offsets, const int32_t* start_positions,
                            const Kv8& cache, int num_sms, int32_t* dev_err, cudaStream_t stream) {
  return launch_pdl(
      cache.format == kKv8E4m3 ? kv8_read_kernel<kKv8E4m3> : kv8_read_kernel<kKv8Int8>,
      dim3(unit_grid(num_tokens, cache.batch, num_sms, kReadCtas)), dim3(kThreads), 0, stream, k,
      v, num_tokens, token_offsets, start_positions, cache, dev_err);
}

}  // namespace pkv
