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

#include "kv8.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kHalf = kHeadDim / 2;
constexpr int kThreads = 32 * kNumKvHeads;  // a warp to a kv head
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ bool finite_bf16(uint32_t h) { return (h & 0x7F80u) != 0x7F80u; }

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
// 2i + 1 of V.
template <int kFmt>
__global__ void __launch_bounds__(kThreads)
    kv8_append_kernel(const uint16_t* __restrict__ k_new, const uint16_t* __restrict__ v_new,
                      const Kv8 c, const int32_t* __restrict__ positions,
                      const int32_t* __restrict__ slots, RopeFreqs freqs,
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
  // threads (as in kv_append_kernel).
  __shared__ double2 s_cs[kHalf];
  RopeCS cs;
  if (freqs.table_theta == nullptr || pos < 0 || pos >= kRopeTablePositions) {
    if (h == 0) {
      const RopeCS f = rope_cs(freqs, false, pos, i);
      s_cs[i] = make_double2(f.c64, f.s64);
    }
    __syncthreads();
    cs.c64 = s_cs[i].x;
    cs.s64 = s_cs[i].y;
    cs.c32 = static_cast<float>(cs.c64);
    cs.s32 = static_cast<float>(cs.s64);
    cs.have64 = true;
  } else {
    cs = rope_cs(freqs, table_ok, pos, i);
  }

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
      rotate_pair_rope(freqs, table_ok, pos, i, cs, x1[k], x2[k], &y1, &y2);
      q_out[o] = y1;
      q_out[o + kHalf] = y2;
    }
  }
  if (!page_ok) {
    if (tid == 0) record_error(dev_err, pos_ok ? kErrPage : kErrPosition);
    return;
  }

  uint16_t y1, y2;
  rotate_pair_rope(freqs, table_ok, pos, i, cs, k1, k2, &y1, &y2);
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
  const uint32_t w = encode4<kFmt>(bf16_to_float(y1) * fk, bf16_to_float(y2) * fk,
                                   __uint_as_float(v1 << 16) * fv, __uint_as_float(v2 << 16) * fv);
  uint8_t* kd = c.pool + block_at(page, 0, h) + slot * kHeadDim;
  uint8_t* vd = c.pool + block_at(page, 1, h) + slot * kHeadDim;
  kd[i] = static_cast<uint8_t>(w);
  kd[i + kHalf] = static_cast<uint8_t>(w >> 8);
  reinterpret_cast<uint16_t*>(vd)[i] = static_cast<uint16_t>(w >> 16);
}

// A unit is one page of one sequence.  Units are numbered so that a sequence's
// first is off[b] / 16 + 2 b: n tokens touch at most n / 16 + 2 pages, so the
// ranges of numbers do not meet (some numbers name no page), and the sequence of
// a unit is found by search, without a prefix sum.
struct Unit {
  int b, page;          // sequence, page of it; b < 0: none
  int64_t row0;         // row of k and v of the token in slot 0 of the page
  int s0, s1;           // slots [s0, s1) are the call's
  int64_t pool_page;
};

__host__ __device__ inline int64_t unit_count(int num_tokens, int batch) {
  return num_tokens / kPageSize + 2 * static_cast<int64_t>(batch);
}

// Found by a whole warp (the same in every lane); `report`: one warp of the unit
// reports what is wrong with it.
__device__ __forceinline__ Unit find_unit(int64_t u, const Kv8& c,
                                          const int32_t* __restrict__ off,
                                          const int32_t* __restrict__ starts, int num_tokens,
                                          int32_t* dev_err, bool report, int lane) {
  auto first = [&](int b) { return static_cast<int64_t>(off[b] / kPageSize) + 2ll * b; };
  int lo = 0, n = c.batch;
  while (n > 1) {  // 32 places at a time
    const int step = (n + 31) / 32, at = lane * step;
    const unsigned below = __ballot_sync(kFull, at < n && first(lo + min(at, n - 1)) <= u);
    const int cut = max(__popc(below) - 1, 0) * step;
    lo += cut;
    n = min(step, n - cut);
  }
  Unit r;
  r.b = -1;
  r.page = 0;
  r.row0 = 0;
  r.s0 = r.s1 = 0;
  r.pool_page = -1;
  const int o0 = off[lo], o1 = off[lo + 1];
  if (o0 < 0 || o1 < o0 || o1 > num_tokens) {
    if (report && lane == 0) record_error(dev_err, kErrOffsets);
    return r;
  }
  const int64_t start = starts[lo], end = start + (o1 - o0);
  const int64_t limit = static_cast<int64_t>(c.max_blocks) * kPageSize;
  const int64_t p0 = start > 0 ? start : 0, p1 = end < limit ? end : limit;
  if (o1 > o0 && (p0 != start || p1 != end) && report && lane == 0)
    record_error(dev_err, kErrPosition);
  const int64_t page = p0 / kPageSize + (u - first(lo));
  if (u < first(lo) || p1 <= p0 || page * kPageSize >= p1) return r;
  r.page = static_cast<int>(page);
  r.s0 = max(static_cast<int>(p0 - page * kPageSize), 0);
  r.s1 = p1 - page * kPageSize < kPageSize ? static_cast<int>(p1 - page * kPageSize) : kPageSize;
  r.row0 = o0 + page * kPageSize - start;
  r.pool_page = c.block_table[static_cast<int64_t>(lo) * c.max_blocks + page];
  if (r.pool_page < 0 || r.pool_page >= c.num_pages) {
    if (report && lane == 0) record_error(dev_err, kErrPage);
    return r;
  }
  r.b = lo;
  return r;
}

// Offsets that do not begin at 0 and end at the number of tokens.
__device__ __forceinline__ void check_ends(const Kv8& c, const int32_t* off, int num_tokens,
                                           int32_t* dev_err) {
  if (blockIdx.x == 0 && threadIdx.x == 0 && (off[0] != 0 || off[c.batch] != num_tokens))
    record_error(dev_err, kErrOffsets);
}

// RoPE of the 8 pairs (x1, x2) = dims (8 q + p, 32 + 8 q + p) of a row, in place:
// FP32 with both ends of its error bound rounded to bf16, the pairs where these
// differ (or that are outside FP32's comfort) again in FP64 (rotate_pair).
__device__ __forceinline__ void rotate8(const RopeFreqs& f, bool table_ok, int pos, int q,
                                        uint4& x1, uint4& x2) {
  uint32_t* a = &x1.x;
  uint32_t* b = &x2.x;
  const int i0 = 8 * q;
  float c[8], sn[8];
  if (table_ok) {
    const float4* t = reinterpret_cast<const float4*>(f.table32 + pos * kHalf + i0);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 cs = t[e];
      c[2 * e] = cs.x;
      sn[2 * e] = cs.y;
      c[2 * e + 1] = cs.z;
      sn[2 * e + 1] = cs.w;
    }
  } else {
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      double s64, c64;
      sincos(__dmul_rn(static_cast<double>(pos), f.inv_freq[i0 + e]), &s64, &c64);
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (p == e) {
          c[p] = static_cast<float>(c64);
          sn[p] = static_cast<float>(s64);
        }
    }
  }
  uint32_t bad = 0, o1[4], o2[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float y1[2], y2[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = 2 * e + h;
      const float u = __uint_as_float(h ? (a[e] & 0xFFFF0000u) : (a[e] << 16));
      const float v = __uint_as_float(h ? (b[e] & 0xFFFF0000u) : (b[e] << 16));
      y1[h] = fmaf(u, c[p], -(v * sn[p]));
      y2[h] = fmaf(v, c[p], u * sn[p]);
      const float s0 = fabsf(u) + fabsf(v);
      const float m1 = s0 + fabsf(y1[h]), m2 = s0 + fabsf(y2[h]);
      const uint32_t lo = cvt_bf16x2_rn(fmaf(m1, -0x1p-22f, y1[h]), fmaf(m2, -0x1p-22f, y2[h]));
      const uint32_t hi = cvt_bf16x2_rn(fmaf(m1, 0x1p-22f, y1[h]), fmaf(m2, 0x1p-22f, y2[h]));
      // 2^-100 <= s0 <= 2^100
      const bool in_range = __float_as_uint(s0) - 0x0D800000u <= 0x71800000u - 0x0D800000u;
      if (lo != hi || !in_range) bad |= 1u << p;
    }
    o1[e] = cvt_bf16x2_rn(y1[0], y1[1]);
    o2[e] = cvt_bf16x2_rn(y2[0], y2[1]);
  }
  while (bad != 0) {
    const int p = __ffs(bad) - 1;
    bad &= bad - 1;
    uint32_t wa = 0, wb = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e == p >> 1) {
        wa = a[e];
        wb = b[e];
      }
    const int sh = 16 * (p & 1);
    double c64, s64;
    if (table_ok) {
      const double2 t = f.table64[pos * kHalf + i0 + p];
      c64 = t.x;
      s64 = t.y;
    } else {
      sincos(__dmul_rn(static_cast<double>(pos), f.inv_freq[i0 + p]), &s64, &c64);
    }
    uint16_t y1, y2;
    rotate_pair(static_cast<uint16_t>(wa >> sh), static_cast<uint16_t>(wb >> sh), c64, s64, &y1,
                &y2);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e == p >> 1) {
        o1[e] = (o1[e] & ~(0xFFFFu << sh)) | (static_cast<uint32_t>(y1) << sh);
        o2[e] = (o2[e] & ~(0xFFFFu << sh)) | (static_cast<uint32_t>(y2) << sh);
      }
  }
  x1 = make_uint4(o1[0], o1[1], o1[2], o1[3]);
  x2 = make_uint4(o2[0], o2[1], o2[2], o2[3]);
}

// Zero the values of 8 that are not finite; true when there were some.
__device__ __forceinline__ bool drop_nonfinite(uint4& x) {
  const uint32_t m0 = nonfinite_halves(x.x), m1 = nonfinite_halves(x.y),
                 m2 = nonfinite_halves(x.z), m3 = nonfinite_halves(x.w);
  x = make_uint4(x.x & ~m0, x.y & ~m1, x.z & ~m2, x.w & ~m3);
  return (m0 | m1 | m2 | m3) != 0u;
}

// The larger magnitude of each half, over the words.
__device__ __forceinline__ uint32_t top_halves(uint32_t top, const uint4& x) {
  top = __vmaxu2(top, __vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu));
  return __vmaxu2(top, __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
}

template <int kFmt>
__device__ __forceinline__ uint2 encode8(const uint4& x, float f) {
  const float2 a = bf16x2_to_float2(x.x), b = bf16x2_to_float2(x.y), c = bf16x2_to_float2(x.z),
               d = bf16x2_to_float2(x.w);
  return make_uint2(encode4<kFmt>(a.x * f, a.y * f, b.x * f, b.y * f),
                    encode4<kFmt>(c.x * f, c.y * f, d.x * f, d.y * f));
}

// Warp h of a CTA takes the K and the V block of kv head h of a unit: lane 4 r +
// q holds dims [8 q, 8 q + 8) and [32 + 8 q, 32 + 8 q + 8) of slots r and r + 8.
template <int kFmt>
__global__ void __launch_bounds__(kThreads)
    kv8_write_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                     int num_tokens, const int32_t* __restrict__ off,
                     const int32_t* __restrict__ starts, const Kv8 c, RopeFreqs freqs,
                     int32_t* dev_err) {
  const int lane = threadIdx.x & 31, h = threadIdx.x >> 5;
  const int r = lane >> 2, q = lane & 3;
  wait_for_prior_grids();
  allow_dependent_grids();
  check_ends(c, off, num_tokens, dev_err);
  const bool tag_ok = rope_table_ready(freqs);
  const int64_t units = unit_count(num_tokens, c.batch);
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit t = find_unit(u, c, off, starts, num_tokens, dev_err, h == 0, lane);
    if (t.b < 0) continue;
    uint4 x[2][2][2];  // [K|V][slot r, r + 8][dims 8 q, 32 + 8 q]
    bool in[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int slot = r + 8 * s;
      in[s] = slot >= t.s0 && slot < t.s1;
      const int64_t at = (t.row0 + slot) * (kNumKvHeads * kHeadDim) + h * kHeadDim + 8 * q;
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        x[0][s][d] = x[1][s][d] = make_uint4(0u, 0u, 0u, 0u);
        if (in[s]) {
          x[0][s][d] = __ldcs(reinterpret_cast<const uint4*>(k + at + kHalf * d));
          x[1][s][d] = __ldcs(reinterpret_cast<const uint4*>(v + at + kHalf * d));
        }
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int pos = t.page * kPageSize + r + 8 * s;
      if (in[s]) rotate8(freqs, tag_ok && pos < kRopeTablePositions, pos, q, x[0][s][0], x[0][s][1]);
    }
    bool dropped = false;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint32_t top = 0;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          dropped |= drop_nonfinite(x[kv][s][d]);
          top = top_halves(top, x[kv][s][d]);
        }
      top = __reduce_max_sync(kFull, max(top & 0xFFFFu, top >> 16));
      const uint32_t old =
          t.s0 > 0 ? stored_scale(c.scales[scale_at(t.pool_page, kv, h)]) : 0u;
      const uint32_t e = settle_scale<kFmt>(c, t.pool_page, kv, h, top, t.s0, old, lane);
      const float f = scale_inverse(e);
      uint8_t* block = c.pool + block_at(t.pool_page, kv, h);
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (in[s])
#pragma unroll
          for (int d = 0; d < 2; ++d)
            *reinterpret_cast<uint2*>(block + (r + 8 * s) * kHeadDim + kHalf * d + 8 * q) =
                encode8<kFmt>(x[kv][s][d], f);
    }
    if (dropped) record_error(dev_err, kErrValue);
  }
}

// Warp h of a CTA reads the K and the V block of kv head h of a unit: lane 4 r +
// q holds dims [16 q, 16 q + 16) of slots r and r + 8.
template <int kFmt>
__global__ void __launch_bounds__(kThreads)
    kv8_read_kernel(uint16_t* __restrict__ k, uint16_t* __restrict__ v, int num_tokens,
                    const int32_t* __restrict__ off, const int32_t* __restrict__ starts,
                    const Kv8 c, int32_t* dev_err) {
  const int lane = threadIdx.x & 31, h = threadIdx.x >> 5;
  const int r = lane >> 2, q = lane & 3;
  wait_for_prior_grids();
  allow_dependent_grids();
  check_ends(c, off, num_tokens, dev_err);
  const int64_t units = unit_count(num_tokens, c.batch);
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit t = find_unit(u, c, off, starts, num_tokens, dev_err, h == 0, lane);
    if (t.b < 0) continue;
    uint4 w[2][2];
    bool in[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      in[s] = r + 8 * s >= t.s0 && r + 8 * s < t.s1;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)
        if (in[s])
          w[kv][s] = __ldcs(reinterpret_cast<const uint4*>(c.pool + block_at(t.pool_page, kv, h)) +
                            lane + 32 * s);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const float f = scale_value(stored_scale(c.scales[scale_at(t.pool_page, kv, h)]));
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (!in[s]) continue;
        widen16<kFmt>(w[kv][s], f,
                      reinterpret_cast<uint4*>((kv == 0 ? k : v) +
                                               (t.row0 + r + 8 * s) * (kNumKvHeads * kHeadDim) +
                                               h * kHeadDim + 16 * q));
      }
    }
  }
}

int unit_grid(int num_tokens, int batch, int num_sms, int per_sm) {
  return static_cast<int>(std::min<int64_t>(unit_count(num_tokens, batch),
                                            static_cast<int64_t>(num_sms) * per_sm));
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
  return launch_pdl(
      cache.format == kKv8E4m3 ? kv8_write_kernel<kKv8E4m3> : kv8_write_kernel<kKv8Int8>,
      dim3(unit_grid(num_tokens, cache.batch, num_sms, 8)), dim3(kThreads), 0, stream, k, v,
      num_tokens, token_offsets, start_positions, cache, freqs, dev_err);
}

cudaError_t launch_kv8_read(uint16_t* k, uint16_t* v, int num_tokens,
                            const int32_t* token_offsets, const int32_t* start_positions,
                            const Kv8& cache, int num_sms, int32_t* dev_err, cudaStream_t stream) {
  return launch_pdl(
      cache.format == kKv8E4m3 ? kv8_read_kernel<kKv8E4m3> : kv8_read_kernel<kKv8Int8>,
      dim3(unit_grid(num_tokens, cache.batch, num_sms, 8)), dim3(kThreads), 0, stream, k, v,
      num_tokens, token_offsets, start_positions, cache, dev_err);
}

}  // namespace pkv
