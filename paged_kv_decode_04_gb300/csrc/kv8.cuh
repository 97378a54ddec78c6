// kv8.cuh -- the 8-bit cache: codes, scales and where a block stands.
//
// Pool [pages][K|V][8 kv heads][16 tokens][64] of 8-bit codes: a block, the 16
// tokens of one page, K or V and one kv head, is 1 KiB in a row, which its scale
// (uint8 [pages][K|V][8]) serves, and a page is one TMA box of 16 KiB.  A value
// is code * 2^(scale - 127), the code an e4m3 float or a signed integer.
// Powers of two make the products with the scales exact: a bf16 value has 8
// significant bits and a code at most 7, so dividing by a scale loses nothing
// before the one rounding to a code, every cached value is a bf16 number, and a
// block that needs a larger scale has its codes rounded again without another
// error than that rounding.  e4m3 loses no precision to it (a float's relative
// precision does not depend on the scale), an integer up to one bit of 7.  Scales
// begin at 2^-124, where the smallest e4m3 code is still a bf16 number.
#pragma once

#include <stdint.h>

#include "pkv_device.cuh"

namespace pkv {

constexpr int kBlockBytes = kPageSize * kHeadDim;            // 1 KiB
constexpr int kPage8Bytes = 2 * kNumKvHeads * kBlockBytes;   // 16 KiB
constexpr int kPageScales = 2 * kNumKvHeads;
constexpr int kScaleBias = 127, kLeastScale = 3, kMostScale = 240;

// Bytes from the pool's start to a block, and its scale's place.
__device__ __forceinline__ int64_t block_at(int64_t page, int kv, int g) {
  return page * kPage8Bytes + (kv * kNumKvHeads + g) * kBlockBytes;
}
__device__ __forceinline__ int64_t scale_at(int64_t page, int kv, int g) {
  return page * kPageScales + kv * kNumKvHeads + g;
}

// 2^(scale - 127) and its inverse, for scales in [3, 240].
__device__ __forceinline__ float scale_value(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ float scale_inverse(uint32_t e) {
  return __uint_as_float((254u - e) << 23);
}

// Any byte as a scale that the writers store (others count as the nearest).
__device__ __forceinline__ uint32_t stored_scale(uint32_t e) {
  return min(max(e, static_cast<uint32_t>(kLeastScale)), static_cast<uint32_t>(kMostScale));
}

// Scale of the smallest power of two that takes the bf16 magnitude `bits` to at
// most the largest code: 448 = 1.75 x 2^8, 127 = 1.984375 x 2^6.
template <int kFmt>
__device__ __forceinline__ uint32_t needed_scale(uint32_t bits) {
  const int e = static_cast<int>(bits >> 7), m = static_cast<int>(bits & 0x7Fu);
  const int s = kFmt == kKv8E4m3 ? e - 8 + (m > 96 ? 1 : 0) : e - 6 + (m > 126 ? 1 : 0);
  return static_cast<uint32_t>(min(max(s, kLeastScale), kMostScale));
}

// Four values times f (the scale's inverse; exact products) as codes, the first in
// the low byte.  Past the largest code (scales end at 240) e4m3 codes saturate;
// integers do where kClamp.
template <int kFmt, bool kClamp>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float f) {
  if constexpr (kFmt == kKv8E4m3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * f), "f"(a * f));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * f), "f"(c * f));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  } else {
    // 1.5 x 2^23 + y holds y, rounded once to nearest even, in its low bits
    auto code = [f](float y) {
      return __float_as_uint(kClamp ? fminf(fmaxf(y * f, -127.f), 127.f) + 12582912.f
                                    : fmaf(y, f, 12582912.f));
    };
    return prmt(prmt(code(a), code(b), 0x0040u), prmt(code(c), code(d), 0x0040u), 0x5410u);
  }
}

// Two floats as f16 (round to nearest even), `lo` in the low half.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Two e4m3 codes as two f16 values (exact; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
  return r;
}

// The four codes of a word as f16 pairs: (0, 1) and (2, 3).
template <int kFmt>
__device__ __forceinline__ void decode_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kFmt == kKv8E4m3) {
    lo = e4m3x2_to_f16x2(static_cast<uint16_t>(w & 0xFFFFu));
    hi = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
  } else {
    // the f16 0x6400 + u is 1024 + u; u = code + 128
    const uint32_t u = w ^ 0x80808080u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(prmt(u, 0x64646464u, 0x4140u)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(prmt(u, 0x64646464u, 0x4342u)), "r"(0x64806480u));
  }
}

// The four codes of a word as floats.
template <int kFmt>
__device__ __forceinline__ float4 decode4(uint32_t w) {
  if constexpr (kFmt == kKv8E4m3) {
    uint32_t lo, hi;
    decode_f16<kFmt>(w, lo, hi);
    float4 f;
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, "
        "y;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(lo));
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, "
        "y;\n\t}" : "=f"(f.z), "=f"(f.w) : "r"(hi));
    return f;
  } else {
    // 2^23 + u, u = code + 128
    const uint32_t u = w ^ 0x80808080u;
    auto value = [u](uint32_t sel) {
      return __uint_as_float(prmt(u, 0x4B000000u, sel)) - 8388736.f;
    };
    return make_float4(value(0x7540u), value(0x7541u), value(0x7542u), value(0x7543u));
  }
}

// 8 codes times a scale's value as bf16 (exact).
template <int kFmt>
__device__ __forceinline__ uint4 widen8(const uint2& codes, float scale) {
  const float4 a = decode4<kFmt>(codes.x), b = decode4<kFmt>(codes.y);
  return make_uint4(pack_bf16x2(a.x * scale, a.y * scale), pack_bf16x2(a.z * scale, a.w * scale),
                    pack_bf16x2(b.x * scale, b.y * scale), pack_bf16x2(b.z * scale, b.w * scale));
}

// A warp rounds the first `rows` tokens of a block again, under a scale larger
// by `up`.
template <int kFmt>
__device__ __forceinline__ void rescale_rows(uint8_t* block, int rows, uint32_t up, int lane) {
  const float f = up > 126u ? 0.f : __uint_as_float((127u - up) << 23);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if ((lane >> 2) + 8 * h >= rows) continue;
    uint4* at = reinterpret_cast<uint4*>(block) + lane + 32 * h;
    uint4 w = *at;
    uint32_t* x = &w.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = decode4<kFmt>(x[i]);
      x[i] = encode4<kFmt, false>(v.x, v.y, v.z, v.w, f);
    }
    *at = w;
  }
}

}  // namespace pkv
