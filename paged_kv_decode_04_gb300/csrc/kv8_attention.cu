// kv8_attention.cu -- attention of one new token, or of chunks of a few, per
// sequence over the 8-bit paged cache, streaming its pages once.
//
// One CTA per (sequence, range of the pages that its queries see): a producer
// warp brings whole pages (16 KiB, all kv heads, one TMA box, and the 16 bytes of
// their scales) into a ring in shared memory, and warp g of eight takes kv head
// g's blocks of every page.  So a page is one copy and one barrier for all heads,
// and the heads' states never meet.
//
// mma.sync m16n8k16 in f16, FP32 accumulators, for a page (16 tokens) and a kv
// head; codes become f16 exactly (one instruction for two e4m3 codes):
//   S^T = K Q^T    tokens as M, query rows as N.  A lane reads 16 codes in a row
//                  of K for its four k-steps; which dims share a k-step does not
//                  matter, as Q's fragments take the same ones.  Q enters as f16
//                  times the power of two that takes its row's largest magnitude
//                  to [2^14, 2^15): exact for values down to 2^-31 of it (bf16
//                  has 8 significant bits, f16 24 bits below that magnitude).
//   O^T += V^T P^T dims as M.  V^T comes through ldmatrix on 8-bit elements,
//                  transposed, four tokens to a lane's word; K's rows are read
//                  in the order that gives P those tokens.
// The scales of a block stay out of the products: K's goes into the factor of
// the scores, V's multiplies the page's own product, added to the accumulators in
// FP32; so weights and codes of f16 keep their range whatever the scales are.
// Weights are 2^(s - m + 7), m the running reference of decode_page.cuh (which
// moves when a score passes it by 8, so they stay below 2^15), and enter the
// product as two f16 terms (22 significant bits, 2^-32 of the reference's weight
// at the least); for one token the terms are the columns 0-3 and 4-7 of one MMA.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "kv8.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "visible.cuh"

namespace pkv {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kWarps = kNumKvHeads;            // and one that loads
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStages = 6, kCtas = 2;
constexpr int kOffScales = kStages * kPage8Bytes;
constexpr int kOffMeta = kOffScales + kStages * kPageScales;
constexpr int kOffBars = kOffMeta + kStages * 8;
constexpr size_t kSmem = 1024 + kOffBars + 2 * 8 * kStages;
static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "the CTAs of an SM fit");

constexpr float kMoveLog2 = 8.f;   // a score this far above the reference moves it
constexpr float kLift = 7.f;       // weights are 2^(s - m + kLift) <= 2^15
constexpr float kLowestFloat = -3.402823466e38f;

// D = A B (+ D), FP32 accumulators.  (Not volatile: the compiler may interleave the
// chains of two pages.)
__device__ __forceinline__ void mma_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Two 16 x 16 matrices of bytes, transposed: lane l gives the address of row
// l & 15 of matrix l >> 4 and gets, of each, columns l / 4 and l / 4 + 8 of rows
// 4 (l & 3) .. + 3.
__device__ __forceinline__ void ldsm_b8_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t w) {
  float2 f;
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, "
      "y;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(w));
  return f;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// A lane's places in the fragments.
struct Lane {
  int fg, ft;          // fragment row and column group
  int tok;             // token of row fg of S^T; row fg + 8 is token tok + 2
  uint32_t k0, k1;     // this lane's 16 codes of both rows of a K block
  uint32_t v0, v1;     // this lane's rows of V's matrices of dims 0-31 and 32-63
  __device__ __forceinline__ explicit Lane(int lane) {
    fg = lane >> 2;
    ft = lane & 3;
    tok = 4 * (fg >> 1) + (fg & 1);
    // 16-byte chunk c of row r lies at chunk c ^ (r / 2 mod 4) (TMA's 64-byte
    // swizzle)
    auto at = [](int r, int c) {
      return static_cast<uint32_t>(r * kHeadDim + ((c ^ ((r >> 1) & 3)) << 4));
    };
    k0 = at(tok, ft);
    k1 = at(tok + 2, ft);
    v0 = at(lane & 15, lane >> 4);
    v1 = at(lane & 15, 2 + (lane >> 4));
  }
};

// Online softmax of 8 query rows (columns of S^T) of a warp.
struct State {
  float m[2], l[2];    // of columns 2 ft, 2 ft + 1: reference, this lane's share of the sum
  float2 o[4][2];      // O^T: dims 16 mt + fg (+ 8), columns 2 ft, 2 ft + 1
  __device__ __forceinline__ void reset() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) o[mt][0] = o[mt][1] = make_float2(0.f, 0.f);
  }
};

// Q^T as B fragments of a row of q: column fg's dims 16 ft + 4 kk + {0, 1} and
// {2, 3}.  Returns the power of two that undoes the row's own (the same in the
// row's four lanes).
__device__ __forceinline__ float load_q(const uint16_t* row, int ft, uint32_t (&qb)[4][2]) {
  uint32_t w[8];
  if (row != nullptr) {
    const uint4 a = reinterpret_cast<const uint4*>(row)[2 * ft];
    const uint4 b = reinterpret_cast<const uint4*>(row)[2 * ft + 1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0u;
  }
  uint32_t top = 0;  // largest finite magnitude
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu & ~nonfinite_halves(w[i]));
  top = max(top & 0xFFFFu, top >> 16);
  top = max(top, __shfl_xor_sync(kFull, top, 1));
  top = max(top, __shfl_xor_sync(kFull, top, 2));
  // 2^(14 - exponent), within normal numbers
  const int up = top == 0 ? 0 : min(max(14 + 127 - static_cast<int>(top >> 7), -126), 126);
  const float f = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = bf16x2_to_float2(w[i]);
    qb[i >> 1][i & 1] = pack_f16x2(x.x * f, x.y * f);
  }
  return __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
}

// A K block's rows as A fragments of the four k-steps.
template <int kFmt>
__device__ __forceinline__ void load_k(uint32_t kt, const Lane& P, uint32_t (&ka)[4][4]) {
  const uint4 x = lds128(kt + P.k0), y = lds128(kt + P.k1);
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    decode_f16<kFmt>(a[kk], ka[kk][0], ka[kk][2]);
    decode_f16<kFmt>(b[kk], ka[kk][1], ka[kk][3]);
  }
}

template <int kFmt>
__device__ __forceinline__ void load_v(uint32_t vt, const Lane& P, uint32_t (&va)[4][4]) {
  uint32_t r[8];
  ldsm_b8_trans(vt + P.v0, *reinterpret_cast<uint32_t(*)[4]>(&r[0]));
  ldsm_b8_trans(vt + P.v1, *reinterpret_cast<uint32_t(*)[4]>(&r[4]));
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    decode_f16<kFmt>(r[2 * mt], va[mt][0], va[mt][2]);
    decode_f16<kFmt>(r[2 * mt + 1], va[mt][1], va[mt][3]);
  }
}

// Move the references of S's rows to what the masked scores x of two pages ask for;
// f: the factors of the pages' scores, of columns 2 ft and 2 ft + 1.
__device__ __forceinline__ void move_reference(const float (&x)[2][4], const float (&f)[2][2],
                                               State& S) {
  float mx0 = fmaxf(fmaxf(x[0][0], x[0][2]) * f[0][0], fmaxf(x[1][0], x[1][2]) * f[1][0]);
  float mx1 = fmaxf(fmaxf(x[0][1], x[0][3]) * f[0][1], fmaxf(x[1][1], x[1][3]) * f[1][1]);
  if (!__any_sync(kFull, mx0 > S.m[0] + kMoveLog2 || mx1 > S.m[1] + kMoveLog2)) return;
#pragma unroll
  for (int i = 4; i <= 16; i <<= 1) {
    mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, i));
    mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, i));
  }
  const float m0 = fmaxf(S.m[0], mx0), m1 = fmaxf(S.m[1], mx1);
  // (0 until the row has seen a score above -inf)
  const float2 alpha = make_float2(fast_exp2(S.m[0] - fmaxf(m0, kLowestFloat)),
                                   fast_exp2(S.m[1] - fmaxf(m1, kLowestFloat)));
  S.l[0] *= alpha.x;
  S.l[1] *= alpha.y;
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    S.o[mt][0] = fmul2(S.o[mt][0], alpha);
    S.o[mt][1] = fmul2(S.o[mt][1], alpha);
  }
  S.m[0] = m0;
  S.m[1] = m1;
}

// A page's weights as the B fragment of the second product: columns 0-3 the first
// terms of the four rows, columns 4-7 (lanes ft >= 2, which hold the same scores)
// their second ones.
__device__ __forceinline__ void page_weights(const float (&x)[4], const float (&f)[2], int ft,
                                             State& S, uint32_t& b0, uint32_t& b1) {
  const float d0 = kLift - fmaxf(S.m[0], kLowestFloat), d1 = kLift - fmaxf(S.m[1], kLowestFloat);
  const float p0 = fast_exp2(fmaf(x[0], f[0], d0)), p1 = fast_exp2(fmaf(x[1], f[1], d1));
  const float p2 = fast_exp2(fmaf(x[2], f[0], d0)), p3 = fast_exp2(fmaf(x[3], f[1], d1));
  S.l[0] += p0 + p2;
  S.l[1] += p1 + p3;
  const uint32_t h0 = pack_f16x2(p0, p1), h1 = pack_f16x2(p2, p3);
  const float2 f0 = f16x2_to_float2(h0), f1 = f16x2_to_float2(h1);
  const uint32_t l0 = pack_f16x2(p0 - f0.x, p1 - f0.y), l1 = pack_f16x2(p2 - f1.x, p3 - f1.y);
  b0 = transpose8x8(ft < 2 ? h0 : l0);
  b1 = transpose8x8(ft < 2 ? h1 : l1);
}

// O += sv * V^T P^T of a page.
template <int kFmt>
__device__ __forceinline__ void add_values(uint32_t vt, const Lane& P, float sv, uint32_t b0,
                                           uint32_t b1, State& S) {
  uint32_t va[4][4];
  load_v<kFmt>(vt, P, va);
  const float2 s2 = make_float2(sv, sv);
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    float t[4];
    mma_new(t, va[mt], b0, b1);
    S.o[mt][0] = ffma2(make_float2(t[0], t[1]), s2, S.o[mt][0]);
    S.o[mt][1] = ffma2(make_float2(t[2], t[3]), s2, S.o[mt][1]);
  }
}

// Zero the V rows of a block whose tokens are not in `vis`: their codes may be
// NaN, and 0 x NaN is not 0.
__device__ __forceinline__ void hide_v(uint32_t vt, uint32_t vis, int lane) {
#pragma unroll
  for (int i = lane; i < kPageSize * 4; i += 32)
    if (!((vis >> (i >> 2)) & 1u)) sts128_zero(vt + i * 16);
  fence_proxy_async_smem();  // the ring's next copy comes after these writes
  __syncwarp();
}

// The ring of a CTA.
struct Ring {
  uint32_t base;
  __device__ __forceinline__ uint32_t page(int st) const { return base + st * kPage8Bytes; }
  __device__ __forceinline__ uint32_t scales(int st) const {
    return base + kOffScales + st * kPageScales;
  }
  __device__ __forceinline__ uint32_t meta(int st) const { return base + kOffMeta + st * 8; }
  __device__ __forceinline__ uint32_t full(int st) const { return base + kOffBars + st * 8; }
  __device__ __forceinline__ uint32_t empty(int st) const {
    return base + kOffBars + (kStages + st) * 8;
  }
};

// The ring's stages in turn, and the parity of their barriers' phases.
struct Turn {
  int stage = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// The producer warp: pages [r0, r1) of the list page_of, ids 32 at a time.
template <typename PageOf>
__device__ __forceinline__ void load_pages(const Ring& R, const CUtensorMap* map,
                                           const MaskedArgs& a, int b, int r0, int r1, int lane,
                                           const PageOf& page_of) {
  const int n = r1 - r0;
  auto load_ids = [&](int k0) {
    int pid = -1;
    if (k0 + lane < n) {
      pid = a.block_table[static_cast<int64_t>(b) * a.max_blocks + page_of(r0 + k0 + lane)];
      if (pid < 0 || pid >= a.num_pages) {
        record_error(a.dev_err, kErrPage);
        pid = -1;
      }
    }
    return pid;
  };
  const uint64_t policy = l2_policy_evict_first();
  int ids = load_ids(0), ids_next = load_ids(32);
  int k = 0;
  Turn T;
  for (; k < n; ++k, T.next()) {
    const int st = T.stage;
    if (k >= kStages) {
      const bool ok = mbar_wait_bounded(R.empty(st), T.phase ^ 1, a.wait_ns);
      if (!__all_sync(kFull, ok)) {
        if (lane == 0) record_error(a.dev_err, kErrTimeout);
        break;
      }
    }
    const int pid = __shfl_sync(kFull, ids, k & 31);
    if (lane == 0) {
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(R.meta(st)), "r"(page_of(r0 + k)),
                   "r"(pid)
                   : "memory");
      if (pid >= 0) {
        mbar_arrive_expect_tx(R.full(st), kPage8Bytes + kPageScales);
        tma_load_3d(R.page(st), map, R.full(st), 0, 0, pid, policy);
        bulk_load(R.scales(st), a.scales + static_cast<int64_t>(pid) * kPageScales, kPageScales,
                  R.full(st), policy);
      } else {
        mbar_arrive(R.full(st));  // keep the stage's phase sequence in step
      }
    }
    __syncwarp();
    if ((k & 31) == 31) {
      ids = ids_next;
      ids_next = load_ids(k + 33);
    }
  }
  // every copy has landed before the CTA ends (full limit)
  for (int j = k > kStages ? k - kStages : 0; j < k; ++j)
    mbar_wait_bounded(R.full(j % kStages), (j / kStages) & 1);
}

__device__ __forceinline__ Ring make_ring(uint8_t* raw, const CUtensorMap* map) {
  const Ring R{(smem_addr(raw) + 1023u) & ~1023u};
  if (threadIdx.x == 0) {
    tma_prefetch_desc(map);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(R.full(s), 1);
      mbar_init(R.empty(s), kWarps);
    }
    fence_barrier_init();
  }
  __syncthreads();
  return R;
}

// Column 2 ft + j of S as a row's output or, where the row has several ranges, as
// its partial result number `part`.
__device__ __forceinline__ void put_row(const State& S, int j, int fg, uint16_t* out, bool partial,
                                        float* acc, float* ml, int64_t part) {
  if (partial) {
    float* dst = acc + part * kHeadDim + fg;
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[8 * i] = j == 0 ? S.o[i >> 1][i & 1].x : S.o[i >> 1][i & 1].y;
    if (fg == 0) *reinterpret_cast<float2*>(ml + 2 * part) = make_float2(S.m[j], S.l[j]);
  } else {
    const float inv = S.l[j] > 0.f || S.l[j] != S.l[j] ? 1.f / S.l[j] : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      out[fg + 8 * i] = static_cast<uint16_t>(pack_bf16x2(
          (j == 0 ? S.o[i >> 1][i & 1].x : S.o[i >> 1][i & 1].y) * inv, 0.f));
  }
}

// One token a sequence; grid (ranges, batch).
template <int kFmt>
__global__ void __launch_bounds__(kThreads, kCtas)
    paged8_decode_kernel(const __grid_constant__ CUtensorMap map, const MaskedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, g = tid >> 5;
  const int split = blockIdx.x, b = blockIdx.y;
  const Ring R = make_ring(smem_raw, &map);
  wait_for_prior_grids();
  allow_dependent_grids();
  const Visible V(clamped_len(a, b, tid == 0 && split == 0), a.window, a.sinks);
  const int r0 = static_cast<int>(static_cast<int64_t>(V.n) * split / a.num_splits);
  const int r1 = static_cast<int>(static_cast<int64_t>(V.n) * (split + 1) / a.num_splits);
  if (g == kWarps) {
    load_pages(R, &map, a, b, r0, r1, lane, [&](int i) { return V.page(i); });
    return;
  }

  const Lane P(lane);
  uint32_t qb[4][2];
  const int64_t row0 = static_cast<int64_t>(b) * kNumQHeads + g * kGroup;
  const float undo = load_q(a.q + (row0 + (P.fg & 3)) * kHeadDim, P.ft, qb);
  // factors of the scores of columns 2 ft and 2 ft + 1
  const int h = (2 * P.ft) & 3;
  const float c0 = a.scale_log2 * __shfl_sync(kFull, undo, 4 * h);
  const float c1 = a.scale_log2 * __shfl_sync(kFull, undo, 4 * h + 4);
  State S;
  S.reset();
  // Two pages at a time: one alone is a chain of latencies (copy, products, weights,
  // products), and what is checked is checked once for both.
  const int n = r1 - r0;
  Turn T;
  for (int k = 0; k < n; k += 2) {
    const int st0 = T.stage, phase0 = T.phase;
    T.next();
    const int st1 = T.stage, phase1 = T.phase;
    T.next();
    bool ready = mbar_wait_bounded(R.full(st0), phase0, a.wait_ns);
    if (k + 1 < n) ready &= mbar_wait_bounded(R.full(st1), phase1, a.wait_ns);
    if (!__all_sync(kFull, ready)) {
      if (lane == 0) record_error(a.dev_err, kErrTimeout);
      break;
    }
    // seen tokens of the pages (none where there is none, or it was not read)
    auto seen = [&](int st, bool there) {
      const uint2 meta = lds64(R.meta(st));
      if (!there || static_cast<int>(meta.y) < 0) return 0u;
      return V.whole(meta.x) ? 0xFFFFu : V.mask(meta.x);
    };
    const uint32_t vis0 = seen(st0, true), vis1 = seen(st1, k + 1 < n);
    const uint32_t kt0 = R.page(st0) + g * kBlockBytes, kt1 = R.page(st1) + g * kBlockBytes;
    constexpr uint32_t kV = kNumKvHeads * kBlockBytes;
    const float sk0 = scale_value(lds8(R.scales(st0) + g));
    const float sk1 = scale_value(lds8(R.scales(st1) + g));
    const float sv0 = scale_value(lds8(R.scales(st0) + kNumKvHeads + g));
    const float sv1 = scale_value(lds8(R.scales(st1) + kNumKvHeads + g));
    // (a factor of 0 would make NaN of a masked score)
    const float f[2][2] = {{fmaxf(c0 * sk0, 0x1p-126f), fmaxf(c1 * sk0, 0x1p-126f)},
                           {fmaxf(c0 * sk1, 0x1p-126f), fmaxf(c1 * sk1, 0x1p-126f)}};
    float s[2][4];
    uint32_t b[2][2];
    auto scores = [&](uint32_t kt, float (&x)[4]) {
      uint32_t ka[4][4];
      load_k<kFmt>(kt, P, ka);
      mma_new(x, ka[0], qb[0][0], qb[0][1]);
#pragma unroll
      for (int kk = 1; kk < 4; ++kk) mma_add(x, ka[kk], qb[kk][0], qb[kk][1]);
    };
    if ((vis0 & vis1) == 0xFFFFu) {
      scores(kt0, s[0]);
      scores(kt1, s[1]);
      move_reference(s, f, S);
      page_weights(s[0], f[0], P.ft, S, b[0][0], b[0][1]);
      page_weights(s[1], f[1], P.ft, S, b[1][0], b[1][1]);
      add_values<kFmt>(kt0 + kV, P, sv0, b[0][0], b[0][1], S);
      add_values<kFmt>(kt1 + kV, P, sv1, b[1][0], b[1][1], S);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t vis = i == 0 ? vis0 : vis1, kt = i == 0 ? kt0 : kt1;
        s[i][0] = s[i][1] = s[i][2] = s[i][3] = -INFINITY;
        if (vis == 0u) continue;
        scores(kt, s[i]);
        if (!((vis >> P.tok) & 1u)) s[i][0] = s[i][1] = -INFINITY;
        if (!((vis >> (P.tok + 2)) & 1u)) s[i][2] = s[i][3] = -INFINITY;
        if constexpr (kFmt == kKv8E4m3) hide_v(kt + kV, vis, lane);
      }
      // (the scales of a page that was not read may be anything)
      const float g2[2][2] = {{vis0 ? f[0][0] : 1.f, vis0 ? f[0][1] : 1.f},
                              {vis1 ? f[1][0] : 1.f, vis1 ? f[1][1] : 1.f}};
      move_reference(s, g2, S);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        page_weights(s[i], g2[i], P.ft, S, b[i][0], b[i][1]);
        if ((i == 0 ? vis0 : vis1) != 0u)
          add_values<kFmt>((i == 0 ? kt0 : kt1) + kV, P, i == 0 ? sv0 : sv1, b[i][0], b[i][1], S);
      }
    }
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(R.empty(st0));
      if (k + 1 < n) mbar_arrive(R.empty(st1));
    }
  }

  // the terms' columns meet; lanes ft < 2 hold heads 2 ft and 2 ft + 1
#pragma unroll
  for (int i = 4; i <= 16; i <<= 1) {
    S.l[0] += __shfl_xor_sync(kFull, S.l[0], i);
    S.l[1] += __shfl_xor_sync(kFull, S.l[1], i);
  }
#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      S.o[mt][e].x += __shfl_xor_sync(kFull, S.o[mt][e].x, 2);
      S.o[mt][e].y += __shfl_xor_sync(kFull, S.o[mt][e].y, 2);
    }
  if (P.ft >= 2) return;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t row = row0 + 2 * P.ft + j;
    put_row(S, j, P.fg, a.out + row * kHeadDim, a.num_splits > 1, a.part_acc, a.part_ml,
            row * a.num_splits + split);
  }
}

// Chunks of at most four tokens: the 16 query rows of a kv head (row = 4 token +
// head) as M of both products, tokens and then dims as N.  Rows fg and fg + 8 of a
// lane are of tokens fg / 4 and 2 + fg / 4.  The scores' fragment of a page is the
// weights' of the second product as it stands.  grid (ranges, batch).  kBeside:
// launched right after the tcgen05 kernel of the same call, as short_chunk.cu's
// kernel is: it starts at once, and its first CTA and those without a short chunk
// end after that grid.
template <int kFmt, bool kBeside>
__global__ void __launch_bounds__(kThreads, kCtas)
    paged8_short_chunk_kernel(const __grid_constant__ CUtensorMap map, const MaskedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, g = tid >> 5;
  const int split = blockIdx.x, b = blockIdx.y;
  const Ring R = make_ring(smem_raw, &map);
  if constexpr (!kBeside) wait_for_prior_grids();
  allow_dependent_grids();
  const int o0 = a.token_offsets[b], o1 = a.token_offsets[b + 1];
  const bool bad_offsets = o0 < 0 || o1 < o0 || o1 > a.num_tokens;
  if (bad_offsets && !kBeside && tid == 0) record_error(a.dev_err, kErrOffsets);
  if (bad_offsets || o1 == o0 || o1 - o0 > kShortTokens) {
    if constexpr (kBeside) wait_for_prior_grids();
    return;
  }
  const int nt = o1 - o0;
  const int L = clamped_len(a, b, tid == 0 && split == 0);
  const int pos0 = L - nt;
  if (pos0 < 0 && tid == 0 && split == 0) record_error(a.dev_err, kErrPosition);
  // pages that some row sees: those of the sinks, then those of the windows
  const int end = pos0 + nt, p_first = max(pos0, 0);
  const int lo = p_first >= a.window ? p_first - a.window + 1 : 0;
  const int w0 = lo / kPageSize;
  const int ns = min((min(a.sinks, lo) + kPageSize - 1) / kPageSize, w0);
  const int pages = end > 0 ? ns + (end + kPageSize - 1) / kPageSize - w0 : 0;
  const int r0 = static_cast<int>(static_cast<int64_t>(pages) * split / a.short_splits);
  const int r1 = static_cast<int>(static_cast<int64_t>(pages) * (split + 1) / a.short_splits);
  if (g == kWarps) {
    load_pages(R, &map, a, b, r0, r1, lane, [&](int i) { return i < ns ? i : w0 + (i - ns); });
    if (kBeside && blockIdx.x == 0 && blockIdx.y == 0) wait_for_prior_grids();
    return;
  }

  const Lane P(lane);
  uint32_t qa[4][4];  // A fragments: [k-step][row fg, fg + 8 of dims {0, 1}, then {2, 3}]
  float c[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int tok = 2 * i + (P.fg >> 2);
    uint32_t qb[4][2];
    c[i] = a.scale_log2 *
           load_q(tok < nt ? a.q + (static_cast<int64_t>(o0 + tok) * kNumQHeads + g * kGroup +
                                    (P.fg & 3)) * kHeadDim
                           : nullptr,
                  P.ft, qb);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      qa[kk][i] = qb[kk][0];
      qa[kk][2 + i] = qb[kk][1];
    }
  }
  float2 o[8][2];  // dims 8 nt + 2 ft, + 1 of rows fg and fg + 8
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = make_float2(0.f, 0.f);
  // bits of a page's slots below token x (as a distance from the page's first)
  auto below = [](int64_t x) {
    return x <= 0 ? 0u : (x >= kPageSize ? 0xFFFFu : (1u << static_cast<int>(x)) - 1u);
  };
  // tokens of the page at `base` that positions p0 to p1 see, taken together
  auto seen_by = [&](int base, int p0, int p1) {
    return below(static_cast<int64_t>(p1) + 1 - base) &
           ((0xFFFFu & ~below(static_cast<int64_t>(p0) - a.window + 1 - base)) |
            below(static_cast<int64_t>(a.sinks) - base));
  };
  Turn T;
  for (int k = 0; k < r1 - r0; ++k, T.next()) {
    const int st = T.stage;
    const bool ready = mbar_wait_bounded(R.full(st), T.phase, a.wait_ns);
    if (!__all_sync(kFull, ready)) {
      if (lane == 0) record_error(a.dev_err, kErrTimeout);
      break;
    }
    const uint2 meta = lds64(R.meta(st));
    if (static_cast<int>(meta.y) >= 0) {
      const uint32_t kt = R.page(st) + g * kBlockBytes, vt = kt + kNumKvHeads * kBlockBytes;
      const float sk = scale_value(lds8(R.scales(st) + g));
      const float sv = scale_value(lds8(R.scales(st) + kNumKvHeads + g));
      const int base = static_cast<int>(meta.x) * kPageSize;
      // does every row see the whole page?
      const bool whole = base + kPageSize - 1 <= pos0 &&
                         (static_cast<int64_t>(base) > static_cast<int64_t>(end) - 1 - a.window ||
                          base + kPageSize <= a.sinks);
      // s[j][2 i + e]: row fg + 8 i, token 4 ft + 2 j + e
      float s[2][4];
      {
        const uint4 x = lds128(kt + P.k0), y = lds128(kt + P.k1);
        const uint32_t k0[4] = {x.x, x.y, x.z, x.w}, k1[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint32_t b0, b1, d0, d1;
          decode_f16<kFmt>(k0[kk], b0, b1);
          decode_f16<kFmt>(k1[kk], d0, d1);
          if (kk == 0) {
            mma_new(s[0], qa[kk], b0, b1);
            mma_new(s[1], qa[kk], d0, d1);
          } else {
            mma_add(s[0], qa[kk], b0, b1);
            mma_add(s[1], qa[kk], d0, d1);
          }
        }
      }
      const float f[2] = {c[0] * sk, c[1] * sk};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] *= f[e >> 1];
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int p = pos0 + 2 * i + (P.fg >> 2);
          const uint32_t vis = seen_by(base, p, p) >> (4 * P.ft);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!((vis >> (2 * j + e)) & 1u)) s[j][2 * i + e] = -INFINITY;
        }
        if constexpr (kFmt == kKv8E4m3) hide_v(vt, seen_by(base, pos0, end - 1), lane);
      }
      // the running reference of both rows
      float mx[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        mx[i] = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
      if (__any_sync(kFull, mx[0] > m[0] + kMoveLog2 || mx[1] > m[1] + kMoveLog2)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(kFull, mx[i], 1));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(kFull, mx[i], 2));
          const float top = fmaxf(m[i], mx[i]);
          const float alpha = fast_exp2(m[i] - fmaxf(top, kLowestFloat));
          l[i] *= alpha;
#pragma unroll
          for (int d = 0; d < 8; ++d) o[d][i] = fmul2(o[d][i], make_float2(alpha, alpha));
          m[i] = top;
        }
      }
      // weights as two f16 terms
      uint32_t hi[4], lo2[4];  // A fragments: row fg of tokens {0, 1}, row fg + 8, then {2, 3}
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float d = kLift - fmaxf(m[i], kLowestFloat);
          const float p0 = fast_exp2(s[j][2 * i] + d), p1 = fast_exp2(s[j][2 * i + 1] + d);
          l[i] += p0 + p1;
          const uint32_t w = pack_f16x2(p0, p1);
          const float2 r = f16x2_to_float2(w);
          hi[2 * j + i] = w;
          lo2[2 * j + i] = pack_f16x2(p0 - r.x, p1 - r.y);
        }
      uint32_t vb[8];
      ldsm_b8_trans(vt + P.v0, *reinterpret_cast<uint32_t(*)[4]>(&vb[0]));
      ldsm_b8_trans(vt + P.v1, *reinterpret_cast<uint32_t(*)[4]>(&vb[4]));
      const float2 s2 = make_float2(sv, sv);
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        uint32_t b0, b1;
        decode_f16<kFmt>(vb[d], b0, b1);
        float t[4];
        mma_new(t, hi, b0, b1);
        mma_add(t, lo2, b0, b1);
        o[d][0] = ffma2(make_float2(t[0], t[1]), s2, o[d][0]);
        o[d][1] = ffma2(make_float2(t[2], t[3]), s2, o[d][1]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(R.empty(st));
  }

#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(kFull, l[i], 1);
    l[i] += __shfl_xor_sync(kFull, l[i], 2);
    const int tok = 2 * i + (P.fg >> 2), h = P.fg & 3;
    if (tok >= nt) continue;
    if (a.short_splits > 1) {
      const int64_t part = short_part_row(b, g, tok * kGroup + h) * a.short_splits + split;
      float2* dst = reinterpret_cast<float2*>(a.short_acc + part * kHeadDim) + P.ft;
#pragma unroll
      for (int d = 0; d < 8; ++d) dst[4 * d] = o[d][i];
      if (P.ft == 0) *reinterpret_cast<float2*>(a.short_ml + 2 * part) = make_float2(m[i], l[i]);
    } else {
      const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;
      uint32_t* dst = reinterpret_cast<uint32_t*>(
                          a.out + (static_cast<int64_t>(o0 + tok) * kNumQHeads + g * kGroup + h) *
                                      kHeadDim) + P.ft;
#pragma unroll
      for (int d = 0; d < 8; ++d) dst[4 * d] = pack_bf16x2(o[d][i].x * inv, o[d][i].y * inv);
    }
  }
}

// Combine a row's ranges, added in an order that does not change.  Up to kFewRanges
// of them a warp to a row; more take a CTA to a row, warp w the ranges w, w +
// kMergeWarps, ... (each step of a sum is an L2 latency: the 304 ranges of one
// sequence of 30011 tokens took 33 us with one warp, 9 with eight and a maximum over
// all ranges first).
constexpr int kMergeRows = 4, kMergeWarps = 16, kFewRanges = 16;
__global__ void __launch_bounds__(32 * kMergeRows) merge8_few_kernel(const MaskedArgs a) {
  allow_dependent_grids();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeRows + (threadIdx.x >> 5);
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + row * a.num_splits;
  const float2* acc =
      reinterpret_cast<const float2*>(a.part_acc) + row * a.num_splits * (kHeadDim / 2) + lane;
  reinterpret_cast<uint32_t*>(a.out + row * kHeadDim)[lane] =
      merge_ranges(ml, acc, a.num_splits, lane);
}

__global__ void __launch_bounds__(32 * kMergeWarps) merge8_many_kernel(const MaskedArgs a) {
  __shared__ float2 s_ml[kMergeWarps];
  __shared__ float2 s_o[kMergeWarps][kHeadDim / 2];
  allow_dependent_grids();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, splits = a.num_splits;
  const int64_t row = blockIdx.x;
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + row * splits;
  const float2* acc =
      reinterpret_cast<const float2*>(a.part_acc) + row * splits * (kHeadDim / 2) + lane;
  // this warp's state; a range that saw no token has a sum of 0
  float M = -INFINITY, L = 0.f;
  float2 O = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int s0 = w; s0 < splits; s0 += 32 * kMergeWarps) {
    // lane i: (max, sum) of range s0 + i kMergeWarps
    const int mine = s0 + lane * kMergeWarps;
    const float2 x = mine < splits ? __ldcg(ml + mine) : make_float2(-INFINITY, 0.f);
    float top = x.y != 0.f ? x.x : -INFINITY;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, i));
    top = fmaxf(top, M);
    const float old = M == -INFINITY ? 1.f : fast_exp2(M - top);
    // (-inf: a NaN row)
    const float wt = x.y == 0.f ? 0.f : x.x == -INFINITY ? 1.f : fast_exp2(x.x - top);
    float sum = x.y == 0.f ? 0.f : x.y * wt;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(kFull, sum, i);
    L = L * old + sum;
    O.x *= old;
    O.y *= old;
    M = top;
#pragma unroll 1
    for (int e0 = 0; e0 < 32 && s0 + e0 * kMergeWarps < splits; e0 += 16) {
      float2 v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int s = s0 + (e0 + e) * kMergeWarps;
        v[e] = s < splits ? __ldcg(acc + static_cast<int64_t>(s) * (kHeadDim / 2))
                          : make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float f = __shfl_sync(kFull, wt, e0 + e);
        if (f != 0.f) {  // (what a range without tokens left is not read)
          O.x = fmaf(v[e].x, f, O.x);
          O.y = fmaf(v[e].y, f, O.y);
        }
      }
    }
  }
  s_o[w][lane] = O;
  if (lane == 0) s_ml[w] = make_float2(M, L);
  __syncthreads();
  if (w > 0) return;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kMergeWarps; ++i) top = fmaxf(top, s_ml[i].x);
  L = 0.f;
  O = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kMergeWarps; ++i) {
    if (s_ml[i].y == 0.f) continue;
    const float f = s_ml[i].x == -INFINITY ? 1.f : fast_exp2(s_ml[i].x - top);
    L = fmaf(s_ml[i].y, f, L);
    O.x = fmaf(s_o[i][lane].x, f, O.x);
    O.y = fmaf(s_o[i][lane].y, f, O.y);
  }
  const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
  reinterpret_cast<uint32_t*>(a.out + row * kHeadDim)[lane] = pack_bf16x2(O.x * inv, O.y * inv);
}

// Launch a streaming kernel, opting in to its shared memory once per device.
template <auto kKernel>
cudaError_t launch(const CUtensorMap& map, const MaskedArgs& a, int splits, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  const unsigned long long bit = 1ull << (device & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    err = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(kSmem));
    if (err != cudaSuccess) return err;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  return launch_pdl(kKernel, dim3(splits, a.batch), dim3(kThreads), kSmem, stream, map, a);
}

}  // namespace

cudaError_t launch_decode8(const CUtensorMap& page_map, const MaskedArgs& args, int format,
                           cudaStream_t stream) {
  const cudaError_t err =
      format == kKv8E4m3
          ? launch<paged8_decode_kernel<kKv8E4m3>>(page_map, args, args.num_splits, stream)
          : launch<paged8_decode_kernel<kKv8Int8>>(page_map, args, args.num_splits, stream);
  if (err != cudaSuccess || args.num_splits == 1) return err;
  static_assert(kNumQHeads % kMergeRows == 0, "whole CTAs of rows");
  if (args.num_splits > kFewRanges)
    return launch_pdl(merge8_many_kernel, dim3(args.batch * kNumQHeads), dim3(32 * kMergeWarps), 0,
                      stream, args);
  return launch_pdl(merge8_few_kernel, dim3(args.batch * (kNumQHeads / kMergeRows)),
                    dim3(32 * kMergeRows), 0, stream, args);
}

cudaError_t launch_short_chunks8(const CUtensorMap& page_map, const MaskedArgs& args, int format,
                                 bool beside, cudaStream_t stream) {
  const int n = args.short_splits;
  if (format == kKv8E4m3)
    return beside ? launch<paged8_short_chunk_kernel<kKv8E4m3, true>>(page_map, args, n, stream)
                  : launch<paged8_short_chunk_kernel<kKv8E4m3, false>>(page_map, args, n, stream);
  return beside ? launch<paged8_short_chunk_kernel<kKv8Int8, true>>(page_map, args, n, stream)
                : launch<paged8_short_chunk_kernel<kKv8Int8, false>>(page_map, args, n, stream);
}

}  // namespace pkv
