// kv8_attention.cu -- attention of one new token, or of chunks of a few, per
// sequence over the 8-bit paged cache, streaming its pages once.
//
// In a CTA a producer warp brings whole pages (16 KiB, all kv heads, one TMA box, and the
// 16 bytes of their scales) into a ring in shared memory, and warp g of eight takes kv
// head g's blocks of every page.  So a page is one copy and one barrier for all heads,
// and the heads' states never meet.
//
// A CTA takes a range of one sequence's pages (grid (ranges, sequences)) or, kShared,
// an even share of the batch's: the pages that the queries see, counted on from sequence
// to sequence, are dealt out to two CTAs an SM, CTA c of N the pages [c T / N,
// (c + 1) T / N) of T, which it works out from the lengths (a sum and a scan of them in
// every CTA).  A sequence that lies in one CTA is answered there; of the others each CTA
// leaves a partial result (two at most), which the merge kernel combines.
//
// Bound by memory, in the middle by latencies: one token for 256 sequences of 1024 to
// 2048 tokens (409 MB) 72 us, 5.7 TB/s; 64 x 4 new tokens over 1024 to 2048 (104 MB) 35
// us without the launches around (22 without the arithmetic).  There a scheduler's time
// counts: an MMA takes 8.3 cycles of it in which nothing else is issued (with 8 FMAs
// 17.7), so a page and head take 24 x 8.3 + 250, and an SM with two of the longest CTAs
// 29 us.  Two pages at a time, as for one token, or the next page's loads during this
// one's products hide latencies that are hidden already: 42 and 40.
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
// V's factors stay at 2^72 or below, as 2^31 tokens' codes times weights of 2^15 then
// sum to less than 2^127: where a block seen has a larger scale the accumulators, and
// the factors after it, are in larger units, and the row's sum is told at the end.
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
constexpr int kStages = 6, kCtas = kStream8Ctas;
constexpr int kOffScales = kStages * kPage8Bytes;
constexpr int kOffMeta = kOffScales + kStages * kPageScales;
constexpr int kOffBars = kOffMeta + kStages * 8;
constexpr size_t kSmem = 1024 + kOffBars + 2 * 8 * kStages;
static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "the CTAs of an SM fit");

constexpr float kMoveLog2 = 8.f;   // a score this far above the reference moves it
constexpr float kLift = 7.f;       // weights are 2^(s - m + kLift) <= 2^15
constexpr float kLowestFloat = -3.402823466e38f;
constexpr float kTopFactor = 0x1p72f;  // the largest factor of V

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
    // two tokens to a row of eight 16-byte chunks, chunk c of row r at chunk c ^ (r mod
    // 8) (TMA's 128-byte swizzle; boxes with rows of 64 bytes took 76 us for the 256
    // sequences above, these 71)
    auto at = [](int t, int c) {
      const int r = t >> 1;
      return static_cast<uint32_t>(r * 128 + (((4 * (t & 1) + c) ^ r) << 4));
    };
    k0 = at(tok, ft);
    k1 = at(tok + 2, ft);
    v0 = at(lane & 15, lane >> 4);
    v1 = at(lane & 15, 2 + (lane >> 4));
  }
};

// Accumulators of n pairs in units of 1 / down become such that a block of V whose
// scale's value is sv, a power of two, can be added: with the factor sv * down.
template <int n>
__device__ __forceinline__ void raise_units(float sv, float& down, float2 (&o)[n][2]) {
  const float factor = sv * down;
  if (factor <= kTopFactor) return;
  // kTopFactor / factor
  const float f = __uint_as_float(((127u + 127u + 72u) - (__float_as_uint(factor) >> 23)) << 23);
#pragma unroll
  for (int i = 0; i < n; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) o[i][j] = fmul2(o[i][j], make_float2(f, f));
  down *= f;
}
// A row's reference and sum beside accumulators in units of 1 / down: l 2^m is the same.
__device__ __forceinline__ void tell_units(float down, float& m, float& l) {
  m += static_cast<float>(127 - static_cast<int>(__float_as_uint(down) >> 23));
  l *= down;
}

// Online softmax of 8 query rows (columns of S^T) of a warp.
struct State {
  float m[2], l[2];    // of columns 2 ft, 2 ft + 1: reference, this lane's share of the sum
  float2 o[4][2];      // O^T: dims 16 mt + fg (+ 8), columns 2 ft, 2 ft + 1
  float down;          // ... in units of 1 / down
  __device__ __forceinline__ void reset() {
    down = 1.f;
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

// Move the references of S's rows to what the masked scores x of two pages ask for, and
// the accumulators' units to what sv does, the larger of their V scales' values; f: the
// factors of the pages' scores, of columns 2 ft and 2 ft + 1.
__device__ __forceinline__ void move_reference(const float (&x)[2][4], const float (&f)[2][2],
                                               float sv, State& S) {
  float mx0 = fmaxf(fmaxf(x[0][0], x[0][2]) * f[0][0], fmaxf(x[1][0], x[1][2]) * f[1][0]);
  float mx1 = fmaxf(fmaxf(x[0][1], x[0][3]) * f[0][1], fmaxf(x[1][1], x[1][3]) * f[1][1]);
  if (!__any_sync(kFull, mx0 > S.m[0] + kMoveLog2 || mx1 > S.m[1] + kMoveLog2 ||
                             sv * S.down > kTopFactor))
    return;
  raise_units(sv, S.down, S.o);
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
  for (int i = lane; i < kPageSize * 4; i += 32) {
    const int r = i >> 3, c = (i & 7) ^ r;
    if (!((vis >> (2 * r + (c >> 2))) & 1u)) sts128_zero(vt + i * 16);
  }
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

// The producer warp: pages [r0, r1) of a sequence's list, ids 32 at a time.  k counts
// the pages of all segments.  False: a wait ran out.
template <typename Seq>
__device__ __forceinline__ bool load_pages(const Ring& R, const CUtensorMap* map,
                                           const MaskedArgs& a, int b, const Seq& seq, int r0,
                                           int r1, int lane, Turn& T, int& k) {
  const int n = r1 - r0;
  auto load_ids = [&](int k0) {
    int pid = -1;
    if (k0 + lane < n) {
      pid = a.block_table[static_cast<int64_t>(b) * a.max_blocks + seq.page(r0 + k0 + lane)];
      if (pid < 0 || pid >= a.num_pages) {
        record_error(a.dev_err, kErrPage);
        pid = -1;
      }
    }
    return pid;
  };
  const uint64_t policy = l2_policy_evict_first();
  int ids = load_ids(0), ids_next = load_ids(32);
  for (int i = 0; i < n; ++i, ++k, T.next()) {
    const int st = T.stage;
    if (k >= kStages) {
      const bool ok = mbar_wait_bounded(R.empty(st), T.phase ^ 1, a.wait_ns);
      if (!__all_sync(kFull, ok)) return false;
    }
    const int pid = __shfl_sync(kFull, ids, i & 31);
    if (lane == 0) {
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(R.meta(st)), "r"(seq.page(r0 + i)),
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
    if ((i & 31) == 31) {
      ids = ids_next;
      ids_next = load_ids(i + 33);
    }
  }
  return true;
}

// Every copy has landed before the CTA ends (full limit): the last ones of k.
__device__ __forceinline__ void drain(const Ring& R, int k) {
  for (int j = k > kStages ? k - kStages : 0; j < k; ++j)
    mbar_wait_bounded(R.full(j % kStages), (j / kStages) & 1);
}

// The CTA's part of the work, dealt out as above, or with num_splits one range of one
// sequence.
struct Part {
  int64_t u0, u1;  // pages [u0, u1) of all
  int64_t base;    // pages before sequence b, the first of them
  int b;
};
constexpr int kLeastPages = 4;  // of a CTA, while there are fewer than all of them need
// Sequences up to this long are not cut: a part that would begin in one begins behind it
// (256 of 200 tokens in tables of 2048, cold: 25 us, 29 with cuts everywhere).
constexpr int kWholePages = 16;

// CTAs that share `total` pages, and the first page of one.
__device__ __forceinline__ int64_t parts_of(int64_t total, int ctas) {
  return max(1ll, min(static_cast<long long>(ctas), static_cast<long long>(total / kLeastPages)));
}
__device__ __forceinline__ int64_t part_start(int64_t total, int64_t parts, int64_t c) {
  return total * c / parts;
}

// make(b): sequence b's list.  By all threads of the CTA, some sequences in a row each.
// The first CTA writes the sequences' bases, and the total behind them, for the merge.
template <typename Make>
__device__ __forceinline__ Part share_out(const MaskedArgs& a, const Make& make) {
  __shared__ int64_t s_warp[kThreads / 32];
  __shared__ Part s_part;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += make(b).n;
  int64_t incl = sum;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const int64_t y = __shfl_up_sync(kFull, incl, x);
    if (lane >= x) incl += y;
  }
  if (lane == 31) s_warp[w] = incl;
  __syncthreads();
  int64_t base = incl - sum, total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < w) base += s_warp[i];
    total += s_warp[i];
  }
  const int64_t parts = parts_of(total, gridDim.x);
  Part p = {0, 0, 0, 0};
  if (blockIdx.x < parts) {
    p.u0 = part_start(total, parts, blockIdx.x);
    p.u1 = part_start(total, parts, blockIdx.x + 1);
  }
  auto holds = [](int64_t from, int64_t n, int64_t u) { return from <= u && u < from + n; };
  if (holds(base, sum, p.u0) || holds(base, sum, p.u1) || blockIdx.x == 0)
    for (int b = b0; b < b1; ++b) {
      const int n = make(b).n;
      auto moved = [&](int64_t u) { return n <= kWholePages && u > base ? base + n : u; };
      if (holds(base, n, p.u0)) {
        s_part.u0 = moved(p.u0);
        const bool behind = s_part.u0 == base + n;
        s_part.b = b + behind;
        s_part.base = behind ? s_part.u0 : base;
      }
      if (holds(base, n, p.u1)) s_part.u1 = moved(p.u1);
      if (blockIdx.x == 0) a.part_bases[b] = base;
      base += n;
    }
  if (blockIdx.x == 0 && tid == 0) a.part_bases[a.batch] = total;
  __syncthreads();
  if (p.u0 < p.u1) {
    p.b = s_part.b;
    p.base = s_part.base;
    p.u0 = s_part.u0;
    if (p.u1 < total) p.u1 = s_part.u1;
  }
  return p;
}

// Call f(b, list, r0, r1, slot) for the CTA's segments: pages [r0, r1) of sequence b,
// slot -1 where these are all of them, else the place of the partial result.  Ends
// when f returns false.
template <bool kShared, typename Make, typename F>
__device__ __forceinline__ void each_segment(int num_splits, const Part& p, const Make& make,
                                             const F& f) {
  if constexpr (!kShared) {
    const int b = blockIdx.y;
    const auto seq = make(b);
    const int r0 = static_cast<int>(static_cast<int64_t>(seq.n) * blockIdx.x / num_splits);
    const int r1 = static_cast<int>(static_cast<int64_t>(seq.n) * (blockIdx.x + 1) / num_splits);
    f(b, seq, r0, r1, num_splits > 1 ? b * num_splits + static_cast<int>(blockIdx.x) : -1);
  } else {
    int64_t base = p.base;
    for (int b = p.b; base < p.u1 && p.u0 < p.u1; ++b) {
      const auto seq = make(b);
      if (seq.n == 0) continue;
      const int r0 = p.u0 > base ? static_cast<int>(p.u0 - base) : 0;
      const int r1 = p.u1 - base < seq.n ? static_cast<int>(p.u1 - base) : seq.n;
      const bool all = r0 == 0 && r1 == seq.n;
      // (a part's first segment, or its last, which begins its sequence)
      if (!f(b, seq, r0, r1, all ? -1 : 2 * static_cast<int>(blockIdx.x) + (r0 == 0 ? 1 : 0)))
        return;
      base += seq.n;
    }
  }
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
__device__ __forceinline__ void put_row(const State& S, int j, int fg, uint16_t* out, float* acc,
                                        float* ml, int64_t part) {
  if (part >= 0) {
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

// Zero rows of a kv head's group for a token that sees nothing.
__device__ __forceinline__ void put_zeros(uint16_t* out, int lane) {
#pragma unroll
  for (int h = 0; h < kGroup; ++h) reinterpret_cast<uint32_t*>(out + h * kHeadDim)[lane] = 0u;
}

// One token of a kv head's group over n pages of the ring, V saying what it sees: q and
// out its four rows, part their place in the partial results or -1.  False: a wait ran
// out.
template <int kFmt>
__device__ __forceinline__ bool attend_one(const MaskedArgs& a, const Ring& R, const Lane& P,
                                           Turn& T, int g, int lane, const Visible& V, int n,
                                           const uint16_t* q, uint16_t* out, float* acc, float* ml,
                                           int64_t part) {
  uint32_t qb[4][2];
  const float undo = load_q(q + (P.fg & 3) * kHeadDim, P.ft, qb);
  // factors of the scores of columns 2 ft and 2 ft + 1
  const int h = (2 * P.ft) & 3;
  const float c0 = a.scale_log2 * __shfl_sync(kFull, undo, 4 * h);
  const float c1 = a.scale_log2 * __shfl_sync(kFull, undo, 4 * h + 4);
  State S;
  S.reset();
  bool ok = true;
  // Two pages at a time: one alone is a chain of latencies (copy, products, weights,
  // products), and what is checked is checked once for both.
  for (int k = 0; k < n; k += 2) {
    const int st0 = T.stage, phase0 = T.phase;
    T.next();
    const int st1 = T.stage, phase1 = T.phase;
    if (k + 1 < n) T.next();
    bool ready = mbar_wait_bounded(R.full(st0), phase0, a.wait_ns);
    if (k + 1 < n) ready &= mbar_wait_bounded(R.full(st1), phase1, a.wait_ns);
    if (!__all_sync(kFull, ready)) {
      if (lane == 0) record_error(a.dev_err, kErrTimeout);
      ok = false;
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
      move_reference(s, f, fmaxf(sv0, sv1), S);
      page_weights(s[0], f[0], P.ft, S, b[0][0], b[0][1]);
      page_weights(s[1], f[1], P.ft, S, b[1][0], b[1][1]);
      add_values<kFmt>(kt0 + kV, P, sv0 * S.down, b[0][0], b[0][1], S);
      add_values<kFmt>(kt1 + kV, P, sv1 * S.down, b[1][0], b[1][1], S);
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
      // (the scales of a page that was not read, or is not seen, may be anything)
      const float g2[2][2] = {{vis0 ? f[0][0] : 1.f, vis0 ? f[0][1] : 1.f},
                              {vis1 ? f[1][0] : 1.f, vis1 ? f[1][1] : 1.f}};
      move_reference(s, g2, fmaxf(vis0 ? sv0 : 0.f, vis1 ? sv1 : 0.f), S);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        page_weights(s[i], g2[i], P.ft, S, b[i][0], b[i][1]);
        if ((i == 0 ? vis0 : vis1) == 0u) continue;
        const float sv = i == 0 ? sv0 : sv1;
        add_values<kFmt>((i == 0 ? kt0 : kt1) + kV, P, sv * S.down, b[i][0], b[i][1], S);
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
  tell_units(S.down, S.m[0], S.l[0]);
  tell_units(S.down, S.m[1], S.l[1]);
#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      S.o[mt][e].x += __shfl_xor_sync(kFull, S.o[mt][e].x, 2);
      S.o[mt][e].y += __shfl_xor_sync(kFull, S.o[mt][e].y, 2);
    }
  if (P.ft < 2) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      put_row(S, j, P.fg, out + (2 * P.ft + j) * kHeadDim, acc, ml,
              part < 0 ? -1 : part + 2 * P.ft + j);
  }
  return ok;
}

// One token a sequence.  Grid: the CTAs that share the work, or (num_splits, batch).
template <int kFmt, bool kShared>
__global__ void __launch_bounds__(kThreads, kCtas)
    paged8_decode_kernel(const __grid_constant__ CUtensorMap map, const MaskedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, g = tid >> 5;
  const Ring R = make_ring(smem_raw, &map);
  wait_for_prior_grids();
  allow_dependent_grids();
  const bool report = blockIdx.x == 0 && (kShared || tid == 0);
  auto make = [&](int b) { return Visible(clamped_len(a, b, report), a.window, a.sinks); };
  Part part = {0, 0, 0, 0};
  if constexpr (kShared) part = share_out(a, make);
  Turn T;
  if (g == kWarps) {
    int k = 0;
    each_segment<kShared>(a.num_splits, part, make,
                 [&](int b, const Visible& V, int r0, int r1, int) {
                   const bool ok = load_pages(R, &map, a, b, V, r0, r1, lane, T, k);
                   if (!ok && lane == 0) record_error(a.dev_err, kErrTimeout);
                   return ok;
                 });
    drain(R, k);
    return;
  }

  // (while the first copies are on their way)
  if constexpr (kShared)
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x)
      if (make(b).n == 0)
        put_zeros(a.out + (static_cast<int64_t>(b) * kNumQHeads + g * kGroup) * kHeadDim, lane);
  const Lane P(lane);
  each_segment<kShared>(a.num_splits, part, make, [&](int b, const Visible& V, int r0, int r1,
                                                      int slot) {
    const int64_t row = (static_cast<int64_t>(b) * kNumQHeads + g * kGroup) * kHeadDim;
    return attend_one<kFmt>(a, R, P, T, g, lane, V, r1 - r0, a.q + row, a.out + row, a.part_acc,
                            a.part_ml,
                            slot < 0 ? -1 : static_cast<int64_t>(slot) * kNumQHeads + g * kGroup);
  });
}

// Chunks of at most four tokens: the 16 query rows of a kv head (row = 4 token +
// head) as M of both products, tokens and then dims as N.  Rows fg and fg + 8 of a
// lane are of tokens fg / 4 and 2 + fg / 4.  The scores' fragment of a page is the
// weights' of the second product as it stands.  Grid: the CTAs that share the work, or
// (short_splits, batch).  kBeside: launched right after the tcgen05 kernel of the same
// call, as short_chunk.cu's kernel is: it starts at once, and its first CTA and those
// without pages end after that grid.
constexpr int kShortRows = kShortTokens * kGroup;

// A short chunk and the pages that some row of it sees: those of the sinks, then those
// of the windows (no pages, and no tokens, of a sequence without a short chunk).
struct ShortList {
  int o0, nt, pos0, ns, w0, n;
  __device__ __forceinline__ int page(int i) const { return i < ns ? i : w0 + (i - ns); }
  __device__ __forceinline__ ShortList(const MaskedArgs& a, int b, bool report,
                                       bool report_offsets) {
    o0 = a.token_offsets[b];
    const int o1 = a.token_offsets[b + 1];
    const bool bad = o0 < 0 || o1 < o0 || o1 > a.num_tokens;
    if (bad && report_offsets) record_error(a.dev_err, kErrOffsets);
    nt = bad || o1 - o0 > kShortTokens ? 0 : o1 - o0;
    pos0 = ns = w0 = n = 0;
    if (nt == 0) return;
    const int L = clamped_len(a, b, report);
    pos0 = L - nt;
    if (pos0 < 0 && report) record_error(a.dev_err, kErrPosition);
    const int first = max(pos0, 0), lo = first >= a.window ? first - a.window + 1 : 0;
    w0 = lo / kPageSize;
    ns = min((min(a.sinks, lo) + kPageSize - 1) / kPageSize, w0);
    n = L > 0 ? ns + (L + kPageSize - 1) / kPageSize - w0 : 0;
  }
};

template <int kFmt, bool kBeside, bool kShared>
__global__ void __launch_bounds__(kThreads, kCtas)
    paged8_short_chunk_kernel(const __grid_constant__ CUtensorMap map, const MaskedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, g = tid >> 5;
  const Ring R = make_ring(smem_raw, &map);
  if constexpr (!kBeside) wait_for_prior_grids();
  allow_dependent_grids();
  const bool report = blockIdx.x == 0 && (kShared || tid == 0);
  auto make = [&](int b) { return ShortList(a, b, report, !kBeside && report); };
  Part part = {0, 0, 0, 0};
  if constexpr (kShared) part = share_out(a, make);
  Turn T;
  if (g == kWarps) {
    int k = 0;
    each_segment<kShared>(a.short_splits, part, make,
                 [&](int b, const ShortList& V, int r0, int r1, int) {
                   const bool ok = load_pages(R, &map, a, b, V, r0, r1, lane, T, k);
                   if (!ok && lane == 0) record_error(a.dev_err, kErrTimeout);
                   return ok;
                 });
    drain(R, k);
    if (kBeside && ((blockIdx.x == 0 && blockIdx.y == 0) || k == 0)) wait_for_prior_grids();
    return;
  }

  // (while the first copies are on their way)
  if constexpr (kShared)
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
      const ShortList V = make(b);
      for (int t = 0; t < V.nt && V.n == 0; ++t)
        put_zeros(a.out + (static_cast<int64_t>(V.o0 + t) * kNumQHeads + g * kGroup) * kHeadDim,
                  lane);
    }
  const Lane P(lane);
  each_segment<kShared>(a.short_splits, part, make, [&](int b, const ShortList& V, int r0, int r1,
                                                  int slot) {
    const int nt = V.nt, o0 = V.o0, pos0 = V.pos0, end = V.pos0 + V.nt;
    if (nt == 0) return true;
    // A token by itself would leave three quarters of the MMAs empty: a chunk of 509
    // tokens beside 63 single ones over 1024 to 2047 took 62 us so, 51 with this.
    if (nt == 1) {
      const int64_t row = (static_cast<int64_t>(o0) * kNumQHeads + g * kGroup) * kHeadDim;
      return attend_one<kFmt>(
          a, R, P, T, g, lane, Visible(end, a.window, a.sinks), r1 - r0, a.q + row, a.out + row,
          a.short_acc, a.short_ml,
          slot < 0 ? -1 : (static_cast<int64_t>(slot) * kNumKvHeads + g) * kShortRows);
    }
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
    bool ok = true;
    float down = 1.f;
    float2 o[8][2];  // dims 8 nt + 2 ft, + 1 of rows fg and fg + 8, in units of 1 / down
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
    for (int k = 0; k < r1 - r0; ++k, T.next()) {
      const int st = T.stage;
      const bool ready = mbar_wait_bounded(R.full(st), T.phase, a.wait_ns);
      if (!__all_sync(kFull, ready)) {
        if (lane == 0) record_error(a.dev_err, kErrTimeout);
        ok = false;
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
        raise_units(sv, down, o);
        const float2 s2 = make_float2(sv * down, sv * down);
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
      tell_units(down, m[i], l[i]);
      const int tok = 2 * i + (P.fg >> 2), h = P.fg & 3;
      if (tok >= nt) continue;
      if (slot >= 0) {
        const int64_t row =
            (static_cast<int64_t>(slot) * kNumKvHeads + g) * kShortRows + tok * kGroup + h;
        float2* dst = reinterpret_cast<float2*>(a.short_acc + row * kHeadDim) + P.ft;
#pragma unroll
        for (int d = 0; d < 8; ++d) dst[4 * d] = o[d][i];
        if (P.ft == 0) *reinterpret_cast<float2*>(a.short_ml + 2 * row) = make_float2(m[i], l[i]);
      } else {
        const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;
        uint32_t* dst = reinterpret_cast<uint32_t*>(
                            a.out + (static_cast<int64_t>(o0 + tok) * kNumQHeads + g * kGroup + h) *
                                        kHeadDim) + P.ft;
#pragma unroll
        for (int d = 0; d < 8; ++d) dst[4 * d] = pack_bf16x2(o[d][i].x * inv, o[d][i].y * inv);
      }
    }
    return ok;
  });
}

// The partial results of a sequence's rows: how many, and the place of each.
template <bool kShared>
struct Pieces {
  int n;          // 1 where the sequence has none: it was answered at once
  int64_t first;  // its range or part
  __device__ __forceinline__ Pieces(const MaskedArgs& a, int num_splits, int b) {
    n = num_splits;
    first = static_cast<int64_t>(b) * num_splits;
    if constexpr (kShared) {
      const int64_t base = a.part_bases[b], past = a.part_bases[b + 1];
      const int64_t total = a.part_bases[a.batch];
      n = 1;
      if (past - base <= kWholePages) return;
      const int64_t parts = parts_of(total, a.part_ctas);
      // the part that holds page u is the last one that starts at or before it
      first = ((base + 1) * parts - 1) / total;
      n = static_cast<int>((past * parts - 1) / total - first) + 1;
    }
  }
  __device__ __forceinline__ int slot(int i) const {
    const int c = static_cast<int>(first) + i;
    return kShared ? 2 * c + (i == 0 ? 1 : 0) : c;
  }
};

// Row r of sequence b (decode: query head; chunks: kv head, token, head of the group)
// in the partial results and in the output; false: there is no such row.
template <bool kChunk>
__device__ __forceinline__ bool merged_row(const MaskedArgs& a, int b, int r, uint16_t*& out) {
  if constexpr (kChunk) {
    const int o0 = a.token_offsets[b], o1 = a.token_offsets[b + 1];
    const int g = r / kShortRows, tok = r % kShortRows / kGroup, h = r % kGroup;
    if (o0 < 0 || o1 > a.num_tokens || o1 <= o0 || o1 - o0 > kShortTokens || tok >= o1 - o0)
      return false;
    out = a.out + (static_cast<int64_t>(o0 + tok) * kNumQHeads + g * kGroup + h) * kHeadDim;
  } else {
    out = a.out + (static_cast<int64_t>(b) * kNumQHeads + r) * kHeadDim;
  }
  return true;
}

// Combine a row's partial results, added in an order that does not change.  Where few
// are expected a warp takes a row; else a CTA does, warp w the results w, w +
// kWarpsOfRow, ... (each step of a sum is an L2 latency: 304 of one sequence of 30011
// tokens took 33 us with one warp), of sixteen warps while the rows are few, of four
// where these would take several waves (cold, 4 tokens of 8 sequences of 2048: 30 us
// with sixteen, 23.5 with four; of 2 of 30000: 35 and 39).  grid (rows / 4 or rows,
// batch).
constexpr int kMergeRows = 4, kFewPieces = 16, kFewRows = 256;
template <bool kChunk, bool kShared, int kWarpsOfRow>
__global__ void __launch_bounds__(32 * (kWarpsOfRow == 1 ? kMergeRows : kWarpsOfRow))
    merge8_kernel(const MaskedArgs a) {
  constexpr bool kMany = kWarpsOfRow > 1;
  constexpr int kRows = kChunk ? kNumKvHeads * kShortRows : kNumQHeads;
  __shared__ float2 s_ml[kWarpsOfRow];
  __shared__ float2 s_o[kWarpsOfRow][kHeadDim / 2];
  allow_dependent_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.y;
  const int r = kMany ? blockIdx.x : blockIdx.x * kMergeRows + warp, w = kMany ? warp : 0;
  const int num_splits = kChunk ? a.short_splits : a.num_splits;
  // The offsets are the call's input: grids before the call's own were waited for by its
  // first one, before this one could start.
  uint16_t* out;
  const bool there = merged_row<kChunk>(a, b, r, out);
  wait_for_prior_grids();
  if (!there) return;  // (the same for a row's warps)
  const Pieces<kShared> P(a, num_splits, b);
  if (P.n == 1) return;
  const float2* all_ml = reinterpret_cast<const float2*>(kChunk ? a.short_ml : a.part_ml) + r;
  const float2* all_acc = reinterpret_cast<const float2*>(kChunk ? a.short_acc : a.part_acc) +
                          static_cast<int64_t>(r) * (kHeadDim / 2) + lane;
  // this warp's state; a result that saw no token has a sum of 0
  float M = -INFINITY, L = 0.f;
  float2 O = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int s0 = w; s0 < P.n; s0 += 32 * kWarpsOfRow) {
    // lane i: the place, and (max, sum), of result s0 + i kWarpsOfRow
    const int mine = s0 + lane * kWarpsOfRow;
    const int at = mine < P.n ? P.slot(mine) : 0;
    const float2 x = mine < P.n ? __ldcg(all_ml + static_cast<int64_t>(at) * kRows)
                                : make_float2(-INFINITY, 0.f);
    // (of 16 results at most, half at a time leaves registers for more warps)
    constexpr int kAhead = kMany || kShared ? 16 : 8;
    float2 v[kAhead];
    auto load = [&](int e0) {
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int64_t place = __shfl_sync(kFull, at, e0 + e);
        v[e] = s0 + (e0 + e) * kWarpsOfRow < P.n
                   ? __ldcg(all_acc + place * (kRows * kHeadDim / 2))
                   : make_float2(0.f, 0.f);
      }
    };
    load(0);
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
    for (int e0 = 0;;) {
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const float f = __shfl_sync(kFull, wt, e0 + e);
        if (f != 0.f) {  // (what a range without tokens left is not read)
          O.x = fmaf(v[e].x, f, O.x);
          O.y = fmaf(v[e].y, f, O.y);
        }
      }
      e0 += kAhead;
      if (e0 == 32 || s0 + e0 * kWarpsOfRow >= P.n) break;
      load(e0);
    }
  }
  if constexpr (kMany) {
    s_o[w][lane] = O;
    if (lane == 0) s_ml[w] = make_float2(M, L);
    __syncthreads();
    if (w > 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kWarpsOfRow; ++i) top = fmaxf(top, s_ml[i].x);
    L = 0.f;
    O = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kWarpsOfRow; ++i) {
      if (s_ml[i].y == 0.f) continue;
      const float f = s_ml[i].x == -INFINITY ? 1.f : fast_exp2(s_ml[i].x - top);
      L = fmaf(s_ml[i].y, f, L);
      O.x = fmaf(s_o[i][lane].x, f, O.x);
      O.y = fmaf(s_o[i][lane].y, f, O.y);
    }
  }
  const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
  reinterpret_cast<uint32_t*>(out)[lane] = pack_bf16x2(O.x * inv, O.y * inv);
}

template <bool kChunk, bool kShared>
cudaError_t launch_merge(const MaskedArgs& a, int pieces, cudaStream_t stream) {
  constexpr int kRows = kChunk ? kNumKvHeads * kShortRows : kNumQHeads;
  if (pieces > kFewPieces && kRows * a.batch <= kFewRows)
    return launch_pdl(merge8_kernel<kChunk, kShared, 16>, dim3(kRows, a.batch), dim3(32 * 16), 0,
                      stream, a);
  if (pieces > kFewPieces)
    return launch_pdl(merge8_kernel<kChunk, kShared, 4>, dim3(kRows, a.batch), dim3(32 * 4), 0,
                      stream, a);
  return launch_pdl(merge8_kernel<kChunk, kShared, 1>, dim3(kRows / kMergeRows, a.batch),
                    dim3(32 * kMergeRows), 0, stream, a);
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
  return launch_pdl(kKernel, splits > 0 ? dim3(splits, a.batch) : dim3(a.part_ctas), dim3(kThreads),
                    kSmem, stream, map, a);
}

// (shared: the pieces of a sequence where all are of a length)
template <int kFmt>
cudaError_t launch_decode(const CUtensorMap& map, const MaskedArgs& a, cudaStream_t stream) {
  const int n = a.num_splits;
  const cudaError_t err = n > 0 ? launch<paged8_decode_kernel<kFmt, false>>(map, a, n, stream)
                                : launch<paged8_decode_kernel<kFmt, true>>(map, a, n, stream);
  if (err != cudaSuccess || n == 1) return err;
  return n > 0 ? launch_merge<false, false>(a, n, stream)
               : launch_merge<false, true>(a, a.part_ctas / a.batch, stream);
}

template <int kFmt, bool kBeside>
cudaError_t launch_short(const CUtensorMap& map, const MaskedArgs& a, cudaStream_t stream) {
  const int n = a.short_splits;
  const cudaError_t err =
      n > 0 ? launch<paged8_short_chunk_kernel<kFmt, kBeside, false>>(map, a, n, stream)
            : launch<paged8_short_chunk_kernel<kFmt, kBeside, true>>(map, a, n, stream);
  if (err != cudaSuccess || n == 1) return err;
  return n > 0 ? launch_merge<true, false>(a, n, stream)
               : launch_merge<true, true>(a, a.part_ctas / a.batch, stream);
}

}  // namespace

cudaError_t launch_decode8(const CUtensorMap& page_map, const MaskedArgs& args, int format,
                           cudaStream_t stream) {
  return format == kKv8E4m3 ? launch_decode<kKv8E4m3>(page_map, args, stream)
                            : launch_decode<kKv8Int8>(page_map, args, stream);
}

cudaError_t launch_short_chunks8(const CUtensorMap& page_map, const MaskedArgs& args, int format,
                                 bool beside, cudaStream_t stream) {
  if (format == kKv8E4m3)
    return beside ? launch_short<kKv8E4m3, true>(page_map, args, stream)
                  : launch_short<kKv8E4m3, false>(page_map, args, stream);
  return beside ? launch_short<kKv8Int8, true>(page_map, args, stream)
                : launch_short<kKv8Int8, false>(page_map, args, stream);
}

}  // namespace pkv
