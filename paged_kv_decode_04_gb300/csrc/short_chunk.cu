// short_chunk.cu -- attention of chunks of at most kShortTokens new tokens
// (drafted tokens to verify, or the single tokens beside a prompt's chunk)
// over the paged cache.
//
// Such a chunk reads its whole cache for 16 query rows of a kv head, so it is
// bound by memory, and a 128-row MMA tile would be mostly padding: a unit of
// the tcgen05 kernel costs the same for 16 rows as for 128: with cold caches 64
// sequences of 5 to 16 tokens over 2048 take 65-68 us there, of 4 tokens 53 us
// here (256 over 512: 102 and 59 us).  This kernel
// streams pages as the one-token kernels do: one CTA per (sequence, kv head,
// range of the pages), 4 warps taking every 4th page through private rings of
// 4 KiB tiles, mma.sync with the tokens of a page as M and the query rows as
// N (row = 4 token + head, 8 rows = 2 tokens to an n-tile).
//
// A query at position p sees token t when t <= p and (t > p - window or
// t < sinks), so the rows of a page differ in what they see only near the end
// of the sequence, of the window and of the sinks.  There the scores of unseen
// tokens become -inf, and non-finite V values become zero in shared memory
// (0 x NaN is NaN); a row that sees such a value gets it at the end.
// Weights enter the product with V as two bf16 terms (16 significant bits), as
// in the one-token kernels, so a single token's result has their precision
// whichever call makes it.  The second term costs the 64 x 4 tokens over 2048
// 42.3 -> 43.3 us; moving the terms between the lanes with shuffles instead of
// movmatrix 44.7.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "decode_page.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// Tiles in flight per warp, and CTAs per SM: three of deep rings next to a long
// chunk, whose CTAs keep some SMs to themselves (fewer CTAs to an SM leave
// less behind when those SMs come free: 63 single tokens beside a chunk of
// 509 took 52 us, with four CTAs of shallow rings 65 us), four of shallow
// rings where every chunk may be short (64 x 4 tokens: 45 us, with three 53).
constexpr int kDeep = 4, kShallow = 3;
__host__ __device__ constexpr int ctas_per_sm(int stages) { return stages == kDeep ? 3 : 4; }
__host__ __device__ constexpr int ring_bytes(int stages) { return kWarps * stages * kTileBytes; }
constexpr int kTiles = kShortTokens / 2;         // n-tiles of 8 query rows
constexpr int kRows = kShortTokens * kGroup;     // query rows of a kv head
constexpr size_t smem_bytes(int stages) { return 1024 + ring_bytes(stages) + 8 * kWarps * stages; }
static_assert(kWarps * kRows * (2 + kHeadDim) * 4 <= ring_bytes(kShallow), "states fit in the ring");

// Online-softmax state of a warp for one n-tile (see AttnState).
struct TileState {
  float m_ref[2], l_run[2];
  float oacc[4][4];
};

// An 8 x 8 matrix of 16-bit values, lane l holding columns 2 (l & 3) and + 1 of
// row l / 4, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Fold a page's masked scores of one n-tile into S.  va: the page's V^T
// fragments (4 tiles of 16 dims).
__device__ __forceinline__ void fold_tile(const float (&s)[4], const uint32_t (&va)[4][4], float c,
                                          TileState& S) {
  float mx0 = fmaxf(s[0], s[2]) * c;
  float mx1 = fmaxf(s[1], s[3]) * c;
  const bool grow = mx0 > S.m_ref[0] + kRescaleLog2 || mx1 > S.m_ref[1] + kRescaleLog2;
  if (__any_sync(kFullMask, grow)) {
#pragma unroll
    for (int x = 4; x <= 16; x <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(kFullMask, mx0, x));
      mx1 = fmaxf(mx1, __shfl_xor_sync(kFullMask, mx1, x));
    }
    const float mx[2] = {mx0, mx1};
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const float m_new = fmaxf(S.m_ref[rr], mx[rr]);
      // (a row that has seen no token keeps its zeros)
      const float alpha = m_new == -INFINITY ? 1.f : fast_exp2(S.m_ref[rr] - m_new);
      S.l_run[rr] *= alpha;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        S.oacc[mt][rr] *= alpha;
        S.oacc[mt][2 + rr] *= alpha;
      }
      S.m_ref[rr] = m_new;
    }
  }
  float p[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float m = S.m_ref[e & 1] == -INFINITY ? 0.f : S.m_ref[e & 1];
    p[e] = fast_exp2(fmaf(s[e], c, -m));
  }
  S.l_run[0] += p[0] + p[2];
  S.l_run[1] += p[1] + p[3];
  // The weights of tokens fg and fg + 8 (rows 2ft, 2ft + 1) as hi + lo bf16
  // terms, transposed into P^T fragments (tokens 2ft, 2ft + 1 of row fg)
  const uint32_t h0 = pack_bf16x2(p[0], p[1]), h1 = pack_bf16x2(p[2], p[3]);
  const uint32_t l0 = pack_bf16x2(p[0] - __uint_as_float(h0 << 16),
                                  p[1] - __uint_as_float(h0 & 0xFFFF0000u));
  const uint32_t l1 = pack_bf16x2(p[2] - __uint_as_float(h1 << 16),
                                  p[3] - __uint_as_float(h1 & 0xFFFF0000u));
  const uint32_t th0 = transpose8x8(h0), th1 = transpose8x8(h1);
  const uint32_t tl0 = transpose8x8(l0), tl1 = transpose8x8(l1);
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) mma_16816_bf16(S.oacc[mt], va[mt], th0, th1);
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) mma_16816_bf16(S.oacc[mt], va[mt], tl0, tl1);
}

// Place of query row r of (sequence, kv head) among the partials.
__device__ __forceinline__ int64_t part_row(int b, int g, int r) {
  return (static_cast<int64_t>(b) * kNumKvHeads + g) * kRows + r;
}

// kBeside: launched right after the tcgen05 kernel of the same call, whose
// CTAs let this grid start only after their own wait for the prior grids and
// write other rows: this grid starts at once.  Its first CTA waits for that one
// before it ends, and so do the CTAs without a short chunk, so this grid ends
// last and what follows sees both.  A CTA that has streamed ends at once and
// leaves its place to the next (509 tokens beside 63 single ones: 44.6 us, with
// every CTA waiting 47.7; 2 x 400 beside 40 of 4000: 84 and 97).  CTAs without
// a chunk that do not wait either let later grids in under the last items: 2 x
// 4096 over 8192 356.9 us against 354.7, 10 x 100 beside 64 of 4000 133 against
// 129.
template <bool kBeside, int kStages>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(kStages))
    paged_short_chunk_kernel(const __grid_constant__ CUtensorMap pool_map, const MaskedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.x % kNumKvHeads, split = blockIdx.x / kNumKvHeads, b = blockIdx.y;
  const uint32_t bar0 = smem_addr(smem + ring_bytes(kStages)) + warp * kStages * 8;
  const uint32_t tile0 = smem_addr(smem) + warp * kStages * kTileBytes;
  if (tid == 0) tma_prefetch_desc(&pool_map);
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_barrier_init();
  }
  __syncwarp();
  if constexpr (!kBeside) wait_for_prior_grids();
  allow_dependent_grids();

  const int o0 = a.token_offsets[b], o1 = a.token_offsets[b + 1];
  const bool bad_offsets = o0 < 0 || o1 < o0 || o1 > a.num_tokens;
  if (bad_offsets && !kBeside && tid == 0) record_error(a.dev_err, kErrOffsets);
  if (bad_offsets || o1 == o0 || o1 - o0 > kShortTokens) {
    if constexpr (kBeside) wait_for_prior_grids();
    return;
  }
  const int n = o1 - o0, tiles = (n + 1) >> 1;
  const int Lmax = a.max_blocks * kPageSize;
  int L = a.seq_lens[b];
  if (L < 0 || L > Lmax) {
    if (tid == 0) record_error(a.dev_err, kErrSeqLen);
    L = L < 0 ? 0 : Lmax;
  }
  const int pos0 = L - n;
  if (pos0 < 0 && tid == 0) record_error(a.dev_err, kErrPosition);
  // pages that some row sees: those of the sinks, then those of the windows
  const int p_first = max(pos0, 0);
  const int lo = p_first >= a.window ? p_first - a.window + 1 : 0;
  const int w0 = lo / kPageSize;
  const int ns = min((min(a.sinks, lo) + kPageSize - 1) / kPageSize, w0);
  const int pages = L > 0 ? ns + (L + kPageSize - 1) / kPageSize - w0 : 0;
  const int r0 = static_cast<int>(static_cast<int64_t>(pages) * split / a.short_splits);
  const int r1 = static_cast<int>(static_cast<int64_t>(pages) * (split + 1) / a.short_splits);
  const int nw = r1 - r0 > warp ? (r1 - r0 - warp + kWarps - 1) / kWarps : 0;  // this warp's
  auto page_of = [&](int k) {
    const int i = r0 + warp + kWarps * k;
    return i < ns ? i : w0 + (i - ns);
  };
  // tokens of a page that position p sees
  auto seen_by = [&](int base, int p) {
    auto below = [](int64_t x) {
      return x <= 0 ? 0u : (x >= kPageSize ? 0xFFFFu : (1u << static_cast<int>(x)) - 1u);
    };
    return below(static_cast<int64_t>(p) + 1 - base) &
           ((0xFFFFu & ~below(static_cast<int64_t>(p) - a.window + 1 - base)) |
            below(static_cast<int64_t>(a.sinks) - base));
  };

  // lane l: id of the warp's page 32 i + l, of this block of 32 and the next
  auto load_ids = [&](int k0) {
    int pid = -1;
    if (k0 + lane < nw) {
      pid = a.block_table[static_cast<int64_t>(b) * a.max_blocks + page_of(k0 + lane)];
      if (pid < 0 || pid >= a.num_pages) {
        record_error(a.dev_err, kErrPage);
        pid = -1;
      }
    }
    return pid;
  };
  int ids = load_ids(0), ids_next = load_ids(32);
  const uint64_t policy = l2_policy_evict_first();
  auto issue = [&](int k, int pid) {  // lane 0
    const uint32_t bar = bar0 + 8 * (k % kStages);
    if (pid >= 0) {
      mbar_arrive_expect_tx(bar, kTileBytes);
      tma_load_3d(tile0 + (k % kStages) * kTileBytes, &pool_map, bar, g * kHeadDim, 0, pid, policy);
    } else {
      mbar_arrive(bar);  // keep the stage's phase sequence in step
    }
  };
  for (int k = 0; k < kStages && k < nw; ++k) {
    const int pid = __shfl_sync(kFullMask, ids, k);
    if (lane == 0) issue(k, pid);
  }

  const LaneGeom G(lane);
  // Q^T fragments of the n-tiles: column fg is query row 8 i + fg (rows of no
  // token: zeros)
  uint32_t qb[kTiles][4][2];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    const int tok = 2 * i + (G.fg >> 2);
    const uint32_t* qw = reinterpret_cast<const uint32_t*>(
        a.q + (static_cast<int64_t>(o0 + tok) * kNumQHeads + g * kGroup + (G.fg & 3)) * kHeadDim);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      qb[i][kk][0] = tok < n ? qw[kk * 8 + G.ft] : 0u;
      qb[i][kk][1] = tok < n ? qw[kk * 8 + 4 + G.ft] : 0u;
    }
  }
  const float c = a.scale_log2;
  TileState S[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    S[i].m_ref[0] = S[i].m_ref[1] = -INFINITY;
    S[i].l_run[0] = S[i].l_run[1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[i].oacc[mt][e] = 0.f;
  }
  bool nonfinite = false;  // a V value that some row sees was replaced
  const int last_lo = max(L - 1, 0) >= a.window ? L - a.window : 0;  // of the last row's window
  for (int k = 0; k < nw; ++k) {
    const int st = k % kStages;
    const bool there = mbar_wait_bounded(bar0 + 8 * st, (k / kStages) & 1, a.wait_ns);
    if (!__all_sync(kFullMask, there)) {
      // give up, but not before this warp's copies have landed (full limit)
      if (lane == 0) {
        record_error(a.dev_err, kErrTimeout);
        for (int j = k; j < k + kStages && j < nw; ++j)
          mbar_wait_bounded(bar0 + 8 * (j % kStages), (j / kStages) & 1);
      }
      __syncwarp();
      break;
    }
    if (__shfl_sync(kFullMask, ids, k & 31) >= 0) {
      const uint32_t kt = tile0 + st * kTileBytes, vt = kt + kPageSize * kRowBytes;
      const int base = page_of(k) * kPageSize;
      // every row sees the whole page?
      const bool whole = base + kPageSize - 1 <= pos0 &&
                         (base >= last_lo || base + kPageSize <= a.sinks);
      uint32_t ka[4][4];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        ldsm_x4(kt + G.k_row + (static_cast<uint32_t>((2 * kk + G.k_chunk) ^ G.lr) << 4), ka[kk]);
      float s[kTiles][4];
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
        if (i < tiles) {
          s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_16816_bf16(s[i], ka[kk], qb[i][kk][0], qb[i][kk][1]);
        }
      if (!whole) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          // this lane's two rows are of one token
          const uint32_t vis = seen_by(base, pos0 + 2 * i + (G.ft >> 1));
          if (!((vis >> G.fg) & 1u)) s[i][0] = s[i][1] = -INFINITY;
          if (!((vis >> (G.fg + 8)) & 1u)) s[i][2] = s[i][3] = -INFINITY;
        }
        for (int j = lane; j < kPageSize * 8; j += 32) {
          const uint32_t at = vt + (j >> 3) * kRowBytes + ((j & 7) << 4);
          const uint4 v = lds128(at);
          const uint32_t m0 = nonfinite_halves(v.x), m1 = nonfinite_halves(v.y),
                         m2 = nonfinite_halves(v.z), m3 = nonfinite_halves(v.w);
          if ((m0 | m1 | m2 | m3) != 0u) {
            if (base + (j >> 3) < L) nonfinite = true;
            sts128(at, v.x & ~m0, v.y & ~m1, v.z & ~m2, v.w & ~m3);
          }
        }
        __syncwarp();
      }
      uint32_t va[4][4];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
        ldsm_x4_trans(vt + G.v_row + (static_cast<uint32_t>((2 * mt + G.v_chunk) ^ G.lr) << 4),
                      va[mt]);
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
        if (i < tiles) fold_tile(s[i], va, c, S[i]);
    }
    __syncwarp();
    // refill the stage with the page kStages ahead
    const int kn = k + kStages;
    const int pid = __shfl_sync(kFullMask, (kn & ~31) == (k & ~31) ? ids : ids_next, kn & 31);
    if (lane == 0 && kn < nw) {
      fence_proxy_async_smem();
      issue(kn, pid);
    }
    if ((k & 31) == 31) {
      ids = ids_next;
      ids_next = load_ids((k & ~31) + 64);
    }
  }

  // ---- the warps' states through shared memory
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int x = 4; x <= 16; x <<= 1) {
      S[i].l_run[0] += __shfl_xor_sync(kFullMask, S[i].l_run[0], x);
      S[i].l_run[1] += __shfl_xor_sync(kFullMask, S[i].l_run[1], x);
    }
  const bool any_nonfinite = __syncthreads_or(nonfinite) != 0;  // every warp is done with its ring
  float* sm_m = reinterpret_cast<float*>(smem);
  float* sm_l = sm_m + kWarps * kRows;
  float* sm_o = sm_l + kWarps * kRows;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    const int r = warp * kRows + 8 * i + 2 * G.ft;
    if (G.fg == 0) {
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        sm_m[r + rr] = S[i].m_ref[rr];
        sm_l[r + rr] = S[i].l_run[rr];
      }
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      float* op = sm_o + r * kHeadDim + 16 * mt + G.fg;
      op[0] = S[i].oacc[mt][0];
      op[kHeadDim] = S[i].oacc[mt][1];
      op[8] = S[i].oacc[mt][2];
      op[kHeadDim + 8] = S[i].oacc[mt][3];
    }
  }
  __syncthreads();
  for (int r = warp; r < n * kGroup; r += kWarps) {
    float M = -INFINITY;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) M = fmaxf(M, sm_m[x * kRows + r]);
    float Ls = 0.f;
    float2 O = make_float2(0.f, 0.f);
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      const float ms = sm_m[x * kRows + r], ls = sm_l[x * kRows + r];
      if (ls == 0.f) continue;  // saw no token
      const float wt = ms == -INFINITY ? 1.f : fast_exp2(ms - M);  // (-inf: a NaN row)
      Ls += ls * wt;
      const float2 os =
          *reinterpret_cast<const float2*>(sm_o + (x * kRows + r) * kHeadDim + 2 * lane);
      O.x = fmaf(wt, os.x, O.x);
      O.y = fmaf(wt, os.y, O.y);
    }
    // seen values that are not finite: some were replaced, or a product with
    // them is NaN (a row whose sum is stays so)
    if (any_nonfinite || __any_sync(kFullMask, (O.x != O.x || O.y != O.y) && Ls == Ls))
      set_nonfinite(
          O, a.pool, a.num_pages, a.block_table + static_cast<int64_t>(b) * a.max_blocks, g, lane,
          r0, r1, [&](int i) { return i < ns ? i : w0 + (i - ns); },
          [&](int page) { return seen_by(page * kPageSize, pos0 + r / kGroup); });
    const int64_t row =
        static_cast<int64_t>(o0 + r / kGroup) * kNumQHeads + g * kGroup + r % kGroup;
    if (a.short_splits > 1) {
      const int64_t part = part_row(b, g, r) * a.short_splits + split;
      *reinterpret_cast<float2*>(a.short_acc + part * kHeadDim + 2 * lane) = O;
      if (lane == 0) *reinterpret_cast<float2*>(a.short_ml + 2 * part) = make_float2(M, Ls);
    } else {
      const float inv = Ls > 0.f || Ls != Ls ? 1.f / Ls : 0.f;
      reinterpret_cast<uint32_t*>(a.out + row * kHeadDim)[lane] =
          pack_bf16x2(O.x * inv, O.y * inv);
    }
  }
  if (kBeside && blockIdx.x == 0 && blockIdx.y == 0) wait_for_prior_grids();
}

// grid (kv heads x tokens, batch): combine the ranges of a short chunk's rows,
// added in order; a warp to a row, lane l holding dims 2l and 2l + 1, with the
// loads of eight ranges in flight.  (Every step of the sum is an L2 latency:
// with four warps for all rows of a kv head, 4 tokens over 2048 took 39 us,
// this way 14 us.)
__global__ void __launch_bounds__(32 * kGroup) merge_short_kernel(const MaskedArgs a) {
  allow_dependent_grids();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31, g = blockIdx.x % kNumKvHeads, b = blockIdx.y;
  const int r = blockIdx.x / kNumKvHeads * kGroup + (threadIdx.x >> 5);
  const int o0 = a.token_offsets[b], o1 = a.token_offsets[b + 1];
  if (o0 < 0 || o1 > a.num_tokens || o1 <= o0 || o1 - o0 > kShortTokens) return;
  if (r >= (o1 - o0) * kGroup) return;
  const int64_t first = part_row(b, g, r) * a.short_splits;
  const float2* ml = reinterpret_cast<const float2*>(a.short_ml) + first;
  const float2* acc = reinterpret_cast<const float2*>(a.short_acc) + first * (kHeadDim / 2) + lane;
  const int64_t row = static_cast<int64_t>(o0 + r / kGroup) * kNumQHeads + g * kGroup + r % kGroup;
  reinterpret_cast<uint32_t*>(a.out + row * kHeadDim)[lane] =
      merge_ranges(ml, acc, a.short_splits, lane);
}

template <bool kBeside, int kStages>
cudaError_t launch(const CUtensorMap& pool_map, const MaskedArgs& args, cudaStream_t stream) {
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  static std::atomic<unsigned long long> done{0};
  const unsigned long long bit = 1ull << (device & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    err = cudaFuncSetAttribute(paged_short_chunk_kernel<kBeside, kStages>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(smem_bytes(kStages)));
    if (err != cudaSuccess) return err;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  return launch_pdl(paged_short_chunk_kernel<kBeside, kStages>,
                    dim3(kNumKvHeads * args.short_splits, args.batch), dim3(kThreads),
                    smem_bytes(kStages),
                    stream, pool_map, args);
}

}  // namespace

cudaError_t launch_short_chunks(const CUtensorMap& pool_map, const MaskedArgs& args, bool beside,
                                cudaStream_t stream) {
  const bool all_short = args.num_tokens <= static_cast<int64_t>(kShortTokens) * args.batch;
  const cudaError_t err =
      all_short ? (beside ? launch<true, kShallow>(pool_map, args, stream)
                          : launch<false, kShallow>(pool_map, args, stream))
                : launch<true, kDeep>(pool_map, args, stream);
  if (err != cudaSuccess || args.short_splits == 1) return err;
  return launch_pdl(merge_short_kernel, dim3(kNumKvHeads * kShortTokens, args.batch),
                    dim3(32 * kGroup), 0, stream, args);
}

}  // namespace pkv
