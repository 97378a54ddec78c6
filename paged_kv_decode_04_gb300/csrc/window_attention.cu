// window_attention.cu -- one-token attention over the paged cache that sees a
// sliding window and sink tokens only, or that adds every token's weight to
// a running mass.
//
// The query of sequence b stands at position L - 1 and sees token t when
// t < L and (t >= L - window or t < sinks).  The pages that hold such tokens
// form a list, sink pages first, then the window's; one CTA per (sequence,
// kv head, range of that list), 4 warps taking every 4th page of the range
// through a private ring of 4 KiB tiles (16 K rows, 16 V rows) filled by TMA,
// with the per-page tensor-core math of decode_page.cuh.  Masked tokens of
// the list's ragged pages lose their score, and their V rows are zeroed in
// shared memory.  The page ids of a warp's next 32 pages sit in its lanes.
//
// Weights (kScored): w_{j,t} = 2^(s_{j,t} - M_j) / l_j needs the row's final
// maximum and sum, so the page loop keeps the scores, 4 floats a token: in
// shared memory when one CTA has the whole list and it fits, else in the
// workspace; a last pass over them turns them into weights and adds the sum
// over the 4 query rows to mass.  One thread adds each token's, so there are
// no atomics and the same inputs give the same bits.  The scores of a page that
// was not read (bad id, wait run out) are a NaN of their own, and its tokens'
// mass is stored as it was loaded: adding 0 would not do, since 0 x NaN (a row
// with a NaN key) is NaN.  (A store under the condition instead keeps loads
// from being gathered: 128 sequences of 2048 took 75.9 us, this way 73.2.)
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "decode_page.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "visible.cuh"

namespace pkv {

namespace {

// Warps of a CTA, tiles in flight per warp and CTAs per SM of the instances.
// The scores of 2048 tokens take 32 KiB, so with weights two CTAs share an SM,
// and eight warps each with rings of two keep as many bytes in flight as four
// CTAs of four warps do without: 128 sequences of 2048 took 72.7 us (5.8 TB/s),
// with four warps and rings of four 80.5 us, with one CTA of eight warps and
// rings of three 85 us, with the scores in the workspace and three CTAs 86 us.
// Without weights 256 sequences of 1004 visible tokens took 86.5 us (6.1 TB/s,
// 90 % of the measured copy rate), with three CTAs of rings of four 87.4 us.
template <bool kScored>
struct Shape {
  static constexpr int kWarps = kScored ? 8 : 4;
  static constexpr int kStages = kScored ? 2 : 3;
  static constexpr int kCtas = kScored ? 2 : 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRingBytes = kWarps * kStages * kTileBytes;
};
constexpr int kMergeThreads = 32 * kGroup;  // one warp per query row of a kv head
constexpr int kPageScoreBytes = kPageSize * kGroup * 4;
constexpr int kMassTokens = 1024;  // tokens of one CTA of merge_scored_kernel
constexpr uint32_t kNotRead = 0xFFC0DEADu;  // (products give the NaN 0x7FFFFFFF)

template <bool kScored>
constexpr size_t win_smem(int score_pages) {
  using Sh = Shape<kScored>;
  static_assert(Sh::kWarps * (2 * kGroup + kGroup * kHeadDim) * 4 <= Sh::kRingBytes,
                "end-of-CTA merge scratch must fit in the ring");
  static_assert(Sh::kWarps >= kGroup, "a warp for each query row");
  return 1024 /* alignment slack */ + Sh::kRingBytes + 8 * Sh::kWarps * Sh::kStages +
         static_cast<size_t>(score_pages) * kPageScoreBytes;
}

// Shared memory of an SM, a KiB of it taken by each CTA.
constexpr size_t kSmemOfSm = 228 * 1024;
static_assert(Shape<true>::kCtas * (win_smem<true>(kScoredSmemPages) + 1024) <= kSmemOfSm,
              "the scores kept in shared memory leave room for every CTA of an SM");

template <bool kScored>
__global__ void __launch_bounds__(Shape<kScored>::kThreads, Shape<kScored>::kCtas)
    paged_window_kernel(const __grid_constant__ CUtensorMap pool_map, const MaskedArgs a) {
  constexpr int kWarps = Shape<kScored>::kWarps, kStages = Shape<kScored>::kStages;
  constexpr int kThreads = Shape<kScored>::kThreads, kRingBytes = Shape<kScored>::kRingBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.x % kNumKvHeads, split = blockIdx.x / kNumKvHeads, b = blockIdx.y;
  const uint32_t bar0 = smem_addr(smem + kRingBytes) + warp * kStages * 8;
  const uint32_t tile0 = smem_addr(smem) + warp * kStages * kTileBytes;
  if (tid == 0) tma_prefetch_desc(&pool_map);
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_barrier_init();
  }
  __syncwarp();
  wait_for_prior_grids();
  allow_dependent_grids();

  const Visible V(clamped_len(a, b, tid == 0 && blockIdx.x == 0), a.window, a.sinks);
  const int r0 = static_cast<int>(static_cast<int64_t>(V.n) * split / a.num_splits);
  const int r1 = static_cast<int>(static_cast<int64_t>(V.n) * (split + 1) / a.num_splits);
  const int nw = r1 - r0 > warp ? (r1 - r0 - warp + kWarps - 1) / kWarps : 0;  // this warp's pages

  // lane l: id of the warp's page 32 i + l, of this block of 32 and the next
  auto page_of = [&](int k) { return V.page(r0 + warp + kWarps * k); };
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
  uint32_t qb[4][2];
  load_q_frags(a.q + (static_cast<int64_t>(b) * kNumQHeads + g * kGroup) * kHeadDim, G, qb);
  const float c = a.scale_log2;
  // scores of token t and row r at 4 t + r: of the range's pages in shared
  // memory, or of the sequence in the workspace
  float* scores = nullptr;
  if constexpr (kScored)
    scores = a.scores == nullptr
                 ? reinterpret_cast<float*>(smem + kRingBytes + 8 * kWarps * kStages)
                 : a.scores + (static_cast<int64_t>(b) * kNumKvHeads + g) * a.max_blocks *
                                  (kPageSize * kGroup);

  auto keep_scores = [&](int page, const float (&s)[4]) {
    // (the pages of a weighted call's list are the sequence's: no window)
    if (G.ft >= 2) return;
    float* sp = scores + static_cast<int64_t>(a.scores == nullptr ? page - r0 : page) *
                             (kPageSize * kGroup) + 2 * G.ft;
    *reinterpret_cast<float2*>(sp + G.fg * kGroup) = make_float2(s[0], s[1]);
    *reinterpret_cast<float2*>(sp + (G.fg + 8) * kGroup) = make_float2(s[2], s[3]);
  };

  AttnState S;
  S.reset();
  for (int k = 0; k < nw; ++k) {
    const int st = k % kStages;
    const bool ready = mbar_wait_bounded(bar0 + 8 * st, (k / kStages) & 1, a.wait_ns);
    if (!__all_sync(kFullMask, ready)) {
      // give up, but not before this warp's copies have landed (full limit)
      if (lane == 0) {
        record_error(a.dev_err, kErrTimeout);
        for (int j = k; j < k + kStages && j < nw; ++j)
          mbar_wait_bounded(bar0 + 8 * (j % kStages), (j / kStages) & 1);
      }
      __syncwarp();
      if constexpr (kScored) {
        const float x = __uint_as_float(kNotRead);
        const float none[4] = {x, x, x, x};
        for (int j = k; j < nw; ++j) keep_scores(page_of(j), none);
      }
      break;
    }
    const int page = page_of(k);
    const bool live = __shfl_sync(kFullMask, ids, k & 31) >= 0;
    float s[4];
    if (live) {
      const uint32_t kt = tile0 + st * kTileBytes;
      page_scores(kt, qb, G, s);
      const uint32_t vis = V.mask(page);
      if (vis != 0xFFFFu) {
        if (!((vis >> G.fg) & 1u)) s[0] = s[1] = -INFINITY;
        if (!((vis >> (G.fg + 8)) & 1u)) s[2] = s[3] = -INFINITY;
        for (int i = lane; i < kPageSize * 8; i += 32)
          if (!((vis >> (i >> 3)) & 1u))
            sts128_zero(kt + (kPageSize + (i >> 3)) * kRowBytes + ((i & 7) << 4));
        __syncwarp();
      }
      fold_page(kt, s, c, G, S);
    } else {
      s[0] = s[1] = s[2] = s[3] = __uint_as_float(kNotRead);
    }
    if constexpr (kScored) keep_scores(page, s);
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
  reduce_row_sums(S);
  __syncthreads();  // every warp is done with its ring
  float* sm_m = reinterpret_cast<float*>(smem);
  float* sm_l = sm_m + kWarps * kGroup;
  float* sm_o = sm_l + kWarps * kGroup;
  if (G.ft < 2) {
    if (G.fg == 0) {
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        sm_m[warp * kGroup + 2 * G.ft + rr] = S.m_ref[rr];
        sm_l[warp * kGroup + 2 * G.ft + rr] = S.l_run[rr];
      }
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      float* o0 = sm_o + (warp * kGroup + 2 * G.ft) * kHeadDim + 16 * mt + G.fg;
      o0[0] = S.oacc[mt][0];
      o0[kHeadDim] = S.oacc[mt][1];
      o0[8] = S.oacc[mt][2];
      o0[kHeadDim + 8] = S.oacc[mt][3];
    }
  }
  __syncthreads();

  const int r = warp;  // the first 4 warps <-> 4 query rows
  float M = -INFINITY, inv = 0.f;
  if (r < kGroup) {
#pragma unroll
    for (int x = 0; x < kWarps; ++x) M = fmaxf(M, sm_m[x * kGroup + r]);
    float Ls = 0.f;
    float2 O = make_float2(0.f, 0.f);
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      const float ms = sm_m[x * kGroup + r];
      const float ls = sm_l[x * kGroup + r];
      if (ls == 0.f) continue;  // saw no token
      const float wt = ms == -INFINITY ? 1.f : fast_exp2(ms - M);  // (-inf: a NaN row)
      Ls += ls * wt;
      const float2 os =
          *reinterpret_cast<const float2*>(sm_o + (x * kGroup + r) * kHeadDim + 2 * lane);
      O.x = fmaf(wt, os.x, O.x);
      O.y = fmaf(wt, os.y, O.y);
    }
    // seen values that are not finite (a row whose sum is NaN stays so)
    if (__any_sync(kFullMask, (O.x != O.x || O.y != O.y) && Ls == Ls))
      set_nonfinite(
          O, a.pool, a.num_pages, a.block_table + static_cast<int64_t>(b) * a.max_blocks, g, lane,
          r0, r1, [&](int i) { return V.page(i); }, [&](int page) { return V.mask(page); });
    const int64_t row = static_cast<int64_t>(b) * kNumQHeads + g * kGroup + r;
    if (a.num_splits > 1) {
      const int64_t part = row * a.num_splits + split;
      *reinterpret_cast<float2*>(a.part_acc + part * kHeadDim + 2 * lane) = O;
      if (lane == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * part) = make_float2(M, Ls);
    } else {
      inv = Ls > 0.f || Ls != Ls ? 1.f / Ls : 0.f;
      reinterpret_cast<uint32_t*>(a.out + row * kHeadDim)[lane] = pack_bf16x2(O.x * inv, O.y * inv);
    }
  }
  if (a.num_splits > 1) return;
  if constexpr (kScored) {
    __syncthreads();  // the states have been read
    if (lane == 0 && r < kGroup) {
      sm_m[r] = M == -INFINITY ? 0.f : M;
      sm_l[r] = inv;
    }
    __syncthreads();
    const float4 Ms = *reinterpret_cast<const float4*>(sm_m);
    const float4 Is = make_float4(sm_l[0], sm_l[1], sm_l[2], sm_l[3]);
    float* mass = a.mass + (static_cast<int64_t>(b) * kNumKvHeads + g) * a.mass_stride;
    for (int t = tid; t < V.L; t += kThreads) {
      const float4 x = reinterpret_cast<const float4*>(scores)[t];
      const float old = mass[t];
      const float m =
          old +
          ((fast_exp2(fmaf(x.x, c, -Ms.x)) * Is.x + fast_exp2(fmaf(x.y, c, -Ms.y)) * Is.y) +
           (fast_exp2(fmaf(x.z, c, -Ms.z)) * Is.z + fast_exp2(fmaf(x.w, c, -Ms.w)) * Is.w));
      mass[t] = __float_as_uint(x.x) != kNotRead ? m : old;
    }
  }
}

// Maximum and sum of a row over its ranges: the same in every lane.
__device__ __forceinline__ float2 row_stats(const MaskedArgs& a, int64_t row, int lane) {
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + row * a.num_splits;
  float M = -INFINITY, L = 0.f;
  for (int s = lane; s < a.num_splits; s += 32) {
    const float2 x = __ldcg(ml + s);
    if (x.y != 0.f) M = fmaxf(M, x.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
  for (int s = lane; s < a.num_splits; s += 32) {
    const float2 x = __ldcg(ml + s);
    if (x.y != 0.f) L += x.y * (x.x == -INFINITY ? 1.f : fast_exp2(x.x - M));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(kFullMask, L, o);
  return make_float2(M, L);
}

// Combine a row's ranges, added in order: lane l holds dims 2l and 2l + 1.
__device__ __forceinline__ void merge_out(const MaskedArgs& a, int64_t row, float2 st, int lane) {
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + row * a.num_splits;
  const float2* acc =
      reinterpret_cast<const float2*>(a.part_acc) + row * a.num_splits * (kHeadDim / 2) + lane;
  float2 O = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < a.num_splits; ++s) {
    const float2 x = __ldcg(ml + s);
    const float2 v = __ldcg(acc + static_cast<int64_t>(s) * (kHeadDim / 2));
    const float wt = x.y == 0.f ? 0.f : x.x == -INFINITY ? 1.f : fast_exp2(x.x - st.x);
    if (x.y != 0.f) {
      O.x = fmaf(v.x, wt, O.x);
      O.y = fmaf(v.y, wt, O.y);
    }
  }
  const float inv = st.y > 0.f || st.y != st.y ? 1.f / st.y : 0.f;
  reinterpret_cast<uint32_t*>(a.out + row * kHeadDim)[lane] = pack_bf16x2(O.x * inv, O.y * inv);
}

// grid (8 kv heads, batch), one warp per query row of the head.
__global__ void __launch_bounds__(kMergeThreads) merge_window_kernel(const MaskedArgs a) {
  allow_dependent_grids();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.y) * kNumQHeads + blockIdx.x * kGroup +
                      (threadIdx.x >> 5);
  merge_out(a, row, row_stats(a, row, lane), lane);
}

// grid (8 kv heads x pieces of kMassTokens tokens, batch): every piece works
// out the rows' statistics, the first writes the output, and each adds its
// tokens' weights.
__global__ void __launch_bounds__(kMergeThreads) merge_scored_kernel(const MaskedArgs a) {
  __shared__ float s_m[kGroup], s_inv[kGroup];
  allow_dependent_grids();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int g = blockIdx.x % kNumKvHeads, piece = blockIdx.x / kNumKvHeads, b = blockIdx.y;
  const int L = clamped_len(a, b, false);
  if (piece > 0 && piece * kMassTokens >= L) return;
  const int64_t row = static_cast<int64_t>(b) * kNumQHeads + g * kGroup + r;
  const float2 st = row_stats(a, row, lane);
  if (lane == 0) {
    s_m[r] = st.x == -INFINITY ? 0.f : st.x;
    s_inv[r] = st.y > 0.f || st.y != st.y ? 1.f / st.y : 0.f;
  }
  __syncthreads();
  const int64_t bg = static_cast<int64_t>(b) * kNumKvHeads + g;
  const float4* scores =
      reinterpret_cast<const float4*>(a.scores) + bg * a.max_blocks * kPageSize;
  float* mass = a.mass + bg * a.mass_stride;
  const float c = a.scale_log2;
  const int end = min(L, (piece + 1) * kMassTokens);
  for (int t = piece * kMassTokens + threadIdx.x; t < end; t += kMergeThreads) {
    const float4 x = __ldcg(scores + t);
    const float old = mass[t];
    const float m = old + ((fast_exp2(fmaf(x.x, c, -s_m[0])) * s_inv[0] +
                            fast_exp2(fmaf(x.y, c, -s_m[1])) * s_inv[1]) +
                           (fast_exp2(fmaf(x.z, c, -s_m[2])) * s_inv[2] +
                            fast_exp2(fmaf(x.w, c, -s_m[3])) * s_inv[3]));
    mass[t] = __float_as_uint(x.x) != kNotRead ? m : old;
  }
  if (piece == 0) merge_out(a, row, st, lane);
}

template <bool kScored>
cudaError_t configure(int device) {
  static std::atomic<unsigned long long> done{0};
  const unsigned long long bit = 1ull << (device & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t err = cudaFuncSetAttribute(
      paged_window_kernel<kScored>, cudaFuncAttributeMaxDynamicSharedMemorySize,
      static_cast<int>(win_smem<kScored>(kScored ? kScoredSmemPages : 0)));
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return err;
}

}  // namespace

cudaError_t launch_window_attention(const CUtensorMap& pool_map, const MaskedArgs& args,
                                    int score_pages, cudaStream_t stream) {
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  const bool scored = args.mass != nullptr;
  err = scored ? configure<true>(device) : configure<false>(device);
  if (err != cudaSuccess) return err;
  const dim3 grid(kNumKvHeads * args.num_splits, args.batch);
  err = scored ? launch_pdl(paged_window_kernel<true>, grid, dim3(Shape<true>::kThreads),
                            win_smem<true>(score_pages), stream, pool_map, args)
               : launch_pdl(paged_window_kernel<false>, grid, dim3(Shape<false>::kThreads),
                            win_smem<false>(0), stream, pool_map, args);
  if (err != cudaSuccess || args.num_splits == 1) return err;
  if (!scored)
    return launch_pdl(merge_window_kernel, dim3(kNumKvHeads, args.batch), dim3(kMergeThreads), 0,
                      stream, args);
  const int pieces = (args.max_blocks * kPageSize + kMassTokens - 1) / kMassTokens;
  return launch_pdl(merge_scored_kernel, dim3(kNumKvHeads * pieces, args.batch), dim3(kMergeThreads),
                    0, stream, args);
}

}  // namespace pkv
