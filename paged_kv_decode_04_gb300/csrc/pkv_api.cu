// pkv_api.cu -- the extern "C" boundary of libpkv (declared in include/pkv.h):
// argument checks, the split plan, TMA descriptor encoding, and launches.
// No entry point allocates, frees or synchronizes; everything is enqueued on
// the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "pkv.h"
#include "pkv_internal.h"

using pkv::kHeadDim;
using pkv::kNumKvHeads;
using pkv::kNumQHeads;
using pkv::kPageSize;

namespace pkv {

// The calling thread's limit on each in-kernel wait (pkv_set_wait_limit_ns).
unsigned long long& t_wait_ns_ref() {
  thread_local unsigned long long ns = kDefaultWaitNs;
  return ns;
}

unsigned long long wait_limit_ns() { return t_wait_ns_ref(); }

}  // namespace pkv

namespace {

bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// SM count of the current device, cached per device (-1 when unavailable).
int current_sm_count() {
  static std::atomic<int> cache[64] = {};  // 0 = not queried yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  if (dev < 0 || dev >= 64) return -1;
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v > 0) return v;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  cache[dev].store(v, std::memory_order_relaxed);
  return v;
}

// Split plan: S logical page ranges of pages_per_split pages per sequence,
// one CTA each.  Explicit S is honoured (capped by the table width); S = 0
// aims for about four CTAs per SM across (sequence, kv head, range) while
// keeping at least eight pages per range (measured on one 2048-token
// sequence: 8 pages per range 114.7 us per 16 layers, 4 pages 135.9 us).
bool make_plan(int batch, int max_blocks, int num_splits, pkv::SplitPlan* plan) {
  int S;
  if (num_splits > 0) {
    S = num_splits;
  } else {
    const int sms = current_sm_count();
    if (sms <= 0) return false;
    const long long units = static_cast<long long>(batch) * kNumKvHeads;
    const long long target = 4LL * sms;
    S = static_cast<int>((target + units - 1) / units);
    const int cap = (max_blocks + 7) / 8;
    if (S > cap) S = cap;
    if (S < 1) S = 1;
  }
  if (S > max_blocks) S = max_blocks;
  int pps = (max_blocks + S - 1) / S;
  if (pps > pkv::max_pages_per_split()) pps = pkv::max_pages_per_split();
  plan->pages_per_split = pps;
  plan->num_splits = (max_blocks + pps - 1) / pps;
  return true;
}

size_t plan_workspace(int batch, const pkv::SplitPlan& plan) {
  return pkv::workspace_bytes_for(batch, kNumQHeads, kHeadDim, plan);
}

bool supported_dims(int num_q_heads, int num_kv_heads, int head_dim, int page_size) {
  return num_q_heads == kNumQHeads && num_kv_heads == kNumKvHeads &&
         head_dim == kHeadDim && page_size == kPageSize;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::atomic<EncodeTiledFn> fn{nullptr};
  EncodeTiledFn f = fn.load(std::memory_order_acquire);
  if (f == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                         cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || p == nullptr) {
      cudaGetLastError();
      return nullptr;
    }
    f = reinterpret_cast<EncodeTiledFn>(p);
    fn.store(f, std::memory_order_release);
  }
  return f;
}

// TMA descriptor of the pool viewed as [num_pages][32 rows (K|V x slot)][512]
// bf16, 128-byte swizzled, with a box of one kv head's rows of one page:
// box_rows = 32 takes its K and V rows (a 4 KiB tile), box_rows = 16 its K
// rows (row coordinate 0) or its V rows (row coordinate 16), 2 KiB each.
// Cached per thread for the last (device, pool, pages) of each box height.
bool pool_tensor_map(const void* pool, int64_t num_pages, CUtensorMap* out,
                     int box_rows = 2 * kPageSize) {
  struct Entry {
    int device = -1;
    const void* pool = nullptr;
    int64_t num_pages = 0;
    CUtensorMap map;
  };
  thread_local Entry cached[2];
  if (box_rows != kPageSize && box_rows != 2 * kPageSize) return false;
  Entry& c = cached[box_rows == kPageSize ? 1 : 0];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (c.device == dev && c.pool == pool && c.num_pages == num_pages) {
    *out = c.map;
    return true;
  }
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kNumKvHeads * kHeadDim),
                              static_cast<cuuint64_t>(2 * kPageSize),
                              static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t strides[2] = {
      static_cast<cuuint64_t>(kNumKvHeads * kHeadDim * 2),
      static_cast<cuuint64_t>(2 * kPageSize * kNumKvHeads * kHeadDim * 2)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(kHeadDim),
                             static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUtensorMap m;
  const CUresult r = enc(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(pool),
                         dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return false;
  c.device = dev;
  c.pool = pool;
  c.num_pages = num_pages;
  c.map = m;
  *out = m;
  return true;
}

// TMA descriptor of the pool as the 4-D tensor (dim 64, row 32, kv head 8,
// page) with strides (2 B, 1 KiB, 128 B, 32 KiB) and a box of one whole page:
// the box lands in shared memory as [head][32 rows][64], 128-byte swizzled,
// i.e. each head's 4 KiB tile laid out as in pool_tensor_map's box.
bool pool_page_map(const void* pool, int64_t num_pages, CUtensorMap* out) {
  struct Entry {
    int device = -1;
    const void* pool = nullptr;
    int64_t num_pages = 0;
    CUtensorMap map;
  };
  thread_local Entry cached;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (cached.device == dev && cached.pool == pool && cached.num_pages == num_pages) {
    *out = cached.map;
    return true;
  }
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kHeadDim),
                              static_cast<cuuint64_t>(2 * kPageSize),
                              static_cast<cuuint64_t>(kNumKvHeads),
                              static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t strides[3] = {
      static_cast<cuuint64_t>(kNumKvHeads * kHeadDim * 2),  // next row (slot, K|V)
      static_cast<cuuint64_t>(kHeadDim * 2),                 // next kv head
      static_cast<cuuint64_t>(2 * kPageSize * kNumKvHeads * kHeadDim * 2)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(kHeadDim),
                             static_cast<cuuint32_t>(2 * kPageSize),
                             static_cast<cuuint32_t>(kNumKvHeads), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUtensorMap m;
  const CUresult r = enc(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool),
                         dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return false;
  cached.device = dev;
  cached.pool = pool;
  cached.num_pages = num_pages;
  cached.map = m;
  *out = m;
  return true;
}

// Whole-page boxes pay off once the CTAs (one per sequence range, all heads)
// fill every SM at least once.
bool use_pagebox(long long ctas, int range_pages) {
  const int sms = current_sm_count();
  return sms > 0 && ctas >= sms && range_pages <= pkv::pagebox_max_range_pages();
}

// Launch attention (append == nullptr) or the fused step under `plan`: the
// whole-page kernel when the batch fills the SMs, else the per-(sequence,
// kv head) kernel; then the split merge.
cudaError_t launch_attention(const pkv::SplitPlan& plan, const void* pool, int64_t num_pages,
                             const pkv_bf16* q, const int32_t* block_table, int max_blocks,
                             const int32_t* seq_lens, int batch, float scale, pkv_bf16* out,
                             void* workspace, int32_t* dev_err, cudaStream_t stream,
                             const pkv::AppendArgs* append) {
  pkv::AttnArgs args = {};
  args.q = q;
  args.block_table = block_table;
  args.seq_lens = seq_lens;
  args.out = out;
  const size_t need = pkv::workspace_bytes_for(batch, kNumQHeads, kHeadDim, plan);
  float* ws = static_cast<float*>(workspace);
  const size_t acc_elems = static_cast<size_t>(batch) * kNumQHeads * plan.num_splits * kHeadDim;
  args.part_acc = need > 0 ? ws : nullptr;
  args.part_ml = need > 0 ? ws + acc_elems : nullptr;
  args.dev_err = dev_err;
  args.num_pages = num_pages;
  args.max_blocks = max_blocks;
  args.batch = batch;
  args.scale_log2 = scale * 1.4426950408889634f;
  args.plan = plan;
  args.wait_ns = pkv::wait_limit_ns();
  CUtensorMap map;
  if (use_pagebox(static_cast<long long>(batch) * plan.num_splits, plan.pages_per_split)) {
    if (!pool_page_map(pool, num_pages, &map)) return cudaErrorInvalidValue;
    const cudaError_t err =
        pkv::launch_pagebox_attention(map, args, 0, plan.pages_per_split, stream, append);
    if (err != cudaSuccess) return err;
    return pkv::launch_split_merge(args, 0, stream);
  }
  if (!pool_tensor_map(pool, num_pages, &map)) return cudaErrorInvalidValue;
  return pkv::launch_paged_decode_attention(map, args, stream, append);
}

}  // namespace

extern "C" {

PKV_API int pkv_abi_version(void) { return 1; }

PKV_API unsigned long long pkv_set_wait_limit_ns(unsigned long long ns) {
  const unsigned long long prev = pkv::t_wait_ns_ref();
  pkv::t_wait_ns_ref() = ns;
  return prev;
}

PKV_API const char* pkv_strerror(int status) {
  switch (status) {
    case PKV_OK: return "ok";
    case PKV_EINVAL: return "invalid argument (null pointer, bad size or bad scale/theta)";
    case PKV_EUNSUPPORTED: return "unsupported geometry (needs 32 q heads, 8 kv heads, head dim 64, page size 16)";
    case PKV_EWORKSPACE: return "workspace missing or smaller than pkv_workspace_bytes()";
    case PKV_ECUDA: return "CUDA runtime error (launch failed or no usable device)";
    case PKV_EALIGN: return "pointer alignment requirement violated";
    case 7: return "request rejected: its page budget exceeds the whole pool";
    case 8: return "unknown or already finished request id";
    case PKV_ESCRATCH: return "split partials would exceed the static scratch buffer (PKV_STATIC_SCRATCH_BYTES); use fewer splits";
    default: return "unknown status";
  }
}

PKV_API int pkv_plan_splits(int batch, int num_kv_heads, int max_blocks, int num_splits) {
  if (batch < 1 || max_blocks < 1 || num_splits < 0 || num_kv_heads != kNumKvHeads) return -1;
  pkv::SplitPlan plan;
  if (!make_plan(batch, max_blocks, num_splits, &plan)) return -1;
  return plan.num_splits;
}

PKV_API size_t pkv_workspace_bytes(int batch, int num_q_heads, int num_kv_heads,
                                   int head_dim, int max_blocks, int num_splits) {
  if (batch < 0 || max_blocks < 1 || num_splits < 0 ||
      !supported_dims(num_q_heads, num_kv_heads, head_dim, kPageSize))
    return static_cast<size_t>(-1);
  if (batch == 0) return 0;
  pkv::SplitPlan plan;
  if (!make_plan(batch, max_blocks, num_splits, &plan)) return static_cast<size_t>(-1);
  return plan_workspace(batch, plan);
}

PKV_API int pkv_kv_append(const pkv_bf16* k_new, const pkv_bf16* v_new, pkv_bf16* pool,
                          int64_t num_pages, const int32_t* block_table, int max_blocks,
                          const int32_t* positions, int batch, int num_kv_heads,
                          int head_dim, int page_size, double rope_theta,
                          const pkv_bf16* q_in, pkv_bf16* q_out, int num_q_heads,
                          int32_t* dev_err, pkv_stream_t stream) {
  if (!k_new || !v_new || !pool || !block_table || !positions) return PKV_EINVAL;
  if (batch < 0 || num_pages < 1 || num_pages > INT32_MAX || max_blocks < 1) return PKV_EINVAL;
  if ((q_in == nullptr) != (q_out == nullptr)) return PKV_EINVAL;
  if (!(rope_theta > 0.0) || !isfinite(rope_theta)) return PKV_EINVAL;
  if (num_kv_heads != kNumKvHeads || head_dim != kHeadDim || page_size != kPageSize)
    return PKV_EUNSUPPORTED;
  if (q_in != nullptr && num_q_heads != kNumQHeads) return PKV_EUNSUPPORTED;
  if (batch > INT32_MAX / 2) return PKV_EINVAL;
  if (!aligned(pool, 16) || !aligned(v_new, 4) || !aligned(k_new, 2) || !aligned(q_in, 2) ||
      !aligned(q_out, 2) || !aligned(dev_err, 4))
    return PKV_EALIGN;
  if (batch == 0) return PKV_OK;
  pkv::RopeFreqs freqs;
  if (pkv::prepare_rope(rope_theta, &freqs, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return PKV_ECUDA;
  const cudaError_t err = pkv::launch_kv_append(
      k_new, v_new, pool, num_pages, block_table, max_blocks, positions, nullptr, batch, freqs,
      q_in, q_out, dev_err, reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

PKV_API int pkv_kv_write_prefill(const pkv_bf16* k, const pkv_bf16* v, int num_tokens,
                                 const int32_t* token_offsets, const int32_t* start_positions,
                                 pkv_bf16* pool, int64_t num_pages, const int32_t* block_table,
                                 int max_blocks, int batch, int num_kv_heads, int head_dim,
                                 int page_size, double rope_theta, int32_t* dev_err,
                                 pkv_stream_t stream) {
  if (!k || !v || !token_offsets || !start_positions || !pool || !block_table) return PKV_EINVAL;
  if (num_tokens < 0 || batch < 1 || num_pages < 1 || num_pages > INT32_MAX || max_blocks < 1 ||
      max_blocks > (INT32_MAX / kPageSize))
    return PKV_EINVAL;
  if (!(rope_theta > 0.0) || !isfinite(rope_theta)) return PKV_EINVAL;
  if (num_kv_heads != kNumKvHeads || head_dim != kHeadDim || page_size != kPageSize)
    return PKV_EUNSUPPORTED;
  if (!aligned(pool, 16) || !aligned(v, 16) || !aligned(k, 16) || !aligned(dev_err, 4))
    return PKV_EALIGN;
  if (num_tokens == 0) return PKV_OK;
  pkv::RopeFreqs freqs;
  if (pkv::prepare_rope(rope_theta, &freqs, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return PKV_ECUDA;
  const cudaError_t err = pkv::launch_kv_write_prefill(
      k, v, num_tokens, token_offsets, start_positions, pool, num_pages, block_table, max_blocks,
      batch, freqs, dev_err, pkv::wait_limit_ns(), reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

PKV_API int pkv_paged_decode_attention(const pkv_bf16* q, const pkv_bf16* pool,
                                       int64_t num_pages, const int32_t* block_table,
                                       int max_blocks, const int32_t* seq_lens, int batch,
                                       int num_q_heads, int num_kv_heads, int head_dim,
                                       int page_size, float scale, pkv_bf16* out,
                                       void* workspace, size_t workspace_bytes,
                                       int num_splits, int32_t* dev_err,
                                       pkv_stream_t stream) {
  if (!q || !pool || !block_table || !seq_lens || !out) return PKV_EINVAL;
  if (batch < 0 || batch > 65535 || num_pages < 1 || num_pages > INT32_MAX ||
      max_blocks < 1 || max_blocks > (INT32_MAX / kPageSize) || num_splits < 0)
    return PKV_EINVAL;
  if (!(scale > 0.f) || !isfinite(scale)) return PKV_EINVAL;
  if (!supported_dims(num_q_heads, num_kv_heads, head_dim, page_size)) return PKV_EUNSUPPORTED;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 4) || !aligned(workspace, 16) ||
      !aligned(dev_err, 4))
    return PKV_EALIGN;
  if (batch == 0) return PKV_OK;
  pkv::SplitPlan plan;
  if (!make_plan(batch, max_blocks, num_splits, &plan)) return PKV_ECUDA;
  const size_t need = plan_workspace(batch, plan);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return PKV_EWORKSPACE;
  const cudaError_t err =
      launch_attention(plan, pool, num_pages, q, block_table, max_blocks, seq_lens, batch, scale,
                       out, workspace, dev_err, reinterpret_cast<cudaStream_t>(stream), nullptr);
  return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

PKV_API int pkv_decode_step(const pkv_bf16* q, const pkv_bf16* k_new, const pkv_bf16* v_new,
                            pkv_bf16* pool, int64_t num_pages, const int32_t* block_table,
                            int max_blocks, const int32_t* seq_lens, int batch, int num_q_heads,
                            int num_kv_heads, int head_dim, int page_size, double rope_theta,
                            float scale, pkv_bf16* out, void* workspace, size_t workspace_bytes,
                            int num_splits, int32_t* dev_err, pkv_stream_t stream) {
  if (!q || !k_new || !v_new || !pool || !block_table || !seq_lens || !out) return PKV_EINVAL;
  if (batch < 0 || batch > 65535 || num_pages < 1 || num_pages > INT32_MAX ||
      max_blocks < 1 || max_blocks > (INT32_MAX / kPageSize) || num_splits < 0)
    return PKV_EINVAL;
  if (!(scale > 0.f) || !isfinite(scale)) return PKV_EINVAL;
  if (!(rope_theta > 0.0) || !isfinite(rope_theta)) return PKV_EINVAL;
  if (!supported_dims(num_q_heads, num_kv_heads, head_dim, page_size)) return PKV_EUNSUPPORTED;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 4) || !aligned(workspace, 16) ||
      !aligned(dev_err, 4) || !aligned(v_new, 4) || !aligned(k_new, 2))
    return PKV_EALIGN;
  if (batch == 0) return PKV_OK;
  pkv::SplitPlan plan;
  if (!make_plan(batch, max_blocks, num_splits, &plan)) return PKV_ECUDA;
  const size_t need = plan_workspace(batch, plan);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return PKV_EWORKSPACE;
  pkv::AppendArgs app;
  app.k_new = k_new;
  app.v_new = v_new;
  app.pool = pool;
  if (pkv::prepare_rope(rope_theta, &app.freqs, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return PKV_ECUDA;
  const cudaError_t err =
      launch_attention(plan, pool, num_pages, q, block_table, max_blocks, seq_lens, batch, scale,
                       out, workspace, dev_err, reinterpret_cast<cudaStream_t>(stream), &app);
  return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Attention without a caller workspace: the split-K partials live in a fixed
// device buffer owned by the library (see pkv_paged_decode_attention_static_ws
// in pkv.h for who needs this and the rules of sharing it).

namespace {

static __device__ __align__(256) unsigned char g_static_scratch[PKV_STATIC_SCRATCH_BYTES];

// Device address of g_static_scratch, looked up once per device (with that
// device current) and cached.  In host code the symbol itself is only a
// stand-in for the device object, so its address must never be passed to a
// kernel directly.
void* static_scratch_address(int device) {
  static std::atomic<void*> cache[64] = {};
  if (device < 0 || device >= 64) return nullptr;
  void* p = cache[device].load(std::memory_order_acquire);
  if (p != nullptr) return p;
  if (cudaGetSymbolAddress(&p, g_static_scratch) != cudaSuccess || p == nullptr) {
    cudaGetLastError();
    return nullptr;
  }
  cache[device].store(p, std::memory_order_release);
  return p;
}

}  // namespace

extern "C" PKV_API int pkv_paged_decode_attention_static_ws(
    const pkv_bf16* q, const pkv_bf16* pool, int64_t num_pages, const int32_t* block_table,
    int max_blocks, const int32_t* seq_lens, int batch, int num_q_heads, int num_kv_heads,
    int head_dim, int page_size, float scale, pkv_bf16* out, int num_splits,
    int32_t* dev_err, pkv_stream_t stream) {
  if (!q || !pool || !block_table || !seq_lens || !out) return PKV_EINVAL;
  if (batch < 0 || batch > 65535 || num_pages < 1 || num_pages > INT32_MAX ||
      max_blocks < 1 || max_blocks > (INT32_MAX / kPageSize) || num_splits < 0)
    return PKV_EINVAL;
  if (!(scale > 0.f) || !isfinite(scale)) return PKV_EINVAL;
  if (!supported_dims(num_q_heads, num_kv_heads, head_dim, page_size)) return PKV_EUNSUPPORTED;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 4) || !aligned(dev_err, 4))
    return PKV_EALIGN;
  if (batch == 0) return PKV_OK;
  pkv::SplitPlan plan;
  if (!make_plan(batch, max_blocks, num_splits, &plan)) return PKV_ECUDA;
  const size_t need = plan_workspace(batch, plan);
  if (need > PKV_STATIC_SCRATCH_BYTES) return PKV_ESCRATCH;
  float* ws = nullptr;
  if (need > 0) {
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return PKV_ECUDA;
    ws = static_cast<float*>(static_scratch_address(device));
    if (ws == nullptr) return PKV_ECUDA;
  }
  const cudaError_t err =
      launch_attention(plan, pool, num_pages, q, block_table, max_blocks, seq_lens, batch, scale,
                       out, ws, dev_err, reinterpret_cast<cudaStream_t>(stream), nullptr);
  return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

// ---------------------------------------------------------------------------
// Work plans (include/pkv.h): built on the host by planner.cpp, run by the
// attention kernel's planned instances.

namespace {

struct PlanHeader {
  int32_t magic, batch, max_blocks, num_items, num_merges, num_slots, range_pages, bytes_used;
  int32_t num_shared, shared_pages, num_segs, layout;
};
static_assert(sizeof(PlanHeader) == 4 * pkv::kPlanHeaderWords, "plan header layout");

// True when every index a kernel takes from the plan's body stays inside the
// buffers it addresses: sequences in [0, batch), page ranges inside the table
// and within the page list the launch sizes (range_pages, shared_pages),
// partial slots in [0, num_slots), shared items with 1..16 members.  A plan
// from pkv_plan_build / pkv_plan_build_shared always passes; a hand-made or
// damaged one is refused before anything is launched.
bool plan_body_valid(const PlanHeader& h) {
  const int32_t* w = reinterpret_cast<const int32_t*>(&h) + pkv::kPlanHeaderWords;
  auto seq_ok = [&](int32_t b) { return b >= 0 && b < h.batch; };
  auto range_ok = [&](int32_t p, int32_t n, int32_t cap) {
    return p >= 0 && n >= 0 && n <= cap && static_cast<int64_t>(p) + n <= h.max_blocks;
  };
  const int64_t lmax = static_cast<int64_t>(h.max_blocks) * kPageSize;
  const int32_t* segs = w + static_cast<int64_t>(h.num_items) * pkv::kPlanItemWords +
                        static_cast<int64_t>(h.num_merges) * pkv::kPlanMergeWords +
                        static_cast<int64_t>(h.num_shared) * pkv::kPlanSharedWords;
  for (int i = 0; i < h.num_items; ++i, w += pkv::kPlanItemWords) {
    if (h.num_segs > 0) {
      // a segment plan: every item is a segment CTA, its segments inside the
      // section, their pages summing to the item's, at most range_pages
      if (w[0] != pkv::kPlanKindSegments || w[1] < 0 || w[2] < 1 || w[2] > pkv::kSegMax ||
          static_cast<int64_t>(w[1]) + w[2] > h.num_segs || w[3] < 0 || w[3] > h.range_pages)
        return false;
      int64_t pages = 0;
      for (int k = 0; k < w[2]; ++k) {
        const int32_t* sg = segs + static_cast<int64_t>(w[1] + k) * pkv::kPlanSegWords;
        const int64_t live = (static_cast<int64_t>(sg[1]) + kPageSize - 1) / kPageSize;
        if (!seq_ok(sg[0]) || sg[1] < 0 || sg[1] > lmax || !range_ok(sg[2], sg[3], h.range_pages) ||
            sg[2] + sg[3] > live || (sg[4] != -1 && (sg[4] < 0 || sg[4] >= h.num_slots)))
          return false;
        // partials folded into the output: slots [sg[6], sg[6] + sg[5])
        if (sg[5] < 0 || sg[7] != 0 ||
            (sg[5] == 0 ? sg[6] != 0
                        : (sg[4] != -1 || sg[6] < 0 ||
                           static_cast<int64_t>(sg[6]) + sg[5] > h.num_slots)))
          return false;
        pages += sg[3];
      }
      if (pages != w[3]) return false;
      continue;
    }
    if (w[0] == pkv::kPlanKindRange) {
      if (!seq_ok(w[4]) || !range_ok(w[2], w[3], h.range_pages)) return false;
      if (w[1] != -1 && (w[1] < 0 || w[1] >= h.num_slots)) return false;
    } else if (w[0] == pkv::kPlanKindPacked) {
      if (w[1] != -1) return false;
      for (int k = 0; k < pkv::kPlanWarps; ++k)
        if (w[4 + k] != -1 && (!seq_ok(w[4 + k]) || w[8 + k] < 0 || w[8 + k] > lmax))
          return false;
    } else {
      return false;
    }
  }
  for (int i = 0; i < h.num_merges; ++i, w += pkv::kPlanMergeWords)
    if (!seq_ok(w[0]) || w[1] < 0 || w[2] < 1 ||
        static_cast<int64_t>(w[1]) + w[2] > h.num_slots)
      return false;
  for (int i = 0; i < h.num_shared; ++i, w += pkv::kPlanSharedWords) {
    const int members = w[0];
    if (members < 1 || members > pkv::kSharedMembers || w[2] < 1 ||
        !range_ok(w[1], w[2], h.shared_pages))
      return false;
    for (int m = 0; m < members; ++m)
      if (!seq_ok(w[4 + m]) || w[4 + pkv::kSharedMembers + m] < 0 ||
          w[4 + pkv::kSharedMembers + m] >= h.num_slots)
        return false;
  }
  return true;
}

// The plan's header when it is well formed for this batch and table, else nullptr.
const PlanHeader* plan_header(const void* plan, int batch, int max_blocks) {
  if (plan == nullptr || !aligned(plan, 16)) return nullptr;
  const PlanHeader* h = static_cast<const PlanHeader*>(plan);
  if (h->magic != static_cast<int32_t>(PKV_PLAN_MAGIC) || h->batch != batch ||
      h->max_blocks != max_blocks || h->num_items < 1 || h->num_items > 65535 ||
      h->num_merges < 0 || h->num_merges > batch || h->num_slots < 0 ||
      h->range_pages < 1 || h->range_pages > 1024 || h->num_shared < 0 ||
      h->num_shared > 65535 || h->num_segs < 0 ||
      (h->num_shared > 0 && (h->shared_pages < 1 || h->shared_pages > 1024)))
    return nullptr;
  // the beside layout is for shared-prefix plans only
  if (h->layout != pkv::kPlanLayoutSequential &&
      (h->layout != pkv::kPlanLayoutBeside || h->num_shared < 1))
    return nullptr;
  // bytes_used is exactly the header and the three sections the counts imply
  const int64_t words = pkv::kPlanHeaderWords +
                        static_cast<int64_t>(h->num_items) * pkv::kPlanItemWords +
                        static_cast<int64_t>(h->num_merges) * pkv::kPlanMergeWords +
                        static_cast<int64_t>(h->num_shared) * pkv::kPlanSharedWords +
                        static_cast<int64_t>(h->num_segs) * pkv::kPlanSegWords;
  if (static_cast<int64_t>(h->bytes_used) != 4 * words) return nullptr;
  if (!plan_body_valid(*h)) return nullptr;
  return h;
}

size_t plan_slots_bytes(const PlanHeader& h) {
  return static_cast<size_t>(h.num_slots) * kNumQHeads * (kHeadDim + 2) * sizeof(float);
}

// True when every item of the plan is a range (no packed sequences).
bool plan_has_only_ranges(const PlanHeader& h) {
  const int32_t* item = reinterpret_cast<const int32_t*>(&h) + pkv::kPlanHeaderWords;
  for (int i = 0; i < h.num_items; ++i, item += pkv::kPlanItemWords)
    if (item[0] != pkv::kPlanKindRange) return false;
  return true;
}

// Launch a planned call: the whole-page kernel when the plan is all ranges
// and fills the SMs, else the per-(item, kv head) kernel; then the merge.
cudaError_t launch_planned(const PlanHeader& h, const void* pool, int64_t num_pages,
                           const pkv_bf16* q, const int32_t* block_table, int max_blocks,
                           const int32_t* seq_lens, int batch, float scale, pkv_bf16* out,
                           const void* plan_dev, void* workspace, int32_t* dev_err,
                           cudaStream_t stream, const pkv::AppendArgs* append) {
  pkv::AttnArgs args = {};
  args.q = q;
  args.block_table = block_table;
  args.seq_lens = seq_lens;
  args.out = out;
  float* ws = static_cast<float*>(workspace);
  const size_t slots = static_cast<size_t>(h.num_slots) * kNumQHeads;
  args.part_acc = h.num_slots > 0 ? ws : nullptr;
  args.part_ml = h.num_slots > 0 ? ws + slots * kHeadDim : nullptr;
  const int32_t* words = static_cast<const int32_t*>(plan_dev);
  args.plan_items = reinterpret_cast<const int4*>(words + pkv::kPlanHeaderWords);
  args.plan_merges = reinterpret_cast<const int4*>(
      words + pkv::kPlanHeaderWords + static_cast<size_t>(h.num_items) * pkv::kPlanItemWords);
  args.plan_shared = reinterpret_cast<const int4*>(
      words + pkv::kPlanHeaderWords + static_cast<size_t>(h.num_items) * pkv::kPlanItemWords +
      static_cast<size_t>(h.num_merges) * pkv::kPlanMergeWords);
  args.plan_segs = reinterpret_cast<const int4*>(
      reinterpret_cast<const int32_t*>(args.plan_shared) +
      static_cast<size_t>(h.num_shared) * pkv::kPlanSharedWords);
  args.dev_err = dev_err;
  args.num_pages = num_pages;
  args.max_blocks = max_blocks;
  args.batch = batch;
  args.scale_log2 = scale * 1.4426950408889634f;
  args.plan.num_splits = 1;
  args.plan.pages_per_split = h.range_pages;
  args.wait_ns = pkv::wait_limit_ns();
  CUtensorMap map;
  if (h.num_shared > 0) {
    // shared prefixes first: their partials join the members' own ones in
    // the merge that follows the attention kernel
    if (!pool_tensor_map(pool, num_pages, &map, kPageSize)) return cudaErrorInvalidValue;
    const cudaError_t err =
        pkv::launch_shared_prefix_attention(map, args, h.num_shared, h.shared_pages, stream,
                                            h.layout == pkv::kPlanLayoutBeside);
    if (err != cudaSuccess) return err;
  }
  if (h.num_segs > 0) {
    if (!pool_page_map(pool, num_pages, &map)) return cudaErrorInvalidValue;
    const cudaError_t err =
        pkv::launch_segments_attention(map, args, h.num_items, h.range_pages, stream, append,
                                       h.layout == pkv::kPlanLayoutBeside);
    if (err != cudaSuccess) return err;
    return pkv::launch_split_merge(args, h.num_merges, stream);
  }
  const bool beside = h.layout == pkv::kPlanLayoutBeside;
  if (!beside && use_pagebox(h.num_items, h.range_pages) && plan_has_only_ranges(h)) {
    if (!pool_page_map(pool, num_pages, &map)) return cudaErrorInvalidValue;
    const cudaError_t err = pkv::launch_pagebox_attention(map, args, h.num_items, h.range_pages,
                                                          stream, append);
    if (err != cudaSuccess) return err;
    return pkv::launch_split_merge(args, h.num_merges, stream);
  }
  if (!pool_tensor_map(pool, num_pages, &map)) return cudaErrorInvalidValue;
  return pkv::launch_planned_decode_attention(map, args, h.num_items, h.num_merges,
                                              h.range_pages, stream, append, beside);
}

}  // namespace

extern "C" {

PKV_API const char* pkv_attention_kernels(int batch, int max_blocks, int num_splits,
                                          const void* plan) {
  if (batch < 1 || max_blocks < 1 || num_splits < 0) return nullptr;
  if (plan != nullptr) {
    const PlanHeader* h = plan_header(plan, batch, max_blocks);
    if (h == nullptr) return nullptr;
    if (h->num_segs > 0) {
      if (h->num_shared > 0)
        return h->num_merges > 0
                   ? "paged_decode_shared_kernel+paged_decode_segments_kernel+merge_plan_kernel"
                   : "paged_decode_shared_kernel+paged_decode_segments_kernel";
      return h->num_merges > 0 ? "paged_decode_segments_kernel+merge_plan_kernel"
                               : "paged_decode_segments_kernel";
    }
    const bool pb = h->layout != pkv::kPlanLayoutBeside &&
                    use_pagebox(h->num_items, h->range_pages) && plan_has_only_ranges(*h);
    if (h->num_shared > 0)  // a plan with shared groups always merges
      return pb ? "paged_decode_shared_kernel+paged_decode_pagebox_kernel+merge_plan_kernel"
                : "paged_decode_shared_kernel+paged_decode_kernel+merge_plan_kernel";
    if (h->num_merges > 0)
      return pb ? "paged_decode_pagebox_kernel+merge_plan_kernel"
                : "paged_decode_kernel+merge_plan_kernel";
    return pb ? "paged_decode_pagebox_kernel" : "paged_decode_kernel";
  }
  pkv::SplitPlan p;
  if (!make_plan(batch, max_blocks, num_splits, &p)) return nullptr;
  const bool pb = use_pagebox(static_cast<long long>(batch) * p.num_splits, p.pages_per_split);
  if (p.num_splits > 1)
    return pb ? "paged_decode_pagebox_kernel+merge_splits_kernel"
              : "paged_decode_kernel+merge_splits_kernel";
  return pb ? "paged_decode_pagebox_kernel" : "paged_decode_kernel";
}

PKV_API size_t pkv_plan_bytes(int batch, int max_blocks) {
  return pkv::plan_bytes(batch, max_blocks);
}

PKV_API int pkv_plan_build(const int32_t* seq_lens_host, int batch, int max_blocks, int num_sms,
                           void* plan, size_t plan_bytes) {
  if (num_sms < 0) return PKV_EINVAL;
  if (num_sms == 0) {
    num_sms = current_sm_count();
    if (num_sms <= 0) return PKV_ECUDA;
  }
  return pkv::build_plan(seq_lens_host, batch, max_blocks, num_sms, static_cast<int32_t*>(plan),
                         plan_bytes);
}

PKV_API int pkv_plan_build_shared(const int32_t* seq_lens_host, const int32_t* block_tables_host,
                                  int batch, int max_blocks, int num_sms, int min_shared_pages,
                                  void* plan, size_t plan_bytes) {
  if (num_sms < 0) return PKV_EINVAL;
  if (num_sms == 0) {
    num_sms = current_sm_count();
    if (num_sms <= 0) return PKV_ECUDA;
  }
  return pkv::build_plan_shared(seq_lens_host, block_tables_host, batch, max_blocks, num_sms,
                                min_shared_pages, static_cast<int32_t*>(plan), plan_bytes);
}

PKV_API size_t pkv_plan_workspace_bytes(const void* plan) {
  if (plan == nullptr || !aligned(plan, 16)) return static_cast<size_t>(-1);
  const PlanHeader* h = static_cast<const PlanHeader*>(plan);
  if (h->magic != static_cast<int32_t>(PKV_PLAN_MAGIC) || h->num_slots < 0)
    return static_cast<size_t>(-1);
  return plan_slots_bytes(*h);
}

PKV_API int pkv_paged_decode_attention_planned(
    const pkv_bf16* q, const pkv_bf16* pool, int64_t num_pages, const int32_t* block_table,
    int max_blocks, const int32_t* seq_lens, int batch, int num_q_heads, int num_kv_heads,
    int head_dim, int page_size, float scale, pkv_bf16* out, const void* plan_host,
    const void* plan_dev, void* workspace, size_t workspace_bytes, int32_t* dev_err,
    pkv_stream_t stream) {
  if (!q || !pool || !block_table || !seq_lens || !out || !plan_host || !plan_dev)
    return PKV_EINVAL;
  if (batch < 1 || batch > 65535 || num_pages < 1 || num_pages > INT32_MAX || max_blocks < 1 ||
      max_blocks > (INT32_MAX / kPageSize))
    return PKV_EINVAL;
  if (!(scale > 0.f) || !isfinite(scale)) return PKV_EINVAL;
  if (!supported_dims(num_q_heads, num_kv_heads, head_dim, page_size)) return PKV_EUNSUPPORTED;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 4) || !aligned(workspace, 16) ||
      !aligned(dev_err, 4) || !aligned(plan_dev, 16) || !aligned(plan_host, 16))
    return PKV_EALIGN;
  const PlanHeader* h = plan_header(plan_host, batch, max_blocks);
  if (h == nullptr) return PKV_EINVAL;
  const size_t need = plan_slots_bytes(*h);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return PKV_EWORKSPACE;
  const cudaError_t err =
      launch_planned(*h, pool, num_pages, q, block_table, max_blocks, seq_lens, batch, scale, out,
                     plan_dev, workspace, dev_err, reinterpret_cast<cudaStream_t>(stream),
                     nullptr);
  return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

PKV_API int pkv_decode_step_planned(
    const pkv_bf16* q, const pkv_bf16* k_new, const pkv_bf16* v_new, pkv_bf16* pool,
    int64_t num_pages, const int32_t* block_table, int max_blocks, const int32_t* seq_lens,
    int batch, int num_q_heads, int num_kv_heads, int head_dim, int page_size,
    double rope_theta, float scale, pkv_bf16* out, const void* plan_host, const void* plan_dev,
    void* workspace, size_t workspace_bytes, int32_t* dev_err, pkv_stream_t stream) {
  if (!q || !k_new || !v_new || !pool || !block_table || !seq_lens || !out || !plan_host ||
      !plan_dev)
    return PKV_EINVAL;
  if (batch < 1 || batch > 65535 || num_pages < 1 || num_pages > INT32_MAX || max_blocks < 1 ||
      max_blocks > (INT32_MAX / kPageSize))
    return PKV_EINVAL;
  if (!(scale > 0.f) || !isfinite(scale)) return PKV_EINVAL;
  if (!(rope_theta > 0.0) || !isfinite(rope_theta)) return PKV_EINVAL;
  if (!supported_dims(num_q_heads, num_kv_heads, head_dim, page_size)) return PKV_EUNSUPPORTED;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 4) || !aligned(workspace, 16) ||
      !aligned(dev_err, 4) || !aligned(v_new, 4) || !aligned(k_new, 2) ||
      !aligned(plan_dev, 16) || !aligned(plan_host, 16))
    return PKV_EALIGN;
  const PlanHeader* h = plan_header(plan_host, batch, max_blocks);
  if (h == nullptr) return PKV_EINVAL;
  const size_t need = plan_slots_bytes(*h);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return PKV_EWORKSPACE;
  pkv::AppendArgs app;
  app.k_new = k_new;
  app.v_new = v_new;
  app.pool = pool;
  if (pkv::prepare_rope(rope_theta, &app.freqs, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return PKV_ECUDA;
  const cudaError_t err =
      launch_planned(*h, pool, num_pages, q, block_table, max_blocks, seq_lens, batch, scale, out,
                     plan_dev, workspace, dev_err, reinterpret_cast<cudaStream_t>(stream), &app);
  return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

PKV_API int pkv_decode_steps_planned(
    int layers, const pkv_bf16* q, const pkv_bf16* k_new, const pkv_bf16* v_new, pkv_bf16* pool,
    int64_t num_pages, const int32_t* block_tables, int max_blocks, const int32_t* seq_lens,
    int batch, int num_q_heads, int num_kv_heads, int head_dim, int page_size, double rope_theta,
    float scale, pkv_bf16* out, const void* plan_host, const void* plan_dev, void* workspace,
    size_t workspace_bytes, int32_t* dev_err, pkv_stream_t stream) {
  if (layers < 1) return PKV_EINVAL;
  // layer 0 through the single-layer call checks every argument (the layer
  // strides keep each array's alignment: whole rows of 64 elements) and
  // prepares the RoPE table; the other layers only launch
  const int rc = pkv_decode_step_planned(q, k_new, v_new, pool, num_pages, block_tables,
                                         max_blocks, seq_lens, batch, num_q_heads, num_kv_heads,
                                         head_dim, page_size, rope_theta, scale, out, plan_host,
                                         plan_dev, workspace, workspace_bytes, dev_err, stream);
  if (rc != PKV_OK || layers == 1) return rc;
  const PlanHeader* h = plan_header(plan_host, batch, max_blocks);
  pkv::AppendArgs app;
  app.pool = pool;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (pkv::prepare_rope(rope_theta, &app.freqs, st) != cudaSuccess) return PKV_ECUDA;
  const size_t q_stride = static_cast<size_t>(batch) * kNumQHeads * kHeadDim;
  const size_t kv_stride = static_cast<size_t>(batch) * kNumKvHeads * kHeadDim;
  const size_t bt_stride = static_cast<size_t>(batch) * static_cast<size_t>(max_blocks);
  for (int l = 1; l < layers; ++l) {
    app.k_new = k_new + l * kv_stride;
    app.v_new = v_new + l * kv_stride;
    const cudaError_t err =
        launch_planned(*h, pool, num_pages, q + l * q_stride, block_tables + l * bt_stride,
                       max_blocks, seq_lens, batch, scale, out + l * q_stride, plan_dev,
                       workspace, dev_err, st, &app);
    if (err != cudaSuccess) return PKV_ECUDA;
  }
  return PKV_OK;
}

PKV_API int pkv_kv_write_prefill_layers(int layers, const pkv_bf16* k, const pkv_bf16* v,
                                        int num_tokens, const int32_t* token_offsets,
                                        const int32_t* start_positions, pkv_bf16* pool,
                                        int64_t num_pages, const int32_t* block_tables,
                                        int max_blocks, int batch, int num_kv_heads,
                                        int head_dim, int page_size, double rope_theta,
                                        int32_t* dev_err, pkv_stream_t stream) {
  if (layers < 1) return PKV_EINVAL;
  const int rc = pkv_kv_write_prefill(k, v, num_tokens, token_offsets, start_positions, pool,
                                      num_pages, block_tables, max_blocks, batch, num_kv_heads,
                                      head_dim, page_size, rope_theta, dev_err, stream);
  if (rc != PKV_OK || layers == 1 || num_tokens == 0) return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  pkv::RopeFreqs freqs;
  if (pkv::prepare_rope(rope_theta, &freqs, st) != cudaSuccess) return PKV_ECUDA;
  const size_t kv_stride = static_cast<size_t>(num_tokens) * kNumKvHeads * kHeadDim;
  const size_t bt_stride = static_cast<size_t>(batch) * static_cast<size_t>(max_blocks);
  for (int l = 1; l < layers; ++l) {
    const cudaError_t err = pkv::launch_kv_write_prefill(
        k + l * kv_stride, v + l * kv_stride, num_tokens, token_offsets, start_positions, pool,
        num_pages, block_tables + l * bt_stride, max_blocks, batch, freqs, dev_err,
        pkv::wait_limit_ns(), st);
    if (err != cudaSuccess) return PKV_ECUDA;
  }
  return PKV_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Long contexts: chunks of new tokens, sliding windows with sinks, attention
// weights and eviction by them, and the append at a slot of its own.

namespace {

// Bytes [p, p + n) that a call reads or writes.
struct Span {
  const void* p;
  size_t n;
};

bool overlap(const Span& x, const Span& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return x.p != nullptr && y.p != nullptr && x.n > 0 && y.n > 0 && a < b + y.n && b < a + x.n;
}

// True when an output shares a byte with an input or another output: outputs
// are written while inputs are still read, and in no order among themselves.
template <int kOuts, int kIns>
bool outputs_overlap(const Span (&outs)[kOuts], const Span (&ins)[kIns]) {
  for (int o = 0; o < kOuts; ++o) {
    for (const Span& i : ins)
      if (overlap(outs[o], i)) return true;
    for (int p = 0; p < o; ++p)
      if (overlap(outs[o], outs[p])) return true;
  }
  return false;
}

template <int kOuts, int kIns>
bool workspace_overlaps(const Span& ws, const Span (&outs)[kOuts], const Span (&ins)[kIns]) {
  return outputs_overlap({ws}, outs) || outputs_overlap({ws}, ins);
}

Span ints(const int32_t* p, size_t n) { return {p, n * sizeof(int32_t)}; }

Span pages_span(const pkv_bf16* pool, int64_t num_pages) {
  return {pool, static_cast<size_t>(num_pages) * 2 * kPageSize * kNumKvHeads * kHeadDim *
                    sizeof(pkv_bf16)};
}

// `rows` rows of `row` floats, `stride` floats apart.
Span rows_span(const float* p, size_t rows, int64_t stride, int64_t row) {
  return {p, rows > 0 ? ((rows - 1) * static_cast<size_t>(stride) + row) * sizeof(float) : 0};
}

bool bad_cache(int batch, int64_t num_pages, int max_blocks) {
  return batch < 0 || batch > 65535 || num_pages < 1 || num_pages > INT32_MAX || max_blocks < 1 ||
         max_blocks > (INT32_MAX / kPageSize);
}

// Widest tables of calls with a mass: their kernels step over tokens by up to
// 2^16 in 32 bits.
constexpr int kMaxMassBlocks = (INT32_MAX - (1 << 16)) / kPageSize;

// TMA descriptor of the query rows of a chunk, [num_tokens][32 heads][64] bf16:
// a box of 4 heads of 32 tokens, 128-byte swizzled.
bool chunk_q_map(const void* q, int num_tokens, CUtensorMap* out) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim),
                              static_cast<cuuint64_t>(kNumQHeads),
                              static_cast<cuuint64_t>(num_tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kHeadDim * 2),
                                 static_cast<cuuint64_t>(kNumQHeads * kHeadDim * 2)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(kHeadDim),
                             static_cast<cuuint32_t>(pkv::kGroup),
                             static_cast<cuuint32_t>(pkv::kChunkTileTokens / 2)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Ranges of a one-token call whose sequences see at most `pages` pages: CTAs for
// two an SM (scored: one and a half), but 20 pages a range or more (scored: 48,
// its merge also adds the weights), where a range's streaming is as long as the
// merge it costs.  With cold caches, one sequence of 4093: 14 us in 8 ranges, 37
// in one, 18 in 32; 34 of 403: 12 us in one, 18 in three.  Scored: one of 4093
// 21 us in 8, 31 in one, 23 in 32; 36 of 1076 23 us in one, 33 in two.
int one_token_splits(int batch, long long pages, int num_splits, bool scored) {
  if (num_splits > 0) return static_cast<int>(std::min<long long>(num_splits, pages));
  const int sms = current_sm_count();
  if (sms <= 0) return -1;
  const long long units = static_cast<long long>(batch) * kNumKvHeads;
  long long s = std::min((scored ? 3LL : 4LL) * sms / (2 * units), pages / (scored ? 48 : 20));
  // (weights that do not fit shared memory go through the workspace anyway: 45
  // sequences of 9593 took 154 us in one range, 139 in two)
  if (scored && pages > pkv::kScoredSmemPages) s = std::max(s, 2LL);
  return static_cast<int>(std::max(1LL, s));
}

long long window_pages(int max_blocks, int window, int sinks) {
  const long long seen = (static_cast<long long>(window) + kPageSize - 2) / kPageSize + 1;
  return std::min<long long>(
      max_blocks, seen + (static_cast<long long>(sinks) + kPageSize - 1) / kPageSize);
}

// Ranges and CTAs of a chunk call.  Chunks of more than kShortTokens tokens
// are cut into tiles of up to 64, so there are at most tokens / 64 + the
// number of such chunks of them.
struct ChunkPlan {
  int num_splits, short_splits, grid;  // grid 0: no long chunk is possible
  size_t long_parts, short_parts;      // rows of partials
  size_t workspace;
};

bool chunk_plan(int num_tokens, int batch, int max_blocks, int window, int sinks, int num_splits,
                ChunkPlan* plan) {
  const long long chunks = std::min(batch, num_tokens / (pkv::kShortTokens + 1));
  const long long items =
      chunks > 0 ? (num_tokens / pkv::kChunkTileTokens + chunks) * kNumKvHeads : 0;
  constexpr int kKvPages = pkv::kChunkKvTokens / kPageSize;
  long long kv = (max_blocks + kKvPages - 1) / kKvPages;  // most kv tiles of an item
  long long pages = max_blocks;                           // most pages of a short chunk
  if (window > 0) {
    kv = std::min(kv, (static_cast<long long>(window) + pkv::kChunkTileTokens - 2) /
                              pkv::kChunkKvTokens + 2 +
                          (static_cast<long long>(sinks) + pkv::kChunkKvTokens - 1) /
                              pkv::kChunkKvTokens);
    pages = window_pages(max_blocks, static_cast<int>(std::min<long long>(
                                         static_cast<long long>(window) + pkv::kShortTokens - 1,
                                         INT32_MAX)), sinks);
  }
  const int sms = current_sm_count();
  long long s = num_splits;
  if (s == 0) {
    if (sms <= 0) return false;
    // (items bounds their number; chunks of one length make this many, and more
    // ranges than CTAs of a wave cost little, fewer leave SMs idle: 8 chunks of
    // 64 tokens over 16384 took 142 us in one range, 87 us in two)
    const long long each = (num_tokens + chunks - 1) / std::max(chunks, 1LL);
    const long long likely =
        chunks * ((each + pkv::kChunkTileTokens - 1) / pkv::kChunkTileTokens) * kNumKvHeads;
    s = std::max(1LL, std::min(sms / std::max(likely, 1LL), kv / 8));
    // long caches whose last round of items would leave a third of the SMs idle:
    // three ranges (2 x 700 tokens over 16384, 176 items: 252 -> 202 us; 6 x 128
    // over 16384, 96 items: 139 -> 107; but 5 x 256 over 6000, 160 items: 68 ->
    // 83, where the merge costs more)
    const long long rounds = (likely + sms - 1) / sms;
    if (s == 1 && kv >= 64 && 2 * rounds * sms >= 3 * likely) s = 3;
  }
  s = std::min(s, std::max(kv, 1LL));
  plan->num_splits = static_cast<int>(items > 0 ? s : 1);
  // short chunks: one wave of the CTAs that fit (short_chunk.cu: three per SM
  // beside a long chunk, else four), eight pages a range or more; more tokens
  // than short chunks of this batch can have mean a long one, or a padded q: one
  // sequence gets its ranges all the same.  (32 x 4 tokens over 4096: 69 us in
  // one range, 58 us in two; 64 x 4 over 2048 53 and 60.  One sequence of 4
  // tokens in a q of 8 rows, over 2048, 16384 and 131072: 17, 28 and 69 us, in
  // one range 30, 155 and 1350; a long chunk pays the merge, 1 us.)
  long long t = num_splits;
  if (t == 0) {
    const bool a_long_one = num_tokens > pkv::kShortTokens * static_cast<long long>(batch);
    const long long most = a_long_one ? std::max(batch - 1, 1) : std::min(batch, num_tokens);
    t = std::max(1LL, std::min((a_long_one ? 3LL : 4LL) * sms / (most * kNumKvHeads),
                               (pages + 7) / 8));
  }
  plan->short_splits = static_cast<int>(std::min(t, pages));
  plan->grid = static_cast<int>(std::min<long long>(sms > 0 ? sms : 1, items * s));
  plan->long_parts = plan->num_splits > 1
                         ? static_cast<size_t>(num_tokens) * kNumQHeads * plan->num_splits
                         : 0;
  plan->short_parts = plan->short_splits > 1 ? static_cast<size_t>(batch) * pkv::kShortTokens *
                                                   kNumQHeads * plan->short_splits
                                             : 0;
  plan->workspace = (plan->long_parts + plan->short_parts) * (kHeadDim + 2) * sizeof(float);
  return true;
}

size_t part_bytes(int batch, int splits) {
  return splits > 1 ? static_cast<size_t>(batch) * kNumQHeads * splits * (kHeadDim + 2) *
                          sizeof(float)
                    : 0;
}

// Scores of a call that wants the weights, when shared memory does not hold
// them: four floats for every token of the tables and kv head.
size_t score_bytes(int batch, int max_blocks, int splits) {
  if (splits == 1 && max_blocks <= pkv::kScoredSmemPages) return 0;
  return static_cast<size_t>(batch) * kNumKvHeads * max_blocks * kPageSize * pkv::kGroup *
         sizeof(float);
}

Span heads_span(const pkv_bf16* p, int rows, int heads = kNumQHeads) {
  return {p, static_cast<size_t>(rows) * heads * kHeadDim * sizeof(pkv_bf16)};
}

}  // namespace

extern "C" {

PKV_API int pkv_kv_append_at(const pkv_bf16* k_new, const pkv_bf16* v_new, pkv_bf16* pool,
                             int64_t num_pages, const int32_t* block_table, int max_blocks,
                             const int32_t* positions, const int32_t* slots, int batch,
                             int num_kv_heads, int head_dim, int page_size, double rope_theta,
                             const pkv_bf16* q_in, pkv_bf16* q_out, int num_q_heads,
                             int32_t* dev_err, pkv_stream_t stream) {
  if (!k_new || !v_new || !pool || !block_table || !positions || !slots) return PKV_EINVAL;
  if (bad_cache(batch, num_pages, max_blocks)) return PKV_EINVAL;
  if ((q_in == nullptr) != (q_out == nullptr)) return PKV_EINVAL;
  if (!(rope_theta > 0.0) || !isfinite(rope_theta)) return PKV_EINVAL;
  if (num_kv_heads != kNumKvHeads || head_dim != kHeadDim || page_size != kPageSize)
    return PKV_EUNSUPPORTED;
  if (q_in != nullptr && num_q_heads != kNumQHeads) return PKV_EUNSUPPORTED;
  if (!aligned(pool, 16) || !aligned(v_new, 4) || !aligned(k_new, 2) || !aligned(q_in, 2) ||
      !aligned(q_out, 2) || !aligned(positions, 4) || !aligned(slots, 4) ||
      !aligned(block_table, 4) || !aligned(dev_err, 4))
    return PKV_EALIGN;
  const size_t rows = static_cast<size_t>(batch);
  // (the pool is the caller's: a page that is not appended to may hold inputs)
  const Span ins[] = {heads_span(k_new, batch, kNumKvHeads),
                      heads_span(v_new, batch, kNumKvHeads),
                      heads_span(q_in, batch),
                      ints(block_table, rows * max_blocks),
                      ints(positions, rows),
                      ints(slots, rows)};
  const Span outs[] = {heads_span(q_out, batch), ints(dev_err, 1)};
  if (outputs_overlap(outs, ins)) return PKV_EINVAL;
  if (overlap(outs[0], pages_span(pool, num_pages)) ||
      overlap(outs[1], pages_span(pool, num_pages)))
    return PKV_EINVAL;
  if (batch == 0) return PKV_OK;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  pkv::RopeFreqs freqs;
  if (pkv::prepare_rope(rope_theta, &freqs, st) != cudaSuccess) return PKV_ECUDA;
  const cudaError_t err =
      pkv::launch_kv_append(k_new, v_new, pool, num_pages, block_table, max_blocks, positions,
                            slots, batch, freqs, q_in, q_out, dev_err, st);
  return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

PKV_API size_t pkv_chunk_workspace_bytes(int num_tokens, int batch, int num_q_heads,
                                         int num_kv_heads, int head_dim, int max_blocks,
                                         int window, int sinks, int num_splits) {
  if (num_tokens < 0 || bad_cache(batch, 1, max_blocks) || window < 0 || sinks < 0 ||
      num_splits < 0 || !supported_dims(num_q_heads, num_kv_heads, head_dim, kPageSize))
    return static_cast<size_t>(-1);
  if (num_tokens == 0 || batch == 0) return 0;
  ChunkPlan plan;
  if (!chunk_plan(num_tokens, batch, max_blocks, window, sinks, num_splits, &plan))
    return static_cast<size_t>(-1);
  return plan.workspace;
}

PKV_API int pkv_paged_chunk_attention(
    const pkv_bf16* q, int num_tokens, const int32_t* token_offsets, const pkv_bf16* pool,
    int64_t num_pages, const int32_t* block_table, int max_blocks, const int32_t* seq_lens,
    int batch, int num_q_heads, int num_kv_heads, int head_dim, int page_size, int window,
    int sinks, float scale, pkv_bf16* out, void* workspace, size_t workspace_bytes,
    int num_splits, int32_t* dev_err, pkv_stream_t stream) {
  if (!q || !token_offsets || !pool || !block_table || !seq_lens || !out) return PKV_EINVAL;
  if (num_tokens < 0 || bad_cache(batch, num_pages, max_blocks) || window < 0 || sinks < 0 ||
      num_splits < 0)
    return PKV_EINVAL;
  if (!(scale > 0.f) || !isfinite(scale)) return PKV_EINVAL;
  if (!supported_dims(num_q_heads, num_kv_heads, head_dim, page_size)) return PKV_EUNSUPPORTED;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
      !aligned(token_offsets, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(dev_err, 4))
    return PKV_EALIGN;
  const size_t seqs = static_cast<size_t>(batch);
  const Span ins[] = {heads_span(q, num_tokens), ints(token_offsets, seqs + 1),
                      pages_span(pool, num_pages), ints(block_table, seqs * max_blocks),
                      ints(seq_lens, seqs)};
  const Span outs[] = {heads_span(out, num_tokens), ints(dev_err, 1)};
  if (outputs_overlap(outs, ins)) return PKV_EINVAL;
  if (batch == 0 || num_tokens == 0) return PKV_OK;
  ChunkPlan plan;
  if (!chunk_plan(num_tokens, batch, max_blocks, window, sinks, num_splits, &plan))
    return PKV_ECUDA;
  if (plan.workspace > 0 && (workspace == nullptr || workspace_bytes < plan.workspace))
    return PKV_EWORKSPACE;
  if (workspace_overlaps({workspace, plan.workspace}, outs, ins)) return PKV_EINVAL;
  pkv::MaskedArgs a = {};
  a.q = q;
  a.pool = pool;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.token_offsets = token_offsets;
  a.out = out;
  a.dev_err = dev_err;
  a.num_pages = num_pages;
  a.max_blocks = max_blocks;
  a.batch = batch;
  a.num_tokens = num_tokens;
  a.window = window > 0 ? window : INT32_MAX;
  a.sinks = sinks;
  a.num_splits = plan.num_splits;
  a.short_splits = plan.short_splits;
  // partials: accumulators of the long and of the short chunks, then the
  // (max, sum) pairs
  a.part_acc = static_cast<float*>(workspace);
  a.short_acc = a.part_acc + plan.long_parts * kHeadDim;
  a.part_ml = a.short_acc + plan.short_parts * kHeadDim;
  a.short_ml = a.part_ml + plan.long_parts * 2;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.wait_ns = pkv::wait_limit_ns();
  CUtensorMap q_map, page_map, pool_map;
  if (!chunk_q_map(q, num_tokens, &q_map) ||
      !pool_tensor_map(pool, num_pages, &page_map, kPageSize) ||
      !pool_tensor_map(pool, num_pages, &pool_map))
    return PKV_ECUDA;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t err = cudaSuccess;
  if (plan.grid > 0) err = pkv::launch_chunk_attention(q_map, page_map, a, plan.grid, st);
  if (err == cudaSuccess) err = pkv::launch_short_chunks(pool_map, a, plan.grid > 0, st);
  if (err == cudaSuccess && plan.grid > 0 && a.num_splits > 1) err = pkv::launch_chunk_merge(a, st);
  return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

PKV_API size_t pkv_window_workspace_bytes(int batch, int num_q_heads, int num_kv_heads,
                                          int head_dim, int max_blocks, int window, int sinks,
                                          int num_splits) {
  if (bad_cache(batch, 1, max_blocks) || window < 1 || sinks < 0 || num_splits < 0 ||
      !supported_dims(num_q_heads, num_kv_heads, head_dim, kPageSize))
    return static_cast<size_t>(-1);
  if (batch == 0) return 0;
  const int splits =
      one_token_splits(batch, window_pages(max_blocks, window, sinks), num_splits, false);
  return splits < 1 ? static_cast<size_t>(-1) : part_bytes(batch, splits);
}

PKV_API int pkv_paged_window_attention(
    const pkv_bf16* q, const pkv_bf16* pool, int64_t num_pages, const int32_t* block_table,
    int max_blocks, const int32_t* seq_lens, int batch, int num_q_heads, int num_kv_heads,
    int head_dim, int page_size, int window, int sinks, float scale, pkv_bf16* out,
    void* workspace, size_t workspace_bytes, int num_splits, int32_t* dev_err,
    pkv_stream_t stream) {
  if (!q || !pool || !block_table || !seq_lens || !out) return PKV_EINVAL;
  if (bad_cache(batch, num_pages, max_blocks) || window < 1 || sinks < 0 || num_splits < 0)
    return PKV_EINVAL;
  if (!(scale > 0.f) || !isfinite(scale)) return PKV_EINVAL;
  if (!supported_dims(num_q_heads, num_kv_heads, head_dim, page_size)) return PKV_EUNSUPPORTED;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 4) || !aligned(workspace, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(dev_err, 4))
    return PKV_EALIGN;
  const size_t seqs = static_cast<size_t>(batch);
  const Span ins[] = {heads_span(q, batch), pages_span(pool, num_pages),
                      ints(block_table, seqs * max_blocks), ints(seq_lens, seqs)};
  const Span outs[] = {heads_span(out, batch), ints(dev_err, 1)};
  if (outputs_overlap(outs, ins)) return PKV_EINVAL;
  if (batch == 0) return PKV_OK;
  const int splits =
      one_token_splits(batch, window_pages(max_blocks, window, sinks), num_splits, false);
  if (splits < 1) return PKV_ECUDA;
  const size_t need = part_bytes(batch, splits);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return PKV_EWORKSPACE;
  if (workspace_overlaps({workspace, need}, outs, ins)) return PKV_EINVAL;
  pkv::MaskedArgs a = {};
  a.q = q;
  a.pool = pool;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.dev_err = dev_err;
  a.num_pages = num_pages;
  a.max_blocks = max_blocks;
  a.batch = batch;
  a.num_tokens = batch;
  a.window = window;
  a.sinks = sinks;
  a.num_splits = splits;
  if (need > 0) {
    a.part_acc = static_cast<float*>(workspace);
    a.part_ml = a.part_acc + static_cast<size_t>(batch) * kNumQHeads * splits * kHeadDim;
  }
  a.scale_log2 = scale * 1.4426950408889634f;
  a.wait_ns = pkv::wait_limit_ns();
  CUtensorMap map;
  if (!pool_tensor_map(pool, num_pages, &map)) return PKV_ECUDA;
  const cudaError_t err =
      pkv::launch_window_attention(map, a, 0, reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

PKV_API size_t pkv_scored_workspace_bytes(int batch, int num_q_heads, int num_kv_heads,
                                          int head_dim, int max_blocks, int num_splits) {
  if (bad_cache(batch, 1, max_blocks) || max_blocks > kMaxMassBlocks || num_splits < 0 ||
      !supported_dims(num_q_heads, num_kv_heads, head_dim, kPageSize))
    return static_cast<size_t>(-1);
  if (batch == 0) return 0;
  const int splits = one_token_splits(batch, max_blocks, num_splits, true);
  return splits < 1 ? static_cast<size_t>(-1)
                    : part_bytes(batch, splits) + score_bytes(batch, max_blocks, splits);
}

PKV_API int pkv_paged_scored_attention(
    const pkv_bf16* q, const pkv_bf16* pool, int64_t num_pages, const int32_t* block_table,
    int max_blocks, const int32_t* seq_lens, int batch, int num_q_heads, int num_kv_heads,
    int head_dim, int page_size, float scale, pkv_bf16* out, float* mass, int64_t mass_stride,
    void* workspace, size_t workspace_bytes, int num_splits, int32_t* dev_err,
    pkv_stream_t stream) {
  if (!q || !pool || !block_table || !seq_lens || !out || !mass) return PKV_EINVAL;
  if (bad_cache(batch, num_pages, max_blocks) || max_blocks > kMaxMassBlocks || num_splits < 0 ||
      mass_stride < static_cast<int64_t>(max_blocks) * kPageSize)
    return PKV_EINVAL;
  if (!(scale > 0.f) || !isfinite(scale)) return PKV_EINVAL;
  if (!supported_dims(num_q_heads, num_kv_heads, head_dim, page_size)) return PKV_EUNSUPPORTED;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 4) || !aligned(workspace, 16) ||
      !aligned(mass, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(dev_err, 4))
    return PKV_EALIGN;
  const size_t seqs = static_cast<size_t>(batch);
  const Span ins[] = {heads_span(q, batch), pages_span(pool, num_pages),
                      ints(block_table, seqs * max_blocks), ints(seq_lens, seqs)};
  const Span outs[] = {heads_span(out, batch),
                       rows_span(mass, seqs * kNumKvHeads, mass_stride,
                                 static_cast<int64_t>(max_blocks) * kPageSize),
                       ints(dev_err, 1)};
  if (outputs_overlap(outs, ins)) return PKV_EINVAL;
  if (batch == 0) return PKV_OK;
  const int splits = one_token_splits(batch, max_blocks, num_splits, true);
  if (splits < 1) return PKV_ECUDA;
  const size_t parts = part_bytes(batch, splits), keep = score_bytes(batch, max_blocks, splits);
  if (parts + keep > 0 && (workspace == nullptr || workspace_bytes < parts + keep))
    return PKV_EWORKSPACE;
  if (workspace_overlaps({workspace, parts + keep}, outs, ins)) return PKV_EINVAL;
  pkv::MaskedArgs a = {};
  a.q = q;
  a.pool = pool;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.mass = mass;
  a.mass_stride = mass_stride;
  a.dev_err = dev_err;
  a.num_pages = num_pages;
  a.max_blocks = max_blocks;
  a.batch = batch;
  a.num_tokens = batch;
  a.window = INT32_MAX;
  a.num_splits = splits;
  // the scores (16-byte aligned) first, then the partials
  if (keep > 0) a.scores = static_cast<float*>(workspace);
  if (parts > 0) {
    a.part_acc = reinterpret_cast<float*>(static_cast<char*>(workspace) + keep);
    a.part_ml = a.part_acc + static_cast<size_t>(batch) * kNumQHeads * splits * kHeadDim;
  }
  a.scale_log2 = scale * 1.4426950408889634f;
  a.wait_ns = pkv::wait_limit_ns();
  CUtensorMap map;
  if (!pool_tensor_map(pool, num_pages, &map)) return PKV_ECUDA;
  const cudaError_t err =
      pkv::launch_window_attention(map, a, keep > 0 ? 0 : max_blocks,
                                   reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

PKV_API int pkv_kv_evict(const float* mass, int64_t mass_stride, pkv_bf16* pool,
                         int64_t num_pages, const int32_t* block_table, int max_blocks,
                         const int32_t* seq_lens, int batch, int num_kv_heads, int head_dim,
                         int page_size, int budget, int sinks, int recent,
                         const int32_t* dst_block_table, int dst_max_blocks, int32_t* new_lens,
                         float* new_mass, int64_t new_mass_stride, int32_t* kept,
                         int32_t* dev_err, pkv_stream_t stream) {
  if (!mass || !pool || !block_table || !seq_lens || !dst_block_table || !new_lens ||
      !new_mass || !kept)
    return PKV_EINVAL;
  if (bad_cache(batch, num_pages, max_blocks) || bad_cache(batch, num_pages, dst_max_blocks) ||
      max_blocks > kMaxMassBlocks || dst_max_blocks > kMaxMassBlocks || budget < 1 || sinks < 0 ||
      recent < 0 || sinks > budget || recent > budget - sinks ||
      budget > static_cast<int64_t>(dst_max_blocks) * kPageSize ||
      mass_stride < static_cast<int64_t>(max_blocks) * kPageSize || new_mass_stride < budget)
    return PKV_EINVAL;
  if (num_kv_heads != kNumKvHeads || head_dim != kHeadDim || page_size != kPageSize)
    return PKV_EUNSUPPORTED;
  if (!aligned(pool, 16) || !aligned(mass, 4) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(dst_block_table, 4) || !aligned(new_lens, 4) ||
      !aligned(new_mass, 4) || !aligned(kept, 4) || !aligned(dev_err, 4))
    return PKV_EALIGN;
  const size_t seqs = static_cast<size_t>(batch), rows = seqs * kNumKvHeads;
  const Span ins[] = {rows_span(mass, rows, mass_stride,
                                static_cast<int64_t>(max_blocks) * kPageSize),
                      pages_span(pool, num_pages), ints(seq_lens, seqs),
                      ints(block_table, seqs * max_blocks),
                      ints(dst_block_table, seqs * dst_max_blocks)};
  const Span outs[] = {ints(new_lens, seqs),
                       rows_span(new_mass, rows, new_mass_stride, new_mass_stride),
                       ints(kept, rows * budget), ints(dev_err, 1)};
  if (outputs_overlap(outs, ins)) return PKV_EINVAL;
  if (batch == 0) return PKV_OK;
  pkv::EvictArgs a = {};
  a.mass = mass;
  a.pool = pool;
  a.block_table = block_table;
  a.dst_block_table = dst_block_table;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.new_mass = new_mass;
  a.kept = kept;
  a.dev_err = dev_err;
  a.num_pages = num_pages;
  a.mass_stride = mass_stride;
  a.new_mass_stride = new_mass_stride;
  a.max_blocks = max_blocks;
  a.dst_max_blocks = dst_max_blocks;
  a.batch = batch;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  const int sms = current_sm_count();
  if (sms <= 0) return PKV_ECUDA;
  const cudaError_t err = pkv::launch_kv_evict(a, sms, reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

}  // extern "C"
