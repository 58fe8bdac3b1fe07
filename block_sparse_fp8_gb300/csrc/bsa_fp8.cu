// Block-sparse FP8 attention prefill over a paged KV cache, for GB300 (sm_103a): host entry
// points of the C ABI (include/bsa_fp8.h) and the exported active-tile list kernel.
//
//   * bsa_compact_kernel -- one warp per (b, h, qt) task writes the ascending list of active
//     KV tiles (warp ballot stream compaction; hpc-ops Block-Sparse FP8 Attention, section
//     活跃 tile 列表).  The attention kernel runs the same device function on its own tasks.
//   * attn::bsa_attention_kernel (bsa_attention.cuh) -- the persistent prefill kernel.
//   * quant::quantize_rows_kernel / quant::append_kv_kernel (bsa_quant.cuh) -- the quantise
//     step that produces the prefill's e4m3 inputs.
//   * decode (bsa_decode.cuh), gather (bsa_gather.cuh), merge (bsa_merge.cuh) -- serving: the next
//     token's attention over the cache, the cache read back, the join of attention results.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "bsa_attention.cuh"
#include "bsa_attention_wide.cuh"
#include "bsa_common.cuh"
#include "bsa_decode.cuh"
#include "bsa_decode_fp4.cuh"
#include "bsa_fp4.cuh"
#include "bsa_fp8.h"
#include "bsa_gather.cuh"
#include "bsa_merge.cuh"
#include "bsa_pages.cuh"
#include "bsa_quant.cuh"
#include "bsa_rope.cuh"
#include "ptx_sm103.cuh"

namespace bsa {

constexpr int COMPACT_WARPS = 4;

__global__ void __launch_bounds__(COMPACT_WARPS * 32) bsa_compact_kernel(const Params p,
                                                                        int *tile_lists,
                                                                        int *tile_counts) {
  __shared__ uint32_t bitmaps[COMPACT_WARPS][KB_MAX / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long task = (long long)blockIdx.x * COMPACT_WARPS + warp;
  const long long ntasks = (long long)p.B * p.N1 * p.Qb;
  if (task >= ntasks) return;
  const int qt = (int)(task % p.Qb);
  const int h = (int)((task / p.Qb) % p.N1);
  const int b = (int)(task / ((long long)p.Qb * p.N1));
  TaskGeo g = task_geometry(p, b, qt);
  int *list = tile_lists + task * p.Kb;
  int n = compact_task(p, b, h, qt, g.kend, list, bitmaps[warp]);
  for (int t = n + lane; t < p.Kb; t += 32) list[t] = -1;
  if (lane == 0) tile_counts[task] = n;
}

// ------------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------------

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

static bool aligned16(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

static int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

// Checks only host-visible facts: dims, scalars, pointer nullness and alignment.
static bsa_status_t validate_dims(const bsa_fp8_dims_t *d) {
  if (!d) return BSA_ERR_INVALID_ARGUMENT;
  if (d->D != HEAD_DIM) return BSA_ERR_INVALID_ARGUMENT;
  if (d->page_size != 32 && d->page_size != 64) return BSA_ERR_INVALID_ARGUMENT;
  if (d->B < 0 || d->N1 < 1 || d->N2 < 1 || d->N1 % d->N2 != 0 || d->N1 / d->N2 > 16)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->max_q_len < 0 || d->max_kv_len < 0 || d->total_q < 0 || d->num_pages < 0 ||
      d->max_pages_per_seq < 0)
    return BSA_ERR_INVALID_ARGUMENT;
  if ((long long)d->max_pages_per_seq * d->page_size < d->max_kv_len)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->k_scale_kind != BSA_SCALE_PER_TENSOR && d->k_scale_kind != BSA_SCALE_PER_TOKEN_HEAD)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->v_scale_kind != BSA_SCALE_PER_TENSOR && d->v_scale_kind != BSA_SCALE_PER_HEAD)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->causal != 0 && d->causal != 1) return BSA_ERR_INVALID_ARGUMENT;
  if (d->q_layout != BSA_Q_TND && d->q_layout != BSA_Q_NTD) return BSA_ERR_INVALID_ARGUMENT;
  if (d->kv_layout != BSA_KV_HND && d->kv_layout != BSA_KV_NHD) return BSA_ERR_INVALID_ARGUMENT;
  if (d->tiles_per_step < 0 || d->tiles_per_step > 2) return BSA_ERR_INVALID_ARGUMENT;
  if (cdiv(d->max_kv_len, TILE) > KB_MAX) return BSA_ERR_UNSUPPORTED;
  // task indices are int; the work-item counter runs past the last task by up to one claim
  // per pipeline, so keep the count well inside int range
  if ((long long)d->B * d->N1 * cdiv(d->max_q_len, TILE) > (1LL << 30))
    return BSA_ERR_UNSUPPORTED;
  return BSA_OK;
}

struct DeviceInfo {
  int state = 0;  // 0 unknown, 1 supported, 2 unsupported
  int num_sms = 0;
  int smem_per_sm = 0;        // shared memory of one SM
  int smem_reserved = 0;      // shared memory the system reserves per resident block
  size_t smem_attr = 0;  // dynamic shared memory the attention kernel is enabled for
  size_t smem_attr_wide = 0;  // ... and the 256-wide macro-block kernel
  bool decode_attr = false;   // the decode kernels' shared memory is enabled
};

static DeviceInfo g_devices[64];
static std::mutex g_devices_mu;

// sm_103 only; caches the SM count and raises the attention kernel's shared-memory limit.
static bsa_status_t check_device(size_t attn_smem, int *num_sms, int *per_sm = nullptr,
                                 bool wide = false) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
  if (dev < 0 || dev >= 64) return BSA_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_devices_mu);
  DeviceInfo &di = g_devices[dev];
  if (di.state == 0) {
    int major = 0, minor = 0, sms = 0, smem_sm = 0, smem_res = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&smem_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) !=
            cudaSuccess ||
        cudaDeviceGetAttribute(&smem_res, cudaDevAttrReservedSharedMemoryPerBlock, dev) !=
            cudaSuccess)
      return BSA_ERR_CUDA;
    di.state = (major == 10 && minor == 3) ? 1 : 2;
    di.num_sms = sms;
    di.smem_per_sm = smem_sm;
    di.smem_reserved = smem_res;
    if (di.state == 1) {
      // The softmax warpgroups raise their registers with setmaxnreg.inc, drawing on what the
      // CTA was launched with; that only completes if the launch allocation covers the
      // whole split, so refuse to launch a build where it does not.
      cudaFuncAttributes fa, fw;
      if (cudaFuncGetAttributes(&fa, attn::bsa_attention_kernel) != cudaSuccess ||
          cudaFuncGetAttributes(&fw, attn_wide::bsa_attention_wide_kernel) != cudaSuccess)
        return BSA_ERR_CUDA;
      if (fa.numRegs * attn::NTHREADS < attn::SPLIT_REGS ||
          fw.numRegs * attn_wide::NTHREADS < attn_wide::SPLIT_REGS)
        di.state = 2;
    }
  }
  if (di.state != 1) return BSA_ERR_UNSUPPORTED;
  size_t &attr = wide ? di.smem_attr_wide : di.smem_attr;
  if (attn_smem > attr) {
    const cudaError_t e =
        wide ? cudaFuncSetAttribute(attn_wide::bsa_attention_wide_kernel,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)attn_smem)
             : cudaFuncSetAttribute(attn::bsa_attention_kernel,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)attn_smem);
    if (e != cudaSuccess) return BSA_ERR_CUDA;
    attr = attn_smem;
  }
  if (num_sms) *num_sms = di.num_sms;
  if (per_sm) *per_sm = 1;  // one CTA per SM: it holds the SM's registers and all of TMEM
  return BSA_OK;
}

// Limit of one bounded wait inside the prefill kernel; 0 selects the default.
static std::atomic<unsigned long long> g_wait_limit_ns{0};

static Params make_params(const bsa_fp8_dims_t *d) {
  Params p;
  memset(&p, 0, sizeof(p));
  const unsigned long long lim = g_wait_limit_ns.load(std::memory_order_relaxed);
  p.wait_limit_ns = lim ? lim : WAIT_LIMIT_NS;
  p.B = d->B;
  p.N1 = d->N1;
  p.N2 = d->N2;
  p.G = d->N1 / d->N2;
  p.ps = d->page_size;
  p.max_q_len = d->max_q_len;
  p.max_kv_len = d->max_kv_len;
  p.num_pages = d->num_pages;
  p.L = d->max_pages_per_seq;
  p.T = d->total_q;
  p.Qb = cdiv(d->max_q_len, TILE);
  p.Kb = cdiv(d->max_kv_len, TILE);
  p.k_per_token = d->k_scale_kind == BSA_SCALE_PER_TOKEN_HEAD;
  p.v_per_head = d->v_scale_kind == BSA_SCALE_PER_HEAD;
  p.causal = d->causal;
  p.q_ntd = d->q_layout == BSA_Q_NTD;
  p.kv_nhd = d->kv_layout == BSA_KV_NHD;
  p.qd_tok = p.q_ntd ? 1 : d->N1;
  p.qd_head = p.q_ntd ? d->total_q : 1;
  return p;
}

static bool encode_map(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims,
                       const cuuint64_t *strides, const cuuint32_t *box,
                       CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void *>(base),
                  dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, promotion,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace bsa

using namespace bsa;

// one int: the work-item counter the persistent CTAs claim work from (padded to 256 bytes)
static constexpr size_t WORKSPACE_BYTES = 256;

namespace {

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// Split-KV plan.  When the (b, h, q-tile) tasks cannot occupy half of the pipelines (two per
// SM), each task's active list is cut into S slices (work items) that run on separate
// pipelines and are merged afterwards.  S = min(8, pipelines / tasks, Kb / 16): a slice covers
// at least 16 KV tiles of the task's range.  Splitting costs a partial write and a merge per
// task, which measured more than it saved once every pipeline already had a task.
struct SplitPlan {
  int splits = 1;
  size_t bytes = WORKSPACE_BYTES;           // workspace needed
  size_t off_cnt = 0, off_ml = 0, off_o = 0;
};

SplitPlan plan_splits(const Params &p, int num_sms, bool allow) {
  SplitPlan plan;
  const long long ntasks = (long long)p.B * p.N1 * p.Qb;
  const long long pipes = (long long)attn::NPIPE * std::max(num_sms, 1);
  if (!allow || ntasks <= 0 || 2 * ntasks > pipes) return plan;
  const int best = (int)std::min<long long>(std::min<long long>(attn::MAX_SPLITS, pipes / ntasks),
                                             p.Kb / 16);
  if (best <= 1) return plan;
  const long long items = ntasks * best;
  plan.splits = best;
  plan.off_cnt = WORKSPACE_BYTES;
  plan.off_ml = plan.off_cnt + round256((size_t)ntasks * TILE * 2 * sizeof(int));
  plan.off_o = plan.off_ml + round256((size_t)items * TILE * 2 * 2 * sizeof(float));
  plan.bytes = plan.off_o + (size_t)items * TILE * HEAD_DIM * sizeof(float);
  return plan;
}

}  // namespace

extern "C" size_t bsa_fp8_prefill_workspace_size(const bsa_fp8_dims_t *dims) {
  if (validate_dims(dims) != BSA_OK) return 0;
  int num_sms = 0;
  if (check_device(0, &num_sms) != BSA_OK) return WORKSPACE_BYTES;
  return plan_splits(make_params(dims), num_sms, dims->tiles_per_step != 2).bytes;
}

extern "C" bsa_status_t bsa_fp8_set_wait_limit_ns(unsigned long long ns) {
  g_wait_limit_ns.store(ns, std::memory_order_relaxed);
  return BSA_OK;
}

extern "C" const char *bsa_status_string(bsa_status_t status) {
  switch (status) {
    case BSA_OK: return "ok";
    case BSA_ERR_INVALID_ARGUMENT: return "invalid argument";
    case BSA_ERR_UNSUPPORTED: return "unsupported (device or size)";
    case BSA_ERR_CUDA: return "CUDA error";
    case BSA_ERR_WORKSPACE: return "workspace too small";
  }
  return "unknown status";
}

extern "C" bsa_status_t bsa_fp8_compact_tiles(const bsa_fp8_dims_t *dims, const int *cu_seqlens_q,
                                              const int *seqused_kv, const uint8_t *block_mask,
                                              const int *sparse_indices,
                                              const int *sparse_seq_len, int *tile_lists,
                                              int *tile_counts, int *dev_status, void *stream) {
  bsa_status_t st = validate_dims(dims);
  if (st != BSA_OK) return st;
  if (block_mask && sparse_indices) return BSA_ERR_INVALID_ARGUMENT;
  if (sparse_indices && !sparse_seq_len) return BSA_ERR_INVALID_ARGUMENT;
  Params p = make_params(dims);
  const long long ntasks = (long long)p.B * p.N1 * p.Qb;
  if (ntasks == 0 || p.Kb == 0) return BSA_OK;
  if (!cu_seqlens_q || !tile_lists || !tile_counts) return BSA_ERR_INVALID_ARGUMENT;
  st = check_device(0, nullptr);
  if (st != BSA_OK) return st;
  p.cu_seqlens_q = cu_seqlens_q;
  p.seqused_kv = seqused_kv;
  p.block_mask = block_mask;
  p.sparse_indices = sparse_indices;
  p.sparse_seq_len = sparse_seq_len;
  p.dev_status = dev_status;
  const long long blocks = (ntasks + COMPACT_WARPS - 1) / COMPACT_WARPS;
  bsa_compact_kernel<<<(unsigned)blocks, COMPACT_WARPS * 32, 0, (cudaStream_t)stream>>>(
      p, tile_lists, tile_counts);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

// ------------------------------------------------------------------------------------------
// The workspace of bsa_fp8_prefill_noalloc, for callers that cannot allocate device memory:
// this file-scope array, 256 bytes on every device that loads the library.
// ------------------------------------------------------------------------------------------

namespace {

constexpr size_t NOALLOC_SCRATCH_BYTES = 256;
static_assert(NOALLOC_SCRATCH_BYTES >= WORKSPACE_BYTES,
              "the array must hold the unsplit prefill's workspace");
static __device__ __align__(256) unsigned char g_noalloc_scratch[NOALLOC_SCRATCH_BYTES];

// Host code cannot pass g_noalloc_scratch itself to a kernel (on the host that name is only a
// stand-in for the device symbol): look up the device address with the device current and
// reuse it.  The address belongs to the context the module was loaded into, so it is cached
// together with that context's ID and looked up again when the ID changes (a device reset or
// a recreated primary context loads the module afresh, possibly at another address).
struct NoallocAddr {
  unsigned long long ctx_id = 0;
  void *ptr = nullptr;
};
NoallocAddr g_noalloc_addr[64];
std::mutex g_noalloc_mu;

struct CtxFns {
  PFN_cuCtxGetCurrent_v4000 get_current = nullptr;
  PFN_cuCtxGetId_v12000 get_id = nullptr;
};

const CtxFns &ctx_fns() {
  static CtxFns fns;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &ptr, 4000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fns.get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(ptr);
    ptr = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fns.get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(ptr);
  });
  return fns;
}

// Called after check_device(), so the device's primary context is current.
bsa_status_t noalloc_scratch(void **addr) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
  if (dev < 0 || dev >= 64) return BSA_ERR_UNSUPPORTED;
  const CtxFns &fns = ctx_fns();
  CUcontext ctx = nullptr;
  unsigned long long id = 0;
  if (!fns.get_current || !fns.get_id || fns.get_current(&ctx) != CUDA_SUCCESS || !ctx ||
      fns.get_id(ctx, &id) != CUDA_SUCCESS)
    return BSA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  NoallocAddr &a = g_noalloc_addr[dev];
  if (!a.ptr || a.ctx_id != id) {
    void *ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_noalloc_scratch) != cudaSuccess || !ptr) {
      (void)cudaGetLastError();  // leave no pending error behind for the caller
      return BSA_ERR_CUDA;
    }
    a.ptr = ptr;
    a.ctx_id = id;
  }
  *addr = a.ptr;
  return BSA_OK;
}

}  // namespace

// The prefill.  With `noalloc` it ignores workspace / workspace_bytes and uses the library's
// own array instead (never split-KV); otherwise the caller's workspace must hold the split
// plan's bytes.  With `check_only` it returns after every check (the tensor maps' encoding
// included), before anything is queued.
static bsa_status_t prefill_impl(const bsa_fp8_dims_t *dims, const void *q, const void *k_pages,
                                 const void *v_pages, const float *q_descale,
                                 const float *k_descale, const float *v_descale,
                                 const int *cu_seqlens_q, const int *seqused_kv,
                                 const int *block_table, const uint8_t *block_mask,
                                 const int *sparse_indices, const int *sparse_seq_len,
                                 float softmax_scale, float p_scale, void *out_bf16,
                                 float *lse_f32, void *workspace, size_t workspace_bytes,
                                 int *dev_status, void *stream, bool noalloc,
                                 bool check_only = false) {
  bsa_status_t st = validate_dims(dims);
  if (st != BSA_OK) return st;
  if (block_mask && sparse_indices) return BSA_ERR_INVALID_ARGUMENT;
  if (sparse_indices && !sparse_seq_len) return BSA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(softmax_scale)) return BSA_ERR_INVALID_ARGUMENT;
  if (std::isnan(p_scale) || std::isinf(p_scale)) return BSA_ERR_INVALID_ARGUMENT;
  if (p_scale <= 0.f) p_scale = 256.f;
  Params p = make_params(dims);
  const long long ntasks = (long long)p.B * p.N1 * p.Qb;
  if (ntasks == 0 || p.T == 0) return BSA_OK;
  if (!q || !k_pages || !v_pages || !q_descale || !k_descale || !v_descale || !cu_seqlens_q ||
      !block_table || !out_bf16)
    return BSA_ERR_INVALID_ARGUMENT;
  if (p.num_pages < 1 || p.L < 1) return BSA_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) ||
      (p.k_per_token && !aligned16(k_descale)) || !aligned16(out_bf16) ||
      (reinterpret_cast<uintptr_t>(lse_f32) & 3u) != 0)
    return BSA_ERR_INVALID_ARGUMENT;
  if (!noalloc && (!workspace || workspace_bytes < WORKSPACE_BYTES ||
                   (reinterpret_cast<uintptr_t>(workspace) & 3u) != 0))
    return BSA_ERR_WORKSPACE;
  // 256-wide macro blocks (two list tiles per online-softmax step) run their own kernel
  const bool wide = dims->tiles_per_step == 2;
  const size_t smem = wide ? attn_wide::smem_bytes(p.Kb) : attn::smem_bytes(p.Kb);
  int num_sms = 0, per_sm = 1;
  st = check_device(smem, &num_sms, &per_sm, wide);
  if (st != BSA_OK) return st;
  if (noalloc) {
    // the library's own array, looked up only once every argument has been checked
    st = noalloc_scratch(&workspace);
    if (st != BSA_OK) return st;
    workspace_bytes = NOALLOC_SCRATCH_BYTES;
  }
  // the array-backed entry point never splits: its array holds the item counter only; nor do
  // macro blocks (a slice boundary would cut a pair)
  const SplitPlan plan = plan_splits(p, num_sms, !noalloc && !wide);
  if (workspace_bytes < plan.bytes ||
      (plan.splits > 1 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
    return BSA_ERR_WORKSPACE;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.splits = plan.splits;
  if (plan.splits > 1) {
    p.row_cnt = reinterpret_cast<int *>(ws + plan.off_cnt);
    p.part_ml = reinterpret_cast<float *>(ws + plan.off_ml);
    p.part_o = reinterpret_cast<float *>(ws + plan.off_o);
  }

  p.q_descale = q_descale;
  p.k_descale = k_descale;
  p.v_descale = v_descale;
  p.cu_seqlens_q = cu_seqlens_q;
  p.seqused_kv = seqused_kv;
  p.block_table = block_table;
  p.block_mask = block_mask;
  p.sparse_indices = sparse_indices;
  p.sparse_seq_len = sparse_seq_len;
  p.out = static_cast<__nv_bfloat16 *>(out_bf16);
  p.lse = lse_f32;
  p.dev_status = dev_status;
  p.task_counter = static_cast<int *>(workspace);
  p.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);
  p.log2_pscale = (float)std::log2((double)p_scale);
  p.ln_pscale = (float)std::log((double)p_scale);

  // Tensor maps, innermost dimension first.  Either layout puts one 128-token Q box of a head,
  // or one page of a KV head, into shared memory as consecutive 128-byte rows.
  CUtensorMap tq, tk, tv;
  if (!p.q_ntd) {  // [T, N1, 128]: dims (d, head, token), box (128, 1, 128)
    cuuint64_t gd[3] = {HEAD_DIM, (cuuint64_t)p.N1, (cuuint64_t)p.T};
    cuuint64_t gs[2] = {HEAD_DIM, (cuuint64_t)p.N1 * HEAD_DIM};
    cuuint32_t box[3] = {HEAD_DIM, 1, TILE};
    if (!encode_map(&tq, q, 3, gd, gs, box)) return BSA_ERR_CUDA;
  } else {         // [N1, T, 128]: dims (d, token, head), box (128, 128, 1)
    cuuint64_t gd[3] = {HEAD_DIM, (cuuint64_t)p.T, (cuuint64_t)p.N1};
    cuuint64_t gs[2] = {HEAD_DIM, (cuuint64_t)p.T * HEAD_DIM};
    cuuint32_t box[3] = {HEAD_DIM, TILE, 1};
    if (!encode_map(&tq, q, 3, gd, gs, box)) return BSA_ERR_CUDA;
  }
  if (!p.kv_nhd) {  // [P, N2, ps, 128]: dims (d, slot, head, page), box (128, ps, 1, 1)
    cuuint64_t gd[4] = {HEAD_DIM, (cuuint64_t)p.ps, (cuuint64_t)p.N2, (cuuint64_t)p.num_pages};
    cuuint64_t gs[3] = {HEAD_DIM, (cuuint64_t)p.ps * HEAD_DIM,
                        (cuuint64_t)p.N2 * p.ps * HEAD_DIM};
    cuuint32_t box[4] = {HEAD_DIM, (cuuint32_t)p.ps, 1, 1};
    if (!encode_map(&tk, k_pages, 4, gd, gs, box)) return BSA_ERR_CUDA;
    if (!encode_map(&tv, v_pages, 4, gd, gs, box)) return BSA_ERR_CUDA;
  } else {          // [P, ps, N2, 128]: dims (d, head, slot, page), box (128, 1, ps, 1)
    cuuint64_t gd[4] = {HEAD_DIM, (cuuint64_t)p.N2, (cuuint64_t)p.ps, (cuuint64_t)p.num_pages};
    cuuint64_t gs[3] = {HEAD_DIM, (cuuint64_t)p.N2 * HEAD_DIM,
                        (cuuint64_t)p.ps * p.N2 * HEAD_DIM};
    cuuint32_t box[4] = {HEAD_DIM, 1, (cuuint32_t)p.ps, 1};
    if (!encode_map(&tk, k_pages, 4, gd, gs, box)) return BSA_ERR_CUDA;
    if (!encode_map(&tv, v_pages, 4, gd, gs, box)) return BSA_ERR_CUDA;
  }
  if (check_only) return BSA_OK;  // every check done, the tensor maps included
  // persistent grid: one CTA per SM (two pipelines each)
  const long long items = ntasks * plan.splits;
  const long long grid = std::min<long long>(items, (long long)per_sm * num_sms);
  // the item counter, and with split-KV the per-row completion counters, start at zero
  const size_t zero_bytes = plan.splits > 1 ? plan.off_ml : sizeof(int);
  if (cudaMemsetAsync(workspace, 0, zero_bytes, (cudaStream_t)stream) != cudaSuccess)
    return BSA_ERR_CUDA;
  if (wide)
    attn_wide::bsa_attention_wide_kernel<<<(unsigned)grid, attn_wide::NTHREADS, smem,
                                           (cudaStream_t)stream>>>(p, tq, tk, tv);
  else
    attn::bsa_attention_kernel<<<(unsigned)grid, attn::NTHREADS, smem, (cudaStream_t)stream>>>(
        p, tq, tk, tv);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

extern "C" bsa_status_t bsa_fp8_prefill(const bsa_fp8_dims_t *dims, const void *q,
                                        const void *k_pages, const void *v_pages,
                                        const float *q_descale, const float *k_descale,
                                        const float *v_descale, const int *cu_seqlens_q,
                                        const int *seqused_kv, const int *block_table,
                                        const uint8_t *block_mask, const int *sparse_indices,
                                        const int *sparse_seq_len, float softmax_scale,
                                        float p_scale, void *out_bf16, float *lse_f32,
                                        void *workspace, size_t workspace_bytes,
                                        int *dev_status, void *stream) {
  return prefill_impl(dims, q, k_pages, v_pages, q_descale, k_descale, v_descale, cu_seqlens_q,
                      seqused_kv, block_table, block_mask, sparse_indices, sparse_seq_len,
                      softmax_scale, p_scale, out_bf16, lse_f32, workspace, workspace_bytes,
                      dev_status, stream, false);
}

extern "C" bsa_status_t bsa_fp8_prefill_host(const bsa_fp8_dims_t *dims,
                                             const bsa_fp8_tensors_t *host,
                                             const bsa_fp8_tensors_t *dev, float softmax_scale,
                                             float p_scale, void *workspace,
                                             size_t workspace_bytes, int *dev_status,
                                             void *stream) {
  if (!host || !dev) return BSA_ERR_INVALID_ARGUMENT;
  bsa_status_t st = validate_dims(dims);
  if (st != BSA_OK) return st;
  const Params p = make_params(dims);
  // an empty problem queues nothing, as bsa_fp8_prefill launches nothing for it
  const bool empty = (long long)p.B * p.N1 * p.Qb == 0 || p.T == 0;
  // every tensor of the device set has its host counterpart, and the reverse
  if (!empty && (!host->q || !host->k_pages || !host->v_pages || !host->q_descale ||
                 !host->k_descale || !host->v_descale || !host->cu_seqlens_q ||
                 !host->block_table || !host->out_bf16))
    return BSA_ERR_INVALID_ARGUMENT;
  if (!empty && (!host->seqused_kv != !dev->seqused_kv || !host->block_mask != !dev->block_mask ||
                 !host->sparse_indices != !dev->sparse_indices ||
                 !host->sparse_seq_len != !dev->sparse_seq_len || !host->lse_f32 != !dev->lse_f32))
    return BSA_ERR_INVALID_ARGUMENT;
  const auto run = [&](bool check_only) {
    return prefill_impl(dims, dev->q, dev->k_pages, dev->v_pages, dev->q_descale,
                        dev->k_descale, dev->v_descale, dev->cu_seqlens_q, dev->seqused_kv,
                        dev->block_table, dev->block_mask, dev->sparse_indices,
                        dev->sparse_seq_len, softmax_scale, p_scale, dev->out_bf16,
                        dev->lse_f32, workspace, workspace_bytes, dev_status, stream, false,
                        check_only);
  };
  st = run(true);
  if (st != BSA_OK || empty) return st;

  const size_t T = (size_t)p.T, N1 = (size_t)p.N1, N2 = (size_t)p.N2, B = (size_t)p.B;
  const size_t cache_rows = (size_t)p.num_pages * N2 * (size_t)p.ps;
  const size_t tasks = B * N1 * (size_t)p.Qb;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto copy = [&](const void *dst, const void *src, size_t bytes, cudaMemcpyKind kind) {
    if (!src || bytes == 0) return true;
    if (cudaMemcpyAsync(const_cast<void *>(dst), src, bytes, kind, s) == cudaSuccess) return true;
    cudaGetLastError();  // leave no pending error behind
    return false;
  };
  const cudaMemcpyKind in = cudaMemcpyHostToDevice;
  const bool queued =
      copy(dev->q, host->q, T * N1 * HEAD_DIM, in) &&
      copy(dev->k_pages, host->k_pages, cache_rows * HEAD_DIM, in) &&
      copy(dev->v_pages, host->v_pages, cache_rows * HEAD_DIM, in) &&
      copy(dev->q_descale, host->q_descale, T * N1 * sizeof(float), in) &&
      copy(dev->k_descale, host->k_descale, (p.k_per_token ? cache_rows : 1) * sizeof(float),
           in) &&
      copy(dev->v_descale, host->v_descale, (p.v_per_head ? N2 : 1) * sizeof(float), in) &&
      copy(dev->cu_seqlens_q, host->cu_seqlens_q, (B + 1) * sizeof(int), in) &&
      copy(dev->seqused_kv, host->seqused_kv, B * sizeof(int), in) &&
      copy(dev->block_table, host->block_table, B * (size_t)p.L * sizeof(int), in) &&
      copy(dev->block_mask, host->block_mask, tasks * (size_t)p.Kb, in) &&
      copy(dev->sparse_indices, host->sparse_indices, tasks * (size_t)p.Kb * sizeof(int), in) &&
      copy(dev->sparse_seq_len, host->sparse_seq_len, tasks * sizeof(int), in);
  if (!queued) return BSA_ERR_CUDA;
  st = run(false);
  if (st != BSA_OK) return st;
  const cudaMemcpyKind out = cudaMemcpyDeviceToHost;
  if (!copy(host->out_bf16, dev->out_bf16, T * N1 * HEAD_DIM * 2, out) ||
      !copy(host->lse_f32, dev->lse_f32, N1 * T * sizeof(float), out))
    return BSA_ERR_CUDA;
  return BSA_OK;
}

// ------------------------------------------------------------------------------------------
// quantise step
// ------------------------------------------------------------------------------------------

namespace {

// grid for `rows` half-warp rows (two per half-warp step): enough blocks to cover them, at
// most as many as are resident at once
template <typename Kernel>
bsa_status_t quant_grid(Kernel kernel, long long rows, unsigned *grid) {
  int num_sms = 0, per_sm = 0;
  const bsa_status_t st = check_device(0, &num_sms);
  if (st != BSA_OK) return st;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, quant::THREADS, 0) !=
      cudaSuccess)
    return BSA_ERR_CUDA;
  const long long per_block = 2 * (quant::THREADS / 16);
  const long long need = (rows + per_block - 1) / per_block;
  *grid = (unsigned)std::max<long long>(
      1, std::min<long long>(need, (long long)std::max(per_sm, 1) * num_sms));
  return BSA_OK;
}

}  // namespace

static bsa_status_t quantize_rows_impl(const void *x_bf16, long long rows, void *codes_e4m3,
                                       float *descale, void *stream, bool ue8m0) {
  if (rows < 0) return BSA_ERR_INVALID_ARGUMENT;
  if (rows == 0) return BSA_OK;
  if (!x_bf16 || !codes_e4m3 || !descale || !aligned16(x_bf16) || !aligned16(codes_e4m3))
    return BSA_ERR_INVALID_ARGUMENT;
  unsigned grid = 0;
  const bsa_status_t st = quant_grid(quant::quantize_rows_kernel, rows, &grid);
  if (st != BSA_OK) return st;
  quant::quantize_rows_kernel<<<grid, quant::THREADS, 0, (cudaStream_t)stream>>>(
      static_cast<const uint4 *>(x_bf16), rows, static_cast<uint2 *>(codes_e4m3), descale,
      ue8m0);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

extern "C" bsa_status_t bsa_fp8_quantize_rows(const void *x_bf16, long long rows,
                                              void *codes_e4m3, float *descale, void *stream) {
  return quantize_rows_impl(x_bf16, rows, codes_e4m3, descale, stream, false);
}

extern "C" bsa_status_t bsa_fp8_quantize_rows_ue8m0(const void *x_bf16, long long rows,
                                                    void *codes_e4m3, float *descale,
                                                    void *stream) {
  return quantize_rows_impl(x_bf16, rows, codes_e4m3, descale, stream, true);
}

// The tokens' places come from the table or, with `slots`, from slot_map.
static bsa_status_t append_impl(const bsa_fp8_append_dims_t *d, bool slots, const void *k_new_bf16,
                                const void *v_new_bf16, const int *cu_seqlens_new,
                                const int *cache_seqlens, const int *block_table,
                                const int *slot_map, const float *k_scale, const float *v_scale,
                                void *k_pages, void *v_pages, float *k_descale, int *dev_status,
                                void *stream) {
  if (!d || d->D != HEAD_DIM || (d->page_size != 32 && d->page_size != 64) || d->B < 0 ||
      d->N2 < 1 || d->num_pages < 0 || d->max_pages_per_seq < 0 || d->total_new < 0)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->k_scale_kind != BSA_SCALE_PER_TOKEN_HEAD && d->k_scale_kind != BSA_SCALE_PER_TENSOR)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->v_scale_kind != BSA_SCALE_PER_HEAD && d->v_scale_kind != BSA_SCALE_PER_TENSOR)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->kv_layout != BSA_KV_HND && d->kv_layout != BSA_KV_NHD) return BSA_ERR_INVALID_ARGUMENT;
  if (d->k_descale_rule != BSA_DESCALE_AMAX && d->k_descale_rule != BSA_DESCALE_UE8M0)
    return BSA_ERR_INVALID_ARGUMENT;
  const long long rows = (long long)d->total_new * d->N2;
  if (rows == 0 || (!slots && d->B == 0)) return BSA_OK;
  const bool k_tok = d->k_scale_kind == BSA_SCALE_PER_TOKEN_HEAD;
  if (slots ? !slot_map : !cu_seqlens_new || !cache_seqlens || !block_table)
    return BSA_ERR_INVALID_ARGUMENT;
  if (!k_new_bf16 || !v_new_bf16 || !v_scale || !k_pages || !v_pages ||
      (k_tok ? !k_descale : !k_scale))
    return BSA_ERR_INVALID_ARGUMENT;
  if (!aligned16(k_new_bf16) || !aligned16(v_new_bf16) || !aligned16(k_pages) ||
      !aligned16(v_pages))
    return BSA_ERR_INVALID_ARGUMENT;
  unsigned grid = 0;
  const bsa_status_t st = quant_grid(quant::append_kv_kernel, rows, &grid);
  if (st != BSA_OK) return st;
  quant::AppendParams p;
  p.k_new = static_cast<const uint4 *>(k_new_bf16);
  p.v_new = static_cast<const uint4 *>(v_new_bf16);
  p.cu_new = cu_seqlens_new;
  p.cache_len = cache_seqlens;
  p.block_table = block_table;
  p.slot_map = slot_map;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_pages = static_cast<uint2 *>(k_pages);
  p.v_pages = static_cast<uint2 *>(v_pages);
  p.k_descale = k_descale;
  p.dev_status = dev_status;
  p.B = d->B;
  p.N2 = d->N2;
  p.ps = d->page_size;
  p.num_pages = d->num_pages;
  p.L = d->max_pages_per_seq;
  p.total_new = d->total_new;
  p.k_per_token = k_tok ? 1 : 0;
  p.v_per_head = d->v_scale_kind == BSA_SCALE_PER_HEAD ? 1 : 0;
  p.kv_nhd = d->kv_layout == BSA_KV_NHD ? 1 : 0;
  p.k_ue8m0 = d->k_descale_rule == BSA_DESCALE_UE8M0 ? 1 : 0;
  quant::append_kv_kernel<<<grid, quant::THREADS, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

extern "C" bsa_status_t bsa_fp8_append_kv(const bsa_fp8_append_dims_t *d, const void *k_new_bf16,
                                          const void *v_new_bf16, const int *cu_seqlens_new,
                                          const int *cache_seqlens, const int *block_table,
                                          const float *k_scale, const float *v_scale,
                                          void *k_pages, void *v_pages, float *k_descale,
                                          int *dev_status, void *stream) {
  return append_impl(d, false, k_new_bf16, v_new_bf16, cu_seqlens_new, cache_seqlens, block_table,
                     nullptr, k_scale, v_scale, k_pages, v_pages, k_descale, dev_status, stream);
}

extern "C" bsa_status_t bsa_fp8_append_kv_slots(const bsa_fp8_append_dims_t *d,
                                                const void *k_new_bf16, const void *v_new_bf16,
                                                const int *slot_map, const float *k_scale,
                                                const float *v_scale, void *k_pages,
                                                void *v_pages, float *k_descale, int *dev_status,
                                                void *stream) {
  return append_impl(d, true, k_new_bf16, v_new_bf16, nullptr, nullptr, nullptr, slot_map, k_scale,
                     v_scale, k_pages, v_pages, k_descale, dev_status, stream);
}

extern "C" bsa_status_t bsa_fp8_prefill_noalloc(
    const bsa_fp8_dims_t *dims, const void *q, const void *k_pages, const void *v_pages,
    const float *q_descale, const float *k_descale, const float *v_descale,
    const int *cu_seqlens_q, const int *seqused_kv, const int *block_table,
    const uint8_t *block_mask, const int *sparse_indices, const int *sparse_seq_len,
    float softmax_scale, float p_scale, void *out_bf16, float *lse_f32, int *dev_status,
    void *stream) {
  // every argument is checked as bsa_fp8_prefill checks it; the array is looked up after that
  return prefill_impl(dims, q, k_pages, v_pages, q_descale, k_descale, v_descale, cu_seqlens_q,
                      seqused_kv, block_table, block_mask, sparse_indices, sparse_seq_len,
                      softmax_scale, p_scale, out_bf16, lse_f32, nullptr, 0, dev_status, stream,
                      true);
}

// ------------------------------------------------------------------------------------------
// serving: decode, cache read-back, merge
// ------------------------------------------------------------------------------------------

namespace {

// byte strides of a page, a KV head and a slot inside the page pool
void pool_strides(int kv_layout, int N2, int page_size, int row, long long *page, long long *head,
                  long long *slot) {
  *page = (long long)N2 * page_size * row;
  *head = kv_layout == BSA_KV_NHD ? row : (long long)page_size * row;
  *slot = kv_layout == BSA_KV_NHD ? (long long)N2 * row : row;
}

bsa_status_t validate_decode(const bsa_fp8_decode_dims_t *d, bool fp4) {
  if (!d || d->D != HEAD_DIM || (d->page_size != 32 && d->page_size != 64))
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->B < 0 || d->N1 < 1 || d->N2 < 1 || d->N1 % d->N2 != 0 || d->N1 / d->N2 > 16)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->max_kv_len < 0 || d->num_pages < 0 || d->max_pages_per_seq < 0)
    return BSA_ERR_INVALID_ARGUMENT;
  if ((long long)d->max_pages_per_seq * d->page_size < d->max_kv_len)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->k_scale_kind != BSA_SCALE_PER_TENSOR &&
      d->k_scale_kind != (fp4 ? BSA_SCALE_PER_HEAD : BSA_SCALE_PER_TOKEN_HEAD))
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->v_scale_kind != BSA_SCALE_PER_TENSOR && d->v_scale_kind != BSA_SCALE_PER_HEAD)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->kv_layout != BSA_KV_HND && d->kv_layout != BSA_KV_NHD) return BSA_ERR_INVALID_ARGUMENT;
  if (d->q_type != BSA_QTYPE_BF16 && d->q_type != BSA_QTYPE_E4M3) return BSA_ERR_INVALID_ARGUMENT;
  if (d->q_stride < (long long)d->N1 * HEAD_DIM ||
      d->q_stride % (d->q_type == BSA_QTYPE_E4M3 ? 16 : 8) != 0)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->sparse != 0 && d->sparse != 1) return BSA_ERR_INVALID_ARGUMENT;
  const long long kb = cdiv(d->max_kv_len, TILE);
  if (kb > KB_MAX) return BSA_ERR_UNSUPPORTED;
  // rows of a 4-bit pool are counted in 32 bits
  if (fp4 && (long long)d->num_pages * d->N2 * d->page_size > 0xffffffffLL)
    return BSA_ERR_UNSUPPORTED;
  // tile counts and grid sizes are int
  if ((long long)d->B * d->N1 > (1LL << 30) || (long long)d->B * d->N2 * (kb + 1) > (1LL << 30))
    return BSA_ERR_UNSUPPORTED;
  return BSA_OK;
}

// Grid of the decode kernel and where its workspace arrays lie.  The grid depends on the SM count
// and an upper bound of the tiles only: the host does not know the lengths.
struct DecodePlan {
  int grid = 0;
  bool whole = false;  // runs are whole tasks: nothing is joined
  size_t off_o = 0, off_counts = 0, off_tiles = 0, bytes = 0;
};

DecodePlan plan_decode(const bsa_fp8_decode_dims_t *d, int num_sms, bool fp4) {
  DecodePlan plan;
  const int ctas = fp4 ? decode4::CTAS_PER_SM : decode::CTAS_PER_SM;
  const long long tasks = (long long)d->B * d->N2, kb = cdiv(d->max_kv_len, TILE);
  const long long resident = (long long)ctas * std::max(num_sms, 1);
  // One CTA goes through up to four tiles about as fast as a cut task's are joined (one sequence of
  // 300 tokens 5.2 us against 5.8, 16 of 512 6.2 against 8.9); with eight, or with more
  // tasks than CTAs, an even cut is faster (64 of 300 11.9 us against 12.4).
  plan.whole = kb <= decode::WHOLE_TILES && tasks <= resident;
  // (a task without a tile is one piece of work all the same: 512 idle ones 5 us, on one CTA 700)
  plan.grid = (int)std::max<long long>(
      1, std::min<long long>(resident, plan.whole ? tasks : tasks * std::max(kb, 1LL)));
  const size_t slots = plan.whole ? 0 : 2 * (size_t)plan.grid;
  plan.off_o = round256(slots * decode::MAX_G * sizeof(float2));
  plan.off_counts = plan.off_o + slots * (size_t)(d->N1 / d->N2) * HEAD_DIM * sizeof(float);
  plan.off_tiles = plan.off_counts + (d->sparse ? round256((size_t)tasks * sizeof(int2)) : 0);
  plan.bytes = std::max(WORKSPACE_BYTES, plan.off_tiles + (d->sparse ? (size_t)tasks * (size_t)kb *
                                                                           sizeof(uint32_t)
                                                                     : 0));
  return plan;
}

// Enables the decode kernels' dynamic shared memory on the current device, once.
bsa_status_t enable_decode() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_devices_mu);
  DeviceInfo &di = g_devices[dev];  // check_device has bounded dev
  if (di.decode_attr) return BSA_OK;
  const auto enable = [](const void *kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) ==
           cudaSuccess;
  };
  const auto enable_all = [&](auto params) {  // the kernels that take such parameters
    using P = decltype(params);
    return enable((const void *)decode::decode_kernel<1, false, P>, decode::SMEM_BYTES) &&
           enable((const void *)decode::decode_kernel<2, false, P>, decode::SMEM_BYTES) &&
           enable((const void *)decode::decode_kernel<1, true, P>, decode::SMEM_BYTES) &&
           enable((const void *)decode::decode_kernel<2, true, P>, decode::SMEM_BYTES) &&
           enable((const void *)decode4::decode_kernel<1, false, P>, decode4::SMEM_BYTES) &&
           enable((const void *)decode4::decode_kernel<2, false, P>, decode4::SMEM_BYTES) &&
           enable((const void *)decode4::decode_kernel<1, true, P>, decode4::SMEM_BYTES) &&
           enable((const void *)decode4::decode_kernel<2, true, P>, decode4::SMEM_BYTES);
  };
  if (!enable_all(decode::Params()) || !enable_all(decode::PackedParams())) {
    (void)cudaGetLastError();  // leave no pending error behind
    return BSA_ERR_CUDA;
  }
  di.decode_attr = true;
  return BSA_OK;
}

// A launch that may begin while the kernel before it on the stream runs; it waits for that
// kernel's writes itself (griddepcontrol.wait).
template <bool CLUSTER = false, typename... Args>  // CLUSTER: the grid is one cluster
bool launch_dependent(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, void *stream,
                      const Args &...args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = grid.x;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER && grid.x > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return true;
  (void)cudaGetLastError();  // leave no pending error behind
  return false;
}

}  // namespace

static size_t decode_workspace_size(const bsa_fp8_decode_dims_t *dims, bool fp4) {
  if (validate_decode(dims, fp4) != BSA_OK) return 0;
  int num_sms = 0;
  if (check_device(0, &num_sms) != BSA_OK) return WORKSPACE_BYTES;
  return plan_decode(dims, num_sms, fp4).bytes;
}

extern "C" size_t bsa_fp8_decode_workspace_size(const bsa_fp8_decode_dims_t *dims) {
  return decode_workspace_size(dims, false);
}

extern "C" size_t bsa_fp4_decode_workspace_size(const bsa_fp8_decode_dims_t *dims) {
  return decode_workspace_size(dims, true);
}

// The launches of a decode: the tile lists where there are some, the attention, the join.
template <bool FP4, typename P>
static bsa_status_t launch_decode(const P &p, const DecodePlan &plan, bool lists, int num_sms,
                                  void *stream) {
  const bool wide = p.G > 8;  // two blocks of eight query heads per KV head
  if (lists && !launch_dependent(p.block_mask ? decode::plan_kernel<true, P>
                                              : decode::plan_kernel<false, P>,
                                 dim3((unsigned)(p.B * p.N2)),
                                 decode::PLAN_THREADS, (size_t)p.Kb * sizeof(uint32_t), stream, p))
    return BSA_ERR_CUDA;
  if constexpr (FP4) {
    const auto kernel =
        lists ? (wide ? decode4::decode_kernel<2, true, P> : decode4::decode_kernel<1, true, P>)
              : (wide ? decode4::decode_kernel<2, false, P> : decode4::decode_kernel<1, false, P>);
    if (!launch_dependent(kernel, dim3((unsigned)plan.grid), decode4::THREADS,
                          decode4::SMEM_BYTES, stream, p))
      return BSA_ERR_CUDA;
  } else {
    // Tensor maps of the pools: a box is a warp's 32 slots of one page and head, in shared memory
    // consecutive 128-byte rows in either layout.  L2 fetches no more than those rows: in NHD pages
    // the next 128 bytes are another head's, wanted at another time (16 sequences of 8K tokens x 8
    // heads: 65.9 us with 256-byte promotion, 50.3 without; HND 47.4 either way).
    CUtensorMap tk, tv;
    memset(&tk, 0, sizeof(tk));
    memset(&tv, 0, sizeof(tv));
    if (p.Kb > 0) {
      const cuuint64_t H = (cuuint64_t)p.N2, S = (cuuint64_t)p.ps;
      const bool nhd = p.kv_nhd != 0;
      const cuuint64_t gd[4] = {HEAD_DIM, nhd ? H : S, nhd ? S : H, (cuuint64_t)p.num_pages};
      const cuuint64_t gs[3] = {HEAD_DIM, gd[1] * HEAD_DIM, H * S * HEAD_DIM};
      const cuuint32_t box[4] = {HEAD_DIM, nhd ? 1u : (cuuint32_t)decode::TOK,
                                 nhd ? (cuuint32_t)decode::TOK : 1u, 1};
      const CUtensorMapL2promotion row = CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
      if (!encode_map(&tk, p.k_pages, 4, gd, gs, box, row) ||
          !encode_map(&tv, p.v_pages, 4, gd, gs, box, row))
        return BSA_ERR_CUDA;
    }
    const auto kernel =
        lists ? (wide ? decode::decode_kernel<2, true, P> : decode::decode_kernel<1, true, P>)
              : (wide ? decode::decode_kernel<2, false, P> : decode::decode_kernel<1, false, P>);
    if (!launch_dependent(kernel, dim3((unsigned)plan.grid), decode::THREADS, decode::SMEM_BYTES,
                          stream, p, tk, tv))
      return BSA_ERR_CUDA;
  }
  if (plan.whole || p.Kb <= 1) return BSA_OK;  // no task is cut
  // The join, 62 registers.  Beside two CTAs of the kernels for up to eight heads (220 registers,
  // with lists 214) an SM has room for one block of four warps or two of two; the kernels for more
  // heads (255) leave none.  Blocks that find no room start as attention CTAs end.  The more heads and
  // tasks there are, the fewer warps a block has.
  const long long tasks = (long long)p.B * p.N2;
  const bool by_task = tasks < plan.grid;
  const int warps = !by_task ? 4 : tasks * p.G <= num_sms ? 8 : tasks * p.G <= 2 * num_sms ? 4 : 2;
  if (!launch_dependent(lists ? decode::join_kernel<true, P> : decode::join_kernel<false, P>,
                        by_task ? dim3((unsigned)tasks, (unsigned)p.G) : dim3((unsigned)plan.grid),
                        warps * 32, 0, stream, p, by_task, plan.grid))
    return BSA_ERR_CUDA;
  return BSA_OK;
}

// Both cache formats' decode; k_scales and v_scales are the block scales of 4-bit pages.  With
// `packed` the queries are total_q rows, found by cu_seqlens_q; without, a row a sequence.
template <bool FP4>
static bsa_status_t decode_impl(const bsa_fp8_decode_dims_t *d, bool packed, int total_q,
                                const int *cu_seqlens_q, const void *q, const float *q_descale,
                                const void *k_pages, const void *v_pages, const void *k_scales,
                                const void *v_scales,
                                const float *k_descale, const float *v_descale,
                                const int *seqused_kv, const int *block_table,
                                const uint8_t *block_mask, const int *sparse_indices,
                                const int *sparse_seq_len, float softmax_scale, void *out_bf16,
                                float *lse_f32, void *workspace, size_t workspace_bytes,
                                int *dev_status, void *stream) {
  bsa_status_t st = validate_decode(d, FP4);
  if (st != BSA_OK) return st;
  if (block_mask && sparse_indices) return BSA_ERR_INVALID_ARGUMENT;
  if (sparse_indices && !sparse_seq_len) return BSA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(softmax_scale)) return BSA_ERR_INVALID_ARGUMENT;
  if (packed && total_q < 0) return BSA_ERR_INVALID_ARGUMENT;
  if (packed ? total_q == 0 : d->B == 0) return BSA_OK;
  if (packed && !cu_seqlens_q) return BSA_ERR_INVALID_ARGUMENT;
  // a batch of empty sequences only (max_kv_len = 0) has no cache and no tiles to name
  const bool none = d->max_kv_len == 0 || d->B == 0;
  if (!none && (d->sparse != 0) != (block_mask || sparse_indices)) return BSA_ERR_INVALID_ARGUMENT;
  const bool k_tok = d->k_scale_kind == BSA_SCALE_PER_TOKEN_HEAD;
  const bool e4m3 = d->q_type == BSA_QTYPE_E4M3;
  if (!q || (d->B && !seqused_kv) || !out_bf16 || e4m3 != (q_descale != nullptr))
    return BSA_ERR_INVALID_ARGUMENT;
  if (!none && (!k_pages || !v_pages || !k_descale || !v_descale || !block_table ||
                d->num_pages < 1))
    return BSA_ERR_INVALID_ARGUMENT;
  if (FP4 && ((!none && (!k_scales || !v_scales)) || !aligned16(k_scales) || !aligned16(v_scales)))
    return BSA_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) ||
      (k_tok && !aligned16(k_descale)) || !aligned16(out_bf16) ||
      (reinterpret_cast<uintptr_t>(lse_f32) & 3u) != 0)
    return BSA_ERR_INVALID_ARGUMENT;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return BSA_ERR_WORKSPACE;
  int num_sms = 0;
  st = check_device(0, &num_sms);
  if (st != BSA_OK) return st;
  const DecodePlan plan = plan_decode(d, num_sms, FP4);
  if (workspace_bytes < plan.bytes) return BSA_ERR_WORKSPACE;
  st = enable_decode();
  if (st != BSA_OK) return st;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  decode::PackedParams p;
  memset(&p, 0, sizeof(p));
  p.q = q;
  p.q_descale = q_descale;
  p.k_pages = static_cast<const uint8_t *>(k_pages);
  p.v_pages = static_cast<const uint8_t *>(v_pages);
  p.k_scales = static_cast<const uint8_t *>(k_scales);
  p.v_scales = static_cast<const uint8_t *>(v_scales);
  p.k_descale = k_descale;
  p.v_descale = v_descale;
  p.seqused_kv = seqused_kv;
  p.block_table = block_table;
  p.block_mask = block_mask;
  p.sparse_indices = sparse_indices;
  p.sparse_seq_len = sparse_seq_len;
  p.out = static_cast<__nv_bfloat16 *>(out_bf16);
  p.lse = lse_f32;
  p.dev_status = dev_status;
  p.cu_q = cu_seqlens_q;
  p.rows = total_q;
  p.q_stride = d->q_stride;
  p.kv_nhd = d->kv_layout == BSA_KV_NHD;
  p.whole = plan.whole;
  const unsigned long long lim = g_wait_limit_ns.load(std::memory_order_relaxed);
  p.wait_limit_ns = lim ? lim : WAIT_LIMIT_NS;
  p.B = d->B;
  p.N1 = d->N1;
  p.N2 = d->N2;
  p.G = d->N1 / d->N2;
  p.ps = d->page_size;
  p.num_pages = d->num_pages;
  p.L = d->max_pages_per_seq;
  p.Kb = cdiv(d->max_kv_len, TILE);
  p.max_kv_len = d->max_kv_len;
  p.q_e4m3 = e4m3;
  p.k_per_token = k_tok;
  p.k_per_head = d->k_scale_kind == BSA_SCALE_PER_HEAD;
  p.v_per_head = d->v_scale_kind == BSA_SCALE_PER_HEAD;
  p.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);
  p.ps_shift = d->page_size == 64 ? 6 : 5;
  p.part_ml = reinterpret_cast<float2 *>(ws);
  p.part_o = reinterpret_cast<float *>(ws + plan.off_o);
  p.counts = reinterpret_cast<int2 *>(ws + plan.off_counts);
  p.tiles = reinterpret_cast<uint32_t *>(ws + plan.off_tiles);
  if (d->B == 0)
    return launch_dependent(decode::clear_kernel, dim3((unsigned)std::min(total_q, num_sms)),
                            decode::THREADS, 0, stream, p)
               ? BSA_OK
               : BSA_ERR_CUDA;
  const bool lists = d->sparse && !none;
  return packed ? launch_decode<FP4>(p, plan, lists, num_sms, stream)
                : launch_decode<FP4>(static_cast<const decode::Params &>(p), plan, lists,
                                     num_sms, stream);
}

extern "C" bsa_status_t bsa_fp8_decode(const bsa_fp8_decode_dims_t *d, const void *q,
                                       const float *q_descale, const void *k_pages,
                                       const void *v_pages, const float *k_descale,
                                       const float *v_descale, const int *seqused_kv,
                                       const int *block_table, const uint8_t *block_mask,
                                       const int *sparse_indices, const int *sparse_seq_len,
                                       float softmax_scale, void *out_bf16, float *lse_f32,
                                       void *workspace, size_t workspace_bytes, int *dev_status,
                                       void *stream) {
  return decode_impl<false>(d, false, 0, nullptr, q, q_descale, k_pages, v_pages, nullptr, nullptr,
                            k_descale, v_descale, seqused_kv, block_table, block_mask,
                            sparse_indices, sparse_seq_len, softmax_scale, out_bf16, lse_f32,
                            workspace, workspace_bytes, dev_status, stream);
}

extern "C" bsa_status_t bsa_fp8_decode_rows(
    const bsa_fp8_decode_dims_t *d, int total_q, const int *cu_seqlens_q, const void *q,
    const float *q_descale, const void *k_pages, const void *v_pages, const float *k_descale,
    const float *v_descale, const int *seqused_kv, const int *block_table,
    const uint8_t *block_mask, const int *sparse_indices, const int *sparse_seq_len,
    float softmax_scale, void *out_bf16, float *lse_f32, void *workspace, size_t workspace_bytes,
    int *dev_status, void *stream) {
  return decode_impl<false>(d, true, total_q, cu_seqlens_q, q, q_descale, k_pages, v_pages, nullptr,
                            nullptr, k_descale, v_descale, seqused_kv, block_table, block_mask,
                            sparse_indices, sparse_seq_len, softmax_scale, out_bf16, lse_f32,
                            workspace, workspace_bytes, dev_status, stream);
}

extern "C" bsa_status_t bsa_fp4_decode(
    const bsa_fp8_decode_dims_t *d, const void *q, const float *q_descale, const void *k_pages,
    const void *v_pages, const void *k_scales, const void *v_scales, const float *k_descale,
    const float *v_descale, const int *seqused_kv, const int *block_table,
    const uint8_t *block_mask, const int *sparse_indices, const int *sparse_seq_len,
    float softmax_scale, void *out_bf16, float *lse_f32, void *workspace, size_t workspace_bytes,
    int *dev_status, void *stream) {
  return decode_impl<true>(d, false, 0, nullptr, q, q_descale, k_pages, v_pages, k_scales, v_scales,
                           k_descale, v_descale, seqused_kv, block_table, block_mask,
                           sparse_indices, sparse_seq_len, softmax_scale, out_bf16, lse_f32,
                           workspace, workspace_bytes, dev_status, stream);
}

extern "C" bsa_status_t bsa_fp4_decode_rows(
    const bsa_fp8_decode_dims_t *d, int total_q, const int *cu_seqlens_q, const void *q,
    const float *q_descale, const void *k_pages, const void *v_pages, const void *k_scales,
    const void *v_scales, const float *k_descale, const float *v_descale, const int *seqused_kv,
    const int *block_table, const uint8_t *block_mask, const int *sparse_indices,
    const int *sparse_seq_len, float softmax_scale, void *out_bf16, float *lse_f32, void *workspace,
    size_t workspace_bytes, int *dev_status, void *stream) {
  return decode_impl<true>(d, true, total_q, cu_seqlens_q, q, q_descale, k_pages, v_pages, k_scales,
                           v_scales, k_descale, v_descale, seqused_kv, block_table, block_mask,
                           sparse_indices, sparse_seq_len, softmax_scale, out_bf16, lse_f32,
                           workspace, workspace_bytes, dev_status, stream);
}

template <bool FP4>
static bsa_status_t gather_impl(const bsa_fp8_gather_dims_t *d, const void *k_pages,
                                const void *v_pages, const void *k_scales, const void *v_scales,
                                const float *k_descale, const float *v_descale,
                                const int *cu_seqlens, const int *cache_starts,
                                const int *block_table, void *k_out, void *v_out, int *dev_status,
                                void *stream) {
  if (!d || d->D != HEAD_DIM || (d->page_size != 32 && d->page_size != 64) || d->B < 0 ||
      d->N2 < 1 || d->num_pages < 0 || d->max_pages_per_seq < 0 || d->total < 0)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->k_scale_kind != (FP4 ? BSA_SCALE_PER_HEAD : BSA_SCALE_PER_TOKEN_HEAD) &&
      d->k_scale_kind != BSA_SCALE_PER_TENSOR)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->v_scale_kind != BSA_SCALE_PER_HEAD && d->v_scale_kind != BSA_SCALE_PER_TENSOR)
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->kv_layout != BSA_KV_HND && d->kv_layout != BSA_KV_NHD) return BSA_ERR_INVALID_ARGUMENT;
  if (d->out_type != BSA_OUT_BF16 && d->out_type != BSA_OUT_FP32) return BSA_ERR_INVALID_ARGUMENT;
  if (d->total == 0 || d->B == 0) return BSA_OK;
  if ((!k_out && !v_out) || !cu_seqlens || !block_table) return BSA_ERR_INVALID_ARGUMENT;
  if ((k_out && (!k_pages || !k_descale)) || (v_out && (!v_pages || !v_descale)))
    return BSA_ERR_INVALID_ARGUMENT;
  if (FP4 && ((k_out && !k_scales) || (v_out && !v_scales))) return BSA_ERR_INVALID_ARGUMENT;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned16(k_pages) || !aligned16(v_pages))
    return BSA_ERR_INVALID_ARGUMENT;
  int num_sms = 0;
  const bsa_status_t st = check_device(0, &num_sms);
  if (st != BSA_OK) return st;
  gather::Params p;
  memset(&p, 0, sizeof(p));
  p.k_pages = static_cast<const uint8_t *>(k_pages);
  p.v_pages = static_cast<const uint8_t *>(v_pages);
  p.k_scales = static_cast<const uint8_t *>(k_scales);
  p.v_scales = static_cast<const uint8_t *>(v_scales);
  p.k_descale = k_descale;
  p.v_descale = v_descale;
  p.cu_seqlens = cu_seqlens;
  p.cache_starts = cache_starts;
  p.block_table = block_table;
  p.k_out = k_out;
  p.v_out = v_out;
  p.dev_status = dev_status;
  pool_strides(d->kv_layout, d->N2, d->page_size, FP4 ? fp4::ROW_BYTES : HEAD_DIM, &p.page_bytes,
               &p.head_bytes, &p.slot_bytes);
  p.B = d->B;
  p.N2 = d->N2;
  p.ps = d->page_size;
  p.num_pages = d->num_pages;
  p.L = d->max_pages_per_seq;
  p.total = d->total;
  p.k_per_token = d->k_scale_kind == BSA_SCALE_PER_TOKEN_HEAD;
  p.k_per_head = d->k_scale_kind == BSA_SCALE_PER_HEAD;
  p.v_per_head = d->v_scale_kind == BSA_SCALE_PER_HEAD;
  // a block's tokens: as many as leave every SM four rounds of its four resident blocks, so that a
  // lookup serves many rows and the last round is short (8 sequences of 100 to 5000 tokens
  // in fp32: 45 us with one round, 37 with two, 35 with four, 37 with eight)
  p.tokens = gather::MAX_TOKENS;
  while (p.tokens > 1 && cdiv(d->total, p.tokens) < 16 * num_sms) p.tokens /= 2;
  const unsigned grid = (unsigned)cdiv(d->total, p.tokens);
  const bool f32 = d->out_type == BSA_OUT_FP32;
  const auto kernel = FP4 ? (f32 ? gather::gather_fp4_kernel<true> : gather::gather_fp4_kernel<false>)
                          : (f32 ? gather::gather_kernel<true> : gather::gather_kernel<false>);
  kernel<<<grid, gather::THREADS, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

extern "C" bsa_status_t bsa_fp8_gather_kv(const bsa_fp8_gather_dims_t *d, const void *k_pages,
                                          const void *v_pages, const float *k_descale,
                                          const float *v_descale, const int *cu_seqlens,
                                          const int *cache_starts, const int *block_table,
                                          void *k_out, void *v_out, int *dev_status,
                                          void *stream) {
  return gather_impl<false>(d, k_pages, v_pages, nullptr, nullptr, k_descale, v_descale,
                            cu_seqlens, cache_starts, block_table, k_out, v_out, dev_status,
                            stream);
}

extern "C" bsa_status_t bsa_fp4_gather_kv(const bsa_fp8_gather_dims_t *d, const void *k_pages,
                                          const void *v_pages, const void *k_scales,
                                          const void *v_scales, const float *k_descale,
                                          const float *v_descale, const int *cu_seqlens,
                                          const int *cache_starts, const int *block_table,
                                          void *k_out, void *v_out, int *dev_status,
                                          void *stream) {
  return gather_impl<true>(d, k_pages, v_pages, k_scales, v_scales, k_descale, v_descale,
                           cu_seqlens, cache_starts, block_table, k_out, v_out, dev_status,
                           stream);
}

static bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

extern "C" bsa_status_t bsa_fp8_merge_states(int count, const void *const *outs,
                                             const float *const *lses, int T, int N1,
                                             void *out_bf16, float *lse_f32, void *stream) {
  if (count < 1 || count > BSA_MAX_MERGE || !outs || !lses || T < 0 || N1 < 1 ||
      (long long)T * N1 > 0x7fffffffLL)
    return BSA_ERR_INVALID_ARGUMENT;
  if (T == 0) return BSA_OK;
  if (!out_bf16 || !aligned16(out_bf16) || (reinterpret_cast<uintptr_t>(lse_f32) & 3u) != 0)
    return BSA_ERR_INVALID_ARGUMENT;
  merge::Params p;
  memset(&p, 0, sizeof(p));
  for (int i = 0; i < count; ++i) {
    if (!outs[i] || !lses[i] || !aligned16(outs[i]) ||
        (reinterpret_cast<uintptr_t>(lses[i]) & 3u) != 0)
      return BSA_ERR_INVALID_ARGUMENT;
    p.outs[i] = static_cast<const __nv_bfloat16 *>(outs[i]);
    p.lses[i] = lses[i];
  }
  // an element is written once its own sources have been read, not its neighbours'
  const size_t nz = (size_t)T * N1 * 4, nl = lse_f32 ? nz : 0, no = (size_t)T * N1 * HEAD_DIM * 2;
  if (overlap(out_bf16, no, lse_f32, nl)) return BSA_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < count; ++i)
    if ((out_bf16 != outs[i] && overlap(out_bf16, no, outs[i], no)) ||
        (lse_f32 != lses[i] && overlap(lse_f32, nl, lses[i], nz)) ||
        overlap(out_bf16, no, lses[i], nz) || overlap(lse_f32, nl, outs[i], no))
      return BSA_ERR_INVALID_ARGUMENT;
  int num_sms = 0;
  const bsa_status_t st = check_device(0, &num_sms);
  if (st != BSA_OK) return st;
  p.out = static_cast<__nv_bfloat16 *>(out_bf16);
  p.lse = lse_f32;
  p.T = T;
  p.N1 = N1;
  // tiles of up to 32 heads and 256 rows, smaller ones while they do not give every SM sixteen
  // (8192 tokens x 32 heads in two parts: 36.7 us with four an SM, 34.5 with eight, 33.9 with
  // sixteen, 36.5 with thirty-two)
  p.head_shift = 0;
  while (p.head_shift < 5 && (1 << p.head_shift) < N1) ++p.head_shift;
  int rows = merge::MAX_ROWS;
  while (rows > 32 && (long long)T * N1 / rows < 16 * num_sms) rows /= 2;
  p.tok_shift = 0;
  while ((1 << (p.tok_shift + p.head_shift)) < rows) ++p.tok_shift;
  p.head_tiles = cdiv(N1, 1 << p.head_shift);
  const unsigned grid = (unsigned)((long long)cdiv(T, 1 << p.tok_shift) * p.head_tiles);
  // a kernel for each number of parts (five parts in the kernel for eight: 255 us at 16K x 64, in
  // their own 231)
  using Kernel = void (*)(const merge::Params);
  static const Kernel kernels[BSA_MAX_MERGE] = {
      merge::merge_kernel<1>, merge::merge_kernel<2>, merge::merge_kernel<3>,
      merge::merge_kernel<4>, merge::merge_kernel<5>, merge::merge_kernel<6>,
      merge::merge_kernel<7>, merge::merge_kernel<8>};
  kernels[count - 1]<<<grid, merge::THREADS, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

// ------------------------------------------------------------------------------------------
// around attention: rotary positions, pages, tokens into the 4-bit cache
// ------------------------------------------------------------------------------------------

extern "C" bsa_status_t bsa_rope_frequencies(int rotary_dim, int scaling, double base, double factor,
                                             double context, double slow, double fast,
                                             const double *inv_freq, uint64_t *freqs) {
  if (rotary_dim < 16 || rotary_dim > HEAD_DIM || rotary_dim % 16 != 0 || !freqs)
    return BSA_ERR_INVALID_ARGUMENT;
  if (!inv_freq) {
    if (scaling < BSA_ROPE_NONE || scaling > BSA_ROPE_PARTS || !std::isfinite(base) || base <= 0 ||
        (scaling != BSA_ROPE_NONE && (!std::isfinite(factor) || factor <= 0)))
      return BSA_ERR_INVALID_ARGUMENT;
    if (scaling == BSA_ROPE_PARTS && (!std::isfinite(context) || context <= 0 ||
                                      !std::isfinite(slow) || !std::isfinite(fast) || slow >= fast))
      return BSA_ERR_INVALID_ARGUMENT;
  }
  const double R = rotary_dim, two_pi = 6.283185307179586476925;
  if (!inv_freq && scaling == BSA_ROPE_BASE) {
    base *= std::pow(factor, R / (R - 2));
    if (!std::isfinite(base) || base <= 0) return BSA_ERR_INVALID_ARGUMENT;
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f;
    if (inv_freq) {
      f = inv_freq[i];
    } else {
      f = std::pow(base, -2.0 * i / R);
      if (scaling == BSA_ROPE_LINEAR) f /= factor;
      if (scaling == BSA_ROPE_PARTS) {
        const double turns = context * f / two_pi;
        const double w = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
        f = f * w + f / factor * (1 - w);
      }
    }
    if (!std::isfinite(f)) return BSA_ERR_INVALID_ARGUMENT;
    // turns a position, less whole ones: positions are whole numbers.  In (-1, 1), times 2^64; a
    // negative one counts down from 2^64.
    const double turns = std::fmod(f / two_pi, 1.0);
    const double size = std::floor(std::fabs(turns) * 0x1p64 + 0.5);
    const uint64_t u = size >= 0x1p64 ? 0u : (uint64_t)size;
    freqs[i] = turns < 0 ? 0u - u : u;
  }
  return BSA_OK;
}

namespace {

bool rope_dims_ok(const bsa_rope_dims_t *d) {
  return d && d->D == HEAD_DIM && d->T >= 0 && d->N1 >= 1 && d->N2 >= 0 &&
         d->N1 <= (1 << 20) && d->N2 <= (1 << 20) && d->rotary_dim >= 16 &&
         d->rotary_dim <= HEAD_DIM && d->rotary_dim % 16 == 0 &&
         (d->layout == BSA_ROPE_HALF || d->layout == BSA_ROPE_INTERLEAVED);
}

// from token to token: rows side by side at least, 16-byte vectors
bool rope_stride_ok(long long stride, int heads) {
  return stride >= (long long)heads * HEAD_DIM && stride % 8 == 0;
}

// T rows of `bytes` each, `stride` bytes apart, at `at`
struct Rows {
  const void *at;
  long long stride;
  size_t bytes;
  size_t span(int T) const { return (size_t)(T - 1) * (size_t)stride + bytes; }
};

// Whether two sets of rows share a byte.  Rows that lie between one another are told apart by their
// places modulo the stride, which has to be the same; otherwise they count as overlapping.
bool rows_overlap(const Rows &a, const Rows &b, int T) {
  if (!overlap(a.at, a.span(T), b.at, b.span(T))) return false;
  if (T == 1 || a.stride != b.stride) return true;
  const uintptr_t s = (uintptr_t)a.stride;
  const uintptr_t d = (reinterpret_cast<uintptr_t>(b.at) % s + s -
                       reinterpret_cast<uintptr_t>(a.at) % s) % s;  // from a's row up to b's
  return d < a.bytes || s - d < b.bytes;
}

bsa_status_t rope_params(const bsa_rope_dims_t *d, const void *q, const void *k,
                         const int *positions, const uint64_t *freqs, float amplitude,
                         rope::Params *p, unsigned *grid) {
  int num_sms = 0;
  const bsa_status_t st = check_device(0, &num_sms);
  if (st != BSA_OK) return st;
  memset(p, 0, sizeof(*p));
  p->q = static_cast<const __nv_bfloat16 *>(q);
  p->k = static_cast<const __nv_bfloat16 *>(k);
  p->positions = positions;
  p->freqs = reinterpret_cast<const unsigned long long *>(freqs);
  p->q_stride = d->q_stride;
  p->k_stride = d->k_stride;
  p->N1 = d->N1;
  p->N2 = d->N2;
  p->R = d->rotary_dim;
  p->interleaved = d->layout == BSA_ROPE_INTERLEAVED;
  p->amplitude = amplitude;
  // heads that one thread serves with its sines and cosines: as many as leave every SM eight warps
  const int heads = d->N1 + d->N2;
  p->heads = 1;
  while (p->heads < 8 && (long long)d->T * cdiv(heads, 2 * p->heads) * rope::LANES >=
                             (long long)num_sms * 256)
    p->heads *= 2;
  p->groups = cdiv(heads, p->heads);
  const long long units = (long long)d->T * p->groups;
  if (units > 0x7ffffff0LL) return BSA_ERR_UNSUPPORTED;  // (more rows than any memory holds)
  p->units = (uint32_t)units;
  p->by_groups = Divisor::of((uint32_t)p->groups);
  *grid = (unsigned)cdiv(units, rope::THREADS / rope::LANES);
  return BSA_OK;
}

}  // namespace

extern "C" bsa_status_t bsa_rope(const bsa_rope_dims_t *d, const void *q, const void *k,
                                 const int *positions, const uint64_t *freqs, float amplitude,
                                 void *q_out, void *k_out, void *stream) {
  if (!rope_dims_ok(d) || !std::isfinite(amplitude)) return BSA_ERR_INVALID_ARGUMENT;
  if (!rope_stride_ok(d->q_stride, d->N1) || !rope_stride_ok(d->q_out_stride, d->N1) ||
      (d->N2 && (!rope_stride_ok(d->k_stride, d->N2) || !rope_stride_ok(d->k_out_stride, d->N2))))
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->T == 0) return BSA_OK;
  if (!q || !q_out || !positions || !freqs || (d->N2 != 0) != (k != nullptr) ||
      (d->N2 != 0) != (k_out != nullptr) || !aligned16(q) || !aligned16(k) || !aligned16(q_out) ||
      !aligned16(k_out) || (reinterpret_cast<uintptr_t>(freqs) & 7u) != 0)
    return BSA_ERR_INVALID_ARGUMENT;
  // a tensor may be turned where it lies; any other overlap would read what is written
  const size_t q_bytes = (size_t)d->N1 * HEAD_DIM * 2, k_bytes = (size_t)d->N2 * HEAD_DIM * 2;
  const Rows qi = {q, d->q_stride * 2, q_bytes}, qo = {q_out, d->q_out_stride * 2, q_bytes},
             ki = {k, d->k_stride * 2, k_bytes}, ko = {k_out, d->k_out_stride * 2, k_bytes};
  const auto same = [](const Rows &a, const Rows &b) { return a.at == b.at && a.stride == b.stride; };
  if (!same(qo, qi) && rows_overlap(qo, qi, d->T)) return BSA_ERR_INVALID_ARGUMENT;
  if (k && ((!same(ko, ki) && rows_overlap(ko, ki, d->T)) || rows_overlap(qo, ki, d->T) ||
            rows_overlap(ko, qi, d->T) || rows_overlap(qo, ko, d->T)))
    return BSA_ERR_INVALID_ARGUMENT;
  rope::Params p;
  unsigned grid = 0;
  const bsa_status_t st = rope_params(d, q, k, positions, freqs, amplitude, &p, &grid);
  if (st != BSA_OK) return st;
  p.q_out = static_cast<__nv_bfloat16 *>(q_out);
  p.k_out = static_cast<__nv_bfloat16 *>(k_out);
  p.q_out_stride = d->q_out_stride;
  p.k_out_stride = d->k_out_stride;
  rope::rope_kernel<false><<<grid, rope::THREADS, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

extern "C" bsa_status_t bsa_rope_quantize(const bsa_rope_dims_t *d, const void *q,
                                          const int *positions, const uint64_t *freqs,
                                          float amplitude, int descale_rule, void *codes_e4m3,
                                          float *descale, void *stream) {
  if (!rope_dims_ok(d) || d->N2 != 0 || !std::isfinite(amplitude) ||
      !rope_stride_ok(d->q_stride, d->N1) ||
      (descale_rule != BSA_DESCALE_AMAX && descale_rule != BSA_DESCALE_UE8M0))
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->T == 0) return BSA_OK;
  if (!q || !positions || !freqs || !codes_e4m3 || !descale || !aligned16(q) ||
      !aligned16(codes_e4m3) || (reinterpret_cast<uintptr_t>(freqs) & 7u) != 0)
    return BSA_ERR_INVALID_ARGUMENT;
  const Rows in = {q, d->q_stride * 2, (size_t)d->N1 * HEAD_DIM * 2};
  if (overlap(codes_e4m3, (size_t)d->T * d->N1 * HEAD_DIM, q, in.span(d->T)))
    return BSA_ERR_INVALID_ARGUMENT;
  rope::Params p;
  unsigned grid = 0;
  const bsa_status_t st = rope_params(d, q, nullptr, positions, freqs, amplitude, &p, &grid);
  if (st != BSA_OK) return st;
  p.codes = static_cast<uint2 *>(codes_e4m3);
  p.descale = descale;
  p.ue8m0 = descale_rule == BSA_DESCALE_UE8M0;
  rope::rope_kernel<true><<<grid, rope::THREADS, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

namespace {

bool pages_dims_ok(const bsa_pages_dims_t *d) {
  return d && d->B >= 0 && (d->page_size == 32 || d->page_size == 64) && d->num_pages >= 0 &&
         d->max_pages_per_seq >= 0 && d->total >= 0 &&
         (long long)d->num_pages * d->page_size <= 0x7fffffffLL &&
         (long long)d->max_pages_per_seq * d->page_size <= 0x7fffffffLL;
}

pages::Params pages_params(const bsa_pages_dims_t *d, int *block_table, int *free_pages,
                           int *free_count, int *dev_status) {
  pages::Params p;
  memset(&p, 0, sizeof(p));
  p.block_table = block_table;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.dev_status = dev_status;
  p.B = d->B;
  p.ps_shift = d->page_size == 64 ? 6 : 5;
  p.num_pages = d->num_pages;
  p.L = d->max_pages_per_seq;
  p.total = d->total;
  return p;
}

}  // namespace

extern "C" bsa_status_t bsa_assign_pages(const bsa_pages_dims_t *d, const int *new_lens,
                                         const int *cache_seqlens, int *block_table,
                                         int *free_pages, int *free_count, int *cu_seqlens,
                                         int *seqused_kv, int *positions, int *slot_map,
                                         int *dev_status, void *stream) {
  if (!pages_dims_ok(d)) return BSA_ERR_INVALID_ARGUMENT;
  if (d->B == 0 && d->total == 0) {  // nothing but the one offset
    if (!cu_seqlens) return BSA_OK;
    int num_sms = 0;
    const bsa_status_t st = check_device(0, &num_sms);
    if (st != BSA_OK) return st;
    if (cudaMemsetAsync(cu_seqlens, 0, sizeof(int), (cudaStream_t)stream) == cudaSuccess)
      return BSA_OK;
    (void)cudaGetLastError();  // leave no pending error behind
    return BSA_ERR_CUDA;
  }
  if (!free_count || !cu_seqlens || (d->total && (!positions || !slot_map)) ||
      (d->num_pages && !free_pages) || (d->B && (!new_lens || !cache_seqlens || !seqused_kv)) ||
      (d->B && d->max_pages_per_seq && !block_table))
    return BSA_ERR_INVALID_ARGUMENT;
  // the lengths are read to the end of the call
  const size_t nb = (size_t)d->B * sizeof(int);
  if (d->B && (overlap(seqused_kv, nb, cache_seqlens, nb) || overlap(seqused_kv, nb, new_lens, nb) ||
               overlap(cu_seqlens, nb + sizeof(int), cache_seqlens, nb) ||
               overlap(cu_seqlens, nb + sizeof(int), new_lens, nb)))
    return BSA_ERR_INVALID_ARGUMENT;
  int num_sms = 0;
  const bsa_status_t st = check_device(0, &num_sms);
  if (st != BSA_OK) return st;
  pages::Params p = pages_params(d, block_table, free_pages, free_count, dev_status);
  p.new_lens = new_lens;
  p.cache_seqlens = cache_seqlens;
  p.cu_seqlens = cu_seqlens;
  p.seqused_kv = seqused_kv;
  p.positions = positions;
  p.slot_map = slot_map;
  p.fill = d->total <= pages::FEW_ROWS || d->B == 0;
  if (!launch_dependent<true>(pages::assign_kernel,
                              dim3(p.fill ? 1u : pages::CLUSTER), pages::THREADS, 0,
                              stream, p))
    return BSA_ERR_CUDA;
  if (p.fill) return BSA_OK;
  return launch_dependent(pages::fill_kernel, dim3((unsigned)cdiv(d->total, pages::FILL_ROWS)),
                          pages::FILL_THREADS, 0, stream, p)
             ? BSA_OK
             : BSA_ERR_CUDA;
}

extern "C" bsa_status_t bsa_release_pages(const bsa_pages_dims_t *d, const int *seq_lens,
                                          const int *keep_lens, const int *block_table,
                                          int *free_pages, int *free_count, int *lens_out,
                                          int *dev_status, void *stream) {
  if (!pages_dims_ok(d)) return BSA_ERR_INVALID_ARGUMENT;
  if (d->B == 0) return BSA_OK;
  if (!seq_lens || !keep_lens || !free_count || !lens_out || (d->num_pages && !free_pages) ||
      (d->max_pages_per_seq && !block_table))
    return BSA_ERR_INVALID_ARGUMENT;
  // a length is written where it was read from or where none is read
  const size_t nb = (size_t)d->B * sizeof(int);
  if ((lens_out != seq_lens && overlap(lens_out, nb, seq_lens, nb)) ||
      (lens_out != keep_lens && overlap(lens_out, nb, keep_lens, nb)))
    return BSA_ERR_INVALID_ARGUMENT;
  int num_sms = 0;
  const bsa_status_t st = check_device(0, &num_sms);
  if (st != BSA_OK) return st;
  pages::Params p =
      pages_params(d, const_cast<int *>(block_table), free_pages, free_count, dev_status);
  p.seq_lens = seq_lens;
  p.keep_lens = keep_lens;
  p.lens_out = lens_out;
  return launch_dependent<true>(pages::release_kernel,
                                dim3(d->num_pages <= pages::FEW_PAGES ? 1u : pages::CLUSTER),
                                pages::THREADS, 0, stream, p)
             ? BSA_OK
             : BSA_ERR_CUDA;
}

extern "C" bsa_status_t bsa_fp4_append_kv(const bsa_fp4_append_dims_t *d, const void *k_new_bf16,
                                          const void *v_new_bf16, const int *slot_map,
                                          const float *k_descale, const float *v_descale,
                                          void *k_pages, void *v_pages, void *k_scales,
                                          void *v_scales, int *dev_status, void *stream) {
  if (!d || d->D != HEAD_DIM || (d->page_size != 32 && d->page_size != 64) || d->N2 < 1 ||
      d->N2 > (1 << 20) || d->num_pages < 0 || d->total_new < 0 ||
      (d->k_scale_kind != BSA_SCALE_PER_TENSOR && d->k_scale_kind != BSA_SCALE_PER_HEAD) ||
      (d->v_scale_kind != BSA_SCALE_PER_TENSOR && d->v_scale_kind != BSA_SCALE_PER_HEAD) ||
      (d->kv_layout != BSA_KV_HND && d->kv_layout != BSA_KV_NHD) ||
      !rope_stride_ok(d->k_stride, d->N2) || !rope_stride_ok(d->v_stride, d->N2))
    return BSA_ERR_INVALID_ARGUMENT;
  if (d->total_new == 0) return BSA_OK;
  if (!k_new_bf16 || !v_new_bf16 || !slot_map || !k_descale || !v_descale || !k_pages ||
      !v_pages || !k_scales || !v_scales || !aligned16(k_new_bf16) || !aligned16(v_new_bf16) ||
      !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_scales) || !aligned16(v_scales))
    return BSA_ERR_INVALID_ARGUMENT;
  int num_sms = 0;
  const bsa_status_t st = check_device(0, &num_sms);
  if (st != BSA_OK) return st;
  fp4::AppendParams p;
  memset(&p, 0, sizeof(p));
  p.k_new = static_cast<const __nv_bfloat16 *>(k_new_bf16);
  p.v_new = static_cast<const __nv_bfloat16 *>(v_new_bf16);
  p.k_stride = d->k_stride;
  p.v_stride = d->v_stride;
  p.slot_map = slot_map;
  p.k_descale = k_descale;
  p.v_descale = v_descale;
  p.k_pages = static_cast<uint8_t *>(k_pages);
  p.v_pages = static_cast<uint8_t *>(v_pages);
  p.k_scales = static_cast<uint8_t *>(k_scales);
  p.v_scales = static_cast<uint8_t *>(v_scales);
  p.dev_status = dev_status;
  const long long rows = (long long)d->total_new * d->N2;
  if (rows > 0x7ffffff0LL) return BSA_ERR_UNSUPPORTED;  // (more rows than any memory holds)
  p.rows = (uint32_t)rows;
  p.heads = Divisor::of((uint32_t)d->N2);
  p.N2 = d->N2;
  p.ps_shift = d->page_size == 64 ? 6 : 5;
  p.num_pages = d->num_pages;
  p.k_per_head = d->k_scale_kind == BSA_SCALE_PER_HEAD;
  p.v_per_head = d->v_scale_kind == BSA_SCALE_PER_HEAD;
  p.kv_nhd = d->kv_layout == BSA_KV_NHD;
  fp4::append_kernel<<<(unsigned)cdiv(rows, fp4::THREADS / fp4::BLOCKS), fp4::THREADS, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}
