// What the files with C entry points share: the handle, the launch wrapper, tensor
// maps, argument helpers and the device status (internal; not part of the C ABI).
#pragma once

#include <cstdint>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "../../include/ckl.h"
#include "common.cuh"

namespace ckl {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct ProfRec {
  int kernel;
  int ev;
  double flops, bytes;
};

enum KernelId {
  KID_MASK = 0, KID_GATHER, KID_LSE, KID_COMBINE, KID_GRAD, KID_REPAIR, KID_FIXUP, KID_DH,
  KID_DW, KID_LOSS, KID_TKMAX, KID_TKTHRESH, KID_TKEMIT, KID_TKSELECT, KID_VP_MERGE,
  KID_DH_F32, KID_TO_BF16, KID_VP_GATHER, KID_VP_REDUCE,
  KID_EMBED, KID_EMBED_SORT, KID_EMBED_GRAD, KID_EMBED_JOIN, KID_ACT8_PACK, KID_ACT8_UNPACK,
  KID_NORM_FWD, KID_NORM_BWD, KID_NORM_DGAIN, KID_WGRAD_PARTS, KID_WGRAD, KID_WGRAD_SUM,
  KID_EMBED_ZERO, KID_COUNT
};
// bf16 backward: a profiled "dh_gemm" range also holds the next chunk's teacher
// kernel, and a "dw_gemm" range the chunk's dH split reduction, both launched
// behind the contraction as dependents (no event may stand between the two).
inline const char* const kKernelNames[KID_COUNT] = {"mask_count", "teacher_topk", "lse_gemm", "lse_combine",
                                       "grad_gemm", "row_repair", "topk_fixup", "dh_gemm",
                                       "dw_gemm", "loss_finalize", "cache_max_gemm",
                                       "cache_threshold", "cache_emit_gemm", "cache_select",
                                       "vp_merge", "dh_reduce_f32", "dh_to_bf16",
                                       "vp_all_gather", "vp_all_reduce", "embed", "embed_sort",
                                       "embed_grad", "embed_join", "act8_pack", "act8_unpack",
                                       "norm_fwd", "norm_bwd", "norm_dgain", "weight_grad_parts",
                                       "act8_weight_grad",
                                       "weight_grad_sum", "embed_zero"};

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

}  // namespace ckl

struct ckl_ctx {
  int device = 0;
  ckl_dtype dtype = CKL_F32;
  int64_t V = 0, d = 0, K = 0, max_chunk = 0;
  int num_sms = 0;
  unsigned* d_status = nullptr;  // device status word
  unsigned* h_status = nullptr;  // pinned
  float* h_loss = nullptr;       // pinned
  int64_t launches = 0;
  int recompute = 0;  // bf16: form the logits again in the backward (1) or keep exp(z) (0)
  ckl::EncodeTiledFn encode = nullptr;
  // profiling
  bool prof = false;
  std::vector<cudaEvent_t> ev;  // pairs: ev[2i], ev[2i+1]
  int ev_used = 0;
  std::vector<ckl::ProfRec> recs;
  // host-input calls: inputs are copied chunk by chunk on their own stream
  cudaStream_t copy_stream = nullptr;
  cudaEvent_t copy_start = nullptr;
  std::vector<cudaEvent_t> chunk_ready;
};

namespace ckl {

struct DeviceGuard {
  int prev = -1;
  bool ok = false;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) return;
    ok = (prev == dev) || cudaSetDevice(dev) == cudaSuccess;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// 2-D tensor map (bf16, or fp32 when f32 is set): `inner` contiguous elements per
// row, `outer` rows `row_bytes` apart, box of box_inner x box_outer, 128-byte
// swizzle, zero fill outside the tensor (loads) / clipping (stores).
inline bool make_map(const ckl_ctx* h, CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
              uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, bool f32 = false) {
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = h->encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                               2, const_cast<void*>(base),
                               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 3-D tensor map (bf16, or fp32 when f32 is set) of `outer` planes of rows x inner, dense;
// boxes of box x box x 1, 128-byte swizzle, zero fill outside (loads) / clipping (stores).
inline bool make_map_planes(const ckl_ctx* h, CUtensorMap* m, const void* base, uint64_t inner,
                            uint64_t rows, uint64_t outer, uint32_t box, bool f32 = false) {
  const uint64_t es = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {inner, rows, outer};
  const cuuint64_t strides[2] = {inner * es, inner * rows * es};
  const cuuint32_t boxes[3] = {box, box, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return h->encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                   const_cast<void*>(base), dims, strides, boxes, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Every launch (and every caller-supplied collective) is wrapped in an NVTX range
// named after its kernel, so a timeline tool shows the call's structure; with no
// tool attached a range costs a few nanoseconds.
struct Launcher {
  ckl_ctx* h;
  cudaStream_t s;
  template <class F>
  cudaError_t operator()(int kid, double flops, double bytes, F&& f) {
    struct Range {
      explicit Range(const char* n) { nvtxRangePushA(n); }
      ~Range() { nvtxRangePop(); }
    } range(kKernelNames[kid]);
    int slot = -1;
    if (h->prof && h->ev_used * 2 + 1 < (int)h->ev.size()) {
      slot = h->ev_used++;
      cudaEventRecord(h->ev[2 * slot], s);
    }
    f();
    cudaError_t e = cudaGetLastError();
    if (slot >= 0) {
      cudaEventRecord(h->ev[2 * slot + 1], s);
      h->recs.push_back(ProfRec{kid, slot, flops, bytes});
    }
    h->launches++;
    return e;
  }
  // A caller-supplied collective: profiled under `kid`, not counted as a launch.
  template <class F>
  int collective(int kid, double bytes, F&& f) {
    nvtxRangePushA(kKernelNames[kid]);
    struct Pop {
      ~Pop() { nvtxRangePop(); }
    } pop;
    int slot = -1;
    if (h->prof && h->ev_used * 2 + 1 < (int)h->ev.size()) {
      slot = h->ev_used++;
      cudaEventRecord(h->ev[2 * slot], s);
    }
    const int rc = f();
    if (slot >= 0) {
      cudaEventRecord(h->ev[2 * slot + 1], s);
      h->recs.push_back(ProfRec{kid, slot, 0.0, bytes});
    }
    return rc;
  }
};

inline ckl_status fold_status(unsigned dev) {
  if (dev & ST_INDEX_RANGE) return CKL_ERR_INDEX_RANGE;
  if (dev & ST_TIMEOUT) return CKL_ERR_TIMEOUT;
  if (dev & ST_INTERNAL) return CKL_ERR_INTERNAL;
  return CKL_OK;
}

// Copy the loss and the device status to pinned host memory, wait, clear the
// status word.
inline ckl_status sync_and_read(ckl_ctx* h, cudaStream_t s, const float* loss_dev, float* loss_host) {
  if (loss_dev && cudaMemcpyAsync(h->h_loss, loss_dev, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return CKL_ERR_CUDA;
  if (cudaMemcpyAsync(h->h_status, h->d_status, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemsetAsync(h->d_status, 0, 4, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return CKL_ERR_CUDA;
  if (loss_host && loss_dev) *loss_host = *h->h_loss;
  return fold_status(*h->h_status);
}

}  // namespace ckl
