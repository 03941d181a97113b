// C ABI of the operators around the loss: the embedding (the other end of a tied LM
// head), 8-bit activation checkpoints with the weight gradient that reads one, and the
// RMS norm that keeps its input in one. Argument checks, workspace plans and launches;
// the kernels are in k_embed.cu, k_act8.cu and k_wgrad.cu.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "ctx.h"
#include "k_ops.h"
#include "kernels.h"

using namespace ckl;

namespace {

ckl_status cuda_status(cudaError_t err) {
  if (err == cudaSuccess) return CKL_OK;
  std::fprintf(stderr, "ckl: CUDA error: %s\n", cudaGetErrorString(err));
  return CKL_ERR_CUDA;
}

// Set the handle's device, and see that a call that is to wait does not run on a stream whose work
// is being captured: to wait would spoil the capture, so nothing is enqueued.
ckl_status enter(DeviceGuard& guard, cudaStream_t s, int wait) {
  if (!guard.ok) return CKL_ERR_CUDA;
  cudaGetLastError();
  if (!wait) return CKL_OK;
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  const cudaError_t err = cudaStreamIsCapturing(s, &capture);
  if (err == cudaSuccess && capture == cudaStreamCaptureStatusNone) return CKL_OK;
  cudaGetLastError();
  return err == cudaSuccess || err == cudaErrorStreamCaptureImplicit ? CKL_ERR_INVALID_ARG
                                                                     : cuda_status(err);
}

size_t elem(const ckl_ctx* h) { return h->dtype == CKL_BF16 ? 2 : 4; }

// ------------------------------------------------------------------ embedding
ckl_status check_ids(const ckl_ctx* h, const int32_t* ids, int64_t T, int64_t V_total, int64_t v0,
                     float scale) {
  if (!h || T < 0 || (T > 0 && !ids)) return CKL_ERR_INVALID_ARG;
  if (v0 < 0 || V_total > INT32_MAX || v0 + h->V > V_total || !std::isfinite(scale))
    return CKL_ERR_INVALID_ARG;
  if (T > INT32_MAX) return CKL_ERR_UNSUPPORTED;
  if (ids && !aligned(ids, 4)) return CKL_ERR_ALIGNMENT;
  return CKL_OK;
}

EmbedIds ids_of(const ckl_ctx* h, const int32_t* ids, const uint8_t* mask, int64_t T,
                int64_t V_total, int64_t v0) {
  return EmbedIds{ids, mask, T, (int32_t)V_total, (int32_t)v0, (int32_t)h->V, h->d_status};
}

struct EmbedGradPlan {
  EmbedShape shape{};
  size_t off_a = 0, off_b = 0, off_part = 0, total = 0;
};

EmbedGradPlan embed_grad_plan(const ckl_ctx* h, int64_t T) {
  EmbedGradPlan p;
  p.shape = embed_shape(T, (int)h->d, h->num_sms);
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes, 256); return at; };
  p.off_a = take((size_t)T * 8);
  p.off_b = take((size_t)T * 8);
  p.off_part = take((size_t)((T + p.shape.tile() - 1) / p.shape.tile()) * 2 * h->d * 4);
  p.total = o;
  return p;
}

// ------------------------------------------------------------------ 8-bit checkpoints
ckl_status check_act8(const ckl_ctx* h, int64_t T, int64_t cols, int fmt, const void* q,
                      const void* scale) {
  if (!h || T < 0 || cols < 1 || (fmt != CKL_ACT8_INT8 && fmt != CKL_ACT8_E4M3))
    return CKL_ERR_INVALID_ARG;
  if (cols % 8 != 0 || cols > (1 << 20) || T > INT32_MAX) return CKL_ERR_UNSUPPORTED;
  if (T > 0 && (!q || !scale)) return CKL_ERR_INVALID_ARG;
  if (q && !aligned(q, 16)) return CKL_ERR_ALIGNMENT;
  return CKL_OK;
}

// The contraction runs over `chunk` tokens at a time, so that the bf16 copy of the checkpoint, and
// of fp32 handles each of the three bf16 parts of dY, stays below kWgradChunkBytes whatever T and n
// are (or at kWgradChunkStep tokens, where so many alone are more). (Chunks small enough to stay in L2, each unpacked
// behind the contraction of the one before, measured slower: 32768 x 2880 x 2880 in one chunk 478 us
// from a cool start and 560 under the power limit, in chunks of 96 MB 487 and 571, of 48 MB 502 and
// 592: every contraction has its own start and end.)
struct WgradPlan {
  int64_t chunk = 0, parts = 0;
  int n_split = 1;
  size_t off_x = 0, off_parts = 0, off_sum = 0, total = 0;
};

constexpr int64_t kWgradChunkBytes = 256 << 20;  // of a bf16 copy
constexpr int64_t kWgradChunkStep = 4096;        // tokens: whole accumulator ranges of the kernel

WgradPlan wgrad_plan(const ckl_ctx* h, int64_t T, int64_t n, int64_t cols) {
  WgradPlan p;
  p.parts = h->dtype == CKL_BF16 ? 1 : 3;
  const int64_t widest = p.parts > 1 ? std::max(n, cols) : cols;  // of the copies that are made
  const int64_t fit = kWgradChunkBytes / (widest * 2) / kWgradChunkStep * kWgradChunkStep;
  p.chunk = std::max<int64_t>(1, std::min(T, std::max(fit, kWgradChunkStep)));
  p.n_split = wgrad_split(n, cols, p.parts * ((p.chunk + 63) / 64), h->num_sms);
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes, 256); return at; };
  if (T == 0) return p;
  p.off_x = take((size_t)p.chunk * cols * 2);
  if (p.parts > 1) p.off_parts = take((size_t)p.chunk * n * 2 * p.parts);
  if (p.n_split > 1) p.off_sum = take((size_t)p.n_split * n * cols * 4);
  p.total = o;
  return p;
}

ckl_status check_wgrad(const ckl_ctx* h, int64_t T, int64_t n, int64_t cols) {
  if (!h || T < 0 || n < 1 || cols < 1) return CKL_ERR_INVALID_ARG;
  if (n % 8 != 0 || cols % 8 != 0 || n > (1 << 20) || cols > (1 << 20) ||
      T > (int64_t)INT32_MAX / 4)
    return CKL_ERR_UNSUPPORTED;
  return CKL_OK;
}

}  // namespace

extern "C" {

ckl_status ckl_act8_weight_grad_workspace_bytes(ckl_handle h, int64_t T, int64_t n, int64_t cols,
                                                size_t* bytes) {
  const ckl_status st = check_wgrad(h, T, n, cols);
  if (st != CKL_OK || !bytes) return st != CKL_OK ? st : CKL_ERR_INVALID_ARG;
  *bytes = wgrad_plan(h, T, n, cols).total;
  return CKL_OK;
}

ckl_status ckl_act8_weight_grad(ckl_handle h, const void* dY, int64_t T, int64_t n, const void* q,
                                const uint8_t* scale, int64_t cols, ckl_act8_format fmt,
                                int accumulate, float* dW, void* workspace, size_t workspace_bytes,
                                void* stream, int wait) {
  ckl_status st = check_wgrad(h, T, n, cols);
  if (st == CKL_OK) st = check_act8(h, T, cols, fmt, q, scale);
  if (st != CKL_OK) return st;
  if (!dW || (T > 0 && !dY)) return CKL_ERR_INVALID_ARG;
  if (!aligned(dW, 16) || (dY && !aligned(dY, 16))) return CKL_ERR_ALIGNMENT;
  const WgradPlan P = wgrad_plan(h, T, n, cols);
  if (P.total && (!workspace || !aligned(workspace, 256) || workspace_bytes < P.total))
    return CKL_ERR_WORKSPACE;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = enter(guard, s, wait)) != CKL_OK) return st;
  cudaError_t err = cudaSuccess;
  auto chk = [&](cudaError_t e) { if (e != cudaSuccess && err == cudaSuccess) err = e; };
  if (T == 0) {
    if (!accumulate) chk(cudaMemsetAsync(dW, 0, (size_t)n * cols * 4, s));
  } else {
    unsigned char* base = static_cast<unsigned char*>(workspace);
    Launcher L{h, s};
    const size_t es = elem(h);
    const int nb = (int)((cols + 31) / 32);
    float* out = P.n_split > 1 ? reinterpret_cast<float*>(base + P.off_sum) : dW;
    void* x = base + P.off_x;
    for (int64_t t0 = 0; t0 < T && err == cudaSuccess; t0 += P.chunk) {
      const int64_t Tc = std::min(P.chunk, T - t0);
      const bool add = accumulate || t0 > 0;
      const void* a = static_cast<const unsigned char*>(dY) + (size_t)(t0 * n) * es;
      chk(L(KID_ACT8_UNPACK, 0, (double)Tc * cols * (2.0 + 33.0 / 32), [&] {
        launch_act8_unpack(true, static_cast<const uint8_t*>(q) + t0 * cols, scale + t0 * nb, Tc,
                           (int)cols, fmt, x, s);
      }));
      if (P.parts > 1) {
        uint16_t* parts = reinterpret_cast<uint16_t*>(base + P.off_parts);
        chk(L(KID_WGRAD_PARTS, 0, (double)Tc * n * 10,
              [&] { launch_split3(static_cast<const float*>(a), Tc * n, parts, s); }));
        a = parts;
      }
      CUtensorMap ma, mb, mc;
      if (!make_map_planes(h, &ma, a, n, Tc, P.parts, 64) ||
          !make_map(h, &mb, x, cols, Tc, (uint64_t)cols * 2, 64, 64) ||
          !make_map_planes(h, &mc, out, cols, n, P.n_split, 32, true))
        return CKL_ERR_CUDA;
      WgradArgs p{};
      p.n = (int)n; p.cols = (int)cols;
      p.kb_part = (int)((Tc + 63) / 64);
      p.n_kb = (int)P.parts * p.kb_part;
      // a short last chunk takes as many of the ranges as it has steps for
      const int range = (p.n_kb + P.n_split - 1) / P.n_split;
      p.n_split = (p.n_kb + range - 1) / range;
      p.kb_split = range;
      p.add = P.n_split == 1 && add;
      p.status = h->d_status;
      chk(L(KID_WGRAD, 2.0 * Tc * n * cols, 0,
            [&] { chk(launch_wgrad(ma, mb, mc, p, h->num_sms, s)); }));
      if (P.n_split > 1)
        chk(L(KID_WGRAD_SUM, 0, 4.0 * n * cols * (p.n_split + 1), [&] {
          chk(launch_wgrad_sum(out, p.n_split, n * cols, add, dW, s));
        }));
    }
  }
  if ((st = cuda_status(err)) != CKL_OK) return st;
  return wait ? sync_and_read(h, s, nullptr, nullptr) : CKL_OK;
}

ckl_status ckl_embed(ckl_handle h, const int32_t* ids, const uint8_t* mask, const void* W,
                     int64_t T, int64_t V_total, int64_t v0, float scale, void* out, void* stream,
                     int wait) {
  ckl_status st = check_ids(h, ids, T, V_total, v0, scale);
  if (st != CKL_OK) return st;
  if (!W || (T > 0 && !out)) return CKL_ERR_INVALID_ARG;
  if (!aligned(W, 16) || (out && !aligned(out, 16))) return CKL_ERR_ALIGNMENT;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = enter(guard, s, wait)) != CKL_OK) return st;
  if (T > 0) {
    Launcher L{h, s};
    st = cuda_status(L(KID_EMBED, 0, (double)T * h->d * 2 * elem(h), [&] {
      launch_embed(ids_of(h, ids, mask, T, V_total, v0), h->dtype == CKL_BF16, W, (int)h->d, scale,
                   out, false, s);
    }));
    if (st != CKL_OK) return st;
  }
  return wait ? sync_and_read(h, s, nullptr, nullptr) : CKL_OK;
}

ckl_status ckl_embed_vp_workspace_bytes(ckl_handle h, int64_t T, size_t* bytes) {
  if (!h || !bytes || T < 0) return CKL_ERR_INVALID_ARG;
  *bytes = align_up((size_t)T * h->d * 4, 256);
  return CKL_OK;
}

ckl_status ckl_embed_vocab_parallel(ckl_handle h, const ckl_vocab_group* g, const int32_t* ids,
                                    const uint8_t* mask, const void* W_shard, int64_t T,
                                    float scale, void* out, void* workspace,
                                    size_t workspace_bytes, void* stream, int wait) {
  if (!h || !g || g->world < 1 || g->rank < 0 || g->rank >= g->world || !g->all_reduce_sum)
    return CKL_ERR_INVALID_ARG;
  if (h->dtype != CKL_BF16) return CKL_ERR_UNSUPPORTED;
  ckl_status st = check_ids(h, ids, T, g->V_total, g->v0, scale);
  if (st != CKL_OK) return st;
  if (!W_shard || (T > 0 && !out)) return CKL_ERR_INVALID_ARG;
  if (!aligned(W_shard, 16) || (out && !aligned(out, 16))) return CKL_ERR_ALIGNMENT;
  const size_t need = align_up((size_t)T * h->d * 4, 256);
  if (T > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return CKL_ERR_WORKSPACE;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = enter(guard, s, wait)) != CKL_OK) return st;
  if (T > 0) {
    Launcher L{h, s};
    float* buf = static_cast<float*>(workspace);
    // one rank's row and zeros from the others: the sum is exact in any order
    cudaError_t err = L(KID_EMBED, 0, (double)T * h->d * 6, [&] {
      launch_embed(ids_of(h, ids, mask, T, g->V_total, g->v0), true, W_shard, (int)h->d, scale, buf,
                   true, s);
    });
    // made even after a failed launch: the ranks' calls stay matched
    const int rc = L.collective(KID_VP_REDUCE, (double)T * h->d * 4,
                                [&] { return g->all_reduce_sum(g->user, buf, T * h->d, s); });
    if (err == cudaSuccess && rc == 0)
      err = L(KID_TO_BF16, 0, (double)T * h->d * 6, [&] {
        launch_f32_to_bf16(buf, T * h->d, static_cast<uint16_t*>(out), s);
      });
    if ((st = cuda_status(err)) != CKL_OK) return st;
    if (rc != 0) return CKL_ERR_COLLECTIVE;
  }
  return wait ? sync_and_read(h, s, nullptr, nullptr) : CKL_OK;
}

ckl_status ckl_embed_grad_workspace_bytes(ckl_handle h, int64_t T, size_t* bytes) {
  if (!h || !bytes || T < 0) return CKL_ERR_INVALID_ARG;
  *bytes = embed_grad_plan(h, T).total;
  return CKL_OK;
}

ckl_status ckl_embed_grad(ckl_handle h, const int32_t* ids, const uint8_t* mask, const void* dX,
                          int64_t T, int64_t V_total, int64_t v0, float scale, int accumulate,
                          float* dW, void* workspace, size_t workspace_bytes, void* stream,
                          int wait) {
  ckl_status st = check_ids(h, ids, T, V_total, v0, scale);
  if (st != CKL_OK) return st;
  if (!dW || (T > 0 && !dX)) return CKL_ERR_INVALID_ARG;
  if (!aligned(dW, 16) || (dX && !aligned(dX, 16))) return CKL_ERR_ALIGNMENT;
  const EmbedGradPlan P = embed_grad_plan(h, T);
  if (T > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < P.total))
    return CKL_ERR_WORKSPACE;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = enter(guard, s, wait)) != CKL_OK) return st;
  cudaError_t err = cudaSuccess;
  auto chk = [&](cudaError_t e) { if (e != cudaSuccess && err == cudaSuccess) err = e; };
  const int d = (int)h->d, V = (int)h->V;
  if (T == 0) {
    if (!accumulate) chk(cudaMemsetAsync(dW, 0, (size_t)V * d * 4, s));
  } else if (embed_grad_is_few(T)) {
    Launcher L{h, s};
    if (!accumulate)
      chk(L(KID_EMBED_ZERO, 0, 4.0 * V * d, [&] { launch_embed_zero(dW, (int64_t)V * d, s); }));
    chk(L(KID_EMBED_GRAD, 0, (double)T * d * elem(h), [&] {
      chk(launch_embed_grad_few(ids_of(h, ids, mask, T, V_total, v0), h->dtype == CKL_BF16, dX, d,
                                scale, accumulate != 0, dW, s));
    }));
  } else {
    unsigned char* base = static_cast<unsigned char*>(workspace);
    uint64_t* a = reinterpret_cast<uint64_t*>(base + P.off_a);
    uint64_t* b = reinterpret_cast<uint64_t*>(base + P.off_b);
    float* part = reinterpret_cast<float*>(base + P.off_part);
    const uint64_t* sorted = embed_sort_result(T, V) ? b : a;
    Launcher L{h, s};
    const int64_t n_fill = accumulate ? 0 : (int64_t)V * d;
    chk(L(KID_EMBED_SORT, 0, (double)T * 12 + 4.0 * n_fill, [&] {
      chk(launch_embed_sort(ids_of(h, ids, mask, T, V_total, v0), a, b, dW, n_fill, s));
    }));
    chk(L(KID_EMBED_GRAD, 0, (double)T * d * elem(h), [&] {
      chk(launch_embed_grad(sorted, T, V, h->dtype == CKL_BF16, dX, d, P.shape, scale,
                            accumulate != 0, dW, part, s));
    }));
    if (T > P.shape.tile())  // a row may span tiles
      chk(L(KID_EMBED_JOIN, 0, 0, [&] {
        chk(launch_embed_join(sorted, T, V, d, P.shape, scale, accumulate != 0, dW, part, s));
      }));
  }
  if ((st = cuda_status(err)) != CKL_OK) return st;
  return wait ? sync_and_read(h, s, nullptr, nullptr) : CKL_OK;
}

ckl_status ckl_act8_pack(ckl_handle h, const void* X, int64_t T, int64_t cols, ckl_act8_format fmt,
                         void* q, uint8_t* scale, void* stream) {
  ckl_status st = check_act8(h, T, cols, fmt, q, scale);
  if (st != CKL_OK) return st;
  if (T > 0 && !X) return CKL_ERR_INVALID_ARG;
  if (X && !aligned(X, 16)) return CKL_ERR_ALIGNMENT;
  if (T == 0) return CKL_OK;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = enter(guard, s, 0)) != CKL_OK) return st;
  Launcher L{h, s};
  return cuda_status(L(KID_ACT8_PACK, 0, (double)T * cols * (elem(h) + 33.0 / 32), [&] {
    launch_act8_pack(h->dtype == CKL_BF16, X, T, (int)cols, fmt, static_cast<uint8_t*>(q), scale, s);
  }));
}

ckl_status ckl_act8_unpack(ckl_handle h, const void* q, const uint8_t* scale, int64_t T,
                           int64_t cols, ckl_act8_format fmt, void* out, void* stream) {
  ckl_status st = check_act8(h, T, cols, fmt, q, scale);
  if (st != CKL_OK) return st;
  if (T > 0 && !out) return CKL_ERR_INVALID_ARG;
  if (out && !aligned(out, 16)) return CKL_ERR_ALIGNMENT;
  if (T == 0) return CKL_OK;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = enter(guard, s, 0)) != CKL_OK) return st;
  Launcher L{h, s};
  return cuda_status(L(KID_ACT8_UNPACK, 0, (double)T * cols * (elem(h) + 33.0 / 32), [&] {
    launch_act8_unpack(h->dtype == CKL_BF16, static_cast<const uint8_t*>(q), scale, T, (int)cols,
                       fmt, out, s);
  }));
}

ckl_status ckl_norm(ckl_handle h, const void* X, const void* residual, const void* gain, int64_t T,
                    float eps, ckl_act8_format fmt, void* sum, void* Y, void* q, uint8_t* scale,
                    float* rstd, void* stream) {
  if (!h || T < 0 || !gain || !(eps > 0.f) || !std::isfinite(eps)) return CKL_ERR_INVALID_ARG;
  if (fmt != CKL_ACT8_INT8 && fmt != CKL_ACT8_E4M3) return CKL_ERR_INVALID_ARG;
  if (T > INT32_MAX) return CKL_ERR_UNSUPPORTED;
  if (T > 0 && (!X || !Y || (residual && !sum))) return CKL_ERR_INVALID_ARG;
  if ((q != nullptr) != (scale != nullptr) || (T > 0 && q && !rstd)) return CKL_ERR_INVALID_ARG;
  if (residual && sum == Y && T > 0) return CKL_ERR_INVALID_ARG;
  for (const void* p : {X, residual, gain, (const void*)sum, (const void*)Y, (const void*)q})
    if (p && !aligned(p, 16)) return CKL_ERR_ALIGNMENT;
  if (rstd && !aligned(rstd, 4)) return CKL_ERR_ALIGNMENT;
  if (T == 0) return CKL_OK;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (const ckl_status st = enter(guard, s, 0); st != CKL_OK) return st;
  NormArgs a{};
  a.x = X; a.res = residual; a.gain = gain; a.T = T; a.d = (int)h->d; a.eps = eps; a.fmt = fmt;
  a.sum = sum; a.y = Y; a.q = static_cast<uint8_t*>(q); a.e = scale; a.rstd = rstd;
  Launcher L{h, s};
  const double per = elem(h) * (residual ? 4.0 : 2.0) + (q ? 33.0 / 32 : 0.0);
  cudaError_t set = cudaSuccess;
  const cudaError_t err = L(KID_NORM_FWD, 0, (double)T * h->d * per, [&] {
    set = launch_norm_fwd(a, h->dtype == CKL_BF16, h->num_sms, s);
  });
  return cuda_status(err != cudaSuccess ? err : set);
}

ckl_status ckl_norm_bwd_workspace_bytes(ckl_handle h, int64_t T, size_t* bytes) {
  if (!h || !bytes || T < 0) return CKL_ERR_INVALID_ARG;
  *bytes = (size_t)norm_part_rows(T, (int)h->d, h->dtype == CKL_BF16, h->num_sms) * h->d * 4;
  return CKL_OK;
}

ckl_status ckl_norm_bwd(ckl_handle h, const void* dY, const void* q, const uint8_t* scale,
                        const float* rstd, const void* gain, const void* d_sum, int64_t T,
                        ckl_act8_format fmt, int accumulate, void* dX, float* dgain,
                        void* workspace, size_t workspace_bytes, void* stream) {
  ckl_status st = check_act8(h, T, h ? h->d : 0, fmt, q, scale);
  if (st != CKL_OK) return st;
  if (!gain || !dgain || (T > 0 && (!dY || !rstd || !dX))) return CKL_ERR_INVALID_ARG;
  for (const void* p : {dY, gain, d_sum, (const void*)dX})
    if (p && !aligned(p, 16)) return CKL_ERR_ALIGNMENT;
  if (!aligned(dgain, 4) || (rstd && !aligned(rstd, 4))) return CKL_ERR_ALIGNMENT;
  const int d = (int)h->d;
  const int64_t rows = norm_part_rows(T, d, h->dtype == CKL_BF16, h->num_sms);
  if (T > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < (size_t)rows * d * 4))
    return CKL_ERR_WORKSPACE;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = enter(guard, s, 0)) != CKL_OK) return st;
  if (T == 0) return accumulate ? CKL_OK : cuda_status(cudaMemsetAsync(dgain, 0, (size_t)d * 4, s));
  NormArgs a{};
  a.x = dY; a.res = d_sum; a.gain = gain; a.T = T; a.d = d; a.fmt = fmt; a.y = dX;
  a.q = const_cast<uint8_t*>(static_cast<const uint8_t*>(q));
  a.e = const_cast<uint8_t*>(scale);
  a.rstd = const_cast<float*>(rstd);
  a.part = static_cast<float*>(workspace);
  Launcher L{h, s};
  const double per = elem(h) * (d_sum ? 3.0 : 2.0) + 33.0 / 32;
  cudaError_t set = cudaSuccess;
  cudaError_t err = L(KID_NORM_BWD, 0, (double)T * d * per,
                      [&] { set = launch_norm_bwd(a, h->dtype == CKL_BF16, h->num_sms, s); });
  if (err == cudaSuccess) err = set;
  if (err == cudaSuccess)
    err = L(KID_NORM_DGAIN, 0, (double)rows * d * 4,
            [&] { set = launch_norm_dgain(a.part, rows, d, accumulate != 0, dgain, s); });
  return cuda_status(err != cudaSuccess ? err : set);
}

}  // extern "C"
