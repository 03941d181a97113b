// 8-bit activation checkpoints (pack, unpack) and the RMS norm that writes one in its
// forward pass and reads it in its backward pass. The format is described in ops.cuh.
//
//   forward   s = round(x + r);  rstd = 1 / sqrt(mean(s^2) + eps);  y = round(s rstd g)
//             kept for the backward: the checkpoint of s and rstd (1.03 bytes an element and
//             4 a row, against 2 or 4 bytes an element for s itself)
//   backward  h = s' rstd with s' the checkpoint's values;  a = dY g;
//             dX = round(rstd (a - h mean(a h)) + dS);  dg = sum over rows of dY h
//             (dX is the gradient of x and of r; dS the gradient that reaches s from
//             elsewhere, as s is the residual stream that the next layer adds to)
// Everything is held in fp32 between the loads and the one rounding of each output.
// All of these are bound by memory. A row is read once, kept in registers (16-byte loads,
// one vector of eight columns a lane, four lanes to an 8-bit block) while its sum goes
// round the warps that share it, and written from there.
#include "common.cuh"
#include "k_ops.h"
#include "ops.cuh"

namespace ckl {

namespace {

constexpr int kSlab = 128;  // vectors of eight columns a warp handles of one row (pack, unpack)

template <typename T>
__global__ void __launch_bounds__(256)
    act8_pack_kernel(const T* __restrict__ X, int64_t rows, int nvec, int slabs, int fmt,
                     uint8_t* __restrict__ q, uint8_t* __restrict__ e) {
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = w / slabs;
  if (t >= rows) return;
  const int v0 = (int)(w - t * slabs) * kSlab + lane;
  const int nb = (nvec + 3) / 4;
  Raw8<T> r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = v0 + i * 32;
    r[i] = v < nvec ? load8(X + (t * nvec + v) * 8) : zero8<T>();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = v0 + i * 32;
    float f[8];
    to_f32(r[i], f);
    const uint32_t byte = act8_scale_byte(quad_max(amax_bits8(f)), fmt);
    if (v < nvec) {
      *reinterpret_cast<uint2*>(q + (t * nvec + v) * 8) = act8_encode(f, byte, fmt);
      if ((lane & 3) == 0) e[t * nb + (v >> 2)] = (uint8_t)byte;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256)
    act8_unpack_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ e, int64_t rows,
                       int nvec, int slabs, int fmt, T* __restrict__ out) {
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = w / slabs;
  if (t >= rows) return;
  const int v0 = (int)(w - t * slabs) * kSlab + lane;
  const int nb = (nvec + 3) / 4;
  uint2 c[4];
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = v0 + i * 32;
    if (v < nvec) {
      c[i] = *reinterpret_cast<const uint2*>(q + (t * nvec + v) * 8);
      b[i] = e[t * nb + (v >> 2)];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = v0 + i * 32;
    if (v >= nvec) break;
    float f[8];
    act8_decode(c[i], act8_scale(b[i]), fmt, f);
    store8(out + (t * nvec + v) * 8, from_f32<T>(f));
  }
}

// Sum over the WPR warps of a row (all threads of the block call it; each row group r of the
// block has its own line of `red`).
template <int WPR>
__device__ __forceinline__ float row_add(float v, float (*red)[32], int r, int lw, int lane) {
  v = warp_add(v);
  if (WPR == 1) return v;
  if (lane == 0) red[r][lw] = v;
  __syncthreads();
  float t = red[r][0];
#pragma unroll
  for (int w = 1; w < WPR; ++w) t += red[r][w];
  return t;
}

// WPR warps share a row, each lane holding VPT vectors of eight columns. Blocks of eight
// warps (8 / WPR rows), or of one row where it takes 32 warps.
template <int WPR>
constexpr int kNormThreads = WPR > 8 ? WPR * 32 : 256;

template <typename T, int WPR, int VPT>
__global__ void __launch_bounds__(kNormThreads<WPR>) norm_fwd_kernel(const NormArgs a) {
  constexpr int R = kNormThreads<WPR> / 32 / WPR;
  __shared__ float red[R][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = warp / WPR, lw = warp % WPR;
  const int64_t t = (int64_t)blockIdx.x * R + r;
  const int nvec = a.d / 8, nb = (nvec + 3) / 4;
  const bool row_ok = t < a.T;
  const T* x = (const T*)a.x + t * a.d;
  const T* res = (const T*)a.res + t * a.d;
  Raw8<T> s[VPT];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = (i * WPR + lw) * 32 + lane;
    s[i] = row_ok && v < nvec ? load8(x + v * 8) : zero8<T>();
    if (a.res && row_ok && v < nvec) {
      float f[8], g[8];
      to_f32(s[i], f);
      to_f32(load8(res + v * 8), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += g[j];
      s[i] = from_f32<T>(f);
    }
    float f[8];
    to_f32(s[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
  }
  ss = row_add<WPR>(ss, red, r, lw, lane);
  const float rstd = 1.f / sqrtf(ss / (float)a.d + a.eps);
  if (a.rstd && row_ok && lw == 0 && lane == 0) a.rstd[t] = rstd;
  T* sum = (T*)a.sum + t * a.d;
  T* y = (T*)a.y + t * a.d;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = (i * WPR + lw) * 32 + lane;
    const bool ok = row_ok && v < nvec;
    float f[8];
    to_f32(s[i], f);
    if (a.q) {
      const uint32_t byte = act8_scale_byte(quad_max(amax_bits8(f)), a.fmt);
      if (ok) {
        *reinterpret_cast<uint2*>(a.q + t * a.d + v * 8) = act8_encode(f, byte, a.fmt);
        if ((lane & 3) == 0) a.e[t * nb + (v >> 2)] = (uint8_t)byte;
      }
    }
    if (!ok) continue;
    if (a.res) store8(sum + v * 8, s[i]);
    float g[8];
    to_f32(load8((const T*)a.gain + v * 8), g);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * g[j];
    store8(y + v * 8, from_f32<T>(f));
  }
}

// A block walks rows in steps of the grid and keeps its columns' share of dg in registers;
// each row group leaves one line of partial sums, added up by norm_dgain_kernel.
template <typename T, int WPR, int VPT>
__global__ void __launch_bounds__(kNormThreads<WPR>) norm_bwd_kernel(const NormArgs a) {
  constexpr int R = kNormThreads<WPR> / 32 / WPR;
  __shared__ float red[2][R][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = warp / WPR, lw = warp % WPR;
  const int nvec = a.d / 8, nb = (nvec + 3) / 4;
  const float inv_d = 1.f / (float)a.d;
  Raw8<T> g[VPT];
  float dg[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = (i * WPR + lw) * 32 + lane;
    g[i] = v < nvec ? load8((const T*)a.gain + v * 8) : zero8<T>();
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = 0.f;
  }
  int flip = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * R; t0 < a.T; t0 += (int64_t)gridDim.x * R, flip ^= 1) {
    const int64_t t = t0 + r;
    const bool row_ok = t < a.T;
    const float rstd = row_ok ? a.rstd[t] : 0.f;
    Raw8<T> dy[VPT];
    uint2 q[VPT];
    uint32_t e[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = (i * WPR + lw) * 32 + lane;
      dy[i] = zero8<T>();
      q[i] = make_uint2(0u, 0u);
      e[i] = 1u;
      if (row_ok && v < nvec) {
        dy[i] = load8((const T*)a.x + t * a.d + v * 8);
        q[i] = *reinterpret_cast<const uint2*>(a.q + t * a.d + v * 8);
        e[i] = a.e[t * nb + (v >> 2)];
      }
    }
    float c = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float h[8], d[8], w[8];
      act8_decode(q[i], act8_scale(e[i]), a.fmt, h);
      to_f32(dy[i], d);
      to_f32(g[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float dh = d[j] * (h[j] * rstd);
        dg[i][j] += dh;
        c = fmaf(dh, w[j], c);
      }
    }
    c = row_add<WPR>(c, red[flip], r, lw, lane) * inv_d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = (i * WPR + lw) * 32 + lane;
      if (!row_ok || v >= nvec) continue;
      float h[8], d[8], w[8];
      act8_decode(q[i], act8_scale(e[i]), a.fmt, h);
      to_f32(dy[i], d);
      to_f32(g[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = rstd * (d[j] * w[j] - h[j] * rstd * c);
      if (a.res) {
        float p[8];
        to_f32(load8((const T*)a.res + t * a.d + v * 8), p);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] += p[j];
      }
      store8((T*)a.y + t * a.d + v * 8, from_f32<T>(d));
    }
  }
  float* out = a.part + ((int64_t)blockIdx.x * R + r) * a.d;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = (i * WPR + lw) * 32 + lane;
    if (v < nvec) store8(out + v * 8, from_f32<float>(dg[i]));
  }
}

// 32 columns per block; each of 32 warps adds every 32nd line, then the warps' sums in order.
__global__ void __launch_bounds__(1024)
    norm_dgain_kernel(const float* __restrict__ part, int64_t rows, int d, bool accumulate,
                      float* __restrict__ out) {
  __shared__ float red[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  float acc = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int64_t r = warp; r < rows; r += 32) acc += part[r * d + c];
  }
  red[warp][lane] = acc;
  __syncthreads();
  if (warp == 0 && c < d) {
    for (int w = 1; w < 32; ++w) acc += red[w][lane];
    out[c] = accumulate ? out[c] + acc : acc;
  }
}

// Warps per row: the fewest whose lanes hold the row in at most four vectors each; rows of
// more than 1024 vectors take a block of 32 warps (handles have at most 3200 vectors).
int warps_per_row(int nvec) {
  for (int w = 1; w <= 8; w *= 2)
    if (nvec <= w * 128) return w;
  return 32;
}

template <typename F>
void pick_norm(int nvec, F&& f) {  // f(integral_constant WPR, integral_constant VPT)
  const int wpr = warps_per_row(nvec), vpt = (nvec + wpr * 32 - 1) / (wpr * 32);
  auto with = [&](auto w) {
    switch (vpt) {
      case 1: f(w, std::integral_constant<int, 1>{}); break;
      case 2: f(w, std::integral_constant<int, 2>{}); break;
      case 3: f(w, std::integral_constant<int, 3>{}); break;
      default: f(w, std::integral_constant<int, 4>{}); break;
    }
  };
  switch (wpr) {
    case 1: with(std::integral_constant<int, 1>{}); break;
    case 2: with(std::integral_constant<int, 2>{}); break;
    case 4: with(std::integral_constant<int, 4>{}); break;
    case 8: with(std::integral_constant<int, 8>{}); break;
    default: with(std::integral_constant<int, 32>{}); break;
  }
}

int rows_per_block(int nvec) {
  const int w = warps_per_row(nvec);
  return w > 8 ? 1 : 8 / w;
}

int64_t norm_bwd_blocks(int64_t T, int d, int num_sms) {
  const int R = rows_per_block(d / 8);
  const int64_t need = (T + R - 1) / R, most = (int64_t)num_sms * 4;
  return need < most ? need : most;
}

}  // namespace

void launch_act8_pack(bool bf16, const void* X, int64_t T, int cols, int fmt, uint8_t* q,
                      uint8_t* e, cudaStream_t s) {
  const int nvec = cols / 8, slabs = (nvec + kSlab - 1) / kSlab;
  const unsigned blocks = (unsigned)((T * slabs + 7) / 8);
  if (bf16)
    act8_pack_kernel<uint16_t><<<blocks, 256, 0, s>>>((const uint16_t*)X, T, nvec, slabs, fmt, q, e);
  else
    act8_pack_kernel<float><<<blocks, 256, 0, s>>>((const float*)X, T, nvec, slabs, fmt, q, e);
}

void launch_act8_unpack(bool bf16, const uint8_t* q, const uint8_t* e, int64_t T, int cols,
                        int fmt, void* out, cudaStream_t s) {
  const int nvec = cols / 8, slabs = (nvec + kSlab - 1) / kSlab;
  const unsigned blocks = (unsigned)((T * slabs + 7) / 8);
  if (bf16)
    act8_unpack_kernel<uint16_t><<<blocks, 256, 0, s>>>(q, e, T, nvec, slabs, fmt, (uint16_t*)out);
  else
    act8_unpack_kernel<float><<<blocks, 256, 0, s>>>(q, e, T, nvec, slabs, fmt, (float*)out);
}

void launch_norm_fwd(const NormArgs& a, bool bf16, cudaStream_t s) {
  const int R = rows_per_block(a.d / 8);
  const unsigned blocks = (unsigned)((a.T + R - 1) / R);
  pick_norm(a.d / 8, [&](auto w, auto v) {
    constexpr int WPR = decltype(w)::value, VPT = decltype(v)::value;
    if (bf16) norm_fwd_kernel<uint16_t, WPR, VPT><<<blocks, kNormThreads<WPR>, 0, s>>>(a);
    else norm_fwd_kernel<float, WPR, VPT><<<blocks, kNormThreads<WPR>, 0, s>>>(a);
  });
}

int64_t norm_part_rows(int64_t T, int d, int num_sms) {
  return norm_bwd_blocks(T, d, num_sms) * rows_per_block(d / 8);
}

void launch_norm_bwd(const NormArgs& a, bool bf16, int num_sms, cudaStream_t s) {
  const unsigned blocks = (unsigned)norm_bwd_blocks(a.T, a.d, num_sms);
  pick_norm(a.d / 8, [&](auto w, auto v) {
    constexpr int WPR = decltype(w)::value, VPT = decltype(v)::value;
    if (bf16) norm_bwd_kernel<uint16_t, WPR, VPT><<<blocks, kNormThreads<WPR>, 0, s>>>(a);
    else norm_bwd_kernel<float, WPR, VPT><<<blocks, kNormThreads<WPR>, 0, s>>>(a);
  });
}

void launch_norm_dgain(const float* part, int64_t rows, int d, bool accumulate, float* out,
                       cudaStream_t s) {
  norm_dgain_kernel<<<(unsigned)((d + 31) / 32), 1024, 0, s>>>(part, rows, d, accumulate, out);
}

}  // namespace ckl
