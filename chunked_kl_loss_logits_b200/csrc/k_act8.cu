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
// All of these are bound by memory. A row is read once, kept in registers (one vector of
// eight columns a lane, four lanes to an 8-bit block) while its sum goes round the warps that
// share it, and written from there.
#include "common.cuh"
#include "k_ops.h"
#include "ops.cuh"

namespace ckl {

namespace {

constexpr int kNoCkpt = -1;
constexpr int kSlab = 128;  // vectors of eight columns a warp handles of one row (pack, unpack)

// One warp for 128 vectors of a row, four in flight per lane; four lanes make an 8-bit block.
// Bound by memory: 32768 x 2880 bf16, pack 50 us (5.7 TB/s), unpack 46 us (6.2 TB/s), where a copy
// runs at 6.1. Codes by conversion instructions instead of one fused operation: 59 us.
template <typename T, int FMT>
__global__ void __launch_bounds__(256)
    act8_pack_kernel(const T* __restrict__ X, int64_t rows, int nvec, int slabs,
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
    const uint32_t byte = act8_scale_byte<FMT>(quad_max(amax_bits8(r[i])));
    if (v < nvec) {
      *reinterpret_cast<uint2*>(q + (t * nvec + v) * 8) = act8_encode<FMT>(f, byte);
      if ((lane & 3) == 0) e[t * nb + (v >> 2)] = (uint8_t)byte;
    }
  }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(256)
    act8_unpack_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ e, int64_t rows,
                       int nvec, int slabs, T* __restrict__ out) {
  griddep_launch_dependents();
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
    act8_decode<FMT>(c[i], act8_scale(b[i]), f);
    store8(out + (t * nvec + v) * 8, from_f32<T>(f));
  }
}

// The norm kernels: a block of WPR warps walks rows in steps of the grid, each lane with VPT
// vectors of eight columns. What it needs of the rows ahead is on its way to shared memory
// (cp.async, each thread its own vectors, so that nothing but the row sum is synchronised): two
// rows, as four keep fewer blocks on an SM (272 us against 275 for both passes below; 4096 x 2048
// without a residual, forward: two rows 11.0 us, three 11.4, four 12.0).
// 32768 x 2880 bf16 with a residual: forward 148 us (5.75 TB/s), backward 121 us (5.5 TB/s). Rows in
// registers alone, several to a block, took 173 and 215 us: the sums of dg leave room for too few
// warps to keep HBM busy without copies under way. Asking L2 for the scales of the rows ahead
// cost 8 us. Rows of 4 or 7 vectors a lane (above 8192 columns) spill registers, 24 to 172 bytes
// forward and 108 to 700 backward: 8192 bf16 rows with a residual run backward at 5.6 TB/s at 8192 columns,
// 4.2 at 16384 and 1.9 at 24000, forward at 5.3, 5.4 and 4.7.
template <typename T, int WPR, int VPT, bool BWD>
struct NormCfg {
  static constexpr int kThreads = WPR * 32;
  // Blocks per SM, in warps: 36 forward, 24 backward, whose sums of dg are in registers; 32 where a
  // power of two fills them at one vector a lane. 64 million elements backward with d_sum, in us with
  // 32 and with 24 warps: bf16 d = 256 96 and 95, 512 87 and 85, 1024 84 and 82, 2048 85 and 84,
  // 4096 87 and 99; fp32 137, 162, 173, 169, 138 and 137, 160, 170, 164, 152. So it gains at 16 warps a
  // row (d = 4096) and costs 1 to 3% below, without d_sum up to 8% (fp32 d = 512: 13%); rows of 6 or
  // 12 warps lose 3%.
  static constexpr bool kEven = VPT == 1 && (WPR & (WPR - 1)) == 0;
  static constexpr int kWant = (!BWD ? 36 : kEven ? 32 : 24) / WPR;
  static constexpr int kPerSm = kWant < 1 ? 1 : kWant > 16 ? 16 : kWant;
  static constexpr size_t kStage = (size_t)kThreads * VPT * (2 * sizeof(Raw8<T>) + (BWD ? 8 : 0));
  static constexpr size_t kRoom = 200 * 1024 / kPerSm;
  static constexpr int kDepth = kRoom / kStage >= 2 ? 2 : 1;
  static constexpr size_t kSmem = kStage * kDepth;
  static_assert(kSmem <= 200 * 1024, "shared memory per block");
};

// Sum over the WPR warps of a row (all threads of the block call it, `red` in turn).
template <int WPR>
__device__ __forceinline__ float row_add(float v, float* red, int warp, int lane) {
  v = warp_add(v);
  if (WPR == 1) return v;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float t = red[0];
#pragma unroll
  for (int w = 1; w < WPR; ++w) t += red[w];
  return t;
}

template <typename T, int WPR, int VPT, int FMT>  // FMT: the checkpoint's format or kNoCkpt
__global__ void __launch_bounds__(WPR * 32, NormCfg<T, WPR, VPT, false>::kPerSm)
    norm_fwd_kernel(const NormArgs a) {
  using C = NormCfg<T, WPR, VPT, false>;
  constexpr int D = C::kDepth;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[2][WPR];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nvec = a.d / 8, nb = (nvec + 3) / 4;
  Raw8<T>* xs = reinterpret_cast<Raw8<T>*>(smem) + threadIdx.x;  // [stage][x, res][i] of this thread
  auto slot = [&](int stage, int which, int i) {
    return xs + ((stage * 2 + which) * VPT + i) * C::kThreads;
  };
  auto vec = [&](int i) { return (i * WPR + warp) * 32 + lane; };
  auto fetch = [&](int64_t t, int stage) {
    if (t < a.T) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (vec(i) >= nvec) break;
        copy8(slot(stage, 0, i), (const T*)a.x + t * a.d + vec(i) * 8);
        if (a.res) copy8(slot(stage, 1, i), (const T*)a.res + t * a.d + vec(i) * 8);
      }
    }
    cp_async_commit();
  };
  const int64_t step = gridDim.x;
#pragma unroll
  for (int u = 0; u < D; ++u) fetch(blockIdx.x + u * step, u);
  Raw8<T> g[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    g[i] = vec(i) < nvec ? load8((const T*)a.gain + vec(i) * 8) : zero8<T>();
  int stage = 0, flip = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += step, flip ^= 1) {
    cp_async_wait<D - 1>();
    Raw8<T> s[VPT];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const bool ok = vec(i) < nvec;
      s[i] = ok ? *slot(stage, 0, i) : zero8<T>();
      float f[8];
      to_f32(s[i], f);
      if (a.res && ok) {
        float p[8];
        to_f32(*slot(stage, 1, i), p);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += p[j];
        s[i] = from_f32<T>(f);
        to_f32(s[i], f);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
    }
    fetch(t + D * step, stage);
    if (++stage == D) stage = 0;
    ss = row_add<WPR>(ss, red[flip], warp, lane);
    const float rstd = 1.f / sqrtf(ss / (float)a.d + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const bool ok = vec(i) < nvec;
      float f[8];
      to_f32(s[i], f);
      if (FMT != kNoCkpt) {
        const uint32_t byte = act8_scale_byte<FMT>(quad_max(amax_bits8(s[i])));
        if (ok) {
          *reinterpret_cast<uint2*>(a.q + t * a.d + vec(i) * 8) = act8_encode<FMT>(f, byte);
          if ((lane & 3) == 0) a.e[t * nb + (vec(i) >> 2)] = (uint8_t)byte;
        }
      }
      if (!ok) continue;
      if (a.res) store8((T*)a.sum + t * a.d + vec(i) * 8, s[i]);
      float w[8];
      to_f32(g[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * w[j];
      store8((T*)a.y + t * a.d + vec(i) * 8, from_f32<T>(f));
    }
  }
  cp_async_wait<0>();
}

// Keeps its columns' share of dg in registers and leaves it as one line of partial sums, added
// up by norm_dgain_kernel.
template <typename T, int WPR, int VPT, int FMT>
__global__ void __launch_bounds__(WPR * 32, NormCfg<T, WPR, VPT, true>::kPerSm)
    norm_bwd_kernel(const NormArgs a) {
  using C = NormCfg<T, WPR, VPT, true>;
  constexpr int D = C::kDepth;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[2][WPR];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nvec = a.d / 8, nb = (nvec + 3) / 4;
  const float inv_d = 1.f / (float)a.d;
  Raw8<T>* xs = reinterpret_cast<Raw8<T>*>(smem) + threadIdx.x;  // [stage][dY, dS][i]
  uint2* qs = reinterpret_cast<uint2*>(smem + (size_t)D * 2 * VPT * C::kThreads * sizeof(Raw8<T>)) +
              threadIdx.x;                                       // [stage][i]
  auto slot = [&](int stage, int which, int i) {
    return xs + ((stage * 2 + which) * VPT + i) * C::kThreads;
  };
  auto qslot = [&](int stage, int i) { return qs + (stage * VPT + i) * C::kThreads; };
  auto vec = [&](int i) { return (i * WPR + warp) * 32 + lane; };
  auto fetch = [&](int64_t t, int stage) {
    if (t < a.T) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (vec(i) >= nvec) break;
        copy8(slot(stage, 0, i), (const T*)a.x + t * a.d + vec(i) * 8);
        cp_async<8>(qslot(stage, i), a.q + t * a.d + vec(i) * 8);
        if (a.res) copy8(slot(stage, 1, i), (const T*)a.res + t * a.d + vec(i) * 8);
      }
    }
    cp_async_commit();
  };
  const int64_t step = gridDim.x;
  griddep_launch_dependents();
#pragma unroll
  for (int u = 0; u < D; ++u) fetch(blockIdx.x + u * step, u);
  Raw8<T> g[VPT];
  float dg[VPT][8];
  uint32_t e[VPT];
  float rstd = a.rstd[blockIdx.x];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    g[i] = vec(i) < nvec ? load8((const T*)a.gain + vec(i) * 8) : zero8<T>();
    e[i] = vec(i) < nvec ? a.e[(int64_t)blockIdx.x * nb + (vec(i) >> 2)] : 1u;
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = 0.f;
  }
  int stage = 0, flip = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += step, flip ^= 1) {
    const bool more = t + step < a.T;
    const float next_rstd = more ? a.rstd[t + step] : 0.f;
    uint32_t next_e[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      next_e[i] = more && vec(i) < nvec ? a.e[(t + step) * nb + (vec(i) >> 2)] : 1u;
    cp_async_wait<D - 1>();
    float ay[VPT][8], h[VPT][8];  // a = dY gain and h of the text above
    float c = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const bool ok = vec(i) < nvec;
      act8_decode<FMT>(ok ? *qslot(stage, i) : make_uint2(0u, 0u), act8_scale(e[i]) * rstd, h[i]);
      float d[8], w[8];
      to_f32(ok ? *slot(stage, 0, i) : zero8<T>(), d);
      to_f32(g[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ay[i][j] = d[j] * w[j];
        dg[i][j] = fmaf(d[j], h[i][j], dg[i][j]);
        c = fmaf(ay[i][j], h[i][j], c);
      }
    }
    c = row_add<WPR>(c, red[flip], warp, lane) * inv_d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (vec(i) >= nvec) continue;
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = rstd * fmaf(-h[i][j], c, ay[i][j]);
      if (a.res) {
        float p[8];
        to_f32(*slot(stage, 1, i), p);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] += p[j];
      }
      store8((T*)a.y + t * a.d + vec(i) * 8, from_f32<T>(d));
    }
    fetch(t + D * step, stage);
    if (++stage == D) stage = 0;
    rstd = next_rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) e[i] = next_e[i];
  }
  cp_async_wait<0>();
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (vec(i) < nvec) store8(a.part + (int64_t)blockIdx.x * a.d + vec(i) * 8, from_f32<float>(dg[i]));
}

// 32 columns per block; each of 32 warps adds every 32nd line, then the warps' sums in order.
__global__ void __launch_bounds__(1024)
    norm_dgain_kernel(const float* part, int64_t rows, int d, bool accumulate, float* out) {
  __shared__ float red[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  float acc = 0.f;
  griddep_wait();
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

// Warps per row and vectors per lane: one vector a lane up to 16 warps (4096 columns), then as
// many vectors as it takes (handles have at most 3200, in fp32 1600).
template <typename T, typename F>
void pick_norm(int nvec, F&& f) {  // f(integral_constant WPR, integral_constant VPT)
#define CKL_NORM_CASE(W, V)          \
  if (nvec <= W * 32 * V)            \
    return f(std::integral_constant<int, W>{}, std::integral_constant<int, V>{});
  CKL_NORM_CASE(1, 1)
  CKL_NORM_CASE(2, 1)
  CKL_NORM_CASE(3, 1)
  CKL_NORM_CASE(4, 1)
  CKL_NORM_CASE(6, 1)
  CKL_NORM_CASE(8, 1)
  CKL_NORM_CASE(12, 1)
  CKL_NORM_CASE(16, 1)
  CKL_NORM_CASE(16, 2)
  CKL_NORM_CASE(16, 4)
  if constexpr (sizeof(T) == 2) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 7>{});
#undef CKL_NORM_CASE
}

template <typename T, bool BWD>
int64_t norm_blocks(int64_t T_, int d, int num_sms) {
  int per_sm = 1;
  pick_norm<T>(d / 8, [&](auto w, auto v) {
    per_sm = NormCfg<T, decltype(w)::value, decltype(v)::value, BWD>::kPerSm;
  });
  const int64_t most = (int64_t)num_sms * per_sm;
  return T_ < most ? T_ : most;
}

template <typename T, int FMT>
cudaError_t norm_fwd(const NormArgs& a, int num_sms, cudaStream_t s) {
  const unsigned blocks = (unsigned)norm_blocks<T, false>(a.T, a.d, num_sms);
  cudaError_t err = cudaErrorInvalidValue;
  pick_norm<T>(a.d / 8, [&](auto w, auto v) {
    constexpr int WPR = decltype(w)::value, VPT = decltype(v)::value;
    using C = NormCfg<T, WPR, VPT, false>;
    static std::atomic<uint64_t> attr_set{0};
    err = smem_once(norm_fwd_kernel<T, WPR, VPT, FMT>, C::kSmem, attr_set);
    if (err == cudaSuccess)
      norm_fwd_kernel<T, WPR, VPT, FMT><<<blocks, C::kThreads, C::kSmem, s>>>(a);
  });
  return err;
}

template <typename T, int FMT>
cudaError_t norm_bwd(const NormArgs& a, int num_sms, cudaStream_t s) {
  const unsigned blocks = (unsigned)norm_blocks<T, true>(a.T, a.d, num_sms);
  cudaError_t err = cudaErrorInvalidValue;
  pick_norm<T>(a.d / 8, [&](auto w, auto v) {
    constexpr int WPR = decltype(w)::value, VPT = decltype(v)::value;
    using C = NormCfg<T, WPR, VPT, true>;
    static std::atomic<uint64_t> attr_set{0};
    err = smem_once(norm_bwd_kernel<T, WPR, VPT, FMT>, C::kSmem, attr_set);
    if (err == cudaSuccess)
      norm_bwd_kernel<T, WPR, VPT, FMT><<<blocks, C::kThreads, C::kSmem, s>>>(a);
  });
  return err;
}

template <typename T, int FMT>
void pack(const void* X, int64_t rows, int nvec, uint8_t* q, uint8_t* e, cudaStream_t s) {
  const int slabs = (nvec + kSlab - 1) / kSlab;
  act8_pack_kernel<T, FMT><<<(unsigned)((rows * slabs + 7) / 8), 256, 0, s>>>(
      static_cast<const T*>(X), rows, nvec, slabs, q, e);
}

template <typename T, int FMT>
void unpack(const uint8_t* q, const uint8_t* e, int64_t rows, int nvec, void* out, cudaStream_t s) {
  const int slabs = (nvec + kSlab - 1) / kSlab;
  act8_unpack_kernel<T, FMT><<<(unsigned)((rows * slabs + 7) / 8), 256, 0, s>>>(
      q, e, rows, nvec, slabs, static_cast<T*>(out));
}

}  // namespace

void launch_act8_pack(bool bf16, const void* X, int64_t T, int cols, int fmt, uint8_t* q,
                      uint8_t* e, cudaStream_t s) {
  if (fmt == kActInt8)
    bf16 ? pack<uint16_t, kActInt8>(X, T, cols / 8, q, e, s) : pack<float, kActInt8>(X, T, cols / 8, q, e, s);
  else
    bf16 ? pack<uint16_t, kActE4m3>(X, T, cols / 8, q, e, s) : pack<float, kActE4m3>(X, T, cols / 8, q, e, s);
}

void launch_act8_unpack(bool bf16, const uint8_t* q, const uint8_t* e, int64_t T, int cols,
                        int fmt, void* out, cudaStream_t s) {
  if (fmt == kActInt8)
    bf16 ? unpack<uint16_t, kActInt8>(q, e, T, cols / 8, out, s)
         : unpack<float, kActInt8>(q, e, T, cols / 8, out, s);
  else
    bf16 ? unpack<uint16_t, kActE4m3>(q, e, T, cols / 8, out, s)
         : unpack<float, kActE4m3>(q, e, T, cols / 8, out, s);
}

cudaError_t launch_norm_fwd(const NormArgs& a, bool bf16, int num_sms, cudaStream_t s) {
  if (!a.q)
    return bf16 ? norm_fwd<uint16_t, kNoCkpt>(a, num_sms, s) : norm_fwd<float, kNoCkpt>(a, num_sms, s);
  if (a.fmt == kActInt8)
    return bf16 ? norm_fwd<uint16_t, kActInt8>(a, num_sms, s)
                : norm_fwd<float, kActInt8>(a, num_sms, s);
  return bf16 ? norm_fwd<uint16_t, kActE4m3>(a, num_sms, s) : norm_fwd<float, kActE4m3>(a, num_sms, s);
}

int64_t norm_part_rows(int64_t T, int d, bool bf16, int num_sms) {
  return bf16 ? norm_blocks<uint16_t, true>(T, d, num_sms) : norm_blocks<float, true>(T, d, num_sms);
}

cudaError_t launch_norm_bwd(const NormArgs& a, bool bf16, int num_sms, cudaStream_t s) {
  if (a.fmt == kActInt8)
    return bf16 ? norm_bwd<uint16_t, kActInt8>(a, num_sms, s)
                : norm_bwd<float, kActInt8>(a, num_sms, s);
  return bf16 ? norm_bwd<uint16_t, kActE4m3>(a, num_sms, s) : norm_bwd<float, kActE4m3>(a, num_sms, s);
}

cudaError_t launch_norm_dgain(const float* part, int64_t rows, int d, bool accumulate, float* out,
                              cudaStream_t s) {
  return launch_behind(norm_dgain_kernel, dim3((unsigned)((d + 31) / 32)), 1024, 0, s, part, rows,
                       d, accumulate, out);
}

}  // namespace ckl
