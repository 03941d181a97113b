// Device helpers of the operators around the loss (embedding, 8-bit activation
// checkpoints, norm): eight neighbouring elements at a time, warp reductions, and
// the 8-bit block format.
//
// The 8-bit format. A row's columns are cut into blocks of 32 (the last one may be
// shorter). A block with largest magnitude A keeps one byte e + 127 and a code per
// element, value = code * 2^e, where e >= -126 is the smallest exponent with
// A <= M * 2^e; M is the largest code (int8: 127, e4m3: 448). Scaling by 2^-e is exact,
// so a code is the one rounding (to nearest, ties to even) of its element: off by at
// most half a step, 2^(e-1) < A / 127 for int8, and by at most 2^-4 of the value for
// e4m3 above its subnormals. A power of two costs int8 up to one bit against a free
// scale; in return every value has at most 8 significant bits and is exact in bf16, so
// the matrix product that reads a checkpoint adds no rounding of its own. A block that
// holds an infinity or a NaN gets the byte 255 and reads back as NaN.
#pragma once

#include <cuda_fp8.h>

#include <atomic>

#include "common.cuh"

namespace ckl {

// Allow `fn` its dynamic shared memory: once per device (a bit of `set` per ordinal), so a
// call made during stream capture changes no attribute.
template <typename F>
cudaError_t smem_once(F* fn, size_t bytes, std::atomic<uint64_t>& set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t{1} << dev) : 0;
  if (bit && (set.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) set.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launch behind the kernel just enqueued on s, which it may overlap up to its griddep_wait(): the
// kernel calls that before it touches what the one before wrote or reads what that may write (and
// takes no such pointer as const __restrict__: its loads are not read-only for the kernel's life).
template <typename... P, typename... A>
cudaError_t launch_behind(void (*fn)(P...), dim3 grid, unsigned threads, size_t smem,
                          cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

constexpr int kActInt8 = 0, kActE4m3 = 1;  // ckl_act8_format
constexpr int kActBlock = 32;

template <typename T>
struct Raw8;  // eight elements as loaded
template <>
struct Raw8<uint16_t> {
  uint4 u;
};
template <>
struct Raw8<float> {
  float4 a, b;
};

__device__ __forceinline__ Raw8<uint16_t> load8(const uint16_t* p) {
  return {*reinterpret_cast<const uint4*>(p)};
}
__device__ __forceinline__ Raw8<float> load8(const float* p) {
  return {reinterpret_cast<const float4*>(p)[0], reinterpret_cast<const float4*>(p)[1]};
}
__device__ __forceinline__ void to_f32(const Raw8<uint16_t>& r, float (&v)[8]) {
  v[0] = lo_bf16(r.u.x); v[1] = hi_bf16(r.u.x);
  v[2] = lo_bf16(r.u.y); v[3] = hi_bf16(r.u.y);
  v[4] = lo_bf16(r.u.z); v[5] = hi_bf16(r.u.z);
  v[6] = lo_bf16(r.u.w); v[7] = hi_bf16(r.u.w);
}
__device__ __forceinline__ void to_f32(const Raw8<float>& r, float (&v)[8]) {
  v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
  v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
template <typename T>
__device__ __forceinline__ Raw8<T> from_f32(const float (&v)[8]);
template <>
__device__ __forceinline__ Raw8<uint16_t> from_f32<uint16_t>(const float (&v)[8]) {
  return {make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7]))};
}
template <>
__device__ __forceinline__ Raw8<float> from_f32<float>(const float (&v)[8]) {
  return {make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7])};
}
__device__ __forceinline__ void store8(uint16_t* p, const Raw8<uint16_t>& r) {
  *reinterpret_cast<uint4*>(p) = r.u;
}
__device__ __forceinline__ void store8(float* p, const Raw8<float>& r) {
  reinterpret_cast<float4*>(p)[0] = r.a;
  reinterpret_cast<float4*>(p)[1] = r.b;
}
template <typename T>
__device__ __forceinline__ Raw8<T> zero8() {
  const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  return from_f32<T>(z);
}

// Copies of 16 or 8 bytes to shared memory that go on while the thread does; a thread waits for
// its own, in groups.
template <int N>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  static_assert(N == 16 || N == 8, "");
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Wait until at most N of this thread's groups are under way.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Eight elements by cp.async, and back from there.
__device__ __forceinline__ void copy8(Raw8<uint16_t>* dst, const uint16_t* src) {
  cp_async<16>(dst, src);
}
__device__ __forceinline__ void copy8(Raw8<float>* dst, const float* src) {
  cp_async<16>(&dst->a, src);
  cp_async<16>(&dst->b, src + 4);
}

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Bits of the largest magnitude among eight elements (a NaN's bits are above every other's).
__device__ __forceinline__ uint32_t amax_bits8(const Raw8<float>& r) {
  uint32_t m = 0;
  const float v[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}
__device__ __forceinline__ uint32_t amax_bits8(const Raw8<uint16_t>& r) {
  constexpr uint32_t k = 0x7FFF7FFFu;  // two elements at a time
  const uint32_t m = __vmaxu2(__vmaxu2(r.u.x & k, r.u.y & k), __vmaxu2(r.u.z & k, r.u.w & k));
  return max(m << 16, m & 0xFFFF0000u);
}
// The same over the four lanes of a block (the whole warp calls it).
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}
// Scale byte of a block: 127 = 1.984375 * 2^6 and 448 = 1.75 * 2^8, so the smallest
// exponent follows from the magnitude's own exponent and fraction bits.
template <int FMT>
__device__ __forceinline__ uint32_t act8_scale_byte(uint32_t amax) {
  const int ex = (int)(amax >> 23);
  if (ex == 255) return 255u;
  const uint32_t frac = amax & 0x7FFFFFu;
  const int b = FMT == kActInt8 ? ex - 6 + (frac > 0x7E0000u) : ex - 8 + (frac > 0x600000u);
  return (uint32_t)max(b, 1);
}
// Codes of eight elements under the block's scale byte.
template <int FMT>
__device__ __forceinline__ uint2 act8_encode(const float (&x)[8], uint32_t byte) {
  if (byte == 255u) return make_uint2(0u, 0u);
  const float inv = __uint_as_float((254u - byte) << 23);  // 2^-e
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x[i];
  if (byte >= 247u) {
    // the largest magnitudes of fp32 and bf16 would round up to 2^128: the code below it
    const float lim = (FMT == kActE4m3 ? 240.f : byte >= 249u ? 63.f : 127.f) *
                      __uint_as_float(byte << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], -lim), lim);
  }
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (FMT == kActInt8) {
      // 1.5 * 2^23 + x / 2^e is rounded to a whole number, whose two's complement is in the low
      // bits (conversion instructions run at a quarter of the rate)
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(fmaf(v[4 * j + i], inv, 12582912.f));
      w[j] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    } else {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * j] * inv, v[4 * j + 1] * inv),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(
          make_float2(v[4 * j + 2] * inv, v[4 * j + 3] * inv), __NV_SATFINITE, __NV_E4M3);
      w[j] = lo | hi << 16;
    }
  }
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ float act8_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : byte << 23);
}
template <int FMT>
__device__ __forceinline__ void act8_decode(uint2 q, float scale, float (&v)[8]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (FMT == kActInt8) {
      // a code's byte with its sign bit flipped, in the low bits of 2^23, is 2^23 + 128 + code
      const uint32_t x = w[j] ^ 0x80808080u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[4 * j + i] = (__uint_as_float(__byte_perm(x, 0x4B000000u, 0x7550 + i)) - 8388736.f) * scale;
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __half2 h(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j] >> (16 * i)),
                                                   __NV_E4M3));
        const float2 f = __half22float2(h);
        v[4 * j + 2 * i] = f.x * scale;
        v[4 * j + 2 * i + 1] = f.y * scale;
      }
    }
  }
}

}  // namespace ckl
