// Weight gradient of a linear layer whose input is kept as an 8-bit checkpoint:
//
//     dW[n][c] (+)= sum_t dY[t][n] X'[t][c],    X'[t][c] = code[t][c] * 2^e[t][c / 32]
//
// on the tensor cores, the codes turned into bf16 on their way into shared memory. X' has
// at most 8 significant bits, so bf16 holds it exactly. bf16 dY enters as it is; fp32 dY is
// cut into three bf16 parts of 8 bits each (their sum is dY exactly) that are contracted one
// after the other, so both types get exact products and fp32 sums.
//
// Bound by the tensor cores: 2 T n c operations (three times that for fp32) against T (2n + c)
// bytes, a thousand operations a byte at n = c = 2880. Reading the codes in the contraction
// instead of a bf16 copy saves writing that copy and reading it back (4 T c bytes).
//
// Work unit: a 256 x 256 tile of dW and a range of tokens, by a CTA pair
// (tcgen05.mma.cta_group::2), 64 tokens a step. Both operands are MN-major: dY by TMA, X' by
// two groups of four warps of each CTA that take the steps in turn: codes come to shared memory
// by cp.async (they need no alignment beyond 8 bytes, which a TMA copy would) and scales to
// registers, four of the group's steps ahead, are converted, and stored in the 128-byte
// swizzle that the MMA reads. The tensor cores cut the running sum at each step instead of rounding it: a relative
// error that grows with the number of steps (1e-6 at 2048 tokens, 1.5e-5 at 32768). So a
// tile's sum is taken out after kFlush steps, and added up in fp32 by the epilogue; the parts
// of an fp32 dY are contracted smallest first, which keeps their errors as small as they are.
// Roles, per CTA (480 threads):
//   warp 0      TMA producer of dY (both CTAs; completion on the even CTA's `full`)
//   warp 1      allocates TMEM; in the even CTA one thread issues the MMAs
//   warps 2..5  epilogue: the CTA's 128 accumulator rows, while the MMAs fill the other one
//   warps 6..13 converters (both CTAs; each warp arrives on its CTA's `conv`)
//   warp 14     publisher (both CTAs): waits for `conv`, makes the converters' stores visible to
//               the tensor cores (fence.proxy.async), arrives on the even CTA's `full`. Done by
//               the converters themselves, the fence waits for the loads they have in flight:
//               1428 us at 32768 x 2880 x 2880 where the publisher's take 966.
// Every wait is bounded (common.cuh).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "k_ops.h"
#include "ops.cuh"

namespace ckl {

namespace {

constexpr int kBM = 128;                      // dY columns (rows of dW) per CTA
constexpr int kBK = 64;                       // tokens a step
constexpr int kBN = 256, kBNH = kBN / 2;      // X' columns of the pair, of a CTA
constexpr int kStages = 5;
constexpr int kAtom = 64 * 128;               // 64 (MN) x 64 (K) bf16
constexpr int kABytes = 2 * kAtom, kBBytes = 2 * kAtom, kStageBytes = kABytes + kBBytes;
constexpr int kTmemCols = 512, kAccCols = 256;
constexpr int kConvWarps = 8, kGroups = 2;    // converter warps; groups that take steps in turn
constexpr int kDepth = 4;                     // steps of its own a group loads ahead
constexpr int kGroupWarps = kConvWarps / kGroups;
constexpr int kPass = kBK / (kGroupWarps * 4);  // tokens a converter thread has of a step
constexpr int kWgThreads = (7 + kConvWarps) * 32;
constexpr int kFlush = 64;                    // steps (of 64 tokens) one accumulator sums
constexpr int kRawBytes = kBK * kBNH;         // the codes of a step
constexpr int kWgSmem = 1024 + kStages * kStageBytes + kGroups * kDepth * kRawBytes + 256;
static_assert(kWgSmem <= 232448, "shared memory per CTA");
constexpr uint16_t kPair = 0x3;

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* m,
                                                 uint32_t bar_cluster, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// *dst += v in L2, with nothing to wait for. One thread makes all additions to an element, in
// its program's order, so the sums do not depend on timing.
__device__ __forceinline__ void red_add4(float4* dst, const float4& v) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}
// Copy of N bytes (8 or 16) to shared memory, tracked per thread in groups.
template <int N>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct WgTile {
  int mt, nt, split, kb0, kb1;
};
__device__ __forceinline__ WgTile wg_tile(const WgradArgs& p, int n_m, int n_n, int tile) {
  WgTile c;
  c.mt = tile % n_m;  // neighbouring pairs share the X' columns
  const int r = tile / n_m;
  c.nt = r % n_n;
  c.split = r / n_n;
  c.kb0 = c.split * p.kb_split;
  c.kb1 = min(p.n_kb, c.kb0 + p.kb_split);
  return c;
}

// 16 codes of a token from column c into shared memory, and their scale. Loads are
// unconditional (what is past the last token or column reads the last one's); V16: rows of
// codes start on 16-byte boundaries (cols % 16 == 0).
template <bool V16>
__device__ __forceinline__ void load_codes(const WgradArgs& p, int64_t t, int c, uint4* dst,
                                           uint32_t& e) {
  t = min(t, p.T - 1);
  const uint8_t* src = p.q + t * p.cols;
  e = p.e[t * p.nb + min(c >> 5, p.nb - 1)];
  if (V16) {
    cp_async<16>(dst, src + min(c, p.cols - 16));
  } else {
    cp_async<8>(dst, src + min(c, p.cols - 8));
    cp_async<8>(reinterpret_cast<uint2*>(dst) + 1, src + min(c + 8, p.cols - 8));
  }
}

// Four codes to bf16. int8: a code's byte with its sign bit flipped, in the low bits of
// 2^23, is 2^23 + 128 + code.
template <int FMT>
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w, float scale) {
  float f[4];
  if (FMT == kActInt8) {
    w ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = (__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7550 + i)) - 8388736.f) * scale;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2 h(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3));
      const float2 v = __half22float2(h);
      f[2 * i] = v.x * scale;
      f[2 * i + 1] = v.y * scale;
    }
  }
  return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}

template <int FMT, bool V16>
__global__ void __launch_bounds__(kWgThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap tmA, const WgradArgs p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes +
                                                kGroups * kDepth * kRawBytes);  // even CTA's in use
  uint64_t* empty = full + kStages;     // both CTAs
  uint64_t* conv = empty + kStages;     // both CTAs
  uint64_t* tfull = conv + kStages;     // [2] both CTAs
  uint64_t* tempty = tfull + 2;         // [2] even CTA's in use
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int n_m = (p.n + 2 * kBM - 1) / (2 * kBM), n_n = (p.cols + kBN - 1) / kBN;
  const int n_tiles = n_m * n_n * p.n_split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1 + 2);  // the byte count of dY, the publishers
      mbar_init(&empty[s], 1);
      mbar_init(&conv[s], kGroupWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * 4);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tmA);
  if (warp == 1) tmem_alloc_pair(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ dY producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < n_tiles; tile += n_pairs) {
        const WgTile c = wg_tile(p, n_m, n_n, tile);
        const int row0 = c.mt * 2 * kBM + (int)rank * kBM;
        for (int kb = c.kb0; kb < c.kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
          unsigned char* sA = smem + stage * kStageBytes;
          const uint32_t fbar = cluster_map(&full[stage], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kABytes);
          const int part = kb / p.kb_part, t0 = (kb - part * p.kb_part) * kBK;
#pragma unroll
          for (int a = 0; a < 2; ++a)
            tma_load_3d_pair(sA + a * kAtom, &tmA, fbar, row0 + a * 64, t0, part);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
      // no copy is in flight when the CTA exits
      for (int s = 0; s < kStages; ++s) {
        if (!((issued >> s) & 1u)) continue;
        const long long t0 = clock64();
        while (!mbar_try_wait(&empty[s], (issued_phase >> s) & 1u)) {
          if (clock64() - t0 > kWaitCycles) { atomicOr(p.status, (unsigned)ST_TIMEOUT); break; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = umma_idesc_bf16(2 * kBM, kBN, true, true);
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < n_tiles; tile += n_pairs) {
        const WgTile c = wg_tile(p, n_m, n_n, tile);
        for (int kf = c.kb0; ok && kf < c.kb1; kf += kFlush, ++it) {
          const int buf = it & 1;
          if (!mbar_wait(&tempty[buf], ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + (uint32_t)(buf * kAccCols);
          for (int kb = kf; kb < min(kf + kFlush, c.kb1); ++kb) {
            if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) { ok = false; break; }
            tc_fence_after();
            const uint32_t a0 = smem_u32(smem + stage * kStageBytes), b0 = a0 + kABytes;
  #pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)
              umma_bf16_pair(d_tmem, umma_desc_sw128(a0 + kk * 2048, kAtom, 1024),
                             umma_desc_sw128(b0 + kk * 2048, kAtom, 1024), idesc,
                             (kb > kf || kk > 0) ? 1u : 0u);
            umma_commit_pair_mc(&empty[stage], kPair);
            if (++stage == kStages) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          umma_commit_pair_mc(&tfull[buf], kPair);
        }
      }
      umma_commit_pair(done);
      const long long t0 = clock64();
      while (!mbar_try_wait(done, 0)) {
        if (clock64() - t0 > kWaitCycles) { atomicOr(p.status, (unsigned)ST_TIMEOUT); break; }
      }
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    int it = 0;
    bool ok = true;
    for (int tile = pair; ok && tile < n_tiles; tile += n_pairs) {
      const WgTile c = wg_tile(p, n_m, n_n, tile);
      for (int kf = c.kb0; kf < c.kb1; kf += kFlush, ++it) {
        const int buf = it & 1;
        if (!mbar_wait(&tfull[buf], (uint32_t)(it >> 1) & 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool add = p.add || kf > c.kb0;
        const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * kAccCols);
        const int row = c.mt * 2 * kBM + (int)rank * kBM + q * 32 + lane;
        float* out = p.out + ((int64_t)c.split * p.n + row) * p.cols;
#pragma unroll 1
        for (int cc = 0; cc < kBN / 32; ++cc) {
          const int cb = c.nt * kBN + cc * 32;
          if (cb >= p.cols) break;
          float v[32];
          tmem_ld32(taddr + cc * 32, v);
          if (row >= p.n) continue;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (cb + 4 * j >= p.cols) break;  // cols % 8 == 0: whole vectors
            float4* dst = reinterpret_cast<float4*>(out + cb + 4 * j);
            const float4 o = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            if (add) red_add4(dst, o);
            else *dst = o;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_map(&tempty[buf], 0));
      }
    }
  } else if (warp == 6 + kConvWarps) {
    // ------------------------------------------------------------ publisher
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < n_tiles; tile += n_pairs) {
        const WgTile c = wg_tile(p, n_m, n_n, tile);
        for (int kb = c.kb0; kb < c.kb1; ++kb) {
          if (!mbar_wait(&conv[stage], phase, abort_flag, p.status)) { ok = false; break; }
          fence_proxy_async_smem();
          mbar_arrive_cluster(cluster_map(&full[stage], 0));
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ converters
    // Group g has every kGroups-th step. Eight neighbouring threads read 128 neighbouring
    // codes of a token: a thread has 16 of each of the tokens r0, r0 + 4 kGroupWarps, ... and
    // reads back from shared memory only what it copied there itself.
    const int g = (warp - 6) / kGroupWarps, ct = threadIdx.x - (6 + g * kGroupWarps) * 32;
    const int seg = ct & 7, r0 = ct >> 3;
    uint4* raw = reinterpret_cast<uint4*>(smem + kStages * kStageBytes + g * kDepth * kRawBytes) + ct;
    unsigned char* dst0 = smem + kABytes + (seg >> 2) * kAtom + r0 * 128;
    int cnt = 0;  // steps of the tiles before
    bool ok = true;
    for (int tile = pair; ok && tile < n_tiles; tile += n_pairs) {
      const WgTile c = wg_tile(p, n_m, n_n, tile);
      const int col = c.nt * kBN + (int)rank * kBNH + seg * 16;
      const int first = c.kb0 + (g - cnt % kGroups + kGroups) % kGroups;
      uint32_t e[kDepth][kPass];
      auto token = [&](int kb, int h) {
        return (int64_t)(kb % p.kb_part) * kBK + r0 + 4 * kGroupWarps * h;
      };
      auto slot = [&](int u, int h) { return raw + u * (kRawBytes / 16) + h * 32 * kGroupWarps; };
      auto fetch = [&](int kb, int u) {
#pragma unroll
        for (int h = 0; h < kPass; ++h)
          load_codes<V16>(p, token(min(kb, c.kb1 - 1), h), col, slot(u, h), e[u][h]);
        cp_async_commit();
      };
#pragma unroll
      for (int u = 0; u < kDepth; ++u) fetch(first + u * kGroups, u);
      for (int kb0 = first; ok && kb0 < c.kb1; kb0 += kDepth * kGroups) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
          const int kb = kb0 + u * kGroups;
          if (!ok || kb >= c.kb1) break;
          const int at = cnt + kb - c.kb0, stage = at % kStages;
          const uint32_t phase = (uint32_t)(at / kStages) & 1u;
          cp_async_wait<kDepth - 1>();
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
#pragma unroll
          for (int h = 0; h < kPass; ++h) {
            const bool in = token(kb, h) < p.T;  // past the last token: zeros, as dY has there
            const float scale = act8_scale(in ? e[u][h] : 1u);
            const uint4 q = in ? *slot(u, h) : make_uint4(0u, 0u, 0u, 0u);
            const uint2 a = codes_to_bf16<FMT>(q.x, scale), b = codes_to_bf16<FMT>(q.y, scale);
            const uint2 d = codes_to_bf16<FMT>(q.z, scale), f = codes_to_bf16<FMT>(q.w, scale);
            const uint4 lo = make_uint4(a.x, a.y, b.x, b.y), hi = make_uint4(d.x, d.y, f.x, f.y);
            // 16-byte chunk i of row r sits at i ^ (r % 8); the second atom's threads store
            // their halves in the other order, so that eight threads meet eight banks
            uint4* dst = reinterpret_cast<uint4*>(dst0 + stage * kStageBytes +
                                                  h * 4 * kGroupWarps * 128);
            const int i = 2 * (seg & 3), sw = (r0 + 4 * kGroupWarps * h) & 7, odd = seg >> 2;
            dst[(i + odd) ^ sw] = odd ? hi : lo;
            dst[(i + 1 - odd) ^ sw] = odd ? lo : hi;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&conv[stage]);
          fetch(kb + kDepth * kGroups, u);
        }
      }
      cp_async_wait<0>();
      cnt += c.kb1 - c.kb0;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// fp32 -> three bf16 parts, cut (not rounded) after 8 significant bits each, so that they add
// up to the value exactly and none overflows; the part of the lowest bits first.
__global__ void __launch_bounds__(256) split3_kernel(const float* __restrict__ x, int64_t n8,
                                                     uint16_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  float v[8];
  to_f32(load8(x + i * 8), v);
#pragma unroll
  for (int part = 0; part < 3; ++part) {
    float h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool fin = isfinite(v[j]);
      h[j] = fin ? __uint_as_float(__float_as_uint(v[j]) & 0xFFFF0000u) : v[j];
      v[j] = fin ? v[j] - h[j] : 0.f;
    }
    store8(out + ((int64_t)(2 - part) * n8 + i) * 8, from_f32<uint16_t>(h));
  }
}

// out (+)= the sum of n_split partial results, in order.
__global__ void __launch_bounds__(256)
    wgrad_sum_kernel(const float4* __restrict__ part, int n_split, int64_t n4, bool add,
                     float4* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  float4 s = part[i];
  for (int k = 1; k < n_split; ++k) {
    const float4 b = part[k * n4 + i];
    s = make_float4(s.x + b.x, s.y + b.y, s.z + b.z, s.w + b.w);
  }
  if (add) {
    const float4 o = out[i];
    s = make_float4(o.x + s.x, o.y + s.y, o.z + s.z, o.w + s.w);
  }
  out[i] = s;
}

template <int FMT, bool V16>
cudaError_t launch_one(const CUtensorMap& a, const WgradArgs& p, int num_sms, cudaStream_t s) {
  const int n_tiles = (p.n + 2 * kBM - 1) / (2 * kBM) * ((p.cols + kBN - 1) / kBN) * p.n_split;
  static std::atomic<uint64_t> attr_set{0};
  cudaError_t e = smem_once(wgrad_kernel<FMT, V16>, kWgSmem, attr_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kWgThreads, 1, 1);
  cfg.dynamicSmemBytes = kWgSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // As many pairs as can be resident at once (cached; concurrent first calls agree).
  static std::atomic<int> cached_pairs{0};
  int pairs = cached_pairs.load(std::memory_order_relaxed);
  if (pairs == 0) {
    cfg.gridDim = dim3((unsigned)(2 * num_sms), 1, 1);
    if (cudaOccupancyMaxActiveClusters(&pairs, wgrad_kernel<FMT, V16>, &cfg) != cudaSuccess ||
        pairs < 1)
      pairs = std::max(1, num_sms / 2);
    cached_pairs.store(pairs, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3((unsigned)(2 * std::min(n_tiles, pairs)), 1, 1);
  return cudaLaunchKernelEx(&cfg, wgrad_kernel<FMT, V16>, a, p);
}

}  // namespace

// Splits of the tokens: enough that the tiles fill the pairs evenly, weighed against writing
// and reading a partial dW for each (both in seconds, at the measured rates).
int wgrad_split(int64_t n, int64_t cols, int64_t n_kb, int num_sms) {
  const int64_t tiles = (n + 255) / 256 * ((cols + kBN - 1) / kBN);
  const int pairs = std::max(1, num_sms / 2);
  const double step = 2.0 * 256 * 256 * kBK / (1.6e15 / 74), part = 8.0 * n * cols / 6.5e12;
  int best = 1;
  double cost = 1e300;
  for (int s = 1; s <= 64 && (s == 1 || n_kb / s >= 4); ++s) {
    const int64_t waves = (tiles * s + pairs - 1) / pairs, kb = (n_kb + s - 1) / s;
    const double c = (double)waves * (double)kb * step + (s > 1 ? s * part : 0.0);
    if (c < cost * 0.98) { cost = c; best = s; }
  }
  const int64_t kps = (n_kb + best - 1) / best;  // no split without a step
  return (int)((n_kb + kps - 1) / kps);
}

cudaError_t launch_wgrad(const CUtensorMap& a, const WgradArgs& p, int fmt, int num_sms,
                         cudaStream_t s) {
  const bool v16 = p.cols % 16 == 0;
  if (fmt == kActInt8)
    return v16 ? launch_one<kActInt8, true>(a, p, num_sms, s)
               : launch_one<kActInt8, false>(a, p, num_sms, s);
  return v16 ? launch_one<kActE4m3, true>(a, p, num_sms, s)
             : launch_one<kActE4m3, false>(a, p, num_sms, s);
}

void launch_split3(const float* x, int64_t n, uint16_t* out, cudaStream_t s) {
  split3_kernel<<<(unsigned)((n / 8 + 255) / 256), 256, 0, s>>>(x, n / 8, out);
}

void launch_wgrad_sum(const float* part, int n_split, int64_t n, bool add, float* out,
                      cudaStream_t s) {
  wgrad_sum_kernel<<<(unsigned)((n / 4 + 255) / 256), 256, 0, s>>>(
      reinterpret_cast<const float4*>(part), n_split, n / 4, add, reinterpret_cast<float4*>(out));
}

}  // namespace ckl
