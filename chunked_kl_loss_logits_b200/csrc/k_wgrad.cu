// Weight gradient of a linear layer whose input is kept as an 8-bit checkpoint:
//
//     dW[n][c] (+)= sum_t dY[t][n] X'[t][c],    X'[t][c] = code[t][c] * 2^e[t][c / 32]
//
// on the tensor cores. X' has at most 8 significant bits, so bf16 holds it exactly (from 2^-126
// on; below that to 2^-134): it is
// unpacked to a bf16 workspace first. bf16 dY enters as it is; fp32 dY is cut into three bf16
// parts of 8 bits each that are contracted one after the other, so both types get exact products
// and fp32 sums. (The parts add up to dY exactly from 2^-110 on; of a smaller number they leave out
// what lies below bf16's smallest, 2^-133.)
//
// Bound by the tensor cores: 2 T n c operations (three times that for fp32) against T (2n + c)
// bytes, a thousand operations a byte at n = c = 2880.
//
// Work unit: a 256 x 256 tile of dW and a range of tokens, by a CTA pair
// (tcgen05.mma.cta_group::2), 64 tokens a step. Both operands are MN-major as they lie in
// memory, and come by TMA. The tensor cores cut the running sum at each step instead of
// rounding it: a relative error that grows with the number of steps (1.2e-6 at 2048 tokens, 3e-5
// at 32768). So an accumulator sums kFlush steps only, and the epilogue warps, whose registers
// hold the CTA's 128 x 256 share of the tile, add it up there in fp32 while the MMAs fill
// the other accumulator. (Adding to dW in L2 instead costs 25 us every 64 steps at 32768 x 2880 x
// 2880.) The parts of an fp32 dY are contracted smallest first, which keeps their errors as
// small as they are. Roles, per CTA (320 threads):
//   warp 0      TMA producer (both CTAs; completion on the even CTA's `full`)
//   warp 1      allocates TMEM; in the even CTA one thread issues the MMAs
//   warps 2..9  epilogue: 32 accumulator rows by 128 columns each
// Every wait is bounded (common.cuh).
//
// Converting the codes inside the contraction (by further warps, from the codes in shared
// memory or in registers) was measured and not kept: 570 us and more at 32768 x 2880 x 2880, where
// unpacking first took 488 then, both over 25 calls from a cool start (477 now; 560 under the power
// limit, at which the two were not compared). The extra passes over shared memory (codes in and
// out, bf16 in) take bandwidth that the MMA needs for its operands; unpacking first moves 3 bytes a
// code through HBM and L2 instead. The epilogue's 128 sums a thread leave the 168 registers short
// by 24 bytes, which are spilled.
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
constexpr int kStages = 6;
constexpr int kAtom = 64 * 128;               // 64 (MN) x 64 (K) bf16
constexpr int kABytes = 2 * kAtom, kBBytes = 2 * kAtom, kStageBytes = kABytes + kBBytes;
constexpr int kEpiWarps = 8;                  // two per lane quarter of TMEM, 128 columns each
constexpr int kWgThreads = (2 + kEpiWarps) * 32;
constexpr int kTmemCols = 512, kAccCols = 256;
constexpr int kFlush = 16;                    // steps (of 64 tokens) one accumulator sums
constexpr int kBox = 32 * 128;                // a staged 32 x 32 fp32 box of an epilogue warp
constexpr int kWgSmem = 1024 + kStages * kStageBytes + kEpiWarps * kBox + 256;
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
// Store or add a staged box at (column c0, row c1) of plane c2; rows and columns outside are
// not written.
__device__ __forceinline__ void tma_put_3d(const CUtensorMap* m, const void* src, int c0, int c1,
                                           int c2, bool add) {
  if (add)
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group"
        " [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(m)),
        "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
            reinterpret_cast<uint64_t>(m)),
        "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// sum += 16 consecutive f32 columns of this thread's TMEM lane (warp-collective).
__device__ __forceinline__ void tmem_add16(uint32_t taddr, float* sum) {
  uint32_t r[16];
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) sum[i] += __uint_as_float(r[i]);
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

__global__ void __launch_bounds__(kWgThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmC, const WgradArgs p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* boxes = smem + kStages * kStageBytes;  // one for each epilogue warp
  uint64_t* full = reinterpret_cast<uint64_t*>(boxes + kEpiWarps * kBox);  // even CTA's in use
  uint64_t* empty = full + kStages;     // both CTAs
  uint64_t* tfull = empty + kStages;    // [2] both CTAs
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
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < n_tiles; tile += n_pairs) {
        const WgTile c = wg_tile(p, n_m, n_n, tile);
        const int row0 = c.mt * 2 * kBM + (int)rank * kBM, col0 = c.nt * kBN + (int)rank * kBNH;
        for (int kb = c.kb0; kb < c.kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
          unsigned char* sA = smem + stage * kStageBytes;
          const uint32_t fbar = cluster_map(&full[stage], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
          const int part = kb / p.kb_part, t0 = (kb - part * p.kb_part) * kBK;
#pragma unroll
          for (int a = 0; a < 2; ++a)
            tma_load_3d_pair(sA + a * kAtom, &tmA, fbar, row0 + a * 64, t0, part);
#pragma unroll
          for (int a = 0; a < 2; ++a)
            tma_load_2d_pair(sA + kABytes + a * kAtom, &tmB, fbar, col0 + a * 64, t0);
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
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;           // TMEM lane quarter this warp may access
    const int half = (warp - 2) >> 2;  // its 128 of the accumulator's 256 columns
    unsigned char* box = boxes + (warp - 2) * kBox;
    int it = 0;
    bool ok = true;
    for (int tile = pair; ok && tile < n_tiles; tile += n_pairs) {
      const WgTile c = wg_tile(p, n_m, n_n, tile);
      const int row0 = c.mt * 2 * kBM + (int)rank * kBM + q * 32;  // this warp's rows of dW
      const int col0 = c.nt * kBN + half * 128;
      float sum[128];  // this thread's row: the accumulators taken out so far
#pragma unroll
      for (int j = 0; j < 128; ++j) sum[j] = 0.f;
      for (int kf = c.kb0; kf < c.kb1; kf += kFlush, ++it) {
        const int buf = it & 1;
        if (!mbar_wait(&tfull[buf], (uint32_t)(it >> 1) & 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t taddr =
            tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * kAccCols + half * 128);
#pragma unroll
        for (int cc = 0; cc < 8; ++cc) tmem_add16(taddr + cc * 16, &sum[cc * 16]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_map(&tempty[buf], 0));
      }
      if (!ok) break;
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        if (col0 + cc * 32 < p.cols && row0 < p.n) {
          if (lane == 0) bulk_wait_read<0>();  // the box's previous contents have been read
          __syncwarp();
          uint4* rowp = reinterpret_cast<uint4*>(box + lane * 128);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            rowp[j ^ (lane & 7)] = make_uint4(
                __float_as_uint(sum[cc * 32 + 4 * j]), __float_as_uint(sum[cc * 32 + 4 * j + 1]),
                __float_as_uint(sum[cc * 32 + 4 * j + 2]), __float_as_uint(sum[cc * 32 + 4 * j + 3]));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_put_3d(&tmC, box, col0 + cc * 32, row0, c.split, p.add);
            bulk_commit();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
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
// up to the value exactly (but for bits below 2^-133) and none overflows; the part of the lowest
// bits first.
__global__ void __launch_bounds__(256) split3_kernel(const float* __restrict__ x, int64_t n8,
                                                     uint16_t* __restrict__ out) {
  griddep_launch_dependents();
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
    wgrad_sum_kernel(const float4* part, int n_split, int64_t n4, bool add, float4* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  griddep_wait();
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

cudaError_t launch_wgrad(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c,
                         const WgradArgs& p, int num_sms, cudaStream_t s) {
  const int n_tiles = (p.n + 2 * kBM - 1) / (2 * kBM) * ((p.cols + kBN - 1) / kBN) * p.n_split;
  static std::atomic<uint64_t> attr_set{0};
  cudaError_t e = smem_once(wgrad_kernel, kWgSmem, attr_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kWgThreads, 1, 1);
  cfg.dynamicSmemBytes = kWgSmem;
  cfg.stream = s;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // As many pairs as can be resident at once (cached; concurrent first calls agree).
  static std::atomic<int> cached_pairs{0};
  int pairs = cached_pairs.load(std::memory_order_relaxed);
  if (pairs == 0) {
    cfg.gridDim = dim3((unsigned)(2 * num_sms), 1, 1);
    if (cudaOccupancyMaxActiveClusters(&pairs, wgrad_kernel, &cfg) != cudaSuccess ||
        pairs < 1)
      pairs = std::max(1, num_sms / 2);
    cached_pairs.store(pairs, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3((unsigned)(2 * std::min(n_tiles, pairs)), 1, 1);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, wgrad_kernel, a, b, c, p);
}

void launch_split3(const float* x, int64_t n, uint16_t* out, cudaStream_t s) {
  split3_kernel<<<(unsigned)((n / 8 + 255) / 256), 256, 0, s>>>(x, n / 8, out);
}

cudaError_t launch_wgrad_sum(const float* part, int n_split, int64_t n, bool add, float* out,
                             cudaStream_t s) {
  return launch_behind(wgrad_sum_kernel, dim3((unsigned)((n / 4 + 255) / 256)), 256, 0, s,
                       reinterpret_cast<const float4*>(part), n_split, n / 4, add,
                       reinterpret_cast<float4*>(out));
}

}  // namespace ckl
