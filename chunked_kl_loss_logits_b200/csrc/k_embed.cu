// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   out[t] = round(scale * W[id_t])
//   gradient  dW[v] (+)= scale * sum over { t : id_t = v } of dX[t]
//
// W is the V x d matrix of the LM head where the two are tied, and dW the fp32 buffer the
// fused loss wrote, so the gradient can be added in place. Both are bound by memory: the
// forward moves a row in and a row out per token; the gradient reads dX once and reads and
// writes the rows of the ids that occur. Atomic adds would read and write dW once per
// token and make the sums' order, hence their last bits, change from run to run; instead
// the tokens are sorted by (id, position) and each thread walks `tile` neighbouring sorted
// tokens with eight columns of the running row sum in registers.
#include "common.cuh"
#include "k_ops.h"
#include "ops.cuh"

namespace ckl {

namespace {

// The token's row among those held here, or V (mask 0, another rank's row, or out of range).
__device__ __forceinline__ int32_t token_row(const EmbedIds& a, int64_t t, bool& bad) {
  if (a.mask && a.mask[t] == 0) return a.V;
  const int32_t id = a.ids[t];
  if (id < 0 || id >= a.V_total) {
    bad = true;
    return a.V;
  }
  const int32_t r = id - a.v0;
  return r >= 0 && r < a.V ? r : a.V;
}

// One warp per (token, 128 vectors of 8 columns).
template <typename T, typename To>
__global__ void __launch_bounds__(256) embed_kernel(const EmbedIds a, const T* __restrict__ W,
                                                    int nvec, int slabs, float scale,
                                                    To* __restrict__ out) {
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = w / slabs;
  if (t >= a.T) return;
  const int v0 = (int)(w - t * slabs) * 128 + lane;
  bool bad = false;
  const int32_t row = token_row(a, t, bad);
  if (bad && lane == 0) atomicOr(a.status, (unsigned)ST_INDEX_RANGE);
  const bool have = row < a.V;
  const T* src = W + (int64_t)(have ? row : 0) * nvec * 8;
  To* dst = out + t * nvec * 8;
  Raw8<T> r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = v0 + i * 32;
    r[i] = have && v < nvec ? load8(src + (int64_t)v * 8) : zero8<T>();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = v0 + i * 32;
    if (v >= nvec) break;
    float f[8];
    to_f32(r[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = have ? f[j] * scale : 0.f;
    store8(dst + (int64_t)v * 8, from_f32<To>(f));
  }
}

// ------------------------------------------------------------------ sort
// Stable least-significant-digit radix sort by one cluster of CTAs. Each of the cluster's
// warps owns a contiguous range of the items, so "count per (digit, warp), prefix over
// digits, then over warps" gives every item its place, and equal keys keep their order.
// The digit counts of the other CTAs are read from their shared memory.
constexpr int kSortWarps = 32;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;
constexpr size_t kSortSmem = (size_t)(kSortWarps * kMaxBins + 2 * kMaxBins + 32) * 4;

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kSortWarps * 32, 1)
    embed_sort_kernel(const EmbedIds a, int n_pass, int bits, int cluster, uint64_t* buf_a,
                      uint64_t* buf_b) {
  extern __shared__ uint32_t sm[];
  uint32_t* hist = sm;                          // [warp][bin] counts, then places
  uint32_t* tot = sm + kSortWarps * kMaxBins;   // [bin] this CTA's counts (read by the others)
  uint32_t* base = tot + kMaxBins;              // [bin] first place of this CTA's items
  uint32_t* wsum = base + kMaxBins;             // [32]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank();
  const int bins = 1 << bits;
  const int64_t per = ((a.T + (int64_t)cluster * kSortWarps * 32 - 1) /
                       ((int64_t)cluster * kSortWarps * 32)) * 32;
  const int64_t i0 = min(a.T, ((int64_t)rank * kSortWarps + warp) * per);
  const int64_t i1 = min(a.T, i0 + per);
  uint32_t* myhist = hist + warp * bins;
  bool bad = false;

  for (int p = 0; p < n_pass; ++p) {
    const uint64_t* in = (p & 1) ? buf_a : buf_b;  // pass 0 reads the ids
    uint64_t* out = (p & 1) ? buf_b : buf_a;
    const int shift = 32 + p * bits;
    auto item = [&](int64_t i) -> uint64_t {
      if (p == 0) return (uint64_t)(uint32_t)token_row(a, i, bad) << 32 | (uint64_t)i;
      return __ldcg(reinterpret_cast<const unsigned long long*>(in) + i);
    };
    for (int b = lane; b < bins; b += 32) myhist[b] = 0;
    __syncwarp();
    for (int64_t i = i0 + lane; i < i1; i += 32)
      atomicAdd(&myhist[(uint32_t)(item(i) >> shift) & (bins - 1)], 1u);
    __syncthreads();
    uint32_t mine = 0;
    if (tid < bins) {
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = hist[w * bins + tid];
        hist[w * bins + tid] = mine;
        mine += c;
      }
      tot[tid] = mine;
    }
    cluster_sync();
    uint32_t before = 0, all = 0;
    if (tid < bins) {
      for (int r = 0; r < cluster; ++r) {
        const uint32_t c = ld_cluster_u32(cluster_map(tot + tid, (uint32_t)r));
        if (r < rank) before += c;
        all += c;
      }
    }
    // exclusive prefix of `all` over the bins (threads past the bins hold 0)
    uint32_t incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    if (tid < bins) {
      uint32_t pre = 0;
      for (int w = 0; w < warp; ++w) pre += wsum[w];
      base[tid] = pre + incl - all + before;
    }
    __syncthreads();
    for (int64_t ib = i0; ib < i1; ib += 32) {
      const int64_t i = ib + lane;
      const unsigned act = __ballot_sync(0xffffffffu, i < i1);
      if (i < i1) {
        const uint64_t it = item(i);
        const uint32_t dg = (uint32_t)(it >> shift) & (bins - 1);
        const unsigned same = __match_any_sync(act, dg);
        const uint32_t at = myhist[dg];
        __syncwarp(act);
        if (lane == __ffs(same) - 1) myhist[dg] = at + __popc(same);
        out[base[dg] + at + __popc(same & ((1u << lane) - 1))] = it;
      }
      __syncwarp();
    }
    // every item is in place, and no CTA still reads another's counts, before the next pass
    cluster_sync();
  }
  if (bad) atomicOr(a.status, (unsigned)ST_INDEX_RANGE);
}

// ------------------------------------------------------------------ gradient
__device__ __forceinline__ int32_t key_of(uint64_t it) { return (int32_t)(it >> 32); }

__device__ __forceinline__ void add_row8(float* dst, const float (&v)[8], float scale,
                                         bool accumulate) {
  float o[8];
  if (accumulate) {
    to_f32(load8(dst), o);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] += scale * v[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = scale * v[j];
  }
  store8(dst, from_f32<float>(o));
}

// One thread per (tile of sorted tokens, 8 columns). A row all of whose tokens lie in the
// tile is finished here. Of a row whose tokens span tiles, the sum of this tile's share goes
// to part: slot 0 where the row began in an earlier tile, slot 1 where it begins here.
template <typename T>
__global__ void __launch_bounds__(256)
    embed_grad_kernel(const uint64_t* __restrict__ sorted, int64_t n, int32_t V,
                      const T* __restrict__ dX, int nvec, int tile_n, float scale, bool accumulate,
                      float* __restrict__ dW, float* __restrict__ part) {
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t tile = idx / nvec;
  const int64_t i0 = tile * tile_n;
  if (i0 >= n) return;
  const int64_t col = (idx - tile * nvec) * 8, d = (int64_t)nvec * 8;
  const int64_t i1 = min(n, i0 + tile_n);
  const int32_t next = i1 < n ? key_of(sorted[i1]) : -1;
  int32_t cur = key_of(sorted[i0]);
  bool head = i0 > 0 && key_of(sorted[i0 - 1]) == cur;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto flush = [&](bool tail) {
    if (cur == V) return;
    if (!head && !tail) {
      add_row8(dW + (int64_t)cur * d + col, acc, scale, accumulate);
    } else {
      store8(part + (tile * 2 + (head ? 0 : 1)) * d + col, from_f32<float>(acc));
    }
  };
  for (int64_t ib = i0; ib < i1 && cur != V; ib += 4) {
    int32_t key[4];
    Raw8<T> r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      key[u] = V;
      if (ib + u < i1) {
        const uint64_t it = sorted[ib + u];
        key[u] = key_of(it);
        if (key[u] != V) r[u] = load8(dX + (int64_t)(uint32_t)it * d + col);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (ib + u >= i1) break;
      if (key[u] != cur) {
        flush(false);
        cur = key[u];
        head = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
      }
      if (cur == V) break;  // the tokens without a row come last
      float f[8];
      to_f32(r[u], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += f[j];
    }
  }
  flush(cur == next);
}

// One CTA per tile; works where a row that spans tiles begins in it: adds up the row's
// partial sums, each of the eight warps a contiguous share of them, then the eight in order.
__global__ void __launch_bounds__(256)
    embed_join_kernel(const uint64_t* __restrict__ sorted, int64_t n, int32_t V, int d, int tile_n,
                      float scale, bool accumulate, float* __restrict__ dW,
                      const float* __restrict__ part) {
  __shared__ float4 red[8][32][2];
  const int64_t tile = blockIdx.x, i0 = tile * tile_n, i1 = i0 + tile_n;
  if (i1 >= n) return;
  const int32_t cur = key_of(sorted[i1 - 1]);
  if (cur == V || key_of(sorted[i1]) != cur) return;
  if (key_of(sorted[i0]) == cur && i0 > 0 && key_of(sorted[i0 - 1]) == cur) return;
  int64_t lo = i1, hi = n;  // the row's end: first sorted token past i1 with another key
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (key_of(sorted[mid]) == cur) lo = mid + 1; else hi = mid;
  }
  const int64_t n_part = (lo - 1) / tile_n - tile + 1;  // slot 1 of this tile, slot 0 of the others
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t share = (n_part + 7) / 8;
  const int64_t p0 = min(n_part, warp * share), p1 = min(n_part, p0 + share);
  for (int c0 = 0; c0 < d; c0 += 256) {
    const int col = c0 + lane * 8;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (col < d) {
#pragma unroll 4
      for (int64_t p = p0; p < p1; ++p) {
        float f[8];
        to_f32(load8(part + ((tile + p) * 2 + (p == 0 ? 1 : 0)) * d + col), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += f[j];
      }
    }
    const Raw8<float> mine = from_f32<float>(acc);
    red[warp][lane][0] = mine.a;
    red[warp][lane][1] = mine.b;
    __syncthreads();
    if (warp == 0 && col < d) {
      for (int w = 1; w < 8; ++w) {
        const Raw8<float> o{red[w][lane][0], red[w][lane][1]};
        float f[8];
        to_f32(o, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += f[j];
      }
      add_row8(dW + (int64_t)cur * d + col, acc, scale, accumulate);
    }
    __syncthreads();
  }
}

// Digits of the sort: bits of the largest key (V), in as few equal digits as fit the bins.
void sort_digits(int32_t V, int& n_pass, int& bits) {
  int need = 1;
  while (need < 31 && (V >> need) != 0) ++need;
  n_pass = (need + kMaxDigitBits - 1) / kMaxDigitBits;
  bits = (need + n_pass - 1) / n_pass;
}

}  // namespace

void launch_embed(const EmbedIds& a, bool bf16, const void* W, int d, float scale, void* out,
                  bool out_f32, cudaStream_t s) {
  const int nvec = d / 8, slabs = (nvec + 127) / 128;
  const unsigned blocks = (unsigned)((a.T * slabs + 7) / 8);
  if (!bf16)
    embed_kernel<float, float><<<blocks, 256, 0, s>>>(a, (const float*)W, nvec, slabs, scale,
                                                      (float*)out);
  else if (out_f32)
    embed_kernel<uint16_t, float><<<blocks, 256, 0, s>>>(a, (const uint16_t*)W, nvec, slabs, scale,
                                                         (float*)out);
  else
    embed_kernel<uint16_t, uint16_t><<<blocks, 256, 0, s>>>(a, (const uint16_t*)W, nvec, slabs,
                                                            scale, (uint16_t*)out);
}

int embed_sort_result(int32_t V) {
  int n_pass, bits;
  sort_digits(V, n_pass, bits);
  return n_pass % 2 == 0 ? 1 : 0;
}

cudaError_t launch_embed_sort(const EmbedIds& a, uint64_t* buf_a, uint64_t* buf_b, cudaStream_t s) {
  int n_pass, bits;
  sort_digits(a.V, n_pass, bits);
  int cluster = 1;  // about a thousand items per CTA, at most the portable cluster size
  while (cluster < 8 && (int64_t)cluster * 1024 < a.T) cluster *= 2;
  static std::atomic<uint64_t> attr_set{0};
  cudaError_t e = smem_once(embed_sort_kernel, kSortSmem, attr_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)cluster, 1, 1);
  cfg.blockDim = dim3(kSortWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = kSortSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, embed_sort_kernel, a, n_pass, bits, cluster, buf_a, buf_b);
}

// Longer tiles mean fewer partial rows, shorter ones more threads: the longest that still
// fills the GPU's threads once.
int embed_tile(int64_t T, int d, int num_sms) {
  int tile = 32;
  while (tile > 4 && (T + tile - 1) / tile * (d / 8) < (int64_t)num_sms * 2048) tile /= 2;
  return tile;
}

void launch_embed_grad(const uint64_t* sorted, int64_t T, int32_t V, bool bf16, const void* dX,
                       int d, int tile, float scale, bool accumulate, float* dW, float* part,
                       cudaStream_t s) {
  const int64_t threads = (T + tile - 1) / tile * (d / 8);
  const unsigned blocks = (unsigned)((threads + 255) / 256);
  if (bf16)
    embed_grad_kernel<uint16_t><<<blocks, 256, 0, s>>>(sorted, T, V, (const uint16_t*)dX, d / 8,
                                                       tile, scale, accumulate, dW, part);
  else
    embed_grad_kernel<float><<<blocks, 256, 0, s>>>(sorted, T, V, (const float*)dX, d / 8, tile,
                                                    scale, accumulate, dW, part);
}

void launch_embed_join(const uint64_t* sorted, int64_t T, int32_t V, int d, int tile, float scale,
                       bool accumulate, float* dW, const float* part, cudaStream_t s) {
  const int64_t tiles = (T + tile - 1) / tile;
  embed_join_kernel<<<(unsigned)tiles, 256, 0, s>>>(sorted, T, V, d, tile, scale, accumulate, dW,
                                                    part);
}

}  // namespace ckl
