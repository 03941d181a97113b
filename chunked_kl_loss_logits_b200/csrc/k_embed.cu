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
// the tokens are sorted by (id, position) and each thread walks neighbouring sorted tokens
// with eight columns of the running row sum in registers. Some hundred tokens need no sort at
// all, and of a few thousand each finds its place by comparing itself with all.
#include <algorithm>

#include "common.cuh"
#include "k_ops.h"
#include "ops.cuh"

namespace ckl {

namespace {

// A token's row among those held here, or V (mask 0, another rank's row, or out of range).
__device__ __forceinline__ int32_t row_of(const EmbedIds& a, int32_t id, uint8_t keep, bool& bad) {
  const bool in = id >= 0 && id < a.V_total;
  bad |= keep && !in;
  const int32_t r = keep && in ? id - a.v0 : -1;
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
  const int32_t row = row_of(a, a.ids[t], a.mask ? a.mask[t] : 1, bad);
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

// Zeros for dW where it is overwritten: a block's share, 16 vectors of 16 bytes a thread.
constexpr int kFill = 16;
template <int THREADS>
__device__ __forceinline__ void fill_zeros(float4* dst, int64_t n, int64_t block) {
  const int64_t i0 = block * (THREADS * kFill), i1 = min(n, i0 + THREADS * kFill);
#pragma unroll 8
  for (int64_t i = i0 + threadIdx.x; i < i1; i += THREADS) dst[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// ------------------------------------------------------------------ sort
// Stable least-significant-digit radix sort by one cluster of CTAs. Each of the cluster's
// warps owns a contiguous range of the items, so "count per (digit, warp), prefix over
// digits, then over warps" gives every item its place, and equal keys keep their order.
// The digit counts of the other CTAs are read from their shared memory. 32768 tokens, 18-bit
// keys in two digits: 14 us, for this plan a chain of latencies (cluster barriers, counts of the others,
// the scattered stores) on 8 of the SMs rather than work. 16 CTAs take a tenth less (1.4 us of a call of 117), but a
// cluster of more than 8 is a size that a kernel has to ask for and a device may refuse.
constexpr int kSortCtas = 8;
constexpr int kSortWarps = 32;
constexpr int kBatch = 4;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;
constexpr size_t kSortSmem = (size_t)(kSortWarps * kMaxBins + 2 * kMaxBins + 32) * 4;

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// The two halves of a cluster barrier: what a thread read or wrote before it arrives is done for
// those that have waited.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The first cluster sorts. The others (where dW is to be overwritten) zero dW meanwhile.
__global__ void __launch_bounds__(kSortWarps * 32, 1)
    embed_sort_kernel(const EmbedIds a, int n_pass, int bits, uint64_t* buf_a, uint64_t* buf_b,
                      float4* fill, int64_t n_fill) {
  extern __shared__ uint32_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  if (blockIdx.x >= kSortCtas) {
    fill_zeros<kSortWarps * 32>(fill, n_fill, blockIdx.x - kSortCtas);
    return;
  }
  uint32_t* hist = sm;                          // [warp][bin] counts, then places
  uint32_t* tot = sm + kSortWarps * kMaxBins;   // [bin] this CTA's counts (read by the others)
  uint32_t* base = tot + kMaxBins;              // [bin] first place of this CTA's items
  uint32_t* wsum = base + kMaxBins;             // [32]
  const int rank = (int)cluster_ctarank();
  const int bins = 1 << bits;
  constexpr int64_t kThreads = kSortCtas * kSortWarps * 32;
  const int64_t per = (a.T + kThreads - 1) / kThreads * 32;
  const int64_t i0 = min(a.T, ((int64_t)rank * kSortWarps + warp) * per);
  const int64_t i1 = min(a.T, i0 + per);
  uint32_t* myhist = hist + warp * bins;
  bool bad = false;

  for (int p = 0; p < n_pass; ++p) {
    const uint64_t* in = (p & 1) ? buf_a : buf_b;  // pass 0 reads the ids
    uint64_t* out = (p & 1) ? buf_b : buf_a;
    const int shift = 32 + p * bits;
    // kBatch items a lane at a time; a warp's range of at most one batch stays in registers
    uint64_t it[kBatch];
    auto load = [&](int64_t ib) {
      if (p == 0) {
        int32_t id[kBatch];
        uint8_t keep[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int64_t i = min(ib + j * 32 + lane, i1 - 1);
          id[j] = a.ids[i];
          keep[j] = a.mask ? a.mask[i] : 1;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          it[j] = (uint64_t)(uint32_t)row_of(a, id[j], keep[j], bad) << 32 |
                  (uint64_t)(ib + j * 32 + lane);
      } else {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          it[j] = __ldcg(reinterpret_cast<const unsigned long long*>(in) +
                         min(ib + j * 32 + lane, i1 - 1));
      }
    };
    auto digit = [&](uint64_t v) { return (uint32_t)(v >> shift) & (uint32_t)(bins - 1); };
    if (i0 < i1) load(i0);
    for (int b = lane; b < bins; b += 32) myhist[b] = 0;
    __syncwarp();
#pragma unroll 1
    for (int64_t ib = i0; ib < i1; ib += kBatch * 32) {
      if (ib > i0) load(ib);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (ib + j * 32 + lane < i1) atomicAdd(&myhist[digit(it[j])], 1u);
    }
    __syncthreads();
    if (tid < bins) {
      uint32_t mine = 0;
#pragma unroll 8
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
#pragma unroll
      for (int r = 0; r < kSortCtas; ++r) {
        const uint32_t c = ld_cluster_u32(cluster_map(tot + tid, (uint32_t)r));
        if (r < rank) before += c;
        all += c;
      }
    }
    // the other CTAs' counts are read: after the last pass nothing else keeps a CTA from leaving.
    // The arrival releases, so that no read is still under way when the CTA it reads from leaves.
    const bool last = p == n_pass - 1;
    if (last) cluster_arrive();
    // exclusive prefix of `all` over the bins (threads past the bins hold 0)
    uint32_t incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    const uint32_t pre = __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane] : 0u);
    if (tid < bins) base[tid] = pre + incl - all + before;
    __syncthreads();
#pragma unroll 1
    for (int64_t ib = i0; ib < i1; ib += kBatch * 32) {
      if (i1 - i0 > kBatch * 32) load(ib);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (ib + j * 32 >= i1) break;
        const bool have = ib + j * 32 + lane < i1;
        const unsigned act = __ballot_sync(0xffffffffu, have);
        if (have) {
          const uint32_t dg = digit(it[j]);
          const unsigned same = __match_any_sync(act, dg);
          const uint32_t at = myhist[dg];
          __syncwarp(act);
          if (lane == __ffs(same) - 1) myhist[dg] = at + __popc(same);
          out[base[dg] + at + __popc(same & ((1u << lane) - 1))] = it[j];
        }
        __syncwarp();
      }
    }
    // every item is in place, and no CTA still reads another's counts, before the next pass
    if (last) cluster_wait();
    else cluster_sync();
  }
  if (bad) atomicOr(a.status, (unsigned)ST_INDEX_RANGE);
}

// A few thousand tokens: every token's place is the number of tokens before it, those of smaller rows and
// the earlier ones of its own, counted by comparing with all; a warp counts for four tokens. The whole
// gradient of 2048 tokens of 512 columns takes 8.4 us so, 13.9 with the cluster's sort; 4096 11.7 and 16.7;
// 6000, whose blocks no longer have an SM each, 17.7 and 18.4, 8192 21.5 and 19.7.
constexpr int kRankMax = 4096;
constexpr int kRankTokens = 32;  // of a block

__global__ void __launch_bounds__(256)
    embed_rank_kernel(const EmbedIds a, int blocks, uint64_t* out, float4* fill, int64_t n_fill) {
  __shared__ uint4 keys[kRankMax / 4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = (int)a.T;
  griddep_launch_dependents();
  if ((int)blockIdx.x >= blocks) {
    fill_zeros<256>(fill, n_fill, blockIdx.x - blocks);
    return;
  }
  uint32_t* key = reinterpret_cast<uint32_t*>(keys);
  const int padded = (n + 127) / 128 * 128;
  bool bad = false;
#pragma unroll 4
  for (int j = tid; j < padded; j += 256)  // past the last token: a key above every other
    key[j] = j < n ? (uint32_t)row_of(a, a.ids[j], a.mask ? a.mask[j] : 1, bad) : ~0u;
  if (bad && blockIdx.x == 0) atomicOr(a.status, (unsigned)ST_INDEX_RANGE);
  __syncthreads();
  const int i0 = (int)blockIdx.x * kRankTokens + warp * 4;
  if (i0 >= n) return;
  uint32_t mine[4], place[4] = {0, 0, 0, 0};
#pragma unroll
  for (int t = 0; t < 4; ++t) mine[t] = key[i0 + t];  // (padded: in bounds)
  const int here = i0 / 128;  // the 128 tokens that hold these four
  auto count = [&](int v, uint32_t more) {  // of 128 tokens, equal rows counted where more = 1
    const uint4 k = keys[v * 32 + lane];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t lim = mine[t] + more;
      place[t] += (k.x < lim) + (k.y < lim) + (k.z < lim) + (k.w < lim);
    }
  };
#pragma unroll 4
  for (int v = 0; v < here; ++v) count(v, 1);
#pragma unroll 4
  for (int v = here + 1; v < padded / 128; ++v) count(v, 0);
  const uint4 k = keys[here * 32 + lane];
  const int j = here * 128 + lane * 4;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int i = i0 + t;
    place[t] += (k.x < mine[t] + (j < i)) + (k.y < mine[t] + (j + 1 < i)) +
                (k.z < mine[t] + (j + 2 < i)) + (k.w < mine[t] + (j + 3 < i));
    place[t] = __reduce_add_sync(0xffffffffu, place[t]);
    if (lane == t && i < n) out[place[t]] = (uint64_t)mine[t] << 32 | (uint32_t)i;
  }
}

// ------------------------------------------------------------------ gradient
__device__ __forceinline__ int32_t key_of(uint64_t it) { return (int32_t)(it >> 32); }

// dst (+)= scale * v. The addition is made in L2, so that the thread does not wait for the old
// value (121 us against 125 for the call at 32768 x 2880); a call adds to an element once, so it is
// the sum of two numbers either way (an L2 addition takes subnormal numbers for zero).
__device__ __forceinline__ void add_row8(float* dst, const float (&v)[8], float scale,
                                         bool accumulate) {
  float o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = scale * v[j];
  if (!accumulate) {
    store8(dst, from_f32<float>(o));
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; j += 4)
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst + j), "f"(o[j]),
                 "f"(o[j + 1]), "f"(o[j + 2]), "f"(o[j + 3])
                 : "memory");
}

// A group of `lanes` threads walks `run` sorted tokens, each thread with eight columns of the
// running sum; a CTA has 256 / lanes neighbouring groups, its tile, and lanes * 8 columns. A
// row all of whose tokens a group meets is finished by it. Of a row whose tokens span groups,
// each group's share goes to shared memory, and the group in which the row begins adds the
// shares up in order; of a row that spans tiles the tile's sum goes to part: slot 0 where the
// row began in an earlier tile, slot 1 where it begins here.
// 32768 tokens of 2880 columns, 13 thousand different ids of 201088: 90 us, 5.5 TB/s; 8 rows of
// dX ahead instead of 4 (fewer CTAs an SM) 140 us, 5 CTAs an SM (spills) 110 us.
constexpr int kHead = 1, kTail = 2;  // flags of a group: a share of a row that began before; a row begins, goes on
constexpr int kThrough = 4;          // with kHead: the row also goes on
constexpr int kAhead = 4;            // rows of dX loaded at a time

template <typename T>
__global__ void __launch_bounds__(256)
    embed_grad_kernel(const uint64_t* sorted, int64_t n, int32_t V,
                      const T* __restrict__ dX, int nvec, EmbedShape shape, float scale,
                      bool accumulate, float* dW, float* part) {
  __shared__ float4 head_sum[256][2];
  __shared__ int flags[256];
  const int lanes = shape.lanes, groups = 256 / lanes;
  const int g = threadIdx.x / lanes, l = threadIdx.x % lanes;
  const int64_t tile = blockIdx.x / shape.slabs;  // a tile's slabs run side by side
  const int vec = (int)(blockIdx.x - tile * shape.slabs) * lanes + l;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t i0 = (tile * groups + g) * shape.run;
  const int64_t i1 = min(n, i0 + shape.run);
  const int64_t col = (int64_t)vec * 8, d = (int64_t)nvec * 8;
  const bool on = vec < nvec;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  int32_t cur = V;
  int flag = 0;
  auto put_head = [&] {
    const Raw8<float> r = from_f32<float>(acc);
    head_sum[threadIdx.x][0] = r.a;
    head_sum[threadIdx.x][1] = r.b;
  };
  if (i0 < n) {
    const int32_t next = i1 < n ? key_of(sorted[i1]) : -1;
    cur = key_of(sorted[i0]);
    bool head = i0 > 0 && key_of(sorted[i0 - 1]) == cur;
    for (int64_t ib = i0; ib < i1 && cur != V; ib += kAhead) {
      int32_t key[kAhead];
      Raw8<T> r[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        key[u] = V;
        if (ib + u < i1) {
          const uint64_t it = sorted[ib + u];
          key[u] = key_of(it);
          if (on && key[u] != V) r[u] = load8(dX + (int64_t)(uint32_t)it * d + col);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (ib + u >= i1) break;
        if (key[u] != cur) {
          if (head) {
            put_head();
            flag = kHead;
          } else if (on) {
            add_row8(dW + (int64_t)cur * d + col, acc, scale, accumulate);
          }
          cur = key[u];
          head = false;
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = 0.f;
        }
        if (cur == V) break;  // the tokens without a row come last
        float f[8];
        to_f32(r[u], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += on ? f[j] : 0.f;
      }
    }
    if (cur != V) {
      const bool tail = cur == next;
      if (head) {
        put_head();
        flag = kHead | (tail ? kThrough : 0);
      } else if (tail) {
        flag |= kTail;  // the sum stays in acc
      } else if (on) {
        add_row8(dW + (int64_t)cur * d + col, acc, scale, accumulate);
      }
    }
  }
  if (l == 0) flags[g] = flag;
  __syncthreads();
  const bool begins = flag & kTail, goes_on = g == 0 && (flag & kHead);
  if (!begins && !goes_on) return;  // (a group can be both: two rows)
  auto follow = [&](int j, bool more) {  // add the shares of the groups from j on; still going on?
    for (; j < groups && more; ++j) {
      const Raw8<float> o{head_sum[j * lanes + l][0], head_sum[j * lanes + l][1]};
      float f[8];
      to_f32(o, f);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += f[k];
      more = flags[j] & kThrough;
    }
    return more;
  };
  float* mine = part + tile * 2 * d + col;
  if (begins) {
    if (follow(g + 1, true)) {
      if (on) store8(mine + d, from_f32<float>(acc));
    } else if (on) {
      add_row8(dW + (int64_t)cur * d + col, acc, scale, accumulate);
    }
  }
  if (goes_on) {
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    follow(0, true);
    if (on) store8(mine, from_f32<float>(acc));
  }
}

// One CTA per (tile, 256 columns); works where a row that spans tiles begins in the tile: adds
// up the row's partial sums, each of the eight warps a contiguous share of them, then the
// eight in order.
__global__ void __launch_bounds__(256)
    embed_join_kernel(const uint64_t* sorted, int64_t n, int32_t V, int d, int tile_n, float scale,
                      bool accumulate, float* dW, const float* part) {
  __shared__ float4 red[8][32][2];
  const int64_t tile = blockIdx.x, i0 = tile * tile_n, i1 = i0 + tile_n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  if (i1 >= n) return;
  // the first keys of the 32 tiles after this one, a lane each, beside those that tell whether a
  // row begins here and goes on: one round of loads
  auto first_key = [&](int64_t k) {
    return (tile + k) * tile_n < n ? key_of(sorted[(tile + k) * tile_n]) : -1;
  };
  int32_t ahead = first_key(1 + lane);
  const int32_t cur = key_of(sorted[i1 - 1]), first = key_of(sorted[i0]);
  const int32_t before = i0 > 0 ? key_of(sorted[i0 - 1]) : -1;
  unsigned same = __ballot_sync(0xffffffffu, ahead == cur);
  if (cur == V || !(same & 1u) || (first == cur && before == cur)) return;
  int64_t n_part = 1;  // slot 1 of this tile, slot 0 of the tiles that begin with the row
  while (same == 0xffffffffu) {
    n_part += 32;
    same = __ballot_sync(0xffffffffu, first_key(n_part + lane) == cur);
  }
  n_part += __ffs(~same) - 1;
  const int64_t share = (n_part + 7) / 8;
  const int64_t p0 = min(n_part, warp * share), p1 = min(n_part, p0 + share);
  const int col = blockIdx.y * 256 + lane * 8;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (col < d) {
#pragma unroll 8
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
}

// Few tokens: no sort. A token's CTA compares its row with every other token's. The row's c tokens
// have c CTAs: the one of the m-th takes the m-th of every c slabs of 256 columns. Its warps
// take a slab each where it has many, or share one slab's tokens: each a contiguous part of them in
// order of position, and the parts are added up in order. One launch instead of three, each of
// which waits for the one before. d = 2880, added to dW, against the places counted as below, in us:
// 64 tokens 3.0 and 5.5, 256 3.6 and 5.7, 512 4.9 and 8.8; 512 tokens of one row 7.8 and 7.5. With 1024
// tokens it still gains (7.0 and 9.8), but one row that takes them all costs 14.9 and 8.9.
// Every thread waits for the launch before it, also where it writes nothing: a batch without a token
// of these rows would otherwise be done before the zeros are, for all that follows it.
constexpr int kFew = 512;
constexpr int kFewWords = kFew / 32;

template <typename T>
__global__ void __launch_bounds__(256)
    embed_grad_few_kernel(const EmbedIds a, const T* __restrict__ dX, int nvec, float scale,
                          bool accumulate, float* dW) {
  static_assert(kFewWords <= 32, "a word of the tokens' bits for each lane");
  __shared__ uint32_t has[kFewWords];  // bit j: token j has this row
  __shared__ uint16_t list[kFew];      // those tokens
  __shared__ float4 sums[8][32][2];
  const int n = (int)a.T, i = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool bad = false, ignore = false;
  const int32_t row = row_of(a, a.ids[i], a.mask ? a.mask[i] : 1, bad);
  if (bad && threadIdx.x == 0) atomicOr(a.status, (unsigned)ST_INDEX_RANGE);
  if (row == a.V) {
    griddep_wait();
    return;
  }
  uint32_t mine[kFewWords / 8];
#pragma unroll
  for (int k = 0; k < kFewWords / 8; ++k) {
    const int j = k * 256 + (int)threadIdx.x;
    const bool same = j < n && row_of(a, a.ids[j], a.mask ? a.mask[j] : 1, ignore) == row;
    mine[k] = __ballot_sync(0xffffffffu, same);
    if (lane == 0) has[k * 8 + warp] = mine[k];
  }
  __syncthreads();
  const uint32_t word = lane < kFewWords ? has[lane] : 0u;
  const uint32_t below = lane < i / 32 ? ~0u : lane > i / 32 ? 0u : (1u << (i & 31)) - 1u;
  const int m = (int)__reduce_add_sync(0xffffffffu, __popc(word & below));
  int upto = __popc(word);  // tokens in the words up to this lane's
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  const int c = __shfl_sync(0xffffffffu, upto, 31), slabs = (nvec + 31) / 32;
  if (m >= slabs) {
    griddep_wait();
    return;
  }
#pragma unroll
  for (int k = 0; k < kFewWords / 8; ++k) {
    const int before = __shfl_sync(0xffffffffu, upto - __popc(word), k * 8 + warp);
    if (mine[k] >> lane & 1u)
      list[before + __popc(mine[k] & ((1u << lane) - 1u))] = (uint16_t)(k * 256 + threadIdx.x);
  }
  __syncthreads();
  const int ns = (slabs - m + c - 1) / c;  // slabs of this CTA
  const int per = ns > 4 ? 1 : ns > 2 ? 2 : ns > 1 ? 4 : 8;  // warps for a slab
  const int group = warp / per, sub = warp % per, share = (c + per - 1) / per;
  const int p0 = min(c, sub * share), p1 = min(c, p0 + share);
  bool waited = false;
  for (int q = group; q < ns; q += 8 / per) {  // (at most one where warps share a slab)
    const int vec = (m + q * c) * 32 + lane;
    const bool on = vec < nvec;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (on) {
#pragma unroll 8
      for (int p = p0; p < p1; ++p) {
        float f[8];
        to_f32(load8(dX + ((int64_t)list[p] * nvec + vec) * 8), f);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += f[k];
      }
    }
    if (per > 1 && c > 1) {
      const Raw8<float> r = from_f32<float>(acc);
      sums[warp][lane][0] = r.a;
      sums[warp][lane][1] = r.b;
    } else if (on && sub == 0) {
      if (!waited) griddep_wait();  // the zeros are written
      waited = true;
      add_row8(dW + ((int64_t)row * nvec + vec) * 8, acc, scale, accumulate);
    }
  }
  if (per == 1 || c == 1) {
    if (!waited) griddep_wait();
    return;
  }
  __syncthreads();
  const int vec = (m + group * c) * 32 + lane;
  if (sub != 0 || group >= ns || vec >= nvec) {
    griddep_wait();
    return;
  }
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int w = 0; w < per && w * share < c; ++w) {
    const Raw8<float> o{sums[warp + w][lane][0], sums[warp + w][lane][1]};
    float f[8];
    to_f32(o, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] += f[k];
  }
  griddep_wait();
  add_row8(dW + ((int64_t)row * nvec + vec) * 8, acc, scale, accumulate);
}

__global__ void __launch_bounds__(256) embed_zero_kernel(float4* dst, int64_t n) {
  griddep_launch_dependents();
  fill_zeros<256>(dst, n, blockIdx.x);
}

template <int THREADS>
unsigned fill_blocks(int64_t n) {  // n floats
  return (unsigned)((n / 4 + THREADS * kFill - 1) / (THREADS * kFill));
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

int embed_sort_result(int64_t T, int32_t V) {
  if (T <= kRankMax) return 0;
  int n_pass, bits;
  sort_digits(V, n_pass, bits);
  return n_pass % 2 == 0 ? 1 : 0;
}

cudaError_t launch_embed_sort(const EmbedIds& a, uint64_t* buf_a, uint64_t* buf_b, float* fill,
                              int64_t n_fill, cudaStream_t s) {
  // Blocks of zeros, many more than fit at once, as not every SM gets as many (one block per SM with a
  // fixed share: 58 us for 262 MB beside the sort of a cluster, this 41).
  if (a.T <= kRankMax) {
    const int blocks = (int)((a.T + kRankTokens - 1) / kRankTokens);
    embed_rank_kernel<<<(unsigned)blocks + fill_blocks<256>(n_fill), 256, 0, s>>>(
        a, blocks, buf_a, reinterpret_cast<float4*>(fill), n_fill / 4);
    return cudaSuccess;
  }
  int n_pass, bits;
  sort_digits(a.V, n_pass, bits);
  static std::atomic<uint64_t> attr_set{0};
  cudaError_t e = smem_once(embed_sort_kernel, kSortSmem, attr_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSortCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  const unsigned zero = fill_blocks<kSortWarps * 32>(n_fill);
  cfg.gridDim = dim3(kSortCtas * (1 + (zero + kSortCtas - 1) / kSortCtas), 1, 1);
  cfg.blockDim = dim3(kSortWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = kSortSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, embed_sort_kernel, a, n_pass, bits, buf_a, buf_b,
                            reinterpret_cast<float4*>(fill), n_fill / 4);
}

bool embed_grad_is_few(int64_t T) { return T <= kFew; }

cudaError_t launch_embed_grad_few(const EmbedIds& a, bool bf16, const void* dX, int d, float scale,
                                  bool accumulate, float* dW, cudaStream_t s) {
  const dim3 grid((unsigned)a.T);
  auto launch = [&](auto kernel, auto* x) {
    // it reads ids and dX before its wait: behind the zeros only, whose launch waited for those
    if (!accumulate) return launch_behind(kernel, grid, 256, 0, s, a, x, d / 8, scale, accumulate, dW);
    kernel<<<grid, 256, 0, s>>>(a, x, d / 8, scale, accumulate, dW);
    return cudaSuccess;
  };
  return bf16 ? launch(embed_grad_few_kernel<uint16_t>, (const uint16_t*)dX)
              : launch(embed_grad_few_kernel<float>, (const float*)dX);
}

void launch_embed_zero(float* dst, int64_t n, cudaStream_t s) {
  embed_zero_kernel<<<fill_blocks<256>(n), 256, 0, s>>>(reinterpret_cast<float4*>(dst), n / 4);
}

// Lanes of a group: as many as a row has vectors of eight columns, or the most of 32, 16 and 8 that
// leave at most a quarter idle (at d = 2880: 32 lanes 12 of 384 idle, 90 us; 8 lanes none, 164 us, as
// they read 128 bytes of a row at a time). Tokens of a group: the most, up to 16, that still give every SM two
// rounds of eight CTAs (a longer walk leaves fewer partial sums, a shorter one more in parallel).
EmbedShape embed_shape(int64_t T, int d, int num_sms) {
  const int nvec = d / 8;
  EmbedShape p;
  p.lanes = 1;
  if (nvec < 8) {
    while (p.lanes < nvec) p.lanes *= 2;
  } else {
    p.lanes = 32;
    while (p.lanes > 8 && (nvec + p.lanes - 1) / p.lanes * p.lanes * 3 > nvec * 4) p.lanes /= 2;
  }
  p.slabs = (nvec + p.lanes - 1) / p.lanes;
  p.run = 16;
  auto tiles = [&] { return (T + (int64_t)p.tile() - 1) / p.tile(); };
  while (p.run > 4 && tiles() * p.slabs < (int64_t)num_sms * 16) p.run /= 2;
  return p;
}

cudaError_t launch_embed_grad(const uint64_t* sorted, int64_t T, int32_t V, bool bf16,
                              const void* dX, int d, const EmbedShape& p, float scale,
                              bool accumulate, float* dW, float* part, cudaStream_t s) {
  const dim3 grid((unsigned)((T + p.tile() - 1) / p.tile() * p.slabs));
  return bf16 ? launch_behind(embed_grad_kernel<uint16_t>, grid, 256, 0, s, sorted, T, V,
                              (const uint16_t*)dX, d / 8, p, scale, accumulate, dW, part)
              : launch_behind(embed_grad_kernel<float>, grid, 256, 0, s, sorted, T, V,
                              (const float*)dX, d / 8, p, scale, accumulate, dW, part);
}

cudaError_t launch_embed_join(const uint64_t* sorted, int64_t T, int32_t V, int d,
                              const EmbedShape& p, float scale, bool accumulate, float* dW,
                              const float* part, cudaStream_t s) {
  const dim3 grid((unsigned)((T + p.tile() - 1) / p.tile()), (unsigned)((d + 255) / 256));
  return launch_behind(embed_join_kernel, grid, 256, 0, s, sorted, T, V, d, p.tile(), scale,
                       accumulate, dW, part);
}

}  // namespace ckl
