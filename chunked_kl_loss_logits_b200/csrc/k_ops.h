// Host-side launchers of the operators around the loss (internal; not part of the
// C ABI). Element types: bf16 (bits) or fp32, chosen by `bf16`.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ckl {

// ---- embedding (k_embed.cu)
struct EmbedIds {
  const int32_t* ids;   // T token ids in [0, V_total)
  const uint8_t* mask;  // T bytes or NULL; the id of a token with mask 0 is not looked at
  int64_t T;
  int32_t V_total;      // ids are checked against it
  int32_t v0, V;        // the rows held here: ids v0 .. v0 + V - 1
  unsigned* status;
};
// out[t] = scale * W[ids[t] - v0] in the element type (or fp32 with out_f32); zeros for
// masked tokens and for ids of other rows.
void launch_embed(const EmbedIds& a, bool bf16, const void* W, int d, float scale, void* out,
                  bool out_f32, cudaStream_t s);
// (row, position) of every token in ascending order, as row << 32 | position; the row is V for
// tokens that have none here. The result is in `b` where embed_sort_result is 1, else in `a`.
// The same launch zeroes n_fill floats (a multiple of 8) at `fill`.
int embed_sort_result(int64_t T, int32_t V);
cudaError_t launch_embed_sort(const EmbedIds& a, uint64_t* buf_a, uint64_t* buf_b, float* fill,
                              int64_t n_fill, cudaStream_t s);
// dW[row] (+)= scale * sum of the row's dX where that needs no sort (few tokens, by embed_grad_is_few).
// Where dW is overwritten it follows launch_embed_zero (launch_behind).
bool embed_grad_is_few(int64_t T);
cudaError_t launch_embed_grad_few(const EmbedIds& a, bool bf16, const void* dX, int d, float scale,
                                  bool accumulate, float* dW, cudaStream_t s);
void launch_embed_zero(float* dst, int64_t n, cudaStream_t s);  // n: a multiple of 8
// How the gradient is shared out: groups of `lanes` threads walk `run` sorted tokens each,
// 256 / lanes groups make a CTA's tile, `slabs` CTAs cover the columns.
struct EmbedShape {
  int lanes, run, slabs;
  __host__ __device__ int tile() const { return 256 / lanes * run; }
};
EmbedShape embed_shape(int64_t T, int d, int num_sms);
// dW[row] (+)= scale * sum of the row's dX, in order of position. part: 2 fp32 rows for each
// tile, the sums of rows whose tokens span tiles; launch_embed_join adds those up.
// Both are launched behind the kernel before them (launch_behind).
cudaError_t launch_embed_grad(const uint64_t* sorted, int64_t T, int32_t V, bool bf16,
                              const void* dX, int d, const EmbedShape& p, float scale,
                              bool accumulate, float* dW, float* part, cudaStream_t s);
cudaError_t launch_embed_join(const uint64_t* sorted, int64_t T, int32_t V, int d,
                              const EmbedShape& p, float scale, bool accumulate, float* dW,
                              const float* part, cudaStream_t s);

// ---- 8-bit checkpoints and the norm (k_act8.cu)
void launch_act8_pack(bool bf16, const void* X, int64_t T, int cols, int fmt, uint8_t* q,
                      uint8_t* e, cudaStream_t s);
void launch_act8_unpack(bool bf16, const uint8_t* q, const uint8_t* e, int64_t T, int cols,
                        int fmt, void* out, cudaStream_t s);
struct NormArgs {
  const void* x;         // forward: input; backward: dY
  const void* res;       // forward: residual or NULL; backward: gradient of the sum or NULL
  const void* gain;
  int64_t T;
  int d;
  float eps;
  int fmt;
  void* sum;             // forward: x + res (with res)
  void* y;               // forward: output; backward: dX
  uint8_t *q, *e;        // checkpoint (forward: NULL for none)
  float* rstd;
  float* part;           // backward: dgain partials, norm_part_rows x d
};
cudaError_t launch_norm_fwd(const NormArgs& a, bool bf16, int num_sms, cudaStream_t s);
int64_t norm_part_rows(int64_t T, int d, bool bf16, int num_sms);
cudaError_t launch_norm_bwd(const NormArgs& a, bool bf16, int num_sms, cudaStream_t s);
// out[c] (+)= sum over rows of part[r][c], in a fixed order; behind norm_bwd (launch_behind)
cudaError_t launch_norm_dgain(const float* part, int64_t rows, int d, bool accumulate, float* out,
                              cudaStream_t s);

// ---- weight gradient from a checkpoint (k_wgrad.cu)
struct WgradArgs {
  int n, cols;      // dY columns, X' columns
  int kb_part;      // 64-token steps of one part of dY
  int n_kb;         // steps in all (parts x kb_part)
  int n_split, kb_split;
  int add;          // add to the result (n_split == 1 only)
  unsigned* status;
};
int wgrad_split(int64_t n, int64_t cols, int64_t n_kb, int num_sms);
// a: the bf16 parts of dY as a (n, T, parts) tensor, boxes of 64 x 64 x 1; b: X' in bf16 as
// a (cols, T) tensor, boxes of 64 x 64; c: dW or the n_split partial results as an fp32
// (cols, n, n_split) tensor, boxes of 32 x 32 x 1. Both this and the sum of the partial results
// are launched behind the kernel before them (launch_behind).
cudaError_t launch_wgrad(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c,
                         const WgradArgs& p, int num_sms, cudaStream_t s);
void launch_split3(const float* x, int64_t n, uint16_t* out, cudaStream_t s);
cudaError_t launch_wgrad_sum(const float* part, int n_split, int64_t n, bool add, float* out,
                             cudaStream_t s);

}  // namespace ckl
