// Kernel arguments of the norms of queries and keys with their rotation.
#pragma once

#include "row_ops.cuh"

namespace bam {

// The queries (side 0) or the keys (side 1).
struct NormSide {
  const uint16_t* x;
  const uint16_t* g;   // backward: gradient of the output
  uint16_t* y;         // output, or the gradient of x
  const float* w;      // [64] or [heads, 64]
  float* dw;           // backward
  int64_t xs[3], gs[3], ys[3];  // strides over batch, head, token, in 16-byte words
  int heads;
};

struct NormArgs {
  NormSide side[2];
  const int* positions;  // [B, T] or null: the token's index
  float* part;           // backward: [ctas, part rows, 64] sums of one CTA
  unsigned tokens;       // B * T
  float eps;
  unsigned T;
  Divisor by_T;
  int per_head;
  int large;             // some place needs more than 32 bits
  int passes;            // of a part, kNormPass heads each: the queries' and then the keys'
  unsigned parts;        // of a tile's passes
  unsigned ctas;         // of the launch, a multiple of parts
  RopeArgs rope;
};

constexpr int kNormPass = 4;  // heads of a pass
// Rows of a CTA's sums of the weights' gradients: its heads, or q and k.
__host__ __device__ inline int norm_part_rows(const NormArgs& a) {
  return a.per_head ? kNormPass * a.passes : 2;
}

// The most CTAs of a backward launch and the most passes of a part.
constexpr int kNormMaxCtas = 152 * 16 / kNormPass;
constexpr int kNormMaxPasses = 64 / kNormPass;

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st);
// Chooses passes, parts and CTAs for `sms` SMs.
void norm_bwd_config(NormArgs* a, int sms);
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_bwd_finish(const NormArgs& a, cudaStream_t st);

}  // namespace bam
