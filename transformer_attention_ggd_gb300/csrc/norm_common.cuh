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
  int64_t xs[3], gs[3], ys[3];  // element strides over batch, head, token
  int heads;
};

struct NormArgs {
  NormSide side[2];
  const int* positions;  // [B, T] or null: the token's index
  float* part;           // backward: [ctas, part rows, 64] sums of one CTA
  unsigned tokens;       // B * T
  float eps;
  unsigned T;
  int per_head;
  int heads;             // of a unit: q then k heads, a multiple of 4
  int parts;             // units of a token tile
  int ctas;              // backward: CTAs of the launch, a multiple of parts
  RopeArgs rope;
};

// Rows of a CTA's sums of the weights' gradients: its heads, or q and k.
__host__ __device__ inline int norm_part_rows(const NormArgs& a) { return a.per_head ? a.heads : 2; }

// The most CTAs of a backward launch and the most heads of its units.
constexpr int kNormMaxCtas = 152 * 3;
constexpr int kNormMaxHeads = 64;

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st);
// Chooses heads, parts and ctas for `sms` SMs.
void norm_bwd_config(NormArgs* a, int sms);
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_bwd_finish(const NormArgs& a, cudaStream_t st);

}  // namespace bam
