// Attention of a tree of drafted tokens over a paged cache.
//
//   z[t, j] = c_t q_t . k_j + b_h(pos_t - pos_j),   o_t = softmax_j(z) V
//
// over the committed keys j < len (pos_j = j) and over node t's ancestors and
// itself (pos = len + depth).
#include "table_eval.cuh"
#include "tree_common.cuh"

namespace bam {
namespace {

constexpr int kTreeThreads = 128;

// Starts the call and checks the lengths.
__global__ void bam_tree_prep_kernel(const TreeArgs a) {
  if (threadIdx.x == 0) status_begin_call(a.c.status);
  __syncthreads();
  bool ok = true;
  for (int b = threadIdx.x; b < a.c.B; b += blockDim.x) {
    int len, n;
    ok &= cache_lengths(a.c, b, &len, &n);
  }
  if (!ok) record_bad_arg(a.c.status);
}

// One CTA per row (b, h, t); a thread takes every 128th key and keeps its own
// running maximum, sum and output.
__global__ void __launch_bounds__(kTreeThreads) bam_tree_kernel(const TreeArgs a) {
  __shared__ int jump[kTreeMax], depth[kTreeMax], parent[kTreeMax];
  __shared__ bool seen[kTreeMax];
  __shared__ float q[kHeadDim];
  __shared__ float red[kTreeThreads / 32][2 + kHeadDim];
  const CacheArgs& c = a.c;
  const int t = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  int len, n;
  cache_lengths(c, b, &len, &n);
  if (t >= n) return;
  const int* par = c.parents ? c.parents + static_cast<size_t>(b) * c.N : nullptr;
  bool ok = tree_depths(par, n, jump, depth);
  const int i = threadIdx.x;
  int p = par && i < n ? par[i] : i - 1;
  if (p < -1 || p >= i) p = -1;
  parent[i] = p;
  seen[i] = false;
  const size_t row = (static_cast<size_t>(b) * a.H + h) * c.N + t;
  if (i < kHeadDim) q[i] = __uint_as_float(static_cast<uint32_t>(a.q[row * kHeadDim + i]) << 16);
  __syncthreads();
  if (i == 0)
    for (int x = t; x >= 0; x = parent[x]) seen[x] = true;
  __syncthreads();

  const int pos = len + depth[t];
  float cl = 0.125f;
  if (a.ssmax) cl *= a.s[h] * logf(static_cast<float>(pos + 1));
  cl *= static_cast<float>(kLog2e);
  const float al = a.alpha[h], be = a.beta[h], mu = a.mu[h];
  const int hk = h / (a.H / c.Hkv);
  float m = -INFINITY, l = 0.0f, o[kHeadDim];
#pragma unroll
  for (int x = 0; x < kHeadDim; ++x) o[x] = 0.0f;
  for (int j = i; j < len + n; j += kTreeThreads) {
    if (j >= len && !seen[j - len]) continue;
    int pg = c.block_table[static_cast<size_t>(b) * c.max_blocks + j / c.page];
    if (pg < 0 || pg >= c.num_pages) {
      ok = false;
      pg = 0;
    }
    const size_t at = ((static_cast<size_t>(pg) * c.Hkv + hk) * c.page + j % c.page) * kHeadDim;
    float dot = 0.0f;
    for (int x = 0; x < kHeadDim; ++x)
      dot = fmaf(q[x], __uint_as_float(static_cast<uint32_t>(a.k_pages[at + x]) << 16), dot);
    const int d = j < len ? pos - j : depth[t] - depth[j - len];
    float bias, g1, g2;
    bias_terms<false>(d, al, be, mu, a.eps, a.prior, &bias, &g1, &g2);
    const float z = fmaf(dot, cl, to_f32_finite(bias * static_cast<float>(kLog2e)));
    const float mn = fmaxf(m, z);
    const float base = mn == -INFINITY ? 0.0f : mn;
    const float corr = ex2_approx(m - base), w = ex2_approx(z - base);
    l = l * corr + w;
#pragma unroll
    for (int x = 0; x < kHeadDim; ++x)
      o[x] = o[x] * corr + w * __uint_as_float(static_cast<uint32_t>(a.v_pages[at + x]) << 16);
    m = mn;
  }
  if (!ok) record_bad_arg(c.status);
  // Merge the lanes, then the warps.
  for (int off = 16; off; off >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, off), l2 = __shfl_xor_sync(0xffffffffu, l, off);
    const float mn = fmaxf(m, m2), base = mn == -INFINITY ? 0.0f : mn;
    const float e1 = ex2_approx(m - base), e2 = ex2_approx(m2 - base);
    l = l * e1 + l2 * e2;
#pragma unroll
    for (int x = 0; x < kHeadDim; ++x)
      o[x] = o[x] * e1 + __shfl_xor_sync(0xffffffffu, o[x], off) * e2;
    m = mn;
  }
  if ((i & 31) == 0) {
    red[i >> 5][0] = m;
    red[i >> 5][1] = l;
    for (int x = 0; x < kHeadDim; ++x) red[i >> 5][2 + x] = o[x];
  }
  __syncthreads();
  if (i < kHeadDim) {
    float M = -INFINITY, L = 0.0f, O = 0.0f;
    for (int w = 0; w < kTreeThreads / 32; ++w) M = fmaxf(M, red[w][0]);
    const float base = M == -INFINITY ? 0.0f : M;
    for (int w = 0; w < kTreeThreads / 32; ++w) {
      const float e = ex2_approx(red[w][0] - base);
      L += red[w][1] * e;
      O += red[w][2 + i] * e;
    }
    if (a.o_fp32)
      static_cast<float*>(a.o)[row * kHeadDim + i] = O / L;
    else
      static_cast<uint16_t*>(a.o)[row * kHeadDim + i] =
          static_cast<uint16_t>(pack_bf16x2(O / L, 0.0f) & 0xFFFFu);
    if (a.lse && i == 0) a.lse[row] = (M + log2f(L)) * kLn2f;
  }
}

}  // namespace

cudaError_t launch_tree_prep(const TreeArgs& a, cudaStream_t st) {
  return launch_k(bam_tree_prep_kernel, dim3(1), dim3(256), 0, st, false, a);
}

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t st) {
  return launch_k(bam_tree_kernel, dim3(a.c.N, a.H, a.c.B), dim3(kTreeThreads), 0, st, false, a);
}

}  // namespace bam
