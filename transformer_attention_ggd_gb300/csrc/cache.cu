// Writing a paged cache: appending keys and values with their rotation by
// position, and keeping the accepted path of a draft.
//
// Both are copies (a token's head vector is 128 bytes of K and of V): the
// append reads and writes 2 * 128 * (2 Hkv + H) bytes a token and is bound by
// HBM for prompts and by latency for single tokens; the keep moves a few rows
// a sequence and is always bound by latency.
#include "tree_common.cuh"

namespace bam {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 32;  // most tokens of one CTA
constexpr int kAppendRows = 4;     // rows of a thread in flight

// One rotated pair: (a, b) -> (a cos - b sin, b cos + a sin), in fp32, rounded
// once to bf16 by the caller.
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
  const float x = a * cs.x - b * cs.y;
  b = b * cs.x + a * cs.y;
  a = x;
}

__device__ __forceinline__ void unpack8(const uint4& w, float* f) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(x[i] << 16);
    f[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// One CTA: up to 32 tokens of one sequence and a run of its heads (queries,
// then keys, then values).  The cosines and sines of the tokens are computed
// once and serve all heads.  Four lanes hold a row, 32 bytes each: for pairs
// (x_f, x_{f + dims/2}) a lane takes the two 16-byte chunks that pair up.
__global__ void __launch_bounds__(kAppendThreads) bam_kv_append_kernel(const AppendArgs a) {
  __shared__ float2 cs[kAppendTokens][kHeadDim / 2];
  __shared__ int64_t slot_row[kAppendTokens];  // row of head 0 in the pages, -1: not written
  __shared__ int depth[kTreeMax], jump[kTreeMax];
  const CacheArgs& c = a.c;
  const int tiles = (c.N + a.tokens - 1) / a.tokens;
  const int b = blockIdx.x / tiles;
  const int t0 = (blockIdx.x % tiles) * a.tokens;
  const int cap = c.page * c.max_blocks;
  const int raw = __ldg(c.lens + b);
  const int rawn = c.draft_lens ? __ldg(c.draft_lens + b) : c.N;
  const int len = min(max(raw, 0), cap);
  const int n = min(max(rawn, 0), c.N);
  bool ok = raw == len && rawn == n;
  const int nt = min(a.tokens, n - t0);
  if (nt <= 0) {
    if (!ok && t0 == 0 && blockIdx.y == 0 && threadIdx.x == 0) record_bad_arg(c.status);
    return;
  }
  if (c.parents) ok &= tree_depths(c.parents + static_cast<size_t>(b) * c.N, n, jump, depth);
  for (int x = threadIdx.x; x < nt; x += kAppendThreads) {
    const int64_t slot = static_cast<int64_t>(len) + t0 + x;
    int64_t row = -1;
    if (slot < cap) {
      const int pg = __ldg(c.block_table + static_cast<size_t>(b) * c.max_blocks + slot / c.page);
      if (pg >= 0 && pg < c.num_pages)
        row = static_cast<int64_t>(pg) * c.Hkv * c.page + slot % c.page;
    }
    ok &= row >= 0;
    slot_row[x] = row;
  }
  if (!ok && blockIdx.y == 0) record_bad_arg(c.status);
  const int half = a.dims / 2;
  for (int x = threadIdx.x; x < nt * half; x += kAppendThreads) {
    const int t = x / half, f = x % half;
    const uint64_t pos = static_cast<uint64_t>(len) + (c.parents ? depth[t0 + t] : t0 + t);
    // The phase wraps modulo 2^64, one turn: an exact reduction.  Its top 32
    // bits, signed, are the angle in units of 2^-31 half turns.
    const int top = static_cast<int>((pos * a.freq[f]) >> 32);
    float s, co;
    sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &co);
    cs[t][f] = make_float2(co, s);
  }
  __syncthreads();

  const int heads = a.H + 2 * c.Hkv;
  const int h0 = blockIdx.y * a.heads;
  const int nrow = nt * min(a.heads, heads - h0);
  const int u = threadIdx.x & 3;
  const int nh = a.dims / 16;
  const int c0 = a.interleaved || u >= nh ? 2 * u : u;
  const int c1 = a.interleaved || u >= nh ? 2 * u + 1 : u + nh;
  const bool rotated = u < nh;
  for (int r0 = threadIdx.x >> 2; r0 < nrow; r0 += kAppendRows * (kAppendThreads / 4)) {
    uint4 w[kAppendRows][2];
#pragma unroll
    for (int x = 0; x < kAppendRows; ++x) {
      const int r = r0 + x * (kAppendThreads / 4);
      if (r >= nrow) break;
      const int h = h0 + r / nt, t = t0 + r % nt;
      const uint16_t* src;
      if (h < a.H)
        src = a.q + b * a.qs[0] + h * a.qs[1] + t * a.qs[2];
      else if (h < a.H + c.Hkv)
        src = a.k + b * a.ks[0] + (h - a.H) * a.ks[1] + t * a.ks[2];
      else
        src = a.v + b * a.vs[0] + (h - a.H - c.Hkv) * a.vs[1] + t * a.vs[2];
      w[x][0] = *reinterpret_cast<const uint4*>(src + 8 * c0);
      w[x][1] = *reinterpret_cast<const uint4*>(src + 8 * c1);
    }
#pragma unroll
    for (int x = 0; x < kAppendRows; ++x) {
      const int r = r0 + x * (kAppendThreads / 4);
      if (r >= nrow) break;
      const int h = h0 + r / nt, t = r % nt;
      if (rotated && h < a.H + c.Hkv) {
        float f0[8], f1[8];
        unpack8(w[x][0], f0);
        unpack8(w[x][1], f1);
        if (a.interleaved) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            turn(f0[2 * y], f0[2 * y + 1], cs[t][8 * u + y]);
            turn(f1[2 * y], f1[2 * y + 1], cs[t][8 * u + 4 + y]);
          }
        } else {
#pragma unroll
          for (int y = 0; y < 8; ++y) turn(f0[y], f1[y], cs[t][8 * u + y]);
        }
        w[x][0] = pack8(f0);
        w[x][1] = pack8(f1);
      }
      uint16_t* dst;
      if (h < a.H) {
        dst = a.q_out + ((static_cast<int64_t>(b) * a.H + h) * c.N + t0 + t) * kHeadDim;
      } else {
        const int64_t row = slot_row[t];
        if (row < 0) continue;
        const int hk = h < a.H + c.Hkv ? h - a.H : h - a.H - c.Hkv;
        dst = (h < a.H + c.Hkv ? a.k_pages : a.v_pages) +
              (row + static_cast<int64_t>(hk) * c.page) * kHeadDim;
      }
      *reinterpret_cast<uint4*>(dst + 8 * c0) = w[x][0];
      *reinterpret_cast<uint4*>(dst + 8 * c1) = w[x][1];
    }
  }
}

constexpr int kKeepThreads = 256;
constexpr int kKeepBatch = 16;  // rows that a warp holds in registers

// One cluster per sequence; a warp takes one head of K or of V at a time.
// Node m of the path moves from slot a_m to slot m <= a_m.  A slot that is
// written may be an earlier node's source but never a later one's
// (a_m' >= m' > m), so a warp that reads a batch of rows before it writes
// them, batches in order, moves them in place.
__global__ void __launch_bounds__(kKeepThreads) bam_kv_keep_kernel(const KeepArgs a) {
  __shared__ int path[kTreeMax];
  __shared__ int64_t src_row[kTreeMax], dst_row[kTreeMax];
  __shared__ int count;
  const CacheArgs& c = a.c;
  const int b = blockIdx.y;
  int len, n;
  bool ok = cache_lengths(c, b, &len, &n);
  int acc = __ldg(a.accepted + b);
  if (acc < -1 || acc >= n) {
    ok = false;
    acc = -1;
  }
  if (threadIdx.x == 0) {
    // Root to node, from the deep end: the depth is known after the walk.
    const int* par = c.parents ? c.parents + static_cast<size_t>(b) * c.N : nullptr;
    int m = 0;
    if (par) {
      for (int i = acc; i >= 0;) {
        path[m++] = i;
        const int p = __ldg(par + i);
        if (p < -1 || p >= i) ok = false;
        i = p < i ? p : -1;
      }
    } else {
      m = acc + 1;  // a chain: every node is where it belongs
    }
    count = m;
  }
  __syncthreads();
  const int m = count;
  bool pages_ok = true;
  if (c.parents) {
    for (int x = threadIdx.x; x < m; x += kKeepThreads) {
      const int s = len + path[m - 1 - x], d = len + x;
      const int ps = __ldg(c.block_table + static_cast<size_t>(b) * c.max_blocks + s / c.page);
      const int pd = __ldg(c.block_table + static_cast<size_t>(b) * c.max_blocks + d / c.page);
      pages_ok &= ps >= 0 && ps < c.num_pages && pd >= 0 && pd < c.num_pages;
      src_row[x] = static_cast<int64_t>(ps) * c.Hkv * c.page + s % c.page;
      dst_row[x] = static_cast<int64_t>(pd) * c.Hkv * c.page + d % c.page;
    }
  }
  pages_ok = __syncthreads_and(pages_ok);
  if (blockIdx.x == 0 && threadIdx.x == 0 && !(ok && pages_ok)) record_bad_arg(c.status);

  if (c.parents && pages_ok) {
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kKeepThreads / 32);
    for (int hv = blockIdx.x * (kKeepThreads / 32) + (threadIdx.x >> 5); hv < 2 * c.Hkv;
         hv += warps) {
      uint16_t* pool = hv < c.Hkv ? a.k_pages : a.v_pages;
      const int64_t head = static_cast<int64_t>(hv < c.Hkv ? hv : hv - c.Hkv) * c.page;
      for (int m0 = 0; m0 < m; m0 += kKeepBatch) {
        uint4 w[kKeepBatch / 4];
#pragma unroll
        for (int x = 0; x < kKeepBatch / 4; ++x) {
          const int i = m0 + 4 * x + (lane >> 3);
          if (i < m)
            w[x] = reinterpret_cast<const uint4*>(pool + (src_row[i] + head) * kHeadDim)[lane & 7];
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < kKeepBatch / 4; ++x) {
          const int i = m0 + 4 * x + (lane >> 3);
          if (i < m && src_row[i] != dst_row[i])
            reinterpret_cast<uint4*>(pool + (dst_row[i] + head) * kHeadDim)[lane & 7] = w[x];
        }
        __syncwarp();
      }
    }
  }
  // new_lens may be cache_lens: written when every CTA of the sequence has
  // read its length.
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x == 0) a.new_lens[b] = len + (pages_ok ? m : 0);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& args, cudaStream_t st) {
  AppendArgs a = args;
  const int heads = a.H + 2 * a.c.Hkv;
  // Tokens and heads of a CTA: about four rows a thread once there are enough
  // rows for two CTAs per SM.
  a.tokens = a.c.N < kAppendTokens ? a.c.N : kAppendTokens;
  const int tiles = (a.c.N + a.tokens - 1) / a.tokens;
  const int64_t ctas = static_cast<int64_t>(a.c.B) * tiles;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  int split = 1;
  while (split < heads && ctas * split < 2 * 152 &&
         static_cast<int64_t>(a.tokens) * ((heads + split - 1) / split) > kAppendThreads / 4)
    ++split;
  a.heads = (heads + split - 1) / split;
  dim3 grid(static_cast<unsigned>(ctas), (heads + a.heads - 1) / a.heads);
  return launch_k(bam_kv_append_kernel, grid, dim3(kAppendThreads), 0, st, false, a);
}

cudaError_t launch_keep(const KeepArgs& a, cudaStream_t st) {
  const int warps = kKeepThreads / 32;
  int x = (2 * a.c.Hkv + warps - 1) / warps;
  if (x > 8) x = 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(x, a.c.B);
  cfg.blockDim = dim3(kKeepThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = x;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, bam_kv_keep_kernel, a);
}

}  // namespace bam
