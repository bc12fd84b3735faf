// Norms of queries and keys with their rotation by position, and the gradients.
//
//   r = 1 / sqrt(mean(x^2) + eps),   n = x r,   y = R(pos) (w n)
//   dn = R(-pos) dy,  dw = sum dn n,  dx = r (w dn - n mean(w dn n))
//
// per head vector x of 64 values.  A row is read and written once: 256 bytes
// forward, 384 backward, against some 500 and 1000 instructions of a lane, so
// both are bound by HBM.  1 / rms is computed again in the backward pass (x is
// read there anyway), so nothing is kept between the passes.
//
// Four lanes hold a row, 16 values each; a tile is 16 tokens, whose angles are
// computed once for the heads of a unit (a sine and cosine cost as much as a
// value's whole path).
#include "norm_common.cuh"

namespace bam {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;       // of a tile
constexpr int kPass = 4;          // heads of a pass: 64 rows of 4 lanes
constexpr int kFwdRows = 4;       // passes of a forward unit, loaded at once
constexpr int kFinishThreads = 1024;

// This thread's place: token t of the tile, head h of each pass, its chunks.
struct Lane {
  int t, h, u4, c0, c1;
  bool rotated;
};
__device__ __forceinline__ Lane lane_of(const RopeArgs& r) {
  Lane l;
  l.u4 = threadIdx.x & 3;
  l.t = (threadIdx.x >> 2) & (kTokens - 1);
  l.h = threadIdx.x / (4 * kTokens);
  const int nh = r.dims / 16;
  l.rotated = l.u4 < nh;
  const bool apart = l.rotated && !r.interleaved;
  l.c0 = apart ? l.u4 : 2 * l.u4;
  l.c1 = apart ? l.u4 + nh : 2 * l.u4 + 1;
  return l;
}

// Cosines and sines of a tile's tokens, by the whole block.
__device__ __forceinline__ void tile_angles(const NormArgs& a, unsigned tile,
                                            float4 (*cs)[kHeadDim / 4]) {
  const int half = a.rope.dims / 2;
  for (int y = threadIdx.x; y < kTokens * (kHeadDim / 2); y += kThreads) {
    const int t = y / (kHeadDim / 2), f = y % (kHeadDim / 2);
    const unsigned n = tile * kTokens + t;
    if (f >= half) continue;
    // (places behind the last token hold zeros, which any angle leaves zero)
    const int pos = n >= a.tokens ? 0 : a.positions ? __ldg(a.positions + n) : static_cast<int>(n % a.T);
    reinterpret_cast<float2*>(cs[t])[f] =
        rope_angle(static_cast<uint64_t>(static_cast<int64_t>(pos)), a.rope.freq[f]);
  }
}

struct Row {
  uint4 v[2];
};
__device__ __forceinline__ Row load_row(const uint16_t* p, const int64_t* st, unsigned b, int h,
                                        unsigned t, const Lane& l) {
  const uint16_t* src = p + b * st[0] + h * st[1] + t * st[2];
  Row r;
  r.v[0] = *reinterpret_cast<const uint4*>(src + 8 * l.c0);
  r.v[1] = *reinterpret_cast<const uint4*>(src + 8 * l.c1);
  return r;
}
__device__ __forceinline__ void store_row(uint16_t* p, const int64_t* st, unsigned b, int h,
                                          unsigned t, const Lane& l, const float* f) {
  uint16_t* dst = p + b * st[0] + h * st[1] + t * st[2];
  *reinterpret_cast<uint4*>(dst + 8 * l.c0) = pack8(f);
  *reinterpret_cast<uint4*>(dst + 8 * l.c1) = pack8(f + 8);
}
__device__ __forceinline__ void load_weight(const NormArgs& a, const NormSide& s, int h,
                                            const Lane& l, float* w) {
  const float* p = s.w + (a.per_head ? h * kHeadDim : 0);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float4* q = reinterpret_cast<const float4*>(p + 8 * (c ? l.c1 : l.c0));
    const float4 x = __ldg(q), y = __ldg(q + 1);
    w[8 * c] = x.x, w[8 * c + 1] = x.y, w[8 * c + 2] = x.z, w[8 * c + 3] = x.w;
    w[8 * c + 4] = y.x, w[8 * c + 5] = y.y, w[8 * c + 6] = y.z, w[8 * c + 7] = y.w;
  }
}

// A unit is a tile of tokens and up to 16 heads (the queries' and then the
// keys', in one row of numbers); all its rows are on their way before its angles are
// computed.
__global__ void __launch_bounds__(kThreads, 4) bam_qk_norm_fwd_kernel(const NormArgs a) {
  __shared__ float4 cs[kTokens][kHeadDim / 4];
  const Lane l = lane_of(a.rope);
  const unsigned tile = blockIdx.x / a.parts;
  const int part = static_cast<int>(blockIdx.x - tile * a.parts);
  const unsigned n = tile * kTokens + l.t;
  const bool live = n < a.tokens;
  const unsigned b = live ? n / a.T : 0, t = n - b * a.T;
  const int h0 = part * a.heads + l.h, H = a.side[0].heads;
  const int end = min((part + 1) * a.heads, H + a.side[1].heads);
  Row x[kFwdRows];
#pragma unroll
  for (int y = 0; y < kFwdRows; ++y) {
    const int hh = h0 + kPass * y;
    if (!live || hh >= end) continue;
    const NormSide& s = a.side[hh >= H];
    x[y] = load_row(s.x, s.xs, b, hh >= H ? hh - H : hh, t, l);
  }
  if (a.rope.dims) {
    tile_angles(a, tile, cs);
    __syncthreads();
  }
  float4 r[4];
  if (l.rotated) {
#pragma unroll
    for (int z = 0; z < 4; ++z) r[z] = cs[l.t][4 * l.u4 + z];
  }
#pragma unroll
  for (int y = 0; y < kFwdRows; ++y) {
    const int hh = h0 + kPass * y;
    if (__all_sync(0xffffffffu, hh >= end)) break;
    const bool on = live && hh < end;
    float f[16];
    if (!on) x[y].v[0] = x[y].v[1] = make_uint4(0, 0, 0, 0);
    unpack8(x[y].v[0], f);
    unpack8(x[y].v[1], f + 8);
    float scale;
    const float inv = row_rms_inv(f, a.eps, &scale);
    if (!on) continue;
    const NormSide& s = a.side[hh >= H];
    const int h = hh >= H ? hh - H : hh;
    float w[16];
    load_weight(a, s, h, l, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = f[i] * inv * w[i];
    if (l.rotated) turn_row(f, f + 8, r, a.rope.interleaved, 1.0f);
    store_row(s.y, s.ys, b, h, t, l, f);
  }
}

// A CTA takes every (ctas / parts)-th tile of one part of the heads, a pass of
// four heads after the other with the next pass's rows on their way, and sums
// the weights' gradients in shared memory: a warp's eight rows belong to one
// head, so they are joined by shuffles (halving the values each lane holds), and
// a place in shared memory has one warp that adds to it.  The order of every sum
// is fixed.
__global__ void __launch_bounds__(kThreads, 2) bam_qk_norm_bwd_kernel(const NormArgs a) {
  extern __shared__ __align__(16) float acc[];  // [rows][2 token halves][64]
  __shared__ float4 cs[kTokens][kHeadDim / 4];
  grid_dep_trigger();
  const Lane l = lane_of(a.rope);
  const int lane = threadIdx.x & 31, wt = (threadIdx.x >> 5) & 1;
  const int part = blockIdx.x % a.parts, H = a.side[0].heads;
  const int first = part * a.heads, end = min(first + a.heads, H + a.side[1].heads);
  const int passes = (end - first + kPass - 1) / kPass;
  const int acc_rows = a.per_head ? a.heads : 2 * kPass;
  for (int y = threadIdx.x; y < acc_rows * 2 * kHeadDim; y += kThreads) acc[y] = 0.0f;
  const unsigned tiles = (a.tokens + kTokens - 1) / kTokens;
  const unsigned step = a.ctas / a.parts;
  unsigned tile = blockIdx.x / a.parts;
  int pass = 0;
  Row x, g;
  auto load = [&](unsigned tl, int ps, Row& xr, Row& gr) {
    const unsigned n = tl * kTokens + l.t;
    const int hh = first + kPass * ps + l.h;
    if (tl >= tiles || n >= a.tokens || hh >= end) {
      xr.v[0] = xr.v[1] = gr.v[0] = gr.v[1] = make_uint4(0, 0, 0, 0);
      return;
    }
    const unsigned b = n / a.T, t = n - b * a.T;
    const NormSide& s = a.side[hh >= H];
    const int h = hh >= H ? hh - H : hh;
    xr = load_row(s.x, s.xs, b, h, t, l);
    gr = load_row(s.g, s.gs, b, h, t, l);
  };
  load(tile, 0, x, g);
  float4 r[4];
  while (tile < tiles) {
    const int next_pass = pass + 1 == passes ? 0 : pass + 1;
    const unsigned next_tile = next_pass ? tile : tile + step;
    Row xn, gn;
    load(next_tile, next_pass, xn, gn);
    if (pass == 0) {
      __syncthreads();  // the last tile's angles are no longer read; the sums are zeroed
      if (a.rope.dims) tile_angles(a, tile, cs);
      __syncthreads();
      if (l.rotated) {
#pragma unroll
        for (int z = 0; z < 4; ++z) r[z] = cs[l.t][4 * l.u4 + z];
      }
    }
    const unsigned n = tile * kTokens + l.t;
    const int hh = first + kPass * pass + l.h;
    const bool on = n < a.tokens && hh < end;
    const NormSide& s = a.side[hh >= H];
    const int h = hh >= H ? hh - H : hh;
    float f[16], d[16], w[16];
    unpack8(x.v[0], f);
    unpack8(x.v[1], f + 8);
    unpack8(g.v[0], d);
    unpack8(g.v[1], d + 8);
    float scale;
    const float inv = row_rms_inv(f, a.eps, &scale);
    if (l.rotated) turn_row(d, d + 8, r, a.rope.interleaved, -1.0f);
    if (on)
      load_weight(a, s, h, l, w);
    else
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = 0.0f;
    float dot = 0.0f, v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      f[i] *= inv;         // n
      v[i] = d[i] * f[i];  // dn n: this row's part of dw
      d[i] *= w[i];
      dot = fmaf(d[i], f[i], dot);
    }
    dot = row_sum(dot) * (1.0f / kHeadDim);
    if (on) {
      const float back = inv * scale;
      float dx[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) dx[i] = back * (d[i] - f[i] * dot);
      const unsigned b = n / a.T;
      store_row(s.y, s.ys, b, h, n - b * a.T, l, dx);
    }
    // Sum of the warp's eight rows: each step hands over half of the values.
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float send = lane & 16 ? v[i] : v[i + 8];
      const float keep = lane & 16 ? v[i + 8] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float send = lane & 8 ? v[i] : v[i + 4];
      const float keep = lane & 8 ? v[i + 4] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 8);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float send = lane & 4 ? v[i] : v[i + 2];
      const float keep = lane & 4 ? v[i + 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 4);
    }
    if (hh < end) {
      const int row = a.per_head ? hh - first : (hh >= H ? kPass : 0) + l.h;
      const int chunk = lane & 16 ? l.c1 : l.c0;
      float* p = acc + (2 * row + wt) * kHeadDim + 8 * chunk + (lane & 8 ? 4 : 0) + (lane & 4 ? 2 : 0);
      p[0] += v[0];
      p[1] += v[1];
    }
    x = xn;
    g = gn;
    pass = next_pass;
    tile = next_tile;
  }
  __syncthreads();
  const int rows = norm_part_rows(a);
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * rows * kHeadDim;
  for (int y = threadIdx.x; y < rows * kHeadDim; y += kThreads) {
    const int row = y / kHeadDim, d = y % kHeadDim;
    float sum = 0.0f;
    if (a.per_head) {
      sum = acc[2 * row * kHeadDim + d] + acc[(2 * row + 1) * kHeadDim + d];
    } else {
#pragma unroll
      for (int z = 0; z < 2 * kPass; ++z) sum += acc[(2 * kPass * row + z) * kHeadDim + d];
    }
    out[y] = sum;
  }
}

// One block a row of the weights' gradients: the CTAs' sums, in 64 bits.
__global__ void __launch_bounds__(kFinishThreads) bam_qk_norm_finish_kernel(const NormArgs a) {
  __shared__ double sums[kFinishThreads];
  grid_dep_wait();
  const int H = a.side[0].heads, d = threadIdx.x % kHeadDim, group = threadIdx.x / kHeadDim;
  constexpr int kGroups = kFinishThreads / kHeadDim;
  const int rows = norm_part_rows(a);
  const int hh = blockIdx.x;  // the head, or q or k
  const int part = a.per_head ? hh / a.heads : 0, step = a.per_head ? a.parts : 1;
  const int row = a.per_head ? hh % a.heads : hh;
  double sum = 0.0;
#pragma unroll 4
  for (int c = part + group * step; c < a.ctas; c += kGroups * step)
    sum += a.part[(static_cast<int64_t>(c) * rows + row) * kHeadDim + d];
  sums[threadIdx.x] = sum;
  __syncthreads();
  if (group == 0) {
    for (int y = 1; y < kGroups; ++y) sum += sums[y * kHeadDim + d];
    const int k = a.per_head ? hh >= H : hh;
    const int h = a.per_head ? (hh >= H ? hh - H : hh) : 0;
    a.side[k].dw[h * kHeadDim + d] = static_cast<float>(sum);
  }
}

int round4(int x) { return (x + kPass - 1) / kPass * kPass; }

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& args, cudaStream_t st) {
  NormArgs a = args;
  const int all = a.side[0].heads + a.side[1].heads, most = kPass * kFwdRows;
  a.parts = (all + most - 1) / most;
  a.heads = round4((all + a.parts - 1) / a.parts);
  a.parts = (all + a.heads - 1) / a.heads;
  const int64_t units = (a.tokens + kTokens - 1) / kTokens * a.parts;
  if (units > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch_k(bam_qk_norm_fwd_kernel, dim3(static_cast<unsigned>(units)), dim3(kThreads), 0, st,
                  false, a);
}

void norm_bwd_config(NormArgs* a, int sms) {
  const int all = a->side[0].heads + a->side[1].heads;
  const int64_t tiles = (a->tokens + kTokens - 1) / kTokens;
  int most = 2 * sms;
  if (most > kNormMaxCtas) most = kNormMaxCtas;
  // As many heads a unit as leave every CTA a few units.
  a->heads = round4(all < kNormMaxHeads ? all : kNormMaxHeads);
  while (a->heads > kPass && tiles * ((all + a->heads - 1) / a->heads) < 2 * most)
    a->heads = round4(a->heads / 2);
  a->parts = (all + a->heads - 1) / a->heads;
  int64_t per_part = most / a->parts;
  if (per_part > tiles) per_part = tiles;
  if (per_part < 1) per_part = 1;
  a->ctas = static_cast<int>(per_part) * a->parts;
}

cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(a.per_head ? a.heads : 2 * kPass) * 2 * kHeadDim * 4;
  return launch_k(bam_qk_norm_bwd_kernel, dim3(a.ctas), dim3(kThreads), smem, st, false, a);
}

cudaError_t launch_norm_bwd_finish(const NormArgs& a, cudaStream_t st) {
  const int rows = a.per_head ? a.side[0].heads + a.side[1].heads : 2;
  return launch_k(bam_qk_norm_finish_kernel, dim3(rows), dim3(kFinishThreads), 0, st, true, a);
}

}  // namespace bam
