// Norms of queries and keys with their rotation by position, and the gradients.
//
//   r = 1 / sqrt(mean(x^2) + eps),   n = x r,   y = R(pos) (w n)
//   dn = R(-pos) dy,  dw = sum dn n,  dx = r (w dn - n mean(w dn n))
//
// per head vector x of 64 values.  A row is read and written once: 256 bytes
// forward, 384 backward, so both are bound by HBM as far as their instructions
// let them: some 200 and 300 of a warp for eight rows, where a copy has 30.  1 / rms is
// computed again in the backward pass (x is read there anyway), so nothing is
// kept between the passes.
//
// Four lanes hold a row, 16 values each, as pairs for f32x2 arithmetic; a tile is 8 or 16
// tokens, whose angles are computed once for all heads (a sine and cosine cost as
// much as a value's whole path), and a CTA goes through the heads of a token in
// order, as they lie in a projection's output.
//
// Measured on the device: 4 x 16383 tokens, 32 and 8 heads, out of a projection's output:
// forward 111 us (0.67 GB, 6.0 TB/s; a copy along the same path takes 101), backward
// 167 us (1.0 GB, 6.0 TB/s); 8 x 512 tokens, 12 and 12 heads: 21 us both calls.
#include "norm_common.cuh"

namespace bam {
namespace {

// Tokens of a thread in a tile, eight apart: two share a head's weights and, backward, the
// sum of its gradient.
constexpr int kFwdSlots = 1, kBwdSlots = 2;
constexpr int kPass = kNormPass;  // heads of a pass, a warp of eight rows each
constexpr int kThreads = 32 * kPass;
constexpr int kFwdStages = 3, kBwdStages = 2;  // passes whose rows are on their way
constexpr int kFinishThreads = 1024;
// Resident CTAs of an SM (forward 6, 7 and 8 take 111, 112 and 111 us in the first case
// above, backward 3, 4 and 5 174, 168 and 182).
constexpr int kFwdResident = 32 / kNormPass, kBwdResident = 16 / kNormPass;

// This thread's place: tokens t and t + 8 of the tile, head h of each pass.
struct Lane : RowLane {
  int t, h;
};
template <int kTurn>
__device__ __forceinline__ Lane lane_of(const RopeArgs& r) {
  return Lane{row_lane<kTurn>(threadIdx.x & 3, r.dims), static_cast<int>(threadIdx.x >> 2) & 7,
              static_cast<int>(threadIdx.x >> 5)};
}

// Cosines and sines (times `sign`) of a tile's tokens, by the whole block.
template <int kSlots>
struct Angles {
  float cos[8 * kSlots][kHeadDim / 2];
  float sin[8 * kSlots][kHeadDim / 2];
};
template <int kSlots>
__device__ __forceinline__ void tile_angles(const NormArgs& a, unsigned tile, float sign,
                                            uint64_t freq, Angles<kSlots>& cs) {
  constexpr int kTokens = 8 * kSlots;
  const int half = a.rope.dims / 2;
  for (int y = threadIdx.x; y < kTokens * (kHeadDim / 2); y += kThreads) {
    const int t = y / (kHeadDim / 2), f = y % (kHeadDim / 2);
    const unsigned n = tile * kTokens + t;
    if (f >= half) continue;
    // (places behind the last token hold zeros, which any angle leaves zero)
    const int pos = n >= a.tokens ? 0
                    : a.positions ? __ldg(a.positions + n)
                                  : static_cast<int>(n - a.T * divide(n, a.by_T));
    const float2 x = rope_angle(static_cast<uint64_t>(static_cast<int64_t>(pos)), freq);
    cs.cos[t][f] = x.x;
    cs.sin[t][f] = sign * x.y;
  }
}

// A CTA's tiles, every `step`-th from `tile` on, and passes; the queries' passes come
// first.
struct Span {
  unsigned tile, tiles, step;
  int first, last, nq;
};
template <int kSlots>
__device__ __forceinline__ Span span_of(const NormArgs& a) {
  constexpr int kTokens = 8 * kSlots;
  Span s;
  s.tiles = (a.tokens + kTokens - 1) / kTokens;
  s.tile = blockIdx.x / a.parts;
  s.step = a.ctas / a.parts;
  s.nq = (a.side[0].heads + kPass - 1) / kPass;
  s.first = static_cast<int>(blockIdx.x - s.tile * a.parts) * a.passes;
  s.last = min(s.first + a.passes, s.nq + (a.side[1].heads + kPass - 1) / kPass);
  return s;
}

// A walk over them: places of this thread's rows in kN tensors, in 16-byte words (32 bits
// where that is enough: fewer registers, see launch_norm_fwd).  `strides` gives those of
// a side's tensor.  A pass further on a side is kPass heads further; places are worked
// out anew for a tile and for a side.
template <int kN, int kSlots, class Off>
struct Walk {
  unsigned tile;
  int pass, side, h;
  bool live[kSlots];
  Off at[kN][kSlots];
  __device__ __forceinline__ bool on(const NormArgs& a, int y) const {
    return live[y] && h < a.side[side].heads;
  }
};
template <int kN, int kSlots, class Off, class F>
__device__ __forceinline__ void walk_to(Walk<kN, kSlots, Off>& w, const NormArgs& a, const Span& s,
                                        const Lane& l, F strides) {
  w.side = w.pass >= s.nq;
  w.h = kPass * (w.pass - (w.side ? s.nq : 0)) + l.h;
#pragma unroll
  for (int y = 0; y < kSlots; ++y) {
    const unsigned n = 8 * (w.tile * kSlots + y) + l.t;
    w.live[y] = w.tile < s.tiles && n < a.tokens;
    const unsigned b = w.live[y] ? divide(n, a.by_T) : 0, t = w.live[y] ? n - b * a.T : 0;
#pragma unroll
    for (int x = 0; x < kN; ++x) {
      const int64_t* st = strides(a.side[w.side], x);
      w.at[x][y] = static_cast<Off>(st[0]) * b + static_cast<Off>(st[1]) * w.h + static_cast<Off>(st[2]) * t;
    }
  }
}
template <int kN, int kSlots, class Off, class F>
__device__ __forceinline__ void walk_on(Walk<kN, kSlots, Off>& w, const NormArgs& a, const Span& s,
                                        const Lane& l, F strides) {
  ++w.pass;
  if (w.pass != s.last && w.pass != s.nq) {
    w.h += kPass;
#pragma unroll
    for (int x = 0; x < kN; ++x) {
      const Off step = static_cast<Off>(strides(a.side[w.side], x)[1]) * kPass;
#pragma unroll
      for (int y = 0; y < kSlots; ++y) w.at[x][y] += step;
    }
    return;
  }
  if (w.pass == s.last) {
    w.pass = s.first;
    w.tile += s.step;
  }
  walk_to(w, a, s, l, strides);
}

// Rows on their way: every thread copies its own chunks into a ring and reads them back, kStages passes
// later (in registers, one pass ahead, backward took 192 us in the first case above).
template <int kN, int kSlots, int kStages>
struct Ring {
  uint4 v[kStages][kSlots][kN][2][kThreads];
};
template <class Off>
__device__ __forceinline__ void copy_row(uint4 (&dst)[2][kThreads], const uint16_t* p, Off at, bool on, const Lane& l) {
  const uint4* src = reinterpret_cast<const uint4*>(p) + (on ? at : 0);
  copy_chunk(&dst[0][threadIdx.x], src + (on ? l.c0 : 0), on);
  copy_chunk(&dst[1][threadIdx.x], src + (on ? l.c1 : 0), on);
}
__device__ __forceinline__ void read_row(const uint4 (&src)[2][kThreads], F2x8& f) {
  const uint4 v[2] = {src[0][threadIdx.x], src[1][threadIdx.x]};
  unpack_row(v, f);
}
template <class Off>
__device__ __forceinline__ void store_row(uint16_t* p, Off at, const Lane& l, const F2x8& f) {
  uint4 v[2];
  pack_row(f, v);
  uint4* dst = reinterpret_cast<uint4*>(p) + at;
  dst[l.c0] = v[0];
  dst[l.c1] = v[1];
}
// A CTA takes its tiles and passes in turn (Span); the rows of the next passes are on their way
// while one is turned and stored.
template <int kTurn, class Off>
__global__ void __launch_bounds__(kThreads, kFwdResident) bam_qk_norm_fwd_kernel(const NormArgs a) {
  __shared__ __align__(16) Angles<kFwdSlots> cs;
  __shared__ __align__(16) Ring<1, kFwdSlots, kFwdStages> ring;
  const Lane l = lane_of<kTurn>(a.rope);
  // this thread's frequency (read once: lanes read the launch's arguments one after the other)
  const uint64_t freq = a.rope.freq[threadIdx.x % (kHeadDim / 2)];
  const Span sp = span_of<kFwdSlots>(a);
  auto xs = [](const NormSide& s, int) { return s.xs; };
  auto ys = [](const NormSide& s, int) { return s.ys; };
  constexpr int kSlots = kFwdSlots;
  Walk<1, kSlots, Off> at, ahead;
  at.tile = ahead.tile = sp.tile;
  at.pass = ahead.pass = sp.first;
  walk_to(ahead, a, sp, l, xs);
  walk_to(at, a, sp, l, ys);
  auto load = [&](int stage) {  // of the next pass
#pragma unroll
    for (int y = 0; y < kSlots; ++y)
      copy_row(ring.v[stage][y][0], a.side[ahead.side].x, ahead.at[0][y], ahead.on(a, y), l);
    copies_commit();
    walk_on(ahead, a, sp, l, xs);
  };
#pragma unroll
  for (int stage = 0; stage < kFwdStages; ++stage) load(stage);
  int stage = 0;
  while (at.tile < sp.tiles) {
    if (kTurn != kNoTurn && at.pass == sp.first) {
      __syncthreads();  // the last tile's angles are no longer read
      tile_angles(a, at.tile, 1.0f, freq, cs);
      __syncthreads();
    }
    F2x8 w;
    load_weight(a.side[at.side].w + (a.per_head && at.on(a, 0) ? at.h * kHeadDim : 0), l, w);
    copies_wait<kFwdStages - 1>();
    F2x8 x[kSlots];
#pragma unroll
    for (int y = 0; y < kSlots; ++y) read_row(ring.v[stage][y][0], x[y]);
    load(stage);
    if (++stage == kFwdStages) stage = 0;
#pragma unroll
    for (int y = 0; y < kSlots; ++y) {
      F2x8& f = x[y];
      float scale;
      const float inv = row_rms_inv(f, a.eps, &scale);
      const uint64_t inv2 = f2_both(inv);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = fmul2(fmul2(f[i], inv2), w[i]);
      turn_values<kTurn>(f, cs.cos[8 * y + l.t], cs.sin[8 * y + l.t], l);
      if (at.on(a, y)) store_row(a.side[at.side].y, at.at[0][y], l, f);
    }
    walk_on(at, a, sp, l, ys);
  }
  copies_wait<0>();  // (no copy outlives its block)
}

// Sum of a warp's eight rows of 16 values (f32x2 pairs): each step hands over half of
// them; this lane ends with the pair whose number is made of its lane bits 4, 3, 2.
__device__ __forceinline__ uint64_t sum_rows(F2x8& v, int lane) {
#pragma unroll
  for (int n = 4, bit = 16; n >= 1; n >>= 1, bit >>= 1) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool up = lane & bit;
      const uint64_t send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = fadd2(keep, __shfl_xor_sync(0xffffffffu, send, bit));
    }
  }
  return v[0];
}

// As the forward kernel.  With r = 1 / rms, d = dn r and u = w d:
// dw gathers d x, and dx = u - x r^2 mean(u x).  The sums of the weights'
// gradients stay in registers as long as they belong to one row of them (a
// side's passes of a tile, or one pass with weights of each head); a warp's eight rows
// are then joined by shuffles and added to shared memory, where every place has
// one warp that adds to it.  The order of every sum is fixed.
template <int kTurn, class Off>
__global__ void __launch_bounds__(kThreads, kBwdResident) bam_qk_norm_bwd_kernel(const NormArgs a) {
  extern __shared__ __align__(16) float acc[];  // [rows][64], a warp adds to each
  __shared__ __align__(16) Angles<kBwdSlots> cs;
  __shared__ __align__(16) Ring<2, kBwdSlots, kBwdStages> ring;
  grid_dep_trigger();
  const Lane l = lane_of<kTurn>(a.rope);
  const int lane = threadIdx.x & 31;
  // this thread's frequency (read once: lanes read the launch's arguments one after the other)
  const uint64_t freq = a.rope.freq[threadIdx.x % (kHeadDim / 2)];
  const int acc_rows = kPass * (a.per_head ? a.passes : 2);
  // (each place is zeroed by a thread of the warp that adds to it)
  for (int y = 0; y < acc_rows / kPass; ++y)
    reinterpret_cast<uint64_t*>(acc + (kPass * y + l.h) * kHeadDim)[lane] = 0;
  __syncwarp();
  const Span sp = span_of<kBwdSlots>(a);
  auto xs = [](const NormSide& s, int x) { return x ? s.gs : s.xs; };
  auto ys = [](const NormSide& s, int) { return s.ys; };
  constexpr int kSlots = kBwdSlots;
  Walk<2, kSlots, Off> ahead;
  Walk<1, kSlots, Off> at;
  at.tile = ahead.tile = sp.tile;
  at.pass = ahead.pass = sp.first;
  walk_to(ahead, a, sp, l, xs);
  walk_to(at, a, sp, l, ys);
  auto load = [&](int stage) {  // of the next pass
#pragma unroll
    for (int y = 0; y < kSlots; ++y) {
      const bool on = ahead.on(a, y);
      copy_row(ring.v[stage][y][0], a.side[ahead.side].x, ahead.at[0][y], on, l);
      copy_row(ring.v[stage][y][1], a.side[ahead.side].g, ahead.at[1][y], on, l);
    }
    copies_commit();
    walk_on(ahead, a, sp, l, xs);
  };
#pragma unroll
  for (int stage = 0; stage < kBwdStages; ++stage) load(stage);
  int stage = 0;
  F2x8 sum;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0;
  while (at.tile < sp.tiles) {
    if (kTurn != kNoTurn && at.pass == sp.first) {
      __syncthreads();  // the last tile's angles are no longer read
      tile_angles(a, at.tile, -1.0f, freq, cs);
      __syncthreads();
    }
    F2x8 w;
    load_weight(a.side[at.side].w + (a.per_head && at.on(a, 0) ? at.h * kHeadDim : 0), l, w);
    copies_wait<kBwdStages - 1>();
#pragma unroll
    for (int y = 0; y < kSlots; ++y) {
      F2x8 f, d;
      read_row(ring.v[stage][y][0], f);
      read_row(ring.v[stage][y][1], d);
      float scale;
      const float inv = row_rms_inv(f, a.eps, &scale);
      turn_values<kTurn>(d, cs.cos[8 * y + l.t], cs.sin[8 * y + l.t], l);
      const uint64_t inv2 = f2_both(inv);
      uint64_t dot0 = 0, dot1 = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = fmul2(d[i], inv2);
        sum[i] = ffma2(d[i], f[i], sum[i]);
        d[i] = fmul2(d[i], w[i]);
        if (i & 1)
          dot1 = ffma2(d[i], f[i], dot1);
        else
          dot0 = ffma2(d[i], f[i], dot0);
      }
      const float dot = row_sum(f2_sum(fadd2(dot0, dot1))) * (1.0f / kHeadDim);
      const uint64_t back = f2_both(-dot * inv * inv);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = ffma2(f[i], back, d[i]);
      if (__any_sync(0xffffffffu, scale != 1.0f)) {
        const uint64_t s2 = f2_both(scale);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = fmul2(d[i], s2);
      }
      if (at.on(a, y)) store_row(a.side[at.side].y, at.at[0][y], l, d);
    }
    load(stage);
    if (++stage == kBwdStages) stage = 0;
    const int pass = at.pass, side = at.side;
    walk_on(at, a, sp, l, ys);
    if (a.per_head || at.pass == sp.first || at.side != side) {
      const uint64_t v = sum_rows(sum, lane);
      const int row = kPass * (a.per_head ? pass - sp.first : side) + l.h;
      const int pair = (lane & 16 ? 4 : 0) + (lane & 8 ? 2 : 0) + (lane & 4 ? 1 : 0);
      uint64_t* p = reinterpret_cast<uint64_t*>(acc + row * kHeadDim + 8 * (pair >= 4 ? l.c1 : l.c0) +
                                                2 * (pair & 3));
      *p = fadd2(*p, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = 0;
    }
  }
  copies_wait<0>();  // (no copy outlives its block)
  __syncthreads();
  const int rows = norm_part_rows(a);
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * rows * kHeadDim;
  for (int y = threadIdx.x; y < rows * kHeadDim; y += kThreads) {
    const int row = y / kHeadDim, d = y % kHeadDim;
    float total = 0.0f;
    const int from = a.per_head ? row : kPass * row, n = a.per_head ? 1 : kPass;
    for (int z = from; z < from + n; ++z) total += acc[z * kHeadDim + d];
    out[y] = total;
  }
}

// Sum with the rounding errors carried along (TwoSum).
__device__ __forceinline__ void add_carried(float& sum, float& err, float x) {
  const float t = sum + x, z = t - sum;
  err += (sum - (t - z)) + (x - z);
  sum = t;
}

constexpr int kFinishDims = 16;  // of a block

// A block takes 16 places of a row of the weights' gradients: the CTAs' sums, as if in 48
// bits (fp64 would take 10 us here).
__global__ void __launch_bounds__(kFinishThreads) bam_qk_norm_finish_kernel(const NormArgs a) {
  __shared__ float2 sums[kFinishThreads];
  grid_dep_wait();
  constexpr int kBlocks = kHeadDim / kFinishDims, kGroups = kFinishThreads / kFinishDims;
  const int out = blockIdx.x / kBlocks;  // row of the weights: queries' first
  const int d = blockIdx.x % kBlocks * kFinishDims + threadIdx.x % kFinishDims;
  const int group = threadIdx.x / kFinishDims, H = a.side[0].heads;
  const int rows = norm_part_rows(a);
  const int k = out >= (a.per_head ? H : 1);  // side, and the head of its weights
  const int h = a.per_head ? out - (k ? H : 0) : 0;
  const int pass = (k ? (H + kPass - 1) / kPass : 0) + h / kPass;
  const int part = a.per_head ? pass / a.passes : 0, step = a.per_head ? a.parts : 1;
  const int row = a.per_head ? kPass * (pass % a.passes) + h % kPass : k;
  float sum = 0.0f, err = 0.0f;
#pragma unroll 8
  for (int c = part + group * step; c < a.ctas; c += kGroups * step)
    add_carried(sum, err, a.part[(static_cast<int64_t>(c) * rows + row) * kHeadDim + d]);
  // a warp's two groups, then the warps' sums
  add_carried(sum, err, __shfl_down_sync(0xffffffffu, sum, kFinishDims));
  err += __shfl_down_sync(0xffffffffu, err, kFinishDims);
  sums[threadIdx.x] = make_float2(sum, err);
  __syncthreads();
  if (group == 0) {
#pragma unroll 8
    for (int y = 2; y < kGroups; y += 2) {
      const float2 x = sums[y * kFinishDims + threadIdx.x];
      add_carried(sum, err, x.x);
      err += x.y;
    }
    // (the error of an infinite sum is NaN)
    a.side[k].dw[h * kHeadDim + d] = isinf(sum) ? sum : sum + err;
  }
}

// A launch of at most `resident` CTAs an SM: as many passes a part as leave a quarter of them a part of a
// tile, so that angles serve many heads (8 x 512 tokens, both calls: 21 us; all of them 25, half 22).
void split_passes(NormArgs* a, int slots, int sms, int resident, int most_ctas) {
  int all = 0;
  for (int k = 0; k < 2; ++k) all += (a->side[k].heads + kPass - 1) / kPass;
  const int64_t tiles = (static_cast<int64_t>(a->tokens) + 8 * slots - 1) / (8 * slots);
  int most = resident * sms;
  if (most > most_ctas) most = most_ctas;
  if (most < 1) most = 1;
  a->passes = all < kNormMaxPasses ? all : kNormMaxPasses;
  while (a->passes > 1 && tiles * ((all + a->passes - 1) / a->passes) < most / 4)
    a->passes = (a->passes + 1) / 2;
  a->parts = (all + a->passes - 1) / a->passes;
  int64_t each = most / a->parts;
  if (each > tiles) each = tiles;
  if (each < 1) each = 1;
  each = (tiles + (tiles + each - 1) / each - 1) / ((tiles + each - 1) / each);  // no more than the longest needs
  a->ctas = static_cast<unsigned>(each) * a->parts;
}

constexpr int turn_of(const RopeArgs& r) { return r.dims == 0 ? kNoTurn : r.interleaved ? kPairs : kHalves; }

typedef void (*Kernel)(NormArgs);
template <class Off>
constexpr Kernel fwd_kernel[] = {bam_qk_norm_fwd_kernel<kNoTurn, Off>,
                                 bam_qk_norm_fwd_kernel<kHalves, Off>, bam_qk_norm_fwd_kernel<kPairs, Off>};

// The sums of the weights' gradients of 16 passes, and beside them the rings and angles, take 53 KB
// of shared memory: more than a launch has without a limit of its own.
template <int kTurn, class Off>
cudaError_t launch_bwd(const NormArgs& a, cudaStream_t st) {
  constexpr size_t kMost = static_cast<size_t>(kPass) * kNormMaxPasses * kHeadDim * 4;
  static bool limit_set[64] = {};
  const cudaError_t e = smem_limit_once(bam_qk_norm_bwd_kernel<kTurn, Off>, kMost, limit_set);
  if (e != cudaSuccess) return e;
  const size_t smem = static_cast<size_t>(kPass * (a.per_head ? a.passes : 2)) * kHeadDim * 4;
  return launch_k(bam_qk_norm_bwd_kernel<kTurn, Off>, dim3(a.ctas), dim3(kThreads), smem, st, false, a);
}
template <class Off>
cudaError_t launch_bwd(const NormArgs& a, cudaStream_t st) {
  switch (turn_of(a.rope)) {
    case kHalves: return launch_bwd<kHalves, Off>(a, st);
    case kPairs: return launch_bwd<kPairs, Off>(a, st);
    default: return launch_bwd<kNoTurn, Off>(a, st);
  }
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& args, cudaStream_t st) {
  NormArgs a = args;
  split_passes(&a, kFwdSlots, sm_count(), kFwdResident, 1 << 30);
  const int turn = turn_of(a.rope);
  return launch_k(a.large ? fwd_kernel<uint64_t>[turn] : fwd_kernel<uint32_t>[turn], dim3(a.ctas),
                  dim3(kThreads), 0, st, false, a);
}

void norm_bwd_config(NormArgs* a, int sms) { split_passes(a, kBwdSlots, sms, kBwdResident, kNormMaxCtas); }

cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t st) {
  return a.large ? launch_bwd<uint64_t>(a, st) : launch_bwd<uint32_t>(a, st);
}

cudaError_t launch_norm_bwd_finish(const NormArgs& a, cudaStream_t st) {
  const int rows = a.per_head ? a.side[0].heads + a.side[1].heads : 2;
  return launch_k(bam_qk_norm_finish_kernel, dim3(rows * (kHeadDim / kFinishDims)), dim3(kFinishThreads), 0, st, true, a);
}

}  // namespace bam
