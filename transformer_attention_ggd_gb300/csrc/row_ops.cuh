// Head vectors of 64 bf16 values, four lanes a row with 16 values each, as the
// row-wise operators (append, norms) take them: unpacking, the rotation of a
// pair by an angle, the norm of a row, and the angles of a tile of tokens.
#pragma once

#include "bam_common.cuh"

namespace bam {

// Rotation by position: turns per position of pair f, times 2^64 (see
// bam_rope).  dims is 0 without rotation.
struct RopeArgs {
  int dims, interleaved;
  uint64_t freq[kHeadDim / 2];
};

#ifdef __CUDACC__

// One rotated pair: (a, b) -> (a cos - b sin, b cos + a sin), in fp32, rounded
// once to bf16 by the caller.
__device__ __forceinline__ void turn(float& a, float& b, float co, float si) {
  const float x = a * co - b * si;
  b = b * co + a * si;
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

// The (cosine, sine) of pair frequency `freq` at position pos: the phase wraps
// modulo 2^64, one turn, which is an exact reduction.  Its top 32 bits, signed,
// are the angle in units of 2^-31 half turns.
__device__ __forceinline__ float2 rope_angle(uint64_t pos, uint64_t freq) {
  const int top = static_cast<int>((pos * freq) >> 32);
  float s, co;
  sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &co);
  return make_float2(co, s);
}

// Turns a lane's 16 values (two chunks of 8) by the angles of its eight pairs, r: their
// (cosine, sine), two in each float4.
// Interleaved pairs lie inside a chunk, the others across the two.
__device__ __forceinline__ void turn_row(float* f0, float* f1, const float4* r, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      turn(f0[4 * z], f0[4 * z + 1], r[z].x, r[z].y);
      turn(f0[4 * z + 2], f0[4 * z + 3], r[z].z, r[z].w);
      turn(f1[4 * z], f1[4 * z + 1], r[2 + z].x, r[2 + z].y);
      turn(f1[4 * z + 2], f1[4 * z + 3], r[2 + z].z, r[2 + z].w);
    }
  } else {
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      turn(f0[2 * z], f1[2 * z], r[z].x, r[z].y);
      turn(f0[2 * z + 1], f1[2 * z + 1], r[z].z, r[z].w);
    }
  }
}

// Sum over the four lanes of a row.
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

constexpr float kBigSquares = 1e38f;
constexpr float kDownScale = 0x1p-68f;

// How a lane's two chunks of 8 values are turned: not at all, as pairs (x_f,
// x_{f + dims/2}) that lie across them, or as neighbouring pairs inside each.
enum : int { kNoTurn = 0, kHalves = 1, kPairs = 2 };

// A lane's 16 values as f32x2 pairs.
typedef uint64_t F2x8[8];
__device__ __forceinline__ void unpack_row(const uint4* v, F2x8& f) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t x[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[4 * c + i] = f2_pack(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xFFFF0000u));
  }
}
__device__ __forceinline__ void pack_row(const F2x8& f, uint4* v) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      f2_unpack(f[4 * c + i], lo, hi);
      x[i] = pack_bf16x2(lo, hi);
    }
    v[c] = make_uint4(x[0], x[1], x[2], x[3]);
  }
}
__device__ __forceinline__ uint64_t f2_both(float x) { return f2_pack(x, x); }
__device__ __forceinline__ float f2_sum(uint64_t x) {
  float lo, hi;
  f2_unpack(x, lo, hi);
  return lo + hi;
}
// One of the four lanes of a row: its two chunks of 8 values (where it can, one of the
// row's first and one of its last four: an access then covers 64 bytes of the row.
// Chunks side by side took twice the sectors: 164 instead of 139 us forward, 4 x 16383
// tokens, 40 heads), and which of them are turned (kHalves: turn0 for both).
struct RowLane {
  int u4, c0, c1;
  bool turn0, turn1;
};
template <int kTurn>
__device__ __forceinline__ RowLane row_lane(int u4, int dims) {
  RowLane l = {u4, u4, u4 + 4, false, false};
  if (kTurn == kHalves) {
    const int nh = dims / 16;
    l.turn0 = u4 < nh;
    l.c0 = l.turn0 ? u4 : 2 * u4;
    l.c1 = l.turn0 ? u4 + nh : 2 * u4 + 1;
  }
  if (kTurn == kPairs) {
    l.turn0 = 8 * l.c0 < dims;
    l.turn1 = 8 * l.c1 < dims;
  }
  return l;
}

// Turns a lane's values by its token's angles, 32 cosines and 32 sines in shared memory
// (they are read for every row: in registers they would take 32).
template <int kTurn>
__device__ __forceinline__ void turn_values(F2x8& f, const float* cos, const float* sin,
                                            const RowLane& l) {
  if (kTurn == kHalves) {
    if (!l.turn0) return;
    const float* pc = cos + 8 * l.u4;
    const float* ps = sin + 8 * l.u4;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      uint64_t c[2], s[2];
      ld_f2x2(pc + 2 * i, c[0], c[1]);
      ld_f2x2(ps + 2 * i, s[0], s[1]);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint64_t x0 = f[i + y], x1 = f[4 + i + y];
        f[i + y] = ffma2(x1, s[y] ^ 0x8000000080000000ull, fmul2(x0, c[y]));
        f[4 + i + y] = ffma2(x0, s[y], fmul2(x1, c[y]));
      }
    }
  }
  if (kTurn == kPairs) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!(h ? l.turn1 : l.turn0)) continue;
      const float4 c = *reinterpret_cast<const float4*>(cos + 4 * (h ? l.c1 : l.c0));
      const float4 s = *reinterpret_cast<const float4*>(sin + 4 * (h ? l.c1 : l.c0));
      const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        float x0, x1;
        f2_unpack(f[4 * h + y], x0, x1);
        turn(x0, x1, cv[y], sv[y]);
        f[4 * h + y] = f2_pack(x0, x1);
      }
    }
  }
}

// 1 / sqrt(mean(x^2) + eps) of each row, by whole warps.  A row whose squares
// leave fp32 (values above 1e18) is scaled by 2^-68 first; the values in f are
// then scaled too and *scale is 2^-68, else 1: f * result is the normalised row
// either way, and result * *scale is 1 / rms.
__device__ __forceinline__ float row_rms_inv(F2x8& f, float eps, float* scale) {
  uint64_t s0 = fmul2(f[0], f[0]), s1 = fmul2(f[1], f[1]);
#pragma unroll
  for (int i = 2; i < 8; i += 2) {
    s0 = ffma2(f[i], f[i], s0);
    s1 = ffma2(f[i + 1], f[i + 1], s1);
  }
  float ss = row_sum(f2_sum(fadd2(s0, s1)));
  *scale = 1.0f;
  const bool big = ss > kBigSquares;
  if (__any_sync(0xffffffffu, big)) {
    const float down = big ? kDownScale : 1.0f;
    const uint64_t d2 = f2_both(down);
    uint64_t s2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] = fmul2(f[i], d2);
      s2 = ffma2(f[i], f[i], s2);
    }
    ss = row_sum(f2_sum(s2));
    eps *= down * down;
    *scale = down;
  }
  return rsqrtf(ss * (1.0f / kHeadDim) + eps);
}

// A chunk of 16 bytes, global -> shared, asynchronously; zeros where it is not `on`.
__device__ __forceinline__ void copy_chunk(uint4* dst, const uint4* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A row's weights.
__device__ __forceinline__ void load_weight(const float* p, const RowLane& l, F2x8& w) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float* q = p + 8 * (c ? l.c1 : l.c0);
    ld_f2x2(q, w[4 * c], w[4 * c + 1]);
    ld_f2x2(q + 4, w[4 * c + 2], w[4 * c + 3]);
  }
}

#endif  // __CUDACC__

}  // namespace bam
