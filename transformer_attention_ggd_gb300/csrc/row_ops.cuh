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

// Turns a lane's 16 values (two chunks of 8) by the angles of its eight pairs;
// `sign` -1 turns back.  r: the pairs' (cosine, sine), two in each float4.
// Interleaved pairs lie inside a chunk, the others across the two.
__device__ __forceinline__ void turn_row(float* f0, float* f1, const float4* r, bool interleaved,
                                         float sign) {
  if (interleaved) {
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      turn(f0[4 * z], f0[4 * z + 1], r[z].x, sign * r[z].y);
      turn(f0[4 * z + 2], f0[4 * z + 3], r[z].z, sign * r[z].w);
      turn(f1[4 * z], f1[4 * z + 1], r[2 + z].x, sign * r[2 + z].y);
      turn(f1[4 * z + 2], f1[4 * z + 3], r[2 + z].z, sign * r[2 + z].w);
    }
  } else {
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      turn(f0[2 * z], f1[2 * z], r[z].x, sign * r[z].y);
      turn(f0[2 * z + 1], f1[2 * z + 1], r[z].z, sign * r[z].w);
    }
  }
}

// Sum over the four lanes of a row.
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// 1 / sqrt(mean(x^2) + eps) of each row, by whole warps.  A row whose squares
// leave fp32 (values above 1e18) is scaled by 2^-68 first; the values in f are
// then scaled too and *scale is 2^-68, else 1: f * result is the normalised row
// either way, and result * *scale is 1 / rms.
__device__ __forceinline__ float row_rms_inv(float (&f)[16], float eps, float* scale) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
  ss = row_sum(ss);
  *scale = 1.0f;
  const bool big = ss > 1e38f;
  if (__any_sync(0xffffffffu, big)) {
    constexpr float kDown = 3.3881317890172014e-21f;  // 2^-68
    const float down = big ? kDown : 1.0f;
    float s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      f[i] *= down;
      s2 = fmaf(f[i], f[i], s2);
    }
    ss = row_sum(s2);
    eps *= down * down;
    *scale = down;
  }
  return rsqrtf(ss * (1.0f / kHeadDim) + eps);
}

#endif  // __CUDACC__

}  // namespace bam
