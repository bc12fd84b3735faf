// Decode over a paged cache whose first keys a whole batch shares and whose own
// keys may carry positions and accumulated weights, on sm_103a.
#include "shared_common.cuh"
#include "table_eval.cuh"

namespace bam {
namespace {

constexpr int kWarps = 4;                    // consumer warps; a producer warp beside them
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStages = 4;
constexpr int kKeys = 64;                    // of a stage: a box of a page
constexpr int kWarpKeys = kKeys / kWarps;
constexpr int kRows = 16;                    // of an item
constexpr int kBoxBytes = kKeys * kHeadDim * 2;
constexpr int kBiasStride = 24;
constexpr float kRescale = 8.0f;

struct RowInfo {
  float alpha, beta, mu, c;  // c: logit scale, log2 units
  int pos;
  int row;                   // b * H + h, or -1
};

struct __align__(1024) SharedSmem {
  uint8_t k[kStages][kBoxBytes];
  uint8_t v[kStages][kBoxBytes];
  int kpos[kStages][kKeys];
  float bias[kWarps][kRows][kBiasStride];
  RowInfo rows[kRows];
  uint64_t full[kStages];
  uint64_t empty[kStages];
  int abort_flag;
};

enum : int {
  kSiteSharedProducer = 90,
  kSiteSharedConsumer = 91,
  kSiteSharedPos = 92  // debug build: bounds of a copy of positions
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kPrepThreads = 256;

// Starts the call and, for the prefix in tiles, fills the table over the distances that its
// keys have from the queries.
__global__ void __launch_bounds__(kPrepThreads) bam_shared_prep_kernel(const SharedArgs a) {
  __shared__ int2 range;
  grid_dep_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) status_begin_call(a.c.status);
  if (!a.table) return;
  bool ok = true;
  const int P = prefix_len(a, &ok);
  if (P == 0) return;
  if (threadIdx.x == 0) range = make_int2(0x7FFFFFFF, -1);
  __syncthreads();
  int lo = 0x7FFFFFFF, hi = -1;
  for (int b = threadIdx.x; b < a.c.B; b += kPrepThreads) {
    const int pos = query_pos(a, b, P, &ok);
    lo = min(lo, pos);
    hi = max(hi, pos);
  }
  atomicMin(&range.x, lo);
  atomicMax(&range.y, hi);
  __syncthreads();
  const int h = blockIdx.y, from = range.x - P + 1;
  const float alpha = a.alpha[h], beta = a.beta[h], mu = a.mu[h];
  for (int d = from + blockIdx.x * kPrepThreads + threadIdx.x; d <= range.y; d += gridDim.x * kPrepThreads) {
    float b, g1, g2;
    bias_terms<false>(d, alpha, beta, mu, a.eps, a.prior, &b, &g1, &g2);
    b = to_f32_finite(b * static_cast<float>(kLog2e));
#pragma unroll
    for (int k = 0; k < kTabCopies; ++k)
      a.table[(static_cast<int64_t>(k) * a.H + h) * a.tab_len + (a.tab_top - d) + k] = b;
  }
}

// An item is up to 16 rows (the heads of one sequence that share a key head, or rows
// of all sequences over the prefix) and one part of their keys.  kTwo: more than 8
// rows.  kParts: bf16 parts of a weight.
template <bool kTwo, int kParts>
__global__ void __launch_bounds__(kThreads) bam_shared_kernel(const __grid_constant__ CUtensorMap tk,
                                                              const __grid_constant__ CUtensorMap tv,
                                                              const SharedArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SharedSmem& sm = *reinterpret_cast<SharedSmem*>(smem_raw + ((0u - smem_u32(smem_raw)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = a.c.Hkv;
  // The item.
  const bool few = a.npsplit && a.copies == 0;  // the prefix's rows are one item's
  const int64_t pitems = few ? static_cast<int64_t>(a.npsplit) * Hkv : 0;
  int64_t item = blockIdx.x;
  const bool prefix = item < pitems;
  int sp, hk, b = 0, r0, nrows;
  if (prefix) {
    sp = static_cast<int>(item % a.npsplit);
    hk = static_cast<int>(item / a.npsplit);
    r0 = 0;
    nrows = a.c.B * a.group;
  } else {
    item -= pitems;
    const int blocks = (a.group + kRows - 1) / kRows;
    sp = static_cast<int>(item % a.nsplit);
    item /= a.nsplit;
    r0 = static_cast<int>(item % blocks) * kRows;
    item /= blocks;
    hk = static_cast<int>(item % Hkv);
    b = static_cast<int>(item / Hkv);
    nrows = min(kRows, a.group - r0);
  }
  bool ok_arg = true;
  const int P = prefix_len(a, &ok_arg);
  const int len = prefix ? P : own_len(a, b, &ok_arg);
  const int chunk = prefix ? part_keys(len, a.npsplit, kPrefixLeast) : part_keys(len, a.nsplit, kOwnLeast);
  const int kbeg = min(len, sp * chunk), kend = min(len, kbeg + chunk);
  const int nst = kend > kbeg ? (kend - kbeg + kKeys - 1) / kKeys : 0;
  const bool marked = !prefix && a.key_pos;
  volatile int* ab = &sm.abort_flag;

  if (threadIdx.x < kRows) {
    const int i = threadIdx.x;
    RowInfo r = {1.0f, 0.0f, 0.0f, 0.0f, 0, -1};
    if (i < nrows) {
      const int rb = prefix ? (r0 + i) / a.group : b;
      const int h = hk * a.group + (prefix ? (r0 + i) % a.group : r0 + i);
      r.pos = query_pos(a, rb, P, &ok_arg);
      r.alpha = __ldg(a.alpha + h);
      r.beta = __ldg(a.beta + h);
      r.mu = __ldg(a.mu + h);
      r.c = shared_scale(a, h, r.pos);
      r.row = rb * a.H + h;
    }
    sm.rows[i] = r;
  }
  if (threadIdx.x == 0) {
    // Behind the prefix in tiles: the kernel before has waited for the call's start.
    if (!a.copies) grid_dep_wait();
    sm.abort_flag = *reinterpret_cast<volatile int*>(&a.c.status->abort);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], kWarps);
    }
    fence_barrier_init();
  }
  __syncthreads();
  if (!ok_arg) record_bad_arg(a.c.status);

  float o[8][4], m[2] = {kNoMax, kNoMax}, l[2] = {0.0f, 0.0f};
#pragma unroll
  for (int d = 0; d < 8; ++d)
#pragma unroll
    for (int x = 0; x < 4; ++x) o[d][x] = 0.0f;

  if (warp == kWarps) {
    if (lane == 0) {
      bool ok = *ab == 0, bad_page = false;
      int issued = 0;
      const int* table = prefix ? a.prefix_table
                                : a.c.block_table + static_cast<size_t>(b) * a.c.max_blocks;
      for (int it = 0; ok && it < nst; ++it) {
        const int s = it % kStages;
        if (it >= kStages &&
            !mbar_wait(&sm.empty[s], (it / kStages - 1) & 1, a.c.status, ab, kSiteSharedProducer))
          break;
        const int kb = kbeg + it * kKeys;
        int pg = __ldg(table + kb / a.c.page);
        if (pg < 0 || pg >= a.c.num_pages) {
          bad_page = true;
          pg = 0;
        }
        const int in = kb % a.c.page, ph = pg * Hkv + hk;
        mbar_arrive_expect_tx(&sm.full[s], 2 * kBoxBytes + (marked ? kKeys * 4 : 0));
        tma_load_3d(sm.k[s], &tk, &sm.full[s], 0, in, ph);
        tma_load_3d(sm.v[s], &tv, &sm.full[s], 0, in, ph);
        if (marked) {
          const int* seg = a.key_pos + static_cast<size_t>(ph) * a.c.page;
          ok = bulk_load_checked(sm.kpos[s], seg + in, kKeys * 4, &sm.full[s], seg, seg + a.c.page,
                                 a.c.status, ab, kSiteSharedPos);
        }
        issued = it + 1;
      }
      for (int it = max(0, issued - kStages); it < issued; ++it)
        mbar_drain(&sm.full[it % kStages], (it / kStages) & 1);
      if (bad_page) record_bad_arg(a.c.status);
    }
  } else {
    const int rq = lane >> 2, cq = 2 * (lane & 3);  // this lane's rows rq, rq + 8; its columns
    uint32_t qf[4][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = sm.rows[rq + 8 * x].row;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + static_cast<int64_t>(row) * kHeadDim);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        qf[ks][x] = row >= 0 ? __ldg(src + (16 * ks + cq) / 2) : 0u;
        qf[ks][x + 2] = row >= 0 ? __ldg(src + (16 * ks + cq) / 2 + 4) : 0u;
      }
    }
    const float c0 = sm.rows[rq].c, c1 = sm.rows[rq + 8].c;
    float* zrow[2] = {nullptr, nullptr};
    if (marked) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = sm.rows[rq + 8 * x].row;
        if (row >= 0) zrow[x] = a.z + row * a.zstride;
      }
    }
    const int key0 = kWarpKeys * warp, bkey = lane & 15;
    bool ok = *ab == 0, bad_pos = false;
    for (int it = 0; ok && it < nst; ++it) {
      const int s = it % kStages;
      ok = mbar_wait(&sm.full[s], (it / kStages) & 1, a.c.status, ab, kSiteSharedConsumer);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int kb = kbeg + it * kKeys + key0;  // this warp's first key
      const int valid = kend - kb;
      const uint32_t kt = smem_u32(sm.k[s]), vt = smem_u32(sm.v[s]);
      // S
      float sacc[2][4];
#pragma unroll
      for (int oc = 0; oc < 2; ++oc) {
#pragma unroll
        for (int x = 0; x < 4; ++x) sacc[oc][x] = 0.0f;
        const int row = key0 + 8 * oc + (lane & 7);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t kf[4];
          ldsm_x4(kt + row * 128 + (((4 * hf + (lane >> 3)) ^ (row & 7)) << 4), kf);
          mma_bf16(sacc[oc], qf[2 * hf], kf[0], kf[1]);
          mma_bf16(sacc[oc], qf[2 * hf + 1], kf[2], kf[3]);
        }
      }
      // The bias of the warp's 16 keys: lane key, rows in turn.
      {
        const int kp = marked ? sm.kpos[s][key0 + bkey] : (prefix ? 0 : P) + kb + bkey;
        for (int r = lane >> 4; r < nrows; r += 2) {
          int d = sm.rows[r].pos - kp;
          if (d < 0) {
            bad_pos |= bkey < valid;
            d = 0;
          }
          float bb, g1, g2;
          bias_terms<false>(d, sm.rows[r].alpha, sm.rows[r].beta, sm.rows[r].mu, a.eps, a.prior,
                            &bb, &g1, &g2);
          sm.bias[warp][r][bkey] = to_f32_finite(bb * static_cast<float>(kLog2e));
        }
        __syncwarp();
      }
#pragma unroll
      for (int x = 0; x < (kTwo ? 2 : 1); ++x) {
        float z[2][2], mx = -INFINITY;
        const float c = x ? c1 : c0;
#pragma unroll
        for (int oc = 0; oc < 2; ++oc) {
          const float2 bi = *reinterpret_cast<const float2*>(&sm.bias[warp][rq + 8 * x][8 * oc + cq]);
          z[oc][0] = fmaf(sacc[oc][2 * x], c, bi.x);
          z[oc][1] = fmaf(sacc[oc][2 * x + 1], c, bi.y);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if (8 * oc + cq + y >= valid) z[oc][y] = -INFINITY;
            mx = fmaxf(mx, z[oc][y]);
          }
          if (zrow[x])
            *reinterpret_cast<float2*>(zrow[x] + kb + 8 * oc + cq) = make_float2(z[oc][0], z[oc][1]);
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (mx > m[x] + kRescale) {
          const float corr = ex2_approx(m[x] - mx);
          l[x] *= corr;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            o[d][2 * x] *= corr;
            o[d][2 * x + 1] *= corr;
          }
          m[x] = mx;
        }
#pragma unroll
        for (int oc = 0; oc < 2; ++oc) {
          sacc[oc][2 * x] = ex2_approx(z[oc][0] - m[x]);
          sacc[oc][2 * x + 1] = ex2_approx(z[oc][1] - m[x]);
          l[x] += sacc[oc][2 * x] + sacc[oc][2 * x + 1];
        }
      }
      // Weights as bf16 parts: all but the last cut off, none of them negative or, where
      // the weight is not, zero (an infinite value then stays one: no inf - inf, no 0 * inf).
      uint32_t pf[kParts][4];
#pragma unroll
      for (int oc = 0; oc < 2; ++oc)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float p0 = kTwo || x == 0 ? sacc[oc][2 * x] : 0.0f;
          float p1 = kTwo || x == 0 ? sacc[oc][2 * x + 1] : 0.0f;
          float least0 = p0 * 0x1p-28f, least1 = p1 * 0x1p-28f;
#pragma unroll
          for (int y = 0; y < kParts - 1; ++y) {
            const uint32_t w0 = __float_as_uint(p0), w1 = __float_as_uint(p1);
            pf[y][2 * oc + x] = __byte_perm(w0, w1, 0x7632);
            p0 = fmaxf(p0 - __uint_as_float(w0 & 0xFFFF0000u), least0);
            p1 = fmaxf(p1 - __uint_as_float(w1 & 0xFFFF0000u), least1);
            least0 *= 0x1p-8f;
            least1 *= 0x1p-8f;
          }
          pf[kParts - 1][2 * oc + x] = pack_bf16x2(p0, p1);
        }
      // What lies behind the last key (anything) has no effect: weight 0 times 0.
      if (valid < kWarpKeys) {
        const int from = max(valid, 0);
        for (int y = lane; y < (kWarpKeys - from) * 8; y += 32)
          *reinterpret_cast<uint4*>(sm.v[s] + (key0 + from) * 128 + 16 * y) = make_uint4(0, 0, 0, 0);
        __syncwarp();
      }
      const int vrow = key0 + (lane & 15);
#pragma unroll
      for (int dd = 0; dd < 4; ++dd) {
        uint32_t vf[4];
        ldsm_x4_t(vt + vrow * 128 + (((2 * dd + (lane >> 4)) ^ (vrow & 7)) << 4), vf);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int p = kParts - 1; p >= 0; --p) mma_bf16(t, pf[p], vf[2 * y], vf[2 * y + 1]);
#pragma unroll
          for (int x = 0; x < 4; ++x) o[2 * dd + y][x] += t[x];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[s]);
    }
    if (bad_pos) record_bad_arg(a.c.status);
  }
  __syncthreads();
  // The prefix's parts are written when this grid ends: the join waits for this grid alone.
  if (a.copies && blockIdx.x == gridDim.x - 1) grid_dep_wait();
  grid_dep_trigger();
  if (*ab) return;
  // Join the four warps in the ring's memory: every copy into it has been waited for.
  float* red_o = reinterpret_cast<float*>(sm.k[0]);          // [warp][row][64]
  float2* red_ml = reinterpret_cast<float2*>(sm.v[0]);       // [warp][row]
  if (warp < kWarps) {
    const int rq = lane >> 2, cq = 2 * (lane & 3);
#pragma unroll
    for (int x = 0; x < (kTwo ? 2 : 1); ++x) {
      float sum = l[x];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int r = rq + 8 * x;
      if ((lane & 3) == 0) red_ml[warp * kRows + r] = make_float2(m[x], sum);
#pragma unroll
      for (int d = 0; d < 8; ++d)
        *reinterpret_cast<float2*>(red_o + (warp * kRows + r) * kHeadDim + 8 * d + cq) =
            make_float2(o[d][2 * x], o[d][2 * x + 1]);
    }
  }
  __syncthreads();
  const int slot = prefix ? a.nsplit + sp : sp;
  for (int y = threadIdx.x; y < nrows * kHeadDim; y += kThreads) {
    const int r = y / kHeadDim, d = y % kHeadDim;
    float M = kNoMax, L = 0.0f, O = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_ml[w * kRows + r].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = red_ml[w * kRows + r];
      const float f = ex2_approx(ml.x - M);
      L += ml.y * f;
      O += red_o[(w * kRows + r) * kHeadDim + d] * f;
    }
    const int64_t at = static_cast<int64_t>(sm.rows[r].row) * a.slots + slot;
    a.part[at * kHeadDim + d] = O;
    if (d == 0) a.ml[at] = make_float2(M, L);
  }
}

constexpr int kJoinWarps = 4;

// One block a row: joins the parts of its keys.
__global__ void __launch_bounds__(32 * kJoinWarps) bam_shared_join_kernel(const SharedArgs a) {
  __shared__ float2 red[kJoinWarps];
  __shared__ float2 red_o[kJoinWarps][32];
  grid_dep_wait();
  grid_dep_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const int64_t base = row * a.slots;
  const bool aborted = *reinterpret_cast<volatile int*>(&a.c.status->abort) != 0;
  float M = kNoMax;
  for (int s = threadIdx.x; s < a.slots; s += 32 * kJoinWarps) M = fmaxf(M, a.ml[base + s].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  if (lane == 0) red[warp].x = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, red[w].x);
  float L = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll 4
  for (int s = warp; s < a.slots; s += kJoinWarps) {
    const float2 ml = a.ml[base + s];
    if (ml.y == 0.0f) continue;  // no key, or no weight
    const float2 o = reinterpret_cast<const float2*>(a.part + (base + s) * kHeadDim)[lane];
    const float f = ex2_approx(ml.x - M);
    L += ml.y * f;
    o0 += o.x * f;
    o1 += o.y * f;
  }
  __syncthreads();
  red[warp].y = L;
  red_o[warp][lane] = make_float2(o0, o1);
  __syncthreads();
  if (warp) return;
  L = o0 = o1 = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    L += red[w].y;
    o0 += red_o[w][lane].x;
    o1 += red_o[w][lane].y;
  }
  float lse2 = M + __log2f(L), inv = 1.0f / L;
  if (L == 0.0f) {
    bool ok = true;
    const int keys = prefix_len(a, &ok) + own_len(a, static_cast<int>(row / a.H), &ok);
    if (keys == 0) {  // no key at all: nothing to weigh
      lse2 = -INFINITY;
      inv = 0.0f;
    }  // else every logit was -inf: 0 / 0
  }
  if (aborted) lse2 = inv = __int_as_float(0x7fc00000);
  o0 *= inv;
  o1 *= inv;
  if (a.o_fp32)
    reinterpret_cast<float2*>(static_cast<float*>(a.o) + row * kHeadDim)[lane] = make_float2(o0, o1);
  else
    reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + row * kHeadDim)[lane] = pack_bf16x2(o0, o1);
  if (lane == 0) {
    if (a.lse) a.lse[row] = lse2 * kLn2f;
    // for the weights, in the first part's place
    if (a.z) a.ml[base] = make_float2(lse2, 0.0f);
  }
}

constexpr int kWeighThreads = 256;
constexpr int kWeighKeys = 4 * kWeighThreads;

// w_j <- decay w_j + sum over the heads of the group of exp(z_j - lse).
__global__ void __launch_bounds__(kWeighThreads) bam_shared_weigh_kernel(const SharedArgs a) {
  grid_dep_wait();
  if (*reinterpret_cast<volatile int*>(&a.c.status->abort)) return;
  const int hk = blockIdx.y, b = blockIdx.z;
  bool ok = true;
  const int len = own_len(a, b, &ok);
  const int j = blockIdx.x * kWeighKeys + 4 * threadIdx.x;
  if (j >= len) return;
  float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int g = 0; g < a.group; ++g) {
    const int64_t row = static_cast<int64_t>(b) * a.H + hk * a.group + g;
    const float lse = a.ml[row * a.slots].x;
    const float4 z = *reinterpret_cast<const float4*>(a.z + row * a.zstride + j);
    w[0] += ex2_approx(z.x - lse);
    w[1] += ex2_approx(z.y - lse);
    w[2] += ex2_approx(z.z - lse);
    w[3] += ex2_approx(z.w - lse);
  }
  const int pg = __ldg(a.c.block_table + static_cast<size_t>(b) * a.c.max_blocks + j / a.c.page);
  if (pg < 0 || pg >= a.c.num_pages) return;
  float* dst = a.key_weight + (static_cast<int64_t>(pg) * a.c.Hkv + hk) * a.c.page + j % a.c.page;
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (j + x < len) dst[x] = fmaf(a.decay, dst[x], w[x]);
}

}  // namespace

void shared_split(SharedArgs* a, int64_t Pmax, int64_t Tmax) {
  const int blocks = (a->group + kRows - 1) / kRows;
  int chunk;
  decode_split(a->c.B * a->c.Hkv * blocks, static_cast<int>(Tmax), &a->nsplit, &chunk);
  a->npsplit = a->copies = a->tab_len = 0;
  if (Pmax > 0) {
    if (static_cast<int64_t>(a->c.B) * a->group <= kFewRows)
      decode_split(a->c.Hkv, static_cast<int>(Pmax), &a->npsplit, &chunk);
    else
      prefix_split(a, Pmax, Tmax);
  }
  a->slots = a->nsplit + a->npsplit * (a->copies > 1 ? a->copies : 1);
}

cudaError_t launch_shared_prep(const SharedArgs& a, cudaStream_t st) {
  dim3 grid(1, 1);
  if (a.table) {
    const int64_t blocks = (static_cast<int64_t>(a.tab_top) + kPrepThreads) / kPrepThreads;
    const int64_t most = (8 * sm_count() + a.H - 1) / a.H;
    grid = dim3(static_cast<unsigned>(blocks < most ? blocks : most), a.H);
  }
  return launch_k(bam_shared_prep_kernel, grid, dim3(kPrepThreads), 0, st, false, a);
}

template <bool kTwo, int kParts>
cudaError_t launch_main(const CUtensorMap& tk, const CUtensorMap& tv, const SharedArgs& a,
                        int64_t items, cudaStream_t st) {
  const size_t smem = sizeof(SharedSmem) + 1024;
  static bool limit_set[64] = {};
  const cudaError_t e = smem_limit_once(bam_shared_kernel<kTwo, kParts>, smem, limit_set);
  if (e != cudaSuccess) return e;
  return launch_k(bam_shared_kernel<kTwo, kParts>, dim3(static_cast<unsigned>(items)), dim3(kThreads),
                  smem, st, true, tk, tv, a);
}

cudaError_t launch_shared(const CUtensorMap& tk, const CUtensorMap& tv, const SharedArgs& a,
                          cudaStream_t st) {
  const int blocks = (a.group + kRows - 1) / kRows;
  const bool few = a.npsplit && a.copies == 0;
  const int64_t items = static_cast<int64_t>(a.nsplit) * a.c.B * a.c.Hkv * blocks +
                        (few ? static_cast<int64_t>(a.npsplit) * a.c.Hkv : 0);
  if (items > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const bool two = a.group > 8 || (few && a.c.B * a.group > 8);
  if (a.o_fp32)
    return two ? launch_main<true, 3>(tk, tv, a, items, st) : launch_main<false, 3>(tk, tv, a, items, st);
  return two ? launch_main<true, 2>(tk, tv, a, items, st) : launch_main<false, 2>(tk, tv, a, items, st);
}

cudaError_t launch_shared_join(const SharedArgs& a, cudaStream_t st) {
  return launch_k(bam_shared_join_kernel, dim3(a.c.B * a.H), dim3(32 * kJoinWarps), 0, st, true, a);
}

cudaError_t launch_shared_weigh(const SharedArgs& a, cudaStream_t st) {
  const unsigned tiles = static_cast<unsigned>((a.zstride + kWeighKeys - 1) / kWeighKeys);
  return launch_k(bam_shared_weigh_kernel, dim3(tiles, a.c.Hkv, a.c.B), dim3(kWeighThreads), 0, st, true, a);
}

}  // namespace bam
