// Decode over a paged cache whose first keys a whole batch shares and whose own
// keys may carry positions and accumulated weights, on sm_103a.
//
//   z[r, j] = c_r q_r . k_j + b_h(pos_r - pos_j),  o = sum_j exp(z - lse) v_j,
//   w_j <- decay w_j + sum over the heads r of j's key head of exp(z[r, j] - lse_r)
//
// 256 bytes a key and key head, 256 flops a key and row of up to 16 rows: bound by HBM as far as the
// logits' instructions let it (with marks 12 bytes a key more, and 8 a row and key for the logits,
// which stay in L2).  The first kernel starts the call and fills the prefix's table of biases;
// the prefix goes in tiles (prefix.cu) where nine or more rows share it; the main kernel takes
// what is left on mma.sync, whose 16 rows the heads of a group fill as far as they do; the
// last one joins the parts of a row and, in blocks of its own, adds to the weights, which need every row's sum:
// each takes it from the parts (two kernels in turn took 2.5 us longer in small calls).
//
// Positions of kept keys are any numbers, so that the own keys' biases are evaluated where they
// are needed (20 instructions and two special functions; windows of a table in order of
// positions took 160 us where this takes 151).
//
// Measured: 64 caches of 8192 keys, 12 heads, with weights 151 us (0.85 GB, 5.7 TB/s); one of
// 131072, 32 and 8 heads, 65 us, with fp32 output 71; 4 sequences of 40 keys behind 1000, 12 heads, 12 us.
#include "shared_common.cuh"

namespace bam {
namespace {

// A row's prior, ready to be evaluated:
//   b log2(e) = -log2(e) 2^y,  y = beta (log2 u - log2 alpha),  u = |d - mu| (at least eps where beta <= 0),
// or, with the theta prior, y = theta_beta log2(|d - mu| + eps) + theta_alpha log2(e).
struct __align__(16) BiasRow {
  float beta, mu;
  float least, add;  // u = max(|d - mu|, least) + add
  float e, l;        // log2 alpha: integer part and the rest
  float hi, lo;      // theta_alpha log2(e) as a sum of two floats
};
__device__ __forceinline__ BiasRow bias_row(const SharedArgs& a, int h) {
  BiasRow r;
  const float alpha = __ldg(a.alpha + h);
  r.beta = __ldg(a.beta + h);
  r.mu = __ldg(a.mu + h);
  r.least = r.add = r.e = r.l = r.hi = r.lo = 0.0f;
  if (a.prior == kPriorTheta) {
    r.mu = 2.0f * sinhf(r.mu);
    r.add = a.eps;
    constexpr float kL2eHi = 1.44269502162933349609375f, kL2eLo = 1.925962989091e-08f;  // log2(e)
    r.hi = alpha * kL2eHi;
    r.lo = fmaf(alpha, kL2eHi, -r.hi) + alpha * kL2eLo;
  } else {
    if (r.beta <= 0.0f) r.least = a.eps;
    int e;
    const float m = frexpf(alpha, &e);
    r.e = static_cast<float>(e);
    r.l = log2f(m);
  }
  return r;
}
// b(d) log2(e) to a few 1e-7 relative: the exponent y is a sum of two floats (its large part beta times
// an integer is split exactly), and 2^y is 2^n, exact, times exp2 of the rest.
__device__ __forceinline__ float bias_value(float d, const BiasRow& r) {
  const float u = fmaxf(fabsf(d - r.mu), r.least) + r.add;
  const int bits = __float_as_int(u);
  const float e = static_cast<float>((bits >> 23) - 126) - r.e;
  const float l = __log2f(__int_as_float((bits & 0x007FFFFF) | 0x3F000000)) - r.l;  // u's mantissa in [1/2, 1)
  const float p = r.beta * e, q = fmaf(r.beta, e, -p), t = r.beta * l;
  const float s1 = p + t, v1 = s1 - p, e1 = (p - (s1 - v1)) + (t - v1);
  const float s2 = s1 + r.hi, v2 = s2 - s1, e2 = (s1 - (s2 - v2)) + (r.hi - v2);
  const float y = fminf(fmaxf(s2, -120.0f), 400.0f), n = floorf(y);
  const float f = (y - n) + (e1 + e2 + q + r.lo);
  const float scale = __int_as_float((static_cast<int>(fminf(n, 127.0f)) + 127) << 23);
  const float b = -ex2_approx(f) * scale * (n > 127.0f ? 3.0e38f : 1.0f) * 1.44269504088896341f;
  return u == 0.0f ? 0.0f : fmaxf(b, -3.0e38f);
}

constexpr int kWarps = 4;                    // of a CTA, each on items of its own
constexpr int kThreads = 32 * kWarps;
constexpr int kResident = 3;                 // CTAs of an SM
constexpr int kStages = 2;                   // of a warp's ring
constexpr int kKeys = 32;                    // of a stage
constexpr int kRows = 16;                    // of an item
constexpr int kBoxBytes = kKeys * kHeadDim * 2;
constexpr int kBiasStride = kKeys + 8;       // floats: 8-byte reads of four rows hit all banks
constexpr float kRescale = 8.0f;

template <bool kTwo>
struct __align__(1024) SharedSmem {
  uint8_t k[kWarps][kStages][kBoxBytes];
  uint8_t v[kWarps][kStages][kBoxBytes];
  int kpos[kWarps][kStages][kKeys];
  float bias[kWarps][kTwo ? kRows : kRows / 2][kBiasStride];
  BiasRow rows[kWarps][kRows];
  uint64_t full[kWarps][kStages];
  int abort_flag;
};

enum : int {
  kSiteSharedTile = 91,
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

// The next item of the call, behind the status words.
__device__ __forceinline__ unsigned* item_counter(DevStatus* st) {
  return reinterpret_cast<unsigned*>(st) + 32;
}
static_assert(kFewRows <= kRows / 2);
static_assert(sizeof(DevStatus) <= 128 && kStatusBytes >= 256, "place of the item counter");

constexpr int kPrepThreads = 256;

// Starts the call and, for a prefix in tiles, fills its table over the distances that its keys have
// from the queries.
__global__ void __launch_bounds__(kPrepThreads) bam_shared_prep_kernel(const SharedArgs a) {
  __shared__ int least, most;  // position of any query
  grid_dep_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    status_begin_call(a.c.status);
    *item_counter(a.c.status) = 0;
  }
  if (!a.table) return;
  bool ok = true;
  const int P = prefix_len(a, &ok);
  if (P == 0) return;
  if (threadIdx.x == 0) least = 0x7FFFFFFF, most = -1;
  __syncthreads();
  int lo = 0x7FFFFFFF, hi = -1;
  for (int b = threadIdx.x; b < a.c.B; b += kPrepThreads) {
    const int pos = query_pos(a, b, P, &ok);
    lo = min(lo, pos);
    hi = max(hi, pos);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if ((threadIdx.x & 31) == 0) {
    atomicMin(&least, lo);
    atomicMax(&most, hi);
  }
  __syncthreads();
  const int h = blockIdx.y;
  const BiasRow row = bias_row(a, h);
  float* tab = a.table + static_cast<int64_t>(h) * a.tab_len + a.tab_top;
  const int64_t copy = static_cast<int64_t>(a.H) * a.tab_len + 1;
  for (int d = least - P + 1 + blockIdx.x * kPrepThreads + threadIdx.x; d <= most;
       d += gridDim.x * kPrepThreads) {
    const float b = bias_value(static_cast<float>(d), row);
#pragma unroll
    for (int k = 0; k < kTabCopies; ++k) tab[k * copy - d] = b;
  }
}

// An item: up to 16 rows (the heads of one sequence that share a key head, or all rows over the
// prefix, up to 8) and one part of their keys.
struct Item {
  bool on, prefix;
  int sp, hk, b, r0, nrows;
  int kbeg, kend, P;
};
__device__ __forceinline__ Item item_at(const SharedArgs& a, int64_t id, bool* ok) {
  const int64_t pitems = a.npsplit && a.copies == 0 ? static_cast<int64_t>(a.npsplit) * a.c.Hkv : 0;
  const int blocks = (a.group + kRows - 1) / kRows;
  Item x;
  x.P = prefix_len(a, ok);
  x.on = id < pitems + static_cast<int64_t>(a.nsplit) * a.c.B * a.c.Hkv * blocks;
  x.prefix = id < pitems;
  int len = 0, chunk = 64;
  x.b = x.r0 = 0;
  if (x.prefix) {
    x.sp = static_cast<int>(id % a.npsplit);
    x.hk = static_cast<int>(id / a.npsplit);
    x.nrows = a.c.B * a.group;
    len = x.P;
    chunk = part_keys(len, a.npsplit);
  } else {
    // (the counts of items and of their factors fit 32 bits)
    unsigned y = static_cast<unsigned>(id - pitems);
    x.sp = static_cast<int>(y % a.nsplit);
    y /= a.nsplit;
    if (blocks > 1) {
      x.r0 = static_cast<int>(y % blocks) * kRows;
      y /= blocks;
    }
    x.hk = static_cast<int>(y % a.c.Hkv);
    x.b = static_cast<int>(y / a.c.Hkv);
    x.nrows = min(kRows, a.group - x.r0);
    if (x.on) {
      len = own_len(a, x.b, ok);
      chunk = part_keys(len, a.nsplit);
    }
  }
  x.kbeg = static_cast<int>(min(static_cast<int64_t>(len), static_cast<int64_t>(x.sp) * chunk));
  x.kend = min(len, x.kbeg + chunk);
  return x;
}
// Row `i` of an item: sequence and query head.
__device__ __forceinline__ int item_row(const SharedArgs& a, const Item& x, int i, int* b, int* h) {
  *b = x.prefix ? i / a.group : x.b;
  *h = x.hk * a.group + (x.prefix ? i - *b * a.group : x.r0 + i);
  return *b * a.H + *h;
}
__device__ __forceinline__ int64_t item_slot(const SharedArgs& a, const Item& x, int row) {
  return static_cast<int64_t>(row) * a.slots + (x.prefix ? a.nsplit + x.sp : x.sp);
}

// Every warp takes items by itself, from a counter that the call's first kernel sets to 0 (which warp
// computes an item changes nothing in it), and runs through their keys in tiles of 32; the next
// tiles, of the next item too, are on their way meanwhile.  Nothing is joined in
// a CTA: items of a few hundred keys, whose start a CTA of its own each paid for, took 24 us
// where these take 15 (64 sequences of up to 512 keys, 12 heads).  kTwo: more than 8 rows.  kParts: bf16 parts of
// a weight.
template <bool kTwo, int kParts>
__global__ void __launch_bounds__(kThreads, kResident)
    bam_shared_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                      const SharedArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SharedSmem<kTwo>& sm = *reinterpret_cast<SharedSmem<kTwo>*>(smem_raw + ((0u - smem_u32(smem_raw)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = a.c.Hkv;
  volatile int* ab = &sm.abort_flag;
  DevStatus* const status = a.c.status;
  if (threadIdx.x == 0) {
    // Behind the prefix in tiles: the kernel before has waited for the call's start.
    if (!a.copies) grid_dep_wait();
    sm.abort_flag = *reinterpret_cast<volatile int*>(&status->abort);
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[w][s], 1);
    fence_barrier_init();
  }
  __syncthreads();
  const bool marked = a.key_pos;
  bool ok_arg = true, bad_page = false, bad_pos = false;
  bool ok = *ab == 0;

  // The next item with keys (one without leaves an empty part).
  auto fetch = [&]() {
    for (;;) {
      unsigned id = 0;
      if (lane == 0) id = atomicAdd(item_counter(status), 1u);
      id = __shfl_sync(0xffffffffu, id, 0);
      const Item x = item_at(a, id, &ok_arg);
      if (!x.on || x.kend > x.kbeg) return x;
      if (lane < x.nrows) {
        int b, h;
        a.ml[item_slot(a, x, item_row(a, x, lane, &b, &h))] = make_float2(kNoMax, 0.0f);
      }
    }
  };
  // The walk of the copies: item, first key of the next tile, its page, and the page after it.
  Item ld;
  int ld_key = 0, ld_in = 0, ld_blk = 0, ld_page = 0, issued = 0;
  const int* ld_table = nullptr;
  auto begin = [&](const Item& x) {
    ld = x;
    if (!x.on) return;
    ld_key = x.kbeg;
    ld_blk = ld_key / a.c.page;
    ld_in = ld_key - ld_blk * a.c.page;
    ld_table = x.prefix ? a.prefix_table : a.c.block_table + static_cast<size_t>(x.b) * a.c.max_blocks;
    ld_page = __ldg(ld_table + ld_blk);
  };
  auto issue = [&]() {
    int pg = ld_page;
    if (pg < 0 || pg >= a.c.num_pages) {
      bad_page = true;
      pg = 0;
    }
    if (lane == 0) {
      const int s = issued % kStages, ph = pg * Hkv + ld.hk;
      const bool pos = marked && !ld.prefix;
      uint64_t* bar = &sm.full[warp][s];
      mbar_arrive_expect_tx(bar, 2 * kBoxBytes + (pos ? kKeys * 4 : 0));
      tma_load_3d(sm.k[warp][s], &tk, bar, 0, ld_in, ph);
      tma_load_3d(sm.v[warp][s], &tv, bar, 0, ld_in, ph);
      if (pos) {
        const int* seg = a.key_pos + static_cast<size_t>(ph) * a.c.page;
        bulk_load_checked(sm.kpos[warp][s], seg + ld_in, kKeys * 4, bar, seg, seg + a.c.page, status, ab,
                          kSiteSharedPos);
      }
    }
    ++issued;
    ld_key += kKeys;
    ld_in += kKeys;
    if (ld_in == a.c.page) {
      ld_in = 0;
      ++ld_blk;
      if (ld_key < ld.kend) ld_page = __ldg(ld_table + ld_blk);
    }
  };

  Item cur = fetch();
  begin(cur);
  int used = 0;
  const int rq = lane >> 2, cq = 2 * (lane & 3);  // this lane's rows rq, rq + 8; its columns
  while (ok && cur.on) {
    bool have_next = false;
    Item next = cur;
    // Rows: lane i holds row i's parameters; products take the queries of rows rq and rq + 8.
    float scale = 0.0f;
    int pos = 0, row = -1;
    if (lane < cur.nrows) {
      int b, h;
      row = item_row(a, cur, lane, &b, &h);
      pos = query_pos(a, b, cur.P, &ok_arg);
      scale = shared_scale(a, h, pos);
      sm.rows[warp][lane] = bias_row(a, h);
    }
    __syncwarp();
    const bool tile_marked = marked && !cur.prefix;
    uint32_t qf[4][4];
    float c[2];
    float* zrow[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = __shfl_sync(0xffffffffu, row, rq + 8 * x);
      c[x] = __shfl_sync(0xffffffffu, scale, rq + 8 * x);
      zrow[x] = tile_marked && r >= 0 ? a.z + r * a.zstride : nullptr;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + static_cast<int64_t>(r) * kHeadDim);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        qf[ks][x] = r >= 0 ? __ldg(src + (16 * ks + cq) / 2) : 0u;
        qf[ks][x + 2] = r >= 0 ? __ldg(src + (16 * ks + cq) / 2 + 4) : 0u;
      }
    }
    float o[8][4], m[2] = {kNoMax, kNoMax}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[d][x] = 0.0f;

    for (int kb = cur.kbeg; kb < cur.kend; kb += kKeys) {
      while (issued - used < kStages) {
        if (ld.on && ld_key >= ld.kend) {
          if (have_next) break;
          next = fetch();
          have_next = true;
          begin(next);
        }
        if (!ld.on) break;
        issue();
      }
      const int s = used % kStages;
      ok = mbar_wait(&sm.full[warp][s], (used / kStages) & 1, status, ab, kSiteSharedTile);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int valid = cur.kend - kb;
      const bool full = valid >= kKeys;
      // The bias, a key a lane and rows in turn, handed over in shared memory.  (Out of a table that
      // the call's first kernel fills it took 160 instead of 151 us for 64 caches of 8192 keys, and 80
      // instead of 66 for one of 131072.)
      {
        const int kp = tile_marked ? sm.kpos[warp][s][lane] : (cur.prefix ? 0 : cur.P) + kb + lane;
#pragma unroll 2
        for (int r = 0; r < cur.nrows; ++r) {
          int d = __shfl_sync(0xffffffffu, pos, r) - kp;
          if (d < 0 || (tile_marked && kp < 0)) {
            bad_pos |= lane < valid;
            d = max(d, 0);
          }
          sm.bias[warp][r][lane] = bias_value(static_cast<float>(d), sm.rows[warp][r]);
        }
        __syncwarp();
      }
      const uint32_t kt = smem_u32(sm.k[warp][s]), vt = smem_u32(sm.v[warp][s]);
      // S
      float sacc[4][4];
#pragma unroll
      for (int oc = 0; oc < 4; ++oc) {
#pragma unroll
        for (int x = 0; x < 4; ++x) sacc[oc][x] = 0.0f;
        const int kr = 8 * oc + (lane & 7);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t kf[4];
          ldsm_x4(kt + kr * 128 + (((4 * hf + (lane >> 3)) ^ (kr & 7)) << 4), kf);
          mma_bf16(sacc[oc], qf[2 * hf], kf[0], kf[1]);
          mma_bf16(sacc[oc], qf[2 * hf + 1], kf[2], kf[3]);
        }
      }
#pragma unroll
      for (int x = 0; x < (kTwo ? 2 : 1); ++x) {
        float mx = -INFINITY;
#pragma unroll
        for (int oc = 0; oc < 4; ++oc) {
          const float2 bi = *reinterpret_cast<const float2*>(&sm.bias[warp][rq + 8 * x][8 * oc + cq]);
          float z0 = fmaf(sacc[oc][2 * x], c[x], bi.x), z1 = fmaf(sacc[oc][2 * x + 1], c[x], bi.y);
          if (!full) {
            if (8 * oc + cq >= valid) z0 = -INFINITY;
            if (8 * oc + cq + 1 >= valid) z1 = -INFINITY;
          }
          mx = fmax3(mx, z0, z1);
          if (zrow[x]) *reinterpret_cast<float2*>(zrow[x] + kb + 8 * oc + cq) = make_float2(z0, z1);
          sacc[oc][2 * x] = z0;
          sacc[oc][2 * x + 1] = z1;
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
        for (int oc = 0; oc < 4; ++oc) {
          sacc[oc][2 * x] = ex2_approx(sacc[oc][2 * x] - m[x]);
          sacc[oc][2 * x + 1] = ex2_approx(sacc[oc][2 * x + 1] - m[x]);
          l[x] += sacc[oc][2 * x] + sacc[oc][2 * x + 1];
        }
      }
      // Weights as bf16 parts: all but the last cut off, none of them negative or, where
      // the weight is not, zero (an infinite value then stays one: no inf - inf, no 0 * inf).  The last
      // bit of a weight, set, makes sure of the second part; a third has a least value.
      uint32_t pf[2][kParts][4];  // of 16 keys each
#pragma unroll
      for (int oc = 0; oc < 4; ++oc)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t(&w)[kParts][4] = pf[oc >> 1];
          const int at = 2 * (oc & 1) + x;
          if (!kTwo && x) {
#pragma unroll
            for (int y = 0; y < kParts; ++y) w[y][at] = 0;
            continue;
          }
          uint32_t w0 = __float_as_uint(sacc[oc][2 * x]) | 1u, w1 = __float_as_uint(sacc[oc][2 * x + 1]) | 1u;
          float p0 = __uint_as_float(w0), p1 = __uint_as_float(w1);
          const float least0 = p0 * 0x1p-36f, least1 = p1 * 0x1p-36f;
#pragma unroll
          for (int y = 0; y < kParts - 1; ++y) {
            w[y][at] = __byte_perm(w0, w1, 0x7632);
            p0 -= __uint_as_float(w0 & 0xFFFF0000u);
            p1 -= __uint_as_float(w1 & 0xFFFF0000u);
            if (y == 1) p0 = fmaxf(p0, least0), p1 = fmaxf(p1, least1);
            w0 = __float_as_uint(p0), w1 = __float_as_uint(p1);
          }
          w[kParts - 1][at] = pack_bf16x2(p0, p1);
        }
      // What lies behind the last key (anything) has no effect: weight 0 times 0.
      if (valid < kKeys) {
        for (int y = lane; y < (kKeys - valid) * 8; y += 32)
          *reinterpret_cast<uint4*>(sm.v[warp][s] + valid * 128 + 16 * y) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();  // the next copy comes into the same place
        __syncwarp();
      }
#pragma unroll
      for (int dd = 0; dd < 4; ++dd) {
        uint32_t vf[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int vr = 16 * h + (lane & 15);
          ldsm_x4_t(vt + vr * 128 + (((2 * dd + (lane >> 4)) ^ (vr & 7)) << 4), vf[h]);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if (kParts < 3) {
#pragma unroll
            for (int p = kParts - 1; p >= 0; --p)
#pragma unroll
              for (int h = 0; h < 2; ++h) mma_bf16(o[2 * dd + y], pf[h][p], vf[h][2 * y], vf[h][2 * y + 1]);
          } else {
            // The tensor core's sums cut off their last place in every step: for fp32 output a
            // tile's are added outside.
            float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int p = kParts - 1; p >= 0; --p)
#pragma unroll
              for (int h = 0; h < 2; ++h) mma_bf16(t, pf[h][p], vf[h][2 * y], vf[h][2 * y + 1]);
#pragma unroll
            for (int x = 0; x < (kTwo ? 4 : 2); ++x) o[2 * dd + y][x] += t[x];
          }
        }
      }
      __syncwarp();
      ++used;
    }
    if (!ok) break;
    // This part of each row.
#pragma unroll
    for (int x = 0; x < (kTwo ? 2 : 1); ++x) {
      float sum = l[x];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int r = __shfl_sync(0xffffffffu, row, rq + 8 * x);
      if (r < 0) continue;
      const int64_t at = item_slot(a, cur, r);
      if ((lane & 3) == 0) a.ml[at] = make_float2(m[x], sum);
#pragma unroll
      for (int d = 0; d < 8; ++d)
        *reinterpret_cast<float2*>(a.part + at * kHeadDim + 8 * d + cq) =
            make_float2(o[d][2 * x], o[d][2 * x + 1]);
    }
    __syncwarp();
    if (!have_next) {
      next = fetch();
      begin(next);
    }
    cur = next;
  }
  if (lane == 0)  // given up: what is still on its way
    for (; used < issued; ++used) mbar_drain(&sm.full[warp][used % kStages], (used / kStages) & 1);
  if (!ok_arg || bad_page || bad_pos) record_bad_arg(status);
  // The prefix's parts are written when this grid ends: the join waits for this grid alone.
  if (a.copies && blockIdx.x == gridDim.x - 1) grid_dep_wait();
}

// Joins the parts of a row's keys, kWarpsRow warps a row, kEndWarps a block.
template <int kWarpsRow, int kEndWarps>
__device__ __forceinline__ void join_rows(const SharedArgs& a, int64_t block) {
  constexpr int kRowsBlock = kEndWarps / kWarpsRow;
  __shared__ float red_m[kRowsBlock][kWarpsRow], red_l[kRowsBlock][kWarpsRow];
  __shared__ float2 red_o[kRowsBlock][kWarpsRow][32];
  const int64_t rows = static_cast<int64_t>(a.c.B) * a.H;
  if (block * kRowsBlock >= rows) return;
  grid_dep_wait();
  const int lane = threadIdx.x & 31, part = (threadIdx.x >> 5) % kWarpsRow, rb = (threadIdx.x >> 5) / kWarpsRow;
  const int64_t row_raw = block * kRowsBlock + rb;
  const int64_t row = min(row_raw, rows - 1), base = row * a.slots;
  const bool aborted = *reinterpret_cast<volatile int*>(&a.c.status->abort) != 0;
  float M = kNoMax;
  for (int s = 32 * part + lane; s < a.slots; s += 32 * kWarpsRow) M = fmaxf(M, a.ml[base + s].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  if (kWarpsRow > 1) {
    if (lane == 0) red_m[rb][part] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarpsRow; ++w) M = fmaxf(M, red_m[rb][w]);
  }
  float L = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll 8
  for (int s = part; s < a.slots; s += kWarpsRow) {
    const float2 ml = a.ml[base + s];
    const float2 o = reinterpret_cast<const float2*>(a.part + (base + s) * kHeadDim)[lane];
    const bool none = ml.y == 0.0f;  // no key, or no weight: nothing is there
    const float f = none ? 0.0f : ex2_approx(ml.x - M);
    L += ml.y * f;
    o0 = none ? o0 : fmaf(o.x, f, o0);
    o1 = none ? o1 : fmaf(o.y, f, o1);
  }
  if (kWarpsRow > 1) {
    if (lane == 0) red_l[rb][part] = L;
    red_o[rb][part][lane] = make_float2(o0, o1);
    __syncthreads();
    L = o0 = o1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarpsRow; ++w) {
      L += red_l[rb][w];
      o0 += red_o[rb][w][lane].x;
      o1 += red_o[rb][w][lane].y;
    }
  }
  if (part || row_raw >= rows) return;
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
  if (a.lse && lane == 0) a.lse[row] = lse2 * kLn2f;
}

constexpr int kWeighFours = 2;  // of a thread
constexpr int weigh_keys_of(int warps) { return 4 * kWeighFours * 32 * warps; }
constexpr int kWeighRows = 64;  // whose sums are at hand at a time

// w_j <- decay w_j + sum over the heads of the group of exp(z_j - lse), for a run of a sequence's keys.  A
// row's maximum and sum stay apart: z less the maximum is as exact as z, while maximum + log2(sum) is a
// number of the logits' size, whose last place may be more than log2(sum) (far from every key).
template <int kEndWarps>
__device__ __forceinline__ void weigh_keys(const SharedArgs& a, unsigned block) {
  constexpr int kEndThreads = 32 * kEndWarps, kWeighKeys = 4 * kWeighFours * kEndThreads;
  __shared__ float2 row_ml[kWeighRows];  // maximum, 1 / sum
  const int hk = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
  bool ok = true;
  const int len = own_len(a, b, &ok);
  const int64_t begin = static_cast<int64_t>(block) * kWeighKeys;
  if (begin >= len) return;
  const int j0 = static_cast<int>(begin) + 4 * threadIdx.x;
  // What no kernel of the call writes is on its way before the logits are there.
  float* at[kWeighFours];
  float4 old[kWeighFours];
#pragma unroll
  for (int x = 0; x < kWeighFours; ++x) {
    const int j = j0 + 4 * kEndThreads * x;
    at[x] = nullptr;
    if (j >= len) continue;
    const int pg = __ldg(a.c.block_table + static_cast<size_t>(b) * a.c.max_blocks + j / a.c.page);
    if (pg < 0 || pg >= a.c.num_pages) continue;
    at[x] = a.key_weight + (static_cast<int64_t>(pg) * a.c.Hkv + hk) * a.c.page + j % a.c.page;
    old[x] = *reinterpret_cast<const float4*>(at[x]);
  }
  grid_dep_wait();
  if (*reinterpret_cast<volatile int*>(&a.c.status->abort)) return;
  const int64_t row0 = static_cast<int64_t>(b) * a.H + hk * a.group;
  float w[kWeighFours][4] = {};
  float4 z[kWeighFours];
  auto load = [&](int g) {
#pragma unroll
    for (int x = 0; x < kWeighFours; ++x)
      if (at[x]) z[x] = *reinterpret_cast<const float4*>(a.z + (row0 + g) * a.zstride + j0 + 4 * kEndThreads * x);
  };
  load(0);
  for (int g0 = 0; g0 < a.group; g0 += kWeighRows) {
    const int rows = min(kWeighRows, a.group - g0);
    if (g0 > 0) __syncthreads();
    for (int g = threadIdx.x >> 5; g < rows; g += kEndWarps) {
      // From the row's parts, as the join has it (which runs beside this).
      const float2* ml = a.ml + (row0 + g0 + g) * a.slots;
      float M = kNoMax, L = 0.0f;
#pragma unroll 4
      for (int s = lane; s < a.slots; s += 32) M = fmaxf(M, ml[s].x);
#pragma unroll
      for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
#pragma unroll 4
      for (int s = lane; s < a.slots; s += 32) {
        const float2 p = ml[s];
        L += p.y == 0.0f ? 0.0f : p.y * ex2_approx(p.x - M);
      }
#pragma unroll
      for (int x = 16; x; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
      if (lane == 0) row_ml[g] = make_float2(M, 1.0f / L);
    }
    __syncthreads();
    for (int g = 0; g < rows; ++g) {
      const float2 ml = row_ml[g];
#pragma unroll
      for (int x = 0; x < kWeighFours; ++x) {
        if (!at[x]) continue;
        w[x][0] = fmaf(ex2_approx(z[x].x - ml.x), ml.y, w[x][0]);
        w[x][1] = fmaf(ex2_approx(z[x].y - ml.x), ml.y, w[x][1]);
        w[x][2] = fmaf(ex2_approx(z[x].z - ml.x), ml.y, w[x][2]);
        w[x][3] = fmaf(ex2_approx(z[x].w - ml.x), ml.y, w[x][3]);
      }
      if (g0 + g + 1 < a.group) load(g0 + g + 1);
    }
  }
#pragma unroll
  for (int x = 0; x < kWeighFours; ++x) {
    if (!at[x]) continue;
    const float o[4] = {old[x].x, old[x].y, old[x].z, old[x].w};
    const int left = len - (j0 + 4 * kEndThreads * x);
#pragma unroll
    for (int y = 0; y < 4; ++y) w[x][y] = fmaf(a.decay, o[y], w[x][y]);
    if (left >= 4) {
      *reinterpret_cast<float4*>(at[x]) = make_float4(w[x][0], w[x][1], w[x][2], w[x][3]);
    } else {
#pragma unroll
      for (int y = 0; y < 3; ++y)
        if (y < left) at[x][y] = w[x][y];
    }
  }
}

// The end of a call: blocks that join rows and, with weights, behind them blocks that add to them; both
// need nothing but the parts.
template <int kWarpsRow, int kEndWarps>
__global__ void __launch_bounds__(32 * kEndWarps) bam_shared_end_kernel(const SharedArgs a, unsigned joins) {
  // (every sequence and key head has `joins` of the joining blocks)
  if (blockIdx.x < joins)
    join_rows<kWarpsRow, kEndWarps>(a, (static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y) * joins + blockIdx.x);
  else
    weigh_keys<kEndWarps>(a, blockIdx.x - joins);
}

}  // namespace

// Parts of up to `most` keys of each of `rows` item rows: two items a warp, or up to six of 512
// keys and more, so that the last ones end alike.
constexpr int kItemsFew = 2, kItemsMany = 6, kItemKeys = 512;
static int split_keys(int64_t rows, int64_t most) {
  const int64_t warps = 152 * kResident * kWarps;
  const int64_t few = (kItemsFew * warps + rows - 1) / rows, many = (kItemsMany * warps + rows - 1) / rows;
  int64_t n = most / kItemKeys > few ? most / kItemKeys : few;
  if (n > many) n = many;
  const int64_t cap = (most + kLeastKeys - 1) / kLeastKeys;
  return static_cast<int>(n < cap ? n : cap);
}

void shared_split(SharedArgs* a, int64_t Pmax, int64_t Tmax) {
  const int blocks = (a->group + kRows - 1) / kRows;
  a->nsplit = split_keys(static_cast<int64_t>(a->c.B) * a->c.Hkv * blocks, Tmax);
  a->npsplit = a->copies = a->tab_len = a->spills = 0;
  if (Pmax > 0) {
    if (static_cast<int64_t>(a->c.B) * a->group <= kFewRows)
      a->npsplit = split_keys(a->c.Hkv, Pmax);
    else
      prefix_split(a, Pmax, Tmax);
  }
  a->slots = a->nsplit + a->npsplit;
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
  const size_t smem = sizeof(SharedSmem<kTwo>) + 1024;
  static bool limit_set[64] = {};
  const cudaError_t e = smem_limit_once(bam_shared_kernel<kTwo, kParts>, smem, limit_set);
  if (e != cudaSuccess) return e;
  int64_t ctas = (items + kWarps - 1) / kWarps;
  const int64_t most = static_cast<int64_t>(sm_count()) * kResident;
  if (ctas > most) ctas = most;
  return launch_k(bam_shared_kernel<kTwo, kParts>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads),
                  smem, st, true, tk, tv, a);
}

cudaError_t launch_shared(const CUtensorMap& tk, const CUtensorMap& tv, const SharedArgs& a,
                          cudaStream_t st) {
  const int blocks = (a.group + kRows - 1) / kRows;
  const bool few = a.npsplit && a.copies == 0;
  const int64_t items = static_cast<int64_t>(a.nsplit) * a.c.B * a.c.Hkv * blocks +
                        (few ? static_cast<int64_t>(a.npsplit) * a.c.Hkv : 0);
  if (items > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const bool two = a.group > 8;
  if (a.o_fp32)
    return two ? launch_main<true, 3>(tk, tv, a, items, st) : launch_main<false, 3>(tk, tv, a, items, st);
  return two ? launch_main<true, 2>(tk, tv, a, items, st) : launch_main<false, 2>(tk, tv, a, items, st);
}

cudaError_t launch_shared_end(const SharedArgs& a, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.c.B) * a.H, heads = a.z ? static_cast<int64_t>(a.c.B) * a.c.Hkv : 1;
  auto launch = [&](auto* kernel, int warps, int block) {  // of a row, of a block
    const int64_t blocks = (rows * warps + block - 1) / block, joins = (blocks + heads - 1) / heads;
    const int64_t tiles = a.z ? (a.zstride + weigh_keys_of(block) - 1) / weigh_keys_of(block) : 0;
    const dim3 grid(static_cast<unsigned>(joins + tiles), a.z ? a.c.Hkv : 1, a.z ? a.c.B : 1);
    return launch_k(kernel, grid, dim3(32 * block), 0, st, true, a, static_cast<unsigned>(joins));
  };
  // (8192 rows of 7 parts: 7 us by a warp each, 12 by four; 768 rows of 55: 10 and 7)
  if (a.slots <= 4 || (a.slots <= 16 && rows > 2048)) return launch(bam_shared_end_kernel<1, 8>, 1, 8);
  if (a.slots <= 64) return launch(bam_shared_end_kernel<4, 8>, 4, 8);
  // (96 rows of 8192 keys in 129 parts: 15.2 us with eight warps a row, 16.8 with 32; of 65536 in some
  // hundred: 57 and 54)
  if (a.slots <= 192) return launch(bam_shared_end_kernel<8, 8>, 8, 8);
  return launch(bam_shared_end_kernel<32, 32>, 32, 32);
}

}  // namespace bam
