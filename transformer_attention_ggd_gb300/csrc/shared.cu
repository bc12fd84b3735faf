// Decode over a paged cache whose first keys a whole batch shares and whose own
// keys may carry positions and accumulated weights, on sm_103a.
#include "shared_common.cuh"
#include "table_eval.cuh"

namespace bam {
namespace {

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
static_assert(sizeof(DevStatus) <= 128 && kStatusBytes >= 256, "place of the item counter");

constexpr int kPrepThreads = 256;

// Starts the call and fills the table, if there is one, up to the largest distance.
__global__ void __launch_bounds__(kPrepThreads) bam_shared_prep_kernel(const SharedArgs a) {
  __shared__ int most;  // position of any query, at most
  grid_dep_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    status_begin_call(a.c.status);
    *item_counter(a.c.status) = 0;
  }
  if (!a.table) return;
  bool ok = true;
  const int P = prefix_len(a, &ok);
  if (threadIdx.x == 0) most = -1;
  __syncthreads();
  int hi = -1;
  for (int b = threadIdx.x; b < a.c.B; b += kPrepThreads) hi = max(hi, query_pos(a, b, P, &ok));
  atomicMax(&most, hi);
  __syncthreads();
  const int h = blockIdx.y, copies = a.copies ? kTabCopies : 1;
  const float alpha = a.alpha[h], beta = a.beta[h], mu = a.mu[h];
  for (int d = blockIdx.x * kPrepThreads + threadIdx.x; d <= most; d += gridDim.x * kPrepThreads) {
    float b, g1, g2;
    bias_terms<false>(d, alpha, beta, mu, a.eps, a.prior, &b, &g1, &g2);
    b = to_f32_finite(b * static_cast<float>(kLog2e));
    for (int k = 0; k < copies; ++k)
      a.table[(static_cast<int64_t>(k) * a.H + h) * a.tab_len + (a.tab_top - d) + k] = b;
  }
}

// An item: up to 16 rows (the heads of one sequence that share a key head, or all rows of a
// few over the prefix) and one part of their keys.
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
// a CTA: items of a few hundred keys, whose start a CTA of its own each paid for, took 24 instead of
// XX us (64 sequences of up to 512 keys, 12 heads).  kTwo: more than 8 rows.  kParts: bf16 parts of
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
    float alpha = 1.0f, beta = 0.0f, mu = 0.0f, scale = 0.0f;
    int pos = 0, row = -1;
    if (lane < cur.nrows) {
      int b, h;
      row = item_row(a, cur, lane, &b, &h);
      pos = query_pos(a, b, cur.P, &ok_arg);
      alpha = __ldg(a.alpha + h);
      beta = __ldg(a.beta + h);
      mu = __ldg(a.mu + h);
      scale = shared_scale(a, h, pos);
    }
    const bool tile_marked = marked && !cur.prefix;
    uint32_t qf[4][4];
    float c[2];
    float* zrow[2];
    const float* brow[2];
    int rpos[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = __shfl_sync(0xffffffffu, row, rq + 8 * x);
      c[x] = __shfl_sync(0xffffffffu, scale, rq + 8 * x);
      zrow[x] = tile_marked && r >= 0 ? a.z + r * a.zstride : nullptr;
      rpos[x] = __shfl_sync(0xffffffffu, pos, rq + 8 * x);
      brow[x] = a.table && r >= 0 ? a.table + static_cast<int64_t>(r % a.H) * a.tab_len + (a.tab_top - rpos[x])
                                  : nullptr;
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
      // The bias.  Out of the table: each lane that of its logits.  Else it is evaluated, a key a
      // lane and rows in turn, and handed over in shared memory.
      const int kfirst = (cur.prefix ? 0 : cur.P) + kb;  // position of the tile's first key, without marks
      if (!a.table) {
        const int kp = tile_marked ? sm.kpos[warp][s][lane] : kfirst + lane;
#pragma unroll 2
        for (int r = 0; r < cur.nrows; ++r) {
          int d = __shfl_sync(0xffffffffu, pos, r) - kp;
          if (d < 0) {
            bad_pos |= lane < valid;
            d = 0;
          }
          float bb, g1, g2;
          bias_terms<false>(d, __shfl_sync(0xffffffffu, alpha, r), __shfl_sync(0xffffffffu, beta, r),
                            __shfl_sync(0xffffffffu, mu, r), a.eps, a.prior, &bb, &g1, &g2);
          sm.bias[warp][r][lane] = to_f32_finite(bb * static_cast<float>(kLog2e));
        }
        __syncwarp();
      }
      float2 bias[kTwo ? 2 : 1][4];
#pragma unroll
      for (int x = 0; x < (kTwo ? 2 : 1); ++x) {
#pragma unroll
        for (int oc = 0; oc < 4; ++oc) {
          float2 bi = make_float2(0.0f, 0.0f);
          if (!a.table) {
            bi = *reinterpret_cast<const float2*>(&sm.bias[warp][rq + 8 * x][8 * oc + cq]);
          } else if (brow[x]) {
            // brow: this row's table at the query's position; a key's entry is its position further.
            int k0 = kfirst + 8 * oc + cq, k1 = k0 + 1;
            if (tile_marked) {
              const int2 kp = *reinterpret_cast<const int2*>(&sm.kpos[warp][s][8 * oc + cq]);
              k0 = max(min(kp.x, rpos[x]), 0);
              k1 = max(min(kp.y, rpos[x]), 0);
              bad_pos |= (kp.x > rpos[x] && 8 * oc + cq < valid) || (kp.y > rpos[x] && 8 * oc + cq + 1 < valid);
            }
            bi = make_float2(__ldg(brow[x] + k0), __ldg(brow[x] + k1));
          }
          bias[x][oc] = bi;
        }
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
          float z0 = fmaf(sacc[oc][2 * x], c[x], bias[x][oc].x);
          float z1 = fmaf(sacc[oc][2 * x + 1], c[x], bias[x][oc].y);
          if (8 * oc + cq >= valid) z0 = -INFINITY;
          if (8 * oc + cq + 1 >= valid) z1 = -INFINITY;
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
      // the weight is not, zero (an infinite value then stays one: no inf - inf, no 0 * inf).
      uint32_t pf[2][kParts][4];  // of 16 keys each
#pragma unroll
      for (int oc = 0; oc < 4; ++oc)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t(&w)[kParts][4] = pf[oc >> 1];
          float p0 = kTwo || x == 0 ? sacc[oc][2 * x] : 0.0f;
          float p1 = kTwo || x == 0 ? sacc[oc][2 * x + 1] : 0.0f;
          float least0 = p0 * 0x1p-28f, least1 = p1 * 0x1p-28f;
#pragma unroll
          for (int y = 0; y < kParts - 1; ++y) {
            const uint32_t w0 = __float_as_uint(p0), w1 = __float_as_uint(p1);
            w[y][2 * (oc & 1) + x] = __byte_perm(w0, w1, 0x7632);
            p0 = fmaxf(p0 - __uint_as_float(w0 & 0xFFFF0000u), least0);
            p1 = fmaxf(p1 - __uint_as_float(w1 & 0xFFFF0000u), least1);
            least0 *= 0x1p-8f;
            least1 *= 0x1p-8f;
          }
          w[kParts - 1][2 * (oc & 1) + x] = pack_bf16x2(p0, p1);
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
          float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int p = kParts - 1; p >= 0; --p)
#pragma unroll
            for (int h = 0; h < 2; ++h) mma_bf16(t, pf[h][p], vf[h][2 * y], vf[h][2 * y + 1]);
#pragma unroll
          for (int x = 0; x < 4; ++x) o[2 * dd + y][x] += t[x];
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

constexpr int kJoinThreads = 256;
constexpr int kJoinFew = 16;  // slots of a row, at most, that one warp joins

// Joins the parts of a row's keys: eight rows a block, a warp each, or one row.
template <int kWarpsRow>
__global__ void __launch_bounds__(kJoinThreads) bam_shared_join_kernel(const SharedArgs a) {
  constexpr int kRowsBlock = kJoinThreads / 32 / kWarpsRow;
  __shared__ float red_m[kJoinThreads / 32], red_l[kJoinThreads / 32];
  __shared__ float2 red_o[kJoinThreads / 32][32];
  grid_dep_wait();
  grid_dep_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % kWarpsRow;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsBlock + warp / kWarpsRow;
  if (row >= static_cast<int64_t>(a.c.B) * a.H) return;  // (whole blocks if a row has one)
  const int64_t base = row * a.slots;
  const bool aborted = *reinterpret_cast<volatile int*>(&a.c.status->abort) != 0;
  float M = kNoMax;
  for (int s = 32 * part + lane; s < a.slots; s += 32 * kWarpsRow) M = fmaxf(M, a.ml[base + s].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  if (kWarpsRow > 1) {
    if (lane == 0) red_m[warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarpsRow; ++w) M = fmaxf(M, red_m[w]);
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
    if (lane == 0) red_l[warp] = L;
    red_o[warp][lane] = make_float2(o0, o1);
    __syncthreads();
    if (warp) return;
    L = o0 = o1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarpsRow; ++w) {
      L += red_l[w];
      o0 += red_o[w][lane].x;
      o1 += red_o[w][lane].y;
    }
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

// Parts of up to `most` keys of each of `rows` item rows: two items a warp, or up to six of 512
// keys and more, so that the last ones end alike.
static int split_keys(int64_t rows, int64_t most) {
  const int64_t warps = 152 * kResident * kWarps;
  const int64_t two = (2 * warps + rows - 1) / rows, six = (6 * warps + rows - 1) / rows;
  int64_t n = most / 512 > two ? most / 512 : two;
  if (n > six) n = six;
  const int64_t cap = (most + kLeastKeys - 1) / kLeastKeys;
  return static_cast<int>(n < cap ? n : cap);
}

void shared_split(SharedArgs* a, int64_t Pmax, int64_t Tmax) {
  const int blocks = (a->group + kRows - 1) / kRows;
  a->nsplit = split_keys(static_cast<int64_t>(a->c.B) * a->c.Hkv * blocks, Tmax);
  a->npsplit = a->copies = 0;
  if (Pmax > 0) {
    if (static_cast<int64_t>(a->c.B) * a->group <= kFewRows)
      a->npsplit = split_keys(a->c.Hkv, Pmax);
    else
      prefix_split(a, Pmax);
  }
  a->slots = a->nsplit + a->npsplit * (a->copies > 1 ? a->copies : 1);
  // The table holds every distance below `top`, and room for windows that reach past the last
  // key.  Where it would hold more than a few keys have (one long sequence; positions far
  // beyond what a bounded cache holds), the bias of each key is evaluated instead: XX
  const int64_t reach = Pmax + Tmax;
  const int64_t top = a->max_pos > 0 ? (a->max_pos > Pmax ? a->max_pos : Pmax) : reach;
  a->use_table = a->copies || top <= 8192 || 4 * top <= a->c.B * reach;
  a->tab_top = static_cast<int>(top - 1);
  a->tab_len = static_cast<int>((top + 72 + 63) / 64 * 64);
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
  const bool two = a.group > 8 || (few && a.c.B * a.group > 8);
  if (a.o_fp32)
    return two ? launch_main<true, 3>(tk, tv, a, items, st) : launch_main<false, 3>(tk, tv, a, items, st);
  return two ? launch_main<true, 2>(tk, tv, a, items, st) : launch_main<false, 2>(tk, tv, a, items, st);
}

cudaError_t launch_shared_join(const SharedArgs& a, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.c.B) * a.H;
  constexpr int kWide = kJoinThreads / 32;
  if (a.slots <= kJoinFew)
    return launch_k(bam_shared_join_kernel<1>, dim3(static_cast<unsigned>((rows + kWide - 1) / kWide)),
                    dim3(kJoinThreads), 0, st, true, a);
  return launch_k(bam_shared_join_kernel<kWide>, dim3(static_cast<unsigned>(rows)), dim3(kJoinThreads), 0,
                  st, true, a);
}

cudaError_t launch_shared_weigh(const SharedArgs& a, cudaStream_t st) {
  const unsigned tiles = static_cast<unsigned>((a.zstride + kWeighKeys - 1) / kWeighKeys);
  return launch_k(bam_shared_weigh_kernel, dim3(tiles, a.c.Hkv, a.c.B), dim3(kWeighThreads), 0, st, true, a);
}

}  // namespace bam
