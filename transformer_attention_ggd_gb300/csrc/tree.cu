// Attention of a tree of drafted tokens over a paged cache, on sm_103a.
//
//   z[t, j] = c_t q_t . k_j + b_h(pos_t - pos_j),   o_t = softmax_j(z) V
//
// over the committed keys j < len (pos_j = j) and over node t's ancestors and
// itself (pos = len + depth).  All nodes and the query heads that share a key
// head read the same keys, so K and V are read once for all of them: 256
// bytes a key against 256 flops a row, that is one flop a byte and row.  Up to
// 128 rows the call is bound by HBM (the card's ridge is near 290).
//
// Work is cut into tiles of 64 keys and dealt out evenly: the plan kernel sums
// the tiles of all sequences, whose lengths only the device knows, and each
// CTA takes an equal run of them, across heads and sequences.  A (sequence,
// key head) that lies in one CTA is written by it; one that is cut leaves a
// partial maximum, sum and output per CTA, which the combine kernel joins.
// Ragged batches and a single long sequence keep every SM busy alike.
#include "table_eval.cuh"
#include "tree_common.cuh"

namespace bam {
namespace {

constexpr int kSoftWarps = 4;
constexpr int kTreeThreads = 32 * (kSoftWarps + 2);  // and the producer and the MMA issuer
constexpr int kRowsMax = 128;      // rows of an item: lanes of Tensor Memory
constexpr int kKvBytes = kTreeTile * kHeadDim * 2;  // 8 KB of K (and of V) a tile
constexpr int kQBytes = kRowsMax * kHeadDim * 2;
constexpr int kMergeStride = 68;  // floats of a merge row: 16-byte reads of 32 rows spread over the banks
constexpr int kNear = 32 + 2 * kTreeMax;  // a warp's table entries of the draft's distances
constexpr int kMaxStages = 8;
constexpr float kRescale = 8.0f;  // log2 units by which a weight may exceed 1
constexpr float kNoMax = -3.4e38f;  // below every logit (the table is clamped at -3e38)

// Tensor Memory columns of a CTA (256): S, the parts of P, O.
constexpr uint32_t kTmemCols = 256, kColP = 64, kColO = 192;

enum : int {
  kSiteTreeProducer = 60,
  kSiteTreeTable = 61,
  kSiteTreeMmaQ = 62,
  kSiteTreeMmaS = 63,
  kSiteTreeMmaK = 64,
  kSiteTreeMmaP = 65,
  kSiteTreeSoftS = 66,
  kSiteTreeSoftK = 67,
  kSiteTreeSoftPV = 68,
  kSiteTreeSoftEnd = 69,
  kSiteTreeMerge = 70
};

// Depths and ancestors of a sequence's nodes; every softmax warp has its own,
// so that the warps need no barrier among themselves.
struct TreeInfo {
  uint32_t seen[kTreeMax][kTreeMax / 32];  // a node's ancestors, and itself
  int jump[kTreeMax];
  int depth[kTreeMax];
  float near[kNear];  // [head of the warp's rows][distance < n]
};

struct __align__(16) TreeSmem {
  TreeInfo info[kSoftWarps];
  float4 merge_ml[kRowsMax];
  uint64_t full[kMaxStages];   // K, V and table windows of a stage have arrived
  uint64_t empty[kMaxStages];  // its P V is done
  uint64_t q_full;             // the item's queries are in shared memory
  uint64_t s_full, s_free;     // S is complete; S is in registers
  uint64_t p_full, pv_done;    // P is in Tensor Memory; P V is done
  uint64_t merge_full, merge_free;  // the item's parts are in shared memory; are read
  uint64_t mma_final;
  uint32_t odd[2][kTreeMax / 32];  // nodes whose value is not finite, by item parity
  uint32_t tmem_base;
  int abort_flag;
  int find;
};

// ---------------------------------------------------------------- plan and table

// Block (0, 0) starts the call and sums the sequences' tiles; the blocks
// together write the table of b_h(d) for the distances that occur.
__global__ void __launch_bounds__(256) bam_tree_prep_kernel(const TreeArgs a) {
  grid_dep_trigger();
  __shared__ int64_t sum[256];
  const CacheArgs& c = a.c;
  const int tid = threadIdx.x;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (tid == 0) {
      status_begin_call(c.status);
      a.plan[0] = 0;
    }
    __syncthreads();
    int64_t base = 0;
    bool ok = true;
    for (int b0 = 0; b0 < c.B; b0 += 256) {
      int64_t x = 0;
      if (b0 + tid < c.B) {
        int len, n;
        ok &= cache_lengths(c, b0 + tid, &len, &n);
        if (n > 0)
          x = static_cast<int64_t>(c.Hkv) * ((a.group * n + a.rows - 1) / a.rows) *
              ((len + n + kTreeTile - 1) / kTreeTile);
      }
      sum[tid] = x;
      __syncthreads();
      for (int off = 1; off < 256; off <<= 1) {
        const int64_t y = tid >= off ? sum[tid - off] : 0;
        __syncthreads();
        sum[tid] += y;
        __syncthreads();
      }
      if (b0 + tid < c.B) a.plan[b0 + tid + 1] = base + sum[tid];
      base += sum[255];
      __syncthreads();
    }
    if (!ok) record_bad_arg(c.status);
  }
  // Largest position of the batch: farther distances are not needed.
  int far = 0;
  for (int b = tid; b < c.B; b += 256) {
    int len, n;
    cache_lengths(c, b, &len, &n);
    far = max(far, len + n);
  }
  __shared__ int most;
  if (tid == 0) most = 0;
  __syncthreads();
  far = __reduce_max_sync(0xffffffffu, far);
  if ((tid & 31) == 0) atomicMax(&most, far);
  __syncthreads();
  const int d = blockIdx.x * 256 + tid;
  const int h = blockIdx.y;
  if (d > min(most, a.tab_zero)) return;
  float b, g1, g2;
  bias_terms<false>(d, a.alpha[h], a.beta[h], a.mu[h], a.eps, a.prior, &b, &g1, &g2);
  a.table[static_cast<size_t>(h) * a.tab_len + a.tab_zero - d] =
      to_f32_finite(b * static_cast<float>(kLog2e));
}

// ---------------------------------------------------------------- walking the plan

// CTAs that take part: each gets at least `least` tiles.
__device__ __forceinline__ int active_ctas(int64_t all, int ctas, int least) {
  const int64_t n = (all + least - 1) / least;
  return n < 1 ? 1 : n < ctas ? static_cast<int>(n) : ctas;
}
__device__ __forceinline__ int64_t range_beg(int64_t all, int active, int cta) {
  return all * cta / active;
}
// The CTA whose range holds tile x.
__device__ __forceinline__ int range_owner(int64_t all, int active, int64_t x) {
  return static_cast<int>(((x + 1) * active - 1) / all);
}

struct Item {
  int b, hk, rb;
  int len, n, tiles;
  int t0, t1;      // tiles of this CTA
  int64_t first;   // global index of the item's tile 0
};

// The item that tile x belongs to; `b` is a sequence at or before it.
__device__ __forceinline__ Item item_at(const TreeArgs& a, int b, int64_t x, int64_t end) {
  while (__ldcg(a.plan + b + 1) <= x) ++b;
  Item it;
  it.b = b;
  cache_lengths(a.c, b, &it.len, &it.n);
  it.tiles = (it.len + it.n + kTreeTile - 1) / kTreeTile;
  const int nrb = (a.group * it.n + a.rows - 1) / a.rows;
  const int64_t local = x - __ldcg(a.plan + b);
  const int idx = static_cast<int>(local / it.tiles);
  it.hk = idx / nrb;
  it.rb = idx - it.hk * nrb;
  it.t0 = static_cast<int>(local - static_cast<int64_t>(idx) * it.tiles);
  it.first = x - it.t0;
  it.t1 = static_cast<int>(min(static_cast<int64_t>(it.tiles), it.t0 + (end - x)));
  return it;
}

// Depth and ancestors of the n nodes of sequence b, by one warp (four nodes a
// lane).  Each round doubles the chains that the jump pointers span.  Returns
// false in a lane that met a parent outside [-1, i).
__device__ __forceinline__ bool tree_info(const CacheArgs& c, int b, int n, TreeInfo& ti) {
  constexpr int kPer = kTreeMax / 32;
  const int lane = threadIdx.x & 31;
  bool ok = true, more = false;
  __syncwarp();
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int i = 32 * x + lane;
    uint32_t w[kPer];
    int p = -1, d = 0;
#pragma unroll
    for (int y = 0; y < kPer; ++y) w[y] = x == y ? 1u << lane : 0u;
    if (!c.parents) {
      d = i;
#pragma unroll
      for (int y = 0; y < kPer; ++y) w[y] = x > y ? ~0u : x == y ? ~0u >> (31 - lane) : 0u;
    } else if (i < n) {
      p = __ldg(c.parents + static_cast<size_t>(b) * c.N + i);
      ok &= p >= -1 && p < i;
      if (p < -1 || p >= i) p = -1;
      d = p >= 0;
    }
    more |= p >= 0;
    ti.jump[i] = p;
    ti.depth[i] = d;
    *reinterpret_cast<uint4*>(ti.seen[i]) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  while (__any_sync(0xffffffffu, more)) {
    int p[kPer], dp[kPer];
    uint4 v[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int j = ti.jump[32 * x + lane];
      p[x] = -1;
      dp[x] = 0;
      v[x] = make_uint4(0, 0, 0, 0);
      if (j >= 0) {
        p[x] = ti.jump[j];
        dp[x] = ti.depth[j];
        v[x] = *reinterpret_cast<const uint4*>(ti.seen[j]);
      }
    }
    __syncwarp();
    more = false;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int i = 32 * x + lane;
      uint4* w = reinterpret_cast<uint4*>(ti.seen[i]);
      *w = make_uint4(w->x | v[x].x, w->y | v[x].y, w->z | v[x].z, w->w | v[x].w);
      ti.depth[i] += dp[x];
      ti.jump[i] = p[x];
      more |= p[x] >= 0;
    }
    __syncwarp();
  }
  return ok;
}

__device__ __forceinline__ bool odd_exp(uint32_t half) { return (half & 0x7F80u) == 0x7F80u; }

// Floats of one head's table window for a tile and n nodes: 64 keys against
// n positions at most, from a 16-byte boundary.
__host__ __device__ __forceinline__ int window_floats(int n) {
  return (3 + kTreeTile + n - 1 + 3) & ~3;
}

// Bytes of the query buffer, which also holds the copies' outputs at an
// item's end (24.5 KB for three copies of 32 rows, 17 KB for one of 64).
__host__ __device__ constexpr int q_bytes(int ks) {
  return ks == 1 ? kQBytes : ((kRowsMax - kRowsMax / ks) * kMergeStride * 4 + 1023) / 1024 * 1024;
}
static_assert(q_bytes(2) >= kQBytes && q_bytes(4) >= kQBytes, "queries");

// N columns (16, 32 or 64) of this warp's lanes of Tensor Memory.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t* r) {
  if constexpr (N == 16) {
    tmem_ld_32x32b_x16(taddr, r);
    tmem_ld_wait();
    reg_fence16(r);
  } else {
    tmem_ld_32x32b_x32(taddr, r);
    if (N == 64) tmem_ld_32x32b_x32(taddr + 32, r + 32);
    tmem_ld_wait();
    reg_fence32(r);
    if (N == 64) reg_fence32(r + 32);
  }
}

// D[tmem] (+)= A[tmem] * B[smem] for the 128 / KS lanes of one copy; the other
// lanes of D keep their values.
template <int KS>
__device__ __forceinline__ void umma_ts_lanes(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                              uint32_t idesc, uint32_t accumulate, int copy) {
  uint32_t off[4];  // a bit per lane: not written
#pragma unroll
  for (int x = 0; x < 4; ++x) off[x] = x / (4 / KS) == copy ? 0u : 0xFFFFFFFFu;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n}\n" ::"r"(
          d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate), "r"(off[0]), "r"(off[1]), "r"(off[2]),
      "r"(off[3])
      : "memory");
}

// ---------------------------------------------------------------- attention

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, DevStatus* st,
                                          volatile int* ab, int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, st, ab, site));
}

// Visibility of the 64 keys of a tile that starts at j0 to a node: committed
// keys, then the bits of its ancestors.
__device__ __forceinline__ uint64_t tile_mask(const uint32_t* seen, int j0, int len) {
  const uint64_t lo = static_cast<uint64_t>(seen[1]) << 32 | seen[0];
  const uint64_t hi = static_cast<uint64_t>(seen[3]) << 32 | seen[2];
  const int i = j0 - len;  // node of the tile's first key
  if (i <= 0) {
    const int k = -i;  // 0 .. 63 committed keys in the tile
    return k ? (lo << k) | ((1ull << k) - 1) : lo;
  }
  if (i >= 128) return 0;
  if (i >= 64) return hi >> (i - 64);
  return lo >> i | hi << (64 - i);
}

// One CTA walks its run of tiles; two CTAs share an SM, so that one's
// hand-offs are covered by the other's work.  Roles: four softmax warps, a
// producer warp (TMA loads of K and V, bulk copies of the table windows of
// the item's heads, into a ring), and a thread that issues the products:
//   S = Q K^T   128 x 64 x 64, Q and K from shared memory (K-major),
//   O += P V    128 x 64 x 64, P from Tensor Memory, V from shared memory.
// All 128 lanes are computed whatever the number of rows: at 64 keys a tile
// the two products take 256 cycles of an SM's tensor core, its share of HBM
// delivers the tile's 16 KB in about 700.  The next tile's S runs while the
// softmax works on this tile's.
//
// KS (1, 2, 4): an item of at most 128 / KS rows fills Tensor Memory KS times
// over, and each copy of a row works on its own 64 / KS keys of every tile,
// with its own maximum, sum and output, which are joined at the item's end.
// The products cost the same (a step of P V adds to the lanes of its keys'
// copy only), and the softmax, a thread per row and copy, takes a KS-th of
// the time.  The softmax needs no exchange between threads; O is rescaled
// only when a row's maximum grows by more than 8.
//
// PARTS: bf16 parts of a weight in the product with V.  With one, the sum
// that normalises is that of the rounded weights, so that the rounding of a
// weight that dominates its row cancels; three carry 24 bits.
template <int PARTS, int KS>
__global__ void __launch_bounds__(kTreeThreads, 2)
    bam_tree_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                    const TreeArgs a) {
  constexpr int nw = kSoftWarps;
  constexpr int kRows = kRowsMax / KS;   // rows of an item
  constexpr int kGroups = kRows / 32;    // warps of a copy
  constexpr int kCols = kTreeTile / KS;  // keys of a tile for one copy
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* const sq = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  float* const merge = reinterpret_cast<float*>(sq);  // [KS - 1][kRows][kMergeStride], after Q's use
  uint8_t* const kv = sq + q_bytes(KS);  // [stages][K, V]
  float* const win = reinterpret_cast<float*>(kv + a.stages * 2 * kKvBytes);
  TreeSmem& sm = *reinterpret_cast<TreeSmem*>(win + a.stages * a.win_stage);
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* ab = &sm.abort_flag;

  if (threadIdx.x == 0) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.q_full, nw);
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.s_free, nw);
    mbar_init(&sm.p_full, nw);
    mbar_init(&sm.pv_done, 1);
    mbar_init(&sm.merge_full, nw);
    mbar_init(&sm.merge_free, nw);
    mbar_init(&sm.mma_final, 1);
    fence_barrier_init();
    sm.find = 0;
  }
  if (warp == nw + 1) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  grid_dep_wait();  // plan and table
  grid_dep_trigger();
  if (threadIdx.x == 0) sm.abort_flag = *reinterpret_cast<volatile int*>(&c.status->abort);
  const int64_t all = __ldcg(a.plan + c.B);
  const int active = active_ctas(all, a.ctas, a.least);
  const int cta = blockIdx.x;
  int64_t beg = 0, end = 0;
  if (all > 0 && cta < active) {
    beg = range_beg(all, active, cta);
    end = range_beg(all, active, cta + 1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (beg < end) {
    int before = 0;
    for (int b = threadIdx.x; b < c.B; b += blockDim.x) before += __ldcg(a.plan + b + 1) <= beg;
    if (before) atomicAdd(&sm.find, before);
  }
  __syncthreads();
  const uint32_t tm = sm.tmem_base;
  int b = sm.find;

  if (warp == nw) {
    // ---------------------------------------------------------------- producer
    bool ok = *ab == 0, bad_page = false;
    int issued = 0, s = 0, phase = 1;
    for (int64_t x = beg; ok && x < end;) {
      const Item it = item_at(a, b, x, end);
      b = it.b;
      const int r0 = it.rb * kRows, r1 = min(r0 + kRows, a.group * it.n);
      const int g0 = r0 / it.n, heads = (r1 - 1) / it.n - g0 + 1;
      const int y0 = a.tab_zero - (it.len + it.n - 1);  // entry of key 0 for the last position
      const int nwin = window_floats(it.n);
      const float* trow = a.table + static_cast<size_t>(it.hk * a.group + g0) * a.tab_len;
      int pages = 0;
      for (int t = it.t0; t < it.t1; ++t) {
        const int ahead = (t - it.t0) & 31;
        if (ahead == 0 && t + lane < it.t1) {
          // page numbers of the next 32 tiles, one a lane
          pages = __ldg(c.block_table + static_cast<size_t>(it.b) * c.max_blocks +
                        (t + lane) * kTreeTile / c.page);
          if (pages < 0 || pages >= c.num_pages) {
            bad_page = true;
            pages = 0;
          }
        }
        const int pg = __shfl_sync(0xffffffffu, pages, ahead);
        if (issued >= a.stages) {
          ok = warp_wait(&sm.empty[s], phase, c.status, ab, kSiteTreeProducer);
          if (!ok) break;
        }
        uint8_t* dst = kv + s * 2 * kKvBytes;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.full[s], 2 * kKvBytes + heads * nwin * 4);
          const int row = t * kTreeTile % c.page, plane = pg * c.Hkv + it.hk;
          tma_load_3d(dst, &tk, &sm.full[s], 0, row, plane);
          tma_load_3d(dst + kKvBytes, &tv, &sm.full[s], 0, row, plane);
        }
        __syncwarp();
        for (int g = lane; g < heads; g += 32) {
          const float* tr = trow + static_cast<size_t>(g) * a.tab_len;
          ok &= bulk_load_checked(win + s * a.win_stage + g * nwin, tr + ((y0 + t * kTreeTile) & ~3),
                                  nwin * 4, &sm.full[s], tr, tr + a.tab_len, c.status, ab,
                                  kSiteTreeTable);
        }
        ++issued;
        if (++s == a.stages) {
          s = 0;
          phase ^= 1;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      x += it.t1 - it.t0;
    }
    // Copies in flight land before the CTA leaves.
    for (int i = max(0, issued - a.stages); i < issued; ++i)
      mbar_drain(&sm.full[i % a.stages], (i / a.stages) & 1);
    if (bad_page) record_bad_arg(c.status);
  } else if (warp == nw + 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t id_s = idesc_bf16(128, 64, false, false), id_o = idesc_bf16(128, 64, false, true);
      const uint64_t qd = sdesc_sw128(smem_u32(sq), 16, 1024);
      const uint64_t kd = sdesc_sw128(smem_u32(kv), 16, 1024);
      const uint64_t vd = sdesc_sw128(smem_u32(kv + kKvBytes), 16384, 1024);
      constexpr uint64_t kStageDesc = 2 * kKvBytes >> 4;
      bool ok = *ab == 0;
      int g = 0, item = 0;     // tiles and items so far
      int s = 0, phase = 0;    // ring slot of the tile whose S comes next
      auto issue_s = [&]() {
        if (g > 0) ok = ok && mbar_wait(&sm.s_free, (g - 1) & 1, c.status, ab, kSiteTreeMmaS);
        ok = ok && mbar_wait(&sm.full[s], phase, c.status, ab, kSiteTreeMmaK);
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ss(tm, qd + 2 * kk, kd + kStageDesc * s + 2 * kk, id_s, kk > 0 ? 1u : 0u);
        umma_commit(&sm.s_full);
        ++g;
        if (++s == a.stages) {
          s = 0;
          phase ^= 1;
        }
      };
      for (int64_t x = beg; ok && x < end; ++item) {
        const Item it = item_at(a, b, x, end);
        b = it.b;
        ok = mbar_wait(&sm.q_full, item & 1, c.status, ab, kSiteTreeMmaQ);
        if (!ok) break;
        issue_s();
        for (int t = it.t0; ok && t < it.t1; ++t) {
          const int sv = (s == 0 ? a.stages : s) - 1, gv = g - 1;  // this tile
          if (t + 1 < it.t1) issue_s();
          ok = ok && mbar_wait(&sm.p_full, gv & 1, c.status, ab, kSiteTreeMmaP);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int part = 0; part < PARTS; ++part)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              // 16 keys; they belong to copy kk / (4 / KS).
              constexpr int kSteps = 4 / KS;
              umma_ts_lanes<KS>(tm + kColO, tm + kColP + 32 * part + 8 * kk,
                                vd + kStageDesc * sv + 128 * kk, id_o,
                                (t > it.t0 || part > 0 || kk % kSteps > 0) ? 1u : 0u, kk / kSteps);
            }
          umma_commit(&sm.pv_done);
          umma_commit(&sm.empty[sv]);
        }
        x += it.t1 - it.t0;
      }
      umma_commit(&sm.mma_final);
      mbar_drain(&sm.mma_final, 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int rg = warp % kGroups, copy = warp / kGroups;
    const int k0 = copy * kCols;  // first key of this copy in a tile
    const uint32_t lanes = tm + tmem_lane_base(warp);
    const uint32_t tS = lanes + k0, tP = lanes + kColP + k0 / 2, tO = lanes + kColO;
    TreeInfo& ti = sm.info[warp];
    bool ok = *ab == 0, args_ok = true;
    int last_b = -1, g = 0, item = 0, s = 0, phase = 0;
    for (int64_t x = beg; ok && x < end; ++item) {
      const Item it = item_at(a, b, x, end);
      b = it.b;
      if (it.b != last_b) args_ok &= tree_info(c, it.b, it.n, ti);
      last_b = it.b;
      const int n = it.n, len = it.len;
      const int r0 = it.rb * kRows, r1 = min(r0 + kRows, a.group * n);
      const int rw = r0 + 32 * rg;  // first row of the warp
      const int g0 = r0 / n, nwin = window_floats(n);
      const int r = rw + lane;
      const bool live = r < r1, warp_live = rw < r1;
      const int hg = (live ? r : warp_live ? rw : r0) / n;
      const int node = live ? r - hg * n : 0;
      const int head = it.hk * a.group + hg, depth = ti.depth[node];
      float m = kNoMax, l = 0.0f, le = 0.0f;  // log2 units; sums of rounded and of exact weights
      float cs = 0.125f * static_cast<float>(kLog2e);
      if (a.ssmax) cs *= __ldg(a.s + head) * logf(static_cast<float>(len + depth + 1));
      const int woff = (hg - g0) * nwin + ((a.tab_zero - (len + n - 1)) & 3) + (n - 1 - depth) + k0;
      const size_t orow = (static_cast<size_t>(it.b) * a.H + head) * c.N + node;
      const float* near = ti.near + depth;  // table entry of an ancestor: near[-its depth]
      if (warp_live) {
        // This thread's query row, 16-byte chunks swizzled as the product
        // reads them.  The previous item's last S is done: its warps waited
        // for it.
        const uint4* src = reinterpret_cast<const uint4*>(a.q + orow * kHeadDim);
        uint4 w[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) w[y] = live ? __ldg(src + y) : make_uint4(0, 0, 0, 0);
        if (it.t1 * kTreeTile > len) {
          // Some tile holds drafted keys: their distances' table entries.
          const int h0 = rw / n;
          const int cnt = ((min(rw + 32, r1) - 1) / n - h0 + 1) * n;
          const float* tab = a.table + static_cast<size_t>(it.hk * a.group + h0) * a.tab_len + a.tab_zero;
          __syncwarp();
          for (int y = lane; y < cnt; y += 32)
            ti.near[y] = __ldcg(tab + static_cast<size_t>(y / n) * a.tab_len - y % n);
          near += (hg - h0) * n;
        }
#pragma unroll
        for (int y = 0; y < 8; ++y)
          *reinterpret_cast<uint4*>(sq + threadIdx.x * 128 + ((y ^ (threadIdx.x & 7)) << 4)) = w[y];
      }
      if (warp == 0 && lane < kTreeMax / 32) sm.odd[item & 1][lane] = 0;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full);

      for (int t = it.t0; ok && t < it.t1; ++t, ++g) {
        const int j0 = t * kTreeTile;
        const bool tail = j0 + kTreeTile > len;  // holds keys that not every row sees
        ok = warp_wait(&sm.s_full, g & 1, c.status, ab, kSiteTreeSoftS) &&
             warp_wait(&sm.full[s], phase, c.status, ab, kSiteTreeSoftK);
        if (!ok) break;
        tc_fence_after();
        const float* w = win + s * a.win_stage + woff;
        uint64_t z[kCols / 2];
        if (warp_live) {
          uint32_t sv[kCols];
          tmem_ld_cols<kCols>(tS, sv);
          const uint64_t c2 = f2_pack(cs, cs);
          if (!tail) {
#pragma unroll
            for (int y = 0; y < kCols / 2; ++y)
              z[y] = ffma2(f2_pack(__uint_as_float(sv[2 * y]), __uint_as_float(sv[2 * y + 1])), c2,
                           f2_pack(w[2 * y], w[2 * y + 1]));
          } else {
            const uint64_t vis = live ? tile_mask(ti.seen[node], j0, len) >> k0 : 0;
#pragma unroll
            for (int y = 0; y < kCols / 2; ++y) {
              float e[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int k = 2 * y + h, i = j0 + k0 + k - len;
                // Loads of keys out of sight stay in range and are not used.
                const int back = min(ti.depth[min(max(i, 0), kTreeMax - 1)], depth);
                const float bias = i < 0 ? w[k] : near[-back];
                const float v = fmaf(__uint_as_float(sv[k]), cs, bias);
                e[h] = vis >> k & 1 ? v : -INFINITY;
              }
              z[y] = f2_pack(e[0], e[1]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_free);

        if (tail && warp == 0) {
          // Rows of V behind the draft hold anything, and a drafted value that
          // is not finite must not meet the weight 0 of a row that does not
          // see it: zeros here.  The latter are added to O at the item's end.
          uint8_t* vt = kv + s * 2 * kKvBytes + kKvBytes;
          bool any = false;
#pragma unroll 4
          for (int y = 0; y < kKvBytes / 512; ++y) {
            const int chunk = 32 * y + lane, i = j0 + (chunk >> 3) - len;
            if (i < 0) continue;
            uint4* p = reinterpret_cast<uint4*>(vt + chunk * 16);
            uint4 v = *p;
            uint32_t* u = reinterpret_cast<uint32_t*>(&v);
            bool fix = i >= n;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t keep = i >= n ? 0u : 0xFFFFFFFFu;
              if (odd_exp(u[h])) keep &= 0xFFFF0000u;
              if (odd_exp(u[h] >> 16)) keep &= 0x0000FFFFu;
              fix |= keep != 0xFFFFFFFFu;
              if (i < n && keep != 0xFFFFFFFFu) atomicOr(&sm.odd[item & 1][i >> 5], 1u << (i & 31));
              u[h] &= keep;
            }
            if (fix) *p = v;
            any |= fix;
          }
          if (any) fence_proxy_async_smem();
          __syncwarp();
        }

        bool resc = false;
        float scale = 1.0f;
        if (warp_live) {
          float mq[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float lo, hi;
            f2_unpack(z[y], lo, hi);
            mq[y] = fmaxf(lo, hi);
          }
#pragma unroll
          for (int y = 4; y < kCols / 2; ++y) {
            float lo, hi;
            f2_unpack(z[y], lo, hi);
            mq[y & 3] = fmax3(mq[y & 3], lo, hi);
          }
          const float m_new = fmaxf(m, fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])));
          resc = m_new > m + kRescale;
          if (resc) {
            scale = ex2_approx(m - m_new);
            l *= scale;
            le *= scale;
            m = m_new;
          }
        }
        if (g > 0) {
          // The previous P V is done: P may be overwritten, O is at rest.
          ok = warp_wait(&sm.pv_done, (g - 1) & 1, c.status, ab, kSiteTreeSoftPV);
          if (!ok) break;
          tc_fence_after();
        }
        if (warp_live) {
          const uint64_t negm2 = f2_pack(-m, -m);
          float lr[4] = {0.f, 0.f, 0.f, 0.f};
          uint64_t le2[2] = {0ull, 0ull};
          constexpr int kBatch = kCols / 2 < 16 ? kCols / 2 : 16;
#pragma unroll
          for (int q = 0; q < kCols / 2 / kBatch; ++q) {
            uint32_t pk[PARTS][kBatch];
#pragma unroll
            for (int y = 0; y < kBatch; ++y) {
              float p0, p1;
              f2_unpack(fadd2(z[kBatch * q + y], negm2), p0, p1);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              le2[y & 1] = fadd2(le2[y & 1], f2_pack(p0, p1));
#pragma unroll
              for (int part = 0; part < PARTS; ++part) {
                const uint32_t u = pack_bf16x2(p0, p1);
                pk[part][y] = u;
                if (PARTS == 1) {
                  add_bf16x2_f32(u, lr[2 * (y & 1)], lr[2 * (y & 1) + 1]);
                } else {
                  p0 -= __uint_as_float(u << 16);
                  p1 -= __uint_as_float(u & 0xFFFF0000u);
                }
              }
            }
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
              if (kBatch == 16)
                tmem_st_32x32b_x16(tP + 32 * part + 16 * q, pk[part]);
              else
                tmem_st_32x32b_x8(tP + 32 * part, pk[part]);
            }
          }
          float b0, b1;
          f2_unpack(fadd2(le2[0], le2[1]), b0, b1);
          le += b0 + b1;
          l += (lr[0] + lr[1]) + (lr[2] + lr[3]);
          if (t > it.t0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll
            for (int hb = 0; hb < 2; ++hb) {
              uint32_t ov[32];
              tmem_ld_cols<32>(tO + 32 * hb, ov);
#pragma unroll
              for (int y = 0; y < 32; ++y) ov[y] = __float_as_uint(__uint_as_float(ov[y]) * scale);
              tmem_st_32x32b_x32(tO + 32 * hb, ov);
            }
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full);
        if (++s == a.stages) {
          s = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      ok = warp_wait(&sm.pv_done, (g - 1) & 1, c.status, ab, kSiteTreeSoftEnd);
      if (!ok) break;
      tc_fence_after();
      const float norm = PARTS == 1 ? l : le;
      float M = m, L = norm, LE = le, f[KS];  // joined over the copies
      f[0] = 1.0f;
      if (KS > 1) {
        // The other copies' outputs, maxima and sums go through the buffer of
        // Q, which the item's products no longer read.
        if (copy > 0) {
          if (warp_live) {
            const int mr = (copy - 1) * kRows + 32 * rg + lane;
            sm.merge_ml[mr] = make_float4(m, norm, le, 0.0f);
#pragma unroll
            for (int hb = 0; hb < 2; ++hb) {
              uint32_t ov[32];
              tmem_ld_cols<32>(tO + 32 * hb, ov);
#pragma unroll
              for (int y = 0; y < 8; ++y)
                *reinterpret_cast<uint4*>(merge + mr * kMergeStride + 32 * hb + 4 * y) =
                    make_uint4(ov[4 * y], ov[4 * y + 1], ov[4 * y + 2], ov[4 * y + 3]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.merge_full);
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.merge_full);
          ok = warp_wait(&sm.merge_full, item & 1, c.status, ab, kSiteTreeMerge);
          if (!ok) break;
          float4 ml[KS];
#pragma unroll
          for (int y = 1; y < KS; ++y) {
            ml[y] = sm.merge_ml[(y - 1) * kRows + 32 * rg + lane];
            M = fmaxf(M, ml[y].x);
          }
          f[0] = ex2_approx(m - M);
          L *= f[0];
          LE *= f[0];
#pragma unroll
          for (int y = 1; y < KS; ++y) {
            f[y] = ex2_approx(ml[y].x - M);
            L += ml[y].y * f[y];
            LE += ml[y].z * f[y];
          }
        }
      }
      if (copy == 0 && warp_live) {
        const bool whole = it.t0 == 0 && it.t1 == it.tiles;
        const uint32_t* odd = sm.odd[item & 1];
        const bool any_odd = (odd[0] | odd[1] | odd[2] | odd[3]) != 0;
        const size_t prow =
            static_cast<size_t>(2 * cta + (it.t0 == 0 ? 1 : 0)) * kRows + 32 * rg + lane;
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
          uint32_t ov[32];
          tmem_ld_cols<32>(tO + 32 * hb, ov);
          float* o = reinterpret_cast<float*>(ov);
          if (!live) continue;
          if (KS > 1) {
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] *= f[0];
#pragma unroll
            for (int cp = 1; cp < KS; ++cp) {
              const float4* src = reinterpret_cast<const float4*>(
                  merge + ((cp - 1) * kRows + 32 * rg + lane) * kMergeStride + 32 * hb);
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                const float4 v = src[y];
                o[4 * y] = fmaf(v.x, f[cp], o[4 * y]);
                o[4 * y + 1] = fmaf(v.y, f[cp], o[4 * y + 1]);
                o[4 * y + 2] = fmaf(v.z, f[cp], o[4 * y + 2]);
                o[4 * y + 3] = fmaf(v.w, f[cp], o[4 * y + 3]);
              }
            }
          }
          if (any_odd) {
            // Values that are not finite, for the nodes that see them.
            for (int i = 0; i < n; ++i) {
              if (!(odd[i >> 5] >> (i & 31) & 1) || !(ti.seen[node][i >> 5] >> (i & 31) & 1)) continue;
              const int slot = len + i;
              int pg = __ldg(c.block_table + static_cast<size_t>(it.b) * c.max_blocks + slot / c.page);
              if (pg < 0 || pg >= c.num_pages) pg = 0;
              const uint32_t* v = reinterpret_cast<const uint32_t*>(
                  a.v_pages +
                  ((static_cast<size_t>(pg) * c.Hkv + it.hk) * c.page + slot % c.page) * kHeadDim +
                  32 * hb);
#pragma unroll
              for (int y = 0; y < 16; ++y) {
                const uint32_t u = __ldg(v + y);
                if (odd_exp(u)) o[2 * y] += __uint_as_float(u << 16);
                if (odd_exp(u >> 16)) o[2 * y + 1] += __uint_as_float(u & 0xFFFF0000u);
              }
            }
          }
          if (!whole) {
            float4* dst = reinterpret_cast<float4*>(a.part + prow * kHeadDim + 32 * hb);
#pragma unroll
            for (int y = 0; y < 8; ++y)
              dst[y] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
          } else {
            const float inv = 1.0f / L;
            if (PARTS > 1) {
              float4* dst =
                  reinterpret_cast<float4*>(static_cast<float*>(a.o) + orow * kHeadDim + 32 * hb);
#pragma unroll
              for (int y = 0; y < 8; ++y)
                dst[y] = make_float4(o[4 * y] * inv, o[4 * y + 1] * inv, o[4 * y + 2] * inv,
                                     o[4 * y + 3] * inv);
            } else {
              uint4* dst =
                  reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + orow * kHeadDim + 32 * hb);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                float* e = o + 8 * y;
                dst[y] = make_uint4(pack_bf16x2(e[0] * inv, e[1] * inv),
                                    pack_bf16x2(e[2] * inv, e[3] * inv),
                                    pack_bf16x2(e[4] * inv, e[5] * inv),
                                    pack_bf16x2(e[6] * inv, e[7] * inv));
              }
            }
          }
        }
        if (live) {
          if (!whole)
            a.part_ml[prow] = make_float4(M, L, LE, 0.0f);
          else if (a.lse)
            a.lse[orow] = (M + log2f(LE)) * kLn2f;
        }
      }
      if (KS > 1) {
        // The next item's queries may overwrite the parts.
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.merge_free);
        ok = warp_wait(&sm.merge_free, item & 1, c.status, ab, kSiteTreeMerge);
      }
      // O has been read before the next item's products overwrite it: they
      // wait for its p_full, on which every warp arrives after this.
      tc_fence_before();
      x += it.t1 - it.t0;
    }
    if (!args_ok) record_bad_arg(c.status);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == nw + 1) {
    tc_fence_after();
    tmem_dealloc(tm, kTmemCols);
  }
}

// One warp per row (b, h, t): joins the parts of an item that was cut.
__global__ void __launch_bounds__(256) bam_tree_combine_kernel(const TreeArgs a) {
  grid_dep_wait();
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(c.B) * a.H * c.N;
  const int64_t all = __ldcg(a.plan + c.B);
  const int active = active_ctas(all, a.ctas, a.least);
  const bool gave_up = *reinterpret_cast<volatile int*>(&c.status->abort) != 0;
  for (int64_t row = blockIdx.x * 8ll + (threadIdx.x >> 5); row < rows; row += gridDim.x * 8ll) {
    const int t = static_cast<int>(row % c.N);
    const int h = static_cast<int>(row / c.N % a.H);
    const int b = static_cast<int>(row / c.N / a.H);
    int len, n;
    cache_lengths(c, b, &len, &n);
    if (t >= n) continue;
    float2 v;
    float lse;
    if (gave_up) {
      lse = __int_as_float(0x7fc00000);
      v = make_float2(lse, lse);
    } else {
      const int g = h % a.group, r = g * n + t, rb = r / a.rows;
      const int nrb = (a.group * n + a.rows - 1) / a.rows;
      const int tiles = (len + n + kTreeTile - 1) / kTreeTile;
      const int64_t first =
          __ldcg(a.plan + b) + static_cast<int64_t>(h / a.group * nrb + rb) * tiles;
      const int c0 = range_owner(all, active, first);
      const int c1 = range_owner(all, active, first + tiles - 1);
      if (c0 == c1) continue;
      const int rr = r - rb * a.rows;
      auto part_row = [&](int cta) {
        return static_cast<size_t>(2 * cta + (cta == c0 ? 1 : 0)) * a.rows + rr;
      };
      float M = kNoMax, L = 0.0f, LE = 0.0f;
      for (int x = c0 + lane; x <= c1; x += 32) M = fmaxf(M, __ldcg(a.part_ml + part_row(x)).x);
#pragma unroll
      for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      v = make_float2(0.0f, 0.0f);
#pragma unroll 4
      for (int x = c0; x <= c1; ++x) {
        const size_t pr = part_row(x);
        const float4 ml = __ldcg(a.part_ml + pr);
        const float2 y = __ldcg(reinterpret_cast<const float2*>(a.part + pr * kHeadDim) + lane);
        const float f = ex2_approx(ml.x - M);
        L += ml.y * f;
        LE += ml.z * f;
        v.x += y.x * f;
        v.y += y.y * f;
      }
      v.x /= L;
      v.y /= L;
      lse = (M + log2f(LE)) * kLn2f;
    }
    if (a.o_fp32)
      reinterpret_cast<float2*>(static_cast<float*>(a.o) + row * kHeadDim)[lane] = v;
    else
      reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + row * kHeadDim)[lane] =
          pack_bf16x2(v.x, v.y);
    if (a.lse && lane == 0) a.lse[row] = lse;
  }
}

constexpr size_t kSmemTwo = 113 * 1024;  // a CTA's share when two fit an SM
constexpr size_t kSmemOne = 227 * 1024;

// Shared memory of a CTA besides its ring stages, and of one stage.
size_t smem_fixed(const TreeArgs& a) {
  return 1024 + q_bytes(kRowsMax / a.rows) + sizeof(TreeSmem);
}
size_t smem_stage(const TreeArgs& a) {
  return 2 * kKvBytes + static_cast<size_t>(a.win_stage) * 4;
}

template <int PARTS, int KS>
cudaError_t launch_copies(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a,
                          cudaStream_t st) {
  static bool limit_set[64] = {};
  auto kernel = bam_tree_kernel<PARTS, KS>;
  const cudaError_t e = smem_limit_once(kernel, kSmemOne, limit_set);
  if (e != cudaSuccess) return e;
  return launch_k(kernel, dim3(a.ctas), dim3(kTreeThreads), smem_fixed(a) + a.stages * smem_stage(a),
                  st, true, tk, tv, a);
}

template <int PARTS>
cudaError_t launch_parts(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a,
                         cudaStream_t st) {
  switch (a.rows) {
    case 32:
      return launch_copies<PARTS, 4>(tk, tv, a, st);
    case 64:
      return launch_copies<PARTS, 2>(tk, tv, a, st);
    default:
      return launch_copies<PARTS, 1>(tk, tv, a, st);
  }
}

}  // namespace

// Ring and grid of the call, from its sizes.  Returns false when a stage does
// not fit (more heads share a key head than its windows have room for).
bool tree_config(TreeArgs* a, int sms) {
  // Most heads and floats that a stage's windows hold, over the node counts.
  a->win_stage = 0;
  for (int n = 1; n <= a->c.N; ++n) {
    int heads = (a->rows + n - 2) / n + 1;
    if (heads > a->group) heads = a->group;
    if (heads * window_floats(n) > a->win_stage) a->win_stage = heads * window_floats(n);
  }
  const size_t fixed = smem_fixed(*a), stage = smem_stage(*a);
  int per_sm = 2;
  size_t budget = kSmemTwo;
  if (fixed + 3 * stage > budget) {
    per_sm = 1;
    budget = kSmemOne;
  }
  a->stages = static_cast<int>((budget - fixed) / stage);
  if (a->stages > kMaxStages) a->stages = kMaxStages;
  a->ctas = per_sm * sms < kTreeCtas ? per_sm * sms : kTreeCtas;
  a->least = 1;
  return a->stages >= 2 && a->ctas >= 1;
}

cudaError_t launch_tree_prep(const TreeArgs& a, cudaStream_t st) {
  return launch_k(bam_tree_prep_kernel, dim3(a.tab_zero / 256 + 1, a.H), dim3(256), 0, st, false, a);
}

cudaError_t launch_tree(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a,
                        cudaStream_t st) {
  return a.o_fp32 ? launch_parts<3>(tk, tv, a, st) : launch_parts<1>(tk, tv, a, st);
}

cudaError_t launch_tree_combine(const TreeArgs& a, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.c.B) * a.H * a.c.N;
  const int64_t want = (rows + 7) / 8;
  const int grid = static_cast<int>(want < 152 * 8 ? want : 152 * 8);
  return launch_k(bam_tree_combine_kernel, dim3(grid), dim3(256), 0, st, true, a);
}

}  // namespace bam
