// Attention of a tree of drafted tokens over a paged cache, on sm_103a.
//
//   z[t, j] = c_t q_t . k_j + b_h(pos_t - pos_j),   o_t = softmax_j(z) V
//
// over the committed keys j < len (pos_j = j) and over node t's ancestors and
// itself (pos = len + depth).  All nodes and the query heads that share a key
// head read the same keys, so K and V are read once for all of them: 256
// bytes a key against 256 flops a row, that is one flop a byte and row.  Up to
// 128 rows the call is bound by HBM (the card's ridge is near 290), until the
// softmax is: 9 instructions a logit, two warps a scheduler.
//
// The bias depends on the distance alone.  A table per head holds it, and a
// row reads its keys' entries from a window of the table that is staged with
// the keys.
//
// Work is cut into tiles of 64 or 128 keys and dealt out evenly: the plan
// kernel sums the tiles of all sequences, whose lengths only the device knows,
// and each CTA takes an equal run of them, across heads and sequences.  A
// (sequence, key head) that lies in one CTA is written by it; one that is cut
// leaves a partial maximum, sum and output per CTA, which the combine kernel
// joins.  Ragged batches and a single long sequence keep every SM busy alike.
//
// Measured (HBM copy 6.70 TB/s, L2 129 MB; a call with its three kernels, in a
// graph): 64 sequences of 32768 keys at most, 12 heads, 32 nodes 442 us (3.2 GB,
// 7.3 TB/s with what L2 keeps); 32 of 16384, 8 key heads, one node, 4 heads a
// key head 101 us (537 MB); one of 131072, 12 heads, 64 nodes 87 us (403 MB); 4
// of 20000, 12 heads, 128 nodes 72 us (249 MB); one of 500, 7 nodes 13.4 us.
// fp32 output: 8 of 4096, 16 nodes 29 us (51 MB); 131 and 102 us for the third
// and the fourth.
#include "table_eval.cuh"
#include "tree_common.cuh"

namespace bam {
namespace {

constexpr int kSoftWarps = 4;
constexpr int kTreeThreads = 32 * (kSoftWarps + 2);  // and the producer and the MMA issuer
constexpr int kRowsMax = 128;      // rows of an item: lanes of Tensor Memory
constexpr int kBox = 64;                             // keys of a TMA box: pages are multiples of it
constexpr int kBoxBytes = kBox * kHeadDim * 2;
constexpr int kQBytes = kRowsMax * kHeadDim * 2;
constexpr int kMaxStages = 8;
constexpr float kRescale = 8.0f;  // log2 units by which a weight may exceed 1
constexpr float kNoMax = -3.4e38f;  // below every logit (the table is clamped at -3e38)

// Tensor Memory columns of a CTA: S, P, O.
constexpr uint32_t kTmemCols = 256, kColO = 192;

enum : int {
  kSiteTreeProducer = 60,
  kSiteTreeItem = 61,
  kSiteTreeTable = 62,
  kSiteTreeMmaItem = 63,
  kSiteTreeMmaS = 64,
  kSiteTreeMmaK = 65,
  kSiteTreeMmaP = 66,
  kSiteTreeSoftItem = 67,
  kSiteTreeSoftS = 68,
  kSiteTreeSoftK = 69,
  kSiteTreeSoftPV = 70,
  kSiteTreeSoftEnd = 71,
  kSiteTreeMerge = 72
};

// One CTA's share of an item: rows r0 .. r1 - 1 of sequence b and key head
// hk against tiles t0 .. t1 - 1 of its len + n keys.
struct Item {
  int b, hk, r0, r1, g0;  // g0: head of row r0
  int len, n;
  int t0, t1, tiles;  // t1 == 0: no more items
  int tree;           // which of the two TreeInfo buffers
};

// Ancestors of a sequence's nodes (a bit each, the node itself among them)
// and their depths.
struct TreeInfo {
  uint4* seen;
  int* depth;
};

// What the producer prepares of an item besides its queries.
struct ItemInfo {
  Item* it;
  float* s;     // the Scalable-Softmax factor of each of its heads
  float* near;  // [head of the item's][distance < n] table entries
};

struct __align__(16) TreeSmem {
  Item item[2];
  uint64_t k_full[kMaxStages];   // a slot's K and table windows have arrived
  uint64_t v_full[kMaxStages];   // its V has
  uint64_t s_free[kMaxStages];   // its S and its windows are in registers
  uint64_t v_empty[kMaxStages];  // its P V is done
  uint64_t item_full[2];       // an item's queries and info are in shared memory
  uint64_t item_empty[2];      // the softmax warps are done with them
  uint64_t s_full;             // S is complete
  uint64_t p_full, pv_done;    // P is in Tensor Memory; P V is done
  uint64_t merge[2];           // what two copies, then two pairs, exchange is there
  uint64_t mma_final;
  uint32_t odd[2][kTreeMax / 32];  // nodes whose value is not finite, by item parity
  uint32_t tmem_base;
  int abort_flag;
};

// ---------------------------------------------------------------- plan and table

// Units of an item: its fixed cost, then one for a tile of committed keys and
// tail_cost for one that holds drafted keys.  A tile belongs to the CTA that
// its last unit is dealt to.
__device__ __forceinline__ int item_units(int tile, int tail_cost, int len, int n) {
  const int tiles = (len + n + tile - 1) / tile;
  return kItemCost + tiles + (tail_cost - 1) * (tiles - len / tile);
}
// Tiles of an item that end at or before its unit `at`; `plain` of them hold
// committed keys alone.
__device__ __forceinline__ int tiles_before(int tail_cost, int plain, int at) {
  const int y = at - kItemCost;
  return y <= 0 ? 0 : y <= plain ? y : plain + (y - plain) / tail_cost;
}

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
              item_units(a.tile, a.tail_cost, len, n);
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
  const int far_d = min(most, a.tab_zero);  // farthest distance
  for (int h = blockIdx.y; h < a.H; h += gridDim.y) {
    const float al = __ldg(a.alpha + h), be = __ldg(a.beta + h), mu = __ldg(a.mu + h);
    float* row = a.table + static_cast<size_t>(h) * a.tab_len + a.tab_zero;
    for (int d = blockIdx.x * 256 + tid; d <= far_d; d += gridDim.x * 256) {
      float b, g1, g2;
      bias_terms<false>(d, al, be, mu, a.eps, a.prior, &b, &g1, &g2);
      row[-d] = to_f32_finite(b * static_cast<float>(kLog2e));
    }
  }
}

// ---------------------------------------------------------------- walking the plan

// CTAs that take part: each gets two units or more, if there are as many, so that
// every CTA between the first and the last of an item gets one of its tiles.
static_assert(kTailCost <= 2, "a CTA could get no tile of an item between its first and last");
__device__ __forceinline__ int active_ctas(int64_t all, int ctas) {
  const int64_t n = all >> 1;
  return n < 1 ? 1 : n < ctas ? static_cast<int>(n) : ctas;
}
// (A 64-bit division is a hundred instructions; all * cta fits 32 bits in all
// but the largest calls.)
__device__ __forceinline__ int64_t range_beg(int64_t all, int active, int cta) {
  if (all < (1 << 22))
    return static_cast<uint32_t>(all) * static_cast<uint32_t>(cta) / static_cast<uint32_t>(active);
  return all * cta / active;
}
// The CTA whose range holds unit x.
__device__ __forceinline__ int range_owner(int64_t all, int active, int64_t x) {
  if (all < (1 << 22))
    return static_cast<int>((static_cast<uint32_t>(x + 1) * static_cast<uint32_t>(active) - 1) /
                            static_cast<uint32_t>(all));
  return static_cast<int>(((x + 1) * active - 1) / all);
}

constexpr int kPer = kTreeMax / 32;  // nodes of a lane

// This lane's parents: of nodes lane, lane + 32, ... (-1 behind node n - 1).
__device__ __forceinline__ void tree_parents(const CacheArgs& c, int b, int n, int* par) {
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int i = 32 * x + (threadIdx.x & 31);
    par[x] = c.parents && i < n ? __ldg(c.parents + static_cast<size_t>(b) * c.N + i) : -1;
  }
}
// Depth and ancestors of a sequence's nodes, by one warp, for `nodes` (a
// multiple of 32) entries.  Each round doubles the chains that the jump
// pointers span.  Returns false in a lane that met a parent outside [-1, i).
__device__ __forceinline__ bool tree_info(bool chain, const int* par, int nodes,
                                          const TreeInfo& ti, int* jump) {
  const int lane = threadIdx.x & 31;
  bool ok = true, more = false;
  __syncwarp();
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int i = 32 * x + lane;
    if (32 * x >= nodes) break;
    uint32_t w[kPer];
    int p = par[x], d;
#pragma unroll
    for (int y = 0; y < kPer; ++y) w[y] = x == y ? 1u << lane : 0u;
    if (chain) {
      d = i;
#pragma unroll
      for (int y = 0; y < kPer; ++y) w[y] = x > y ? ~0u : x == y ? ~0u >> (31 - lane) : 0u;
    } else {
      ok &= p >= -1 && p < i;
      if (p < -1 || p >= i) p = -1;
      d = p >= 0;
    }
    more |= p >= 0;
    jump[i] = p;
    ti.depth[i] = d;
    ti.seen[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  while (__any_sync(0xffffffffu, more)) {
    int p[kPer], dp[kPer];
    uint4 v[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      if (32 * x >= nodes) break;
      const int j = jump[32 * x + lane];
      p[x] = -1;
      dp[x] = 0;
      v[x] = make_uint4(0, 0, 0, 0);
      if (j >= 0) {
        p[x] = jump[j];
        dp[x] = ti.depth[j];
        v[x] = ti.seen[j];
      }
    }
    __syncwarp();
    more = false;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      if (32 * x >= nodes) break;
      const int i = 32 * x + lane;
      const uint4 w = ti.seen[i];
      ti.seen[i] = make_uint4(w.x | v[x].x, w.y | v[x].y, w.z | v[x].z, w.w | v[x].w);
      ti.depth[i] += dp[x];
      jump[i] = p[x];
      more |= p[x] >= 0;
    }
    __syncwarp();
  }
  return ok;
}
__device__ __forceinline__ bool tree_sees(const TreeInfo& ti, int node, int i) {
  return reinterpret_cast<const uint32_t*>(ti.seen + node)[i >> 5] >> (i & 31) & 1;
}

__device__ __forceinline__ bool odd_exp(uint32_t half) { return (half & 0x7F80u) == 0x7F80u; }

// Floats of one head's table window for a tile and n nodes: its keys against
// n positions at most, from a 16-byte boundary.
__host__ __device__ __forceinline__ int window_floats(int tile, int n) {
  return (3 + tile + n - 1 + 3) & ~3;
}

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

// True when phase `parity` is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// As mbar_wait, without its call: the slow path of a call would keep the
// caller's live registers (a row of S, here) in local memory.
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, DevStatus* st,
                                          volatile int* ab, int site) {
#ifdef BAM_DEBUG
  if (*reinterpret_cast<volatile int*>(&st->giveup) > 0 && atomicSub(&st->giveup, 1) == 1) {
    raise_abort(st, ab, site);
    return false;
  }
#endif
  if (mbar_test(bar, parity)) return true;
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t it = 1; !mbar_try_wait_sleep(bar, parity, kWaitSleepNs); ++it) {
    if ((it & 3u) != 0) continue;
    if (*ab) return false;
    if (*reinterpret_cast<volatile int*>(&st->abort)) {
      *ab = 1;
      return false;
    }
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitLimitNs) {
      raise_abort(st, ab, site);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, DevStatus* st,
                                          volatile int* ab, int site) {
  return __all_sync(0xffffffffu, tree_wait(bar, parity, st, ab, site));
}

// Visibility of the 64 keys from j0 on to a node: committed keys, then the
// bits of its ancestors.
__device__ __forceinline__ uint64_t tile_mask(uint4 seen, int j0, int len) {
  const uint64_t lo = static_cast<uint64_t>(seen.y) << 32 | seen.x;
  const uint64_t hi = static_cast<uint64_t>(seen.w) << 32 | seen.z;
  const int i = j0 - len;  // node of the tile's first key
  if (i <= 0) {
    const int k = -i;  // committed keys among them
    return k >= 64 ? ~0ull : k ? (lo << k) | ((1ull << k) - 1) : lo;
  }
  if (i >= 128) return 0;
  if (i >= 64) return hi >> (i - 64);
  return lo >> i | hi << (64 - i);
}

// 16 bytes global -> shared, or zeros, asynchronously.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Keys of a tile: as many as S and the parts of P leave Tensor Memory for, and no
// more than 64 columns a thread.  128 against 64 keys where both fit, a call:
// 442 and 463 us with 64 sequences of 32768 keys and 32 rows, 87 and 88 with 64
// rows and 131072 keys, 50 and 59 with 8 rows and 100 keys, 101 and 103 with 4
// rows and 16384; 13.4 and 12.6 with 7 rows and one sequence of 500.
__host__ __device__ constexpr int tree_tile(int parts, int ks) {
  return parts == 1 && ks > 1 ? 128 : 64;
}

// A tile with drafted keys keeps its logits in registers where they are few;
// else they go back to Tensor Memory between the maximum and the weights.
__host__ __device__ constexpr bool tree_once(int parts, int ks) {
  return tree_tile(parts, ks) / ks * parts <= 48;
}
__host__ __device__ constexpr int tree_tail_cost(int parts, int ks) {
  return tree_once(parts, ks) ? 1 : kTailCost;
}

// The tensor core cuts off the last place of O in every step of a product (16
// keys, a part of their weights), toward zero, so that over thousands of steps
// the sum falls short: with positive values of like weight, 304 sequences, by
// 4e-4 after 512 tiles of three parts and 6e-3 after 16384 tiles of one.  After a
// run of tiles O is therefore added to a sum in fp32 outside of Tensor Memory.
// Tiles of a run for each copy, that is 96 steps or 256 to 512: what is lost is then
// below 1e-5 and 3e-5 (bf16 output rounds by 2^-9 to 2^-8).  Runs of 4, 8 and 16 and no end
// of a run took 139, 131, 128 and 121 us with three parts (131072 keys, 64 nodes); with
// one part 64 and 16 took 442 and 461 (64 sequences of 32768 keys), 71.7 and 79.0 (4
// chains of 128 nodes, 20000 keys).
constexpr int kRunParts = 8, kRunOne = 64;

// Sizes of a kernel with PARTS parts of a weight and KS copies of a row.
template <int PARTS, int KS>
struct Shape {
  static constexpr int kRows = kRowsMax / KS;        // rows of an item
  static constexpr int kGroups = kRows / 32;         // warps of a copy
  static constexpr int kTile = tree_tile(PARTS, KS);  // keys of a tile
  static constexpr int kCols = kTile / KS;           // of which one copy's
  static constexpr bool kOnce = tree_once(PARTS, KS);
  static constexpr int kTailCost = tree_tail_cost(PARTS, KS);
  static constexpr int kTileBytes = kTile * kHeadDim * 2;
  static constexpr int kPCols = kTile / 2;           // columns of a part of P
  static constexpr int kRun = (PARTS > 1 ? kRunParts : kRunOne) * KS;
  static constexpr uint32_t kColP = kTile;
  static_assert(kColP + kPCols * PARTS <= kColO, "Tensor Memory");
  static_assert((kRun & (kRun - 1)) == 0 && kRun > kTreeMax / kTile + 1, "a tail lies in one run");
};

// The CTA's shared memory.  What grows with the nodes of a draft is laid out
// for the call's N, so that small drafts leave room for the ring.
extern __shared__ __align__(16) uint8_t tree_smem_raw[];
struct View {
  uint8_t* sq;  // two query tiles
  uint8_t* sk;  // [stages] tiles of K
  uint8_t* sv;  // [stages] tiles of V
  float* win;   // [stages] table windows
  TreeSmem* sm;
  uint8_t* nodes;   // TreeInfo [2], jump
  float* near;      // [2][near]
  float* s;         // [2][kRows]
  float2* merge_ml; // [kRowsMax]
};
template <class S>
__device__ __forceinline__ View smem_view(const TreeArgs& a) {
  View v;
  v.sq = tree_smem_raw + ((0u - smem_u32(tree_smem_raw)) & 1023u);
  v.sk = v.sq + 2 * kQBytes;
  v.sv = v.sk + a.stages * S::kTileBytes;
  v.win = reinterpret_cast<float*>(v.sv + a.stages * S::kTileBytes);
  v.sm = reinterpret_cast<TreeSmem*>(v.win + a.stages * a.win_stage);
  v.nodes = reinterpret_cast<uint8_t*>(v.sm + 1);
  v.near = reinterpret_cast<float*>(v.nodes + a.nodes * 44);
  v.s = v.near + 2 * a.near;
  v.merge_ml = reinterpret_cast<float2*>(v.s + 2 * S::kRows);
  return v;
}
__device__ __forceinline__ TreeInfo tree_view(const TreeArgs& a, const View& v, int which) {
  return TreeInfo{reinterpret_cast<uint4*>(v.nodes) + which * a.nodes,
                  reinterpret_cast<int*>(v.nodes + 32 * a.nodes) + which * a.nodes};
}
__device__ __forceinline__ int* jump_view(const TreeArgs& a, const View& v) {
  return reinterpret_cast<int*>(v.nodes + 40 * a.nodes);
}
template <class S>
__device__ __forceinline__ ItemInfo info_view(const TreeArgs& a, const View& v, int k) {
  const int x = k & 1;
  return ItemInfo{v.sm->item + x, v.s + x * S::kRows, v.near + x * a.near};
}

// What a softmax warp carries from tile to tile.
struct SoftState {
  int g, s, phase;  // tile of the CTA, its ring slot and phase
  int t;            // tile of the item
  float m, l;       // running maximum (log2 units) and sum of the weights
  bool first;       // the item's first tile
  bool ok;
};

// The sum of an item's tiles before the run in Tensor Memory: output, weights, and
// the maximum that they are relative to.  In local memory (the indexes vary), as
// a thread has no 64 registers left.
struct SoftSum {
  float o[64], l, m;
};

// A softmax thread's row of the item in buffer k & 1.
struct SoftRow {
  int rr, copy, k0;  // row of the item, copy, the copy's first key in a tile
  uint32_t lanes;    // the warp's lanes of Tensor Memory
  bool live, warp_live;
  int node, hrel, depth;  // hrel: head within the item
  float cs;          // logit scale, log2 units
  int woff;          // its place in a table window
};
template <class S>
__device__ __forceinline__ SoftRow soft_row(const TreeArgs& a, const View& v, int k) {
  const TreeSmem& sm = *v.sm;
  const ItemInfo info = info_view<S>(a, v, k);
  const Item& it = *info.it;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = it.n;
  SoftRow r;
  r.rr = 32 * (warp % S::kGroups) + lane;
  r.copy = warp / S::kGroups;
  r.k0 = r.copy * S::kCols;
  r.lanes = sm.tmem_base + tmem_lane_base(warp);
  r.warp_live = it.r0 + 32 * (warp % S::kGroups) < it.r1;
  r.live = it.r0 + r.rr < it.r1;
  const int head = r.live ? (it.r0 + r.rr) / n : it.g0;
  r.node = r.live ? it.r0 + r.rr - head * n : 0;
  r.hrel = head - it.g0;
  r.depth = tree_view(a, v, it.tree).depth[r.node];
  r.cs = 0.125f * static_cast<float>(kLog2e);
  if (a.ssmax) r.cs *= info.s[r.hrel] * logf(static_cast<float>(it.len + r.depth + 1));
  r.woff = r.hrel * window_floats(S::kTile, n) + ((a.tab_zero - (it.len + n - 1)) & 3) +
           (n - 1 - r.depth) + r.k0;
  return r;
}

// N / 2 columns of P (bf16 pairs) of this warp's lanes.
template <int N>
__device__ __forceinline__ void tmem_st_pairs(uint32_t taddr, const uint32_t* r) {
  if constexpr (N == 16)
    tmem_st_32x32b_x8(taddr, r);
  else
    tmem_st_32x32b_x16(taddr, r);
}

// The start of a tile: S and the windows are there.
__device__ __forceinline__ bool soft_begin(const TreeArgs& a, TreeSmem& sm, SoftState& st) {
  volatile int* ab = &sm.abort_flag;
  st.ok = __all_sync(0xffffffffu,
                     tree_wait(&sm.s_full, st.g & 1, a.c.status, ab, kSiteTreeSoftS) &&
                         tree_wait(&sm.k_full[st.s], st.phase, a.c.status, ab, kSiteTreeSoftK));
  if (st.ok) tc_fence_after();
  return st.ok;
}
__device__ __forceinline__ void soft_free_s(TreeSmem& sm, const SoftState& st) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.s_free[st.s]);
}
// Takes the tile's maximum mx into account and waits until the previous P V
// is done (P may then be overwritten, and O is at rest).  `scale`: what O has
// to be multiplied by.
__device__ __forceinline__ bool soft_max(const TreeArgs& a, TreeSmem& sm, const SoftRow& row,
                                         SoftState& st, float mx, float& scale) {
  volatile int* ab = &sm.abort_flag;
  scale = 1.0f;
  const float m_new = fmaxf(st.m, mx);
  if (row.warp_live && m_new > st.m + kRescale) {
    scale = ex2_approx(st.m - m_new);
    st.l *= scale;
    st.m = m_new;
  }
  if (st.g > 0) {
    st.ok = warp_wait(&sm.pv_done, (st.g - 1) & 1, a.c.status, ab, kSiteTreeSoftPV);
    if (st.ok) tc_fence_after();
  }
  return st.ok;
}
// The end of a tile: O scaled if need be, P complete.
__device__ __forceinline__ void soft_finish(const TreeArgs& a, TreeSmem& sm, const SoftRow& row,
                                            SoftState& st, float scale) {
  if (row.warp_live) {
    if (!st.first && __any_sync(0xffffffffu, scale != 1.0f)) {
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t ov[16];
        tmem_ld_cols<16>(row.lanes + kColO + 16 * q, ov);
#pragma unroll
        for (int y = 0; y < 16; ++y) ov[y] = __float_as_uint(__uint_as_float(ov[y]) * scale);
        tmem_st_32x32b_x16(row.lanes + kColO + 16 * q, ov);
      }
    }
    tmem_st_wait();
  }
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.p_full);
  if (++st.s == a.stages) {
    st.s = 0;
    st.phase ^= 1;
  }
  ++st.g;
  --st.t;
  st.first = false;
}
// Between two tiles, at the end of a run: adds O and l to the sum of the runs
// before (if `held`).  The next product overwrites O; it waits for the next
// tile's p_full.  kAhead, for short runs: what was held is on its way while the
// last product ends and while columns are added (131 against 136 us with three
// parts, 131072 keys and 64 nodes; with one part the code costs more than it saves).
template <bool kAhead>
__device__ __forceinline__ void soft_hold(const TreeArgs& a, TreeSmem& sm, const SoftRow& row,
                                          SoftState& st, SoftSum& sum, bool held) {
  constexpr int kCols = kAhead ? 32 : 16;
  float o[kCols];
  auto fetch = [&](int col) __attribute__((always_inline)) {
#pragma unroll
    for (int y = 0; y < kCols; ++y) o[y] = held ? sum.o[col + y] : 0.0f;
  };
  if (kAhead) fetch(0);
  st.ok = warp_wait(&sm.pv_done, (st.g - 1) & 1, a.c.status, &sm.abort_flag, kSiteTreeSoftPV);
  if (!st.ok) return;
  tc_fence_after();
  if (row.warp_live) {
    const float f = held ? ex2_approx(sum.m - st.m) : 0.0f;
#pragma unroll 1
    for (int col = 0; col < 64; col += kCols) {
      if (!kAhead) fetch(col);
      uint32_t ov[kCols];
      tmem_ld_cols<kCols>(row.lanes + kColO + col, ov);
#pragma unroll
      for (int y = 0; y < kCols; ++y)
        sum.o[col + y] = fmaf(o[y], f, __uint_as_float(ov[y]));
      if (kAhead) fetch((col + kCols) & 63);
    }
    sum.l = held ? fmaf(sum.l, f, st.l) : st.l;
    sum.m = st.m;
    st.l = 0.0f;
  }
  tc_fence_before();
}
// Two weights and their bf16 parts; l2 gathers the exact ones.  Three parts
// are cut off, not rounded: 8 bits each are the weight's 24, and none is
// negative.  None is less than 2^-26 of the weight (two such floors are half of
// its last place), so that an infinite value meets no zero that turns it into
// NaN; those of a weight of zero are zero, so that a key out of sight adds
// nothing, however large its value.
template <int PARTS, int N>
__device__ __forceinline__ void soft_weights(uint64_t z, uint64_t negm2, uint64_t& l2,
                                             uint32_t (*pk)[N], int y) {
  float p0, p1;
  f2_unpack(fadd2(z, negm2), p0, p1);
  p0 = ex2_approx(p0);
  p1 = ex2_approx(p1);
  l2 = fadd2(l2, f2_pack(p0, p1));
  if (PARTS == 1) {
    pk[0][y] = pack_bf16x2(p0, p1);
    return;
  }
  const float least0 = p0 * 0x1p-26f, least1 = p1 * 0x1p-26f;
#pragma unroll
  for (int part = 0; part < PARTS; ++part) {
    const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
    pk[part][y] = __byte_perm(u0, u1, 0x7632);
    p0 = fmaxf(p0 - __uint_as_float(u0 & 0xFFFF0000u), least0);
    p1 = fmaxf(p1 - __uint_as_float(u1 & 0xFFFF0000u), least1);
  }
}

// A tile of which every row sees every key.
template <int PARTS, int KS>
__device__ __forceinline__ void soft_tile(const TreeArgs& a, const View& v, const SoftRow& row,
                                          SoftState& st) {
  using S = Shape<PARTS, KS>;
  TreeSmem& sm = *v.sm;
  if (!soft_begin(a, sm, st)) return;
  uint64_t z[S::kCols / 2];
  float mx = kNoMax, scale;
  if (row.warp_live) {
    const float* w = v.win + st.s * a.win_stage + row.woff;
    uint32_t sv[S::kCols];
    tmem_ld_cols<S::kCols>(row.lanes + row.k0, sv);
    const uint64_t c2 = f2_pack(row.cs, row.cs);
#pragma unroll
    for (int y = 0; y < S::kCols / 2; ++y)
      z[y] = ffma2(f2_pack(__uint_as_float(sv[2 * y]), __uint_as_float(sv[2 * y + 1])), c2,
                   f2_pack(w[2 * y], w[2 * y + 1]));
  }
  soft_free_s(sm, st);
  if (row.warp_live) {
    float mq[4];
#pragma unroll
    for (int y = 0; y < S::kCols / 2; ++y) {
      float lo, hi;
      f2_unpack(z[y], lo, hi);
      mq[y & 3] = y < 4 ? fmaxf(lo, hi) : fmax3(mq[y & 3], lo, hi);
    }
    mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
  }
  if (!soft_max(a, sm, row, st, mx, scale)) return;
  if (row.warp_live) {
    const uint64_t negm2 = f2_pack(-st.m, -st.m);
    uint64_t l2[2] = {0ull, 0ull};
    constexpr int kBatch = S::kCols < 32 ? S::kCols / 2 : 16;  // column pairs
#pragma unroll
    for (int q = 0; q < S::kCols / 2 / kBatch; ++q) {
      uint32_t pk[PARTS][kBatch];
#pragma unroll
      for (int y = 0; y < kBatch; ++y)
        soft_weights<PARTS, kBatch>(z[kBatch * q + y], negm2, l2[y & 1], pk, y);
#pragma unroll
      for (int part = 0; part < PARTS; ++part)
        tmem_st_pairs<2 * kBatch>(row.lanes + S::kColP + row.k0 / 2 + S::kPCols * part + kBatch * q,
                                  pk[part]);
    }
    float b0, b1;
    f2_unpack(fadd2(l2[0], l2[1]), b0, b1);
    st.l += b0 + b1;
  }
  soft_finish(a, sm, row, st, scale);
}

// 16 logits of a tile with keys that not every row sees, from column kk on.
// nc: committed keys among the copy's columns (not clamped); the n nodes of
// the draft follow them.
__device__ __forceinline__ void tail_logits(uint32_t taddr, const SoftRow& row, const float* w,
                                            const float* near, const int* depth, uint64_t vis,
                                            int kk, int nc, int n, float* z) {
  if (kk >= nc + n) {  // behind the draft
#pragma unroll
    for (int y = 0; y < 16; ++y) z[y] = -INFINITY;
    return;
  }
  uint32_t sv[16];
  tmem_ld_cols<16>(taddr + kk, sv);
  if (kk + 16 <= nc) {  // committed
#pragma unroll
    for (int y = 0; y < 16; ++y) z[y] = fmaf(__uint_as_float(sv[y]), row.cs, w[kk + y]);
    return;
  }
  const uint32_t bits = static_cast<uint32_t>(vis >> kk);
#pragma unroll
  for (int y = 0; y < 16; ++y) {
    // A column outside the draft reads a neighbouring word of shared memory as
    // its depth; kept within the table it stays harmless, and is not used.
    const unsigned back = min(static_cast<unsigned>(depth[kk + y - nc]),
                              static_cast<unsigned>(row.depth));
    const float* from = kk + y < nc ? w + kk + y : near - back;
    const float x = fmaf(__uint_as_float(sv[y]), row.cs, *from);
    z[y] = bits >> y & 1 ? x : -INFINITY;
  }
}

// A tile with keys that not every row sees, 16 columns at a time.
template <int PARTS, int KS>
__device__ __forceinline__ void soft_tail(const TreeArgs& a, const View& v, const SoftRow& row,
                                          SoftState& st, int k) {
  using S = Shape<PARTS, KS>;
  TreeSmem& sm = *v.sm;
  volatile int* ab = &sm.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ItemInfo info = info_view<S>(a, v, k);
  const TreeInfo ti = tree_view(a, v, info.it->tree);
  const int n = info.it->n, len = info.it->len, j0 = st.t * S::kTile;
  if (!soft_begin(a, sm, st)) return;
  const float* w = v.win + st.s * a.win_stage + row.woff;
  const float* near = info.near + row.hrel * n + row.depth;  // of an ancestor: near[-its depth]
  const uint64_t vis = row.live ? tile_mask(ti.seen[row.node], j0 + row.k0, len) : 0;
  const int nc = len - j0 - row.k0;
  constexpr bool kOnce = S::kOnce;
  constexpr int kBlocks = S::kCols / 16;
  float z[kOnce ? S::kCols : 16];
  float mx = kNoMax, scale;
  if (row.warp_live) {
    if constexpr (kOnce) {
#pragma unroll
      for (int q = 0; q < kBlocks; ++q)
        tail_logits(row.lanes + row.k0, row, w, near, ti.depth, vis, 16 * q, nc, n, z + 16 * q);
#pragma unroll
      for (int y = 0; y < S::kCols; y += 2) mx = fmax3(mx, z[y], z[y + 1]);
    } else {
#pragma unroll 1
      for (int q = 0; q < kBlocks; ++q) {
        tail_logits(row.lanes + row.k0, row, w, near, ti.depth, vis, 16 * q, nc, n, z);
        tmem_st_32x32b_x16(row.lanes + row.k0 + 16 * q, reinterpret_cast<const uint32_t*>(z));
#pragma unroll
        for (int y = 0; y < 16; y += 2) mx = fmax3(mx, z[y], z[y + 1]);
      }
      tmem_st_wait();
    }
  }
  if (kOnce) soft_free_s(sm, st);
  // Rows of V behind the draft hold anything, and a drafted value that is not
  // finite must not meet the weight 0 of a row that does not see it: zeros
  // here, a quarter of the rows by each warp.  The latter are added to O at
  // the item's end.
  st.ok = warp_wait(&sm.v_full[st.s], st.phase, a.c.status, ab, kSiteTreeSoftK);
  if (!st.ok) return;
  {
    constexpr int kQuarter = S::kTile / kSoftWarps;
    const int first = j0 + kQuarter * warp - len;  // node of the quarter's first row
    uint8_t* const rows = v.sv + st.s * S::kTileBytes + kQuarter * warp * 128 + 16 * (lane & 7);
    bool any = false;
#pragma unroll 2
    for (int y = lane >> 3; y < kQuarter; y += 4) {
      const int i = first + y;
      if (i < 0) continue;
      uint4* const p = reinterpret_cast<uint4*>(rows + y * 128);
      if (i >= n) {
        *p = make_uint4(0, 0, 0, 0);
        any = true;
        continue;
      }
      uint4 x = *p;
      uint32_t* u = reinterpret_cast<uint32_t*>(&x);
      bool fix = false;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const bool lo = odd_exp(u[h]), hi = odd_exp(u[h] >> 16);
        fix |= lo | hi;
        u[h] &= (lo ? 0xFFFF0000u : 0xFFFFFFFFu) & (hi ? 0x0000FFFFu : 0xFFFFFFFFu);
      }
      if (fix) {
        atomicOr(&sm.odd[k & 1][i >> 5], 1u << (i & 31));
        *p = x;
        any = true;
      }
    }
    if (any) fence_proxy_async_smem();
    __syncwarp();
  }
  if (!soft_max(a, sm, row, st, mx, scale)) return;
  if (row.warp_live) {
    uint64_t l2 = 0ull;
    const uint64_t negm2 = f2_pack(-st.m, -st.m);
    auto weights = [&](const float* zz, int q) __attribute__((always_inline)) {
      uint32_t pk[PARTS][8];
#pragma unroll
      for (int y = 0; y < 8; ++y)
        soft_weights<PARTS, 8>(f2_pack(zz[2 * y], zz[2 * y + 1]), negm2, l2, pk, y);
#pragma unroll
      for (int part = 0; part < PARTS; ++part)
        tmem_st_pairs<16>(row.lanes + S::kColP + row.k0 / 2 + S::kPCols * part + 8 * q, pk[part]);
    };
    if constexpr (kOnce) {
#pragma unroll
      for (int q = 0; q < kBlocks; ++q) weights(z + 16 * q, q);
    } else {
#pragma unroll 1
      for (int q = 0; q < kBlocks; ++q) {
        tmem_ld_cols<16>(row.lanes + row.k0 + 16 * q, reinterpret_cast<uint32_t*>(z));
        weights(z, q);
      }
    }
    float b0, b1;
    f2_unpack(l2, b0, b1);
    st.l += b0 + b1;
  }
  if (!kOnce) soft_free_s(sm, st);
  soft_finish(a, sm, row, st, scale);
}

// o += the infinities and NaN among 2 W columns of the value of node i (zeros
// stood for them in the products), from column col on.
template <int W>
__device__ __forceinline__ void add_odd(const TreeArgs& a, int b, int hk, int len, int i, int col,
                                        float* o) {
  const CacheArgs& c = a.c;
  const int at = len + i;
  int pg = __ldg(c.block_table + static_cast<size_t>(b) * c.max_blocks + at / c.page);
  if (pg < 0 || pg >= c.num_pages) pg = 0;
  const uint32_t* vr = reinterpret_cast<const uint32_t*>(
      a.v_pages + ((static_cast<size_t>(pg) * c.Hkv + hk) * c.page + at % c.page) * kHeadDim + col);
#pragma unroll
  for (int y = 0; y < W; ++y) {
    const uint32_t u = __ldg(vr + y);
    if (odd_exp(u)) o[2 * y] += __uint_as_float(u << 16);
    if (odd_exp(u >> 16)) o[2 * y + 1] += __uint_as_float(u & 0xFFFF0000u);
  }
}

// o += x g, x being 4 N floats that another copy has handed over: chunks of 16
// bytes, swizzled by the row.
template <int N>
__device__ __forceinline__ void join_row(const uint8_t* row, int swz, float g, float* o) {
#pragma unroll
  for (int y = 0; y < N; ++y) {
    const float4 x = *reinterpret_cast<const float4*>(row + ((y ^ swz) << 4));
    o[4 * y] = fmaf(x.x, g, o[4 * y]);
    o[4 * y + 1] = fmaf(x.y, g, o[4 * y + 1]);
    o[4 * y + 2] = fmaf(x.z, g, o[4 * y + 2]);
    o[4 * y + 3] = fmaf(x.w, g, o[4 * y + 3]);
  }
}
template <int N>
__device__ __forceinline__ void hand_row(uint8_t* row, int swz, const float* o) {
#pragma unroll
  for (int y = 0; y < N; ++y)
    *reinterpret_cast<float4*>(row + ((y ^ swz) << 4)) =
        make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
}

// The item's end.  The copies of a row join by halves, through the buffer of
// the item's queries, which its products no longer read: two copies exchange
// 32 columns, and with four copies two pairs then exchange 16 (in the places
// that they have read), so that each ends with 64 / KS columns of the sum.
template <int PARTS, int KS>
__device__ __forceinline__ bool soft_end(const TreeArgs& a, const View& v, const SoftRow& row,
                                         const SoftState& st, const SoftSum& sum, int k) {
  using S = Shape<PARTS, KS>;
  TreeSmem& sm = *v.sm;
  const CacheArgs& c = a.c;
  volatile int* ab = &sm.abort_flag;
  const int lane = threadIdx.x & 31;
  constexpr int kOwn = 64 / KS < 32 ? 64 / KS : 32;  // columns at a time
  if (!warp_wait(&sm.pv_done, (st.g - 1) & 1, c.status, ab, kSiteTreeSoftEnd)) return false;
  tc_fence_after();
  const Item& it = sm.item[k & 1];
  const bool whole = it.t0 == 0 && it.t1 == it.tiles;
  const uint32_t* odd = sm.odd[k & 1];
  auto any_odd = [&]() { return (odd[0] | odd[1] | odd[2] | odd[3]) != 0; };
  const size_t orow =
      (static_cast<size_t>(it.b) * a.H + it.hk * a.group + it.g0 + row.hrel) * c.N + row.node;
  const size_t part = 2 * blockIdx.x + (it.t0 == 0 ? 1 : 0);
  float M = st.m, L = st.l;
  const bool held = it.t1 - it.t0 > S::kRun;
  const float kept = held ? ex2_approx(sum.m - M) : 0.0f;
  if (held) L = fmaf(sum.l, kept, L);
  // 32 columns of this lane's output, with what the runs before left of them.
  auto load = [&](int col, uint32_t* ov) __attribute__((always_inline)) {
    tmem_ld_cols<32>(row.lanes + kColO + col, ov);
    if (held) {
#pragma unroll
      for (int y = 0; y < 32; ++y)
        ov[y] = __float_as_uint(fmaf(sum.o[col + y], kept, __uint_as_float(ov[y])));
    }
  };
  // Columns col .. col + kOwn - 1 of the row's output.
  auto put = [&](float* o, int col) __attribute__((always_inline)) {
    if (!whole) {  // left to the combine kernel
      float4* dst = reinterpret_cast<float4*>(a.part) + (part * 16 + col / 4) * S::kRows + row.rr;
#pragma unroll
      for (int y = 0; y < kOwn / 4; ++y)
        dst[y * S::kRows] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
      // A sum with its sign bit set: drafted values that are not finite are
      // still to be added (here their part's factor could turn them into NaN).
      if (col == 0) a.part_ml[part * S::kRows + row.rr] = make_float2(M, any_odd() ? -L : L);
      return;
    }
    if (any_odd()) {
      const TreeInfo ti = tree_view(a, v, it.tree);
#pragma unroll 1
      for (int i = 0; i < it.n; ++i)
        if ((odd[i >> 5] >> (i & 31) & 1) && tree_sees(ti, row.node, i))
          add_odd<kOwn / 2>(a, it.b, it.hk, it.len, i, col, o);
    }
    const float inv = 1.0f / L;
    if (PARTS > 1) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.o) + orow * kHeadDim + col);
#pragma unroll
      for (int y = 0; y < kOwn / 4; ++y)
        dst[y] = make_float4(o[4 * y] * inv, o[4 * y + 1] * inv, o[4 * y + 2] * inv,
                             o[4 * y + 3] * inv);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + orow * kHeadDim + col);
#pragma unroll
      for (int y = 0; y < kOwn / 8; ++y) {
        const float* e = o + 8 * y;
        dst[y] = make_uint4(pack_bf16x2(e[0] * inv, e[1] * inv), pack_bf16x2(e[2] * inv, e[3] * inv),
                            pack_bf16x2(e[4] * inv, e[5] * inv), pack_bf16x2(e[6] * inv, e[7] * inv));
      }
    }
    if (col == 0 && a.lse) a.lse[orow] = (M + log2f(L)) * kLn2f;
  };
  uint32_t ov[32];
  float* o = reinterpret_cast<float*>(ov);
  if (KS == 1) {
#pragma unroll 1
    for (int col = 0; col < 64 && row.warp_live; col += 32) {
      load(col, ov);
      if (row.live) put(o, col);
    }
  } else {
    uint8_t* const merge = v.sq + (k & 1) * kQBytes;  // 128 rows of 128 bytes
    const int mine = threadIdx.x, other = mine ^ S::kRows, swz = mine & 7;
    int col = 32 * (row.copy & 1);  // of o[0]
    if (row.warp_live) {
      load(col ^ 32, ov);
      hand_row<8>(merge + mine * 128, swz, o);
      v.merge_ml[mine] = make_float2(M, L);
      load(col, ov);
    }
    // The next maximum and sum, and what is kept of both.
    auto join = [&](int from, float& f, float& g) {
      const float2 ml = v.merge_ml[from];
      const float m2 = fmaxf(M, ml.x);
      f = ex2_approx(M - m2);
      g = ex2_approx(ml.x - m2);
      L = L * f + ml.y * g;
      M = m2;
    };
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.merge[0]);
    if (!warp_wait(&sm.merge[0], k & 1, c.status, ab, kSiteTreeMerge)) return false;
    float f, g;
    if (row.warp_live) {
      join(other, f, g);
#pragma unroll
      for (int y = 0; y < 32; ++y) o[y] *= f;
      join_row<8>(merge + other * 128, swz, g, o);
    }
    if (KS == 4) {
      if (row.warp_live) {
        v.merge_ml[other] = make_float2(M, L);
        if (row.copy & 2) {
          hand_row<4>(merge + other * 128, swz, o);
#pragma unroll
          for (int y = 0; y < 16; ++y) o[y] = o[y + 16];
          col += 16;
        } else {
          hand_row<4>(merge + other * 128, swz, o + 16);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.merge[1]);
      if (!warp_wait(&sm.merge[1], k & 1, c.status, ab, kSiteTreeMerge)) return false;
      if (row.warp_live) {
        join(other ^ 64, f, g);
#pragma unroll
        for (int y = 0; y < 16; ++y) o[y] *= f;
        join_row<4>(merge + (other ^ 64) * 128, swz, g, o);
      }
    }
    if (row.live) put(o, col);
  }
  // O has been read before the next item's products overwrite it: they wait
  // for its p_full, on which every warp arrives after this.
  tc_fence_before();
  return true;
}

// One CTA walks its run of tiles; two CTAs share an SM, so that one's
// hand-offs are covered by the other's work.  Roles:
//   producer warp   walks the plan; prepares each item one ahead (queries,
//                   the tree's ancestors) in one of two buffers, and loads K
//                   and V (TMA) and the table windows of the item's heads
//                   (bulk copies) into a ring of tiles;
//   MMA thread      S = Q K^T  (128 x tile x 64, Q and K from shared memory),
//                   O += P V   (128 x 64 x tile, P from Tensor Memory);
//   softmax warps   four, a thread per lane of Tensor Memory.
// Queries come by asynchronous copies of 16 bytes; TMA boxes of 32 rows were 2%
// faster with 100 nodes and 2% slower with one.
// All 128 lanes are computed whatever the number of rows: the two products of
// 64 keys take 256 cycles of an SM's tensor core, its share of HBM delivers
// their 16 KB in about 700.  S runs a tile ahead of the softmax.
//
// KS (1, 2, 4): an item of at most 128 / KS rows fills Tensor Memory KS times
// over, and each copy of a row works on its own KS-th of the keys of every
// tile, with its own maximum, sum and output, which are joined at the item's
// end.  The products cost the same (a step of P V adds to the lanes of its
// keys' copy only), and the softmax takes a KS-th of the time.  With copies a
// tile is 128 keys: a tile's hand-offs (about 1000 cycles) then weigh half.
// The softmax needs no exchange between threads; O is rescaled only when a
// row's maximum grows by more than 8.
//
// PARTS: bf16 parts of a weight in the product with V.  One rounds a weight by
// at most 2^-8, which moves an output by as much as its own rounding to bf16
// does; three carry 24 bits, for fp32 output.  Sums are of the exact weights.
// Measured against 64 bits: 0.0017 to 0.0020 relative for bf16 output (0.0016 to
// 0.0017 are its own rounding), 4e-7 to 1e-6 for fp32 output, up to 7e-6 where
// thousands of positive values have about the same weight (kRunParts).
template <int PARTS, int KS>
__global__ void __launch_bounds__(kTreeThreads, 2)
    bam_tree_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                    const __grid_constant__ TreeArgs a) {
  using S = Shape<PARTS, KS>;
  constexpr int kRows = S::kRows, kTile = S::kTile, kTileBytes = S::kTileBytes;
  const View v = smem_view<S>(a);
  uint8_t *const sq = v.sq, *const sk = v.sk, *const sv_ring = v.sv;
  float* const win = v.win;
  TreeSmem& sm = *v.sm;
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kProducer = kSoftWarps, kMma = kSoftWarps + 1;
  volatile int* ab = &sm.abort_flag;

  if (threadIdx.x == 0) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.s_free[s], kSoftWarps);
      mbar_init(&sm.v_empty[s], 1);
    }
    mbar_init(&sm.s_full, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sm.item_full[x], 1);
      mbar_init(&sm.item_empty[x], kSoftWarps);
    }
    mbar_init(&sm.p_full, kSoftWarps);
    mbar_init(&sm.pv_done, 1);
    mbar_init(&sm.merge[0], kSoftWarps);
    mbar_init(&sm.merge[1], kSoftWarps);
    mbar_init(&sm.mma_final, 1);
    fence_barrier_init();
    sm.abort_flag = 0;
  }
  if (warp == kMma) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sm.tmem_base;
  // The plan, the table and the status words come from the previous kernel
  // (a wait that looks at an abort word before it is cleared would give up).
  // With few sequences (one a lane) the producer makes the plan itself, and its
  // first loads of keys and queries, which no kernel of the call writes, do not
  // wait: 17.4 instead of 18.5 us for 16 sequences of 360 keys, 13.4 instead of
  // 14.5 for one of 500, 86.8 instead of 89.6 for one of 131072; 44.0 against 43.7 at
  // 13 of 9001.
  grid_dep_trigger();
  if (warp != kProducer || c.B > 32) grid_dep_wait();

  if (warp == kProducer) {
    // ---------------------------------------------------------------- producer
    bool ok = true, args_ok = true;
    bool early = c.B <= 32;  // the previous kernel has not been waited for
    // 32 sequences a time, one a lane: where they begin and end, their lengths.
    int b = 0, b0 = 0, len_l = 0, n_l = 0;
    int64_t beg_l = 0, end_l = 0;
    auto fetch = [&]() {
      const int y = min(b0 + lane, c.B - 1);
      beg_l = __ldcg(a.plan + y);
      end_l = __ldcg(a.plan + y + 1);
      cache_lengths(c, y, &len_l, &n_l);
    };
    int64_t all;
    if (early) {
      if (lane < c.B) cache_lengths(c, lane, &len_l, &n_l);
      end_l = n_l > 0 ? static_cast<int64_t>(c.Hkv) * ((a.group * n_l + kRows - 1) / kRows) *
                            item_units(kTile, S::kTailCost, len_l, n_l)
                      : 0;
      beg_l = end_l;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, end_l, off);
        if (lane >= off) end_l += y;
      }
      beg_l = end_l - beg_l;
      all = __shfl_sync(0xffffffffu, end_l, 31);
    } else {
      all = __ldcg(a.plan + c.B);
    }
    const int active = active_ctas(all, a.ctas), cta = blockIdx.x;
    int64_t x = 0, end = 0;
    if (all > 0 && cta < active) {
      x = range_beg(all, active, cta);
      end = range_beg(all, active, cta + 1);
    }
    if (!early && x < end) {
      // The sequence that unit x lies in: how many end at or before it.
      int hi = c.B;
      while (hi - b > 32) {
        const int step = (hi - b + 31) / 32, y = min(b + (lane + 1) * step, hi);
        const int full = __popc(__ballot_sync(0xffffffffu, __ldcg(a.plan + y) <= x));
        b += full * step;
        hi = min(hi, b + step);
      }
      b += __popc(__ballot_sync(0xffffffffu, b + lane < hi && __ldcg(a.plan + b + lane + 1) <= x));
      b0 = b;
      fetch();
    }
    int issued = 0, s = 0, phase = 1, k = 0, last_b = -1, tree = 1;
    Item it;
    int units = 0, plain = 0;  // of an item of the sequence
    CutItem cut{0, 0, 0, 0, 0, 0};
    int64_t seq_end = x;  // of the sequence that the last item was of
    for (;; ++k) {
      const ItemInfo info = info_view<S>(a, v, k);
      if (!ok) break;
      it.t0 = it.t1 = 0;
      if (x < end) {
        int at = 0;  // place of unit x in its item
        if (x < seq_end) {
          it.r0 += kRows;
          if (it.r0 >= a.group * it.n) {
            it.r0 = 0;
            ++it.hk;
          }
        } else {
          // The sequence of unit x, at b or behind it.
          for (;;) {
            const unsigned ends = __ballot_sync(0xffffffffu, b0 + lane >= b && end_l > x);
            if (ends) {
              b = b0 + __ffs(ends) - 1;
              break;
            }
            b = b0 += 32;
            fetch();
          }
          it.b = b;
          it.len = __shfl_sync(0xffffffffu, len_l, b - b0);
          it.n = __shfl_sync(0xffffffffu, n_l, b - b0);
          seq_end = __shfl_sync(0xffffffffu, end_l, b - b0);
          const int64_t local = x - __shfl_sync(0xffffffffu, beg_l, b - b0);
          it.tiles = (it.len + it.n + kTile - 1) / kTile;
          plain = it.len / kTile;
          units = item_units(kTile, S::kTailCost, it.len, it.n);
          it.hk = it.r0 = 0;
          if (local > 0) {
            const int idx = local < (1 << 30) ? static_cast<int>(local) / units
                                              : static_cast<int>(local / units);
            at = static_cast<int>(local - static_cast<int64_t>(idx) * units);
            const int nrb = (a.group * it.n + kRows - 1) / kRows;
            it.hk = idx / nrb;
            it.r0 = (idx - it.hk * nrb) * kRows;
          }
        }
        it.r1 = min(it.r0 + kRows, a.group * it.n);
        const int stop = static_cast<int>(min(static_cast<int64_t>(units), at + (end - x)));
        x += stop - at;
        it.t0 = tiles_before(S::kTailCost, plain, at);
        it.t1 = tiles_before(S::kTailCost, plain, stop);
        // (none: the share ends before the end of the item's next tile)
        if (it.t1 <= it.t0) it.t1 = 0;
        if (it.t0 == 0 && it.t1 > 0) {  // do other CTAs go on with it?
          cut.n = 0;
          if (stop < units)
            cut = CutItem{it.b, it.hk, it.r0, it.n, cta,
                          range_owner(all, active, x + (units - stop) - 1)};
          if (a.by_item && lane == 0)
            a.cut[(it.b * c.Hkv + it.hk) * a.nrb_most + it.r0 / kRows] = cut;
        }
      }
      const int n = it.n, len = it.len;
      const int g0 = it.t1 ? it.r0 / n : 0, heads = it.t1 ? (it.r1 - 1) / n - g0 + 1 : 0;
      it.g0 = g0;
      const float* trow = a.table + static_cast<size_t>(it.hk * a.group + g0) * a.tab_len;
      const int y0 = a.tab_zero - (len + n - 1);  // entry of key 0 for the last position
      const int nwin = window_floats(kTile, n);
      // The table windows of tile t into slot sl.
      auto issue_windows = [&](int t, int sl) {
        for (int g = lane; g < heads; g += 32) {
          const float* tr = trow + static_cast<size_t>(g) * a.tab_len;
          ok &= bulk_load_checked(win + sl * a.win_stage + g * nwin, tr + ((y0 + t * kTile) & ~3),
                                  nwin * 4, &sm.k_full[sl], tr, tr + a.tab_len, c.status, ab,
                                  kSiteTreeTable);
        }
        ok = __all_sync(0xffffffffu, ok);
      };
      // Tiles are issued as slots are free; `wait` waits for them.  The last
      // tiles come first: where the prior falls off with distance, as it mostly
      // does, the first tiles then hold the largest logits, and O is hardly
      // ever rescaled.
      int t = it.t1 - 1, pages = 0, page_rows = 0;
      auto issue_tiles = [&](bool wait) {
        for (; t >= it.t0; --t) {
          if (issued >= a.stages) {
            if (!wait) {
              const bool free = mbar_test(&sm.s_free[s], phase) && mbar_test(&sm.v_empty[s], phase);
              if (!__all_sync(0xffffffffu, free)) return;
            } else {
              ok = warp_wait(&sm.s_free[s], phase, c.status, ab, kSiteTreeProducer);
              if (!ok) return;
            }
          }
          constexpr int kBoxes = kTile / kBox, kAhead = 32 / kBoxes;
          const int ahead = (it.t1 - 1 - t) % kAhead;
          if (ahead == 0) {
            // pages of the boxes of the next tiles and their rows in them, one a lane
            const int tl = t - lane / kBoxes, key = tl * kTile + lane % kBoxes * kBox;
            pages = page_rows = 0;
            if (tl >= it.t0 && key < len + n) {
              const int blk = key / c.page;
              page_rows = key - blk * c.page;
              pages = __ldg(c.block_table + static_cast<size_t>(it.b) * c.max_blocks + blk);
              if (pages < 0 || pages >= c.num_pages) {
                args_ok = false;
                pages = 0;
              }
            }
          }
          // Boxes that hold no key are not loaded: their rows of S are out of
          // sight and their rows of V are made zero.
          const int boxes = min(kBoxes, (len + n - t * kTile + kBox - 1) / kBox);
          int plane[kBoxes], row[kBoxes];
#pragma unroll
          for (int x2 = 0; x2 < kBoxes; ++x2) {
            plane[x2] = __shfl_sync(0xffffffffu, pages, ahead * kBoxes + x2) * c.Hkv + it.hk;
            row[x2] = __shfl_sync(0xffffffffu, page_rows, ahead * kBoxes + x2);
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.k_full[s], boxes * kBoxBytes + heads * nwin * 4);
#pragma unroll
            for (int x2 = 0; x2 < kBoxes; ++x2)
              if (x2 < boxes)
                tma_load_3d(sk + s * kTileBytes + x2 * kBoxBytes, &tk, &sm.k_full[s], 0,
                            row[x2], plane[x2]);
          }
          __syncwarp();
          if (!early) issue_windows(t, s);
          if (ok && wait && issued >= a.stages)
            ok = warp_wait(&sm.v_empty[s], phase, c.status, ab, kSiteTreeProducer);
          // (after a give-up the slot's V copy is still armed, so that the
          // copies can be drained alike)
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.v_full[s], ok ? boxes * kBoxBytes : 0);
#pragma unroll
            for (int x2 = 0; x2 < kBoxes; ++x2)
              if (ok && x2 < boxes)
                tma_load_3d(sv_ring + s * kTileBytes + x2 * kBoxBytes, &tv, &sm.v_full[s], 0,
                            row[x2], plane[x2]);
          }
          __syncwarp();
          ++issued;
          if (++s == a.stages) {
            s = 0;
            phase ^= 1;
          }
          if (!ok) return;
        }
      };
      // What the item's preparation needs is on its way while tiles are issued.
      int par[kPer];
      if (it.t1 && it.b != last_b) tree_parents(c, it.b, n, par);
      const float s_lane =
          a.ssmax && lane < heads ? __ldg(a.s + it.hk * a.group + g0 + lane) : 1.0f;
      issue_tiles(false);
      if (k >= 2) {
        ok = ok && warp_wait(&sm.item_empty[k & 1], (k / 2 - 1) & 1, c.status, ab, kSiteTreeItem);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) break;
      if (it.t1 == 0) {
        if (early) grid_dep_wait();
        early = false;
        if (lane == 0) {
          if (!a.by_item && cta < active) a.cut[cta] = cut;
          *info.it = it;
          mbar_arrive(&sm.item_full[k & 1]);
        }
        break;
      }
      // Queries: the item's rows, once for each copy, 16-byte chunks swizzled
      // as the product reads them; eight lanes a row.  Without shared heads, or
      // with all N nodes drafted, the rows lie one after the other.
      {
        const int nrows = it.r1 - it.r0, padded = (nrows + 31) & ~31;
        const int ch = lane & 7, r4 = lane >> 3;
        const uint32_t dst = smem_u32(sq + (k & 1) * kQBytes) + r4 * 128 + ((ch ^ r4) << 4);
        const uint16_t* base =
            a.q + (static_cast<size_t>(it.b) * a.H + it.hk * a.group) * c.N * kHeadDim + 8 * ch;
        // Row rr = r4 + 4 x of the item, from `src` (any address if it is none).
        auto copy = [&](int rr, const uint16_t* src) __attribute__((always_inline)) {
          const uint32_t d = (dst ^ ((rr & 4) << 4)) + (rr - r4) * 128;
#pragma unroll
          for (int cp = 0; cp < KS; ++cp) cp_async16(d + cp * kRows * 128, src, rr < nrows);
        };
        if (a.group == 1 || n == c.N) {
          const uint16_t* src = base + static_cast<size_t>(it.r0 + r4) * kHeadDim;
#pragma unroll 4
          for (int rr = r4; rr < padded; rr += 4, src += 4 * kHeadDim)
            copy(rr, rr < nrows ? src : base);
        } else {
          int hg = (it.r0 + r4) / n, node = it.r0 + r4 - hg * n;
#pragma unroll 2
          for (int rr = r4; rr < padded; rr += 4) {
            copy(rr, rr < nrows ? base + (static_cast<size_t>(hg) * c.N + node) * kHeadDim : base);
            for (node += 4; node >= n; node -= n) ++hg;
          }
        }
      }
      if (a.ssmax) {
        if (lane < heads) info.s[lane] = s_lane;
        for (int h = lane + 32; h < heads; h += 32)
          info.s[h] = __ldg(a.s + it.hk * a.group + g0 + h);
      }
      if (it.b != last_b) {
        tree ^= 1;
        args_ok &= tree_info(!c.parents, par, a.nodes, tree_view(a, v, tree), jump_view(a, v));
        last_b = it.b;
      }
      it.tree = tree;
      if (early) {
        grid_dep_wait();
        early = false;
        for (int i = 0; i < issued; ++i) issue_windows(it.t1 - 1 - i, i);
      }
      // Some tile holds drafted keys: their distances' table entries.
      if (it.t1 * kTile > len) {
        for (int h = 0; h < heads; ++h)
          for (int y = lane; y < n; y += 32)
            cp_async4(smem_u32(info.near + h * n + y),
                      trow + static_cast<size_t>(h) * a.tab_len + a.tab_zero - y);
      }
      if (lane == 0) *info.it = it;
      if (lane < kTreeMax / 32) sm.odd[k & 1][lane] = 0;
      cp_async_wait();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_full[k & 1]);
      issue_tiles(true);
      if (!ok) break;
    }
    // Copies in flight land before the CTA leaves.
    cp_async_wait();
    for (int i = max(0, issued - a.stages); i < issued; ++i) {
      mbar_drain(&sm.k_full[i % a.stages], (i / a.stages) & 1);
      mbar_drain(&sm.v_full[i % a.stages], (i / a.stages) & 1);
    }
    if (!args_ok) record_bad_arg(c.status);
  } else if (warp == kMma) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t id_s = idesc_bf16(128, kTile, false, false);
      const uint32_t id_o = idesc_bf16(128, 64, false, true);
      const uint64_t qd = sdesc_sw128(smem_u32(sq), 16, 1024);
      const uint64_t kd = sdesc_sw128(smem_u32(sk), 16, 1024);
      const uint64_t vd = sdesc_sw128(smem_u32(sv_ring), 16384, 1024);
      constexpr uint64_t kSlotDesc = kTileBytes >> 4, kQDesc = kQBytes >> 4;
      // Two places in the same sequence of tiles: S runs ahead of P V.
      struct Place {
        int k, left, g, s, phase;  // item, its tiles to come, tile, ring slot and phase
        int run;                   // tiles of the item that O is to take on
      };
      Place ps{-1, 0, 0, 0, 0, 0}, pv{-1, 0, 0, 0, 0, 0};
      bool ok = true;
      auto advance = [&](Place& p) {
        --p.left;
        ++p.g;
        p.run = (p.run + 1) & (S::kRun - 1);
        if (++p.s == a.stages) {
          p.s = 0;
          p.phase ^= 1;
        }
      };
      // Puts p on the next tile; false at the end or when a wait gave up.
      auto enter = [&](Place& p) {
        if (p.left > 0) return true;
        ++p.k;
        p.run = 0;
        ok = ok && tree_wait(&sm.item_full[p.k & 1], (p.k >> 1) & 1, c.status, ab, kSiteTreeMmaItem);
        if (!ok) return false;
        const Item& it = sm.item[p.k & 1];
        p.left = it.t1 - it.t0;
        return it.t1 > 0;
      };
      auto issue_s = [&]() {
        if (ps.g > 0) {  // the S before it has been read
          const int q = (ps.s == 0 ? a.stages : ps.s) - 1;
          ok = ok && tree_wait(&sm.s_free[q], ps.s == 0 ? ps.phase ^ 1 : ps.phase, c.status, ab,
                               kSiteTreeMmaS);
        }
        ok = ok && tree_wait(&sm.k_full[ps.s], ps.phase, c.status, ab, kSiteTreeMmaK);
        if (!ok) return;
        tc_fence_after();
        const uint64_t q0 = qd + kQDesc * (ps.k & 1), k0 = kd + kSlotDesc * ps.s;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ss(tm, q0 + 2 * kk, k0 + 2 * kk, id_s, kk > 0 ? 1u : 0u);
        umma_commit(&sm.s_full);
        advance(ps);
      };
      bool more = enter(ps);  // tiles whose S is to come
      if (more) issue_s();
      while (ok && ps.g > pv.g) {
        // The next tile's S goes first if its item and keys are there (the
        // softmax reads this tile's S before it writes P).
        if (more &&
            (ps.left > 0 || mbar_test(&sm.item_full[(ps.k + 1) & 1], ((ps.k + 1) >> 1) & 1))) {
          more = enter(ps);
          if (more && mbar_test(&sm.k_full[ps.s], ps.phase)) issue_s();
        }
        const bool behind = ps.g == pv.g + 1;
        if (!enter(pv)) break;
        ok = ok && tree_wait(&sm.v_full[pv.s], pv.phase, c.status, ab, kSiteTreeMmaK) &&
             tree_wait(&sm.p_full, pv.g & 1, c.status, ab, kSiteTreeMmaP);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk) {
            // 16 keys; they belong to copy kk / kSteps.
            constexpr int kSteps = kTile / 16 / KS;
            umma_ts_lanes<KS>(tm + kColO, tm + S::kColP + S::kPCols * part + 8 * kk,
                              vd + kSlotDesc * pv.s + 128 * kk, id_o,
                              (pv.run > 0 || part > 0 || kk % kSteps > 0) ? 1u : 0u, kk / kSteps);
          }
        umma_commit(&sm.pv_done);
        umma_commit(&sm.v_empty[pv.s]);
        advance(pv);
        if (behind && more) {
          more = enter(ps);
          if (more) issue_s();
        }
      }
      umma_commit(&sm.mma_final);
      mbar_drain(&sm.mma_final, 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    SoftState st{0, 0, 0, 0, 0.0f, 0.0f, true, true};
    SoftSum sum;
    for (int k = 0;; ++k) {
      st.ok = warp_wait(&sm.item_full[k & 1], (k >> 1) & 1, c.status, ab, kSiteTreeSoftItem);
      if (!st.ok) break;
      const Item& it = sm.item[k & 1];
      const int t0 = it.t0, plain = it.len / S::kTile;  // tiles without drafted keys
      st.t = it.t1 - 1;
      if (st.t < 0) break;
      st.m = kNoMax;
      st.l = 0.0f;
      st.first = true;
      const SoftRow row = soft_row<S>(a, v, k);
      // (the tail ends within the first run)
      int stop = st.t - S::kRun;
      while (st.ok && st.t >= max(plain, t0)) soft_tail<PARTS, KS>(a, v, row, st, k);
      for (bool held = false; st.ok; held = true, stop -= S::kRun) {
        const int last = max(stop + 1, t0);
        while (st.ok && st.t >= last) soft_tile<PARTS, KS>(a, v, row, st);
        if (!st.ok || st.t < t0) break;
        soft_hold<(PARTS > 1)>(a, sm, row, st, sum, held);
      }
      if (!st.ok || !soft_end<PARTS, KS>(a, v, row, st, sum, k)) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[k & 1]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tm, kTmemCols);
  }
}

// Joins the parts of the items that were cut: blocks (x, .) the one of record x.
// A warp takes half the columns of four rows, a lane four columns (a chunk) of
// one row, of every kSplit-th part.  kSplit 4 is for items of many parts: one
// sequence of 131072 keys, 12 heads (26 parts an item) 95 us with 1, 87 with 4;
// 4 chains of 128 nodes over 20000 keys (7 parts) 71.6 with 1, 78.6 with 4.
constexpr int kJoinThreads = 128, kJoinParts = 8;  // parts in flight
constexpr int kJoinRows = kJoinThreads / 16;       // rows of a block
template <int kSplit>
__global__ void __launch_bounds__(kJoinThreads* kSplit) bam_tree_combine_kernel(const TreeArgs a) {
  const CacheArgs& c = a.c;
  const int tid = threadIdx.x % kJoinThreads, split = threadIdx.x / kJoinThreads;
  const int warp = tid >> 5, lane = tid & 31;
  bool used = true;  // the record is of an item that there is
  if (a.by_item) {
    int len, n;
    cache_lengths(c, blockIdx.x / a.nrb_most / c.Hkv, &len, &n);
    used = static_cast<int>(blockIdx.x % a.nrb_most) * a.rows < a.group * n;
  }
  grid_dep_wait();
  if (*reinterpret_cast<volatile int*>(&c.status->abort) != 0) {
    // A wait of the call gave up: NaN in every row.
    const float nan = __int_as_float(0x7fc00000);
    const int64_t rows = static_cast<int64_t>(c.B) * a.H * c.N;
    const int64_t first = static_cast<int64_t>(blockIdx.y * gridDim.x + blockIdx.x) * 4 + warp;
    for (int64_t row = first; split == 0 && row < rows; row += static_cast<int64_t>(gridDim.x) * gridDim.y * 4) {
      int len, n;
      cache_lengths(c, static_cast<int>(row / c.N / a.H), &len, &n);
      if (row % c.N >= n) continue;
      if (a.o_fp32)
        reinterpret_cast<float2*>(a.o)[row * 32 + lane] = make_float2(nan, nan);
      else
        reinterpret_cast<uint32_t*>(a.o)[row * 32 + lane] = pack_bf16x2(nan, nan);
      if (a.lse && lane == 0) a.lse[row] = nan;
    }
    return;
  }
  if (!used) return;
  const CutItem it = a.cut[blockIdx.x];
  if (!a.by_item && blockIdx.x >= active_ctas(__ldcg(a.plan + c.B), a.ctas)) return;
  if (it.n == 0) return;
  const int c0 = it.first;
  const int rr = kJoinRows * blockIdx.y + 4 * (warp >> 1) + (lane & 3);
  const int chunk = 8 * (warp & 1) + (lane >> 2);
  const int r = it.r0 + rr, rows = a.group * it.n;
  const bool on = r < rows;
  float M = kNoMax, L = 0.0f;
  unsigned odd = 0;  // its top bit: the sign of a part's sum
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float4* part = reinterpret_cast<const float4*>(a.part);
  for (int x0 = c0 + split; on && x0 <= it.last; x0 += kJoinParts * kSplit) {
    float2 ml[kJoinParts];
    float4 p[kJoinParts];
#pragma unroll
    for (int u = 0; u < kJoinParts; ++u) {
      ml[u] = make_float2(kNoMax, 0.0f);
      const int x = x0 + u * kSplit;
      if (x > it.last) continue;
      const size_t at = 2 * x + (x == c0 ? 1 : 0);
      ml[u] = __ldcg(a.part_ml + at * a.rows + rr);
      p[u] = __ldcg(part + (at * 16 + chunk) * a.rows + rr);
    }
    float m = M;
#pragma unroll
    for (int u = 0; u < kJoinParts; ++u) m = fmaxf(m, ml[u].x);
    const float old = ex2_approx(M - m);
    M = m;
    L *= old;
    v = make_float4(v.x * old, v.y * old, v.z * old, v.w * old);
#pragma unroll
    for (int u = 0; u < kJoinParts; ++u) {
      if (x0 + u * kSplit > it.last) continue;
      const float f = ex2_approx(ml[u].x - m);
      odd |= __float_as_uint(ml[u].y);
      L = fmaf(fabsf(ml[u].y), f, L);
      v.x = fmaf(p[u].x, f, v.x);
      v.y = fmaf(p[u].y, f, v.y);
      v.z = fmaf(p[u].z, f, v.z);
      v.w = fmaf(p[u].w, f, v.w);
    }
  }
  if (kSplit > 1) {
    __shared__ float4 sv[kSplit][kJoinThreads];
    __shared__ float2 sml[kSplit][kJoinThreads];
    sv[split][tid] = v;
    sml[split][tid] = make_float2(M, odd >> 31 ? -L : L);
    __syncthreads();
    if (split > 0) return;
    float m = M;
#pragma unroll
    for (int u = 1; u < kSplit; ++u) m = fmaxf(m, sml[u][tid].x);
    const float old = ex2_approx(M - m);
    L *= old;
    v = make_float4(v.x * old, v.y * old, v.z * old, v.w * old);
    M = m;
#pragma unroll
    for (int u = 1; u < kSplit; ++u) {
      const float2 ml = sml[u][tid];
      const float4 p = sv[u][tid];
      const float f = ex2_approx(ml.x - m);
      odd |= __float_as_uint(ml.y);
      L = fmaf(fabsf(ml.y), f, L);
      v = make_float4(fmaf(p.x, f, v.x), fmaf(p.y, f, v.y), fmaf(p.z, f, v.z), fmaf(p.w, f, v.w));
    }
  }
  if (!on) return;
  const float inv = 1.0f / L;
  const int h = r / it.n;
  if (odd >> 31) {
    // The row's node and its ancestors.
    int len, n, i = r - h * it.n;
    cache_lengths(c, it.b, &len, &n);
    while (i >= 0) {
      add_odd<2>(a, it.b, it.hk, len, i, 4 * chunk, reinterpret_cast<float*>(&v));
      const int p = c.parents ? __ldg(c.parents + static_cast<size_t>(it.b) * c.N + i) : i - 1;
      i = p < i ? p : -1;
    }
  }
  const size_t orow = (static_cast<size_t>(it.b) * a.H + it.hk * a.group + h) * c.N + (r - h * it.n);
  if (a.o_fp32)
    reinterpret_cast<float4*>(a.o)[orow * 16 + chunk] =
        make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  else
    reinterpret_cast<uint2*>(a.o)[orow * 16 + chunk] =
        make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
  if (a.lse && chunk == 0) a.lse[orow] = (M + log2f(L)) * kLn2f;
}

constexpr size_t kSmemTwo = 113 * 1024;  // a CTA's share when two fit an SM
constexpr size_t kSmemOne = 227 * 1024;

// Shared memory of a CTA besides its ring stages, and of one stage.
size_t smem_fixed(const TreeArgs& a) {
  return 1024 + 2 * kQBytes + sizeof(TreeSmem) + 44 * static_cast<size_t>(a.nodes) +
         8 * static_cast<size_t>(a.near) + 8 * a.rows + 8 * kRowsMax;
}
size_t smem_stage(const TreeArgs& a) {
  return 2 * static_cast<size_t>(a.tile) * kHeadDim * 2 + static_cast<size_t>(a.win_stage) * 4;
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
// not fit (more heads share a key head than its windows have room for).  From 16
// query heads a key head on, with few nodes, the windows of 128-key tiles leave
// room for one CTA an SM instead of two: 64 single tokens over 16384 keys take
// 169 us with 64 query and 4 key heads, 108 with 32 and 4.
bool tree_config(TreeArgs* a, int sms) {
  a->tile = tree_tile(a->o_fp32 ? 3 : 1, kRowsMax / a->rows);
  // Most heads and floats that a stage's windows hold, over the node counts.
  a->win_stage = a->near = 0;
  a->nodes = (a->c.N + 31) & ~31;
  for (int n = 1; n <= a->c.N; ++n) {
    int heads = (a->rows + n - 2) / n + 1;
    if (heads > a->group) heads = a->group;
    const int floats = heads * window_floats(a->tile, n);
    if (floats > a->win_stage) a->win_stage = floats;
    if (heads * n > a->near) a->near = (heads * n + 3) & ~3;
  }
  const size_t fixed = smem_fixed(*a), stage = smem_stage(*a);
  int per_sm = 2;
  size_t budget = kSmemTwo;
  if (fixed + 2 * stage > budget) {
    per_sm = 1;
    budget = kSmemOne;
  }
  a->stages = static_cast<int>((budget - fixed) / stage);
  if (a->stages > kMaxStages) a->stages = kMaxStages;
  a->ctas = per_sm * sms < kTreeCtas ? per_sm * sms : kTreeCtas;
  // Records of the items or of the CTAs, whichever are fewer.
  a->nrb_most = (a->group * a->c.N + a->rows - 1) / a->rows;
  a->by_item = static_cast<int64_t>(a->c.B) * a->c.Hkv * a->nrb_most <= a->ctas;
  a->tail_cost = tree_tail_cost(a->o_fp32 ? 3 : 1, kRowsMax / a->rows);
  return a->stages >= 2 && a->ctas >= 1;
}

cudaError_t launch_tree_prep(const TreeArgs& a, cudaStream_t st) {
  // It asks for the attention kernel's division of an SM's memory, whose CTAs can
  // then start beside it: 86.8 instead of 88.8 us with 131072 keys.
  static bool divided[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const bool cached = dev >= 0 && dev < 64;
  if (e == cudaSuccess && !(cached && divided[dev])) {
    e = cudaFuncSetAttribute(bam_tree_prep_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess && cached) divided[dev] = true;
  }
  if (e != cudaSuccess) return e;
  // At most about four blocks an SM, however long the table is: the attention
  // kernel starts when the last block has started.
  const int want = a.tab_zero / 256 + 1, y = a.H < 608 ? a.H : 608;
  const int most = (608 + y - 1) / y;
  return launch_k(bam_tree_prep_kernel, dim3(want < most ? want : most, y), dim3(256), 0, st, false, a);
}

cudaError_t launch_tree(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a,
                          cudaStream_t st) {
  return a.o_fp32 ? launch_parts<3>(tk, tv, a, st) : launch_parts<1>(tk, tv, a, st);
}

cudaError_t launch_tree_combine(const TreeArgs& a, cudaStream_t st) {
  const int records = a.by_item ? a.c.B * a.c.Hkv * a.nrb_most : a.ctas;
  const dim3 grid(records, a.rows / kJoinRows);
  if (records * 8 < a.ctas)  // mostly more than eight parts an item
    return launch_k(bam_tree_combine_kernel<4>, grid, dim3(4 * kJoinThreads), 0, st, true, a);
  return launch_k(bam_tree_combine_kernel<1>, grid, dim3(kJoinThreads), 0, st, true, a);
}

}  // namespace bam
