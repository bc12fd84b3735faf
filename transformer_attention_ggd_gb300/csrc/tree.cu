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

constexpr int kConsumers = 4;  // warps
constexpr int kTreeThreads = 32 * (kConsumers + 1);
constexpr int kKvBytes = kTreeTile * kHeadDim * 2;  // 8 KB of K (and of V) a tile
constexpr int kMaxStages = 8;
constexpr int kMergeStride = 72;  // floats of a merge row: 8-byte stores of 8 rows hit all banks
constexpr float kRescale = 8.0f;  // log2 units by which a weight may exceed 1
constexpr float kNoMax = -3.4e38f;  // below every logit (the table is clamped at -3e38)

enum : int {
  kSiteTreeProducer = 60,
  kSiteTreeConsumer = 61,
  kSiteTreeTable = 62
};

struct __align__(16) TreeSmem {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint32_t seen[kTreeMax][kTreeMax / 32];  // ancestors of each node, and itself
  int jump[kTreeMax];
  int depth[kTreeMax];
  int node[kTreeMax];  // of the item's rows: node (-1: no row) and query head
  int head[kTreeMax];
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

// ---------------------------------------------------------------- matrix instructions

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory");
}
__device__ __forceinline__ bool consumer_or(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "n"(32 * kConsumers)
      : "memory");
  return r != 0;
}

// Depth and ancestors of the nodes of sequence b, by the consumer threads
// (one node each).  Each round doubles the chains that the jump pointers
// span.  Returns false in a thread whose node had a parent outside [-1, i).
__device__ __forceinline__ bool tree_seen(const CacheArgs& c, int b, int n, TreeSmem& sm) {
  const int i = threadIdx.x;
  bool ok = true;
  int p = -1, d = 0;
  uint32_t w[kTreeMax / 32];
#pragma unroll
  for (int x = 0; x < kTreeMax / 32; ++x) w[x] = i / 32 == x ? 1u << (i & 31) : 0u;
  if (!c.parents) {
    d = i;
#pragma unroll
    for (int x = 0; x < kTreeMax / 32; ++x)
      w[x] = i / 32 > x ? 0xFFFFFFFFu : i / 32 == x ? 0xFFFFFFFFu >> (31 - (i & 31)) : 0u;
  } else if (i < n) {
    p = __ldg(c.parents + static_cast<size_t>(b) * c.N + i);
    ok = p >= -1 && p < i;
    if (!ok) p = -1;
    d = p >= 0;
  }
  consumer_sync();  // the previous sequence's words are no longer read
  for (;;) {
    sm.jump[i] = p;
    sm.depth[i] = d;
    *reinterpret_cast<uint4*>(sm.seen[i]) = make_uint4(w[0], w[1], w[2], w[3]);
    if (!consumer_or(p >= 0)) break;
    int dp = 0, pp = -1;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (p >= 0) {
      dp = sm.depth[p];
      pp = sm.jump[p];
      v = *reinterpret_cast<const uint4*>(sm.seen[p]);
    }
    consumer_sync();
    d += dp;
    p = pp;
    w[0] |= v.x;
    w[1] |= v.y;
    w[2] |= v.z;
    w[3] |= v.w;
  }
  return ok;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ bool odd_exp(uint32_t half) { return (half & 0x7F80u) == 0x7F80u; }

// Floats of one head's table window for a tile and n nodes: 64 keys against
// n positions at most, from a 16-byte boundary.
__host__ __device__ __forceinline__ int window_floats(int n) {
  return (3 + kTreeTile + n - 1 + 3) & ~3;
}

// ---------------------------------------------------------------- attention

// A consumer warp holds 16 * MT rows of an item (row group warp % RG) and one
// of kConsumers / RG equal parts of the keys of every tile.  Its products are
// bf16 m16n8k16 with fp32 accumulators: S = Q K^T, the softmax on the
// accumulators, and O += P V with the weights as the next product's left
// operand, without leaving registers.  (Whole tiles dealt out to the warps in
// turn were slower, 915 against 746 us at B64 H12 N32 T32768: a slot of the
// ring may then serve one warp only, since a wait names a phase by its parity,
// and each warp had a single slot.)
//
// The running maximum is only raised when a logit exceeds it by more than 8
// (a weight is at most 2^8), so most tiles need no exchange between lanes.
// PARTS: bf16 parts of a weight in the product with V (1: its rounding, at
// most 2^-8 of the weight, is of the size of the output's own; 3: 24 bits).
template <int MT, int RG, int PARTS>
__global__ void __launch_bounds__(kTreeThreads, 2)
    bam_tree_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                    const TreeArgs a) {
  constexpr int kRows = 16 * MT * RG;
  constexpr int kStreams = kConsumers / RG;  // parts of a tile's keys
  constexpr int kKeys = kTreeTile / kStreams;
  constexpr int NT = kKeys < 32 ? kKeys / 8 : 4;  // 8-key column tiles of S at a time
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* const kv = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);  // [stages][K, V]
  float* const win = reinterpret_cast<float*>(kv + a.stages * 2 * kKvBytes);
  float* const merge = win + a.stages * a.win_stage;  // [streams][rows][kMergeStride]
  float2* const merge_ml = reinterpret_cast<float2*>(merge + kStreams * kRows * kMergeStride);
  TreeSmem& sm = *reinterpret_cast<TreeSmem*>(merge_ml + kStreams * kRows);
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* ab = &sm.abort_flag;

  if (threadIdx.x == 0) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], kConsumers);
    }
    fence_barrier_init();
    sm.find = 0;
  }
  grid_dep_wait();  // plan and table
  grid_dep_trigger();
  if (threadIdx.x == 0) sm.abort_flag = *reinterpret_cast<volatile int*>(&c.status->abort);
  const int64_t all = __ldcg(a.plan + c.B);
  const int active = active_ctas(all, a.ctas, a.least);
  const int cta = blockIdx.x;
  if (all == 0 || cta >= active) return;
  const int64_t beg = range_beg(all, active, cta), end = range_beg(all, active, cta + 1);
  __syncthreads();
  {
    int before = 0;
    for (int b = threadIdx.x; b < c.B; b += kTreeThreads) before += __ldcg(a.plan + b + 1) <= beg;
    if (before) atomicAdd(&sm.find, before);
  }
  __syncthreads();
  int b = sm.find;

  if (warp == kConsumers) {
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
          ok = mbar_wait(&sm.empty[s], phase, c.status, ab, kSiteTreeProducer);
          ok = __all_sync(0xffffffffu, ok);
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
      }
      x += it.t1 - it.t0;
    }
    // On the give-up path consumers may not have waited for every copy.
    if (!__all_sync(0xffffffffu, ok) || *ab) {
      for (int i = max(0, issued - a.stages); i < issued; ++i)
        mbar_drain(&sm.full[i % a.stages], (i / a.stages) & 1);
    }
    if (bad_page) record_bad_arg(c.status);
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int rg = warp % RG, stream = warp / RG;
  const int quad = lane & 3;
  const int key0 = stream * kKeys;  // first key of this warp in a tile
  int s = 0, phase = 0;
  bool ok = *ab == 0, args_ok = true;
  int last_b = -1;
  for (int64_t x = beg; x < end;) {
    const Item it = item_at(a, b, x, end);
    b = it.b;
    if (it.b != last_b) args_ok &= tree_seen(c, it.b, it.n, sm);
    last_b = it.b;
    const int n = it.n, len = it.len;
    const int r0 = it.rb * kRows, r1 = min(r0 + kRows, a.group * n);
    const int g0 = r0 / n;
    const int nwin = window_floats(n);
    const int rem = (a.tab_zero - (len + n - 1)) & 3;
    // This lane's rows: 2 of each 16.
    float cs[MT][2], m[MT][2], l[MT][2], o[MT][8][4];
    int woff[MT][2];
    uint32_t q[MT][4][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = r0 + 16 * (MT * rg + mt) + 8 * hf + (lane >> 2);
        const bool live = r < r1;
        const int g = live ? r / n : g0;
        const int t = live ? r - g * n : 0;
        const int pos = len + sm.depth[t];
        float cl = 0.125f;
        const int head = it.hk * a.group + g;
        if (a.ssmax) cl *= __ldg(a.s + head) * logf(static_cast<float>(pos + 1));
        cs[mt][hf] = cl * static_cast<float>(kLog2e);
        woff[mt][hf] = (g - g0) * nwin + rem + (len + n - 1 - pos) + 2 * quad;
        if (quad == 0 && stream == 0) {
          const int rr = 16 * (MT * rg + mt) + 8 * hf + (lane >> 2);
          sm.node[rr] = live ? t : -1;
          sm.head[rr] = head;
        }
        m[mt][hf] = kNoMax;
        l[mt][hf] = 0.0f;
        const uint32_t* qr = reinterpret_cast<const uint32_t*>(
            a.q + ((static_cast<size_t>(it.b) * a.H + head) * c.N + t) * kHeadDim);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          q[mt][kk][hf] = live ? __ldg(qr + 8 * kk + quad) : 0u;
          q[mt][kk][2 + hf] = live ? __ldg(qr + 8 * kk + 4 + quad) : 0u;
        }
      }
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.0f;
    }
    consumer_sync();  // rows' nodes and heads; the previous item's join is over
    const bool rows_live = r0 + 16 * MT * rg < r1;

    for (int t = it.t0; t < it.t1; ++t) {
      if (ok) ok = mbar_wait(&sm.full[s], phase, c.status, ab, kSiteTreeConsumer);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t ks = smem_u32(kv + s * 2 * kKvBytes), vs = ks + kKvBytes;
      const float* w = win + s * a.win_stage + key0;
      const int j0 = t * kTreeTile + key0;
      const bool tail = j0 + kKeys > len;  // holds keys that not every row sees
      bool odd = false;
#pragma unroll 1
      for (int ch = 0; rows_live && ch < kKeys / (8 * NT); ++ch) {
        float z[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[mt][nt][e] = 0.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            uint32_t kb[4];
            ldsm_x4(ks + (key0 + (ch * NT + nt) * 8 + (lane & 7)) * 128 +
                        (((4 * kk + (lane >> 3)) ^ (lane & 7)) << 4),
                    kb);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma_bf16(z[mt][nt], q[mt][2 * kk], kb);
              mma_bf16(z[mt][nt], q[mt][2 * kk + 1], kb + 2);
            }
          }
        }
        bool raise = false;
        if (!tail) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const float* wr = w + woff[mt][hf] + ch * NT * 8;
              float mx = kNoMax;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float& z0 = z[mt][nt][2 * hf];
                float& z1 = z[mt][nt][2 * hf + 1];
                z0 = fmaf(z0, cs[mt][hf], wr[8 * nt]);
                z1 = fmaf(z1, cs[mt][hf], wr[8 * nt + 1]);
                mx = fmax3(mx, z0, z1);
              }
              raise |= mx > m[mt][hf] + kRescale;
            }
          }
        } else {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int rr = 16 * (MT * rg + mt) + 8 * hf + (lane >> 2);
              const int nd = sm.node[rr];
              const float* wr = w + woff[mt][hf] + ch * NT * 8;
              // table entry of an ancestor at depth x: near + x
              const float* near = a.table + static_cast<size_t>(sm.head[rr]) * a.tab_len +
                                  a.tab_zero - (nd >= 0 ? sm.depth[nd] : 0);
              float mx = kNoMax;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float& zz = z[mt][nt][2 * hf + e];
                  const int j = j0 + (ch * NT + nt) * 8 + 2 * quad + e, i = j - len;
                  if (i < 0) {
                    zz = fmaf(zz, cs[mt][hf], wr[8 * nt + e]);
                  } else if (nd >= 0 && i < n && (sm.seen[nd][i >> 5] >> (i & 31) & 1)) {
                    zz = fmaf(zz, cs[mt][hf], __ldcg(near + sm.depth[i]));
                  } else {
                    zz = -INFINITY;
                  }
                  mx = fmaxf(mx, zz);
                }
              }
              raise |= mx > m[mt][hf] + kRescale;
            }
          }
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              float mx = kNoMax;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mx = fmax3(mx, z[mt][nt][2 * hf], z[mt][nt][2 * hf + 1]);
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
              if (mx > m[mt][hf]) {
                const float corr = ex2_approx(m[mt][hf] - mx);
                l[mt][hf] *= corr;
#pragma unroll
                for (int nt = 0; nt < 8; ++nt) {
                  o[mt][nt][2 * hf] *= corr;
                  o[mt][nt][2 * hf + 1] *= corr;
                }
                m[mt][hf] = mx;
              }
            }
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = ex2_approx(z[mt][nt][e] - m[mt][e >> 1]);
              z[mt][nt][e] = p;
              l[mt][e >> 1] += p;
            }
        // 16 keys at a time: two column tiles of S are the left operand.
#pragma unroll
        for (int k2 = 0; k2 < NT / 2; ++k2) {
          uint32_t pa[MT][PARTS][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float lo = z[mt][2 * k2 + (e >> 1)][2 * (e & 1)];
              float hi = z[mt][2 * k2 + (e >> 1)][2 * (e & 1) + 1];
#pragma unroll
              for (int part = 0; part < PARTS; ++part) {
                const uint32_t pk = pack_bf16x2(lo, hi);
                pa[mt][part][e] = pk;
                lo -= bf16_lo(pk);
                hi -= bf16_hi(pk);
              }
            }
          }
          const int kb = (ch * NT + 2 * k2) * 8;  // first key, from this warp's
#pragma unroll
          for (int dp = 0; dp < 4; ++dp) {
            uint32_t vb[4];
            ldsm_x4_t(vs + (key0 + kb + (lane & 15)) * 128 + (((2 * dp + (lane >> 4)) ^ (lane & 7)) << 4),
                      vb);
            if (tail) {
              // Rows behind the draft hold anything: zeros.  A drafted value
              // that is not finite is zero here (a weight of 0 would turn it
              // into NaN for the rows that do not see it) and is added below
              // to those that do.
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int i = j0 + kb + 8 * (y & 1) + 2 * quad - len;
                uint32_t keep = 0xFFFFFFFFu;
                if (i >= n || (i >= 0 && odd_exp(vb[y]))) keep &= 0xFFFF0000u;
                if (i + 1 >= n || (i + 1 >= 0 && odd_exp(vb[y] >> 16))) keep &= 0x0000FFFFu;
                odd |= (i >= 0 && i < n && !(keep & 1u)) || (i + 1 >= 0 && i + 1 < n && !(keep >> 31));
                vb[y] &= keep;
              }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
              for (int part = 0; part < PARTS; ++part) {
                mma_bf16(o[mt][2 * dp], pa[mt][part], vb);
                mma_bf16(o[mt][2 * dp + 1], pa[mt][part], vb + 2);
              }
            }
          }
        }
      }
      if (tail && __any_sync(0xffffffffu, odd)) {
        const uint8_t* vt = kv + s * 2 * kKvBytes + kKvBytes;
#pragma unroll 1
        for (int j = max(len, j0); j < min(len + n, j0 + kKeys); ++j) {
          const int row = j - t * kTreeTile, i = j - len;
#pragma unroll
          for (int nt = 0; nt < 8; ++nt) {
            const uint32_t v =
                *reinterpret_cast<const uint32_t*>(vt + row * 128 + ((nt ^ (row & 7)) << 4) + 4 * quad);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                const int nd = sm.node[16 * (MT * rg + mt) + 8 * hf + (lane >> 2)];
                if (nd >= 0 && (sm.seen[nd][i >> 5] >> (i & 31) & 1)) {
                  if (odd_exp(v)) o[mt][nt][2 * hf] += bf16_lo(v);
                  if (odd_exp(v >> 16)) o[mt][nt][2 * hf + 1] += bf16_hi(v);
                }
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[s]);
      if (++s == a.stages) {
        s = 0;
        phase ^= 1;
      }
    }

    // Join the parts of the keys in shared memory.  After a give-up the values mean
    // nothing, but every warp comes here for every item, so the barriers match.
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        l[mt][hf] += __shfl_xor_sync(0xffffffffu, l[mt][hf], 1);
        l[mt][hf] += __shfl_xor_sync(0xffffffffu, l[mt][hf], 2);
        const int rr = stream * kRows + 16 * (MT * rg + mt) + 8 * hf + (lane >> 2);
        if (quad == 0) merge_ml[rr] = make_float2(m[mt][hf], l[mt][hf]);
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
          *reinterpret_cast<float2*>(merge + rr * kMergeStride + 8 * nt + 2 * quad) =
              make_float2(o[mt][nt][2 * hf], o[mt][nt][2 * hf + 1]);
      }
    }
    consumer_sync();
    const bool whole = it.t0 == 0 && it.t1 == it.tiles;
    const int slot = 2 * cta + (it.t0 == 0 ? 1 : 0);
    for (int e = threadIdx.x; e < kRows * 16; e += 32 * kConsumers) {
      const int rr = e >> 4, col = (e & 15) * 4, r = r0 + rr;
      if (r >= r1) break;
      float M = kNoMax, L = 0.0f;
#pragma unroll
      for (int st = 0; st < kStreams; ++st) M = fmaxf(M, merge_ml[st * kRows + rr].x);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int st = 0; st < kStreams; ++st) {
        const float2 ml = merge_ml[st * kRows + rr];
        const float4 y = *reinterpret_cast<const float4*>(merge + (st * kRows + rr) * kMergeStride + col);
        const float f = ex2_approx(ml.x - M);
        L += ml.y * f;
        v.x += y.x * f;
        v.y += y.y * f;
        v.z += y.z * f;
        v.w += y.w * f;
      }
      if (whole) {
        const int g = r / n, nd = r - g * n;
        const size_t row = (static_cast<size_t>(it.b) * a.H + it.hk * a.group + g) * c.N + nd;
        v.x /= L;
        v.y /= L;
        v.z /= L;
        v.w /= L;
        if (PARTS > 1) {
          *reinterpret_cast<float4*>(static_cast<float*>(a.o) + row * kHeadDim + col) = v;
        } else {
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + row * kHeadDim + col) =
              make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
        if (a.lse && col == 0) a.lse[row] = (M + log2f(L)) * kLn2f;
      } else {
        const size_t row = static_cast<size_t>(slot) * kRows + rr;
        *reinterpret_cast<float4*>(a.part + row * kHeadDim + col) = v;
        if (col == 0) a.part_ml[row] = make_float2(M, L);
      }
    }
    x += it.t1 - it.t0;
  }
  if (!args_ok) record_bad_arg(c.status);
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
      float M = kNoMax, L = 0.0f;
      for (int x = c0 + lane; x <= c1; x += 32) M = fmaxf(M, __ldcg(a.part_ml + part_row(x)).x);
#pragma unroll
      for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      v = make_float2(0.0f, 0.0f);
#pragma unroll 4
      for (int x = c0; x <= c1; ++x) {
        const size_t pr = part_row(x);
        const float2 ml = __ldcg(a.part_ml + pr);
        const float2 y = __ldcg(reinterpret_cast<const float2*>(a.part + pr * kHeadDim) + lane);
        const float f = ex2_approx(ml.x - M);
        L += ml.y * f;
        v.x += y.x * f;
        v.y += y.y * f;
      }
      v.x /= L;
      v.y /= L;
      lse = (M + log2f(L)) * kLn2f;
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
size_t smem_fixed(int rows) {
  const int streams = rows <= 32 ? kConsumers : kConsumers * 32 / rows;
  return 1024 + static_cast<size_t>(streams) * rows * (kMergeStride * 4 + 8) + sizeof(TreeSmem);
}
size_t smem_stage(const TreeArgs& a) {
  return 2 * kKvBytes + static_cast<size_t>(a.win_stage) * 4;
}

template <int MT, int RG, int PARTS>
cudaError_t launch_rows(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a,
                        cudaStream_t st) {
  static bool limit_set[64] = {};
  auto kernel = bam_tree_kernel<MT, RG, PARTS>;
  const cudaError_t e = smem_limit_once(kernel, kSmemOne, limit_set);
  if (e != cudaSuccess) return e;
  return launch_k(kernel, dim3(a.ctas), dim3(kTreeThreads),
                  smem_fixed(a.rows) + a.stages * smem_stage(a), st, true, tk, tv, a);
}

template <int PARTS>
cudaError_t launch_parts(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a,
                         cudaStream_t st) {
  switch (a.rows) {
    case 16:
      return launch_rows<1, 1, PARTS>(tk, tv, a, st);
    case 32:
      return launch_rows<2, 1, PARTS>(tk, tv, a, st);
    case 64:
      return launch_rows<2, 2, PARTS>(tk, tv, a, st);
    default:
      return launch_rows<2, 4, PARTS>(tk, tv, a, st);
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
  const size_t fixed = smem_fixed(a->rows), stage = smem_stage(*a);
  int per_sm = 2;
  size_t budget = kSmemTwo;
  if (fixed + 3 * stage > budget) {
    per_sm = 1;
    budget = kSmemOne;
  }
  a->stages = static_cast<int>((budget - fixed) / stage);
  if (a->stages > kMaxStages) a->stages = kMaxStages;
  a->ctas = per_sm * sms < kTreeCtas ? per_sm * sms : kTreeCtas;
  a->least = 2;
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
