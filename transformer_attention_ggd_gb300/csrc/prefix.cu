// Attention of all rows of a batch over a prefix that it shares, on sm_103a.
//
//   z[r, j] = c_r q_r . k_j + b_h(pos_r - j),   partial (max, sum, exp(z - max) V)
//
// The rows of a key head are the B * group (sequence, query head) pairs that read it, 128
// at a time; an item is such a block and a part of the prefix's keys, so that K and V
// are read once for 128 rows: 256 bytes a key against 256 flops a row and key, on
// tcgen05.  Rows stand at positions of their own, so that each has its own window of its
// head's table of biases: 4 bytes a row and key out of L2, staged with the keys.
//
// A tile of 64 keys is a chain of S = Q K^T, softmax, O += P V, each of which waits for the one
// before; so that a processor has more than one under way, its CTA takes a part's tiles in turn
// with three chains, each with a maximum, a sum and an O of its own, which are joined at the end.  A chain: four warps, a thread a row (its lane of Tensor Memory), which
// also copy their rows' windows; P lies over S, and the next S is issued right behind the
// product that reads P, so that one wait and one arrival a tile are all that a chain needs.
// One more warp copies K and V by TMA into rings, one issues the products.
//
// With up to 64 rows a row stands in two or four lanes, each with its part of a tile's keys and
// zeros for the weights of the others: 32 rows over 32768 keys of 12 heads take 33 us with four
// lanes a row, 40 with two, 63 with one; 64 rows 40 with two, 61 with one.
//
// The weights enter P V as sums of bf16 parts: three for fp32 output, two (16 bits, as for own keys) for bf16
// output.  One part, 8 bits, took 47.5 and 78.0 us where two take 49.0 and 81.4 (the cases below, bf16 output), and
// put a sequence's error down to how many others it shares the prefix with.
//
// Measured, of the whole call: 64 sequences, 12 heads, 32768 keys: 49 us, of it 29 in this kernel
// (100 MB at 3.5 TB/s); 256 sequences, 32 and 8 heads, 8111 keys: 81 us, of it 61 here, and with fp32 output 105
// and 86, with the tensor pipe busy for a fifth of it: the softmax of 128 rows is what lasts.  A tile takes
// 1.2 us a processor with fp32 output, with bf16 output and one part a weight 0.9; without the copies of the windows,
// which come at 5 TB/s out of L2 beside 2.5 TB/s of keys, the first call took 45 instead of 47, the second 47
// instead of 73 (one part) and 93 instead of 104 (fp32).  One chain a
// CTA and two CTAs a processor took 52 and 109 us.  The issuing thread is chosen by elect.sync: chosen
// by its lane it took 60 us where it took 51.
#include "shared_common.cuh"

namespace bam {
namespace {

constexpr int kTile = 64;                      // keys
constexpr int kLanes = 128;
constexpr int kBoxBytes = kTile * kHeadDim * 2, kQBytes = kLanes * kHeadDim * 2;
constexpr int kMaxStages = 8;
constexpr int kSmemMost = 224 * 1024;
constexpr int kChains = 3;                     // (four, with bf16 output: 50 us where three take 47)
constexpr int kSoft = 4 * kChains;             // their warps
constexpr int kThreads = 32 * (kSoft + 2);
constexpr int kOutStride = kHeadDim + 4;       // floats
constexpr float kRescale = 8.0f;               // log2 units by which a weight may exceed 1
constexpr uint32_t kTmemCols = 512;

enum : int {
  kSitePrefixProducer = 94,
  kSitePrefixQ = 95,
  kSitePrefixK = 96,
  kSitePrefixP = 98,
  kSitePrefixS = 99,
  kSitePrefixTable = 103  // debug build: bounds of a copy of a window
};

// kParts: bf16 parts of a weight.
template <int kCopies, int kParts>
struct Shape {
  static constexpr int kWin = kTile / kCopies;       // keys of a lane in a tile
  static constexpr int kRows = kLanes / kCopies;     // rows of an item
  static constexpr int kWinStride = kWin + 4;        // floats: 16-byte reads of eight rows hit all banks
  static constexpr int kWinBytes = kLanes * kWinStride * 4;
  // Columns of a chain: O, then S and, over it, P.
  static constexpr uint32_t kColS = kHeadDim, kChainCols = kHeadDim + (kParts == 3 ? 96 : 64);
  static_assert(kChains * kChainCols <= kTmemCols);
  // Shared memory: Q, rings of K and V, a window of each chain; in the end, outputs and their
  // maxima and sums.
  static constexpr int kBoxes = (kSmemMost - kQBytes - kChains * kWinBytes) / kBoxBytes;
  static constexpr int kVStages = (kBoxes + 1) / 2 < kMaxStages ? (kBoxes + 1) / 2 : kMaxStages;
  static constexpr int kKStages = kBoxes / 2 < kMaxStages ? kBoxes / 2 : kMaxStages;
  static constexpr int kK = kQBytes, kV = kK + kKStages * kBoxBytes, kW = kV + kVStages * kBoxBytes;
  static constexpr int kOutBytes = kChains * kLanes * kOutStride * 4, kMl = kOutBytes;
  static constexpr int kUsed = kW + kChains * kWinBytes, kEnd = kMl + kChains * kLanes * 8;
  static constexpr int kSmem = kUsed > kEnd ? kUsed : kEnd;
  static_assert(kSmem <= kSmemMost && kKStages >= kChains);
};
// O leaves the accumulator, which cuts off its last place in every step, after as many tiles (96
// steps for fp32 output, 512 for bf16).
__host__ __device__ constexpr int flush_tiles(bool fp32) { return fp32 ? 8 : 64; }

struct PrefixBars {
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t q_full, s_full[kChains], p_full[kChains], final;
  uint32_t win[kLanes];  // where each lane's window begins in the table, in 16-byte words
  uint32_t tmem;
  int abort_flag;
};

// 16 bytes global -> shared, asynchronously.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, DevStatus* st,
                                          volatile int* ab, int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, st, ab, site));
}

template <int kN>
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t* r) {
  if constexpr (kN == 32) tmem_ld_32x32b_x32(at, r);
  if constexpr (kN == 16) tmem_ld_32x32b_x16(at, r);
  tmem_ld_wait();
  if constexpr (kN == 32) reg_fence32(r);
  if constexpr (kN == 16) reg_fence16(r);
}
// Barrier of the softmax warps.
constexpr int kSoftBarrier = 1;
__device__ __forceinline__ void soft_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// A row of the item: query head h of sequence b, or none.
struct RowAt {
  bool on;
  int b, h;
};
__device__ __forceinline__ RowAt row_at(const SharedArgs& a, int hk, int64_t row) {
  RowAt r;
  r.on = row < static_cast<int64_t>(a.c.B) * a.group;
  r.b = r.on ? static_cast<int>(row / a.group) : 0;
  r.h = hk * a.group + (r.on ? static_cast<int>(row - static_cast<int64_t>(r.b) * a.group) : 0);
  return r;
}

// Where a tile's keys are: its page and place in it.
struct Walk {
  int blk, in, next;  // next: the page, on its way
  __device__ __forceinline__ Walk(const SharedArgs& a, int kbeg, int tiles)
      : blk(kbeg / a.c.page), in(kbeg - blk * a.c.page), next(tiles ? __ldg(a.prefix_table + blk) : 0) {}
  __device__ __forceinline__ void advance(const SharedArgs& a, bool more) {
    in += kTile;
    if (in == a.c.page) {
      in = 0;
      ++blk;
      if (more) next = __ldg(a.prefix_table + blk);
    }
  }
};

template <int kCopies, int kParts>
__global__ void __launch_bounds__(kThreads, 1)
    bam_prefix_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                      const SharedArgs a) {
  using S = Shape<kCopies, kParts>;
  constexpr int kFlush = flush_tiles(kParts == 3), kWin = S::kWin;
  constexpr int kKStages = S::kKStages, kVStages = S::kVStages;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ PrefixBars bars;
  uint8_t* const smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* ab = &bars.abort_flag;
  DevStatus* const status = a.c.status;

  // The item: a part of the keys of a block of rows of a key head.
  const int blocks = static_cast<int>((static_cast<int64_t>(a.c.B) * a.group + S::kRows - 1) / S::kRows);
  const int sp = blockIdx.x % a.npsplit;
  const int rb = blockIdx.x / a.npsplit % blocks, hk = blockIdx.x / a.npsplit / blocks;
  bool ok_arg = true;
  const int P = prefix_len(a, &ok_arg);
  const int chunk = part_keys(P, a.npsplit);
  const int kbeg = min(P, sp * chunk), kend = min(P, kbeg + chunk);
  const int tiles = (kend - kbeg + kTile - 1) / kTile;
  const int64_t row0 = static_cast<int64_t>(rb) * S::kRows;

  if (threadIdx.x == 0) {
    bars.abort_flag = 0;
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&bars.k_full[s], 1);
      mbar_init(&bars.k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&bars.v_full[s], 1);
      mbar_init(&bars.v_empty[s], 1);
    }
    for (int g = 0; g < kChains; ++g) {
      mbar_init(&bars.s_full[g], 1);
      mbar_init(&bars.p_full[g], 4);
    }
    mbar_init(&bars.q_full, 4);
    mbar_init(&bars.final, 1);
    fence_barrier_init();
  }
  if (warp == kSoft) {
    tmem_alloc(&bars.tmem, kTmemCols);
    tmem_relinquish();
  }
  // A lane's row and window: it begins on a 16-byte boundary in the copy of the table that is
  // shifted by as much as is missing.
  const int ln = threadIdx.x % kLanes, c = ln / S::kRows;
  const RowAt r = row_at(a, hk, row0 + ln % S::kRows);
  int pos = 0;
  if (warp < kSoft) {
    pos = r.on ? query_pos(a, r.b, P, &ok_arg) : 0;
    const int y = a.tab_top - (r.on ? pos : max(P - 1, 0)) + kbeg + c * kWin, k = (4 - (y & 3)) & 3;
    if (warp < 4)
      bars.win[ln] = static_cast<uint32_t>((static_cast<int64_t>(k) * a.H + (r.on ? r.h : 0)) * (a.tab_len / 4) +
                                           (y + k) / 4);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;

  if (warp == kSoft + 1) {
    // ------------------------------------------------------------ K and V, in the order of their use
    if (elect_one()) {
      bool bad_page = false, ok = true;
      int k_issued = 0, v_issued = 0;
      Walk kw(a, kbeg, tiles), vw(a, kbeg, tiles);
      auto load = [&](Walk& w, const CUtensorMap* map, uint64_t* full, uint8_t* dst, bool more) {
        int pg = w.next;
        if (pg < 0 || pg >= a.c.num_pages) {
          bad_page = true;
          pg = 0;
        }
        mbar_arrive_expect_tx(full, kBoxBytes);
        tma_load_3d(dst, map, full, 0, w.in, pg * a.c.Hkv + hk);
        w.advance(a, more);
      };
      for (int it = 0; ok && it < tiles + kChains - 1; ++it) {
        if (it < tiles) {
          const int s = it % kKStages;
          if (it >= kKStages)
            ok = mbar_wait(&bars.k_empty[s], (it / kKStages - 1) & 1, status, ab, kSitePrefixProducer);
          if (!ok) break;
          load(kw, &tk, &bars.k_full[s], smem + S::kK + s * kBoxBytes, it + 1 < tiles);
          k_issued = it + 1;
        }
        const int iv = it - (kChains - 1);
        if (iv >= 0) {
          const int s = iv % kVStages;
          if (iv >= kVStages)
            ok = mbar_wait(&bars.v_empty[s], (iv / kVStages - 1) & 1, status, ab, kSitePrefixProducer);
          if (!ok) break;
          load(vw, &tv, &bars.v_full[s], smem + S::kV + s * kBoxBytes, iv + 1 < tiles);
          v_issued = iv + 1;
        }
      }
      for (int it = max(0, k_issued - kKStages); it < k_issued; ++it)
        mbar_drain(&bars.k_full[it % kKStages], (it / kKStages) & 1);
      for (int it = max(0, v_issued - kVStages); it < v_issued; ++it)
        mbar_drain(&bars.v_full[it % kVStages], (it / kVStages) & 1);
      if (bad_page) {
        grid_dep_wait();  // (the call's start clears what fresh memory held)
        record_bad_arg(status);
      }
    }
    __syncwarp();
  } else if (warp == kSoft) {
    // ------------------------------------------------------------ products
    if (elect_one()) {
      const uint32_t idS = idesc_bf16(kLanes, kTile, false, false);
      const uint32_t idO = idesc_bf16(kLanes, kHeadDim, false, true);
      const uint64_t qd = sdesc_sw128(smem_u32(smem), 16, 1024);
      auto issue_s = [&](int it, uint32_t chain) {
        const int s = it % kKStages;
        if (!mbar_wait(&bars.k_full[s], (it / kKStages) & 1, status, ab, kSitePrefixK)) return false;
        tc_fence_after();
        const uint64_t kd = sdesc_sw128(smem_u32(smem + S::kK + s * kBoxBytes), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < kHeadDim / 16; ++kk)
          umma_ss(chain + S::kColS, qd + 2 * kk, kd + 2 * kk, idS, kk > 0);
        umma_commit(&bars.k_empty[s]);
        return true;
      };
      bool ok = tiles == 0 || mbar_wait(&bars.q_full, 0, status, ab, kSitePrefixQ);
      tc_fence_after();
      for (int g = 0; ok && g < min(kChains, tiles); ++g) {
        ok = issue_s(g, tmem + g * S::kChainCols);
        if (ok) umma_commit(&bars.s_full[g]);
      }
      int g = 0, n = 0;  // chain, and its tile
      for (int it = 0; ok && it < tiles; ++it) {
        const uint32_t chain = tmem + g * S::kChainCols;
        const int s = it % kVStages;
        ok = mbar_wait(&bars.v_full[s], (it / kVStages) & 1, status, ab, kSitePrefixK) &&
             mbar_wait(&bars.p_full[g], n & 1, status, ab, kSitePrefixP);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = sdesc_sw128(smem_u32(smem + S::kV + s * kBoxBytes), 16384, 1024);
#pragma unroll
        for (int p = kParts - 1; p >= 0; --p)
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            umma_ts(chain, chain + S::kColS + 32 * p + 8 * kk, vd + 128 * kk, idO,
                    n % kFlush != 0 || p < kParts - 1 || kk > 0);
        umma_commit(&bars.v_empty[s]);
        // (products of one thread and shape run in their order: P is read before S covers it)
        if (it + kChains < tiles) ok = issue_s(it + kChains, chain);
        if (ok) umma_commit(&bars.s_full[g]);
        if (++g == kChains) g = 0, ++n;
      }
      // Every product is done before Tensor Memory is freed.
      umma_commit(&bars.final);
      mbar_drain(&bars.final, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int g = warp / 4;
    const int64_t row = static_cast<int64_t>(r.b) * a.H + r.h;
    const uint32_t tl = tmem + tmem_lane_base(warp & 3) + g * S::kChainCols;
    if (g == 0) {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint4 w = r.on ? __ldg(reinterpret_cast<const uint4*>(a.q + row * kHeadDim) + x)
                             : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(smem + ln * 128 + 16 * (x ^ (ln & 7))) = w;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.q_full);
    }
    const float cr = r.on ? shared_scale(a, r.h, pos) : 0.0f;
    const uint64_t cr2 = f2_pack(cr, cr);
    float m = kNoMax, l = 0.0f, m_out = kNoMax;  // m_out: the maximum that what has left O is relative to
    bool ok = true;
    // What has left O, of this lane.
    float4* const spill =
        reinterpret_cast<float4*>(a.spill + (((row * a.npsplit + sp) * kChains + g) * kCopies + c) * kHeadDim);
    // O (behind a flush: and what left before), 16 columns at a time.
    auto take = [&](int x, bool more, float4* v) {
      uint32_t o[16];
      tmem_ld<16>(tl + 16 * x, o);
      const float f = ex2_approx(m_out - m);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        v[y] = make_float4(__uint_as_float(o[4 * y]), __uint_as_float(o[4 * y + 1]),
                           __uint_as_float(o[4 * y + 2]), __uint_as_float(o[4 * y + 3]));
        if (more && r.on) {
          const float4 w = spill[4 * x + y];
          v[y] = make_float4(fmaf(w.x, f, v[y].x), fmaf(w.y, f, v[y].y), fmaf(w.z, f, v[y].z),
                             fmaf(w.w, f, v[y].w));
        }
      }
    };
    float* const wins = reinterpret_cast<float*>(smem + S::kW + g * S::kWinBytes);
    constexpr int kChunks = kWin / 4, kStep = 32 / kChunks;  // 16-byte words of a window; windows at a time
    const uint4* const src = reinterpret_cast<const uint4*>(a.table) + lane % kChunks;
    const int first = 32 * (warp & 3) + lane / kChunks;
    const uint32_t dst = smem_u32(wins + first * S::kWinStride) + 16 * (lane % kChunks);
    auto windows = [&](int it) {  // of this warp's rows, for a tile
#pragma unroll
      for (int x = 0; x < kChunks; ++x) {
        const uint4* from = src + (bars.win[first + kStep * x] + it * (kTile / 4));
#ifdef BAM_DEBUG
        if (from + 1 > reinterpret_cast<const uint4*>(a.table) + static_cast<int64_t>(a.H) * a.tab_len) {
          raise_error(status, ab, kSitePrefixTable, BAM_DEV_BOUNDS);
          continue;
        }
#endif
        copy16(dst + x * kStep * S::kWinStride * 4, from);
      }
    };
    grid_dep_wait();  // the table, and the call's start
    if (threadIdx.x == 0) grid_dep_trigger();
    if (g < tiles) windows(g);
    int n = 0;
    for (int it = g; it < tiles; it += kChains, ++n) {
      copies_wait();
      // S; and P V of the chain's last tile: O is at rest.
      ok = warp_wait(&bars.s_full[g], n & 1, status, ab, kSitePrefixS);
      if (!ok) break;
      tc_fence_after();
      __syncwarp();  // (and the windows, copied by other lanes)
      constexpr int kLoad = kWin < 32 ? kWin : 32;
      uint64_t z[kWin / 2];
#pragma unroll
      for (int q = 0; q < kWin; q += kLoad) {
        uint32_t sv[kLoad];
        tmem_ld<kLoad>(tl + S::kColS + c * kWin + q, sv);
        const float* win = wins + ln * S::kWinStride + q;
#pragma unroll
        for (int x = 0; x < kLoad / 2; x += 2) {
          uint64_t b0, b1;
          ld_f2x2(win + 2 * x, b0, b1);
          z[q / 2 + x] =
              ffma2(f2_pack(__uint_as_float(sv[2 * x]), __uint_as_float(sv[2 * x + 1])), cr2, b0);
          z[q / 2 + x + 1] =
              ffma2(f2_pack(__uint_as_float(sv[2 * x + 2]), __uint_as_float(sv[2 * x + 3])), cr2, b1);
        }
      }
      __syncwarp();
      const int valid = kend - kbeg - it * kTile;  // keys of the tile
      if (valid < kTile) {
        // What lies behind the last key (anything) has no effect: weight 0 times 0.
        const int vs = it % kVStages;
        ok = warp_wait(&bars.v_full[vs], (it / kVStages) & 1, status, ab, kSitePrefixK);
        if (!ok) break;
        for (int y = ln; y < (kTile - valid) * 8; y += kLanes)
          *reinterpret_cast<uint4*>(smem + S::kV + vs * kBoxBytes + valid * 128 + 16 * y) =
              make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        const int lim = valid - c * kWin;
#pragma unroll
        for (int x = 0; x < kWin / 2; ++x) {
          float z0, z1;
          f2_unpack(z[x], z0, z1);
          z[x] = f2_pack(2 * x < lim ? z0 : -INFINITY, 2 * x + 1 < lim ? z1 : -INFINITY);
        }
      }
      float mq[4];
#pragma unroll
      for (int x = 0; x < kWin / 2; ++x) {
        float z0, z1;
        f2_unpack(z[x], z0, z1);
        mq[x % 4] = x < 4 ? fmaxf(z0, z1) : fmax3(mq[x % 4], z0, z1);
      }
      const float mx = fmax3(fmaxf(mq[0], mq[1]), mq[2], mq[3]);
      const bool fresh = n % kFlush == 0;  // O starts anew with this tile
      if (fresh && n > 0) {
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          float4 v[4];
          __syncwarp();
          take(x, n > kFlush, v);
          if (r.on)
#pragma unroll
            for (int y = 0; y < 4; ++y) spill[4 * x + y] = v[y];
        }
        __syncwarp();
        m_out = m;
      }
      const bool grow = mx > m + kRescale;
      float scale = 1.0f;
      if (grow) {
        scale = ex2_approx(m - mx);
        l *= scale;
        m = mx;
      }
      const uint64_t negm2 = f2_pack(-m, -m);
      const uint64_t minus = f2_pack(-1.0f, -1.0f);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int q = 0; q < kWin / 2; q += 8) {  // pairs
        uint32_t pk[kParts][8];
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          float p0, p1;
          f2_unpack(fadd2(z[q + y], negm2), p0, p1);
          p0 = ex2_approx(p0);
          p1 = ex2_approx(p1);
          sum[y & 1] = fadd2(sum[y & 1], f2_pack(p0, p1));
          // Each part is the rounding of what the last left.
          uint64_t left = f2_pack(p0, p1);
#pragma unroll
          for (int p = 0; p < kParts; ++p) {
            const uint32_t w = pack_bf16x2(p0, p1);
            pk[p][y] = w;
            if (p + 1 < kParts) {
              left = ffma2(f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)), minus, left);
              f2_unpack(left, p0, p1);
            }
          }
        }
#pragma unroll
        for (int p = 0; p < kParts; ++p)
          tmem_st_32x32b_x8(tl + S::kColS + 32 * p + c * (kWin / 2) + q, pk[p]);
      }
      if (kCopies > 1) {  // the other copies' keys
        const uint32_t zero[8] = {};
#pragma unroll
        for (int x = 1; x < kCopies; ++x)
#pragma unroll
          for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int q = 0; q < kWin / 2; q += 8)
              tmem_st_32x32b_x8(tl + S::kColS + 32 * p + (c + x) % kCopies * (kWin / 2) + q, zero);
      }
      {
        float s0, s1;
        f2_unpack(fadd2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      if (!fresh && __any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t o[32];
          tmem_ld<32>(tl + 32 * x, o);
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * scale);
          tmem_st_32x32b_x32(tl + 32 * x, o);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.p_full[g]);
      if (it + kChains < tiles) windows(it + kChains);
    }
    // All chains are done: nothing reads Q and the rings any more, and outputs take their place.
    if (ok && n) {
      ok = warp_wait(&bars.s_full[g], n & 1, status, ab, kSitePrefixS);
      tc_fence_after();
    }
    copies_wait();
    soft_sync(kSoftBarrier, 32 * kSoft);
    float* const out = reinterpret_cast<float*>(smem);
    float2* const ml = reinterpret_cast<float2*>(smem + S::kMl);
    if (ok) {
      ml[g * kLanes + ln] = make_float2(m, l);
      if (n)
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          float4 v[4];
          __syncwarp();
          take(x, n > kFlush, v);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            *reinterpret_cast<float4*>(out + (g * kLanes + ln) * kOutStride + 16 * x + 4 * y) = v[y];
        }
    }
    soft_sync(kSoftBarrier, 32 * kSoft);
    if (ok) {
      for (int i = threadIdx.x; i < S::kRows * (kHeadDim / 4); i += 32 * kSoft) {
        const int lr = i / (kHeadDim / 4), x = i % (kHeadDim / 4);
        const RowAt ro = row_at(a, hk, row0 + lr);
        if (!ro.on) break;
        float M = kNoMax, L = 0.0f;
#pragma unroll
        for (int y = 0; y < kChains * kCopies; ++y) M = fmaxf(M, ml[y * S::kRows + lr].x);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int y = 0; y < kChains * kCopies; ++y) {
          const float2 w = ml[y * S::kRows + lr];
          if (w.y == 0.0f) continue;  // no key, or no weight: nothing is there
          const float f = ex2_approx(w.x - M);
          const float4 v = *reinterpret_cast<const float4*>(out + (y * S::kRows + lr) * kOutStride + 4 * x);
          L = fmaf(w.y, f, L);
          o = make_float4(fmaf(v.x, f, o.x), fmaf(v.y, f, o.y), fmaf(v.z, f, o.z), fmaf(v.w, f, o.w));
        }
        const int64_t slot = (static_cast<int64_t>(ro.b) * a.H + ro.h) * a.slots + a.nsplit + sp;
        reinterpret_cast<float4*>(a.part + slot * kHeadDim)[x] = o;
        if (x == 0) a.ml[slot] = make_float2(M, L);
      }
    }
    if (!ok_arg) record_bad_arg(status);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoft) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int kCopies, int kParts>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const SharedArgs& a, cudaStream_t st) {
  using S = Shape<kCopies, kParts>;
  const int64_t blocks = (static_cast<int64_t>(a.c.B) * a.group + S::kRows - 1) / S::kRows;
  const int64_t items = blocks * a.c.Hkv * a.npsplit;
  if (items > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const size_t smem = S::kSmem + 1024;
  static bool limit_set[64] = {};
  const cudaError_t e = smem_limit_once(bam_prefix_kernel<kCopies, kParts>, smem, limit_set);
  if (e != cudaSuccess) return e;
  return launch_k(bam_prefix_kernel<kCopies, kParts>, dim3(static_cast<unsigned>(items)), dim3(kThreads),
                  smem, st, true, tk, tv, a);
}

}  // namespace

void prefix_split(SharedArgs* a, int64_t Pmax, int64_t Tmax) {
  const int64_t rows = static_cast<int64_t>(a->c.B) * a->group;
  a->copies = rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
  const int64_t base = (rows * a->copies + kLanes - 1) / kLanes * a->c.Hkv;
  // The parts that end first, if an item's start and end cost as much as kItemCost tiles.
  constexpr int kItemCost = 8;  // (4 to 28 measured the same)
  const int64_t ctas = 152, tiles = (Pmax + kTile - 1) / kTile;
  int64_t best = INT64_MAX;
  a->npsplit = 1;
  for (int64_t n = 1; n <= 2 * ctas && n * kLeastKeys < Pmax + kLeastKeys; ++n) {
    const int64_t cost = (base * n + ctas - 1) / ctas * ((tiles + n - 1) / n + kItemCost);
    if (cost < best) {
      best = cost;
      a->npsplit = static_cast<int>(n);
    }
  }
  // (of either output: the workspace is one size)
  a->spills = part_keys(static_cast<int>(Pmax), a->npsplit) > flush_tiles(true) * kChains * kTile
                  ? a->npsplit * kChains * a->copies
                  : 0;
  // Distances of the prefix's keys, and behind them windows that reach past the last key.
  const int64_t top = a->max_pos > 0 ? (a->max_pos > Pmax ? a->max_pos : Pmax) : Pmax + Tmax;
  a->tab_top = static_cast<int>(top - 1);
  a->tab_len = static_cast<int>((top + kTile + 8 + 63) / 64 * 64);
}

cudaError_t launch_prefix(const CUtensorMap& tk, const CUtensorMap& tv, const SharedArgs& a,
                          cudaStream_t st) {
  if (a.o_fp32)
    return a.copies == 4   ? launch<4, 3>(tk, tv, a, st)
           : a.copies == 2 ? launch<2, 3>(tk, tv, a, st)
                           : launch<1, 3>(tk, tv, a, st);
  return a.copies == 4   ? launch<4, 2>(tk, tv, a, st)
         : a.copies == 2 ? launch<2, 2>(tk, tv, a, st)
                         : launch<1, 2>(tk, tv, a, st);
}

}  // namespace bam
