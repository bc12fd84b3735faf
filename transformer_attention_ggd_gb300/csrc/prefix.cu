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
// Warps 0-7: softmax, two threads a row (its lane of Tensor Memory), each with half of a tile's
// keys; they exchange their maxima.  Warp 8: K and V by TMA and the windows by
// asynchronous 16-byte copies, into a ring (a bulk copy per window took 4.4 us a tile).
// Warp 9, one thread: S = Q K^T (Q in Tensor Memory) and O += P V (P in Tensor Memory).
//
// With up to 64 rows a row stands in two or four lanes, each with its part of a tile's keys and
// zeros for the weights of the others.
#include "shared_common.cuh"

namespace bam {
namespace {

constexpr int kSoftWarps = 8;
constexpr int kCopyWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
constexpr int kThreads = 32 * (kSoftWarps + 2);
constexpr int kTile = 64;                      // keys
constexpr int kLanes = 128;
constexpr int kBoxBytes = kTile * kHeadDim * 2;
constexpr int kMaxStages = 5;
constexpr int kResident = 2;                   // CTAs of an SM
constexpr int kSmemMost = 111 * 1024;
constexpr float kRescale = 8.0f;               // log2 units by which a weight may exceed 1

// Tensor Memory columns: S, O, P (up to three parts), Q.
constexpr uint32_t kTmemCols = 256, kColS = 0, kColO = 64, kColP = 128, kColQ = 224;

enum : int {
  kSitePrefixProducer = 94,
  kSitePrefixQ = 95,
  kSitePrefixK = 96,
  kSitePrefixSFree = 97,
  kSitePrefixP = 98,
  kSitePrefixS = 99,
  kSitePrefixWin = 100,
  kSitePrefixPV = 101,
  kSitePrefixPair = 102,
  kSitePrefixTable = 103  // debug build: bounds of a copy of a window
};

template <int kCopies>
struct Shape {
  static constexpr int kWin = kTile / kCopies;       // keys of a lane in a tile
  static constexpr int kCols = kWin / 2;             // of a thread
  static constexpr int kRows = kLanes / kCopies;     // rows of an item
  static constexpr int kWinStride = kWin + 4;        // floats: 16-byte reads of eight rows hit all banks
  static constexpr int kWinBytes = kLanes * kWinStride * 4;
  // Rings: windows are free again when they have been read, K when S is there, V last.
  static constexpr int kWinStages = 2;
  static constexpr int kBoxes = (kSmemMost - kWinStages * kWinBytes) / kBoxBytes;
  static constexpr int kVStages = (kBoxes + 1) / 2 < kMaxStages ? (kBoxes + 1) / 2 : kMaxStages;
  static constexpr int kKStages = kBoxes / 2 < kMaxStages ? kBoxes / 2 : kMaxStages;
  static constexpr int kV = kKStages * kBoxBytes, kW = kV + kVStages * kBoxBytes;  // behind the K ring
  static constexpr int kSmem = kW + kWinStages * kWinBytes;
};

struct PrefixBars {
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t win_full[2], win_empty[2];
  uint64_t q_full, s_full, s_free, p_full, pv_done, final, pair[4];
  float max[2][2][kLanes];  // of a row's halves, by the tile's parity
  uint32_t win[kLanes];  // where each lane's window begins in the table, in 16-byte words
  uint32_t tmem;
  int abort_flag;
};

// 16 bytes global -> shared, asynchronously; arrive_copied: the barrier's phase also waits for this
// thread's copies so far (one of the arrivals that it counts).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_copied(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, DevStatus* st,
                                          volatile int* ab, int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, st, ab, site));
}

template <int kN>
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t* r) {
  if constexpr (kN == 32) tmem_ld_32x32b_x32(at, r);
  if constexpr (kN == 16) tmem_ld_32x32b_x16(at, r);
  if constexpr (kN == 8) tmem_ld_32x32b_x8(at, r);
  tmem_ld_wait();
  if constexpr (kN == 32) reg_fence32(r);
  if constexpr (kN == 16) reg_fence16(r);
  if constexpr (kN == 8) reg_fence8(r);
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

// kParts: bf16 parts of a weight.  O leaves the accumulator, which cuts off its last place in every
// step, after kFlush tiles (96 steps for fp32 output, 512 for bf16).
template <int kCopies, int kParts>
__global__ void __launch_bounds__(kThreads, kResident)
    bam_prefix_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                      const SharedArgs a) {
  using S = Shape<kCopies>;
  constexpr int kCols = S::kCols, kFlush = kParts == 3 ? 8 : 128;
  constexpr int kKStages = S::kKStages, kVStages = S::kVStages, kWinStages = S::kWinStages;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ PrefixBars bars;
  uint8_t* const ring = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
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
    for (int s = 0; s < kWinStages; ++s) {
      mbar_init(&bars.win_full[s], 32);
      mbar_init(&bars.win_empty[s], kSoftWarps);
    }
    mbar_init(&bars.q_full, kSoftWarps);
    mbar_init(&bars.s_full, 1);
    mbar_init(&bars.s_free, kSoftWarps);
    mbar_init(&bars.p_full, kSoftWarps);
    mbar_init(&bars.pv_done, 1);
    mbar_init(&bars.final, 1);
    for (int x = 0; x < 4; ++x) mbar_init(&bars.pair[x], 2);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars.tmem, kTmemCols);
    tmem_relinquish();
  }
  // A lane's row and window: it begins on a 16-byte boundary in the copy of the table that is
  // shifted by as much as is missing.
  const int ln = threadIdx.x % kLanes, half = threadIdx.x / kLanes, c = ln / S::kRows;
  const RowAt r = row_at(a, hk, row0 + ln % S::kRows);
  int pos = 0;
  if (warp < kSoftWarps) {
    pos = r.on ? query_pos(a, r.b, P, &ok_arg) : 0;
    const int y = a.tab_top - (r.on ? pos : max(P - 1, 0)) + kbeg + c * S::kWin, k = (4 - (y & 3)) & 3;
    bars.win[ln] = static_cast<uint32_t>((static_cast<int64_t>(k) * a.H + (r.on ? r.h : 0)) * (a.tab_len / 4) +
                                         (y + k) / 4);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;

  if (warp == kCopyWarp) {
    // ------------------------------------------------------------ copies
    constexpr int kChunks = S::kWin / 4, kStep = 32 / kChunks;  // 16-byte words of a window; windows at a time
    const int chunk = lane % kChunks;
    const uint4* src = reinterpret_cast<const uint4*>(a.table) + chunk;
    uint32_t win[kLanes / kStep];
#pragma unroll
    for (int x = 0; x < kLanes / kStep; ++x) win[x] = bars.win[lane / kChunks + kStep * x];
    const uint32_t dst = smem_u32(ring + S::kW) + 16 * chunk + lane / kChunks * S::kWinStride * 4;
    bool bad_page = false;
    int k_issued = 0, v_issued = 0, blk = kbeg / a.c.page, in = kbeg - blk * a.c.page;
    int next = tiles ? __ldg(a.prefix_table + blk) : 0;  // the next tile's page, on its way
    for (int it = 0; it < tiles; ++it) {
      const int ks = it % kKStages, vs = it % kVStages, s = it % kWinStages;
      if (it >= kKStages &&
          !warp_wait(&bars.k_empty[ks], (it / kKStages - 1) & 1, status, ab, kSitePrefixProducer))
        break;
      int pg = next;
      if (pg < 0 || pg >= a.c.num_pages) {
        bad_page = true;
        pg = 0;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars.k_full[ks], kBoxBytes);
        tma_load_3d(ring + ks * kBoxBytes, &tk, &bars.k_full[ks], 0, in, pg * a.c.Hkv + hk);
      }
      k_issued = it + 1;
      if (it >= kVStages &&
          !warp_wait(&bars.v_empty[vs], (it / kVStages - 1) & 1, status, ab, kSitePrefixProducer))
        break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars.v_full[vs], kBoxBytes);
        tma_load_3d(ring + S::kV + vs * kBoxBytes, &tv, &bars.v_full[vs], 0, in, pg * a.c.Hkv + hk);
      }
      v_issued = it + 1;
      in += kTile;
      if (in == a.c.page) {
        in = 0;
        if (it + 1 < tiles) next = __ldg(a.prefix_table + ++blk);
      }
      if (it >= kWinStages &&
          !warp_wait(&bars.win_empty[s], (it / kWinStages - 1) & 1, status, ab, kSitePrefixProducer))
        break;
      if (it == 0) {
        grid_dep_wait();  // the table, and the call's start
        grid_dep_trigger();
      }
      __syncwarp();
#pragma unroll
      for (int x = 0; x < kLanes / kStep; ++x) {
#ifdef BAM_DEBUG
        if (src + win[x] + 1 > reinterpret_cast<const uint4*>(a.table) + static_cast<int64_t>(a.H) * a.tab_len) {
          raise_error(status, ab, kSitePrefixTable, BAM_DEV_BOUNDS);
          continue;
        }
#endif
        copy16(dst + s * S::kWinBytes + x * kStep * S::kWinStride * 4, src + win[x]);
      }
      src += kTile / 4;
      arrive_copied(&bars.win_full[s]);
    }
    if (tiles == 0) {
      grid_dep_wait();
      grid_dep_trigger();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0) {
      for (int it = max(0, k_issued - kKStages); it < k_issued; ++it)
        mbar_drain(&bars.k_full[it % kKStages], (it / kKStages) & 1);
      for (int it = max(0, v_issued - kVStages); it < v_issued; ++it)
        mbar_drain(&bars.v_full[it % kVStages], (it / kVStages) & 1);
    }
    __syncwarp();
    if (bad_page) record_bad_arg(status);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      const uint32_t idS = idesc_bf16(kLanes, kTile, false, false);
      const uint32_t idO = idesc_bf16(kLanes, kHeadDim, false, true);
      auto issue_s = [&](int it) {
        const int s = it % kKStages;
        if (!mbar_wait(&bars.k_full[s], (it / kKStages) & 1, status, ab, kSitePrefixK)) return false;
        tc_fence_after();
        const uint64_t kd = sdesc_sw128(smem_u32(ring + s * kBoxBytes), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < kHeadDim / 16; ++kk)
          umma_ts(tmem + kColS, tmem + kColQ + 8 * kk, kd + 2 * kk, idS, kk > 0);
        umma_commit(&bars.s_full);
        umma_commit(&bars.k_empty[s]);
        return true;
      };
      bool ok = tiles == 0 || mbar_wait(&bars.q_full, 0, status, ab, kSitePrefixQ);
      tc_fence_after();
      if (ok && tiles) ok = issue_s(0);
      for (int it = 0; ok && it < tiles; ++it) {
        if (it + 1 < tiles) {
          ok = mbar_wait(&bars.s_free, it & 1, status, ab, kSitePrefixSFree);
          if (ok) ok = issue_s(it + 1);
          if (!ok) break;
        }
        const int s = it % kVStages;
        ok = mbar_wait(&bars.v_full[s], (it / kVStages) & 1, status, ab, kSitePrefixK) &&
             mbar_wait(&bars.p_full, it & 1, status, ab, kSitePrefixP);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = sdesc_sw128(smem_u32(ring + S::kV + s * kBoxBytes), 16384, 1024);
#pragma unroll
        for (int p = kParts - 1; p >= 0; --p)
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            umma_ts(tmem + kColO, tmem + kColP + 32 * p + 8 * kk, vd + 128 * kk, idO,
                    it % kFlush != 0 || p < kParts - 1 || kk > 0);
        umma_commit(&bars.pv_done);
        umma_commit(&bars.v_empty[s]);
      }
      // Every product is done before Tensor Memory is freed.
      umma_commit(&bars.final);
      mbar_drain(&bars.final, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int64_t row = static_cast<int64_t>(r.b) * a.H + r.h;
    const uint32_t tl = tmem + tmem_lane_base(warp);
    float cr = 0.0f;
    {
      uint32_t q[32];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint4 w = r.on ? __ldg(reinterpret_cast<const uint4*>(a.q + row * kHeadDim) + x)
                             : make_uint4(0, 0, 0, 0);
        q[4 * x] = w.x, q[4 * x + 1] = w.y, q[4 * x + 2] = w.z, q[4 * x + 3] = w.w;
      }
      if (half == 0) tmem_st_32x32b_x32(tl + kColQ, q);
      if (kCopies > 1 && half == 1) {  // weights of the other copies' keys
        uint32_t zero[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) zero[x] = 0;
#pragma unroll
        for (int p = 0; p < kParts; ++p) tmem_st_32x32b_x32(tl + kColP + 32 * p, zero);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.q_full);
      if (r.on) cr = shared_scale(a, r.h, pos);
    }
    const int64_t slot = row * a.slots + a.nsplit + sp * kCopies + c;
    float m = kNoMax, l = 0.0f, m_out = kNoMax;  // m_out: the maximum that what has left O is relative to
    bool first = true, ok = true;
    // Adds this half of O's columns to the row's partial output.
    auto flush = [&]() {
      float4* out = reinterpret_cast<float4*>(a.part + slot * kHeadDim) + 8 * half;
      const float f = ex2_approx(m_out - m);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t o[16];
        __syncwarp();
        tmem_ld<16>(tl + kColO + 32 * half + 16 * x, o);
        if (r.on) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float4 v = make_float4(__uint_as_float(o[4 * y]), __uint_as_float(o[4 * y + 1]),
                                   __uint_as_float(o[4 * y + 2]), __uint_as_float(o[4 * y + 3]));
            if (!first) {
              const float4 w = out[4 * x + y];
              v = make_float4(fmaf(w.x, f, v.x), fmaf(w.y, f, v.y), fmaf(w.z, f, v.z), fmaf(w.w, f, v.w));
            }
            out[4 * x + y] = v;
          }
        }
      }
      __syncwarp();
      m_out = m;
      first = false;
    };
    const int col = c * S::kWin + half * kCols;  // this thread's first key in a tile
    uint64_t* const pair = &bars.pair[warp & 3];
    const uint64_t cr2 = f2_pack(cr, cr);
    for (int it = 0; it < tiles; ++it) {
      const int s = it % kWinStages, vs = it % kVStages;
      ok = warp_wait(&bars.s_full, it & 1, status, ab, kSitePrefixS) &&
           warp_wait(&bars.win_full[s], (it / kWinStages) & 1, status, ab, kSitePrefixWin);
      if (!ok) break;
      tc_fence_after();
      uint64_t z[kCols / 2];
      {
        uint32_t sv[kCols];
        tmem_ld<kCols>(tl + kColS + col, sv);
        const float* win =
            reinterpret_cast<const float*>(ring + S::kW + s * S::kWinBytes) + ln * S::kWinStride + half * kCols;
#pragma unroll
        for (int x = 0; x < kCols / 2; x += 2) {
          uint64_t b0, b1;
          ld_f2x2(win + 2 * x, b0, b1);
          z[x] = ffma2(f2_pack(__uint_as_float(sv[2 * x]), __uint_as_float(sv[2 * x + 1])), cr2, b0);
          z[x + 1] = ffma2(f2_pack(__uint_as_float(sv[2 * x + 2]), __uint_as_float(sv[2 * x + 3])), cr2, b1);
        }
      }
      tc_fence_before();
      const int valid = kend - kbeg - it * kTile;  // keys of the tile
      if (valid < kTile) {
        // What lies behind the last key (anything) has no effect: weight 0 times 0.
        ok = warp_wait(&bars.v_full[vs], (it / kVStages) & 1, status, ab, kSitePrefixK);
        if (!ok) break;
        for (int y = threadIdx.x; y < (kTile - valid) * 8; y += 32 * kSoftWarps)
          *reinterpret_cast<uint4*>(ring + S::kV + vs * kBoxBytes + valid * 128 + 16 * y) =
              make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.s_free);
        mbar_arrive(&bars.win_empty[s]);
      }
      if (valid < kTile) {
        const int lim = valid - col;
#pragma unroll
        for (int x = 0; x < kCols / 2; ++x) {
          float z0, z1;
          f2_unpack(z[x], z0, z1);
          z[x] = f2_pack(2 * x < lim ? z0 : -INFINITY, 2 * x + 1 < lim ? z1 : -INFINITY);
        }
      }
      constexpr int kChains = kCols / 2 < 4 ? kCols / 2 : 4;
      float mq[kChains];
#pragma unroll
      for (int x = 0; x < kCols / 2; ++x) {
        float z0, z1;
        f2_unpack(z[x], z0, z1);
        mq[x % kChains] = x < kChains ? fmaxf(z0, z1) : fmax3(mq[x % kChains], z0, z1);
      }
      float mx = mq[0];
#pragma unroll
      for (int x = 1; x < kChains; ++x) mx = fmaxf(mx, mq[x]);
      // The row's maximum: of both halves.
      bars.max[it & 1][half][ln] = mx;
      __syncwarp();
      if (lane == 0) mbar_arrive(pair);
      ok = warp_wait(pair, it & 1, status, ab, kSitePrefixPair);
      if (!ok) break;
      mx = fmaxf(mx, bars.max[it & 1][half ^ 1][ln]);
      if (it > 0) {
        // P V of the last tile: it has read P, and O is at rest.
        ok = warp_wait(&bars.pv_done, (it - 1) & 1, status, ab, kSitePrefixPV);
        if (!ok) break;
        tc_fence_after();
      }
      const bool fresh = it % kFlush == 0;  // O starts anew with this tile
      if (fresh && it > 0) flush();
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
      constexpr int kStep = kCols / 2 < 8 ? kCols / 2 : 8;  // pairs at a time (4 or 8)
#pragma unroll
      for (int q = 0; q < kCols / 2; q += kStep) {
        uint32_t pk[kParts][kStep];
#pragma unroll
        for (int y = 0; y < kStep; ++y) {
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
          if constexpr (kStep == 8)
            tmem_st_32x32b_x8(tl + kColP + 32 * p + col / 2 + q, pk[p]);
          else
            tmem_st_32x32b_x4(tl + kColP + 32 * p + col / 2 + q, pk[p]);
      }
      {
        float s0, s1;
        f2_unpack(fadd2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      if (!fresh && __any_sync(0xffffffffu, grow)) {  // each half its columns of O
        uint32_t o[32];
        tmem_ld<32>(tl + kColO + 32 * half, o);
#pragma unroll
        for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * scale);
        tmem_st_32x32b_x32(tl + kColO + 32 * half, o);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.p_full);
    }
    if (ok && tiles) {
      ok = warp_wait(&bars.pv_done, (tiles - 1) & 1, status, ab, kSitePrefixPV);
      tc_fence_after();
      if (ok) flush();
    }
    if (ok) {
      // The row's sum: of both halves.
      if (half == 1) bars.max[tiles & 1][1][ln] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(pair);
      ok = warp_wait(pair, tiles & 1, status, ab, kSitePrefixPair);
      if (ok && r.on && half == 0) a.ml[slot] = make_float2(m, l + bars.max[tiles & 1][1][ln]);
    }
    if (!ok_arg) {
      grid_dep_wait();  // (the call's start clears what fresh memory held)
      record_bad_arg(status);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int kCopies, int kParts>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const SharedArgs& a, cudaStream_t st) {
  using S = Shape<kCopies>;
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
  constexpr int kItemCost = 8;
  const int64_t ctas = 152 * kResident, tiles = (Pmax + kTile - 1) / kTile;
  int64_t best = INT64_MAX;
  a->npsplit = 1;
  for (int64_t n = 1; n <= 2 * ctas && n * kLeastKeys < Pmax + kLeastKeys; ++n) {
    const int64_t cost = (base * n + ctas - 1) / ctas * ((tiles + n - 1) / n + kItemCost);
    if (cost < best) {
      best = cost;
      a->npsplit = static_cast<int>(n);
    }
  }
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
  return a.copies == 4   ? launch<4, 1>(tk, tv, a, st)
         : a.copies == 2 ? launch<2, 1>(tk, tv, a, st)
                         : launch<1, 1>(tk, tv, a, st);
}

}  // namespace bam
