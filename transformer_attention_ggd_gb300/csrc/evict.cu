// Eviction from a paged cache: of each sequence and key head the first keys, the
// last ones and, of the rest, those of the largest accumulated weight stay, in
// order.
//
// It reads the weights once (4 bytes a key) and moves the keys, values, positions
// and weights that stay (264 bytes a key, read and written): bound by HBM, with
// the choice of the keys before it.
//
// Choice: the weight of the last key that stays is found digit by digit (11, 11
// and 10 bits, from the highest) in histograms of the weights, which stay in shared
// memory; keys of exactly that weight stay from the lowest slot on.  Then every warp
// counts what it keeps of a run of slots, and writes their rows behind what the
// warps before it keep.  Long sequences are dealt to a cluster of CTAs, a run of slots each.
//
// Measured: 64 sequences, 12 heads, 4352 -> 4096 keys, to other pages: 290 us, of which 25 for
// the choice (1.66 GB moved at 6.3 TB/s); one sequence, 12 heads, 131072 -> 65536: 104 us, 33 for the
// choice, which is a chain of latencies: three digits of 5 us, each of a histogram and two meetings
// of the cluster; 8 sequences of 600 -> 512: 10 us, two kernels of dependent steps.  In place, where keys
// in front of the first that leaves stay where they are: 309 us with weights that all differ (94% of the rows
// kept move: 1.5 GB), 125 where the ones that leave have equal weights and lie at the end (30%), 134 for the long
// sequence (all), 18 for the small ones.
#include "shared_common.cuh"

namespace bam {
namespace {

// Threads of a selecting CTA for short runs of slots and for long ones (96 CTAs with 16384 each take
// 48 us with the few, 33 with the many; 768 with 4352 each 25 and 36).
constexpr int kSelFew = 256, kSelMany = 512;
constexpr int kSelRun = 8192;                       // slots, at most, for the few
constexpr int kSelPer = 4;                          // slots of a thread in a chunk
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kCacheMost = 40960;                   // weights in shared memory, at most
constexpr int kSlotsCta = 4096;                     // of a CTA of a cluster, at least
constexpr int kMoveRows = 8;                        // rows of a thread in a wave

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The int at `p` of this CTA's shared memory in CTA `rank` of the cluster.
__device__ __forceinline__ int cluster_load(const int* p, int rank) {
  uint32_t at;
  int x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}

__device__ __forceinline__ int4 cluster_load4(const int* p, int rank) {
  uint32_t at;
  int4 x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(at)
               : "memory");
  return x;
}

// Order of the weights as unsigned numbers: NaN above everything, -0 as 0.
__device__ __forceinline__ uint32_t weight_order(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t x = __float_as_uint(w + 0.0f);
  return x & 0x80000000u ? ~x : x | 0x80000000u;
}

// Exclusive prefix sums over the block.
template <int kSelThreads>
__device__ __forceinline__ int block_scan(int x, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w)
    if (w < warp) before += warp_sums[w];
  __syncthreads();
  return before + s - x;
}

// A cluster chooses the keys of a sequence and key head.
template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, 1280 / kSelThreads) bam_kv_evict_select_kernel(const EvictArgs a) {
  constexpr int kSelChunk = kSelThreads * kSelPer, kSelWarps = kSelThreads / 32;
  constexpr int kSelAhead = kSelThreads == kSelFew ? 2 : 4;  // chunks whose weights are on their way
  constexpr int kBinThreads = kSelThreads < kBins / 4 ? kSelThreads : kBins / 4;
  constexpr int kThreadBins = kBins / kBinThreads;  // in fours
  extern __shared__ __align__(16) uint32_t cache[];  // orders of this CTA's weights
  __shared__ __align__(16) int hist[kBins];
  __shared__ int warp_sums[kSelWarps];
  __shared__ int2 kept_by[kSelWarps];
  __shared__ int s_bin, s_need, s_over, s_ties, s_first;
  grid_dep_trigger();
  const CacheArgs& c = a.c;
  const int rank = blockIdx.x % a.cluster, hk = blockIdx.x / a.cluster, b = blockIdx.y;
  const int cap = c.page * c.max_blocks, raw = __ldg(c.lens + b);
  const int len = min(max(raw, 0), cap), kept = min(len, a.budget);
  const int* table = c.block_table + static_cast<size_t>(b) * c.max_blocks;
  const int* out = a.out_table ? a.out_table + static_cast<size_t>(b) * a.out_blocks : nullptr;
  // Pages of all used blocks, by every CTA: all of a sequence's CTAs decide alike.
  bool pages_ok = true;
  const int blocks = static_cast<int>(divide(len + c.page - 1, a.by_page));
  const int out_blocks = out ? static_cast<int>(divide(kept + c.page - 1, a.by_page)) : 0;
  for (int i = threadIdx.x; i < blocks + out_blocks; i += kSelThreads) {
    const int pg = __ldg(i < blocks ? table + i : out + (i - blocks));
    pages_ok &= pg >= 0 && pg < c.num_pages;
  }
  pages_ok = __syncthreads_and(pages_ok);
  const int64_t head = static_cast<int64_t>(b) * c.Hkv + hk;
  if (threadIdx.x == 0 && rank == 0 && !(raw == len && pages_ok)) record_bad_arg(c.status);
  unsigned* list = a.list + head * a.budget;
  // Row of a slot in the pages.
  auto row_of = [&](int slot) {
    const unsigned blk = divide(slot, a.by_page);
    return (static_cast<unsigned>(__ldg(table + blk)) * c.Hkv + hk) * c.page + (slot - blk * c.page);
  };
  if (!pages_ok || len <= a.budget) {  // (the same in every CTA of the cluster)
    if (threadIdx.x == 0 && rank == 0) a.count[head] = make_int2(pages_ok ? len : -1 - len, out ? 0 : len);
    if (pages_ok && out)
      for (int i = rank * kSelThreads + threadIdx.x; i < len; i += a.cluster * kSelThreads) list[i] = row_of(i);
    return;
  }
  // This CTA's slots: a run of whole fours.
  const int per = ((len + a.cluster - 1) / a.cluster + kSelPer - 1) / kSelPer * kSelPer;
  const int begin = min(len, rank * per), end = min(len, begin + per);
  const int lo = a.sink, hi = len - a.recent;   // the candidates
  const int inner = min(hi, end);               // end of those of this CTA
  int need = a.budget - a.sink - a.recent;      // of them
  // Orders of four slots from i on, which lie in one page.
  auto orders_of = [](const float4& f) {
    return make_uint4(weight_order(f.x), weight_order(f.y), weight_order(f.z), weight_order(f.w));
  };
  auto orders = [&](int i) {
    return i - begin < a.cached ? *reinterpret_cast<const uint4*>(cache + (i - begin))
                                : orders_of(*reinterpret_cast<const float4*>(a.key_weight + row_of(i)));
  };
  uint32_t threshold = 0;
  int shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3 && need > 0; ++pass) {
    const int bits = pass < 2 ? 11 : 10, up = shift;  // bits above `up` are known
    shift -= bits;
    for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    auto add = [&](int i, const uint4& q) {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      const bool all = i >= lo && i + 4 <= inner;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (!all && (i + x < lo || i + x >= inner)) continue;
        if (pass > 0 && ((w[x] ^ threshold) >> up) != 0) continue;
        atomicAdd(&hist[(w[x] >> shift) & ((1 << bits) - 1)], 1);
      }
    };
    if (pass == 0) {
      // The weights, some on their way at a time.
      for (int i = begin + kSelPer * threadIdx.x; i < end; i += kSelAhead * kSelChunk) {
        float4 f[kSelAhead];
#pragma unroll
        for (int y = 0; y < kSelAhead; ++y)
          if (i + y * kSelChunk < end)
            f[y] = *reinterpret_cast<const float4*>(a.key_weight + row_of(i + y * kSelChunk));
#pragma unroll
        for (int y = 0; y < kSelAhead; ++y) {
          const int j = i + y * kSelChunk;
          if (j >= end) break;
          const uint4 w = orders_of(f[y]);
          if (j - begin < a.cached) *reinterpret_cast<uint4*>(cache + (j - begin)) = w;
          add(j, w);
        }
      }
    } else {
      for (int i = begin + kSelPer * threadIdx.x; i < end; i += kSelChunk) add(i, orders(i));
    }
    if (a.cluster > 1)
      cluster_sync();
    else
      __syncthreads();
    // Thread 0 has the highest bins.
    int n[kThreadBins], sum = 0;  // from the highest on
    const int top = kBins - kThreadBins * static_cast<int>(threadIdx.x + 1);
#pragma unroll
    for (int x = 0; x < kThreadBins; x += 4) {
      n[x] = n[x + 1] = n[x + 2] = n[x + 3] = 0;
      if (top < 0) continue;
      const int* p = hist + top + kThreadBins - 4 - x;
      int4 v = *reinterpret_cast<const int4*>(p);
      if (a.cluster > 1) {
        int4 y[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          y[r] = r < a.cluster ? cluster_load4(p, r) : make_int4(0, 0, 0, 0);
        v = make_int4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) v.x += y[r].x, v.y += y[r].y, v.z += y[r].z, v.w += y[r].w;
      }
      n[x] = v.w, n[x + 1] = v.z, n[x + 2] = v.y, n[x + 3] = v.x;
      sum += v.x + v.y + v.z + v.w;
    }
    int above = block_scan<kSelThreads>(sum, warp_sums);
#pragma unroll
    for (int x = 0; x < kThreadBins; ++x) {
      if (above < need && need <= above + n[x]) {
        s_bin = top + kThreadBins - 1 - x;
        s_need = need - above;
      }
      above += n[x];
    }
    if (a.cluster > 1)
      cluster_sync();  // (the histograms are no longer read)
    else
      __syncthreads();
    threshold |= static_cast<uint32_t>(s_bin) << shift;
    need = s_need;
    __syncthreads();
  }
  // `need` of the keys whose weight is the threshold stay, the lowest slots first (none of the
  // candidates if none is needed).
  const bool any = a.budget > a.sink + a.recent;
  auto classify = [&](int i0, bool (&over)[kSelPer], bool (&tie)[kSelPer]) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (i0 < end && any) q = orders(i0);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const bool all = i0 >= lo && i0 + kSelPer <= inner && any;
#pragma unroll
    for (int x = 0; x < kSelPer; ++x) {
      const int i = i0 + x;
      over[x] = w[x] > threshold;
      tie[x] = w[x] == threshold;
      if (!all) {
        const bool in = i < end, candidate = in && i >= lo && i < hi;
        over[x] = in && (!candidate || (any && over[x]));
        tie[x] = candidate && any && tie[x];
      }
    }
  };
  // Each warp has a run of slots; what is kept before it is counted first.
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int run = ((per + kSelWarps - 1) / kSelWarps + 127) / 128 * 128;
  const int wbegin = min(end, begin + warp * run), wend = min(end, wbegin + run);
  int at = 0, ties = 0;
  {
    int n = 0, t = 0;
    for (int i0 = wbegin + kSelPer * lane; i0 < wend; i0 += 32 * kSelPer) {
      bool over[kSelPer], tie[kSelPer];
      classify(i0, over, tie);
#pragma unroll
      for (int x = 0; x < kSelPer; ++x) n += over[x], t += tie[x];
    }
    n = __reduce_add_sync(0xffffffffu, n);
    t = __reduce_add_sync(0xffffffffu, t);
    if (lane == 0) kept_by[warp] = make_int2(n, t);
    if (threadIdx.x == 0) s_first = len;
    __syncthreads();
    n = t = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      const int2 k = kept_by[w];
      if (w < warp) at += k.x, ties += k.y;
      n += k.x, t += k.y;
    }
    if (a.cluster > 1) {
      if (threadIdx.x == 0) s_over = n, s_ties = t;
      cluster_sync();
      const bool before = lane < rank;
      at += __reduce_add_sync(0xffffffffu, before ? cluster_load(&s_over, lane) : 0);
      ties += __reduce_add_sync(0xffffffffu, before ? cluster_load(&s_ties, lane) : 0);
    }
  }
  int first = len;
  for (int base = wbegin; base < wend; base += 32 * kSelPer) {
    const int i0 = base + lane * kSelPer;
    bool over[kSelPer], tie[kSelPer];
    classify(i0, over, tie);
    int n = 0;  // of both, 16 bits each
#pragma unroll
    for (int x = 0; x < kSelPer; ++x) n += over[x] + (tie[x] << 16);
    int scan = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, scan, d);
      if (lane >= d) scan += y;
    }
    const int total = __shfl_sync(0xffffffffu, scan, 31);
    scan -= n;
    int tie_rank = ties + (scan >> 16);
    int dst = at + (scan & 0xFFFF) + min(tie_rank, need);
    if (n > 0) {
      const unsigned row = row_of(i0);
#pragma unroll
      for (int x = 0; x < kSelPer; ++x) {
        const bool keep = over[x] || (tie[x] && tie_rank < need);
        tie_rank += tie[x];
        if (keep) {
          if (dst != i0 + x && first == len) first = dst;
          list[dst++] = row + x;
        }
      }
    }
    at += total & 0xFFFF;
    ties += total >> 16;
  }
  // The first key that moves.
  __syncthreads();
  if (first < len) atomicMin(&s_first, first);
  if (a.cluster > 1)
    cluster_sync();
  else
    __syncthreads();
  if (threadIdx.x == 0 && rank == 0) {
    int f = s_first;
    for (int r = 1; r < a.cluster; ++r) f = min(f, cluster_load(&s_first, r));
    a.count[head] = make_int2(kept, out ? 0 : min(f, kept));
  }
  if (a.cluster > 1) cluster_sync();  // (no CTA ends while another reads it)
}

// CTAs move the keys (z 0) or the values (z 1) of one sequence and key head.  In place they
// are a cluster and go in waves: every CTA reads its rows of the wave, the
// cluster meets, and they are written.  Row m goes from a slot >= m to slot m, so
// that a row that is written was the source of an earlier row, if of any, which has
// been read.  The numbers of the next wave's rows are on their way meanwhile; the rows
// themselves are read behind this wave's writes.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) bam_kv_evict_move_kernel(const EvictArgs a) {
  constexpr int kStep = kThreads / 8, kWave = kStep * kMoveRows;  // eight lanes a row
  grid_dep_wait();
  const CacheArgs& c = a.c;
  const int rank = blockIdx.x % a.cluster, hk = blockIdx.x / a.cluster, b = blockIdx.y;
  const bool values = blockIdx.z;
  const int64_t head = static_cast<int64_t>(b) * c.Hkv + hk;
  const int2 cnt = a.count[head];
  if (blockIdx.x == 0 && !values && threadIdx.x == 0) a.new_lens[b] = cnt.x >= 0 ? cnt.x : -1 - cnt.x;
  const int* table = a.out_table ? a.out_table + static_cast<size_t>(b) * a.out_blocks
                                 : c.block_table + static_cast<size_t>(b) * c.max_blocks;
  const unsigned* list = a.list + head * a.budget;
  uint4* pool = reinterpret_cast<uint4*>(values ? a.v_pages : a.k_pages);
  uint32_t* side = values ? reinterpret_cast<uint32_t*>(a.key_weight) : reinterpret_cast<uint32_t*>(a.key_pos);
  const int u = threadIdx.x & 7, n = cnt.x, step = kWave * a.cluster;
  uint4 w[kMoveRows];
  uint32_t mark[kMoveRows];
  unsigned src[kMoveRows];
  auto fetch = [&](int64_t m) {  // rows' places
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) src[x] = m + x * kStep < n ? __ldg(list + m + x * kStep) : 0;
  };
  int64_t m0 = cnt.y + static_cast<int64_t>(rank) * kWave + (threadIdx.x >> 3);
  fetch(m0);
  // (every CTA of a cluster goes through as many waves)
  for (int64_t wave = cnt.y; wave < n; wave += step, m0 += step) {
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) {
      if (m0 + x * kStep >= n) break;
      w[x] = pool[static_cast<int64_t>(src[x]) * 8 + u];
      if (u == 0) mark[x] = side[src[x]];
    }
    fetch(m0 + step);
    if (!a.out_table) cluster_sync();
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) {
      const int64_t m = m0 + x * kStep;
      if (m >= n) break;
      const unsigned blk = divide(static_cast<unsigned>(m), a.by_page);
      const int64_t row = (static_cast<int64_t>(__ldg(table + blk)) * c.Hkv + hk) * c.page + (m - blk * c.page);
      pool[row * 8 + u] = w[x];
      if (u == 0) side[row] = mark[x];
    }
  }
}

template <class F>
cudaError_t launch_cluster(F* kernel, dim3 grid, int threads, size_t smem, int cluster, bool pdl,
                           const EvictArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& args, cudaStream_t st) {
  EvictArgs a = args;
  const int64_t heads = static_cast<int64_t>(a.c.B) * a.c.Hkv, cap = static_cast<int64_t>(a.c.page) * a.c.max_blocks;
  // A cluster for what shared memory does not hold, and where CTAs are few (12 heads of 131072 slots: 33 us
  // with eight CTAs each, 40 with the four that hold them).
  a.cluster = 1;
  while (a.cluster < kMaxCluster &&
         (cap > static_cast<int64_t>(kCacheMost) * a.cluster ||
          (heads * a.cluster < 2 * sm_count() && cap > static_cast<int64_t>(2 * kSlotsCta) * a.cluster)))
    a.cluster *= 2;
  const int64_t per = ((cap + a.cluster - 1) / a.cluster + kSelPer - 1) / kSelPer * kSelPer;
  a.cached = static_cast<int>(per < kCacheMost ? per : kCacheMost);
  static bool few_set[64] = {}, many_set[64] = {};
  const bool few = per <= kSelRun;
  const cudaError_t e = few ? smem_limit_once(bam_kv_evict_select_kernel<kSelFew>, kCacheMost * 4, few_set)
                            : smem_limit_once(bam_kv_evict_select_kernel<kSelMany>, kCacheMost * 4, many_set);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.c.Hkv * a.cluster, a.c.B);
  const size_t smem = static_cast<size_t>(a.cached) * 4;
  return few ? launch_cluster(bam_kv_evict_select_kernel<kSelFew>, grid, kSelFew, smem, a.cluster, false, a, st)
             : launch_cluster(bam_kv_evict_select_kernel<kSelMany>, grid, kSelMany, smem, a.cluster, false, a, st);
}

cudaError_t launch_evict_move(const EvictArgs& args, cudaStream_t st) {
  EvictArgs a = args;
  const int64_t chains = 2 * static_cast<int64_t>(a.c.B) * a.c.Hkv;
  a.cluster = 1;
  if (a.out_table) {
    // Nothing that is read is written: any number of CTAs.
    while (a.cluster < 64 && chains * a.cluster < 8 * sm_count() && a.budget > 128 * static_cast<int64_t>(a.cluster))
      a.cluster *= 2;
    return launch_k(bam_kv_evict_move_kernel<128>, dim3(a.cluster * a.c.Hkv, a.c.B, 2), dim3(128), 0, st, true, a);
  }
  // Small CTAs for many short chains (16000 of 512 rows: 282 us, with large ones 345; 16 of them 21 and 15);
  // else large ones (1536 of 4096 rows, 30% of which move: 125 us with the choice, with small ones 133), and as
  // many a chain as a cluster takes.
  const bool many = chains >= 4 * sm_count() && a.budget <= 2048;
  while (a.cluster < kMaxCluster && chains * a.cluster < 2 * sm_count() &&
         a.budget > 512 * static_cast<int64_t>(a.cluster))
    a.cluster *= 2;
  const dim3 grid(a.cluster * a.c.Hkv, a.c.B, 2);
  if (many) return launch_cluster(bam_kv_evict_move_kernel<128>, grid, 128, 0, a.cluster, true, a, st);
  return launch_cluster(bam_kv_evict_move_kernel<512>, grid, 512, 0, a.cluster, true, a, st);
}

}  // namespace bam
