// Eviction from a paged cache: of each sequence and key head the first keys, the
// last ones and, of the rest, those of the largest accumulated weight stay, in
// order.
#include "shared_common.cuh"

namespace bam {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelPer = 4;        // slots of a thread in a chunk
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 8;      // rows of a thread in a wave
constexpr int kMoveWave = kMoveThreads / 8 * kMoveRows;

// Order of the weights as unsigned numbers: NaN above everything, -0 as 0.
__device__ __forceinline__ uint32_t weight_order(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t x = __float_as_uint(w + 0.0f);
  return x & 0x80000000u ? ~x : x | 0x80000000u;
}

// Exclusive prefix sums over the block of two counts packed in a 64-bit word.
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* warp_sums, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  uint64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  __syncthreads();
  *total = all;
  return before + s - x;
}

// One block a sequence and key head: the weight of the last kept key by a radix
// search from the highest bits, then the list of the slots that stay.
__global__ void __launch_bounds__(kSelThreads) bam_kv_evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[256];
  __shared__ uint64_t warp_sums[kSelThreads / 32];
  __shared__ int s_bin, s_need;
  grid_dep_trigger();
  const CacheArgs& c = a.c;
  const int hk = blockIdx.x, b = blockIdx.y;
  const int cap = c.page * c.max_blocks, raw = __ldg(c.lens + b);
  const int len = min(max(raw, 0), cap), kept = min(len, a.budget);
  bool ok = raw == len, pages_ok = true;
  const int* table = c.block_table + static_cast<size_t>(b) * c.max_blocks;
  const int* out = a.out_table ? a.out_table + static_cast<size_t>(b) * a.out_blocks : nullptr;
  for (int i = threadIdx.x; i * static_cast<int64_t>(c.page) < len; i += kSelThreads) {
    const int pg = __ldg(table + i);
    pages_ok &= pg >= 0 && pg < c.num_pages;
  }
  if (out) {
    for (int i = threadIdx.x; i * static_cast<int64_t>(c.page) < kept; i += kSelThreads) {
      const int pg = __ldg(out + i);
      pages_ok &= pg >= 0 && pg < c.num_pages;
    }
  }
  pages_ok = __syncthreads_and(pages_ok);
  int2* count = a.count + static_cast<int64_t>(b) * c.Hkv + hk;
  if (threadIdx.x == 0 && !(ok && pages_ok)) record_bad_arg(c.status);
  int* list = a.list + (static_cast<int64_t>(b) * c.Hkv + hk) * a.budget;
  if (!pages_ok || len <= a.budget) {
    if (threadIdx.x == 0) *count = make_int2(pages_ok ? len : -1 - len, out ? 0 : len);
    if (pages_ok && out)
      for (int i = threadIdx.x; i < len; i += kSelThreads) list[i] = i;
    return;
  }
  auto weight = [&](int slot) {
    const int pg = __ldg(table + slot / c.page);
    return weight_order(a.key_weight[(static_cast<int64_t>(pg) * c.Hkv + hk) * c.page + slot % c.page]);
  };
  const int lo = a.sink, hi = len - a.recent;
  int need = a.budget - a.sink - a.recent;  // of [lo, hi), which holds more
  uint32_t prefix = 0;                      // the threshold's leading bits
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = lo + threadIdx.x; i < hi; i += kSelThreads) {
        const uint32_t w = weight(i);
        if (shift == 24 || (w >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&hist[(w >> shift) & 255], 1);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        int left = need, bin = 255;
        while (hist[bin] < left) left -= hist[bin--];
        s_bin = bin;
        s_need = left;
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(s_bin) << shift;
      need = s_need;
    }
  }
  // `need` of the keys whose weight is the threshold stay, the lowest slots first.
  const bool none = a.budget == a.sink + a.recent;
  int at = 0, ties = 0, first = len;
  for (int base = 0; base < len; base += kSelThreads * kSelPer) {
    const int i0 = base + threadIdx.x * kSelPer;
    bool over[kSelPer], tie[kSelPer];
    int n = 0, t = 0;
#pragma unroll
    for (int x = 0; x < kSelPer; ++x) {
      const int i = i0 + x;
      over[x] = tie[x] = false;
      if (i < lo || (i >= hi && i < len)) {
        over[x] = true;
      } else if (i < len && !none) {
        const uint32_t w = weight(i);
        over[x] = w > prefix;
        tie[x] = w == prefix;
      }
      n += over[x];
      t += tie[x];
    }
    uint64_t total;
    const uint64_t scan =
        block_scan(static_cast<uint64_t>(n) << 32 | static_cast<uint32_t>(t), warp_sums, &total);
    int tie_rank = ties + static_cast<int>(scan & 0xFFFFFFFFu);
    int dst = at + static_cast<int>(scan >> 32) + min(tie_rank, need) ;
#pragma unroll
    for (int x = 0; x < kSelPer; ++x) {
      const bool keep = over[x] || (tie[x] && tie_rank < need);
      tie_rank += tie[x];
      if (keep) {
        if (dst != i0 + x && first == len) first = dst;
        list[dst++] = i0 + x;
      }
    }
    at += static_cast<int>(total >> 32);
    ties += static_cast<int>(total & 0xFFFFFFFFu);
  }
  // The first key that moves.
  __syncthreads();
  if (threadIdx.x == 0) s_need = len;
  __syncthreads();
  atomicMin(&s_need, first);
  __syncthreads();
  if (threadIdx.x == 0) *count = make_int2(kept, out ? 0 : min(s_need, kept));
}

// A cluster moves the keys (z 0) or the values (z 1) of one sequence and key head,
// in waves: every CTA reads its rows of the wave, the cluster meets, and they are
// written.  Row m goes from slot list[m] >= m to slot m, so a row that is written
// was the source of an earlier row, if of any, which has been read.
__global__ void __launch_bounds__(kMoveThreads) bam_kv_evict_move_kernel(const EvictArgs a) {
  grid_dep_wait();
  const CacheArgs& c = a.c;
  const int rank = blockIdx.x % a.cluster, hk = blockIdx.x / a.cluster, b = blockIdx.y;
  const bool values = blockIdx.z;
  const int2 cnt = a.count[static_cast<int64_t>(b) * c.Hkv + hk];
  if (blockIdx.x == 0 && !values && threadIdx.x == 0) a.new_lens[b] = cnt.x >= 0 ? cnt.x : -1 - cnt.x;
  const int* table = c.block_table + static_cast<size_t>(b) * c.max_blocks;
  const int* dst_table = a.out_table ? a.out_table + static_cast<size_t>(b) * a.out_blocks : table;
  const int* list = a.list + (static_cast<int64_t>(b) * c.Hkv + hk) * a.budget;
  uint4* pool = reinterpret_cast<uint4*>(values ? a.v_pages : a.k_pages);
  uint32_t* side = values ? reinterpret_cast<uint32_t*>(a.key_weight) : reinterpret_cast<uint32_t*>(a.key_pos);
  const int u = threadIdx.x & 7;
  for (int64_t m0 = cnt.y; m0 < cnt.x; m0 += static_cast<int64_t>(kMoveWave) * a.cluster) {
    uint4 w[kMoveRows];
    uint32_t mark[kMoveRows];
    const int64_t first = m0 + rank * kMoveWave + (threadIdx.x >> 3);
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) {
      const int64_t m = first + x * (kMoveThreads / 8);
      if (m >= cnt.x) break;
      const int slot = list[m];
      const int pg = __ldg(table + slot / c.page);
      const int64_t row = (static_cast<int64_t>(pg) * c.Hkv + hk) * c.page + slot % c.page;
      w[x] = pool[row * 8 + u];
      if (u == 0) mark[x] = side[row];
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) {
      const int64_t m = first + x * (kMoveThreads / 8);
      if (m >= cnt.x) break;
      const int slot = static_cast<int>(m);
      const int pg = __ldg(dst_table + slot / c.page);
      const int64_t row = (static_cast<int64_t>(pg) * c.Hkv + hk) * c.page + slot % c.page;
      pool[row * 8 + u] = w[x];
      if (u == 0) side[row] = mark[x];
    }
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t st) {
  return launch_k(bam_kv_evict_select_kernel, dim3(a.c.Hkv, a.c.B), dim3(kSelThreads), 0, st, false, a);
}

cudaError_t launch_evict_move(const EvictArgs& args, cudaStream_t st) {
  EvictArgs a = args;
  a.cluster = 1;
  while (a.cluster < 8 && 2 * static_cast<int64_t>(a.c.B) * a.c.Hkv * a.cluster < 4 * sm_count()) a.cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.cluster * a.c.Hkv, a.c.B, 2);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, bam_kv_evict_move_kernel, a);
}

}  // namespace bam
