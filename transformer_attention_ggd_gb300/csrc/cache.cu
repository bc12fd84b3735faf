// Writing a paged cache: appending keys and values with their rotation by
// position, and keeping the accepted path of a draft.
//
// Both are copies (a token's head vector is 128 bytes of K and of V): the
// append reads and writes 2 * 128 * (2 Hkv + H) bytes a token and is bound by
// HBM for prompts and by latency for single tokens; the keep moves a few rows
// a sequence and is always bound by latency.  Measured on the device: prompts
// of up to 8192 tokens, 8 sequences, 12 heads 92 us (453 MB, 4.9 TB/s); 64
// drafts of 48 nodes, 32 and 8 heads 10.1 us (28 MB); 8 single tokens 3.0 us;
// keep of 256 sequences, 64 nodes 4.1 us.
#include "tree_common.cuh"

namespace bam {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 16;  // most tokens of a unit
constexpr int kAppendRows = 4;     // rows of a thread
constexpr int kAppendPass = kAppendThreads / 4;  // rows in flight per load: four lanes a row
// CTAs of an SM in a long call: 1, 2 and 3 took 134, 92 and 106 us for prompts
// of up to 8192 tokens, 12 heads, 8 sequences (453 MB: 68 us).
constexpr int kAppendResident = 2;

// One rotated pair: (a, b) -> (a cos - b sin, b cos + a sin), in fp32, rounded
// once to bf16 by the caller.
__device__ __forceinline__ void turn(float& a, float& b, float co, float si) {
  const float x = a * co - b * si;
  b = b * co + a * si;
  a = x;
}

__device__ __forceinline__ void unpack8(const uint4& w, float* f) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(x[i] << 16);
    f[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// A unit is up to 16 tokens of one sequence and a run of the heads of its
// queries, keys or values, 256 rows at most: four lanes hold a row, 32 bytes
// each, and a thread has up to four rows, of one token.  For pairs
// (x_f, x_{f + dims/2}) a lane takes the two 16-byte chunks that pair up.
struct AppendUnit {
  int b, tile;
  int kind, h0, heads;  // kind: 0 queries, 1 keys, 2 values
};
__device__ __forceinline__ AppendUnit append_unit(const AppendArgs& a, int64_t bt, int part) {
  AppendUnit x;
  x.b = static_cast<int>(bt / a.tiles);
  x.tile = static_cast<int>(bt - static_cast<int64_t>(x.b) * a.tiles);
  x.kind = part < a.q_parts ? 0 : part < a.q_parts + a.kv_parts ? 1 : 2;
  const int i = part - (x.kind == 0 ? 0 : x.kind == 1 ? a.q_parts : a.q_parts + a.kv_parts);
  x.h0 = i * a.heads;
  x.heads = min(a.heads, (x.kind == 0 ? a.H : a.c.Hkv) - x.h0);
  return x;
}
// Committed length and tokens of sequence b, clamped; false if out of range.
__device__ __forceinline__ bool append_lengths(const CacheArgs& c, int b, int& len, int& n) {
  const int cap = c.page * c.max_blocks;
  const int raw = __ldg(c.lens + b);
  const int rawn = c.draft_lens ? __ldg(c.draft_lens + b) : c.N;
  len = min(max(raw, 0), cap);
  n = min(max(rawn, 0), c.N);
  return raw == len && rawn == n;
}

// The parent of this thread's node of sequence b.
__device__ __forceinline__ int append_parent(const CacheArgs& c, int b) {
  return c.parents && threadIdx.x < c.N
             ? __ldg(c.parents + static_cast<size_t>(b) * c.N + threadIdx.x)
             : -1;
}

// This thread's place in a unit: token t, heads h, h + step, ...
struct AppendLane {
  int t, h, step, c0, c1;
};
// Loads this thread's rows of a unit whose tokens below n count.
__device__ __forceinline__ void append_load(const AppendArgs& a, const AppendUnit& x, int n,
                                            const AppendLane& ln, uint4 (&w)[kAppendRows][2]) {
  const int tok = x.tile * a.tokens + ln.t;
  if (tok >= n) return;
  const uint16_t* base = x.kind == 0 ? a.q : x.kind == 1 ? a.k : a.v;
  const int64_t* st = x.kind == 0 ? a.qs : x.kind == 1 ? a.ks : a.vs;
  const uint16_t* src = base + x.b * st[0] + (x.h0 + ln.h) * st[1] + tok * st[2];
  const int64_t step = ln.step * st[1];
#pragma unroll
  for (int y = 0; y < kAppendRows; ++y, src += step) {
    if (ln.h + y * ln.step >= x.heads) break;
    w[y][0] = *reinterpret_cast<const uint4*>(src + 8 * ln.c0);
    w[y][1] = *reinterpret_cast<const uint4*>(src + 8 * ln.c1);
  }
}

// A CTA takes every gridDim-th token tile (ragged prompts then load all SMs
// alike), its heads one unit after the other, so that the tile's slots and
// angles serve them all; the next unit's rows are on their way while this
// one's are turned and stored.  A call of so few units that each has a CTA
// loads all N tokens' rows before it knows which count: the lengths, slots,
// depths and angles then take no time of their own.
template <bool kRun>
__global__ void __launch_bounds__(kAppendThreads, kRun ? 2 : 3) bam_kv_append_kernel(const AppendArgs a) {
  __shared__ float4 cs[kAppendTokens][kHeadDim / 4];  // two (cosine, sine) pairs each
  __shared__ int64_t slot_row[kAppendTokens];  // row of head 0 in the pages, -1: not written
  __shared__ int depth[kTreeMax], jump[kTreeMax];
  const CacheArgs& c = a.c;
  const int u4 = threadIdx.x & 3, nh = a.dims / 16, half = a.dims / 2;
  const bool rotated = u4 < nh;
  AppendLane ln;
  ln.t = (threadIdx.x >> 2) & (a.tokens - 1);  // a.tokens is a power of two
  ln.h = (threadIdx.x >> 2) / a.tokens;
  ln.step = kAppendPass / a.tokens;
  ln.c0 = a.interleaved || !rotated ? 2 * u4 : u4;
  ln.c1 = a.interleaved || !rotated ? 2 * u4 + 1 : u4 + nh;
  const int cap = c.page * c.max_blocks;
  const int split = a.q_parts + 2 * a.kv_parts;
  int64_t bt = kRun ? blockIdx.x : blockIdx.x / split;
  int part = kRun ? 0 : static_cast<int>(blockIdx.x - bt * split);
  const int64_t tiles = static_cast<int64_t>(c.B) * a.tiles;
  AppendUnit x = append_unit(a, bt, part);
  uint4 w[kAppendRows][2], wn[kAppendRows][2];
  int len, n, par = -1, last_b = -1, last_tile = -1;
  if (!kRun) {
    append_load(a, x, c.N, ln, w);
    par = append_parent(c, x.b);
  }
  bool ok = append_lengths(c, x.b, len, n);
  if (kRun) append_load(a, x, n, ln, w);
  for (;;) {
    // The unit after this one.
    AppendUnit xn = x;
    int len_n = len, n_n = n;
    bool more = false;
    if (kRun) {
      if (++part == split) {
        part = 0;
        bt += gridDim.x;
      }
      more = bt < tiles;
      if (more) {
        xn = append_unit(a, bt, part);
        if (xn.b != x.b) ok &= append_lengths(c, xn.b, len_n, n_n);
        append_load(a, xn, n_n, ln, wn);
      }
    }
    const int t0 = x.tile * a.tokens, nt = min(a.tokens, n - t0);
    if (nt > 0 && (x.b != last_b || x.tile != last_tile)) {
      if (last_b >= 0) __syncthreads();  // the last tile's slots and angles are no longer read
      const int64_t slot = static_cast<int64_t>(len) + t0 + threadIdx.x;
      const int blk = static_cast<int>(slot) / c.page;
      int pg = -1;
      if (threadIdx.x < nt && slot < cap)
        pg = __ldg(c.block_table + static_cast<size_t>(x.b) * c.max_blocks + blk);
      if (c.parents && x.b != last_b) {
        if (kRun) par = append_parent(c, x.b);
        ok &= tree_depths(par, n, jump, depth);
      }
      if (threadIdx.x < nt) {
        int64_t row = -1;
        if (pg >= 0 && pg < c.num_pages)
          row = static_cast<int64_t>(pg) * c.Hkv * c.page + (static_cast<int>(slot) - blk * c.page);
        ok &= row >= 0;
        slot_row[threadIdx.x] = row;
      }
      for (int y = threadIdx.x; y < nt * (kHeadDim / 2); y += kAppendThreads) {
        const int t = y / (kHeadDim / 2), f = y % (kHeadDim / 2);
        if (f >= half) continue;
        const uint64_t pos = static_cast<uint64_t>(len) + (c.parents ? depth[t0 + t] : t0 + t);
        // The phase wraps modulo 2^64, one turn: an exact reduction.  Its top
        // 32 bits, signed, are the angle in units of 2^-31 half turns.
        const int top = static_cast<int>((pos * a.freq[f]) >> 32);
        float s, co;
        sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &co);
        reinterpret_cast<float2*>(cs[t])[f] = make_float2(co, s);
      }
      __syncthreads();
      last_b = x.b;
      last_tile = x.tile;
    }
    const int64_t row = ln.t < nt ? (x.kind == 0 ? 0 : slot_row[ln.t]) : -1;
    if (row >= 0) {
      uint16_t* dst;
      int64_t hs;  // elements from a head to the next
      if (x.kind == 0) {
        hs = static_cast<int64_t>(c.N) * kHeadDim;
        dst = a.q_out + (static_cast<int64_t>(x.b) * a.H + x.h0 + ln.h) * hs +
              static_cast<int64_t>(t0 + ln.t) * kHeadDim;
      } else {
        hs = static_cast<int64_t>(c.page) * kHeadDim;
        dst = (x.kind == 1 ? a.k_pages : a.v_pages) + row * kHeadDim + (x.h0 + ln.h) * hs;
      }
      hs *= ln.step;
      if (rotated && x.kind < 2) {
        float4 r[4];  // eight (cosine, sine) pairs
#pragma unroll
        for (int y = 0; y < 4; ++y) r[y] = cs[ln.t][4 * u4 + y];
#pragma unroll
        for (int y = 0; y < kAppendRows; ++y) {
          if (ln.h + y * ln.step >= x.heads) break;
          float f0[8], f1[8];
          unpack8(w[y][0], f0);
          unpack8(w[y][1], f1);
          if (a.interleaved) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              turn(f0[4 * z], f0[4 * z + 1], r[z].x, r[z].y);
              turn(f0[4 * z + 2], f0[4 * z + 3], r[z].z, r[z].w);
              turn(f1[4 * z], f1[4 * z + 1], r[2 + z].x, r[2 + z].y);
              turn(f1[4 * z + 2], f1[4 * z + 3], r[2 + z].z, r[2 + z].w);
            }
          } else {
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              turn(f0[2 * z], f1[2 * z], r[z].x, r[z].y);
              turn(f0[2 * z + 1], f1[2 * z + 1], r[z].z, r[z].w);
            }
          }
          w[y][0] = pack8(f0);
          w[y][1] = pack8(f1);
        }
      }
#pragma unroll
      for (int y = 0; y < kAppendRows; ++y, dst += hs) {
        if (ln.h + y * ln.step >= x.heads) break;
        *reinterpret_cast<uint4*>(dst + 8 * ln.c0) = w[y][0];
        *reinterpret_cast<uint4*>(dst + 8 * ln.c1) = w[y][1];
      }
    }
    if (!more) break;
    x = xn;
    len = len_n;
    n = n_n;
#pragma unroll
    for (int y = 0; y < kAppendRows; ++y) {
      w[y][0] = wn[y][0];
      w[y][1] = wn[y][1];
    }
  }
  if (!ok) record_bad_arg(c.status);
}

constexpr int kKeepThreads = 256;
constexpr int kKeepBatch = 16;  // rows that a warp holds in registers

// One cluster per sequence; a warp takes one head of K or of V at a time.
// Node m of the path moves from slot a_m to slot m <= a_m.  A slot that is
// written may be an earlier node's source but never a later one's
// (a_m' >= m' > m), so a warp that reads a batch of rows before it writes
// them, batches in order, moves them in place.
__global__ void __launch_bounds__(kKeepThreads) bam_kv_keep_kernel(const KeepArgs a) {
  __shared__ int par[kTreeMax], path[kTreeMax];
  __shared__ int64_t src_row[kTreeMax], dst_row[kTreeMax];
  __shared__ int count;
  const CacheArgs& c = a.c;
  const int b = blockIdx.y;
  if (c.parents && threadIdx.x < c.N)
    par[threadIdx.x] = __ldg(c.parents + static_cast<size_t>(b) * c.N + threadIdx.x);
  int len, n;
  bool ok = cache_lengths(c, b, &len, &n);
  int acc = __ldg(a.accepted + b);
  if (acc < -1 || acc >= n) {
    ok = false;
    acc = -1;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    // Root to node, from the deep end: the depth is known after the walk.
    int m = 0;
    if (c.parents) {
      for (int i = acc; i >= 0;) {
        path[m++] = i;
        const int p = par[i];
        if (p < -1 || p >= i) ok = false;
        i = p < i ? p : -1;
      }
    } else {
      m = acc + 1;  // a chain: every node is where it belongs
    }
    count = m;
  }
  __syncthreads();
  const int m = count;
  bool pages_ok = true;
  for (int x = threadIdx.x; x < m; x += kKeepThreads) {
    const int s = len + (c.parents ? path[m - 1 - x] : x), d = len + x;
    const int ps = __ldg(c.block_table + static_cast<size_t>(b) * c.max_blocks + s / c.page);
    const int pd = __ldg(c.block_table + static_cast<size_t>(b) * c.max_blocks + d / c.page);
    pages_ok &= ps >= 0 && ps < c.num_pages && pd >= 0 && pd < c.num_pages;
    src_row[x] = static_cast<int64_t>(ps) * c.Hkv * c.page + s % c.page;
    dst_row[x] = static_cast<int64_t>(pd) * c.Hkv * c.page + d % c.page;
  }
  pages_ok = __syncthreads_and(pages_ok);
  if (blockIdx.x == 0 && threadIdx.x == 0 && !(ok && pages_ok)) record_bad_arg(c.status);

  if (c.parents && pages_ok) {
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kKeepThreads / 32);
    for (int hv = blockIdx.x * (kKeepThreads / 32) + (threadIdx.x >> 5); hv < 2 * c.Hkv;
         hv += warps) {
      uint16_t* pool = hv < c.Hkv ? a.k_pages : a.v_pages;
      const int64_t head = static_cast<int64_t>(hv < c.Hkv ? hv : hv - c.Hkv) * c.page;
      for (int m0 = 0; m0 < m; m0 += kKeepBatch) {
        uint4 w[kKeepBatch / 4];
#pragma unroll
        for (int x = 0; x < kKeepBatch / 4; ++x) {
          const int i = m0 + 4 * x + (lane >> 3);
          if (i < m)
            w[x] = reinterpret_cast<const uint4*>(pool + (src_row[i] + head) * kHeadDim)[lane & 7];
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < kKeepBatch / 4; ++x) {
          const int i = m0 + 4 * x + (lane >> 3);
          if (i < m && src_row[i] != dst_row[i])
            reinterpret_cast<uint4*>(pool + (dst_row[i] + head) * kHeadDim)[lane & 7] = w[x];
        }
        __syncwarp();
      }
    }
  }
  // new_lens may be cache_lens: written when every CTA of the sequence has
  // read its length.
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x == 0) a.new_lens[b] = len + (pages_ok ? m : 0);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& args, cudaStream_t st) {
  AppendArgs a = args;
  a.tokens = 1;
  while (a.tokens < a.c.N && a.tokens < kAppendTokens) a.tokens *= 2;
  a.tiles = (a.c.N + a.tokens - 1) / a.tokens;
  // Heads of a unit: what fits, in equal parts.
  const int most = kAppendRows * kAppendPass / a.tokens;
  const int big = a.H > a.c.Hkv ? a.H : a.c.Hkv, parts = (big + most - 1) / most;
  a.heads = (big + parts - 1) / parts;
  a.q_parts = (a.H + a.heads - 1) / a.heads;
  a.kv_parts = (a.c.Hkv + a.heads - 1) / a.heads;
  const int64_t tiles = static_cast<int64_t>(a.c.B) * a.tiles;
  const int64_t units = tiles * (a.q_parts + 2 * a.kv_parts);
  // Token tiles dealt to resident CTAs once there are enough of them.  A CTA per
  // unit takes 97 instead of 92 us for the prompts above and 25.7 instead of
  // 20.3 for 200 drafts of 48 nodes; resident CTAs take 4.2 instead of 3.0 for 8
  // single tokens and 11.1 instead of 10.1 for 64 drafts of 48 nodes.
  const int64_t run = static_cast<int64_t>(sm_count()) * kAppendResident;
  if (tiles > run)
    return launch_k(bam_kv_append_kernel<true>, dim3(static_cast<unsigned>(run)),
                    dim3(kAppendThreads), 0, st, false, a);
  if (units > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch_k(bam_kv_append_kernel<false>, dim3(static_cast<unsigned>(units)),
                  dim3(kAppendThreads), 0, st, false, a);
}

cudaError_t launch_keep(const KeepArgs& a, cudaStream_t st) {
  const int warps = kKeepThreads / 32;
  int x = (2 * a.c.Hkv + warps - 1) / warps;
  if (x > 8) x = 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(x, a.c.B);
  cfg.blockDim = dim3(kKeepThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = x;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, bam_kv_keep_kernel, a);
}

}  // namespace bam
