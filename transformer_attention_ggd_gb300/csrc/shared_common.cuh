// Shared by the kernels of the bounded cache: decode over a shared prefix and
// over keys with positions and weights, and eviction.
#pragma once

#include "tree_common.cuh"

namespace bam {

struct SharedArgs {
  CacheArgs c;               // the sequences' own keys (N, draft_lens, parents unused)
  const uint16_t* q;         // [B, H, 64]
  const int* prefix_table;   // [prefix_blocks] or null: no prefix
  const int* prefix_len;     // [1]
  int prefix_blocks;
  const int* q_pos;          // [B] position of each query, or null: behind prefix and own keys
  const int* key_pos;        // [num_pages, Hkv, page] or null: slots in order behind the prefix
  float* key_weight;         // with key_pos
  float decay;
  int max_pos;               // positions are below it (with key_pos)
  const float* alpha;
  const float* beta;
  const float* mu;
  const float* s;
  float eps;
  int prior, ssmax;
  void* o;                   // [B, H, 64]
  int o_fp32;
  float* lse;                // [B, H] or null
  float2* ml;                // [B * H, slots]: maximum (log2 units) and sum of each part
  float* part;               // [B * H, slots, 64]: its unnormalised output
  float* z;                  // [B, H, zstride] logits (log2 units) of own keys, with key_pos
  int H, group;
  int nsplit;                // parts of a sequence's own keys
  int npsplit;               // of the prefix
  int copies;                // of a row, each with its part of a tile's keys; 0: few rows, no tiles
  int slots;                 // of a row: nsplit + npsplit
  int64_t zstride;           // max_blocks * page
  float* spill;              // [B * H, spills, 64]: what leaves the accumulators of a prefix in tiles
  int spills;
  // For a prefix in tiles: the table of b_h(d) log2(e).  Entry y of copy k of head h, at
  // [(k * H + h) * tab_len + y + k], holds d = tab_top - y.
  float* table;
  int tab_top, tab_len;
};

constexpr int kLeastKeys = 64;    // of a part, at least
// Keys of each of `parts` parts of n keys: whole tiles of 64.
__host__ __device__ inline int part_keys(int n, int parts) {
  const int each = ((n + parts - 1) / parts + 63) / 64 * 64;
  return each > kLeastKeys ? each : kLeastKeys;
}
// Rows of a key head over the prefix, at most, that go with the own keys instead of in tiles.  8 rows, 12
// key heads and 1024, 8192 and 65536 keys: 12, 16 and 54 us without tiles, 14, 19 and 62 with them;
// 12 rows and 1024 and 8192: 14 and 23, 15 and 21; 16 rows, 32768: 58 and 38.
constexpr int kFewRows = 8;

constexpr float kNoMax = -3.4e38f;  // below every logit (the bias is clamped at -3e38)

#ifdef __CUDACC__
// Own length of sequence b and length of the prefix, clamped.
__device__ __forceinline__ int own_len(const SharedArgs& a, int b, bool* ok) {
  const int cap = a.c.page * a.c.max_blocks, raw = __ldg(a.c.lens + b);
  const int len = min(max(raw, 0), cap);
  *ok &= raw == len;
  return len;
}
__device__ __forceinline__ int prefix_len(const SharedArgs& a, bool* ok) {
  if (!a.prefix_table) return 0;
  const int cap = a.c.page * a.prefix_blocks, raw = __ldg(a.prefix_len);
  const int len = min(max(raw, 0), cap);
  *ok &= raw == len;
  return len;
}
// Position of the query of sequence b (-1 when there is no key at all), not before the
// prefix's last key.
__device__ __forceinline__ int query_pos(const SharedArgs& a, int b, int P, bool* ok) {
  if (a.q_pos) {
    const int raw = __ldg(a.q_pos + b), pos = max(min(raw, a.max_pos - 1), max(P - 1, 0));
    *ok &= raw == pos;
    return pos;
  }
  return P + own_len(a, b, ok) - 1;
}
// Logit scale of head h at position pos, log2 units.
__device__ __forceinline__ float shared_scale(const SharedArgs& a, int h, int pos) {
  const float c = a.ssmax ? __ldg(a.s + h) * logf(static_cast<float>(pos + 1)) : 1.0f;
  return c * (0.125f * 1.44269504088896341f);
}
#endif

struct EvictArgs {
  CacheArgs c;
  uint16_t* k_pages;
  uint16_t* v_pages;
  int* key_pos;
  float* key_weight;
  const int* out_table;  // [B, out_blocks] or null: in place
  int out_blocks;
  int* new_lens;
  int budget, sink, recent;
  Divisor by_page;
  // Of each sequence and key head: the rows of the pages that stay, in order, how many they are
  // (-1 - length: the sequence stays as it is) and the first that moves.
  unsigned* list;        // [B, Hkv, budget]
  int2* count;           // [B, Hkv]
  int cluster;           // CTAs that share a sequence and key head (of its keys or values, moving)
  int cached;            // weights of a selecting CTA that stay in shared memory
};

cudaError_t launch_shared_prep(const SharedArgs& a, cudaStream_t st);
cudaError_t launch_shared(const CUtensorMap& tk, const CUtensorMap& tv, const SharedArgs& a,
                          cudaStream_t st);
cudaError_t launch_shared_end(const SharedArgs& a, cudaStream_t st);
cudaError_t launch_prefix(const CUtensorMap& tk, const CUtensorMap& tv, const SharedArgs& a,
                          cudaStream_t st);
// Splits of the own and prefix keys and the table's size; fills nsplit, npsplit, copies,
// slots, spills, tab_top, tab_len.
void shared_split(SharedArgs* a, int64_t Pmax, int64_t Tmax);
void prefix_split(SharedArgs* a, int64_t Pmax, int64_t Tmax);

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t st);
cudaError_t launch_evict_move(const EvictArgs& a, cudaStream_t st);

}  // namespace bam
