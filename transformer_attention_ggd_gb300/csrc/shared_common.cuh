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
  int nsplit, chunk;         // parts of the own keys, keys of a part
  int npsplit, pchunk;       // of the prefix
  int slots;                 // nsplit + npsplit
  int64_t zstride;           // max_blocks * page
};

constexpr float kNoMax = -3.4e38f;  // below every logit (the bias is clamped at -3e38)

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
  int* list;             // [B, Hkv, budget] slots kept, ascending
  int2* count;           // [B, Hkv] kept keys (-1: left as they were) and the first that moves
  int cluster;           // CTAs that share a chain of moves
};

cudaError_t launch_shared_prep(const SharedArgs& a, cudaStream_t st);
cudaError_t launch_shared(const CUtensorMap& tk, const CUtensorMap& tv, const SharedArgs& a,
                          cudaStream_t st);
cudaError_t launch_shared_join(const SharedArgs& a, cudaStream_t st);
cudaError_t launch_shared_weigh(const SharedArgs& a, cudaStream_t st);
// Splits of the own and prefix keys; fills nsplit, chunk, npsplit, pchunk, slots.
void shared_split(SharedArgs* a, int64_t Pmax, int64_t Tmax);

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t st);
cudaError_t launch_evict_move(const EvictArgs& a, cudaStream_t st);

}  // namespace bam
