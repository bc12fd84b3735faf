// Shared by the paged-cache operators for drafted tokens (append, tree
// attention, keep): kernel argument blocks, checks of what only the device
// reads, and the depths and ancestors of a draft's nodes.
#pragma once

#include "row_ops.cuh"

namespace bam {

constexpr int kTreeMax = 128;  // nodes of a draft with parents
constexpr int kMaxPosition = 1 << 28;  // positions of keys and queries stay below

// A paged cache and the drafts behind its committed keys.
struct CacheArgs {
  const int* block_table;  // [B, max_blocks]
  const int* lens;         // [B] committed keys
  const int* draft_lens;   // [B] or null: N each
  const int* parents;      // [B, N] or null: a chain
  DevStatus* status;
  int B, Hkv, N, page, max_blocks, num_pages;
};

struct AppendArgs {
  CacheArgs c;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* q;
  uint16_t* q_out;
  uint16_t* k_pages;
  uint16_t* v_pages;
  int64_t ks[3], vs[3], qs[3];  // element strides over batch, head, token
  int H;                        // query heads (0 without q)
  int tokens, heads;            // tokens (a power of two) and heads of a unit of work
  int tiles;                    // token tiles of a sequence
  int q_parts, kv_parts;        // units of a token tile: of its queries, of its keys
  RopeArgs rope;
  // With `extended` alone:
  const float* q_weight;        // norms (null: none), [64] or [heads, 64]
  const float* k_weight;
  const int* first_pos;         // [B] position of each sequence's token 0, or null: lens
  int* key_pos;                 // [num_pages, Hkv, page] or null
  float* key_weight;
  float norm_eps;
  int per_head, max_pos, extended;
};

struct KeepArgs {
  CacheArgs c;
  uint16_t* k_pages;
  uint16_t* v_pages;
  const int* accepted;
  int* new_lens;
  int* key_pos;       // [num_pages, Hkv, page] or null: no marks
  float* key_weight;
};

// Tree attention: the rows of a (sequence, key head) are its group * n
// (query head, node) pairs, row r = (head r / n, node r % n), taken `rows` at
// a time; such an item reads the tiles of 64 or 128 keys that hold the sequence's
// len + n keys.  An item counts as kItemCost units and those of its tiles;
// the plan is the running sum of the sequences' units over all their items,
// and CTA c of `active` takes units [W c / active, W (c+1) / active) of the W
// in all.
// An item's fixed cost, in units of a tile of committed keys.  3, 4 and 7
// measured 45.3, 44.0 and 44.5 us (13 sequences of 9001 keys, 21 nodes), 100.6,
// 101.4 and 103.5 (32 of 16384, single tokens), 29.4, 29.4 and 31.1 (8 of 4096,
// fp32 output), 13.8, 13.4 and 13.2 (one of 500, 7 nodes).
constexpr int kItemCost = 4;
// Units of a tile with drafted keys where its logits do not stay in registers.
// 1 and 2 measured 74.2 and 71.7 us (4 chains of 128 nodes, 20000 keys), 45.2 and
// 44.0 (13 of 9001, 21 nodes), 116.3 and 118.3 (100 of 600, 40 nodes, 8 heads a
// key head, fp32 output).
constexpr int kTailCost = 2;
constexpr int kTreeCtas = 304;   // most CTAs (two per SM)

// An item that lies in CTAs `first` to `last`; n is 0 if it lies in one.  In a call
// of few items there is a record of each (by_item), in one of many a record of
// the one that begins in each CTA and goes on in others.
struct CutItem {
  int b, hk, r0, n, first, last;
};

struct TreeArgs {
  CacheArgs c;
  const uint16_t* q;  // [B, H, N, 64]
  const uint16_t* v_pages;
  const float* alpha;
  const float* beta;
  const float* mu;
  const float* s;
  void* o;
  float* lse;
  int64_t* plan;      // [B + 1] first unit of each sequence, and W
  float* table;       // [H, tab_len]: entry y is b_h(tab_zero - y) * log2(e)
  float* part;        // [2 * kTreeCtas, 16, rows, 4] partial outputs, by four columns
  float2* part_ml;    // [2 * kTreeCtas, rows]: maximum (log2 units), sum (sign bit: odd values to come)
  CutItem* cut;       // [kTreeCtas]
  int by_item, nrb_most;  // nrb_most: items of a sequence and key head, at most
  float eps;
  int H, group, prior, ssmax, o_fp32;
  int tab_len, tab_zero;
  int rows;           // rows of an item, at most: 32, 64 or 128
  int tile;           // keys of a tile, 64 or 128
  int tail_cost;      // units of a tile that holds drafted keys
  int ctas;           // CTAs of the launch
  int stages;         // ring stages
  int win_stage;      // floats of a stage's table windows
  int nodes, near;    // nodes (a multiple of 32) and table entries that an item keeps
};

// Rows of an item for `rows` (head, node) pairs: Tensor Memory's 128, or the half
// or quarter that holds them all; they then stand there two or four times, each
// copy with its part of the keys.  Against 128 always, a call: 442 and 515 us
// with 32 rows and 64 sequences of 32768 keys, 101 and 112 with 4 rows and
// 16384 keys, 87 and 91 with 64 rows and 131072, 50 and 78 with 8 rows and 256
// sequences of 100; 13.4 and 12.8 with 7 rows and one sequence of 500.
inline int tree_rows(int64_t rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }
// Table row: distances 0 .. Tmax at entries Tmax .. 0 and, behind entry
// Tmax, room for windows that reach past the last key.
inline int tree_table_zero(int Tmax) { return (Tmax + 63) / 64 * 64; }
inline int tree_table_len(int Tmax) { return tree_table_zero(Tmax) + 64 + kTreeMax + 128; }

cudaError_t launch_append(const AppendArgs& a, cudaStream_t st);
cudaError_t launch_keep(const KeepArgs& a, cudaStream_t st);
bool tree_config(TreeArgs* a, int sms);
cudaError_t launch_tree_prep(const TreeArgs& a, cudaStream_t st);
cudaError_t launch_tree(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a,
                        cudaStream_t st);
cudaError_t launch_tree_combine(const TreeArgs& a, cudaStream_t st);

#ifdef __CUDACC__

enum : int { kSiteCacheArg = 50 };

// Records an argument that only the device reads and that was out of range.
// The operators of one launch have no earlier kernel that initialises a fresh
// status area, so the recording thread does; every thread that gets here
// writes the same words, so their order does not matter.
__device__ __forceinline__ void record_bad_arg(DevStatus* st) {
  volatile DevStatus* v = st;
  if (v->magic[0] == kStatusMagic0 && v->magic[1] == kStatusMagic1) {
    if (atomicCAS(&st->code, BAM_DEV_OK, BAM_DEV_BAD_ARG) == BAM_DEV_OK) v->site = kSiteCacheArg;
    return;
  }
  v->abort = 0;
  v->code = BAM_DEV_BAD_ARG;
  v->site = kSiteCacheArg;
  v->block = 0;
  v->giveup = 0;
  __threadfence();
  v->magic[0] = kStatusMagic0;
  v->magic[1] = kStatusMagic1;
}

// Committed length and draft nodes of sequence b, clamped into their ranges.
// Returns false when a value was out of range.
__device__ __forceinline__ bool cache_lengths(const CacheArgs& c, int b, int* len, int* n) {
  const int cap = c.page * c.max_blocks;
  const int raw = __ldg(c.lens + b);
  const int rawn = c.draft_lens ? __ldg(c.draft_lens + b) : c.N;
  *len = min(max(raw, 0), cap);
  *n = min(min(max(rawn, 0), c.N), cap - *len);
  return raw == *len && rawn == *n;
}

// Depths of the first n <= kTreeMax nodes, by all threads of a block of at
// least kTreeMax threads, thread i with node i's parent: each round doubles
// the distance that a node's jump pointer spans, so the deepest chain takes
// log2(depth) rounds.  `jump` holds kTreeMax ints of shared memory, as
// `depth`.  Ends with a block barrier.  Returns false in a thread whose node
// had a parent outside [-1, i).
__device__ __forceinline__ bool tree_depths(int parent, int n, int* jump, int* depth) {
  const int i = threadIdx.x;
  const bool ok = i >= n || (parent >= -1 && parent < i);
  int p = i < n && ok ? parent : -1;
  int d = p >= 0 ? 1 : 0;
  if (i < kTreeMax) {
    jump[i] = p;
    depth[i] = d;
  }
  while (__syncthreads_or(p >= 0)) {
    int dp = 0, pp = -1;
    if (p >= 0) {
      dp = depth[p];
      pp = jump[p];
    }
    __syncthreads();
    d += dp;
    p = pp;
    if (i < kTreeMax) {
      jump[i] = p;
      depth[i] = d;
    }
  }
  return ok;
}

#endif  // __CUDACC__

}  // namespace bam
