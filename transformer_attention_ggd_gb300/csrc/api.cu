// C ABI of the GGD-BAM attention library (declarations and contracts in
// include/bam_attn.h): argument validation, workspace layout, TMA tensor-map
// encoding and kernel launches.  No allocation, no host fallback: every step
// of the computation runs in the kernels of this library.
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>
#include <utility>

#include <cudaTypedefs.h>

#include "../../include/bam_attn.h"
#include "bam_common.cuh"
#include "norm_common.cuh"
#include "shared_common.cuh"
#include "tree_common.cuh"

static_assert(BAM_PRIOR_THETA == bam::kPriorTheta, "prior codes of the ABI and the kernels");

namespace bam {
namespace {

std::atomic<uint64_t> g_launches{0};
std::mutex g_prof_mu;
cudaEvent_t g_prof_before[BAM_KERNEL_COUNT] = {};
cudaEvent_t g_prof_after[BAM_KERNEL_COUNT] = {};

// Runs `launch` bracketed by the instrumentation events of kernel `which`.
template <class F>
cudaError_t launch_kernel(int which, cudaStream_t st, F launch) {
  cudaEvent_t before = nullptr, after = nullptr;
  {
    std::lock_guard<std::mutex> g(g_prof_mu);
    before = g_prof_before[which];
    after = g_prof_after[which];
  }
  // Under stream capture the records are external, so that they become
  // event-record nodes of the graph (timestamps on every replay) rather than
  // internal dependencies.
  unsigned flags = cudaEventRecordDefault;
  if (before || after) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(st, &cs);
    if (e != cudaSuccess) return e;
    if (cs == cudaStreamCaptureStatusActive) flags = cudaEventRecordExternal;
  }
  if (before) {
    cudaError_t e = cudaEventRecordWithFlags(before, st, flags);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = launch();
  g_launches.fetch_add(1, std::memory_order_relaxed);
  if (e != cudaSuccess) return e;
  if (after) e = cudaEventRecordWithFlags(after, st, flags);
  return e;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// [BH, T, 64] bf16 viewed as a 3-D tensor (64, T, BH); boxes of `rows` x 64
// (128 by default) with the 128-byte swizzle that the tcgen05 K-major /
// MN-major operands expect.  Rows past T inside a head read as zeros.
bool encode_rows(CUtensorMap* m, const void* base, int BH, int T, unsigned rows = 128) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(T),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(kHeadDim) * 2,
                           static_cast<cuuint64_t>(T) * kHeadDim * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(kHeadDim), rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// fp32 [BH, T, 64] accumulator as a 3-D tensor (64, T, BH) in boxes of 32
// columns x `rows` (128 by default; 128-byte rows, 128-byte swizzle) for TMA
// reductions and stores.
bool encode_acc_rows(CUtensorMap* m, void* base, int BH, int T, unsigned rows = 128) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(T),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(kHeadDim) * 4,
                           static_cast<cuuint64_t>(T) * kHeadDim * 4};
  cuuint32_t box[3] = {32, rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bam_status check_sizes(int B, int H, int T, int D) {
  if (B < 1 || H < 1 || T < 1 || D < 1) return BAM_ERR_INVALID_ARG;
  if (D != kHeadDim) return BAM_ERR_UNSUPPORTED;
  if (T > (1 << 28)) return BAM_ERR_UNSUPPORTED;
  const int64_t BH = static_cast<int64_t>(B) * H;
  const int64_t nqb = (T + 255) / 256;
  if (BH > (1 << 24) || BH * nqb >= (int64_t(1) << 31)) return BAM_ERR_UNSUPPORTED;
  if (H > 65535) return BAM_ERR_UNSUPPORTED;
  return BAM_OK;
}

bam_status check_params(const bam_params* p) {
  if (!p || !p->alpha || !p->beta || !p->mu) return BAM_ERR_INVALID_ARG;
  if (p->ssmax && !p->s) return BAM_ERR_INVALID_ARG;
  if (!(p->eps > 0.0f) || !std::isfinite(p->eps)) return BAM_ERR_INVALID_ARG;
  if ((p->causal != 0 && p->causal != 1) || (p->ssmax != 0 && p->ssmax != 1))
    return BAM_ERR_INVALID_ARG;
  if (p->prior != BAM_PRIOR_ALPHA && p->prior != BAM_PRIOR_THETA) return BAM_ERR_INVALID_ARG;
  return BAM_OK;
}

// Workspace layouts.
struct FwdWs {
  size_t table, total;
};
FwdWs fwd_ws(int H, int T, int causal) {
  const TableGeom g = table_geom(T, causal);
  FwdWs w;
  w.table = kStatusBytes;
  w.total = w.table + align256((kTabCopies * static_cast<size_t>(H) * g.len + kTabPadFloats) * 4);
  return w;
}

struct BwdWs {
  size_t table, delta, dq_acc, rowacc, total;
};
BwdWs bwd_ws(int B, int H, int T, int causal) {
  const TableGeom g = table_geom(T, causal);
  const size_t BH = static_cast<size_t>(B) * H;
  BwdWs w;
  w.table = kStatusBytes;
  w.delta =
      w.table + align256((3 * kTabCopies * static_cast<size_t>(H) * g.len + kTabPadFloats) * 4);
  w.dq_acc = w.delta + align256(BH * T * 4);
  w.rowacc = w.dq_acc + align256(BH * T * kHeadDim * 4);
  w.total = w.rowacc + align256(BH * T * 8 * 4);
  return w;
}

struct DecWs {
  size_t table, part, total;
  int nsplit, chunk, tab_len;
};
DecWs dec_ws(int B, int H, int Tkv) {
  DecWs w;
  decode_split(B * H, Tkv, &w.nsplit, &w.chunk);
  w.tab_len = decode_table_len(Tkv);
  w.table = kStatusBytes;
  w.part = w.table + align256(static_cast<size_t>(H) * w.tab_len * 4);
  w.total = w.part + align256(static_cast<size_t>(B) * H * w.nsplit * (2 + kHeadDim) * 4);
  return w;
}

struct TreeWs {
  size_t plan, table, ml, cut, part, total;
  int rows;
};
TreeWs tree_ws(int B, int H, int Hkv, int N, int Tmax) {
  TreeWs w;
  w.rows = tree_rows(static_cast<int64_t>(H / Hkv) * N);
  w.plan = kStatusBytes;
  w.table = w.plan + align256((static_cast<size_t>(B) + 1) * 8);
  w.ml = w.table + align256(static_cast<size_t>(H) * tree_table_len(Tmax) * 4);
  w.cut = w.ml + align256(2 * kTreeCtas * static_cast<size_t>(w.rows) * 8);
  w.part = w.cut + align256(kTreeCtas * sizeof(CutItem));
  w.total = w.part + align256(2 * kTreeCtas * static_cast<size_t>(w.rows) * kHeadDim * 4);
  return w;
}

bam_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (!ws || !aligned(ws, 256) || ws_bytes < need) return BAM_ERR_WORKSPACE;
  return BAM_OK;
}

// Sizes and pointers of a paged cache with drafts behind its committed keys.
bam_status check_cache(int B, int H, int Hkv, int N, int page, int max_blocks, int num_pages,
                       int D, const void* block_table, const void* cache_lens,
                       const void* draft_lens, const void* parents) {
  if (B < 1 || H < 1 || Hkv < 1 || N < 1 || D < 1 || max_blocks < 1 || num_pages < 1)
    return BAM_ERR_INVALID_ARG;
  if (page < 64 || page % 64 != 0 || H % Hkv != 0) return BAM_ERR_INVALID_ARG;
  if (!block_table || !aligned(block_table, 4) || !cache_lens || !aligned(cache_lens, 4) ||
      !aligned(draft_lens, 4) || !aligned(parents, 4))
    return BAM_ERR_INVALID_ARG;
  if (D != kHeadDim) return BAM_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(page) * max_blocks > (1 << 28) || N > (1 << 28) || B > 65535 ||
      H > 65535 || static_cast<int64_t>(num_pages) * Hkv > 0x7FFFFFFF)
    return BAM_ERR_UNSUPPORTED;
  return BAM_OK;
}

// False when the rotation is not a valid one (null: none).
bool fill_rope(const bam_rope* rope, RopeArgs* a) {
  a->dims = a->interleaved = 0;
  if (!rope || rope->dims == 0) return true;
  if (rope->dims < 0 || rope->dims > kHeadDim || rope->dims % 16 != 0 ||
      (rope->interleaved != 0 && rope->interleaved != 1) || !(rope->base >= 1.0) ||
      !std::isfinite(rope->base))
    return false;  // (below 1, turns per position exceed what a double's fraction holds)
  a->dims = rope->dims;
  a->interleaved = rope->interleaved;
  // base^(-2 f / dims) by repeated products: their 2^-48 is 2^-23 turns at
  // position 2^28.
  const double ratio = std::pow(rope->base, -2.0 / rope->dims);
  double per = 1.0 / 6.283185307179586477;
  for (int f = 0; f < rope->dims / 2; ++f, per *= ratio) {
    // (per is below 1: base is at least 1)
    a->freq[f] = static_cast<uint64_t>(per * 18446744073709551616.0);
  }
  return true;
}

// The smallest eps of a norm: below it, squares that fp32 loses would count.
constexpr float kNormEpsMin = 1e-30f;

bool norm_ok(const bam_qk_norm* n) {
  return n && n->q_weight && n->k_weight && aligned(n->q_weight, 16) && aligned(n->k_weight, 16) &&
         n->eps >= kNormEpsMin && std::isfinite(n->eps) && (n->per_head == 0 || n->per_head == 1);
}

// Three element strides (batch, head, token) of a tensor of rows of 64; an output's
// rows must not overlap: sorted by stride, each spans what lies below it.
bool strides_ok(const int64_t* st, const int64_t* dims, bool output) {
  for (int x = 0; x < 3; ++x)
    if (st[x] < 0 || st[x] % 8 != 0) return false;
  if (!output) return true;
  int order[3] = {0, 1, 2};
  for (int x = 0; x < 2; ++x)
    for (int y = 0; y < 2; ++y)
      if (st[order[y]] > st[order[y + 1]]) std::swap(order[y], order[y + 1]);
  int64_t span = kHeadDim;
  for (int x : order) {
    if (dims[x] == 1) continue;
    if (st[x] < span) return false;
    span = st[x] * (dims[x] - 1) + span;
  }
  return true;
}

// The sides of a norm: x, g (backward), y from `ptrs` (queries', keys'), strides from
// `strides` in the same order (null: dense).
bam_status fill_norm(NormArgs* a, const void* const (*ptrs)[2], int tensors, const int64_t* strides,
                     const int* positions, int B, int H, int Hkv, int T, int D,
                     const bam_qk_norm* norm, const bam_rope* rope) {
  if (B < 1 || H < 1 || Hkv < 1 || T < 1 || D < 1) return BAM_ERR_INVALID_ARG;
  if (D != kHeadDim) return BAM_ERR_UNSUPPORTED;
  if (H > 65535 || Hkv > 65535 || static_cast<int64_t>(B) * T > 0x7FFFFFFF) return BAM_ERR_UNSUPPORTED;
  if (!norm_ok(norm) || !fill_rope(rope, &a->rope) || !aligned(positions, 4)) return BAM_ERR_INVALID_ARG;
  for (int x = 0; x < tensors; ++x) {
    for (int k = 0; k < 2; ++k) {
      if (!ptrs[x][k] || !aligned(ptrs[x][k], 16)) return BAM_ERR_INVALID_ARG;
      NormSide& s = a->side[k];
      s.heads = k ? Hkv : H;
      int64_t* st = x == 0 ? s.xs : x == tensors - 1 ? s.ys : s.gs;
      const int64_t dims[3] = {B, s.heads, T};
      const int64_t dense[3] = {static_cast<int64_t>(s.heads) * T * kHeadDim,
                                static_cast<int64_t>(T) * kHeadDim, kHeadDim};
      std::memcpy(st, strides ? strides + 3 * (2 * x + k) : dense, sizeof(dense));
      if (!strides_ok(st, dims, x == tensors - 1)) return BAM_ERR_INVALID_ARG;
      // (a walk goes up to a pass past the last head)
      unsigned __int128 most = 0;
      for (int y = 0; y < 3; ++y) {
        st[y] /= 8;
        most += static_cast<unsigned __int128>(st[y]) * (dims[y] + (y == 1 ? 2 * kNormPass : 0));
      }
      if (most >> 32) a->large = 1;
      if (most >> 60) return BAM_ERR_INVALID_ARG;
    }
  }
  for (int k = 0; k < 2; ++k) {
    NormSide& s = a->side[k];
    s.x = static_cast<const uint16_t*>(ptrs[0][k]);
    s.g = static_cast<const uint16_t*>(ptrs[1][k]);
    s.y = static_cast<uint16_t*>(const_cast<void*>(ptrs[tensors - 1][k]));
    s.w = k ? norm->k_weight : norm->q_weight;
  }
  a->positions = positions;
  a->tokens = static_cast<unsigned>(static_cast<int64_t>(B) * T);
  a->T = T;
  a->by_T = divisor_of(a->T);
  a->eps = norm->eps;
  a->per_head = norm->per_head;
  return BAM_OK;
}

// Workspace of the norms' backward: sums of every CTA it may have.
size_t norm_ws(int H, int Hkv) {
  const int64_t all = (H + kNormPass - 1) / kNormPass + (Hkv + kNormPass - 1) / kNormPass;
  const int64_t ctas = all > kNormMaxCtas ? all : kNormMaxCtas;  // (each part has one at least)
  const int64_t rows = kNormPass * (all < kNormMaxPasses ? all : kNormMaxPasses);
  return align256(static_cast<size_t>(ctas * rows) * kHeadDim * 4);
}

struct SharedWs {
  size_t ml, part, z, spill, table, total;
};
SharedWs shared_ws(const SharedArgs& a, bool marked) {
  SharedWs w;
  const size_t rows = static_cast<size_t>(a.c.B) * a.H;
  w.ml = kStatusBytes;
  w.part = w.ml + align256(rows * a.slots * 8);
  w.z = w.part + align256(rows * a.slots * kHeadDim * 4);
  w.spill = w.z + (marked ? align256(rows * a.zstride * 4) : 0);
  w.table = w.spill + align256(rows * a.spills * kHeadDim * 4);
  w.total = w.table;
  if (a.copies)
    w.total += align256((kTabCopies * static_cast<size_t>(a.H) * a.tab_len + kTabPadFloats) * 4);
  return w;
}

// Sizes of a decode over a shared prefix of up to Pmax keys and Tmax own ones.
bam_status check_shared(int64_t B, int64_t H, int64_t Hkv, int64_t Pmax, int64_t Tmax, int64_t max_pos,
                        int D, SharedArgs* a) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || Pmax < 0 || Tmax < 1 || max_pos < 0 || D < 1)
    return BAM_ERR_INVALID_ARG;
  if (D != kHeadDim) return BAM_ERR_UNSUPPORTED;
  if (Pmax + Tmax > (1 << 28) || max_pos > (1 << 28) || B > 65535 || H > 65535 || B * H > (1 << 24))
    return BAM_ERR_UNSUPPORTED;
  a->c.B = static_cast<int>(B);
  a->c.Hkv = static_cast<int>(Hkv);
  a->H = static_cast<int>(H);
  a->group = static_cast<int>(H / Hkv);
  a->max_pos = static_cast<int>(max_pos);
  a->zstride = (Tmax + 63) / 64 * 64;
  shared_split(a, Pmax, Tmax);
  // (windows are found by 32 bits of 16-byte words)
  if (a->copies && static_cast<int64_t>(a->H) * a->tab_len > INT64_C(0x7FFFFFFF)) return BAM_ERR_UNSUPPORTED;
  return BAM_OK;
}

struct EvictWs {
  size_t count, list, total;
};
EvictWs evict_ws(int B, int Hkv, int budget) {
  EvictWs w;
  const size_t rows = static_cast<size_t>(B) * Hkv;
  w.count = kStatusBytes;
  w.list = w.count + align256(rows * 8);
  w.total = w.list + align256(rows * budget * 4);
  return w;
}

inline bam_status cuda_status(cudaError_t e) { return e == cudaSuccess ? BAM_OK : BAM_ERR_CUDA; }

}  // namespace
}  // namespace bam

namespace bam {
// Lets entry points defined in other files count their launches.
void note_launches(int n) { g_launches.fetch_add(static_cast<uint64_t>(n), std::memory_order_relaxed); }
}  // namespace bam

namespace bam {
namespace {

// bam_attn_decode and its ragged form (lens: device int32 [B], or null).
// Paged form: block_table non-null, kc/vc [num_pages, H, page, D], Tkv the
// longest sequence a block-table row can hold (max_blocks * page).
struct Paging {
  const int* block_table = nullptr;
  int page = 0, max_blocks = 0, num_pages = 0;
};

bam_status decode_impl(const void* q, const void* kc, const void* vc, const int* lens, void* o,
                       int o_fp32, float* lse, int B, int H, int Tkv, int D,
                       const bam_params* p, void* ws, size_t ws_bytes, cudaStream_t stream,
                       const Paging& pg = Paging()) {
  bam_status s = check_sizes(B, H, Tkv, D);
  if (s != BAM_OK) return s;
  if ((s = check_params(p)) != BAM_OK) return s;
  if (!q || !kc || !vc || !o) return BAM_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kc, 16) || !aligned(vc, 16) || !aligned(o, 16) ||
      (lse && !aligned(lse, 4)))
    return BAM_ERR_INVALID_ARG;
  const DecWs w = dec_ws(B, H, Tkv);
  if ((s = check_ws(ws, ws_bytes, w.total)) != BAM_OK) return s;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  DevStatus* status = reinterpret_cast<DevStatus*>(wsb);
  float* table = reinterpret_cast<float*>(wsb + w.table);

  TableArgs ta{table, p->alpha, p->beta, p->mu, status, p->eps, H, w.tab_len, 0, Tkv,
               kTableDecode, p->prior};
  cudaError_t e = launch_kernel(BAM_KERNEL_TABLE, stream, [&] { return launch_table(ta, stream); });
  if (e != cudaSuccess) return BAM_ERR_CUDA;

  DecodeArgs da;
  da.q = static_cast<const uint16_t*>(q);
  da.kc = static_cast<const uint16_t*>(kc);
  da.vc = static_cast<const uint16_t*>(vc);
  da.lens = lens;
  da.block_table = pg.block_table;
  da.page = pg.page;
  da.max_blocks = pg.max_blocks;
  da.num_pages = pg.num_pages;
  da.table = table;
  da.s = p->s;
  da.part = reinterpret_cast<float*>(wsb + w.part);
  da.o = o;
  da.lse = lse;
  da.status = status;
  da.B = B;
  da.H = H;
  da.Tkv = Tkv;
  da.nsplit = w.nsplit;
  da.chunk = w.chunk;
  da.tab_len = w.tab_len;
  da.ssmax = p->ssmax;
  da.o_fp32 = o_fp32 ? 1 : 0;
  e = launch_kernel(BAM_KERNEL_DECODE, stream, [&] { return launch_decode(da, stream); });
  if (e != cudaSuccess) return BAM_ERR_CUDA;
  e = launch_kernel(BAM_KERNEL_DECODE_COMBINE, stream,
                    [&] { return launch_decode_combine(da, stream); });
  return cuda_status(e);
}

bool marks_ok(const bam_marks* m) {
  return m && m->key_pos && m->key_weight && aligned(m->key_pos, 16) && aligned(m->key_weight, 16) &&
         m->max_pos >= 1 && m->max_pos <= kMaxPosition;
}

// bam_kv_append_paged, and with `extended` bam_kv_append_norm_paged.
bam_status append_impl(const void* k, const void* v, const void* q, void* q_out,
                       const int64_t* strides, void* k_pages, void* v_pages, const int* block_table,
                       const int* cache_lens, const int* new_lens, const int* parents, int B, int H,
                       int Hkv, int N, int page, int max_blocks, int num_pages, int D,
                       const bam_qk_norm* norm, const bam_rope* rope, const int* first_pos,
                       const bam_marks* marks, bool extended, void* ws, size_t ws_bytes,
                       cudaStream_t stream) {
  bam_status s = check_cache(B, H, Hkv, N, page, max_blocks, num_pages, D, block_table, cache_lens,
                             new_lens, parents);
  if (s != BAM_OK) return s;
  if (!k || !v || !k_pages || !v_pages || !q != !q_out) return BAM_ERR_INVALID_ARG;
  for (const void* x : {k, v, q, static_cast<const void*>(q_out),
                        static_cast<const void*>(k_pages), static_cast<const void*>(v_pages)})
    if (!aligned(x, 16)) return BAM_ERR_INVALID_ARG;
  if (parents && N > kTreeMax) return BAM_ERR_UNSUPPORTED;
  AppendArgs a = {};
  if (!fill_rope(rope, &a.rope)) return BAM_ERR_INVALID_ARG;
  for (int x = 0; x < 9; ++x) {
    const int h = x < 6 ? Hkv : H;
    const int64_t dense[3] = {static_cast<int64_t>(h) * N * kHeadDim,
                              static_cast<int64_t>(N) * kHeadDim, kHeadDim};
    const int64_t v64 = strides ? strides[x] : dense[x % 3];
    if (x >= 6 && !q) break;
    if (v64 < 0 || v64 % 8 != 0) return BAM_ERR_INVALID_ARG;
    (x < 3 ? a.ks : x < 6 ? a.vs : a.qs)[x % 3] = v64;
  }
  if (norm && !norm_ok(norm)) return BAM_ERR_INVALID_ARG;
  if (marks && !marks_ok(marks)) return BAM_ERR_INVALID_ARG;
  if (!aligned(first_pos, 4)) return BAM_ERR_INVALID_ARG;
  if ((s = check_ws(ws, ws_bytes, BAM_CACHE_WORKSPACE_BYTES)) != BAM_OK) return s;
  if (norm) {
    a.q_weight = norm->q_weight;
    a.k_weight = norm->k_weight;
    a.norm_eps = norm->eps;
    a.per_head = norm->per_head;
  }
  if (marks) {
    a.key_pos = marks->key_pos;
    a.key_weight = marks->key_weight;
    a.max_pos = marks->max_pos;
  }
  a.first_pos = first_pos;
  a.extended = extended;
  a.c = CacheArgs{block_table, cache_lens, new_lens, parents, static_cast<DevStatus*>(ws),
                  B, Hkv, N, page, max_blocks, num_pages};
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_pages = static_cast<uint16_t*>(k_pages);
  a.v_pages = static_cast<uint16_t*>(v_pages);
  a.H = q ? H : 0;
  return cuda_status(
      launch_kernel(BAM_KERNEL_KV_APPEND, stream, [&] { return launch_append(a, stream); }));
}

// bam_kv_keep_paged, and with `marks` bam_kv_keep_marks_paged.
bam_status keep_impl(void* k_pages, void* v_pages, const int* block_table, const int* cache_lens,
                     const int* draft_lens, const int* parents, const int* accepted, int* new_lens,
                     const bam_marks* marks, int B, int Hkv, int N, int page, int max_blocks, int num_pages,
                     int D, void* ws, size_t ws_bytes, cudaStream_t stream) {
  bam_status s = check_cache(B, Hkv, Hkv, N, page, max_blocks, num_pages, D, block_table,
                             cache_lens, draft_lens, parents);
  if (s != BAM_OK) return s;
  if (N > kTreeMax) return BAM_ERR_UNSUPPORTED;
  if (!k_pages || !v_pages || !accepted || !new_lens || !aligned(k_pages, 16) ||
      !aligned(v_pages, 16) || !aligned(accepted, 4) || !aligned(new_lens, 4))
    return BAM_ERR_INVALID_ARG;
  if ((s = check_ws(ws, ws_bytes, BAM_CACHE_WORKSPACE_BYTES)) != BAM_OK) return s;
  KeepArgs a = {};
  a.c = CacheArgs{block_table, cache_lens, draft_lens, parents, static_cast<DevStatus*>(ws),
                  B, Hkv, N, page, max_blocks, num_pages};
  a.k_pages = static_cast<uint16_t*>(k_pages);
  a.v_pages = static_cast<uint16_t*>(v_pages);
  a.accepted = accepted;
  a.new_lens = new_lens;
  if (marks) {
    a.key_pos = marks->key_pos;
    a.key_weight = marks->key_weight;
  }
  return cuda_status(
      launch_kernel(BAM_KERNEL_KV_KEEP, stream, [&] { return launch_keep(a, stream); }));
}

}  // namespace

// For bam_attn_decode_noalloc (decode_noalloc.cu): the argument checks, the
// scratch size and the launches of bam_attn_decode, on caller-given scratch.
bam_status decode_args_ok(const void* q, const void* kc, const void* vc, void* o, float* lse,
                          int B, int H, int Tkv, int D, const bam_params* p) {
  bam_status s = check_sizes(B, H, Tkv, D);
  if (s != BAM_OK) return s;
  if ((s = check_params(p)) != BAM_OK) return s;
  if (!q || !kc || !vc || !o) return BAM_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kc, 16) || !aligned(vc, 16) || !aligned(o, 16) ||
      (lse && !aligned(lse, 4)))
    return BAM_ERR_INVALID_ARG;
  return BAM_OK;
}
size_t decode_scratch_bytes(int B, int H, int Tkv) { return dec_ws(B, H, Tkv).total; }
bam_status decode_plain(const void* q, const void* kc, const void* vc, void* o, int o_fp32,
                        float* lse, int B, int H, int Tkv, int D, const bam_params* p,
                        void* scratch, size_t scratch_bytes, cudaStream_t stream) {
  return decode_impl(q, kc, vc, nullptr, o, o_fp32, lse, B, H, Tkv, D, p, scratch, scratch_bytes,
                     stream);
}
// Reads and clears the status words at `st` (device memory) after
// synchronising `stream`; the sticky-error rules of bam_attn_check_status.
bam_status read_and_clear_status(void* st_dev, cudaStream_t stream) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return BAM_ERR_CUDA;
  DevStatus st;
  if (cudaMemcpy(&st, st_dev, sizeof(st), cudaMemcpyDeviceToHost) != cudaSuccess)
    return BAM_ERR_CUDA;
  // A status area no call has initialised holds no error.
  if (st.magic[0] != kStatusMagic0 || st.magic[1] != kStatusMagic1) return BAM_OK;
  // Clears abort, code, site and block; the magic and the debug count stay.
  if (cudaMemset(st_dev, 0, 4 * sizeof(int)) != cudaSuccess) return BAM_ERR_CUDA;
  if (st.code == BAM_DEV_BAD_ARG && st.abort == 0) return BAM_ERR_INVALID_ARG;
  if (st.code == BAM_DEV_BOUNDS) return BAM_ERR_BOUNDS;
  if (st.code != BAM_DEV_OK || st.abort != 0) return BAM_ERR_TIMEOUT;
  return BAM_OK;
}
// Debug builds: arms the give-up count of the status words at `st_dev`.
bam_status arm_giveup(void* st_dev, int n) {
#ifdef BAM_DEBUG
  DevStatus st;
  if (cudaDeviceSynchronize() != cudaSuccess) return BAM_ERR_CUDA;
  if (cudaMemcpy(&st, st_dev, sizeof(st), cudaMemcpyDeviceToHost) != cudaSuccess)
    return BAM_ERR_CUDA;
  if (st.magic[0] != kStatusMagic0 || st.magic[1] != kStatusMagic1) {
    std::memset(&st, 0, sizeof(st));
    st.magic[0] = kStatusMagic0;
    st.magic[1] = kStatusMagic1;
  }
  st.giveup = n;
  if (cudaMemcpy(st_dev, &st, sizeof(st), cudaMemcpyHostToDevice) != cudaSuccess)
    return BAM_ERR_CUDA;
  return BAM_OK;
#else
  (void)st_dev;
  (void)n;
  return BAM_ERR_UNSUPPORTED;
#endif
}
}  // namespace bam

using namespace bam;

extern "C" {

size_t bam_attn_workspace_size(int op, int B, int H, int T, int D) {
  if (check_sizes(B, H, T, D) != BAM_OK) return 0;
  switch (op) {
    case BAM_OP_FWD:
      // the larger of the causal and non-causal layouts
      return fwd_ws(H, T, 0).total;
    case BAM_OP_BWD:
      return bwd_ws(B, H, T, 0).total;
    case BAM_OP_DECODE:
      return dec_ws(B, H, T).total;
    default:
      return 0;
  }
}

bam_status bam_attn_fwd(const void* q, const void* k, const void* v, void* o, int o_fp32,
                        float* lse, int B, int H, int T, int D, const bam_params* p, void* ws,
                        size_t ws_bytes, cudaStream_t stream) {
  bam_status s = check_sizes(B, H, T, D);
  if (s != BAM_OK) return s;
  if ((s = check_params(p)) != BAM_OK) return s;
  if (!q || !k || !v || !o) return BAM_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      (lse && !aligned(lse, 4)))
    return BAM_ERR_INVALID_ARG;
  const FwdWs w = fwd_ws(H, T, p->causal);
  if ((s = check_ws(ws, ws_bytes, w.total)) != BAM_OK) return s;
  const int BH = B * H;
  CUtensorMap tq, tk, tv;
  if (!encode_rows(&tq, q, BH, T) || !encode_rows(&tk, k, BH, T) || !encode_rows(&tv, v, BH, T))
    return BAM_ERR_CUDA;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  DevStatus* status = reinterpret_cast<DevStatus*>(wsb);
  float* table = reinterpret_cast<float*>(wsb + w.table);
  const TableGeom g = table_geom(T, p->causal);

  TableArgs ta{table, p->alpha, p->beta, p->mu, status, p->eps, H, g.len, g.off, 0,
               kTableByDistance, p->prior};
  cudaError_t e = launch_kernel(BAM_KERNEL_TABLE, stream, [&] { return launch_table(ta, stream); });
  if (e != cudaSuccess) return BAM_ERR_CUDA;

  FwdArgs fa;
  fa.o = o;
  fa.lse = lse;
  fa.table = table;
  fa.s = p->s;
  fa.status = status;
  fa.B = B;
  fa.H = H;
  fa.T = T;
  fa.causal = p->causal;
  fa.ssmax = p->ssmax;
  fa.o_fp32 = o_fp32 ? 1 : 0;
  fa.tab_len = g.len;
  fa.tab_off = g.off;
  // O by TMA stores: fp32 in 32-column boxes, bf16 in 64-column boxes; 128
  // rows a box for the paired kernel, 32 (one warp's rows) for the
  // single-tile kernel.
  CUtensorMap to, to32;
  if (!(o_fp32 ? encode_acc_rows(&to, o, BH, T) : encode_rows(&to, o, BH, T)) ||
      !(o_fp32 ? encode_acc_rows(&to32, o, BH, T, 32) : encode_rows(&to32, o, BH, T, 32)))
    return BAM_ERR_CUDA;
  e = launch_kernel(BAM_KERNEL_FWD, stream,
                    [&] { return launch_fwd(tq, tk, tv, to, to32, fa, stream); });
  return cuda_status(e);
}

bam_status bam_attn_decode(const void* q, const void* kc, const void* vc, void* o, int o_fp32,
                           float* lse, int B, int H, int Tkv, int D, const bam_params* p,
                           void* ws, size_t ws_bytes, cudaStream_t stream) {
  return decode_impl(q, kc, vc, nullptr, o, o_fp32, lse, B, H, Tkv, D, p, ws, ws_bytes, stream);
}

bam_status bam_attn_decode_paged(const void* q, const void* k_pages, const void* v_pages,
                                 const int* block_table, const int* cache_lens, void* o,
                                 int o_fp32, float* lse, int B, int H, int page, int max_blocks,
                                 int num_pages, int D, const bam_params* p, void* ws,
                                 size_t ws_bytes, cudaStream_t stream) {
  if (!block_table || !aligned(block_table, 4) || !cache_lens || !aligned(cache_lens, 4))
    return BAM_ERR_INVALID_ARG;
  if (page < 64 || page % 64 != 0 || max_blocks < 1 || num_pages < 1) return BAM_ERR_INVALID_ARG;
  const int64_t tmax = static_cast<int64_t>(page) * max_blocks;
  if (tmax > (1 << 28)) return BAM_ERR_UNSUPPORTED;
  Paging pg;
  pg.block_table = block_table;
  pg.page = page;
  pg.max_blocks = max_blocks;
  pg.num_pages = num_pages;
  return decode_impl(q, k_pages, v_pages, cache_lens, o, o_fp32, lse, B, H,
                     static_cast<int>(tmax), D, p, ws, ws_bytes, stream, pg);
}

bam_status bam_attn_decode_varlen(const void* q, const void* kc, const void* vc,
                                  const int* cache_lens, void* o, int o_fp32, float* lse, int B,
                                  int H, int Tmax, int D, const bam_params* p, void* ws,
                                  size_t ws_bytes, cudaStream_t stream) {
  if (!cache_lens || !aligned(cache_lens, 4)) return BAM_ERR_INVALID_ARG;
  return decode_impl(q, kc, vc, cache_lens, o, o_fp32, lse, B, H, Tmax, D, p, ws, ws_bytes,
                     stream);
}

bam_status bam_kv_append_paged(const void* k, const void* v, const void* q, void* q_out,
                               const int64_t* strides, void* k_pages, void* v_pages,
                               const int* block_table, const int* cache_lens,
                               const int* new_lens, const int* parents, int B, int H, int Hkv,
                               int N, int page, int max_blocks, int num_pages, int D,
                               const bam_rope* rope, void* ws, size_t ws_bytes,
                               cudaStream_t stream) {
  return append_impl(k, v, q, q_out, strides, k_pages, v_pages, block_table, cache_lens, new_lens,
                     parents, B, H, Hkv, N, page, max_blocks, num_pages, D, nullptr, rope, nullptr,
                     nullptr, false, ws, ws_bytes, stream);
}

bam_status bam_kv_append_norm_paged(const void* k, const void* v, const void* q, void* q_out,
                                    const int64_t* strides, void* k_pages, void* v_pages,
                                    const int* block_table, const int* cache_lens,
                                    const int* new_lens, const int* parents, int B, int H, int Hkv,
                                    int N, int page, int max_blocks, int num_pages, int D,
                                    const bam_qk_norm* norm, const bam_rope* rope,
                                    const int* first_pos, const bam_marks* marks, void* ws,
                                    size_t ws_bytes, cudaStream_t stream) {
  return append_impl(k, v, q, q_out, strides, k_pages, v_pages, block_table, cache_lens, new_lens,
                     parents, B, H, Hkv, N, page, max_blocks, num_pages, D, norm, rope, first_pos,
                     marks, true, ws, ws_bytes, stream);
}

bam_status bam_qk_norm_fwd(const void* q, const void* k, void* q_out, void* k_out,
                           const int64_t* strides, const int* positions, int B, int H, int Hkv,
                           int T, int D, const bam_qk_norm* norm, const bam_rope* rope,
                           cudaStream_t stream) {
  NormArgs a = {};
  const void* ptrs[2][2] = {{q, k}, {q_out, k_out}};
  const bam_status s = fill_norm(&a, ptrs, 2, strides, positions, B, H, Hkv, T, D, norm, rope);
  if (s != BAM_OK) return s;
  return cuda_status(
      launch_kernel(BAM_KERNEL_QK_NORM, stream, [&] { return launch_norm_fwd(a, stream); }));
}

size_t bam_qk_norm_workspace_size(int B, int H, int Hkv, int T, int D) {
  if (B < 1 || H < 1 || Hkv < 1 || T < 1 || D != kHeadDim || H > 65535 || Hkv > 65535 ||
      static_cast<int64_t>(B) * T > 0x7FFFFFFF)
    return 0;
  return norm_ws(H, Hkv);
}

bam_status bam_qk_norm_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out,
                           void* dq, void* dk, const int64_t* strides, float* dq_weight,
                           float* dk_weight, const int* positions, int B, int H, int Hkv, int T,
                           int D, const bam_qk_norm* norm, const bam_rope* rope, void* ws,
                           size_t ws_bytes, cudaStream_t stream) {
  NormArgs a = {};
  const void* ptrs[3][2] = {{q, k}, {dq_out, dk_out}, {dq, dk}};
  bam_status s = fill_norm(&a, ptrs, 3, strides, positions, B, H, Hkv, T, D, norm, rope);
  if (s != BAM_OK) return s;
  if (!dq_weight || !dk_weight || !aligned(dq_weight, 4) || !aligned(dk_weight, 4))
    return BAM_ERR_INVALID_ARG;
  if ((s = check_ws(ws, ws_bytes, norm_ws(H, Hkv))) != BAM_OK) return s;
  a.side[0].dw = dq_weight;
  a.side[1].dw = dk_weight;
  a.part = static_cast<float*>(ws);
  norm_bwd_config(&a, sm_count());
  cudaError_t e =
      launch_kernel(BAM_KERNEL_QK_NORM_BWD, stream, [&] { return launch_norm_bwd(a, stream); });
  if (e != cudaSuccess) return BAM_ERR_CUDA;
  return cuda_status(launch_kernel(BAM_KERNEL_QK_NORM_FINISH, stream,
                                   [&] { return launch_norm_bwd_finish(a, stream); }));
}

size_t bam_attn_shared_workspace_size(int B, int H, int Hkv, int Pmax, int Tmax, int max_pos, int D) {
  SharedArgs a = {};
  if (check_shared(B, H, Hkv, Pmax, Tmax, max_pos, D, &a) != BAM_OK) return 0;
  return shared_ws(a, max_pos > 0).total;
}

bam_status bam_attn_decode_shared_paged(const void* q, const void* k_pages, const void* v_pages,
                                        const int* block_table, const int* cache_lens,
                                        const int* prefix_table, const int* prefix_len,
                                        const int* q_pos, const bam_marks* marks, float decay,
                                        void* o, int o_fp32, float* lse, int B, int H, int Hkv,
                                        int page, int max_blocks, int prefix_blocks, int num_pages,
                                        int D, const bam_params* p, void* ws, size_t ws_bytes,
                                        cudaStream_t stream) {
  bam_status s = check_cache(B, H, Hkv, 1, page, max_blocks, num_pages, D, block_table, cache_lens,
                             nullptr, nullptr);
  if (s != BAM_OK) return s;
  if ((s = check_params(p)) != BAM_OK) return s;
  if (!q || !k_pages || !v_pages || !o) return BAM_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(o, 16) ||
      !aligned(lse, 4) || !aligned(prefix_table, 4) || !aligned(prefix_len, 4) || !aligned(q_pos, 4))
    return BAM_ERR_INVALID_ARG;
  if (!prefix_table != !prefix_len || !prefix_table != (prefix_blocks == 0) || prefix_blocks < 0)
    return BAM_ERR_INVALID_ARG;
  if (!marks != !q_pos || (marks && !marks_ok(marks)) || !(decay >= 0.0f && decay <= 1.0f))
    return BAM_ERR_INVALID_ARG;
  SharedArgs a = {};
  if ((s = check_shared(B, H, Hkv, static_cast<int64_t>(prefix_blocks) * page,
                        static_cast<int64_t>(max_blocks) * page, marks ? marks->max_pos : 0, D, &a)) !=
      BAM_OK)
    return s;
  const SharedWs w = shared_ws(a, marks != nullptr);
  if ((s = check_ws(ws, ws_bytes, w.total)) != BAM_OK) return s;
  // Pages in boxes of 32 keys, and of a tile of 64 for the prefix.
  CUtensorMap tk, tv, tk64, tv64;
  if (!encode_rows(&tk, k_pages, num_pages * Hkv, page, 32) ||
      !encode_rows(&tv, v_pages, num_pages * Hkv, page, 32) ||
      (a.copies && (!encode_rows(&tk64, k_pages, num_pages * Hkv, page, 64) ||
                    !encode_rows(&tv64, v_pages, num_pages * Hkv, page, 64))))
    return BAM_ERR_CUDA;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  a.c = CacheArgs{block_table, cache_lens, nullptr, nullptr, static_cast<DevStatus*>(ws),
                  B, Hkv, 1, page, max_blocks, num_pages};
  a.q = static_cast<const uint16_t*>(q);
  a.prefix_table = prefix_table;
  a.prefix_len = prefix_len;
  a.prefix_blocks = prefix_blocks;
  a.q_pos = q_pos;
  if (marks) {
    a.key_pos = marks->key_pos;
    a.key_weight = marks->key_weight;
    a.z = reinterpret_cast<float*>(wsb + w.z);
  }
  a.decay = decay;
  a.alpha = p->alpha;
  a.beta = p->beta;
  a.mu = p->mu;
  a.s = p->s;
  a.eps = p->eps;
  a.prior = p->prior;
  a.ssmax = p->ssmax;
  a.o = o;
  a.o_fp32 = o_fp32 ? 1 : 0;
  a.lse = lse;
  a.ml = reinterpret_cast<float2*>(wsb + w.ml);
  a.part = reinterpret_cast<float*>(wsb + w.part);
  if (a.copies) {
    a.spill = reinterpret_cast<float*>(wsb + w.spill);
    a.table = reinterpret_cast<float*>(wsb + w.table);
  }
  cudaError_t e =
      launch_kernel(BAM_KERNEL_SHARED_PREP, stream, [&] { return launch_shared_prep(a, stream); });
  if (e != cudaSuccess) return BAM_ERR_CUDA;
  if (a.copies) {
    e = launch_kernel(BAM_KERNEL_PREFIX, stream, [&] { return launch_prefix(tk64, tv64, a, stream); });
    if (e != cudaSuccess) return BAM_ERR_CUDA;
  }
  e = launch_kernel(BAM_KERNEL_SHARED, stream, [&] { return launch_shared(tk, tv, a, stream); });
  if (e != cudaSuccess) return BAM_ERR_CUDA;
  return cuda_status(
      launch_kernel(BAM_KERNEL_SHARED_END, stream, [&] { return launch_shared_end(a, stream); }));
}

size_t bam_kv_evict_workspace_size(int B, int Hkv, int Tmax, int budget) {
  if (B < 1 || Hkv < 1 || Tmax < 1 || budget < 1 || B > 65535 || Hkv > 65535 || Tmax > (1 << 28))
    return 0;
  return evict_ws(B, Hkv, budget < Tmax ? budget : Tmax).total;
}

bam_status bam_kv_evict_paged(void* k_pages, void* v_pages, const int* block_table,
                              const int* cache_lens, const bam_marks* marks, const int* out_table,
                              int* new_lens, int B, int Hkv, int page, int max_blocks,
                              int out_blocks, int num_pages, int D, int budget, int sink,
                              int recent, void* ws, size_t ws_bytes, cudaStream_t stream) {
  bam_status s = check_cache(B, Hkv, Hkv, 1, page, max_blocks, num_pages, D, block_table, cache_lens,
                             nullptr, nullptr);
  if (s != BAM_OK) return s;
  if (!k_pages || !v_pages || !new_lens || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(new_lens, 4) || !aligned(out_table, 4) || !marks_ok(marks))
    return BAM_ERR_INVALID_ARG;
  if (budget < 1 || sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > budget)
    return BAM_ERR_INVALID_ARG;
  // (rows of the pages are numbered with 32 bits: more than any device holds)
  if (static_cast<int64_t>(num_pages) * Hkv > 0xFFFFFFFFll / page) return BAM_ERR_UNSUPPORTED;
  const int Tmax = page * max_blocks;
  if (budget > Tmax) budget = Tmax;  // no sequence is longer: nothing leaves
  if (!out_table != (out_blocks == 0) || out_blocks < 0 ||
      (out_table && static_cast<int64_t>(out_blocks) * page < budget))
    return BAM_ERR_INVALID_ARG;
  const EvictWs w = evict_ws(B, Hkv, budget);
  if ((s = check_ws(ws, ws_bytes, w.total)) != BAM_OK) return s;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  EvictArgs a = {};
  a.c = CacheArgs{block_table, cache_lens, nullptr, nullptr, static_cast<DevStatus*>(ws),
                  B, Hkv, 1, page, max_blocks, num_pages};
  a.k_pages = static_cast<uint16_t*>(k_pages);
  a.v_pages = static_cast<uint16_t*>(v_pages);
  a.key_pos = marks->key_pos;
  a.key_weight = marks->key_weight;
  a.out_table = out_table;
  a.out_blocks = out_blocks;
  a.new_lens = new_lens;
  a.budget = budget;
  a.sink = sink;
  a.recent = recent;
  a.count = reinterpret_cast<int2*>(wsb + w.count);
  a.list = reinterpret_cast<unsigned*>(wsb + w.list);
  a.by_page = divisor_of(static_cast<unsigned>(page));
  cudaError_t e =
      launch_kernel(BAM_KERNEL_EVICT_SELECT, stream, [&] { return launch_evict_select(a, stream); });
  if (e != cudaSuccess) return BAM_ERR_CUDA;
  return cuda_status(
      launch_kernel(BAM_KERNEL_EVICT_MOVE, stream, [&] { return launch_evict_move(a, stream); }));
}

size_t bam_attn_tree_workspace_size(int B, int H, int Hkv, int N, int Tmax, int D) {
  if (B < 1 || H < 1 || Hkv < 1 || N < 1 || Tmax < 1 || D != kHeadDim || H % Hkv != 0 ||
      N > kTreeMax || B > 65535 || H > 65535 || Tmax > (1 << 28))
    return 0;
  return tree_ws(B, H, Hkv, N, Tmax).total;
}

bam_status bam_attn_decode_tree_paged(const void* q, const void* k_pages, const void* v_pages,
                                      const int* block_table, const int* cache_lens,
                                      const int* draft_lens, const int* parents, void* o,
                                      int o_fp32, float* lse, int B, int H, int Hkv, int N,
                                      int page, int max_blocks, int num_pages, int D,
                                      const bam_params* p, void* ws, size_t ws_bytes,
                                      cudaStream_t stream) {
  bam_status s = check_cache(B, H, Hkv, N, page, max_blocks, num_pages, D, block_table, cache_lens,
                             draft_lens, parents);
  if (s != BAM_OK) return s;
  if (N > kTreeMax) return BAM_ERR_UNSUPPORTED;
  if ((s = check_params(p)) != BAM_OK) return s;
  if (!q || !k_pages || !v_pages || !o) return BAM_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(o, 16) ||
      (lse && !aligned(lse, 4)))
    return BAM_ERR_INVALID_ARG;
  const int Tmax = page * max_blocks;
  const TreeWs w = tree_ws(B, H, Hkv, N, Tmax);
  if ((s = check_ws(ws, ws_bytes, w.total)) != BAM_OK) return s;
  // Pages as rows of 64 dimensions, in boxes of one tile of 64 keys.
  CUtensorMap tk, tv;
  if (!encode_rows(&tk, k_pages, num_pages * Hkv, page, 64) ||
      !encode_rows(&tv, v_pages, num_pages * Hkv, page, 64))
    return BAM_ERR_CUDA;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  TreeArgs a = {};
  a.c = CacheArgs{block_table, cache_lens, draft_lens, parents, static_cast<DevStatus*>(ws),
                  B, Hkv, N, page, max_blocks, num_pages};
  a.q = static_cast<const uint16_t*>(q);
  a.v_pages = static_cast<const uint16_t*>(v_pages);
  a.alpha = p->alpha;
  a.beta = p->beta;
  a.mu = p->mu;
  a.s = p->s;
  a.o = o;
  a.lse = lse;
  a.plan = reinterpret_cast<int64_t*>(wsb + w.plan);
  a.table = reinterpret_cast<float*>(wsb + w.table);
  a.part_ml = reinterpret_cast<float2*>(wsb + w.ml);
  a.cut = reinterpret_cast<CutItem*>(wsb + w.cut);
  a.part = reinterpret_cast<float*>(wsb + w.part);
  a.eps = p->eps;
  a.H = H;
  a.group = H / Hkv;
  a.prior = p->prior;
  a.ssmax = p->ssmax;
  a.o_fp32 = o_fp32 ? 1 : 0;
  a.tab_len = tree_table_len(Tmax);
  a.tab_zero = tree_table_zero(Tmax);
  a.rows = w.rows;
  if (!tree_config(&a, sm_count())) return BAM_ERR_CUDA;
  cudaError_t e =
      launch_kernel(BAM_KERNEL_TREE_PREP, stream, [&] { return launch_tree_prep(a, stream); });
  if (e != cudaSuccess) return BAM_ERR_CUDA;
  e = launch_kernel(BAM_KERNEL_TREE, stream, [&] { return launch_tree(tk, tv, a, stream); });
  if (e != cudaSuccess) return BAM_ERR_CUDA;
  return cuda_status(launch_kernel(BAM_KERNEL_TREE_COMBINE, stream,
                                   [&] { return launch_tree_combine(a, stream); }));
}

bam_status bam_kv_keep_paged(void* k_pages, void* v_pages, const int* block_table,
                             const int* cache_lens, const int* draft_lens, const int* parents,
                             const int* accepted, int* new_lens, int B, int Hkv, int N, int page,
                             int max_blocks, int num_pages, int D, void* ws, size_t ws_bytes,
                             cudaStream_t stream) {
  return keep_impl(k_pages, v_pages, block_table, cache_lens, draft_lens, parents, accepted, new_lens, nullptr,
                   B, Hkv, N, page, max_blocks, num_pages, D, ws, ws_bytes, stream);
}

bam_status bam_kv_keep_marks_paged(void* k_pages, void* v_pages, const int* block_table,
                                   const int* cache_lens, const int* draft_lens, const int* parents,
                                   const int* accepted, int* new_lens, const bam_marks* marks, int B,
                                   int Hkv, int N, int page, int max_blocks, int num_pages, int D,
                                   void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!marks_ok(marks)) return BAM_ERR_INVALID_ARG;
  return keep_impl(k_pages, v_pages, block_table, cache_lens, draft_lens, parents, accepted, new_lens, marks,
                   B, Hkv, N, page, max_blocks, num_pages, D, ws, ws_bytes, stream);
}

static bam_status bounded_call(int op, const void* words) {
  // Words of each operator, the place of its strides' flag (-1: none) and their number.
  constexpr int kWords[] = {26, 14, 20, 25, 20, 19}, kFlag[] = {4, 4, 6, -1, -1, -1},
                kSteps[] = {9, 12, 18, 0, 0, 0};
  const int x = op - BAM_CALL_KV_APPEND_NORM, flag = kFlag[x];
  int64_t w[26], steps[18];
  std::memcpy(w, words, kWords[x] * sizeof(int64_t));
  const int64_t* strides = nullptr;
  if (flag >= 0) {
    if (w[flag] != 0 && w[flag] != 1) return BAM_ERR_INVALID_ARG;
    if (w[flag]) {
      std::memcpy(steps, static_cast<const char*>(words) + kWords[x] * sizeof(int64_t),
                  kSteps[x] * sizeof(int64_t));
      strides = steps;
    }
  }
  bool fits = true;
  auto p = [&](int i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(w[i])); };
  auto ip = [&](int i) { return static_cast<int*>(p(i)); };
  auto fp = [&](int i) { return static_cast<float*>(p(i)); };
  auto n = [&](int i) {
    fits &= w[i] == static_cast<int>(w[i]);
    return static_cast<int>(w[i]);
  };
  auto norm = [&](int i) { return static_cast<const bam_qk_norm*>(p(i)); };
  auto rope = [&](int i) { return static_cast<const bam_rope*>(p(i)); };
  auto marks = [&](int i) { return static_cast<const bam_marks*>(p(i)); };
  auto st = [&](int i) { return static_cast<cudaStream_t>(p(i)); };
  auto sz = [&](int i) { return static_cast<size_t>(w[i]); };
  constexpr int kFirst[] = {11, 6, 10, 13, 7, 9}, kInts[] = {8, 5, 5, 8, 10, 7};
  int i[10];
  for (int y = 0; y < kInts[x]; ++y) i[y] = n(kFirst[x] + y);
  const int o_fp32 = op == BAM_CALL_DECODE_SHARED ? n(11) : 0;
  float decay = 0.0f;
  if (op == BAM_CALL_DECODE_SHARED) {  // its bits
    const int bits = n(9);
    std::memcpy(&decay, &bits, sizeof(decay));
  }
  if (!fits) return BAM_ERR_INVALID_ARG;
  switch (op) {
    case BAM_CALL_KV_APPEND_NORM:
      return bam_kv_append_norm_paged(p(0), p(1), p(2), p(3), strides, p(5), p(6), ip(7), ip(8), ip(9),
                                      ip(10), i[0], i[1], i[2], i[3], i[4], i[5], i[6], i[7], norm(19),
                                      rope(20), ip(21), marks(22), p(23), sz(24), st(25));
    case BAM_CALL_QK_NORM_FWD:
      return bam_qk_norm_fwd(p(0), p(1), p(2), p(3), strides, ip(5), i[0], i[1], i[2], i[3], i[4],
                             norm(11), rope(12), st(13));
    case BAM_CALL_QK_NORM_BWD:
      return bam_qk_norm_bwd(p(0), p(1), p(2), p(3), p(4), p(5), strides, fp(7), fp(8), ip(9), i[0],
                             i[1], i[2], i[3], i[4], norm(15), rope(16), p(17), sz(18), st(19));
    case BAM_CALL_DECODE_SHARED:
      return bam_attn_decode_shared_paged(p(0), p(1), p(2), ip(3), ip(4), ip(5), ip(6), ip(7), marks(8),
                                          decay, p(10), o_fp32, fp(12), i[0], i[1], i[2], i[3], i[4],
                                          i[5], i[6], i[7], static_cast<const bam_params*>(p(21)), p(22),
                                          sz(23), st(24));
    case BAM_CALL_KV_KEEP_MARKS:
      return bam_kv_keep_marks_paged(p(0), p(1), ip(2), ip(3), ip(4), ip(5), ip(6), ip(7), marks(8), i[0], i[1],
                                     i[2], i[3], i[4], i[5], i[6], p(16), sz(17), st(18));
    default:
      return bam_kv_evict_paged(p(0), p(1), ip(2), ip(3), marks(4), ip(5), ip(6), i[0], i[1], i[2], i[3],
                                i[4], i[5], i[6], i[7], i[8], i[9], p(17), sz(18), st(19));
  }
}

bam_status bam_paged_call(int op, const void* words) {
  constexpr int kWords[] = {23, 22, 18}, kStrides = 4;  // place of the append's strides
  if (words && op > BAM_CALL_KV_KEEP && op <= BAM_CALL_KV_KEEP_MARKS) return bounded_call(op, words);
  if (!words || op < BAM_CALL_KV_APPEND || op > BAM_CALL_KV_KEEP) return BAM_ERR_INVALID_ARG;
  int64_t w[23], strides[9];
  std::memcpy(w, words, kWords[op] * sizeof(int64_t));
  bool fits = true;
  auto p = [&](int x) { return reinterpret_cast<void*>(static_cast<uintptr_t>(w[x])); };
  auto ip = [&](int x) { return static_cast<const int*>(p(x)); };
  auto n = [&](int x) {
    fits &= w[x] == static_cast<int>(w[x]);
    return static_cast<int>(w[x]);
  };
  auto st = [&](int x) { return static_cast<cudaStream_t>(p(x)); };
  auto sz = [&](int x) { return static_cast<size_t>(w[x]); };
  int i[8];
  const int first = op == BAM_CALL_KV_APPEND ? 11 : op == BAM_CALL_DECODE_TREE ? 10 : 8;
  const int ints = op == BAM_CALL_KV_KEEP ? 7 : 8;
  for (int x = 0; x < ints; ++x) i[x] = n(first + x);
  const int o_fp32 = op == BAM_CALL_DECODE_TREE ? n(8) : 0;
  if (!fits) return BAM_ERR_INVALID_ARG;
  switch (op) {
    case BAM_CALL_KV_APPEND:
      if (w[kStrides] != 0 && w[kStrides] != 1) return BAM_ERR_INVALID_ARG;
      if (w[kStrides])
        std::memcpy(strides, static_cast<const char*>(words) + sizeof(w), sizeof(strides));
      return bam_kv_append_paged(p(0), p(1), p(2), p(3), w[kStrides] ? strides : nullptr, p(5), p(6),
                                 ip(7), ip(8), ip(9), ip(10), i[0], i[1], i[2], i[3], i[4], i[5],
                                 i[6], i[7], static_cast<const bam_rope*>(p(19)), p(20), sz(21),
                                 st(22));
    case BAM_CALL_DECODE_TREE:
      return bam_attn_decode_tree_paged(p(0), p(1), p(2), ip(3), ip(4), ip(5), ip(6), p(7), o_fp32,
                                        static_cast<float*>(p(9)), i[0], i[1], i[2], i[3], i[4],
                                        i[5], i[6], i[7], static_cast<const bam_params*>(p(18)),
                                        p(19), sz(20), st(21));
    default:
      return bam_kv_keep_paged(p(0), p(1), ip(2), ip(3), ip(4), ip(5), ip(6),
                               static_cast<int*>(p(7)), i[0], i[1], i[2], i[3], i[4], i[5], i[6],
                               p(15), sz(16), st(17));
  }
}

bam_status bam_attn_bwd(const void* q, const void* k, const void* v, const void* o, int o_fp32,
                        const float* lse, const void* dO, void* dq, void* dk, void* dv,
                        float* dalpha, float* dbeta, float* dmu, float* ds, int B, int H, int T,
                        int D, const bam_params* p, void* ws, size_t ws_bytes,
                        cudaStream_t stream) {
  bam_status s = check_sizes(B, H, T, D);
  if (s != BAM_OK) return s;
  if ((s = check_params(p)) != BAM_OK) return s;
  if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv || !dalpha || !dbeta || !dmu ||
      !ds)
    return BAM_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      !aligned(dO, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) ||
      !aligned(lse, 16))
    return BAM_ERR_INVALID_ARG;
  const BwdWs w = bwd_ws(B, H, T, p->causal);
  if ((s = check_ws(ws, ws_bytes, w.total)) != BAM_OK) return s;
  const int BH = B * H;
  CUtensorMap tq, tk, tv, tdo;
  if (!encode_rows(&tq, q, BH, T) || !encode_rows(&tk, k, BH, T) ||
      !encode_rows(&tv, v, BH, T) || !encode_rows(&tdo, dO, BH, T))
    return BAM_ERR_CUDA;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  DevStatus* status = reinterpret_cast<DevStatus*>(wsb);
  float* table = reinterpret_cast<float*>(wsb + w.table);
  const TableGeom g = table_geom(T, p->causal);

  BwdArgs ba;
  ba.tab = TableArgs{table, p->alpha, p->beta, p->mu, status, p->eps, H, g.len, g.off, 0,
                     kTableBackward, p->prior};
  ba.o = o;
  ba.dO = static_cast<const uint16_t*>(dO);
  ba.lse = lse;
  ba.table = table;
  ba.alpha = p->alpha;
  ba.beta = p->beta;
  ba.s = p->s;
  ba.delta = reinterpret_cast<float*>(wsb + w.delta);
  ba.dq_acc = reinterpret_cast<float*>(wsb + w.dq_acc);
  ba.rowacc = reinterpret_cast<float*>(wsb + w.rowacc);
  ba.dq = static_cast<uint16_t*>(dq);
  ba.dk = static_cast<uint16_t*>(dk);
  ba.dv = static_cast<uint16_t*>(dv);
  ba.dalpha = dalpha;
  ba.dbeta = dbeta;
  ba.dmu = dmu;
  ba.ds = ds;
  ba.status = status;
  ba.B = B;
  ba.H = H;
  ba.T = T;
  ba.nkb = (T + 127) / 128;
  ba.causal = p->causal;
  ba.ssmax = p->ssmax;
  ba.o_fp32 = o_fp32 ? 1 : 0;
  ba.tab_len = g.len;
  ba.tab_off = g.off;
  cudaError_t e =
      launch_kernel(BAM_KERNEL_BWD_PREP, stream, [&] { return launch_bwd_prep(ba, stream); });
  if (e != cudaSuccess) return BAM_ERR_CUDA;
  CUtensorMap tdq, tdk, tdv;
  if (!encode_acc_rows(&tdq, ba.dq_acc, BH, T) || !encode_rows(&tdk, dk, BH, T) ||
      !encode_rows(&tdv, dv, BH, T))
    return BAM_ERR_CUDA;
  e = launch_kernel(BAM_KERNEL_BWD, stream,
                    [&] { return launch_bwd(tq, tk, tv, tdo, tdq, tdk, tdv, ba, stream); });
  if (e != cudaSuccess) return BAM_ERR_CUDA;
  e = launch_kernel(BAM_KERNEL_BWD_FINAL, stream, [&] { return launch_bwd_final(ba, stream); });
  return cuda_status(e);
}

bam_status bam_attn_check_status(void* ws, cudaStream_t stream) {
  if (!ws || !aligned(ws, 256)) return BAM_ERR_WORKSPACE;
  return read_and_clear_status(ws, stream);
}

bam_status bam_attn_debug_arm_giveup(void* ws, int n) {
  if (n < 0) return BAM_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256)) return BAM_ERR_WORKSPACE;
  return arm_giveup(ws, n);
}

int bam_attn_debug_build(void) {
#ifdef BAM_DEBUG
  return 1;
#else
  return 0;
#endif
}

const char* bam_status_string(bam_status s) {
  switch (s) {
    case BAM_OK:
      return "ok";
    case BAM_ERR_INVALID_ARG:
      return "invalid argument";
    case BAM_ERR_UNSUPPORTED:
      return "unsupported size or option";
    case BAM_ERR_CUDA:
      return "CUDA error";
    case BAM_ERR_TIMEOUT:
      return "device-side wait gave up";
    case BAM_ERR_WORKSPACE:
      return "workspace missing, misaligned or too small";
    case BAM_ERR_BOUNDS:
      return "a bulk copy failed its bounds check (debug build)";
  }
  return "unknown status";
}

bam_status bam_attn_profile_events(int which, cudaEvent_t before, cudaEvent_t after) {
  if (which < 0 || which >= BAM_KERNEL_COUNT) return BAM_ERR_INVALID_ARG;
  std::lock_guard<std::mutex> g(g_prof_mu);
  g_prof_before[which] = before;
  g_prof_after[which] = after;
  return BAM_OK;
}

uint64_t bam_attn_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

}  // extern "C"
