// Host side of the calls around a paged K/V cache: argument checks (nothing
// is launched when one fails) and launches.  Included by hs2.cu, whose
// helpers (tensor maps, shared-memory limits, launch accounting) it uses.
#pragma once

#include "cache_weights.cuh"
#include "evict.cuh"
#include "norm_rope.cuh"
#include "tree_attn.cuh"
#include "varlen.cuh"

namespace hs2 {
namespace {

constexpr int kMaxSeqs = 4096;
constexpr int kMaxGroup = 16;  // query heads per KV head

// Strides of [tokens][H][128] rows: positive, `align` elements, no overlap.
int check_rows(int64_t tok, int64_t head, int H, int64_t align) {
  if (tok <= 0 || head <= 0) return HS2_ERR_INVALID_ARG;
  if (tok % align || head % align || head < HD || tok < static_cast<int64_t>(H) * head) return HS2_ERR_UNSUPPORTED;
  return HS2_OK;
}

int log2_of(int page) {
  switch (page) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
  }
}

bool overlap(const void* a, const void* b, uint64_t bytes) {
  const uint64_t x = reinterpret_cast<uint64_t>(a), y = reinterpret_cast<uint64_t>(b);
  return x < y ? y - x < bytes : x - y < bytes;
}

// table: whether the call reads the page table.
int check_cache(const hs2_cache* c, bool table) {
  if (!c || !c->k || !c->v) return HS2_ERR_INVALID_ARG;
  if (c->Hkv <= 0 || c->n_pages <= 0 || c->reserved != 0) return HS2_ERR_INVALID_ARG;
  if (c->kv_dtype != HS2_KV_BF16 && c->kv_dtype != HS2_KV_E4M3) return HS2_ERR_INVALID_ARG;
  const bool kv8 = c->kv_dtype == HS2_KV_E4M3;
  if (kv8 && (!c->k_scale || !c->v_scale)) return HS2_ERR_INVALID_ARG;
  if (c->d != HD || log2_of(c->page) < 0 || c->Hkv > 256) return HS2_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->n_pages) * c->page > (int64_t(1) << 31) - 256) return HS2_ERR_UNSUPPORTED;
  if (int rc = check_rows(c->tok_stride, c->head_stride, c->Hkv, kv8 ? 16 : 8)) return rc;
  if (!aligned16(c->k) || !aligned16(c->v)) return HS2_ERR_UNSUPPORTED;
  if (kv8 && ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) & 3u))
    return HS2_ERR_UNSUPPORTED;
  if (table) {
    if (!c->page_table || c->n_seqs <= 0 || c->max_pages <= 0) return HS2_ERR_INVALID_ARG;
    if (c->n_seqs > kMaxSeqs || static_cast<int64_t>(c->max_pages) * c->page > (int64_t(1) << 30))
      return HS2_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(c->page_table) & 3u) return HS2_ERR_UNSUPPORTED;
  }
  return HS2_OK;
}

// 3-D map over e4m3 codes [tokens][heads][128], a box of one head's codes of
// box_t tokens, swizzled (128 bytes) where the tensor cores read them.
int make_map_codes(CUtensorMap* m, const void* base, int64_t L, int H, int64_t tok_stride, int64_t head_stride,
                   int box_t, bool swizzled) {
  EncodeTiledFn enc = encode_fn();
  if (!enc || (g_flags & FLAG_FAIL_TMAP)) return HS2_ERR_CUDA;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(HD), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(L)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride), static_cast<cuuint64_t>(tok_stride)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(HD), 1u, static_cast<cuuint32_t>(box_t)};
  const cuuint32_t es[3] = {1u, 1u, 1u};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE,
                         swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? HS2_OK : HS2_ERR_CUDA;
}

// A map over a pool of the cache, one box per page.
int make_pool_map(CUtensorMap* m, const hs2_cache* c, const void* pool, bool codes_swizzled = false) {
  const int tokens = c->n_pages * c->page;
  return c->kv_dtype == HS2_KV_E4M3
             ? make_map_codes(m, pool, tokens, c->Hkv, c->tok_stride, c->head_stride, c->page,
                              codes_swizzled)
             : make_map(m, pool, tokens, c->Hkv, c->tok_stride, c->head_stride, 1, c->page);
}

int check_group(int Hq, int Hkv) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv) return HS2_ERR_INVALID_ARG;
  return Hq / Hkv > kMaxGroup ? HS2_ERR_UNSUPPORTED : HS2_OK;
}

int check_draft(const hs2_cache* c, const hs2_draft* d) {
  if (!d || d->n_tok < 0 || d->reserved != 0 || !d->cu_draft || !d->ctx_len) return HS2_ERR_INVALID_ARG;
  if (d->max_draft < 1 || d->max_draft > 64) return HS2_ERR_INVALID_ARG;
  if (int rc = check_group(d->Hq, c->Hkv)) return rc;
  if (int rc = check_rows(d->q_tok_stride, d->q_head_stride, d->Hq, 8)) return rc;
  if (((reinterpret_cast<uintptr_t>(d->cu_draft) | reinterpret_cast<uintptr_t>(d->ctx_len)) & 3u) ||
      (reinterpret_cast<uintptr_t>(d->mask) & 7u))
    return HS2_ERR_UNSUPPORTED;
  return HS2_OK;
}

// rows: of a token tile (query rows of one KV head)
TreeParams tree_params(const hs2_cache* c, const hs2_draft* d, int rows) {
  TreeParams p{};
  p.B = c->n_seqs;
  p.Hq = d->Hq;
  p.Hkv = c->Hkv;
  p.G = d->Hq / c->Hkv;
  p.R = rows / p.G;
  p.page_log2 = log2_of(c->page);
  p.n_pages = c->n_pages;
  p.max_pages = c->max_pages;
  p.max_len = static_cast<int64_t>(c->max_pages) * c->page;
  p.n_tok = d->n_tok;
  p.max_draft = d->max_draft;
  p.table = c->page_table;
  p.cu = d->cu_draft;
  p.ctx = d->ctx_len;
  p.mask = d->mask;
  p.q_tok = d->q_tok_stride;
  p.q_head = d->q_head_stride;
  p.scale_log2 = scale_log2(HD);
  p.ksc = c->k_scale;
  p.vsc = c->v_scale;
  p.limit_ns = g_wait_limit_ns;
  p.flags = g_flags;
  return p;
}

// Workspace of the tree attention: per CTA two parts of up to 128 rows
// (un-normalised O, then (m, l)) and the unit its last part begins.
struct TreePlan {
  int ctas;
  size_t ml_off, unit_off, bytes;
};

TreePlan tree_plan() {
  TreePlan t{};
  t.ctas = sm_count();
  t.ml_off = static_cast<size_t>(t.ctas) * 2 * 128 * 128 * sizeof(float);
  t.unit_off = t.ml_off + static_cast<size_t>(t.ctas) * 2 * 128 * sizeof(float2);
  t.bytes = t.unit_off + static_cast<size_t>(t.ctas) * sizeof(int4);
  return t;
}

template <int TOK>
int launch_norm_rope(const NormRopeParams& p, bool kv8, bool pairs, cudaStream_t st) {
  const Range range("hs2 qk_norm_rope");
  const unsigned grid = static_cast<unsigned>((p.n + TOK - 1) / TOK);
  if (kv8 && pairs)
    qk_norm_rope_kernel<true, true, TOK><<<grid, NR_THREADS, 0, st>>>(p);
  else if (kv8)
    qk_norm_rope_kernel<true, false, TOK><<<grid, NR_THREADS, 0, st>>>(p);
  else if (pairs)
    qk_norm_rope_kernel<false, true, TOK><<<grid, NR_THREADS, 0, st>>>(p);
  else
    qk_norm_rope_kernel<false, false, TOK><<<grid, NR_THREADS, 0, st>>>(p);
  return launched();
}

// Clusters of `ctas` CTAs of cache_evict_kernel that run at once on the current
// device (a GPC's SMs are shared out in whole clusters), asked once per device.
int active_clusters(int ctas) {
  static std::mutex mu;
  static int known[128][EV_MAX_CTAS + 1];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 0;
  std::lock_guard<std::mutex> lock(mu);
  int& n = known[dev][ctas];
  if (n == 0) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ctas);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(EV_THREADS);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, cache_evict_kernel<false, EV_THREADS>, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = sm_count() / ctas;
    }
  }
  return n;
}

template <typename K>
int launch_evict(K kernel, const EvictParams& p, const hs2_cache* c, int ctas, int threads, uint32_t smem,
                 cudaStream_t st) {
  if (int rc = set_smem(kernel, smem)) return rc;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ctas);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(c->Hkv), static_cast<unsigned>(c->n_seqs));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return HS2_ERR_CUDA;
  }
  return launched();
}

// The attention, then the join of split units; the second kernel's launch
// overlaps the first one's run (it waits on the device for its end).
template <bool KV8, int RB>
int launch_tree(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p, int ctas,
                int most_rows, cudaStream_t st) {
  constexpr uint32_t smem = TreeSmem<KV8, RB>::BYTES;
  if (int rc = set_smem(tree_attn_kernel<KV8, RB>, smem)) return rc;
  tree_attn_kernel<KV8, RB><<<static_cast<unsigned>(ctas), tr_threads(KV8), smem, st>>>(mq, mk, mv, p);
  if (int rc = launched()) return rc;
  const int rows = std::min(p.R * p.G, most_rows);  // of a unit
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(std::min(rows, 32)));
  cfg.blockDim = dim3(32 * TM_WARPS);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, tree_merge_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return HS2_ERR_CUDA;
  }
  return launched();
}

template <bool KV8>
int launch_weights(const CUtensorMap& mq, const CUtensorMap& mk, const WeightParams& p, cudaStream_t st) {
  constexpr uint32_t smem = WeightSmem<KV8>::BYTES;
  if (int rc = set_smem(cache_weights_kernel<KV8>, smem)) return rc;
  cache_weights_kernel<KV8><<<static_cast<unsigned>(sm_count()), CW_THREADS, smem, st>>>(mq, mk, p);
  return launched();
}

}  // namespace
}  // namespace hs2

extern "C" {

int hs2_qk_norm_rope(const hs2_cache* cache, const hs2_rope* rope, const void* q, const void* k, const void* v,
                     const void* q_weight, const void* k_weight, const double* inv_freq, const int32_t* positions,
                     const int32_t* slots, void* q_out, void* stream) {
  using namespace hs2;
  int rc = check_cache(cache, false);
  if (rc) return rc;
  if (!rope || rope->n < 0 || rope->Hq <= 0 || rope->reserved != 0) return HS2_ERR_INVALID_ARG;
  if (rope->interleaved != 0 && rope->interleaved != 1) return HS2_ERR_INVALID_ARG;
  if (!(rope->eps >= 0.f)) return HS2_ERR_INVALID_ARG;
  if (rope->rot <= 0 || rope->rot > HD) return HS2_ERR_INVALID_ARG;
  if (rope->rot % 16 || rope->Hq > kMaxGroup * 256) return HS2_ERR_UNSUPPORTED;
  if ((rc = check_rows(rope->q_tok_stride, rope->q_head_stride, rope->Hq, 8))) return rc;
  if ((rc = check_rows(rope->out_tok_stride, rope->out_head_stride, rope->Hq, 8))) return rc;
  // the key and value rows may be views into wider rows (no check that a
  // token's heads end before the next token: both only step over them)
  if (rope->kv_tok_stride <= 0 || rope->kv_head_stride <= 0) return HS2_ERR_INVALID_ARG;
  if (rope->kv_tok_stride % 8 || rope->kv_head_stride % 8 || rope->kv_head_stride < HD) return HS2_ERR_UNSUPPORTED;
  if (rope->n == 0) return HS2_OK;
  if (!q || !k || !v || !inv_freq || !positions || !q_out) return HS2_ERR_INVALID_ARG;
  if ((q_weight == nullptr) != (k_weight == nullptr)) return HS2_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out)) return HS2_ERR_UNSUPPORTED;
  if (!aligned16(q_weight) || !aligned16(k_weight)) return HS2_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(inv_freq) & 7u) ||
      ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slots)) & 3u))
    return HS2_ERR_UNSUPPORTED;
  // in place only as itself: rows are read before they are written one by one
  if (q == q_out && (rope->q_tok_stride != rope->out_tok_stride || rope->q_head_stride != rope->out_head_stride))
    return HS2_ERR_INVALID_ARG;
  NormRopeParams p{};
  p.n = rope->n;
  p.Hq = rope->Hq;
  p.Hkv = cache->Hkv;
  p.rot = rope->rot;
  p.eps = rope->eps;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_tok = rope->q_tok_stride;
  p.q_head = rope->q_head_stride;
  p.kv_tok = rope->kv_tok_stride;
  p.kv_head = rope->kv_head_stride;
  p.out_tok = rope->out_tok_stride;
  p.out_head = rope->out_head_stride;
  p.wq = static_cast<const __nv_bfloat16*>(q_weight);
  p.wk = static_cast<const __nv_bfloat16*>(k_weight);
  p.inv_freq = inv_freq;
  p.pos = positions;
  p.slots = slots;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.kc = static_cast<uint8_t*>(cache->k);
  p.vc = static_cast<uint8_t*>(cache->v);
  p.ksc = cache->k_scale;
  p.vsc = cache->v_scale;
  p.c_tok = cache->tok_stride;
  p.c_head = cache->head_stride;
  p.n_slots = static_cast<int64_t>(cache->n_pages) * cache->page;
  // a CTA per token until that fills the GPU a few times over, then a warp per
  // token (norm_rope.cuh has both sides' times)
  const bool kv8 = cache->kv_dtype == HS2_KV_E4M3, pairs = rope->interleaved != 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return p.n >= sm_count() * 16 ? launch_norm_rope<8>(p, kv8, pairs, st) : launch_norm_rope<1>(p, kv8, pairs, st);
}

int hs2_cache_evict(const hs2_cache* cache, const int32_t* seq_len, const float* acc, float* acc_out,
                    int64_t acc_stride, int32_t keep, int32_t recent, int32_t* idx, int32_t* new_len, void* stream) {
  using namespace hs2;
  if (int rc = check_cache(cache, true)) return rc;
  if (!seq_len || !acc || !idx || !new_len) return HS2_ERR_INVALID_ARG;
  if (keep < 1 || recent < 0 || recent > keep) return HS2_ERR_INVALID_ARG;
  if (acc_stride <= 0 || acc_stride % 4) return HS2_ERR_INVALID_ARG;
  if (keep > (1 << 24) || acc_stride > (int64_t(1) << 31)) return HS2_ERR_UNSUPPORTED;
  if (!aligned16(acc) || (acc_out && !aligned16(acc_out))) return HS2_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(seq_len) | reinterpret_cast<uintptr_t>(idx) |
       reinterpret_cast<uintptr_t>(new_len)) & 3u)
    return HS2_ERR_UNSUPPORTED;
  // the CTAs of a row have to read the same lengths and weights, whichever rows are done
  const uint64_t acc_bytes = static_cast<uint64_t>(acc_stride) * 4u * static_cast<uint64_t>(cache->n_seqs) * cache->Hkv;
  if (overlap(seq_len, new_len, static_cast<uint64_t>(cache->n_seqs) * 4u)) return HS2_ERR_INVALID_ARG;
  if (acc_out && acc_out != acc && overlap(acc, acc_out, acc_bytes)) return HS2_ERR_INVALID_ARG;
  EvictParams p{};
  const bool kv8 = cache->kv_dtype == HS2_KV_E4M3;
  p.Hkv = cache->Hkv;
  p.page_log2 = log2_of(cache->page);
  p.n_pages = cache->n_pages;
  p.max_pages = cache->max_pages;
  p.keep = keep;
  p.recent = recent;
  p.k = static_cast<uint8_t*>(cache->k);
  p.v = static_cast<uint8_t*>(cache->v);
  p.tok_b = cache->tok_stride * (kv8 ? 1 : 2);
  p.head_b = cache->head_stride * (kv8 ? 1 : 2);
  p.ksc = cache->k_scale;
  p.vsc = cache->v_scale;
  p.table = cache->page_table;
  p.len = seq_len;
  p.acc = acc;
  p.acc_out = acc_out;
  p.acc_stride = acc_stride;
  p.idx = idx;
  p.new_len = new_len;
  // CTAs a row: as many as let every row run at once, up to a portable cluster
  // (16 rows of up to 131072 positions: two waves of clusters of 8 take 80 us, one of
  // clusters of 6 53).  More rows than SMs: smaller CTAs, two an SM (256 rows of
  // 2000: 69 us against 88).
  const int64_t rows = static_cast<int64_t>(cache->n_seqs) * cache->Hkv;
  int ctas = EV_MAX_CTAS;
  while (ctas > 1 && rows > active_clusters(ctas)) --ctas;
  // shared memory for the longest part a row of this cache can have, and its pages
  const int64_t longest = std::min<int64_t>(acc_stride, static_cast<int64_t>(cache->max_pages) * cache->page);
  const int64_t part = ((longest + ctas - 1) / ctas + 3) & ~int64_t(3);
  p.part_cap = static_cast<int>(std::min<int64_t>(part, EV_MAX_PART));
  p.table_cap = std::min(cache->max_pages, EV_MAX_TABLE);
  const uint32_t smem = static_cast<uint32_t>(sizeof(EvictSmem)) + static_cast<uint32_t>(p.part_cap + p.table_cap) * 4u;
  const Range range("hs2 cache_evict");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows > active_clusters(1))
    return kv8 ? launch_evict(cache_evict_kernel<true, EV_THREADS_MANY>, p, cache, ctas, EV_THREADS_MANY, smem, st)
               : launch_evict(cache_evict_kernel<false, EV_THREADS_MANY>, p, cache, ctas, EV_THREADS_MANY, smem, st);
  return kv8 ? launch_evict(cache_evict_kernel<true, EV_THREADS>, p, cache, ctas, EV_THREADS, smem, st)
             : launch_evict(cache_evict_kernel<false, EV_THREADS>, p, cache, ctas, EV_THREADS, smem, st);
}

int hs2_varlen_attn(const hs2_varlen* shape, const void* q, const void* k, const void* v, const int32_t* cu_q,
                    const int32_t* cu_k, void* o, float* lse, void* stream) {
  using namespace hs2;
  const hs2_varlen* s = shape;
  if (!s || s->n_seqs <= 0 || s->total_q < 0 || s->total_k < 0) return HS2_ERR_INVALID_ARG;
  if (int rc = check_group(s->Hq, s->Hkv)) return rc;
  if (s->d != HD || s->n_seqs > kMaxSeqs) return HS2_ERR_UNSUPPORTED;
  if (int rc = check_rows(s->q_tok_stride, s->q_head_stride, s->Hq, 8)) return rc;
  if (int rc = check_rows(s->kv_tok_stride, s->kv_head_stride, s->Hkv, 8)) return rc;
  if (!cu_q) return HS2_ERR_INVALID_ARG;
  if (s->total_q == 0) return HS2_OK;
  if (!q || !o || (s->total_k > 0 && (!k || !v))) return HS2_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      ((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(cu_k)) & 3u))
    return HS2_ERR_UNSUPPORTED;
  VarlenParams p{};
  p.B = s->n_seqs;
  p.total_q = s->total_q;
  p.total_k = s->total_k;
  p.Hq = s->Hq;
  p.Hkv = s->Hkv;
  p.G = s->Hq / s->Hkv;
  p.rows_tok = 128 / p.G;
  p.cu_q = cu_q;
  p.cu_k = cu_k ? cu_k : cu_q;
  p.scale_log2 = scale_log2(HD);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.o_tok = s->q_tok_stride;
  p.o_head = s->q_head_stride;
  p.lse = lse;
  p.limit_ns = g_wait_limit_ns;
  p.flags = g_flags;
  // at least one item per KV head for every tile (pair) any split of total_q
  // tokens into n_seqs sequences can have; single tiles while all of them run
  // at once (7 short prompts: 12.4 us, in pairs 14.4)
  const int64_t singles = s->total_q / p.rows_tok + s->n_seqs;
  p.tiles = singles * s->Hkv <= sm_count() ? 1 : 2;
  const int64_t items = p.tiles == 1 ? singles : s->total_q / (2 * p.rows_tok) + s->n_seqs;
  if (items * s->Hkv > (int64_t(1) << 31) - 1) return HS2_ERR_UNSUPPORTED;
  CUtensorMap mq, mk, mv;
  if (int rc = make_map(&mq, q, s->total_q, s->Hq, s->q_tok_stride, s->q_head_stride, p.G, p.rows_tok)) return rc;
  mk = mv = mq;  // without keys no tile of them is loaded
  if (s->total_k > 0) {
    if (int rc = make_map(&mk, k, s->total_k, s->Hkv, s->kv_tok_stride, s->kv_head_stride, 1, 128)) return rc;
    if (int rc = make_map(&mv, v, s->total_k, s->Hkv, s->kv_tok_stride, s->kv_head_stride, 1, 128)) return rc;
  }
  if (int rc = set_smem(varlen_attn_kernel, VL_SMEM)) return rc;
  const Range range("hs2 varlen_attn");
  varlen_attn_kernel<<<static_cast<unsigned>(items * s->Hkv), FL_THREADS, VL_SMEM, static_cast<cudaStream_t>(stream)>>>(
      mq, mk, mv, p);
  return launched();
}

int hs2_tree_attn_workspace(const hs2_cache* cache, const hs2_draft* draft, size_t* workspace_bytes) {
  using namespace hs2;
  if (int rc = check_cache(cache, true)) return rc;
  if (int rc = check_draft(cache, draft)) return rc;
  if (!workspace_bytes) return HS2_ERR_INVALID_ARG;
  *workspace_bytes = tree_plan().bytes;
  return HS2_OK;
}

int hs2_tree_attn(const hs2_cache* cache, const hs2_draft* draft, const void* q, void* o, float* lse,
                  void* workspace, size_t workspace_bytes, void* stream) {
  using namespace hs2;
  if (int rc = check_cache(cache, true)) return rc;
  if (int rc = check_draft(cache, draft)) return rc;
  if (draft->n_tok == 0) return HS2_OK;
  if (!q || !o || !workspace) return HS2_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return HS2_ERR_UNSUPPORTED;
  const TreePlan plan = tree_plan();
  if (workspace_bytes < plan.bytes) return HS2_ERR_WORKSPACE;
  // blocks of 32 rows where they hold a sequence's drafted tokens (blocks of 64
  // lost: e4m3, 48 rows over 4 x 32768 tokens 145 us, 124 in one block)
  const int most = draft->max_draft * (draft->Hq / cache->Hkv);
  const int rb = most <= 32 ? 32 : 128;
  TreeParams p = tree_params(cache, draft, rb);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.lse = lse;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(w);
  p.part_ml = reinterpret_cast<float2*>(w + plan.ml_off);
  p.part_unit = reinterpret_cast<int4*>(w + plan.unit_off);
  CUtensorMap mq, mk, mv;
  if (int rc = make_map(&mq, q, draft->n_tok, draft->Hq, draft->q_tok_stride, draft->q_head_stride, p.G, p.R))
    return rc;
  // blocks of 32 rows take K's codes as they are, a full block converts them
  if (int rc = make_pool_map(&mk, cache, cache->k, rb == 32)) return rc;
  if (int rc = make_pool_map(&mv, cache, cache->v)) return rc;
  const Range range("hs2 tree_attn");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool kv8 = cache->kv_dtype == HS2_KV_E4M3;
  if (rb == 32)
    return kv8 ? launch_tree<true, 32>(mq, mk, mv, p, plan.ctas, most, st)
               : launch_tree<false, 32>(mq, mk, mv, p, plan.ctas, most, st);
  return kv8 ? launch_tree<true, 128>(mq, mk, mv, p, plan.ctas, most, st)
             : launch_tree<false, 128>(mq, mk, mv, p, plan.ctas, most, st);
}

int hs2_cache_weights(const hs2_cache* cache, const hs2_draft* draft, const void* q, const float* lse,
                      const uint8_t* counted, float* acc, int64_t acc_stride, void* stream) {
  using namespace hs2;
  if (int rc = check_cache(cache, true)) return rc;
  if (int rc = check_draft(cache, draft)) return rc;
  if (acc_stride <= 0 || acc_stride % 4) return HS2_ERR_INVALID_ARG;
  if (draft->n_tok == 0) return HS2_OK;
  if (!q || !lse || !acc) return HS2_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(acc) || (reinterpret_cast<uintptr_t>(lse) & 3u)) return HS2_ERR_UNSUPPORTED;
  WeightParams p{};
  p.t = tree_params(cache, draft, CW_ROWS);
  p.lse = lse;
  p.counted = counted;
  p.acc = acc;
  p.acc_stride = acc_stride;
  p.t.max_len = std::min(p.t.max_len, acc_stride);
  p.t.q = static_cast<const __nv_bfloat16*>(q);
  CUtensorMap mq, mk;
  if (int rc = make_map(&mq, q, draft->n_tok, draft->Hq, draft->q_tok_stride, draft->q_head_stride, p.t.G, p.t.R))
    return rc;
  if (int rc = make_pool_map(&mk, cache, cache->k, true)) return rc;
  const Range range("hs2 cache_weights");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cache->kv_dtype == HS2_KV_E4M3 ? launch_weights<true>(mq, mk, p, st) : launch_weights<false>(mq, mk, p, st);
}

}  // extern "C"
