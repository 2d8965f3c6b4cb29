// Host side of the calls around a paged K/V cache: argument checks (nothing
// is launched when one fails) and launches.  Included by hs2.cu, whose
// helpers (tensor maps, shared-memory limits, launch accounting) it uses.
#pragma once

#include "evict.cuh"
#include "norm_rope.cuh"

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

template <bool KV8, bool PAIRS>
int launch_norm_rope(const NormRopeParams& p, dim3 grid, cudaStream_t st) {
  const Range range("hs2 qk_norm_rope");
  qk_norm_rope_kernel<KV8, PAIRS><<<grid, NR_THREADS, 0, st>>>(p);
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
  if ((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight)) & 1u) return HS2_ERR_UNSUPPORTED;
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
  // one token a CTA until that fills the GPU several times over
  p.tok_per_cta = p.n >= sm_count() * 8 * NR_MAX_TOK ? NR_MAX_TOK : 1;
  const dim3 grid(static_cast<unsigned>((p.n + p.tok_per_cta - 1) / p.tok_per_cta));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cache->kv_dtype == HS2_KV_E4M3)
    return rope->interleaved ? launch_norm_rope<true, true>(p, grid, st) : launch_norm_rope<true, false>(p, grid, st);
  return rope->interleaved ? launch_norm_rope<false, true>(p, grid, st) : launch_norm_rope<false, false>(p, grid, st);
}

int hs2_cache_evict(const hs2_cache* cache, const int32_t* seq_len, const float* acc, float* acc_out,
                    int64_t acc_stride, int32_t keep, int32_t recent, int32_t* idx, int32_t* new_len, void* stream) {
  using namespace hs2;
  if (int rc = check_cache(cache, true)) return rc;
  if (!seq_len || !acc || !idx || !new_len) return HS2_ERR_INVALID_ARG;
  if (keep < 1 || recent < 0 || recent > keep || new_len == seq_len) return HS2_ERR_INVALID_ARG;
  if (acc_stride <= 0 || acc_stride % 4) return HS2_ERR_INVALID_ARG;
  if (keep > (1 << 24)) return HS2_ERR_UNSUPPORTED;
  if (!aligned16(acc) || (acc_out && !aligned16(acc_out))) return HS2_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(seq_len) | reinterpret_cast<uintptr_t>(idx) |
       reinterpret_cast<uintptr_t>(new_len)) & 3u)
    return HS2_ERR_UNSUPPORTED;
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
  // shared memory for the longest part a row of this cache can have
  const int64_t longest = std::min<int64_t>(acc_stride, static_cast<int64_t>(cache->max_pages) * cache->page);
  const int64_t part = ((longest + EV_CTAS - 1) / EV_CTAS + 3) & ~int64_t(3);
  p.part_cap = static_cast<int>(std::min<int64_t>(part, EV_MAX_PART));
  const uint32_t smem = static_cast<uint32_t>(sizeof(EvictSmem)) + static_cast<uint32_t>(p.part_cap) * 4u;
  const dim3 grid(EV_CTAS, static_cast<unsigned>(cache->Hkv), static_cast<unsigned>(cache->n_seqs));
  const Range range("hs2 cache_evict");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (kv8) {
    if (int rc = set_smem(cache_evict_kernel<true>, smem)) return rc;
    cache_evict_kernel<true><<<grid, EV_THREADS, smem, st>>>(p);
  } else {
    if (int rc = set_smem(cache_evict_kernel<false>, smem)) return rc;
    cache_evict_kernel<false><<<grid, EV_THREADS, smem, st>>>(p);
  }
  return launched();
}

}  // extern "C"
