// Causal grouped-query attention over packed prompts of different lengths.
// Per sequence o_i = softmax_{j <= i + nk - nq} (q_i . k_j / sqrt(d)) v_j.
//
// The pipeline is kernel (1)'s (flash.cuh: TMA loads, one MMA-issuing thread,
// two softmax warpgroups taking turns, S / P / O in tensor memory); what
// differs is the shape of the work:
//
//   rows     a tile's 128 rows are 128 / G tokens times the G query heads of a
//            KV head, so a short prompt fills tiles (100 tokens at G = 8 are
//            800 rows, 7 tiles, where tiles of one head would be 8 of them,
//            each 100 / 128 full) and its K and V are loaded once for all
//            heads; a CTA takes two consecutive tiles of one KV head;
//   order    CTA -> (KV head, item), items longest first over all sequences:
//            item k lies at level p (the p-th tile pair of its sequence) with
//            C(p + 1) <= k < C(p), C(p) = sum_b max(0, pairs_b - p), found by
//            a binary search that one warp makes while the others set up.
//            Only the sequences' total and their number size the grid, so the
//            lengths stay on the device; the surplus CTAs (fewer than the
//            sequences times the KV heads) come last and leave at once;
//   edges    keys behind a sequence's end are other sequences' or padding: a
//            score there is replaced by -inf (whatever it was) and the V rows
//            are zeroed in shared memory by an otherwise idle warp before
//            the last product reads them.
//
// Bound by the tensor cores and the serial chain through the softmax, as
// kernel (1) is; short prompts by the latency of a CTA's few steps.
#pragma once

#include "attn_tile.cuh"

namespace hs2 {

struct VarlenParams {
  int B, total_q, total_k, Hq, Hkv, G, rows_tok;
  const int32_t *cu_q, *cu_k;
  float scale_log2;
  __nv_bfloat16* o;
  int64_t o_tok, o_head;
  float* lse;  // [Hq][total_q] or null
  uint64_t limit_ns;
  uint32_t flags;
};

struct VarlenBars {
  uint64_t q_full;
  uint64_t full_k[FL_STAGES], full_v[FL_STAGES], empty_k[FL_STAGES], empty_v[FL_STAGES];
  uint64_t v_raw;  // the last V tile landed, its rows behind the sequence not yet zeroed
  uint64_t s_full[2], p_ready[2], o_done[2];
  uint64_t fin;
  uint32_t tmem_slot;
  int abort;
  int item_g, item_b, item_pair;  // item_g < 0: nothing to do
  int q0, nq, k0, nk;
};
static_assert(sizeof(VarlenBars) <= 256, "barrier area");
static_assert(4096 * 4 <= 2 * TILE_BYTES, "the item search borrows the first K/V stage");

// One warp finds this CTA's item (see the order above); scratch holds B ints.
__device__ __forceinline__ void varlen_find_item(const VarlenParams& p, int* scratch, VarlenBars* bars) {
  const int lane = threadIdx.x & 31;
  const int per = 2 * p.rows_tok;
  bool ok = true;
  int most = 0;
  int64_t sum = 0;
  for (int b = lane; b < p.B; b += 32) {
    const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
    ok &= q0 >= 0 && q0 <= q1 && q1 <= p.total_q && k0 >= 0 && k0 <= k1 && k1 <= p.total_k;
    const int n = ok ? (q1 - q0 + per - 1) / per : 0;
    scratch[b] = n;
    most = max(most, n);
    sum += n;
  }
  ok = __all_sync(0xffffffffu, ok);
  most = __reduce_max_sync(0xffffffffu, most);
  const unsigned total = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(sum));  // <= total_q / per + B
  const int g = ok && total > 0 ? static_cast<int>(blockIdx.x / total) : p.Hkv;
  if (!ok && lane == 0 && blockIdx.x == 0) report(HS2_ERR_INDEX, 701);
  if (g >= p.Hkv) {
    if (lane == 0) bars->item_g = -1;
    return;
  }
  const unsigned k = blockIdx.x % total;
  __syncwarp();
  auto at_least = [&](int level) {  // C(level)
    unsigned c = 0;
    for (int b = lane; b < p.B; b += 32) c += static_cast<unsigned>(max(0, scratch[b] - level));
    return __reduce_add_sync(0xffffffffu, c);
  };
  int lo = 0, hi = most;  // C(lo) > k >= C(hi)
  unsigned c_hi = 0;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const unsigned c = at_least(mid);
    if (c > k) {
      lo = mid;
    } else {
      hi = mid;
      c_hi = c;
    }
  }
  unsigned r = k - c_hi;  // rank among the sequences with more than lo pairs
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const unsigned m = __ballot_sync(0xffffffffu, b < p.B && scratch[b] > lo);
    const unsigned c = __popc(m);
    if (r < c) {
      if ((m >> lane & 1u) && __popc(m & ((1u << lane) - 1u)) == static_cast<int>(r)) {
        bars->item_g = g;
        bars->item_b = b;
        bars->item_pair = lo;
        bars->q0 = p.cu_q[b];
        bars->nq = p.cu_q[b + 1] - p.cu_q[b];
        bars->k0 = p.cu_k[b];
        bars->nk = p.cu_k[b + 1] - p.cu_k[b];
      }
      return;
    }
    r -= c;
  }
}

__global__ void __launch_bounds__(FL_THREADS, 1)
    varlen_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const VarlenParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  VarlenBars* bars = reinterpret_cast<VarlenBars*>(smem + FL_BAR_OFF);
  const uint32_t q_base = smem_u32(smem + FL_Q_OFF);
  const uint32_t kv_base = smem_u32(smem + FL_KV_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    for (int s = 0; s < FL_STAGES; ++s) {
      mbar_init(&bars->full_k[s], 1);
      mbar_init(&bars->full_v[s], 1);
      mbar_init(&bars->empty_k[s], 1);
      mbar_init(&bars->empty_v[s], 1);
    }
    mbar_init(&bars->v_raw, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->p_ready[x], 4);
      mbar_init(&bars->o_done[x], 1);
    }
    mbar_init(&bars->fin, 1);
    bars->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 2) {
    varlen_find_item(p, reinterpret_cast<int*>(smem + FL_KV_OFF), bars);
    fence_proxy_async_smem();  // TMA writes the borrowed stage after the barrier
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;

  // ---- this CTA's two tiles (B may be absent); tile x reads key tiles 0 .. n_x - 1
  const int g = bars->item_g;
  const bool work = g >= 0;
  const int R = p.rows_tok;
  const int nq = bars->nq, nk = bars->nk, q0 = bars->q0, k0 = bars->k0;
  const int tok0 = work ? bars->item_pair * 2 * R : 0;
  const int off = nk - nq;
  const bool has_b = work && tok0 + R < nq;
  auto key_tiles = [&](int x) {
    const int last = min(nq, tok0 + (x + 1) * R) - 1;
    return max(0, last + off + 1 + 127) >> 7;
  };
  const int nA = work ? key_tiles(0) : 0;
  const int nB = has_b ? key_tiles(1) : 0;
  const int n = max(nA, nB);
  const int v_rows = nk - (n - 1) * 128;  // rows of the last tile that are keys
  const bool fix = n > 0 && v_rows < 128;

  if (warp == 0) {
    // =========================================================== TMA loads
    if (lane == 0 && !(p.flags & FLAG_SKIP_LOADS) && n > 0) {
      const int nqt = has_b ? 2 : 1;
      const uint32_t half = static_cast<uint32_t>(R * p.G) * 128u;
      mbar_arrive_expect_tx(&bars->q_full, static_cast<uint32_t>(nqt) * 2u * half);
      for (int x = 0; x < nqt; ++x) {
        uint8_t* qd = smem + FL_Q_OFF + x * TILE_BYTES;
        tma_load_3d(qd, &tmQ, &bars->q_full, 0, g * p.G, q0 + tok0 + x * R);
        tma_load_3d(qd + HALF_BYTES, &tmQ, &bars->q_full, 64, g * p.G, q0 + tok0 + x * R);
      }
      int last = -1;
      for (int j = 0; j < n; ++j) {
        const int s = j % FL_STAGES;
        const uint32_t par = ((j / FL_STAGES) - 1) & 1;
        if (j >= FL_STAGES && !mbar_wait(&bars->empty_k[s], par, p.limit_ns, abort_flag, 711)) break;
        uint8_t* kd = smem + FL_KV_OFF + s * 2 * TILE_BYTES;
        mbar_arrive_expect_tx(&bars->full_k[s], TILE_BYTES);
        tma_load_3d(kd, &tmK, &bars->full_k[s], 0, g, k0 + j * 128);
        tma_load_3d(kd + HALF_BYTES, &tmK, &bars->full_k[s], 64, g, k0 + j * 128);
        if (j >= FL_STAGES && !mbar_wait(&bars->empty_v[s], par, p.limit_ns, abort_flag, 712)) {
          wait_done(&bars->full_k[s], (j / FL_STAGES) & 1, p.limit_ns, 713);
          break;
        }
        // a last tile to be mended reaches full_v through warp 2
        uint64_t* vbar = fix && j == n - 1 ? &bars->v_raw : &bars->full_v[s];
        mbar_arrive_expect_tx(vbar, TILE_BYTES);
        tma_load_3d(kd + TILE_BYTES, &tmV, vbar, 0, g, k0 + j * 128);
        tma_load_3d(kd + TILE_BYTES + HALF_BYTES, &tmV, vbar, 64, g, k0 + j * 128);
        last = j;
      }
      // never leave a TMA write in flight into memory the CTA gives back
      for (int u = max(0, last - FL_STAGES + 1); u <= last; ++u) {
        const int s = u % FL_STAGES;
        wait_done(&bars->full_k[s], (u / FL_STAGES) & 1, p.limit_ns, 714);
        if (fix && u == n - 1)
          wait_done(&bars->v_raw, 0, p.limit_ns, 715);
        else
          wait_done(&bars->full_v[s], (u / FL_STAGES) & 1, p.limit_ns, 715);
      }
      wait_done(&bars->q_full, 0, p.limit_ns, 716);
    }
  } else if (warp == 1) {
    // ========================================================== MMA issue
    if (lane == 0 && n > 0) {
      const int nx[2] = {nA, nB};
      auto issue_s = [&](int x, int j) {
        const uint32_t kb = kv_base + (j % FL_STAGES) * 2 * TILE_BYTES;
        const uint32_t qb = q_base + x * TILE_BYTES;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t koff = (kk >> 2) * HALF_BYTES + (kk & 3) * 32;
          umma_ss(tmem + x * 128, sdesc_sw128(qb + koff, 16, 1024), sdesc_sw128(kb + koff, 16, 1024), IDESC_S,
                  kk > 0 ? 1u : 0u);
        }
        umma_commit(&bars->s_full[x]);
      };
      auto issue_pv = [&](int x, int j) {
        const uint32_t vb = kv_base + (j % FL_STAGES) * 2 * TILE_BYTES + TILE_BYTES;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, sdesc_sw128(vb + kk * 2048, HALF_BYTES, 1024),
                  IDESC_PV, (j > 0 || kk > 0) ? 1u : 0u);
        if (j == nx[x] - 1) umma_commit(&bars->o_done[x]);
      };
      bool ok = mbar_wait(&bars->q_full, 0, p.limit_ns, abort_flag, 721);
      if (ok) ok = mbar_wait(&bars->full_k[0], 0, p.limit_ns, abort_flag, 722);
      if (ok) {
        tc_fence_after();
        for (int x = 0; x < 2; ++x)
          if (nx[x] > 0) issue_s(x, 0);
        umma_commit(&bars->empty_k[0]);
      }
      for (int j = 0; j < n && ok; ++j) {
        const int s = j % FL_STAGES;
        if (!mbar_wait(&bars->full_v[s], (j / FL_STAGES) & 1, p.limit_ns, abort_flag, 723)) break;
        if (j + 1 < n &&
            !mbar_wait(&bars->full_k[(j + 1) % FL_STAGES], ((j + 1) / FL_STAGES) & 1, p.limit_ns, abort_flag, 724))
          break;
        for (int x = 0; x < 2 && ok; ++x) {
          if (j >= nx[x]) continue;
          if (!mbar_wait(&bars->p_ready[x], j & 1, p.limit_ns, abort_flag, 726)) {
            ok = false;
            break;
          }
          tc_fence_after();
          issue_pv(x, j);
          if (j + 1 < nx[x]) issue_s(x, j + 1);
        }
        if (ok) {
          umma_commit(&bars->empty_v[s]);
          if (j + 1 < n) umma_commit(&bars->empty_k[(j + 1) % FL_STAGES]);
        }
      }
      umma_commit(&bars->fin);
      wait_done(&bars->fin, 0, p.limit_ns, 727);
    }
  } else if (warp == 2) {
    // ==================================== V rows behind the sequence's end
    if (fix && !(p.flags & FLAG_SKIP_LOADS)) {
      const int s = (n - 1) % FL_STAGES;
      if (warp_wait(&bars->v_raw, 0, p.limit_ns, abort_flag, 731)) {
        zero_rows(kv_base + s * 2 * TILE_BYTES + TILE_BYTES, v_rows, lane, 32);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->full_v[s]);
      }
    }
  } else if (warp >= 4 && work) {
    // ============================================ softmax / rescale / epilogue
    const int x = (warp >= 8) ? 1 : 0;
    const int nX = x ? nB : nA;
    const int r = threadIdx.x - 128 - 128 * x;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_off + x * 128;
    const uint32_t o_tm = tmem + lane_off + 256 + x * 128;
    const int first = tok0 + x * R;
    const int i_row = first + r / p.G;      // the row's query within its sequence
    const int h = g * p.G + r % p.G;
    const int limit = i_row + off;          // its last visible key
    RowState st;
    bool ok = true;
    for (int j = 0; j < nX; ++j) {
      if (!warp_wait(&bars->s_full[x], j & 1, p.limit_ns, abort_flag, 741)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t sr[4][32];
      load_scores(s_tm, sr);
      if (j * 128 + 127 > first + off) mask_after(sr, limit - j * 128);
      float alpha;
      const bool resc = softmax_tile(s_tm, sr, p.scale_log2, st, alpha);
      // P V(j - 1) completed before S(j): s_full's commit covers it
      if (j > 0 && __any_sync(0xffffffffu, resc)) rescale_row(o_tm, alpha);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->p_ready[x]);
    }
    // ---- epilogue; a tile without a visible key writes zeros
    const bool row_live = (x == 0 || has_b) && r < R * p.G && i_row < nq;
    if (ok && (nX == 0 || warp_wait(&bars->o_done[x], 0, p.limit_ns, abort_flag, 742))) {
      tc_fence_after();
      const float inv = st.l == 0.f ? 0.f : 1.f / st.l;
      __nv_bfloat16* orow =
          p.o + static_cast<int64_t>(q0 + i_row) * p.o_tok + static_cast<int64_t>(h) * p.o_head;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t orr[32];
        if (nX > 0) {
          tmem_ld32(o_tm + c * 32, orr);
          tmem_ld_wait();
          reg_fence(orr);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) orr[e] = 0u;
        }
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          pk[e] = pack_bf16x2(__uint_as_float(orr[2 * e]) * inv, __uint_as_float(orr[2 * e + 1]) * inv);
        if (row_live) {
          uint4* dst = reinterpret_cast<uint4*>(orow + c * 32);
#pragma unroll
          for (int v4 = 0; v4 < 4; ++v4)
            dst[v4] = make_uint4(pk[4 * v4], pk[4 * v4 + 1], pk[4 * v4 + 2], pk[4 * v4 + 3]);
        }
      }
      if (row_live && p.lse)
        p.lse[static_cast<int64_t>(h) * p.total_q + q0 + i_row] = (st.m + log2f(st.l)) * 0.69314718055994530942f;
    }
  }

  // ---- teardown: every role has drained its asynchronous work
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace hs2
