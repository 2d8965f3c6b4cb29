// Causal grouped-query attention over packed prompts of different lengths.
// Per sequence o_i = softmax_{j <= i + nk - nq} (q_i . k_j / sqrt(d)) v_j.
//
// The pipeline is kernel (1)'s (flash.cuh: TMA loads, one MMA-issuing lane,
// two softmax warpgroups taking turns, S / P / O in tensor memory); what
// differs is the shape of the work:
//
//   rows     a tile's 128 rows are 128 / G tokens times the G query heads of a
//            KV head, so a short prompt fills tiles (100 tokens at G = 8 are
//            800 rows, 7 tiles, where tiles of one head would be 8 of them,
//            each 100 / 128 full) and its K and V are loaded once for all
//            heads; an item is two consecutive tiles of one KV head, or one
//            where few prompts leave SMs free (the chain of a single tile is
//            shorter);
//   order    index -> (KV head, item), items longest first over all sequences:
//            item k lies at level p (the p-th tile pair of its sequence) with
//            C(p + 1) <= k < C(p), C(p) = sum_b max(0, pairs_b - p), found by
//            a binary search of one warp. Only the sequences' total and their
//            number size the grid, so the lengths stay on the device; surplus
//            indexes (fewer than the sequences times the KV heads) come last;
//   overlap  a CTA goes on to the next index that no CTA has started yet
//            (cluster launch control: it cancels that CTA's launch and does its
//            work), so the order stays the hardware's and the next item's
//            queries and first keys load while the last one is still in its
//            softmax and its epilogue;
//   edges    keys behind a sequence's end are other sequences' or padding: a
//            score there is replaced by -inf (whatever it was) and the V rows
//            are zeroed in shared memory by an otherwise idle warp before
//            the last product reads them.
//
// Bound by the tensor cores and the serial chain through the softmax, as
// kernel (1) is (32/8 heads: one prompt of 32768 tokens 7.9 ms, 1110 TFLOP/s; 32
// prompts of up to 4096 425 us, 965); short prompts by the latency of a CTA's
// few steps (7 of them 12.4 us).
#pragma once

#include "attn_tile.cuh"

namespace hs2 {

struct VarlenParams {
  int B, total_q, total_k, Hq, Hkv, G, rows_tok;
  int tiles;  // of an item: 2, or 1 where that still leaves SMs free
  const int32_t *cu_q, *cu_k;
  float scale_log2;
  __nv_bfloat16* o;
  int64_t o_tok, o_head;
  float* lse;  // [Hq][total_q] or null
  uint64_t limit_ns;
  uint32_t flags;
};

// What the other roles need to know of an item; nq < 0: there is none left.
struct VarlenItem {
  int g, tok0;         // KV head, first token of its tiles
  int q0, nq, k0, nk;  // the sequence's rows
};

constexpr int VL_ITEMS = 2;    // items known ahead
constexpr int VL_READERS = 11;  // arrivals that give an item's slot back: 8 softmax warps, loads, products, warp 2

struct VarlenBars {
  uint64_t q_full, q_empty;
  uint64_t full_k[FL_STAGES], full_v[FL_STAGES], empty_k[FL_STAGES], empty_v[FL_STAGES];
  uint64_t v_raw[FL_STAGES];  // a V tile landed whose rows behind the sequence are not yet zeroed
  uint64_t s_full[2], p_ready[2], o_done[2];
  uint64_t item_full[VL_ITEMS], item_empty[VL_ITEMS];
  uint64_t loads_done;  // an item's loads are all under way
  uint64_t next_full;   // an answer to "which index next" has come
  uint64_t fin;
  uint32_t tmem_slot;
  int abort;
  VarlenItem item[VL_ITEMS];
  alignas(16) uint32_t next[4];
};
constexpr uint32_t VL_BAR_BYTES = 512;
static_assert(sizeof(VarlenBars) <= VL_BAR_BYTES, "barrier area");
constexpr uint32_t VL_PAIRS_OFF = FL_BAR_OFF + VL_BAR_BYTES;           // int [4096]: tile pairs of each sequence
constexpr uint32_t VL_SMEM = VL_PAIRS_OFF + 4096 * 4 + 1024;           // + alignment slack
static_assert(VL_SMEM <= 232448, "shared memory of one CTA");

// An item's tiles: tile x reads key tiles 0 .. n_x - 1.
struct VarlenTiles {
  int nA, nB, n;
  bool has_b;
  int v_rows;  // rows of the last key tile that are keys
  bool fix;    // it has others
  __device__ __forceinline__ VarlenTiles(const VarlenItem& it, int R, int tiles) {
    const int off = it.nk - it.nq;
    has_b = tiles > 1 && it.tok0 + R < it.nq;
    auto key_tiles = [&](int x) { return max(0, min(it.nq, it.tok0 + (x + 1) * R) + off + 127) >> 7; };
    nA = key_tiles(0);
    nB = has_b ? key_tiles(1) : 0;
    n = max(nA, nB);
    v_rows = it.nk - (n - 1) * 128;
    fix = n > 0 && v_rows < 128;
  }
};

// One warp counts the tile pairs of each sequence; returns their sum (0 where
// an entry of cu_q or cu_k is bad) and the most of one sequence.
__device__ __forceinline__ unsigned varlen_count(const VarlenParams& p, int* pairs, int& most) {
  const int lane = threadIdx.x & 31;
  const int per = p.tiles * p.rows_tok;
  bool ok = true;
  most = 0;
  unsigned sum = 0;  // <= total_q / per + B
  for (int b = lane; b < p.B; b += 32) {
    const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
    ok &= q0 >= 0 && q0 <= q1 && q1 <= p.total_q && k0 >= 0 && k0 <= k1 && k1 <= p.total_k;
    const int n = ok ? (q1 - q0 + per - 1) / per : 0;
    pairs[b] = n;
    most = max(most, n);
    sum += static_cast<unsigned>(n);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (!__all_sync(0xffffffffu, ok)) {
    if (lane == 0 && blockIdx.x == 0) report(HS2_ERR_INDEX, 701);
    return 0;
  }
  return sum;
}

// One warp finds the item of index `index` (see the order above); each lane
// reads only the counts that it wrote itself.  False: there is no such item.
__device__ __forceinline__ bool varlen_find(const VarlenParams& p, const int* pairs, unsigned total, int most,
                                            unsigned index, VarlenItem* item) {
  const int lane = threadIdx.x & 31, per = p.tiles * p.rows_tok;
  if (total == 0 || index / total >= static_cast<unsigned>(p.Hkv)) return false;
  const unsigned g = index / total, k = index - g * total;
  auto at_least = [&](int level) {  // C(level)
    unsigned c = 0;
    for (int b = lane; b < p.B; b += 32) c += static_cast<unsigned>(max(0, pairs[b] - level));
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
    const unsigned m = __ballot_sync(0xffffffffu, b < p.B && pairs[b] > lo);
    const unsigned c = __popc(m);
    if (r < c) {
      if ((m >> lane & 1u) && __popc(m & ((1u << lane) - 1u)) == static_cast<int>(r)) {
        const int q0 = p.cu_q[b], k0 = p.cu_k[b];
        *item = VarlenItem{static_cast<int>(g), lo * per, q0, p.cu_q[b + 1] - q0, k0, p.cu_k[b + 1] - k0};
      }
      break;
    }
    r -= c;
  }
  __syncwarp();
  return true;
}

// Asks for the index of a CTA of this grid that has not been launched yet, whose
// launch is then cancelled; the answer (16 bytes) completes on `bar`.
__device__ __forceinline__ void ask_next(uint32_t* answer, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}

// The answer's index, or -1: no CTA is left to be launched.
__device__ __forceinline__ int next_index(const uint32_t* answer) {
  int index;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t.reg .b32 x;\n\t"
      "ld.shared.b128 a, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "mov.b32 x, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 x, a;\n\t"
      "mov.b32 %0, x;\n\t}"
      : "=r"(index)
      : "r"(smem_u32(answer))
      : "memory");
  return index;
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
  const int R = p.rows_tok;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < FL_STAGES; ++s) {
      mbar_init(&bars->full_k[s], 1);
      mbar_init(&bars->full_v[s], 1);
      mbar_init(&bars->empty_k[s], 1);
      mbar_init(&bars->empty_v[s], 1);
      mbar_init(&bars->v_raw[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->p_ready[x], 4);
      mbar_init(&bars->o_done[x], 1);
    }
    for (int s = 0; s < VL_ITEMS; ++s) {
      mbar_init(&bars->item_full[s], 1);
      mbar_init(&bars->item_empty[s], VL_READERS);
    }
    mbar_init(&bars->loads_done, 1);
    mbar_init(&bars->next_full, 1);
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
  int most = 0;
  unsigned total = 0;
  int* pairs = reinterpret_cast<int*>(smem + VL_PAIRS_OFF);
  if (warp == 3) total = varlen_count(p, pairs, most);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;

  // the it-th item of this CTA, for a reader (a warp or one thread of it);
  // false: there is none, or a wait ran out
  auto item_of = [&](int it, VarlenItem& item) {
    const int s = it % VL_ITEMS;
    if (!mbar_wait(&bars->item_full[s], (it / VL_ITEMS) & 1, p.limit_ns, abort_flag, 702)) return false;
    item = bars->item[s];
    return item.nq >= 0;
  };

  // registers move to the softmax warpgroups: 2 x 192 + 120 = 3 x 168
  if (warp >= 4) {
    reg_acquire<192>();
    // ============================================ softmax / rescale / epilogue
    const int x = (warp >= 8) ? 1 : 0;
    const int r = threadIdx.x - 128 - 128 * x;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_off + x * 128;
    const uint32_t o_tm = tmem + lane_off + 256 + x * 128;
    const int tok_r = r / p.G, head_r = r % p.G;
    int ns = 0, no = 0;  // waits taken on s_full[x] and o_done[x]
    VarlenItem item;
    bool ok = true;
    for (int it = 0; ok && __all_sync(0xffffffffu, item_of(it, item)); ++it) {
      const VarlenTiles t(item, R, p.tiles);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->item_empty[it % VL_ITEMS]);
      const int nX = x ? t.nB : t.nA;
      const int first = item.tok0 + x * R, off = item.nk - item.nq;
      const int i_row = first + tok_r;        // the row's query within its sequence
      const int h = item.g * p.G + head_r;
      const int limit = i_row + off;          // its last visible key
      RowState st;
      for (int j = 0; j < nX; ++j) {
        if (!(ok = warp_wait(&bars->s_full[x], ns++ & 1, p.limit_ns, abort_flag, 741))) break;
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
      if (ok && nX > 0) ok = warp_wait(&bars->o_done[x], no++ & 1, p.limit_ns, abort_flag, 742);
      if (!ok) break;
      const bool row_live = (x == 0 || t.has_b) && r < R * p.G && i_row < item.nq;
      tc_fence_after();
      const float inv = st.l == 0.f ? 0.f : 1.f / st.l;
      __nv_bfloat16* orow =
          p.o + static_cast<int64_t>(item.q0 + i_row) * p.o_tok + static_cast<int64_t>(h) * p.o_head;
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
        p.lse[static_cast<int64_t>(h) * p.total_q + item.q0 + i_row] =
            (st.m + log2f(st.l)) * 0.69314718055994530942f;
    }
  } else {
    reg_release<120>();
    if (warp == 3) {
      // ================================================================ items
      unsigned index = blockIdx.x;
      for (int it = 0;; ++it) {
        const int s = it % VL_ITEMS;
        if (it >= VL_ITEMS &&
            !warp_wait(&bars->item_empty[s], (it / VL_ITEMS - 1) & 1, p.limit_ns, abort_flag, 703))
          break;
        const bool left = static_cast<int>(index) >= 0 && varlen_find(p, pairs, total, most, index, &bars->item[s]);
        if (lane == 0) {
          if (!left) bars->item[s].nq = -1;
          mbar_arrive(&bars->item_full[s]);
        }
        if (!left) break;
        // the next index once this item's loads are on their way: soon enough to
        // load the next one behind them, late enough not to take an item that
        // another CTA would start sooner
        if (!warp_wait(&bars->loads_done, it & 1, p.limit_ns, abort_flag, 705)) break;
        if (lane == 0) ask_next(bars->next, &bars->next_full);
        if (!__all_sync(0xffffffffu, wait_done(&bars->next_full, it & 1, p.limit_ns, 704))) break;
        index = static_cast<unsigned>(next_index(bars->next));
        fence_proxy_async_smem();  // read before the next answer is written
        __syncwarp();
      }
    } else if (warp == 0) {
      // =========================================================== TMA loads
      if (lane == 0 && !(p.flags & FLAG_SKIP_LOADS)) {
        VarlenItem item;
        int u = 0, nq_loads = 0;  // key tiles and query loads so far
        uint32_t raw_used = 0, raw_uses = 0;  // stages last filled through v_raw, and how often (mod 2)
        bool ok = true, k_alone = false;
        for (int it = 0; ok && item_of(it, item); ++it) {
          const VarlenTiles t(item, R, p.tiles);
          if (t.n > 0) {
            const int nqt = t.has_b ? 2 : 1;
            const uint32_t half = static_cast<uint32_t>(R * p.G) * 128u;
            if (nq_loads > 0 && !mbar_wait(&bars->q_empty, (nq_loads - 1) & 1, p.limit_ns, abort_flag, 711)) break;
            ++nq_loads;
            mbar_arrive_expect_tx(&bars->q_full, static_cast<uint32_t>(nqt) * 2u * half);
            for (int x = 0; x < nqt; ++x) {
              uint8_t* qd = smem + FL_Q_OFF + x * TILE_BYTES;
              tma_load_3d(qd, &tmQ, &bars->q_full, 0, item.g * p.G, item.q0 + item.tok0 + x * R);
              tma_load_3d(qd + HALF_BYTES, &tmQ, &bars->q_full, 64, item.g * p.G, item.q0 + item.tok0 + x * R);
            }
            for (int j = 0; j < t.n; ++j, ++u) {
              const int s = u % FL_STAGES;
              const uint32_t par = ((u / FL_STAGES) - 1) & 1;
              if (u >= FL_STAGES && !mbar_wait(&bars->empty_k[s], par, p.limit_ns, abort_flag, 712)) {
                ok = false;
                break;
              }
              uint8_t* kd = smem + FL_KV_OFF + s * 2 * TILE_BYTES;
              mbar_arrive_expect_tx(&bars->full_k[s], TILE_BYTES);
              tma_load_3d(kd, &tmK, &bars->full_k[s], 0, item.g, item.k0 + j * 128);
              tma_load_3d(kd + HALF_BYTES, &tmK, &bars->full_k[s], 64, item.g, item.k0 + j * 128);
              if (u >= FL_STAGES && !mbar_wait(&bars->empty_v[s], par, p.limit_ns, abort_flag, 713)) {
                ok = false;
                k_alone = true;  // K(u) in flight, V(u) not
                break;
              }
              // a last tile to be mended reaches full_v through warp 2
              const bool mend = t.fix && j == t.n - 1;
              uint64_t* vbar = mend ? &bars->v_raw[s] : &bars->full_v[s];
              raw_used = (raw_used & ~(1u << s)) | (mend ? 1u << s : 0u);
              raw_uses ^= mend ? 1u << s : 0u;
              mbar_arrive_expect_tx(vbar, TILE_BYTES);
              tma_load_3d(kd + TILE_BYTES, &tmV, vbar, 0, item.g, item.k0 + j * 128);
              tma_load_3d(kd + TILE_BYTES + HALF_BYTES, &tmV, vbar, 64, item.g, item.k0 + j * 128);
            }
          }
          if (!ok) break;
          mbar_arrive(&bars->loads_done);
          mbar_arrive(&bars->item_empty[it % VL_ITEMS]);
        }
        // never leave a TMA write in flight into memory the CTA gives back
        if (k_alone) wait_done(&bars->full_k[u % FL_STAGES], (u / FL_STAGES) & 1, p.limit_ns, 714);
        for (int v = max(0, u - FL_STAGES); v < u; ++v) {
          const int s = v % FL_STAGES;
          if (!(k_alone && s == u % FL_STAGES)) wait_done(&bars->full_k[s], (v / FL_STAGES) & 1, p.limit_ns, 715);
          if (raw_used >> s & 1u)
            wait_done(&bars->v_raw[s], ~(raw_uses >> s) & 1u, p.limit_ns, 716);
          else
            wait_done(&bars->full_v[s], (v / FL_STAGES) & 1, p.limit_ns, 717);
        }
        if (nq_loads > 0) wait_done(&bars->q_full, (nq_loads - 1) & 1, p.limit_ns, 718);
      }
    } else if (warp == 1) {
      // ========================================================== MMA issue
      // the warp walks together, its elected lane issues (as one lane's branch
      // every case took 5 to 7% longer)
      VarlenItem item;
      int u = 0, nq_loads = 0;
      uint32_t np = 0;  // by tile of the item: P tiles so far (mod 2)
      auto issue_s = [&](int x, int tile) {
        const uint64_t da = sdesc_sw128(q_base + x * TILE_BYTES, 16, 1024);
        const uint64_t db = sdesc_sw128(kv_base + (tile % FL_STAGES) * 2 * TILE_BYTES, 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t koff = ((kk >> 2) * HALF_BYTES + (kk & 3) * 32) >> 4;
            umma_ss(tmem + x * 128, da + koff, db + koff, IDESC_S, kk > 0 ? 1u : 0u);
          }
          umma_commit(&bars->s_full[x]);
        }
        __syncwarp();
      };
      auto issue_pv = [&](int x, int tile, bool first, bool last) {
        const uint64_t db =
            sdesc_sw128(kv_base + (tile % FL_STAGES) * 2 * TILE_BYTES + TILE_BYTES, HALF_BYTES, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, db + kk * (2048 >> 4), IDESC_PV,
                    (!first || kk > 0) ? 1u : 0u);
          if (last) umma_commit(&bars->o_done[x]);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      auto k_landed = [&](int tile) {
        return warp_wait(&bars->full_k[tile % FL_STAGES], (tile / FL_STAGES) & 1, p.limit_ns, abort_flag, 721);
      };
      bool ok = true;
      for (int it = 0; ok && __all_sync(0xffffffffu, item_of(it, item)); ++it) {
        const VarlenTiles t(item, R, p.tiles);
        const int n = t.n;
        if (n > 0) {
          ok = warp_wait(&bars->q_full, nq_loads++ & 1, p.limit_ns, abort_flag, 722) && k_landed(u);
          if (!ok) break;
          tc_fence_after();
          if (t.nA > 0) issue_s(0, u);
          if (t.nB > 0) issue_s(1, u);
          commit(&bars->empty_k[u % FL_STAGES]);
          if (n == 1) commit(&bars->q_empty);
        }
        // The first product of a tile writes over the last item's O without a
        // barrier of its own: it waits for P, and the warps of that tile write P
        // after they have read O.  (A barrier with a phase an item, waited for by
        // its parity, would not do: a warpgroup without a tile, or with one that
        // sees no key, is up to two items ahead, so that two phases may end before
        // this warp looks.)
        for (int j = 0; j < n && ok; ++j) {
          const int tile = u + j, s = tile % FL_STAGES;
          ok = warp_wait(&bars->full_v[s], (tile / FL_STAGES) & 1, p.limit_ns, abort_flag, 724) &&
               (j + 1 >= n || k_landed(tile + 1));
          for (int x = 0; x < 2 && ok; ++x) {
            const int nx = x ? t.nB : t.nA;
            if (j >= nx) continue;
            if (!(ok = warp_wait(&bars->p_ready[x], (np >> x) & 1, p.limit_ns, abort_flag, 725))) break;
            np ^= 1u << x;
            tc_fence_after();
            issue_pv(x, tile, j == 0, j == nx - 1);
            if (j + 1 < nx) issue_s(x, tile + 1);
          }
          if (ok) {
            commit(&bars->empty_v[s]);
            if (j + 1 < n) commit(&bars->empty_k[(tile + 1) % FL_STAGES]);
            if (j + 2 == n) commit(&bars->q_empty);  // every score product is queued
          }
        }
        u += n;
        if (ok && lane == 0) mbar_arrive(&bars->item_empty[it % VL_ITEMS]);
      }
      commit(&bars->fin);
      wait_done(&bars->fin, 0, p.limit_ns, 726);
    } else if (warp == 2) {
      // ==================================== V rows behind the sequence's end
      if (!(p.flags & FLAG_SKIP_LOADS)) {
        VarlenItem item;
        int u = 0;
        uint32_t uses = 0;  // of each stage's v_raw, mod 2
        for (int it = 0; __all_sync(0xffffffffu, item_of(it, item)); ++it) {
          const VarlenTiles t(item, R, p.tiles);
          u += t.n;
          if (t.fix) {
            const int s = (u - 1) % FL_STAGES;
            if (!warp_wait(&bars->v_raw[s], uses >> s & 1u, p.limit_ns, abort_flag, 731)) break;
            uses ^= 1u << s;
            zero_rows(kv_base + s * 2 * TILE_BYTES + TILE_BYTES, t.v_rows, lane, 32);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->full_v[s]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->item_empty[it % VL_ITEMS]);
        }
      }
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
