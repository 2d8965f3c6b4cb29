// Eviction from the paged cache by collected attention weight: per sequence
// and KV head the keep - recent heaviest positions of [0, n - recent) (ties to
// the lower position) and the last `recent`, moved to positions 0 .. keep - 1.
//
// One cluster of CTAs per (sequence, KV head).  Bound by memory (the row of
// weights is read once, the kept K and V rows are read and written once; 256
// rows of 2000 tokens cut to 1152 69 us, 4.5 TB/s) and, for few rows, by the
// latency of its steps (8 rows of 32768 18 us).
//   select   each CTA holds its contiguous part of the row as order-preserving
//            32-bit keys in shared memory (parts too long for it are read from
//            global memory again) and the cluster finds the k-th largest key
//            by a radix search of 11 + 11 + 10 bits: a histogram per CTA and
//            pass, added up through distributed shared memory;
//   list     a CTA's warps own contiguous pieces of its part; counts of larger
//            and equal keys before each piece (over the cluster, then over the
//            CTA) give every kept position its place, so the list comes out
//            ascending without a sort;
//   move     the cluster takes the list in ascending batches.  The new place of
//            a row is never behind its old one, so once a batch is in registers
//            (one cluster barrier) it can be stored without touching a row
//            that a later batch reads: the move needs no second buffer.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"
#include "topk_select.cuh"

namespace hs2 {

constexpr int EV_THREADS = 1024;      // of a CTA that has an SM to itself
constexpr int EV_THREADS_MANY = 512;  // where there are more rows than SMs: two CTAs an SM overlap
constexpr int EV_MAX_CTAS = 8;  // CTAs of a cluster
constexpr int EV_BINS = 2048;
constexpr int EV_COARSE = 64;   // groups of 32 bins
constexpr int EV_ROWS = 8;      // 16-byte pieces in flight per thread
constexpr int EV_MAX_PART = 40960;  // keys a CTA holds in shared memory
constexpr int EV_MAX_TABLE = 8192;  // page table entries held there

struct EvictParams {
  int Hkv, page_log2, n_pages, max_pages, keep, recent, part_cap, table_cap;
  uint8_t *k, *v;
  int64_t tok_b, head_b;  // bytes
  float *ksc, *vsc;
  const int32_t *table, *len;
  const float* acc;
  float* acc_out;
  int64_t acc_stride;
  int32_t *idx, *new_len;
};

struct EvictSmem {
  uint32_t hist[3][EV_BINS];      // this CTA's counts of each pass, read by the other CTAs
  uint32_t coarse[3][EV_COARSE];  // the same, 32 bins together
  uint32_t part[EV_MAX_CTAS * EV_COARSE];
  uint32_t warp_gt[32], warp_eq[32];
  uint32_t cta_gt, cta_eq;    // read by the other CTAs
  uint32_t sh[2];
  uint32_t keys[];  // this CTA's part of the row, then its page table
};

// Sums BINS counts over the cluster and finds the bin that holds rank k from the
// top down: out = (bin, count in the bins above it).  BINS is 32 or 64.
template <int THREADS, int BINS>
__device__ __forceinline__ void ev_find(cooperative_groups::cluster_group& cl, uint32_t* counts, int ctas, uint32_t k,
                                        uint32_t* part, uint32_t* out) {
  static_assert(THREADS / BINS >= EV_MAX_CTAS && BINS <= EV_COARSE, "a thread reads one count");
  const int tid = threadIdx.x, bin = tid % BINS, r = tid / BINS;
  if (r < EV_MAX_CTAS) part[tid] = r < ctas ? cl.map_shared_rank(counts, r)[bin] : 0u;
  __syncthreads();
  if (tid < 32) {  // lane l: bins from the top down
    constexpr int PER = BINS / 32;
    uint32_t c[PER], sum = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      c[q] = 0;
#pragma unroll
      for (int i = 0; i < EV_MAX_CTAS; ++i) c[q] += part[i * BINS + BINS - 1 - (PER * tid + q)];
      sum += c[q];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (tid >= o) incl += y;
    }
    uint32_t run = incl - sum;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      if (run < k && run + c[q] >= k) {
        out[0] = static_cast<uint32_t>(BINS - 1 - (PER * tid + q));
        out[1] = run;
      }
      run += c[q];
    }
  }
  __syncthreads();
}

template <bool KV8, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) cache_evict_kernel(const EvictParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cl = cg::this_cluster();
  extern __shared__ __align__(16) uint8_t ev_raw[];
  EvictSmem& sm = *reinterpret_cast<EvictSmem*>(ev_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cl.block_rank()), ctas = static_cast<int>(cl.num_blocks());
  const int g = blockIdx.y, b = blockIdx.z;
  const int64_t row = static_cast<int64_t>(b) * p.Hkv + g;
  const int n = p.len[b];
  int32_t* idx = p.idx + row * p.keep;
  const float* acc = p.acc + row * p.acc_stride;
  float* acc_out = p.acc_out ? p.acc_out + row * p.acc_stride : nullptr;

  // the same decision in every CTA of the cluster
  if (n < 0 || n > (static_cast<int64_t>(p.max_pages) << p.page_log2) || n > p.acc_stride) {
    if (tid == 0 && rank == 0) report(HS2_ERR_INDEX, 601);
    return;
  }
  if (rank == 0 && g == 0 && tid == 0) p.new_len[b] = min(n, p.keep);
  if (n <= p.keep) {
    for (int i = rank * THREADS + tid; i < p.keep; i += ctas * THREADS) idx[i] = i < n ? i : -1;
    if (acc_out && acc_out != acc)
      for (int i = rank * THREADS + tid; i < n; i += ctas * THREADS) acc_out[i] = acc[i];
    return;
  }

  // the sequence's pages, where they fit
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.max_pages;
  {
    const int pages = (n + (1 << p.page_log2) - 1) >> p.page_log2;
    if (pages <= p.table_cap) {
      int32_t* held_table = reinterpret_cast<int32_t*>(sm.keys + p.part_cap);
      for (int i = tid; i < pages; i += THREADS) held_table[i] = table[i];
      table = held_table;  // read after the cluster's barriers below
    }
  }

  // ---- select: the k-th largest key of the candidates
  const int n_c = n - p.recent, k = p.keep - p.recent;  // n_c > k >= 0
  const int part = ((n_c + ctas - 1) / ctas + 3) & ~3;
  const int lo = min(n_c, rank * part), cnt = min(n_c, lo + part) - lo;
  const bool held = part <= p.part_cap;
  auto key_at = [&](int i) { return held ? sm.keys[i] : order_key(acc[lo + i]); };
  uint32_t T = 0, krem = 0;
  if (k > 0) {
    if (held) {
      const float4* a4 = reinterpret_cast<const float4*>(acc + lo);
      for (int i = tid; i < (cnt + 3) / 4; i += THREADS) {
        const float4 x = a4[i];  // the tail stays inside the row: acc_stride is a multiple of 4
        reinterpret_cast<uint4*>(sm.keys)[i] =
            make_uint4(order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w));
      }
    }
    for (int i = tid; i < 3 * EV_BINS / 4; i += THREADS)
      reinterpret_cast<uint4*>(sm.hist[0])[i] = make_uint4(0, 0, 0, 0);
    uint32_t prefix = 0, pmask = 0;
    krem = static_cast<uint32_t>(k);
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t dmask = pass == 2 ? 1023u : 2047u;
      uint32_t* hist = sm.hist[pass];
      __syncthreads();
      for (int i = tid; i < cnt; i += THREADS) {
        const uint32_t key = key_at(i);
        if ((key & pmask) == prefix) atomicAdd(&hist[(key >> shift) & dmask], 1u);
      }
      __syncthreads();
      if (tid < EV_BINS / 4) {  // groups of 32 bins: eight lanes add up four bins each
        const uint4 x = reinterpret_cast<const uint4*>(hist)[tid];
        uint32_t c = (x.x + x.y) + (x.z + x.w);
        c += __shfl_xor_sync(0xffffffffu, c, 1);
        c += __shfl_xor_sync(0xffffffffu, c, 2);
        c += __shfl_xor_sync(0xffffffffu, c, 4);
        if ((tid & 7) == 0) sm.coarse[pass][tid >> 3] = c;
      }
      cl.sync();  // each pass has counts of its own, so one barrier a pass is enough
      // the group that holds rank krem from the top, then the bin in it; both
      // from the sums over the cluster, so that few words cross it
      ev_find<THREADS, EV_COARSE>(cl, sm.coarse[pass], ctas, krem, sm.part, sm.sh);
      const uint32_t group = sm.sh[0], above = sm.sh[1];
      __syncthreads();
      ev_find<THREADS, 32>(cl, hist + 32 * group, ctas, krem - above, sm.part, sm.sh);
      if (tid == 0) {
        sm.sh[0] += 32 * group;
        sm.sh[1] += above;
      }
      __syncthreads();
      prefix |= sm.sh[0] << shift;
      pmask |= dmask << shift;
      krem -= sm.sh[1];
    }
    T = prefix;

    // ---- list: warp w owns [w * piece, (w + 1) * piece) of this CTA's part
    const int piece = ((cnt + THREADS / 32 - 1) / (THREADS / 32) + 31) & ~31;
    const int w_lo = min(cnt, warp * piece), w_hi = min(cnt, w_lo + piece);
    uint32_t gt = 0, eq = 0;
    for (int i = w_lo + lane; i < w_hi; i += 32) {
      const uint32_t key = key_at(i);
      gt += key > T;
      eq += key == T;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
      sm.warp_gt[warp] = gt;
      sm.warp_eq[warp] = eq;
    }
    __syncthreads();
    if (warp == 0) {
      const bool own = lane < THREADS / 32;
      const uint32_t a = __reduce_add_sync(0xffffffffu, own ? sm.warp_gt[lane] : 0u);
      const uint32_t c = __reduce_add_sync(0xffffffffu, own ? sm.warp_eq[lane] : 0u);
      if (lane == 0) {
        sm.cta_gt = a;
        sm.cta_eq = c;
      }
    }
    cl.sync();
    // counts before this warp's piece: the CTA's warps and the cluster's CTAs before
    static_assert(THREADS <= 32 * 32, "a lane per warp");
    uint32_t gt_before = 0, eq_before = 0;
    if (lane < warp) {
      gt_before = sm.warp_gt[lane];
      eq_before = sm.warp_eq[lane];
    }
    if (lane < rank) {
      gt_before += *cl.map_shared_rank(&sm.cta_gt, lane);
      eq_before += *cl.map_shared_rank(&sm.cta_eq, lane);
    }
    gt_before = __reduce_add_sync(0xffffffffu, gt_before);
    eq_before = __reduce_add_sync(0xffffffffu, eq_before);
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t key = i < w_hi ? key_at(i) : 0u;
      const bool is_gt = i < w_hi && key > T, is_eq = i < w_hi && key == T;
      const uint32_t mg = __ballot_sync(0xffffffffu, is_gt), me = __ballot_sync(0xffffffffu, is_eq);
      const uint32_t eq_rank = eq_before + __popc(me & below);
      if (is_gt || (is_eq && eq_rank < krem))
        idx[gt_before + __popc(mg & below) + min(eq_rank, krem)] = lo + i;
      gt_before += __popc(mg);
      eq_before += __popc(me);
    }
  }
  if (rank == ctas - 1)
    for (int i = tid; i < p.recent; i += THREADS) idx[k + i] = n - p.recent + i;
  cl.sync();  // the list is complete; no CTA reads another's shared memory any more

  // ---- move: batches of rows, in ascending order, by the whole cluster
  constexpr int PIECES = KV8 ? 16 : 32;  // 16-byte pieces of a K row and a V row
  // token of the pools that holds position pos, or -1
  auto token_of = [&](int pos) -> int64_t {
    const int pg = table[pos >> p.page_log2];
    if (pg < 0 || pg >= p.n_pages) {
      report(HS2_ERR_INDEX, 602);
      return -1;
    }
    return (static_cast<int64_t>(pg) << p.page_log2) + (pos & ((1 << p.page_log2) - 1));
  };
  const int piece = tid % PIECES;
  uint8_t* base = (piece < PIECES / 2 ? p.k : p.v) + static_cast<int64_t>(g) * p.head_b + (piece % (PIECES / 2)) * 16;
  const int step = ctas * (THREADS / PIECES);  // rows the cluster's threads cover at once
  const int row0 = rank * (THREADS / PIECES) + tid / PIECES;
  const int batch = step * EV_ROWS;
  const int ctid = rank * THREADS + tid;  // scalars of row ctid of a batch
  int old[EV_ROWS];  // old positions of the batch's rows, read a batch ahead
  // (-1 for what is no position: weights that change under the call leave holes in the list)
  auto listed = [&](int i) {
    const int x = i < p.keep ? idx[i] : -1;
    return x < n ? x : -1;
  };
  auto olds_of = [&](int i0) {
#pragma unroll
    for (int e = 0; e < EV_ROWS; ++e) old[e] = listed(i0 + e * step + row0);
  };
  olds_of(0);
  auto scalar_of = [&](int i0) { return ctid < batch ? listed(i0 + ctid) : -1; };
  int was_next = scalar_of(0);
  for (int i0 = 0; i0 < p.keep; i0 += batch) {
    uint4 data[EV_ROWS];
    uint32_t have = 0;
#pragma unroll
    for (int e = 0; e < EV_ROWS; ++e) {
      if (old[e] >= 0) {
        const int64_t tok = token_of(old[e]);
        if (tok >= 0) {
          data[e] = *reinterpret_cast<const uint4*>(base + tok * p.tok_b);
          have |= 1u << e;
        }
      }
    }
    olds_of(i0 + batch);
    float x_acc = 0.f, x_ks = 0.f, x_vs = 0.f;
    int64_t from = -1;
    const int is = i0 + ctid, was = was_next;
    was_next = scalar_of(i0 + batch);
    if (was >= 0) {
      x_acc = acc[was];
      if (KV8 && (from = token_of(was)) >= 0) {
        x_ks = p.ksc[from * p.Hkv + g];
        x_vs = p.vsc[from * p.Hkv + g];
      }
    }
    cl.sync();  // the batch is in registers
#pragma unroll
    for (int e = 0; e < EV_ROWS; ++e) {
      if (have >> e & 1u) {
        const int64_t tok = token_of(i0 + e * step + row0);
        if (tok >= 0) *reinterpret_cast<uint4*>(base + tok * p.tok_b) = data[e];
      }
    }
    if (was >= 0) {
      if (acc_out) acc_out[is] = x_acc;
      if (KV8 && from >= 0) {
        const int64_t to = token_of(is);
        if (to >= 0) {
          p.ksc[to * p.Hkv + g] = x_ks;
          p.vsc[to * p.Hkv + g] = x_vs;
        }
      }
    }
  }
  // acc_out may be acc: every kept weight is read by now
  if (acc_out)
    for (int i = p.keep + ctid; i < n; i += ctas * THREADS) acc_out[i] = 0.f;
}

}  // namespace hs2
