// The attention weight that cached tokens collect from drafted queries:
//   acc[b][g][j] += sum over counted rows r and heads h of g of
//                   exp(q_rh . k_j / sqrt(d) - lse[h][r])   (0 where j is masked)
//
// As kernel (2) (importance.cuh) the keys lie on the MMA's M dimension: D =
// K tile (128 keys x d) * Q^T (d x up to CW_ROWS query rows), so TMEM lane r holds
// key r against every row and the thread that owns it adds its row up in
// registers, with no reduction between threads and no atomics: each position
// is written by one thread, in a fixed order.
//
// K is read once (256 B a key and KV head, 132 B as e4m3).  Work is split as
// in tree_attn.cuh, but by (sequence, KV head): a CTA takes an equal stretch of
// all key tiles, and for more than CW_ROWS rows walks its part of a sequence
// once per CW_ROWS rows (adding to what it wrote; the K tiles then come from
// L2).  Two pairs of epilogue warpgroups take the even and the odd tiles, each
// warpgroup half of the columns (with one a tile 32 columns took 700 cycles of
// mostly waiting); the second hands its sums to the first through shared memory.
//
// e4m3: the codes are an operand of the product as they arrive (kind::f8f6f4).
// A query row times a power of two is the sum of three e5m2 rows (split_queries),
// so twelve products of 32 give the scores that eight of 16 give in bf16; the
// key's scale and the row's power of two multiply them afterwards.  Turning the
// codes into bf16 instead took 245 us for 32 tokens (256 rows) over 2 sequences
// of up to 131072, where this takes 204 (two e4m3 parts, which lost bits, 188).
//
// Bound by memory at few rows (4 x 32768 tokens of 64/8 heads, 8 rows: bf16 51
// us, 5.4 TB/s; e4m3 49 us, 3.0 TB/s, there the steps of a tile are longer than
// its load), then by the sums (512 rows: 186 and 250 us), of which the
// exponentials are a large part: 16 a clock and SM on the MUFU unit, so where all
// 32 columns of a chunk count four of its sixteen pairs take the degree-4
// polynomial on the FMA pipes instead (2.6e-6; the cubic that kernel (2) mixes in
// is exact only to 7.5e-5; none of them 213 and 254 us, eight 204 and 269).
#pragma once

#include "tree_attn.cuh"

namespace hs2 {

constexpr int CW_ROWS = 256;     // query rows of a pass (128: 222 us for 192 with 512 rows of a bf16 cache)
constexpr int CW_MAX_ITEMS = 7;  // K tiles in the ring, at most
constexpr int CW_THREADS = 640;  // loads, products, queries and a spare warp; two warpgroups for each tile parity

struct WeightParams {
  TreeParams t;          // geometry, table, cu, ctx, mask, scales, limits
  const float* lse;      // [Hq][n_tok]
  const uint8_t* counted;
  float* acc;            // [B][Hkv][acc_stride]
  int64_t acc_stride;
};

struct WeightBars {
  uint64_t full[CW_MAX_ITEMS], empty[CW_MAX_ITEMS];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], s_empty[2];
  uint64_t rows_ready[2];
  uint64_t part_full[2], part_empty[2];  // the second column half's sums of a tile
  uint64_t fin;
  int first, count;   // as in TreeBars; a unit is a (sequence, KV head) here
  int b, unit, offset, row0, T, ctx;
  int each, more;
  uint32_t tmem_slot;
  int abort;
};
static_assert(sizeof(WeightBars) <= 512, "barrier area");

template <bool KV8>
struct WeightSmem {
  static constexpr int QR = CW_ROWS;
  static constexpr int ITEMS = KV8 ? 7 : 4;
  static_assert(ITEMS <= CW_MAX_ITEMS, "ring");
  static constexpr uint32_t SLOT = KV8 ? RAW_BYTES : TILE_BYTES;
  static constexpr uint32_t QPART = QR * 128u;  // half of d in bf16, or one of the three e5m2 parts
  static constexpr uint32_t ITEM = (KV8 ? 3 : 2) * QPART;  // after Q
  static constexpr uint32_t BAR = ITEM + ITEMS * SLOT;
  // per epilogue warpgroup and segment parity, for each column (query row):
  static constexpr uint32_t BITS = BAR + 512u;                // uint64 [2][2][QR]: the drafted keys it sees
  static constexpr uint32_t NLSE = BITS + 2 * 2 * QR * 8u;    // float [2][2][QR]: -lse * log2(e), -inf: none
  static constexpr uint32_t LIVE = NLSE + 2 * 2 * QR * 4u;    // uint32 [2][2][QR / 32]: the columns that collect
  static constexpr uint32_t PART = LIVE + 2 * 2 * QR / 8u;    // float [2][128]
  static constexpr uint32_t QSC = PART + 1024u;               // e4m3: float [2][QR], what a column's scores are multiplied by
  static constexpr uint32_t BYTES = QSC + (KV8 ? 2 * QR * 4u : 0u);
  static_assert(BYTES <= 232448u, "shared memory of one CTA");
};

// Walks one CTA's stretch: segments are (sequence, KV head, key tiles t0 .. t1,
// token tile m); all token tiles of a key range come one after another.
struct WeightWalk {
  int b, g, m, row0, T, ctx, tiles, mtiles, t0, t1;
  int left;
  __device__ __forceinline__ void load(const TreeParams& p) {
    tree_seq(p, b, row0, T, ctx);
    sizes(p);
  }
  __device__ __forceinline__ void sizes(const TreeParams& p) {
    tiles = T ? (ctx + T + 127) >> 7 : 0;
    mtiles = (T + p.R - 1) / p.R;
  }
  __device__ __forceinline__ bool begin(const TreeParams& p, const WeightBars* bars) {
    left = bars->count;
    if (left <= 0) return false;
    b = bars->b;
    g = bars->unit;
    m = 0;
    row0 = bars->row0;
    T = bars->T;
    ctx = bars->ctx;
    sizes(p);
    t0 = bars->offset;
    t1 = min(tiles, t0 + left);
    return true;
  }
  __device__ __forceinline__ bool next(const TreeParams& p) {
    if (++m < mtiles) return true;
    m = 0;
    left -= t1 - t0;
    if (left <= 0) return false;
    if (++g == p.Hkv) {
      g = 0;
      do {
        ++b;
        load(p);
      } while (T == 0);
    }
    t0 = 0;
    t1 = min(tiles, left);
    return true;
  }
  __device__ __forceinline__ int n() const { return t1 - t0; }
};

// Adds 32 columns' weights of one key to sum.  ALL: every column collects, so
// that some exponentials may leave the MUFU unit (the polynomial has no zero
// for a column that does not; skipping such columns eight at a time cost more
// in branches than it saved).  Else those of the bits of `live` do: the others'
// scores may be anything in bf16 (a row that is left out, TMEM behind the rows),
// an infinity or a NaN too, so they are replaced; e4m3 queries that are left out
// enter the product as zeros (replacing their scores here took 66 us for 49).
template <bool KV8, bool ALL>
__device__ __forceinline__ void weights_add(const uint32_t (&sr)[32], uint64_t f2, const float* nlse,
                                            const float* qsc, uint32_t live, uint64_t (&sum)[4]) {
  const float4* nl4 = reinterpret_cast<const float4*>(nlse);
  const float4* qs4 = reinterpret_cast<const float4*>(qsc);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float4 nl = nl4[e];  // broadcast
    const float4 qs = KV8 ? qs4[e] : make_float4(1.f, 1.f, 1.f, 1.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = 4 * e + 2 * i, pair = 2 * e + i;
      uint64_t score = f2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
      if (KV8) score = f2_mul(score, i ? f2_pack(qs.z, qs.w) : f2_pack(qs.x, qs.y));
      uint64_t x = f2_fma(score, f2, i ? f2_pack(nl.z, nl.w) : f2_pack(nl.x, nl.y));
      if (!ALL && !KV8) {
        float a, b;
        f2_unpack(x, a, b);
        x = f2_pack(live >> c & 1u ? a : -INFINITY, live >> (c + 1) & 1u ? b : -INFINITY);
      }
      const bool poly = ALL && pair % 4 == 1;
      sum[pair & 3] = f2_add(sum[pair & 3], poly ? exp2_fma_nan_x2<4>(x) : ex2_x2(x));
    }
  }
}

template <bool KV8>
__global__ void __launch_bounds__(CW_THREADS, 1)
    cache_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const WeightParams wp) {
  using SM = WeightSmem<KV8>;
  constexpr int QR = SM::QR, ITEMS = SM::ITEMS;
  const TreeParams& p = wp.t;
  extern __shared__ __align__(1024) uint8_t weights_smem[];
  uint8_t* smem = weights_smem;
  WeightBars* bars = reinterpret_cast<WeightBars*>(smem + SM::BAR);
  const uint32_t q_base = smem_u32(smem);
  const uint32_t item_base = smem_u32(smem + SM::ITEM);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort;
  if (q_base & 1023u) {
    if (threadIdx.x == 0) report(HS2_ERR_CUDA, 900);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < ITEMS; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->q_full, KV8 ? 16 : 1);
    mbar_init(&bars->q_empty, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->s_empty[x], 8);
      mbar_init(&bars->rows_ready[x], 8);
      mbar_init(&bars->part_full[x], 4);
      mbar_init(&bars->part_empty[x], 4);
    }
    mbar_init(&bars->fin, 1);
    bars->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_slot, 2 * QR);
    tmem_relinquish();
  }
  if (warp == 2) tree_split(p, bars, false, 0, 901);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;

  if (warp == 0) {
    // ======================================================== K tiles by TMA
    WeightWalk w;
    const bool work = !(p.flags & FLAG_SKIP_LOADS) && w.begin(p, bars);
    const int page = 1 << p.page_log2, per_tile = 128 >> p.page_log2;
    int item = 0;
    bool ok = work;
    while (ok) {
      const int len = w.ctx + w.T;
      const int32_t* table = p.table + static_cast<int64_t>(w.b) * p.max_pages;
      auto page_of = [&](int t) {
        const int at = t * 128 + lane * page;
        return (t < w.t1 && lane < per_tile && at < len) ? table[at >> p.page_log2] : 0;
      };
      int pg = page_of(w.t0);
      for (int t = w.t0; t < w.t1; ++t, ++item) {
        const int next_pg = page_of(t + 1);
        const int slot = item % ITEMS;
        if (item >= ITEMS && !warp_wait(&bars->empty[slot], ((item / ITEMS) - 1) & 1, p.limit_ns, abort_flag, 911)) {
          ok = false;
          break;
        }
        const int keys = min(128, len - t * 128);
        const int pages = (keys + page - 1) >> p.page_log2;
        if (lane == 0)
          mbar_arrive_expect_tx(&bars->full[slot], static_cast<uint32_t>(pages << p.page_log2) * (KV8 ? 128u : 256u));
        __syncwarp();
        if (lane < pages) {
          if (pg < 0 || pg >= p.n_pages) {
            report(HS2_ERR_INDEX, 912);
            pg = p.n_pages;
          }
          uint8_t* dst = smem + SM::ITEM + slot * SM::SLOT + lane * page * 128;
          tma_load_3d(dst, &tmK, &bars->full[slot], 0, w.g, pg << p.page_log2);
          if (!KV8) tma_load_3d(dst + HALF_BYTES, &tmK, &bars->full[slot], 64, w.g, pg << p.page_log2);
        }
        pg = next_pg;
      }
      if (!ok || !w.next(p)) break;
    }
    __syncwarp();
    if (lane == 0 && work)
      for (int u = max(0, item - ITEMS); u < item; ++u)
        wait_done(&bars->full[u % ITEMS], (u / ITEMS) & 1, p.limit_ns, 913);
  } else if (warp == 1) {
    // ========================================================== MMA issue
    // by the elected lane of a warp that walks together (as one lane's branch the
    // issue took longer than the load of a tile: e4m3, 8 rows 56 us for 44)
    WeightWalk w;
    if (w.begin(p, bars)) {
      int item = 0, seg = 0;
      uint32_t used = 0, uses = 0;  // by tile parity: whether a tile was issued, and how many (mod 2)
      bool ok = true;
      while (ok) {
        if (!(ok = warp_wait(&bars->q_full, seg & 1, p.limit_ns, abort_flag, 921))) break;
        const int rows = min(p.R, w.T - w.m * p.R) * p.G;
        const uint32_t cols = static_cast<uint32_t>((rows + 15) & ~15);
        const uint32_t idesc = KV8 ? idesc_f8_f32(128, static_cast<int>(cols), 0, 1)
                                   : idesc_bf16_f32(128, static_cast<int>(cols), 0, 0);
        const int n = w.n();
        for (int j = 0; j < n; ++j, ++item) {
          const int x = j & 1, slot = item % ITEMS;
          ok = warp_wait(&bars->full[slot], (item / ITEMS) & 1, p.limit_ns, abort_flag, 922) &&
               (!(used >> x & 1u) ||
                warp_wait(&bars->s_empty[x], ~(uses >> x) & 1u, p.limit_ns, abort_flag, 923));
          if (!ok) break;
          used |= 1u << x;
          uses ^= 1u << x;
          tc_fence_after();
          const uint64_t da = sdesc_sw128(item_base + slot * SM::SLOT, 16, 1024), db = sdesc_sw128(q_base, 16, 1024);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < (KV8 ? 12 : 8); ++kk) {  // e4m3: the same keys times each part of the queries
              const uint32_t koff = (KV8 ? 0 : (kk >> 2) * HALF_BYTES) + (kk & 3) * 32;
              const uint32_t qoff = (kk >> 2) * SM::QPART + (kk & 3) * 32;
              if (KV8)
                umma_ss_f8(tmem + x * QR, da + (koff >> 4), db + (qoff >> 4), idesc, kk > 0 ? 1u : 0u);
              else
                umma_ss(tmem + x * QR, da + (koff >> 4), db + (qoff >> 4), idesc, kk > 0 ? 1u : 0u);
            }
            umma_commit(&bars->s_full[x]);
            umma_commit(&bars->empty[slot]);
            if (j == n - 1) umma_commit(&bars->q_empty);
          }
          __syncwarp();
        }
        if (!ok) break;
        ++seg;
        if (!w.next(p)) break;
      }
      if (elect_one()) umma_commit(&bars->fin);
      __syncwarp();
      wait_done(&bars->fin, 0, p.limit_ns, 924);
    }
  } else if (warp == 3) {
    // ========================================= bf16: queries by TMA
    WeightWalk w;
    if (!KV8 && lane == 0 && !(p.flags & FLAG_SKIP_LOADS) && w.begin(p, bars)) {
      const uint32_t half = static_cast<uint32_t>(p.R * p.G) * 128u;
      int seg = 0;
      do {
        if (seg > 0 && !mbar_wait(&bars->q_empty, (seg - 1) & 1, p.limit_ns, abort_flag, 931)) break;
        mbar_arrive_expect_tx(&bars->q_full, 2 * half);
        tma_load_3d(smem, &tmQ, &bars->q_full, 0, w.g * p.G, w.row0 + w.m * p.R);
        tma_load_3d(smem + SM::QPART, &tmQ, &bars->q_full, 64, w.g * p.G, w.row0 + w.m * p.R);
        ++seg;
      } while (w.next(p));
      wait_done(&bars->q_full, (seg - 1) & 1, p.limit_ns, 932);
    }
  } else if (warp >= 4) {
    // ===== sums: thread r of a warpgroup owns key r of tiles x, x + 2, ..., and
    // half of the columns
    const int x = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1;
    const int r = (threadIdx.x - 128) & 127;
    const uint32_t s_tm = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + x * QR;
    float* part = reinterpret_cast<float*>(smem + SM::PART) + x * 128 + r;
    int ns = 0, seg = 0, np = 0;
    WeightWalk w;
    bool ok = w.begin(p, bars);
    while (ok) {
      const int rows = min(p.R, w.T - w.m * p.R) * p.G;
      // this segment's query rows: what each sees, and its log-sum.  A buffer is
      // written again two segments later, after every warp passed the barrier
      // of the segment between.
      const int area = x * 2 + (seg & 1);
      uint64_t* row_bits = reinterpret_cast<uint64_t*>(smem + SM::BITS) + area * QR;
      float* row_nlse = reinterpret_cast<float*>(smem + SM::NLSE) + area * QR;
      uint32_t* live = reinterpret_cast<uint32_t*>(smem + SM::LIVE) + area * (QR / 32);
      // the log-sum of column c < rows, -inf where it does not collect
      auto row_lse = [&](int c) {
        const int64_t row = w.row0 + w.m * p.R + c / p.G;
        const float l = wp.lse[static_cast<int64_t>(w.g * p.G + c % p.G) * p.n_tok + row];
        return !wp.counted || wp.counted[row] ? l : -INFINITY;  // both loads under way at once
      };
      {
        const int c = 128 * half + r;
        uint64_t bits = 0;
        float nl = -INFINITY;
        const int t = w.m * p.R + c / p.G;
        if (c < rows) {
          const int64_t row = w.row0 + t;
          bits = p.mask ? p.mask[row] : (2ull << t) - 1;
          if (w.T < 64) bits &= (1ull << w.T) - 1;
          const float l = row_lse(c);
          if (l != -INFINITY) nl = -l * 1.44269504088896340736f;
        }
        row_bits[c] = bits;
        row_nlse[c] = nl;
        const uint32_t m = __ballot_sync(0xffffffffu, nl != -INFINITY);
        if (lane == 0) live[c >> 5] = m;
      }
      const float* qsc = reinterpret_cast<float*>(smem + SM::QSC) + (seg & 1) * QR;
      if (KV8) {  // both tile parities' warps write the queries, when the last segment's products are done
        if (seg > 0 && !warp_wait(&bars->q_empty, (seg - 1) & 1, p.limit_ns, abort_flag, 945)) break;
        uint4 raw[QR / 32];
        load_queries<QR / 32, 16>(p, w.g, w.row0 + w.m * p.R, rows, warp - 4, raw);
#pragma unroll
        for (int s = 0; s < QR / 32; ++s) {
          const int c = 32 * s + 2 * (warp - 4) + (lane >> 4);
          if (c < rows && row_lse(c) == -INFINITY) raw[s] = make_uint4(0, 0, 0, 0);
        }
        split_queries<QR / 32, 16, 1>(raw, smem, SM::QPART, const_cast<float*>(qsc), rows, warp - 4);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(KV8 ? &bars->q_full : &bars->rows_ready[x]);
      if (!warp_wait(KV8 ? &bars->q_full : &bars->rows_ready[x], seg & 1, p.limit_ns, abort_flag, 942)) break;
      ++seg;
      const int len = w.ctx + w.T, n = w.n();
      const int32_t* table = p.table + static_cast<int64_t>(w.b) * p.max_pages;
      float* acc = wp.acc + (static_cast<int64_t>(w.b) * p.Hkv + w.g) * wp.acc_stride;
      // this thread's key of tile j: the sum so far and (e4m3) the page, both
      // read before they are needed: the sum and the scale one tile of this
      // warpgroup ahead, the page two
      auto page_of = [&](int j) {
        const int at = (w.t0 + j) * 128 + r;
        return KV8 && j < n && at < len ? table[at >> p.page_log2] : -1;
      };
      auto fetch = [&](int j, int pg, float& old, float& f) {
        const int at = (w.t0 + j) * 128 + r;
        old = !half && j < n && at < len ? acc[at] : 0.f;
        f = p.scale_log2;
        if (KV8) {
          f = 0.f;  // a page outside the pools reads as zeros
          if (pg >= 0 && pg < p.n_pages)
            f = p.ksc[((static_cast<int64_t>(pg) << p.page_log2) + (at & ((1 << p.page_log2) - 1))) * p.Hkv + w.g];
        }
      };
      float old_next, f_next;
      fetch(x, page_of(x), old_next, f_next);
      int pg_next = page_of(x + 2);
      for (int j = x; j < n; j += 2, ++ns) {
        const int at = (w.t0 + j) * 128 + r;
        const float old = old_next, f = KV8 ? f_next * p.scale_log2 : f_next;
        fetch(j + 2, pg_next, old_next, f_next);
        pg_next = page_of(j + 4);
        if (!(ok = warp_wait(&bars->s_full[x], ns & 1, p.limit_ns, abort_flag, 941))) break;
        tc_fence_after();
        const int d = at - w.ctx;  // >= 0: a drafted key
        const bool drafted = __any_sync(0xffffffffu, d >= 0);
        uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
        const uint64_t ff = f2_pack(f, f);
        const int chunks = (rows + 31) / 32, mid = (chunks + 1) / 2;
        const int c_end = half ? chunks : mid;
#pragma unroll 1
        for (int c = half ? mid : 0; c < c_end; ++c) {
          const int c0 = 32 * c;
          uint32_t sr[32];
          tmem_ld32(s_tm + c0, sr);
          tmem_ld_wait();
          reg_fence(sr);
          const uint32_t collect = live[c];
          if (KV8 && c0 + 32 > rows) {  // columns behind the rows may hold anything
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c0 + e >= rows) sr[e] = 0u;
          }
          if (drafted) {  // not every row sees the key
            const bool in_reach = d < 64;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const bool seen = d < 0 || (in_reach && (row_bits[c0 + e] >> (d & 63) & 1u));
              const float score = __uint_as_float(sr[e]) * (KV8 ? qsc[c0 + e] : 1.f);
              const float y = ex2_approx(fmaf(score, f, row_nlse[c0 + e]));
              sum[e & 3] = f2_add(sum[e & 3], f2_pack(seen && (KV8 || (collect >> e & 1u)) ? y : 0.f, 0.f));
            }
          } else if (collect == 0xffffffffu) {
            weights_add<KV8, true>(sr, ff, row_nlse + c0, qsc + c0, collect, sum);
          } else {
            weights_add<KV8, false>(sr, ff, row_nlse + c0, qsc + c0, collect, sum);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->s_empty[x]);
        float s0, s1, s2, s3;
        f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
        f2_unpack(f2_add(sum[2], sum[3]), s2, s3);
        float total = (s0 + s1) + (s2 + s3);
        if (chunks > 1) {
          if (half) {
            if (np > 0 && !(ok = warp_wait(&bars->part_empty[x], (np - 1) & 1, p.limit_ns, abort_flag, 943))) break;
            *part = total;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->part_full[x]);
          } else {
            if (!(ok = warp_wait(&bars->part_full[x], np & 1, p.limit_ns, abort_flag, 944))) break;
            total += *part;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->part_empty[x]);
          }
          ++np;
        }
        if (!half && at < len) acc[at] = old + total;
      }
      if (!ok || !w.next(p)) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * QR);
  }
}

}  // namespace hs2
