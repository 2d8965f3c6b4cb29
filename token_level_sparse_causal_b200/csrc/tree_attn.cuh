// Attention of drafted tokens over a paged cache: each of a sequence's T
// drafted tokens (T * G query rows per KV head) sees all committed tokens and
// the drafted ones its mask names; T = 1 is ordinary decoding.
//
// Bound by memory: K and V are read once (512 B per key and KV head in bf16,
// 264 B as e4m3 with scales), and at T * G <= 128 rows one pass over them
// serves all rows.  So the design is about keeping loads in flight (bf16,
// 4 x 32768 tokens of 64/8 heads: T = 1 92 us, 5.8 TB/s; T = 16 106 us, 5.1):
//
//   work     the unit is (sequence, KV head, tile of RB / G tokens); all units'
//            key tiles (128 keys) are laid end to end and every CTA (one per
//            SM, persistent) takes an equal stretch, whatever the lengths: one
//            long context is spread over all SMs, many short ones are packed.
//            A stretch that holds only part of a unit leaves (m, l, O) in the
//            workspace and tree_merge_kernel joins the parts in key order, so
//            results do not depend on timing;
//   ring     one ring of tiles in the order the products use them, K0 K1 V0 K2
//            V1 K3 ..., filled by TMA through the page table (a box per page)
//            without regard to unit borders: loads of the next unit run while
//            the last one finishes;
//   overlap  even and odd key tiles of a unit are two independent softmaxes
//            (own S, P, O in tensor memory, own warpgroup) that take turns on
//            the tensor core as in flash.cuh; their O join in the epilogue,
//            where each warpgroup writes half of the columns;
//   few rows a tile's 128 rows are 4 blocks of 32, copies of the unit's
//            rows where those fit, and block k keeps only its share of the
//            tile's keys (the rest of its P is zero): all warps share one row's
//            exponentials, instead of one warp taking all of them (bf16, 64
//            short sequences 36 -> 32.5 us, one of 2048 tokens 14 -> 13; e4m3
//            with the codes as below 121 -> 92 us). Each block is a
//            softmax of its own; the epilogue adds the blocks' O, each block a
//            share of the columns;
//   e4m3     codes arrive by TMA; eight warps turn them into bf16 (exact; unlike
//            f16 it leaves Q and P their whole range), another fetches the
//            scales; the K scale multiplies the scores, the V scale multiplies
//            P before its rounding.  Few rows: K's codes are the products'
//            operand as they are, the queries sums of three e5m2 rows
//            (split_queries), and only V is converted (4 x 32768 tokens, T = 1:
//            107 -> 92 us); for a full block the split of 128 rows costs more
//            than it saves (64 short sequences, T = 6: 52 us, 62 with it).
//            Bound by the conversion and the softmax with its scales, not by
//            memory: 2.4 TB/s at 128 rows, 3.0 at 8;
//   edges    columns without a visible key become -inf whatever they hold, V
//            rows behind the last key are zeroed before the product.
#pragma once

#include <cuda_fp16.h>

#include "attn_tile.cuh"
#include "quantize.cuh"

namespace hs2 {

constexpr int TR_MAX_ITEMS = 6;  // tiles of 32 KB in the ring, at most
constexpr int TR_MAX_RAW = 5;    // e4m3: tiles of codes, 16 KB, in a ring, at most
constexpr int TR_OVERHEAD = 3;   // what a unit costs beside its key tiles, in tiles (see tree_split)
constexpr int TR_SCALES = 8;     // e4m3: key tiles whose scales are held or on their way
constexpr uint32_t RAW_BYTES = 128u * 128u;
constexpr int TR_CONV = 256;     // e4m3: converting threads (4 sequences up to 131072, T = 16: 330 us, 128 of them 430)
__host__ __device__ constexpr int tr_threads(bool kv8) { return 384 + (kv8 ? TR_CONV : 0); }

// What a call's kernels share: the unit geometry.
struct TreeParams {
  int B, Hq, Hkv, G, R, page_log2, n_pages, max_pages, n_tok, max_draft;
  int64_t max_len;  // tokens of a sequence, drafted ones with them: what the table (and acc) can hold
  const int32_t *table, *cu, *ctx;
  const uint64_t* mask;
  float scale_log2;
  const float *ksc, *vsc;  // e4m3 only
  const __nv_bfloat16* q;  // where the queries are split (else by TMA)
  int64_t q_tok, q_head;   // of q and o
  __nv_bfloat16* o;
  float* lse;
  float* part_o;    // [CTA][2][128][128], un-normalised
  float2* part_ml;  // [CTA][2][128]
  int4* part_unit;  // [CTA]: (first row, tokens, KV head, last CTA) of the unit whose first part this CTA holds
  uint64_t limit_ns;
  uint32_t flags;
};

struct TreeBars {
  uint64_t full[TR_MAX_ITEMS], empty[TR_MAX_ITEMS];
  uint64_t k8_full[TR_MAX_RAW], k8_empty[TR_MAX_RAW], v8_full[2], v8_empty[2];  // e4m3
  uint64_t sc_full[TR_SCALES], sc_empty[TR_SCALES];
  uint64_t q_full, q_empty;
  uint64_t qsc_read;  // few rows, e4m3: every softmax warp has a segment's row scales (and has seen q_full's phase)
  uint64_t v_raw[TR_MAX_ITEMS];  // a V tile landed whose rows behind the sequence are not yet zeroed
  uint64_t s_full[2], p_ready[2], o_done[2];
  uint64_t ml_ready, o_free;
  uint64_t x_ready[2], x_free[2];  // the exchange of O between row blocks, per warpgroup
  uint64_t fin;
  int first, count;          // this CTA's stretch, in units of a key tile's cost
  int b, unit, offset;       // where it begins: sequence, its unit, cost inside the unit
  int row0, T, ctx;          // its sequence
  int each, more;     // cost of a CTA; the first `more` CTAs have one more
  uint32_t tmem_slot;
  int abort;
};
constexpr uint32_t TR_BAR_BYTES = 704;
static_assert(sizeof(TreeBars) <= TR_BAR_BYTES, "barrier area");

// RB: rows of a block (32 or 128); a unit has RB / G tokens.
template <bool KV8, int RB>
struct TreeSmem {
  static_assert(RB == 32 || RB == 128, "four blocks or one");
  static constexpr int BLOCKS = 128 / RB;
  static constexpr bool CODES = KV8 && BLOCKS > 1;  // K's codes are the products' operand
  static constexpr int ITEMS = CODES ? 2 : KV8 ? 3 : BLOCKS > 1 ? 5 : 6;  // CODES: V tiles only
  static constexpr int K8 = CODES ? 3 : 5, V8 = CODES ? 2 : 0;  // rings of codes; else K's and V's in one
  static_assert(ITEMS <= TR_MAX_ITEMS && K8 <= TR_MAX_RAW && V8 <= TR_MAX_RAW, "rings");
  static constexpr uint32_t ITEM = CODES ? 3 * HALF_BYTES : TILE_BYTES;  // after Q: three parts of it, or two halves
  static constexpr uint32_t K8_AT = ITEM + ITEMS * TILE_BYTES;
  static constexpr uint32_t V8_AT = K8_AT + (KV8 ? K8 * RAW_BYTES : 0u);
  static constexpr uint32_t SCALE = V8_AT + V8 * RAW_BYTES;
  static constexpr uint32_t BAR = SCALE + (KV8 ? TR_SCALES * 1024u : 0u);
  static constexpr uint32_t ML = BAR + TR_BAR_BYTES;     // float2 [2][128]
  static constexpr uint32_t EXCH = ML + 2048u;   // float [2][128 - RB][32]
  static constexpr uint32_t QSC = EXCH + 2u * (128 - RB) * 128u;  // CODES: float [RB], what a row's scores are times
  static constexpr uint32_t BYTES = QSC + (CODES ? RB * 4u : 0u);
  static_assert(BYTES <= 232448u, "shared memory of one CTA");
};

// A sequence's lengths; a bad entry counts as no drafted tokens (tree_split looks
// at cu_draft as a whole, for sequences that would share rows).
__device__ __forceinline__ bool tree_seq(const TreeParams& p, int b, int& row0, int& T, int& ctx) {
  const int64_t r0 = p.cu[b], t = static_cast<int64_t>(p.cu[b + 1]) - r0, c = p.ctx[b];
  const bool ok = r0 >= 0 && t >= 0 && t <= p.max_draft && r0 + t <= p.n_tok && c >= 0 && c + t <= p.max_len;
  row0 = ok ? static_cast<int>(r0) : 0;
  T = ok ? static_cast<int>(t) : 0;
  ctx = ok ? static_cast<int>(c) : 0;
  return ok;
}

// Walks the segments (parts of units) of one CTA's stretch; every role of the
// CTA walks the same ones.
struct TreeWalk {
  int b, g, m;          // unit
  int row0, T, ctx;     // its sequence
  int tiles, mtiles;    // key tiles of the unit, token tiles of the sequence
  int t0, t1;           // the segment's key tiles
  int left, pos;        // cost left in the stretch from the unit's begin on, and where that lies in all

  __device__ __forceinline__ void load(const TreeParams& p) {
    tree_seq(p, b, row0, T, ctx);
    sizes(p);
  }
  __device__ __forceinline__ void sizes(const TreeParams& p) {
    tiles = T ? (ctx + T + 127) >> 7 : 0;
    mtiles = T <= p.R ? (T > 0 ? 1 : 0) : (T + p.R - 1) / p.R;
  }
  __device__ __forceinline__ bool begin(const TreeParams& p, const TreeBars* bars) {
    left = bars->count;
    if (left <= 0) return false;
    pos = bars->first;
    b = bars->b;
    row0 = bars->row0;
    T = bars->T;
    ctx = bars->ctx;
    sizes(p);
    g = mtiles == 1 ? bars->unit : bars->unit / mtiles;
    m = bars->unit - g * mtiles;
    const int f = bars->offset;
    pos = bars->first - f;
    left = bars->count + f;
    t0 = max(0, f - TR_OVERHEAD);
    t1 = min(tiles, left - TR_OVERHEAD);
    return t1 > t0 || advance(p);
  }
  // to the next unit of which the stretch holds a tile
  __device__ __forceinline__ bool next(const TreeParams& p) { return advance(p); }
  __device__ __forceinline__ bool advance(const TreeParams& p) {
    left -= TR_OVERHEAD + tiles;
    pos += TR_OVERHEAD + tiles;
    if (left <= TR_OVERHEAD) return false;  // the next unit's first tile is the next CTA's
    if (++m == mtiles) {
      m = 0;
      if (++g == p.Hkv) {
        g = 0;
        do {
          ++b;
          load(p);
        } while (T == 0);  // cost is left, so a sequence with some follows
      }
    }
    t0 = 0;
    t1 = min(tiles, left - TR_OVERHEAD);
    return true;
  }
  // the stretch ends with this unit, or inside it
  __device__ __forceinline__ bool last() const { return left <= 2 * TR_OVERHEAD + tiles; }
  __device__ __forceinline__ int n() const { return t1 - t0; }
  __device__ __forceinline__ int rows(const TreeParams& p) const { return min(p.R, T - m * p.R) * p.G; }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
  // rows of the segment's last tile that are keys (128: all)
  __device__ __forceinline__ int last_rows() const { return t1 == tiles ? ctx + T - (tiles - 1) * 128 : 128; }
};

// One warp splits all key tiles evenly over the CTAs and finds where this CTA's
// stretch begins.  units: a sequence's keys count once per token tile.  over:
// cost of a unit beside its tiles (queries to load, a pipeline to fill, an O to
// write); without it the CTAs with many short sequences came in last (64 of up to
// 500 tokens: 34 us, 42 without).
template <typename Bars>
__device__ __forceinline__ void tree_split(const TreeParams& p, Bars* bars, bool units, int over, int where) {
  const int lane = threadIdx.x & 31;
  struct Seq {
    int row0, T, ctx;
    int64_t cost;
  };
  bool ascends = true;  // cu_draft, within [0, n_tok]
  auto look = [&](int b) {
    Seq q{0, 0, 0, 0};
    if (b < p.B) {
      const int r0 = p.cu[b], r1 = p.cu[b + 1];
      ascends &= r0 >= 0 && r0 <= r1 && r1 <= p.n_tok;
      if (!tree_seq(p, b, q.row0, q.T, q.ctx) && blockIdx.x == 0) report(HS2_ERR_INDEX, where);
      const int mtiles = !units || q.T <= p.R ? 1 : (q.T + p.R - 1) / p.R;
      if (q.T) q.cost = static_cast<int64_t>(((q.ctx + q.T + 127) >> 7) + over) * (p.Hkv * mtiles);
    }
    return q;
  };
  const Seq mine = look(lane);  // the first 32 sequences, used twice
  int64_t total64 = mine.cost;
  for (int b = lane + 32; b < p.B; b += 32) total64 += look(b).cost;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total64 += __shfl_xor_sync(0xffffffffu, total64, o);
  // a sequence that begins before the last one's end: its rows would be two
  // sequences', written by both, so nothing is done (reported by look)
  if (!__all_sync(0xffffffffu, ascends)) total64 = 0;
  if (total64 > 0x7fffffff) {  // only by sequences that share pages; no part of it is done
    if (lane == 0 && blockIdx.x == 0) report(HS2_ERR_INDEX, where);
    total64 = 0;
  }
  const unsigned total = static_cast<unsigned>(total64), ctas = gridDim.x;
  const int each = static_cast<int>(total / ctas), more = static_cast<int>(total % ctas);
  const int c = blockIdx.x;
  const int first = c * each + min(c, more), count = each + (c < more ? 1 : 0);
  if (lane == 0) {
    bars->first = first;
    bars->count = count;
    bars->each = each;
    bars->more = more;
  }
  if (count == 0) return;
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const Seq q = b0 == 0 ? mine : look(b0 + lane);
    const int w = static_cast<int>(q.cost);
    int incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const bool here = first >= before + incl - w && first < before + incl;
    if (here) {
      const unsigned cost = (static_cast<unsigned>(q.ctx + q.T + 127) >> 7) + over;
      const unsigned rest = static_cast<unsigned>(first - (before + incl - w)), unit = rest / cost;
      bars->b = b0 + lane;
      bars->unit = static_cast<int>(unit);
      bars->offset = static_cast<int>(rest - unit * cost);
      bars->row0 = q.row0;
      bars->T = q.T;
      bars->ctx = q.ctx;
    }
    if (__any_sync(0xffffffffu, here)) return;
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// The tile that is item u of a segment of n tiles (K0 K1 V0 K2 V1 ... ): its
// index, and whether it is a V tile.
__device__ __forceinline__ void tree_item(int u, int n, int& tile, bool& is_v) {
  if (u == 0 || n == 1) {
    tile = 0;
    is_v = u == 1;
  } else if (u == 1) {
    tile = 1;
    is_v = false;
  } else if (u >= 2 * n - 2) {  // the last two V follow each other
    tile = u - n;
    is_v = true;
  } else {
    is_v = (u & 1) == 0;
    tile = is_v ? (u - 2) >> 1 : (u + 1) >> 1;
  }
}

// Columns of key tile j (first key at `base`) that a row with draft bits
// `bits` sees, as 4 words.
__device__ __forceinline__ void tree_visible(int ctx, int base, uint64_t bits, uint32_t (&w)[4]) {
  const int d = ctx - base;  // columns before the first drafted key
  uint64_t lo = 0, hi = 0;
  if (d >= 128) {
    lo = hi = ~0ull;
  } else if (d >= 64) {
    const int s = d - 64;
    lo = ~0ull;
    hi = ((1ull << s) - 1) | (bits << s);
  } else if (d > 0) {
    lo = ((1ull << d) - 1) | (bits << d);
    hi = bits >> (64 - d);
  } else if (d > -64) {
    lo = bits >> -d;
  }
  w[0] = static_cast<uint32_t>(lo);
  w[1] = static_cast<uint32_t>(lo >> 32);
  w[2] = static_cast<uint32_t>(hi);
  w[3] = static_cast<uint32_t>(hi >> 32);
}

// Sixteen e4m3 codes -> sixteen bf16 values (exact, NaN stays NaN).  The
// conversion instructions beat shifting the bits into place (525 against 673
// cycles a tile of 128 x 128 by 128 threads).
__device__ __forceinline__ void e4m3x16_to_bf16(uint4 raw, uint4& a, uint4& b) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t f[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t h = e4m3x2_to_f16x2(w[q >> 1] >> (16 * (q & 1)));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[q] = pack_bf16x2(v.x, v.y);
  }
  a = make_uint4(f[0], f[1], f[2], f[3]);
  b = make_uint4(f[4], f[5], f[6], f[7]);
}

// A raw tile of 128 rows of codes -> a bf16 tile in two 128-byte-swizzled
// halves, by THREADS threads (pt); rows from `keys` on become zeros.  No
// branch, so that a thread's rows overlap.
template <int THREADS>
__device__ __forceinline__ void convert_tile(uint32_t raw_tile, uint32_t tile, int keys, int pt) {
  constexpr int STEP = THREADS / 8, ROWS = 128 / STEP;
  const int c8 = pt & 7, row0 = pt >> 3;
  // lanes 0-3 and 4-7 of a row store their two chunks in opposite order, so
  // that a store touches every bank once
  const bool flip = c8 >= 4;
  const uint32_t src = raw_tile + row0 * 128 + c8 * 16;
  // a step keeps row & 7, so the chunks' places only move by whole rows
  const uint32_t dst1 = tile + sw128_chunk_offset(row0, 2 * c8 + (flip ? 1 : 0), 128);
  const uint32_t dst2 = tile + sw128_chunk_offset(row0, 2 * c8 + (flip ? 0 : 1), 128);
  constexpr int BATCH = 4;  // rows in registers
#pragma unroll
  for (int b0 = 0; b0 < ROWS; b0 += BATCH) {
    uint4 raw[BATCH];
#pragma unroll
    for (int it = 0; it < BATCH; ++it) raw[it] = ld_shared_v4(src + (b0 + it) * STEP * 128);
#pragma unroll
    for (int it = 0; it < BATCH; ++it) {
      if (row0 + STEP * (b0 + it) >= keys) raw[it] = make_uint4(0, 0, 0, 0);
      uint4 a, b;
      e4m3x16_to_bf16(raw[it], a, b);
      st_shared_v4(dst1 + (b0 + it) * STEP * 128, flip ? b : a);
      st_shared_v4(dst2 + (b0 + it) * STEP * 128, flip ? a : b);
    }
  }
}

// Query rows of a tile, 16 bytes a lane and step: WARPS warps (w) take 2 rows each
// a step, rows [0, rows) exist, those behind them are zeros.
template <int STEPS, int WARPS>
__device__ __forceinline__ void load_queries(const TreeParams& p, int g, int64_t row0, int rows, int w,
                                             uint4 (&raw)[STEPS]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int c = 2 * WARPS * s + 2 * w + (lane >> 4);
    raw[s] = make_uint4(0, 0, 0, 0);
    if (c < rows)
      raw[s] = *reinterpret_cast<const uint4*>(p.q + (row0 + c / p.G) * p.q_tok + (g * p.G + c % p.G) * p.q_head +
                                               8 * (lane & 15));
  }
}

// Those rows as sums of three e5m2 rows (K-major, 128-byte swizzle, the parts
// `part` bytes apart).  A row is scaled by the power of two that brings its
// maximum to [2^14, 2^15), or less for a row of zeros or nearly so; qsc gets the
// inverse.  The first two parts leave at most the last of a bf16 value's 8 bits,
// so the three are exact where the value is not below 2^-23 of its row's maximum
// (2^-9 scaled; e5m2's smallest step is 2^-16), else off by at most 2^-31 of it.
// Two e4m3 parts, which reach down to 2^-9 only, were off by up to 2^-17 of the
// maximum, and with one large dimension among small ones so were the scores.
// Steps that begin at `upto` or behind are left out; COPIES copies of the tile
// are written.
template <int STEPS, int WARPS, int COPIES>
__device__ __forceinline__ void split_queries(const uint4 (&raw)[STEPS], uint8_t* smem, uint32_t part, float* qsc,
                                              int upto, int w) {
  const int lane = threadIdx.x & 31, l16 = lane & 15;
  constexpr int STEP = 2 * WARPS;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    if (STEP * s >= upto) break;
    const int c = STEP * s + 2 * w + (lane >> 4);
    const uint32_t v[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
    uint32_t top = 0;  // the exponents' maximum, in bits 7 .. 14
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, max(v[e] & 0x7f80u, (v[e] >> 16) & 0x7f80u));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    // not below 2^-104: the inverse times log2(e) / sqrt(d) has to stay a normal
    // number (as a subnormal it became 0, and 0 times a masked key's -inf a NaN)
    const uint32_t eb = max(top >> 7, 23u);
    const float up = __uint_as_float((268u - eb) << 23);
    uint32_t codes[3][2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x = __uint_as_float(v[e] << 16) * up, y = __uint_as_float(v[e] & 0xffff0000u) * up;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint32_t a = e5m2x2_from_f32(x, y);
        codes[i][e >> 1] = (e & 1) ? codes[i][e >> 1] | a << 16 : a;
        const uint32_t h = e5m2x2_to_f16x2(a);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        x -= f.x;
        y -= f.y;
      }
    }
#pragma unroll
    for (int k = 0; k < COPIES; ++k) {
      uint8_t* dst = smem + k * STEPS * STEP * 128 + sw128_chunk_offset(c, l16 >> 1, 0) + 8 * (l16 & 1);
#pragma unroll
      for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2*>(dst + i * part) = make_uint2(codes[i][0], codes[i][1]);
    }
    // the codes saturate: a row with an infinity or a NaN is made NaN by its scale
    if (l16 == 0) qsc[c] = __uint_as_float(eb == 255u ? 0x7fffffffu : (eb - 14u) << 23);
  }
}

template <bool KV8, int RB>
__global__ void __launch_bounds__(tr_threads(KV8), 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const TreeParams p) {
  using SM = TreeSmem<KV8, RB>;
  constexpr int ITEMS = SM::ITEMS, K8 = SM::K8, V8 = SM::V8, BLOCKS = SM::BLOCKS;
  constexpr bool CODES = SM::CODES;
  extern __shared__ __align__(1024) uint8_t tree_smem[];
  uint8_t* smem = tree_smem;
  TreeBars* bars = reinterpret_cast<TreeBars*>(smem + SM::BAR);
  float2* ml = reinterpret_cast<float2*>(smem + SM::ML);
  float* scales = reinterpret_cast<float*>(smem + SM::SCALE);  // [slot][K, V][128]
  const uint32_t q_base = smem_u32(smem);
  const uint32_t item_base = smem_u32(smem + SM::ITEM);
  const uint32_t exch_base = smem_u32(smem + SM::EXCH);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort;
  // tree_merge_kernel may be set up meanwhile; it waits for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (q_base & 1023u) {  // the swizzled tiles need it; the whole CTA leaves
    if (threadIdx.x == 0) {
      p.part_unit[blockIdx.x] = make_int4(0, 0, 0, -1);
      report(HS2_ERR_CUDA, 800);
    }
    return;
  }

  // Warp 0 sets up the barriers, finds the stretch and goes straight on to its
  // loads (it arrives at the CTA's barrier without waiting there).
  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < ITEMS; ++s) {
        mbar_init(&bars->full[s], KV8 ? TR_CONV / 32 : 1);
        mbar_init(&bars->empty[s], 1);
        mbar_init(&bars->v_raw[s], 1);
      }
      if (KV8) {
        for (int s = 0; s < K8; ++s) {
          mbar_init(&bars->k8_full[s], 1);
          mbar_init(&bars->k8_empty[s], CODES ? 1 : TR_CONV / 32);
        }
        for (int s = 0; s < V8; ++s) {
          mbar_init(&bars->v8_full[s], 1);
          mbar_init(&bars->v8_empty[s], TR_CONV / 32);
        }
        for (int s = 0; s < TR_SCALES; ++s) {
          mbar_init(&bars->sc_full[s], 32);
          mbar_init(&bars->sc_empty[s], 4);
        }
      }
      mbar_init(&bars->q_full, CODES ? TR_CONV / 32 : 1);
      mbar_init(&bars->q_empty, 1);
      mbar_init(&bars->qsc_read, 8);
      for (int x = 0; x < 2; ++x) {
        mbar_init(&bars->s_full[x], 1);
        mbar_init(&bars->p_ready[x], 4);
        mbar_init(&bars->o_done[x], 1);
      }
      for (int x = 0; x < 2; ++x) {
        mbar_init(&bars->x_ready[x], 4);
        mbar_init(&bars->x_free[x], 4);
      }
      mbar_init(&bars->ml_ready, 8);
      mbar_init(&bars->o_free, 8);
      mbar_init(&bars->fin, 1);
      bars->abort = 0;
      fence_mbar_init();
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    __syncwarp();
    tree_split(p, bars, true, TR_OVERHEAD, 801);
    __syncwarp();
    asm volatile("bar.arrive 1, %0;" ::"n"(tr_threads(KV8)) : "memory");
  } else {
    if (warp == 1) {
      tmem_alloc(&bars->tmem_slot, 512);
      tmem_relinquish();
    }
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(tr_threads(KV8)) : "memory");
    tc_fence_after();
  }
  const uint32_t tmem = bars->tmem_slot;  // not warp 0's to read
  // Registers move to the two softmax warpgroups (a row of scores is 128 of
  // them); the shares of all warpgroups add up to no more than the CTA was
  // launched with: 2 x 208 + 88 = 3 x 168; with an e4m3 cache (640 threads of
  // 96, the scores read in quarters) 2 x 136 + 3 x 64 <= 5 x 96.
  if (warp >= 4 && warp < 12) {
    reg_acquire<KV8 ? 136 : 208>();
    // ============================================ softmax / rescale / epilogue
    const int x = (warp >= 8) ? 1 : 0;
    const int r = threadIdx.x - 128 - 128 * x;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_off + x * 128;
    const uint32_t o_tm = tmem + lane_off + 256;  // O of x at + 128 x
    const int block = r / RB, row_r = r % RB;  // this thread's keys of a tile, its query row
    constexpr int SHARE = 32 / BLOCKS;         // of 32 columns of O, those a block writes
    const int tok_r = row_r / p.G, head_r = row_r % p.G;
    // waits taken on s_full[x] and o_done[1]; segments; tiles; exchanges
    int ns = 0, no1 = 0, seg = 0, ti = 0, ex = 0;
    TreeWalk w;
    bool ok = w.begin(p, bars);
    if (threadIdx.x == 128) p.part_unit[blockIdx.x] = make_int4(0, 0, 0, -1);  // also if a wait runs out below
    while (ok) {
      const int n = w.n();
      const int t = w.m * p.R + tok_r;
      const bool row_live = row_r < p.R * p.G && t < w.T;
      const bool warp_live = (warp & 3) * 32 % RB < w.rows(p);
      uint64_t bits = 0;
      if (row_live) {
        bits = p.mask ? p.mask[w.row0 + t] : (2ull << t) - 1;  // t = 63: 2 << 63 = 0, minus 1: all
        if (w.T < 64) bits &= (1ull << w.T) - 1;
      }
      float scale = p.scale_log2;
      if (CODES) {
        if (!(ok = warp_wait(&bars->q_full, seg & 1, p.limit_ns, abort_flag, 847))) break;
        scale *= reinterpret_cast<const float*>(smem + SM::QSC)[row_r];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->qsc_read);
      }
      RowState st;
      for (int j = x; j < n; j += 2, ++ns) {
        if (!(ok = warp_wait(&bars->s_full[x], ns & 1, p.limit_ns, abort_flag, 841))) break;
        tc_fence_after();
        const float* sc_s = nullptr;
        if (KV8) {
          const int slot = (ti + j) % TR_SCALES;
          if (!(ok = warp_wait(&bars->sc_full[slot], ((ti + j) / TR_SCALES) & 1, p.limit_ns, abort_flag, 842))) break;
          sc_s = scales + slot * 256;
        }
        if (warp_live) {
          const int base = (w.t0 + j) * 128;
          const int q0 = block * (RB / 32);
          const float* vs_s = KV8 ? sc_s + 128 : nullptr;
          uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
          float alpha;
          bool resc;
          if (base + 128 > w.ctx) {
            tree_visible(w.ctx, base, bits, vis);
            resc = softmax_quarters<RB / 32, KV8, true>(s_tm, q0, scale, sc_s, vs_s, vis, st, alpha);
          } else {
            resc = softmax_quarters<RB / 32, KV8, false>(s_tm, q0, scale, sc_s, vs_s, vis, st, alpha);
          }
          // P V(j - 2) completed before S(j): s_full's commit covers it
          if (j >= 2 && __any_sync(0xffffffffu, resc)) rescale_row(o_tm + 128 * x, alpha);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars->p_ready[x]);
          if (KV8) mbar_arrive(&bars->sc_empty[(ti + j) % TR_SCALES]);
        }
      }
      if (!ok) break;
      // ---- epilogue: join the O of the even and the odd tiles and of the row
      // blocks.  Once O is done the (m, l) area is free: this segment's products
      // waited (o_free) for every warp to be through with the last segment's.
      ok = warp_wait(&bars->o_done[0], seg & 1, p.limit_ns, abort_flag, 843);
      if (ok && n > 1) ok = warp_wait(&bars->o_done[1], no1++ & 1, p.limit_ns, abort_flag, 845);
      if (!ok) break;
      ml[x * 128 + r] = make_float2(st.m, st.l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->ml_ready);
      if (!(ok = warp_wait(&bars->ml_ready, seg & 1, p.limit_ns, abort_flag, 844))) break;
      tc_fence_after();
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int k = 0; k < 2 * BLOCKS; ++k) M = fmaxf(M, ml[k * RB + row_r].x);
#pragma unroll
      for (int k = 0; k < 2 * BLOCKS; ++k) {
        const float2 q = ml[k * RB + row_r];
        L += q.x == -INFINITY ? q.y : q.y * ex2_approx(q.x - M);  // without a max: 0, or the NaN of its scores
      }
      const float ma = ml[r].x, mb = ml[128 + r].x;
      const float wa = ma == -INFINITY ? 0.f : ex2_approx(ma - M);
      const float wb = mb == -INFINITY ? 0.f : ex2_approx(mb - M);
      const uint64_t wa2 = f2_pack(wa, wa), wb2 = f2_pack(wb, wb);
      const bool whole = w.whole();
      const float inv = !whole ? 1.f : (L == 0.f ? 0.f : 1.f / L);
      const int64_t row = w.row0 + t;
      const int h = w.g * p.G + head_r;
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (w.t0 == 0 ? 1 : 0);
#pragma unroll 1
      for (int c = 2 * x; c < 2 * x + 2; ++c) {  // this warpgroup's half of the columns
        uint64_t v[16];
        if (warp_live) {
          uint32_t oa[32], ob[32];
          tmem_ld32(o_tm + c * 32, oa);
          if (!KV8 && n > 1) tmem_ld32(o_tm + 128 + c * 32, ob);
          tmem_ld_wait();
          reg_fence(oa);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            v[e] = f2_mul(f2_pack(__uint_as_float(oa[2 * e]), __uint_as_float(oa[2 * e + 1])), wa2);
          if (n > 1) {
            if (KV8) {  // fewer registers: one after the other
              tmem_ld32(o_tm + 128 + c * 32, ob);
              tmem_ld_wait();
            }
            reg_fence(ob);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              v[e] = f2_fma(f2_pack(__uint_as_float(ob[2 * e]), __uint_as_float(ob[2 * e + 1])), wb2, v[e]);
          }
        }
        if (BLOCKS > 1) {
          // Each block takes SHARE of the 32 columns and hands the others'
          // theirs through shared memory: [taker][giver][row][SHARE], the
          // 16-byte chunks XOR-ed with the row so that a store or load of
          // eight lanes meets every bank once.
          const uint32_t area = exch_base + static_cast<uint32_t>(x * (128 - RB)) * 128u;
          auto place = [&](int taker, int giver) {
            return area + static_cast<uint32_t>((taker * (BLOCKS - 1) + giver) * RB + row_r) * (SHARE * 4u);
          };
          auto chunk = [&](int q) {
            return static_cast<uint32_t>(q ^ ((row_r >> 2) & (SHARE / 4 - 1))) << 4;
          };
          if (ex > 0 && !(ok = warp_wait(&bars->x_free[x], (ex - 1) & 1, p.limit_ns, abort_flag, 846))) break;
          if (warp_live) {
#pragma unroll
            for (int k = 0; k < BLOCKS; ++k) {  // columns SHARE k ..: to block k
              if (k == block) continue;
              const uint32_t at = place(k, block < k ? block : block - 1);
#pragma unroll
              for (int q = 0; q < SHARE / 4; ++q) {
                const uint64_t lo = v[k * (SHARE / 2) + 2 * q], hi = v[k * (SHARE / 2) + 2 * q + 1];
                st_shared_v4(at + chunk(q), make_uint4(static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32),
                                                       static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)));
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->x_ready[x]);
          if (!(ok = warp_wait(&bars->x_ready[x], ex & 1, p.limit_ns, abort_flag, 848))) break;
          if (warp_live) {
            uint64_t mine[SHARE / 2];
#pragma unroll
            for (int k = 0; k < BLOCKS; ++k)
              if (k == block) {
#pragma unroll
                for (int e = 0; e < SHARE / 2; ++e) mine[e] = v[k * (SHARE / 2) + e];
              }
#pragma unroll
            for (int k = 0; k < BLOCKS - 1; ++k) {
              const uint32_t at = place(block, k);
#pragma unroll
              for (int q = 0; q < SHARE / 4; ++q) {
                const uint4 y = ld_shared_v4(at + chunk(q));
                mine[2 * q] = f2_add(mine[2 * q], f2_pack(__uint_as_float(y.x), __uint_as_float(y.y)));
                mine[2 * q + 1] = f2_add(mine[2 * q + 1], f2_pack(__uint_as_float(y.z), __uint_as_float(y.w)));
              }
            }
#pragma unroll
            for (int e = 0; e < SHARE / 2; ++e) v[e] = mine[e];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->x_free[x]);
          ++ex;
        }
        if (!warp_live || !row_live) continue;
        const int col = c * 32 + block * SHARE;  // SHARE columns from here on, in v
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(p.o + row * p.q_tok + static_cast<int64_t>(h) * p.q_head + col);
#pragma unroll
          for (int q = 0; q < SHARE / 8; ++q) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float y0, y1;
              f2_unpack(f2_mul(v[4 * q + e], f2_pack(inv, inv)), y0, y1);
              o[e] = pack_bf16x2(y0, y1);
            }
            dst[q] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        } else {
          ulonglong2* dst = reinterpret_cast<ulonglong2*>(p.part_o + (slot * 128 + row_r) * 128 + col);
#pragma unroll
          for (int q = 0; q < SHARE / 4; ++q) dst[q] = make_ulonglong2(v[2 * q], v[2 * q + 1]);
        }
      }
      if (!ok) break;
      if (row_live && x == 0 && block == 0) {
        if (!whole)
          p.part_ml[slot * 128 + row_r] = make_float2(M, L);
        else if (p.lse)
          p.lse[static_cast<int64_t>(h) * p.n_tok + row] = (M + log2f(L)) * 0.69314718055994530942f;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->o_free);
      ti += n;
      ++seg;
      // the stretch's last segment may be a unit's first part
      if (threadIdx.x == 128 && w.last()) {
        const bool head = w.t0 == 0 && w.t1 < w.tiles;
        // the CTA with the unit's last tile (its segment begins at tile 0)
        const int end = w.pos + TR_OVERHEAD + w.tiles - 1, big = bars->more * (bars->each + 1);
        const int last = end < big ? end / (bars->each + 1) : bars->more + (end - big) / bars->each;
        p.part_unit[blockIdx.x] = make_int4(w.row0 + w.m * p.R, min(p.R, w.T - w.m * p.R), w.g, head ? last : -1);
      }
      if (!w.next(p)) break;
    }
  } else {
    reg_release<KV8 ? 64 : 88>();
    if (warp == 0) {
      // =========================================================== TMA loads
      TreeWalk w;
      const bool work = !(p.flags & FLAG_SKIP_LOADS) && w.begin(p, bars);
      const int page = 1 << p.page_log2, per_tile = 128 >> p.page_log2;
      int item = 0, kc = 0, vc = 0;  // in one ring, or (CODES) K and V in rings of their own
      uint32_t raw_used = 0, raw_uses = 0;  // slots last filled through v_raw, and how often (mod 2)
      bool ok = work;
      while (ok) {
        const int n = w.n(), len = w.ctx + w.T;
        const int32_t* table = p.table + static_cast<int64_t>(w.b) * p.max_pages;
        // each lane's page of an item, read one item ahead of its use
        auto page_of = [&](int u) {
          int tile;
          bool is_v;
          tree_item(u, n, tile, is_v);
          const int at = (w.t0 + tile) * 128 + lane * page;
          return (u < 2 * n && lane < per_tile && at < len) ? table[at >> p.page_log2] : 0;
        };
        int pg = page_of(0);
        for (int u = 0; u < 2 * n; ++u, ++item) {
          int tile;
          bool is_v;
          tree_item(u, n, tile, is_v);
          const int next_pg = page_of(u + 1);
          const bool v8 = CODES && is_v;
          const int ring = !KV8 ? ITEMS : v8 ? V8 : K8, at = !CODES ? item : is_v ? vc : kc;
          const int slot = at % ring;
          uint64_t* full = !KV8 ? bars->full : v8 ? bars->v8_full : bars->k8_full;
          uint64_t* empty = !KV8 ? bars->empty : v8 ? bars->v8_empty : bars->k8_empty;
          if (at >= ring && !warp_wait(&empty[slot], ((at / ring) - 1) & 1, p.limit_ns, abort_flag, 812)) {
            ok = false;
            break;
          }
          const int keys = min(128, len - (w.t0 + tile) * 128);
          const int pages = (keys + page - 1) >> p.page_log2;  // the rest of the tile is not loaded
          // a last V tile to be mended reaches `full` through warp 2
          const bool mend = !KV8 && is_v && tile == n - 1 && w.last_rows() < 128;
          uint64_t* bar = mend ? &bars->v_raw[slot] : &full[slot];
          raw_used = (raw_used & ~(1u << slot)) | (mend ? 1u << slot : 0u);
          raw_uses ^= mend ? 1u << slot : 0u;
          if (lane == 0)
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(pages << p.page_log2) * (KV8 ? 128u : 256u));
          __syncwarp();
          if (lane < pages) {
            if (pg < 0 || pg >= p.n_pages) {
              report(HS2_ERR_INDEX, 813);
              pg = p.n_pages;  // behind the pools: reads as zeros
            }
            const CUtensorMap* map = is_v ? &tmV : &tmK;
            uint8_t* dst = smem + lane * page * 128 +
                           (!KV8 ? SM::ITEM + slot * TILE_BYTES : (v8 ? SM::V8_AT : SM::K8_AT) + slot * RAW_BYTES);
            const int tok = pg << p.page_log2;
            tma_load_3d(dst, map, bar, 0, w.g, tok);
            if (!KV8) tma_load_3d(dst + HALF_BYTES, map, bar, 64, w.g, tok);
          }
          (is_v ? vc : kc) += 1;
          pg = next_pg;
        }
        if (!ok || !w.next(p)) break;
      }
      // never leave a TMA write in flight into memory the CTA gives back
      __syncwarp();
      if (lane == 0 && work && KV8) {
        const int in_k8 = CODES ? kc : item;
        for (int u = max(0, in_k8 - K8); u < in_k8; ++u)
          wait_done(&bars->k8_full[u % K8], (u / K8) & 1, p.limit_ns, 814);
        if constexpr (CODES)
          for (int u = max(0, vc - V8); u < vc; ++u) wait_done(&bars->v8_full[u % V8], (u / V8) & 1, p.limit_ns, 817);
      } else if (lane == 0 && work) {
        for (int u = max(0, item - ITEMS); u < item; ++u)
          if (raw_used >> (u % ITEMS) & 1u)
            wait_done(&bars->v_raw[u % ITEMS], ~(raw_uses >> (u % ITEMS)) & 1u, p.limit_ns, 819);
          else
            wait_done(&bars->full[u % ITEMS], (u / ITEMS) & 1, p.limit_ns, 820);
      }
    } else if (warp == 1) {
      // ========================================================== MMA issue
      TreeWalk w;
      if (w.begin(p, bars)) {  // the warp walks together, its elected lane issues
        int item = 0, vc = 0, seg = 0;  // next item, or (CODES) K tile, next V tile
        uint32_t np = 0;  // by tile parity: tiles so far (mod 2)
        bool ok = true;
        auto wait_for = [&](uint64_t* bar, uint32_t parity, int where) {
          return warp_wait(bar, parity, p.limit_ns, abort_flag, where);
        };
        auto wait_item = [&](int u) {  // (CODES) of K only
          if constexpr (CODES) return wait_for(&bars->k8_full[u % K8], (u / K8) & 1, 821);
          return wait_for(&bars->full[u % ITEMS], (u / ITEMS) & 1, 821);
        };
        auto issue_s = [&](int x, int u, bool last) {
          const uint64_t da = sdesc_sw128(q_base, 16, 1024);
          const uint64_t db = sdesc_sw128(CODES ? smem_u32(smem + SM::K8_AT) + (u % K8) * RAW_BYTES
                                                : item_base + (u % ITEMS) * TILE_BYTES, 16, 1024);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < (CODES ? 12 : 8); ++kk) {  // CODES: the same keys times each part of the queries
              const uint32_t step = (kk & 3) * 32 >> 4, part = (kk >> 2) * HALF_BYTES >> 4;
              if (CODES)
                umma_ss_f8(tmem + x * 128, da + part + step, db + step, idesc_f8_f32(128, 128, 1, 0),
                           kk > 0 ? 1u : 0u);
              else
                umma_ss(tmem + x * 128, da + part + step, db + part + step, IDESC_S, kk > 0 ? 1u : 0u);
            }
            umma_commit(&bars->s_full[x]);
            umma_commit(CODES ? &bars->k8_empty[u % K8] : &bars->empty[u % ITEMS]);
            if (last) umma_commit(&bars->q_empty);
          }
          __syncwarp();
        };
        auto issue_pv = [&](int x, int u, bool first, bool last) {
          const uint64_t db = sdesc_sw128(item_base + (u % ITEMS) * TILE_BYTES, HALF_BYTES, 1024);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, db + kk * (2048 >> 4), IDESC_PV,
                      (!first || kk > 0) ? 1u : 0u);
            umma_commit(&bars->empty[u % ITEMS]);
            if (last) umma_commit(&bars->o_done[x]);
          }
          __syncwarp();
        };
        while (ok) {
          const int n = w.n();
          ok = wait_for(&bars->q_full, seg & 1, 822) && wait_item(item);
          if (!ok) break;
          tc_fence_after();
          issue_s(0, item++, n == 1);
          if (n > 1) {
            if (!(ok = wait_item(item))) break;
            tc_fence_after();
            issue_s(1, item++, n == 2);
          }
          for (int j = 0; j < n; ++j) {
            const int x = j & 1;
            // V(j) and K(j + 2) normally landed long ago: nothing but P stands
            // between its arrival and the products.  A K(j + 2) that is converted
            // may not be there yet, so P V does not wait for it.
            if constexpr (CODES)
              ok = wait_for(&bars->full[vc % ITEMS], (vc / ITEMS) & 1, 827) && (j + 2 >= n || wait_item(item));
            else
              ok = wait_item(item) && (KV8 || j + 2 >= n || wait_item(item + 1));
            // the last segment's O has been read
            if (ok && j == 0 && seg > 0) ok = wait_for(&bars->o_free, (seg - 1) & 1, 824);
            if (ok) ok = wait_for(&bars->p_ready[x], (np >> x) & 1, 825);
            np ^= 1u << x;
            if (!ok) break;
            tc_fence_after();
            issue_pv(x, CODES ? vc++ : item++, j < 2, j + 2 >= n);
            if (j + 2 < n) {
              if (KV8 && !CODES) {
                if (!(ok = wait_item(item))) break;
                tc_fence_after();
              }
              issue_s(x, item++, j + 3 == n);
            }
          }
          ++seg;
          if (!ok || !w.next(p)) break;
        }
        if (elect_one()) umma_commit(&bars->fin);
        __syncwarp();
        wait_done(&bars->fin, 0, p.limit_ns, 826);
      }
    } else if (warp == 3) {
      // ======================= a segment's queries, once the last one's products
      // have read theirs (the K / V loads above do not wait for that)
      TreeWalk w;
      if (!CODES && lane == 0 && !(p.flags & FLAG_SKIP_LOADS) && w.begin(p, bars)) {
        const uint32_t half = static_cast<uint32_t>(p.R * p.G) * 128u;
        int seg = 0;
        do {
          if (seg > 0 && !mbar_wait(&bars->q_empty, (seg - 1) & 1, p.limit_ns, abort_flag, 816)) break;
          mbar_arrive_expect_tx(&bars->q_full, 2 * BLOCKS * half);
          for (int k = 0; k < BLOCKS; ++k) {  // the same rows for every block
            uint8_t* dst = smem + k * RB * 128;
            tma_load_3d(dst, &tmQ, &bars->q_full, 0, w.g * p.G, w.row0 + w.m * p.R);
            tma_load_3d(dst + HALF_BYTES, &tmQ, &bars->q_full, 64, w.g * p.G, w.row0 + w.m * p.R);
          }
          ++seg;
        } while (w.next(p));
        wait_done(&bars->q_full, (seg - 1) & 1, p.limit_ns, 815);
      }
    } else if (warp == 2) {
      TreeWalk w;
      if (!(p.flags & FLAG_SKIP_LOADS) && w.begin(p, bars)) {
        if (!KV8) {
          // ================================ V rows behind the sequence's last key
          int item = 0;
          uint32_t uses = 0;  // of each slot's v_raw, mod 2
          do {
            item += 2 * w.n();
            if (w.last_rows() < 128) {
              const int slot = (item - 1) % ITEMS;  // a segment's last item is its last V tile
              if (!warp_wait(&bars->v_raw[slot], uses >> slot & 1u, p.limit_ns, abort_flag, 831)) break;
              uses ^= 1u << slot;
              zero_rows(item_base + slot * TILE_BYTES, w.last_rows(), lane, 32);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars->full[slot]);
            }
          } while (w.next(p));
        } else {
          // ============ scales of the keys: asynchronous copies, several tiles ahead
          int ti = 0;
          bool ok = true;
          do {
            const int len = w.ctx + w.T;
            const int32_t* table = p.table + static_cast<int64_t>(w.b) * p.max_pages;
            int pg[4];  // pages of this lane's keys, read one tile ahead
            auto pages_of = [&](int t) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int at = t * 128 + lane + 32 * e;
                pg[e] = (t < w.t1 && at < len) ? table[at >> p.page_log2] : -1;
              }
            };
            pages_of(w.t0);
            for (int t = w.t0; t < w.t1; ++t, ++ti) {
              const int slot = ti % TR_SCALES;
              if (ti >= TR_SCALES && !warp_wait(&bars->sc_empty[slot], ((ti / TR_SCALES) - 1) & 1, p.limit_ns,
                                                abort_flag, 832)) {
                ok = false;
                break;
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int at = t * 128 + lane + 32 * e;
                const bool have = pg[e] >= 0 && pg[e] < p.n_pages;  // a page outside the pools reads as zeros
                const int64_t tok =
                    have ? (static_cast<int64_t>(pg[e]) << p.page_log2) + (at & ((1 << p.page_log2) - 1)) : 0;
                const uint32_t dst = smem_u32(scales + slot * 256 + lane + 32 * e);
                cp_async_4(dst, p.ksc + tok * p.Hkv + w.g, have ? 4u : 0u);
                cp_async_4(dst + 512, p.vsc + tok * p.Hkv + w.g, have ? 4u : 0u);
              }
              cp_async_arrive(&bars->sc_full[slot]);
              pages_of(t + 1);
            }
          } while (ok && w.next(p));
          cp_async_wait_all();  // nothing may be on its way into memory the CTA gives back
        }
      }
    } else {
      // ==== e4m3: codes to bf16, K's and V's or (CODES) V's, and a segment's queries
      // to sums of codes
      TreeWalk w;
      if (KV8 && !(p.flags & FLAG_SKIP_LOADS) && w.begin(p, bars)) {
        const int pt = threadIdx.x - 384;
        const uint32_t raw_base = smem_u32(smem + (CODES ? SM::V8_AT : SM::K8_AT));
        constexpr int RAWS = CODES ? V8 : K8;
        uint64_t* raw_full = CODES ? bars->v8_full : bars->k8_full;
        uint64_t* raw_empty = CODES ? bars->v8_empty : bars->k8_empty;
        int at = 0, seg = 0;
        bool ok = true;
        do {
          if constexpr (CODES) {
            constexpr int STEPS = RB * 32 / (2 * TR_CONV);
            uint4 raw[STEPS];
            load_queries<STEPS, TR_CONV / 32>(p, w.g, w.row0 + w.m * p.R, w.rows(p), pt >> 5, raw);
            // the last segment's products have read its queries, the softmax its scales
            if (seg > 0 && !(warp_wait(&bars->q_empty, (seg - 1) & 1, p.limit_ns, abort_flag, 816) &&
                             warp_wait(&bars->qsc_read, (seg - 1) & 1, p.limit_ns, abort_flag, 818)))
              break;
            split_queries<STEPS, TR_CONV / 32, BLOCKS>(raw, smem, HALF_BYTES, reinterpret_cast<float*>(smem + SM::QSC),
                                                       RB, pt >> 5);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->q_full);
            ++seg;
          }
          const int n = w.n(), len = w.ctx + w.T;
          for (int u = 0; u < (CODES ? n : 2 * n) && ok; ++u, ++at) {
            int tile = u;
            bool is_v = true;
            if (!CODES) tree_item(u, n, tile, is_v);
            const int keys = len - (w.t0 + tile) * 128;  // rows from here on are behind the sequence
            const int rs = at % RAWS, cs = at % ITEMS;
            ok = warp_wait(&raw_full[rs], (at / RAWS) & 1, p.limit_ns, abort_flag, 851) &&
                 (at < ITEMS || warp_wait(&bars->empty[cs], ((at / ITEMS) - 1) & 1, p.limit_ns, abort_flag, 852));
            if (!ok) break;
            convert_tile<TR_CONV>(raw_base + rs * RAW_BYTES, item_base + cs * TILE_BYTES, keys, pt);
            fence_proxy_async_smem();
            __syncwarp();  // one arrival per warp: 256 of them would take longer than the conversion
            if (lane == 0) {
              mbar_arrive(&bars->full[cs]);
              mbar_arrive(&raw_empty[rs]);
            }
          }
        } while (ok && w.next(p));
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

// Adds a part (m, l) = q, O = v to a row's (M, L), acc.
__device__ __forceinline__ void merge_part(float& M, float& L, float4& acc, float2 q, float4 v) {
  const float m = fmaxf(M, q.x);
  const float keep = M == -INFINITY ? 0.f : ex2_approx(M - m), w = q.x == -INFINITY ? 0.f : ex2_approx(q.x - m);
  L = (M == -INFINITY ? L : L * keep) + (q.x == -INFINITY ? q.y : q.y * w);  // without a max: 0, or a NaN that stays
  acc.x = fmaf(v.x, w, acc.x * keep);
  acc.y = fmaf(v.y, w, acc.y * keep);
  acc.z = fmaf(v.z, w, acc.z * keep);
  acc.w = fmaf(v.w, w, acc.w * keep);
  M = m;
}

// Joins the parts of the units that several CTAs share: block (c, y) takes rows
// y, y + gridDim.y, ... of the unit whose first part CTA c holds.  A row's parts
// are spread over 1, 2, 4 or 8 warps, so that a long chain of parts is read at
// once; the warps' sums meet in shared memory, in a fixed order.
constexpr int TM_WARPS = 8;
__global__ void __launch_bounds__(32 * TM_WARPS) tree_merge_kernel(const TreeParams p) {
  __shared__ float4 acc_s[TM_WARPS][32];
  __shared__ float2 ml_s[TM_WARPS];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched beside tree_attn_kernel's end
  const int c = blockIdx.x;
  const int4 u = p.part_unit[c];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = u.y * p.G;
  if (u.w < 0 || static_cast<int>(blockIdx.y) >= rows) return;
  const int n = u.w - c + 1;
  const int per_row = n <= 2 ? 1 : n <= 4 ? 2 : n <= 8 ? 4 : 8;  // warps of a row
  const int sub = warp / per_row, wk = warp % per_row;
  for (int i0 = 0; static_cast<int>(blockIdx.y) + i0 * static_cast<int>(gridDim.y) < rows; i0 += TM_WARPS / per_row) {
    const int r = blockIdx.y + (i0 + sub) * gridDim.y;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) {
      // parts in key order: slot 1 of CTA c, then slot 0 of CTAs c + 1 .. last
      auto slot = [&](int k) { return (static_cast<int64_t>(c + k) * 2 + (k == 0 ? 1 : 0)) * 128 + r; };
      for (int k0 = wk; k0 < n; k0 += 4 * per_row) {
        float4 v[4];
        float2 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = k0 + i * per_row;
          q[i] = make_float2(-INFINITY, 0.f);
          v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < n) {
            q[i] = p.part_ml[slot(k)];
            v[i] = reinterpret_cast<const float4*>(p.part_o + slot(k) * 128)[lane];
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) merge_part(M, L, acc, q[i], v[i]);
      }
    }
    acc_s[warp][lane] = acc;
    if (lane == 0) ml_s[warp] = make_float2(M, L);
    __syncthreads();
    if (wk == 0 && r < rows) {
      for (int k = 1; k < per_row; ++k) merge_part(M, L, acc, ml_s[warp + k], acc_s[warp + k][lane]);
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const int h = u.z * p.G + r % p.G;
      const int64_t row = u.x + r / p.G;
      *reinterpret_cast<uint2*>(p.o + row * p.q_tok + static_cast<int64_t>(h) * p.q_head + lane * 4) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (lane == 0 && p.lse)
        p.lse[static_cast<int64_t>(h) * p.n_tok + row] = (M + log2f(L)) * 0.69314718055994530942f;
    }
    __syncthreads();
  }
}

}  // namespace hs2
