// The softmax of one 128 x 128 score tile held in tensor memory, as the
// attention kernels around a cache run it: thread r of a softmax warpgroup
// owns query row r (TMEM lane r).  Log2 domain, reference max updated only when
// a row's max grows by more than 8 (P stays below 256 and O / l is exact up to
// rounding), row max in 8 chains of 3-input max, arguments and sums as packed
// f32x2, sums and reference in fp32; P is rounded to bf16 once, for the
// product (its sum is of the unrounded values).
#pragma once

#include "common.cuh"
#include "flash.cuh"

namespace hs2 {

struct RowState {
  float m = -INFINITY;  // reference max, log2 units
  float l = 0.f;        // sum of 2^(s - m)
};

__device__ __forceinline__ void load_scores(uint32_t s_tm, uint32_t (&sr)[4][32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_ld32(s_tm + 32 * c, sr[c]);
  tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < 4; ++c) reg_fence(sr[c]);
}

// Columns c > last hold no visible key.
__device__ __forceinline__ void mask_after(uint32_t (&sr)[4][32], int last) {
#pragma unroll
  for (int c = 0; c < 128; ++c)
    if (c > last) sr[c >> 5][c & 31] = __float_as_uint(-INFINITY);
}

// Moves the reference max to a row max of `mx` (scaled) where that grew by more
// than 8; returns whether, with what l and O have to be multiplied by.
__device__ __forceinline__ bool update_max(float mx, RowState& st, float& alpha) {
  const float m_new = fmaxf(st.m, mx);
  alpha = 1.f;
  const bool resc = m_new > st.m + 8.f;
  if (resc) {
    alpha = ex2_approx(st.m - m_new);
    st.m = m_new;
  }
  st.l *= alpha;
  return resc;
}

__device__ __forceinline__ float max32(const uint32_t (&v)[32]) {
  float mx2[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t* u = &v[q * 16];
    float m = fmax3(__uint_as_float(u[0]), __uint_as_float(u[1]), __uint_as_float(u[2]));
#pragma unroll
    for (int e = 0; e < 6; ++e) m = fmax3(m, __uint_as_float(u[3 + 2 * e]), __uint_as_float(u[4 + 2 * e]));
    mx2[q] = fmaxf(m, __uint_as_float(u[15]));
  }
  return fmaxf(mx2[0], mx2[1]);
}

// P of a tile with its row in registers, over the scores' first 64 columns;
// returns whether this row's O has to be multiplied by alpha.
__device__ __forceinline__ bool softmax_tile(uint32_t s_tm, const uint32_t (&sr)[4][32], float sc, RowState& st,
                                             float& alpha) {
  const float mx = fmaxf(fmaxf(max32(sr[0]), max32(sr[1])), fmaxf(max32(sr[2]), max32(sr[3])));
  const bool resc = update_max(mx * sc, st, alpha);
  const float mu = (st.m == -INFINITY) ? 0.f : st.m;
  const uint64_t sc2 = f2_pack(sc, sc), nmu2 = f2_pack(-mu, -mu);
  uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint64_t a2 =
          f2_fma(f2_pack(__uint_as_float(sr[c][2 * e]), __uint_as_float(sr[c][2 * e + 1])), sc2, nmu2);
      const uint64_t p2 = ex2_x2(a2);
      sum2[e & 1] = f2_add(sum2[e & 1], p2);
      float e0, e1;
      f2_unpack(p2, e0, e1);
      pk[e] = pack_bf16x2(e0, e1);
    }
    tmem_st16(s_tm + c * 16, pk);
  }
  float a0, a1, b0, b1;
  f2_unpack(sum2[0], a0, a1);
  f2_unpack(sum2[1], b0, b1);
  st.l += (a0 + a1) + (b0 + b1);
  return resc;
}

// The same for NQ quarters (32 columns each) of a tile from quarter q0 on, the
// other columns' P set to zero; optionally (SCALED) with a K and a V scale per
// key in shared memory ([128] each: scores are multiplied by the K scale, and P
// times the V scale is what is rounded, the sum is of P), and (MASKED) with the
// visible columns in 4 words.  A whole tile's scores are read from tensor
// memory twice, a quarter ahead of its use, so that a row takes 64 registers,
// and in loops of two quarters: unrolled, with the mask's code among it, the
// warps waited for instructions more than for anything else (3.5 of 13 cycles
// an instruction).
template <int NQ, bool SCALED, bool MASKED>
__device__ __forceinline__ bool softmax_quarters(uint32_t s_tm, int q0, float sc, const float* kscale,
                                                 const float* vscale, const uint32_t (&vis)[4], RowState& st,
                                                 float& alpha) {
  static_assert(NQ == 1 || NQ == 4, "quarters");
  uint32_t buf[2][32];
  auto issue = [&](int q, uint32_t(&sr)[32]) { tmem_ld32(s_tm + 32 * q, sr); };
  auto arrived = [&](uint32_t(&sr)[32]) {
    tmem_ld_wait();
    reg_fence(sr);
  };
  // scores of quarter q as they enter the softmax
  auto prepare = [&](int q, uint32_t(&sr)[32]) {
    if (SCALED) {
      const ulonglong2* ks = reinterpret_cast<const ulonglong2*>(kscale + 32 * q);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const ulonglong2 k2 = ks[e];  // broadcast
        float a0, a1, a2, a3;
        f2_unpack(f2_mul(f2_pack(__uint_as_float(sr[4 * e]), __uint_as_float(sr[4 * e + 1])), k2.x), a0, a1);
        f2_unpack(f2_mul(f2_pack(__uint_as_float(sr[4 * e + 2]), __uint_as_float(sr[4 * e + 3])), k2.y), a2, a3);
        sr[4 * e] = __float_as_uint(a0);
        sr[4 * e + 1] = __float_as_uint(a1);
        sr[4 * e + 2] = __float_as_uint(a2);
        sr[4 * e + 3] = __float_as_uint(a3);
      }
    }
    if (MASKED) {
      const uint32_t w = q < 2 ? (q ? vis[1] : vis[0]) : (q == 2 ? vis[2] : vis[3]);
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (!(w >> e & 1u)) sr[e] = __float_as_uint(-INFINITY);
    }
  };
  float mx = -INFINITY;
  issue(q0, buf[0]);
#pragma unroll 1
  for (int h = 0; h < (NQ == 4 ? 2 : 1); ++h) {
    const int q = q0 + 2 * h;
    arrived(buf[0]);
    if (NQ > 1) issue(q + 1, buf[1]);
    prepare(q, buf[0]);
    mx = fmaxf(mx, max32(buf[0]));
    if (NQ > 1) {
      arrived(buf[1]);
      if (NQ == 4) issue(h == 0 ? q + 2 : q0, buf[0]);  // at last quarter 0 again
      prepare(q + 1, buf[1]);
      mx = fmaxf(mx, max32(buf[1]));
    }
  }
  const bool resc = update_max(mx * sc, st, alpha);
  const float mu = (st.m == -INFINITY) ? 0.f : st.m;
  const uint64_t sc2 = f2_pack(sc, sc), nmu2 = f2_pack(-mu, -mu);
  uint64_t sum2[2] = {0ull, 0ull};
  // P of quarter q, over scores that this thread has read for the last time (a
  // quarter on its way to registers lies behind them)
  auto weigh = [&](int q, const uint32_t(&sr)[32]) {
    const ulonglong2* vs = reinterpret_cast<const ulonglong2*>(vscale + 32 * q);
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint64_t a2 = f2_fma(f2_pack(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), sc2, nmu2);
      uint64_t p2 = ex2_x2(a2);
      sum2[e & 1] = f2_add(sum2[e & 1], p2);
      if (SCALED) p2 = f2_mul(p2, (e & 1) ? vs[e >> 1].y : vs[e >> 1].x);
      float e0, e1;
      f2_unpack(p2, e0, e1);
      pk[e] = pack_bf16x2(e0, e1);
    }
    tmem_st16(s_tm + 16 * q, pk);
  };
#pragma unroll 1
  for (int h = 0; h < (NQ == 4 ? 2 : 1); ++h) {
    const int q = q0 + 2 * h;
    if (NQ == 4) {
      arrived(buf[0]);
      issue(q + 1, buf[1]);
      prepare(q, buf[0]);
    }
    weigh(q, buf[0]);
    if (NQ == 4) {
      arrived(buf[1]);
      if (h == 0) issue(q + 2, buf[0]);
      prepare(q + 1, buf[1]);
    }
    if (NQ > 1) weigh(q + 1, buf[1]);
  }
  if (NQ < 4) {
    uint32_t zero[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) zero[e] = 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < q0 || q >= q0 + NQ) tmem_st16(s_tm + q * 16, zero);
  }
  float a0, a1, b0, b1;
  f2_unpack(sum2[0], a0, a1);
  f2_unpack(sum2[1], b0, b1);
  st.l += (a0 + a1) + (b0 + b1);
  return resc;
}

// O row times alpha in tensor memory (warp-uniform call).
__device__ __forceinline__ void rescale_row(uint32_t o_tm, float alpha) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t orr[32];
    tmem_ld32(o_tm + c * 32, orr);
    tmem_ld_wait();
    reg_fence(orr);
#pragma unroll
    for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
    tmem_st32(o_tm + c * 32, orr);
  }
}

// Zeroes rows [first, 128) of a V tile in shared memory (two 128-byte-swizzled
// halves), for the tensor core: a weight of zero times whatever lies behind a
// sequence's last key must be zero, also where that is an infinity or a NaN.
__device__ __forceinline__ void zero_rows(uint32_t tile, int first, int thread, int threads) {
  for (int i = first * 16 + thread; i < 128 * 16; i += threads)
    st_shared_v4(tile + sw128_chunk_offset(i >> 4, i & 15, 128), make_uint4(0, 0, 0, 0));
}

}  // namespace hs2
