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

// P of the tile over the scores' first 64 columns; returns whether this row's
// O has to be multiplied by alpha.  With a V scale per key (VSCALE) P times
// the scale is what is rounded; the sum is of P.
template <bool VSCALE>
__device__ __forceinline__ bool softmax_tile(uint32_t s_tm, const uint32_t (&sr)[4][32], float sc,
                                             const float* vscale, RowState& st, float& alpha) {
  float mx8[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t* v = &sr[q >> 1][(q & 1) * 16];
    float m = fmax3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
#pragma unroll
    for (int e = 0; e < 6; ++e) m = fmax3(m, __uint_as_float(v[3 + 2 * e]), __uint_as_float(v[4 + 2 * e]));
    mx8[q] = fmaxf(m, __uint_as_float(v[15]));
  }
  const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
  const float m_new = fmaxf(st.m, mx * sc);
  alpha = 1.f;
  const bool resc = m_new > st.m + 8.f;
  if (resc) {
    alpha = ex2_approx(st.m - m_new);
    st.m = m_new;
  }
  const float mu = (st.m == -INFINITY) ? 0.f : st.m;
  st.l *= alpha;
  const uint64_t sc2 = f2_pack(sc, sc), nmu2 = f2_pack(-mu, -mu);
  uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint64_t a2 =
          f2_fma(f2_pack(__uint_as_float(sr[c][2 * e]), __uint_as_float(sr[c][2 * e + 1])), sc2, nmu2);
      uint64_t p2 = ex2_x2(a2);
      sum2[e & 1] = f2_add(sum2[e & 1], p2);
      if (VSCALE) p2 = f2_mul(p2, reinterpret_cast<const uint64_t*>(vscale)[c * 16 + e]);
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
