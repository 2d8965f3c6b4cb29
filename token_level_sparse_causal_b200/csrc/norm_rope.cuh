// Norms of queries and keys per head, position rotation and cache write in
// one pass over a projection's rows (the step before attention):
//
//   y = x * rsqrt(mean(x^2) + eps) * w
//   (y_a, y_b) -> (y_a cos u - y_b sin u, y_b cos u + y_a sin u),  u = t * inv_freq[f]
//
// with the rotated query written to q_out and the rotated key and the value
// written to their cache slots (bf16, or e4m3 codes with scale amax / 448).
//
// Bound by memory: every row is read once (256 B) and written once (256 B, or
// 128 B + 4 B in an e4m3 cache).  A half-warp holds one row, 8 values (16 B) a
// lane, so the norm and the row's amax are four shuffles and the partner
// dimension of the half-split rotation lies rot / 16 lanes away; each half-warp
// has the loads of four rows in flight while it works on four others.  32768
// tokens of 64/8 heads: 207 us, 6.5 TB/s into a bf16 cache, 6.2 into e4m3.
//
// A half-warp stays with one token, so its lane's eight sines and cosines and
// the weights sit in registers for all of the token's heads: read from shared
// memory for every row they made the shared-memory pipe the bound (32768 tokens
// of 64/8 heads took 331 us).  Few tokens: a CTA per token, its heads over all
// half-warps (512 tokens 8.2 us, a warp per token 12.3); many: a warp per token
// (4096 tokens 36 us, a CTA per token 44).  The angle in turns,
// t * inv_freq / (2 pi), is formed and reduced in 64 bits (at t = 2^20 an fp32
// product would be off by 0.06 rad) once per token; sine and cosine of the
// reduced turn are fp32.  Everything else is fp32 with one rounding at the store.
#pragma once

#include "common.cuh"
#include "quantize.cuh"

namespace hs2 {

constexpr int NR_THREADS = 256;
constexpr int NR_HALFWARPS = NR_THREADS / 16;
// rows in flight per half-warp: few tokens have few rows per half-warp
__host__ __device__ constexpr int nr_rows(int tok) { return tok == 1 ? 2 : 4; }

struct NormRopeParams {
  int n, Hq, Hkv, rot;
  float eps;
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_tok, q_head, kv_tok, kv_head, out_tok, out_head;
  const __nv_bfloat16 *wq, *wk;  // both null: no norm
  const double* inv_freq;
  const int32_t *pos, *slots;
  __nv_bfloat16* q_out;
  uint8_t *kc, *vc;  // cache pools
  float *ksc, *vsc;  // e4m3 only, [slots][Hkv]
  int64_t c_tok, c_head, n_slots;
};

// The eight values of a lane's 16 bytes, as fp32 pairs.
__device__ __forceinline__ void bf16x8_to_f32x2(uint4 v, uint64_t (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = f2_pack(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
}

// TOK: tokens per CTA, NR_HALFWARPS / TOK half-warps each.  A half-warp walks
// its share of the token's query heads, then of the key heads, then of the
// value heads: three loops of their own, so that none carries the others'
// choices (one loop over all heads took 159 instructions a row pair).
template <bool KV8, bool PAIRS, int TOK>
__global__ void __launch_bounds__(NR_THREADS, 3) qk_norm_rope_kernel(const NormRopeParams p) {
  constexpr int STEP = NR_HALFWARPS / TOK;  // half-warps of a token
  constexpr int NR_ROWS = nr_rows(TOK);
  __shared__ __align__(16) float cos_s[TOK][64], sin_s[TOK][64];
  const int tid = threadIdx.x, l = tid & 15, hw = tid >> 4;
  const int tl = hw / STEP;
  const int t = blockIdx.x * TOK + tl;
  const bool here = t < p.n;
  const int h_first = hw % STEP;

  // rows h_first, h_first + STEP, ... of a token: NR_ROWS of them from `row` on
  uint4 raw[NR_ROWS];
  auto load = [&](const __nv_bfloat16* row, int64_t stride, int left) {
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i)  // not .nc: q_out may be q
      raw[i] = i * STEP < left ? *reinterpret_cast<const uint4*>(row + i * stride) : make_uint4(0, 0, 0, 0);
  };
  const int64_t q_step = STEP * p.q_head, kv_step = STEP * p.kv_head;
  const __nv_bfloat16* q_row = p.q + static_cast<int64_t>(t) * p.q_tok + h_first * p.q_head + l * 8;
  const int64_t kv_off = static_cast<int64_t>(t) * p.kv_tok + h_first * p.kv_head + l * 8;
  const int q_left = here ? p.Hq - h_first : 0, kv_left = here ? p.Hkv - h_first : 0;
  load(q_row, q_step, q_left);  // in flight while the angles are computed

  const int half = p.rot >> 1;
  for (int i = tid; i < TOK * 64; i += NR_THREADS) {
    const int tt = blockIdx.x * TOK + (i >> 6), f = i & 63;
    if (tt < p.n && f < half) {
      double turn = static_cast<double>(p.pos[tt]) * (p.inv_freq[f] * 0.15915494309189533577);  // 1 / (2 pi)
      turn -= rint(turn);
      sincospif(2.0f * static_cast<float>(turn), &sin_s[i >> 6][f], &cos_s[i >> 6][f]);
    }
  }
  int64_t slot = t;
  if (here && p.slots) slot = p.slots[t];
  const bool store = here && slot >= 0 && slot < p.n_slots;
  if (here && !store && slot != -1 && l == 0 && h_first == 0) report(HS2_ERR_INDEX, 501);
  __syncthreads();

  // this lane's angles: half-split pairs have their partner hl lanes away and
  // add its value times -sin (first half) or sin (second half); dimensions
  // that are not rotated have cos 1 and sin 0.  Interleaved pairs (a, b) are
  // (a, b) cos + (b, a) (-sin, sin).
  const int hl = p.rot >> 4;  // lanes per half
  const bool rotated = l < 2 * hl;
  const int partner = (tid & 16) | (!rotated ? l : (l < hl ? l + hl : l - hl));
  uint64_t cs2[4], sn2[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int f = PAIRS ? 4 * l + e : 8 * (l < hl ? l : l - hl) + 2 * e;
    const float c0 = rotated ? cos_s[tl][f] : 1.f, s0 = rotated ? sin_s[tl][f] : 0.f;
    if (PAIRS) {
      cs2[e] = f2_pack(c0, c0);
      sn2[e] = f2_pack(-s0, s0);
    } else {
      const float c1 = rotated ? cos_s[tl][f + 1] : 1.f, s1 = rotated ? sin_s[tl][f + 1] : 0.f;
      cs2[e] = f2_pack(c0, c1);
      sn2[e] = l < hl ? f2_pack(-s0, -s1) : f2_pack(s0, s1);
    }
  }
  const bool norm = p.wq != nullptr;
  uint64_t w2[4];
  auto weights = [&](const __nv_bfloat16* w) {
    if (norm) bf16x8_to_f32x2(*reinterpret_cast<const uint4*>(w + l * 8), w2);
  };

  // norm and rotation of one row; every lane of the warp takes part
  auto turn_row = [&](uint4 v, uint64_t (&x2)[4]) {
    bf16x8_to_f32x2(v, x2);
    if (norm) {
      uint64_t s2 = f2_mul(x2[0], x2[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) s2 = f2_fma(x2[e], x2[e], s2);
      float s0, s1;
      f2_unpack(s2, s0, s1);
      float ss = s0 + s1;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(fmaf(ss, 1.f / 128.f, p.eps));
      const uint64_t r2 = f2_pack(r, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) x2[e] = f2_mul(f2_mul(x2[e], r2), w2[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, b;
      f2_unpack(x2[e], a, b);
      const uint64_t y2 = PAIRS ? f2_pack(b, a)
                                : f2_pack(__shfl_sync(0xffffffffu, a, partner), __shfl_sync(0xffffffffu, b, partner));
      x2[e] = f2_fma(y2, sn2[e], f2_mul(x2[e], cs2[e]));
    }
  };
  auto to_bf16 = [&](const uint64_t (&x2)[4]) {
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, b;
      f2_unpack(x2[e], a, b);
      o[e] = pack_bf16x2(a, b);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  };
  // one row of an e4m3 cache
  auto quantize = [&](const uint64_t (&x2)[4], bool live, uint8_t* dst, float* dst_scale) {
    float x[8], a = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f2_unpack(x2[e], x[2 * e], x[2 * e + 1]);
#pragma unroll
    for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(x[e]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const float scale = a > 0.f ? a / 448.0f : 1.0f;
    if (live) {
      uint32_t c[4];
      e4m3_codes(x, scale, c);
      *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      if (l == 0) *dst_scale = scale;
    }
  };

  // every lane of a warp makes the same number of steps (its two half-warps
  // have different heads, and the shuffles take the whole warp)
  constexpr int AT_ONCE = NR_ROWS * STEP;
  weights(p.wq);
  __nv_bfloat16* o_row = p.q_out + static_cast<int64_t>(t) * p.out_tok + h_first * p.out_head + l * 8;
  const int64_t o_step = STEP * p.out_head;
  for (int h0 = 0; h0 < p.Hq; h0 += AT_ONCE) {
    uint4 cur[NR_ROWS];
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i) cur[i] = raw[i];
    q_row += NR_ROWS * q_step;
    if (h0 + AT_ONCE < p.Hq)
      load(q_row, q_step, q_left - h0 - AT_ONCE);
    else
      load(p.k + kv_off, kv_step, kv_left);
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i) {
      uint64_t x2[4];
      turn_row(cur[i], x2);
      if (h0 + i * STEP < q_left) *reinterpret_cast<uint4*>(o_row + i * o_step) = to_bf16(x2);
    }
    o_row += NR_ROWS * o_step;
  }
  weights(p.wk);
  const int64_t at0 = slot * p.c_tok + h_first * p.c_head + l * 8;
  for (int h0 = 0; h0 < p.Hkv; h0 += AT_ONCE) {
    uint4 cur[NR_ROWS];
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i) cur[i] = raw[i];
    if (h0 + AT_ONCE < p.Hkv)
      load(p.k + kv_off + (h0 + AT_ONCE) * p.kv_head, kv_step, kv_left - h0 - AT_ONCE);
    else
      load(p.v + kv_off, kv_step, kv_left);
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i) {
      const int h = h0 + i * STEP;
      const bool live = store && h < kv_left;
      uint64_t x2[4];
      turn_row(cur[i], x2);
      const int64_t at = at0 + h * p.c_head;
      if (KV8)
        quantize(x2, live, p.kc + at, p.ksc + slot * p.Hkv + h_first + h);
      else if (live)
        *reinterpret_cast<uint4*>(p.kc + at * 2) = to_bf16(x2);
    }
  }
  for (int h0 = 0; h0 < p.Hkv; h0 += AT_ONCE) {
    uint4 cur[NR_ROWS];
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i) cur[i] = raw[i];
    if (h0 + AT_ONCE < p.Hkv) load(p.v + kv_off + (h0 + AT_ONCE) * p.kv_head, kv_step, kv_left - h0 - AT_ONCE);
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i) {
      const int h = h0 + i * STEP;
      const bool live = store && h < kv_left;
      const int64_t at = at0 + h * p.c_head;
      if (KV8) {
        uint64_t x2[4];
        bf16x8_to_f32x2(cur[i], x2);
        quantize(x2, live, p.vc + at, p.vsc + slot * p.Hkv + h_first + h);
      } else if (live) {
        *reinterpret_cast<uint4*>(p.vc + at * 2) = cur[i];  // a value row is copied as it is
      }
    }
  }
}

}  // namespace hs2
