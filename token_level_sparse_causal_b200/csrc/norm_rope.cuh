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
// has the loads of four heads in flight while it works on four others.
//
// A half-warp stays with one token, so its lane's eight sines and cosines and
// the weights sit in registers for all of the token's heads: read from shared
// memory for every row they made the shared-memory pipe the bound (32768 tokens
// of 64/8 heads took 331 us; 1.34 GB are 205 us).  Few tokens: a CTA per token,
// its heads over all half-warps; many: a warp per token.  The angle in turns,
// t * inv_freq / (2 pi), is formed and reduced in 64 bits (at t = 2^20 an fp32
// product would be off by 0.06 rad) once per token; sine and cosine of the
// reduced turn are fp32.  Everything else is fp32 with one rounding at the store.
#pragma once

#include "common.cuh"
#include "quantize.cuh"

namespace hs2 {

constexpr int NR_THREADS = 256;
constexpr int NR_HALFWARPS = NR_THREADS / 16;
constexpr int NR_ROWS = 4;  // rows in flight per half-warp

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

// TOK: tokens per CTA, NR_HALFWARPS / TOK half-warps each.
template <bool KV8, bool PAIRS, int TOK>
__global__ void __launch_bounds__(NR_THREADS) qk_norm_rope_kernel(const NormRopeParams p) {
  constexpr int STEP = NR_HALFWARPS / TOK;  // half-warps of a token
  __shared__ __align__(16) float cos_s[TOK][64], sin_s[TOK][64];
  const int tid = threadIdx.x, l = tid & 15, hw = tid >> 4;
  const int tl = hw / STEP;
  const int t = blockIdx.x * TOK + tl;
  const int H = p.Hq + 2 * p.Hkv;
  const bool norm = p.wq != nullptr;
  const bool here = t < p.n;

  const __nv_bfloat16* qrow = p.q + static_cast<int64_t>(t) * p.q_tok + l * 8;
  const __nv_bfloat16* krow = p.k + static_cast<int64_t>(t) * p.kv_tok + l * 8;
  const __nv_bfloat16* vrow = p.v + static_cast<int64_t>(t) * p.kv_tok + l * 8;
  uint4 raw[NR_ROWS];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i) {
      const int h = h0 + i * STEP;
      const __nv_bfloat16* src = h < p.Hq           ? qrow + h * p.q_head
                                 : h < p.Hq + p.Hkv ? krow + (h - p.Hq) * p.kv_head
                                                    : vrow + (h - p.Hq - p.Hkv) * p.kv_head;
      // not .nc: q_out may be q
      raw[i] = (here && h < H) ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
    }
  };
  const int h_first = hw % STEP;
  load(h_first);  // in flight while the angles are computed

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
  // that are not rotated have cos 1 and sin 0
  const int hl = p.rot >> 4;  // lanes per half
  const bool rotated = l < 2 * hl;
  const int partner = (tid & 16) | (!rotated ? l : (l < hl ? l + hl : l - hl));
  constexpr int NF = PAIRS ? 4 : 8;
  float cs[NF], sn[NF];
#pragma unroll
  for (int e = 0; e < NF; ++e) {
    const int f = (PAIRS ? 4 * l : 8 * (l < hl ? l : l - hl)) + e;
    cs[e] = rotated ? cos_s[tl][f] : 1.f;
    sn[e] = rotated ? sin_s[tl][f] : 0.f;
    if (!PAIRS && l < hl) sn[e] = -sn[e];
  }
  // q's weights, then k's once the heads come to them
  uint64_t w2[4] = {0, 0, 0, 0};
  int w_of = -1;

  // every lane of a warp makes the same number of steps (its two half-warps
  // have different heads, and the shuffles below take the whole warp)
  for (int h0 = h_first; h0 - h_first < H; h0 += NR_ROWS * STEP) {
    uint4 cur[NR_ROWS];
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i) cur[i] = raw[i];
    load(h0 + NR_ROWS * STEP);
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i) {
      const int h = h0 + i * STEP;
      const bool live = here && h < H;
      const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
      uint64_t x2[4];
      bf16x8_to_f32x2(cur[i], x2);
      if (norm) {
        uint64_t s2 = f2_mul(x2[0], x2[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) s2 = f2_fma(x2[e], x2[e], s2);
        float s0, s1;
        f2_unpack(s2, s0, s1);
        float ss = s0 + s1;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!is_v) {
          const int which = is_q ? 0 : 1;
          if (w_of != which) {
            bf16x8_to_f32x2(*reinterpret_cast<const uint4*>((which ? p.wk : p.wq) + l * 8), w2);
            w_of = which;
          }
          const float r = rsqrtf(fmaf(ss, 1.f / 128.f, p.eps));
          const uint64_t r2 = f2_pack(r, r);
#pragma unroll
          for (int e = 0; e < 4; ++e) x2[e] = f2_mul(f2_mul(x2[e], r2), w2[e]);
        }
      }
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) f2_unpack(x2[e], x[2 * e], x[2 * e + 1]);
      if (PAIRS) {
        if (!is_v) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = a * cs[e % NF] - b * sn[e % NF];
            x[2 * e + 1] = b * cs[e % NF] + a * sn[e % NF];
          }
        }
      } else {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner);
        if (!is_v) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = fmaf(y[e], sn[e % NF], x[e] * cs[e % NF]);
        }
      }
      uint4 out = cur[i];  // a value row is copied as it is
      if (!is_v) {
        out.x = pack_bf16x2(x[0], x[1]);
        out.y = pack_bf16x2(x[2], x[3]);
        out.z = pack_bf16x2(x[4], x[5]);
        out.w = pack_bf16x2(x[6], x[7]);
      }
      if (live && is_q)
        *reinterpret_cast<uint4*>(p.q_out + static_cast<int64_t>(t) * p.out_tok + h * p.out_head + l * 8) = out;
      const bool cached = live && !is_q && store;
      const int g = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
      const int64_t at = slot * p.c_tok + g * p.c_head + l * 8;
      if (KV8) {
        if (!__any_sync(0xffffffffu, cached)) continue;
        float a = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(x[e]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        const float scale = a > 0.f ? a / 448.0f : 1.0f;
        if (cached) {
          uint32_t c[4];
          e4m3_codes(x, scale, c);
          *reinterpret_cast<uint2*>((is_v ? p.vc : p.kc) + at) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
          if (l == 0) (is_v ? p.vsc : p.ksc)[slot * p.Hkv + g] = scale;
        }
      } else if (cached) {
        *reinterpret_cast<uint4*>((is_v ? p.vc : p.kc) + at * 2) = out;
      }
    }
  }
}

}  // namespace hs2
