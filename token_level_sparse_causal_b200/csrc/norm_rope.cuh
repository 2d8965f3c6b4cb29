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
// has the loads of four rows in flight before it works on the first.  The
// rot / 2 angles of a token are shared by all its heads: a CTA takes all heads
// of a few tokens and computes each angle once, into shared memory.  The angle
// in turns, t * inv_freq / (2 pi), is formed and reduced in 64 bits (at
// t = 2^20 an fp32 product would be off by 0.06 rad); sine and cosine of the
// reduced turn are fp32.  Everything else is fp32 with one rounding at the
// store.
#pragma once

#include "common.cuh"
#include "quantize.cuh"

namespace hs2 {

constexpr int NR_THREADS = 256;
constexpr int NR_MAX_TOK = 4;  // tokens per CTA
constexpr int NR_ROWS = 4;     // rows in flight per half-warp

struct NormRopeParams {
  int n, Hq, Hkv, rot, tok_per_cta;
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

template <bool KV8, bool PAIRS>
__global__ void __launch_bounds__(NR_THREADS) qk_norm_rope_kernel(const NormRopeParams p) {
  __shared__ __align__(16) float cos_s[NR_MAX_TOK][64], sin_s[NR_MAX_TOK][64];
  __shared__ __align__(16) float w_s[2][128];
  const int tid = threadIdx.x, l = tid & 15, hw = tid >> 4;
  const int t0 = blockIdx.x * p.tok_per_cta;
  const int nt = min(p.tok_per_cta, p.n - t0);
  const int H = p.Hq + 2 * p.Hkv;
  const int units = nt * H;
  const bool norm = p.wq != nullptr;

  uint4 raw[NR_ROWS];
  auto load = [&](int u0) {
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i) {
      const int u = u0 + i * (NR_THREADS / 16);
      raw[i] = make_uint4(0, 0, 0, 0);
      if (u < units) {
        const int t = t0 + u / H, h = u % H;
        const __nv_bfloat16* src;
        if (h < p.Hq)
          src = p.q + static_cast<int64_t>(t) * p.q_tok + static_cast<int64_t>(h) * p.q_head;
        else if (h < p.Hq + p.Hkv)
          src = p.k + static_cast<int64_t>(t) * p.kv_tok + static_cast<int64_t>(h - p.Hq) * p.kv_head;
        else
          src = p.v + static_cast<int64_t>(t) * p.kv_tok + static_cast<int64_t>(h - p.Hq - p.Hkv) * p.kv_head;
        raw[i] = *reinterpret_cast<const uint4*>(src + l * 8);  // not .nc: q_out may be q
      }
    }
  };
  load(hw);  // in flight while the angles are computed

  const int half = p.rot >> 1;
  for (int i = tid; i < nt * half; i += NR_THREADS) {
    const int t = i / half, f = i % half;
    double turn = static_cast<double>(p.pos[t0 + t]) * (p.inv_freq[f] * 0.15915494309189533577);  // 1 / (2 pi)
    turn -= rint(turn);
    sincospif(2.0f * static_cast<float>(turn), &sin_s[t][f], &cos_s[t][f]);
  }
  if (norm && tid < 128) {
    w_s[0][tid] = __bfloat162float(p.wq[tid]);
    w_s[1][tid] = __bfloat162float(p.wk[tid]);
  }
  __syncthreads();

  // half-split pairs: this lane's partner dimension and its angles
  const int hl = p.rot >> 4;  // lanes per half
  const bool rotated = l < 2 * hl;
  const int partner = (tid & 16) | (!rotated ? l : (l < hl ? l + hl : l - hl));
  const int f0 = PAIRS ? (rotated ? 4 * l : 0) : (rotated ? 8 * (l < hl ? l : l - hl) : 0);
  const float sgn = l < hl ? -1.f : 1.f;

  for (int u0 = hw; u0 < units; u0 += NR_ROWS * (NR_THREADS / 16)) {
    uint4 cur[NR_ROWS];
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i) cur[i] = raw[i];
    load(u0 + NR_ROWS * (NR_THREADS / 16));
#pragma unroll
    for (int i = 0; i < NR_ROWS; ++i) {
      // the rows of a warp's two halves differ, so every shuffle names its half
      const int u = u0 + i * (NR_THREADS / 16);
      const bool live = u < units;
      const int tl = live ? u / H : 0, h = live ? u % H : 0;
      const int t = t0 + tl;
      const bool is_v = h >= p.Hq + p.Hkv, is_k = h >= p.Hq && !is_v;
      const uint32_t w4[4] = {cur[i].x, cur[i].y, cur[i].z, cur[i].w};
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w4[e] << 16);
        x[2 * e + 1] = __uint_as_float(w4[e] & 0xFFFF0000u);
      }
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!is_v) {
          const float r = rsqrtf(fmaf(ss, 1.f / 128.f, p.eps));
          const float* w = w_s[is_k ? 1 : 0] + l * 8;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
        }
      }
      if (PAIRS) {
        if (!is_v && rotated) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float c = cos_s[tl][f0 + e], s = sin_s[tl][f0 + e];
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = a * c - b * s;
            x[2 * e + 1] = b * c + a * s;
          }
        }
      } else {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner);
        if (!is_v && rotated) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * cos_s[tl][f0 + e] + sgn * y[e] * sin_s[tl][f0 + e];
        }
      }
      if (live && !is_v && !is_k) {
        uint4 out;
        out.x = pack_bf16x2(x[0], x[1]);
        out.y = pack_bf16x2(x[2], x[3]);
        out.z = pack_bf16x2(x[4], x[5]);
        out.w = pack_bf16x2(x[6], x[7]);
        *reinterpret_cast<uint4*>(p.q_out + static_cast<int64_t>(t) * p.out_tok +
                                  static_cast<int64_t>(h) * p.out_head + l * 8) = out;
      }
      const bool cache_row = live && (is_v || is_k);
      if (KV8 ? __any_sync(0xffffffffu, cache_row) : cache_row) {
        int64_t slot = t;
        if (cache_row && p.slots) slot = p.slots[t];
        bool store = cache_row;
        if (cache_row && (slot < 0 || slot >= p.n_slots)) {
          if (slot != -1 && l == 0) report(HS2_ERR_INDEX, 501);
          store = false;
        }
        const int g = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
        uint8_t* base = is_v ? p.vc : p.kc;
        const int64_t at = slot * p.c_tok + static_cast<int64_t>(g) * p.c_head + l * 8;
        if (KV8) {
          float a = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(x[e]));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
          const float scale = a > 0.f ? a / 448.0f : 1.0f;
          if (store) {
            uint32_t c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = e4m3x2_from_f32(x[2 * e] / scale, x[2 * e + 1] / scale);
            *reinterpret_cast<uint2*>(base + at) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
            if (l == 0) (is_v ? p.vsc : p.ksc)[slot * p.Hkv + g] = scale;
          }
        } else if (store) {
          uint4 out = cur[i];  // a value row is copied as it is
          if (is_k) {
            out.x = pack_bf16x2(x[0], x[1]);
            out.y = pack_bf16x2(x[2], x[3]);
            out.z = pack_bf16x2(x[4], x[5]);
            out.w = pack_bf16x2(x[6], x[7]);
          }
          *reinterpret_cast<uint4*>(base + at * 2) = out;
        }
      }
    }
  }
}

}  // namespace hs2
