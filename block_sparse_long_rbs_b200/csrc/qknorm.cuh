// Per-head norm of queries and keys with the position rotation in the same
// pass: for a head row x of 128 values of the token at position p,
//   y = rot_p(w * x / sqrt(mean(x^2) + eps)),
// w the 128 norm weights of the queries or of the keys (ones when absent) and
// rot_p the rotation of pair m by p theta^(-2m/128) (pairs (m, m + 64) or
// (2m, 2m + 1)).  Everything between the bf16 input and the bf16 output is
// fp32: one rounding per value.
//
// The angle is formed in turns, t = p (f_m / 2 pi), in fp64 and reduced there
// (t - rint(t), exact); only the remainder in [-1/2, 1/2] is rounded to fp32
// (2^-26 turns at most, an angle error below 1e-7 at any position) and goes to
// sincospi.  f_m = f_base r^step with eight bases and eight powers, so a thread
// forms its eight frequencies with eight products.
//
// Eight threads share a head row: thread c holds the 16-byte chunks c and
// c + 8, which are both halves of its rotate-half pairs and whole interleaved
// pairs alike, so neither style moves data between threads; three shuffles
// give the row's sum of squares.  A unit is one token and up to `per` heads of
// its queries or of its keys: the thread's sines, cosines and weights are
// formed once per unit and the loads of four heads are issued together.
// Bound by memory: 512 bytes per head row.
#pragma once

#include "common.cuh"

namespace rbs {

struct QkNormArgs {
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *qo, *ko;
  int64_t qb, qs, qh, kb, ks, kh, qob, qos, qoh, kob, kos, koh;
  const uint4 *wq, *wk;  // 128 bf16 weights each, or null for ones
  const int32_t* pos;
  int64_t pos_b;  // elements between batch entries' positions (0: shared)
  int L, Hq, Hkv;
  int per, nq, nk;  // heads of a unit; units per token of queries and of keys
  int64_t units;    // B * L * (nq + nk)
  float eps;
  double base[8], step[8];  // frequencies in turns per position: base[c] * step[i]
};

constexpr int kQkThreads = 128;
constexpr int kQkHeads = 4;  // head rows whose loads are in flight together

template <int STYLE>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const __grid_constant__ QkNormArgs a) {
  const int c = threadIdx.x & 7;
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * (kQkThreads / 8) + (threadIdx.x >> 3);
  const bool live = u0 < a.units;  // a whole group of eight threads is live or not
  const int64_t u = live ? u0 : a.units - 1;
  const int per_tok = a.nq + a.nk;
  const int64_t tok = u / per_tok;
  int part = static_cast<int>(u - tok * per_tok);
  const int b = static_cast<int>(tok / a.L), t = static_cast<int>(tok - static_cast<int64_t>(b) * a.L);
  const bool is_q = part < a.nq;
  if (!is_q) part -= a.nq;
  const int h0 = part * a.per, h1 = min(h0 + a.per, is_q ? a.Hq : a.Hkv);
  const int64_t sh = is_q ? a.qh : a.kh, dh = is_q ? a.qoh : a.koh;
  const __nv_bfloat16* src = is_q ? a.q + b * a.qb + t * a.qs : a.k + b * a.kb + t * a.ks;
  __nv_bfloat16* dst = is_q ? a.qo + b * a.qob + t * a.qos : a.ko + b * a.kob + t * a.kos;
  uint4 x[kQkHeads][2];
  auto load = [&](int h) {
#pragma unroll
    for (int v = 0; v < kQkHeads; ++v) {
      const uint4* p = reinterpret_cast<const uint4*>(src + min(h + v, h1 - 1) * sh);
      x[v][0] = p[c];
      x[v][1] = p[c + 8];
    }
  };
  load(h0);
  const int32_t p = __ldg(a.pos + b * a.pos_b + t);
  uint4 w[2] = {};
  const uint4* wp = is_q ? a.wq : a.wk;
  if (wp != nullptr) {
    w[0] = __ldg(wp + c);
    w[1] = __ldg(wp + c + 8);
  }
  double f = a.base[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) f = c == i ? a.base[i] : f;
  f *= static_cast<double>(p);
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double turns = f * a.step[i];
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &sn[i], &cs[i]);
  }
  float wf[16];
  {
    const uint32_t ww[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      wf[2 * i] = wp != nullptr ? bf16lo(ww[i]) : 1.f;
      wf[2 * i + 1] = wp != nullptr ? bf16hi(ww[i]) : 1.f;
    }
  }
  // every group runs the same number of head passes as the widest unit, so
  // the shuffles below always have the whole warp
  for (int base = 0; base < a.per; base += kQkHeads) {
    if (base > 0) load(min(h0 + base, h1 - 1));
#pragma unroll
    for (int v = 0; v < kQkHeads; ++v) {
      const uint32_t xw[8] = {x[v][0].x, x[v][0].y, x[v][0].z, x[v][0].w, x[v][1].x, x[v][1].y, x[v][1].z, x[v][1].w};
      float y[16], ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[2 * i] = bf16lo(xw[i]);
        y[2 * i + 1] = bf16hi(xw[i]);
        ss = fmaf(y[2 * i], y[2 * i], ss);
        ss = fmaf(y[2 * i + 1], y[2 * i + 1], ss);
      }
      ss += __shfl_xor_sync(0xffffffffu, ss, 1);
      ss += __shfl_xor_sync(0xffffffffu, ss, 2);
      ss += __shfl_xor_sync(0xffffffffu, ss, 4);
      const float r = rsqrtf(fmaf(ss, 1.f / 128.f, a.eps));
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] *= r * wf[i];
      uint32_t o[8];
      if (STYLE == 0) {  // pairs (8c + i, 64 + 8c + i)
        float lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          lo[i] = fmaf(y[i], cs[i], -y[8 + i] * sn[i]);
          hi[i] = fmaf(y[i], sn[i], y[8 + i] * cs[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[i] = pack_bf16x2(lo[2 * i], lo[2 * i + 1]);
          o[4 + i] = pack_bf16x2(hi[2 * i], hi[2 * i + 1]);
        }
      } else {  // pairs (2m, 2m + 1), m = 4c + i and 32 + 4c + i
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = pack_bf16x2(fmaf(y[2 * i], cs[i], -y[2 * i + 1] * sn[i]), fmaf(y[2 * i], sn[i], y[2 * i + 1] * cs[i]));
      }
      if (live && h0 + base + v < h1) {
        uint4* d = reinterpret_cast<uint4*>(dst + (h0 + base + v) * dh);
        d[c] = make_uint4(o[0], o[1], o[2], o[3]);
        d[c + 8] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

}  // namespace rbs
