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
// and goes to the approximate sine and cosine, whose absolute error on
// [-pi, pi] is below 2^-20.5: with the angle's own rounding an output is off by
// less than 2^-19 of its pair's size before its rounding to bf16 (2^-8).
// f_m = f_base r^step with eight bases and eight powers, so a thread forms its
// eight frequencies with eight products.
//
// Eight threads share a head row: thread c holds the 16-byte chunks c and
// c + 8, which are both halves of its rotate-half pairs and whole interleaved
// pairs alike, so neither style moves data between threads; three shuffles
// give the row's sum of squares.  A unit is one token and up to `per` heads of
// its queries or of its keys.  With lo, hi the members of a pair, per unit
//   A = w_lo cos, B = w_hi sin, C = w_lo sin, D = w_hi cos
// and per row r = 1 / sqrt(mean + eps) the outputs are r (A lo - B hi) and
// r (C lo + D hi), two pairs at a time in packed fp32; the loads of four heads
// are issued together.
// Bound by memory: 512 bytes per head row (16,384 tokens of 32 + 4 heads: 53 us,
// 5.7 TB/s of the 6.46 a copy reaches, with 44 and 52 bytes of spilled registers
// in the two styles; 64 tokens: 3.1 us, the launch).
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
__global__ void __launch_bounds__(kQkThreads, 5) qk_norm_rope_kernel(const __grid_constant__ QkNormArgs a) {
  const int c = threadIdx.x & 7;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * (kQkThreads / 8) + (threadIdx.x >> 3);
  if (u >= a.units) return;  // the eight threads of a unit stay together
  const uint32_t group = 0xffu << (threadIdx.x & 24);
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
  uint4 w[2] = {make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u),
                make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u)};  // ones
  const uint4* wp = is_q ? a.wq : a.wk;
  if (wp != nullptr) {
    w[0] = __ldg(wp + c);
    w[1] = __ldg(wp + c + 8);
  }
  // pairs of a thread: lo[i], hi[i], i = 0 .. 7, two to a float2.  Rotate-half:
  // (8c + i, 64 + 8c + i); interleaved: the halves of its eight words.
  auto unpack = [](const uint4& x0, const uint4& x1, float2 (&lo)[4], float2 (&hi)[4]) {
    const uint32_t q0[4] = {x0.x, x0.y, x0.z, x0.w}, q1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (STYLE == 0) {
        lo[i] = make_float2(bf16lo(q0[i]), bf16hi(q0[i]));
        hi[i] = make_float2(bf16lo(q1[i]), bf16hi(q1[i]));
      } else {
        const uint32_t e0 = i < 2 ? q0[2 * i] : q1[2 * i - 4], e1 = i < 2 ? q0[2 * i + 1] : q1[2 * i - 3];
        lo[i] = make_float2(bf16lo(e0), bf16lo(e1));
        hi[i] = make_float2(bf16hi(e0), bf16hi(e1));
      }
    }
  };
  float2 A[4], B[4], C[4], D[4];  // B negated
  {
    double f = a.base[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) f = c == i ? a.base[i] : f;
    f *= static_cast<double>(p);
    float2 wl[4], wh[4];
    unpack(w[0], w[1], wl, wh);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float sn[2], cs[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const double turns = f * a.step[2 * i + k];
        __sincosf(6.283185307179586f * static_cast<float>(turns - rint(turns)), &sn[k], &cs[k]);
      }
      const float2 s2 = make_float2(sn[0], sn[1]), c2 = make_float2(cs[0], cs[1]);
      A[i] = fmul2(wl[i], c2);
      B[i] = fmul2(wh[i], make_float2(-s2.x, -s2.y));
      C[i] = fmul2(wl[i], s2);
      D[i] = fmul2(wh[i], c2);
    }
  }
  for (int h = h0; h < h1; h += kQkHeads) {
    if (h > h0) load(h);
#pragma unroll
    for (int v = 0; v < kQkHeads; ++v) {
      float2 lo[4], hi[4], sq = make_float2(0.f, 0.f);
      unpack(x[v][0], x[v][1], lo, hi);
#pragma unroll
      for (int i = 0; i < 4; ++i) sq = ffma2(hi[i], hi[i], ffma2(lo[i], lo[i], sq));
      float ss = sq.x + sq.y;
      ss += __shfl_xor_sync(group, ss, 1);
      ss += __shfl_xor_sync(group, ss, 2);
      ss += __shfl_xor_sync(group, ss, 4);
      const float r = rsqrtf(fmaf(ss, 1.f / 128.f, a.eps));
      const float2 r2 = make_float2(r, r);
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = fmul2(ffma2(lo[i], A[i], fmul2(hi[i], B[i])), r2);
        const float2 z = fmul2(ffma2(lo[i], C[i], fmul2(hi[i], D[i])), r2);
        if (STYLE == 0) {
          o[i] = pack_bf16x2(y.x, y.y);
          o[4 + i] = pack_bf16x2(z.x, z.y);
        } else {
          o[2 * i] = pack_bf16x2(y.x, z.x);
          o[2 * i + 1] = pack_bf16x2(y.y, z.y);
        }
      }
      if (h + v < h1) {
        uint4* d = reinterpret_cast<uint4*>(dst + (h + v) * dh);
        d[c] = make_uint4(o[0], o[1], o[2], o[3]);
        d[c + 8] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

}  // namespace rbs
