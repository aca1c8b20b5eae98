// A paged key/value cache held in 4 bits: pages and slots from request
// lengths, writing and reading tokens, and attention over the cache.
//
// Format.  A key or value (one token, one KV head, 128 dims) is eight groups
// of 16 dims; a group holds e2m1 codes q (0, .5, 1, 1.5, 2, 3, 4, 6 and their
// negatives) and one e4m3 scale s:  x ~ q s g, g = the cache's k_scale or
// v_scale, a power of two.  s = e4m3(amax / (6 g)) to nearest even (448 at
// most), q = e2m1(x / (s g)) to nearest even (6 at most).  q s has six
// significant bits and lies between 2^-10 and 2688, so it is exact in bf16
// and in fp16, and g only shifts it.  A group holding a NaN or an infinity
// gets the scale NaN and reads back as NaN.
//
// Layout.  A (page, KV head) is page_size / 16 sub-blocks of 16 tokens, 2304
// contiguous bytes each, ordered as the 16-row matrix instruction wants its
// operands, so attention moves a sub-block with plain 16-byte copies and each
// lane reads its fragment of the codes with two 16-byte loads:
//   [0, 1024)     key codes: token 8h + r, chunk j: at 512 h + 64 r + 16 j,
//                 byte 2s + e: dims 16s + 8e + 2j (low half), + 1 (high half)
//   [1024, 2048)  value codes: token 8h + 2j + i: at 512 h + 64 r + 16 j + 8 i,
//                 byte s: dims 16s + r (low half), 16s + 8 + r (high half)
//   [2048, 2176)  key scales: token t, group s: at 8 t + s
//   [2176, 2304)  value scales: token 2a + i, group s: at 16 a + 2 s + i
// No byte is shared by two tokens: tokens are written without reading.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace rbs {

constexpr int kSubTokens = 16;
constexpr int kSubBytes = 2304;

// ---------------------------------------------------------------------------
// pages and slots

struct ExtendArgs {
  int32_t* table;  // [B, max_pages], rows table_b apart
  int64_t table_b;
  int B, max_pages, page, max_new;
  const int32_t *old_lens, *new_lens, *free_pages, *free_head;
  int64_t num_free;
  int32_t *slots, *pos, *head_out;
};

constexpr int kExtThreads = 256;

// Sum of v over the threads before this one; total receives the block's sum.
__device__ __forceinline__ int64_t block_exclusive_scan(int64_t v, int64_t* warp_sums, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // the previous use of warp_sums is over
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int64_t before = 0;
  total = 0;
  for (int i = 0; i < warps; ++i) {
    if (i < warp) before += warp_sums[i];
    total += warp_sums[i];
  }
  return before + x - v;
}

// Pages of request b before and after the call, with the lengths made safe:
// a request never shrinks and never passes its row of the table.
__device__ __forceinline__ void extend_pages(const ExtendArgs& a, int b, int& old_len, int& new_len, int& had, int& has,
                                             bool& bad) {
  const int64_t most = static_cast<int64_t>(a.max_pages) * a.page;
  const int o = a.old_lens[b], n = a.new_lens[b];
  old_len = static_cast<int>(min(static_cast<int64_t>(max(o, 0)), most));
  new_len = static_cast<int>(min(static_cast<int64_t>(max(n, old_len)), most));
  bad = o != old_len || n != new_len || new_len - old_len > a.max_new;
  had = (old_len + a.page - 1) / a.page;
  has = (new_len + a.page - 1) / a.page;
}

// Bound by the launch: 64 requests and one token each 3.0 us, 4,096 tokens each
// 4.5 us.
// CTAs split requests' output rows (blockIdx.y: slices of one request's slots
// and pages).  Each sums the page counts of the requests before its own from
// the lengths; the entries a CTA writes to the table are never read by another
// one (new tokens of an old page take its entry from before the call, those of
// a new page the free list), so one launch does it all.
__global__ void __launch_bounds__(kExtThreads) kv4_extend_kernel(const __grid_constant__ ExtendArgs a, int per_cta) {
  __shared__ int64_t sums[kExtThreads / 32];
  __shared__ int64_t first[kExtThreads];
  const int b0 = blockIdx.x * per_cta, b1 = min(b0 + per_cta, a.B);
  const bool last = blockIdx.x == gridDim.x - 1 && blockIdx.y == 0;
  int64_t carry = 0;
  const int need_to = last ? a.B : b1;
  for (int base = 0; base < need_to; base += kExtThreads) {
    const int b = base + threadIdx.x;
    int64_t v = 0;
    if (b < a.B) {
      int o, n, had, has;
      bool bad;
      extend_pages(a, b, o, n, had, has, bad);
      v = has - had;
      if (bad && last) raise_error(RBS_DEVERR_LENGTH);
    }
    int64_t total;
    const int64_t before = block_exclusive_scan(v, sums, total);
    if (b >= b0 && b < b1) first[b - b0] = carry + before;
    carry += total;
  }
  const int64_t head = *a.free_head;
  if (last && threadIdx.x == 0) {
    const int64_t end = head + carry;
    if (head < 0 || end > a.num_free) raise_error(RBS_DEVERR_PAGES);
    *a.head_out = static_cast<int32_t>(min(max(end, static_cast<int64_t>(0)), a.num_free));
  }
  __syncthreads();
  auto free_page = [&](int64_t i) -> int32_t { return i >= 0 && i < a.num_free ? __ldg(a.free_pages + i) : -1; };
  // (request, entry) pairs of this CTA, entries in slices over blockIdx.y
  const int stride = gridDim.y * kExtThreads;
  for (int b = b0; b < b1; ++b) {
    int old_len, new_len, had, has;
    bool bad;
    extend_pages(a, b, old_len, new_len, had, has, bad);
    const int64_t f = head + first[b - b0];
    int32_t* row = a.table + b * a.table_b;
    for (int e = had + blockIdx.y * kExtThreads + threadIdx.x; e < has; e += stride) row[e] = free_page(f + e - had);
    // (64 bits: a step past a max_new near 2^31 would come out negative, and write there)
    for (int64_t i = blockIdx.y * kExtThreads + threadIdx.x; i < a.max_new; i += stride) {
      int32_t slot = -1, pos = -1;
      if (i < new_len - old_len) {
        const int p = old_len + static_cast<int>(i), e = p / a.page;
        const int32_t pg = e < had ? row[e] : free_page(f + e - had);
        pos = p;
        // (an entry that is no page of any cache gives no slot)
        if (pg >= 0 && pg <= (INT32_MAX - a.page) / a.page) slot = pg * a.page + (p - e * a.page);
      }
      a.slots[static_cast<int64_t>(b) * a.max_new + i] = slot;
      a.pos[static_cast<int64_t>(b) * a.max_new + i] = pos;
    }
  }
}

// ---------------------------------------------------------------------------
// writing and reading tokens

struct Kv4IoArgs {
  uint8_t* data;
  int64_t num_slots;
  int Hkv, page;
  const int32_t* slots;  // [B, L]
  __nv_bfloat16 *k, *v;  // inputs of the writer, outputs of the reader
  int64_t kb, ks, kh, vb, vs, vh;
  int L;
  int64_t rows;  // B * L * Hkv
  float kg, vg, kg_inv, vg_inv;  // the cache's powers of two and their inverses
};

constexpr int kIoThreads = 256;

// Where a token's bytes lie: the sub-block of its (page, head) and the token in it.
__device__ __forceinline__ uint8_t* kv4_sub(uint8_t* data, int Hkv, int page, int32_t slot, int h, int& t) {
  const int pg = slot / page, off = slot - pg * page;
  t = off & 15;
  return data + ((static_cast<int64_t>(pg) * Hkv + h) * (page >> 4) + (off >> 4)) * kSubBytes;
}

// e2m1 codes of two values, the first in the low half.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 d;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %2, %1;\n\tcvt.u32.u8 %0, d;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
// Two e2m1 codes (the low byte of w) as f16x2.
__device__ __forceinline__ uint32_t e2m1x2_f16(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b8 d;\n\tcvt.u8.u32 d, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_bits(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
__device__ __forceinline__ float e4m3_value(uint32_t bits) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(bits)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(r & 0xffffu)));
}

// 16 bf16 values -> their scale bits; q: their codes, pairs (i, i + 1) for
// keys or (i, i + 8) for values, one byte each.
template <bool KEY>
__device__ __forceinline__ uint32_t quantise16(const uint4& x0, const uint4& x1, float g_inv, uint32_t (&q)[8]) {
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  // the largest size by its bits, two values at a time: infinities and NaN are
  // above every finite one
  uint32_t top = w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
  top = max(top & 0xffffu, top >> 16);
  const bool finite = top < 0x7f80u;
  // g is a power of two: an exact shift (a result below fp32's normal range is
  // below any code)
  const float amax = __uint_as_float(top << 16) * g_inv;
  // amax / 6 on a border between two scales is exact (the border has 5
  // significant bits and amax 8), so ties go to the even scale
  const uint32_t s8 = finite ? e4m3_bits(__fdiv_rn(amax, 6.f)) : 0x7fu;
  const float s = e4m3_value(s8);
  const bool zero = !finite || s8 == 0;
  // x / s as x times 1 / s, off by at most 2^-22 relative, then brought to
  // multiples of 2^-11: x has 8 significant bits and a border between two codes
  // (1, 3, 5, 7 quarters or halves, 5) times s at most 7, so a quotient that is
  // not on a border is 2^-8 of it, 2^-10 at least, away from it and stays on
  // its side, and one that is on a border becomes it: ties go to the even code
  // (a value above s's range is infinite here at most, and 6 below)
  const float inv = zero ? 0.f : __frcp_rn(s);
  const float2 g2 = make_float2(g_inv, g_inv), inv2 = make_float2(inv, inv);
  const float2 up = make_float2(0x1p12f, 0x1p12f), down = make_float2(-0x1p12f, -0x1p12f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = i >> 1;  // values: words j and 4 + j, halves i % 2
    float2 y = KEY ? make_float2(bf16lo(w[i]), bf16hi(w[i]))
                   : make_float2(i & 1 ? bf16hi(w[j]) : bf16lo(w[j]), i & 1 ? bf16hi(w[4 + j]) : bf16lo(w[4 + j]));
    const uint32_t sign = (__float_as_uint(y.x) >> 28 & 8u) | (__float_as_uint(y.y) >> 24 & 0x80u);
    y = fadd2(fadd2(fmul2(fmul2(y, g2), inv2), up), down);
    // (the sum loses the sign of what becomes zero)
    q[i] = zero ? 0u : e2m1x2(y.x, y.y) | sign;
  }
  return s8;
}

// Eight neighbouring lanes with eight bytes each, lo and hi: lane i's byte k
// becomes lane k's byte i, by one exchange for each of the lane's three bits.
__device__ __forceinline__ void transpose8(uint32_t& lo, uint32_t& hi, int lane, uint32_t group) {
  const bool b2 = lane & 4, b1 = lane & 2, b0 = lane & 1;
  uint32_t got = __shfl_xor_sync(group, b2 ? lo : hi, 4);
  if (b2) lo = got; else hi = got;
  // pairs of bytes: the lane whose bit is clear keeps bytes 0, 1 of both words
  uint32_t mine = __byte_perm(lo, hi, b1 ? 0x7632 : 0x5410);
  got = __shfl_xor_sync(group, __byte_perm(lo, hi, b1 ? 0x5410 : 0x7632), 2);
  lo = __byte_perm(b1 ? got : mine, b1 ? mine : got, 0x5410);
  hi = __byte_perm(b1 ? got : mine, b1 ? mine : got, 0x7632);
  // single bytes: bytes 0 and 2 of both
  mine = __byte_perm(lo, hi, b0 ? 0x7531 : 0x6420);
  got = __shfl_xor_sync(group, __byte_perm(lo, hi, b0 ? 0x6420 : 0x7531), 1);
  lo = __byte_perm(b0 ? got : mine, b0 ? mine : got, 0x5140);
  hi = __byte_perm(b0 ? got : mine, b0 ? mine : got, 0x7362);
}

// One thread per (token, head, group of dims), eight neighbours to a token's
// row, which move their bytes to the layout's order among themselves: a thread
// writes (reads) eight bytes of the row's key codes and eight of its value
// codes.  512 + 144 bytes per row have to move; measured: 16,384 tokens of 4 KV
// heads written and read back in 23.3 us (13.3 at a copy's rate), the writer with
// 69% of the issue slots taken; 64 tokens in 5.9 us, two launches.
__global__ void __launch_bounds__(kIoThreads) kv4_append_kernel(const __grid_constant__ Kv4IoArgs a) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kIoThreads / 8) + (threadIdx.x >> 3);
  const int s = threadIdx.x & 7;
  if (row >= a.rows) return;
  const int64_t tok = row / a.Hkv;
  const int h = static_cast<int>(row - tok * a.Hkv);
  const int32_t slot = __ldg(a.slots + tok);
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    raise_error(RBS_DEVERR_SLOT);
    return;
  }
  const int64_t b = tok / a.L, l = tok - b * a.L;
  const uint4* kp = reinterpret_cast<const uint4*>(a.k + b * a.kb + l * a.ks + h * a.kh) + 2 * s;
  const uint4* vp = reinterpret_cast<const uint4*>(a.v + b * a.vb + l * a.vs + h * a.vh) + 2 * s;
  const uint4 k0 = ldg_stream(kp), k1 = ldg_stream(kp + 1), v0 = ldg_stream(vp), v1 = ldg_stream(vp + 1);
  int t;
  uint8_t* sub = kv4_sub(a.data, a.Hkv, a.page, slot, h, t);
  const int hh = t >> 3, r = t & 7, j = r >> 1, i = r & 1;
  const uint32_t group = 0xffu << (threadIdx.x & 24);
  auto word = [](const uint32_t* q) { return q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24; };
  uint32_t q[8];
  sub[2048 + 8 * t + s] = static_cast<uint8_t>(quantise16<true>(k0, k1, a.kg_inv, q));
  {
    // byte 2 j + e from every group: lane 2 j + e then has byte e of chunk j of all of them
    const uint32_t m[8] = {q[0], q[4], q[1], q[5], q[2], q[6], q[3], q[7]};
    uint32_t lo = word(m), hi = word(m + 4);
    transpose8(lo, hi, s, group);
    // bytes of e = 0 and e = 1 alternate: the even lane takes groups 0 .. 3, the odd one 4 .. 7
    const uint32_t got = __shfl_xor_sync(group, s & 1 ? lo : hi, 1);
    const uint32_t x = s & 1 ? got : lo, y = s & 1 ? hi : got;
    *reinterpret_cast<uint2*>(sub + 512 * hh + 64 * r + 8 * s) = make_uint2(__byte_perm(x, y, 0x5140), __byte_perm(x, y, 0x7362));
  }
  sub[2176 + 16 * (t >> 1) + 2 * s + i] = static_cast<uint8_t>(quantise16<false>(v0, v1, a.vg_inv, q));
  {
    uint32_t lo = word(q), hi = word(q + 4);
    transpose8(lo, hi, s, group);  // lane r: dims r and r + 8 of every group
    *reinterpret_cast<uint2*>(sub + 1024 + 512 * hh + 64 * s + 16 * j + 8 * i) = make_uint2(lo, hi);
  }
}

__global__ void __launch_bounds__(kIoThreads) kv4_load_kernel(const __grid_constant__ Kv4IoArgs a) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kIoThreads / 8) + (threadIdx.x >> 3);
  const int s = threadIdx.x & 7;
  if (row >= a.rows) return;
  const int64_t tok = row / a.Hkv;
  const int h = static_cast<int>(row - tok * a.Hkv);
  const int32_t slot = __ldg(a.slots + tok);
  const int64_t b = tok / a.L, l = tok - b * a.L;
  uint4* kp = reinterpret_cast<uint4*>(a.k + b * a.kb + l * a.ks + h * a.kh) + 2 * s;
  uint4* vp = reinterpret_cast<uint4*>(a.v + b * a.vb + l * a.vs + h * a.vh) + 2 * s;
  uint32_t ko[8] = {}, vo[8] = {};
  if (slot >= a.num_slots) raise_error(RBS_DEVERR_SLOT);
  if (slot >= 0 && slot < a.num_slots) {
    int t;
    const uint8_t* sub = kv4_sub(a.data, a.Hkv, a.page, slot, h, t);
    const int hh = t >> 3, r = t & 7, j = r >> 1, i = r & 1;
    const float ks = e4m3_value(sub[2048 + 8 * t + s]) * a.kg, vs = e4m3_value(sub[2176 + 16 * (t >> 1) + 2 * s + i]) * a.vg;
    const uint32_t group = 0xffu << (threadIdx.x & 24);
    {
      const uint2 w = *reinterpret_cast<const uint2*>(sub + 512 * hh + 64 * r + 8 * s);
      const uint32_t x = __byte_perm(w.x, w.y, 0x6420), y = __byte_perm(w.x, w.y, 0x7531);
      const uint32_t got = __shfl_xor_sync(group, s & 1 ? x : y, 1);
      uint32_t lo = s & 1 ? got : x, hi = s & 1 ? y : got;
      transpose8(lo, hi, s, group);  // byte 2 j + e of this group
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t f = e2m1x2_f16(((k < 4 ? lo : hi) >> (8 * (k & 3))) & 0xffu);
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
        ko[4 * (k & 1) + (k >> 1)] = pack_bf16x2(v.x * ks, v.y * ks);
      }
    }
    float lo[8], hi[8];
    {
      const uint2 w = *reinterpret_cast<const uint2*>(sub + 1024 + 512 * hh + 64 * s + 16 * j + 8 * i);
      uint32_t x = w.x, y = w.y;
      transpose8(x, y, s, group);  // byte r of this group
#pragma unroll
      for (int rr = 0; rr < 8; ++rr) {
        const uint32_t f = e2m1x2_f16(((rr < 4 ? x : y) >> (8 * (rr & 3))) & 0xffu);
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
        lo[rr] = v.x * vs;
        hi[rr] = v.y * vs;
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      vo[q] = pack_bf16x2(lo[2 * q], lo[2 * q + 1]);
      vo[4 + q] = pack_bf16x2(hi[2 * q], hi[2 * q + 1]);
    }
  }
  kp[0] = make_uint4(ko[0], ko[1], ko[2], ko[3]);
  kp[1] = make_uint4(ko[4], ko[5], ko[6], ko[7]);
  vp[0] = make_uint4(vo[0], vo[1], vo[2], vo[3]);
  vp[1] = make_uint4(vo[4], vo[5], vo[6], vo[7]);
}

}  // namespace rbs
