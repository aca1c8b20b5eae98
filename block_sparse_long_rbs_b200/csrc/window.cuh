// Sliding-window attention with sinks on the 5th-generation tensor core:
// query p sees the keys s <= p with p - W < s, and the first S keys.
//
// A work item is T = 128 / G tokens of one (batch, KV head): the 128 rows of
// the tile are the (token, q head) pairs of the G q heads that share the KV
// head.  The keys an item needs span T + W - 1 positions, so a narrow window
// wastes little of a tile (128 tokens of one head would span 127 + W), and a
// key tile is read once for all G heads.  Key tiles of 64 start at the item's
// own first visible key (TMA rows may start anywhere).  Up to 16 sinks share a
// tile with the window's first 48 keys; more sinks get tiles of their own.
//
// Two CTAs per SM, each a whole pipeline on half of the SM's tensor and shared
// memory: while one CTA's softmax waits for its products or its epilogue
// stores, the other one has the tensor core and the issue slots.  Within a
// CTA two S buffers let S_{g+1} run under the softmax of tile g.
// Roles (256 threads):
//   warps 0-3  softmax: a thread owns one row (its TMEM lane).  It reads the 64
//              scores, masks them in tiles that some row sees only in part,
//              takes the maximum (the running maximum moves, and O is rescaled,
//              only when it grows by more than 2^8), writes
//              P = exp2(S c - m) as bf16 pairs over the scores (2^-8 relative:
//              V is bf16 and both operands of a product have one type; V's
//              range does not fit fp16), and at the end
//              stages O / l for a TMA store and writes the LSE.
//   warp 4     Q and K producer, warp 5 V producer (TMA, one lane)
//   warp 6     TMEM allocator, issuer of S = Q K^T (both operands in shared memory)
//   warp 7     issuer of O += P V (P in TMEM, V MN-major in shared memory)
//              and of the outputs' stores
// TMEM columns: S buffers [0, 64) and [64, 128), O [128, 256).
//
// No single unit is full: per 64 scores of two rows a scheduler has 1024 cycles
// of exponentials (16 a clock and SM), and the two warps that share it overlap
// them with only part of their other work (1890 cycles per pair of tiles
// measured: exponentials 60% busy, the tensor core 59%, issue 53%); a division
// of the work that overlaps more of it has not been found among those below (the
// products need 1280: 48 cycles per K = 16 step of S at N = 64, where shared
// memory is the limit, and 64 of P V).  16,384 tokens, window 4096, 32 q / 4 KV
// heads: 860 us (980 us when repeated until the power limit lowers the clock).
// Measured and left, against 890 us then: one CTA with two row tiles on shared
// key tiles (1056 us: the two run in step, and their exponentials collide), key
// tiles of 128 in that form (1120 us), a quarter of the exponentials as a
// polynomial (915 us), two warps per row with the maximum agreed between them
// (1005 us).
// A narrow window is bound by what an item costs beside its tiles: 65,536
// tokens, window 128, 16,384 items of three tiles: 365 to 385 us (443 while the
// 128 registers a thread may have did not suffice and 28 bytes were spilled; the
// outputs' way to memory was 120 us of that).  Measured and left there: no
// exponentials for 32 columns that no row of a warp sees (5% slower: spills),
// stores of each softmax warp's own rows, 32 dims at a time, without warp 7
// (1% slower on both windows).
//
// Masked scores are replaced before the softmax, so NaN keys stay out.  A masked
// value still meets its zero weight in the product, and zero times a NaN or an
// infinity is NaN.  The keys that some row of an item does not see are few: the
// window's edges (fewer than T keys each) and what the last step of 16 keys holds
// past the last token (the copies fill what lies past the sinks with zeros).  Warp 7
// looks through those before their product and sets what is not finite there to
// zero; where it found some, each row adds those that it does see (whatever
// their weights, they make the sum non-finite) to its outputs at the end.  The
// look is hidden behind the softmax (380 us for the narrow window with it, 385
// before); an item that has to give values back pays for T alone, however long
// the prompt is: with such values in every key the narrow window takes 1.4 ms
// (0.33 without, both in single calls) and the wide one 1.07 (0.86).
// Every mbarrier wait is bounded, as in attention.cuh.
#pragma once

#include "common.cuh"

namespace rbs {

struct WinArgs {
  // Q boxes of T tokens x G heads, O's the same (ordered by stride), K / V boxes of 64, 16 and 48 keys
  // tmVs, tmVt (64 keys): values that end with the sinks, zeros past them
  CUtensorMap tmQ, tmO, tmK, tmV, tmKs, tmVs, tmKw, tmVw, tmVt;
  const __nv_bfloat16* V;
  __nv_bfloat16* O;
  int64_t vb, vs, vh, ob, os, oh;
  int o_seq_inner;  // O's token stride is the smaller one: its box is T tokens inside G heads
  float* lse;  // [B, Hq, Lq] or null
  int B, G, Hkv, Lq, Lk, T, nt;  // T tokens per item, nt items per (batch, KV head)
  int64_t q_off;
  int W, S;
  int items;
  float inv_nt, inv_hkv;
  float scale_log2;
  uint64_t wait_ns;
  int stall_after;  // testing only: the K producer stops after this many tiles (< 0: never)
};

constexpr int kWinThreads = 256;
constexpr int kWinKeys = 64;    // keys of a tile
constexpr int kWinSinkRows = 16;  // rows that sinks take in a shared first tile
constexpr int kWinNS = 2;       // K and V ring depth

struct WinSmem {
  static constexpr int kQBytes = 128 * 256;
  static constexpr int kKVBytes = kWinKeys * 256;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kQBytes;
  static constexpr int kV = kK + kWinNS * kKVBytes;
  static constexpr int kO = kV + kWinNS * kKVBytes;  // 64 dims of the outputs, on their way to the store
  static constexpr int kBar = kO + 128 * 128;
  // no slack for alignment: the block's dynamic shared memory starts at a
  // multiple of 1024 (checked)
  static constexpr int kAlloc = kBar + 256;
  static constexpr uint32_t kTmemCols = 256;
  __host__ __device__ static constexpr uint32_t col_s(int buf) { return buf * kWinKeys; }
  static constexpr uint32_t kColO = 128;
};
static_assert(2 * (WinSmem::kAlloc + 1024) <= 228 * 1024, "two CTAs per SM");

enum : int {
  kWbQFull = 0,
  kWbQEmpty = 1,
  kWbKFull = 2,                // + stage
  kWbVFull = kWbKFull + kWinNS,
  kWbSFull = kWbVFull + kWinNS,  // + S buffer
  kWbPFull = kWbSFull + 2,       // + S buffer
  kWbPVDone = kWbPFull + 2,      // + tile mod 4
  kWbOFull = kWbPVDone + 4,
  kWbOEmpty = kWbOFull + 1,
  kWbStoreFull = kWbOEmpty + 1,  // 64 dims of the outputs are staged
  kWbStoreEmpty = kWbStoreFull + 1,
  kWbDrain = kWbStoreEmpty + 1,  // + issuer
  kWbNum = kWbDrain + 2
};
static_assert(kWbNum * 8 + 16 <= 256, "barrier area");

// One item's key tiles.  Positions fit 32 bits (q_off + Lq < 2^31, checked by
// the host).
struct WinItem {
  int b, kvh, t0;      // batch, KV head, first token
  int p0, p1;          // positions of the first and last token
  int lo;              // first key of the window part
  int sinks;           // sinks before the window part
  int n_sink;          // tiles of sinks alone
  bool merged;         // the first tile holds the sinks and 48 window keys
  int n;               // tiles
};

// n / d by the reciprocal and a correction; the quotient is off by one at most
// while it stays below 2^22, and the loops mend any other.
__device__ __forceinline__ int win_div(int n, int d, float inv, int& rem) {
  int q = static_cast<int>(static_cast<float>(n) * inv);
  rem = n - q * d;
  while (rem < 0) { --q; rem += d; }
  while (rem >= d) { ++q; rem -= d; }
  return q;
}

__device__ __forceinline__ WinItem win_item(const WinArgs& a, int w) {
  WinItem x;
  int i;
  // a token tile's KV heads side by side (against one head after another: 2% off
  // the wide window, 1% off the narrow one)
  const int bt = win_div(w, a.Hkv, a.inv_hkv, x.kvh);
  x.b = win_div(bt, a.nt, a.inv_nt, i);
  x.t0 = (a.nt - 1 - i) * a.T;  // the last tokens, with the most keys, first
  x.p0 = static_cast<int>(a.q_off) + x.t0;
  x.p1 = min(x.p0 + a.T, static_cast<int>(a.q_off) + a.Lq) - 1;
  const int hi = min(x.p1, a.Lk - 1);
  x.lo = max(0, x.p0 - a.W + 1);
  if (x.lo < a.S) x.lo = 0;  // the sinks are, or adjoin, the window's first keys
  x.sinks = min(min(a.S, x.lo), a.Lk);
  const int len = max(0, hi - x.lo + 1);
  x.merged = x.sinks > 0 && x.sinks <= kWinSinkRows && len > 0;
  x.n_sink = x.merged ? 0 : (x.sinks + kWinKeys - 1) / kWinKeys;
  x.n = x.n_sink + ((x.merged ? kWinSinkRows : 0) + len + kWinKeys - 1) / kWinKeys;
  return x;
}

// Key of tile t's column 0 (of a merged first tile: what column 16 would give, minus 16).
__device__ __forceinline__ int win_key0(const WinItem& x, int t) {
  if (t < x.n_sink) return t * kWinKeys;
  return x.lo - (x.merged ? kWinSinkRows : 0) + (t - x.n_sink) * kWinKeys;
}

// Columns [c0, c1) of a value tile in shared memory, by a whole warp: stays
// zero (of either sign) while all of them are finite, since 0 times a value
// that is not is NaN.
__device__ __forceinline__ void window_look(uint32_t tile, int c0, int c1, uint32_t& acc) {
  const int lane = threadIdx.x & 31;
#pragma unroll 2
  for (int c = c0 + (lane >> 3); c < c1; c += 4) {
    const uint32_t at = tile + c * 128 + (lane & 7) * 16;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t w[4];
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at + hf * (kWinKeys * 128)) : "memory");
#pragma unroll
      for (int k = 0; k < 4; ++k) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w[k]), "r"(0u));
    }
  }
}

// What is not finite in those columns becomes zero.
__device__ __noinline__ void window_scrub(uint32_t tile, int c0, int c1) {
  const int lane = threadIdx.x & 31;
  for (int c = c0 + (lane >> 3); c < c1; c += 4)
    for (int k = 0; k < 8; ++k) {
      const uint32_t at = tile + (k >> 2) * (kWinKeys * 128) + c * 128 + (lane & 7) * 16 + (k & 3) * 4;
      uint32_t w;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
      if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
      if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
    }
  fence_proxy_async_smem();
  __syncwarp();
}

// What window_scrub took from the queries of a warp's 32 rows, back onto half
// hf (64 dims) of their outputs staged at `stage`, a row after the other, two
// dims a lane.  row: this thread's row in the staging buffer, -1 for none;
// t: its token.  Only items whose values window_scrub changed come here; they
// are formed anew from w, to keep the registers of the others.
__device__ __noinline__ void window_restore(const WinArgs& a, int w, int hf, int row, int t, uint32_t stage) {
  const int lane = threadIdx.x & 31;
  const WinItem x = win_item(a, w);
  const __nv_bfloat16* v = a.V + x.b * a.vb + x.kvh * a.vh + 64 * hf + 2 * lane;
  __syncwarp();  // every thread's row is staged
  float2 add = make_float2(0.f, 0.f);  // of values that are not finite alone
  int token = -1;                      // whose they are: the rows of a token's heads share them
  for (int i = 0; i < 32; ++i) {
    const int r = __shfl_sync(0xffffffffu, row, i), p = static_cast<int>(a.q_off) + __shfl_sync(0xffffffffu, t, i);
    if (r < 0) continue;
    auto take = [&](int s0, int s1) {    // keys s0 .. s1
#pragma unroll 4
      for (int s = s0; s <= s1; ++s) {
        const uint32_t y = __ldg(reinterpret_cast<const uint32_t*>(v + s * a.vs));
        if ((y & 0x7f80u) == 0x7f80u) add.x += bf16lo(y);
        if ((y & 0x7f800000u) == 0x7f800000u) add.y += bf16hi(y);
      }
    };
    // the keys of either edge that the row sees: in its window, then its sinks
    // among them (a key taken twice changes nothing)
    if (p != token) {
      token = p;
      add = make_float2(0.f, 0.f);
      const int see = p - a.W + 1, end = min(p, a.Lk - 1), lo_end = min(x.p1 - a.W, end), hi_from = max(x.lo, x.p0 + 1);
      take(max(x.lo, see), lo_end);
      take(x.lo, min(a.S - 1, lo_end));
      take(max(hi_from, see), end);
      take(hi_from, min(a.S - 1, end));
    }
    const uint32_t out = stage + r * 128 + ((((lane >> 2) ^ (r & 7)) << 4) | ((lane & 3) << 2));
    uint32_t o;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(o) : "r"(out) : "memory");
    if (add.x != 0.f) o = (o & 0xffff0000u) | (pack_bf16x2(bf16lo(o) + add.x, 0.f) & 0xffffu);
    if (add.y != 0.f) o = (o & 0xffffu) | (pack_bf16x2(0.f, bf16hi(o) + add.y) & 0xffff0000u);
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(out), "r"(o) : "memory");
  }
}

__global__ void __launch_bounds__(kWinThreads, 2) swa_prefill_kernel(const __grid_constant__ WinArgs a) {
  using L = WinSmem;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  const uint32_t sbase = smem_u32(smem);
  if ((sbase & 1023u) != 0) {  // the swizzled tiles would not be where the products look
    if (threadIdx.x == 0) raise_error(RBS_DEVERR_TIMEOUT);
    return;
  }
  const uint32_t sQ = sbase + L::kQ, sK = sbase + L::kK, sV = sbase + L::kV, bars = sbase + L::kBar;
  auto bar = [&](int k) -> uint32_t { return bars + 8u * k; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBar + kWbNum * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kBar + kWbNum * 8 + 4);
  volatile int* scrubbed = reinterpret_cast<volatile int*>(smem + L::kBar + kWbNum * 8 + 8);  // the item's tiles held values to take out
  const uint64_t limit = a.wait_ns;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(bar(kWbQFull), 1);
    mbar_init(bar(kWbQEmpty), 1);
    for (int s = 0; s < kWinNS; ++s) {
      mbar_init(bar(kWbKFull + s), 1);
      mbar_init(bar(kWbVFull + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kWbSFull + s), 1);
      mbar_init(bar(kWbPFull + s), 4);
    }
    for (int s = 0; s < 4; ++s) mbar_init(bar(kWbPVDone + s), 1);
    mbar_init(bar(kWbOFull), 2);  // the products, and the word on what was taken out of the values
    mbar_init(bar(kWbOEmpty), 4);
    mbar_init(bar(kWbStoreFull), 4);
    mbar_init(bar(kWbStoreEmpty), 1);
    mbar_init(bar(kWbDrain), 1);
    mbar_init(bar(kWbDrain + 1), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  {
    // Q rows past T G and V rows that no copy has filled yet would otherwise
    // hold whatever ran here before: finite zeros once
    uint4* z = reinterpret_cast<uint4*>(smem + L::kQ);
    for (int k = tid; k < L::kBar / 16; k += kWinThreads) z[k] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (warp == 6) {
    tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4 || warp == 5) {
    // ------------------------------------------------------------ Q + K / V producers
    if (lane == 0) {
      const bool isK = warp == 4;
      const CUtensorMap *map = isK ? &a.tmK : &a.tmV, *map_s = isK ? &a.tmKs : &a.tmVs, *map_w = isK ? &a.tmKw : &a.tmVw;
      const uint32_t ring = isK ? sK : sV;
      const int full0 = isK ? kWbKFull : kWbVFull;
      tma_prefetch_desc(map);
      if (isK) tma_prefetch_desc(&a.tmQ);
      const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
      uint32_t nf = 0, nq = 0;
      bool ok = true;
      for (int w = blockIdx.x; w < a.items && ok; w += gridDim.x) {
        const WinItem x = win_item(a, w);
        if (x.n == 0) continue;
        if (isK) {
          if (nq >= 1 && !mbar_wait(bar(kWbQEmpty), (nq - 1) & 1, abort_flag, limit)) break;
          mbar_arrive_expect_tx(bar(kWbQFull), a.T * a.G * 256);
          tma_load_4d_hint(sQ, &a.tmQ, bar(kWbQFull), 0, x.kvh * a.G, x.t0, x.b, pol_q);
          tma_load_4d_hint(sQ + 128 * 128, &a.tmQ, bar(kWbQFull), 64, x.kvh * a.G, x.t0, x.b, pol_q);
          ++nq;
        }
        for (int t = 0; t < x.n; ++t) {
          if (isK && a.stall_after >= 0 && static_cast<int>(nf) >= a.stall_after) { ok = false; break; }
          const int s = nf % kWinNS;
          // the stage's previous tile is consumed: its S (for K) or PV (for V)
          // is complete.  Neither barrier can move past that phase before this
          // load lands, so the parity is unambiguous.
          if (nf >= kWinNS) {
            const uint32_t prev = nf - kWinNS;
            const bool done = isK ? mbar_wait(bar(kWbSFull + (prev & 1)), (prev >> 1) & 1, abort_flag, limit)
                                  : mbar_wait(bar(kWbPVDone + (prev & 3)), (prev >> 2) & 1, abort_flag, limit);
            if (!done) { ok = false; break; }
          }
          mbar_arrive_expect_tx(bar(full0 + s), L::kKVBytes);
          const uint32_t dst = ring + s * L::kKVBytes;
          const int k0 = win_key0(x, t);
          if (t < x.n_sink && !isK) {
            tma_load_4d_hint(dst, &a.tmVt, bar(full0 + s), 0, x.kvh, k0, x.b, pol_kv);
            tma_load_4d_hint(dst + kWinKeys * 128, &a.tmVt, bar(full0 + s), 64, x.kvh, k0, x.b, pol_kv);
          } else if (t == 0 && x.merged) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t d = dst + hf * kWinKeys * 128;
              tma_load_4d_hint(d, map_s, bar(full0 + s), 64 * hf, x.kvh, 0, x.b, pol_kv);
              tma_load_4d_hint(d + kWinSinkRows * 128, map_w, bar(full0 + s), 64 * hf, x.kvh, x.lo, x.b, pol_kv);
            }
          } else {
            tma_load_4d_hint(dst, map, bar(full0 + s), 0, x.kvh, k0, x.b, pol_kv);
            tma_load_4d_hint(dst + kWinKeys * 128, map, bar(full0 + s), 64, x.kvh, k0, x.b, pol_kv);
          }
          ++nf;
        }
      }
      // every load issued must land before the CTA exits
      for (uint32_t s = 0; s < kWinNS; ++s)
        if (s < nf) mbar_drain(bar(full0 + s), ((nf - s + kWinNS - 1) / kWinNS - 1) & 1, limit);
      if (isK && nq > 0) mbar_drain(bar(kWbQFull), (nq - 1) & 1, limit);
    }
  } else if (warp == 6 || warp == 7) {
    // ------------------------------------------------------------ S issuer / PV issuer
    const bool isS = warp == 6;
    constexpr uint32_t idS = idesc_bf16_f32(128, kWinKeys, 0, 0);
    constexpr uint32_t idPV = idesc_bf16_f32(128, 128, 0, 1);
    const uint64_t qdesc = smem_desc(sQ, 16, 1024, kLayoutSW128);
    const uint64_t kdesc0 = smem_desc(sK, 16, 1024, kLayoutSW128);
    const uint64_t vdesc0 = smem_desc(sV, kWinKeys * 128, 1024, kLayoutSW128);
    constexpr uint32_t kStageUnits = L::kKVBytes >> 4, kQHalf = (128 * 128) >> 4, kKHalf = (kWinKeys * 128) >> 4;
    auto wait = [&](int k, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(k), parity, abort_flag, limit)); };
    uint32_t g = 0, it = 0;  // tiles and items so far
    bool ok = true, odd = false;
    for (int w = blockIdx.x; w < a.items && ok; w += gridDim.x) {
      const WinItem x = win_item(a, w);
      if (x.n == 0) continue;
      for (int t = 0; t < x.n; ++t, ++g) {
        const int b = g & 1, s = g % kWinNS;
        if (isS) {
          if (t == 0 && !wait(kWbQFull, it & 1)) { ok = false; break; }
          if (!wait(kWbKFull + s, (g / kWinNS) & 1)) { ok = false; break; }
          // S_g overwrites P_{g-2}: PV_{g-2} must be complete
          if (g >= 2 && !wait(kWbPVDone + ((g - 2) & 3), ((g - 2) >> 2) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint64_t kd = kdesc0 + s * kStageUnits;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ss_warp(tmem + L::col_s(b), qdesc + (kk >> 2) * kQHalf + (kk & 3) * 2, kd + (kk >> 2) * kKHalf + (kk & 3) * 2,
                         idS, kk > 0 ? 1u : 0u);
          umma_commit_warp(bar(kWbSFull + b));
          if (t == x.n - 1) umma_commit_warp(bar(kWbQEmpty));
        } else {
          if (!wait(kWbVFull + s, (g / kWinNS) & 1)) { ok = false; break; }
          // the tile's keys that some row does not see, while its weights are
          // still being formed: at the window's lower edge, and past the first token
          if (t == 0) odd = false;
          const int k0 = win_key0(x, t);
          // steps of 16 keys up to the last one that some row sees
          const int steps = min(kWinKeys / 16, ((t < x.n_sink ? x.sinks - 1 : min(x.p1, a.Lk - 1)) - k0) / 16 + 1);
          if (t >= x.n_sink) {
            const int c0 = t == 0 && x.merged ? kWinSinkRows : 0;
            const int lo_end = min(kWinKeys, x.p1 - a.W + 1 - k0), hi_from = max(c0, x.p0 + 1 - k0), hi_end = min(16 * steps, a.Lk - k0);
            const uint32_t tile = sV + s * L::kKVBytes;
            uint32_t acc = 0;
            window_look(tile, c0, lo_end, acc);
            window_look(tile, hi_from, hi_end, acc);
            if (__any_sync(0xffffffffu, (acc & 0x7fff7fffu) != 0)) {
              window_scrub(tile, c0, lo_end);
              window_scrub(tile, hi_from, hi_end);
              odd = true;
            }
          }
          if (t == x.n - 1 && lane == 0) {
            *scrubbed = odd;
            mbar_arrive(bar(kWbOFull));
          }
          if (!wait(kWbPFull + b, (g >> 1) & 1)) { ok = false; break; }
          if (t == 0 && it > 0 && !wait(kWbOEmpty, (it - 1) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint64_t vd = vdesc0 + s * kStageUnits;
#pragma unroll
          for (int kk = 0; kk < kWinKeys / 16; ++kk)
            if (kk < steps)
              umma_ts_warp(tmem + L::kColO, tmem + L::col_s(b) + kk * 8, vd + kk * (2048 >> 4), idPV, (t == 0 && kk == 0) ? 0u : 1u);
          umma_commit_warp(bar(kWbPVDone + (g & 3)));
          if (t == x.n - 1) umma_commit_warp(bar(kWbOFull));
        }
      }
      if (!isS && ok) {
        // the outputs' stores: the softmax warps stage them while this warp has
        // nothing to issue, the next item's first weights coming after them
        for (int hf = 0; hf < 2 && ok; ++hf) {
          if (!wait(kWbStoreFull, hf)) { ok = false; break; }  // two phases per item
          if (lane == 0) {
            tma_store_4d(&a.tmO, sbase + L::kO, 64 * hf, a.o_seq_inner ? x.t0 : x.kvh * a.G, a.o_seq_inner ? x.kvh * a.G : x.t0, x.b);
            tma_store_commit();
            tma_store_wait_read();
            mbar_arrive(bar(kWbStoreEmpty));
          }
          __syncwarp();
        }
      }
      ++it;
    }
    // drain this issuer's tensor-core work before TMEM is freed
    umma_commit_warp(bar(kWbDrain + (isS ? 0 : 1)));
    mbar_drain(bar(kWbDrain + (isS ? 0 : 1)), 0, limit);
  } else {
    // ------------------------------------------------------------ softmax (warps 0-3)
    const int r = tid;  // row of the tile == TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const float c = a.scale_log2;
    const int tl = r / a.G, gh = r - tl * a.G;  // token and q head of this row
    auto warp_arrive = [&](int k) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(k));
    };
    uint32_t g = 0, it = 0;  // tiles, items
    bool ok = true;
    for (int w = blockIdx.x; w < a.items && ok; w += gridDim.x) {
      const WinItem x = win_item(a, w);
      const int t_row = x.t0 + tl, h = x.kvh * a.G + gh;
      const bool live = tl < a.T && t_row < a.Lq;
      auto write_lse = [&](float z) {
        if (live && a.lse != nullptr) a.lse[(static_cast<int64_t>(x.b) * a.G * a.Hkv + h) * a.Lq + t_row] = z;
      };
      if (x.n == 0) {
        if (live) {
          uint4* dst = reinterpret_cast<uint4*>(a.O + x.b * a.ob + t_row * a.os + h * a.oh);
          for (int k = 0; k < 16; ++k) dst[k] = make_uint4(0, 0, 0, 0);
        }
        write_lse(-INFINITY);
        continue;
      }
      float m_used = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      for (int t = 0; t < x.n; ++t, ++g) {
        const int b = g & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(bar(kWbSFull + b), (g >> 1) & 1, abort_flag, limit))) { ok = false; break; }
        tc_fence_after();
        const uint32_t scol = lane_base + L::col_s(b);
        uint32_t v[2][32];
        tmem_ld32(scol, v[0]);
        tmem_ld32(scol + 32, v[1]);
        tmem_wait_ld();
        const int k0 = win_key0(x, t);
        const bool sink_tile = t < x.n_sink, shared = t == 0 && x.merged;
        if (sink_tile || shared || k0 + kWinKeys - 1 > min(x.p0, a.Lk - 1) || k0 <= x.p1 - a.W) {
          // columns are seen up to hi_c from lo_c on, and below sk_c (sinks): a bit per column
          const int p = x.p0 + tl, hi_c = min(p, a.Lk - 1) - k0, lo_c = sink_tile ? kWinKeys : p - a.W + 1 - k0;
          const int sk_c = sink_tile ? x.sinks - k0 : shared ? x.sinks : a.S - k0;
          auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };  // columns 0 .. n - 1
          const unsigned long long see = below(hi_c + 1) & (~below(lo_c) | below(sk_c));
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t bits = static_cast<uint32_t>(see >> (32 * q));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(bits & (1u << e))) v[q][e] = __float_as_uint(-INFINITY);
          }
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 64; e += 2)
          m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], __uint_as_float(v[e >> 5][e & 31]), __uint_as_float(v[e >> 5][(e & 31) + 1]));
        const float mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
        const float m_new = fmaxf(m_used, mx * c);
        float factor = 1.f;
        bool rescale = false;
        if (t == 0) {
          m_used = m_new;
        } else if (m_new - m_used > 8.f) {
          // a row that has seen no key yet has nothing to scale
          rescale = m_used != -INFINITY;
          factor = ptx_exp2(m_used - m_new);
          m_used = m_new;
        }
        const float m_exp = m_used == -INFINITY ? 0.f : m_used;
        l2.x *= factor;
        l2.y *= factor;
        const float2 c2 = make_float2(c, c), nm2 = make_float2(-m_exp, -m_exp);
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t pw[32];
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          const float2 arg = ffma2(make_float2(__uint_as_float(v[e >> 5][e & 31]), __uint_as_float(v[e >> 5][(e & 31) + 1])), c2, nm2);
          const float2 pv = make_float2(ptx_exp2(arg.x), ptx_exp2(arg.y));
          acc[(e >> 1) & 1] = fadd2(acc[(e >> 1) & 1], pv);
          pw[e >> 1] = pack_bf16x2(pv.x, pv.y);
        }
        tmem_st32(scol, pw);
        l2 = fadd2(l2, fadd2(acc[0], acc[1]));
        if (__any_sync(0xffffffffu, rescale)) {
          // O must hold every earlier tile's product first.  The next phase of
          // PV_{g-1}'s barrier is PV_{g+3}, which needs this tile's P.
          if (!__all_sync(0xffffffffu, mbar_wait(bar(kWbPVDone + ((g - 1) & 3)), ((g - 1) >> 2) & 1, abort_flag, limit))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t o[32];
            tmem_ld32(lane_base + L::kColO + 32 * q, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
            tmem_st32(lane_base + L::kColO + 32 * q, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(kWbPFull + b);
      }
      if (!ok) break;

      // ---- epilogue: O / l -> bf16, LSE
      const float l = l2.x + l2.y;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(kWbOFull), it & 1, abort_flag, limit))) { ok = false; break; }
      tc_fence_after();
      const bool odd = *scrubbed != 0;
      const float2 inv2 = make_float2(inv, inv);
      // this row in the store's box (128-byte swizzle: 16-byte chunk k of row r at k ^ (r % 8))
      const int ro = a.o_seq_inner ? gh * a.T + tl : r;
      uint32_t ow[2][32];  // the row as bf16 pairs
      {
        uint32_t o[32];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tmem_ld32(lane_base + L::kColO + 32 * q, o);
          tmem_wait_ld();
          if (q == 3) {
            tc_fence_before();
            warp_arrive(kWbOEmpty);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 f2 = fmul2(make_float2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), inv2);
            ow[q >> 1][16 * (q & 1) + e] = pack_bf16x2(f2.x, f2.y);
          }
        }
      }
      write_lse(l == 0.f ? -INFINITY : (m_used + log2f(l)) * 0.69314718055994530942f);
      // 64 dims at a time through the staging buffer, whose stores warp 7 issues
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        // the buffer's previous half (two phases per item) has been read
        if (it + hf >= 1 && !__all_sync(0xffffffffu, mbar_wait(bar(kWbStoreEmpty), (hf + 1) & 1, abort_flag, limit))) { ok = false; break; }
        if (tl < a.T) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(sbase + L::kO + ro * 128 + ((k ^ (ro & 7)) << 4)),
                         "r"(ow[hf][4 * k]), "r"(ow[hf][4 * k + 1]), "r"(ow[hf][4 * k + 2]), "r"(ow[hf][4 * k + 3])
                         : "memory");
        }
        if (odd) window_restore(a, w, hf, live ? ro : -1, t_row, sbase + L::kO);
        fence_proxy_async_smem();
        warp_arrive(kWbStoreFull);
      }
      ++it;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 6) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

}  // namespace rbs
