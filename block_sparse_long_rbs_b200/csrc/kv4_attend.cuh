// Attention of new tokens over the 4-bit paged cache.
//
// For query t of request b at position p = start_b + t and q head h of KV
// head h / G:
//   O = sum_s softmax_s(scale q . k_s) v_s  over the cached keys s <= p,
// with a window W also p - W < s or s < S (the S first tokens stay visible).
//
// A work item is (request, KV head, tile of 8 NT query rows), rows being the
// (token, q head of the group) pairs that share the KV head, so a cached byte
// is read once for all of them.  An item's visible sub-blocks (16 tokens)
// form units of eight, one per warp; all items' units in one sequence are cut
// into equal runs, one per CTA, so unequal lengths leave no CTA idle.  An item
// that a CTA holds whole is finished there; parts of items split between CTAs
// go to the workspace as (max, sum, unnormalised output) and
// kv4_combine_kernel joins them in their order, so results do not vary.
//
// A warp works on its own sub-blocks with no barrier: 2304 bytes by 16-byte
// asynchronous copies into its ring, then
//   S^T (16 keys x 8 rows) = K Q^T,  O^T (16 dims x 8 rows) += V^T P^T
// by mma.m16n8k16 in fp16 with fp32 sums: rows of queries are the instruction's
// narrow side, since one token's G rows rarely fill the wide one.  The codes
// become fp16 by the e2m1 conversion, and times their scale stay exact; Q is
// brought to fp16 by a power of two per row (bf16's 8 bits fit fp16's 11; values
// more than 2^26 below the row's largest lose bits that fp32 sums would lose as
// well); P = 2^6 exp2(s - m) is rounded to fp16 once (2^-11 relative), m at most
// 2^8 below the running maximum, so that an update is rare; keys down to 2^-31
// of the largest still count.  Sums and outputs stay in fp32.
// Keys that no row may see get the value scale 0 (their bytes may be
// anything, NaN scales too); a sub-block that some rows see only in part is
// taken once per query token, for that token's rows alone and with the keys it
// may not see set to zero.
// 144 bytes per cached token and KV head have to be read.  Measured: 64 requests of
// 8,192 to 16,384 tokens, 32 q / 4 KV heads (about 456 MB): 118 us, 3.9 TB/s of the
// 6.46 a copy reaches; most of the time goes to instruction issue (61% of the slots, about 400 warp
// instructions per sub-block, of them 88 conversions, 64 scalings, 16 matrix
// instructions), the rest to latencies that four warps per scheduler leave open.
// 32 rows per tile: the outputs
// take 128 registers of every thread, one CTA per SM and two warps per
// scheduler are left, and latency bounds it (four drafted tokens of four requests
// of 65,536 to 131,072 tokens: 131 us for 383,000 tokens in all, 139 for 406,000).
// Spilled registers: 24 bytes of stores there, 64 for 16 rows of one token, 196
// for 16 rows of several, where two CTAs per SM allow 128 registers (what they
// cost apart has not been measured); none for 8 rows.  Measured and left: tiles of 16 rows
// there, reading the cache twice (226 against 165 us); pairs of warps that share
// a sub-block's rows and dims (178 against 133 us: keys converted twice); rings of
// 4 and 6 stages (120 and 118 us for the 64 requests); two chains of products
// for the scores (no change); the next sub-block's scores before this one's
// products (no change, and 16 rows spill: 195 against 173 us for 64 requests of
// two tokens); groups of four warps that each form the scores of their own
// sub-block and a quarter of the dims of all four, P going through shared
// memory, which doubles the warps (138 against 134 us: 634 warp instructions per
// sub-block for 437).
#pragma once

#include <cfloat>
#include <type_traits>

#include "kv4.cuh"

namespace rbs {

constexpr int kAttWarps = 8;
constexpr int kAttThreads = kAttWarps * 32;
constexpr int kAttStages = 5;
constexpr int kAttMaxBatch = 4096;
constexpr float kAttPShift = 6.f;  // P carries 2^6
constexpr float kAttNoMax = -FLT_MAX;  // the running maximum of a row that has seen no key: below every score, and finite

struct Kv4AttArgs {
  const uint8_t* data;
  int64_t num_pages;
  int Hkv, G, page, spp;      // spp: sub-blocks per page
  uint32_t page_bytes;        // of all heads: at most 65535 * 16 * 2304
  uint32_t spp_magic;         // ceil(2^32 / spp); 0 when spp is 1
  const int32_t* table;
  int64_t table_b;
  int max_pages, B, Lq;
  const int32_t *lens, *starts;
  int window, sinks;
  const __nv_bfloat16* q;
  int64_t qb, qs, qh;
  __nv_bfloat16* o;
  int64_t ob, os, oh;
  float* lse;  // [B, Hq, Lq] or null
  float scale_log2;  // softmax scale * log2(e)
  int k_exp;         // k_scale's power of two
  float v_scale;
  int tiles;  // row tiles of 8 NT rows per (request, KV head)
  float *part_o, *part_ml;  // workspace: two slots per CTA
  int ctas;  // CTAs of the main kernel; those past the count of units have none
};

// CTAs that share the units: each has at least one.
__device__ __forceinline__ int att_sharers(const Kv4AttArgs& a, int64_t total) {
  return static_cast<int>(min(total, static_cast<int64_t>(a.ctas)));
}

// A request's visible range for its queries: sub-blocks [0, sink) and
// [lo, hi), and the positions of its queries.
struct AttRange {
  int first_q, len, sink, lo, n;  // n: sub-blocks in all
};

__device__ __forceinline__ AttRange att_range(const Kv4AttArgs& a, int b) {
  AttRange r;
  const int64_t most = static_cast<int64_t>(a.max_pages) * a.page;
  r.len = static_cast<int>(min(static_cast<int64_t>(max(__ldg(a.lens + b), 0)), most));
  r.first_q = a.starts != nullptr ? __ldg(a.starts + b) : r.len - a.Lq;
  const int64_t qmin = max(r.first_q, 0);
  const int64_t qmax = min(static_cast<int64_t>(r.first_q) + a.Lq, static_cast<int64_t>(r.len)) - 1;
  r.sink = r.lo = r.n = 0;
  if (qmax < qmin) return r;
  if (a.window > 0) {
    r.lo = static_cast<int>(max(qmin - a.window + 1, static_cast<int64_t>(0)) >> 4);
    r.sink = static_cast<int>(min((static_cast<int64_t>(a.sinks) + 15) >> 4, static_cast<int64_t>(r.lo)));
  }
  r.n = r.sink + static_cast<int>(qmax >> 4) + 1 - r.lo;
  return r;
}

// Prefix sums of the requests' units into shared memory, prefix[B] their sum.
// A request with nothing visible has one unit, which writes its empty rows.
__device__ __forceinline__ void att_units(const Kv4AttArgs& a, int32_t* prefix, int64_t* sums) {
  int64_t carry = 0;
  for (int base = 0; base < a.B; base += blockDim.x) {
    const int b = base + threadIdx.x;
    int64_t v = 0;
    if (b < a.B) v = max(1, (att_range(a, b).n + kAttWarps - 1) / kAttWarps);
    int64_t total;
    const int64_t before = block_exclusive_scan(v, sums, total);
    if (b < a.B) prefix[b] = static_cast<int32_t>(carry + before);
    carry += total;
  }
  if (threadIdx.x == 0) prefix[a.B] = static_cast<int32_t>(carry);
  __syncthreads();
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same onto zeros.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Four e2m1 pairs (a word) as f16x2 each.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
// Four e4m3 scales (a word) as two f16x2.
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// a times either half of s
__device__ __forceinline__ uint32_t hmul2_half(uint32_t a, uint32_t s, int hi) {
  const __half2 x = *reinterpret_cast<const __half2*>(&a), y = *reinterpret_cast<const __half2*>(&s);
  const __half2 r = __hmul2(x, hi ? __high2half2(y) : __low2half2(y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
  return v;
}

template <int NT>
struct AttSmem {
  static constexpr int kRing = 0;
  static constexpr int kQ = kRing + kAttWarps * kAttStages * kSubBytes;  // Q fragments [8 groups][NT][32 lanes][8 B]
  static constexpr int kQFac = kQ + 8 * NT * 256;                        // float [8 NT]: what brings the rows' products to exponents
  // a warp's part for joining, float [8 rows][128 + 4], lies over its own ring
  static_assert(kAttStages * kSubBytes >= 8 * 132 * 4, "the ring holds it");
  static constexpr int kPos = kQFac + 8 * NT * 4;                        // int [8 NT]: the rows' positions, -1: it sees nothing
  static constexpr int kML = kPos + 8 * NT * 4;                          // float [8 warps][8 NT][2]
  static constexpr int kSums = kML + kAttWarps * 8 * NT * 8;             // int64 [warps]
  static constexpr int kPrefix = kSums + kAttWarps * 8;                  // int32 [B + 1]
  static constexpr int bytes(int B) { return kPrefix + (B + 1) * 4; }
};

// ONE: every request has one query token (Lq == 1).
template <int NT, bool ONE>
__global__ void __launch_bounds__(kAttThreads, NT <= 2 ? 2 : 1) kv4_attend_kernel(const __grid_constant__ Kv4AttArgs a) {
  using L = AttSmem<NT>;
  constexpr int R = 8 * NT;  // rows of a tile
  extern __shared__ __align__(16) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  float* qfac = reinterpret_cast<float*>(smem + L::kQFac);
  int* qpos = reinterpret_cast<int*>(smem + L::kPos);
  float* ml = reinterpret_cast<float*>(smem + L::kML);
  int64_t* sums = reinterpret_cast<int64_t*>(smem + L::kSums);
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + L::kPrefix);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, j = lane & 3;
  const uint32_t ring = sb + L::kRing + warp * kAttStages * kSubBytes;

  att_units(a, prefix, sums);
  if (blockIdx.x == 0)
    for (int b = tid; b < a.B; b += kAttThreads) {
      const int len = __ldg(a.lens + b);
      if (len < 0 || len > static_cast<int64_t>(a.max_pages) * a.page) raise_error(RBS_DEVERR_LENGTH);
    }
  const int HT = a.Hkv * a.tiles;
  const int64_t total = static_cast<int64_t>(prefix[a.B]) * HT;
  const int sharers = att_sharers(a, total), me = min(static_cast<int>(blockIdx.x), sharers);
  int64_t u = total * me / sharers;
  const int64_t u_end = total * min(me + 1, sharers) / sharers;
  bool first_part = true;

  while (u < u_end) {
    // the item of unit u: request (last b with prefix[b] HT <= u), KV head, row tile
    int lo_b = 0, hi_b = a.B - 1;
    const int64_t target = u / HT;
    while (lo_b < hi_b) {
      const int mid = (lo_b + hi_b + 1) >> 1;
      if (prefix[mid] <= target) lo_b = mid; else hi_b = mid - 1;
    }
    const int b = lo_b, nu = prefix[b + 1] - prefix[b];
    const int64_t rem = u - static_cast<int64_t>(prefix[b]) * HT;
    const int ht = static_cast<int>(rem / nu);
    const int ua = static_cast<int>(rem - static_cast<int64_t>(ht) * nu);
    const int ub = static_cast<int>(min(static_cast<int64_t>(nu), ua + (u_end - u)));
    const int kvh = ht / a.tiles, tile = ht - kvh * a.tiles;
    u += ub - ua;
    const AttRange rg = att_range(a, b);
    const int rows = a.G * a.Lq, row0 = tile * R;

    // ---- sub-blocks v = 8 k + warp of units [ua, ub)
    const int v_end = min(ub * kAttWarps, rg.n);
    const int shift = rg.lo - rg.sink;  // from a sub-block's place in the item to its place in the request, past the sinks
    const int32_t* table = a.table + b * a.table_b;
    const uint8_t* head_data = a.data + static_cast<int64_t>(kvh) * a.spp * kSubBytes + 16 * lane;
    const uint32_t ring_lane = ring + 16 * lane;
    // the next sub-block to load: its table entry is fetched one step ahead
    int v_load = ua * kAttWarps + warp, pg_next = 0;
    uint32_t off_next = 0, dst_next = ring_lane;
    auto look = [&]() {
      if (v_load < v_end) {
        const int sub = v_load < rg.sink ? v_load : v_load + shift;
        const int pi = a.spp_magic != 0 ? static_cast<int>(__umulhi(static_cast<uint32_t>(sub), a.spp_magic)) : sub;
        pg_next = __ldg(table + pi);
        off_next = static_cast<uint32_t>(sub - pi * a.spp) * kSubBytes;
      }
    };
    look();
    uint32_t taken = 0;  // bit per stage issued, newest lowest: its page was valid
    auto issue = [&]() {
      bool ok = false;
      if (v_load < v_end) {
        ok = static_cast<uint32_t>(pg_next) < static_cast<uint32_t>(a.num_pages);
        if (!ok && lane == 0) raise_error(RBS_DEVERR_BLOCK_INDEX);
        const uint8_t* src = head_data + (static_cast<uint64_t>(ok ? static_cast<uint32_t>(pg_next) : 0u) * a.page_bytes + off_next);
#pragma unroll
        for (int q = 0; q < 4; ++q) cp_async16(dst_next + 512 * q, src + 512 * q, ok);
        if (lane < 16) cp_async16(dst_next + 2048, src + 2048, ok);
      }
      cp_async_commit();
      taken = (taken << 1) | (ok ? 1u : 0u);
      dst_next = dst_next == ring_lane + (kAttStages - 1) * kSubBytes ? ring_lane : dst_next + kSubBytes;
      v_load += kAttWarps;
      look();
    };
    __syncthreads();  // the previous item's readers are done
#pragma unroll
    for (int q = 0; q < kAttStages - 1; ++q) issue();


    // ---- Q fragments: row n of the tile, dims 16 s + {2j, 2j + 1, 2j + 8, 2j + 9}
    for (int n = warp; n < R; n += kAttWarps) {
      const int row = row0 + n;
      uint2 x = make_uint2(0, 0);
      if (row < rows) {
        const int t = row / a.G, g = row - t * a.G;
        x = *reinterpret_cast<const uint2*>(a.q + b * a.qb + t * a.qs + (kvh * a.G + g) * a.qh + 4 * lane);
      }
      const float v[4] = {bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y)};
      float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      // the row times 2^-e, its largest in [2^11, 2^12); e kept in the range where 2^e and 2^-e are normal
      const int e = (m > 0.f && m < INFINITY) ? max(-126, min(126, static_cast<int>(__float_as_uint(m) >> 23) - 127 - 11)) : 0;
      const float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      // lane holds dims 4 lane .. 4 lane + 3 of group s = lane / 4: k = 4 (lane % 4) ..
      const int s = lane >> 2, k0 = 4 * (lane & 3);
      const uint32_t w0 = pack_f16x2(v[0] * up, v[1] * up), w1 = pack_f16x2(v[2] * up, v[3] * up);
      const uint32_t dst = sb + L::kQ + ((s * NT + (n >> 3)) * 32 + (n & 7) * 4) * 8;
      // pair k, k + 1 belongs to lane (n % 8, (k % 8) / 2), word k / 8
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + ((k0 & 7) >> 1) * 8 + (k0 >> 3) * 4), "r"(w0) : "memory");
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + (((k0 + 2) & 7) >> 1) * 8 + (k0 >> 3) * 4), "r"(w1) : "memory");
      if (lane == 0) {
        // scale_log2 k_scale 2^e, the powers of two in halves that fp32 holds.  A factor outside fp32's
        // range comes from a row whose scores are all negligible (products stay below 2^31), or whose
        // scores fp32 does not hold: the end of the range serves, where 0 or an infinity would make a
        // masked score's -inf, or a product of 0, a NaN.
        const int f = e + a.k_exp, half = f >> 1;
        const float fac = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + half) << 23) * __uint_as_float(static_cast<uint32_t>(127 + f - half) << 23);
        qfac[n] = fminf(fmaxf(fac, FLT_MIN), FLT_MAX);
        const int p = row < rows ? rg.first_q + row / a.G : -1;
        qpos[n] = p < rg.len ? p : -1;
      }
    }
    __syncthreads();

    // ---- this thread's columns of S^T: rows 8 nt + 2j + {0, 1}
    float sc[NT][2];
    float m_run[NT][2], l_run[NT][2], o[8][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sc[nt][i] = qfac[8 * nt + 2 * j + i];
        m_run[nt][i] = kAttNoMax;
        l_run[nt][i] = 0.f;
      }
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q) o[s][nt][q] = 0.f;
    // positions of the tile's live queries: [p_lo, p_hi].  Rows of a padded batch that are past the request's tokens or
    // before its first take part in sub-blocks that the live rows see whole, whatever comes out: they are emptied when
    // the warps join (three live tokens of four over 65,536: 101 us a call against 288 when one such row made every
    // sub-block a partly visible one; four live ones 100).
    const int t_lo = row0 / a.G, t_hi = (min(row0 + R, rows) - 1) / a.G;
    const int p_lo = max(rg.first_q + t_lo, 0);
    const int p_hi = max(0, static_cast<int>(min(static_cast<int64_t>(rg.first_q) + t_hi, static_cast<int64_t>(rg.len) - 1)));
    // sub-blocks that every live row sees whole: below full_sink, and in [full_lo, full_hi)
    const int full_hi = ((p_lo + 1) >> 4) - shift;
    const int full_lo = a.window == 0 ? 0 : static_cast<int>((static_cast<uint32_t>(max(p_hi - a.window + 1, 0)) + 15u) >> 4) - shift;
    const int full_sink = min(rg.sink, a.sinks >> 4);

    // ---- the sub-blocks: products of one, then scores of the next
    uint32_t p0[NT], p1[NT];  // P^T, the second product's operand: keys 2j, 2j + 1 (+ 8) of row r
    bool full = true, valid = true;  // of the sub-block whose P these are
    int tok0 = 0;

    // S^T = K Q^T of a stage, unscaled
    auto scores = [&](uint32_t st, float (&c)[NT][4]) {
      const uint4 ka = lds128(st + 16 * lane), kb = lds128(st + 512 + 16 * lane);
      const uint2 sa = lds64(st + 2048 + 8 * r), sbk = lds64(st + 2048 + 64 + 8 * r);
      uint32_t fa[4], fb[4];  // f16x2 scales of groups (0,1), (2,3), ...
      e4m3x4_f16(sa.x, fa[0], fa[1]);
      e4m3x4_f16(sa.y, fa[2], fa[3]);
      e4m3x4_f16(sbk.x, fb[0], fb[1]);
      e4m3x4_f16(sbk.y, fb[2], fb[3]);
      const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t xa[4], xb[4];
        e2m1x8_f16(wa[w], xa);
        e2m1x8_f16(wb[w], xb);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int s = 2 * w + e;
          const uint32_t a0 = hmul2_half(xa[2 * e], fa[w], e), a1 = hmul2_half(xb[2 * e], fb[w], e);
          const uint32_t a2 = hmul2_half(xa[2 * e + 1], fa[w], e), a3 = hmul2_half(xb[2 * e + 1], fb[w], e);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 qf = lds64(sb + L::kQ + ((s * NT + nt) * 32 + lane) * 8);
            if (s == 0) mma_f16_first(c[nt], a0, a1, a2, a3, qf.x, qf.y);
            else mma_f16(c[nt], a0, a1, a2, a3, qf.x, qf.y);
          }
        }
      }
    };
    // scores -> P of sub-block v, whose page was there or not; c[nt][2 i + q]: key r + 8 i, row column q
    auto weights = [&](float (&c)[NT][4], int v, bool there) {
      valid = there;
      full = there && (v < full_sink || (v >= full_lo && v < full_hi));
      if (!full) {
        tok0 = (v < rg.sink ? v : v + shift) * 16;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int key = tok0 + r + 8 * (q >> 1), p = qpos[8 * nt + 2 * j + (q & 1)];
            const bool see = valid && key <= p && (a.window == 0 || key > p - a.window || key < a.sinks);
            if (!see) c[nt][q] = -INFINITY;
          }
      }
      // exponents of P; the running maximum moves only when a score passes it by 2^8.  The scaled scores are
      // rounded before the maximum is taken off, as the maximum itself was: one rounding for both would leave the
      // difference of a rounded and an exact product, which past 2^28 is more than fp16's exponents hold
      // (in pairs this takes no more instructions).
      auto exponents = [&](int nt, int i) {  // of keys r (i = 0) or r + 8 (i = 2)
        return fadd2(fmul2(make_float2(c[nt][i], c[nt][i + 1]), make_float2(sc[nt][0], sc[nt][1])),
                     make_float2(kAttPShift - m_run[nt][0], kAttPShift - m_run[nt][1]));
      };
      float e[NT][4];
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          const float2 x = exponents(nt, q);
          e[nt][q] = x.x;
          e[nt][q + 1] = x.y;
        }
        up = up || fmaxf(fmax3(e[nt][0], e[nt][1], e[nt][2]), e[nt][3]) > 8.f + kAttPShift;
      }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mx = fmaxf(c[nt][i], c[nt][2 + i]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m_run[nt][i], mx * sc[nt][i]);
            const float f = ptx_exp2(m_run[nt][i] - mn);
            m_run[nt][i] = mn;
            l_run[nt][i] *= f;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
              o[s][nt][i] *= f;
              o[s][nt][2 + i] *= f;
            }
          }
#pragma unroll
          for (int q = 0; q < 4; q += 2) {
            const float2 x = exponents(nt, q);
            e[nt][q] = x.x;
            e[nt][q + 1] = x.y;
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int q = 0; q < 4; ++q) e[nt][q] = ptx_exp2(e[nt][q]);
        l_run[nt][0] += e[nt][0] + e[nt][2];
        l_run[nt][1] += e[nt][1] + e[nt][3];
        p0[nt] = movmatrix_trans(pack_f16x2(e[nt][0], e[nt][1]));
        p1[nt] = movmatrix_trans(pack_f16x2(e[nt][2], e[nt][3]));
      }
    };
    // which of keys k0, k0 + 1 of the sub-block the query at position pt sees, as a mask of scale bytes
    auto keep = [&](int k0, int pt) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = tok0 + k0 + i;
        if (valid && pt < rg.len && key <= pt && (a.window == 0 || key > pt - a.window || key < a.sinks)) m |= 0x00ff00ffu << (8 * i);
      }
      return m;
    };
    // O^T += V^T P^T of a stage; group s is dims 16 s .. 16 s + 15 of the
    // instruction's 16 rows.  All columns, or (part) those of token t alone:
    // 0 times a NaN value is one, so other columns are left out and not given
    // zero weights.
    auto product = [&](auto part, uint32_t st, const uint4& ta, const uint4& tb, int t) {
      bool mine[NT][2];
      if (part)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) mine[nt][i] = (row0 + 8 * nt + 2 * j + i) / a.G == t;
      const uint4 va = lds128(st + 1024 + 16 * lane), vb = lds128(st + 1536 + 16 * lane);
      const uint32_t ya[4] = {ta.x, ta.y, ta.z, ta.w}, yb[4] = {tb.x, tb.y, tb.z, tb.w};
#pragma unroll
      for (int hw = 0; hw < 2; ++hw) {  // groups 4 hw .. 4 hw + 3
        const uint32_t a_0 = hw ? va.y : va.x, a_1 = hw ? va.w : va.z;  // keys 2j, 2j + 1
        const uint32_t b_0 = hw ? vb.y : vb.x, b_1 = hw ? vb.w : vb.z;  // keys 2j + 8, 2j + 9
        uint32_t xl[4], xh[4], zl[4], zh[4];
        constexpr uint32_t k = 0x0f0f0f0fu;
        e2m1x8_f16((a_0 & k) | ((a_1 << 4) & ~k), xl);  // dim r of both keys
        e2m1x8_f16(((a_0 >> 4) & k) | (a_1 & ~k), xh);  // dim r + 8
        e2m1x8_f16((b_0 & k) | ((b_1 << 4) & ~k), zl);
        e2m1x8_f16(((b_0 >> 4) & k) | (b_1 & ~k), zh);
        uint32_t ga[4], gb[4];
        e4m3x4_f16(ya[2 * hw], ga[0], ga[1]);
        e4m3x4_f16(ya[2 * hw + 1], ga[2], ga[3]);
        e4m3x4_f16(yb[2 * hw], gb[0], gb[1]);
        e4m3x4_f16(yb[2 * hw + 1], gb[2], gb[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a0 = hmul2(xl[e], ga[e]), a1 = hmul2(xh[e], ga[e]);
          const uint32_t a2 = hmul2(zl[e], gb[e]), a3 = hmul2(zh[e], gb[e]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (part) {
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(d, a0, a1, a2, a3, p0[nt], p1[nt]);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (mine[nt][q & 1]) o[4 * hw + e][nt][q] += d[q];
            } else {
              mma_f16(o[4 * hw + e][nt], a0, a1, a2, a3, p0[nt], p1[nt]);
            }
          }
        }
      }
    };

    const int v_first = ua * kAttWarps + warp;
    if (v_first < v_end) {
      float c[NT][4];
      cp_async_wait<kAttStages - 2>();
      __syncwarp();  // every lane's copies have landed
      scores(ring, c);
      weights(c, v_first, (taken >> (kAttStages - 2)) & 1u);
      uint32_t st = ring, nx = ring + kSubBytes;
      for (int v = v_first; v < v_end; v += kAttWarps) {
        cp_async_wait<kAttStages - 3>();
        __syncwarp();  // the next stage is there, and the one before this is read out
        issue();
        const uint32_t scales = st + 2176 + 16 * j;
        uint4 ta = lds128(scales), tb = lds128(scales + 64);
        if (ONE) {
          if (!full) {
            const uint32_t ka = keep(2 * j, rg.first_q), kb = keep(2 * j + 8, rg.first_q);
            ta = make_uint4(ta.x & ka, ta.y & ka, ta.z & ka, ta.w & ka);
            tb = make_uint4(tb.x & kb, tb.y & kb, tb.z & kb, tb.w & kb);
          }
          product(std::false_type{}, st, ta, tb, 0);
        } else {
          if (full) {
            product(std::false_type{}, st, ta, tb, 0);
          } else {
            // once per query token, with the keys it sees
            for (int t = t_lo; t <= t_hi; ++t) {
              const uint32_t ka = keep(2 * j, rg.first_q + t), kb = keep(2 * j + 8, rg.first_q + t);
              product(std::true_type{}, st, make_uint4(ta.x & ka, ta.y & ka, ta.z & ka, ta.w & ka),
                      make_uint4(tb.x & kb, tb.y & kb, tb.z & kb, tb.w & kb), t);
            }
          }
        }
        if (v + kAttWarps < v_end) {
          scores(nx, c);
          weights(c, v + kAttWarps, (taken >> (kAttStages - 2)) & 1u);
        }
        st = nx;
        nx = nx == ring + (kAttStages - 1) * kSubBytes ? ring : nx + kSubBytes;
      }
    }
    cp_async_wait<0>();

    // ---- join the warps: row sums over lanes, then every row over the warps
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = l_run[nt][i];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (r == 0) {
          const int n = 8 * nt + 2 * j + i;
          ml[(warp * R + n) * 2] = m_run[nt][i];
          ml[(warp * R + n) * 2 + 1] = l;
        }
      }
    constexpr int kMergeStride = kAttStages * kSubBytes / 4;
    float* merge = reinterpret_cast<float*>(smem + L::kRing);
    const bool whole = ua == 0 && ub == nu;
    const int slot = 2 * blockIdx.x + (first_part ? 0 : 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          merge[warp * kMergeStride + (2 * j + (q & 1)) * 132 + 16 * s + r + 8 * (q >> 1)] = o[s][nt][q];
      __syncthreads();
      // warp w: row w of this group of eight, four dims a lane
      const int n = 8 * nt + warp, row = row0 + n;
      float m = kAttNoMax;
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) m = fmaxf(m, ml[(w * R + n) * 2]);
      float l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) {
        const float f = ptx_exp2(ml[(w * R + n) * 2] - m);
        const float4 x = *reinterpret_cast<const float4*>(merge + w * kMergeStride + warp * 132 + 4 * lane);
        l = fmaf(f, ml[(w * R + n) * 2 + 1], l);
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
      }
      if (row < rows) {
        if (qpos[n] < 0) {  // a row that sees nothing
          m = kAttNoMax;
          l = 0.f;
          acc = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (whole) {
          const float inv = l == 0.f ? 0.f : a.v_scale / l;  // a NaN stays one
          const int t = row / a.G, h = kvh * a.G + row - t * a.G;
          *reinterpret_cast<uint2*>(a.o + b * a.ob + t * a.os + h * a.oh + 4 * lane) =
              make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
          if (a.lse != nullptr && lane == 0)
            a.lse[(static_cast<int64_t>(b) * a.Hkv * a.G + h) * a.Lq + t] =
                l == 0.f ? -INFINITY : (m - kAttPShift + log2f(l)) * 0.69314718055994530942f;
        } else {
          *reinterpret_cast<float4*>(a.part_o + (static_cast<int64_t>(slot) * R + n) * 128 + 4 * lane) = acc;
          if (lane == 0) *reinterpret_cast<float2*>(a.part_ml + (static_cast<int64_t>(slot) * R + n) * 2) = make_float2(m, l);
        }
      }
    }
    first_part = false;
  }
  asm volatile("griddepcontrol.launch_dependents;");
}

// Joins the parts of split items: one CTA of four warps per (request, KV head,
// row tile) and row.  The CTAs whose runs meet the item follow from the same
// prefix sums.  The warps take the parts in turn, four dims a lane, and their
// sums are added in warp order.
constexpr int kAttMaxCtas = 2 * 160;

template <int NT>
__global__ void __launch_bounds__(128) kv4_combine_kernel(const __grid_constant__ Kv4AttArgs a) {
  constexpr int R = 8 * NT;
  __shared__ int64_t sums[4];
  __shared__ float weight[kAttMaxCtas], red[8];
  __shared__ float4 acc_s[4][32];
  extern __shared__ int32_t prefix[];
  const int HT = a.Hkv * a.tiles;
  const int item = blockIdx.x;  // b * HT + ht
  const int b = item / HT, ht = item - b * HT, kvh = ht / a.tiles, tile = ht - kvh * a.tiles;
  const int n = blockIdx.y, rows = a.G * a.Lq, row = tile * R + n;
  att_units(a, prefix, sums);
  const int64_t total = static_cast<int64_t>(prefix[a.B]) * HT;
  const int sharers = att_sharers(a, total);
  const int nu = prefix[b + 1] - prefix[b];
  const int64_t u0 = static_cast<int64_t>(prefix[b]) * HT + static_cast<int64_t>(ht) * nu, u1 = u0 + nu;
  // CTA c holds [total c / sharers, total (c + 1) / sharers): unit u is with the last c whose run begins at or before it
  const int c0 = static_cast<int>(((u0 + 1) * sharers - 1) / total), c1 = static_cast<int>((u1 * sharers - 1) / total);
  // a part is its CTA's first one unless the CTA's run began before the item
  const int first_slot = 2 * c0 + (total * c0 / sharers < u0 ? 1 : 0);
  auto at = [&](int i) { return static_cast<int64_t>(i == 0 ? first_slot : 2 * (c0 + i)) * R + n; };
  const int parts = c1 - c0 + 1;
  // every block waits for the main kernel, so this grid never ends before it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= rows || parts == 1) return;  // one part: written by its CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float m = kAttNoMax;
  for (int i = threadIdx.x; i < parts; i += 128) m = fmaxf(m, a.part_ml[at(i) * 2]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  float l = 0.f;
  for (int i = threadIdx.x; i < parts; i += 128) {
    const float2 x = *reinterpret_cast<const float2*>(a.part_ml + at(i) * 2);
    const float f = ptx_exp2(x.x - m);
    weight[i] = f;
    l = fmaf(f, x.y, l);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if (lane == 0) red[4 + warp] = l;
  __syncthreads();
  l = (red[4] + red[5]) + (red[6] + red[7]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = warp; i < parts; i += 4) {
    const float4 x = *reinterpret_cast<const float4*>(a.part_o + at(i) * 128 + 4 * lane);
    const float f = weight[i];
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, x.z, acc.z);
    acc.w = fmaf(f, x.w, acc.w);
  }
  acc_s[warp][lane] = acc;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    const float4 x = acc_s[w][lane];
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
  }
  const float inv = l == 0.f ? 0.f : a.v_scale / l;
  const int t = row / a.G, h = kvh * a.G + row - t * a.G;
  *reinterpret_cast<uint2*>(a.o + b * a.ob + t * a.os + h * a.oh + 4 * lane) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse != nullptr && lane == 0)
    a.lse[(static_cast<int64_t>(b) * a.Hkv * a.G + h) * a.Lq + t] =
        l == 0.f ? -INFINITY : (m - kAttPShift + log2f(l)) * 0.69314718055994530942f;
}

}  // namespace rbs
