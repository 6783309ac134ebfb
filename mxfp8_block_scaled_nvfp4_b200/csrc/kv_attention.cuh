// Attention over the paged block-scaled cache (kv_cache.cuh).
//
// Query i of sequence b (n queries over L cached tokens) is at position
// p = L - n + i and sees token j iff j < L, j <= p when causal, and
// j > p - window when window > 0:
//   z_j = scale * q . k_hat_j,  m = max z_j,  P_j = exp(z_j - m),
//   out = sum_j P_j v_hat_j / sum_j P_j,  lse = m + ln(sum_j P_j);
// a query that sees nothing gets out = 0 and lse = -inf.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "kv_cache.cuh"

namespace nvfp4 {
namespace kv {

struct AttnArgs {
  const uint8_t* codes[2];
  const uint8_t* scales[2];
  const float* g[2];
  const void* q;
  int64_t q_stride;             // elements between query tokens
  const int32_t* q_start;       // [B + 1] or NULL (query t belongs to sequence t)
  const int32_t* kv_len;        // [B]
  const int32_t* page_table;    // [B, max_pages]
  void* out;                    // [T, Hq, D]
  float* lse;                   // [T, Hq] or NULL
  float scale;
  uint32_t B, T, Hq, heads, G, D, max_q, max_kv, max_pages, num_pages, page_size;
  uint32_t window;              // 0: none
  int causal;
  int32_t chunk;                // tokens a CTA walks (a multiple of 16, at most 2^30)
  uint32_t chunks;              // CTAs a row tile has
  uint32_t tile_rows;           // query rows a CTA holds
  uint64_t scale_bytes;         // of one side
  float2* part_ml;              // [chunks, T, Hq]
  float* part_o;                // [chunks, T, Hq, D]
  FastDiv by_page;
};

// A sequence's queries and cached length; false (and the device error word)
// when its entries are outside what the call's sizes allow.
struct Seq {
  uint32_t t0, n, L;
};
__device__ __forceinline__ bool seq_of(const AttnArgs& a, uint32_t b, Seq& s) {
  int64_t t0 = b, t1 = (int64_t)b + 1;
  if (a.q_start) {
    t0 = __ldg(a.q_start + b);
    t1 = __ldg(a.q_start + b + 1);
  }
  const int64_t L = __ldg(a.kv_len + b);
  if (t0 < 0 || t1 < t0 || t1 > (int64_t)a.T || t1 - t0 > (int64_t)a.max_q || L < 0 || L > (int64_t)a.max_kv) {
    atomicOr(&g_device_error, (unsigned)kDevErrIndex);
    return false;
  }
  s.t0 = (uint32_t)t0;
  s.n = (uint32_t)(t1 - t0);
  s.L = (uint32_t)L;
  return true;
}

// ---------------------------------------------------------------------------
// Split work and partial results
// ---------------------------------------------------------------------------
// The tokens any of a row tile's queries can see are the range [lo, hi); it
// is walked in chunks of `chunk` tokens counted from lo rounded down to 16.
// A tile whose range takes one chunk is finished by its CTA; otherwise chunk c
// leaves (m, l, O) of every row -- O = sum 2^(z_j - m) v_j, l = sum
// 2^(z_j - m), logits z in units of log2 -- at index (c, t, h) of the
// partials, and k_kv_join adds them up.
struct Range {
  int32_t lo, hi;  // hi <= lo: nothing
};
__device__ __forceinline__ Range tile_range(const AttnArgs& a, const Seq& s, uint32_t i0, uint32_t i1) {
  Range r;
  // first and last query's positions; lengths and windows are at most 2^30
  const int32_t p0 = (int32_t)(s.L - s.n + i0), p1 = (int32_t)(s.L - s.n + i1);
  r.lo = a.window ? max(0, p0 - (int32_t)a.window + 1) : 0;
  r.hi = a.causal ? min((int32_t)s.L, p1 + 1) : (int32_t)s.L;
  return r;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 2^k, -126 <= k <= 127.
__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ---------------------------------------------------------------------------
// Few query rows: k_kv_decode
// ---------------------------------------------------------------------------
// The R = n * G rows (queries x heads of one group) of a sequence and a
// key/value head, 8 * NT of them a CTA; four warps take steps of 16 * TS
// tokens in turn, each with its own running maximum, and join at the end.
// Codes go from global memory straight into matrix fragments: a quad of lanes
// loads one token's key row (the order of the elements along D is free as
// long as q's fragments use the same), and a lane's share of a value row is
// the D / 8 consecutive elements of its fragment rows.
//   S^T [16 tokens x 8 rows] = K_hat . q^T      (m16n8k16, fp32)
//   O^T [16 elements x 8 rows] += V_hat^T . P^T
// P^T is S^T's fragment transposed by movmatrix.
//
// Number formats.  NVFP4: code * block scale has six significant bits and
// lies in [2^-10, 2688], so K_hat and V_hat are exact in fp16 (the global
// scales are factors of the logits and of the output).  A query row is scaled
// by a power of two to [2^14, 2^15) and rounds to fp16 exactly (elements
// 2^-28 below the row's largest lose bits that fp32 sums lose too); P is
// rounded to fp16 (2^-11 relative; the weights sum in fp32 unrounded).
// MX modes: code * 2^e spans fp32's exponents, so K_hat and V_hat are bf16
// (exact: at most four significant bits) times 2^-64; a query row is scaled
// to [2^40, 2^41) and split into two bf16 terms when it is fp16 (11 bits = 8
// + 3), and P, scaled by 2^32, into two bf16 terms (16 bits), so nothing
// rounds to fewer bits than fp16 would.
enum { kDecWarps = 4, kDecThreads = kDecWarps * 32 };

template <int MODE, int DP>
struct Geo {
  static constexpr int kbytes = DP / 4 * (int)Fmt<MODE>::bits / 8, kw = kbytes / 4;  // a lane's share of a key row
  static constexpr int vbytes = DP / 8 * (int)Fmt<MODE>::bits / 8, vw = vbytes / 4;  // and of a value row
  static constexpr int ksteps = DP / 16, mtiles = DP / 16;
  static constexpr int krow = DP * (int)Fmt<MODE>::bits / 8, srow = DP / (int)Fmt<MODE>::group;  // a row's bytes
  static constexpr int ts = (MODE == kMX8 || DP == 256) ? 1 : 2;  // 16-token tiles a step: what 255 registers hold
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The four bytes of a word as pairs of e2m1 codes: fp16 pairs (low nibble low).
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
}
// fp16 values of the two e4m3 bytes in the low half of a word.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(b));
  return r;
}
// Nibbles i and i + 4 of a word as bf16 pairs holding 2^-126 times the e2m1
// value: magnitude bits at bf16 bits 6-8, sign at 15 (as e2m1_value).
template <int I>
__device__ __forceinline__ uint32_t e2m1_pair_bf16(uint32_t w) {
  const uint32_t sg = I < 3 ? w << (12 - 4 * I) : w;
  const uint32_t mg = I < 2 ? w << (6 - 4 * I) : w >> (4 * I - 6);
  return (sg & 0x80008000u) | (mg & 0x01C001C0u);
}
// Bytes i and i + 2 of a word as bf16 pairs holding 2^-120 times the e4m3 value.
template <int I>
__device__ __forceinline__ uint32_t e4m3_pair_bf16(uint32_t w) {
  const uint32_t sg = I == 0 ? w << 8 : w;
  const uint32_t mg = I == 0 ? w << 4 : w >> 4;
  return (sg & 0x80008000u) | (mg & 0x07F007F0u);
}
// bf16 of 2^(s - 127 - 64 + up) for an e8m0 byte s (capped at 2^64), `up` the
// power of two that the pair functions above leave out (126 or 120): exponent
// field min(s, 191) - 64 + up, at most 253.
template <int MODE>
__device__ __forceinline__ uint32_t mx_factor(uint32_t s) {
  return (min(s, 191u) + (MODE == kMX8 ? 56u : 62u)) << 7;
}

template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (BYTES == 4) {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (BYTES == 8) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  }
}

// N scale bytes (N < 1: the byte that several lanes share).
template <int N>
__device__ __forceinline__ uint32_t load_scales(const uint8_t* p) {
  if constexpr (N <= 1) return __ldg(p);
  else if constexpr (N == 2) return __ldg(reinterpret_cast<const uint16_t*>(p));
  else return __ldg(reinterpret_cast<const uint32_t*>(p));
}

// A lane's key words and scales of one token row; `row` < 0 gives zeros.
// 32 elements (one piece) is what D is a multiple of.
template <int MODE, int DP>
__device__ __forceinline__ void load_key(const AttnArgs& a, int64_t row, uint32_t c, uint32_t* w, uint32_t& sc) {
  using G = Geo<MODE, DP>;
  constexpr uint32_t bits = Fmt<MODE>::bits, group = Fmt<MODE>::group, per = DP / 4;
  constexpr int piece = G::kbytes < (int)(4 * bits) ? G::kbytes : (int)(4 * bits);  // bytes of at most 32 elements
#pragma unroll
  for (int i = 0; i < G::kw; ++i) w[i] = 0;
  sc = 0;
  if (row < 0) return;
  const uint8_t* p = a.codes[0] + (uint64_t)row * (a.D * bits / 8u) + c * G::kbytes;
#pragma unroll
  for (int i = 0; i < G::kbytes / piece; ++i)
    if (c * per + 32u * i < a.D) load_words<piece>(p + i * piece, w + i * (piece / 4));
  const uint8_t* s = a.scales[0] + (uint64_t)row * (a.D / group);
  if constexpr (MODE == kNV) {
    if constexpr (DP == 64) {
      if (16u * c < a.D) sc = __ldg(s + c);
    } else {
#pragma unroll
      for (int i = 0; i < DP / 128; ++i)
        if (c * per + 32u * i < a.D)
          sc |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(s + c * (per / 16)) + i) << (16 * i);
    }
  } else if constexpr (DP == 64) {
    if (16u * c < a.D) sc = __ldg(s + c / 2);
  } else {
#pragma unroll
    for (int i = 0; i < DP / 128; ++i)
      if (c * per + 32u * i < a.D) sc |= (uint32_t)__ldg(s + c * (DP / 128) + i) << (8 * i);
  }
}

// A lane's value words and scales (byte 0, and byte 1 for a second block) of
// one token row.
template <int MODE, int DP>
__device__ __forceinline__ void load_value(const AttnArgs& a, int64_t row, uint32_t g, uint32_t* w, uint32_t& sc) {
  using G = Geo<MODE, DP>;
  constexpr uint32_t bits = Fmt<MODE>::bits, group = Fmt<MODE>::group, per = DP / 8;
#pragma unroll
  for (int i = 0; i < G::vw; ++i) w[i] = 0;
  sc = 0;
  if (row < 0 || g * per >= a.D) return;
  load_words<G::vbytes>(a.codes[1] + (uint64_t)row * (a.D * bits / 8u) + g * G::vbytes, w);
  const uint8_t* s = a.scales[1] + (uint64_t)row * (a.D / group);
  if constexpr (MODE == kNV && DP == 256)
    sc = __ldg(reinterpret_cast<const uint16_t*>(s) + g);
  else
    sc = __ldg(s + g * per / group);
}

// FAST: D == DP, 16-token tiles lie on one page and rows have 32-bit numbers;
// a step wholly inside the range then loads without a check at fixed offsets
// from one row.  Everything else looks each row up.
template <typename QT, int MODE, int DP, int NT, bool FAST>
struct Decode {
  using G = Geo<MODE, DP>;
  static constexpr int TS = G::ts;
  static constexpr bool kSplitQ = MODE != kNV && std::is_same<QT, __half>::value;
  static constexpr bool kMx = MODE != kNV;

  uint32_t qf[NT][G::ksteps][2], ql[kSplitQ ? NT : 1][kSplitQ ? G::ksteps : 1][2];
  float fz[NT][2];     // logit (log2 units) of an accumulator, for this lane's two columns
  float m[NT][2], l[NT][2];
  float o[NT][G::mtiles][4];
  uint32_t kw[TS][2][G::kw], ks[TS][2], vw[TS][4][G::vw], vs[TS][4];
  uint32_t lane, g, c;

  // Element (within the lane's DP / 4) of k-step s, fragment register j, half e.
  __device__ static constexpr int q_elem(int s, int j, int e) {
    return MODE == kNV ? 4 * s + 2 * j + e : MODE == kMX4 ? 8 * (s / 2) + 2 * (s % 2) + j + 4 * e : 4 * s + j + 2 * e;
  }

  __device__ __forceinline__ void load_q(const AttnArgs& a, const Seq& sq, uint32_t hk, uint32_t r0, uint32_t R) {
    const float gk = a.g[0] ? __ldg(a.g[0]) / kGlobalEncode : 1.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t r = r0 + 8u * nt + g;
      float v[DP / 4];
#pragma unroll
      for (int i = 0; i < DP / 4; ++i) v[i] = 0.0f;
      if (r < R) {
        const uint32_t i = r / a.G, h = hk * a.G + (r - i * a.G);
        const QT* q = static_cast<const QT*>(a.q) + (int64_t)(sq.t0 + i) * a.q_stride + (int64_t)h * a.D + c * (DP / 4);
#pragma unroll
        for (int k = 0; k < DP / 32; ++k)
          if (c * (DP / 4) + 8u * k < a.D) {
            float x[8];
            load8<QT>(q + 8 * k, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * k + e] = x[e];
          }
      }
      float mx = 0.0f;
#pragma unroll
      for (int i = 0; i < DP / 4; ++i) mx = fmaxf(mx, fabsf(v[i]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // 2^e <= mx < 2^(e+1), kept where every factor below is normal
      const int e = mx > 0.0f ? max(-80, (int)((__float_as_uint(mx) >> 23) & 255u) - 127) : 0;
      constexpr int top = kMx ? 40 : 14;
      const float up = pow2(top - e) * (a.scale < 0.0f ? -1.0f : 1.0f);
#pragma unroll
      for (int s = 0; s < G::ksteps; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float x = v[q_elem(s, j, 0)] * up, y = v[q_elem(s, j, 1)] * up;
          if constexpr (!kMx) {
            qf[nt][s][j] = pack_f16x2(x, y);
          } else {
            const uint32_t hi = pack_bf16x2(x, y);
            qf[nt][s][j] = hi;
            if constexpr (kSplitQ)
              ql[nt][s][j] = pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
          }
        }
      // row 8 nt + g's factor, wanted by the lanes of columns 2c, 2c + 1
      const float f = fmaxf(fabsf(a.scale) * kLog2e * pow2(e) * gk * pow2(kMx ? 24 : -14), 1e-37f);
      fz[nt][0] = __shfl_sync(0xffffffffu, f, 8 * c);
      fz[nt][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
    }
  }

  // Row of token j, or -1 where it is outside [lo, hi) or its page is not one.
  __device__ __forceinline__ int64_t row_at(const AttnArgs& a, const int32_t* table, uint32_t hk, int32_t j, const Range& rg) const {
    if (j < rg.lo || j >= rg.hi) return -1;
    const uint32_t pg = a.by_page.div((uint32_t)j);
    const int32_t page = __ldg(table + pg);
    if (page < 0 || (uint32_t)page >= a.num_pages) {
      atomicOr(&g_device_error, (unsigned)kDevErrIndex);
      return -1;
    }
    return (int64_t)(((uint64_t)page * a.heads + hk) * a.page_size + ((uint32_t)j - pg * a.page_size));
  }
  // FAST: row of token 0 of a 16-token tile on page `page`.
  __device__ __forceinline__ uint32_t tile_row(const AttnArgs& a, int32_t page, uint32_t hk, int32_t j0) const {
    return ((uint32_t)page * a.heads + hk) * a.page_size + ((uint32_t)j0 - a.by_page.div((uint32_t)j0) * a.page_size);
  }

  // Bit 2t + i of the result: token 16 t + 8 i + g of the step is there.
  __device__ __forceinline__ uint32_t load_keys(const AttnArgs& a, const int32_t* table, uint32_t hk, int32_t j0, const Range& rg,
                                                bool inside, const uint32_t (&rows)[TS]) {
    if (FAST && inside) {
#pragma unroll
      for (int t = 0; t < TS; ++t) {
        const uint8_t* p = a.codes[0] + (uint64_t)(rows[t] + g) * G::krow + c * G::kbytes;
        const uint8_t* q = a.scales[0] + (uint64_t)(rows[t] + g) * G::srow + c * (DP / 4) / Fmt<MODE>::group;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          load_words<G::kbytes>(p + 8 * i * G::krow, kw[t][i]);
          ks[t][i] = load_scales<DP / 4 / Fmt<MODE>::group>(q + 8 * i * G::srow);
        }
      }
      return (1u << (2 * TS)) - 1u;
    }
    uint32_t there = 0;
#pragma unroll
    for (int t = 0; t < TS; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t row = row_at(a, table, hk, j0 + 16 * t + 8 * i + g, rg);
        there |= (row >= 0 ? 1u : 0u) << (2 * t + i);
        load_key<MODE, DP>(a, row, c, kw[t][i], ks[t][i]);
      }
    return there;
  }
  __device__ __forceinline__ void load_values(const AttnArgs& a, const int32_t* table, uint32_t hk, int32_t j0, const Range& rg,
                                              bool inside, const uint32_t (&rows)[TS]) {
    if (FAST && inside) {
#pragma unroll
      for (int t = 0; t < TS; ++t) {
        const uint8_t* p = a.codes[1] + (uint64_t)(rows[t] + 2 * c) * G::krow + g * G::vbytes;
        const uint8_t* q = a.scales[1] + (uint64_t)(rows[t] + 2 * c) * G::srow + g * (DP / 8) / Fmt<MODE>::group;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = (i & 1) + 8 * (i >> 1);
          load_words<G::vbytes>(p + x * G::krow, vw[t][i]);
          vs[t][i] = load_scales<DP / 8 / Fmt<MODE>::group>(q + x * G::srow);
        }
      }
      return;
    }
#pragma unroll
    for (int t = 0; t < TS; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = row_at(a, table, hk, j0 + 16 * t + 2 * c + (i & 1) + 8 * (i >> 1), rg);
        load_value<MODE, DP>(a, row, g, vw[t][i], vs[t][i]);
      }
  }

  __device__ __forceinline__ void step_mma(float (&s)[NT][4], int ks_, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (!kMx) {
        mma_f16(s[nt], a0, a1, a2, a3, qf[nt][ks_][0], qf[nt][ks_][1]);
      } else {
        mma_bf16(s[nt], a0, a1, a2, a3, qf[nt][ks_][0], qf[nt][ks_][1]);
        if constexpr (kSplitQ) mma_bf16(s[nt], a0, a1, a2, a3, ql[nt][ks_][0], ql[nt][ks_][1]);
      }
    }
  }

  // S^T of tile t.
  __device__ __forceinline__ void logits(int t, float (&s)[NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
    if constexpr (MODE == kNV) {
      uint32_t sc[2][DP / 64];  // fp16 pairs (s, s) of the lane's blocks
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int b = 0; b < DP / 64; b += 2) {
          const uint32_t p = e4m3x2_to_f16x2(ks[t][i] >> (8 * b));
          sc[i][b] = __byte_perm(p, 0, 0x1010);
          if (b + 1 < DP / 64) sc[i][b + 1] = __byte_perm(p, 0, 0x3232);
        }
#pragma unroll
      for (int w = 0; w < G::kw; ++w) {
        uint32_t x[4], y[4];
        e2m1x8_to_f16x2(kw[t][0][w], x);
        e2m1x8_to_f16x2(kw[t][1][w], y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = mul_f16x2(x[e], sc[0][w / 2]);
          y[e] = mul_f16x2(y[e], sc[1][w / 2]);
        }
        step_mma(s, 2 * w, x[0], y[0], x[1], y[1]);
        step_mma(s, 2 * w + 1, x[2], y[2], x[3], y[3]);
      }
    } else {
      constexpr int wpb = 32 * (int)Fmt<MODE>::bits / 32;  // words a block
      uint32_t f[2] = {0, 0};
#pragma unroll
      for (int w = 0; w < G::kw; ++w) {
        if (w % wpb == 0)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            f[i] = mx_factor<MODE>((ks[t][i] >> (8 * (w / wpb))) & 255u);
            f[i] |= f[i] << 16;
          }
        const uint32_t a = kw[t][0][w], b = kw[t][1][w];
        if constexpr (MODE == kMX4) {
          step_mma(s, 2 * w, mul_bf16x2(e2m1_pair_bf16<0>(a), f[0]), mul_bf16x2(e2m1_pair_bf16<0>(b), f[1]),
                   mul_bf16x2(e2m1_pair_bf16<1>(a), f[0]), mul_bf16x2(e2m1_pair_bf16<1>(b), f[1]));
          step_mma(s, 2 * w + 1, mul_bf16x2(e2m1_pair_bf16<2>(a), f[0]), mul_bf16x2(e2m1_pair_bf16<2>(b), f[1]),
                   mul_bf16x2(e2m1_pair_bf16<3>(a), f[0]), mul_bf16x2(e2m1_pair_bf16<3>(b), f[1]));
        } else {
          step_mma(s, w, mul_bf16x2(e4m3_pair_bf16<0>(a), f[0]), mul_bf16x2(e4m3_pair_bf16<0>(b), f[1]),
                   mul_bf16x2(e4m3_pair_bf16<1>(a), f[0]), mul_bf16x2(e4m3_pair_bf16<1>(b), f[1]));
        }
      }
    }
  }

  __device__ __forceinline__ void out_mma(int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          const uint32_t (&ph)[NT][2], const uint32_t (&pl)[NT][2]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (!kMx) {
        mma_f16(o[nt][mt], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
      } else {
        mma_bf16(o[nt][mt], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
        mma_bf16(o[nt][mt], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
      }
    }
  }

  // O^T += V_hat^T . P^T of tile t; fragment rows g and g + 8 of m-tile mt are
  // elements (DP / 8) g + 2 mt and the next.
  __device__ __forceinline__ void weigh(int t, const uint32_t (&ph)[NT][2], const uint32_t (&pl)[NT][2]) {
    if constexpr (MODE == kNV) {
#pragma unroll
      for (int w = 0; w < G::vw; ++w) {
        constexpr int wpb = 2;  // words a block
        const int b = DP == 256 ? w / wpb : 0;
        const uint32_t s01 = e4m3x2_to_f16x2(__byte_perm(vs[t][0], vs[t][1], b ? 0x0051 : 0x0040));
        const uint32_t s23 = e4m3x2_to_f16x2(__byte_perm(vs[t][2], vs[t][3], b ? 0x0051 : 0x0040));
        const uint32_t lo = 0x0F0F0F0Fu;
        uint32_t x01[4], y01[4], x23[4], y23[4];
        const uint32_t v0 = vw[t][0][w], v1 = vw[t][1][w], v2 = vw[t][2][w], v3 = vw[t][3][w];
        e2m1x8_to_f16x2((v0 & lo) | ((v1 << 4) & ~lo), x01);
        e2m1x8_to_f16x2(((v0 >> 4) & lo) | (v1 & ~lo), y01);
        e2m1x8_to_f16x2((v2 & lo) | ((v3 << 4) & ~lo), x23);
        e2m1x8_to_f16x2(((v2 >> 4) & lo) | (v3 & ~lo), y23);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          out_mma(4 * w + e, mul_f16x2(x01[e], s01), mul_f16x2(y01[e], s01), mul_f16x2(x23[e], s23),
                  mul_f16x2(y23[e], s23), ph, pl);
      }
    } else {
      const uint32_t f01 = mx_factor<MODE>(vs[t][0]) | (mx_factor<MODE>(vs[t][1]) << 16);
      const uint32_t f23 = mx_factor<MODE>(vs[t][2]) | (mx_factor<MODE>(vs[t][3]) << 16);
#pragma unroll
      for (int w = 0; w < G::vw; ++w)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t sel = hf ? 0x7632u : 0x5410u;
          const uint32_t u = __byte_perm(vw[t][0][w], vw[t][1][w], sel), v = __byte_perm(vw[t][2][w], vw[t][3][w], sel);
          if constexpr (MODE == kMX4) {
            out_mma(4 * w + 2 * hf, mul_bf16x2(e2m1_pair_bf16<0>(u), f01), mul_bf16x2(e2m1_pair_bf16<1>(u), f01),
                    mul_bf16x2(e2m1_pair_bf16<0>(v), f23), mul_bf16x2(e2m1_pair_bf16<1>(v), f23), ph, pl);
            out_mma(4 * w + 2 * hf + 1, mul_bf16x2(e2m1_pair_bf16<2>(u), f01), mul_bf16x2(e2m1_pair_bf16<3>(u), f01),
                    mul_bf16x2(e2m1_pair_bf16<2>(v), f23), mul_bf16x2(e2m1_pair_bf16<3>(v), f23), ph, pl);
          } else {
            out_mma(2 * w + hf, mul_bf16x2(e4m3_pair_bf16<0>(u), f01), mul_bf16x2(e4m3_pair_bf16<1>(u), f01),
                    mul_bf16x2(e4m3_pair_bf16<0>(v), f23), mul_bf16x2(e4m3_pair_bf16<1>(v), f23), ph, pl);
          }
        }
    }
  }
};

template <typename QT, int MODE, int DP, int NT, bool FAST>
__global__ void __launch_bounds__(kDecThreads) k_kv_decode(const __grid_constant__ AttnArgs a) {
  using D = Decode<QT, MODE, DP, NT, FAST>;
  constexpr int TS = D::TS, MT = D::G::mtiles, STEP = 16 * TS, ROWS = 8 * NT;
  __shared__ float sm[kDecWarps][ROWS], sl[kDecWarps][ROWS];
  __shared__ float so[kDecWarps / 2][ROWS * DP];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t tile = blockIdx.x / a.chunks, chunk = blockIdx.x - tile * a.chunks, hk = blockIdx.y, b = blockIdx.z;
  const uint32_t r0 = tile * ROWS;
  Seq s;
  if (!seq_of(a, b, s)) return;
  const uint32_t R = s.n * a.G;
  if (r0 >= R) return;
  const uint32_t i0 = r0 / a.G, i1 = (min(r0 + ROWS, R) - 1u) / a.G;
  const Range rg = tile_range(a, s, i0, i1);
  const int32_t base = rg.lo & ~15;
  const int32_t span = rg.hi > rg.lo ? rg.hi - base : 0;
  if (chunk > 0 && (int64_t)chunk * a.chunk >= span) return;
  const bool whole = span <= a.chunk;
  const int32_t begin = base + (int32_t)chunk * a.chunk;
  const int32_t end = min(rg.hi, begin + a.chunk);
  const Range here{rg.lo, end};
  const int32_t* table = a.page_table + (uint64_t)b * a.max_pages;

  D d;
  d.lane = lane;
  d.g = lane >> 2;
  d.c = lane & 3u;
  d.load_q(a, s, hk, r0, R);
  // what this lane's columns (rows r0 + 8 nt + 2c, + 1) see
  int32_t see_lo[NT][2], see_hi[NT][2];
  int32_t all_lo = rg.lo, all_hi = end;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t i = min(r0 + 8u * nt + 2u * d.c + e, R - 1u) / a.G;
      const Range r = tile_range(a, s, i, i);
      see_lo[nt][e] = r.lo;
      see_hi[nt][e] = r.hi;
      d.m[nt][e] = -INFINITY;
      d.l[nt][e] = 0.0f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) d.o[nt][mt][2 * e] = d.o[nt][mt][2 * e + 1] = 0.0f;
    }
  // tokens every row of the tile sees
  if (a.window) all_lo = tile_range(a, s, i1, i1).lo;
  if (a.causal) all_hi = min(end, tile_range(a, s, i0, i0).hi);

  // The loads of the next step are issued as soon as this one's registers are
  // free: keys after the logits, values after the weighted sum; the page
  // numbers a step earlier still.
  int32_t j0 = begin + (int32_t)warp * STEP;
  int32_t pages[TS];
  auto look = [&](int32_t j) {
#pragma unroll
    for (int t = 0; t < TS; ++t) pages[t] = FAST && j + 16 * t < end ? __ldg(table + a.by_page.div((uint32_t)(j + 16 * t))) : -1;
  };
  uint32_t rows[TS];
  bool inside = false;
  auto find = [&](int32_t j) {
    inside = FAST && j >= rg.lo && j + STEP <= end;
#pragma unroll
    for (int t = 0; t < TS; ++t) {
      inside = inside && (uint32_t)pages[t] < a.num_pages;
      rows[t] = d.tile_row(a, pages[t], hk, j + 16 * t);
    }
  };
  uint32_t there = 0;
  if (j0 < end) {
    look(j0);
    find(j0);
    look(j0 + kDecWarps * STEP);
    there = d.load_keys(a, table, hk, j0, here, inside, rows);
    d.load_values(a, table, hk, j0, here, inside, rows);
  }
  for (; j0 < end; j0 += kDecWarps * STEP) {
    const int32_t jn = j0 + kDecWarps * STEP;
    const uint32_t now = there;
    float sv[TS][NT][4];
#pragma unroll
    for (int t = 0; t < TS; ++t) d.logits(t, sv[t]);
    if (jn < end) {
      find(jn);
      look(jn + kDecWarps * STEP);
      there = d.load_keys(a, table, hk, jn, here, inside, rows);
    }
    const bool full = __all_sync(0xffffffffu, now == (1u << (2 * TS)) - 1u) && j0 >= all_lo && j0 + STEP <= all_hi;
    if (!full) {
#pragma unroll
      for (int t = 0; t < TS; ++t)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int32_t j = j0 + 16 * t + 8 * (e >> 1) + d.g;
            if (!((now >> (2 * t + (e >> 1))) & 1u) || j < see_lo[nt][e & 1] || j >= see_hi[nt][e & 1]) sv[t][nt][e] = -INFINITY;
          }
    }
    // The running maximum moves only when a step exceeds it by 2^8 (weights
    // then lie below 2^8, which fp16 and the sums hold as well as below 1).
    float top[NT][2];
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = -INFINITY;
#pragma unroll
        for (int t = 0; t < TS; ++t) x = fmaxf(x, fmaxf(sv[t][nt][e], sv[t][nt][2 + e]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        top[nt][e] = x * d.fz[nt][e] - (D::kMx ? 32.0f : 0.0f);
        grow = grow || top[nt][e] > d.m[nt][e] + 8.0f;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(d.m[nt][e], top[nt][e]);
          const float f = mn == -INFINITY ? 1.0f : ex2(d.m[nt][e] - mn);
          d.m[nt][e] = mn;
          d.l[nt][e] *= f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            d.o[nt][mt][e] *= f;
            d.o[nt][mt][2 + e] *= f;
          }
        }
    }
    float ref[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) ref[nt][e] = d.m[nt][e] == -INFINITY ? 0.0f : d.m[nt][e];
#pragma unroll
    for (int t = 0; t < TS; ++t) {
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = ex2(fmaf(sv[t][nt][e], d.fz[nt][e & 1], -ref[nt][e & 1]));
          d.l[nt][e & 1] += p[e];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (!D::kMx) {
            ph[nt][i] = transpose8x8(pack_f16x2(p[2 * i], p[2 * i + 1]));
          } else {
            const uint32_t hi = pack_bf16x2(p[2 * i], p[2 * i + 1]);
            const uint32_t lo = pack_bf16x2(p[2 * i] - __uint_as_float(hi << 16), p[2 * i + 1] - __uint_as_float(hi & 0xFFFF0000u));
            ph[nt][i] = transpose8x8(hi);
            pl[nt][i] = transpose8x8(lo);
          }
        }
      }
      d.weigh(t, ph, pl);
    }
    if (jn < end) d.load_values(a, table, hk, jn, here, inside, rows);
  }

  // Join the warps: a common maximum first, then the sums, two warps at a time.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float& l = d.l[nt][e];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      if (d.g == 0) sm[warp][8 * nt + 2 * d.c + e] = d.m[nt][e];
    }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, sm[w][8 * nt + 2 * d.c + e]);
      const float f = d.m[nt][e] == -INFINITY ? 0.0f : ex2(d.m[nt][e] - M);
      d.m[nt][e] = M;
      d.l[nt][e] *= f;
      if (d.g == 0) sl[warp][8 * nt + 2 * d.c + e] = d.l[nt][e];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        d.o[nt][mt][e] *= f;
        d.o[nt][mt][2 + e] *= f;
      }
    }
#pragma unroll
  for (int half = kDecWarps / 2; half > 0; half >>= 1) {
    if (warp >= (uint32_t)half && warp < 2u * half) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          reinterpret_cast<float4*>(so[warp - half])[(nt * MT + mt) * 32 + lane] =
              make_float4(d.o[nt][mt][0], d.o[nt][mt][1], d.o[nt][mt][2], d.o[nt][mt][3]);
    }
    __syncthreads();
    if (warp < (uint32_t)half) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const float4 v = reinterpret_cast<const float4*>(so[warp])[(nt * MT + mt) * 32 + lane];
          d.o[nt][mt][0] += v.x;
          d.o[nt][mt][1] += v.y;
          d.o[nt][mt][2] += v.z;
          d.o[nt][mt][3] += v.w;
        }
    }
    __syncthreads();
  }
  if (warp != 0) return;
  const float fv = D::kMx ? 0x1p64f : (a.g[1] ? __ldg(a.g[1]) / kGlobalEncode : 1.0f);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t r = r0 + 8u * nt + 2u * d.c + e;
      if (r >= R) continue;
      float l = 0.0f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) l += sl[w][8 * nt + 2 * d.c + e];
      const uint32_t i = r / a.G, h = hk * a.G + (r - i * a.G);
      const uint64_t at = (uint64_t)(s.t0 + i) * a.Hq + h;
      const float f = whole ? (l > 0.0f ? fv / l : 0.0f) : fv;
      if (whole) {
        if (a.lse && d.g == 0) a.lse[at] = l > 0.0f ? (d.m[nt][e] + log2f(l)) * kLn2 : -INFINITY;
      } else if (d.g == 0) {
        a.part_ml[(uint64_t)chunk * a.T * a.Hq + at] = make_float2(d.m[nt][e], l);
      }
#pragma unroll
      for (int k = 0; k < DP / 64; ++k) {  // eight elements: m-tiles 4k .. 4k + 3
        const uint32_t el = d.g * (DP / 8) + 8u * k;
        if (el >= a.D) continue;
        float v[8];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          v[2 * x] = d.o[nt][4 * k + x][e] * f;
          v[2 * x + 1] = d.o[nt][4 * k + x][2 + e] * f;
        }
        if (whole)
          store8<QT>(static_cast<QT*>(a.out) + at * a.D + el, v);
        else
          store8<float>(a.part_o + ((uint64_t)chunk * a.T * a.Hq + at) * a.D + el, v);
      }
    }
}

// Join of the partial results of one (query, head): one CTA, a warp for every
// fourth chunk, the row's elements over the lanes.
constexpr int kJoinWarps = 4;
template <typename QT>
__global__ void __launch_bounds__(kJoinWarps * 32) k_kv_join(const __grid_constant__ AttnArgs a) {
  __shared__ float sl[kJoinWarps];
  __shared__ float so[kJoinWarps][256];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  Seq s;
  if (!seq_of(a, b, s) || i >= s.n) return;
  // the row tile this query's row was in
  const uint32_t r0 = (i * a.G + h % a.G) / a.tile_rows * a.tile_rows;
  const uint32_t r1 = min(r0 + a.tile_rows, s.n * a.G) - 1u;
  const Range rg = tile_range(a, s, r0 / a.G, r1 / a.G);
  const int32_t span = rg.hi > rg.lo ? rg.hi - (rg.lo & ~15) : 0;
  if (span <= a.chunk) return;  // finished by its CTA
  const uint32_t nc = ((uint32_t)span + a.chunk - 1u) / a.chunk;
  const uint64_t at = (uint64_t)(s.t0 + i) * a.Hq + h, step = (uint64_t)a.T * a.Hq;
  float m = -INFINITY;
  for (uint32_t c = lane; c < nc; c += 32) m = fmaxf(m, __ldg(&a.part_ml[c * step + at].x));
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  float l = 0.0f, o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.0f;
  const uint32_t d0 = lane * 8u;
#pragma unroll 4
  for (uint32_t c = warp; c < nc; c += kJoinWarps) {
    const float2 ml = __ldg(&a.part_ml[c * step + at]);
    const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - m);
    l += ml.y * f;
    if (d0 < a.D) {
      float v[8];
      load8<float>(a.part_o + (c * step + at) * a.D + d0, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(v[e], f, o[e]);
    }
  }
  if (lane == 0) sl[warp] = l;
  if (d0 < a.D) store8<float>(&so[warp][d0], o);
  __syncthreads();
  if (warp != 0) return;
  l = 0.0f;
  for (int w = 0; w < kJoinWarps; ++w) l += sl[w];
  if (a.lse && lane == 0) a.lse[at] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
  if (d0 >= a.D) return;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = 0.0f;
    for (int w = 0; w < kJoinWarps; ++w) v[e] += so[w][d0 + e];
    v[e] = l > 0.0f ? v[e] / l : 0.0f;
  }
  store8<QT>(static_cast<QT*>(a.out) + at * a.D + d0, v);
}

}  // namespace kv
}  // namespace nvfp4
