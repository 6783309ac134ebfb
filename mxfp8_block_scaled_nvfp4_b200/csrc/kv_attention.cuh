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
#include "qqmm_sm100.cuh"

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
  int32_t chunk;                // k_kv_prefill: tokens a CTA walks (a multiple of 16, at most 2^30)
  uint32_t chunks;              // CTAs a row tile has
  uint32_t tile_rows;           // query rows a CTA holds
  int split;                    // k_kv_decode: 0 where there is no workspace
  uint64_t scale_bytes;         // of one side
  float2* part_ml;              // [chunks, T, Hq]; k_kv_decode: [workers, 2, rows]
  float* part_o;                // [chunks, T, Hq, D]; [workers, 2, rows, D]
  int4* part_head;              // k_kv_decode: [workers]
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
// Ranges and partial results
// ---------------------------------------------------------------------------
// The tokens any of a row tile's queries can see are the range [lo, hi).
// Where several CTAs walk one range, each leaves (m, l, O) of every row --
// O = sum 2^(z_j - m) v_j, l = sum 2^(z_j - m), logits z in units of log2 --
// and a second kernel adds them up.
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

// ln of a row's sum; a row that saw nothing has l = 0, one with a NaN logit
// (a NaN in its query) l = NaN.
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2; }

// The weights are kept times 2^kUp, so that their 16-bit terms (and, in the MX
// modes, the products with very small values) keep their bits.  They reach 2^8
// times that, which fp16 (2^16) and the sums over 2^30 tokens of values below
// 2^73 (2^128) have to hold.
template <int MODE>
constexpr float kUp = MODE == kNV ? 7.0f : 16.0f;

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
// key/value head are cut into tiles of 8 * NT; a tile walks its tokens in
// units of 64 * TS.  All units of all (sequence, tile, head) in that order
// are dealt out in equal runs to as many CTAs as fit the GPU at once, so
// uneven lengths, few heads and one long sequence fill the SMs alike (with a
// grid of equal chunks the last wave stood half empty: one sequence of
// 131072 tokens took 55 us in 2.4 waves, 47 us in one).  A run begins and
// ends anywhere in a range: what it does not cover whole goes to
// k_kv_decode_join.
//
// In a CTA a fifth warp copies the units ahead into shared memory, so loads
// cost the other four neither instructions nor registers: one bulk copy a page
// (or piece of one) and part (K and V codes, K and V scales).  Each of the four
// takes 16 * TS tokens of every unit, with its own running maximum, and they
// join at the end of a range.  Codes go from shared memory straight into
// matrix fragments: a quad of lanes holds one token's key row (the order of
// the elements along D is free as long as q's fragments use the same), and a
// lane's share of a value row is the D / 8 consecutive elements of its
// fragment rows.
//   S^T [16 tokens x 8 rows] = K_hat . q^T      (m16n8k16, fp32)
//   O^T [16 elements x 8 rows] += V_hat^T . P^T
// P^T is S^T's fragment transposed by movmatrix.
//
// Measured (NVFP4, 32 query and 8 key/value heads of 128), in a captured graph:
// 32 x 32768 tokens 196 us, 4.67 TB/s or 71 % of the copy rate; 1 x 131072
// 46 us, of which 5 are spent up to the first unit (lengths, page table, codes:
// three loads one after the other) and 3 in the join.  Calls on a stream take 2
// to 4 us more each (the gap between launches), and seconds of the first case on
// end 214 us: the 1000 W power cap takes the SM clock from 1965 to 1820 MHz.
// Bound by memory and by the decoding instructions (660 for 32 tokens, the ALU
// pipe half busy) alike.
//
// Number formats.  NVFP4: code * block scale has six significant bits and
// lies in [2^-10, 2688], so K_hat and V_hat are exact in fp16 (the global
// scales are factors of the logits and of the output).  A query row is scaled
// by a power of two to [2^14, 2^15) and rounds to fp16 exactly (elements
// 2^-28 below the row's largest lose bits that fp32 sums lose too).  P, times
// 2^7, is rounded to fp16: 16 bits are what one product per code takes, and
// bf16 or fp16 outputs have no more.  That is 2^-11 relative down to weights
// of 2^-21 of the reference, then half a step of fp16's subnormals, 2^-32 of
// it (2^-25 without the factor: 131072 tokens that light beside a heavy one
// lost 2^-8 of the output).  The weights sum in fp32 unrounded.
// MX modes: code * 2^e spans fp32's exponents, so K_hat and V_hat are bf16
// (exact: at most four significant bits; bf16's subnormals end at 2^-133, so
// elements below that, MXFP4 keys below 2^-109, round to multiples of it).  A query
// row is scaled to [2^16, 2^17) and split into two bf16 terms when it is fp16
// (11 bits = 8 + 3), and P, times 2^16, into two bf16 terms (16 bits), so
// nothing rounds to fewer bits than fp16 would.  With scales of at most 2^64
// and 2^30 tokens every sum stays below 2^127.
enum { kDecWarps = 4, kDecThreads = (kDecWarps + 1) * 32 };

template <int MODE, int DP>
struct Geo {
  static constexpr int kbytes = DP / 4 * (int)Fmt<MODE>::bits / 8, kw = kbytes / 4;  // a lane's share of a key row
  static constexpr int vbytes = DP / 8 * (int)Fmt<MODE>::bits / 8, vw = vbytes / 4;  // and of a value row
  static constexpr int ksteps = DP / 16, mtiles = DP / 16;
  static constexpr int krow = DP * (int)Fmt<MODE>::bits / 8, srow = DP / (int)Fmt<MODE>::group;  // a row's bytes
  // 16-token tiles of a warp in a unit, units in shared memory: 34 to 66 KB of
  // them a CTA.  With the fp32 output tiles of the four warps that is 45 to 73 KB
  // (three CTAs an SM) for 8 rows of D <= 128, 53 to 100 KB (two, or one where
  // the registers end first) for 16 rows and for D 256.
  static constexpr int ts = DP == 256 || (MODE == kMX8 && DP == 128) ? 1 : 2;
  static constexpr int unit = 16 * kDecWarps * ts, unit_bytes = 2 * unit * (krow + srow);
  static constexpr int stages = unit_bytes > 26000 ? 2 : unit_bytes > 12000 ? 3 : 4;
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
// The NaN codes (0x7F, 0xFF) read as +-480: finite, so that a weight of zero
// hides them from the queries that do not see their token.  Carrying a NaN to
// those that do costs a check of every code (in the best ways tried 16 x 8192 of
// D 128 took 59.8 us for 58.0, 8 x 6000 of D 256 59.6 for 55.5), for inputs that
// the library leaves open.
template <int I>
__device__ __forceinline__ uint32_t e4m3_pair_bf16(uint32_t w) {
  const uint32_t sg = I == 0 ? w << 8 : w;
  const uint32_t mg = I == 0 ? w << 4 : w >> 4;
  return (sg & 0x80008000u) | (mg & 0x07F007F0u);
}
// MX values take the power of two that the pair functions leave out (2^126,
// 2^120) and the block scale 2^(s - 127), s an e8m0 byte capped at 2^64.  As one
// factor they are a bf16 number up to a scale of 2 (MXFP4) or 2^7 (MXFP8); a
// smaller factor for all would lose small blocks.  So they are two products,
// but for MXFP4 tiles without a larger scale (not BIG): 16 x 8192 tokens 49.2 us
// where two products everywhere take 52.0.  MXFP4 keys, which outlying channels
// put above that, are held times 2^-24, so that 2^25 is their border.  MXFP8
// gains nothing (8 x 6000 of D 256: 64.8 us with the choice, 55.3 without).
template <int MODE>
struct Mx {
  static constexpr uint32_t left_out = MODE == kMX8 ? 120 : 126;
  static constexpr int key_down = MODE == kMX4 ? 24 : 0;  // keys are held times 2^-key_down
  // of a key or a value
  __device__ static constexpr uint32_t up(bool key) { return left_out - (key ? key_down : 0); }
  __device__ static constexpr uint32_t largest(bool key) { return 254u - up(key); }  // scale byte that one factor holds
};
// A block's factor; in a BIG tile what the pair functions leave out is another.
template <bool BIG>
__device__ __forceinline__ uint32_t mx_factor(uint32_t s, uint32_t up) {
  return BIG ? max(min(s, 191u) << 7, 0x40u) : (s + up) << 7;
}
// Nibbles i and i + 4 (MXFP4) or bytes i and i + 2 (MXFP8) of a word times the
// pair f of factors.
template <int MODE, int I, bool BIG>
__device__ __forceinline__ uint32_t mx_pair(uint32_t w, uint32_t f, uint32_t up) {
  uint32_t p;
  if constexpr (MODE == kMX8) p = e4m3_pair_bf16<I>(w);
  else p = e2m1_pair_bf16<I>(w);
  if constexpr (BIG) p = mul_bf16x2(p, (up + 127u) * 0x00800080u);
  return mul_bf16x2(p, f);
}

template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (BYTES == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (BYTES == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
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
  if constexpr (N <= 1) return *p;
  else if constexpr (N == 2) return *reinterpret_cast<const uint16_t*>(p);
  else return *reinterpret_cast<const uint32_t*>(p);
}

// EXACT: D == DP; otherwise a row's elements beyond D read as zero.
template <typename QT, int MODE, int DP, int NT, bool EXACT>
struct Decode {
  using G = Geo<MODE, DP>;
  static constexpr int TS = G::ts;
  static constexpr bool kSplitQ = MODE != kNV && std::is_same<QT, __half>::value;
  static constexpr bool kMx = MODE != kNV;

  uint32_t qf[NT][G::ksteps][2], ql[kSplitQ ? NT : 1][kSplitQ ? G::ksteps : 1][2];
  float fz[NT][2];     // logit (log2 units) of an accumulator, for this lane's two columns
  float m[NT][2], l[NT][2];
  float o[NT][G::mtiles][4];
  uint32_t lane, g, c;
  uint32_t rb, sb, D;  // a row's code and scale bytes, elements

  // Element (within the lane's DP / 4) of k-step s, fragment register j, half e.
  __device__ static constexpr int q_elem(int s, int j, int e) {
    return MODE == kNV ? 4 * s + 2 * j + e : MODE == kMX4 ? 8 * (s / 2) + 2 * (s % 2) + j + 4 * e : 4 * s + j + 2 * e;
  }

  __device__ __forceinline__ void load_q(const AttnArgs& a, const Seq& sq, uint32_t hk, uint32_t r0, uint32_t R, float gk) {
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
      constexpr int top = kMx ? 16 : 14;
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
      const float f = fmaxf(fabsf(a.scale) * kLog2e * pow2(e) * gk * pow2(Mx<MODE>::key_down - top), 1e-37f);
      fz[nt][0] = __shfl_sync(0xffffffffu, f, 8 * c);
      fz[nt][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
    }
  }

  // Fragment row r of a 16-token tile is token r with the last bit turned over
  // where bit 1 is set: a lane column's value rows then lie on both halves of
  // the banks.
  __device__ __forceinline__ static uint32_t token(uint32_t r) { return r ^ ((r >> 1) & 1u); }
  __device__ __forceinline__ uint32_t row_bytes() const { return EXACT ? (uint32_t)G::krow : rb; }
  __device__ __forceinline__ uint32_t scale_bytes() const { return EXACT ? (uint32_t)G::srow : sb; }

  // This lane's key words and scales of token `tok` of a unit.
  __device__ __forceinline__ void load_key(const uint8_t* codes, const uint8_t* scales, uint32_t tok, uint32_t (&w)[G::kw], uint32_t& sc) const {
    constexpr uint32_t per = DP / 4, group = Fmt<MODE>::group;
    const uint8_t* p = codes + tok * row_bytes() + c * G::kbytes;
    const uint8_t* q = scales + tok * scale_bytes() + c * per / group;
    if constexpr (EXACT) {
      load_words<G::kbytes>(p, w);
      sc = load_scales<per / group>(q);
    } else {
      constexpr int piece = per < 32 ? G::kbytes : 4 * (int)Fmt<MODE>::bits;  // bytes of at most 32 elements
#pragma unroll
      for (int i = 0; i < G::kw; ++i) w[i] = 0;
      sc = 0;
#pragma unroll
      for (int i = 0; i < G::kbytes / piece; ++i)
        if (c * per + 32u * i < D) {
          load_words<piece>(p + i * piece, w + i * (piece / 4));
          constexpr int n = per < 32 ? per / group : 32 / group;  // its scales
          sc |= load_scales<n>(q + i * (32 / group)) << (8 * i * (32 / group));
        }
    }
  }
  // And value words and scales (byte 0, and byte 1 for a second block).
  __device__ __forceinline__ void load_value(const uint8_t* codes, const uint8_t* scales, uint32_t tok, uint32_t (&w)[G::vw], uint32_t& sc) const {
    constexpr uint32_t per = DP / 8, group = Fmt<MODE>::group;
#pragma unroll
    for (int i = 0; i < G::vw; ++i) w[i] = 0;
    sc = 0;
    if (!EXACT && g * per >= D) return;
    load_words<G::vbytes>(codes + tok * row_bytes() + g * G::vbytes, w);
    sc = load_scales<per / group>(scales + tok * scale_bytes() + g * per / group);
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

  // S^T of the tile at token `tok0` of a unit.
  __device__ __forceinline__ void logits(const uint8_t* codes, const uint8_t* scales, uint32_t tok0, float (&s)[NT][4]) {
    uint32_t kw[2][G::kw], ks[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) load_key(codes, scales, tok0 + token(g) + 8u * i, kw[i], ks[i]);
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
          const uint32_t p = e4m3x2_to_f16x2(ks[i] >> (8 * b));
          sc[i][b] = __byte_perm(p, 0, 0x1010);
          if (b + 1 < DP / 64) sc[i][b + 1] = __byte_perm(p, 0, 0x3232);
        }
#pragma unroll
      for (int w = 0; w < G::kw; ++w) {
        uint32_t x[4], y[4];
        e2m1x8_to_f16x2(kw[0][w], x);
        e2m1x8_to_f16x2(kw[1][w], y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = mul_f16x2(x[e], sc[0][w / 2]);
          y[e] = mul_f16x2(y[e], sc[1][w / 2]);
        }
        step_mma(s, 2 * w, x[0], y[0], x[1], y[1]);
        step_mma(s, 2 * w + 1, x[2], y[2], x[3], y[3]);
      }
    } else if constexpr (MODE == kMX4) {
      uint32_t most = max(ks[0] & 255u, ks[1] & 255u);
      if constexpr (DP == 256) most = max(most, max(ks[0] >> 8, ks[1] >> 8));
      if (__any_sync(0xffffffffu, most > Mx<MODE>::largest(true))) mx_logits<true>(kw, ks, s);
      else mx_logits<false>(kw, ks, s);
    } else {
      mx_logits<true>(kw, ks, s);
    }
  }

  template <bool BIG>
  __device__ __forceinline__ void mx_logits(const uint32_t (&kw)[2][G::kw], const uint32_t (&ks)[2], float (&s)[NT][4]) {
    constexpr uint32_t up = Mx<MODE>::up(true);
    constexpr int wpb = 32 * (int)Fmt<MODE>::bits / 32;  // words a block
    uint32_t f[2] = {0, 0};
#pragma unroll
    for (int w = 0; w < G::kw; ++w) {
      if (w % wpb == 0)
#pragma unroll
        for (int i = 0; i < 2; ++i) f[i] = mx_factor<BIG>((ks[i] >> (8 * (w / wpb))) & 255u, up) * 0x10001u;
      const uint32_t a = kw[0][w], b = kw[1][w];
      auto k = [&](auto i, uint32_t x, uint32_t by) { return mx_pair<MODE, decltype(i)::value, BIG>(x, by, up); };
      const std::integral_constant<int, 0> i0;
      const std::integral_constant<int, 1> i1;
      if constexpr (MODE == kMX4) {
        const std::integral_constant<int, 2> i2;
        const std::integral_constant<int, 3> i3;
        step_mma(s, 2 * w, k(i0, a, f[0]), k(i0, b, f[1]), k(i1, a, f[0]), k(i1, b, f[1]));
        step_mma(s, 2 * w + 1, k(i2, a, f[0]), k(i2, b, f[1]), k(i3, a, f[0]), k(i3, b, f[1]));
      } else {
        step_mma(s, w, k(i0, a, f[0]), k(i0, b, f[1]), k(i1, a, f[0]), k(i1, b, f[1]));
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

  // O^T += V_hat^T . P^T of the tile at token `tok0`; fragment rows g and g + 8
  // of m-tile mt are elements (DP / 8) g + 2 mt and the next.  Bit i of `in`:
  // the lane's i-th token counts (what a masked place holds must not: P = 0
  // does not hide a NaN).
  __device__ __forceinline__ void weigh(const uint8_t* codes, const uint8_t* scales, uint32_t tok0, uint32_t in, const uint32_t (&ph)[NT][2],
                                        const uint32_t (&pl)[NT][2]) {
    uint32_t vw[4][G::vw], vs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      load_value(codes, scales, tok0 + token(2u * c + (i & 1)) + 8u * (i >> 1), vw[i], vs[i]);
      if (!((in >> i) & 1u)) vs[i] = 0;
    }
    if constexpr (MODE == kNV) {
#pragma unroll
      for (int w = 0; w < G::vw; ++w) {
        constexpr int wpb = 2;  // words a block
        const int b = DP == 256 ? w / wpb : 0;
        const uint32_t s01 = e4m3x2_to_f16x2(__byte_perm(vs[0], vs[1], b ? 0x0051 : 0x0040));
        const uint32_t s23 = e4m3x2_to_f16x2(__byte_perm(vs[2], vs[3], b ? 0x0051 : 0x0040));
        const uint32_t lo = 0x0F0F0F0Fu;
        uint32_t x01[4], y01[4], x23[4], y23[4];
        const uint32_t v0 = vw[0][w], v1 = vw[1][w], v2 = vw[2][w], v3 = vw[3][w];
        e2m1x8_to_f16x2((v0 & lo) | ((v1 << 4) & ~lo), x01);
        e2m1x8_to_f16x2(((v0 >> 4) & lo) | (v1 & ~lo), y01);
        e2m1x8_to_f16x2((v2 & lo) | ((v3 << 4) & ~lo), x23);
        e2m1x8_to_f16x2(((v2 >> 4) & lo) | (v3 & ~lo), y23);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          out_mma(4 * w + e, mul_f16x2(x01[e], s01), mul_f16x2(y01[e], s01), mul_f16x2(x23[e], s23),
                  mul_f16x2(y23[e], s23), ph, pl);
      }
    } else if constexpr (MODE == kMX4) {
      const uint32_t most = max(max(vs[0], vs[1]), max(vs[2], vs[3]));
      if (__any_sync(0xffffffffu, most > Mx<MODE>::largest(false))) mx_weigh<true>(vw, vs, ph, pl);
      else mx_weigh<false>(vw, vs, ph, pl);
    } else {
      mx_weigh<true>(vw, vs, ph, pl);
    }
  }

  template <bool BIG>
  __device__ __forceinline__ void mx_weigh(const uint32_t (&vw)[4][G::vw], const uint32_t (&vs)[4], const uint32_t (&ph)[NT][2],
                                           const uint32_t (&pl)[NT][2]) {
    constexpr uint32_t up = Mx<MODE>::up(false);
    const uint32_t f01 = mx_factor<BIG>(vs[0], up) | (mx_factor<BIG>(vs[1], up) << 16);
    const uint32_t f23 = mx_factor<BIG>(vs[2], up) | (mx_factor<BIG>(vs[3], up) << 16);
#pragma unroll
    for (int w = 0; w < G::vw; ++w)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint32_t sel = hf ? 0x7632u : 0x5410u;
        const uint32_t x = __byte_perm(vw[0][w], vw[1][w], sel), y = __byte_perm(vw[2][w], vw[3][w], sel);
        auto v = [&](auto i, uint32_t c, uint32_t by) { return mx_pair<MODE, decltype(i)::value, BIG>(c, by, up); };
        const std::integral_constant<int, 0> i0;
        const std::integral_constant<int, 1> i1;
        if constexpr (MODE == kMX4) {
          const std::integral_constant<int, 2> i2;
          const std::integral_constant<int, 3> i3;
          out_mma(4 * w + 2 * hf, v(i0, x, f01), v(i1, x, f01), v(i0, y, f23), v(i1, y, f23), ph, pl);
          out_mma(4 * w + 2 * hf + 1, v(i2, x, f01), v(i3, x, f01), v(i2, y, f23), v(i3, y, f23), ph, pl);
        } else {
          out_mma(2 * w + hf, v(i0, x, f01), v(i1, x, f01), v(i0, y, f23), v(i1, y, f23), ph, pl);
        }
      }
  }
};

// A sequence's share of the units: tiles * heads * span of them.
struct Work {
  Seq s;
  int32_t lo, hi, base;  // tokens that any query sees; base: of unit 0
  uint32_t R, tiles, span;
};
// From w.s, which has queries.
template <int ROWS, int UNIT>
__device__ __forceinline__ void lay_out(const AttnArgs& a, Work& w) {
  w.R = w.s.n * a.G;
  w.tiles = (w.R + ROWS - 1u) / ROWS;
  w.lo = tile_range(a, w.s, 0, 0).lo;
  w.hi = tile_range(a, w.s, w.s.n - 1, w.s.n - 1).hi;
  w.base = w.lo & ~(UNIT - 1);
  w.span = w.hi > w.lo ? ((uint32_t)(w.hi - w.base) + UNIT - 1u) / UNIT : 1u;  // an empty range is one unit of nothing
}
template <int ROWS, int UNIT>
__device__ __forceinline__ bool work_of(const AttnArgs& a, uint32_t b, Work& w) {
  if (!seq_of(a, b, w.s) || w.s.n == 0) return false;
  lay_out<ROWS, UNIT>(a, w);
  return true;
}

// A place in the order of all units.
template <int ROWS, int UNIT>
struct Cursor {
  uint32_t b, tile, hk, off;
  Work w;
  // Unit `at` of sequence b, w.s.
  __device__ __forceinline__ void start(const AttnArgs& a, uint32_t at) {
    lay_out<ROWS, UNIT>(a, w);
    const uint32_t q = at / w.span;
    off = at - q * w.span;
    tile = q / a.heads;
    hk = q - tile * a.heads;
  }
  // The next range's first unit; false past the last sequence.
  __device__ __forceinline__ bool next(const AttnArgs& a) {
    off = 0;
    if (++hk < a.heads) return true;
    hk = 0;
    if (++tile < w.tiles) return true;
    tile = 0;
    while (++b < a.B)
      if (work_of<ROWS, UNIT>(a, b, w)) return true;
    return false;
  }
};

__device__ __forceinline__ uint32_t shared_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
               "r"(bar)
               : "memory");
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on the barrier when this thread's copy16s so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Waits with a hint of how long (in ns) the thread may be suspended; by
// default at most 2^17 * 20 us.  A wait for what is still on its way into the
// CTA's memory (kDrainPolls) keeps that limit in test builds too.
constexpr uint32_t kPolls = tc::kWaitLimit / 512u, kDrainPolls = 1u << 17;
__device__ __forceinline__ bool wait_for(uint64_t& bar, uint32_t parity, uint32_t polls = kPolls) {
  for (uint32_t i = 0; i < polls; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(shared_u32(&bar)), "r"(parity), "r"(20000u)
        : "memory");
    if (ok) return true;
  }
  atomicOr(&g_device_error, (unsigned)kDevErrTimeout);
  return false;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <typename QT, int MODE, int DP, int NT, bool EXACT>
__global__ void __launch_bounds__(kDecThreads) k_kv_decode(const __grid_constant__ AttnArgs a) {
  using D = Decode<QT, MODE, DP, NT, EXACT>;
  using G = Geo<MODE, DP>;
  constexpr int TS = D::TS, MT = G::mtiles, ROWS = 8 * NT, UNIT = G::unit, ST = G::stages;
  extern __shared__ __align__(128) uint8_t stage_mem[];  // ST units: K codes, V codes, K scales, V scales
  __shared__ __align__(8) uint64_t full[ST], empty[ST];
  __shared__ uint32_t got[ST][UNIT / 32];                 // a bit for each of the unit's tokens: it is there
  __shared__ uint32_t wsum[kDecWarps + 1], found[5];
  __shared__ volatile int abort_flag;
  __shared__ float sm[kDecWarps][ROWS], sl[kDecWarps][ROWS];
  __shared__ __align__(16) float so[kDecWarps][ROWS * DP];
  __shared__ int64_t rows[UNIT];                          // pages that end inside a 16-token piece: row of each token, or -1
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t rb = a.D * Fmt<MODE>::bits / 8u, sb = a.D / Fmt<MODE>::group;
  const uint32_t v_at = UNIT * rb, ks_at = 2u * v_at, vs_at = ks_at + UNIT * sb, unit_bytes = 2u * UNIT * (rb + sb);
  // All units, then this worker's run [u0, u1) of them and the sequence it
  // begins in.  Up to 32 sequences every warp does it for itself, with nothing
  // to wait for but the lengths; of more, the warps take 32 each in turn.
  Work w;
  // (The caller's bounds keep the number of units below 2^32.)
  auto units_of = [&](uint32_t b) -> uint32_t {
    return b < a.B && work_of<ROWS, UNIT>(a, b, w) ? w.tiles * a.heads * w.span : 0u;
  };
  const float gk = a.g[0] ? __ldg(a.g[0]) / kGlobalEncode : 1.0f, gv = a.g[1] ? __ldg(a.g[1]) / kGlobalEncode : 1.0f;
  const bool few = a.B <= 32u;
  constexpr uint32_t ROUND = 32 * (kDecWarps + 1);
  uint32_t total = 0, mine = 0;
  for (uint32_t b0 = few ? 0u : 32u * warp; b0 < a.B; b0 += ROUND) {
    mine = units_of(b0 + lane);
    total += mine;
  }
  if (threadIdx.x == 0) {
    abort_flag = 0;
    found[0] = a.B;
    for (int i = 0; i < ST; ++i) {
      // without bulk copies every lane arrives
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_u32(&full[i])), "r"(a.page_size % 16u ? 33 : 1));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_u32(&empty[i])), "r"((int)kDecWarps));
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
  if (!few) {
    if (lane == 0) wsum[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int i = 0; i <= kDecWarps; ++i) total += wsum[i];
  }
  const uint32_t workers = min(gridDim.x, total);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x >= workers) {
    if (a.split && threadIdx.x == 0) a.part_head[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  // the first `longer` workers take one unit more than the others
  const uint32_t each = total / workers, longer = total - each * workers;
  const uint32_t u0 = each * blockIdx.x + min(blockIdx.x, longer), u1 = u0 + each + (blockIdx.x < longer ? 1u : 0u);
  Cursor<ROWS, UNIT> at;
  at.b = a.B;
  uint32_t found_at = 0, before = 0;  // units of the sequences before these
  for (uint32_t b0 = few ? 0u : 32u * warp;; b0 += ROUND) {
    const uint32_t v = few ? mine : units_of(b0 + lane);
    uint32_t incl = v;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, x);
      if (lane >= (uint32_t)x) incl += y;
    }
    uint32_t round = 0;
    if (!few) {
      __syncthreads();  // wsum is read
      if (lane == 31) wsum[warp] = incl;
      __syncthreads();
#pragma unroll
      for (int i = 0; i <= kDecWarps; ++i) {
        if ((uint32_t)i < warp) incl += wsum[i];
        round += wsum[i];
      }
      incl += before;
    }
    const uint32_t here = __ballot_sync(0xffffffffu, u0 < incl && u0 >= incl - v);
    if (here) {
      const int src = __ffs(here) - 1;
      at.b = b0 + (uint32_t)src;
      at.w.s.t0 = __shfl_sync(0xffffffffu, w.s.t0, src);
      at.w.s.n = __shfl_sync(0xffffffffu, w.s.n, src);
      at.w.s.L = __shfl_sync(0xffffffffu, w.s.L, src);
      found_at = __shfl_sync(0xffffffffu, incl - v, src);
    }
    if (few) break;
    before += round;
    if (u0 < before || b0 - 32u * warp + ROUND >= a.B) {  // the same for all warps: one of them has it
      if (here && lane == 0) {
        found[0] = at.b;
        found[1] = at.w.s.t0;
        found[2] = at.w.s.n;
        found[3] = at.w.s.L;
        found[4] = found_at;
      }
      __syncthreads();
      at.b = found[0];
      at.w.s = Seq{found[1], found[2], found[3]};
      found_at = found[4];
      break;
    }
  }
  __syncthreads();  // the barriers stand
  if (at.b >= a.B) return;  // the lengths changed meanwhile
  at.start(a, u0 - found_at);
  uint32_t u = u0;
  bool more = true;
  if (!a.split && at.off) {  // without partial results a range belongs to the worker it begins in
    u += at.w.span - at.off;
    more = u < u1 && at.next(a);
  }
  // units of the current range that this worker takes
  auto take = [&]() { return a.split ? min(at.w.span - at.off, u1 - u) : at.w.span; };

  if (warp == kDecWarps) {
    // ------------------------------------------------------------ copies
    // run: tokens that lie together on one page whatever unit they are in
    const uint32_t run = min((uint32_t)UNIT, a.page_size & (0u - a.page_size));
    uint32_t it = 0;
    bool ok = true;
    while (more && ok) {
      const uint32_t n = take();
      const int32_t* table = a.page_table + (uint64_t)at.b * a.max_pages;
      auto row_of = [&](int32_t j) -> int64_t {
        const uint32_t pg = a.by_page.div((uint32_t)j);
        const int32_t page = __ldg(table + pg);
        if ((uint32_t)page < a.num_pages)
          return (int64_t)(((uint64_t)(uint32_t)page * a.heads + at.hk) * a.page_size + ((uint32_t)j - pg * a.page_size));
        atomicOr(&g_device_error, (unsigned)kDevErrIndex);
        return -1;
      };
      // runs of at least 16 tokens: lane = run * 4 + part; else token lane + 32 i
      const uint32_t part = lane & 3u, r = lane >> 2;
      int64_t y[UNIT / 32];  // rows of the unit to come, looked up a unit ahead
      auto look = [&](uint32_t k) {
        const int32_t t0 = at.w.base + (int32_t)((at.off + k) * UNIT);
        if (run >= 16u) {
          const int32_t j = t0 + (int32_t)(r * run);
          y[0] = r * run < (uint32_t)UNIT && j < at.w.hi && j + (int32_t)run > at.w.lo ? row_of(j) : -1;
        } else {
#pragma unroll
          for (int i = 0; i < UNIT / 32; ++i) {
            const int32_t j = t0 + (int32_t)(32u * i + lane);
            y[i] = j >= at.w.lo && j < at.w.hi ? row_of(j) : -1;
          }
        }
      };
      if (n > 0) look(0);
      for (uint32_t k = 0; k < n; ++k, ++it) {
        const uint32_t st = it % ST;
        if (!__all_sync(0xffffffffu, wait_for(empty[st], (it / ST & 1u) ^ 1u) && !abort_flag)) {
          ok = false;
          break;
        }
        if (tc::withheld_stage(it)) {
          if (k + 1 < n) look(k + 1);
          continue;
        }
        const int32_t t0 = at.w.base + (int32_t)((at.off + k) * UNIT);
        const uint32_t bar = shared_u32(&full[st]), dst = shared_u32(stage_mem) + st * unit_bytes;
        if (run >= 16u) {
          const int32_t j = t0 + (int32_t)(r * run);
          const uint32_t cnt = y[0] >= 0 ? min(run, ((uint32_t)(at.w.hi - j) + 15u) & ~15u) : 0u;
          uint32_t tokens = 0;
#pragma unroll
          for (int i = 0; i < UNIT / 32; ++i) {
            const int from = max((int)(r * run) - 32 * i, 0), to = min((int)(r * run + cnt) - 32 * i, 32);
            const uint32_t mask = __reduce_or_sync(0xffffffffu, to > from ? (0xffffffffu >> (32 - to)) & (0xffffffffu << from) : 0u);
            if (lane == 0) got[st][i] = mask;
            tokens += __popc(mask);
          }
          if (lane == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(tokens * 2u * (rb + sb)) : "memory");
          __syncwarp();
          if (cnt) {
            const uint32_t bytes = part < 2u ? rb : sb;
            const uint8_t* src = part == 0 ? a.codes[0] : part == 1 ? a.codes[1] : part == 2 ? a.scales[0] : a.scales[1];
            bulk_copy(dst + (part == 0 ? 0u : part == 1 ? v_at : part == 2 ? ks_at : vs_at) + r * run * bytes, src + (uint64_t)y[0] * bytes,
                      cnt * bytes, bar);
          }
        } else {
          // pages that end inside a 16-token piece: codes by 16-byte pieces of
          // each token's row, scales (rows of any few bytes) by plain loads
#pragma unroll
          for (int i = 0; i < UNIT / 32; ++i) {
            rows[32u * i + lane] = y[i];
            const uint32_t mask = __ballot_sync(0xffffffffu, y[i] >= 0);
            if (lane == 0) got[st][i] = mask;
          }
          __syncwarp();
          const uint32_t per = rb / 16u;
#pragma unroll 4
          for (uint32_t x = lane; x < UNIT * per; x += 32u) {
            const int64_t row = rows[x / per];
            if (row >= 0) {
              const uint64_t from = (uint64_t)row * rb + (x % per) * 16u;
              copy16(dst + x * 16u, a.codes[0] + from);
              copy16(dst + v_at + x * 16u, a.codes[1] + from);
            }
          }
          copies_arrive(bar);
#pragma unroll 4
          for (uint32_t x = lane; x < UNIT * sb; x += 32u) {
            const int64_t row = rows[x / sb];
            if (row >= 0) {
              const uint64_t from = (uint64_t)row * sb + x % sb;
              uint8_t* to = stage_mem + st * unit_bytes + ks_at + x;
              to[0] = __ldg(a.scales[0] + from);
              to[UNIT * sb] = __ldg(a.scales[1] + from);
            }
          }
          __syncwarp();
          if (lane == 0) arrive(bar);
        }
        if (k + 1 < n) look(k + 1);
      }
      u += n;
      more = ok && u < u1 && at.next(a);
    }
    if (!ok && lane == 0) abort_flag = 1;
    // what was asked for has landed before the CTA's memory goes
    for (uint32_t i = it > (uint32_t)ST ? it - ST : 0; i < it; ++i)
      if (!tc::withheld_stage(i)) wait_for(full[i % ST], i / ST & 1u, kDrainPolls);
    return;
  }

  // -------------------------------------------------------------- the rest
  D d;
  d.lane = lane;
  d.g = lane >> 2;
  d.c = lane & 3u;
  d.rb = rb;
  d.sb = sb;
  d.D = a.D;
  if (a.split && threadIdx.x == 0) a.part_head[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  uint32_t it = 0;
  for (uint32_t seg = 0; more; ++seg) {
    const uint32_t n = take(), r0 = at.tile * ROWS, R = at.w.R;
    const Seq s = at.w.s;
    const bool whole = at.off == 0 && n == at.w.span;
    d.load_q(a, s, at.hk, r0, R, gk);
    // what this lane's columns (rows r0 + 8 nt + 2c, + 1) see
    int32_t see_lo[NT][2], see_hi[NT][2];
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
    const uint32_t i0 = r0 / a.G, i1 = (min(r0 + ROWS, R) - 1u) / a.G;
    const int32_t all_lo = max(at.w.lo, tile_range(a, s, i1, i1).lo), all_hi = min(at.w.hi, tile_range(a, s, i0, i0).hi);

    for (uint32_t k = 0; k < n; ++k, ++it) {
      const uint32_t st = it % ST;
      // once a wait has run out nothing is waited for: the sums are void, the host is told
      if (!__any_sync(0xffffffffu, abort_flag) && !__all_sync(0xffffffffu, wait_for(full[st], it / ST & 1u))) abort_flag = 1;
      const uint8_t* mem = stage_mem + st * unit_bytes;
      const uint32_t tok0 = warp * 16u * TS;
      const int32_t j0 = at.w.base + (int32_t)((at.off + k) * UNIT + tok0);
      const uint32_t there = TS == 2 ? got[st][warp] : got[st][warp >> 1] >> (16u * (warp & 1u)) & 0xffffu;
      const bool full_step = there == (TS == 2 ? 0xffffffffu : 0xffffu) && j0 >= all_lo && j0 + 16 * TS <= all_hi;
      float sv[TS][NT][4];
#pragma unroll
      for (int t = 0; t < TS; ++t) d.logits(mem, mem + ks_at, tok0 + 16u * t, sv[t]);
      uint32_t in[TS];  // weigh's tokens that count
#pragma unroll
      for (int t = 0; t < TS; ++t) in[t] = 15u;
      if (!full_step) {
#pragma unroll
        for (int t = 0; t < TS; ++t) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t x = 16u * t + 8u * (e >> 1) + D::token(d.g);
              const int32_t j = j0 + (int32_t)x;
              if (!((there >> x) & 1u) || j < see_lo[nt][e & 1] || j >= see_hi[nt][e & 1]) sv[t][nt][e] = -INFINITY;
            }
          in[t] = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = 16u * t + 8u * (i >> 1) + D::token(2u * d.c + (i & 1));
            const int32_t j = j0 + (int32_t)x;
            in[t] |= ((there >> x) & 1u) && j >= at.w.lo && j < at.w.hi ? 1u << i : 0u;
          }
        }
      }
      // The running maximum moves only when a step exceeds it by 2^8 (weights
      // then lie below 2^(8 + kUp), which 16 bits and the sums hold).
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
          top[nt][e] = x * d.fz[nt][e] - kUp<MODE>;
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
        d.weigh(mem + v_at, mem + vs_at, tok0 + 16u * t, in[t], ph, pl);
      }
      __syncwarp();
      if (lane == 0) arrive(shared_u32(&empty[st]));
    }

    // Join the warps: a common maximum first, then the sums.
    auto sync = [&]() { asm volatile("bar.sync 1, 128;" ::: "memory"); };
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
    sync();
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
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        reinterpret_cast<float4*>(so[warp])[(nt * MT + mt) * 32 + lane] =
            make_float4(d.o[nt][mt][0], d.o[nt][mt][1], d.o[nt][mt][2], d.o[nt][mt][3]);
    sync();
    // eight elements (m-tiles 4k .. 4k + 3) of the lane's columns 2c + e of n-tile nt
    const uint32_t slot = 2u * blockIdx.x + (seg ? 1u : 0u);
    const float fv = D::kMx ? 1.0f : gv;
#pragma unroll 1
    for (uint32_t item = warp; item < NT * (DP / 64) * 2u; item += kDecWarps) {
      const uint32_t e = item & 1u, k = (item >> 1) % (DP / 64), nt = (item >> 1) / (DP / 64);
      const uint32_t lr = 8u * nt + 2u * d.c + e, r = r0 + lr, el = d.g * (DP / 8) + 8u * k;
      if (r >= R || el >= a.D) continue;
      float M = -INFINITY, l = 0.0f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        M = fmaxf(M, sm[w][lr]);
        l += sl[w][lr];
      }
      const uint32_t i = r / a.G, h = at.hk * a.G + (r - i * a.G);
      const uint64_t to = (uint64_t)(s.t0 + i) * a.Hq + h;
      const float f = whole ? (l == 0.0f ? 0.0f : fv / l) : fv;
      if (d.g == 0 && k == 0) {
        if (!whole) a.part_ml[slot * ROWS + lr] = make_float2(M, l);
        else if (a.lse) a.lse[to] = lse_of(M, l);
      }
      float v[8];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        v[2 * x] = v[2 * x + 1] = 0.0f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float4 p = reinterpret_cast<const float4*>(so[w])[(nt * MT + 4u * k + x) * 32u + lane];
          v[2 * x] += e ? p.y : p.x;
          v[2 * x + 1] += e ? p.w : p.z;
        }
        v[2 * x] *= f;
        v[2 * x + 1] *= f;
      }
      if (whole)
        store8<QT>(static_cast<QT*>(a.out) + to * a.D + el, v);
      else
        store8<float>(a.part_o + ((uint64_t)slot * ROWS + lr) * a.D + el, v);
    }
    sync();  // so, sm and sl are read
    if (warp == 0) {
      // The worker that begins a range it does not end says which workers have
      // the rest: the next ones, each in its first slot.
      if (!whole && at.off == 0 && lane == 0) {
        const uint32_t last = u + at.w.span - 1u, many = longer * (each + 1u);
        const uint32_t worker = last < many ? last / (each + 1u) : longer + (last - many) / each;
        a.part_head[2 * blockIdx.x] = make_int4((int)worker + 1, (int)slot, (int)(s.t0 + r0 / a.G), (int)min((uint32_t)ROWS, R - r0));
        a.part_head[2 * blockIdx.x + 1] = make_int4((int)(r0 % a.G), (int)at.hk, 0, 0);
      }
    }
    u += n;
    more = u < u1 && at.next(a);
  }
}

// Join of two rows (2 blockIdx.y, + 1) of the range that worker blockIdx.x
// began and others went on with: four warps a row, one for every fourth part,
// the row's elements over the lanes.
template <typename QT, int ROWS>
__global__ void __launch_bounds__(256) k_kv_decode_join(const __grid_constant__ AttnArgs a) {
  __shared__ float sl[8];
  __shared__ __align__(16) float so[8][256];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 head = a.part_head[2 * blockIdx.x];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, lr = 2u * blockIdx.y + (warp >> 2), w0 = warp & ~3u;
  if (head.x == 0 || 2u * blockIdx.y >= (uint32_t)head.w) return;
  const int4 more = a.part_head[2 * blockIdx.x + 1];
  const uint32_t parts = lr < (uint32_t)head.w ? (uint32_t)head.x - blockIdx.x : 0u, d0 = lane * 8u;
  auto slot = [&](uint32_t k) { return k == 0 ? (uint32_t)head.y : 2u * (blockIdx.x + k); };
  float m = -INFINITY;
  for (uint32_t k = lane; k < parts; k += 32) m = fmaxf(m, a.part_ml[slot(k) * ROWS + lr].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  float l = 0.0f, o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.0f;
#pragma unroll 4
  for (uint32_t k = warp & 3u; k < parts; k += 4u) {
    const float2 ml = a.part_ml[slot(k) * ROWS + lr];
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    if (d0 < a.D) load8_shared<float>(a.part_o + ((uint64_t)slot(k) * ROWS + lr) * a.D + d0, v);
    const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - m);
    l += ml.y * f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = fmaf(v[e], f, o[e]);
  }
  if (lane == 0) sl[warp] = l;
  store8<float>(&so[warp][d0], o);
  __syncthreads();
  if (warp != w0 || parts == 0) return;
  l = sl[w0] + sl[w0 + 1] + sl[w0 + 2] + sl[w0 + 3];
  const uint32_t x = (uint32_t)more.x + lr, i = x / a.G;  // query after the tile's first, head of the group
  const uint64_t at = (uint64_t)((uint32_t)head.z + i) * a.Hq + (uint32_t)more.y * a.G + (x - i * a.G);
  if (a.lse && lane == 0) a.lse[at] = lse_of(m, l);
  if (d0 >= a.D) return;
  const float f = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = (so[w0][d0 + e] + so[w0 + 1][d0 + e] + so[w0 + 2][d0 + e] + so[w0 + 3][d0 + e]) * f;
  store8<QT>(static_cast<QT*>(a.out) + at * a.D + d0, o);
}

// k_kv_prefill's join.  One (query, head): one CTA, a warp for every
// fourth chunk, the row's elements over the lanes.
constexpr int kJoinWarps = 4;
template <typename QT>
__global__ void __launch_bounds__(kJoinWarps * 32) k_kv_join(const __grid_constant__ AttnArgs a) {
  __shared__ float sl[kJoinWarps];
  __shared__ __align__(16) float so[kJoinWarps][256];
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
  if (a.lse && lane == 0) a.lse[at] = lse_of(m, l);
  if (d0 >= a.D) return;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = 0.0f;
    for (int w = 0; w < kJoinWarps; ++w) v[e] += so[w][d0 + e];
    v[e] = l == 0.0f ? 0.0f : v[e] / l;
  }
  store8<QT>(static_cast<QT*>(a.out) + at * a.D + d0, v);
}

}  // namespace kv
}  // namespace nvfp4
