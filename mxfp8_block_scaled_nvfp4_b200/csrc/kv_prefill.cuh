// kv_attention for many query rows: tcgen05 matrix products with S and O in
// tensor memory (formulas and partial results as in kv_attention.cuh).
//
// A CTA holds one or two tiles of 128 query rows (row r of a sequence and a
// key/value head is query r / G, head r % G of the group) and walks the
// tokens in tiles of NT:
//   warps 0-3, 4-7  softmax of query tile 0, 1; thread = row = TMEM lane
//   warps 8-11      producers: cache codes to 16-bit K_hat and V_hat tiles in
//                   shared memory (each decoded once for both query tiles)
//   warp 12         allocates TMEM and issues the MMAs
// Per query tile, S = Q K_hat^T (128 x NT, fp32, TMEM); the softmax threads
// write P as 16-bit pairs over S, and O (128 x D, fp32, TMEM) += P V_hat with
// P as the MMA's TMEM operand.  The two query tiles alternate, so that the
// tensor core works on one while the other's exponentials are taken.
//
// Shared-memory tiles (Q, K, V alike): 8-row groups of ceil(D / 64) boxes of
// 8 rows x 128 bytes, 128-byte swizzled.  Read along D that is a K-major
// operand (Q and K), read along the rows an MN-major one (V), so V needs no
// transpose.
//
// Number formats as in k_kv_decode: NVFP4 exact fp16 operands, P in fp16; MX
// modes exact bf16 operands times 2^-64 and P in two bf16 terms, each with
// its own MMA.  (fp16 queries over an MX cache would need two terms of Q as
// well; they stay with k_kv_decode.)
#pragma once

#include "kv_attention.cuh"
#include "qqmm_sm100.cuh"

namespace nvfp4 {
namespace kv {
namespace pf {

using namespace tc;

constexpr int W_PROD = 8, W_MMA = 12, THREADS = 13 * 32, PROD = 128;
constexpr int ST = 2;  // K and V stages
constexpr int kPolyEvery = 4;  // of so many pairs of exponentials one is a polynomial on the FMA pipes

template <int DP>
struct Shape {
  static constexpr int NQ = DP == 256 ? 1 : 2;        // query tiles a CTA
  static constexpr int NT = DP == 256 ? 64 : 128;     // tokens a tile
  static constexpr uint32_t group = DP / 64 * 1024;   // an 8-row group
  static constexpr uint32_t q_tile = 16 * group;      // 128 rows
  static constexpr uint32_t kv_tile = NT / 8 * group;
  // at least half an SM's: a CTA takes all of TMEM, so one fits at a time
  static constexpr uint32_t bytes = NQ * q_tile + 2 * ST * kv_tile + 1024, smem = bytes < 122880 ? 122880 : bytes;
  static constexpr uint32_t tm_s = 0, tm_o = 256;     // TMEM columns: S of tile t at 128 t, O at 256 + 128 t
};

__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// fp32 accumulate, A K-major and B K- or MN-major, both fp16 or both bf16.
__device__ __forceinline__ uint32_t idesc_f16(bool bf16, bool b_mn, uint32_t n) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&v)[N]);
template <>
__device__ __forceinline__ void tmem_st<16>(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Element (of an octet) at position p of the 16-bit octets that `decode8`
// gives: NVFP4 keeps the order, the MX modes' pairs interleave.
template <int MODE>
__host__ __device__ constexpr int octet(int p) {
  return MODE == kNV ? p : MODE == kMX4 ? (p & 1) * 4 + p / 2 : (p / 4) * 4 + (p & 1) * 2 + (p / 2 % 2);
}
// Eight codes (one word, MXFP8 two) times the scale pair f.
template <int MODE>
__device__ __forceinline__ uint4 decode8(const uint32_t* w, uint32_t f) {
  if constexpr (MODE == kNV) {
    uint32_t v[4];
    e2m1x8_to_f16x2(w[0], v);
    return make_uint4(mul_f16x2(v[0], f), mul_f16x2(v[1], f), mul_f16x2(v[2], f), mul_f16x2(v[3], f));
  } else if constexpr (MODE == kMX4) {
    return make_uint4(mul_bf16x2(e2m1_pair_bf16<0>(w[0]), f), mul_bf16x2(e2m1_pair_bf16<1>(w[0]), f),
                      mul_bf16x2(e2m1_pair_bf16<2>(w[0]), f), mul_bf16x2(e2m1_pair_bf16<3>(w[0]), f));
  } else {
    return make_uint4(mul_bf16x2(e4m3_pair_bf16<0>(w[0]), f), mul_bf16x2(e4m3_pair_bf16<1>(w[0]), f),
                      mul_bf16x2(e4m3_pair_bf16<0>(w[1]), f), mul_bf16x2(e4m3_pair_bf16<1>(w[1]), f));
  }
}

// One thread's share of a K or V tile: units of 32 elements of one token
// (DP / 32 units a token, U a thread, in registers from load to store).  Unit
// u is the same part c of token tok + u * PROD / (DP / 32).
template <int MODE, int DP>
struct Share {
  static constexpr int per_row = DP / 32, U = Shape<DP>::NT * per_row / PROD;
  static constexpr int words = (int)Fmt<MODE>::bits, wo = words / 4;  // of a unit, of an octet
  static constexpr uint32_t step = PROD / per_row;                    // tokens between units (a multiple of 8)
  uint32_t w[U][words], s[U];

  // at: byte offsets of the tokens' code rows and scale rows, < 0 for tokens
  // that are not there: those get another row's codes with a scale of zero
  // (finite numbers that P = 0 meets).
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, const int64_t (*at)[2], uint32_t tok,
                                       uint32_t c, uint32_t D) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t x = at[tok + u * step][0], y = at[tok + u * step][1];
      if (c * 32u < D) {  // the same for all units of a thread
        load_words<4 * words>(codes + (x < 0 ? 0 : x) + c * (4 * words), w[u]);
        s[u] = load_scales<32 / (int)Fmt<MODE>::group>(scales + (x < 0 ? 0 : y) + c * (32 / Fmt<MODE>::group));
        if (x < 0) s[u] = 0;
      } else {
#pragma unroll
        for (int i = 0; i < words; ++i) w[u][i] = 0;
        s[u] = 0;
      }
    }
  }
  // The units' four octets as 16-byte chunks of the tile.  Units 2, 3 (mod 4)
  // of a row lie in another box at the same banks as units 0, 1: they store
  // their octets in another order, so that eight lanes (two rows) always
  // cover eight chunks.
  __device__ __forceinline__ void store(uint32_t base, uint32_t tok, uint32_t c) const {
    const bool swap = per_row >= 4 && (c & 2u);
    const uint32_t row = base + (tok >> 3) * Shape<DP>::group + (c >> 1) * 1024u + (tok & 7u) * 128u;
    uint32_t to[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      to[e] = row + ((((c & 1u) * 4u + (uint32_t)(swap ? e ^ 2 : e)) ^ (tok & 7u)) << 4);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t f[2];
      if constexpr (MODE == kNV) {
        const uint32_t pr = e4m3x2_to_f16x2(s[u]);
        f[0] = __byte_perm(pr, 0, swap ? 0x3232 : 0x1010);
        f[1] = __byte_perm(pr, 0, swap ? 0x1010 : 0x3232);
      } else {
        const uint32_t q = mx_factor<MODE>(s[u]);
        f[0] = f[1] = q | (q << 16);
      }
      uint32_t x[words];
#pragma unroll
      for (int i = 0; i < words; ++i) x[i] = swap ? w[u][i ^ (2 * wo)] : w[u][i];
#pragma unroll
      for (int e = 0; e < 4; ++e) st_shared_v4(to[e] + u * (step / 8u) * Shape<DP>::group, decode8<MODE>(&x[e * wo], f[e / 2]));
    }
  }
};

// tcgen05.ld of 32 columns without its wait; the wait names the registers, so
// that nothing reads them before it.
__device__ __forceinline__ void tmem_ld32_start(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Packed pairs of fp32.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 2^y of a pair on the FMA pipes: y = n + f with n the nearest integer (from
// the low bits of y + 1.5 * 2^23), 2^f by the degree-4 polynomial of least
// relative error on [-1/2, 1/2] (Remez exchange; 2.6e-6, a hundredth of P's
// rounding), n added to the exponent.  y is raised to -126 first, so nothing
// wraps; what is masked becomes 2^-126.
__device__ __forceinline__ uint64_t ex2_poly(uint64_t y2) {
  float y0, y1;
  unpair(y2, y0, y1);
  y2 = pair(fmaxf(y0, -126.0f), fmaxf(y1, -126.0f));
  const uint64_t big = pair(12582912.0f, 12582912.0f), t = add2(y2, big);
  const uint64_t f = fma2(add2(t, pair(-12582912.0f, -12582912.0f)), pair(-1.0f, -1.0f), y2);
  uint64_t p = fma2(f, pair(0.009570102207362652f, 0.009570102207362652f), pair(0.05591785907745361f, 0.05591785907745361f));
  p = fma2(p, f, pair(0.240247443318367f, 0.240247443318367f));
  p = fma2(p, f, pair(0.6931217908859253f, 0.6931217908859253f));
  p = fma2(p, f, pair(0.9999992847442627f, 0.9999992847442627f));
  float t0, t1, p0, p1;
  unpair(t, t0, t1);
  unpair(p, p0, p1);
  return pair(__uint_as_float(__float_as_uint(p0) + (__float_as_uint(t0) << 23)),
              __uint_as_float(__float_as_uint(p1) + (__float_as_uint(t1) << 23)));
}

template <typename QT, int MODE, int DP>
__global__ void __launch_bounds__(THREADS, 1) k_kv_prefill(const __grid_constant__ AttnArgs a) {
  using S = Shape<DP>;
  constexpr int NQ = S::NQ, NT = S::NT;
  constexpr bool kMx = MODE != kNV;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t k_full[ST], k_empty[ST], v_full[ST], v_empty[ST], s_full[2], p_full[2], o_done[2], all_done;
  __shared__ int64_t rows[2][NT][2];  // byte offsets of the tokens' code and scale rows
  __shared__ uint32_t tmem_holder;
  __shared__ volatile int abort_flag;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sq = sbase, sk = sq + NQ * S::q_tile, sv = sk + ST * S::kv_tile;
  const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31u);

  // heaviest tiles first: the last queries of a causal prompt see most
  const uint32_t tiles = gridDim.x / a.chunks, tile = tiles - 1u - blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
  const uint32_t hk = blockIdx.y, b = blockIdx.z, r0 = tile * 128u * NQ;
  Seq s;
  if (!seq_of(a, b, s)) return;
  const uint32_t R = s.n * a.G;
  if (r0 >= R) return;
  const uint32_t rl = min(r0 + 128u * NQ, R) - 1u;
  const Range rg = tile_range(a, s, r0 / a.G, rl / a.G);
  const int32_t base = rg.lo & ~15;
  const int32_t span = rg.hi > rg.lo ? rg.hi - base : 0;
  if (chunk > 0 && (int64_t)chunk * a.chunk >= span) return;
  const bool whole = span <= a.chunk;
  const int32_t begin = base + (int32_t)chunk * a.chunk;
  const int32_t end = min(rg.hi, begin + a.chunk);
  const int32_t iters = end > begin ? (end - begin + NT - 1) / NT : 0;
  const int nq = NQ == 2 && r0 + 128u < R ? 2 : 1;
  const int32_t* table = a.page_table + (uint64_t)b * a.max_pages;
  const uint32_t kchunks = a.D / 16u;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < ST; ++i) {
      mbar_init(smem_u32(&k_full[i]), 4);
      mbar_init(smem_u32(&v_full[i]), 4);
      mbar_init(smem_u32(&k_empty[i]), 1);
      mbar_init(smem_u32(&v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), 4);
      mbar_init(smem_u32(&o_done[i]), 1);
    }
    mbar_init(smem_u32(&all_done), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == W_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_holder)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // pages out of range: the softmax then looks every token up
  int bad = 0;
  if (iters > 0) {
    const uint32_t pg0 = a.by_page.div((uint32_t)max(begin, rg.lo)), pg1 = a.by_page.div((uint32_t)(end - 1));
    for (uint32_t pg = pg0 + threadIdx.x; pg <= pg1; pg += THREADS) bad |= (uint32_t)__ldg(table + pg) >= a.num_pages;
    if (bad) atomicOr(&g_device_error, (unsigned)kDevErrIndex);
  }
  // the query tiles: thread = row
  const int qt = warp >> 2;  // softmax warps: their query tile
  const uint32_t row = (uint32_t)(threadIdx.x & 127u);
  const uint32_t r = r0 + 128u * qt + row;
  float fz = 0.0f;
  if (warp < 4 * nq) {
    const uint32_t i = min(r, R - 1u) / a.G, h = hk * a.G + (min(r, R - 1u) - i * a.G);
    const QT* q = static_cast<const QT*>(a.q) + (int64_t)(s.t0 + i) * a.q_stride + (int64_t)h * a.D;
    float mx = 0.0f;
    for (uint32_t k = 0; k < a.D; k += 8) {
      float x[8];
      load8<QT>(q + k, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
    }
    const int e2 = mx > 0.0f ? max(-80, (int)((__float_as_uint(mx) >> 23) & 255u) - 127) : 0;
    const float up = pow2((kMx ? 40 : 14) - e2) * (a.scale < 0.0f ? -1.0f : 1.0f);
    const float gk = a.g[0] ? __ldg(a.g[0]) / kGlobalEncode : 1.0f;
    fz = fmaxf(fabsf(a.scale) * kLog2e * pow2(e2) * gk * pow2(kMx ? 24 : -14), 1e-37f);
    for (uint32_t o = 0; o < a.D / 8u; ++o) {
      float x[8];
      load8<QT>(q + 8u * o, x);
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float y0 = x[octet<MODE>(2 * e)] * up, y1 = x[octet<MODE>(2 * e + 1)] * up;
        v[e] = kMx ? pack_bf16x2(y0, y1) : pack_f16x2(y0, y1);
      }
      st_shared_v4(sq + qt * S::q_tile + (row >> 3) * S::group + (o >> 3) * 1024u + (row & 7u) * 128u + (((o & 7u) ^ (row & 7u)) << 4),
                   make_uint4(v[0], v[1], v[2], v[3]));
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  tc_fence_before();
  const int any_bad = __syncthreads_or(bad);
  tc_fence_after();
  const uint32_t tmem = tmem_holder;

  if (warp >= W_PROD && warp < W_MMA) {
    // ------------------------------------------------------------ producers
    const uint32_t p = (uint32_t)(threadIdx.x - 32 * W_PROD);
    // Rows of tile n's tokens; true on every producer once any has given up.
    auto look = [&](int32_t n) {
      if (n < iters && p < (uint32_t)NT) {
        const int32_t j = begin + n * NT + (int32_t)p;
        int64_t x = -1;
        if (j >= rg.lo && j < end) {
          const uint32_t pg = a.by_page.div((uint32_t)j);
          const int32_t page = __ldg(table + pg);
          if ((uint32_t)page < a.num_pages)
            x = (int64_t)(((uint64_t)page * a.heads + hk) * a.page_size + ((uint32_t)j - pg * a.page_size));
        }
        rows[n & 1][p][0] = x * (int64_t)(a.D * Fmt<MODE>::bits / 8u);
        rows[n & 1][p][1] = x * (int64_t)(a.D / Fmt<MODE>::group);
      }
      uint32_t stop;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
          "barrier.cta.red.or.pred p, 1, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(stop)
          : "r"((uint32_t)abort_flag)
          : "memory");
      return stop != 0;
    };
    using Sh = Share<MODE, DP>;
    Sh kk, vv;
    const uint32_t tok = p / Sh::per_row, c = p % Sh::per_row;
    look(0);
    if (iters > 0) {
      kk.load(a.codes[0], a.scales[0], rows[0], tok, c, a.D);
      vv.load(a.codes[1], a.scales[1], rows[0], tok, c, a.D);
    }
    look(1);
    for (int32_t n = 0; n < iters; ++n) {
      const uint32_t st = (uint32_t)n % ST, ph = ((uint32_t)n / ST) & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&k_empty[st]), ph ^ 1u)) || abort_flag) abort_flag = 1;
      kk.store(sk + st * S::kv_tile, tok, c);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(smem_u32(&k_full[st]));
      if (n + 1 < iters) kk.load(a.codes[0], a.scales[0], rows[(n + 1) & 1], tok, c, a.D);
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&v_empty[st]), ph ^ 1u)) || abort_flag) abort_flag = 1;
      vv.store(sv + st * S::kv_tile, tok, c);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(smem_u32(&v_full[st]));
      if (n + 1 < iters) vv.load(a.codes[1], a.scales[1], rows[(n + 1) & 1], tok, c, a.D);
      if (look(n + 2)) break;  // rows[n & 1]: every thread read it for tile n before the last look
    }
  } else if (warp == W_MMA) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    const uint32_t id_qk = idesc_f16(kMx, false, NT), id_pv = idesc_f16(kMx, true, a.D);
    bool ok = true;
    auto qk = [&](int t, int32_t n) {
      if (leader) {
        const uint64_t da = smem_desc(sq + t * S::q_tile, 16, S::group, 2);
        const uint64_t db = smem_desc(sk + ((uint32_t)n % ST) * S::kv_tile, 16, S::group, 2);
        for (uint32_t j = 0; j < kchunks; ++j) {
          const uint64_t off = ((j >> 2) * 1024u + (j & 3u) * 32u) >> 4;
          mma_ss(tmem + S::tm_s + 128u * t, da + off, db + off, id_qk, j != 0);
        }
        mma_commit(smem_u32(&s_full[t]));
      }
      __syncwarp();
    };
    auto wait = [&](uint64_t& bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity)) && !abort_flag;
      tc_fence_after();
      return ok;
    };
    if (iters > 0 && wait(k_full[0], 0)) {
      for (int t = 0; t < nq; ++t) qk(t, 0);
      if (leader) mma_commit(smem_u32(&k_empty[0]));
    }
    for (int32_t n = 0; n < iters && ok; ++n) {
      const uint32_t st = (uint32_t)n % ST, ph = ((uint32_t)n / ST) & 1u;
      for (int t = 0; t < nq && ok; ++t) {
        if (t == 0 && !wait(v_full[st], ph)) break;
        if (!wait(p_full[t], (uint32_t)n & 1u)) break;
        if (leader) {
          const uint64_t db = smem_desc(sv + st * S::kv_tile, 1024, S::group, 2);
          const uint32_t pa = tmem + S::tm_s + 128u * t, od = tmem + S::tm_o + 128u * t;
          for (uint32_t j = 0; j < NT / 16; ++j) {
            const uint64_t bj = db + ((j * 2u * S::group) >> 4);
            if constexpr (!kMx) {
              mma_ts(od, pa + 8u * j, bj, id_pv, (n | (int32_t)j) != 0);
            } else {
              const uint32_t pj = pa + 32u * (j >> 1) + 8u * (j & 1u);
              mma_ts(od, pj, bj, id_pv, (n | (int32_t)j) != 0);
              mma_ts(od, pj + 16u, bj, id_pv, 1);
            }
          }
          mma_commit(smem_u32(&o_done[t]));
          if (t == nq - 1) mma_commit(smem_u32(&v_empty[st]));
        }
        __syncwarp();
        if (n + 1 < iters) {
          const uint32_t sn = (uint32_t)(n + 1) % ST;
          if (t == 0 && !wait(k_full[sn], ((uint32_t)(n + 1) / ST) & 1u)) break;
          qk(t, n + 1);
          if (t == nq - 1 && leader) mma_commit(smem_u32(&k_empty[sn]));
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) abort_flag = 1;
    // every MMA issued here has completed before TMEM is released
    if (leader) mma_commit(smem_u32(&all_done));
    __syncwarp();
    mbar_wait(smem_u32(&all_done), 0);
  } else if (warp < 4 * nq) {
    // ------------------------------------------------------------ softmax
    const uint32_t tl = tmem + ((32u * ((uint32_t)warp & 3u)) << 16);
    const uint32_t ts_ = tl + S::tm_s + 128u * qt, to = tl + S::tm_o + 128u * qt;
    const uint32_t i = min(r, R - 1u) / a.G;
    const Range see = tile_range(a, s, i, i);
    const uint32_t f0 = r0 + 128u * qt, f1 = min(f0 + 127u, R - 1u);
    const int32_t all_lo = tile_range(a, s, f1 / a.G, f1 / a.G).lo, all_hi = min(end, tile_range(a, s, f0 / a.G, f0 / a.G).hi);
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int32_t n = 0; n < iters; ++n) {
      const int32_t j0 = begin + n * NT;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s_full[qt]), (uint32_t)n & 1u)) || abort_flag) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool masked = any_bad || j0 < all_lo || j0 + NT > all_hi;
      constexpr int NC = NT / 32;
      uint32_t x[2][32];
      if (masked) {  // minus infinity into S itself; few tiles have a border
#pragma unroll 1
        for (int c = 0; c < NC; ++c) {
          tmem_ld32_start(ts_ + 32u * c, x[0]);
          tmem_ld32_wait(x[0]);
          const int32_t jc = j0 + 32 * c;
          const int32_t lo = see.lo - jc, hi = min(see.hi, end) - jc;
          uint32_t in = (lo <= 0 ? ~0u : lo < 32 ? ~0u << lo : 0u) & (hi >= 32 ? ~0u : hi > 0 ? ~(~0u << hi) : 0u);
          if (any_bad)
            for (int e = 0; e < 32; ++e)
              if (((in >> e) & 1u) && (uint32_t)__ldg(table + a.by_page.div((uint32_t)(jc + e))) >= a.num_pages) in &= ~(1u << e);
          uint32_t y[2][16];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e / 16][e % 16] = (in >> e) & 1u ? x[0][e] : 0xFF800000u;
          tmem_st<16>(ts_ + 32u * c, y[0]);
          tmem_st<16>(ts_ + 32u * c + 16u, y[1]);
        }
        tmem_wait_st();
      }
      float top;
      tmem_ld32_start(ts_, x[0]);
      {
        float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          tmem_ld32_wait(x[c & 1]);
          if (c + 1 < NC) tmem_ld32_start(ts_ + 32u * (c + 1), x[(c + 1) & 1]);
#pragma unroll
          for (int e = 0; e < 32; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              t4[k] = max3(t4[k], __uint_as_float(x[c & 1][e + 2 * k]), __uint_as_float(x[c & 1][e + 2 * k + 1]));
        }
        top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
      }
      tmem_ld32_start(ts_, x[0]);
      top = top * fz - (kMx ? 32.0f : 0.0f);
      // the reference moves only when exceeded by 2^8 (see k_kv_decode)
      if (__any_sync(0xffffffffu, top > m + 8.0f)) {
        const float mn = fmaxf(m, top);
        const float f = mn == -INFINITY ? 1.0f : ex2(m - mn);
        m = mn;
        l *= f;
        if (n > 0) {  // O as of the previous tile
          if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&o_done[qt]), (uint32_t)(n - 1) & 1u))) {
            ok = false;
            break;
          }
          tc_fence_after();
          tmem_ld32_wait(x[0]);  // the load above ends before x[1] waits for others
          for (uint32_t c = 0; c < a.D; c += 32u) {
            tmem_ld32_start(to + c, x[1]);
            tmem_ld32_wait(x[1]);
            uint32_t y[2][16];
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e / 16][e % 16] = __float_as_uint(__uint_as_float(x[1][e]) * f);
            tmem_st<16>(to + c, y[0]);
            tmem_st<16>(to + c + 16u, y[1]);
          }
          tmem_wait_st();
        }
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      const uint64_t fz2 = pair(fz, fz), ref2 = pair(-ref, -ref);
      uint64_t l2[2] = {0, 0};
      auto weights = [&](int c, const uint32_t (&z)[32]) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          uint64_t y = fma2(pair(__uint_as_float(z[2 * e]), __uint_as_float(z[2 * e + 1])), fz2, ref2);
          float p0, p1;
          if (e % kPolyEvery == kPolyEvery - 1) {
            y = ex2_poly(y);
            unpair(y, p0, p1);
          } else {
            unpair(y, p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            y = pair(p0, p1);
          }
          l2[e & 1] = add2(l2[e & 1], y);
          if constexpr (!kMx) {
            hi[e] = pack_f16x2(p0, p1);
          } else {
            hi[e] = pack_bf16x2(p0, p1);
            lo[e] = pack_bf16x2(p0 - __uint_as_float(hi[e] << 16), p1 - __uint_as_float(hi[e] & 0xFFFF0000u));
          }
        }
        if constexpr (!kMx) {
          tmem_st<16>(ts_ + 16u * c, hi);
        } else {
          tmem_st<16>(ts_ + 32u * c, hi);
          tmem_st<16>(ts_ + 32u * c + 16u, lo);
        }
      };
#pragma unroll 1  // twice NC / 2: the loop body stays in the instruction cache
      for (int c = 0; c < NC; c += 2) {
        tmem_ld32_wait(x[0]);
        tmem_ld32_start(ts_ + 32u * (c + 1), x[1]);
        weights(c, x[0]);
        tmem_ld32_wait(x[1]);
        if (c + 2 < NC) tmem_ld32_start(ts_ + 32u * (c + 2), x[0]);
        weights(c + 1, x[1]);
      }
      {
        float s0, s1;
        unpair(add2(l2[0], l2[1]), s0, s1);
        l += s0 + s1;
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(smem_u32(&p_full[qt]));
    }
    if (ok && iters > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&o_done[qt]), (uint32_t)(iters - 1) & 1u)) && !abort_flag;
      tc_fence_after();
    }
    if (!ok) {
      if (lane == 0) abort_flag = 1;
    } else {
      const uint32_t h = hk * a.G + (min(r, R - 1u) - i * a.G);
      const uint64_t at = (uint64_t)(s.t0 + i) * a.Hq + h;
      const float fv = kMx ? 0x1p64f : (a.g[1] ? __ldg(a.g[1]) / kGlobalEncode : 1.0f);
      if (m == -INFINITY) l = 0.0f;  // nothing seen (ex2_poly leaves 2^-126)
      const float f = whole ? (l > 0.0f ? fv / l : 0.0f) : fv;
      if (r < R) {
        if (!whole) a.part_ml[(uint64_t)chunk * a.T * a.Hq + at] = make_float2(m, l);
        else if (a.lse) a.lse[at] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
      for (uint32_t c = 0; c < a.D; c += 32u) {
        float x[32];
        if (iters > 0) {
          tmem_ld32(to + c, x);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 0.0f;
        }
        if (r < R)
#pragma unroll
          for (int o = 0; o < 4; ++o) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[octet<MODE>(e)] = x[8 * o + e] * f;
            if (whole)
              store8<QT>(static_cast<QT*>(a.out) + at * a.D + c + 8 * o, v);
            else
              store8<float>(a.part_o + ((uint64_t)chunk * a.T * a.Hq + at) * a.D + c + 8 * o, v);
          }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

}  // namespace pf
}  // namespace kv
}  // namespace nvfp4
