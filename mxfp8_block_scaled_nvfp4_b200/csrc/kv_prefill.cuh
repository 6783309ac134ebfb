// kv_attention for many query rows: tcgen05 matrix products with S and O in
// tensor memory (formulas and partial results as in kv_attention.cuh).
//
// A CTA holds one or two tiles of 128 query rows (row r of a sequence and a
// key/value head is query r / G, head r % G of the group) and walks the
// tokens in tiles of NT:
//   warps 0-7       producers: cache codes to 16-bit K_hat and V_hat tiles in
//                   shared memory (each decoded once for both query tiles).  A
//                   thread owns a part of a token: it copies its codes and scales
//                   (cp.async) into its own slots a tile ahead and decodes them
//                   from there, so the threads need no barrier; K and V run
//                   through the same loop body, which keeps it small (with the
//                   bodies unrolled the producers waited for instructions)
//   warp 8          allocates TMEM and issues the MMAs
//   warps 12-19, 20-27 softmax of query tile 0, 1; a row (TMEM lane) has two
//                   threads, one for each half of the tile's tokens
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
// Measured: 4096 queries over 8192 tokens (NVFP4, 32 / 8 heads of 128, causal)
// 503 us, 819 TFLOP/s or 49 % of the bf16 burst rate, at an SM clock of 1.83 GHz
// (by the SMs' own counter; 970 W).  With 148 CTAs of two query tiles, a tile of
// 128 tokens takes 2.78 us, about 5000 clocks for 2048 of products (MXFP4 3.38,
// MXFP8 3.95, which have half as many products again), and a CTA 11 us besides:
// the chain from S over the exponentials to P V and the next S bounds it.  Tiles
// of 64 tokens with two S buffers hid more of the chain, but an N = 64 product
// takes as long as an N = 128 one (671 us).
//
// Number formats as in k_kv_decode: NVFP4 exact fp16 operands, P times 2^7 in
// fp16; MX modes exact bf16 operands and P in two bf16 terms, each with its own
// MMA.  (fp16 queries over an MX cache would need two terms of Q as well; they
// stay with k_kv_decode.)
#pragma once

#include "kv_attention.cuh"
#include "qqmm_sm100.cuh"

namespace nvfp4 {
namespace kv {
namespace pf {

using namespace tc;

constexpr int W_MMA = 8, W_SOFT = 12, THREADS = 28 * 32, PROD = 256;

template <int MODE, int DP>
struct Shape {
  static constexpr int NQ = DP == 256 ? 1 : 2;        // query tiles a CTA
  static constexpr int NT = DP == 256 ? 64 : 128;     // tokens a tile
  static constexpr int HC = NT / 2;                   // tokens of a softmax thread
  static constexpr uint32_t group = DP / 64 * 1024;   // an 8-row group
  static constexpr uint32_t q_tile = 16 * group;      // 128 rows
  static constexpr uint32_t kv_tile = NT / 8 * group;
  // tiles in shared memory: two of K and V, but one of V where MXFP8's raw codes take the room
  static constexpr uint32_t st_k = 2, st_v = MODE == kMX8 && DP >= 128 ? 1 : 2;
  static constexpr int EPT = DP * NT / PROD;          // elements of a producer thread: 32 or 64
  static constexpr uint32_t raw_codes = PROD * EPT * Fmt<MODE>::bits / 8u, raw = raw_codes + 8u * PROD;
  static constexpr uint32_t at_k = NQ * q_tile, at_v = at_k + st_k * kv_tile, at_raw = at_v + st_v * kv_tile;
  // at least half an SM's: a CTA takes all of TMEM, so one fits at a time
  static constexpr uint32_t bytes = at_raw + 2 * raw + 1024, smem = bytes < 122880 ? 122880 : bytes;
  static constexpr uint32_t tm_s = 0, tm_o = 256;     // TMEM columns: S of tile t at 128 t, O at 256 + 128 t
};

// Through L1, unlike copy16: a thread's 16-byte pieces are parts of lines that
// its neighbours read too (2048 over 4096 tokens MXFP8 204 us, past L1 214;
// MXFP4 170 and 173, NVFP4 139 and 141; 4096 over 8192 NVFP4 503 and 499).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ void st_shared_u8(uint32_t at, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(v) : "memory");
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
// Eight codes (one word, MXFP8 two) times the pair f of factors.
template <int MODE, bool BIG>
__device__ __forceinline__ uint4 decode8(const uint32_t* w, uint32_t f, uint32_t up) {
  if constexpr (MODE == kNV) {
    uint32_t v[4];
    e2m1x8_to_f16x2(w[0], v);
    return make_uint4(mul_f16x2(v[0], f), mul_f16x2(v[1], f), mul_f16x2(v[2], f), mul_f16x2(v[3], f));
  } else if constexpr (MODE == kMX4) {
    return make_uint4(mx_pair<MODE, 0, BIG>(w[0], f, up), mx_pair<MODE, 1, BIG>(w[0], f, up),
                      mx_pair<MODE, 2, BIG>(w[0], f, up), mx_pair<MODE, 3, BIG>(w[0], f, up));
  } else {
    return make_uint4(mx_pair<MODE, 0, BIG>(w[0], f, up), mx_pair<MODE, 1, BIG>(w[0], f, up),
                      mx_pair<MODE, 0, BIG>(w[1], f, up), mx_pair<MODE, 1, BIG>(w[1], f, up));
  }
}

// A producer thread's slots of one side: its codes, 16-byte piece k at
// [k][thread], and the one or two aligned 32-bit words that hold its scales
// (two where a row's scale bytes are no multiple of four).
template <int MODE, int DP>
struct Raw {
  using S = Shape<MODE, DP>;
  static constexpr int pieces = S::EPT * (int)Fmt<MODE>::bits / 128, units = S::EPT / 32;
  static constexpr uint32_t nb = S::EPT / Fmt<MODE>::group;  // scale bytes
  // Starts the copies of cache row `row`, elements e0 .. e0 + EPT; returns the
  // scales' offset in their first word.
  static __device__ __forceinline__ uint32_t fetch(const AttnArgs& a, const uint8_t* codes, const uint8_t* scales, uint64_t row,
                                                   uint32_t e0, uint32_t at, uint32_t p) {
    const uint8_t* c = codes + row * (a.D * Fmt<MODE>::bits / 8u) + e0 * Fmt<MODE>::bits / 8u;
#pragma unroll
    for (int k = 0; k < pieces; ++k)
      if (e0 + (uint32_t)k * (128u / Fmt<MODE>::bits) < a.D) cp_async16(at + (k * PROD + p) * 16u, c + 16 * k);
    const uint64_t off = row * (a.D / Fmt<MODE>::group) + e0 / Fmt<MODE>::group;
    const uint32_t first = (uint32_t)off & 3u, to = at + S::raw_codes + 8u * p;
    const uint64_t w = off - first;
    if (e0 >= a.D) return first;
    if (w + 8u <= a.scale_bytes) {
      cp_async4(to, scales + w);
      if (first + nb > 4u) cp_async4(to + 4u, scales + w + 4u);
    } else {  // the buffer ends inside the words
      for (uint32_t i = 0; w + i < a.scale_bytes; ++i) st_shared_u8(to + i, __ldg(scales + w + i));
    }
    return first;
  }
  // Decodes the slots into row `tok` of a tile, elements e0 .. e0 + EPT, as
  // 16-byte chunks: eight lanes (eight rows) cover eight chunk places.  up: of
  // the side (Mx).  values: of the values, where drafts that no mask names may
  // hold anything (TREE), and P = 0 does not hide a NaN; what such a key gives is
  // minus infinity before anything reads it, and a key that a query sees may
  // make it NaN.
  template <bool TREE>
  static __device__ __forceinline__ void decode(const AttnArgs& a, uint32_t at, uint32_t p, uint32_t first, bool there, bool values, uint32_t tile,
                                                uint32_t tok, uint32_t e0, uint32_t up) {
    const uint32_t row = tile + (tok >> 3) * S::group + (tok & 7u) * 128u + (e0 >> 6) * 1024u, c0 = (e0 >> 3) & 7u;
    uint32_t s0, s1;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(s0), "=r"(s1) : "r"(at + S::raw_codes + 8u * p));
    uint32_t sc = there ? __funnelshift_r(s0, s1, 8u * first) : 0u;
    if constexpr (TREE && MODE == kNV) {
      if (values) sc = without_nan(sc);
    }
#pragma unroll
    for (int u = 0; u < units; ++u) {
      if (e0 + 32u * u >= a.D) break;
      constexpr int wo = (int)Fmt<MODE>::bits / 4;  // words an octet
      uint32_t w[4 * wo], f[2];
#pragma unroll
      for (int k = 0; k < wo; ++k) {
        const uint4 v = ld_shared_v4(at + ((u * wo + k) * PROD + p) * 16u);
        w[4 * k] = v.x;
        w[4 * k + 1] = v.y;
        w[4 * k + 2] = v.z;
        w[4 * k + 3] = v.w;
      }
      if constexpr (MODE == kNV) {
        const uint32_t pr = e4m3x2_to_f16x2(sc >> (16 * u));
        f[0] = __byte_perm(pr, 0, 0x1010);
        f[1] = __byte_perm(pr, 0, 0x3232);
      } else {
        const uint32_t q = (sc >> (8 * u)) & 255u;
        if (MODE == kMX8 || q > 254u - up) {
          f[0] = mx_factor<true>(q, up) * 0x10001u;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            st_shared_v4(row + (((c0 + (u * 4u + e)) ^ (tok & 7u)) << 4), decode8<MODE, true>(&w[e * wo], f[0], up));
          continue;
        }
        f[0] = f[1] = mx_factor<false>(q, up) * 0x10001u;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        st_shared_v4(row + (((c0 + (u * 4u + e)) ^ (tok & 7u)) << 4), decode8<MODE, false>(&w[e * wo], f[e / 2], up));
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

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
// Barrier of the two warps that share 32 rows.  A warp that gives up, wherever
// it does, arrives once without waiting, after it has set abort_flag: its
// partner may already be at the barrier or get there before it sees the flag,
// and looks at the flag before it gets to the next one.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void pair_leave(int id) { asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory"); }

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
template <typename QT, int MODE, int DP, bool TREE = false>  // TREE: the queries are drafts with masks
__global__ void __launch_bounds__(THREADS, 1) k_kv_prefill(const __grid_constant__ AttnArgs a) {
  using S = Shape<MODE, DP>;
  constexpr int NQ = S::NQ, NT = S::NT;
  constexpr bool kMx = MODE != kNV;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[2][2], empty[2][2], s_full[2], p_full[2], o_done[2], all_done;  // full, empty: [side][stage]
  __shared__ float other[NQ][2][128];  // maxima (later sums) that the two threads of a row exchange
  __shared__ float row_factor[NQ][128];  // logit (log2 units) of an accumulator
  __shared__ float2 slot_ml[TREE && NQ == 2 ? 2 : 1][128];  // maxima and sums that two slots of the same rows exchange
  __shared__ uint32_t tmem_holder;
  __shared__ volatile int abort_flag;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sq = sbase;
  const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31u);

  // heaviest tiles first, over all heads and sequences: the last queries of a
  // causal prompt see most
  const uint32_t per_tile = a.chunks * a.B * a.heads;
  uint32_t at = blockIdx.x;
  const uint32_t tile = gridDim.x / per_tile - 1u - at / per_tile;
  at %= per_tile;
  const uint32_t chunk = at / (a.B * a.heads);
  at %= a.B * a.heads;
  const uint32_t b = at / a.heads, hk = at - b * a.heads, r0 = tile * 128u * NQ;
  Seq s;
  if (!seq_of(a, b, s)) return;
  const uint32_t R = s.n * a.G;
  if (r0 >= R) return;
  const uint32_t rl = min(r0 + 128u * NQ, R) - 1u;
  const Range rg = tile_range(a, s, TREE ? 0u : r0 / a.G, rl / a.G);
  const int32_t base = rg.lo & ~15;
  const int32_t span = rg.hi > rg.lo ? rg.hi - base : 0;
  if (chunk > 0 && (int64_t)chunk * a.chunk >= span) return;
  const bool whole = span <= a.chunk;
  const int32_t begin = base + (int32_t)chunk * a.chunk;
  const int32_t end = min(rg.hi, begin + a.chunk);
  const int32_t iters = end > begin ? (end - begin + NT - 1) / NT : 0;
  const int nq = NQ == 2 && r0 + 128u < R ? 2 : 1;
  // Trees of one query tile: the second tile's S, O and threads take every other
  // tile of tokens (slot t those of remainder t), and the two slots join at the
  // end.  A tile of tokens then takes 1.9 us instead of 2.5 (18 trees of 32
  // drafts over 4096 tokens, 32 / 8 heads of 128: 77 us, 99 without).
  constexpr bool DUAL = TREE && NQ == 2;
  const bool dual = DUAL && nq == 1 && iters > 1;
  const int slots = dual ? 2 : nq;
  const int32_t* table = a.page_table + (uint64_t)b * a.max_pages;
  const uint32_t kchunks = a.D / 16u;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&full[i >> 1][i & 1]), W_MMA);
      mbar_init(smem_u32(&empty[i >> 1][i & 1]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), 8);
      mbar_init(smem_u32(&o_done[i]), 1);
    }
    mbar_init(smem_u32(&all_done), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == W_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_holder)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // The producers' first copies: what a copy waits for (lengths, page table) is
  // long beside them, and so are the queries' way into shared memory below.
  using W = Raw<MODE, DP>;
  const uint32_t p = threadIdx.x, tok = p % NT, e0 = p / NT * S::EPT;
  // tile n's token: its page number is loaded a tile before its row is
  // wanted, its codes and scales a tile before they are decoded
  int32_t page = -1;
  auto page_of = [&](int32_t n) {
    const int32_t j = begin + n * NT + (int32_t)tok;
    page = n < iters && j >= rg.lo && j < end ? __ldg(table + a.by_page.div((uint32_t)j)) : -1;
  };
  uint64_t src_row = 0;
  bool there = false;
  auto fetch = [&](int32_t q) {  // tile q / 2, side q % 2
    const int32_t n = q >> 1;
    uint32_t first = 0;
    if (n < iters) {
      if ((q & 1) == 0) {
        const uint32_t j = (uint32_t)(begin + n * NT) + tok;
        there = (uint32_t)page < a.num_pages;
        src_row = there ? ((uint64_t)(uint32_t)page * a.heads + hk) * a.page_size + (j - a.by_page.div(j) * a.page_size) : 0;
        page_of(n + 1);
      }
      // a token that is not there gets row 0's codes, and zero scales when decoded (finite: P = 0 meets them)
      first = W::fetch(a, q & 1 ? a.codes[1] : a.codes[0], q & 1 ? a.scales[1] : a.scales[0], src_row, e0, sbase + S::at_raw + (q & 1) * S::raw, p) | (there ? 4u : 0u);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return first;
  };
  uint32_t cur = 0, next = 0;
  if (warp < W_MMA) {
    page_of(0);
    cur = fetch(0);
    next = fetch(1);
  }
  // pages out of range: the softmax then looks every token up
  int bad = 0;
  if (iters > 0 && warp < W_SOFT) {  // the softmax warps have the queries to bring in
    const uint32_t pg0 = a.by_page.div((uint32_t)max(begin, rg.lo)), pg1 = a.by_page.div((uint32_t)(end - 1));
    for (uint32_t pg = pg0 + threadIdx.x; pg <= pg1; pg += W_SOFT * 32) bad |= (uint32_t)__ldg(table + pg) >= a.num_pages;
    if (bad) atomicOr(&g_device_error, (unsigned)kDevErrIndex);
  }
  // softmax warps: their query tile, half of the tokens, row of the tile
  const int qt = (warp - W_SOFT) >> 3, half = (warp >> 2) & 1;
  const uint32_t row = (uint32_t)(threadIdx.x & 127u);
  const uint32_t r = r0 + 128u * (dual ? 0 : qt) + row;
  const bool softmax = warp >= W_SOFT && qt < slots;
  if (softmax && qt < nq) {
    // A warp brings 16 rows of the queries in, an octet a lane, so that a load
    // reads whole rows (a row a thread kept the load unit busy for 2 us a tile).
    constexpr uint32_t OPR = DP / 8, RPI = 32 / OPR;  // octets of a row, rows a load
    constexpr int LOADS = 16 / RPI, NB = LOADS < 8 ? LOADS : 8;
    const uint32_t o = (uint32_t)lane % OPR;
    const float gk = a.g[0] ? __ldg(a.g[0]) / kGlobalEncode : 1.0f;
    // n / G: the product with 2^32 / G is the quotient or one less
    const uint32_t inv = a.G == 1u ? ~0u : (uint32_t)((1ull << 32) / a.G);
#pragma unroll 1
    for (int k0 = 0; k0 < LOADS; k0 += NB) {
      uint4 raw[NB];
      const uint32_t rr0 = 16u * ((uint32_t)(warp - W_SOFT) & 7u) + RPI * k0 + (uint32_t)lane / OPR;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const uint32_t rq = min(r0 + 128u * qt + rr0 + RPI * k, R - 1u);
        uint32_t i = __umulhi(rq, inv), h = rq - i * a.G;
        if (h >= a.G) {
          ++i;
          h -= a.G;
        }
        h += hk * a.G;
        const QT* q = static_cast<const QT*>(a.q) + (int64_t)(s.t0 + i) * a.q_stride + (int64_t)h * a.D;
        raw[k] = o < a.D / 8u ? __ldg(reinterpret_cast<const uint4*>(q) + o) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const uint32_t rr = rr0 + RPI * k;
        float x[8], mx = 0.0f;
        unpack8<QT>(raw[k], raw[k], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
        for (uint32_t d = OPR / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const int e2 = mx > 0.0f ? max(-80, (int)((__float_as_uint(mx) >> 23) & 255u) - 127) : 0;
        constexpr int up2 = kMx ? 16 : 14;
        const float up = pow2(up2 - e2) * (a.scale < 0.0f ? -1.0f : 1.0f);
        if (o == 0) row_factor[qt][rr] = fmaxf(fabsf(a.scale) * kLog2e * pow2(e2) * gk * pow2(Mx<MODE>::key_down - up2), 1e-37f);
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y0 = x[octet<MODE>(2 * e)] * up, y1 = x[octet<MODE>(2 * e + 1)] * up;
          v[e] = kMx ? pack_bf16x2(y0, y1) : pack_f16x2(y0, y1);
        }
        if (o < a.D / 8u)
          st_shared_v4(sq + qt * S::q_tile + (rr >> 3) * S::group + (o >> 3) * 1024u + (rr & 7u) * 128u + (((o & 7u) ^ (rr & 7u)) << 4),
                       make_uint4(v[0], v[1], v[2], v[3]));
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  tc_fence_before();
  const int any_bad = __syncthreads_or(bad);
  tc_fence_after();
  const uint32_t tmem = tmem_holder;

  if (warp < W_MMA) {
    // ------------------------------------------------------------ producers
#pragma unroll 1
    for (int32_t q = 0; q < 2 * iters; ++q) {
      const uint32_t side = (uint32_t)q & 1u, n = (uint32_t)q >> 1, nst = side ? S::st_v : S::st_k;
      const uint32_t st = n % nst, ph = n / nst & 1u;
      if (!__all_sync(0xffffffffu, wait_for(empty[side][st], ph ^ 1u) && !abort_flag)) {
        abort_flag = 1;
        break;
      }
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      W::template decode<TREE>(a, sbase + S::at_raw + side * S::raw, p, cur & 3u, (cur & 4u) != 0, side != 0,
                               sbase + (side ? S::at_v : S::at_k) + st * S::kv_tile, tok, e0, Mx<MODE>::up(side == 0));
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0 && !(side == 1 && warp == 0 && withheld_stage(n))) arrive(smem_u32(&full[side][st]));
      cur = next;
      next = fetch(q + 2);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (warp == W_MMA) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    const uint32_t id_qk = idesc_f16(kMx, false, NT), id_pv = idesc_f16(kMx, true, a.D);
    bool ok = true;
    auto qk = [&](int t, int32_t n) {
      if (leader) {
        const uint64_t da = smem_desc(sq + (dual ? 0 : t) * S::q_tile, 16, S::group, 2);
        const uint64_t db = smem_desc(sbase + S::at_k + ((uint32_t)n % S::st_k) * S::kv_tile, 16, S::group, 2);
        for (uint32_t j = 0; j < kchunks; ++j) {
          const uint64_t off = ((j >> 2) * 1024u + (j & 3u) * 32u) >> 4;
          mma_ss(tmem + S::tm_s + 128u * t, da + off, db + off, id_qk, j != 0);
        }
        mma_commit(smem_u32(&s_full[t]));
      }
      __syncwarp();
    };
    auto wait = [&](uint64_t& bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, wait_for(bar, parity) && !abort_flag);
      tc_fence_after();
      return ok;
    };
    // O of slot t, its tile number k, += P V_hat with the V tile in stage st
    auto pv = [&](int t, int32_t k, uint32_t st) {
      const uint64_t db = smem_desc(sbase + S::at_v + st * S::kv_tile, 1024, S::group, 2);
      const uint32_t pa = tmem + S::tm_s + 128u * t, od = tmem + S::tm_o + 128u * t;
      for (uint32_t j = 0; j < NT / 16; ++j) {
        const uint64_t bj = db + ((j * 2u * S::group) >> 4);
        const uint32_t ph = pa + S::HC * (j / (S::HC / 16u)), jh = j % (S::HC / 16u);  // P lies in its half of S
        if constexpr (!kMx) {
          mma_ts(od, ph + 8u * jh, bj, id_pv, (k | (int32_t)j) != 0);
        } else {
          const uint32_t pj = ph + 32u * (jh >> 1) + 8u * (jh & 1u);
          mma_ts(od, pj, bj, id_pv, (k | (int32_t)j) != 0);
          mma_ts(od, pj + 16u, bj, id_pv, 1);
        }
      }
      mma_commit(smem_u32(&o_done[t]));
    };
    if (!dual && iters > 0 && wait(full[0][0], 0)) {
      for (int t = 0; t < nq; ++t) qk(t, 0);
      if (leader) mma_commit(smem_u32(&empty[0][0]));
    }
    for (int32_t n = 0; !dual && n < iters && ok; ++n) {
      const uint32_t st = (uint32_t)n % S::st_v, ph = ((uint32_t)n / S::st_v) & 1u;
      for (int t = 0; t < nq && ok; ++t) {
        if (t == 0 && !wait(full[1][st], ph)) break;
        if (!wait(p_full[t], (uint32_t)n & 1u)) break;
        if (leader) {
          pv(t, n, st);
          if (t == nq - 1) mma_commit(smem_u32(&empty[1][st]));
        }
        __syncwarp();
        if (n + 1 < iters) {
          const uint32_t sn = (uint32_t)(n + 1) % S::st_k;
          if (t == 0 && !wait(full[0][sn], ((uint32_t)(n + 1) / S::st_k) & 1u)) break;
          qk(t, n + 1);  // behind P V in the thread's order: P is read before S takes its place
          if (t == nq - 1 && leader) mma_commit(smem_u32(&empty[0][sn]));
        }
        __syncwarp();
      }
    }
    if constexpr (DUAL) {
      // tile n is slot n % 2's
      auto next_qk = [&](int32_t n) {
        const uint32_t sn = (uint32_t)n % S::st_k;
        if (!wait(full[0][sn], ((uint32_t)n / S::st_k) & 1u)) return;
        qk(n & 1, n);
        if (leader) mma_commit(smem_u32(&empty[0][sn]));
        __syncwarp();
      };
      for (int32_t n = 0; dual && n < 2 && ok; ++n) next_qk(n);
      for (int32_t n = 0; dual && n < iters && ok; ++n) {
        const int t = n & 1;
        const uint32_t st = (uint32_t)n % S::st_v;
        if (!wait(full[1][st], ((uint32_t)n / S::st_v) & 1u) || !wait(p_full[t], (uint32_t)(n >> 1) & 1u)) break;
        if (leader) {
          pv(t, n >> 1, st);
          mma_commit(smem_u32(&empty[1][st]));
        }
        __syncwarp();
        if (n + 2 < iters) next_qk(n + 2);
      }
    }
    if (!ok && lane == 0) abort_flag = 1;
    // every MMA issued here has completed before TMEM is released
    if (leader) mma_commit(smem_u32(&all_done));
    __syncwarp();
    wait_for(all_done, 0, kDrainPolls);
  } else if (softmax) {
    // ------------------------------------------------------------ softmax
    const uint32_t tl = tmem + ((32u * ((uint32_t)warp & 3u)) << 16);
    const uint32_t ts_ = tl + S::tm_s + 128u * qt + S::HC * half, to = tl + S::tm_o + 128u * qt;
    const uint32_t i = min(r, R - 1u) / a.G;
    const float fz = row_factor[dual ? 0 : qt][row];
    const int32_t mine = dual ? (iters - qt + 1) / 2 : iters;  // tiles of this slot
    const Range see = TREE ? tree_range(a, s, i) : tile_range(a, s, i, i);
    const uint32_t f0 = r0 + 128u * qt, f1 = min(f0 + 127u, R - 1u);
    int32_t all_lo = tile_range(a, s, f1 / a.G, f1 / a.G).lo, all_hi = min(end, tile_range(a, s, f0 / a.G, f0 / a.G).hi);
    if constexpr (TREE) {
      const Range all = tree_common(a, s);
      all_lo = all.lo;
      all_hi = min(end, all.hi);
    }
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    auto leave = [&]() {
      abort_flag = 1;
      __threadfence_block();
      pair_leave(2 + 4 * qt + (warp & 3));
      return false;
    };
    for (int32_t n = 0; n < mine; ++n) {
      const int32_t j0 = begin + (dual ? 2 * n + qt : n) * NT + S::HC * half;
      if (!__all_sync(0xffffffffu, wait_for(s_full[qt], (uint32_t)n & 1u) && !abort_flag)) {
        ok = leave();
        break;
      }
      tc_fence_after();
      constexpr int NC = S::HC / 32;
      uint32_t x[32];
      if (any_bad || j0 < all_lo || j0 + S::HC > all_hi) {  // minus infinity into S itself; few tiles have a border
#pragma unroll 1
        for (int c = 0; c < NC; ++c) {
          tmem_ld32_start(ts_ + 32u * c, x);
          tmem_ld32_wait(x);
          const int32_t jc = j0 + 32 * c;
          const int32_t lo = see.lo - jc, hi = min(see.hi, end) - jc;
          uint32_t in = (lo <= 0 ? ~0u : lo < 32 ? ~0u << lo : 0u) & (hi >= 32 ? ~0u : hi > 0 ? ~(~0u << hi) : 0u);
          if constexpr (TREE) in &= tree_bits(a, s, tree_mask(a, s, i), jc);
          if (any_bad)
            for (int e = 0; e < 32; ++e)
              if (((in >> e) & 1u) && (uint32_t)__ldg(table + a.by_page.div((uint32_t)(jc + e))) >= a.num_pages) in &= ~(1u << e);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = (in >> (16 * k + e)) & 1u ? x[16 * k + e] : 0xFF800000u;
            tmem_st<16>(ts_ + 32u * c + 16u * k, y);
          }
        }
        tmem_wait_st();
      }
      float top;
      {
        float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          tmem_ld32_start(ts_ + 32u * c, x);
          tmem_ld32_wait(x);
#pragma unroll
          for (int e = 0; e < 32; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) t4[k] = max3(t4[k], __uint_as_float(x[e + 2 * k]), __uint_as_float(x[e + 2 * k + 1]));
        }
        top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
      }
      tmem_ld32_start(ts_, x);
      // the row's other thread has the other half's maximum
      // (its slot was read before the P that this S followed)
      other[qt][half][row] = top;
      pair_sync(2 + 4 * qt + (warp & 3));
      top = fmaxf(top, other[qt][half ^ 1][row]) * fz - kUp<MODE>;
      tmem_ld32_wait(x);
      // the reference moves only when exceeded by 2^8 (see k_kv_decode)
      if (__any_sync(0xffffffffu, top > m + 8.0f)) {
        const float mn = fmaxf(m, top);
        const float f = mn == -INFINITY ? 1.0f : ex2(m - mn);
        m = mn;
        l *= f;
        if (n > 0) {  // O as of the previous tile, half of the columns each
          if (!__all_sync(0xffffffffu, wait_for(o_done[qt], (uint32_t)(n - 1) & 1u))) {
            ok = leave();
            break;
          }
          tc_fence_after();
          for (uint32_t c = 16u * half; c < a.D; c += 32u) {
            uint32_t y[16];
            tmem_ld16(to + c, y);
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
            tmem_st<16>(to + c, y);
          }
          tmem_wait_st();
        }
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      const uint64_t fz2 = pair(fz, fz), ref2 = pair(-ref, -ref);
      uint64_t l2[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (c > 0) {
          tmem_ld32_start(ts_ + 32u * c, x);
          tmem_ld32_wait(x);
        }
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint64_t y = fma2(pair(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), fz2, ref2);
          float p0, p1;
          unpair(y, p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          l2[e & 1] = add2(l2[e & 1], pair(p0, p1));
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
      if (!__all_sync(0xffffffffu, wait_for(o_done[qt], (uint32_t)(mine - 1) & 1u) && !abort_flag)) ok = leave();
      if (dual && ok && !__all_sync(0xffffffffu, wait_for(o_done[qt ^ 1], (uint32_t)((iters - (qt ^ 1) + 1) / 2 - 1) & 1u) && !abort_flag)) ok = leave();
      tc_fence_after();
    }
    // A warp that gave up arrives at the slots' barrier too.
    auto slots_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(10 + (warp & 3)) : "memory"); };
    if (dual && !ok) asm volatile("bar.arrive %0, 128;" ::"r"(10 + (warp & 3)) : "memory");
    if (ok) {
      // the row's sum (the slots were last read before the last P)
      other[qt][half][row] = l;
      pair_sync(2 + 4 * qt + (warp & 3));
      l += other[qt][half ^ 1][row];
      float f_mine = 1.0f, f_other = 0.0f;  // of the two slots' O
      if (dual) {
        if (half == 0) slot_ml[DUAL ? qt : 0][row] = make_float2(m, l);
        slots_sync();
        const float2 ml = slot_ml[DUAL ? qt ^ 1 : 0][row];
        const float M = fmaxf(m, ml.x);
        f_mine = m == -INFINITY ? 0.0f : ex2(m - M);
        f_other = ml.x == -INFINITY ? 0.0f : ex2(ml.x - M);
        l = l * f_mine + ml.y * f_other;
        m = M;
      }
      const uint32_t h = hk * a.G + (min(r, R - 1u) - i * a.G);
      const uint64_t at = (uint64_t)(s.t0 + i) * a.Hq + h;
      const float fv = kMx ? 1.0f : (a.g[1] ? __ldg(a.g[1]) / kGlobalEncode : 1.0f);
      const float f = whole ? (l == 0.0f ? 0.0f : fv / l) : fv;
      if (r < R && half == 0 && (!dual || qt == 0)) {
        if (!whole) a.part_ml[(uint64_t)chunk * a.T * a.Hq + at] = make_float2(m, l);
        else if (a.lse) a.lse[at] = lse_of(m, l);
      }
      const bool wide = ((whole ? reinterpret_cast<uintptr_t>(a.out) : reinterpret_cast<uintptr_t>(a.part_o)) & 31u) == 0;
      // 16 columns at a time, in turn over the two or four threads that have the row
      for (uint32_t c = 16u * (dual ? 2 * qt + half : half); c < a.D; c += dual ? 64u : 32u) {
        uint32_t y[16];
        if (iters > 0) {
          tmem_ld16(to + c, y);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = 0;
        }
        if constexpr (DUAL) {
          if (dual) {
            uint32_t z[16];
            tmem_ld16(tl + S::tm_o + 128u * (qt ^ 1) + c, z);
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f_mine + __uint_as_float(z[e]) * f_other);
          }
        }
        if (r < R) {
          float v[2][8];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e / 8][octet<MODE>(e % 8)] = __uint_as_float(y[e]) * f;
          if (whole) {
            QT* o = static_cast<QT*>(a.out) + at * a.D + c;
            if (wide) store16<QT, true>(o, v[0], v[1]);
            else store16<QT, false>(o, v[0], v[1]);
          } else {
            float* o = a.part_o + ((uint64_t)chunk * a.T * a.Hq + at) * a.D + c;
            if (wide) store16<float, true>(o, v[0], v[1]);
            else store16<float, false>(o, v[0], v[1]);
          }
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
