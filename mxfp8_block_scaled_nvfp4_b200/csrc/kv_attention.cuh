// Attention over the paged block-scaled cache (kv_cache.cuh).
//
// Query i of sequence b (n queries over L cached tokens) is at position
// p = L - n + i and sees token j iff j < L, j <= p when causal, and
// j > p - window when window > 0:
//   z_j = scale * q . k_hat_j,  m = max z_j,  P_j = exp(z_j - m),
//   out = sum_j P_j v_hat_j / sum_j P_j,  lse = m + ln(sum_j P_j);
// a query that sees nothing gets out = 0 and lse = -inf.
#pragma once

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

// Value of element d of a cache row.
template <int MODE>
__device__ __forceinline__ float cache_value(const AttnArgs& a, int side, uint64_t row, uint32_t d) {
  const uint32_t s = __ldg(a.scales[side] + row * (a.D / Fmt<MODE>::group) + d / Fmt<MODE>::group);
  if constexpr (MODE == kMX8) {
    return e4m3_to_f32(__ldg(a.codes[side] + row * a.D + d)) * ue8m0_to_f32(s);
  } else {
    const uint32_t c = (__ldg(a.codes[side] + row * (a.D / 2u) + d / 2u) >> (4u * (d & 1u))) & 15u;
    return e2m1_value(c) * (MODE == kNV ? e4m3_to_f32(s) : ue8m0_to_f32(s));
  }
}

constexpr int kPlainWarps = 4;

// One CTA per (query, query head); warp w takes tokens w, w + 4, ...; lane l
// holds elements l, l + 32, ... of the row.  The four running (m, l, O) are
// joined at the end.
template <typename T, int MODE>
__global__ void __launch_bounds__(kPlainWarps * 32) k_kv_attention(const __grid_constant__ AttnArgs a) {
  __shared__ float sm[kPlainWarps], sl[kPlainWarps], so[kPlainWarps][256];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t i = blockIdx.x, h = blockIdx.y, b = blockIdx.z, hk = h / a.G;
  Seq s;
  if (!seq_of(a, b, s) || i >= s.n) return;
  const uint32_t t = s.t0 + i;
  const int64_t p = (int64_t)s.L - s.n + i;
  int64_t hi = a.causal ? p + 1 : (int64_t)s.L;
  int64_t lo = a.window ? p - (int64_t)a.window + 1 : 0;
  if (hi > (int64_t)s.L) hi = s.L;
  if (lo < 0) lo = 0;
  const uint32_t nd = a.D / 32u;
  const T* q = static_cast<const T*>(a.q) + (int64_t)t * a.q_stride + (int64_t)h * a.D;
  const float fk = (a.g[0] ? __ldg(a.g[0]) / kGlobalEncode : 1.0f) * a.scale;
  const float fv = a.g[1] ? __ldg(a.g[1]) / kGlobalEncode : 1.0f;
  float qv[8], o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    qv[e] = (uint32_t)e < nd ? Elem<T>::to_f(q[lane + 32u * e]) : 0.0f;
    o[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t j = lo + warp; j < hi; j += kPlainWarps) {
    const uint32_t pg = a.by_page.div((uint32_t)j);
    const int32_t page = __ldg(a.page_table + (uint64_t)b * a.max_pages + pg);
    if (page < 0 || (uint32_t)page >= a.num_pages) {
      atomicOr(&g_device_error, (unsigned)kDevErrIndex);
      continue;
    }
    const uint64_t row = ((uint64_t)page * a.heads + hk) * a.page_size + ((uint32_t)j - pg * a.page_size);
    float z = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if ((uint32_t)e < nd) z = fmaf(qv[e], cache_value<MODE>(a, 0, row, lane + 32u * e), z);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
    z *= fk;
    const float mn = fmaxf(m, z), c = expf(m - mn), pr = expf(z - mn);
    m = mn;
    l = l * c + pr;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if ((uint32_t)e < nd) o[e] = fmaf(pr, cache_value<MODE>(a, 1, row, lane + 32u * e), o[e] * c);
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if ((uint32_t)e < nd) so[warp][lane + 32u * e] = o[e];
  __syncthreads();
  float M = -INFINITY, Lsum = 0.0f;
  for (int w = 0; w < kPlainWarps; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < kPlainWarps; ++w) Lsum += sm[w] == -INFINITY ? 0.0f : sl[w] * expf(sm[w] - M);
  T* out = static_cast<T*>(a.out) + ((uint64_t)t * a.Hq + h) * a.D;
  for (uint32_t d = threadIdx.x; d < a.D; d += kPlainWarps * 32) {
    float v = 0.0f;
    for (int w = 0; w < kPlainWarps; ++w) v += sm[w] == -INFINITY ? 0.0f : so[w][d] * expf(sm[w] - M);
    out[d] = Elem<T>::from_f(Lsum > 0.0f ? v / Lsum * fv : 0.0f);
  }
  if (a.lse && threadIdx.x == 0) a.lse[(uint64_t)t * a.Hq + h] = Lsum > 0.0f ? M + logf(Lsum) : -INFINITY;
}

}  // namespace kv
}  // namespace nvfp4
