// Paged key/value cache held in NVFP4, MXFP8 or MXFP4: writing new tokens
// into their slots and reading slots back.
//
// Layout (K and V alike): codes [pages, heads, page_size, D * bits / 32]
// uint32 words, scales [pages, heads, page_size, D / group] bytes (LINEAR).
// Slot s is row s % page_size of page s / page_size.  A head's rows of one
// page are contiguous, so the attention kernels stream whole pages; a row's
// blocks run along D, so one token is quantized without looking at another.
//
// Mathematics: the per-block arithmetic of k_nvfp4_quantize /
// k_mxfp8_quantize / k_mxfp4_quantize and of the dequantizers, unchanged, so
// codes, scales and values are the same bits those calls give.
//
// Both kernels are bound by memory: reading 65536 NVFP4 rows of 8 x 128 as
// bf16 takes 69 us in a captured graph (5.0 TB/s, 76 % of the copy rate; 71 a
// call), writing 16384 MXFP4 tokens and reading them back 35 (39: two launches).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "quantize.cuh"

namespace nvfp4 {
namespace kv {

// Modes as in nvfp4_mode.
enum { kNV = 0, kMX8 = 1, kMX4 = 2 };

template <int MODE> struct Fmt;
template <> struct Fmt<kNV> { static constexpr uint32_t group = 16, bits = 4; };
template <> struct Fmt<kMX8> { static constexpr uint32_t group = 32, bits = 8; };
template <> struct Fmt<kMX4> { static constexpr uint32_t group = 32, bits = 4; };

constexpr int kRowThreads = 256;

struct RowArgs {
  uint8_t* codes[2];        // K, V
  uint8_t* scales[2];
  const float* g[2];
  const void* x[2];         // write: sources; read: destinations
  int64_t stride[2];        // elements between tokens of x
  const int32_t* slots;
  uint32_t T, heads, D, page_size, num_slots;
  uint32_t units;           // 16-element units of one side: T * heads * D / 16
  FastDiv per_head, per_token, by_page;  // D / 16, heads * D / 16, page_size
};

// Unit u of one side: 16 elements of one row (token t, head h, unit j).
struct Unit {
  uint32_t t, h, j;
};
__device__ __forceinline__ Unit unit_at(const RowArgs& a, uint32_t u) {
  Unit r;
  r.t = a.per_token.div(u);
  const uint32_t w = u - r.t * a.per_token.d;
  r.h = a.per_head.div(w);
  r.j = w - r.h * a.per_head.d;
  return r;
}

// Row index (over pages, heads, page rows) of a slot and head.
__device__ __forceinline__ uint64_t cache_row(const RowArgs& a, uint32_t slot, uint32_t h) {
  const uint32_t page = a.by_page.div(slot), row = slot - page * a.page_size;
  return ((uint64_t)page * a.heads + h) * a.page_size + row;
}

// 16 values rounded to T: 32-byte stores where p allows them (V8; a thread's
// two 16-byte stores fill half of a sector each: reading 65536 NVFP4 rows of
// 8 x 128 took 75 us that way).
template <typename T, bool V8>
__device__ __forceinline__ void store16(T* p, const float (&lo)[8], const float (&hi)[8]) {
  if constexpr (!V8) {
    store8<T>(p, lo);
    store8<T>(p + 8, hi);
  } else if constexpr (sizeof(T) == 4) {
    const float(*h[2])[8] = {&lo, &hi};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float(&v)[8] = *h[i];
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + 8 * i), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                   "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                   : "memory");
    }
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        w[i] = pack_f16x2(lo[2 * i], lo[2 * i + 1]);
        w[4 + i] = pack_f16x2(hi[2 * i], hi[2 * i + 1]);
      } else {
        w[i] = pack_bf16x2(lo[2 * i], lo[2 * i + 1]);
        w[4 + i] = pack_bf16x2(hi[2 * i], hi[2 * i + 1]);
      }
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                 "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  }
}

// One thread per 16 elements; the MX modes' 32-element blocks take two
// neighbouring lanes (units 2i, 2i + 1 of a row: D % 32 == 0).
// V8: 256-bit loads (rows 32-byte aligned).
template <typename T, int MODE, bool V8>
__global__ void __launch_bounds__(kRowThreads) k_kv_write(const __grid_constant__ RowArgs a) {
  const uint32_t u = blockIdx.x * kRowThreads + threadIdx.x;
  const int side = (int)blockIdx.y;
  const bool in = u < a.units;
  const Unit w = unit_at(a, in ? u : 0);
  const int32_t slot = in ? __ldg(a.slots + w.t) : -1;
  const bool store = slot >= 0 && (uint32_t)slot < a.num_slots;
  if (slot >= 0 && !store) atomicOr(&g_device_error, (unsigned)kDevErrIndex);
  float v[16];
  {
    const T* x = static_cast<const T*>(a.x[side]) + (int64_t)w.t * a.stride[side] + (int64_t)w.h * a.D + w.j * 16u;
    RawBlk<T> raw;
    if (store) {
      load_blk<T, V8>(x, raw);
    } else {
#pragma unroll
      for (int i = 0; i < (int)(sizeof(raw.w) / 16); ++i) raw.w[i] = make_uint4(0, 0, 0, 0);
    }
    unpack16<T>(raw, v);
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
  uint32_t s;
  float k;
  if constexpr (MODE == kNV) {
    const float E = a.g[side] ? kGlobalEncode / __ldg(a.g[side]) : 1.0f;
    float t = m / kE2M1Max;
    t = t * E;
    s = f32_to_e4m3(t);
    const float fs = e4m3_to_f32(s);
    k = fs != 0.0f ? E / fs : 0.0f;
  } else {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    s = f32_to_ue8m0_rp(m / (MODE == kMX8 ? kE4M3Max : kE2M1Max));
    k = 1.0f / ue8m0_to_f32(s);
  }
  if (!store) return;
  const uint64_t row = cache_row(a, (uint32_t)slot, w.h);
  uint8_t* codes = a.codes[side] + row * (a.D * Fmt<MODE>::bits / 8u) + w.j * (2u * Fmt<MODE>::bits);
  if constexpr (MODE == kMX8) {
    uint4 q;
    q.x = f32x4_to_e4m3x4(v[0] * k, v[1] * k, v[2] * k, v[3] * k);
    q.y = f32x4_to_e4m3x4(v[4] * k, v[5] * k, v[6] * k, v[7] * k);
    q.z = f32x4_to_e4m3x4(v[8] * k, v[9] * k, v[10] * k, v[11] * k);
    q.w = f32x4_to_e4m3x4(v[12] * k, v[13] * k, v[14] * k, v[15] * k);
    *reinterpret_cast<uint4*>(codes) = q;
  } else {
    uint2 q = make_uint2(0u, 0u);
    if (MODE != kNV || s != 0u) {  // a zero NVFP4 scale stores zero codes
      q.x = scaled_e2m1x8_at(v, 0, k);
      q.y = scaled_e2m1x8_at(v, 8, k);
    }
    *reinterpret_cast<uint2*>(codes) = q;
  }
  const uint32_t blocks = a.D / Fmt<MODE>::group;
  if (MODE == kNV || (w.j & 1u) == 0)
    a.scales[side][row * blocks + w.j * 16u / Fmt<MODE>::group] = (uint8_t)s;
}

// One thread per 16 elements; a negative slot gives a zero row, a slot past
// the cache a zero row and the device error word.
template <typename T, int MODE, bool V8>
__global__ void __launch_bounds__(kRowThreads) k_kv_read(const __grid_constant__ RowArgs a) {
  const uint32_t u = blockIdx.x * kRowThreads + threadIdx.x;
  const int side = (int)blockIdx.y;
  if (u >= a.units) return;
  const Unit w = unit_at(a, u);
  const int32_t slot = __ldg(a.slots + w.t);
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) lo[i] = hi[i] = 0.0f;
  if (slot >= 0 && (uint32_t)slot < a.num_slots) {
    const uint64_t row = cache_row(a, (uint32_t)slot, w.h);
    const uint8_t* codes = a.codes[side] + row * (a.D * Fmt<MODE>::bits / 8u) + w.j * (2u * Fmt<MODE>::bits);
    const uint32_t s = __ldg(a.scales[side] + row * (a.D / Fmt<MODE>::group) + w.j * 16u / Fmt<MODE>::group);
    float f;
    if constexpr (MODE == kNV) {
      const float d = a.g[side] ? __ldg(a.g[side]) / kGlobalEncode : 1.0f;
      f = e4m3_to_f32(s) * d;
    } else {
      f = ue8m0_to_f32(s);
    }
    if constexpr (MODE == kMX8) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(codes));
      float c[4];
      const uint32_t words[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e4m3x4_to_f32(words[i], c);
#pragma unroll
        for (int e = 0; e < 4; ++e) (i < 2 ? lo : hi)[(i & 1) * 4 + e] = c[e] * f;
      }
    } else {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(codes));
      e2m1x8_to_f32(q.x, lo);
      e2m1x8_to_f32(q.y, hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo[i] *= f;
        hi[i] *= f;
      }
    }
  } else if (slot >= 0) {
    atomicOr(&g_device_error, (unsigned)kDevErrIndex);
  }
  T* x = static_cast<T*>(const_cast<void*>(a.x[side])) + (int64_t)w.t * a.stride[side] + (int64_t)w.h * a.D + w.j * 16u;
  store16<T, V8>(x, lo, hi);
}

}  // namespace kv
}  // namespace nvfp4
