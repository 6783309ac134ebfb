// New tokens into the paged block-scaled cache (kv_cache.cuh) with the
// rotation of queries and keys by their positions on the way, and rows of the
// cache to other slots.
//
// Rotation of a head's first `rot` elements, c and s the table's rows of the
// token's position:
//   (a, b) -> (fp32(fp32(a c) - fp32(b s)), fp32(fp32(b c) + fp32(a s)))
// with (a, b) = elements (i, i + rot/2), or (2i, 2i + 1) when interleaved.
// Products and sums are rounded one by one (no fused multiply-add), so that
// the codes of the rotated keys are fixed by the definition; the rotated keys
// are quantized as fp32 numbers, the rotated queries rounded to their type.
#pragma once

#include "common.cuh"
#include "kv_cache.cuh"
#include "norm.cuh"

namespace nvfp4 {
namespace kv {

struct AppendArgs {
  RowArgs r;                // K and V; r.slots
  const void* q;            // [T, Hq, D], q_stride elements between tokens
  void* q_out;              // [T, Hq, D]
  int64_t q_stride;
  const float* cs[2];       // cos, sin [max_pos, rot / 2]
  const int32_t* positions;
  uint32_t max_pos, rot;
  int interleaved;
  uint32_t Hq, q_groups;    // groups of heads that one thread takes
  uint32_t q_units, q_ctas, kv_ctas;  // threads of Q; CTAs of Q, of K and of V
  FastDiv q_per_token;      // q_groups * D / 16
};

__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = u;
}

// Elements e .. e + 8 of a head, rotated.
template <typename T>
__device__ __forceinline__ void turn8(const AppendArgs& a, const T* head, uint32_t pos, uint32_t e, float* v) {
  if (e >= a.rot) return;
  const uint32_t half = a.rot / 2u;
  const float* cr = a.cs[0] + (uint64_t)pos * half;
  const float* sr = a.cs[1] + (uint64_t)pos * half;
  if (a.interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cr + e / 2u)), s = __ldg(reinterpret_cast<const float4*>(sr + e / 2u));
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) turn(v[2 * i], v[2 * i + 1], cc[i], ss[i]);
    return;
  }
  const bool low = e < half;
  const uint32_t at = low ? e : e - half;
  float o[8], c[8], s[8];
  load8<T>(head + (low ? e + half : at), o);
  load8<float>(cr + at, c);
  load8<float>(sr + at, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = __fmul_rn(v[i], c[i]), y = __fmul_rn(o[i], s[i]);
    v[i] = low ? __fsub_rn(x, y) : __fadd_rn(x, y);
  }
}

// A thread's 16 elements of a query head: eight and their partners, so that
// nothing is loaded twice; HEADS heads of a token, which share the angles.
template <typename T, int HEADS>
__device__ __forceinline__ void turn_queries(const AppendArgs& a, uint32_t u) {
  if (u >= a.q_units) return;
  const uint32_t t = a.q_per_token.div(u), y = u - t * a.q_per_token.d;
  const uint32_t grp = a.r.per_head.div(y), j = y - grp * a.r.per_head.d;
  const int32_t slot = __ldg(a.r.slots + t), pos = __ldg(a.positions + t);
  const uint32_t half = a.rot / 2u, D = a.r.D, h0 = grp * HEADS;
  const bool turns = j * 16u < a.rot, pairs = turns && !a.interleaved;
  const uint32_t e0 = pairs ? j * 8u : j * 16u, e1 = pairs ? e0 + half : e0 + 8u;
  const T* q = static_cast<const T*>(a.q) + (int64_t)t * a.q_stride + (int64_t)h0 * D;
  T* out = static_cast<T*>(a.q_out) + ((int64_t)t * a.Hq + h0) * D;
  constexpr int W = sizeof(T) == 4 ? 2 : 1;
  uint4 x[HEADS][2][W];  // (loaded beside slot and position, which may yet say that the token is skipped)
#pragma unroll
  for (int h = 0; h < HEADS; ++h)
    if (h0 + h < a.Hq)
#pragma unroll
      for (int w = 0; w < W; ++w) {
        x[h][0][w] = __ldg(reinterpret_cast<const uint4*>(q + h * D + e0) + w);
        x[h][1][w] = __ldg(reinterpret_cast<const uint4*>(q + h * D + e1) + w);
      }
  if (slot < 0) return;
  if ((uint32_t)slot >= a.r.num_slots || (uint32_t)pos >= a.max_pos) {
    atomicOr(&g_device_error, (unsigned)kDevErrIndex);
    return;
  }
  float c[8], s[8];
  if (turns) {
    load8<float>(a.cs[0] + (uint64_t)pos * half + j * 8u, c);
    load8<float>(a.cs[1] + (uint64_t)pos * half + j * 8u, s);
  }
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    if (h0 + h >= a.Hq) return;
    float v[16];
    {
      float lo[8], hi[8];
      unpack8<T>(x[h][0][0], x[h][0][W - 1], lo);
      unpack8<T>(x[h][1][0], x[h][1][W - 1], hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = lo[i];
        v[8 + i] = hi[i];
      }
    }
    if (pairs) {
#pragma unroll
      for (int i = 0; i < 8; ++i) turn(v[i], v[8 + i], c[i], s[i]);
    } else if (turns) {
#pragma unroll
      for (int i = 0; i < 8; ++i) turn(v[2 * i], v[2 * i + 1], c[i], s[i]);
    }
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = v[i];
      hi[i] = v[8 + i];
    }
    store8<T>(out + h * D + e0, lo);
    store8<T>(out + h * D + e1, hi);
  }
}

// CTAs of Q first, then of K, then of V; of these a thread has 16 elements.
// Bound by memory latency: slot and position, then the angles.  16384 tokens of
// 32 query and 8 key/value heads of 128 to MXFP4, 64 elements turning: 71 us, 76
// % of the copy rate (102 with a thread for every 16 elements of Q and its loads
// behind the slot).  To NVFP4 with all 128 turning, 74 % of it: 74 us, and one
// head a thread / four: 64 tokens 2.8 / 3.0 us, 1024 5.9 / 5.4 (5.9 / 6.1 in
// neighbouring pairs), 2048 14.6 / 12.2, 16384 96 / 75.
template <typename T, int MODE, bool V8, int HEADS>
__global__ void __launch_bounds__(kRowThreads) k_kv_append(const __grid_constant__ AppendArgs a) {
  if (blockIdx.x < a.q_ctas) {
    turn_queries<T, HEADS>(a, blockIdx.x * kRowThreads + threadIdx.x);
    return;
  }
  const uint32_t side = blockIdx.x - a.q_ctas >= a.kv_ctas ? 1u : 0u;
  const uint32_t u = (blockIdx.x - a.q_ctas - side * a.kv_ctas) * kRowThreads + threadIdx.x;
  const bool in = u < a.r.units;
  const Unit w = unit_at(a.r, in ? u : 0u);
  const T* head = static_cast<const T*>(a.r.x[side]) + (int64_t)w.t * a.r.stride[side] + (int64_t)w.h * a.r.D;
  RawBlk<T> raw;
  load_blk<T, V8>(head + w.j * 16u, raw);
  const int32_t slot = in ? __ldg(a.r.slots + w.t) : -1;
  const int32_t pos = in ? __ldg(a.positions + w.t) : 0;
  const bool bad = slot >= 0 && ((uint32_t)slot >= a.r.num_slots || (uint32_t)pos >= a.max_pos);
  if (bad) atomicOr(&g_device_error, (unsigned)kDevErrIndex);
  const bool go = slot >= 0 && !bad;
  float v[16];
  unpack16<T>(raw, v);
  if (go && side == 0) {
    turn8<T>(a, head, (uint32_t)pos, w.j * 16u, v);
    turn8<T>(a, head, (uint32_t)pos, w.j * 16u + 8u, v + 8);
  }
  const float E = MODE == kNV && a.r.g[side] ? kGlobalEncode / __ldg(a.r.g[side]) : 1.0f;
  uint4 q;
  const uint32_t s = norm::encode<MODE>(v, E, q);
  if (!go) return;
  const uint64_t row = cache_row(a.r, (uint32_t)slot, w.h);
  uint8_t* codes = a.r.codes[side] + row * (a.r.D * Fmt<MODE>::bits / 8u) + w.j * (2u * Fmt<MODE>::bits);
  if constexpr (MODE == kMX8) *reinterpret_cast<uint4*>(codes) = q;
  else *reinterpret_cast<uint2*>(codes) = make_uint2(q.x, q.y);
  if (MODE == kNV || (w.j & 1u) == 0)
    a.r.scales[side][row * (a.r.D / Fmt<MODE>::group) + w.j * 16u / Fmt<MODE>::group] = (uint8_t)s;
}

// ---------------------------------------------------------------------------
// Moves.  A thread has one piece (at most 16 bytes of one head's codes or
// scales) of the keys' rows and the same of the values', of one move, or, where
// the moves of a sequence take effect one after the other, of all of them: no
// two threads then touch the same bytes.  Such a thread reads the pieces of
// kMoves moves before it writes them, and takes a piece that an earlier one of
// them writes from there.
// ---------------------------------------------------------------------------
constexpr int kMoves = 8;

struct MoveArgs {
  uint8_t* codes[2];
  uint8_t* scales[2];
  const int32_t* src;
  const int32_t* dst;
  const int32_t* starts;    // [S + 1] or NULL (move s is sequence s)
  uint32_t M, S, heads, page_size, num_slots;
  uint32_t row[2];          // bytes of a row's codes, of its scales
  uint32_t piece;           // bytes of a scale piece: 1, 2, 4, 8 or 16
  uint32_t code_pieces, pieces;  // of a side's row: of its codes; all
  uint32_t units;           // S * heads * pieces
  FastDiv per_seq, per_head, by_page;
};

__device__ __forceinline__ uint4 load_piece(const uint8_t* p, uint32_t bytes) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (bytes == 16u) {
    v = *reinterpret_cast<const uint4*>(p);
  } else if (bytes == 8u) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    v.x = x.x;
    v.y = x.y;
  } else {
    v.x = bytes == 4u ? *reinterpret_cast<const uint32_t*>(p) : bytes == 2u ? *reinterpret_cast<const uint16_t*>(p) : *p;
  }
  return v;
}
__device__ __forceinline__ void store_piece(uint8_t* p, uint32_t bytes, const uint4& v) {
  if (bytes == 16u) *reinterpret_cast<uint4*>(p) = v;
  else if (bytes == 8u) *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
  else if (bytes == 4u) *reinterpret_cast<uint32_t*>(p) = v.x;
  else if (bytes == 2u) *reinterpret_cast<uint16_t*>(p) = (uint16_t)v.x;
  else *p = (uint8_t)v.x;
}

// Bound by memory latency (the indices, then the rows): 32000 rows of 8 x 128 in
// MXFP8 29 us, 71 % of the copy rate.  Through the ordered kernel, whose threads
// take a sequence's moves eight at a time: 105 as 32000 sequences, 34 as 1000 of
// 32, 707 as 32 of 1000.
template <bool ORDERED>
__global__ void __launch_bounds__(kRowThreads) k_kv_move(const __grid_constant__ MoveArgs a) {
  const uint32_t u = blockIdx.x * kRowThreads + threadIdx.x;
  if (u >= a.units) return;
  const uint32_t s = a.per_seq.div(u), y = u - s * a.per_seq.d, h = a.per_head.div(y), p = y - h * a.per_head.d;
  const bool codes = p < a.code_pieces;
  const uint32_t bytes = codes ? 16u : a.piece, row_bytes = a.row[codes ? 0 : 1];
  const uint32_t first = (codes ? p : p - a.code_pieces) * bytes;
  uint8_t* k = (codes ? a.codes[0] : a.scales[0]) + first;
  uint8_t* v = (codes ? a.codes[1] : a.scales[1]) + first;
  auto at = [&](int32_t slot) {
    const uint32_t page = a.by_page.div((uint32_t)slot);
    return (((uint64_t)page * a.heads + h) * a.page_size + ((uint32_t)slot - page * a.page_size)) * row_bytes;
  };
  // whether move m is made
  auto named = [&](int32_t from, int32_t to) {
    if (from < 0 || to < 0) return false;
    if ((uint32_t)from < a.num_slots && (uint32_t)to < a.num_slots) return true;
    atomicOr(&g_device_error, (unsigned)kDevErrIndex);
    return false;
  };
  if constexpr (!ORDERED) {
    const int32_t from = __ldg(a.src + s), to = __ldg(a.dst + s);
    if (!named(from, to)) return;
    const uint64_t x = at(from), z = at(to);
    const uint4 pk = load_piece(k + x, bytes), pv = load_piece(v + x, bytes);
    store_piece(k + z, bytes, pk);
    store_piece(v + z, bytes, pv);
    return;
  }
  const int64_t m0 = __ldg(a.starts + s), m1 = __ldg(a.starts + s + 1);
  if (m0 < 0 || m1 < m0 || m1 > (int64_t)a.M) {
    atomicOr(&g_device_error, (unsigned)kDevErrIndex);
    return;
  }
  for (int64_t m = m0; m < m1; m += kMoves) {
    int32_t from[kMoves], to[kMoves];
    uint4 pk[kMoves], pv[kMoves];
#pragma unroll
    for (int i = 0; i < kMoves; ++i) {
      from[i] = m + i < m1 ? __ldg(a.src + m + i) : -1;
      to[i] = m + i < m1 ? __ldg(a.dst + m + i) : -1;
    }
#pragma unroll
    for (int i = 0; i < kMoves; ++i) {
      if (!named(from[i], to[i])) from[i] = to[i] = -1;
      if (from[i] >= 0) {
        const uint64_t x = at(from[i]);
        pk[i] = load_piece(k + x, bytes);
        pv[i] = load_piece(v + x, bytes);
      }
    }
#pragma unroll
    for (int i = 1; i < kMoves; ++i)
#pragma unroll
      for (int e = 0; e < i; ++e)  // the last of the earlier writes counts
        if (to[e] >= 0 && to[e] == from[i]) {
          pk[i] = pk[e];
          pv[i] = pv[e];
        }
#pragma unroll
    for (int i = 0; i < kMoves; ++i)
      if (from[i] >= 0) {
        const uint64_t z = at(to[i]);
        store_piece(k + z, bytes, pk[i]);
        store_piece(v + z, bytes, pv[i]);
      }
  }
}

}  // namespace kv
}  // namespace nvfp4
