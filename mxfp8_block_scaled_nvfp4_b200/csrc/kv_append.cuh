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
  uint32_t q_units, q_ctas, kv_ctas;  // 16-element units; CTAs of Q, of K and of V
  FastDiv q_per_token;      // Hq * D / 16
};

// Elements 8 i .. 8 i + 8 of a head, rotated.
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
    for (int i = 0; i < 4; ++i) {
      const float x = v[2 * i], y = v[2 * i + 1];
      v[2 * i] = __fsub_rn(__fmul_rn(x, cc[i]), __fmul_rn(y, ss[i]));
      v[2 * i + 1] = __fadd_rn(__fmul_rn(y, cc[i]), __fmul_rn(x, ss[i]));
    }
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

// One thread per 16 elements; CTAs of Q first, then of K, then of V.
template <typename T, int MODE, bool V8>
__global__ void __launch_bounds__(kRowThreads) k_kv_append(const __grid_constant__ AppendArgs a) {
  const bool is_q = blockIdx.x < a.q_ctas;
  const uint32_t side = is_q ? 0u : (blockIdx.x - a.q_ctas) / a.kv_ctas;
  const uint32_t u = (is_q ? blockIdx.x : blockIdx.x - a.q_ctas - side * a.kv_ctas) * kRowThreads + threadIdx.x;
  const bool in = u < (is_q ? a.q_units : a.r.units);
  Unit w;
  {
    const FastDiv& pt = is_q ? a.q_per_token : a.r.per_token;
    const uint32_t x = in ? u : 0u;
    w.t = pt.div(x);
    const uint32_t y = x - w.t * pt.d;
    w.h = a.r.per_head.div(y);
    w.j = y - w.h * a.r.per_head.d;
  }
  const int32_t slot = in ? __ldg(a.r.slots + w.t) : -1;
  const int32_t pos = in ? __ldg(a.positions + w.t) : 0;
  const bool bad = slot >= 0 && ((uint32_t)slot >= a.r.num_slots || (uint32_t)pos >= a.max_pos);
  if (bad) atomicOr(&g_device_error, (unsigned)kDevErrIndex);
  const bool go = slot >= 0 && !bad;
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  if (go) {
    const T* head = static_cast<const T*>(is_q ? a.q : a.r.x[side]) + (int64_t)w.t * (is_q ? a.q_stride : a.r.stride[side]) + (int64_t)w.h * a.r.D;
    RawBlk<T> raw;
    load_blk<T, V8>(head + w.j * 16u, raw);
    unpack16<T>(raw, v);
    if (side == 0) {
      turn8<T>(a, head, (uint32_t)pos, w.j * 16u, v);
      turn8<T>(a, head, (uint32_t)pos, w.j * 16u + 8u, v + 8);
    }
  }
  if (is_q) {
    if (!go) return;
    RawBlk<T> out;
    norm::pack16<T>(v, out);
    norm::store_blk<T, V8>(static_cast<T*>(a.q_out) + (int64_t)u * 16, out);
    return;
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
// Moves: the moves of a sequence take effect one after the other.  A thread
// has one piece (at most 16 bytes of one head's codes or scales) of all rows
// that a sequence moves, so that no two threads touch the same bytes; it reads
// the pieces of kMoves moves before it writes them, and takes a piece that an
// earlier one of them writes from there.
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
  uint32_t code_pieces, pieces;  // of a row and side; of a row
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

__global__ void __launch_bounds__(kRowThreads) k_kv_move(const __grid_constant__ MoveArgs a) {
  const uint32_t u = blockIdx.x * kRowThreads + threadIdx.x;
  if (u >= a.units) return;
  const uint32_t s = a.per_seq.div(u), y = u - s * a.per_seq.d, h = a.per_head.div(y), p = y - h * a.per_head.d;
  int64_t m0 = s, m1 = (int64_t)s + 1;
  if (a.starts) {
    m0 = __ldg(a.starts + s);
    m1 = __ldg(a.starts + s + 1);
    if (m0 < 0 || m1 < m0 || m1 > (int64_t)a.M) {
      atomicOr(&g_device_error, (unsigned)kDevErrIndex);
      return;
    }
  }
  const bool codes = p < 2u * a.code_pieces;
  const uint32_t of_side = codes ? a.code_pieces : a.pieces / 2u - a.code_pieces, i = codes ? p : p - 2u * a.code_pieces;
  const uint32_t side = i >= of_side ? 1u : 0u, bytes = codes ? 16u : a.piece, row_bytes = a.row[codes ? 0 : 1];
  uint8_t* base = (codes ? a.codes[side] : a.scales[side]) + (uint64_t)(i - side * of_side) * bytes;
  auto at = [&](int32_t slot) {
    const uint32_t page = a.by_page.div((uint32_t)slot);
    return base + (((uint64_t)page * a.heads + h) * a.page_size + ((uint32_t)slot - page * a.page_size)) * row_bytes;
  };
  for (int64_t m = m0; m < m1; m += kMoves) {
    int32_t from[kMoves], to[kMoves];
    uint4 v[kMoves];
#pragma unroll
    for (int k = 0; k < kMoves; ++k) {
      from[k] = m + k < m1 ? __ldg(a.src + m + k) : -1;
      to[k] = m + k < m1 ? __ldg(a.dst + m + k) : -1;
      const bool named = from[k] >= 0 && to[k] >= 0;
      if (named && ((uint32_t)from[k] >= a.num_slots || (uint32_t)to[k] >= a.num_slots)) {
        atomicOr(&g_device_error, (unsigned)kDevErrIndex);
        from[k] = to[k] = -1;
      }
      if (!named) from[k] = to[k] = -1;
    }
#pragma unroll
    for (int k = 0; k < kMoves; ++k)
      if (from[k] >= 0) v[k] = load_piece(at(from[k]), bytes);
#pragma unroll
    for (int k = 1; k < kMoves; ++k)
#pragma unroll
      for (int e = 0; e < k; ++e)  // the last of the earlier writes counts
        if (to[e] >= 0 && to[e] == from[k]) v[k] = v[e];
#pragma unroll
    for (int k = 0; k < kMoves; ++k)
      if (from[k] >= 0) store_piece(at(to[k]), bytes, v[k]);
  }
}

}  // namespace kv
}  // namespace nvfp4
