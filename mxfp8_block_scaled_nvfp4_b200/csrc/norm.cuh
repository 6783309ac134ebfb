// Root-mean-square norm in front of a block-scaled product, with the addition
// of the residual stream, and its gradient.
//
// Forward, per row of K elements (T the tensors' type):
//   h = T(x + residual)          (h = x without a residual)
//   r = fp32(1 / sqrt(sum_k h_k^2 / K + eps))
//   y_k = fp32(fp32(h_k r) w_k)
// and y leaves as T(y), or as the codes and scales that the quantizers
// (quantize.cuh) give for the fp32 values y.
// Backward, dy the gradient of y and dh what reaches h past the norm:
//   s = sum_k w_k dy_k h_k,  dx = T(dh + r (w dy - h r^2 s / K)),
//   dw_k = sum over rows of dy_k h_k r.
//
// The sum of squares and the root are in fp64, so that r is the correctly
// rounded one but for about 2^-26 of the rows, whatever order the sum is taken
// in: a step of r moves values across the borders of the 4-bit codes.
#pragma once

#include "common.cuh"
#include "kv_cache.cuh"
#include "quantize.cuh"

namespace nvfp4 {
namespace norm {

// Modes as in nvfp4_mode, and the plain output.
enum { kPlain = 3 };

constexpr int kMaxThreads = 512;  // of a CTA; 16 elements a thread and step

struct Args {
  const void* x;
  const void* residual;  // or NULL
  const void* w;
  void* h;               // or NULL
  void* y;               // kPlain: T, else codes
  float* rstd;           // or NULL
  const float* g;
  ScaleOut so;
  int64_t rows;
  uint32_t K, blocks;    // blocks: K / 16
  uint32_t row_warps;    // warps a row has; the CTA's other warps take other rows
  double eps, per_k;     // per_k: 1 / K
};

struct VjpArgs {
  const void* dy;
  const void* h;
  const void* w;
  const float* rstd;
  const void* dh;        // or NULL
  void* dx;
  float* dw;             // or NULL
  float* part;           // [parts, K]
  uint32_t parts;
  int64_t rows;
  uint32_t K, row_warps;
};

// A block of 16 elements.  Plain loads, not the read-only path: h may take x's
// or the residual's place.
template <typename T, bool V8>
__device__ __forceinline__ void load_rw(const T* p, RawBlk<T>& r) {
  constexpr int n = (int)sizeof(r.w) / 16;
  const uint4* q = reinterpret_cast<const uint4*>(p);
  if constexpr (V8) {
#pragma unroll
    for (int i = 0; i < n; i += 2)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(r.w[i].x), "=r"(r.w[i].y), "=r"(r.w[i].z), "=r"(r.w[i].w), "=r"(r.w[i + 1].x), "=r"(r.w[i + 1].y),
                     "=r"(r.w[i + 1].z), "=r"(r.w[i + 1].w)
                   : "l"(q + i));
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i)
      asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.w[i].x), "=r"(r.w[i].y), "=r"(r.w[i].z), "=r"(r.w[i].w) : "l"(q + i));
  }
}
template <typename T>
__device__ __forceinline__ void zero(RawBlk<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r.w) / 16); ++i) r.w[i] = make_uint4(0, 0, 0, 0);
}
// 16 fp32 values rounded to T.
template <typename T>
__device__ __forceinline__ void pack16(const float (&v)[16], RawBlk<T>& r) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.w[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
  } else {
    uint32_t p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      p[i] = std::is_same<T, __half>::value ? pack_f16x2(v[2 * i], v[2 * i + 1]) : pack_bf16x2(v[2 * i], v[2 * i + 1]);
    r.w[0] = make_uint4(p[0], p[1], p[2], p[3]);
    r.w[1] = make_uint4(p[4], p[5], p[6], p[7]);
  }
}
template <typename T, bool V8>
__device__ __forceinline__ void store_blk(T* p, const RawBlk<T>& r) {
  constexpr int n = (int)sizeof(r.w) / 16;
  uint4* q = reinterpret_cast<uint4*>(p);
  if constexpr (V8) {
#pragma unroll
    for (int i = 0; i < n; i += 2)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q + i), "r"(r.w[i].x), "r"(r.w[i].y), "r"(r.w[i].z),
                   "r"(r.w[i].w), "r"(r.w[i + 1].x), "r"(r.w[i + 1].y), "r"(r.w[i + 1].z), "r"(r.w[i + 1].w)
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) q[i] = r.w[i];
  }
}

// A row's sum over its warps' lanes, the same bits in all of them; `red` has
// a place for each warp, two buffers in turn (one barrier a row).
template <typename F>
__device__ __forceinline__ F row_sum(F v, F* red, uint32_t row_warps, uint32_t first) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (row_warps == 1) return v;
  const uint32_t lane = threadIdx.x & 31u;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < row_warps ? red[first + lane] : F(0);  // at most 16 warps
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return __shfl_sync(0xffffffffu, v, 0);
}
// R rows' sums with one barrier; red [R][warps of a CTA].
template <int R>
__device__ __forceinline__ void row_sums(float (&v)[R], float (*red)[kMaxThreads / 32], uint32_t row_warps, uint32_t first) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < R; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (row_warps == 1) return;
  const uint32_t lane = threadIdx.x & 31u;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < R; ++k) red[k][threadIdx.x >> 5] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < R; ++k) v[k] = lane < row_warps ? red[k][first + lane] : 0.0f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < R; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
#pragma unroll
  for (int k = 0; k < R; ++k) v[k] = __shfl_sync(0xffffffffu, v[k], 0);
}

// Codes and scale byte of this lane's 16 fp32 values (MX: of the lane pair's
// 32); all lanes call it.
template <int OUT>
__device__ __forceinline__ uint32_t encode(const float (&v)[16], float E, uint4& q) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
  uint32_t s;
  if constexpr (OUT == kv::kNV) {
    float t = m / kE2M1Max;
    t = t * E;
    s = f32_to_e4m3(t);
    const float fs = e4m3_to_f32(s);
    const float k = fs != 0.0f ? E / fs : 0.0f;
    q.x = s != 0u ? scaled_e2m1x8_at(v, 0, k) : 0u;  // a zero scale stores zero codes
    q.y = s != 0u ? scaled_e2m1x8_at(v, 8, k) : 0u;
  } else {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    s = f32_to_ue8m0_rp(m / (OUT == kv::kMX8 ? kE4M3Max : kE2M1Max));
    const float k = 1.0f / ue8m0_to_f32(s);
    if constexpr (OUT == kv::kMX8) {
      q.x = f32x4_to_e4m3x4(v[0] * k, v[1] * k, v[2] * k, v[3] * k);
      q.y = f32x4_to_e4m3x4(v[4] * k, v[5] * k, v[6] * k, v[7] * k);
      q.z = f32x4_to_e4m3x4(v[8] * k, v[9] * k, v[10] * k, v[11] * k);
      q.w = f32x4_to_e4m3x4(v[12] * k, v[13] * k, v[14] * k, v[15] * k);
    } else {
      q.x = scaled_e2m1x8_at(v, 0, k);
      q.y = scaled_e2m1x8_at(v, 8, k);
    }
  }
  return s;
}

// Scale bytes of the blocks that a warp's lanes hold, four to a store where
// they lie together.  b: this lane's 16-element block, n of them in a row;
// b's remainder by 32 is the lane.  All lanes call it.
template <int OUT>
__device__ __forceinline__ void put_scales(const ScaleOut& so, uint32_t row, uint32_t b, uint32_t n, uint32_t s) {
  constexpr uint32_t per = OUT == kv::kNV ? 1 : 2;  // lanes a scale
  const uint32_t s1 = __shfl_down_sync(0xffffffffu, s, per), s2 = __shfl_down_sync(0xffffffffu, s, 2 * per),
                 s3 = __shfl_down_sync(0xffffffffu, s, 3 * per);
  const uint32_t c = b / per, cols = so.blocks_per_row, c0 = c & ~3u;
  if (b >= n || b % per) return;
  const bool four = c0 + 4u <= cols && (so.swizzled || cols % 4u == 0);
  if (four && c != c0) return;
  uint8_t* to = so.p + (so.swizzled ? (size_t)swizzled_offset(row, c, so.Cp) : (size_t)row * cols + c);
  if (four) *reinterpret_cast<uint32_t*>(to) = __byte_perm(s | (s1 << 8), s2 | (s3 << 8), 0x5410);
  else *to = (uint8_t)s;
}

// U: 16-element blocks a thread has.  With one, loads and stores are of 32
// bytes, the weights stay in registers and the next row's loads are in flight
// while this row is summed and stored; with four (long rows, and rows that are
// not 32-byte aligned) that would spill.
// A row's warps are one CTA's (several rows a CTA where they are short), so a
// row's sum is one barrier, and the row is read once.  16384 x 8192 bf16 with a
// residual to MXFP8 takes 146 us, 99 % of the copy rate; 4096 x 4096 to NVFP4 21
// us (5.2 TB/s), with half of the issue slots used; one row of 4096 2.3 us.  With
// four blocks a thread 4096 x 16384 to NVFP4 109 us for 67; rows that leave lanes
// without a block, 131072 x 128, 71 for 17 (as plain output 51 for 20.5).
template <typename T, int OUT, int U>
__global__ void __launch_bounds__(kMaxThreads) k_rms_norm(const __grid_constant__ Args a) {
  constexpr bool kAhead = U == 1, V8 = U == 1;
  __shared__ double red[2][kMaxThreads / 32];
  const uint32_t warp = threadIdx.x >> 5, rpc = (blockDim.x >> 5) / a.row_warps;  // rows a CTA
  const uint32_t mine = warp / a.row_warps, first = mine * a.row_warps, span = a.row_warps * 32u;
  const uint32_t b0 = threadIdx.x - first * 32u;  // this thread's blocks: b0 + span u
  const float E = OUT == kv::kNV && a.g ? kGlobalEncode / __ldg(a.g) : 1.0f;
  const T* w = static_cast<const T*>(a.w);
  RawBlk<T> h[U], res, wr;
  auto load = [&](int64_t row, int u) {
    const uint32_t b = b0 + span * u;
    if (row < a.rows && b < a.blocks) {
      const int64_t at = row * a.K + (int64_t)b * 16;
      load_rw<T, V8>(static_cast<const T*>(a.x) + at, h[u]);
      if (a.residual) load_rw<T, V8>(static_cast<const T*>(a.residual) + at, res);
    } else {
      zero(h[u]);
      zero(res);
    }
  };
  const int64_t step = (int64_t)gridDim.x * rpc;
  int64_t row = (int64_t)blockIdx.x * rpc + mine;
  if constexpr (kAhead) {
    load(row, 0);
    if (b0 < a.blocks) load_blk<T, V8>(w + b0 * 16u, wr);
    else zero(wr);
  }
  uint32_t turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * rpc; base < a.rows; base += step, row += step, turn ^= 1u) {
    double sum = 0.0;
    RawBlk<T> cur;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (!kAhead) load(row, u);
      float v[16];
      unpack16<T>(h[u], v);
      if (a.residual) {
        float c[16];
        unpack16<T>(res, c);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += c[i];
        pack16<T>(v, h[u]);
        unpack16<T>(h[u], v);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const double d = (double)v[i];
        sum = fma(d, d, sum);
      }
      const uint32_t b = b0 + span * u;
      if (a.h && row < a.rows && b < a.blocks) store_blk<T, V8>(static_cast<T*>(a.h) + row * a.K + (int64_t)b * 16, h[u]);
    }
    if constexpr (kAhead) {
      cur = h[0];
      load(row + step, 0);
    }
    sum = row_sum(sum, red[turn], a.row_warps, first);
    const float r = (float)rsqrt(fma(sum, a.per_k, a.eps));
    if (a.rstd && b0 == 0 && row < a.rows) a.rstd[row] = r;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t b = b0 + span * u;
      const bool in = row < a.rows && b < a.blocks;
      float v[16], c[16];
      if constexpr (kAhead) {
        unpack16<T>(cur, v);
      } else {
        unpack16<T>(h[u], v);
        if (b < a.blocks) load_blk<T, V8>(w + b * 16u, wr);
        else zero(wr);
      }
      unpack16<T>(wr, c);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = (v[i] * r) * c[i];
      if constexpr (OUT == kPlain) {
        RawBlk<T> y;
        pack16<T>(v, y);
        if (in) store_blk<T, V8>(static_cast<T*>(a.y) + row * a.K + (int64_t)b * 16, y);
      } else {
        uint4 q;
        const uint32_t s = encode<OUT>(v, E, q);
        if (in) {
          const int64_t at = row * a.blocks + b;
          if constexpr (OUT == kv::kMX8) static_cast<uint4*>(a.y)[at] = q;
          else static_cast<uint2*>(a.y)[at] = make_uint2(q.x, q.y);
        }
        put_scales<OUT>(a.so, (uint32_t)row, b, row < a.rows ? a.blocks : 0u, s);
      }
    }
  }
  if constexpr (OUT != kPlain) zero_scale_padding(a.so, (uint32_t)a.rows);
}

// The part of dw that a CTA's rows make stays in registers.  A thread has N
// 16-byte pieces of a row, a row's threads' pieces side by side.  STAGED (pieces
// of 16 elements, K <= 8192): R rows at a time are copied into shared memory a
// step ahead, each thread's pieces into slots of its own, so that no barrier
// stands between copy and use; longer rows are read twice.
// Bound by memory on many rows: 16384 x 8192 bf16 takes 168 us with its dw, 97 %
// of the copy rate (a row at a time from registers 271, from shared memory two
// rows ahead 202, two rows at a time 194, and with packed instructions and a
// row's values kept from the first pass to the second, 20 instead of 34
// instructions an element, this).  2048 x 4096 takes 16 us for 7.7: seven rows
// a CTA are a chain of four steps of 2 us, and dw is 3.4 us more.  Rows read
// twice: 4096 x 16384 175 us for 82.
template <typename T>
constexpr int kVjpRows = sizeof(T) == 4 ? 1 : 2;  // of a step: at K 8192 two stages of 96 KB, 48 KB a row (fp32 96)
template <typename T>
constexpr uint32_t kVjpSmem = 2 * kVjpRows<T> * 3 * 16 * sizeof(T);  // bytes a thread

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// A 16-byte piece as fp32.
template <typename T>
__device__ __forceinline__ void piece_to_f(const uint4& p, float* v) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(p.x);
    v[1] = __uint_as_float(p.y);
    v[2] = __uint_as_float(p.z);
    v[3] = __uint_as_float(p.w);
  } else {
    float x[8];
    unpack8<T>(p, p, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i];
  }
}
template <typename T>
__device__ __forceinline__ uint4 piece_of_f(const float* v) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  } else {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = std::is_same<T, __half>::value ? pack_f16x2(v[2 * i], v[2 * i + 1]) : pack_bf16x2(v[2 * i], v[2 * i + 1]);
    return make_uint4(p[0], p[1], p[2], p[3]);
  }
}

// Pairs of fp32 (the packed instructions round each half as the plain ones do).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\t"
      "mov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
// A 16-byte piece as pairs of fp32.
template <typename T, int P>
__device__ __forceinline__ void pairs_of(const uint4& p, float2 (&v)[P]) {
  float x[2 * P];
  piece_to_f<T>(p, x);
#pragma unroll
  for (int i = 0; i < P; ++i) v[i] = make_float2(x[2 * i], x[2 * i + 1]);
}

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kMaxThreads) k_rms_norm_vjp(const __grid_constant__ VjpArgs a) {
  constexpr int E = 16 / (int)sizeof(T), P = E / 2, N = (STAGED ? 16 : 64) / E, R = STAGED ? kVjpRows<T> : 1;
  constexpr int H = STAGED ? N : 1;  // pieces of a row that stay in registers between its two passes
  extern __shared__ __align__(16) uint4 slots[];  // [step % 2][row][dy, h, dh][piece][thread]
  __shared__ float red[2][R][kMaxThreads / 32];
  const uint32_t warp = threadIdx.x >> 5, rpc = (blockDim.x >> 5) / a.row_warps;
  const uint32_t mine = warp / a.row_warps, first = mine * a.row_warps, span = a.row_warps * 32u;
  const uint32_t p0 = threadIdx.x - first * 32u, pieces = a.K / E;  // this thread's pieces: p0 + span n
  const uint4* w = static_cast<const uint4*>(a.w) + p0;
  const uint4 none = make_uint4(0, 0, 0, 0);
  const int64_t next = (int64_t)gridDim.x * rpc, step = R * next;  // rows row + next k
  int64_t row = (int64_t)blockIdx.x * rpc + mine;
  const uint4* src[3] = {static_cast<const uint4*>(a.dy), static_cast<const uint4*>(a.h), static_cast<const uint4*>(a.dh)};
  bool in[N];
#pragma unroll
  for (int n = 0; n < N; ++n) in[n] = p0 + span * n < pieces;
  float2 acc[N][P];
  // slots of a step's row and tensor
  const uint32_t mem = (uint32_t)__cvta_generic_to_shared(slots) + 16u * threadIdx.x, piece = 16u * blockDim.x;
  auto slot = [&](uint32_t st, int k, int t, int n) { return mem + (((st * R + k) * 3 + t) * N + n) * piece; };
  auto start = [&](int64_t row, uint32_t st) {
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (row + next * k < a.rows) {
        const int64_t at = (row + next * k) * pieces + p0;
#pragma unroll
        for (int t = 0; t < 3; ++t)
          if (t < 2 || a.dh)
#pragma unroll
            for (int n = 0; n < N; ++n)
              if (in[n]) copy_async16(slot(st, k, t, n), src[t] + at + span * n);
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  uint32_t st = 0;
  bool live[R] = {};
  // piece n of tensor t in the step's row k
  auto get = [&](int k, int t, int n) {
    uint4 v = none;
    if (live[k] && in[n] && (t < 2 || a.dh)) {
      if constexpr (STAGED) asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(slot(st, k, t, n)));
      else  // plain loads: dx may take dy's or dh's place
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(src[t] + row * pieces + p0 + span * n));
    }
    return v;
  };
  float2 wf[H][P];
  auto weight = [&](int n) { pairs_of<T, P>(in[n] ? __ldg(w + span * n) : none, wf[n % H]); };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (STAGED) {
    start(row, 0);
#pragma unroll
    for (int n = 0; n < N; ++n) weight(n);
  }
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < P; ++i) acc[n][i] = make_float2(0.0f, 0.0f);
  const float per_k = 1.0f / (float)a.K;
  for (int64_t base = (int64_t)blockIdx.x * rpc; base < a.rows; base += step, row += step, st ^= 1u) {
    float r[R], s[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      live[k] = row + next * k < a.rows;
      r[k] = live[k] ? __ldg(a.rstd + row + next * k) : 0.0f;
    }
    if constexpr (STAGED) {
      start(row + step, st ^ 1u);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    }
    float2 x[R][H][P], d[R][H][P];  // h, and w dy
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float2 rr = make_float2(r[k], r[k]);
      float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if constexpr (!STAGED) weight(n);
        float2 y[P];
        pairs_of<T, P>(get(k, 0, n), y);
        pairs_of<T, P>(get(k, 1, n), x[k][n % H]);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          d[k][n % H][i] = mul2(y[i], wf[n % H][i]);
          part[i & 1] = fma2(d[k][n % H][i], x[k][n % H][i], part[i & 1]);
          acc[n][i] = fma2(y[i], mul2(x[k][n % H][i], rr), acc[n][i]);
        }
      }
      s[k] = (part[0].x + part[0].y) + (part[1].x + part[1].y);
    }
    row_sums<R>(s, red[st], a.row_warps, first);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float f = s[k] * per_k * r[k] * r[k];
      const float2 ff = make_float2(-f, -f), rr = make_float2(r[k], r[k]);
      uint4* dx = static_cast<uint4*>(a.dx) + (row + next * k) * pieces + p0;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if constexpr (!STAGED) {
          weight(n);
          float2 y[P];
          pairs_of<T, P>(get(k, 0, n), y);
          pairs_of<T, P>(get(k, 1, n), x[k][0]);
#pragma unroll
          for (int i = 0; i < P; ++i) d[k][0][i] = mul2(y[i], wf[0][i]);
        }
        float2 g[P];
        pairs_of<T, P>(get(k, 2, n), g);
        float o[E];
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 v = fma2(fma2(x[k][n % H][i], ff, d[k][n % H][i]), rr, g[i]);
          o[2 * i] = v.x;
          o[2 * i + 1] = v.y;
        }
        if (live[k] && in[n]) dx[span * n] = piece_of_f<T>(o);
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (!a.dw) return;
  // the rows that a CTA takes side by side (of at most 256 threads: 16 KB) add up in order
  if (STAGED && rpc > 1) {
    float4* sums = reinterpret_cast<float4*>(slots);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < P; i += 2)
        sums[(n * P + i) / 2 * blockDim.x + threadIdx.x] = make_float4(acc[n][i].x, acc[n][i].y, acc[n][i + 1].x, acc[n][i + 1].y);
    __syncthreads();
    if (mine != 0) return;
    for (uint32_t o = 1; o < rpc; ++o)
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < P; i += 2) {
          const float4 v = sums[(n * P + i) / 2 * blockDim.x + o * span + threadIdx.x];
          acc[n][i].x += v.x;
          acc[n][i].y += v.y;
          acc[n][i + 1].x += v.z;
          acc[n][i + 1].y += v.w;
        }
  }
  float* part = a.part + (uint64_t)blockIdx.x * a.K;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (!in[n]) continue;
#pragma unroll
    for (int i = 0; i < P; i += 2)
      *reinterpret_cast<float4*>(part + (p0 + span * n) * E + 2 * i) = make_float4(acc[n][i].x, acc[n][i].y, acc[n][i + 1].x, acc[n][i + 1].y);
  }
}

// dw: the parts added up, 32 columns a CTA (8 lanes of 4) by 128 groups of
// parts; each group's parts in order, then the groups in a fixed order.
constexpr int kDwThreads = 1024;
__global__ void __launch_bounds__(kDwThreads) k_rms_norm_dw(const __grid_constant__ VjpArgs a) {
  __shared__ float4 sum[kDwThreads / 32][8];
  const uint32_t c = threadIdx.x & 7u, grp = threadIdx.x >> 3, col = blockIdx.x * 32u + c * 4u, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (col < a.K)
#pragma unroll 4
    for (uint32_t p = grp; p < a.parts; p += kDwThreads / 8) {
      const float4 v = *reinterpret_cast<const float4*>(a.part + (uint64_t)p * a.K + col);
      s[0] += v.x;
      s[1] += v.y;
      s[2] += v.z;
      s[3] += v.w;
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s[i] += __shfl_xor_sync(0xffffffffu, s[i], 8);
    s[i] += __shfl_xor_sync(0xffffffffu, s[i], 16);
  }
  if ((threadIdx.x & 31u) < 8u) sum[warp][c] = make_float4(s[0], s[1], s[2], s[3]);
  __syncthreads();
  if (threadIdx.x >= 8u || col >= a.K) return;
  float4 t = sum[0][c];
#pragma unroll
  for (int i = 1; i < kDwThreads / 32; ++i) {
    const float4 v = sum[i][c];
    t.x += v.x;
    t.y += v.y;
    t.z += v.z;
    t.w += v.w;
  }
  *reinterpret_cast<float4*>(a.dw + col) = t;
}

}  // namespace norm
}  // namespace nvfp4
